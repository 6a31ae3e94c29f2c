// Root-mean-square norm over rows of `dim` elements, with the residual's addition
// before it and an output in 8 bits beside or instead of the plain one:
//
//   h_k = x_k + r_k,  rstd = 1 / sqrt(sum_k h_k^2 / dim + eps),  y_k = h_k rstd w_k
//
// Bound by memory: x and r are read, h and y (or its codes) are written, once each.
// A row stays in the registers of the LPR lanes that own it (16 lanes, one wave,
// or several waves of a workgroup), the weights in registers over all rows of a
// workgroup. Everything is fp32 and rounded once when it is stored: the norm is of
// the sum before its rounding. The squares' sum has no cancellation, so unlike a
// variance it needs no second reading; where fp32 cannot hold it, it is made again
// of the values times a power of two. 16384 rows of 4096 bf16 with a residual, to the
// sum and 8 bits: 84 us, 473 MB at 5.6 TB/s. One row of 8192: 3.4 us, one round trip and
// a barrier behind the launch.
#include "zs_e4m3.hpp"
#include "zs_launch.hpp"
#include "zs_launch_rows.hpp"
#include "zs_rows.hpp"

namespace zs {
namespace {

template <int LPR, int VEC>
__device__ __forceinline__ uint32_t col_of(int j, int l) {
  return (uint32_t)(j * LPR + l) * VEC;
}

// VEC weights in fp32, ones where there are none.
template <int VEC>
__device__ __forceinline__ void load_weights(float (&to)[VEC], const void* w, int wdtype, uint32_t c, uint32_t dim) {
  if (!w) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) to[e] = 1.0f;
  } else if (wdtype == ZS_BF16) {
    if constexpr (VEC == 8) {
      Piece<uint16_t, 8> p;
      take_cols<uint16_t, 8>(p, (const uint16_t*)w, c, dim);
#pragma unroll
      for (int e = 0; e < VEC; ++e) to[e] = p.get(e);
    } else {
      Piece<uint16_t, 4> p;
      take_cols<uint16_t, 4>(p, (const uint16_t*)w, c, dim);
#pragma unroll
      for (int e = 0; e < VEC; ++e) to[e] = p.get(e);
    }
  } else {
    Piece<float, VEC> p;
    take_cols<float, VEC>(p, (const float*)w, c, dim);
#pragma unroll
    for (int e = 0; e < VEC; ++e) to[e] = p.get(e);
  }
}

// Whether a row's sum of squares left fp32's range: magnitudes of about 2^64 / sqrt(dim) and
// above make it infinite; below 2^-78 squares may have vanished, and what they add up to matters
// beside an eps below 2^-54. Such a row is summed again times a power of two: 2^-80 leaves
// the largest sum of 2^24 squares below 2^120 and the smallest above 2^-33, 2^90 those
// below 2^-78 below 2^103, and the square of the smallest subnormal 2^-118.
__device__ __forceinline__ bool out_of_range(float s, float eps) {
  return !(s < INFINITY) || (s < 0x1p-78f && eps < 0x1p-54f);
}
__device__ __forceinline__ float factor_of(float s) { return s < 1.0f ? 0x1p90f : 0x1p-80f; }
// 1 / sqrt(mean + eps) for the sum s of the squares of the values times `factor`
__device__ __forceinline__ float rstd_of(float s, float inv_dim, float eps, float factor) {
  return factor / sqrtf(s * inv_dim + eps * factor * factor);
}

struct RmsForward {
  const void *x, *residual, *weight;
  void *sum, *y;
  uint8_t* codes;
  float *scales, *rstd;
  int64_t x_ld, residual_ld, sum_ld, y_ld, codes_ld, scales_ld, rows;
  uint32_t dim;
  int wdtype;
  float eps;
};

// The row's outputs at one piece.
template <typename T, typename R, int VEC, int G, bool NT>
__device__ __forceinline__ void store_row(const RmsForward& a, int64_t row, const float (&h)[VEC], const float (&w)[VEC],
                                          float rstd, uint32_t c) {
  if (a.sum) store_cols<R, VEC, NT>((R*)a.sum + row * a.sum_ld, h, c, a.dim);
  float v[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) v[e] = h[e] * rstd * w[e];
  if (a.y) store_cols<T, VEC, NT>((T*)a.y + row * a.y_ld, v, c, a.dim);
  if (a.codes) store_codes<VEC, G, NT>(a.codes + row * a.codes_ld, a.scales + row * a.scales_ld, v, c, a.dim);
}

template <typename T, typename R, int LPR, int NV, int VEC, bool NT>
__global__ __launch_bounds__(LPR > 256 ? LPR : 256)
void k_rms_fwd(RmsForward a) {
  constexpr int BS = LPR > 256 ? LPR : 256;
  constexpr int RPB = BS / LPR;  // rows in flight per workgroup
  constexpr int NW = LPR / 64;   // waves per row (0 below a wave)
  constexpr int G = LPR < 64 ? LPR : 64;
  constexpr int BLOCK = kScaleBlock / VEC < LPR ? kScaleBlock / VEC : LPR;  // lanes of a block of one scale
  __shared__ float parts[2][BS / 64], again[BS / 64];
  const int l = threadIdx.x % LPR;
  const uint32_t dim = a.dim;
  const int64_t step = (int64_t)gridDim.x * RPB;
  int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / LPR;
  float w[NV][VEC];
#pragma unroll
  for (int j = 0; j < NV; ++j) load_weights<VEC>(w[j], a.weight, a.wdtype, col_of<LPR, VEC>(j, l), dim);
  const float inv_dim = 1.0f / (float)dim;
  // every row group of the workgroup takes the same number of turns (barriers)
  int turn = 0;
  for (int64_t base = (int64_t)blockIdx.x * RPB; base < a.rows; base += step, row += step, turn ^= 1) {
    const bool live = row < a.rows;
    const T* x = (const T*)a.x + row * a.x_ld;
    const R* r = (const R*)a.residual + row * a.residual_ld;
    Piece<T, VEC> px[NV];
    Piece<R, VEC> pr[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      px[j].clear();
      pr[j].clear();
    }
    if (live) {
#pragma unroll
      for (int j = 0; j < NV; ++j) load_cols<T, VEC, NT>(px[j], x, col_of<LPR, VEC>(j, l), dim);
      if (a.residual)
#pragma unroll
        for (int j = 0; j < NV; ++j) load_cols<R, VEC, NT>(pr[j], r, col_of<LPR, VEC>(j, l), dim);
      if (ragged(dim, VEC)) {
#pragma unroll
        for (int j = 0; j < NV; ++j) settle_cols<T, VEC>(px[j], x, col_of<LPR, VEC>(j, l), dim);
        if (a.residual)
#pragma unroll
          for (int j = 0; j < NV; ++j) settle_cols<R, VEC>(pr[j], r, col_of<LPR, VEC>(j, l), dim);
      }
    }
    float h[NV][VEC], s = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        h[j][e] = a.residual ? px[j].get(e) + pr[j].get(e) : px[j].get(e);
        s = fmaf(h[j][e], h[j][e], s);
      }
    s = lane_sum<G>(s);
    bool far = false;  // the same in all waves that meet at a barrier
    if constexpr (NW > 1) {
      if ((threadIdx.x & 63) == 0) parts[turn][threadIdx.x / 64] = s;
      __syncthreads();  // the other turn's entries are read by nobody any more
#pragma unroll
      for (int k = 0; k < RPB; ++k) {
        float t = 0.0f;
#pragma unroll
        for (int i = 0; i < NW; ++i) t += parts[turn][k * NW + i];
        far = far || out_of_range(t, a.eps);
        if (RPB == 1 || k == (int)threadIdx.x / LPR) s = t;
      }
    } else {
      far = out_of_range(s, a.eps);
    }
    float factor = 1.0f;
    if (__any(far)) {  // rows of the workgroup that are in range get the same sum again
      if (out_of_range(s, a.eps)) factor = factor_of(s);
      s = 0.0f;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float x = h[j][e] * factor;
          s = fmaf(x, x, s);
        }
      s = lane_sum<G>(s);
      if constexpr (NW > 1) {
        const int w0 = threadIdx.x / LPR * NW;  // the row's first wave
        if ((threadIdx.x & 63) == 0) again[threadIdx.x / 64] = s;
        __syncthreads();  // the last such turn's entries were read before this turn's first barrier
        s = 0.0f;
#pragma unroll
        for (int i = 0; i < NW; ++i) s += again[w0 + i];
      }
    }
    if (!live) continue;
    const float rstd = rstd_of(s, inv_dim, a.eps, factor);
    if (l == 0 && a.rstd) a.rstd[row] = rstd;
#pragma unroll
    for (int j = 0; j < NV; ++j) store_row<T, R, VEC, BLOCK, NT>(a, row, h[j], w[j], rstd, col_of<LPR, VEC>(j, l));
  }
}

constexpr int kLongBS = 1024;

// Rows longer than the registers of 1024 lanes hold: one workgroup reads the row
// twice (squares, outputs; squares out of range once more). A sum in place is written by the lanes that read
// these elements, in the second reading.
template <typename T, typename R, int VEC>
__global__ __launch_bounds__(kLongBS)
void k_rms_fwd_long(RmsForward a) {
  __shared__ float lds[kLongBS / 64];
  const uint32_t dim = a.dim;
  const float inv_dim = 1.0f / (float)dim;
  const uint32_t turns = (dim + kLongBS * VEC - 1) / (kLongBS * VEC);  // the same for all lanes: blocks' lanes meet
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = (const T*)a.x + row * a.x_ld;
    const R* r = (const R*)a.residual + row * a.residual_ld;
    auto take = [&](uint32_t c, float (&h)[VEC]) {
      Piece<T, VEC> px;
      take_cols<T, VEC>(px, x, c, dim);
#pragma unroll
      for (int e = 0; e < VEC; ++e) h[e] = px.get(e);
      if (a.residual) {
        Piece<R, VEC> pr;
        take_cols<R, VEC>(pr, r, c, dim);
#pragma unroll
        for (int e = 0; e < VEC; ++e) h[e] += pr.get(e);
      }
    };
    auto squares = [&](float factor) {  // of the row, in all lanes
      float s = 0.0f;
      for (uint32_t t = 0; t < turns; ++t) {
        float h[VEC], p = 0.0f;
        take((t * kLongBS + threadIdx.x) * VEC, h);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float x = h[e] * factor;
          p = fmaf(x, x, p);
        }
        s += p;
      }
      s = lane_sum<64>(s);
      if ((threadIdx.x & 63) == 0) lds[threadIdx.x / 64] = s;
      __syncthreads();
      s = 0.0f;
#pragma unroll
      for (int i = 0; i < kLongBS / 64; ++i) s += lds[i];
      __syncthreads();
      return s;
    };
    float s = squares(1.0f), factor = 1.0f;
    if (out_of_range(s, a.eps)) {  // the same in all lanes
      factor = factor_of(s);
      s = squares(factor);
    }
    const float rstd = rstd_of(s, inv_dim, a.eps, factor);
    if (threadIdx.x == 0 && a.rstd) a.rstd[row] = rstd;
    for (uint32_t t = 0; t < turns; ++t) {
      const uint32_t c = (t * kLongBS + threadIdx.x) * VEC;
      float h[VEC], w[VEC];
      take(c, h);
      load_weights<VEC>(w, a.weight, a.wdtype, c, dim);
      store_row<T, R, VEC, kScaleBlock / VEC, false>(a, row, h, w, rstd, c);
    }
  }
}

// As for the layer norm: calls of more bytes than this bypass the caches, and so
// many workgroups of 256 lanes walk over the rows.
constexpr int64_t kStreamBytes = 100000000;
constexpr int64_t kFwdSlots = 1024;

template <typename T, typename R, int VEC>
void run(const RmsForward& a, int64_t bytes, hipStream_t s) {
  const int64_t nvec = ((int64_t)a.dim + VEC - 1) / VEC;
  const bool nt = bytes > kStreamBytes;
  auto go = [&](auto lpr, auto nv) {
    constexpr int LPR = decltype(lpr)::value, NV = decltype(nv)::value, BS = LPR > 256 ? LPR : 256;
    const int64_t need = (a.rows + BS / LPR - 1) / (BS / LPR);
    const int64_t slots = kFwdSlots * 256 / BS, grid = need < slots ? need : slots;
    if (nt) hipLaunchKernelGGL((k_rms_fwd<T, R, LPR, NV, VEC, true>), dim3((unsigned)grid), dim3(BS), 0, s, a);
    else hipLaunchKernelGGL((k_rms_fwd<T, R, LPR, NV, VEC, false>), dim3((unsigned)grid), dim3(BS), 0, s, a);
  };
  using std::integral_constant;
  // by width alone, so that a row gives the same bits whatever the number of rows
  if (nvec <= 16) go(integral_constant<int, 16>{}, integral_constant<int, 1>{});
  else if (nvec <= 32) go(integral_constant<int, 32>{}, integral_constant<int, 1>{});
  else if (nvec <= 64) go(integral_constant<int, 64>{}, integral_constant<int, 1>{});
  else if (nvec <= 128) go(integral_constant<int, 64>{}, integral_constant<int, 2>{});
  else if (nvec <= 192) go(integral_constant<int, 64>{}, integral_constant<int, 3>{});
  else if (nvec <= 256) go(integral_constant<int, 128>{}, integral_constant<int, 2>{});
  else if (nvec <= 512) go(integral_constant<int, 256>{}, integral_constant<int, 2>{});
  else if (nvec <= 1024) go(integral_constant<int, 512>{}, integral_constant<int, 2>{});
  else if (nvec <= 2048) go(integral_constant<int, 1024>{}, integral_constant<int, 2>{});
  else {
    const int64_t grid = a.rows < 2048 ? a.rows : 2048;
    hipLaunchKernelGGL((k_rms_fwd_long<T, R, VEC>), dim3((unsigned)grid), dim3(kLongBS), 0, s, a);
  }
}

}  // namespace

hipError_t launch_rms_norm_forward(const void* x, int dtype, int64_t x_ld, const void* residual, int64_t residual_ld,
                                   void* sum, int64_t sum_ld, int sum_dtype, const void* w, int wdtype, int64_t rows,
                                   int64_t dim, float eps, void* y, int64_t y_ld, uint8_t* codes, int64_t codes_ld,
                                   float* scales, int64_t scales_ld, float* rstd, hipStream_t s) {
  const RmsForward a{x, residual, w, sum, y, codes, scales, rstd, x_ld, residual_ld, sum_ld, y_ld, codes_ld, scales_ld,
                     rows, (uint32_t)dim, wdtype, eps};
  const int64_t t = dtype == ZS_BF16 ? 2 : 4, r = sum_dtype == ZS_BF16 ? 2 : 4;
  const int64_t bytes = rows * dim * (t + (residual ? r : 0) + (sum ? r : 0) + (y ? t : 0) + (codes ? 1 : 0));
  if (dtype == ZS_F32) run<float, float, 4>(a, bytes, s);
  else if (sum_dtype == ZS_F32) run<uint16_t, float, 8>(a, bytes, s);
  else run<uint16_t, uint16_t, 8>(a, bytes, s);
  return hipGetLastError();
}

}  // namespace zs
