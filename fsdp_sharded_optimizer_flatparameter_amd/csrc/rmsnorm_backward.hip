// Gradients of the root-mean-square norm y_k = h_k rstd w_k:
//
//   xh_k = h_k rstd,  c = sum_k dy_k w_k xh_k / dim
//   dh_k = rstd (dy_k w_k - xh_k c) + dres_k,   dw_k = sum_rows dy_k xh_k
//
// dres is the gradient that reaches h past the norm, along the residual stream. h
// is what the forward pass kept, in its own type or in 8 bits with a scale for
// each block of 128 elements. Bound by memory: h, dy and dres are read and dh is
// written once each. A row stays in the registers of the LPR lanes that own it;
// the columns' sums stay in registers over all rows of at most 256 workgroups of
// 16 waves, which leave one row of partial sums each for k_rms_dw to join. 16384 rows of
// 4096 from 8 bits with a residual's gradient: 76 us, 477 MB at 6.3 TB/s, and 4.6 for
// the join. 1201 rows of 1601 fp32: 8.1 and 3.5 us, where three turns of a barrier and
// a round trip count.
#include <type_traits>

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

struct RmsBackward {
  const void *dy, *h, *weight, *dres;
  const float *scales, *rstd;
  void* dh;
  float* partials;
  int64_t dy_ld, h_ld, scales_ld, dres_ld, dh_ld, rows;
  uint32_t dim, pitch;
  int wdtype;
  // with one workgroup alone its sums are the gradient, and no launch joins them
  void* alone;
  int grad_dtype, first;
};

__device__ __forceinline__ void store_alone(const RmsBackward& a, uint32_t c, float sum) {
  if (a.grad_dtype == ZS_BF16) {
    uint16_t* to = (uint16_t*)a.alone + c;
    *to = round_to<uint16_t>(a.first ? sum : sum + bf16_to_f32(*to));
  } else {
    float* to = (float*)a.alone + c;
    *to = a.first ? sum : sum + *to;
  }
}

// One lane's piece of the kept h: of type R, or codes with their block's scale.
template <typename H, int VEC>
struct Kept {
  Piece<H, VEC> p;
  __device__ __forceinline__ void clear() { p.clear(); }
  template <bool NT>
  __device__ __forceinline__ void load(const RmsBackward& a, int64_t row, uint32_t c) {
    load_cols<H, VEC, NT>(p, (const H*)a.h + row * a.h_ld, c, a.dim);
  }
  __device__ __forceinline__ void settle(const RmsBackward& a, int64_t row, uint32_t c) {
    settle_cols<H, VEC>(p, (const H*)a.h + row * a.h_ld, c, a.dim);
  }
  __device__ __forceinline__ float get(int e) const { return p.get(e); }
};
template <int VEC>
struct Kept<uint8_t, VEC> {
  Codes<VEC> p;
  float scale;
  __device__ __forceinline__ void clear() {
    p.clear();
    scale = 0.0f;
  }
  template <bool NT>
  __device__ __forceinline__ void load(const RmsBackward& a, int64_t row, uint32_t c) {
    load_codes<VEC, NT>(p, (const uint8_t*)a.h + row * a.h_ld, c, a.dim);
    scale = 0.0f;
    if (c < a.dim) scale = a.scales[row * a.scales_ld + c / kScaleBlock];
  }
  __device__ __forceinline__ void settle(const RmsBackward& a, int64_t row, uint32_t c) {
    settle_codes<VEC>(p, (const uint8_t*)a.h + row * a.h_ld, c, a.dim);
  }
  __device__ __forceinline__ float get(int e) const { return p.get(e) * scale; }
};

template <int VEC>
__device__ __forceinline__ void load_weights(float (&to)[VEC], const void* w, int wdtype, uint32_t c, uint32_t dim) {
  auto from = [&](auto piece, auto type) {
    using W = decltype(type);
    take_cols<W, VEC>(piece, (const W*)w, c, dim);
#pragma unroll
    for (int e = 0; e < VEC; ++e) to[e] = piece.get(e);
  };
  if (!w) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) to[e] = 1.0f;
  } else if (wdtype == ZS_BF16) {
    from(Piece<uint16_t, VEC>{}, uint16_t{});
  } else {
    from(Piece<float, VEC>{}, float{});
  }
}

template <typename T, typename R, typename H, int LPR, int NV, int VEC, bool NT>
__global__ __launch_bounds__(1024)
void k_rms_bwd(RmsBackward a) {
  constexpr int BS = 1024;
  constexpr int RPB = BS / LPR;
  constexpr int NW = LPR / 64;
  constexpr int G = LPR < 64 ? LPR : 64;
  constexpr int COLS = LPR * NV * VEC;
  __shared__ float sums[2][BS / 64];
  __shared__ __align__(16) float joined[RPB > 1 ? RPB * COLS : 4];
  const int l = threadIdx.x % LPR;
  const uint32_t dim = a.dim;
  const int64_t step = (int64_t)gridDim.x * RPB;
  int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / LPR;
  struct Row {
    Kept<H, VEC> h[NV];
    Piece<T, VEC> dy[NV];
    Piece<R, VEC> dres[NV];
    float rstd;
  };
  auto fetch = [&](int64_t r, Row& to) {
    if (r < a.rows) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const uint32_t c = col_of<LPR, VEC>(j, l);
        to.h[j].template load<NT>(a, r, c);
        load_cols<T, VEC, NT>(to.dy[j], (const T*)a.dy + r * a.dy_ld, c, dim);
        if (a.dres) load_cols<R, VEC, NT>(to.dres[j], (const R*)a.dres + r * a.dres_ld, c, dim);
      }
      to.rstd = a.rstd[r];
    }
  };
  constexpr bool AHEAD = NV == 1;  // two pieces a lane and a row ahead do not fit in 128 registers
  Row next;
  next.rstd = 0.0f;
  if (AHEAD) fetch(row, next);
  float w[NV][VEC], dw[NV][VEC];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    load_weights<VEC>(w[j], a.weight, a.wdtype, col_of<LPR, VEC>(j, l), dim);
#pragma unroll
    for (int e = 0; e < VEC; ++e) dw[j][e] = 0.0f;
  }
  const float inv_dim = 1.0f / (float)dim;
  // every row group of the workgroup takes the same number of turns (barriers)
  int turn = 0;
  for (int64_t base = (int64_t)blockIdx.x * RPB; base < a.rows; base += step, row += step, turn ^= 1) {
    Row now;
    if constexpr (AHEAD) now = next;
    else fetch(row, now);
    const bool live = row < a.rows;
    if (AHEAD) fetch(row + step, next);
    if (ragged(dim, VEC) && live)
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const uint32_t c = col_of<LPR, VEC>(j, l);
        now.h[j].settle(a, row, c);
        settle_cols<T, VEC>(now.dy[j], (const T*)a.dy + row * a.dy_ld, c, dim);
        if (a.dres) settle_cols<R, VEC>(now.dres[j], (const R*)a.dres + row * a.dres_ld, c, dim);
      }
    const float rstd = now.rstd;
    float s = 0.0f;
    if (live) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float g = now.dy[j].get(e), xh = now.h[j].get(e) * rstd;
          s = fmaf(g * w[j][e], xh, s);
          dw[j][e] = fmaf(g, xh, dw[j][e]);
        }
      s = lane_sum<G>(s);
    }
    if constexpr (NW > 1) {
      const int w0 = threadIdx.x / LPR * NW;  // the row's first wave
      if ((threadIdx.x & 63) == 0) sums[turn][threadIdx.x / 64] = s;
      __syncthreads();  // the other turn's entries are read by nobody any more
      s = 0.0f;
#pragma unroll
      for (int i = 0; i < NW; ++i) s += sums[turn][w0 + i];
    }
    if (live) {
      const float c = s * inv_dim;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float v[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float xh = now.h[j].get(e) * rstd;
          v[e] = rstd * (now.dy[j].get(e) * w[j][e] - xh * c);
          if (a.dres) v[e] += now.dres[j].get(e);
        }
        store_cols<R, VEC, NT>((R*)a.dh + row * a.dh_ld, v, col_of<LPR, VEC>(j, l), dim);
      }
    }
  }
  if (!a.partials) return;  // uniform: an argument
  float* pw = a.partials + (int64_t)blockIdx.x * a.pitch;
  if constexpr (RPB > 1) {
    const int mine = threadIdx.x / LPR * COLS;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < VEC; e += 4)
        *reinterpret_cast<f32x4*>(&joined[mine + (j * LPR + l) * VEC + e]) =
            f32x4{dw[j][e], dw[j][e + 1], dw[j][e + 2], dw[j][e + 3]};
    __syncthreads();
    for (uint32_t c = threadIdx.x; c < COLS && c < dim; c += BS) {
      float t = joined[c];
#pragma unroll
      for (int g = 1; g < RPB; ++g) t += joined[g * COLS + c];
      if (a.alone) store_alone(a, c, t);
      else pw[c] = t;
    }
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const uint32_t c = col_of<LPR, VEC>(j, l);
      if (a.alone) {
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          if (c + e < dim) store_alone(a, c + e, dw[j][e]);
      } else if (c < a.pitch) {
        store_piece<float, VEC>(pw + c, dw[j]);  // pitch is a multiple of VEC
      }
    }
  }
}

constexpr int kLongBS = 1024;
constexpr int kMaxParts = 256;  // rows of partial sums: a workgroup of 16 waves per CU

// Rows longer than the registers of 1024 lanes hold, dh alone: one workgroup reads the row twice. A
// gradient in place of dres is written by the lanes that read these elements, in the second reading.
template <typename T, typename R, typename H, int VEC>
__global__ __launch_bounds__(kLongBS)
void k_rms_bwd_long(RmsBackward a) {
  __shared__ float lds[kLongBS / 64];
  const uint32_t dim = a.dim;
  const float inv_dim = 1.0f / (float)dim;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const float rstd = a.rstd[row];
    const T* dy = (const T*)a.dy + row * a.dy_ld;
    auto take = [&](uint32_t c, float (&g)[VEC], float (&xh)[VEC]) {
      Kept<H, VEC> ph;
      Piece<T, VEC> pg;
      float w[VEC];
      ph.template load<false>(a, row, c);
      take_cols<T, VEC>(pg, dy, c, dim);
      if (ragged(dim, VEC)) ph.settle(a, row, c);
      load_weights<VEC>(w, a.weight, a.wdtype, c, dim);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        g[e] = pg.get(e) * w[e];
        xh[e] = ph.get(e) * rstd;
      }
    };
    float s = 0.0f;
    for (uint32_t c = threadIdx.x * VEC; c < dim; c += kLongBS * VEC) {
      float g[VEC], xh[VEC], t = 0.0f;
      take(c, g, xh);
#pragma unroll
      for (int e = 0; e < VEC; ++e) t = fmaf(g[e], xh[e], t);
      s += t;
    }
    s = lane_sum<64>(s);
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x / 64] = s;
    __syncthreads();
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < kLongBS / 64; ++i) s += lds[i];
    __syncthreads();
    const float k = s * inv_dim;
    for (uint32_t c = threadIdx.x * VEC; c < dim; c += kLongBS * VEC) {
      float g[VEC], xh[VEC], v[VEC];
      take(c, g, xh);
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[e] = rstd * (g[e] - xh[e] * k);
      if (a.dres) {
        Piece<R, VEC> pr;
        take_cols<R, VEC>(pr, (const R*)a.dres + row * a.dres_ld, c, dim);
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[e] += pr.get(e);
      }
      store_cols<R, VEC>((R*)a.dh + row * a.dh_ld, v, c, dim);
    }
  }
}

// The columns' sums for such rows: workgroup (tile, g) adds rows g, g + parts,
// ... of 256 pieces of columns.
template <typename T, typename H, int VEC>
__global__ __launch_bounds__(kThreads)
void k_rms_cols(RmsBackward a, int64_t tiles) {
  const int64_t parts = gridDim.x / tiles, tile = blockIdx.x % tiles, g = blockIdx.x / tiles;
  const uint32_t c = ((uint32_t)tile * kThreads + threadIdx.x) * VEC;
  float dw[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) dw[e] = 0.0f;
  for (int64_t row = g; row < a.rows; row += parts) {
    Kept<H, VEC> ph;
    Piece<T, VEC> pg;
    ph.template load<false>(a, row, c);
    take_cols<T, VEC>(pg, (const T*)a.dy + row * a.dy_ld, c, a.dim);
    if (ragged(a.dim, VEC)) ph.settle(a, row, c);
    const float rstd = a.rstd[row];
#pragma unroll
    for (int e = 0; e < VEC; ++e) dw[e] = fmaf(pg.get(e), ph.get(e) * rstd, dw[e]);
  }
  if (c < a.pitch) store_piece<float, VEC>(a.partials + g * (int64_t)a.pitch + c, dw);
}

// Joins the workgroups' partial sums: a wave takes 64 columns, the waves of a
// workgroup every kJoinWaves-th partial, and their sums are added in wave order.
// The grouping depends on the sizes alone.
constexpr int kJoinWaves = 16;
template <typename Gt>
__global__ __launch_bounds__(kJoinWaves * 64)
void k_rms_dw(const float* __restrict__ partials, int64_t pitch, int parts, int64_t dim, Gt* __restrict__ dw, int first) {
  __shared__ float lds[kJoinWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + lane;
  float s = 0.0f, old = 0.0f;
  if (c < dim) {
    if (wave == 0 && !first) {
      if constexpr (sizeof(Gt) == 4) old = dw[c];
      else old = bf16_to_f32(dw[c]);
    }
    constexpr int U = kMaxParts / kJoinWaves;
    float v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = u * kJoinWaves + wave;
      v[u] = k < parts ? partials[(int64_t)k * pitch + c] : 0.0f;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) s += v[u];
  }
  lds[wave][lane] = s;
  __syncthreads();
  if (wave != 0 || c >= dim) return;
#pragma unroll
  for (int i = 1; i < kJoinWaves; ++i) s += lds[i][lane];
  dw[c] = round_to<Gt>(first ? s : s + old);
}

constexpr int64_t kStreamBytes = 100000000;  // calls of more bytes bypass the caches, as for the layer norm

// Returns the number of rows of partial sums, or 0 where they are the gradient already.
template <typename T, typename R, typename H, int VEC>
int run(RmsBackward a, int64_t bytes, hipStream_t s) {
  const int64_t nvec = ((int64_t)a.dim + VEC - 1) / VEC;
  const bool nt = bytes > kStreamBytes;
  int parts = (int)(a.rows < kMaxParts ? a.rows : kMaxParts);
  auto go = [&](auto lpr, auto nv) {
    constexpr int LPR = decltype(lpr)::value, NV = decltype(nv)::value, BS = 1024;
    const int64_t need = (a.rows + BS / LPR - 1) / (BS / LPR);
    const int64_t want = LPR >= 512 && need >= 64 ? (need + 1) / 2 : need;
    parts = (int)(want < kMaxParts ? want : kMaxParts);
    if (parts > 1) a.alone = nullptr;
    else if (a.alone) parts = 0;
    const dim3 grid((unsigned)(parts > 0 ? parts : 1));
    if (nt) hipLaunchKernelGGL((k_rms_bwd<T, R, H, LPR, NV, VEC, true>), grid, dim3(BS), 0, s, a);
    else hipLaunchKernelGGL((k_rms_bwd<T, R, H, LPR, NV, VEC, false>), grid, dim3(BS), 0, s, a);
  };
  using std::integral_constant;
  if (nvec <= 16) go(integral_constant<int, 16>{}, integral_constant<int, 1>{});
  else if (nvec <= 32) go(integral_constant<int, 32>{}, integral_constant<int, 1>{});
  else if (nvec <= 64) go(integral_constant<int, 64>{}, integral_constant<int, 1>{});
  else if (nvec <= 128) go(integral_constant<int, 128>{}, integral_constant<int, 1>{});
  else if (nvec <= 256) go(integral_constant<int, 256>{}, integral_constant<int, 1>{});
  else if (nvec <= 512) go(integral_constant<int, 512>{}, integral_constant<int, 1>{});
  else if (nvec <= 1024) go(integral_constant<int, 1024>{}, integral_constant<int, 1>{});
  else if (nvec <= 2048) go(integral_constant<int, 1024>{}, integral_constant<int, 2>{});
  else {
    const int64_t grid = a.rows < 2048 ? a.rows : 2048;
    hipLaunchKernelGGL((k_rms_bwd_long<T, R, H, VEC>), dim3((unsigned)grid), dim3(kLongBS), 0, s, a);
    if (a.partials) {
      const int64_t tiles = (nvec + kThreads - 1) / kThreads;
      hipLaunchKernelGGL((k_rms_cols<T, H, VEC>), dim3((unsigned)(tiles * parts)), dim3(kThreads), 0, s, a, tiles);
    }
  }
  return parts;
}

}  // namespace

RmsPlan rms_plan(int64_t rows, int64_t dim) {
  RmsPlan p;
  p.pitch = (dim + 7) / 8 * 8;
  p.parts = rows < kMaxParts ? rows : kMaxParts;
  return p;
}

hipError_t launch_rms_norm_backward(const void* dy, int dtype, int64_t dy_ld, const void* h, int h_dtype, int64_t h_ld,
                                    const float* scales, int64_t scales_ld, const void* w, int wdtype,
                                    const float* rstd, const void* dres, int64_t dres_ld, int64_t rows, int64_t dim,
                                    void* dh, int64_t dh_ld, int dh_dtype, void* dw, int grad_dtype, bool first,
                                    void* workspace, hipStream_t s) {
  const RmsPlan p = rms_plan(rows, dim);
  int parts = 0;
  float* partials = dw ? static_cast<float*>(workspace) : nullptr;
  if (rows > 0) {
    const RmsBackward a{dy, h, w, dres, scales, rstd, dh, partials, dy_ld, h_ld, scales_ld, dres_ld, dh_ld, rows,
                        (uint32_t)dim, (uint32_t)p.pitch, wdtype, dw, grad_dtype, (int)first};
    const int64_t t = dtype == ZS_BF16 ? 2 : 4, r = dh_dtype == ZS_BF16 ? 2 : 4, k = h_dtype == ZS_E4M3 ? 1 : r;
    const int64_t bytes = rows * dim * (t + k + r * (dres ? 2 : 1));
    const bool kept8 = h_dtype == ZS_E4M3;
    if (dtype == ZS_F32) parts = kept8 ? run<float, float, uint8_t, 4>(a, bytes, s) : run<float, float, float, 4>(a, bytes, s);
    else if (dh_dtype == ZS_F32) parts = kept8 ? run<uint16_t, float, uint8_t, 8>(a, bytes, s) : run<uint16_t, float, float, 8>(a, bytes, s);
    else parts = kept8 ? run<uint16_t, uint16_t, uint8_t, 8>(a, bytes, s) : run<uint16_t, uint16_t, uint16_t, 8>(a, bytes, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (dw && (parts > 0 || (rows == 0 && first))) {  // without rows the sum is zero
    const dim3 gd((unsigned)((dim + 63) / 64)), bd(kJoinWaves * 64);
    if (grad_dtype == ZS_BF16) hipLaunchKernelGGL((k_rms_dw<uint16_t>), gd, bd, 0, s, partials, p.pitch, parts, dim, (uint16_t*)dw, (int)first);
    else hipLaunchKernelGGL((k_rms_dw<float>), gd, bd, 0, s, partials, p.pitch, parts, dim, (float*)dw, (int)first);
  }
  return hipGetLastError();
}

}  // namespace zs
