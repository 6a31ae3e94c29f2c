// Layer norm over rows of `dim` elements: forward and backward, with the
// reduction of the weight's and the bias's gradient over the rows.
//
//   mean = sum_k x_k / dim,  rstd = 1 / sqrt(sum_k (x_k - mean)^2 / dim + eps)
//   y_k  = (x_k - mean) rstd w_k + b_k
//
//   xh_k = (x_k - mean) rstd,  a = sum_k dy_k w_k / dim,  c = sum_k dy_k w_k xh_k / dim
//   dx_k = rstd (dy_k w_k - a - xh_k c)
//   dw_k = sum_rows dy_k xh_k,  db_k = sum_rows dy_k
//
// Both passes are bound by memory: the forward reads x and writes y, the
// backward reads x and dy and writes dx. A row stays in the registers of the
// LPR lanes that own it (16 lanes, one wave, or several waves of a workgroup),
// so each element is read once; weights are read once per workgroup, which
// walks over rows. Everything is computed in fp32 and rounded once when it is
// stored.
#include "zs_launch.hpp"
#include "zs_rows.hpp"

namespace zs {
namespace {

// Columns of piece j of lane l of a row's LPR lanes: consecutive lanes take
// consecutive pieces, so a wave's access is one contiguous span.
template <int LPR, int VEC>
__device__ __forceinline__ int64_t col_of(int j, int l) {
  return (int64_t)(j * LPR + l) * VEC;
}

template <typename T, int VEC>
__device__ __forceinline__ void load_cols(Piece<T, VEC>& p, const T* row, int64_t c, int64_t dim) {
  if (c + VEC <= dim) p.load(row + c);
  else if (c < dim) p.load_part(row + c, (int)(dim - c));
  else p.clear();
}
template <typename T, int VEC>
__device__ __forceinline__ void store_cols(T* row, const float* v, int64_t c, int64_t dim) {
  if (c + VEC <= dim) store_piece<T, VEC>(row + c, v);
  else if (c < dim) store_part<T, VEC>(row + c, v, (int)(dim - c));
}

// Weight or bias values of a piece; `missing` where the caller passes none.
template <typename W, int VEC>
__device__ __forceinline__ void load_affine(float* f, const W* p, float missing, int64_t c, int64_t dim) {
  if (!p) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) f[e] = missing;
    return;
  }
  Piece<W, VEC> r;
  load_cols<W, VEC>(r, p, c, dim);
#pragma unroll
  for (int e = 0; e < VEC; ++e) f[e] = r.get(e);
}

// Statistics of one part of a row: count, mean and the sum of squared
// distances from that mean. Parts are joined without cancellation:
// M2 = sum_p M2_p + n_p (mean_p - mean)^2.
struct Part {
  float n, mean, m2;
};

template <typename T, typename W, int LPR, int NV, int VEC>
__global__ __launch_bounds__(LPR > 256 ? LPR : 256)
void k_ln_fwd(const T* __restrict__ x, int64_t x_ld, const W* __restrict__ w, const W* __restrict__ b,
              int64_t rows, int64_t dim, float eps, T* __restrict__ y, int64_t y_ld,
              float* __restrict__ mean_out, float* __restrict__ rstd_out) {
  constexpr int BS = LPR > 256 ? LPR : 256;
  constexpr int RPB = BS / LPR;         // rows in flight per workgroup
  constexpr int NW = LPR / 64;          // waves per row (0 below a wave)
  constexpr int G = LPR < 64 ? 16 : 64;
  __shared__ Part parts[2][NW > 1 ? NW : 1];
  const int l = threadIdx.x % LPR;
  float wf[NV][VEC], bf[NV][VEC];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    load_affine<W, VEC>(wf[j], w, 1.0f, col_of<LPR, VEC>(j, l), dim);
    load_affine<W, VEC>(bf[j], b, 0.0f, col_of<LPR, VEC>(j, l), dim);
  }
  const float inv_dim = 1.0f / (float)dim;
  // elements of the row that this wave (or group of 16 lanes) holds
  float cnt = 0.0f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int64_t left = dim - col_of<LPR, VEC>(j, l);
    cnt += (float)(left >= VEC ? VEC : (left > 0 ? left : 0));
  }
  cnt = lane_sum<G>(cnt);
  int turn = 0;
  for (int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / LPR; row < rows;
       row += (int64_t)gridDim.x * RPB, turn ^= 1) {
    Piece<T, VEC> raw[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) load_cols<T, VEC>(raw[j], x + row * x_ld, col_of<LPR, VEC>(j, l), dim);
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < VEC; ++e) s += raw[j].get(e);
    float mean = lane_sum<G>(s) / (cnt > 0.0f ? cnt : 1.0f);
    float m2 = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int64_t left = dim - col_of<LPR, VEC>(j, l);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float d = raw[j].get(e) - mean;
        m2 = e < left ? fmaf(d, d, m2) : m2;
      }
    }
    m2 = lane_sum<G>(m2);
    if constexpr (NW > 1) {
      if ((threadIdx.x & 63) == 0) parts[turn][threadIdx.x / 64] = Part{cnt, mean, m2};
      __syncthreads();  // the other turn's entries are read by nobody any more
      float total = 0.0f;
#pragma unroll
      for (int i = 0; i < NW; ++i) total += parts[turn][i].n * parts[turn][i].mean;
      mean = total * inv_dim;
      m2 = 0.0f;
#pragma unroll
      for (int i = 0; i < NW; ++i) {
        const Part p = parts[turn][i];
        const float d = p.mean - mean;
        m2 += fmaf(p.n * d, d, p.m2);
      }
    }
    const float rstd = 1.0f / sqrtf(m2 * inv_dim + eps);
    if (l == 0) {
      if (mean_out) mean_out[row] = mean;
      if (rstd_out) rstd_out[row] = rstd;
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float v[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[e] = fmaf((raw[j].get(e) - mean) * rstd, wf[j][e], bf[j][e]);
      store_cols<T, VEC>(y + row * y_ld, v, col_of<LPR, VEC>(j, l), dim);
    }
  }
}

// Sum over the workgroup, the same bits in every thread. `lds` holds one value
// per wave and is free again after the second barrier.
template <int BS>
__device__ __forceinline__ float block_sum(float x, float* lds) {
  x = lane_sum<64>(x);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x / 64] = x;
  __syncthreads();
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < BS / 64; ++i) s += lds[i];
  __syncthreads();
  return s;
}

constexpr int kLongBS = 1024;

// Rows longer than the registers of 1024 lanes hold: one workgroup walks over
// the row three times (sum, squared distances, output); the second and third
// reading find most of it in the caches.
template <typename T, typename W, int VEC>
__global__ __launch_bounds__(kLongBS)
void k_ln_fwd_long(const T* __restrict__ x, int64_t x_ld, const W* __restrict__ w, const W* __restrict__ b,
                   int64_t rows, int64_t dim, float eps, T* __restrict__ y, int64_t y_ld,
                   float* __restrict__ mean_out, float* __restrict__ rstd_out) {
  __shared__ float lds[kLongBS / 64];
  const float inv_dim = 1.0f / (float)dim;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const T* xr = x + row * x_ld;
    float s = 0.0f;
    for (int64_t c = (int64_t)threadIdx.x * VEC; c < dim; c += (int64_t)kLongBS * VEC) {
      Piece<T, VEC> p;
      load_cols<T, VEC>(p, xr, c, dim);
      float t = 0.0f;
#pragma unroll
      for (int e = 0; e < VEC; ++e) t += p.get(e);
      s += t;
    }
    const float mean = block_sum<kLongBS>(s, lds) * inv_dim;
    float m2 = 0.0f;
    for (int64_t c = (int64_t)threadIdx.x * VEC; c < dim; c += (int64_t)kLongBS * VEC) {
      Piece<T, VEC> p;
      load_cols<T, VEC>(p, xr, c, dim);
      float t = 0.0f;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float d = p.get(e) - mean;
        t = c + e < dim ? fmaf(d, d, t) : t;
      }
      m2 += t;
    }
    const float rstd = 1.0f / sqrtf(block_sum<kLongBS>(m2, lds) * inv_dim + eps);
    if (threadIdx.x == 0) {
      if (mean_out) mean_out[row] = mean;
      if (rstd_out) rstd_out[row] = rstd;
    }
    for (int64_t c = (int64_t)threadIdx.x * VEC; c < dim; c += (int64_t)kLongBS * VEC) {
      Piece<T, VEC> p;
      float wf[VEC], bf[VEC], v[VEC];
      load_cols<T, VEC>(p, xr, c, dim);
      load_affine<W, VEC>(wf, w, 1.0f, c, dim);
      load_affine<W, VEC>(bf, b, 0.0f, c, dim);
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[e] = fmaf((p.get(e) - mean) * rstd, wf[e], bf[e]);
      store_cols<T, VEC>(y + row * y_ld, v, c, dim);
    }
  }
}

// Backward over the rows of one workgroup: dx, and this workgroup's sums of
// dy xh and dy per column, which go to partials[2 g], partials[2 g + 1] (rows
// of `pitch` fp32) for k_ln_grads to join. The columns' sums stay in registers
// over all rows; the row groups of a workgroup join theirs in LDS in order.
template <typename T, typename W, int LPR, int NV, int VEC>
__global__ __launch_bounds__(LPR > 256 ? LPR : 256)
void k_ln_bwd(const T* __restrict__ dy, int64_t dy_ld, const T* __restrict__ x, int64_t x_ld,
              const W* __restrict__ w, const float* __restrict__ mean_in, const float* __restrict__ rstd_in,
              int64_t rows, int64_t dim, T* __restrict__ dx, int64_t dx_ld, float* __restrict__ partials,
              int64_t pitch) {
  constexpr int BS = LPR > 256 ? LPR : 256;
  constexpr int RPB = BS / LPR;
  constexpr int NW = LPR / 64;
  constexpr int G = LPR < 64 ? 16 : 64;
  __shared__ float2 sums[2][NW > 1 ? NW : 1];
  __shared__ float joined[RPB > 1 ? 2 * LPR * NV * VEC : 1];
  const int l = threadIdx.x % LPR;
  float wf[NV][VEC], dw[NV][VEC], db[NV][VEC];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    load_affine<W, VEC>(wf[j], w, 1.0f, col_of<LPR, VEC>(j, l), dim);
#pragma unroll
    for (int e = 0; e < VEC; ++e) dw[j][e] = db[j][e] = 0.0f;
  }
  const float inv_dim = 1.0f / (float)dim;
  int turn = 0;
  for (int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / LPR; row < rows;
       row += (int64_t)gridDim.x * RPB, turn ^= 1) {
    Piece<T, VEC> rx[NV], rg[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      load_cols<T, VEC>(rx[j], x + row * x_ld, col_of<LPR, VEC>(j, l), dim);
      load_cols<T, VEC>(rg[j], dy + row * dy_ld, col_of<LPR, VEC>(j, l), dim);
    }
    const float mean = mean_in[row], rstd = rstd_in[row];
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float g = rg[j].get(e), xh = (rx[j].get(e) - mean) * rstd, gw = g * wf[j][e];
        s1 += gw;
        s2 = fmaf(gw, xh, s2);
        dw[j][e] = fmaf(g, xh, dw[j][e]);
        db[j][e] += g;
      }
    s1 = lane_sum<G>(s1);
    s2 = lane_sum<G>(s2);
    if constexpr (NW > 1) {
      if ((threadIdx.x & 63) == 0) sums[turn][threadIdx.x / 64] = float2{s1, s2};
      __syncthreads();  // the other turn's entries are read by nobody any more
      s1 = s2 = 0.0f;
#pragma unroll
      for (int i = 0; i < NW; ++i) {
        s1 += sums[turn][i].x;
        s2 += sums[turn][i].y;
      }
    }
    const float a = s1 * inv_dim, c = s2 * inv_dim;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float v[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float xh = (rx[j].get(e) - mean) * rstd;
        v[e] = rstd * (fmaf(rg[j].get(e), wf[j][e], -a) - xh * c);
      }
      store_cols<T, VEC>(dx + row * dx_ld, v, col_of<LPR, VEC>(j, l), dim);
    }
  }
  if (!partials) return;
  if constexpr (RPB > 1) {
    const int grp = threadIdx.x / LPR;
    for (int turn2 = 0; turn2 < RPB; ++turn2) {
      if (grp == turn2) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            const int at = (j * LPR + l) * VEC + e;
            if (turn2 > 0) {
              dw[j][e] = joined[at] + dw[j][e];
              db[j][e] = joined[LPR * NV * VEC + at] + db[j][e];
            }
            if (turn2 + 1 < RPB) {
              joined[at] = dw[j][e];
              joined[LPR * NV * VEC + at] = db[j][e];
            }
          }
      }
      __syncthreads();
    }
    if (grp != RPB - 1) return;
  }
  float* pw = partials + 2 * (int64_t)blockIdx.x * pitch;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int64_t c = col_of<LPR, VEC>(j, l);
    if (c < pitch) {  // pitch is a multiple of VEC
      store_piece<float, VEC>(pw + c, dw[j]);
      store_piece<float, VEC>(pw + pitch + c, db[j]);
    }
  }
}

// Backward of rows longer than the registers of 1024 lanes hold, dx alone.
template <typename T, typename W, int VEC>
__global__ __launch_bounds__(kLongBS)
void k_ln_bwd_long(const T* __restrict__ dy, int64_t dy_ld, const T* __restrict__ x, int64_t x_ld,
                   const W* __restrict__ w, const float* __restrict__ mean_in, const float* __restrict__ rstd_in,
                   int64_t rows, int64_t dim, T* __restrict__ dx, int64_t dx_ld) {
  __shared__ float lds[kLongBS / 64];
  const float inv_dim = 1.0f / (float)dim;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const T *xr = x + row * x_ld, *gr = dy + row * dy_ld;
    const float mean = mean_in[row], rstd = rstd_in[row];
    float s1 = 0.0f, s2 = 0.0f;
    for (int64_t c = (int64_t)threadIdx.x * VEC; c < dim; c += (int64_t)kLongBS * VEC) {
      Piece<T, VEC> px, pg;
      float wf[VEC], t1 = 0.0f, t2 = 0.0f;
      load_cols<T, VEC>(px, xr, c, dim);
      load_cols<T, VEC>(pg, gr, c, dim);
      load_affine<W, VEC>(wf, w, 1.0f, c, dim);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float gw = pg.get(e) * wf[e];
        t1 += gw;
        t2 = fmaf(gw, (px.get(e) - mean) * rstd, t2);
      }
      s1 += t1;
      s2 += t2;
    }
    const float a = block_sum<kLongBS>(s1, lds) * inv_dim, k = block_sum<kLongBS>(s2, lds) * inv_dim;
    for (int64_t c = (int64_t)threadIdx.x * VEC; c < dim; c += (int64_t)kLongBS * VEC) {
      Piece<T, VEC> px, pg;
      float wf[VEC], v[VEC];
      load_cols<T, VEC>(px, xr, c, dim);
      load_cols<T, VEC>(pg, gr, c, dim);
      load_affine<W, VEC>(wf, w, 1.0f, c, dim);
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[e] = rstd * (fmaf(pg.get(e), wf[e], -a) - (px.get(e) - mean) * rstd * k);
      store_cols<T, VEC>(dx + row * dx_ld, v, c, dim);
    }
  }
}

// The columns' sums for such rows: workgroup (tile, g) adds rows g, g + parts,
// ... of 256 pieces of columns.
template <typename T, int VEC>
__global__ __launch_bounds__(kThreads)
void k_ln_cols(const T* __restrict__ dy, int64_t dy_ld, const T* __restrict__ x, int64_t x_ld,
               const float* __restrict__ mean_in, const float* __restrict__ rstd_in, int64_t rows, int64_t dim,
               float* __restrict__ partials, int64_t pitch, int64_t tiles) {
  const int64_t parts = gridDim.x / tiles, tile = blockIdx.x % tiles, g = blockIdx.x / tiles;
  const int64_t c = (tile * kThreads + threadIdx.x) * VEC;
  float dw[VEC], db[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) dw[e] = db[e] = 0.0f;
  for (int64_t row = g; row < rows; row += parts) {
    Piece<T, VEC> px, pg;
    load_cols<T, VEC>(px, x + row * x_ld, c, dim);
    load_cols<T, VEC>(pg, dy + row * dy_ld, c, dim);
    const float mean = mean_in[row], rstd = rstd_in[row];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float d = pg.get(e);
      dw[e] = fmaf(d, (px.get(e) - mean) * rstd, dw[e]);
      db[e] += d;
    }
  }
  float* pw = partials + 2 * g * pitch;
  if (c < pitch) {
    store_piece<float, VEC>(pw + c, dw);
    store_piece<float, VEC>(pw + pitch + c, db);
  }
}

// Joins the workgroups' partial sums: a wave takes 64 columns of dw or db, the
// waves of a workgroup take every kJoinWaves-th partial, and their sums are
// added in wave order. The grouping depends on the sizes alone, so the result
// has the same bits on every call.
constexpr int kJoinWaves = 8;
template <typename Gt>
__global__ __launch_bounds__(kJoinWaves * 64)
void k_ln_grads(const float* __restrict__ partials, int64_t pitch, int parts, int64_t dim, Gt* __restrict__ dw,
                Gt* __restrict__ db, int first) {
  __shared__ float lds[kJoinWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t tiles = (dim + 63) / 64;
  const bool bias = blockIdx.x >= tiles;
  Gt* out = bias ? db : dw;
  if (!out) return;  // uniform across the workgroup
  const int64_t c = ((int64_t)blockIdx.x - (bias ? tiles : 0)) * 64 + lane;
  float s = 0.0f;
  if (c < dim)
    for (int p = wave; p < parts; p += kJoinWaves) s += partials[(2 * (int64_t)p + bias) * pitch + c];
  lds[wave][lane] = s;
  __syncthreads();
  if (wave != 0 || c >= dim) return;
#pragma unroll
  for (int i = 1; i < kJoinWaves; ++i) s += lds[i][lane];
  if (!first) {
    if constexpr (sizeof(Gt) == 4) s += out[c];
    else s += bf16_to_f32(out[c]);
  }
  out[c] = round_to<Gt>(s);
}

// Rows of VEC-element pieces a shape holds.
struct Shape {
  int lpr, nv;
};
constexpr int kVecBf16 = 8, kVecF32 = 4;

template <typename T, typename W, int VEC>
void run_fwd(const T* x, int64_t x_ld, const W* w, const W* b, int64_t rows, int64_t dim, float eps, T* y,
             int64_t y_ld, float* mean, float* rstd, hipStream_t s) {
  const int64_t nvec = (dim + VEC - 1) / VEC;
  auto go = [&](auto lpr, auto nv) {
    constexpr int LPR = decltype(lpr)::value, NV = decltype(nv)::value, BS = LPR > 256 ? LPR : 256;
    const int64_t need = (rows + BS / LPR - 1) / (BS / LPR);
    const int64_t grid = need < 2048 ? need : 2048;
    hipLaunchKernelGGL((k_ln_fwd<T, W, LPR, NV, VEC>), dim3((unsigned)grid), dim3(BS), 0, s, x, x_ld, w, b, rows,
                       dim, eps, y, y_ld, mean, rstd);
  };
  using std::integral_constant;
  if (nvec <= 16) go(integral_constant<int, 16>{}, integral_constant<int, 1>{});
  else if (nvec <= 64) go(integral_constant<int, 64>{}, integral_constant<int, 1>{});
  else if (nvec <= 128) go(integral_constant<int, 64>{}, integral_constant<int, 2>{});
  else if (nvec <= 256) go(integral_constant<int, 64>{}, integral_constant<int, 4>{});
  else if (nvec <= 512) go(integral_constant<int, 256>{}, integral_constant<int, 2>{});
  else if (nvec <= 1024) go(integral_constant<int, 256>{}, integral_constant<int, 4>{});
  else if (nvec <= 2048) go(integral_constant<int, 1024>{}, integral_constant<int, 2>{});
  else {
    const int64_t grid = rows < 2048 ? rows : 2048;
    hipLaunchKernelGGL((k_ln_fwd_long<T, W, VEC>), dim3((unsigned)grid), dim3(kLongBS), 0, s, x, x_ld, w, b, rows,
                       dim, eps, y, y_ld, mean, rstd);
  }
}

template <typename T, typename W, int VEC>
void run_bwd(const T* dy, int64_t dy_ld, const T* x, int64_t x_ld, const W* w, const float* mean, const float* rstd,
             int64_t rows, int64_t dim, T* dx, int64_t dx_ld, float* partials, int parts, int64_t pitch,
             hipStream_t s) {
  const int64_t nvec = (dim + VEC - 1) / VEC;
  auto go = [&](auto lpr, auto nv) {
    constexpr int LPR = decltype(lpr)::value, NV = decltype(nv)::value, BS = LPR > 256 ? LPR : 256;
    hipLaunchKernelGGL((k_ln_bwd<T, W, LPR, NV, VEC>), dim3((unsigned)parts), dim3(BS), 0, s, dy, dy_ld, x, x_ld, w,
                       mean, rstd, rows, dim, dx, dx_ld, partials, pitch);
  };
  using std::integral_constant;
  if (nvec <= 16) go(integral_constant<int, 16>{}, integral_constant<int, 1>{});
  else if (nvec <= 64) go(integral_constant<int, 64>{}, integral_constant<int, 1>{});
  else if (nvec <= 128) go(integral_constant<int, 64>{}, integral_constant<int, 2>{});
  else if (nvec <= 256) go(integral_constant<int, 256>{}, integral_constant<int, 1>{});
  else if (nvec <= 512) go(integral_constant<int, 256>{}, integral_constant<int, 2>{});
  else if (nvec <= 1024) go(integral_constant<int, 1024>{}, integral_constant<int, 1>{});
  else if (nvec <= 2048) go(integral_constant<int, 1024>{}, integral_constant<int, 2>{});
  else {
    const int64_t grid = rows < 2048 ? rows : 2048;
    hipLaunchKernelGGL((k_ln_bwd_long<T, W, VEC>), dim3((unsigned)grid), dim3(kLongBS), 0, s, dy, dy_ld, x, x_ld, w,
                       mean, rstd, rows, dim, dx, dx_ld);
    if (partials) {
      const int64_t tiles = (nvec + kThreads - 1) / kThreads;
      hipLaunchKernelGGL((k_ln_cols<T, VEC>), dim3((unsigned)(tiles * parts)), dim3(kThreads), 0, s, dy, dy_ld, x,
                         x_ld, mean, rstd, rows, dim, partials, pitch, tiles);
    }
  }
}

}  // namespace

LnPlan ln_plan(int64_t rows, int64_t dim) {
  LnPlan p;
  p.pitch = (dim + 7) / 8 * 8;
  p.parts = rows < 512 ? rows : 512;
  return p;
}

hipError_t launch_layer_norm_forward(const void* x, int dtype, int64_t x_ld, const void* w, const void* b, int wdtype,
                                     int64_t rows, int64_t dim, float eps, void* y, int64_t y_ld, float* mean,
                                     float* rstd, hipStream_t s) {
  if (dtype == ZS_BF16) {
    if (wdtype == ZS_BF16) run_fwd<uint16_t, uint16_t, kVecBf16>((const uint16_t*)x, x_ld, (const uint16_t*)w, (const uint16_t*)b, rows, dim, eps, (uint16_t*)y, y_ld, mean, rstd, s);
    else run_fwd<uint16_t, float, kVecBf16>((const uint16_t*)x, x_ld, (const float*)w, (const float*)b, rows, dim, eps, (uint16_t*)y, y_ld, mean, rstd, s);
  } else {
    if (wdtype == ZS_BF16) run_fwd<float, uint16_t, kVecBf16>((const float*)x, x_ld, (const uint16_t*)w, (const uint16_t*)b, rows, dim, eps, (float*)y, y_ld, mean, rstd, s);
    else run_fwd<float, float, kVecF32>((const float*)x, x_ld, (const float*)w, (const float*)b, rows, dim, eps, (float*)y, y_ld, mean, rstd, s);
  }
  return hipGetLastError();
}

hipError_t launch_layer_norm_backward(const void* dy, int64_t dy_ld, const void* x, int64_t x_ld, int dtype,
                                      const void* w, int wdtype, const float* mean, const float* rstd, int64_t rows,
                                      int64_t dim, void* dx, int64_t dx_ld, void* dw, void* db, int grad_dtype,
                                      bool first, void* workspace, hipStream_t s) {
  const LnPlan p = ln_plan(rows, dim);
  const bool grads = dw || db;
  float* partials = grads ? static_cast<float*>(workspace) : nullptr;
  if (rows > 0) {
    const int parts = (int)p.parts;
    if (dtype == ZS_BF16) {
      if (wdtype == ZS_BF16) run_bwd<uint16_t, uint16_t, kVecBf16>((const uint16_t*)dy, dy_ld, (const uint16_t*)x, x_ld, (const uint16_t*)w, mean, rstd, rows, dim, (uint16_t*)dx, dx_ld, partials, parts, p.pitch, s);
      else run_bwd<uint16_t, float, kVecBf16>((const uint16_t*)dy, dy_ld, (const uint16_t*)x, x_ld, (const float*)w, mean, rstd, rows, dim, (uint16_t*)dx, dx_ld, partials, parts, p.pitch, s);
    } else {
      if (wdtype == ZS_BF16) run_bwd<float, uint16_t, kVecBf16>((const float*)dy, dy_ld, (const float*)x, x_ld, (const uint16_t*)w, mean, rstd, rows, dim, (float*)dx, dx_ld, partials, parts, p.pitch, s);
      else run_bwd<float, float, kVecF32>((const float*)dy, dy_ld, (const float*)x, x_ld, (const float*)w, mean, rstd, rows, dim, (float*)dx, dx_ld, partials, parts, p.pitch, s);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (grads && (rows > 0 || first)) {  // without rows the sums are zero
    const dim3 gd((unsigned)(2 * ((dim + 63) / 64))), bd(kJoinWaves * 64);
    if (grad_dtype == ZS_BF16) hipLaunchKernelGGL((k_ln_grads<uint16_t>), gd, bd, 0, s, partials, p.pitch, (int)p.parts, dim, (uint16_t*)dw, (uint16_t*)db, (int)first);
    else hipLaunchKernelGGL((k_ln_grads<float>), gd, bd, 0, s, partials, p.pitch, (int)p.parts, dim, (float*)dw, (float*)db, (int)first);
  }
  return hipGetLastError();
}

}  // namespace zs
