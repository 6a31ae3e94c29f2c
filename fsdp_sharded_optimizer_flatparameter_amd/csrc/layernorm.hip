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
// stored. Means are products with 1 / dim, one rounding more than quotients: a
// row's three quotients in each of its lanes would take 93 instead of 88 us for
// 16384 bf16 rows of 8192, the backward's two 77 instead of 73 for 16384 of 4096.
#include "zs_launch.hpp"
#include "zs_launch_rows.hpp"
#include "zs_rows.hpp"

namespace zs {
namespace {

// Columns of piece j of lane l of a row's LPR lanes: consecutive lanes take
// consecutive pieces, so a wave's access is one contiguous span.
template <int LPR, int VEC>
__device__ __forceinline__ uint32_t col_of(int j, int l) {
  return (uint32_t)(j * LPR + l) * VEC;
}

// Weight or bias values of a piece; `missing` where the caller passes none.
template <typename W, int VEC>
__device__ __forceinline__ void load_affine(Piece<W, VEC>& r, const W* p, float missing, uint32_t c, uint32_t dim) {
  if (p) {
    take_cols<W, VEC>(r, p, c, dim);
  } else {
    r.clear();
#pragma unroll
    for (int e = 0; e < VEC; ++e) r.put(e, round_to<W>(missing));
  }
}

// Statistics of one part of a row: count, mean and the sum of squared
// distances from that mean. Parts are joined without cancellation:
// M2 = sum_p M2_p + n_p (mean_p - mean)^2.
struct Part {
  float n, mean, m2;
};

// A mean from a rounded sum is an ulp or a few off, and where a row has little
// variance 1 / sqrt(eps) makes much of that: elements that all equal 30000 would
// give 0.5 instead of 0. So with |mean| above 16 standard deviations (M2 from
// that mean) the mean is corrected by the mean of the distances from it, and M2
// is taken again: 122 us for 16384 bf16 rows of 8192 that all need it, 88.5
// where none does, 142 and 98 for 8192 fp32 rows of 8192. Below, the error is of
// the size of the other roundings, and adding up the distances of all rows beside
// their squares would cost every call: 92.6 and 100.
__device__ __forceinline__ bool off_center(float n, float mean, float m2) { return m2 * 256.0f < n * mean * mean; }

template <typename T, typename W, int LPR, int NV, int VEC, bool NT>
__global__ __launch_bounds__(LPR > 256 ? LPR : 256)
void k_ln_fwd(const T* __restrict__ x, int64_t x_ld, const W* __restrict__ w, const W* __restrict__ b,
              int64_t rows, uint32_t dim, float eps, T* __restrict__ y, int64_t y_ld,
              float* __restrict__ mean_out, float* __restrict__ rstd_out) {
  constexpr int BS = LPR > 256 ? LPR : 256;
  constexpr int RPB = BS / LPR;         // rows in flight per workgroup
  constexpr int NW = LPR / 64;          // waves per row (0 below a wave)
  constexpr int G = LPR < 64 ? LPR : 64;
  __shared__ Part parts[2][BS / 64];
  const int l = threadIdx.x % LPR;
  const int64_t step = (int64_t)gridDim.x * RPB;
  int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / LPR;
  Piece<W, VEC> wf[NV], bf[NV];  // as they lie in memory: half the registers for bf16
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
    const int left = (int)dim - (int)col_of<LPR, VEC>(j, l);
    cnt += (float)(left >= VEC ? VEC : (left > 0 ? left : 0));
  }
  cnt = lane_sum<G>(cnt);
  const float inv_cnt = 1.0f / (cnt > 0.0f ? cnt : 1.0f);
  Piece<T, VEC> raw[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) raw[j].clear();
  // every row group of the workgroup takes the same number of turns (barriers)
  int turn = 0;
  for (int64_t base = (int64_t)blockIdx.x * RPB; base < rows; base += step, row += step, turn ^= 1) {
    if (row < rows)
#pragma unroll
      for (int j = 0; j < NV; ++j) load_cols<T, VEC, NT>(raw[j], x + row * x_ld, col_of<LPR, VEC>(j, l), dim);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      wf[j].stay_packed();
      bf[j].stay_packed();
    }
    if (ragged(dim, VEC) && row < rows)
#pragma unroll
      for (int j = 0; j < NV; ++j) settle_cols<T, VEC>(raw[j], x + row * x_ld, col_of<LPR, VEC>(j, l), dim);
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < VEC; ++e) s += raw[j].get(e);
    float mean = lane_sum<G>(s) * inv_cnt;
    // sum of f(x - mean) over the elements that the wave (or group) holds
    auto over_distances = [&](auto f) {
      float q = 0.0f;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int left = (int)dim - (int)col_of<LPR, VEC>(j, l);
        if (left >= VEC) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) q = f(raw[j].get(e) - mean, q);
        } else {
#pragma unroll
          for (int e = 0; e < VEC; ++e) q = e < left ? f(raw[j].get(e) - mean, q) : q;
        }
      }
      return lane_sum<G>(q);
    };
    auto squares = [](float d, float q) { return fmaf(d, d, q); };
    float m2 = over_distances(squares);
    if (off_center(cnt, mean, m2)) {
      mean = fmaf(over_distances([](float d, float q) { return q + d; }), inv_cnt, mean);
      m2 = over_distances(squares);
    }
    if constexpr (NW > 1) {
      const int w0 = threadIdx.x / LPR * NW;  // the row's first wave
      if ((threadIdx.x & 63) == 0) parts[turn][threadIdx.x / 64] = Part{cnt, mean, m2};
      __syncthreads();  // the other turn's entries are read by nobody any more
      float total = 0.0f;
#pragma unroll
      for (int i = 0; i < NW; ++i) total += parts[turn][w0 + i].n * parts[turn][w0 + i].mean;
      mean = total * inv_dim;
      m2 = 0.0f;
#pragma unroll
      for (int i = 0; i < NW; ++i) {
        const Part p = parts[turn][w0 + i];
        const float d = p.mean - mean;
        m2 += fmaf(p.n * d, d, p.m2);
      }
      if (off_center((float)dim, mean, m2)) {  // the joined mean is a rounded sum too
        float off = 0.0f;
#pragma unroll 1
        for (int i = 0; i < NW; ++i) off = fmaf(parts[turn][w0 + i].n, parts[turn][w0 + i].mean - mean, off);
        mean = fmaf(off, inv_dim, mean);
        m2 = 0.0f;
#pragma unroll 1
        for (int i = 0; i < NW; ++i) {
          const Part p = parts[turn][w0 + i];
          const float d = p.mean - mean;
          m2 += fmaf(p.n * d, d, p.m2);
        }
      }
    }
    if (row >= rows) continue;
    const float rstd = 1.0f / sqrtf(m2 * inv_dim + eps);
    if (l == 0) {
      if (mean_out) mean_out[row] = mean;
      if (rstd_out) rstd_out[row] = rstd;
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float v[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[e] = fmaf((raw[j].get(e) - mean) * rstd, wf[j].get(e), bf[j].get(e));
      store_cols<T, VEC, NT>(y + row * y_ld, v, col_of<LPR, VEC>(j, l), dim);
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
constexpr int kMaxParts = 256;  // partial sums of the backward pass: a workgroup of 16 waves per CU

// Rows longer than the registers of 1024 lanes hold (four pieces a lane: 32768
// bf16, 16384 fp32; two where bf16 rows have fp32 weights: 16384): one workgroup
// walks over the row three times (sum, squared distances, output); the second
// and third reading find most of it in the caches. (4096 rows of 16384 fp32 took
// 143 us so, 95 in registers.) Two more readings where the mean is corrected:
// 178 instead of 138 us for 4096 bf16 rows of 28672 that all need it.
template <typename T, typename W, int VEC>
__global__ __launch_bounds__(kLongBS)
void k_ln_fwd_long(const T* __restrict__ x, int64_t x_ld, const W* __restrict__ w, const W* __restrict__ b,
                   int64_t rows, uint32_t dim, float eps, T* __restrict__ y, int64_t y_ld,
                   float* __restrict__ mean_out, float* __restrict__ rstd_out) {
  __shared__ float lds[kLongBS / 64];
  const float inv_dim = 1.0f / (float)dim;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const T* xr = x + row * x_ld;
    float s = 0.0f;
    for (uint32_t c = threadIdx.x * VEC; c < dim; c += kLongBS * VEC) {
      Piece<T, VEC> p;
      take_cols<T, VEC>(p, xr, c, dim);
      float t = 0.0f;
#pragma unroll
      for (int e = 0; e < VEC; ++e) t += p.get(e);
      s += t;
    }
    float mean = block_sum<kLongBS>(s, lds) * inv_dim;
    auto over_distances = [&](auto f) {
      float q = 0.0f;
      for (uint32_t c = threadIdx.x * VEC; c < dim; c += kLongBS * VEC) {
        Piece<T, VEC> p;
        take_cols<T, VEC>(p, xr, c, dim);
        float t = 0.0f;
#pragma unroll
        for (int e = 0; e < VEC; ++e) t = c + e < dim ? f(p.get(e) - mean, t) : t;
        q += t;
      }
      return block_sum<kLongBS>(q, lds);
    };
    auto squares = [](float d, float q) { return fmaf(d, d, q); };
    float m2 = over_distances(squares);
    if (off_center((float)dim, mean, m2)) {  // the same in all threads
      mean = fmaf(over_distances([](float d, float q) { return q + d; }), inv_dim, mean);
      m2 = over_distances(squares);
    }
    const float rstd = 1.0f / sqrtf(m2 * inv_dim + eps);
    if (threadIdx.x == 0) {
      if (mean_out) mean_out[row] = mean;
      if (rstd_out) rstd_out[row] = rstd;
    }
    for (uint32_t c = threadIdx.x * VEC; c < dim; c += kLongBS * VEC) {
      Piece<T, VEC> p;
      Piece<W, VEC> wf, bf;
      float v[VEC];
      take_cols<T, VEC>(p, xr, c, dim);
      load_affine<W, VEC>(wf, w, 1.0f, c, dim);
      load_affine<W, VEC>(bf, b, 0.0f, c, dim);
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[e] = fmaf((p.get(e) - mean) * rstd, wf.get(e), bf.get(e));
      store_cols<T, VEC>(y + row * y_ld, v, c, dim);
    }
  }
}

// Backward over the rows of one workgroup: dx, and this workgroup's sums of
// dy xh and dy per column, which go to partials[2 g], partials[2 g + 1] (rows
// of `pitch` fp32) for k_ln_grads to join. The columns' sums stay in registers
// over all rows; the row groups of a workgroup join theirs in LDS in order.
template <typename T, typename W, int LPR, int NV, int VEC, int BS, bool NT>
__global__ __launch_bounds__(BS)
void k_ln_bwd(const T* __restrict__ dy, int64_t dy_ld, const T* __restrict__ x, int64_t x_ld,
              const W* __restrict__ w, const float* __restrict__ mean_in, const float* __restrict__ rstd_in,
              int64_t rows, uint32_t dim, T* __restrict__ dx, int64_t dx_ld, float* __restrict__ partials,
              uint32_t pitch) {
  constexpr int RPB = BS / LPR;
  constexpr int NW = LPR / 64;
  constexpr int G = LPR < 64 ? LPR : 64;
  constexpr int COLS = LPR * NV * VEC;
  __shared__ float2 sums[2][BS / 64];
  __shared__ __align__(16) float joined[2][RPB > 1 ? RPB * COLS : 4];
  const int l = threadIdx.x % LPR;
  const int64_t step = (int64_t)gridDim.x * RPB;
  int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / LPR;
  struct Row {
    Piece<T, VEC> x[NV], dy[NV];
    float mean, rstd;
  };
  auto fetch = [&](int64_t r, Row& to) {
    if (r < rows) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        load_cols<T, VEC, NT>(to.x[j], x + r * x_ld, col_of<LPR, VEC>(j, l), dim);
        load_cols<T, VEC, NT>(to.dy[j], dy + r * dy_ld, col_of<LPR, VEC>(j, l), dim);
      }
      to.mean = mean_in[r];
      to.rstd = rstd_in[r];
    }
  };
  // Two pieces a lane and a row ahead do not fit in 128 registers for bf16 rows. For
  // fp32 rows they do (112), to no clear end: 8192 rows of 8192 took 144 us so
  // and 143 without, of 6144 104 and 108.
  constexpr bool AHEAD = NV == 1;
  Row next;  // the next row is on its way while this one is worked on
  next.mean = next.rstd = 0.0f;
  if (AHEAD) fetch(row, next);
  Piece<W, VEC> wf[NV];
  float dw[NV][VEC], db[NV][VEC];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    load_affine<W, VEC>(wf[j], w, 1.0f, col_of<LPR, VEC>(j, l), dim);
#pragma unroll
    for (int e = 0; e < VEC; ++e) dw[j][e] = db[j][e] = 0.0f;
  }
  const float inv_dim = 1.0f / (float)dim;
  // every row group of the workgroup takes the same number of turns (barriers)
  int turn = 0;
  for (int64_t base = (int64_t)blockIdx.x * RPB; base < rows; base += step, row += step, turn ^= 1) {
    Row now;
    if constexpr (AHEAD) now = next;
    else fetch(row, now);
#pragma unroll
    for (int j = 0; j < NV; ++j) wf[j].stay_packed();
    const bool live = row < rows;
    if (AHEAD) fetch(row + step, next);
    if (ragged(dim, VEC) && live)
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        settle_cols<T, VEC>(now.x[j], x + row * x_ld, col_of<LPR, VEC>(j, l), dim);
        settle_cols<T, VEC>(now.dy[j], dy + row * dy_ld, col_of<LPR, VEC>(j, l), dim);
      }
    const float mean = now.mean, rstd = now.rstd;
    const Piece<T, VEC>*rx = now.x, *rg = now.dy;
    float s1 = 0.0f, s2 = 0.0f;
    if (live) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float g = rg[j].get(e), xh = (rx[j].get(e) - mean) * rstd, gw = g * wf[j].get(e);
          s1 += gw;
          s2 = fmaf(gw, xh, s2);
          dw[j][e] = fmaf(g, xh, dw[j][e]);
          db[j][e] += g;
        }
      s1 = lane_sum<G>(s1);
      s2 = lane_sum<G>(s2);
    }
    if constexpr (NW > 1) {
      const int w0 = threadIdx.x / LPR * NW;  // the row's first wave
      if ((threadIdx.x & 63) == 0) sums[turn][threadIdx.x / 64] = float2{s1, s2};
      __syncthreads();  // the other turn's entries are read by nobody any more
      s1 = s2 = 0.0f;
#pragma unroll
      for (int i = 0; i < NW; ++i) {
        s1 += sums[turn][w0 + i].x;
        s2 += sums[turn][w0 + i].y;
      }
    }
    if (live) {
      const float a = s1 * inv_dim, c = s2 * inv_dim;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float v[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float xh = (rx[j].get(e) - mean) * rstd;
          v[e] = rstd * (fmaf(rg[j].get(e), wf[j].get(e), -a) - xh * c);
        }
        store_cols<T, VEC, NT>(dx + row * dx_ld, v, col_of<LPR, VEC>(j, l), dim);
      }
    }
  }
  if (!partials) return;  // uniform: an argument
  float* pw = partials + 2 * (int64_t)blockIdx.x * pitch;
  if constexpr (RPB > 1) {
    const int mine = threadIdx.x / LPR * COLS;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < VEC; e += 4) {
        const int at = mine + (j * LPR + l) * VEC + e;
        *reinterpret_cast<f32x4*>(&joined[0][at]) = f32x4{dw[j][e], dw[j][e + 1], dw[j][e + 2], dw[j][e + 3]};
        *reinterpret_cast<f32x4*>(&joined[1][at]) = f32x4{db[j][e], db[j][e + 1], db[j][e + 2], db[j][e + 3]};
      }
    __syncthreads();
    for (uint32_t c = threadIdx.x; c < COLS && c < dim; c += BS) {
      float tw = joined[0][c], tb = joined[1][c];
#pragma unroll
      for (int g = 1; g < RPB; ++g) {
        tw += joined[0][g * COLS + c];
        tb += joined[1][g * COLS + c];
      }
      pw[c] = tw;
      pw[pitch + c] = tb;
    }
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const uint32_t c = col_of<LPR, VEC>(j, l);
      if (c < pitch) {  // pitch is a multiple of VEC
        store_piece<float, VEC>(pw + c, dw[j]);
        store_piece<float, VEC>(pw + pitch + c, db[j]);
      }
    }
  }
}

// Backward of rows longer than the registers of 1024 lanes hold (16384
// elements), dx alone. (4096 rows of 16384 fp32 took 310 us so, 155 in
// registers.)
template <typename T, typename W, int VEC>
__global__ __launch_bounds__(kLongBS)
void k_ln_bwd_long(const T* __restrict__ dy, int64_t dy_ld, const T* __restrict__ x, int64_t x_ld,
                   const W* __restrict__ w, const float* __restrict__ mean_in, const float* __restrict__ rstd_in,
                   int64_t rows, uint32_t dim, T* __restrict__ dx, int64_t dx_ld) {
  __shared__ float lds[kLongBS / 64];
  const float inv_dim = 1.0f / (float)dim;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const T *xr = x + row * x_ld, *gr = dy + row * dy_ld;
    const float mean = mean_in[row], rstd = rstd_in[row];
    float s1 = 0.0f, s2 = 0.0f;
    for (uint32_t c = threadIdx.x * VEC; c < dim; c += kLongBS * VEC) {
      Piece<T, VEC> px, pg;
      Piece<W, VEC> wf;
      float t1 = 0.0f, t2 = 0.0f;
      take_cols<T, VEC>(px, xr, c, dim);
      take_cols<T, VEC>(pg, gr, c, dim);
      load_affine<W, VEC>(wf, w, 1.0f, c, dim);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float gw = pg.get(e) * wf.get(e);
        t1 += gw;
        t2 = fmaf(gw, (px.get(e) - mean) * rstd, t2);
      }
      s1 += t1;
      s2 += t2;
    }
    const float a = block_sum<kLongBS>(s1, lds) * inv_dim, k = block_sum<kLongBS>(s2, lds) * inv_dim;
    for (uint32_t c = threadIdx.x * VEC; c < dim; c += kLongBS * VEC) {
      Piece<T, VEC> px, pg;
      Piece<W, VEC> wf;
      float v[VEC];
      take_cols<T, VEC>(px, xr, c, dim);
      take_cols<T, VEC>(pg, gr, c, dim);
      load_affine<W, VEC>(wf, w, 1.0f, c, dim);
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[e] = rstd * (fmaf(pg.get(e), wf.get(e), -a) - (px.get(e) - mean) * rstd * k);
      store_cols<T, VEC>(dx + row * dx_ld, v, c, dim);
    }
  }
}

// The columns' sums for such rows: workgroup (tile, g) adds rows g, g + parts,
// ... of 256 pieces of columns.
template <typename T, int VEC>
__global__ __launch_bounds__(kThreads)
void k_ln_cols(const T* __restrict__ dy, int64_t dy_ld, const T* __restrict__ x, int64_t x_ld,
               const float* __restrict__ mean_in, const float* __restrict__ rstd_in, int64_t rows, uint32_t dim,
               float* __restrict__ partials, uint32_t pitch, int64_t tiles) {
  const int64_t parts = gridDim.x / tiles, tile = blockIdx.x % tiles, g = blockIdx.x / tiles;
  const uint32_t c = ((uint32_t)tile * kThreads + threadIdx.x) * VEC;
  float dw[VEC], db[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) dw[e] = db[e] = 0.0f;
  for (int64_t row = g; row < rows; row += parts) {
    Piece<T, VEC> px, pg;
    take_cols<T, VEC>(px, x + row * x_ld, c, dim);
    take_cols<T, VEC>(pg, dy + row * dy_ld, c, dim);
    const float mean = mean_in[row], rstd = rstd_in[row];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float d = pg.get(e);
      dw[e] = fmaf(d, (px.get(e) - mean) * rstd, dw[e]);
      db[e] += d;
    }
  }
  float* pw = partials + 2 * g * (int64_t)pitch;
  if (c < pitch) {
    store_piece<float, VEC>(pw + c, dw);
    store_piece<float, VEC>(pw + pitch + c, db);
  }
}

// Joins the workgroups' partial sums: a wave takes 64 columns of dw or db, the
// waves of a workgroup take every kJoinWaves-th partial, and their sums are
// added in wave order. The grouping depends on the sizes alone, so the result
// has the same bits on every call.
constexpr int kJoinWaves = 16;
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
  float s = 0.0f, old = 0.0f;
  if (c < dim) {
    if (wave == 0 && !first) {
      if constexpr (sizeof(Gt) == 4) old = out[c];
      else old = bf16_to_f32(out[c]);
    }
    const float* p = partials + (bias ? pitch : 0) + c;
    constexpr int U = kMaxParts / kJoinWaves;
    float v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = u * kJoinWaves + wave;
      v[u] = k < parts ? p[2 * (int64_t)k * pitch] : 0.0f;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) s += v[u];
  }
  lds[wave][lane] = s;
  __syncthreads();
  if (wave != 0 || c >= dim) return;
#pragma unroll
  for (int i = 1; i < kJoinWaves; ++i) s += lds[i][lane];
  out[c] = round_to<Gt>(first ? s : s + old);
}

// Rows that are read and written by a call of more than this many bytes bypass
// the caches: past the memory-side cache nothing of them is left for the next
// kernel, and the plain accesses were slower (16384 rows of 8192 bf16, 537 MB:
// 98.9 against 94.4 us; 8192 rows of 4096, 134 MB: 27.9 against 25.3), below
// it faster (8192 rows of 768 fp32, 50 MB: 9.0 against 10.1 us).
constexpr int64_t kStreamBytes = 100000000;
// Workgroups (of 256 lanes) of the forward pass, 4 per CU, each walking over
// its rows: 88 us for 16384 rows of 8192 bf16 (6.1 TB/s), against 95 with 768,
// 103 with 1280 and 99 with 2048. A row is loaded when the one before it is
// done: with the next row always on its way the same takes 92 us (16384 rows
// of 4096: 49 instead of 45), only 8192 fp32 rows of 8192 gain by it (91
// instead of 93).
constexpr int64_t kFwdSlots = 1024;
constexpr int kVecBf16 = 8, kVecF32 = 4;  // elements of x in 16 bytes

template <typename T, typename W, int VEC>
void run_fwd(const T* x, int64_t x_ld, const W* w, const W* b, int64_t rows, int64_t dim, float eps, T* y,
             int64_t y_ld, float* mean, float* rstd, hipStream_t s) {
  const int64_t nvec = (dim + VEC - 1) / VEC;
  const bool nt = 2 * rows * dim * (int64_t)sizeof(T) > kStreamBytes;
  auto go = [&](auto lpr, auto nv) {
    constexpr int LPR = decltype(lpr)::value, NV = decltype(nv)::value, BS = LPR > 256 ? LPR : 256;
    const int64_t need = (rows + BS / LPR - 1) / (BS / LPR);
    const int64_t slots = kFwdSlots * 256 / BS, grid = need < slots ? need : slots;
    auto launch = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(BS), 0, s, x, x_ld, w, b, rows, (uint32_t)dim, eps, y, y_ld, mean,
                         rstd);
    };
    if (nt) launch(k_ln_fwd<T, W, LPR, NV, VEC, true>);
    else launch(k_ln_fwd<T, W, LPR, NV, VEC, false>);
  };
  using std::integral_constant;
  // Four pieces of bf16 rows with fp32 weights do not fit in 128 registers (4096
  // rows of 28672: 174 us, 143 by the walk).
  constexpr bool FITS = sizeof(T) == 4 || sizeof(W) == 2;
  // By width alone, so that a row gives the same bits whatever the number of
  // rows. One piece a lane is the quickest for one row (8192 bf16: 3.7 us on
  // 1024 or 512 lanes, 4.3 on 256), two to three the fastest for many, with
  // fewer waves that have to meet (16384 rows of 4096 bf16: 48.5 us on 256
  // lanes, 52.7 on 512; 16384 of 1024: 12.5 on 64, 14.1 on 128; 8192 of 768
  // fp32: 9.1 on 64, 11.8 on 256; 16384 of 8192 bf16: 93 on 512 and on 256,
  // 122 on 1024). Four pieces of bf16 rows with bf16 weights spill 4 registers, and
  // are faster all the same: 90 us for 4096 rows of 28672, where the walk takes
  // over 140.
  if (nvec <= 16) go(integral_constant<int, 16>{}, integral_constant<int, 1>{});
  else if (nvec <= 32) go(integral_constant<int, 32>{}, integral_constant<int, 1>{});
  else if (nvec <= 64) go(integral_constant<int, 64>{}, integral_constant<int, 1>{});
  else if (nvec <= 128) go(integral_constant<int, 64>{}, integral_constant<int, 2>{});
  else if (nvec <= 192) go(integral_constant<int, 64>{}, integral_constant<int, 3>{});
  else if (nvec <= 256) go(integral_constant<int, 128>{}, integral_constant<int, 2>{});
  else if (nvec <= 512) go(integral_constant<int, 256>{}, integral_constant<int, 2>{});
  else if (nvec <= 768) go(integral_constant<int, 256>{}, integral_constant<int, 3>{});
  else if (nvec <= 1024) go(integral_constant<int, 512>{}, integral_constant<int, 2>{});
  else if (nvec <= 2048) go(integral_constant<int, 1024>{}, integral_constant<int, 2>{});
  else if (nvec <= 4096 && FITS) go(integral_constant<int, 1024>{}, integral_constant<int, FITS ? 4 : 2>{});
  else {
    const int64_t grid = rows < 2048 ? rows : 2048;
    hipLaunchKernelGGL((k_ln_fwd_long<T, W, VEC>), dim3((unsigned)grid), dim3(kLongBS), 0, s, x, x_ld, w, b, rows,
                       (uint32_t)dim, eps, y, y_ld, mean, rstd);
  }
}

// Returns the number of partial sums per column.
template <typename T, typename W, int VEC>
int run_bwd(const T* dy, int64_t dy_ld, const T* x, int64_t x_ld, const W* w, const float* mean, const float* rstd,
             int64_t rows, int64_t dim, T* dx, int64_t dx_ld, float* partials, int64_t pitch, hipStream_t s) {
  const int64_t nvec = (dim + VEC - 1) / VEC;
  const bool nt = 3 * rows * dim * (int64_t)sizeof(T) > kStreamBytes;
  int parts = (int)(rows < kMaxParts ? rows : kMaxParts);
  auto go = [&](auto lpr, auto nv) {
    constexpr int LPR = decltype(lpr)::value, NV = decltype(nv)::value, BS = 1024;
    const int64_t need = (rows + BS / LPR - 1) / (BS / LPR);
    // long rows: two turns for each workgroup before there are more of them, as
    // their partial sums cost more than the second turn
    const int64_t want = LPR >= 512 && need >= 64 ? (need + 1) / 2 : need;
    parts = (int)(want < kMaxParts ? want : kMaxParts);
    auto launch = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, dim3((unsigned)parts), dim3(BS), 0, s, dy, dy_ld, x, x_ld, w, mean, rstd, rows, dim,
                         dx, dx_ld, partials, pitch);
    };
    if (nt) launch(k_ln_bwd<T, W, LPR, NV, VEC, BS, true>);
    else launch(k_ln_bwd<T, W, LPR, NV, VEC, BS, false>);
  };
  using std::integral_constant;
  // The columns' sums come on top of the rows: two pieces of bf16 rows spill 10 registers
  // (2 with fp32 weights), four of fp32 rows 5 (15 with bf16 weights). 8192 rows
  // of 12288 bf16 take 148 us (1.6 times their floor), and 4096 rows of 16384 fp32
  // half of what the walk takes.
  if (nvec <= 16) go(integral_constant<int, 16>{}, integral_constant<int, 1>{});
  else if (nvec <= 32) go(integral_constant<int, 32>{}, integral_constant<int, 1>{});
  else if (nvec <= 64) go(integral_constant<int, 64>{}, integral_constant<int, 1>{});
  else if (nvec <= 128) go(integral_constant<int, 128>{}, integral_constant<int, 1>{});
  else if (nvec <= 256) go(integral_constant<int, 256>{}, integral_constant<int, 1>{});
  else if (nvec <= 512) go(integral_constant<int, 512>{}, integral_constant<int, 1>{});
  else if (nvec <= 1024) go(integral_constant<int, 1024>{}, integral_constant<int, 1>{});
  else if (nvec <= 2048) go(integral_constant<int, 1024>{}, integral_constant<int, 2>{});
  else if (VEC == 4 && nvec <= 4096) go(integral_constant<int, 1024>{}, integral_constant<int, VEC == 4 ? 4 : 2>{});
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
  return parts;
}

}  // namespace

LnPlan ln_plan(int64_t rows, int64_t dim) {
  LnPlan p;
  p.pitch = (dim + 7) / 8 * 8;
  p.parts = rows < kMaxParts ? rows : kMaxParts;
  return p;
}

hipError_t launch_layer_norm_forward(const void* x, int dtype, int64_t x_ld, const void* w, const void* b, int wdtype,
                                     int64_t rows, int64_t dim, float eps, void* y, int64_t y_ld, float* mean,
                                     float* rstd, hipStream_t s) {
  if (dtype == ZS_BF16) {
    if (wdtype == ZS_BF16) run_fwd<uint16_t, uint16_t, kVecBf16>((const uint16_t*)x, x_ld, (const uint16_t*)w, (const uint16_t*)b, rows, dim, eps, (uint16_t*)y, y_ld, mean, rstd, s);
    else run_fwd<uint16_t, float, kVecBf16>((const uint16_t*)x, x_ld, (const float*)w, (const float*)b, rows, dim, eps, (uint16_t*)y, y_ld, mean, rstd, s);
  } else {
    if (wdtype == ZS_BF16) run_fwd<float, uint16_t, kVecF32>((const float*)x, x_ld, (const uint16_t*)w, (const uint16_t*)b, rows, dim, eps, (float*)y, y_ld, mean, rstd, s);
    else run_fwd<float, float, kVecF32>((const float*)x, x_ld, (const float*)w, (const float*)b, rows, dim, eps, (float*)y, y_ld, mean, rstd, s);
  }
  return hipGetLastError();
}

hipError_t launch_layer_norm_backward(const void* dy, int64_t dy_ld, const void* x, int64_t x_ld, int dtype,
                                      const void* w, int wdtype, const float* mean, const float* rstd, int64_t rows,
                                      int64_t dim, void* dx, int64_t dx_ld, void* dw, void* db, int grad_dtype,
                                      bool first, void* workspace, hipStream_t s) {
  const LnPlan p = ln_plan(rows, dim);
  int parts = 0;
  const bool grads = dw || db;
  float* partials = grads ? static_cast<float*>(workspace) : nullptr;
  if (rows > 0) {
    if (dtype == ZS_BF16) {
      if (wdtype == ZS_BF16) parts = run_bwd<uint16_t, uint16_t, kVecBf16>((const uint16_t*)dy, dy_ld, (const uint16_t*)x, x_ld, (const uint16_t*)w, mean, rstd, rows, dim, (uint16_t*)dx, dx_ld, partials, p.pitch, s);
      else parts = run_bwd<uint16_t, float, kVecBf16>((const uint16_t*)dy, dy_ld, (const uint16_t*)x, x_ld, (const float*)w, mean, rstd, rows, dim, (uint16_t*)dx, dx_ld, partials, p.pitch, s);
    } else {
      if (wdtype == ZS_BF16) parts = run_bwd<float, uint16_t, kVecF32>((const float*)dy, dy_ld, (const float*)x, x_ld, (const uint16_t*)w, mean, rstd, rows, dim, (float*)dx, dx_ld, partials, p.pitch, s);
      else parts = run_bwd<float, float, kVecF32>((const float*)dy, dy_ld, (const float*)x, x_ld, (const float*)w, mean, rstd, rows, dim, (float*)dx, dx_ld, partials, p.pitch, s);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (grads && (rows > 0 || first)) {  // without rows the sums are zero
    const dim3 gd((unsigned)(2 * ((dim + 63) / 64))), bd(kJoinWaves * 64);
    if (grad_dtype == ZS_BF16) hipLaunchKernelGGL((k_ln_grads<uint16_t>), gd, bd, 0, s, partials, p.pitch, parts, dim, (uint16_t*)dw, (uint16_t*)db, (int)first);
    else hipLaunchKernelGGL((k_ln_grads<float>), gd, bd, 0, s, partials, p.pitch, parts, dim, (float*)dw, (float*)db, (int)first);
  }
  return hipGetLastError();
}

}  // namespace zs
