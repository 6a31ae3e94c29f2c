// Softmax cross entropy of a large vocabulary from the hidden states h_i and the
// head's rows w_v, and its gradients, without keeping the logits:
//
//   z_iv = h_i . w_v,  lse_i = log sum_v exp z_iv,  loss_i = lse_i - z_i,label_i
//   g_iv = c_i (exp(z_iv - lse_i) - [v = label_i])      (c_i: the gradient of loss_i)
//   dh_i = sum_v g_iv w_v,  dw_v = sum_i g_iv h_i
//
// All four sums are products on the matrix units (2 n vocab dim operations
// each; the backward pass makes the logits again), which bound both passes for
// more than some hundred tokens; below, reading the head does. The forward's
// tiles leave the maximum and the sum of exponentials of their 128 or 256 rows
// of the head for each token, which a second kernel joins. The backward takes a
// piece of the vocabulary at a time: its g goes to the workspace, from which the
// products for dh (added up in fp32 over the pieces) and for these rows' dw are
// made.
//
// Tokens whose label is outside of the vocabulary count nowhere: those that
// count are moved together first, so the others cost nothing, and nothing that
// their hidden states hold reaches a sum.
//
// Rounding: bf16 products are exact and added in fp32. g is rounded to bf16 for
// gradients in bf16, which are rounded as much themselves; for an fp32
// gradient it is a sum of three bf16 (24 bits; two of them take 2.75 instead of 3.4 ms
// for 8192 tokens, 50257 x 768, but leave dw up to 2.4e-6 off, where fp32 products
// leave 1.6e-6), and the three operands of an fp32 head's gradients are sums of three,
// whose products below 2^-21 of the largest are left out. The loss, and the logits of
// many tokens for the gradients, take fp32 rows as sums of two fp16.
//
// Measured: 8192 tokens, 128256 x 4096 bf16: the loss 6.7 ms (its logits 6.5, 1330
// TFLOP/s), the gradients 21 ms (1230 TFLOP/s); one token: 181 us, 5.8 TB/s; 8192
// tokens, 50257 x 768 into an fp32 accumulator: 3.4 ms, of which the logits 1.06 (600
// TFLOP/s: a tile has 12 stages, then 2.5 GB of g), dh 0.81, dw 1.6 (1210 TFLOP/s).
#include <type_traits>

#include "zs_e4m3.hpp"
#include "zs_gemm.hpp"
#include "zs_launch.hpp"
#include "zs_launch_head.hpp"
#include "zs_rows.hpp"

namespace zs {
namespace {

using Wide = GemmShape<256, 256, 2, 4>;
using Square = GemmShape<128, 128, 2, 2>;
using Narrow = GemmShape<256, 64, 4, 1>;  // at most 64 tokens: the head's rows stream past them

// The smallest products come first: a sum rounds by its size so far.
constexpr Segments kOne{1, 0, 0};
constexpr Segments kOneThree{3, 0x000, 0x012};    // one plane times three
constexpr Segments kThree{3, 0x010, 0x001};       // 2 x 2 planes without the last
constexpr Segments kSix{6, 0x010120, 0x001102};   // 3 x 3 planes, those above 2^-21
constexpr Segments kHalves{3, 0x021, 0x012};      // fp16 planes hi, hi 2^-11, lo 2^11

// What is kept of each token that counts, in the order in which they are moved
// together: its label (-1: none), the gradient of its loss, its log sum of
// exponentials, its row and what the rounding of g at its label left. inverse: the
// place of row i, -1 where it does not count.
struct Tokens {
  int32_t *label, *map, *inverse, *count;
  float *coef, *lse, *rest;
};

// ---------------------------------------------------------------- tokens

// Labels as the caller gives them: -1 for those outside of the vocabulary.
struct Labels {
  const void* p;
  int wide;  // int64, else int32
  int64_t vocab;
  __device__ __forceinline__ int at(int64_t i) const {
    const int64_t id = wide ? ((const int64_t*)p)[i] : (int64_t)((const int32_t*)p)[i];
    return id >= 0 && id < vocab ? (int)id : -1;
  }
};

constexpr int kTokBS = 1024;
constexpr int kTokEach = 4;

// One workgroup walks over the labels, four to a thread, and numbers those that
// count (or, with `gather` 0, keeps every row where it is). Rows that do not
// count get zeros in loss and lse_out where given.
template <typename I>
__global__ __launch_bounds__(kTokBS)
void k_tokens(const I* __restrict__ labels, int64_t n, int64_t vocab, int gather, const float* __restrict__ lse_in,
              const float* __restrict__ dloss, float scale, Tokens t, float* __restrict__ loss,
              float* __restrict__ lse_out) {
  __shared__ int waves[2][kTokBS / 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int base = 0, turn = 0;
  for (int64_t at = 0; at < n; at += kTokBS * kTokEach, turn ^= 1) {
    // of the wave's 256 rows lane l has l, l + 64, ...: whole lines, and their order by masks
    const int64_t first = at + (int64_t)wave * 64 * kTokEach + lane;
    int64_t id[kTokEach];
    float ls[kTokEach], dl[kTokEach];
    uint64_t mask[kTokEach];
    int all_mine = 0;
#pragma unroll
    for (int k = 0; k < kTokEach; ++k) {
      const int64_t i = first + 64 * k;
      id[k] = i < n ? (int64_t)labels[i] : -1;
      ls[k] = lse_in && i < n ? lse_in[i] : 0.0f;
      dl[k] = dloss && i < n ? dloss[i] : 1.0f;
    }
#pragma unroll
    for (int k = 0; k < kTokEach; ++k) {
      const bool counts = id[k] >= 0 && id[k] < vocab;
      mask[k] = __ballot(gather ? counts : first + 64 * k < n);
      all_mine += __popcll(mask[k]);
    }
    if (lane == 0) waves[turn][wave] = all_mine;
    __syncthreads();  // the other turn's entries are read by nobody any more
    int before = base, all = 0;
#pragma unroll
    for (int w = 0; w < kTokBS / 64; ++w) {
      const int c = waves[turn][w];
      before += w < wave ? c : 0;
      all += c;
    }
#pragma unroll
    for (int k = 0; k < kTokEach; ++k) {
      const int64_t i = first + 64 * k;
      const bool counts = id[k] >= 0 && id[k] < vocab;
      const int place = before + __popcll(mask[k] & ((1ull << lane) - 1));
      before += __popcll(mask[k]);
      if (mask[k] >> lane & 1) {
        t.label[place] = counts ? (int32_t)id[k] : -1;
        t.map[place] = (int32_t)i;
        if (lse_in) {
          t.lse[place] = ls[k];
          t.coef[place] = counts ? scale * dl[k] : 0.0f;
        }
      }
      if (i < n) {
        t.inverse[i] = counts ? place : -1;
        if (!counts && loss) loss[i] = 0.0f;
        if (!counts && lse_out) lse_out[i] = 0.0f;
      }
    }
    base += all;
  }
  if (threadIdx.x == 0) *t.count = base;
}

// ---------------------------------------------------------------- layout

__device__ __forceinline__ uint32_t bits_hi(uint32_t a, uint32_t b) {  // upper halves of a (low) and b (high)
  return (a >> 16) | (b & 0xffff0000u);
}

// A value as three bf16 in the upper halves of p: the first cut off (a rounded one could overflow), the
// others what is left, rounded: 24 bits together. Infinities and NaN are whole in the first.
__device__ __forceinline__ void three_planes(float x, uint32_t (&p)[3]) {
  const uint32_t u = __float_as_uint(x);
  const bool whole = (u & 0x7f800000u) == 0x7f800000u;
  p[0] = whole && (u & 0x007fffffu) ? u | 0x00400000u : u & 0xffff0000u;  // a NaN stays one without its lower half
  const float r1 = whole ? 0.0f : x - __uint_as_float(u & 0xffff0000u);
  p[1] = pack_bf16(r1, r1) & 0xffff0000u;
  const float r2 = r1 - __uint_as_float(p[1]);
  p[2] = pack_bf16(r2, r2) & 0xffff0000u;
}

// Rows of `dim` elements as bf16 planes of `dp` elements each, zeros behind dim.
// With `map`, row r is row map[r] of the source, for r below *count, and zeros
// for the rows up to the next multiple of 64.
template <typename T>
__global__ __launch_bounds__(kThreads)
void k_layout(const T* __restrict__ src, int64_t ld, uint32_t dim, int64_t rows, uint16_t* __restrict__ dst, int64_t dp,
              const int32_t* __restrict__ map, const int32_t* __restrict__ count) {
  constexpr int PLANES = sizeof(T) == 4 ? 3 : 1;
  const int64_t per = dp / 8;  // pieces of a row
  const int64_t live = count ? *count : rows, all = count ? (live + 63) / 64 * 64 : rows;
  for (int64_t at = (int64_t)blockIdx.x * kThreads + threadIdx.x; at < all * per; at += (int64_t)gridDim.x * kThreads) {
    const int64_t r = at / per;
    const uint32_t c = (uint32_t)(at % per) * 8;
    Piece<T, 8> p;
    p.clear();
    if (r < live) take_cols<T, 8>(p, src + (map ? (int64_t)map[r] : r) * ld, c, dim);
    uint16_t* to = dst + r * dp * PLANES + c;
    if constexpr (sizeof(T) == 2) {
      st16(u32x4{p.r[0], p.r[1], p.r[2], p.r[3]}, to);
    } else {
      uint32_t v[8][3];
#pragma unroll
      for (int e = 0; e < 8; ++e) three_planes(p.get(e), v[e]);
#pragma unroll
      for (int k = 0; k < 3; ++k)
        st16(u32x4{bits_hi(v[0][k], v[1][k]), bits_hi(v[2][k], v[3][k]), bits_hi(v[4][k], v[5][k]),
                   bits_hi(v[6][k], v[7][k])}, to + k * dp);
    }
  }
}

// fp32 rows for the logits, as fp16: with 2^k the power of two that brings the
// row's largest finite magnitude to [2^14, 2^15), x 2^k = hi + lo, of 11 bits each, lie
// as planes hi, hi 2^-11 and lo 2^11 (so that lo is rarely subnormal), of `dp` elements.
// hi hi' + (hi 2^-11)(lo' 2^11) + (lo 2^11)(hi' 2^-11) is the product of two rows
// within 3 2^-22 |x x'|, where hi 2^-11 is subnormal within 2^-39 of the one's |x| by
// the other's largest, in three products instead of bf16's six. power takes -k.
// Infinities lie in hi alone, so that they meet each value once. A wave takes a row,
// and reads it twice.
//
// BOTH: the three bf16 planes of the gradients' products beside them, with zeros for the
// rows behind the last up to a multiple of 64.
template <bool BOTH>
__global__ __launch_bounds__(kThreads)
void k_layout_half(const float* __restrict__ src, int64_t ld, uint32_t dim, int64_t rows, uint16_t* __restrict__ dst,
                   int64_t dp, int32_t* __restrict__ power, const int32_t* __restrict__ map, const int32_t* __restrict__ count,
                   uint16_t* __restrict__ planes) {
  const int lane = threadIdx.x & 63;
  const int64_t live = count ? *count : rows, all = BOTH && count ? (live + 63) / 64 * 64 : live;
  for (int64_t r = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); r < all; r += (int64_t)gridDim.x * 4) {
    if (BOTH && r >= live) {
      for (int64_t c = lane * 8; c < 3 * dp; c += 64 * 8) *(u32x4*)(planes + r * dp * 3 + c) = u32x4{0u, 0u, 0u, 0u};
      continue;
    }
    const float* from = src + (map ? (int64_t)map[r] : r) * ld;
    float top = 0.0f;
    for (uint32_t c = lane * 8; c < dim; c += 64 * 8) {
      Piece<float, 8> p;
      take_cols<float, 8>(p, from, c, dim);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float x = fabsf(p.get(e));
        top = x < INFINITY ? fmaxf(top, x) : top;
      }
    }
    top = lane_max<32>(top);
    const auto both = __builtin_amdgcn_permlane32_swap(__float_as_uint(top), __float_as_uint(top), false, false);
    top = fmaxf(__uint_as_float(both[0]), __uint_as_float(both[1]));
    const int e = (int)(__float_as_uint(top) >> 23) - 127;
    const int k = top == 0.0f ? 0 : 14 - e > 126 ? 126 : 14 - e;
    const float s = __uint_as_float((uint32_t)(127 + k) << 23);
    if (lane == 0) power[r] = -k;
    for (uint32_t c = lane * 8; c < dp; c += 64 * 8) {
      Piece<float, 8> p;
      p.clear();
      take_cols<float, 8>(p, from, c, dim);
      f16x8 hi, low, lo;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float x = p.get(i) * s;
        hi[i] = (_Float16)x;
        const bool finite = fabsf(x) < INFINITY;
        low[i] = finite ? (_Float16)((float)hi[i] * 0x1p-11f) : (_Float16)0.0f;
        lo[i] = finite ? (_Float16)((x - (float)hi[i]) * 0x1p11f) : (_Float16)0.0f;
      }
      uint16_t* to = dst + r * dp * 3 + c;
      *(f16x8*)to = hi;
      *(f16x8*)(to + dp) = low;
      *(f16x8*)(to + 2 * dp) = lo;
      if constexpr (BOTH) {
        uint32_t t[8][3];
#pragma unroll
        for (int i = 0; i < 8; ++i) three_planes(p.get(i), t[i]);
#pragma unroll
        for (int k = 0; k < 3; ++k)
          *(u32x4*)(planes + r * dp * 3 + k * dp + c) =
              u32x4{bits_hi(t[0][k], t[1][k]), bits_hi(t[2][k], t[3][k]), bits_hi(t[4][k], t[5][k]), bits_hi(t[6][k], t[7][k])};
      }
    }
  }
}

// ---------------------------------------------------------------- products

// Which tile a workgroup takes. Workgroups go round robin over the 8 XCDs, each
// with an L2 of its own: an XCD takes tiles that lie together, eight rows of
// tiles deep, so that its workgroups share both operands' panels.
struct Tile {
  int64_t m, n;
};
__device__ __forceinline__ Tile tile_of(uint32_t id, uint32_t total, uint32_t tm, uint32_t tn) {
  constexpr uint32_t DEEP = 8;
  const uint32_t xcd = id & 7, per = total >> 3, rest = total & 7;
  const uint32_t at = xcd * per + (xcd < rest ? xcd : rest) + (id >> 3);
  const uint32_t g = at / (DEEP * tn), in = at % (DEEP * tn);
  const uint32_t deep = tm - g * DEEP < DEEP ? tm - g * DEEP : DEEP;
  return Tile{g * DEEP + in % deep, in / deep};
}

template <class S>
__device__ __forceinline__ void clear(typename S::Acc& acc) {
#pragma unroll
  for (int i = 0; i < S::TM; ++i)
#pragma unroll
    for (int j = 0; j < S::TN; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
}

__device__ __forceinline__ float join4(float x, bool take_max) {  // over the lanes l, l ^ 16, l ^ 32, l ^ 48
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  const float a0 = __uint_as_float(a[0]), a1 = __uint_as_float(a[1]);
  x = take_max ? fmaxf(a0, a1) : a0 + a1;
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  const float b0 = __uint_as_float(b[0]), b1 = __uint_as_float(b[1]);
  return take_max ? fmaxf(b0, b1) : b0 + b1;
}

constexpr float kLog2e = 1.44269504088896340736f;
__device__ __forceinline__ float exp_of(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }

// Between a wave's accesses to LDS that other lanes of it have written or still read: LDS
// keeps a wave's order, so this tells the compiler alone and costs no instruction.
__device__ __forceinline__ void wave_lds() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// The tiles of one workgroup, one after another: make(at) aims the loop at a tile,
// finish(at) uses its products and says whether all lanes have sent off at least
// kStored stores.
template <class S, GemmMode MA, GemmMode MB, bool HALF = false, typename Make, typename Finish>
__device__ __forceinline__ void tiles_of(char* lds, uint32_t total, uint32_t tm, uint32_t tn, Make&& make, Finish&& finish) {
  TileLoop<S, MA, MB, HALF> loop;
  uint32_t id = blockIdx.x;
  if (id >= total) return;  // uniform
  Tile at = tile_of(id, total, tm, tn);
  make(loop, at);
  loop.preload(lds);
  bool stored = false;
  while (true) {
    typename S::Acc acc;
    clear<S>(acc);
    loop.run(lds, acc, stored);
    const Tile done = at;
    id += gridDim.x;
    if (id < total) {
      at = tile_of(id, total, tm, tn);
      make(loop, at);
      loop.preload(lds);
    }
    stored = finish(done, acc);
    if (id >= total) return;
  }
}

// Partial maxima and sums that a tile leaves for each token: one, joined in LDS, where the
// workgroups that share a CU's 160 KB have room for that beside their stages (8 bytes for each wave
// and token of a tile), else one for each row of waves.
template <class S>
constexpr int parts_of_tile() {
  constexpr int sharing = 2 * S::LDS <= 160 * 1024 ? 2 : 1, joined = S::WM * S::BN * 8;
  return sharing * (S::LDS + joined) <= 160 * 1024 ? 1 : S::WM;
}
static_assert(parts_of_tile<Wide>() == 1 && parts_of_tile<Square>() == 1 && parts_of_tile<Narrow>() == 4,
              "the room for the tiles' maxima in head_plan is for 128 rows of the head, or 64 of a narrow tile's");

// Rows of the tile are rows of the head, columns tokens: a lane holds 4 TM
// logits of each of its TN tokens. PLANES: 0 for the loss, else those of g. HALF:
// the operands are k_layout_half's.
template <class S, int PLANES, bool HALF = false>
__global__ __launch_bounds__(S::THREADS, 2)
void k_logits(GemmSide w, GemmSide h, Segments segs, int steps, int64_t v0, Tokens tok, float2* __restrict__ parts,
              float* __restrict__ own, int64_t np, uint16_t* __restrict__ g, int64_t gp, const int32_t* __restrict__ w_power,
              const int32_t* __restrict__ h_power) {
  __shared__ __align__(1024) char lds[S::LDS];
  constexpr int ROWS = S::BM / S::WM;  // of a wave
  // The waves of a tile join their maxima and sums in LDS, or leave them apart where two
  // workgroups' stages fill it.
  constexpr int APART = parts_of_tile<S>();
  __shared__ float2 joined[PLANES == 0 && APART == 1 ? S::WM * S::BN : 1];
  // The lanes of a store hold 32 bytes each of 16 tokens' rows of g. By way of LDS, where
  // there is room, they are whole lines: 453 instead of 581 us for 8192 tokens, 21760
  // rows of 768 in three planes. The chunk of 16 bytes c of token t lies at place c ^ t.
  constexpr bool LINES = PLANES > 0 && APART == 1;
  constexpr int CHUNKS = ROWS / 8;
  __shared__ __align__(16) u32x4 lines[LINES ? S::WM * S::WN : 1][LINES ? 16 * CHUNKS : 1];
  const int64_t count = *tok.count, written = PLANES ? (count + 63) / 64 * 64 : count;
  const uint32_t tm = (uint32_t)((w.rows + S::BM - 1) / S::BM), tn = (uint32_t)((written + S::BN - 1) / S::BN);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / S::WN, wn = wave % S::WN, q4 = (lane >> 4) * 4;
  auto make = [&](auto& loop, const Tile& at) {
    loop.aim(w, h, at.m * S::BM, at.n * S::BN, segs, steps, 0, segs.count * steps);
  };
  auto finish = [&](const Tile& at, typename S::Acc& acc) {
    const int64_t first = at.m * S::BM + wm * ROWS;  // the wave's first row, from v0 on
    const int left = (int)(w.rows - first) - q4;     // rows of the head from acc[0][.][0] on
    // a wave whose rows and tokens are all there needs no comparison for each logit
    const bool whole = w.rows - first >= ROWS && at.n * S::BN + S::BN <= count;
    const bool whole_tile = w.rows - at.m * S::BM >= S::BM && at.n * S::BN + S::BN <= count;  // the same in all waves
#pragma unroll
    for (int j = 0; j < S::TN; ++j) {
      const int col = wn * (S::BN / S::WN) + j * 16 + (lane & 15);
      const int64_t token = at.n * S::BN + col;
      const bool live = token < count;
      const int label = live ? tok.label[token] : -1;
      const int mine = label >= 0 ? (int)(label - v0 - first) - q4 : -1;  // the label's place among the lane's rows
      const bool hit = __any(mine >= 0 && mine < 16 * S::TM && (mine & 15) < 4);
      auto each = [&](auto f) {
#pragma unroll
        for (int i = 0; i < S::TM; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[i][j][r] = f(acc[i][j][r], 16 * i + r);
      };
      if constexpr (HALF) {
        const int of_token = live ? h_power[token] : 0;
#pragma unroll
        for (int i = 0; i < S::TM; ++i) {
          const int4 of_row = *(const int4*)(w_power + first + q4 + 16 * i);  // whole tiles have a place
          acc[i][j][0] = ldexpf(acc[i][j][0], of_row.x + of_token);
          acc[i][j][1] = ldexpf(acc[i][j][1], of_row.y + of_token);
          acc[i][j][2] = ldexpf(acc[i][j][2], of_row.z + of_token);
          acc[i][j][3] = ldexpf(acc[i][j][3], of_row.w + of_token);
        }
      }
      if constexpr (PLANES == 0) {
        if (!whole) each([&](float z, int row) { return row < left ? z : -INFINITY; });
        if (hit)
          each([&](float z, int row) {
            if (row == mine) own[token] = z;
            return z;
          });
        float top = -INFINITY;
        each([&](float z, int) {
          top = fmaxf(top, z);
          return z;
        });
        top = join4(top, true);
        const float from = top == -INFINITY ? 0.0f : top;  // exp(-inf) = 0 where all are that, not of -inf + inf
        float sum = 0.0f;
        each([&](float z, int) {
          sum += exp_of(z - from);
          return z;
        });
        sum = join4(sum, false);
        if constexpr (APART > 1) {
          if (q4 == 0 && live) parts[(at.m * APART + wm) * np + token] = float2{top, sum};
        } else {
          if (j == 0) __syncthreads();  // nobody reads the last tile's any more
          if (q4 == 0) joined[wm * S::BN + col] = float2{top, sum};
        }
      } else {
        const float lse = live ? tok.lse[token] : 0.0f, coef = live ? tok.coef[token] : 0.0f;
        each([&](float z, int) { return exp_of(z - lse); });
        if (hit) each([&](float p, int row) { return row == mine ? p - 1.0f : p; });
        if (whole) each([&](float p, int) { return coef * p; });
        else each([&](float p, int row) { return live && row < left ? coef * p : 0.0f; });
        if (hit)
          each([&](float d, int row) {
            if (row == mine) tok.rest[token] = d - bf16_lo(pack_bf16(d, d));
            return d;
          });
        if (LINES && whole_tile) {
          u32x4* mine_of = lines[wave];
          const int t = lane & 15;
#pragma unroll
          for (int k = 0; k < PLANES; ++k) {
#pragma unroll
            for (int i = 0; i < S::TM; ++i) {
              f32x4& d = acc[i][j];
              const uint2 v = uint2{pack_bf16(d.x, d.y), pack_bf16(d.z, d.w)};
              if (k + 1 < PLANES)  // what is left for the next plane
                d = f32x4{d.x - bf16_lo(v.x), d.y - bf16_hi(v.x), d.z - bf16_lo(v.y), d.w - bf16_hi(v.y)};
              const int place = (2 * i + (lane >> 5)) ^ (t & (CHUNKS - 1));
              reinterpret_cast<uint2*>(mine_of + t * CHUNKS + place)[lane >> 4 & 1] = v;
            }
            wave_lds();
#pragma unroll
            for (int x = 0; x < 16 * CHUNKS / 64; ++x) {
              const int at16 = x * 64 + lane, t2 = at16 / CHUNKS, c = at16 % CHUNKS;
              const u32x4 v = mine_of[t2 * CHUNKS + (c ^ (t2 & (CHUNKS - 1)))];
              *(u32x4*)(g + (token - t + t2) * gp * PLANES + k * gp + first + c * 8) = v;
            }
            wave_lds();
          }
          continue;
        }
        uint16_t* row = g + token * gp * PLANES + first + q4;
#pragma unroll
        for (int i = 0; i < S::TM; ++i) {
          if (!whole_tile && (token >= written || first + 16 * i >= gp)) continue;
          f32x4 d = acc[i][j];
#pragma unroll
          for (int k = 0; k < PLANES; ++k) {
            const uint2 v = uint2{pack_bf16(d.x, d.y), pack_bf16(d.z, d.w)};
            *(uint2*)(row + 16 * i + k * gp) = v;
            d = f32x4{d.x - bf16_lo(v.x), d.y - bf16_hi(v.x), d.z - bf16_lo(v.y), d.w - bf16_hi(v.y)};
          }
        }
      }
    }
    if constexpr (PLANES == 0 && APART > 1) return false;
    if constexpr (PLANES == 0 && APART == 1) {
      __syncthreads();
      for (int c = threadIdx.x; c < S::BN; c += S::THREADS) {
        const int64_t token = at.n * S::BN + c;
        if (token >= count) continue;
        float top = joined[c].x;
#pragma unroll
        for (int i = 1; i < S::WM; ++i) top = fmaxf(top, joined[i * S::BN + c].x);
        const float from = top == -INFINITY ? 0.0f : top;
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < S::WM; ++i) sum += joined[i * S::BN + c].y * exp_of(joined[i * S::BN + c].x - from);
        parts[at.m * np + token] = float2{top, sum};
      }
      return false;
    }
    return whole_tile && (LINES ? S::TN * 16 * CHUNKS / 64 * PLANES : S::TM * S::TN) >= 16;
  };
  tiles_of<S, K_IN_ROWS, K_IN_ROWS, HALF>(lds, tm * tn, tm, tn, make, finish);
}

// The loss of few tokens: the head's rows stream through registers once, as they
// lie, whatever their type and alignment. A wave takes 16 rows at a time as one
// operand of 16 x 16 products and NT times 16 tokens (the last one's copies behind
// them) as the other; lane l loads 16 bytes of row l % 16, at piece l / 16 of each
// 64 bytes, so a wave's instruction takes 64 bytes of each row. bf16 products take
// 32 values of k, fp32 ones 4: which k a lane holds does not matter as long as both
// operands agree. The tokens' pieces come from the caches. Running maxima and sums
// stay with the lanes over all rows of a wave.
//
// 16-byte loads at odd multiples of 2 bytes take three times as long here (4
// tokens, 41246 rows of 1856: 30 us, and 101 with a row stride of 1857). So a
// wave takes rows of the same parity, every second one where strides are odd,
// leaves the first element of rows that start off the 4-byte grid to a product of
// its own, and takes the tokens from a copy that starts one element later.
constexpr int kFewTokens = 64;
constexpr int kFewWaves = 4096;    // 4 workgroups of 4 waves on each CU
// Rows that the narrow tiles take as they lie are read as fast by them, or faster from some tokens on (16 tokens of
// bf16, 128256 rows of 4096: 181 us, 242 here; 41246 rows of 1856: 44, 45 here; 64 tokens: 46, 104 here); what they would
// have to lay out first is not (41246 rows of 1855, 4 tokens: 100 in all, 41 here; 64: 92, 111 here; fp32, 20 tokens,
// 41246 rows of 1856: over 260, 105 here).
constexpr int kFewAligned = 8;

// KEPT: for fp32 gradients, with the logits of token i and row v in own[i np + v], of `each`
// columns to a part (blockIdx.y), which lie `apart` elements from each other. An error of
// a logit is one of its g relative to it, and the fp32 products round 512 times in a sum of
// 512; so two pieces at a time are taken apart to three bf16 each, whose products round once
// for 32, the small ones into a sum of their own (64 tokens, 5000 x 1027: the gradients
// are 0.3e-6 off, those of the plain fp32 form 1.2e-6; 3 tokens, 5203 x 7616: 47 us, 33 with fp32 products).
template <typename T, int NT, bool KEPT = false>
__global__ __launch_bounds__(kThreads, 3)
void k_logits_few(const T* __restrict__ w, int64_t w_ld, const T* __restrict__ h0, const T* __restrict__ h1, int64_t h_ld,
                  int n, int64_t vocab, uint32_t dim, int64_t groups, Labels labels, float2* __restrict__ parts,
                  float* __restrict__ own, int64_t np, uint32_t each, int64_t apart) {
  constexpr int VEC = 16 / (int)sizeof(T), U = NT == 1 ? 8 : 4;  // values of a piece, pieces of the head on their way
  constexpr uint32_t STEP = 4 * VEC;                             // values of k that a wave's instruction takes of a row
  __shared__ float2 joined[4][16 * NT];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 15, q = lane >> 4;
  int label[NT];
  int64_t token_at[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int i = t * 16 + col;
    label[t] = i < n ? labels.at(i) : -1;
    token_at[t] = (int64_t)(i < n ? i : n - 1) * h_ld;
  }
  if constexpr (KEPT) {
    const uint32_t from = blockIdx.y * each;  // below dim
    w += from;
    h0 += from;
    h1 += from;
    own += blockIdx.y * apart;
    dim = dim - from < each ? dim - from : each;
  }
  const bool paired = sizeof(T) == 2 && (w_ld & 1);
  const int64_t g0 = ((int64_t)blockIdx.x * 4 + wave) * groups;
  float top[NT], sum[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) top[t] = -INFINITY, sum[t] = 0.0f;
  for (int64_t g = g0; g < g0 + groups; ++g) {
    const int64_t first = paired ? (g >> 1) * 32 + (g & 1) : g * 16, step = paired ? 2 : 1;
    if (first >= vocab) break;  // uniform
    const int64_t mine = first + col * step, row = mine < vocab ? mine : first;  // rows behind the last: the first's copies
    const bool shift = sizeof(T) == 2 && (((uint32_t)(uintptr_t)w >> 1) + (uint32_t)(first * w_ld)) & 1;  // uniform
    const T *wr = w + row * w_ld, *h = shift ? h1 : h0;
    f32x4 acc[NT], small[KEPT ? NT : 1];
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int t = 0; t < (KEPT ? NT : 1); ++t) small[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    auto apart3 = [&](bf16x8 (&to)[3], const Piece<T, VEC>& a, const Piece<T, VEC>& b) {
      if constexpr (KEPT) {
        uint32_t p[8][3];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          three_planes(a.get(e), p[e]);
          three_planes(b.get(e), p[4 + e]);
        }
#pragma unroll
        for (int k = 0; k < 3; ++k)
          to[k] = __builtin_bit_cast(bf16x8, u32x4{bits_hi(p[0][k], p[1][k]), bits_hi(p[2][k], p[3][k]),
                                                   bits_hi(p[4][k], p[5][k]), bits_hi(p[6][k], p[7][k])});
      }
    };
    auto multiply3 = [&](int t, const bf16x8 (&a)[3], const bf16x8 (&b)[3]) {
      if constexpr (KEPT) {
        small[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[2], b[0], small[t], 0, 0, 0);
        small[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[0], b[2], small[t], 0, 0, 0);
        small[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[1], b[1], small[t], 0, 0, 0);
        small[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[1], b[0], small[t], 0, 0, 0);
        small[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[0], b[1], small[t], 0, 0, 0);
        acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[0], b[0], acc[t], 0, 0, 0);
      }
    };
    auto multiply = [&](int t, const Piece<T, VEC>& a, const Piece<T, VEC>& b) {
      if constexpr (sizeof(T) == 2) {
        acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b),
                                                         acc[t], 0, 0, 0);
      } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc[t] = __builtin_amdgcn_mfma_f32_16x16x4f32(a.get(e), b.get(e), acc[t], 0, 0, 0);
      }
    };
    if (shift) {
      Piece<T, VEC> a, b;
      a.clear();
      if (q == 0) a.put(0, ld_g(wr));
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        b.clear();
        if (q == 0) b.put(0, ld_g(h0 + token_at[t]));
        multiply(t, a, b);
      }
      ++wr;
    }
    const uint32_t left = dim - (shift ? 1 : 0), whole = left / (U * STEP) * (U * STEP);
    uint32_t k = 0;
    const T* wk = wr + q * VEC;
    Piece<T, VEC> pw[2][U], ph[NT][U];
    auto fetch = [&](Piece<T, VEC> (&to)[U], const T* from) {
#pragma unroll
      for (int u = 0; u < U; ++u) to[u].load(from + u * STEP);
    };
    auto chunk = [&](int which) {
#pragma unroll
      for (int t = 0; t < NT; ++t) fetch(ph[t], h + token_at[t] + q * VEC + k);
      if (k + U * STEP < whole) fetch(pw[which ^ 1], wk + k + U * STEP);
      if constexpr (KEPT) {
#pragma unroll
        for (int u = 0; u < U; u += 2) {
          bf16x8 a[3], b[3];
          apart3(a, pw[which][u], pw[which][u + 1]);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            apart3(b, ph[t][u], ph[t][u + 1]);
            multiply3(t, a, b);
          }
        }
      } else {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int u = 0; u < U; ++u) multiply(t, pw[which][u], ph[t][u]);
      }
      k += U * STEP;
    };
    if (whole) fetch(pw[0], wk);
    while (k < whole) {
      chunk(0);
      if (k < whole) chunk(1);
    }
    for (; k < left; k += STEP) {
      Piece<T, VEC> a, b;
      take_cols<T, VEC>(a, wr, k + q * VEC, left);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        take_cols<T, VEC>(b, h + token_at[t], k + q * VEC, left);
        if constexpr (KEPT) {
          Piece<T, VEC> zero;
          zero.clear();
          bf16x8 a3[3], b3[3];
          apart3(a3, a, zero);
          apart3(b3, b, zero);
          multiply3(t, a3, b3);
        } else {
          multiply(t, a, b);
        }
      }
    }
    // lane l has the wave's rows 4 (l / 16) to 4 (l / 16) + 3 for token l % 16 of each tile
    if constexpr (KEPT) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
        if (t * 16 + col < n) *(f32x4*)(own + (t * 16 + col) * np + first + 4 * q) = acc[t] + small[t];
      continue;
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float m = top[t];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int64_t v = first + (4 * q + r) * step;
        if (v >= vocab) acc[t][r] = -INFINITY;
        else if (v == label[t]) own[t * 16 + col] = acc[t][r];
        m = fmaxf(m, acc[t][r]);
      }
      const float from = m == -INFINITY ? 0.0f : m;
      sum[t] *= exp_of(top[t] - from);
#pragma unroll
      for (int r = 0; r < 4; ++r) sum[t] += exp_of(acc[t][r] - from);
      top[t] = m;
    }
  }
  if constexpr (KEPT) return;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const float all = join4(top[t], true), from = all == -INFINITY ? 0.0f : all;
    const float s = join4(sum[t] * exp_of(top[t] - from), false);
    if (q == 0) joined[wave][t * 16 + col] = float2{all, s};
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kThreads) {
    float m = joined[0][i].x, s = 0.0f;
#pragma unroll
    for (int x = 1; x < 4; ++x) m = fmaxf(m, joined[x][i].x);
    const float from = m == -INFINITY ? 0.0f : m;
#pragma unroll
    for (int x = 0; x < 4; ++x) s += joined[x][i].y * exp_of(joined[x][i].x - from);
    parts[(int64_t)blockIdx.x * np + i] = float2{m, s};
  }
}

// Joins the tiles' maxima and sums: TOKENS tokens and as many groups of tiles as
// fit beside them to a workgroup. Sixteen tokens read whole lines; for few tokens,
// one to a workgroup has all its tiles on their way at once.
//
// PLACED: tokens are where k_tokens put them; otherwise each is in its row.
template <int TOKENS, bool PLACED>
__global__ __launch_bounds__(kThreads)
void k_join_loss(const float2* __restrict__ parts, int64_t tiles, int64_t np, const float* __restrict__ own, Tokens tok,
                 Labels labels, int64_t n, float* __restrict__ loss, float* __restrict__ lse) {
  constexpr int GROUPS = kThreads / TOKENS, U = 8;
  __shared__ float2 lds[GROUPS][TOKENS + 1];
  const int c = threadIdx.x % TOKENS, group = threadIdx.x / TOKENS;
  const int64_t token = (int64_t)blockIdx.x * TOKENS + c, count = PLACED ? *tok.count : n;
  if ((int64_t)blockIdx.x * TOKENS >= count) return;  // uniform
  float top = -INFINITY, sum = 0.0f;
  auto add = [&](const float2* p, int n) {  // n is a constant
    float t = top;
    for (int u = 0; u < n; ++u) t = fmaxf(t, p[u].x);
    const float from = t == -INFINITY ? 0.0f : t;
    sum *= exp_of(top - from);
    for (int u = 0; u < n; ++u) sum = fmaf(p[u].y, exp_of(p[u].x - from), sum);
    top = t;
  };
  if (token < count)
    for (int64_t t = group; t < tiles; t += GROUPS * U) {
      float2 p[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        p[u] = t + GROUPS * u < tiles ? parts[(t + GROUPS * u) * np + token] : float2{-INFINITY, 0.0f};
      add(p, U);
    }
  // a tree over the groups
#pragma unroll
  for (int half = GROUPS / 2; half > 0; half /= 2) {
    if (group >= half && group < 2 * half) lds[group][c] = float2{top, sum};
    __syncthreads();
    if (group < half) add(&lds[group + half][c], 1);
  }
  if (group != 0 || token >= count) return;
  const int64_t i = PLACED ? tok.map[token] : token;
  const bool counts = (PLACED ? tok.label[token] : labels.at(token)) >= 0;
  const float log_sum = logf(sum);
  loss[i] = counts ? log_sum + (top - own[token]) : 0.0f;  // exact where the label's logit is the largest
  if (lse) lse[i] = counts ? top + log_sum : 0.0f;
}

// A product whose sum is split (387 tokens, 260 x 8128 in fp32: the logits' 12 tiles
// take 587 us whole, 38 in 18 parts and 5 to join them), with fp32 rows of its own for each split: the hidden
// states' gradient over one piece (rows of the tile are columns of the hidden states,
// columns tokens), and logits of fewer tiles than CUs (rows of the head, tokens).
template <class S, GemmMode MA, bool HALF>
__global__ __launch_bounds__(S::THREADS, 2)
void k_split(GemmSide a, GemmSide b, int64_t m, Segments segs, int steps, int splits, int add,
             const int32_t* __restrict__ count_of, float* __restrict__ out, int64_t ld, int64_t np,
             const int32_t* __restrict__ a_power, const int32_t* __restrict__ b_power) {
  __shared__ __align__(1024) char lds[S::LDS];
  const int64_t count = *count_of;
  const uint32_t tm = (uint32_t)((m + S::BM - 1) / S::BM), tn = (uint32_t)((count + S::BN - 1) / S::BN);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / S::WN, wn = wave % S::WN;
  const int total = segs.count * steps;
  // the splits of a tile lie behind one another in the tiles' order: tile.n = split * tn + n
  auto make = [&](auto& loop, const Tile& at) {
    const int64_t split = at.n / tn;
    loop.aim(a, b, at.m * S::BM, at.n % tn * S::BN, segs, steps, (int)(total * split / splits),
             (int)(total * (split + 1) / splits));
  };
  auto finish = [&](const Tile& at, typename S::Acc& acc) {
    float* mine = out + (int64_t)(at.n / tn) * np * ld;
#pragma unroll
    for (int j = 0; j < S::TN; ++j) {
      const int64_t token = at.n % tn * S::BN + wn * (S::BN / S::WN) + j * 16 + (lane & 15);
      const int of_token = HALF && token < count ? b_power[token] : 0;
#pragma unroll
      for (int i = 0; i < S::TM; ++i) {
        const int64_t c = at.m * S::BM + wm * (S::BM / S::WM) + i * 16 + (lane >> 4) * 4;
        if (token < count && c < ld) {
          f32x4* to = (f32x4*)(mine + token * ld + c);
          if constexpr (HALF) {
            const int4 of_row = *(const int4*)(a_power + c);  // rows up to a multiple of 256 have a place
            acc[i][j] = f32x4{ldexpf(acc[i][j].x, of_row.x + of_token), ldexpf(acc[i][j].y, of_row.y + of_token),
                              ldexpf(acc[i][j].z, of_row.z + of_token), ldexpf(acc[i][j].w, of_row.w + of_token)};
          }
          *to = add ? *to + acc[i][j] : acc[i][j];
        }
      }
    }
    return false;
  };
  tiles_of<S, MA, K_IN_ROWS, HALF>(lds, tm * tn * splits, tm, tn * splits, make, finish);
}

// The fp32 hidden states' gradient of few tokens: the head's rows stream through
// registers as they lie. A wave takes 64 columns of one part of the rows, 32 rows at
// a time: lane l loads 16 bytes of rows 8 (l / 16) to 8 (l / 16) + 7, and with them g of
// token l % 16 of each tile. 5203 x 7616 and 3, 20 and 64 tokens: 37, 60 and 105 us,
// and the logits in place 47, 66 and 124; the planes of this head and the products with
// them take 61, 107 and 77, whatever the number of tokens.
template <int NT>
__global__ __launch_bounds__(kThreads)
void k_dhidden_few(const float* __restrict__ w, int64_t w_ld, const float* __restrict__ g, int64_t g_ld, Tokens tok,
                   int64_t vc, uint32_t dim, int splits, int add, float* __restrict__ out, int64_t dq, int64_t np) {
  constexpr int U = 8;
  const int lane = threadIdx.x & 63, col = lane & 15, q = lane >> 4, count = *tok.count;
  const int64_t blocks = (dim + 63) / 64, id = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (count == 0 || id >= blocks * splits) return;  // uniform in a wave, and no barriers
  const int64_t split = id / blocks, turns = (vc + 31) / 32;
  const uint32_t c = (uint32_t)(id % blocks) * 64 + col * 4;
  const float* row_of[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) row_of[t] = g + (int64_t)tok.map[t * 16 + col < count ? t * 16 + col : 0] * g_ld + q * U;
  f32x4 acc[NT][4];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[t][e] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  for (int64_t turn = turns * split / splits; turn < turns * (split + 1) / splits; ++turn) {
    const int64_t v0 = turn * 32;
    Piece<float, 4> a[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t v = v0 + q * U + u;  // g is zero for rows behind the last
      load_cols<float, 4>(a[u], w + (v < vc ? v : vc - 1) * w_ld, c, dim);
    }
    f32x4 gv[NT][U / 4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int x = 0; x < U / 4; ++x) gv[t][x] = *(const f32x4*)(row_of[t] + v0 + 4 * x);
    if (ragged(dim, 4))
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t v = v0 + q * U + u;
        settle_cols<float, 4>(a[u], w + (v < vc ? v : vc - 1) * w_ld, c, dim);
      }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          acc[t][e] = __builtin_amdgcn_mfma_f32_16x16x4f32(gv[t][u / 4][u % 4], a[u].get(e), acc[t][e], 0, 0, 0);
  }
  // lane l has tokens 4 (l / 16) to 4 (l / 16) + 3 of each tile
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int token = t * 16 + 4 * q + r;
      if (token < count && c < dq) {
        f32x4* to = (f32x4*)(out + (split * np + token) * dq + c);
        const f32x4 x = {acc[t][0][r], acc[t][1][r], acc[t][2][r], acc[t][3][r]};
        *to = add ? *to + x : x;
      }
    }
}

__device__ __forceinline__ f32x4 sum_of_splits(const float* p, int splits, int64_t apart) {
  f32x4 z = *(const f32x4*)p;
#pragma unroll 4
  for (int k = 1; k < splits; ++k) z += *(const f32x4*)(p + k * apart);
  return z;
}

// Split logits joined, 2048 of a token to a workgroup: their maximum and sum.
constexpr int kJoinRows = 2048;
__global__ __launch_bounds__(kThreads)
void k_join_logits(const float* __restrict__ z, int splits, int64_t ld, int64_t v0, int64_t vc, Tokens tok,
                   float2* __restrict__ parts, float* __restrict__ own, int64_t np) {
  constexpr int N = kJoinRows / (4 * kThreads);
  __shared__ float2 joined[kThreads / 64];
  const int64_t token = blockIdx.x;
  if (token >= *tok.count) return;  // uniform
  const int label = tok.label[token];
  const int64_t mine = label >= 0 ? label - v0 : -1;
  f32x4 x[N];
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int64_t v = (int64_t)blockIdx.y * kJoinRows + (i * kThreads + threadIdx.x) * 4;
    x[i] = f32x4{-INFINITY, -INFINITY, -INFINITY, -INFINITY};
    if (v >= vc) continue;
    const f32x4 y = sum_of_splits(z + token * ld + v, splits, np * ld);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      if (v + r < vc) x[i][r] = y[r];
      if (v + r == mine) own[token] = y[r];
      top = fmaxf(top, x[i][r]);
    }
  }
  auto of_wave = [&](float a, bool take_max) {
    for (int d = 32; d > 0; d /= 2) {
      const float b = __shfl_xor(a, d);
      a = take_max ? fmaxf(a, b) : a + b;
    }
    return a;
  };
  top = of_wave(top, true);
  const float from = top == -INFINITY ? 0.0f : top;  // exp(-inf) = 0 where all are that, not of -inf + inf
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) sum += exp_of(x[i][r] - from);
  sum = of_wave(sum, false);
  if ((threadIdx.x & 63) == 0) joined[threadIdx.x >> 6] = float2{top, sum};
  __syncthreads();
  if (threadIdx.x != 0) return;
  float m = joined[0].x, t = 0.0f;
  for (int k = 1; k < kThreads / 64; ++k) m = fmaxf(m, joined[k].x);
  const float base = m == -INFINITY ? 0.0f : m;
  for (int k = 0; k < kThreads / 64; ++k) t += joined[k].y * exp_of(joined[k].x - base);
  parts[(int64_t)blockIdx.y * np + token] = float2{m, t};
}

// Split logits joined to g, zeros behind the last token up to a multiple of 64 and behind the last row.
// KEPT: the logits are k_logits_few's, in the tokens' rows, and g takes their place in fp32 too.
template <int PLANES, bool KEPT = false>
__global__ __launch_bounds__(kThreads)
void k_join_g(float* __restrict__ z, int splits, int64_t ld, int64_t v0, int64_t vc, Tokens tok, int64_t np,
              uint16_t* __restrict__ g, int64_t gp) {
  const int64_t count = *tok.count, written = (count + 63) / 64 * 64, per = gp / 4;
  for (int64_t at = (int64_t)blockIdx.x * kThreads + threadIdx.x; at < written * per; at += (int64_t)gridDim.x * kThreads) {
    const int64_t token = at / per, v = at % per * 4;
    f32x4 d = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    if (token < count && v < vc) {
      const int64_t mine = (int64_t)tok.label[token] - v0;
      const float lse = tok.lse[token], coef = tok.coef[token];
      const f32x4 x = sum_of_splits(z + (KEPT ? tok.map[token] : token) * ld + v, splits, np * ld);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float p = exp_of(x[r] - lse);
        d[r] = v + r < vc ? coef * (v + r == mine ? p - 1.0f : p) : 0.0f;
        if (v + r == mine) tok.rest[token] = d[r] - bf16_lo(pack_bf16(d[r], d[r]));
      }
    }
    if (KEPT && token < count) *(f32x4*)(z + tok.map[token] * ld + v) = d;
    uint16_t* row = g + token * gp * PLANES + v;
#pragma unroll
    for (int k = 0; k < PLANES; ++k) {
      const uint2 y = uint2{pack_bf16(d.x, d.y), pack_bf16(d.z, d.w)};
      *(uint2*)(row + k * gp) = y;
      d = f32x4{d.x - bf16_lo(y.x), d.y - bf16_hi(y.x), d.z - bf16_lo(y.y), d.w - bf16_hi(y.y)};
    }
  }
}

// The head's gradient for one piece: rows of the tile are columns of the hidden
// states, columns rows of the head. Splits of the sum over the tokens go to matrices
// `apart` elements from each other.
template <class S, typename Gt>
__global__ __launch_bounds__(S::THREADS, 2)
void k_dweight(GemmSide h, GemmSide g, Segments segs, const int32_t* __restrict__ count_of, int64_t v0, int64_t vc,
               uint32_t dim, Gt* __restrict__ dw_of, int64_t dw_ld, int first, int splits, int64_t apart) {
  __shared__ __align__(1024) char lds[S::LDS];
  // Whole tiles are stored by way of LDS, 64 columns of 16 rows at a time and wave: a lane holds 4 columns
  // (3 tokens, 7867 x 8064 bf16: 32 us, 47 from the registers; 70 tokens, 18898 x 5170 added in bf16: 160, 232).
  constexpr int IN = 4, EACH = 16 / sizeof(Gt), FLOATS = IN * 4, CHUNKS = IN * 16 / EACH;
  __shared__ __align__(16) u32x4 lines[S::WM * S::WN][16 * FLOATS];
  const uint32_t tm = (dim + S::BM - 1) / S::BM, tn = (uint32_t)((vc + S::BN - 1) / S::BN);
  const int steps = (int)((*count_of + 63) / 64);  // none: the sums are zero
  const int total = segs.count * steps;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / S::WN, wn = wave % S::WN;
  auto make = [&](auto& loop, const Tile& at) {
    const int64_t split = at.n / tn;
    loop.aim(h, g, at.m * S::BM, at.n % tn * S::BN, segs, steps, (int)(total * split / splits),
             (int)(total * (split + 1) / splits));
  };
  auto finish = [&](const Tile& part, typename S::Acc& acc) {
    const Tile at{part.m, part.n % tn};
    Gt* dw = dw_of + part.n / tn * apart;
    const bool whole = dim - at.m * S::BM >= S::BM && vc - at.n * S::BN >= S::BN;
    if (whole) {
#pragma unroll
      for (int j = 0; j < S::TN; ++j)
#pragma unroll
        for (int part = 0; part < S::TM / IN; ++part) {
          const int t = lane & 15, c0 = wm * (S::BM / S::WM) + part * IN * 16;
          Gt* to = dw + (v0 + at.n * S::BN + wn * (S::BN / S::WN) + j * 16) * dw_ld + at.m * S::BM + c0;
          u32x4* mine = lines[wave];
          u32x4 old[IN * 16 * 16 / EACH / 64];
          if (!first)
#pragma unroll
            for (int x = 0; x < IN * 16 * 16 / EACH / 64; ++x) {
              const int at16 = x * 64 + lane, row = at16 / CHUNKS, c = at16 % CHUNKS;
              old[x] = ld16(to + row * dw_ld + c * EACH);
            }
#pragma unroll
          for (int i = 0; i < IN; ++i) {
            const f32x4 a = acc[part * IN + i][j];
            // four columns lie in one chunk of fp32, or in half of one of two fp32 chunks
            mine[t * FLOATS + ((4 * i + (lane >> 4)) ^ (t & (FLOATS - 1)))] =
                u32x4{__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(a.z), __float_as_uint(a.w)};
          }
          wave_lds();
#pragma unroll
          for (int x = 0; x < IN * 16 * 16 / EACH / 64; ++x) {
            const int at16 = x * 64 + lane, row = at16 / CHUNKS, c = at16 % CHUNKS;
            auto take = [&](int chunk) { return mine[row * FLOATS + (chunk ^ (row & (FLOATS - 1)))]; };
            u32x4 y;
            if constexpr (sizeof(Gt) == 4) {
              y = take(c);
              if (!first)
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) + __uint_as_float(old[x][e]));
            } else {
              const u32x4 lo = take(2 * c), hi = take(2 * c + 1);
              float f[8];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                f[e] = __uint_as_float(lo[e]);
                f[4 + e] = __uint_as_float(hi[e]);
              }
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                if (!first) {
                  f[2 * e] += bf16_lo(old[x][e]);
                  f[2 * e + 1] += bf16_hi(old[x][e]);
                }
                y[e] = pack_bf16(f[2 * e], f[2 * e + 1]);
              }
            }
            st16(y, to + row * dw_ld + c * EACH);
          }
          wave_lds();
        }
      return S::TN * (S::TM / IN) * (IN * 16 * 16 / EACH / 64) >= 16;
    }
#pragma unroll
    for (int j = 0; j < S::TN; ++j) {
      const int64_t v = at.n * S::BN + wn * (S::BN / S::WN) + j * 16 + (lane & 15);
      Gt* row = dw + (v0 + v) * dw_ld;
#pragma unroll
      for (int i = 0; i < S::TM; ++i) {
        const uint32_t c = (uint32_t)(at.m * S::BM) + wm * (S::BM / S::WM) + i * 16 + (lane >> 4) * 4;
        if (v >= vc || c >= dim) continue;
        f32x4 x = acc[i][j];
        if (c + 4 <= dim) {
          if constexpr (sizeof(Gt) == 4) {
            if (!first) {
              const u32x4 old = ld16(row + c);
              x += f32x4{__uint_as_float(old.x), __uint_as_float(old.y), __uint_as_float(old.z), __uint_as_float(old.w)};
            }
            st16(u32x4{__float_as_uint(x.x), __float_as_uint(x.y), __float_as_uint(x.z), __float_as_uint(x.w)}, row + c);
          } else {
            const auto p = (__attribute__((address_space(1))) u32x2_any*)(row + c);
            if (!first) {
              const u32x2 old = *p;
              x += f32x4{bf16_lo(old.x), bf16_hi(old.x), bf16_lo(old.y), bf16_hi(old.y)};
            }
            *p = u32x2{pack_bf16(x.x, x.y), pack_bf16(x.z, x.w)};
          }
        } else {
          for (uint32_t e = 0; c + e < dim; ++e) {
            float y = e == 0 ? x.x : e == 1 ? x.y : x.z;
            if (!first) {
              if constexpr (sizeof(Gt) == 4) y += row[c + e];
              else y += bf16_to_f32(row[c + e]);
            }
            st_g(round_to<Gt>(y), row + c + e);
          }
        }
      }
    }
    return false;
  };
  tiles_of<S, K_IS_ROW, K_IS_ROW>(lds, tm * tn * splits, tm, tn * splits, make, finish);
}

// The splits of the head's gradient, joined and rounded once.
template <typename Gt>
__global__ __launch_bounds__(kThreads)
void k_join_dweight(const float* __restrict__ sums, int splits, int64_t apart, int64_t ld, int64_t vc, uint32_t dim,
                    Gt* __restrict__ dw, int64_t dw_ld, int first) {
  const int64_t per = (ld + 7) / 8;
  for (int64_t at = (int64_t)blockIdx.x * kThreads + threadIdx.x; at < vc * per; at += (int64_t)gridDim.x * kThreads) {
    const int64_t v = at / per;
    const uint32_t c = (uint32_t)(at % per) * 8;
    const float* from = sums + v * ld + c;
    const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f}, a = sum_of_splits(from, splits, apart),
                b = c + 4 < ld ? sum_of_splits(from + 4, splits, apart) : zero;
    float x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    Gt* to = dw + v * dw_ld;
    if (!first) {
      Piece<Gt, 8> p;
      take_cols<Gt, 8>(p, to, c, dim);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] += p.get(e);
    }
    store_cols<Gt, 8>(to, x, c, dim);
  }
}

// The splits' sums, rounded once, back in the tokens' places; zeros where a token
// does not count. GROUPS threads share a piece of 8 columns: with few tokens there
// are few pieces and many splits.
//
// With a head in bf16 their g is one bf16, and a token's largest by far is that at
// its label: what its rounding left, times that row of the head, is added here
// (without: 0.0022 to 0.0025 off the exact result, 0.0017 is bf16's own).
template <typename T, int GROUPS>
__global__ __launch_bounds__(kThreads)
void k_join_dhidden(const float* __restrict__ sums, int splits, int64_t np, int64_t dq, Tokens tok, int64_t n, uint32_t dim,
                    const T* __restrict__ w, int64_t w_ld, T* __restrict__ out, int64_t ld) {
  constexpr int PIECES = kThreads / GROUPS;
  __shared__ float lds[GROUPS > 1 ? GROUPS : 1][PIECES][9];
  const int64_t per = (dim + 7) / 8, all = n * per;
  const int piece = threadIdx.x % PIECES, group = threadIdx.x / PIECES;
  for (int64_t base = (int64_t)blockIdx.x * PIECES; base < all; base += (int64_t)gridDim.x * PIECES) {
    const int64_t at = base + piece, i = at / per;
    const uint32_t c = (uint32_t)(at % per) * 8;
    const int32_t place = at < all ? tok.inverse[i] : -1;
    float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    if (place >= 0) {
      const float* from = sums + (int64_t)place * dq + c;
      const bool both = c + 4 < dq;
#pragma unroll 4
      for (int k = group; k < splits; k += GROUPS) {
        const f32x4 a = *(const f32x4*)(from + (int64_t)k * np * dq);
        const f32x4 b = both ? *(const f32x4*)(from + (int64_t)k * np * dq + 4) : f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[e] += a[e];
          v[4 + e] += b[e];
        }
      }
    }
    if constexpr (GROUPS > 1) {
#pragma unroll
      for (int e = 0; e < 8; ++e) lds[group][piece][e] = v[e];
      __syncthreads();
      if (group == 0)
        for (int x = 1; x < GROUPS; ++x)
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] += lds[x][piece][e];
      __syncthreads();
      if (group != 0) continue;
    }
    if (at >= all) continue;
    if constexpr (sizeof(T) == 2)
      if (place >= 0) {
        const float rest = tok.rest[place];
        Piece<T, 8> p;
        take_cols<T, 8>(p, w + tok.label[place] * w_ld, c, dim);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = fmaf(rest, p.get(e), v[e]);
      }
    store_cols<T, 8>(out + i * ld, v, c, dim);
  }
}

// Zeros in a matrix's rows (a head's gradient without tokens, hidden states' without a vocabulary).
template <typename T>
__global__ __launch_bounds__(kThreads)
void k_zero_rows(T* __restrict__ out, int64_t ld, int64_t rows, uint32_t dim) {
  const int64_t per = (dim + 7) / 8;
  const float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  for (int64_t at = (int64_t)blockIdx.x * kThreads + threadIdx.x; at < rows * per; at += (int64_t)gridDim.x * kThreads)
    store_cols<T, 8>(out + at / per * ld, v, (uint32_t)(at % per) * 8, dim);
}

// ---------------------------------------------------------------- host

int64_t up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }
int64_t least(int64_t a, int64_t b) { return a < b ? a : b; }

unsigned grid_of(int64_t pieces) { return (unsigned)least((pieces + kThreads - 1) / kThreads, 1 << 16); }

// Rows that direct loads take as they lie: on 16-byte boundaries, whole stages
// of k, and 256 of them within 32 bits of offset.
bool as_it_lies(const void* p, int64_t ld, int64_t dim, int dtype) {
  return dtype == ZS_BF16 && dim % kBK == 0 && ld % 8 == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0 &&
         ld <= (1 << 22);
}

Tokens tokens_at(const HeadPlan& p, void* workspace) {
  char* w = static_cast<char*>(workspace);
  return Tokens{(int32_t*)(w + p.label), (int32_t*)(w + p.map), (int32_t*)(w + p.inverse), (int32_t*)(w + p.count),
                (float*)(w + p.coef), (float*)(w + p.lse), (float*)(w + p.rest)};
}

// How a product is made: its tiles, in how many parts of the sum, and how long it
// takes, in stages of the widest tile (1.7 us: 1250 TFLOP/s on 256 CUs), of which a
// round costs some beside its own: first loads, what is done with the products
// (256 x 256, 8 stages: 27 us). 128 x 128 tiles run on a CU at two at once (1.0 us a
// stage, 1070 TFLOP/s) or alone (0.77 us). 256 x 64 ones wait for loads: 0.9 us a
// stage for few, more for many, from HBM 1.6 us for 256 (5.3 TB/s), from the
// memory-side cache about 1. Parts are of eight stages at least, and written and read
// once more.
enum Cut { WIDE, SQUARE, NARROW };
struct Way {
  Cut cut;
  int splits;
  double cost;
};
constexpr double kRoundStages = 10;
Way way_of(int64_t m, int64_t n, int64_t stages, int most = 1, double join = 0.0) {
  auto tiles = [&](int64_t bm, int64_t bn) { return ((m + bm - 1) / bm) * ((n + bn - 1) / bn); };
  const int64_t t[3] = {tiles(256, 256), tiles(128, 128), tiles(256, 64)};
  auto squares = [](int64_t t) { return (double)(t / 512) * 0.6 + (t % 512 == 0 ? 0.0 : t % 512 <= 256 ? 0.45 : 0.6); };
  auto narrows = [](int64_t t) { return t < 220 ? 0.5 : (double)t * 0.0023; };
  Way best{WIDE, 1, 1e300};
  for (int splits = 1; splits <= most; splits += splits < 4 ? 1 : splits / 4 * 2) {  // 1 2 3 4 6 8 12 18 ...
    if (splits > 1 && stages / splits < 8) break;
    const double wide = (double)((t[0] * splits + 255) / 256), square = squares(t[1] * splits), narrow = narrows(t[2] * splits);
    const Cut cut = n <= 64 ? NARROW : square < wide ? SQUARE : WIDE;
    const double rounds = cut == NARROW ? narrow : cut == SQUARE ? square : wide;
    const double cost = rounds * ((double)stages / splits + kRoundStages) +
                        (splits > 1 ? join + (double)m * (double)n * splits * 1.2e-6 : 0.0);
    if (cost < best.cost) best = Way{cut, splits, cost};
  }
  return best;
}
Way way_of_logits(int64_t vc, int64_t n, int64_t stages) { return way_of(vc, n, stages, 32, 4.0); }
Way way_of_dweight(int64_t dim, int64_t vc, int64_t stages) { return way_of(dim, vc, stages, 32, 4.0); }
Way way_of_dhidden(int64_t dim, int64_t n, int64_t stages) { return way_of(dim, n, stages, n <= 64 ? 256 : 32); }

// Parts of the sum for few tokens' hidden states' gradient: 2048 waves, 8 a CU, with 32 rows of the head each at least.
int few_splits(int64_t dim, int64_t rows) {
  const int64_t blocks = (dim + 63) / 64, splits = least(least((2048 + blocks - 1) / blocks, 256), (rows + 31) / 32);
  return (int)(splits < 1 ? 1 : splits);
}
// Workgroups that stream a head of few tokens, and 16-row groups of a wave.
struct FewGrid {
  int64_t groups, grid;
};
FewGrid few_grid(int64_t vocab) {
  const int64_t all = (vocab + 31) / 32 * 2, groups = (all + kFewWaves - 1) / kFewWaves;
  return {groups, groups ? (all + 4 * groups - 1) / (4 * groups) : 0};
}
// Columns of a part of few tokens' fp32 logits, so that there are 2048 waves, with 512 columns each at least.
int64_t few_columns(int64_t rows, int64_t dim) {
  const int64_t most = least(2048 / ((rows + 15) / 16), dim / 512), parts = most < 1 ? 1 : most;
  return up((dim + parts - 1) / parts, 128);
}
int64_t few_parts(int64_t rows, int64_t dim) {
  const int64_t each = few_columns(rows, dim);
  return (dim + each - 1) / each;
}
template <typename F>
void by_tokens(int64_t n, F&& f) {
  if (n <= 16) f(std::integral_constant<int, 1>{});
  else if (n <= 32) f(std::integral_constant<int, 2>{});
  else f(std::integral_constant<int, 4>{});
}

// As many workgroups as 256 CUs hold at once, or tiles, which they then take in turn.
template <class S>
unsigned workgroups(int64_t m, int64_t n, int64_t splits = 1) {
  const int64_t tiles = ((m + S::BM - 1) / S::BM) * ((n + S::BN - 1) / S::BN) * splits;
  return (unsigned)least(tiles, S::LDS <= 80 * 1024 ? 512 : 256);
}

template <typename F>
void with_cut(Cut c, F&& f) {
  if (c == WIDE) f(Wide{});
  else if (c == SQUARE) f(Square{});
  else f(Narrow{});
}

void layout(const void* src, int64_t ld, int dtype, int64_t dim, int64_t rows, uint16_t* dst, int64_t dp,
            const int32_t* map, const int32_t* count, hipStream_t s) {
  const unsigned grid = grid_of(up(rows, 64) * (dp / 8));
  if (dtype == ZS_BF16)
    hipLaunchKernelGGL((k_layout<uint16_t>), dim3(grid), dim3(kThreads), 0, s, (const uint16_t*)src, ld, (uint32_t)dim,
                       rows, dst, dp, map, count);
  else
    hipLaunchKernelGGL((k_layout<float>), dim3(grid), dim3(kThreads), 0, s, (const float*)src, ld, (uint32_t)dim, rows,
                       dst, dp, map, count);
}

void layout_half(const void* src, int64_t ld, int64_t dim, int64_t rows, uint16_t* dst, int64_t dp, int32_t* power,
                 const int32_t* map, const int32_t* count, uint16_t* planes, hipStream_t s) {
  const dim3 grid((unsigned)least((up(rows, 64) + 3) / 4, 4096)), block(kThreads);
  if (planes)
    hipLaunchKernelGGL((k_layout_half<true>), grid, block, 0, s, (const float*)src, ld, (uint32_t)dim, rows, dst, dp, power,
                       map, count, planes);
  else
    hipLaunchKernelGGL((k_layout_half<false>), grid, block, 0, s, (const float*)src, ld, (uint32_t)dim, rows, dst, dp, power,
                       map, count, planes);
}

void number_tokens(const void* labels, int index_type, int64_t n, int64_t vocab, bool gather, const float* lse,
                   const float* dloss, float scale, const Tokens& t, float* loss, float* lse_out, hipStream_t s) {
  if (index_type == ZS_I64)
    hipLaunchKernelGGL((k_tokens<int64_t>), dim3(1), dim3(kTokBS), 0, s, (const int64_t*)labels, n, vocab, (int)gather,
                       lse, dloss, scale, t, loss, lse_out);
  else
    hipLaunchKernelGGL((k_tokens<int32_t>), dim3(1), dim3(kTokBS), 0, s, (const int32_t*)labels, n, vocab, (int)gather,
                       lse, dloss, scale, t, loss, lse_out);
}

void zero_rows(void* p, int dtype, int64_t ld, int64_t rows, int64_t dim, hipStream_t s) {
  const unsigned grid = grid_of(rows * ((dim + 7) / 8));
  if (dtype == ZS_BF16)
    hipLaunchKernelGGL((k_zero_rows<uint16_t>), dim3(grid), dim3(kThreads), 0, s, (uint16_t*)p, ld, rows, (uint32_t)dim);
  else
    hipLaunchKernelGGL((k_zero_rows<float>), dim3(grid), dim3(kThreads), 0, s, (float*)p, ld, rows, (uint32_t)dim);
}

// Rows of the head laid out at a time, and bytes of the logits' gradient of a
// piece (at least 4096 rows of the head, so that their product stays long).
constexpr int64_t kLayoutBytes = 1 << 28;
constexpr int64_t kGradBytes = 1 << 30;
constexpr int64_t kWeightBytes = 1ll << 31;  // of the head's rows of such a piece, where they are laid out
constexpr int64_t kMostPiece = 1 << 20;
// The gradients' logits of fp32 take three products of fp16 pairs instead of six of bf16 planes from this many tokens
// on. For fewer, laying out both costs more than that saves (70 tokens, 18898 x 5170: 361 + 177 us, 161 + 254 with the
// six; 3364 of 4805 tokens, 17606 x 1216: 85 + 514, 46 + 811).
constexpr int64_t kHalfTokens = 512;
// Calls of fewer tokens keep every row where it is in the forward pass.
constexpr int64_t kGatherTokens = 256;

}  // namespace

HeadPlan head_plan(int64_t n, int64_t vocab, int64_t dim, int dtype, int grad_dtype) {
  HeadPlan p{};
  const bool grad = grad_dtype >= 0;
  p.planes = dtype == ZS_F32 ? 3 : 1;
  p.half = dtype == ZS_F32 && (!grad || n >= kHalfTokens);
  p.few = grad && dtype == ZS_F32 && n <= kFewTokens;
  p.gplanes = dtype == ZS_F32 ? 3 : grad_dtype == ZS_F32 ? 3 : 1;
  p.np = up(n, 64);
  p.dp = up(dim, 64);
  p.dq = up(dim, 4);
  const int64_t row = grad ? p.np * p.gplanes * 2 : p.dp * p.planes * 2;
  int64_t most = (grad ? kGradBytes : kLayoutBytes) / (row > 0 ? row : 1);
  if (grad && !p.few) most = least(most, kWeightBytes / (p.dp > 0 ? p.dp * p.planes * (p.half ? 4 : 2) : 1));
  most = most < 4096 ? 4096 : most > kMostPiece ? kMostPiece : most / 256 * 256;
  p.pieces = vocab > 0 ? (vocab + most - 1) / most : 0;
  p.piece = p.pieces ? up((vocab + p.pieces - 1) / p.pieces, 256) : 0;
  p.splits = 1;
  const int64_t zstages = p.dp / kBK * (p.half ? 3 : p.planes == 3 ? 6 : 1);
  // products of planes for the head's gradient
  const int64_t wparts = p.planes == 3 ? (grad_dtype == ZS_F32 ? 6 : 3) : p.gplanes;
  if (grad && p.pieces && n > 0 && dim > 0) {
    // Of pieces of equal size and those whose head's gradient fills rounds of the widest tiles, what takes least.
    const int64_t tm = (dim + 255) / 256, parts = p.planes == 3 ? 6 : 1;
    auto one = [&](int64_t vc) {
      return way_of_logits(vc, n, zstages).cost + way_of_dhidden(dim, n, up(vc, kBK) / kBK * parts).cost +
             way_of_dweight(dim, vc, p.np / kBK * wparts).cost;
    };
    auto all = [&](int64_t piece) {
      const int64_t rest = vocab % piece;
      return (double)(vocab / piece) * one(piece) + (rest ? one(rest) : 0.0);
    };
    double best = all(p.piece);
    for (int64_t rounds = 1; rounds <= 8; ++rounds) {
      const int64_t piece = rounds * 256 / tm * 256;
      if (piece < 4096 || piece > most || piece >= vocab) continue;
      const double cost = all(piece);
      if (cost < best) {
        best = cost;
        p.piece = piece;
      }
    }
    p.splits = p.few ? few_splits(dim, least(p.piece, vocab))
                     : way_of_dhidden(dim, n, up(least(p.piece, vocab), kBK) / kBK * parts).splits;
  }
  p.pieces = p.piece ? (vocab + p.piece - 1) / p.piece : 0;
  // Room for logits and the head's gradient in parts, one after the other: of a piece and of the last one, or, in the
  // forward pass, of the whole head where it lies.
  auto room = [&](int64_t rows) {
    if (rows == 0 || n == 0 || dim == 0) return (int64_t)0;
    const int64_t zs = p.few ? few_parts(rows, dim) : way_of_logits(rows, n, zstages).splits,
                  z = zs > 1 || p.few ? zs * p.np * up(rows, kBK) * 4 : 0;
    const int64_t ws = grad ? way_of_dweight(dim, rows, p.np / kBK * wparts).splits : 1, w = ws > 1 ? ws * rows * p.dq * 4 : 0;
    return z > w ? z : w;
  };
  // The loss of few tokens reads the head as it lies: bf16 on 16-byte boundaries by tiles, others by k_logits_few.
  const bool streams = !grad && n <= kFewTokens, lies = streams && dtype == ZS_BF16;
  const int64_t of_piece = streams ? 0 : room(least(p.piece, vocab)),
                of_other = streams && !lies ? 0 : room(grad && p.piece ? vocab % p.piece : vocab);
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t from = at;
    at = up(at + bytes, 256);
    return from;
  };
  p.label = take(p.np * 4);
  p.map = take(p.np * 4);
  p.inverse = take(p.np * 4);
  p.count = take(4);
  p.coef = take(grad ? p.np * 4 : 0);
  p.lse = take(grad ? p.np * 4 : 0);
  p.rest = take(grad ? p.np * 4 : 0);
  p.own = take(grad ? 0 : p.np * 4);
  const int64_t parts = n <= kFewTokens ? vocab / 64 + 4 : (vocab + 127) / 128;  // 64 or 128 rows of the head each
  p.parts = take(grad ? 0 : parts * p.np * (int64_t)sizeof(float2));
  p.hidden = take(streams && !lies ? 0 : p.np * p.dp * p.planes * 2 * (streams ? 2 : 1));
  p.weight = take(p.few || streams || n == 0 ? 0 : p.piece * p.dp * p.planes * 2);
  p.hpower = take(p.half && !streams ? p.np * 4 : 0);
  p.wpower = take(p.half && !streams ? p.piece * 4 : 0);
  p.hhalf = take(grad && p.half ? p.np * p.dp * 6 : 0);
  p.whalf = take(grad && p.half ? p.piece * p.dp * 6 : 0);
  p.z = take(of_piece > of_other ? of_piece : of_other);
  p.g = take(grad ? p.np * p.piece * p.gplanes * 2 : 0);
  p.dhidden = take(grad ? p.splits * p.np * p.dq * 4 : 0);
  p.bytes = at;
  return p;
}

hipError_t launch_head_forward(const void* hidden, int64_t hidden_ld, int dtype, const void* weight,
                               int64_t weight_ld, const void* labels, int index_type, int64_t n, int64_t vocab,
                               int64_t dim, float* loss, float* lse, void* workspace, hipStream_t s) {
  const HeadPlan p = head_plan(n, vocab, dim, dtype, -1);
  char* ws = static_cast<char*>(workspace);
  const Tokens tok = tokens_at(p, workspace);
  const bool half = p.half;
  const Segments segs = half ? kHalves : kOne;
  int32_t *h_power = (int32_t*)(ws + p.hpower), *w_power = (int32_t*)(ws + p.wpower);
  const bool h_lies = as_it_lies(hidden, hidden_ld, dim, dtype), w_lies = as_it_lies(weight, weight_ld, dim, dtype);
  const Labels given{labels, index_type == ZS_I64, vocab};
  auto join = [&](auto tokens, auto placed, int64_t tiles) {
    constexpr int T = decltype(tokens)::value;
    hipLaunchKernelGGL((k_join_loss<T, decltype(placed)::value>), dim3((unsigned)((n + T - 1) / T)), dim3(kThreads), 0, s,
                       (const float2*)(ws + p.parts), tiles, p.np, (const float*)(ws + p.own), tok, given, n, loss, lse);
  };
  if (n <= (w_lies ? kFewAligned : kFewTokens)) {
    const bool bf16 = dtype == ZS_BF16, w_even = !bf16 || (weight_ld % 2 == 0 && reinterpret_cast<uintptr_t>(weight) % 4 == 0);
    const bool h_even = !bf16 || (hidden_ld % 2 == 0 && reinterpret_cast<uintptr_t>(hidden) % 4 == 0);
    const void *h0 = hidden, *h1 = hidden;
    int64_t h_ld = hidden_ld;
    if (!w_even || !h_even) {  // copies of the tokens on the grid, and from their second element on
      uint16_t* to = (uint16_t*)(ws + p.hidden);
      h0 = to;
      h1 = to + p.np * p.dp;
      h_ld = p.dp;
      layout(hidden, hidden_ld, dtype, dim, n, to, p.dp, nullptr, nullptr, s);
      if (dim > 1)
        layout((const uint16_t*)hidden + 1, hidden_ld, dtype, dim - 1, n, to + p.np * p.dp, p.dp, nullptr, nullptr, s);
    }
    const auto [groups, grid] = few_grid(vocab);
    auto go = [&, groups = groups, grid = grid](auto type, auto tiles) {
      using T = decltype(type);
      hipLaunchKernelGGL((k_logits_few<T, decltype(tiles)::value>), dim3((unsigned)grid), dim3(kThreads), 0, s,
                         (const T*)weight, weight_ld, (const T*)h0, (const T*)h1, h_ld, (int)n, vocab, (uint32_t)dim,
                         groups, given, (float2*)(ws + p.parts), (float*)(ws + p.own), p.np, 0u, (int64_t)0);
    };
    if (grid > 0)
      by_tokens(n, [&](auto tiles) {
        if (bf16) go(uint16_t{}, tiles);
        else go(float{}, tiles);
      });
    join(std::integral_constant<int, 1>{}, std::false_type{}, grid);
    return hipGetLastError();
  }
  const bool gather = n > kGatherTokens;
  number_tokens(labels, index_type, n, vocab, gather, nullptr, nullptr, 0.0f, tok, loss, lse, s);
  GemmSide h{(const uint16_t*)hidden, hidden_ld, 0, n, 0};
  if (gather || !h_lies) {
    uint16_t* to = (uint16_t*)(ws + p.hidden);
    if (half) layout_half(hidden, hidden_ld, dim, n, to, p.dp, h_power, tok.map, tok.count, nullptr, s);
    else layout(hidden, hidden_ld, dtype, dim, n, to, p.dp, tok.map, tok.count, s);
    h = GemmSide{to, p.dp * p.planes, p.dp, p.np, 0};
  }
  const int64_t piece = w_lies ? vocab : least(p.piece, vocab), zq = up(piece, kBK), chunks = (piece + kJoinRows - 1) / kJoinRows;
  const Way way = way_of_logits(piece, n, p.dp / kBK * segs.count);
  const bool split = way.splits > 1;
  float* z = (float*)(ws + p.z);
  int64_t tiles = 0;
  for (int64_t v0 = 0; v0 < vocab; v0 += piece) {
    const int64_t vc = least(piece, vocab - v0);
    GemmSide w{(const uint16_t*)weight + v0 * weight_ld, weight_ld, 0, vc, 0};
    if (!w_lies) {
      uint16_t* to = (uint16_t*)(ws + p.weight);
      const char* from = (const char*)weight + v0 * weight_ld * (half ? 4 : 2);
      if (half) layout_half(from, weight_ld, dim, vc, to, p.dp, w_power, nullptr, nullptr, nullptr, s);
      else layout(from, weight_ld, dtype, dim, vc, to, p.dp, nullptr, nullptr, s);
      w = GemmSide{to, p.dp * p.planes, p.dp, vc, 0};
    }
    float2* parts = (float2*)(ws + p.parts) + tiles * p.np;
    with_cut(way.cut, [&](auto shape) {
      using S = decltype(shape);
      constexpr bool HALVES = !std::is_same_v<S, Narrow>;  // of fp32 few tokens took the head as it lies
      auto go = [&](auto halves) {
        constexpr bool H = HALVES && decltype(halves)::value;
        if (split)
          hipLaunchKernelGGL((k_split<S, K_IN_ROWS, H>), dim3(workgroups<S>(vc, n, way.splits)), dim3(S::THREADS), 0, s, w,
                             h, vc, segs, (int)(p.dp / kBK), way.splits, 0, tok.count, z, zq, p.np, w_power, h_power);
        else
          hipLaunchKernelGGL((k_logits<S, 0, H>), dim3(workgroups<S>(vc, n)), dim3(S::THREADS), 0, s, w, h, segs,
                             (int)(p.dp / kBK), v0, tok, parts, (float*)(ws + p.own), p.np, (uint16_t*)nullptr, (int64_t)0,
                             w_power, h_power);
      };
      if (half) go(std::true_type{});
      else go(std::false_type{});
      tiles += split ? chunks : (vc + S::BM - 1) / S::BM * parts_of_tile<S>();
    });
    if (split) {
      const int64_t of_vc = (vc + kJoinRows - 1) / kJoinRows;
      hipLaunchKernelGGL(k_join_logits, dim3((unsigned)n, (unsigned)of_vc), dim3(kThreads), 0, s, z, way.splits, zq, v0,
                         vc, tok, parts, (float*)(ws + p.own), p.np);
      tiles += of_vc - chunks;
    }
  }
  if (n <= 64) join(std::integral_constant<int, 1>{}, std::true_type{}, tiles);
  else join(std::integral_constant<int, 16>{}, std::true_type{}, tiles);
  return hipGetLastError();
}

hipError_t launch_head_backward(const void* hidden, int64_t hidden_ld, int dtype, const void* weight,
                                int64_t weight_ld, const void* labels, int index_type, const float* lse,
                                const float* dloss, float scale, int64_t n, int64_t vocab, int64_t dim, void* dhidden,
                                int64_t dhidden_ld, void* dweight, int grad_dtype, int64_t dweight_ld, bool first,
                                void* workspace, hipStream_t s) {
  if (n == 0 || vocab == 0) {
    if (n == 0 && first) zero_rows(dweight, grad_dtype, dweight_ld, vocab, dim, s);
    if (vocab == 0) zero_rows(dhidden, dtype, dhidden_ld, n, dim, s);
    return hipGetLastError();
  }
  const HeadPlan p = head_plan(n, vocab, dim, dtype, grad_dtype);
  char* ws = static_cast<char*>(workspace);
  const Tokens tok = tokens_at(p, workspace);
  const Segments segs = p.planes == 3 ? kSix : kOne;
  const Segments wsegs = p.planes == 3 ? (grad_dtype == ZS_F32 ? kSix : kThree) : p.gplanes == 3 ? kOneThree : kOne;
  const bool w_lies = as_it_lies(weight, weight_ld, dim, dtype);
  uint16_t *hp = (uint16_t*)(ws + p.hidden), *gp = (uint16_t*)(ws + p.g);
  float *sums = (float*)(ws + p.dhidden), *z = (float*)(ws + p.z);
  const Way dway = way_of_dhidden(dim, n, up(p.piece < vocab ? p.piece : vocab, kBK) / kBK * segs.count);
  number_tokens(labels, index_type, n, vocab, true, lse, dloss, scale, tok, nullptr, nullptr, s);
  const bool half = p.half;  // the logits' operands are fp16
  const Segments zsegs = half ? kHalves : segs;
  uint16_t *h_half = (uint16_t*)(ws + p.hhalf), *w_half = (uint16_t*)(ws + p.whalf);
  int32_t *h_power = (int32_t*)(ws + p.hpower), *w_power = (int32_t*)(ws + p.wpower);
  if (half) layout_half(hidden, hidden_ld, dim, n, h_half, p.dp, h_power, tok.map, tok.count, hp, s);
  else layout(hidden, hidden_ld, dtype, dim, n, hp, p.dp, tok.map, tok.count, s);
  for (int64_t v0 = 0; v0 < vocab; v0 += p.piece) {
    const int64_t vc = least(p.piece, vocab - v0), vp = up(vc, kBK), ldg = vp * p.gplanes;
    GemmSide w{(const uint16_t*)weight + v0 * weight_ld, weight_ld, 0, vc, dim};
    const float* in_place = (const float*)weight + v0 * weight_ld;  // few tokens' fp32
    if (!w_lies && !p.few) {
      uint16_t* to = (uint16_t*)(ws + p.weight);
      const char* from = (const char*)weight + v0 * weight_ld * (dtype == ZS_F32 ? 4 : 2);
      if (half) layout_half(from, weight_ld, dim, vc, w_half, p.dp, w_power, nullptr, nullptr, to, s);
      else layout(from, weight_ld, dtype, dim, vc, to, p.dp, nullptr, nullptr, s);
      w = GemmSide{to, p.dp * p.planes, p.dp, vc, p.dp};
    }
    const GemmSide h{hp, p.dp * p.planes, p.dp, p.np, p.dp};
    const GemmSide g_rows{gp, ldg, vp, p.np, vp};
    const GemmSide zw = half ? GemmSide{w_half, p.dp * 3, p.dp, vc, 0} : w,
                   zh = half ? GemmSide{h_half, p.dp * 3, p.dp, p.np, 0} : h;
    const Way zway = way_of_logits(vc, n, p.dp / kBK * zsegs.count);
    auto by_planes = [&](auto go) {
      if (p.gplanes == 1) go(std::integral_constant<int, 1>{});
      else go(std::integral_constant<int, 3>{});
    };
    if (p.few)
      by_tokens(n, [&, v0 = v0](auto tiles) {
        const FewGrid f = few_grid(vc);
        const int zparts = (int)few_parts(vc, dim);
        hipLaunchKernelGGL((k_logits_few<float, decltype(tiles)::value, true>), dim3((unsigned)f.grid, (unsigned)zparts),
                           dim3(kThreads), 0, s,
                           in_place, weight_ld, (const float*)hidden, (const float*)hidden, hidden_ld, (int)n, vc,
                           (uint32_t)dim, f.groups, Labels{labels, index_type == ZS_I64, vocab}, (float2*)nullptr, z, vp,
                           (uint32_t)few_columns(vc, dim), p.np * vp);
        hipLaunchKernelGGL((k_join_g<3, true>), dim3(grid_of(p.np * vp / 4)), dim3(kThreads), 0, s, z, zparts, vp, v0, vc, tok,
                           p.np, gp, vp);
        const int64_t waves = (dim + 63) / 64 * p.splits;
        hipLaunchKernelGGL((k_dhidden_few<decltype(tiles)::value>), dim3((unsigned)((waves + 3) / 4)), dim3(kThreads), 0, s,
                           in_place, weight_ld, (const float*)z, vp, tok, vc, (uint32_t)dim, p.splits, (int)(v0 > 0), sums,
                           p.dq, p.np);
      });
    else with_cut(zway.cut, [&](auto shape) {
      using S = decltype(shape);
      auto go = [&](auto planes, auto halves) {
        constexpr bool HALF = decltype(halves)::value && !std::is_same_v<S, Narrow>;  // not for few tokens
        if (zway.splits > 1)
          hipLaunchKernelGGL((k_split<S, K_IN_ROWS, HALF>), dim3(workgroups<S>(vc, n, zway.splits)), dim3(S::THREADS), 0, s,
                             zw, zh, vc, zsegs, (int)(p.dp / kBK), zway.splits, 0, tok.count, z, vp, p.np, w_power, h_power);
        else
          hipLaunchKernelGGL((k_logits<S, decltype(planes)::value, HALF>), dim3(workgroups<S>(vc, n)), dim3(S::THREADS), 0,
                             s, zw, zh, zsegs, (int)(p.dp / kBK), v0, tok, (float2*)nullptr, (float*)nullptr, p.np, gp, vp,
                             w_power, h_power);
      };
      if (half) go(std::integral_constant<int, 3>{}, std::true_type{});
      else by_planes([&](auto planes) { go(planes, std::false_type{}); });
    });
    if (zway.splits > 1 && !p.few)
      by_planes([&](auto planes) {
        hipLaunchKernelGGL((k_join_g<decltype(planes)::value>), dim3(grid_of(p.np * vp / 4)), dim3(kThreads), 0, s, z,
                           zway.splits, vp, v0, vc, tok, p.np, gp, vp);
      });
    if (!p.few) with_cut(dway.cut, [&](auto shape) {
      using S = decltype(shape);
      hipLaunchKernelGGL((k_split<S, K_IS_ROW, false>), dim3(workgroups<S>(dim, n, p.splits)), dim3(S::THREADS), 0, s, w,
                         g_rows, dim, segs, (int)(vp / kBK), p.splits, (int)(v0 > 0), tok.count, sums, p.dq, p.np, w_power,
                         h_power);
    });
    const Way wway = way_of_dweight(dim, vc, p.np / kBK * wsegs.count);
    with_cut(wway.cut == SQUARE ? SQUARE : WIDE, [&](auto shape) {
      using S = std::conditional_t<std::is_same_v<decltype(shape), Square>, Square, Wide>;
      auto go = [&](auto* out, int64_t from, int64_t ld, int alone, int64_t apart) {
        using Gt = std::remove_pointer_t<decltype(out)>;
        hipLaunchKernelGGL((k_dweight<S, Gt>), dim3(workgroups<S>(dim, vc, wway.splits)), dim3(S::THREADS), 0, s, h, g_rows,
                           wsegs, tok.count, from, vc, (uint32_t)dim, out, ld, alone, wway.splits, apart);
      };
      if (wway.splits > 1) go(z, 0, p.dq, 1, vc * p.dq);
      else if (grad_dtype == ZS_BF16) go((uint16_t*)dweight, v0, dweight_ld, (int)first, 0);
      else go((float*)dweight, v0, dweight_ld, (int)first, 0);
    });
    if (wway.splits > 1) {
      auto go = [&](auto* out) {
        using Gt = std::remove_pointer_t<decltype(out)>;
        hipLaunchKernelGGL((k_join_dweight<Gt>), dim3(grid_of(vc * ((p.dq + 7) / 8))), dim3(kThreads), 0, s, z, wway.splits,
                           vc * p.dq, p.dq, vc, (uint32_t)dim, out + v0 * dweight_ld, dweight_ld, (int)first);
      };
      if (grad_dtype == ZS_BF16) go((uint16_t*)dweight);
      else go((float*)dweight);
    }
  }
  auto join = [&](auto type, auto groups) {
    using T = decltype(type);
    constexpr int GROUPS = decltype(groups)::value;
    const unsigned grid = (unsigned)least((n * ((dim + 7) / 8) * GROUPS + kThreads - 1) / kThreads, 1 << 16);
    hipLaunchKernelGGL((k_join_dhidden<T, GROUPS>), dim3(grid), dim3(kThreads), 0, s, sums, p.splits, p.np, p.dq,
                       tok, n, (uint32_t)dim, (const T*)weight, weight_ld, (T*)dhidden, dhidden_ld);
  };
  auto by_splits = [&](auto type) {
    if (p.splits > 4) join(type, std::integral_constant<int, 8>{});
    else join(type, std::integral_constant<int, 1>{});
  };
  if (dtype == ZS_BF16) by_splits(uint16_t{});
  else by_splits(float{});
  return hipGetLastError();
}

}  // namespace zs
