// Embedding lookup with scaling, and its gradient by sorted tokens.
//
//   forward   out_i = scale table[t_i] (+ pos_table[p_i])
//   backward  grad_v = (first ? 0 : grad_v) + scale sum over i with t_i = v of dout_i
//
// Both are bound by memory. The forward copies rows. The backward must not let
// the order of its sums depend on how the hardware interleaves them (tokens
// repeat, the frequent ones thousands of times in a batch), so it sorts the
// positions by token, stably, and adds each token's rows in the order of their
// positions: the sorted list is cut into chunks of equal length, a wave adds
// the rows of one chunk in registers and writes a token's gradient where the
// token's run ends; a run that crosses chunks leaves one partial sum per chunk,
// joined in chunk order by a second kernel.
#include "zs_launch.hpp"
#include "zs_rows.hpp"

namespace zs {
namespace {

__device__ __forceinline__ int64_t id_at(const void* ids, int index_type, int64_t i) {
  return index_type == ZS_I64 ? ld_g(static_cast<const int64_t*>(ids) + i)
                              : (int64_t)ld_g(static_cast<const int32_t*>(ids) + i);
}

// The calling wave's number in the grid, in a scalar register.
__device__ __forceinline__ int64_t wave_id() {
  return (int64_t)blockIdx.x * (kThreads / 64) + __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
}
// a / b for a below 2^32 in 32 bits, where the hardware has no 64-bit divide
__device__ __forceinline__ int64_t quot(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
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

// ---------------------------------------------------------------- forward

// One wave copies one tile of 64 U pieces of a row.
template <typename T, typename O, int VEC, int U>
__global__ __launch_bounds__(kThreads)
void k_embed_fwd(const T* __restrict__ table, int64_t vocab, int64_t dim, int64_t table_ld,
                 const T* __restrict__ pos_table, int64_t pos_rows, int64_t pos_ld, const void* __restrict__ tokens,
                 const void* __restrict__ positions, int index_type, int64_t total, int64_t tiles, float scale,
                 O* __restrict__ out, int64_t out_ld) {
  const int lane = threadIdx.x & 63;
  for (int64_t t = wave_id(); t < total; t += (int64_t)gridDim.x * (kThreads / 64)) {
    const int64_t i = quot(t, tiles);
    const int64_t c0 = (t - i * tiles) * (64 * U * VEC) + lane * VEC;
    const int64_t id = id_at(tokens, index_type, i);
    const bool in = (uint64_t)id < (uint64_t)vocab;  // an id outside of the table selects a row of zeros
    const T* row = table + (in ? id : 0) * table_ld;
    Piece<T, VEC> a[U], p[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (in) load_cols<T, VEC>(a[u], row, c0 + u * 64 * VEC, dim);
      else a[u].clear();
    }
    bool with_pos = false;
    if (pos_table) {
      const int64_t pi = id_at(positions, index_type, i);
      with_pos = (uint64_t)pi < (uint64_t)pos_rows;
      const T* prow = pos_table + (with_pos ? pi : 0) * pos_ld;
      if (with_pos) {
#pragma unroll
        for (int u = 0; u < U; ++u) load_cols<T, VEC>(p[u], prow, c0 + u * 64 * VEC, dim);
      }
    }
    O* orow = out + i * out_ld;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float v[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[e] = with_pos ? fmaf(a[u].get(e), scale, p[u].get(e)) : a[u].get(e) * scale;
      store_cols<O, VEC>(orow, v, c0 + u * 64 * VEC, dim);
    }
  }
}

// ---------------------------------------------------------------- sort

#ifndef FILLG
#define FILLG 512
#endif
#ifndef KW
#define KW 8192
#endif

// Radix sort of (key, position) by digits of kBits bits, lowest first, each pass
// stable. The key of a token that gets no gradient (outside
// of the vocabulary, or the padding token) is `vocab`, behind all others.
constexpr int kBits = 9;
constexpr int kBins = 1 << kBits;
constexpr int kSortRounds = 8;
constexpr int kSortTile = kThreads * kSortRounds;  // entries per workgroup and pass

struct Keys {
  const void* tokens;   // first pass: the tokens themselves
  const uint32_t* keys;  // later passes
  int index_type;
  int64_t vocab, padding;
  __device__ __forceinline__ uint32_t at(int64_t i) const {
    if (keys) return keys[i];
    const int64_t id = id_at(tokens, index_type, i);
    return (uint64_t)id < (uint64_t)vocab && id != padding ? (uint32_t)id : (uint32_t)vocab;
  }
};

// counts[digit][tile]: entries of a tile with that digit
__global__ __launch_bounds__(kThreads)
void k_sort_count(Keys k, int64_t n, int shift, int64_t tiles, uint32_t* __restrict__ counts) {
  __shared__ uint32_t h[kBins];
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    for (int b = threadIdx.x; b < kBins; b += kThreads) h[b] = 0;
    __syncthreads();
    const int64_t i0 = tile * kSortTile;
#pragma unroll
    for (int r = 0; r < kSortRounds; ++r) {
      const int64_t i = i0 + r * kThreads + threadIdx.x;
      if (i < n) atomicAdd(&h[(k.at(i) >> shift) & (kBins - 1)], 1u);
    }
    __syncthreads();
    for (int b = threadIdx.x; b < kBins; b += kThreads) counts[b * tiles + tile] = h[b];
    __syncthreads();
  }
}

// Exclusive sum of v over the workgroup's threads, in thread order; *all gets
// the total. lds: one value per wave and one more.
template <int BS>
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* lds, uint32_t* all) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t s = v;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint32_t y = __shfl_up(s, o, 64);
    if (lane >= o) s += y;
  }
  if (lane == 63) lds[wave] = s;
  __syncthreads();
  uint32_t before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < BS / 64; ++w) {
    if (w < wave) before += lds[w];
    total += lds[w];
  }
  __syncthreads();
  *all = total;
  return before + s - v;
}

// One workgroup per digit: counts[digit][*] become exclusive sums over the
// tiles, totals[digit] their total.
__global__ __launch_bounds__(kThreads)
void k_sort_scan(uint32_t* __restrict__ counts, int64_t tiles, uint32_t* __restrict__ totals) {
  __shared__ uint32_t lds[kThreads / 64];
  uint32_t* c = counts + (int64_t)blockIdx.x * tiles;
  uint32_t run = 0;
  for (int64_t t0 = 0; t0 < tiles; t0 += kThreads) {
    const int64_t t = t0 + threadIdx.x;
    const uint32_t v = t < tiles ? c[t] : 0;
    uint32_t all;
    const uint32_t before = block_scan<kThreads>(v, lds, &all);
    if (t < tiles) c[t] = run + before;
    run += all;
  }
  if (threadIdx.x == 0) totals[blockIdx.x] = run;
}

// Rank of each lane's digit among the wave's earlier entries with the same
// digit: `h` is the wave's own running count per digit. Lanes with live ==
// false take no part.
__device__ __forceinline__ uint32_t wave_rank(uint32_t d, bool live, uint32_t* h) {
  uint64_t same = __ballot(live);
#pragma unroll
  for (int b = 0; b < kBits; ++b) {
    const bool one = (d >> b) & 1u;
    const uint64_t m = __ballot(one);
    same &= one ? m : ~m;
  }
  const int lane = threadIdx.x & 63;
  const int leader = same ? __builtin_ctzll(same) : 0;
  uint32_t before = 0;
  if (live && lane == leader) before = atomicAdd(&h[d], (uint32_t)__popcll(same));
  before = __shfl(before, leader, 64);
  return before + (uint32_t)__popcll(same & ((1ull << lane) - 1));
}

__global__ __launch_bounds__(kThreads)
void k_sort_scatter(Keys k, const uint32_t* __restrict__ pos_in, int64_t n, int shift, int64_t tiles,
                    const uint32_t* __restrict__ counts, const uint32_t* __restrict__ totals,
                    uint32_t* __restrict__ keys_out, uint32_t* __restrict__ pos_out) {
  constexpr int NW = kThreads / 64;
  __shared__ uint32_t hist[NW][kBins];
  __shared__ uint32_t base[kBins];
  __shared__ uint32_t lds[NW];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  static_assert(kBins == 2 * kThreads, "two digits per thread");
  {
    const int b0 = 2 * threadIdx.x;
    const uint32_t v0 = totals[b0], v1 = totals[b0 + 1];
    uint32_t all;
    const uint32_t before = block_scan<kThreads>(v0 + v1, lds, &all);
    base[b0] = before;
    base[b0 + 1] = before + v0;
  }
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    for (int b = threadIdx.x; b < NW * kBins; b += kThreads) (&hist[0][0])[b] = 0;
    __syncthreads();
    const int64_t i0 = tile * kSortTile + wave * (64 * kSortRounds);
    uint32_t key[kSortRounds], rank[kSortRounds];
#pragma unroll
    for (int r = 0; r < kSortRounds; ++r) {
      const int64_t i = i0 + r * 64 + lane;
      key[r] = i < n ? k.at(i) : 0;
      rank[r] = wave_rank((key[r] >> shift) & (kBins - 1), i < n, hist[wave]);
    }
    __syncthreads();
    // where each wave's entries of a digit start
    for (int b = threadIdx.x; b < kBins; b += kThreads) {
      uint32_t at = base[b] + counts[b * tiles + tile];
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const uint32_t c = hist[w][b];
        hist[w][b] = at;
        at += c;
      }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kSortRounds; ++r) {
      const int64_t i = i0 + r * 64 + lane;
      if (i < n) {
        const uint32_t to = hist[wave][(key[r] >> shift) & (kBins - 1)] + rank[r];
        keys_out[to] = key[r];
        pos_out[to] = pos_in ? pos_in[i] : (uint32_t)i;
      }
    }
    __syncthreads();
  }
}

// Zeros into all rows, by the workgroups that `part` of `parts` numbers: tiles
// of kFillTile bytes of the whole table where its rows follow each other
// without gaps, else of each row.
constexpr int kFillTile = 16384;
template <typename Gt, int BS>
__device__ void fill_rows(Gt* grad, int64_t vocab, int64_t dim, int64_t ld, int64_t part, int64_t parts) {
  constexpr int64_t TE = kFillTile / sizeof(Gt);
  constexpr int VEC = 16 / sizeof(Gt);
  if (ld == dim) {
    dim *= vocab;
    vocab = 1;
  }
  const int64_t per_row = (dim + TE - 1) / TE, total = vocab * per_row;
  for (int64_t t = part; t < total; t += parts) {
    const int64_t row = per_row == 1 ? t : t / per_row, c0 = (t - row * per_row) * TE;
    Gt* out = grad + row * ld;
    const int64_t end = c0 + TE < dim ? c0 + TE : dim;
    for (int64_t c = c0 + (int64_t)threadIdx.x * VEC; c < end; c += (int64_t)BS * VEC) {
      if (c + VEC <= end) st16_nt(u32x4{0u, 0u, 0u, 0u}, out + c);
      else
        for (int64_t k = c; k < end; ++k) st_g((Gt)0, out + k);
    }
  }
}

// Up to 1024 R tokens: workgroup 0 sorts them in LDS, in one launch instead of
// three per digit, while the others, where there are any, fill the gradient
// with zeros (`first`).
constexpr int kSmallBS = 1024;
constexpr int kSmallWaves = kSmallBS / 64;
constexpr int64_t kSmallSort = 16 * kSmallBS;
template <int R, typename Gt>
__global__ __launch_bounds__(kSmallBS)
void k_sort_small(Keys k, int n, int passes, uint32_t* __restrict__ keys_out, uint32_t* __restrict__ pos_out,
                  Gt* __restrict__ grad, int64_t dim, int64_t grad_ld) {
  if (blockIdx.x > 0) {
    fill_rows<Gt, kSmallBS>(grad, k.vocab, dim, grad_ld, blockIdx.x - 1, gridDim.x - 1);
    return;
  }
  __shared__ uint32_t skey[R * kSmallBS];
  __shared__ uint16_t spos[R * kSmallBS];  // positions below 2^14
  __shared__ uint32_t hist[kSmallWaves][kBins];
  __shared__ uint32_t base[kBins];
  __shared__ uint32_t lds[kSmallWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t key[R], pos[R];
  // places behind the last token take a key behind all others: they stay last
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int i = (wave * R + r) * 64 + lane;
    pos[r] = i;
    key[r] = i < n ? k.at(i) : 0xffffffffu;
  }
  for (int p = 0; p < passes; ++p) {
    const int shift = p * kBits;
    uint32_t rank[R];
#pragma unroll
    for (int b = 0; b < kBins / 64; ++b) hist[wave][b * 64 + lane] = 0;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup");
#pragma unroll
    for (int r = 0; r < R; ++r) rank[r] = wave_rank((key[r] >> shift) & (kBins - 1), true, hist[wave]);
    __syncthreads();
    // where each digit starts, and each wave's entries within it
    uint32_t run = 0;
    if (threadIdx.x < kBins) {
#pragma unroll
      for (int w = 0; w < kSmallWaves; ++w) {
        const uint32_t c = hist[w][threadIdx.x];
        hist[w][threadIdx.x] = run;
        run += c;
      }
    }
    uint32_t all;
    const uint32_t before = block_scan<kSmallBS>(run, lds, &all);
    if (threadIdx.x < kBins) base[threadIdx.x] = before;
    __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const uint32_t d = (key[r] >> shift) & (kBins - 1);
      const uint32_t to = base[d] + hist[wave][d] + rank[r];
      skey[to] = key[r];
      spos[to] = (uint16_t)pos[r];
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int i = (wave * R + r) * 64 + lane;
      key[r] = skey[i];
      pos[r] = spos[i];
    }
    __syncthreads();
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int i = (wave * R + r) * 64 + lane;
    if (i < n) {
      keys_out[i] = key[r];
      pos_out[i] = pos[r];
    }
  }
}

// ---------------------------------------------------------------- gradient

// The sorted entries are cut into chunks of kWaves K: a workgroup takes one chunk
// and 64 pieces of columns, each of its waves K entries. A wave adds its rows
// in registers and writes the gradient of each token whose run of entries ends
// in it. A run that comes from the wave before is left in LDS for the wave in
// which it starts, which holds its own part in registers and adds the others
// in order; one that comes from the chunk before, or goes on behind the chunk,
// leaves one partial sum in the workspace (rows 2c and 2c + 1 of chunk c),
// joined by k_embed_join.
constexpr int kWaves = 16;

template <typename Gt, int VEC>
__device__ __forceinline__ void put_grad(Gt* row, const float* sum, float scale, bool add, const Piece<Gt, VEC>& old,
                                         int64_t c, int64_t dim) {
  float v[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) v[e] = add ? old.get(e) + sum[e] * scale : sum[e] * scale;
  store_cols<Gt, VEC>(row, v, c, dim);
}

template <typename T, typename Gt, int VEC, int K, bool FIRST>
__global__ __launch_bounds__(kWaves * 64)
void k_embed_chunks(const uint32_t* __restrict__ keys, const uint32_t* __restrict__ pos, int64_t n, uint32_t vocab,
                    int64_t chunks, int64_t coltiles, const T* __restrict__ dout, int64_t dout_ld, int64_t dim,
                    float scale, Gt* __restrict__ grad, int64_t grad_ld, float* __restrict__ partials,
                    int64_t pitch) {
  // rows on their way at once; with them go the gradient's old rows
  constexpr int U = K < 8 ? K : (FIRST || sizeof(Gt) == 2 ? 8 : 4);
  static_assert(K + 2 <= 64 && K % U == 0, "a lane for each entry and its two neighbours");
  __shared__ __align__(16) float heads[kWaves][64 * VEC];
  __shared__ int through[kWaves];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  for (int64_t item = blockIdx.x; item < chunks * coltiles; item += gridDim.x) {
    const int64_t ch = quot(item, coltiles);
    const int64_t c = ((item - ch * coltiles) * 64 + lane) * VEC;
    const int64_t e0 = (ch * kWaves + wave) * K;
    // lane i holds entry e0 - 1 + i; what lies outside the list matches no key
    uint32_t kk = 0xffffffffu, pp = 0;
    {
      const int64_t e = e0 - 1 + lane;
      if (lane < K + 2 && e >= 0 && e < n) {
        kk = keys[e];
        pp = pos[e];
      }
    }
    auto key_at = [&](int u) { return (uint32_t)__builtin_amdgcn_readlane((int)kk, u + 1); };
    // entries with a gradient: they come first in the list
    const int cnt = __popcll(__ballot(lane >= 1 && lane <= K && kk < vocab));
    const bool began = cnt > 0 && key_at(-1) == key_at(0);
    const bool goes = cnt == K && key_at(K) == key_at(K - 1);
    bool whole = began;  // no run has ended in this wave yet
    float acc[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) acc[e] = 0.0f;
#pragma unroll
    for (int u0 = 0; u0 < K; u0 += U) {
      if (u0 >= cnt) break;
      Piece<T, VEC> v[U];
      Piece<Gt, VEC> old[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (u0 + u < cnt) {
          const int64_t row = (uint32_t)__builtin_amdgcn_readlane((int)pp, u0 + u + 1);
          load_cols<T, VEC>(v[u], dout + row * dout_ld, c, dim);
          if (!FIRST && key_at(u0 + u + 1) != key_at(u0 + u))
            load_cols<Gt, VEC>(old[u], grad + (int64_t)key_at(u0 + u) * grad_ld, c, dim);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (u0 + u < cnt) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) acc[e] += v[u].get(e);
          const uint32_t key = key_at(u0 + u);
          if (key_at(u0 + u + 1) != key) {  // the run ends here
            if (whole) {
#pragma unroll
              for (int e = 0; e < VEC; e += 4)
                *reinterpret_cast<f32x4*>(&heads[wave][lane * VEC + e]) = f32x4{acc[e], acc[e + 1], acc[e + 2], acc[e + 3]};
            } else {
              put_grad<Gt, VEC>(grad + (int64_t)key * grad_ld, acc, scale, !FIRST, old[u], c, dim);
            }
            whole = false;
#pragma unroll
            for (int e = 0; e < VEC; ++e) acc[e] = 0.0f;
          }
        }
      }
    }
    if (whole) {  // one run from end to end
#pragma unroll
      for (int e = 0; e < VEC; e += 4)
        *reinterpret_cast<f32x4*>(&heads[wave][lane * VEC + e]) = f32x4{acc[e], acc[e + 1], acc[e + 2], acc[e + 3]};
    }
    if (lane == 0) through[wave] = whole;
    __syncthreads();
    // adds the parts of a run from wave w on; true if it goes on behind the chunk
    auto follow = [&](int w) {
      for (; w < kWaves; ++w) {
#pragma unroll
        for (int e = 0; e < VEC; e += 4) {
          const f32x4 h = *reinterpret_cast<const f32x4*>(&heads[w][lane * VEC + e]);
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[e + q] += h[q];
        }
        if (!through[w]) return false;
      }
      return true;
    };
    if (goes && !whole) {  // a run that starts in this wave and goes on
      if (follow(wave + 1)) {
        if (c < pitch) store_piece<float, VEC>(partials + (2 * ch + 1) * pitch + c, acc);
      } else {
        Piece<Gt, VEC> old;
        Gt* row = grad + (int64_t)key_at(K - 1) * grad_ld;
        if (!FIRST) load_cols<Gt, VEC>(old, row, c, dim);
        put_grad<Gt, VEC>(row, acc, scale, !FIRST, old, c, dim);
      }
    }
    if (wave == 0 && began) {  // one that comes from the chunk before
#pragma unroll
      for (int e = 0; e < VEC; ++e) acc[e] = 0.0f;
      follow(0);
      if (c < pitch) store_piece<float, VEC>(partials + 2 * ch * pitch + c, acc);
    }
    __syncthreads();
  }
}

// One wave per chunk and 64 pieces of columns: a run that starts in this chunk
// and goes on in later ones.
template <typename Gt, int VEC>
__global__ __launch_bounds__(kThreads)
void k_embed_join(const uint32_t* __restrict__ keys, int64_t n, uint32_t vocab, int chunk, int64_t chunks,
                  int64_t coltiles, int64_t dim, float scale, Gt* __restrict__ grad, int64_t grad_ld, int first,
                  const float* __restrict__ partials, int64_t pitch) {
  const int lane = threadIdx.x & 63;
  for (int64_t wv = wave_id(); wv < chunks * coltiles; wv += (int64_t)gridDim.x * (kThreads / 64)) {
    const int64_t ch = quot(wv, coltiles);
    const int64_t c = ((wv - ch * coltiles) * 64 + lane) * VEC;
    const int64_t e1 = (ch + 1) * chunk;
    if (e1 >= n) continue;
    const uint32_t key = keys[e1 - 1], behind = keys[e1], ahead = ch > 0 ? keys[ch * chunk - 1] : 0xffffffffu;
    if (key == vocab || behind != key || ahead == key) continue;  // no run starts here and goes on
    const bool live = c < pitch;
    Gt* row = grad + (int64_t)key * grad_ld;
    Piece<Gt, VEC> old;
    if (!first) load_cols<Gt, VEC>(old, row, c, dim);
    Piece<float, VEC> p;
    if (live) p.load(partials + (2 * ch + 1) * pitch + c);
    else p.clear();
    float sum[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) sum[e] = p.get(e);
    for (int64_t b = ch + 1; b < chunks; b += 64) {
      // the next chunks that begin with this key, 64 at a time
      const uint64_t m = __ballot(b + lane < chunks && keys[(b + lane < chunks ? b + lane : b) * chunk] == key);
      const int more = ~m ? __builtin_ctzll(~m) : 64;
      constexpr int U = 8;
      for (int i = 0; i < more; i += U) {
        Piece<float, VEC> q[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (i + u < more && live) q[u].load(partials + 2 * (b + i + u) * pitch + c);
          else q[u].clear();
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int e = 0; e < VEC; ++e) sum[e] += q[u].get(e);
      }
      if (more < 64) break;
    }
    put_grad<Gt, VEC>(row, sum, scale, !first, old, c, dim);
  }
}

// Zeros into the rows that no token selects. A workgroup takes R (a power of
// two up to 64) rows; each lane below R looks one of them up in the sorted keys.
template <typename Gt, int VEC>
__global__ __launch_bounds__(kThreads)
void k_embed_fill(const uint32_t* __restrict__ keys, int64_t n, int64_t vocab, int R, int64_t groups, int64_t dim,
                  Gt* __restrict__ grad, int64_t grad_ld) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  for (int64_t g = blockIdx.x; g < groups; g += gridDim.x) {
    const int64_t row = g * R + lane;
    bool empty = false;
    if (lane < R && row < vocab) {
      int64_t lo = 0, hi = n;  // first entry not below `row`
      while (lo < hi) {
        const int64_t mid = (lo + hi) >> 1;
        if (keys[mid] < (uint32_t)row) lo = mid + 1;
        else hi = mid;
      }
      empty = lo == n || keys[lo] != (uint32_t)row;
    }
    uint64_t mask = __ballot(empty);
    float z[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) z[e] = 0.0f;
    for (int j = 0; mask; mask &= mask - 1, ++j) {
      if (j % (kThreads / 64) != wave) continue;
      Gt* out = grad + (g * R + __builtin_ctzll(mask)) * grad_ld;
      for (int64_t c = (int64_t)lane * VEC; c < dim; c += 64 * VEC) store_cols<Gt, VEC>(out, z, c, dim);
    }
  }
}

template <typename T, typename Gt>
constexpr int vec_of() { return sizeof(T) == 2 || sizeof(Gt) == 2 ? 8 : 4; }

template <typename T, typename O>
void run_embed_fwd(const T* table, int64_t vocab, int64_t dim, int64_t table_ld, const T* pos_table, int64_t pos_rows,
                   int64_t pos_ld, const void* tokens, const void* positions, int index_type, int64_t n, float scale,
                   O* out, int64_t out_ld, hipStream_t s) {
  constexpr int VEC = vec_of<T, O>();
  auto go = [&](auto uu) {
    constexpr int U = decltype(uu)::value;
    const int64_t tiles = (dim + 64 * U * VEC - 1) / (64 * U * VEC), total = n * tiles;
    hipLaunchKernelGGL((k_embed_fwd<T, O, VEC, U>), dim3((unsigned)grid_for(total, kThreads / 64)), dim3(kThreads), 0,
                       s, table, vocab, dim, table_ld, pos_table, pos_rows, pos_ld, tokens, positions, index_type,
                       total, tiles, scale, out, out_ld);
  };
  const int64_t pieces = (dim + 64 * VEC - 1) / (64 * VEC);
  if (pieces == 1) go(std::integral_constant<int, 1>{});
  else go(std::integral_constant<int, 2>{});
}

template <typename T, typename Gt>
void run_embed_bwd(const EmbedPlan& p, const Keys& tokens, uint32_t* const* keys, uint32_t* const* pos,
                   uint32_t* counts, uint32_t* totals, float* partials, const T* dout, int64_t dout_ld, int64_t n,
                   int64_t vocab, int64_t dim, float scale, Gt* grad, int64_t grad_ld, bool first, hipStream_t s) {
  constexpr int VEC = vec_of<T, Gt>();
  int last = 0;
  if (n <= kSmallSort) {
    // the zeros: a workgroup per CU and a half, or fewer for a small table
    const int64_t tiles = first ? (vocab * dim * (int64_t)sizeof(Gt) + kFillTile - 1) / kFillTile : 0;
    const dim3 gd((unsigned)(1 + (tiles < FILLG ? tiles : FILLG))), bd(kSmallBS);
    auto go = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, gd, bd, 0, s, tokens, (int)n, p.passes, keys[0], pos[0], grad, dim, grad_ld);
    };
    if (n <= kSmallBS) go(k_sort_small<1, Gt>);
    else if (n <= 4 * kSmallBS) go(k_sort_small<4, Gt>);
    else if (n <= 8 * kSmallBS) go(k_sort_small<8, Gt>);
    else go(k_sort_small<16, Gt>);
  } else {
    const dim3 gd((unsigned)grid_for(p.tiles, 1)), bd(kThreads);
    for (int i = 0; i < p.passes; ++i) {
      const int src = (i + 1) & 1, dst = i & 1;
      Keys k = tokens;
      if (i) k.keys = keys[src];
      hipLaunchKernelGGL(k_sort_count, gd, bd, 0, s, k, n, i * kBits, p.tiles, counts);
      hipLaunchKernelGGL(k_sort_scan, dim3(kBins), bd, 0, s, counts, p.tiles, totals);
      hipLaunchKernelGGL(k_sort_scatter, gd, bd, 0, s, k, i ? pos[src] : nullptr, n, i * kBits, p.tiles, counts,
                         totals, keys[dst], pos[dst]);
      last = dst;
    }
    if (first) {
      int R = 1;
      while (R < 64 && vocab / (2 * R) >= 2048) R *= 2;
      const int64_t groups = (vocab + R - 1) / R;
      hipLaunchKernelGGL((k_embed_fill<Gt, VEC>), dim3((unsigned)grid_for(groups, 1)), dim3(kThreads), 0, s,
                         keys[last], n, vocab, R, groups, dim, grad, grad_ld);
    }
  }
  if (n == 0) return;
  const int64_t coltiles = (dim + 64 * VEC - 1) / (64 * VEC), items = p.chunks * coltiles;
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)grid_for(items, 1, kWaves * 64)), dim3(kWaves * 64), 0, s, keys[last],
                       pos[last], n, (uint32_t)vocab, p.chunks, coltiles, dout, dout_ld, dim, scale, grad, grad_ld,
                       partials, p.pitch);
  };
  auto pick = [&](auto f) {
    constexpr bool F = decltype(f)::value;
    if (p.chunk == 4 * kWaves) go(k_embed_chunks<T, Gt, VEC, 4, F>);
    else if (p.chunk == 8 * kWaves) go(k_embed_chunks<T, Gt, VEC, 8, F>);
    else go(k_embed_chunks<T, Gt, VEC, 16, F>);
  };
  if (first) pick(std::true_type{});
  else pick(std::false_type{});
  if (p.chunks > 1)
    hipLaunchKernelGGL((k_embed_join<Gt, VEC>), dim3((unsigned)grid_for(items, kThreads / 64)), dim3(kThreads), 0, s,
                       keys[last], n, (uint32_t)vocab, p.chunk, p.chunks, coltiles, dim, scale, grad, grad_ld,
                       (int)first, partials, p.pitch);
}

}  // namespace

EmbedPlan embed_plan(int64_t n, int64_t vocab, int64_t dim) {
  EmbedPlan p;
  p.pitch = (dim + 7) / 8 * 8;
  const int64_t coltiles = (dim + 511) / 512;
  int k = 4;  // entries per wave
  while (k < 16 && n / k * coltiles > KW) k *= 2;
  p.chunk = k * kWaves;
  p.chunks = (n + p.chunk - 1) / p.chunk;
  p.bits = 1;  // keys are 0 .. vocab
  while (p.bits < 32 && (vocab >> p.bits) != 0) ++p.bits;
  p.passes = (p.bits + kBits - 1) / kBits;
  p.tiles = (n + kSortTile - 1) / kSortTile;
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t r = at;
    at += (bytes + 255) / 256 * 256;
    return r;
  };
  for (int i = 0; i < 2; ++i) {
    p.keys[i] = take(4 * n);
    p.pos[i] = take(4 * n);
  }
  p.counts = take(4 * p.tiles * kBins);
  p.totals = take(4 * kBins);
  p.partials = take(4 * 2 * p.chunks * p.pitch);
  p.bytes = at;
  return p;
}

hipError_t launch_embed_forward(const void* table, int dtype, int64_t vocab, int64_t dim, int64_t table_ld,
                                const void* pos_table, int64_t pos_rows, int64_t pos_ld, const void* tokens,
                                const void* positions, int index_type, int64_t n, float scale, void* out,
                                int out_dtype, int64_t out_ld, hipStream_t s) {
  auto go = [&](auto* t, auto* o) {
    using T = std::remove_pointer_t<decltype(t)>;
    run_embed_fwd(static_cast<const T*>(table), vocab, dim, table_ld, static_cast<const T*>(pos_table), pos_rows,
                  pos_ld, tokens, positions, index_type, n, scale, static_cast<decltype(o)>(out), out_ld, s);
  };
  uint16_t* h = nullptr;
  float* f = nullptr;
  if (dtype == ZS_BF16) out_dtype == ZS_BF16 ? go(h, h) : go(h, f);
  else out_dtype == ZS_BF16 ? go(f, h) : go(f, f);
  return hipGetLastError();
}

hipError_t launch_embed_backward(const void* dout, int dtype, int64_t dout_ld, const void* tokens, int index_type,
                                 int64_t n, int64_t vocab, int64_t dim, int64_t padding_idx, float scale, void* grad,
                                 int grad_dtype, int64_t grad_ld, bool first, void* workspace, hipStream_t s) {
  const EmbedPlan p = embed_plan(n, vocab, dim);
  char* ws = static_cast<char*>(workspace);
  uint32_t *keys[2], *pos[2];
  for (int i = 0; i < 2; ++i) {
    keys[i] = reinterpret_cast<uint32_t*>(ws + p.keys[i]);
    pos[i] = reinterpret_cast<uint32_t*>(ws + p.pos[i]);
  }
  uint32_t* counts = reinterpret_cast<uint32_t*>(ws + p.counts);
  uint32_t* totals = reinterpret_cast<uint32_t*>(ws + p.totals);
  float* partials = reinterpret_cast<float*>(ws + p.partials);
  const Keys k{tokens, nullptr, index_type, vocab, padding_idx};
  auto go = [&](auto* t, auto* g) {
    run_embed_bwd(p, k, keys, pos, counts, totals, partials,
                  static_cast<const std::remove_pointer_t<decltype(t)>*>(dout), dout_ld, n, vocab, dim, scale,
                  static_cast<decltype(g)>(grad), grad_ld, first, s);
  };
  uint16_t* h = nullptr;
  float* f = nullptr;
  if (dtype == ZS_BF16) grad_dtype == ZS_BF16 ? go(h, h) : go(h, f);
  else grad_dtype == ZS_BF16 ? go(f, h) : go(f, f);
  return hipGetLastError();
}

}  // namespace zs
