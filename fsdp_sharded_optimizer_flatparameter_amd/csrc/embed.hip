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
#include "zs_launch_rows.hpp"
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

// ---------------------------------------------------------------- forward

// One wave copies one tile of 64 U pieces of a row. Bound by memory: 16384 rows
// of 4096 bf16, drawn as a text's tokens are (191 MB), take 34 us. The output
// is stored past the caches: 41 us with plain stores, and 9.3 against 9.9 for
// 8192 rows of 768 with their positions.
template <typename T, typename O, int VEC, int U>
__global__ __launch_bounds__(kThreads)
void k_embed_fwd(const T* __restrict__ table, int64_t vocab, uint32_t dim, int64_t table_ld,
                 const T* __restrict__ pos_table, int64_t pos_rows, int64_t pos_ld, const void* __restrict__ tokens,
                 const void* __restrict__ positions, int index_type, int64_t total, int64_t tiles, float scale,
                 O* __restrict__ out, int64_t out_ld) {
  const int lane = threadIdx.x & 63;
  for (int64_t t = wave_id(); t < total; t += (int64_t)gridDim.x * (kThreads / 64)) {
    const int64_t i = quot(t, tiles);
    const uint32_t c0 = (uint32_t)(t - i * tiles) * (64 * U * VEC) + lane * VEC;
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
    const T* prow = pos_table;
    if (pos_table) {
      const int64_t pi = id_at(positions, index_type, i);
      with_pos = (uint64_t)pi < (uint64_t)pos_rows;
      prow = pos_table + (with_pos ? pi : 0) * pos_ld;
      if (with_pos) {
#pragma unroll
        for (int u = 0; u < U; ++u) load_cols<T, VEC>(p[u], prow, c0 + u * 64 * VEC, dim);
      }
    }
    if (ragged(dim, VEC))
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (in) settle_cols<T, VEC>(a[u], row, c0 + u * 64 * VEC, dim);
        if (with_pos) settle_cols<T, VEC>(p[u], prow, c0 + u * 64 * VEC, dim);
      }
    O* orow = out + i * out_ld;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float v[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[e] = with_pos ? fmaf(a[u].get(e), scale, p[u].get(e)) : a[u].get(e) * scale;
      store_cols<O, VEC, true>(orow, v, c0 + u * 64 * VEC, dim);
    }
  }
}

// ---------------------------------------------------------------- zeros

// Stores past the caches from one-wave workgroups with a short piece each keep
// the most writes on their way: the call that writes 128256 x 4096 bf16 took
// 233 us so, 248 with pieces of 8 KiB, 253 with 16 KiB, 240 with 2 KiB, and 250
// with four-wave workgroups or plain stores.
constexpr int64_t kFillBytes = 4096;
// Up to kFillTogether bytes of a gradient are zeroed by the first launch of the
// sort, in all rows, beside the workgroups that sort; of more, kFillBeside bytes
// beside each launch, and after the sort the rows of the rest that no token
// selects. 8192 tokens into 16384 x 1024 fp32 (67 MB): 26.3 us against 29.9 the second
// way; into 50257 x 768 fp32 (154 MB): 38.3, 39.0 all in the first launch;
// 16384 into 128256 x 4096 bf16 (1.05 GB): 211, 222 with nothing beside the
// sort, 216 with 160 MB. (Counted in pieces of kFillBytes: less where rows
// below 64 bytes make them smaller.)
constexpr int64_t kFillTogether = 100000000;
constexpr int64_t kFillBeside = 60000000;

// With `first` the rows that no token selects are zero. The table is cut into
// pieces of about kFillBytes, a wave for each: `step` (up to 64) narrow rows,
// or a part of a wide one.
template <typename Gt>
struct Fill {
  Gt* grad;
  int64_t vocab, ld;
  uint32_t dim, width;  // columns of a piece
  int step, across;     // rows of a piece, pieces across a row
  int64_t begin, end;   // pieces to fill
};
template <typename Gt>
Fill<Gt> fill_plan(Gt* grad, int64_t vocab, int64_t dim, int64_t ld) {
  const int64_t row = dim * (int64_t)sizeof(Gt), fit = kFillBytes / row;
  Fill<Gt> f{grad, vocab, ld, (uint32_t)dim, (uint32_t)dim, (int)(fit < 1 ? 1 : fit > 64 ? 64 : fit),
             (int)((row + kFillBytes - 1) / kFillBytes), 0, 0};
  if (f.across > 1) f.width = kFillBytes / sizeof(Gt);
  f.end = (vocab + f.step - 1) / f.step * f.across;
  return f;
}
// Piece t, without the rows that `touched` marks (none are where it is null).
template <typename Gt>
__device__ __forceinline__ void fill_piece(const Fill<Gt>& f, int64_t t, const uint8_t* touched) {
  constexpr uint32_t VEC = 16 / sizeof(Gt);
  const int lane = threadIdx.x & 63;
  const int64_t g = quot(t, f.across), r0 = g * f.step, row = r0 + lane;
  const uint32_t c0 = (uint32_t)(t - g * f.across) * f.width, c1 = c0 + f.width < f.dim ? c0 + f.width : f.dim;
  for (uint64_t empty = __ballot(lane < f.step && row < f.vocab && !(touched && touched[row])); empty;
       empty &= empty - 1) {
    Gt* out = f.grad + (r0 + __builtin_ctzll(empty)) * f.ld;
    for (uint32_t c = c0 + lane * VEC; c < c1; c += 64 * VEC) {
      if (c + VEC <= c1) st16_nt(u32x4{0u, 0u, 0u, 0u}, out + c);
      else
        for (uint32_t k = c; k < c1; ++k) st_g((Gt)0, out + k);
    }
  }
}

// One-wave workgroups, a piece each.
template <typename Gt>
__global__ __launch_bounds__(64)
void k_embed_fill(Fill<Gt> f, const uint8_t* __restrict__ touched) {
  for (int64_t t = f.begin + blockIdx.x; t < f.end; t += gridDim.x) fill_piece(f, t, touched);
}

// ---------------------------------------------------------------- sort

// Radix sort of (key, position) by digits of up to kBits bits, lowest first, each
// pass stable. The key of a token that gets no gradient (outside of the
// vocabulary, or the padding token) is `vocab`, behind all others.
constexpr int kBits = 9;
// In the passes of up to kPassSort entries also of up to kWideBits, where that
// saves a pass: vocabularies of 2^9 to 2^11 (one pass), of 2^18 to 2^22 (two) and
// from 2^27 (three), as far as the sort by ranges does not take them.
constexpr int kWideBits = 11;
constexpr int kBins = 1 << kBits;
constexpr int kSortRounds = 8;
constexpr int kSortTile = kThreads * kSortRounds;  // entries per workgroup and pass

struct Keys {
  const void* tokens;   // first pass: the tokens themselves
  const uint32_t* keys;  // later passes
  int index_type;
  int64_t vocab, padding;
  __device__ __forceinline__ uint32_t of(int64_t id) const {
    return (uint64_t)id < (uint64_t)vocab && id != padding ? (uint32_t)id : (uint32_t)vocab;
  }
  // The keys of entries i, i + step, ... (the last entry's for those at or past
  // n, which is above 0): all loads are on their way before the first is
  // looked at, without a branch between them.
  template <int N>
  __device__ __forceinline__ void load(uint32_t* out, int64_t i, int64_t step, int64_t n) const {
    auto at = [&](int u) { return i + u * step < n ? i + u * step : n - 1; };
    if (keys) {
#pragma unroll
      for (int u = 0; u < N; ++u) out[u] = ld_g(keys + at(u));
    } else if (index_type == ZS_I64) {
      int64_t id[N];
#pragma unroll
      for (int u = 0; u < N; ++u) id[u] = ld_g(static_cast<const int64_t*>(tokens) + at(u));
#pragma unroll
      for (int u = 0; u < N; ++u) out[u] = of(id[u]);
    } else {
      int32_t id[N];
#pragma unroll
      for (int u = 0; u < N; ++u) id[u] = ld_g(static_cast<const int32_t*>(tokens) + at(u));
#pragma unroll
      for (int u = 0; u < N; ++u) out[u] = of(id[u]);
    }
  }
};

// counts[digit][tile]: entries of a tile with that digit
__global__ __launch_bounds__(kThreads)
void k_sort_count(Keys k, int64_t n, int shift, int64_t tiles, uint32_t* __restrict__ counts,
                  uint8_t* __restrict__ touched) {
  __shared__ uint32_t h[kBins];
  if (touched)  // the first pass clears it
    for (int64_t i = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * 16; i < k.vocab;
         i += (int64_t)gridDim.x * kThreads * 16)
      st16(u32x4{0u, 0u, 0u, 0u}, touched + i);  // the array's room is a multiple of 16
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    for (int b = threadIdx.x; b < kBins; b += kThreads) h[b] = 0;
    __syncthreads();
    const int64_t i0 = tile * kSortTile + threadIdx.x;
    uint32_t key[kSortRounds];
    k.load<kSortRounds>(key, i0, kThreads, n);
#pragma unroll
    for (int r = 0; r < kSortRounds; ++r)
      if (i0 + r * kThreads < n) atomicAdd(&h[(key[r] >> shift) & (kBins - 1)], 1u);
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

// Lanes before this one, among those with live set, that hold the same digit;
// *same gets all that do. A lane that is not live gets nothing of use.
template <int MAXB>
__device__ __forceinline__ uint32_t rank_in_wave(uint32_t d, int bits, bool live, uint64_t* same) {
  uint64_t s = __ballot(live);
#pragma unroll
  for (int b = 0; b < MAXB; ++b) {
    if (b >= bits) break;
    const bool one = (d >> b) & 1u;
    const uint64_t m = __ballot(one);
    s &= one ? m : ~m;
  }
  *same = s;
  return (uint32_t)__popcll(s & ((1ull << (threadIdx.x & 63)) - 1));
}

// The same over several rounds: `h` is the wave's own running count per digit.
__device__ __forceinline__ uint32_t wave_rank(uint32_t d, bool live, uint32_t* h) {
  uint64_t same;
  const uint32_t rank = rank_in_wave<kBits>(d, kBits, live, &same);
  const int leader = same ? __builtin_ctzll(same) : 0;
  uint32_t before = 0;
  if (live && rank == 0) before = atomicAdd(&h[d], (uint32_t)__popcll(same));
  return __shfl(before, leader, 64) + rank;
}

__global__ __launch_bounds__(kThreads)
void k_sort_scatter(Keys k, const uint32_t* __restrict__ pos_in, int64_t n, int shift, int64_t tiles,
                    const uint32_t* __restrict__ counts, const uint32_t* __restrict__ totals,
                    uint32_t* __restrict__ keys_out, uint32_t* __restrict__ pos_out, uint8_t* __restrict__ touched) {
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
    k.load<kSortRounds>(key, i0 + lane, 64, n);
#pragma unroll
    for (int r = 0; r < kSortRounds; ++r) {
      const int64_t i = i0 + r * 64 + lane;
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
        if (touched && key[r] < (uint32_t)k.vocab) touched[key[r]] = 1;  // the last pass sets it
      }
    }
    __syncthreads();
  }
}

// One pass over up to kPassSort entries in one launch: each workgroup counts the
// digits of all entries itself (they lie in L2), those of the tiles before its
// own apart, and then places its own tile, an entry per thread. Counting by
// tiles in a launch of its own, their sums in a second and the placing in a
// third (k_sort_count, k_sort_scan, k_sort_scatter) takes 12 us a pass at any
// of these sizes, this 6 us for 8192 entries and 25 for 65536 (the call for
// 32768 rows of 1024: 80 us either way when the limit was set, 61 now; for
// 65536 of 768: 120 us instead of 94).
// The first pass clears `touched`, a byte per row of the gradient, with `clears`
// workgroups behind the tiles; the last one sets it for each token's row. The
// workgroups behind those fill pieces of the gradient, one for each wave.
constexpr int kPassBS = 1024;
constexpr int kPassWaves = kPassBS / 64;
constexpr int64_t kPassSort = 32768;
constexpr int kClearBytes = kPassBS * 16;  // of `touched`, per workgroup

__device__ __forceinline__ void clear_touched(uint8_t* touched, int64_t vocab, int64_t block) {
  const int64_t i = block * kClearBytes + (int64_t)threadIdx.x * 16;
  if (i < vocab) st16(u32x4{0u, 0u, 0u, 0u}, touched + i);  // the array's room is a multiple of 16
}

// Start of each wave's entries of each digit: hist holds the waves' counts and
// gets the places, `sum` are the thread's digits' entries in the whole list and
// `mine` those before the tile. Digits t and t + kPassBS belong to thread t.
template <int BINS>
__device__ __forceinline__ void place_digits(uint16_t (*hist)[BINS], int bins, const uint32_t* sum,
                                             const uint32_t* mine, uint32_t* lds) {
  constexpr int D = BINS > kPassBS ? BINS / kPassBS : 1;
  uint32_t start = 0;
#pragma unroll
  for (int q = 0; q < D; ++q) {
    const int b = q * kPassBS + threadIdx.x;
    uint32_t all;
    uint32_t at = start + block_scan<kPassBS>(sum[q], lds, &all) + mine[q];
    start += all;
    if (b < bins) {
      uint32_t c[kPassWaves];
#pragma unroll
      for (int w = 0; w < kPassWaves; ++w) c[w] = hist[w][b];
#pragma unroll
      for (int w = 0; w < kPassWaves; ++w) {
        hist[w][b] = (uint16_t)at;  // places stay below 2^15
        at += c[w];
      }
    }
  }
}

template <typename Gt, int MAXB>
__global__ __launch_bounds__(kPassBS)
void k_sort_pass(Keys k, const uint32_t* __restrict__ pos_in, int n, int shift, int bits, int tiles, int clears, int last,
                 uint32_t* __restrict__ keys_out, uint32_t* __restrict__ pos_out, uint8_t* __restrict__ touched,
                 Fill<Gt> fill) {
  // Copies of the counters, each for every so many-th lane and shifted by a
  // bank: frequent tokens have several lanes of a wave count in one place, one
  // after the other (16384 entries: 37.5 us for the call with 8 copies, 42 with
  // one). A counter holds the entries before the tile in its lower half and all
  // in its upper half.
  constexpr int BINS = 1 << MAXB, ROOM = 4096 + 8;
  constexpr int D = BINS > kPassBS ? BINS / kPassBS : 1;
  static_assert(kPassSort < 65536, "16 bits hold a count and a place");
  __shared__ uint32_t counts[ROOM];
  __shared__ uint16_t hist[kPassWaves][BINS];
  __shared__ uint32_t lds[kPassWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if ((int)blockIdx.x >= tiles) {
    const int b = (int)blockIdx.x - tiles;
    if (b < clears) {
      clear_touched(touched, k.vocab, b);
    } else {
      const int64_t t = fill.begin + (int64_t)(b - clears) * kPassWaves + wave;
      if (t < fill.end) fill_piece(fill, t, nullptr);
    }
    return;
  }
  const int bins = 1 << bits, copies = bins <= 512 ? 8 : 4096 / bins;
  auto digit = [&](uint32_t key) { return (key >> shift) & (bins - 1); };
  const int tile0 = blockIdx.x * kPassBS, i = tile0 + threadIdx.x;
  constexpr int U = 8;  // entries on their way per thread
  uint32_t kk[U], key;
  k.load<1>(&key, i, 0, n);
  const uint32_t pos = pos_in ? ld_g(pos_in + (i < n ? i : n - 1)) : (uint32_t)i;
  k.load<U>(kk, threadIdx.x, kPassBS, n);
  for (int b = threadIdx.x; b < copies * (bins + 1); b += kPassBS) counts[b] = 0;
  for (int b = lane; b < bins; b += 64) hist[wave][b] = 0;
  __syncthreads();
  uint32_t* own = counts + (lane & (copies - 1)) * (bins + 1);
  for (int j0 = threadIdx.x; j0 < n; j0 += U * kPassBS) {
    if (j0 != (int)threadIdx.x) k.load<U>(kk, j0, kPassBS, n);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = j0 + u * kPassBS;
      if (j < n) atomicAdd(&own[digit(kk[u])], j < tile0 ? 0x10001u : 0x10000u);
    }
  }
  // rank within the wave, and the wave's count of each digit
  const uint32_t d = digit(key);
  uint64_t same;
  const uint32_t rank = rank_in_wave<MAXB>(d, bits, i < n, &same);
  if (i < n && rank == 0) hist[wave][d] = (uint16_t)__popcll(same);
  __syncthreads();
  uint32_t sum[D], mine[D];
#pragma unroll
  for (int q = 0; q < D; ++q) {
    sum[q] = mine[q] = 0;
    const int b = q * kPassBS + threadIdx.x;
    if (b < bins)
      for (int c = 0; c < copies; ++c) {
        const uint32_t v = counts[c * (bins + 1) + b];
        mine[q] += v & 0xffffu;
        sum[q] += v >> 16;
      }
  }
  place_digits<BINS>(hist, bins, sum, mine, lds);
  __syncthreads();
  if (i < n) {
    const uint32_t to = hist[wave][d] + rank;
    keys_out[to] = key;
    pos_out[to] = pos;
    if (last && touched && key < (uint32_t)k.vocab) touched[key] = 1;
  }
}

// The whole sort in one launch. Each workgroup takes a range of up to kRangeBins
// keys: it looks at all entries (they lie in L2), counts those of the ranges
// before, leaves its own in LDS in their order and sorts these in one pass over
// the whole of their digits. Entries without a gradient are in no range; the
// last workgroup writes their keys behind the others. R: rounds of kPassBS
// entries. The call for 8192 tokens of 768 into 50257 fp32 rows takes 19.7 us
// against 24.4 with two passes, for 2048 12.9 against 15.1 with both passes in
// one workgroup, for 16384 into 2048 rows of 1024 29.5 against 32.2.
// It loses where every workgroup has too much to look at (32768 entries: 49.5
// against 37.1 with 300 keys, 71 against 48 with 256000), or where there are more
// of them than run at once: two per CU up to half of kRangeSort, then one for the
// list's room (16384 entries, 256000 keys: 35.5 against 32.7); and with a table so large
// that its zeros need the time of two passes beside them (16384 into
// 128256 x 4096 bf16: 215 against 210).
constexpr int64_t kRangeSort = 16 * kPassBS;
constexpr int kRangeBits = 9, kRangeBins = 1 << kRangeBits;
constexpr int64_t kRanges = 256;  // workgroups before a range gets more keys; 128 and 64: up to 0.3 us more
constexpr bool by_ranges(int64_t n, int64_t vocab) {
  return n <= kRangeSort && vocab <= kRangeBins * kRanges * (n <= kRangeSort / 2 ? 2 : 1);
}
template <typename Gt, int R>
__global__ __launch_bounds__(kPassBS)
void k_sort_ranges(Keys k, int n, int bits, int ranges, uint32_t* __restrict__ keys_out, uint32_t* __restrict__ pos_out,
                   Fill<Gt> fill) {
  static_assert(R * kPassBS <= 65536, "a position in 16 bits");
  __shared__ uint32_t list[R * kPassBS];
  __shared__ __align__(4) uint16_t hist[kPassWaves][kRangeBins];
  __shared__ uint32_t lds[kPassWaves], within[kPassWaves], under[kPassWaves];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  if ((int)blockIdx.x >= ranges) {
    const int64_t t = fill.begin + (int64_t)((int)blockIdx.x - ranges) * kPassWaves + wave;
    if (t < fill.end) fill_piece(fill, t, nullptr);
    return;
  }
  const int bins = 1 << bits;
  const uint32_t lo = blockIdx.x << bits, vocab = (uint32_t)k.vocab;
  const uint32_t room = vocab - lo < (uint32_t)bins ? vocab - lo : (uint32_t)bins;  // keys of the range
  // a wave's entries are consecutive, so that their order is that of waves, rounds and lanes
  const int rounds = (n + kPassBS - 1) / kPassBS, i0 = wave * rounds * 64 + lane;
  uint32_t key[R];
  constexpr int U = R < 16 ? R : 16;  // entries on their way per thread
#pragma unroll
  for (int r = 0; r < R; r += U)
    if (r < rounds) k.load<U>(key + r, i0 + r * 64, 64, n);
  for (int b = lane; b < bins / 2; b += 64) reinterpret_cast<uint32_t*>(hist[wave])[b] = 0;
  auto live = [&](int r) { return r < rounds && i0 + r * 64 < n; };
  int own = 0, less = 0;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    own += __popcll(__ballot(live(r) && key[r] - lo < room));
    less += __popcll(__ballot(live(r) && key[r] < lo));
  }
  if (lane == 0) {
    within[wave] = own;
    under[wave] = less;
  }
  __syncthreads();
  int at = 0, count = 0;
  uint32_t base = 0;
#pragma unroll
  for (int w = 0; w < kPassWaves; ++w) {
    if (w < wave) at += within[w];
    count += within[w];
    base += under[w];
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const bool in = live(r) && key[r] - lo < room;
    const uint64_t m = __ballot(in);
    if (in) list[at + __popcll(m & ((1ull << lane) - 1))] = (key[r] - lo) << 16 | (uint32_t)(i0 + r * 64);
    at += __popcll(m);
  }
  __syncthreads();
  const int turns = (count + kPassBS - 1) / kPassBS, j0 = wave * turns * 64 + lane;
  for (int j = j0, t = 0; t < turns; ++t, j += 64)
    if (j < count) {
      const uint32_t d = list[j] >> 16;
      atomicAdd(reinterpret_cast<uint32_t*>(hist[wave]) + d / 2, 1u << (d % 2 * 16));
    }
  __syncthreads();
  uint32_t sum = 0;
  if ((int)threadIdx.x < bins)
#pragma unroll
    for (int w = 0; w < kPassWaves; ++w) sum += hist[w][threadIdx.x];
  place_digits<kRangeBins>(hist, bins, &sum, &base, lds);
  __syncthreads();
  for (int j = j0, t = 0; t < turns; ++t, j += 64) {
    const bool on = j < count;
    const uint32_t e = on ? list[j] : 0, d = e >> 16;
    uint64_t same = __ballot(on);
    if (same == 0) break;
    uint32_t rank;
    if (__ballot(on && d != (uint32_t)__builtin_amdgcn_readfirstlane((int)d)) == 0)  // (lane 0 is on)
      rank = (uint32_t)__popcll(same & ((1ull << lane) - 1));
    else
      rank = rank_in_wave<kRangeBits>(d, bits, on, &same);
    const uint32_t start = hist[wave][d];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (on && rank == 0) hist[wave][d] = (uint16_t)(start + __popcll(same));
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (on) {
      keys_out[start + rank] = lo + d;
      pos_out[start + rank] = e & 0xffffu;
    }
  }
  if ((int)blockIdx.x == ranges - 1)
    for (int i = (int)base + count + (int)threadIdx.x; i < n; i += kPassBS) keys_out[i] = vocab;
}

// ---------------------------------------------------------------- gradient

// dout of more bytes than this is read past the caches: 65536 rows of 768 bf16
// (101 MB) 74 instead of 86 us for the call, 32768 of 1024 (67 MB) 61 instead of
// 65; 16384 of 768 (25 MB), which the caches can hold, 37.3 instead of 35.8.
constexpr int64_t kStreamBytes = 60000000;
// Entries per wave are doubled from 4 up to 16 while there are more waves than
// this: 4 for all costs 243 instead of 202 us with 131072 tokens, whose partial
// sums then weigh; fewer waves leave compute units without work.
constexpr int64_t kChunkWaves = 8192;

// Up to this many tokens make one chunk, and the call one launch.
constexpr int64_t kFewTokens = 8 * 8;

// The sorted entries are cut into chunks of kWaves K: a workgroup takes one chunk
// and 64 pieces of columns, each of its waves K entries. A wave adds its rows
// in registers and writes the gradient of each token whose run of entries ends
// in it. A run that comes from the wave before is left in LDS for the wave in
// which it starts, which holds its own part in registers and adds the others
// in order; one that comes from the chunk before, or goes on behind the chunk,
// leaves one partial sum in the workspace (rows 2c and 2c + 1 of chunk c),
// joined by k_embed_join.
constexpr int kWaves = 8;
static_assert(kFewTokens == 8 * kWaves, "one chunk");

template <typename Gt, int VEC>
__device__ __forceinline__ void put_grad(Gt* row, const float* sum, float scale, bool add, const Piece<Gt, VEC>& old,
                                         uint32_t c, uint32_t dim) {
  float v[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) v[e] = add ? old.get(e) + sum[e] * scale : sum[e] * scale;
  store_cols<Gt, VEC>(row, v, c, dim);
}

// With SORT, for the few entries of one chunk, each workgroup sorts the tokens
// itself by counting for each one those that come before it, and that is the
// whole call: 3.2 us for one token instead of 8.1, 7.5 for 64 instead of 10.4
// (128 would take 12.3 instead of 11.0).
template <typename T, typename Gt, int VEC, int K, bool FIRST, bool NT, bool SORT>
__global__ __launch_bounds__(kWaves * 64)
void k_embed_chunks(Keys tokens, const uint32_t* __restrict__ keys, const uint32_t* __restrict__ pos, int64_t n,
                    uint32_t vocab, int64_t chunks, int64_t coltiles, const T* __restrict__ dout, int64_t dout_ld, uint32_t dim,
                    float scale, Gt* __restrict__ grad, int64_t grad_ld, float* __restrict__ partials,
                    uint32_t pitch) {
  // Rows on their way at once; with them go the gradient's old rows (11408 rows
  // of 1728 bf16 into a bf16 accumulator: 34.6 us with 4, 40.0 with 8, which
  // take half of the registers).
  constexpr int U = K < 8 || sizeof(T) * VEC > 16 || !FIRST ? 4 : 8;
  static_assert(K + 2 <= 64 && K % U == 0, "a lane for each entry and its two neighbours");
  __shared__ __align__(16) float heads[kWaves][64 * VEC];
  __shared__ int through[kWaves];
  constexpr int M = SORT ? K * kWaves : 1;
  __shared__ uint32_t skey[M], spos[M];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  if constexpr (SORT) {
    __shared__ __align__(16) uint32_t all[M];
    const int t = threadIdx.x;
    uint32_t key = 0xffffffffu;
    if (t < M) {
      tokens.load<1>(&key, t, 0, n);
      all[t] = t < n ? key : 0xffffffffu;  // the places behind the last count for none
    }
    __syncthreads();
    if (t < n) {
      int rank = 0;
      for (int j = 0; j < (int)n; j += 4) {
        const u32x4 v = *reinterpret_cast<const u32x4*>(&all[j]);
#pragma unroll
        for (int q = 0; q < 4; ++q) rank += v[q] < key || (v[q] == key && j + q < t);
      }
      skey[rank] = key;
      spos[rank] = t;
    }
    __syncthreads();
  }
  for (int64_t item = blockIdx.x; item < chunks * coltiles; item += gridDim.x) {
    const int64_t ch = quot(item, coltiles);
    const uint32_t c = ((uint32_t)(item - ch * coltiles) * 64 + lane) * VEC;
    const int64_t e0 = (ch * kWaves + wave) * K;
    // lane i holds entry e0 - 1 + i; what lies outside the list matches no key
    uint32_t kk = 0xffffffffu, pp = 0;
    {
      const int64_t e = e0 - 1 + lane;
      if (lane < K + 2 && e >= 0 && e < n) {
        kk = SORT ? skey[e] : keys[e];
        pp = SORT ? spos[e] : pos[e];
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
        const int at = u0 + u < cnt ? u0 + u : cnt - 1;  // clamped: the last one again
        const int64_t row = (uint32_t)__builtin_amdgcn_readlane((int)pp, at + 1);
        load_cols<T, VEC, NT>(v[u], dout + row * dout_ld, c, dim);
        if (!FIRST) {
          if (key_at(at + 1) != key_at(at)) load_cols<Gt, VEC>(old[u], grad + (int64_t)key_at(at) * grad_ld, c, dim);
          else old[u].clear();
        }
      }
      if (ragged(dim, VEC)) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int at = u0 + u < cnt ? u0 + u : cnt - 1;
          const int64_t row = (uint32_t)__builtin_amdgcn_readlane((int)pp, at + 1);
          settle_cols<T, VEC>(v[u], dout + row * dout_ld, c, dim);
          if (!FIRST && key_at(at + 1) != key_at(at))
            settle_cols<Gt, VEC>(old[u], grad + (int64_t)key_at(at) * grad_ld, c, dim);
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
        if (c < pitch) store_piece<float, VEC>(partials + (2 * ch + 1) * (int64_t)pitch + c, acc);
      } else {
        Piece<Gt, VEC> old;
        Gt* row = grad + (int64_t)key_at(K - 1) * grad_ld;
        if (!FIRST) take_cols<Gt, VEC>(old, row, c, dim);
        put_grad<Gt, VEC>(row, acc, scale, !FIRST, old, c, dim);
      }
    }
    if (wave == 0 && began) {  // one that comes from the chunk before
#pragma unroll
      for (int e = 0; e < VEC; ++e) acc[e] = 0.0f;
      follow(0);
      if (c < pitch) store_piece<float, VEC>(partials + 2 * ch * (int64_t)pitch + c, acc);
    }
    __syncthreads();
  }
}

// Adds the partial sums at rows 2b, 2(b + 1), ... (count of them) in order.
template <int VEC>
__device__ __forceinline__ void add_partials(float* sum, const float* __restrict__ partials, uint32_t pitch, int64_t b,
                                             int count, uint32_t c, bool live) {
  constexpr int U = 8;  // on their way at once
  for (int i = 0; i < count; i += U) {
    Piece<float, VEC> q[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i + u < count && live) q[u].load(partials + 2 * (b + i + u) * (int64_t)pitch + c);
      else q[u].clear();
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int e = 0; e < VEC; ++e) sum[e] += q[u].get(e);
  }
}

// With many chunks, a run over very many of them (one token in a large part of a
// large batch) would leave its join one long chain: first, a wave for each 64
// chunks (64 g and on) and 64 pieces of columns adds up their partial sums where
// all of them belong to a run from before, into the first one's place. (131072
// tokens of one kind, 1024 wide: 103 us instead of 166; all different: 137.7
// and 137.3. Up to kFoldChunks chunks the chain is no longer than the launch.)
constexpr int kFold = 64;
constexpr int64_t kFoldChunks = 256;
template <int VEC>
__global__ __launch_bounds__(kThreads)
void k_embed_fold(const uint32_t* __restrict__ keys, uint32_t vocab, int chunk, int64_t groups, int64_t coltiles,
                  float* __restrict__ partials, uint32_t pitch) {
  const int lane = threadIdx.x & 63;
  for (int64_t wv = wave_id(); wv < groups * coltiles; wv += (int64_t)gridDim.x * (kThreads / 64)) {
    const int64_t g = quot(wv, coltiles), b = g * kFold;
    const uint32_t c = ((uint32_t)(wv - g * coltiles) * 64 + lane) * VEC;
    const uint32_t key = keys[b * chunk];
    if (key == vocab || b == 0 || keys[b * chunk - 1] != key) continue;
    if (~__ballot(keys[(b + lane) * chunk] == key)) continue;
    float sum[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) sum[e] = 0.0f;
    add_partials<VEC>(sum, partials, pitch, b, kFold, c, c < pitch);
    if (c < pitch) store_piece<float, VEC>(partials + 2 * b * (int64_t)pitch + c, sum);
  }
}

// One wave per chunk and 64 pieces of columns: a run that starts in this chunk
// and goes on in later ones. `groups`: groups of kFold chunks that k_embed_fold
// has been over.
template <typename Gt, int VEC>
__global__ __launch_bounds__(kThreads)
void k_embed_join(const uint32_t* __restrict__ keys, int64_t n, uint32_t vocab, int chunk, int64_t chunks,
                  int64_t groups, int64_t coltiles, uint32_t dim, float scale, Gt* __restrict__ grad, int64_t grad_ld,
                  int first, const float* __restrict__ partials, uint32_t pitch) {
  const int lane = threadIdx.x & 63;
  for (int64_t wv = wave_id(); wv < chunks * coltiles; wv += (int64_t)gridDim.x * (kThreads / 64)) {
    const int64_t ch = quot(wv, coltiles);
    const uint32_t c = ((uint32_t)(wv - ch * coltiles) * 64 + lane) * VEC;
    const int64_t e1 = (ch + 1) * chunk;
    if (e1 >= n) continue;
    const uint32_t key = keys[e1 - 1], behind = keys[e1], ahead = ch > 0 ? keys[ch * chunk - 1] : 0xffffffffu;
    if (key == vocab || behind != key || ahead == key) continue;  // no run starts here and goes on
    const bool live = c < pitch;
    Gt* row = grad + (int64_t)key * grad_ld;
    Piece<Gt, VEC> old;
    if (!first) take_cols<Gt, VEC>(old, row, c, dim);
    Piece<float, VEC> p;
    if (live) p.load(partials + (2 * ch + 1) * (int64_t)pitch + c);
    else p.clear();
    float sum[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) sum[e] = p.get(e);
    for (int64_t b = ch + 1; b < chunks;) {
      // the chunks up to the next group's start that begin with this key
      const int64_t group = b / kFold, end = (group + 1) * kFold < chunks ? (group + 1) * kFold : chunks;
      const uint64_t m = __ballot(b + lane < end && keys[(b + lane < end ? b + lane : b) * chunk] == key);
      const int more = ~m ? __builtin_ctzll(~m) : 64;
      add_partials<VEC>(sum, partials, pitch, b, more == kFold && group < groups ? 1 : more, c, live);
      if (b + more < end) break;
      b = end;
    }
    put_grad<Gt, VEC>(row, sum, scale, !first, old, c, dim);
  }
}

// Elements of a lane's piece: 16 bytes of what is written, so that a wave's
// store covers whole lines. (16384 rows of 4096 bf16 into fp32, 8 elements a
// lane: two stores with gaps took 71 us, 99 past the caches; 4: 50.)
template <typename O>
constexpr int vec_of() { return 16 / sizeof(O); }

template <typename T, typename O>
void run_embed_fwd(const T* table, int64_t vocab, int64_t dim, int64_t table_ld, const T* pos_table, int64_t pos_rows,
                   int64_t pos_ld, const void* tokens, const void* positions, int index_type, int64_t n, float scale,
                   O* out, int64_t out_ld, hipStream_t s) {
  constexpr int VEC = vec_of<O>();
  auto go = [&](auto uu) {
    constexpr int U = decltype(uu)::value;
    const int64_t tiles = (dim + 64 * U * VEC - 1) / (64 * U * VEC), total = n * tiles;
    hipLaunchKernelGGL((k_embed_fwd<T, O, VEC, U>), dim3((unsigned)grid_for(total, kThreads / 64)), dim3(kThreads), 0,
                       s, table, vocab, (uint32_t)dim, table_ld, pos_table, pos_rows, pos_ld, tokens, positions,
                       index_type, total, tiles, scale, out, out_ld);
  };
  // Two pieces a lane: 65 us for 16384 rows of 8192 bf16 (one: 80, four: 70).
  if (dim <= 64 * VEC) go(std::integral_constant<int, 1>{});
  else go(std::integral_constant<int, 2>{});
}

template <typename T, typename Gt>
void run_embed_bwd(const EmbedPlan& p, const Keys& tokens, uint32_t* const* keys, uint32_t* const* pos,
                   uint32_t* counts, uint32_t* totals, uint8_t* touched, float* partials, const T* dout,
                   int64_t dout_ld, int64_t n, int64_t vocab, int64_t dim, float scale, Gt* grad, int64_t grad_ld, bool first, hipStream_t s) {
  constexpr int VEC = vec_of<Gt>();
  int last = 0;
  // What is left to a launch of its own goes by marks of the rows that tokens
  // select, which the first pass clears and the last one sets.
  Fill<Gt> fill = fill_plan(grad, vocab, dim, grad_ld);
  const int64_t pieces = first ? fill.end : 0;
  const bool few = n <= kFewTokens;
  const bool together = first && !few && n <= kPassSort && vocab * dim * (int64_t)sizeof(Gt) <= kFillTogether;
  uint8_t* mark = first && !few && !together ? touched : nullptr;
  const int passes = mark && p.passes < 2 ? 2 : p.passes;
  const bool wide = p.digit > kBits;
  fill.end = 0;
  // The next pieces beside a launch of the sort, a workgroup for every kPassWaves.
  auto beside = [&](int64_t count) {
    fill.begin = fill.end;
    fill.end = fill.begin + count < pieces ? fill.begin + count : pieces;
    return (fill.end - fill.begin + kPassWaves - 1) / kPassWaves;
  };
  if (few) {
    // sorted where they are used
  } else if (by_ranges(n, vocab) && !mark) {
    int bits = 3;  // of a range's keys
    while (bits < kRangeBits && (vocab - 1) >> bits >= kRanges) ++bits;
    const int ranges = (int)(((vocab - 1) >> bits) + 1);
    const int64_t fills = beside(pieces);
    auto sort = [&](auto r) {
      hipLaunchKernelGGL((k_sort_ranges<Gt, decltype(r)::value>), dim3((unsigned)(ranges + fills)), dim3(kPassBS), 0, s,
                         tokens, (int)n, bits, ranges, keys[0], pos[0], fill);
    };
    if (n <= 2 * kPassBS) sort(std::integral_constant<int, 2>{});
    else if (n <= 8 * kPassBS) sort(std::integral_constant<int, 8>{});
    else sort(std::integral_constant<int, kRangeSort / kPassBS>{});
  } else {
    for (int i = 0; i < passes; ++i) {
      const int src = (i + 1) & 1, dst = i & 1;
      Keys k = tokens;
      if (i) k.keys = keys[src];
      const uint32_t* pos_in = i ? pos[src] : nullptr;
      const bool final = i + 1 == passes;
      if (n <= kPassSort) {
        const int tiles = (int)((n + kPassBS - 1) / kPassBS);
        const int clears = i == 0 && mark ? (int)((vocab + kClearBytes - 1) / kClearBytes) : 0;
        const int64_t fills = beside(together ? pieces : kFillBeside / kFillBytes);
        auto pass = [&](auto kernel) {
          hipLaunchKernelGGL(kernel, dim3((unsigned)(tiles + clears + fills)), dim3(kPassBS), 0, s, k, pos_in, (int)n,
                             i * p.digit, p.digit, tiles, clears, (int)final, keys[dst], pos[dst], mark, fill);
        };
        if (wide) pass(k_sort_pass<Gt, kWideBits>);
        else pass(k_sort_pass<Gt, kBits>);
      } else {
        const dim3 gd((unsigned)grid_for(p.tiles, 1)), bd(kThreads);
        hipLaunchKernelGGL(k_sort_count, gd, bd, 0, s, k, n, i * kBits, p.tiles, counts, i == 0 ? mark : nullptr);
        hipLaunchKernelGGL(k_sort_scan, dim3(kBins), bd, 0, s, counts, p.tiles, totals);
        hipLaunchKernelGGL(k_sort_scatter, gd, bd, 0, s, k, pos_in, n, i * kBits, p.tiles, counts, totals, keys[dst],
                           pos[dst], final ? mark : nullptr);
      }
      last = dst;
    }
  }
  if (fill.end < pieces) {
    fill.begin = fill.end;
    fill.end = pieces;
    hipLaunchKernelGGL((k_embed_fill<Gt>), dim3((unsigned)grid_for(fill.end - fill.begin, 1, 64)), dim3(64), 0, s,
                       fill, mark);
  }
  if (n == 0) return;
  const int64_t coltiles = (dim + 64 * VEC - 1) / (64 * VEC), items = p.chunks * coltiles;
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)grid_for(items, 1, kWaves * 64)), dim3(kWaves * 64), 0, s, tokens,
                       keys[last], pos[last], n, (uint32_t)vocab, p.chunks, coltiles, dout, dout_ld, (uint32_t)dim,
                       scale, grad, grad_ld, partials, (uint32_t)p.pitch);
  };
  auto pick = [&](auto f) {
    constexpr bool F = decltype(f)::value;
    if (few) {
      if (p.chunk == 4 * kWaves) go(k_embed_chunks<T, Gt, VEC, 4, F, false, true>);
      else go(k_embed_chunks<T, Gt, VEC, 8, F, false, true>);
    } else if (p.chunk == 4 * kWaves) {
      go(k_embed_chunks<T, Gt, VEC, 4, F, false, false>);
    } else if (p.chunk == 8 * kWaves) {
      go(k_embed_chunks<T, Gt, VEC, 8, F, false, false>);
    } else if (n * dim * (int64_t)sizeof(T) <= kStreamBytes) {
      go(k_embed_chunks<T, Gt, VEC, 16, F, false, false>);
    } else {
      go(k_embed_chunks<T, Gt, VEC, 16, F, true, false>);
    }
  };
  if (first) pick(std::true_type{});
  else pick(std::false_type{});
  const int64_t groups = p.chunks > kFoldChunks ? p.chunks / kFold : 0;
  if (groups > 0)
    hipLaunchKernelGGL((k_embed_fold<VEC>), dim3((unsigned)grid_for(groups * coltiles, kThreads / 64)), dim3(kThreads),
                       0, s, keys[last], (uint32_t)vocab, p.chunk, groups, coltiles, partials, (uint32_t)p.pitch);
  if (p.chunks > 1)
    hipLaunchKernelGGL((k_embed_join<Gt, VEC>), dim3((unsigned)grid_for(items, kThreads / 64)), dim3(kThreads), 0, s,
                       keys[last], n, (uint32_t)vocab, p.chunk, p.chunks, groups, coltiles, (uint32_t)dim, scale,
                       grad, grad_ld, (int)first, partials, (uint32_t)p.pitch);
}

}  // namespace

EmbedPlan embed_plan(int64_t n, int64_t vocab, int64_t dim) {
  EmbedPlan p;
  p.pitch = (dim + 7) / 8 * 8;
  const int64_t coltiles = (dim + 511) / 512;
  int k = 4;  // entries per wave
  while (k < 16 && (n / k * coltiles > kChunkWaves || (n <= kFewTokens && n > k * kWaves))) k *= 2;
  p.chunk = k * kWaves;
  p.chunks = (n + p.chunk - 1) / p.chunk;
  p.bits = 1;  // keys are 0 .. vocab
  while (p.bits < 32 && (vocab >> p.bits) != 0) ++p.bits;
  p.passes = (p.bits + kBits - 1) / kBits;
  p.digit = kBits;
  if (n <= kPassSort) {
    const int fewer = (p.bits + kWideBits - 1) / kWideBits;
    if (fewer < p.passes) p.passes = fewer;
    p.digit = (p.bits + p.passes - 1) / p.passes;
  }
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
  p.touched = take(vocab);
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
  uint8_t* touched = reinterpret_cast<uint8_t*>(ws + p.touched);
  float* partials = reinterpret_cast<float*>(ws + p.partials);
  const Keys k{tokens, nullptr, index_type, vocab, padding_idx};
  auto go = [&](auto* t, auto* g) {
    run_embed_bwd(p, k, keys, pos, counts, totals, touched, partials,
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
