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

// Radix sort of (key, position) by digits of at most kMaxBits bits, lowest
// first, each pass stable. The key of a token that gets no gradient (outside
// of the vocabulary, or the padding token) is `vocab`, behind all others.
constexpr int kMaxBits = 9;
constexpr int kBins = 1 << kMaxBits;
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
void k_sort_count(Keys k, int64_t n, int shift, int bits, int64_t tiles, uint32_t* __restrict__ counts) {
  __shared__ uint32_t h[kBins];
  const int bins = 1 << bits;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    for (int b = threadIdx.x; b < bins; b += kThreads) h[b] = 0;
    __syncthreads();
    const int64_t i0 = tile * kSortTile;
#pragma unroll
    for (int r = 0; r < kSortRounds; ++r) {
      const int64_t i = i0 + r * kThreads + threadIdx.x;
      if (i < n) atomicAdd(&h[(k.at(i) >> shift) & (bins - 1)], 1u);
    }
    __syncthreads();
    for (int b = threadIdx.x; b < bins; b += kThreads) counts[b * tiles + tile] = h[b];
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
__device__ __forceinline__ uint32_t wave_rank(uint32_t d, int bits, bool live, uint32_t* h) {
  uint64_t same = __ballot(live);
  for (int b = 0; b < bits; ++b) {
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
void k_sort_scatter(Keys k, const uint32_t* __restrict__ pos_in, int64_t n, int shift, int bits, int64_t tiles,
                    const uint32_t* __restrict__ counts, const uint32_t* __restrict__ totals,
                    uint32_t* __restrict__ keys_out, uint32_t* __restrict__ pos_out) {
  constexpr int NW = kThreads / 64;
  __shared__ uint32_t hist[NW][kBins];
  __shared__ uint32_t base[kBins];
  __shared__ uint32_t lds[NW];
  const int bins = 1 << bits;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  static_assert(kBins <= 2 * kThreads, "two digits per thread");
  {
    const int b0 = 2 * threadIdx.x;
    const uint32_t v0 = b0 < bins ? totals[b0] : 0, v1 = b0 + 1 < bins ? totals[b0 + 1] : 0;
    uint32_t all;
    const uint32_t before = block_scan<kThreads>(v0 + v1, lds, &all);
    if (b0 < bins) base[b0] = before;
    if (b0 + 1 < bins) base[b0 + 1] = before + v0;
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
      rank[r] = wave_rank((key[r] >> shift) & (bins - 1), bits, i < n, hist[wave]);
    }
    __syncthreads();
    // where each wave's entries of a digit start
    for (int b = threadIdx.x; b < bins; b += kThreads) {
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
        const uint32_t to = hist[wave][(key[r] >> shift) & (bins - 1)] + rank[r];
        keys_out[to] = key[r];
        pos_out[to] = pos_in ? pos_in[i] : (uint32_t)i;
      }
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------- gradient

template <typename T, typename Gt, int VEC>
__device__ __forceinline__ void put_grad(Gt* row, const float* sum, float scale, int first, int64_t c, int64_t dim) {
  float v[VEC];
  if (first) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] = sum[e] * scale;
  } else {
    Piece<Gt, VEC> old;
    load_cols<Gt, VEC>(old, row, c, dim);
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] = old.get(e) + sum[e] * scale;
  }
  store_cols<Gt, VEC>(row, v, c, dim);
}

// One wave: the entries of one chunk, 64 pieces of columns.
template <typename T, typename Gt, int VEC>
__global__ __launch_bounds__(kThreads)
void k_embed_chunks(const uint32_t* __restrict__ keys, const uint32_t* __restrict__ pos, int64_t n, uint32_t vocab,
                    int chunk, int64_t waves, int64_t coltiles, const T* __restrict__ dout, int64_t dout_ld,
                    int64_t dim, float scale, Gt* __restrict__ grad, int64_t grad_ld, int first,
                    float* __restrict__ partials, int64_t pitch) {
  constexpr int U = 8;
  const int lane = threadIdx.x & 63;
  for (int64_t wv = wave_id(); wv < waves; wv += (int64_t)gridDim.x * (kThreads / 64)) {
    const int64_t ch = quot(wv, coltiles);
    const int64_t c = ((wv - ch * coltiles) * 64 + lane) * VEC;
    const int64_t e0 = ch * chunk, e1 = e0 + chunk < n ? e0 + chunk : n;
    uint32_t cur = keys[e0];
    bool before = ch > 0 && keys[e0 - 1] == cur;  // the run began in an earlier chunk
    float acc[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) acc[e] = 0.0f;
    auto flush = [&](bool goes_on) {
      if (cur == vocab) return;
      if (before || goes_on) {
        if (c < pitch) store_piece<float, VEC>(partials + (2 * ch + (before ? 0 : 1)) * pitch + c, acc);
      } else {
        put_grad<T, Gt, VEC>(grad + (int64_t)cur * grad_ld, acc, scale, first, c, dim);
      }
    };
    for (int64_t e = e0; e < e1; e += U) {
      if (keys[e] == vocab) break;  // only entries without a gradient follow
      uint32_t key[U];
      Piece<T, VEC> v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t at = e + u < e1 ? e + u : e1 - 1;  // clamped: loads stay in bounds
        key[u] = keys[at];
        load_cols<T, VEC>(v[u], dout + (int64_t)pos[at] * dout_ld, c, dim);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (e + u >= e1) break;
        if (key[u] != cur) {
          flush(false);
          cur = key[u];
          before = false;
#pragma unroll
          for (int k = 0; k < VEC; ++k) acc[k] = 0.0f;
        }
#pragma unroll
        for (int k = 0; k < VEC; ++k) acc[k] += v[u].get(k);
      }
    }
    flush(e1 < n && keys[e1] == cur);
  }
}

// One wave per chunk and 64 pieces of columns: a run that starts in this chunk
// and goes on in later ones.
template <typename T, typename Gt, int VEC>
__global__ __launch_bounds__(kThreads)
void k_embed_join(const uint32_t* __restrict__ keys, int64_t n, uint32_t vocab, int chunk, int64_t chunks,
                  int64_t waves, int64_t coltiles, int64_t dim, float scale, Gt* __restrict__ grad, int64_t grad_ld,
                  int first, const float* __restrict__ partials, int64_t pitch) {
  const int lane = threadIdx.x & 63;
  for (int64_t wv = wave_id(); wv < waves; wv += (int64_t)gridDim.x * (kThreads / 64)) {
    const int64_t ch = quot(wv, coltiles);
    const int64_t c = ((wv - ch * coltiles) * 64 + lane) * VEC;
    const int64_t e1 = (ch + 1) * chunk;
    if (e1 >= n) continue;
    const uint32_t key = keys[e1 - 1];
    if (key == vocab || keys[e1] != key) continue;             // no run leaves this chunk
    if (ch > 0 && keys[ch * chunk - 1] == key) continue;       // it began earlier
    Piece<float, VEC> p;
    if (c >= pitch) continue;
    p.load(partials + (2 * ch + 1) * pitch + c);
    float sum[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) sum[e] = p.get(e);
    for (int64_t b = ch + 1; b < chunks && keys[b * chunk] == key; ++b) {
      p.load(partials + 2 * b * pitch + c);
#pragma unroll
      for (int e = 0; e < VEC; ++e) sum[e] += p.get(e);
    }
    put_grad<T, Gt, VEC>(grad + (int64_t)key * grad_ld, sum, scale, first, c, dim);
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
void run_embed_bwd(const EmbedPlan& p, const uint32_t* keys, const uint32_t* pos, float* partials, const T* dout,
                   int64_t dout_ld, int64_t n, int64_t vocab, int64_t dim, float scale, Gt* grad, int64_t grad_ld,
                   bool first, hipStream_t s) {
  constexpr int VEC = vec_of<T, Gt>();
  if (first && vocab > 0) {
    int R = 1;
    while (R < 64 && vocab / (2 * R) >= 2048) R *= 2;
    const int64_t groups = (vocab + R - 1) / R;
    hipLaunchKernelGGL((k_embed_fill<Gt, VEC>), dim3((unsigned)grid_for(groups, 1)), dim3(kThreads), 0, s, keys, n,
                       vocab, R, groups, dim, grad, grad_ld);
  }
  if (n == 0) return;
  const int64_t coltiles = (dim + 64 * VEC - 1) / (64 * VEC), waves = p.chunks * coltiles;
  const dim3 gd((unsigned)grid_for(waves, kThreads / 64)), bd(kThreads);
  hipLaunchKernelGGL((k_embed_chunks<T, Gt, VEC>), gd, bd, 0, s, keys, pos, n, (uint32_t)vocab, p.chunk, waves,
                     coltiles, dout, dout_ld, dim, scale, grad, grad_ld, (int)first, partials, p.pitch);
  if (p.chunks > 1)
    hipLaunchKernelGGL((k_embed_join<T, Gt, VEC>), gd, bd, 0, s, keys, n, (uint32_t)vocab, p.chunk, p.chunks, waves,
                       coltiles, dim, scale, grad, grad_ld, (int)first, partials, p.pitch);
}

}  // namespace

EmbedPlan embed_plan(int64_t n, int64_t vocab, int64_t dim) {
  EmbedPlan p;
  p.pitch = (dim + 7) / 8 * 8;
  const int64_t coltiles = (dim + 511) / 512;
  p.chunk = 8;
  while (p.chunk < 128 && n / p.chunk * coltiles > 8192) p.chunk *= 2;
  p.chunks = (n + p.chunk - 1) / p.chunk;
  p.bits = 1;  // keys are 0 .. vocab
  while (p.bits < 32 && (vocab >> p.bits) != 0) ++p.bits;
  p.passes = (p.bits + kMaxBits - 1) / kMaxBits;
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
  int last = 0;
  if (n > 0) {
    const int step = (p.bits + p.passes - 1) / p.passes;
    const dim3 gd((unsigned)grid_for(p.tiles, 1)), bd(kThreads);
    for (int i = 0; i < p.passes; ++i) {
      const int shift = i * step, bits = p.bits - shift < step ? p.bits - shift : step;
      const int src = (i + 1) & 1, dst = i & 1;
      const Keys k{tokens, i ? keys[src] : nullptr, index_type, vocab, padding_idx};
      hipLaunchKernelGGL(k_sort_count, gd, bd, 0, s, k, n, shift, bits, p.tiles, counts);
      hipLaunchKernelGGL(k_sort_scan, dim3(1u << bits), bd, 0, s, counts, p.tiles, totals);
      hipLaunchKernelGGL(k_sort_scatter, gd, bd, 0, s, k, i ? pos[src] : nullptr, n, shift, bits, p.tiles, counts,
                         totals, keys[dst], pos[dst]);
      last = dst;
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  float* partials = reinterpret_cast<float*>(ws + p.partials);
  auto go = [&](auto* t, auto* g) {
    run_embed_bwd(p, keys[last], pos[last], partials, static_cast<const std::remove_pointer_t<decltype(t)>*>(dout),
                  dout_ld, n, vocab, dim, scale, static_cast<decltype(g)>(grad), grad_ld, first, s);
  };
  uint16_t* h = nullptr;
  float* f = nullptr;
  if (dtype == ZS_BF16) grad_dtype == ZS_BF16 ? go(h, h) : go(h, f);
  else grad_dtype == ZS_BF16 ? go(f, h) : go(f, f);
  return hipGetLastError();
}

}  // namespace zs
