// bf16 (or fp16) matrix products D[m, n] = sum_k A[m, k] B[n, k] on the matrix units,
// accumulated in fp32; the epilogue that uses D is the caller's.
//
// Either operand lies in memory as rows of consecutive k (K_IN_ROWS: the logits
// are hidden states times rows of the head) or as one row for each k (K_IS_ROW:
// the gradient of the head is a sum over tokens, and a token's row holds
// consecutive columns of the result). Both are copied to LDS as they lie, by
// loads that go there directly; operands with a row for each k are transposed
// on the way from LDS to registers.
//
// An fp32 operand is a sum of up to three bf16 planes that lie side by side in
// each row, and a product of two such operands the sum of the products of their
// planes that matter: Segments lists them, and the loop over k runs through one
// after another into the same accumulators. Scaled by rows, two fp16 planes do too.
#pragma once

#include "zs_device.hpp"

namespace zs {

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

enum GemmMode { K_IN_ROWS, K_IS_ROW };

// One operand. Rows start on 16-byte boundaries, `ld` elements apart, and hold
// planes of `plane` elements. K_IN_ROWS: `rows` rows of the result, at least 64 *
// steps elements to a plane. K_IS_ROW: `rows` values of k, `cols` columns (a
// multiple of 8).
struct GemmSide {
  const uint16_t* p;
  int64_t ld;
  int64_t plane;
  int64_t rows;
  int64_t cols;
};

// Products of planes: nibble i of a and b is product i's plane of either side.
struct Segments {
  int count;
  uint32_t a, b;
};

constexpr int kBK = 64;  // values of k of a stage

template <int BM_, int BN_, int WM_, int WN_>
struct GemmShape {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_;
  static constexpr int THREADS = WM * WN * 64;
  static constexpr int TM = BM / WM / 16, TN = BN / WN / 16;  // 16 x 16 tiles of a wave
  static constexpr int STAGE_BYTES = (BM + BN) * kBK * 2;
  static constexpr int LDS = 2 * STAGE_BYTES;
  using Acc = f32x4[TM][TN];
};

#ifdef __HIP_DEVICE_COMPILE__  // the host's pass does not know the buffer types
// 16 bytes from byte `off` of each lane behind the buffer's start to LDS, lane l's
// to 16 l behind `lds`. Written out, as behind the builtin the compiler waits for
// all loads before the next transposing read (ds_read_b64_tr_b16), which it
// takes to read what they write; the waits are TileLoop's own. M0 holds the LDS
// address, and needs a wait state before it is used; it is the compiler's, which does
// not take it as clobbered, so it gets its value back.
__device__ __forceinline__ void load_to_lds(u32x4 buffer, uint32_t lds, uint32_t off) {
  uint32_t kept;
  asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\tbuffer_load_dwordx4 %2, %3, 0 offen lds\n\ts_mov_b32 m0, %0"
               : "=&s"(kept)
               : "s"(lds), "v"(off), "s"(buffer)
               : "memory");
}

// The part of an operand that one workgroup reads: SIDE rows (or columns) from
// `start` on, 64 values of k at a time.
//
// K_IN_ROWS: a row's 64 values are 128 bytes, row after row in LDS. The chunk of
// 16 bytes c of row r lies at place c ^ (r & 7): 8 lanes that read the same chunk
// of 8 rows find it in 8 different places. A load to LDS puts lane l's 16 bytes
// 16 l behind the wave's start, so what is permuted is where they come from.
//
// K_IS_ROW: SIDE columns of a row, row after row in LDS. The 16 lanes of a
// transposing read take 32 bytes of 4 rows, the wave of 16 rows: the chunk of 32
// bytes c of row r lies at place c ^ swap(r), with another value of swap for each
// of these rows.
template <class S, int SIDE, GemmMode MODE>
struct SideTile {
  static constexpr int N = SIDE * kBK * 2 / 16 / S::THREADS;  // 16-byte loads of a thread for a stage
  static constexpr int T = SIDE / 16;
  static_assert(N * S::THREADS * 16 == SIDE * kBK * 2, "every thread loads as much");
  const uint16_t* base;
  int64_t ld, plane, rows;
  uint32_t off[N];
  int tid, live;

  static __device__ __forceinline__ int swap(int r) { return ((r & 3) | ((r >> 1) & 12)) & (T - 1); }

  // byte offsets of the thread's loads; values of k from `there` on come as the last one's copies
  __device__ __forceinline__ void offsets_k_is_row(int64_t cols, int there) {
    live = there;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int at = i * S::THREADS + tid, r = at / (SIDE / 8), c = at % (SIDE / 8);
      const int col = (((c >> 1) ^ swap(r)) * 2 + (c & 1)) * 8;
      const int last = (int)(cols < SIDE ? cols : SIDE) - 8;  // columns behind the last are copies; nobody uses them
      off[i] = (uint32_t)((r < live ? r : live - 1) * ld * 2) + (col < last ? col : last) * 2;
    }
  }
  __device__ __forceinline__ void init(const GemmSide& g, int64_t start) {
    tid = threadIdx.x;
    ld = g.ld;
    plane = g.plane;
    rows = g.rows;
    if constexpr (MODE == K_IN_ROWS) {
      base = g.p + start * g.ld;
      const int64_t left = g.rows - start;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int at = i * S::THREADS + tid, r = at >> 3, c = (at & 7) ^ (r & 7);
        off[i] = (uint32_t)((r < left ? r : left - 1) * ld * 2) + c * 16;  // rows behind the last are its copies
      }
    } else {
      base = g.p + start;
      offsets_k_is_row(g.cols - start, kBK);
    }
  }
  // where the values of plane p from k on come from
  __device__ __forceinline__ u32x4 source(int p, int64_t k, int64_t cols_left) {
    const uint16_t* from = base + p * plane + (MODE == K_IN_ROWS ? k : k * ld);
    if constexpr (MODE == K_IS_ROW) {
      const int there = k + kBK <= rows ? kBK : (int)(rows - k);
      if (there != live) offsets_k_is_row(cols_left, there);
    }
    const uint64_t at = (uint64_t)from;
    return u32x4{(uint32_t)at, (uint32_t)(at >> 32) & 0xffffu, 0xffffffffu, 0x00020000u};
  }
  // the thread's load i of N
  __device__ __forceinline__ void load(int i, u32x4 from, char* lds) const {
    load_to_lds(from, (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)lds +
                          (uint32_t)__builtin_amdgcn_readfirstlane((i * S::THREADS + (tid & ~63)) * 16), off[i]);
  }
};

// Fragments of 16 rows (columns) x 32 values of k as the 16x16x32 product takes
// them: lane l has row l % 16, values 8 (l / 16) to 8 (l / 16) + 7.
template <int SIDE, GemmMode MODE>
struct Fragments {
  uint32_t at;  // byte address behind the side's stage
  __device__ __forceinline__ void init(int first) {  // first row of the wave, a multiple of its tiles' 16
    const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
    if constexpr (MODE == K_IN_ROWS) {
      at = (uint32_t)((first + r) * 128 + ((q ^ (r & 7)) * 16));
    } else {
      const int row = 8 * q + (r >> 2);
      constexpr int T = SIDE / 16;
      const int sw = ((row & 3) | ((row >> 1) & 12)) & (T - 1);
      at = (uint32_t)(row * SIDE * 2 + (((first / 16) ^ sw) * 32) + (r & 3) * 8);
    }
  }
  // fragment i of the wave, values 32 kk and on of the stage
  __device__ __forceinline__ bf16x8 get(const char* stage, int i, int kk) const {
    if constexpr (MODE == K_IN_ROWS) {
      return *(const bf16x8*)(stage + (at ^ (kk * 64)) + i * 2048);
    } else {
      const char* p = stage + (at ^ (i * 32)) + kk * 32 * SIDE * 2;
      typedef __attribute__((address_space(3))) bf16x4* ptr;
      const bf16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((ptr)(p));
      const bf16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((ptr)(p + 4 * SIDE * 2));
      return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
  }
};

// This wave's reads of LDS are done, and all its loads but the last N.
template <int N>
__device__ __forceinline__ void wait_reads_and_loads_but() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ void barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}
#endif

// The product of one tile: aim(), preload(), run(). Lane l of the wave at (wm, wn)
// gets in acc[i][j][r] row wm BM / WM + 16 i + 4 (l / 16) + r and column
// wn BN / WN + 16 j + l % 16 of the tile.
//
// A workgroup that makes several tiles sends the first loads of the next off
// before it does what it does with the products of this one: a tile of 12
// stages waits as long for its first loads as it takes for some of its stages.
// `run` leaves LDS to the next tile's loads.
//
// Two stages lie in LDS. The fragments of a step are read during the products of
// the step before, so the one barrier of a stage stands before its last step:
// behind it everybody has read this stage, and the next stage but one can come
// into its place while the last step's and the next stage's products are made.
// A 256 x 256 tile on 8 waves: 1250 TFLOP/s for 16384 x 8192 x 4096 in each of
// the three layouts (1030, 890 and 920 with reads, products and a barrier in
// turn), of the 1490 that the same loop reaches without loads. Stages of 32
// values, four or five in LDS: 1130; loads sent off a few with each step: 1210 to
// 1260; 32 x 32 x 16 products: 1190; of zeros, at the full clock: 1370.
template <class S, GemmMode MA, GemmMode MB, bool HALF = false>  // HALF: the operands are fp16
struct TileLoop {
#ifdef __HIP_DEVICE_COMPILE__
  static constexpr int A_BYTES = S::BM * kBK * 2;
  static constexpr int NA = SideTile<S, S::BM, MA>::N, NB = SideTile<S, S::BN, MB>::N;  // a thread's loads for a stage
  SideTile<S, S::BM, MA> la;
  SideTile<S, S::BN, MB> lb;
  int64_t cols_a, cols_b;
  Segments segs;
  int steps, seg, step, n;  // stages of a segment, the next stage to load, stages of the tile

  // At stages [s0, s1) of the `segs.count * steps` that there are, `steps` to a segment.
  __device__ __forceinline__ void aim(const GemmSide& a, const GemmSide& b, int64_t start_a, int64_t start_b,
                                      const Segments& sg, int per_segment, int s0, int s1) {
    la.init(a, start_a);
    lb.init(b, start_b);
    cols_a = a.cols - start_a;
    cols_b = b.cols - start_b;
    segs = sg;
    steps = per_segment;
    n = s1 - s0;
    seg = n > 0 ? s0 / steps : 0;
    step = n > 0 ? s0 % steps : 0;
  }
  __device__ __forceinline__ void load(char* stage) {  // all of the next stage
    const int64_t k = (int64_t)step * kBK;
    const u32x4 from_a = la.source((segs.a >> (4 * seg)) & 15, k, cols_a);
    const u32x4 from_b = lb.source((segs.b >> (4 * seg)) & 15, k, cols_b);
#pragma unroll
    for (int i = 0; i < NA; ++i) la.load(i, from_a, stage);
#pragma unroll
    for (int i = 0; i < NB; ++i) lb.load(i, from_b, stage + A_BYTES);
    if (++step == steps) step = 0, ++seg;
  }
  __device__ __forceinline__ void preload(char* lds) {
    if (n > 0) load(lds);
    if (n > 1) load(lds + S::STAGE_BYTES);
  }
  // acc += the product. `stored`: at least kStored stores were sent off behind
  // preload(); they need not be done.
  static constexpr int kStored = 16;
  __device__ __forceinline__ void run(char* lds, typename S::Acc& acc, bool stored) {
    if (n <= 0) return;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    Fragments<S::BM, MA> ga;
    Fragments<S::BN, MB> gb;
    ga.init(wave / S::WN * (S::BM / S::WM));
    gb.init(wave % S::WN * (S::BN / S::WN));
    // A stage's products in steps of two rows of tiles, STEPS for each half of its
    // values of k. The fragments of a step are read during the step before.
    constexpr int STEPS = S::TM / 2, LAST = 2 * STEPS - 1;
    bf16x8 fa[2][2], fb[2][S::TN];
    auto read = [&](int u, const char* stage) {  // u is a constant after unrolling
      const int kk = u / STEPS, i = u % STEPS * 2;
      if (i == 0)
#pragma unroll
        for (int j = 0; j < S::TN; ++j) fb[kk][j] = gb.get(stage + A_BYTES, j, kk);
      fa[u & 1][0] = ga.get(stage, i, kk);
      fa[u & 1][1] = ga.get(stage, i + 1, kk);
    };
    auto multiply = [&](int u) {
      const int kk = u / STEPS, i = u % STEPS * 2;
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int j = 0; j < S::TN; ++j) {
          if constexpr (HALF)
            acc[i + x][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, fa[u & 1][x]),
                                                                   __builtin_bit_cast(f16x8, fb[kk][j]), acc[i + x][j], 0, 0, 0);
          else
            acc[i + x][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[u & 1][x], fb[kk][j], acc[i + x][j], 0, 0, 0);
        }
    };
    if (n == 1) wait_reads_and_loads_but<0>();
    else if (stored) wait_reads_and_loads_but<NA + NB + kStored>();
    else wait_reads_and_loads_but<NA + NB>();
    barrier();
    read(0, lds);
    for (int s = 0; s < n; ++s) {
      char* now = lds + (s & 1) * S::STAGE_BYTES;
      const char* next = lds + (~s & 1) * S::STAGE_BYTES;
#pragma unroll
      for (int u = 0; u < LAST; ++u) {
        read(u + 1, now);
        __builtin_amdgcn_sched_barrier(0);
        multiply(u);
        __builtin_amdgcn_sched_barrier(0);
      }
      wait_reads_and_loads_but<0>();
      barrier();  // everybody has read this stage, and everybody's loads of the next are done
      if (s + 1 < n) read(0, next);
      __builtin_amdgcn_sched_barrier(0);
      multiply(LAST);
      __builtin_amdgcn_sched_barrier(0);
      if (s + 2 < n) load(now);
    }
  }
#else
  __device__ void aim(const GemmSide&, const GemmSide&, int64_t, int64_t, const Segments&, int, int, int) {}
  __device__ void preload(char*) {}
  __device__ void run(char*, typename S::Acc&, bool) {}
#endif
};

}  // namespace zs
