// Row access and wave sums shared by the embedding and layer norm kernels.
//
// A row is `dim` consecutive elements at any element-aligned address: odd
// widths and row strides put rows off the 16-byte grid. gfx950 reads and
// writes 16 bytes at any address in one instruction, so a lane's unit of work
// is VEC consecutive elements wherever they start, and only the last, shorter
// piece of a row goes element by element.
#pragma once

#include "zs_device.hpp"

namespace zs {

typedef u32x4 u32x4_any __attribute__((aligned(2)));  // 16 bytes at a 2-byte aligned address
typedef u32x2 u32x2_any __attribute__((aligned(2)));

// 16 bytes at any element-aligned address of global memory. (Not through ld_g:
// a template parameter would drop the typedef's alignment.)
__device__ __forceinline__ u32x4 ld16(const void* p) {
  return *(const __attribute__((address_space(1))) u32x4_any*)p;
}
__device__ __forceinline__ void st16(u32x4 v, void* p) {
  *(__attribute__((address_space(1))) u32x4_any*)p = v;
}
// the same for memory that is touched once
__device__ __forceinline__ u32x4 ld16_nt(const void* p) {
  return __builtin_nontemporal_load((const __attribute__((address_space(1))) u32x4_any*)p);
}
__device__ __forceinline__ void st16_nt(u32x4 v, void* p) {
  __builtin_nontemporal_store(v, (__attribute__((address_space(1))) u32x4_any*)p);
}

// VEC consecutive elements of a row as they lie in memory: 8 bytes, or whole
// 16-byte vectors.
template <typename T, int VEC>
struct Piece {
  static constexpr int B = VEC * (int)sizeof(T);
  static constexpr int N = B / 4;
  static_assert(B == 8 || B % 16 == 0, "an access of 8 or 16 bytes");
  uint32_t r[N];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < N; ++i) r[i] = 0u;
  }
  template <bool NT = false>
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (B == 8) {
      const auto q = (const __attribute__((address_space(1))) u32x2_any*)p;
      const u32x2 v = NT ? __builtin_nontemporal_load(q) : *q;
      r[0] = v.x;
      r[1] = v.y;
    } else {
#pragma unroll
      for (int i = 0; i < N / 4; ++i) {
        const T* q = p + i * (16 / (int)sizeof(T));
        const u32x4 v = NT ? ld16_nt(q) : ld16(q);
        r[4 * i] = v.x;
        r[4 * i + 1] = v.y;
        r[4 * i + 2] = v.z;
        r[4 * i + 3] = v.w;
      }
    }
  }
  // the first n (below VEC) elements, zeros behind them
  __device__ __forceinline__ void load_part(const T* p, int n) {
    clear();
#pragma unroll
    for (int e = 0; e < VEC; ++e)
      if (e < n) put(e, ld_g(p + e));
  }
  // Keeps the piece as it lies in memory from here on: without it the compiler
  // widens values that a loop only reads before the loop and holds them in
  // twice the registers.
  __device__ __forceinline__ void stay_packed() {
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        uint32_t w = r[i];
        asm volatile("" : "+v"(w));
        r[i] = w;
      }
    }
  }
  // every element one place down, a zero behind the last
  __device__ __forceinline__ void drop_first() {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint32_t up = i + 1 < N ? r[i + 1] : 0u;
      r[i] = sizeof(T) == 4 ? up : (r[i] >> 16) | (up << 16);
    }
  }
  __device__ __forceinline__ void put(int e, float x) { r[e] = __float_as_uint(x); }
  __device__ __forceinline__ void put(int e, uint16_t h) { r[e / 2] |= (uint32_t)h << (16 * (e & 1)); }
  __device__ __forceinline__ float get(int e) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(r[e]);
    else return (e & 1) ? bf16_hi(r[e / 2]) : bf16_lo(r[e / 2]);
  }
};

// fp32 -> bf16 by the hardware's conversion (round to nearest even, NaN stays a
// quiet NaN): one instruction for two values, where the integer form takes
// about eleven, which the layer norm kernels, near their VALU bound for bf16
// rows, would feel.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
}

// One value rounded to the row's type.
template <typename T>
__device__ __forceinline__ T round_to(float x) {
  if constexpr (sizeof(T) == 4) return x;
  else return (T)pack_bf16(x, x);
}

// VEC fp32 values stored as a row's elements, each rounded once.
template <typename T, int VEC, bool NT = false>
__device__ __forceinline__ void store_piece(T* p, const float* v) {
  auto st = [](u32x4 x, void* q) {
    if constexpr (NT) st16_nt(x, q);
    else st16(x, q);
  };
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i)
      st(u32x4{__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]), __float_as_uint(v[4 * i + 2]),
                 __float_as_uint(v[4 * i + 3])}, p + 4 * i);
  } else {
#pragma unroll
    for (int i = 0; i < VEC / 8; ++i)
      st(u32x4{pack_bf16(v[8 * i], v[8 * i + 1]), pack_bf16(v[8 * i + 2], v[8 * i + 3]),
                 pack_bf16(v[8 * i + 4], v[8 * i + 5]), pack_bf16(v[8 * i + 6], v[8 * i + 7])}, p + 8 * i);
  }
}
template <typename T, int VEC>
__device__ __forceinline__ void store_part(T* p, const float* v, int n) {
#pragma unroll
  for (int e = 0; e < VEC; ++e)
    if (e < n) st_g(round_to<T>(v[e]), p + e);
}

// The piece of a row at column c; what lies at or past `dim` is zero, or is not
// written. Columns are 32-bit (dim stays below 2^24): with a row's address the
// same for the whole wave, an access then takes it from scalar registers and
// one register of offset, instead of two registers of address for each piece
// that is on its way.
//
// load_cols sends the loads off. The zeros of the lanes behind the row are
// written before the load: written behind it, into the same registers, they
// would have to wait for it, and with them the wave (8192 backward rows of 5376
// bf16, which end in the middle of a wave: 50 us, not 76). Where dim is not a
// multiple of VEC the lane that the row ends in takes the row's last VEC
// elements, and settle_cols, which callers run then where the pieces are
// used, moves them to their places: that has to wait for them (16384 backward
// rows of 4095: 96 us, 163 with its elements loaded one by one).
template <typename T, int VEC, bool NT = false>
__device__ __forceinline__ void load_cols(Piece<T, VEC>& p, const T* row, uint32_t c, uint32_t dim) {
  p.clear();
#pragma unroll
  for (int i = 0; i < Piece<T, VEC>::N; ++i) asm volatile("" : "+v"(p.r[i]));  // now, not behind the load
  const uint32_t end = dim >= VEC ? dim : 0, last = dim - VEC;
  if (c < end) p.template load<NT>(row + (c < last ? c : last));
}
__device__ __forceinline__ bool ragged(uint32_t dim, int vec) { return dim % vec != 0; }
template <typename T, int VEC>
__device__ __forceinline__ void settle_cols(Piece<T, VEC>& p, const T* row, uint32_t c, uint32_t dim) {
  if (dim < VEC) {
    if (c == 0) p.load_part(row, (int)dim);
  } else if (c < dim && c + VEC > dim) {
    for (uint32_t n = c + VEC - dim; n > 0; --n) p.drop_first();
  }
}
// Both, for pieces that are used at once.
template <typename T, int VEC>
__device__ __forceinline__ void take_cols(Piece<T, VEC>& p, const T* row, uint32_t c, uint32_t dim) {
  load_cols<T, VEC>(p, row, c, dim);
  if (ragged(dim, VEC)) settle_cols<T, VEC>(p, row, c, dim);
}
template <typename T, int VEC, bool NT = false>
__device__ __forceinline__ void store_cols(T* row, const float* v, uint32_t c, uint32_t dim) {
  if (c + VEC <= dim) store_piece<T, VEC, NT>(row + c, v);
  else if (c < dim) store_part<T, VEC>(row + c, v, (int)(dim - c));
}

// Sum over the wave's lanes (G = 64) or over each aligned group of G lanes (16, 32),
// the same bits in every lane of the group: pairs of lanes that mirror each
// other are added, so both hold the same sum after each step.
template <int G>
__device__ __forceinline__ float lane_sum(float x) {
  static_assert(G == 16 || G == 32 || G == 64, "16 lanes, half of the wave or the wave");
  auto dpp = [](float v, auto ctrl) {
    return __uint_as_float(__builtin_amdgcn_update_dpp(0u, __float_as_uint(v), decltype(ctrl)::value, 0xf, 0xf, true));
  };
  x += dpp(x, std::integral_constant<int, 0xb1>{});   // lane ^ 1
  x += dpp(x, std::integral_constant<int, 0x4e>{});   // lane ^ 2
  x += dpp(x, std::integral_constant<int, 0x141>{});  // mirrored within 8
  x += dpp(x, std::integral_constant<int, 0x140>{});  // mirrored within 16
  if constexpr (G >= 32) {
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  }
  if constexpr (G == 64) {
    const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(b[0]) + __uint_as_float(b[1]);
  }
  return x;
}

}  // namespace zs
