// Values in 8 bits: e4m3 codes (sign, 4 bits of exponent, 3 of mantissa; the
// largest finite value is 448, there is no infinity) and an fp32 scale for each
// block of 128 consecutive elements of a row. A value is code * scale.
//
// The scale is the smallest power of two, 2^-117 at least, with which the block's
// largest finite magnitude stays within 448; 1 where all are zero. A power of two
// costs no precision, as e4m3 has an exponent of its own, and both the division
// by it and the product with it are exact: packing rounds once, and what is
// unpacked is exact in bf16 too. Infinities and NaN become NaN.
#pragma once

#include "zs_rows.hpp"

namespace zs {

constexpr uint32_t kScaleBlock = 128;

// Largest value over each aligned group of G lanes, in all of them.
template <int G>
__device__ __forceinline__ float lane_max(float x) {
  static_assert(G == 16 || G == 32, "16 lanes or half of the wave");
  auto dpp = [](float v, auto ctrl) {
    return __uint_as_float(__builtin_amdgcn_update_dpp(0u, __float_as_uint(v), decltype(ctrl)::value, 0xf, 0xf, true));
  };
  x = fmaxf(x, dpp(x, std::integral_constant<int, 0xb1>{}));   // lane ^ 1
  x = fmaxf(x, dpp(x, std::integral_constant<int, 0x4e>{}));   // lane ^ 2
  x = fmaxf(x, dpp(x, std::integral_constant<int, 0x141>{}));  // mirrored within 8
  x = fmaxf(x, dpp(x, std::integral_constant<int, 0x140>{}));  // mirrored within 16
  if constexpr (G == 32) {
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  }
  return x;
}

// VEC codes of a row.
template <int VEC>
struct Codes {
  static_assert(VEC == 4 || VEC == 8, "4 or 8 codes");
  static constexpr int N = VEC / 4;
  uint32_t r[N];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < N; ++i) r[i] = 0u;
  }
  __device__ __forceinline__ float get(int e) const {  // e is a constant after unrolling
    const int w = (int)r[e / 4];
    switch (e & 3) {
      case 0: return __builtin_amdgcn_cvt_f32_fp8(w, 0);
      case 1: return __builtin_amdgcn_cvt_f32_fp8(w, 1);
      case 2: return __builtin_amdgcn_cvt_f32_fp8(w, 2);
      default: return __builtin_amdgcn_cvt_f32_fp8(w, 3);
    }
  }
};

typedef uint32_t u32_any __attribute__((aligned(1)));
typedef u32x2 u32x2_bytes __attribute__((aligned(1)));

// The codes of a row at column c, those at or past dim zero (as load_cols and
// settle_cols: the lane that the row ends in takes the row's last VEC codes and
// moves them where they are used).
template <int VEC, bool NT = false>
__device__ __forceinline__ void load_codes(Codes<VEC>& p, const uint8_t* row, uint32_t c, uint32_t dim) {
  p.clear();
#pragma unroll
  for (int i = 0; i < Codes<VEC>::N; ++i) asm volatile("" : "+v"(p.r[i]));
  const uint32_t end = dim >= VEC ? dim : 0, last = dim - VEC;
  if (c < end) {
    const uint8_t* from = row + (c < last ? c : last);
    if constexpr (VEC == 8) {
      const auto q = (const __attribute__((address_space(1))) u32x2_bytes*)from;
      const u32x2 v = NT ? __builtin_nontemporal_load(q) : *q;
      p.r[0] = v.x;
      p.r[1] = v.y;
    } else {
      const auto q = (const __attribute__((address_space(1))) u32_any*)from;
      p.r[0] = NT ? __builtin_nontemporal_load(q) : *q;
    }
  }
}
template <int VEC>
__device__ __forceinline__ void settle_codes(Codes<VEC>& p, const uint8_t* row, uint32_t c, uint32_t dim) {
  if (dim < VEC) {
    if (c == 0)
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        if (e < (int)dim) p.r[e / 4] |= (uint32_t)ld_g(row + e) << (8 * (e & 3));
  } else if (c < dim && c + VEC > dim) {
    for (uint32_t n = c + VEC - dim; n > 0; --n)
#pragma unroll
      for (int i = 0; i < Codes<VEC>::N; ++i)
        p.r[i] = (p.r[i] >> 8) | (i + 1 < Codes<VEC>::N ? p.r[i + 1] << 24 : 0u);
  }
}
template <int VEC>
__device__ __forceinline__ void take_codes(Codes<VEC>& p, const uint8_t* row, uint32_t c, uint32_t dim) {
  load_codes<VEC>(p, row, c, dim);
  if (ragged(dim, VEC)) settle_codes<VEC>(p, row, c, dim);
}

// Codes of VEC values v of a row at column c, of which those at or past dim are
// zero, and their block's scale. The block's G lanes come together.
template <int VEC, int G, bool NT = false>
__device__ __forceinline__ void store_codes(uint8_t* row, float* scales, const float* values, uint32_t c, uint32_t dim) {
  float v[VEC], top = 0.0f;
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    v[e] = values[e];
    top = fmaxf(top, fabsf(v[e]));  // fmaxf passes over NaN
  }
  top = lane_max<G>(top);
  // Infinities are no measure of the others and have no code; a finite value above
  // 240 * 2^120 would be rounded to 2^128.
  constexpr float MOST = 0x1.ep127f;
  if (top > MOST) {
    float finite = 0.0f;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      if (fabsf(v[e]) == INFINITY) v[e] = NAN;
      else if (fabsf(v[e]) > MOST) v[e] = copysignf(MOST, v[e]);
      finite = fmaxf(finite, fabsf(v[e]));
    }
    top = lane_max<G>(finite);
  }
  const uint32_t u = __float_as_uint(top);
  int k = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);  // 448 = 1.75 * 2^8
  k = top == 0.0f ? 0 : k < -117 ? -117 : k;
  const float inverse = __uint_as_float((uint32_t)(127 - k) << 23);
  if (c >= dim) return;
  if (c % kScaleBlock == 0) scales[c / kScaleBlock] = __uint_as_float((uint32_t)(127 + k) << 23);
  uint32_t r[VEC / 4];
#pragma unroll
  for (int i = 0; i < VEC / 4; ++i) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i] * inverse, v[4 * i + 1] * inverse, 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i + 2] * inverse, v[4 * i + 3] * inverse, w, true);
    r[i] = (uint32_t)w;
  }
  if (c + VEC <= dim) {
    if constexpr (VEC == 8) {
      const auto q = (__attribute__((address_space(1))) u32x2_bytes*)(row + c);
      if (NT) __builtin_nontemporal_store(u32x2{r[0], r[1]}, q);
      else *q = u32x2{r[0], r[1]};
    } else {
      const auto q = (__attribute__((address_space(1))) u32_any*)(row + c);
      if (NT) __builtin_nontemporal_store(r[0], q);
      else *q = r[0];
    }
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e)
      if (c + e < dim) st_g((uint8_t)(r[e / 4] >> (8 * (e & 3))), row + c + e);
  }
}

}  // namespace zs
