// Activations in 8 bits: packing rows into e4m3 codes with a scale for each block
// of 128 elements, and back. Bound by memory: packing reads the values and writes
// a byte each, unpacking the reverse. The 16 (bf16) or 32 (fp32) lanes that hold
// a block find its largest magnitude among themselves, so values are read once.
// 16384 rows of 8192 bf16: 71 us each way, 407 MB at 5.7 TB/s.
#include "zs_e4m3.hpp"
#include "zs_launch.hpp"
#include "zs_launch_rows.hpp"
#include "zs_rows.hpp"

namespace zs {
namespace {

// A workgroup takes `1 << shift` lanes to a row: as many as the row's pieces fill,
// 256 at most, which then walk along it, NV pieces at a time.
constexpr int NV = 4;

template <typename T, int VEC, bool NT>
__global__ __launch_bounds__(kThreads)
void k_pack(const T* __restrict__ x, int64_t x_ld, int64_t rows, uint32_t dim, uint8_t* __restrict__ codes,
            int64_t codes_ld, float* __restrict__ scales, int64_t scales_ld, int shift) {
  constexpr int BLOCK = kScaleBlock / VEC;
  const uint32_t lanes = 1u << shift, l = threadIdx.x & (lanes - 1), width = lanes * VEC;
  const int64_t per = kThreads >> shift;
  for (int64_t row = (int64_t)blockIdx.x * per + (threadIdx.x >> shift); row < rows; row += (int64_t)gridDim.x * per) {
    const T* xr = x + row * x_ld;
    for (uint32_t c0 = 0; c0 < dim; c0 += NV * width) {  // the same turns for all lanes of a row
      Piece<T, VEC> p[NV];
#pragma unroll
      for (int j = 0; j < NV; ++j) load_cols<T, VEC, NT>(p[j], xr, c0 + j * width + l * VEC, dim);
      if (ragged(dim, VEC))
#pragma unroll
        for (int j = 0; j < NV; ++j) settle_cols<T, VEC>(p[j], xr, c0 + j * width + l * VEC, dim);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float v[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[e] = p[j].get(e);
        store_codes<VEC, BLOCK, NT>(codes + row * codes_ld, scales + row * scales_ld, v, c0 + j * width + l * VEC, dim);
      }
    }
  }
}

template <typename T, int VEC, bool NT>
__global__ __launch_bounds__(kThreads)
void k_unpack(const uint8_t* __restrict__ codes, int64_t codes_ld, const float* __restrict__ scales, int64_t scales_ld,
              int64_t rows, uint32_t dim, T* __restrict__ out, int64_t out_ld, int shift) {
  const uint32_t lanes = 1u << shift, l = threadIdx.x & (lanes - 1), width = lanes * VEC;
  const int64_t per = kThreads >> shift;
  for (int64_t row = (int64_t)blockIdx.x * per + (threadIdx.x >> shift); row < rows; row += (int64_t)gridDim.x * per) {
    const uint8_t* from = codes + row * codes_ld;
    for (uint32_t c0 = 0; c0 < dim; c0 += NV * width) {
      Codes<VEC> p[NV];
      float scale[NV];
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const uint32_t c = c0 + j * width + l * VEC;
        load_codes<VEC, NT>(p[j], from, c, dim);
        scale[j] = c < dim ? scales[row * scales_ld + c / kScaleBlock] : 0.0f;
      }
      if (ragged(dim, VEC))
#pragma unroll
        for (int j = 0; j < NV; ++j) settle_codes<VEC>(p[j], from, c0 + j * width + l * VEC, dim);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float v[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[e] = p[j].get(e) * scale[j];
        store_cols<T, VEC, NT>(out + row * out_ld, v, c0 + j * width + l * VEC, dim);
      }
    }
  }
}

constexpr int64_t kStreamBytes = 100000000;  // calls of more bytes bypass the caches, as for the layer norm
constexpr int64_t kSlots = 2048;             // workgroups that walk over the rows

// The lanes of a row: a power of two that holds a block's lanes.
int shift_of(int64_t dim, int vec) {
  int shift = vec == 8 ? 4 : 5;
  while (shift < 8 && (int64_t)vec << shift < dim) ++shift;
  return shift;
}

unsigned grid_of(int64_t rows, int shift) {
  const int64_t per = kThreads >> shift, need = (rows + per - 1) / per;
  return (unsigned)(need < kSlots ? need : kSlots);
}

template <typename F>
void either(bool nt, F&& f) {
  if (nt) f(std::true_type{});
  else f(std::false_type{});
}

}  // namespace

hipError_t launch_activation_pack(const void* x, int dtype, int64_t x_ld, int64_t rows, int64_t dim, uint8_t* codes,
                                  int64_t codes_ld, float* scales, int64_t scales_ld, hipStream_t s) {
  either(rows * dim * (dtype == ZS_BF16 ? 3 : 5) > kStreamBytes, [&](auto nt) {
    constexpr bool NT = decltype(nt)::value;
    const int shift = shift_of(dim, dtype == ZS_BF16 ? 8 : 4);
    const dim3 grid(grid_of(rows, shift)), block(kThreads);
    if (dtype == ZS_BF16) hipLaunchKernelGGL((k_pack<uint16_t, 8, NT>), grid, block, 0, s, (const uint16_t*)x, x_ld, rows, (uint32_t)dim, codes, codes_ld, scales, scales_ld, shift);
    else hipLaunchKernelGGL((k_pack<float, 4, NT>), grid, block, 0, s, (const float*)x, x_ld, rows, (uint32_t)dim, codes, codes_ld, scales, scales_ld, shift);
  });
  return hipGetLastError();
}

hipError_t launch_activation_unpack(const uint8_t* codes, int64_t codes_ld, const float* scales, int64_t scales_ld,
                                    int64_t rows, int64_t dim, void* out, int dtype, int64_t out_ld, hipStream_t s) {
  either(rows * dim * (dtype == ZS_BF16 ? 3 : 5) > kStreamBytes, [&](auto nt) {
    constexpr bool NT = decltype(nt)::value;
    const int shift = shift_of(dim, dtype == ZS_BF16 ? 8 : 4);
    const dim3 grid(grid_of(rows, shift)), block(kThreads);
    if (dtype == ZS_BF16) hipLaunchKernelGGL((k_unpack<uint16_t, 8, NT>), grid, block, 0, s, codes, codes_ld, scales, scales_ld, rows, (uint32_t)dim, (uint16_t*)out, out_ld, shift);
    else hipLaunchKernelGGL((k_unpack<float, 4, NT>), grid, block, 0, s, codes, codes_ld, scales, scales_ld, rows, (uint32_t)dim, (float*)out, out_ld, shift);
  });
  return hipGetLastError();
}

}  // namespace zs
