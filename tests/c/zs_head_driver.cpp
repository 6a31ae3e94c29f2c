// Standalone C-ABI driver of the RMS norm, 8-bit activation and loss calls: one
// micro-batch forward and back through libzs with nothing but the HIP runtime
// (no Python, no PyTorch). Test infrastructure: the GPU test writes the
// inputs, runs this program, and checks its outputs.
//
//   zs_head_driver IN OUT
//
// IN (little-endian): int64 n, vocab, dim, then int32 labels[n], bf16 x[n, dim],
//   fp32 residual[n, dim], bf16 weight[dim], bf16 head[vocab, dim].
// OUT: sum[n, dim] fp32, y[n, dim] bf16, codes[n, dim], scales[n, ceil(dim / 128)],
//   rstd[n] fp32 (zs_rms_norm_forward, eps 1e-5), kept[n, dim], kept_scales fp32
//   (zs_activation_pack of the sum), values[n, dim] fp32 (zs_activation_unpack of
//   them), loss[n], lse[n] fp32, dy[n, dim] bf16, dhead[vocab, dim] fp32
//   (zs_linear_cross_entropy_backward, scale 1 / n, first), dh[n, dim] fp32,
//   dweight[dim] fp32 (zs_rms_norm_backward from the kept codes, with the residual
//   as the gradient along the stream).
// Exit status: 0 on success, 2 on a usage or I/O error, 3 on a HIP error, and
// 10 + |status| when an entry point returns an error.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "zs.h"

#define HIP_OK(x)                                                  \
  do {                                                             \
    hipError_t e_ = (x);                                           \
    if (e_ != hipSuccess) {                                        \
      std::fprintf(stderr, "%s: %s\n", #x, hipGetErrorString(e_)); \
      std::exit(3);                                                \
    }                                                              \
  } while (0)
#define ZS_OK_OR_EXIT(x)                                            \
  do {                                                              \
    zs_status s_ = (x);                                             \
    if (s_ != ZS_OK) {                                              \
      std::fprintf(stderr, "%s -> %s\n", #x, zs_status_string(s_)); \
      std::exit(10 - s_ > 255 ? 255 : 10 - s_);                     \
    }                                                               \
  } while (0)

namespace {

std::vector<void*> held;  // freed at the end

template <typename T>
T* dev(size_t count) {
  T* d = nullptr;
  HIP_OK(hipMalloc(&d, count * sizeof(T) + 16));
  held.push_back(d);
  return d;
}
// `count` values of the input file on the device; null where it is too short
template <typename T>
T* read_dev(FILE* f, size_t count) {
  std::vector<T> h(count);
  if (std::fread(h.data(), sizeof(T), count, f) != count) return nullptr;
  T* d = dev<T>(count);
  HIP_OK(hipMemcpy(d, h.data(), count * sizeof(T), hipMemcpyHostToDevice));
  return d;
}
template <typename T>
bool write_dev(FILE* f, const T* d, size_t count) {
  std::vector<T> h(count);
  HIP_OK(hipMemcpy(h.data(), d, count * sizeof(T), hipMemcpyDeviceToHost));
  return std::fwrite(h.data(), sizeof(T), count, f) == count;
}

}  // namespace

int main(int argc, char** argv) {
  if (argc != 3) {
    std::fprintf(stderr, "usage: %s IN OUT\n", argv[0]);
    return 2;
  }
  FILE* in = std::fopen(argv[1], "rb");
  if (!in) return 2;
  int64_t size[3];
  if (std::fread(size, sizeof(int64_t), 3, in) != 3) return 2;
  const int64_t n = size[0], vocab = size[1], dim = size[2], blocks = (dim + 127) / 128;
  if (n < 1 || vocab < 1 || dim < 1) return 2;
  const int32_t* labels = read_dev<int32_t>(in, n);
  const uint16_t* x = read_dev<uint16_t>(in, n * dim);
  const float* residual = read_dev<float>(in, n * dim);
  const uint16_t* weight = read_dev<uint16_t>(in, dim);
  const uint16_t* head = read_dev<uint16_t>(in, vocab * dim);
  std::fclose(in);
  if (!labels || !x || !residual || !weight || !head) return 2;

  hipStream_t s;
  HIP_OK(hipStreamCreate(&s));
  float *sum = dev<float>(n * dim), *values = dev<float>(n * dim), *dh = dev<float>(n * dim), *dhead = dev<float>(vocab * dim);
  uint16_t *y = dev<uint16_t>(n * dim), *dy = dev<uint16_t>(n * dim);
  uint8_t *codes = dev<uint8_t>(n * dim), *kept = dev<uint8_t>(n * dim);
  float *scales = dev<float>(n * blocks), *kept_scales = dev<float>(n * blocks);
  float *rstd = dev<float>(n), *loss = dev<float>(n), *lse = dev<float>(n), *dweight = dev<float>(dim);
  // one workspace for calls in a row on one stream: the largest that any of them needs
  const size_t ws_bytes = std::max({zs_rms_norm_workspace_bytes(n, dim),
                                    zs_linear_cross_entropy_workspace_bytes(n, vocab, dim, ZS_BF16, -1),
                                    zs_linear_cross_entropy_workspace_bytes(n, vocab, dim, ZS_BF16, ZS_F32)});
  void* ws = dev<unsigned char>(ws_bytes);

  ZS_OK_OR_EXIT(zs_rms_norm_forward(x, ZS_BF16, dim, residual, dim, sum, dim, ZS_F32, weight, ZS_BF16, n, dim, 1e-5, y,
                                    dim, codes, dim, scales, blocks, rstd, s));
  ZS_OK_OR_EXIT(zs_activation_pack(sum, ZS_F32, dim, n, dim, kept, dim, kept_scales, blocks, s));
  ZS_OK_OR_EXIT(zs_activation_unpack(kept, dim, kept_scales, blocks, n, dim, values, ZS_F32, dim, s));
  ZS_OK_OR_EXIT(zs_linear_cross_entropy_forward(y, dim, ZS_BF16, head, dim, labels, ZS_I32, n, vocab, dim, loss, lse, ws,
                                                ws_bytes, s));
  ZS_OK_OR_EXIT(zs_linear_cross_entropy_backward(y, dim, ZS_BF16, head, dim, labels, ZS_I32, lse, nullptr, 1.0f / (float)n,
                                                 n, vocab, dim, dy, dim, dhead, ZS_F32, dim, 1, ws, ws_bytes, s));
  ZS_OK_OR_EXIT(zs_rms_norm_backward(dy, ZS_BF16, dim, kept, ZS_E4M3, dim, kept_scales, blocks, weight, ZS_BF16, rstd,
                                     residual, dim, n, dim, dh, dim, ZS_F32, dweight, ZS_F32, 1, ws, ws_bytes, s));
  HIP_OK(hipStreamSynchronize(s));

  FILE* out = std::fopen(argv[2], "wb");
  if (!out) return 2;
  bool ok = write_dev(out, sum, n * dim) && write_dev(out, y, n * dim) && write_dev(out, codes, n * dim) &&
            write_dev(out, scales, n * blocks) && write_dev(out, rstd, n) && write_dev(out, kept, n * dim) &&
            write_dev(out, kept_scales, n * blocks) && write_dev(out, values, n * dim) && write_dev(out, loss, n) &&
            write_dev(out, lse, n) && write_dev(out, dy, n * dim) && write_dev(out, dhead, vocab * dim) &&
            write_dev(out, dh, n * dim) && write_dev(out, dweight, dim);
  ok = std::fclose(out) == 0 && ok;
  if (!ok) return 2;
  for (void* p : held) HIP_OK(hipFree(p));
  HIP_OK(hipStreamDestroy(s));
  std::printf("zs_head_driver ok: n=%lld vocab=%lld dim=%lld\n", (long long)n, (long long)vocab, (long long)dim);
  return 0;
}
