// Standalone C-ABI driver of the embedding and layer norm calls: one
// micro-batch forward and back through libzs with nothing but the HIP runtime
// (no Python, no PyTorch). Test infrastructure: the GPU test writes the
// inputs, runs this program, and checks its outputs.
//
//   zs_rows_driver IN OUT
//
// IN (little-endian): int64 n, vocab, ctx, dim, double scale, then int64
//   tokens[n], positions[n], bf16 table[vocab, dim], pos_table[ctx, dim],
//   weight[dim], bias[dim], dy[n, dim].
// OUT: h[n, dim] bf16 (zs_embed_forward with positions), y[n, dim] bf16, mean[n],
//   rstd[n] fp32 (zs_layer_norm_forward, eps 1e-5), dx[n, dim] bf16, dweight[dim],
//   dbias[dim] fp32 (zs_layer_norm_backward, first), dtable[vocab, dim] fp32
//   (zs_embed_backward of dx by the tokens, first, then the same once more
//   added), dpos[ctx, dim] bf16 (by the positions, first).
// Exit status: 0 on success, 2 on a usage or I/O error, 3 on a HIP error, and
// 10 + |status| when an entry point returns an error.
#include <hip/hip_runtime.h>

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

template <typename T>
T* dev(size_t count) {
  T* d = nullptr;
  HIP_OK(hipMalloc(&d, count * sizeof(T) + 16));
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
  int64_t size[4];
  double scale = 0;
  if (std::fread(size, sizeof(int64_t), 4, in) != 4 || std::fread(&scale, sizeof(scale), 1, in) != 1) return 2;
  const int64_t n = size[0], vocab = size[1], ctx = size[2], dim = size[3];
  if (n < 1 || vocab < 1 || ctx < 1 || dim < 1) return 2;
  const int64_t* tokens = read_dev<int64_t>(in, n);
  const int64_t* positions = read_dev<int64_t>(in, n);
  const uint16_t* table = read_dev<uint16_t>(in, vocab * dim);
  const uint16_t* pos_table = read_dev<uint16_t>(in, ctx * dim);
  const uint16_t* weight = read_dev<uint16_t>(in, dim);
  const uint16_t* bias = read_dev<uint16_t>(in, dim);
  const uint16_t* dy = read_dev<uint16_t>(in, n * dim);
  std::fclose(in);
  if (!tokens || !positions || !table || !pos_table || !weight || !bias || !dy) return 2;

  hipStream_t s;
  HIP_OK(hipStreamCreate(&s));
  uint16_t *h = dev<uint16_t>(n * dim), *y = dev<uint16_t>(n * dim), *dx = dev<uint16_t>(n * dim);
  float *mean = dev<float>(n), *rstd = dev<float>(n), *dw = dev<float>(dim), *db = dev<float>(dim);
  float* dtable = dev<float>(vocab * dim);
  uint16_t* dpos = dev<uint16_t>(ctx * dim);
  // one workspace for calls in a row on one stream: the largest that any of them needs
  size_t ws_bytes = zs_layer_norm_workspace_bytes(n, dim);
  for (int64_t v : {vocab, ctx})
    if (zs_embed_workspace_bytes(n, v, dim) > ws_bytes) ws_bytes = zs_embed_workspace_bytes(n, v, dim);
  void* ws = dev<unsigned char>(ws_bytes);

  ZS_OK_OR_EXIT(zs_embed_forward(table, ZS_BF16, vocab, dim, dim, pos_table, ctx, dim, tokens, positions, ZS_I64, n,
                                 (float)scale, h, ZS_BF16, dim, s));
  ZS_OK_OR_EXIT(zs_layer_norm_forward(h, ZS_BF16, dim, weight, bias, ZS_BF16, n, dim, 1e-5, y, dim, mean, rstd, s));
  ZS_OK_OR_EXIT(zs_layer_norm_backward(dy, dim, h, dim, ZS_BF16, weight, ZS_BF16, mean, rstd, n, dim, dx, dim, dw, db,
                                       ZS_F32, 1, ws, ws_bytes, s));
  for (int first : {1, 0})
    ZS_OK_OR_EXIT(zs_embed_backward(dx, ZS_BF16, dim, tokens, ZS_I64, n, vocab, dim, -1, (float)scale, dtable, ZS_F32,
                                    dim, first, ws, ws_bytes, s));
  ZS_OK_OR_EXIT(zs_embed_backward(dx, ZS_BF16, dim, positions, ZS_I64, n, ctx, dim, -1, 1.0f, dpos, ZS_BF16, dim, 1,
                                  ws, ws_bytes, s));
  HIP_OK(hipStreamSynchronize(s));

  FILE* out = std::fopen(argv[2], "wb");
  if (!out) return 2;
  bool ok = write_dev(out, h, n * dim) && write_dev(out, y, n * dim) && write_dev(out, mean, n) &&
            write_dev(out, rstd, n) && write_dev(out, dx, n * dim) && write_dev(out, dw, dim) &&
            write_dev(out, db, dim) && write_dev(out, dtable, vocab * dim) && write_dev(out, dpos, ctx * dim);
  ok = std::fclose(out) == 0 && ok;
  if (!ok) return 2;
  for (const void* p : {(const void*)tokens, (const void*)positions, (const void*)table, (const void*)pos_table,
                        (const void*)weight, (const void*)bias, (const void*)dy, (const void*)h, (const void*)y,
                        (const void*)dx, (const void*)mean, (const void*)rstd, (const void*)dw, (const void*)db,
                        (const void*)dtable, (const void*)dpos, (const void*)ws})
    HIP_OK(hipFree(const_cast<void*>(p)));
  HIP_OK(hipStreamDestroy(s));
  std::printf("zs_rows_driver ok: n=%lld vocab=%lld ctx=%lld dim=%lld\n", (long long)n, (long long)vocab,
              (long long)ctx, (long long)dim);
  return 0;
}
