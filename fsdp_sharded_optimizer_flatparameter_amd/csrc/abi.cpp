// extern "C" entry points of libzs: argument validation on the host, then the
// launchers. Nothing here allocates memory or keeps state between calls.
#include <cmath>
#include <cstdint>

#include "zs.h"
#include "zs_launch.hpp"
#include "zs_launch_head.hpp"
#include "zs_launch_rows.hpp"

namespace {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// [a, a+na) and [b, b+nb) (bytes) intersect?
inline bool overlaps(const void* a, int64_t na, const void* b, int64_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return na > 0 && nb > 0 && x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}

inline int64_t elem_size(int32_t dtype) { return dtype == ZS_BF16 ? 2 : 4; }

zs_status check_hparams(const zs_adamw_hparams* hp) {
  if (!hp) return ZS_ERR_NULL;
  const double v[5] = {hp->lr, hp->beta1, hp->beta2, hp->eps, hp->weight_decay};
  for (double x : v)
    if (!std::isfinite(x)) return ZS_ERR_HPARAM;
  if (hp->lr < 0 || hp->eps < 0 || hp->weight_decay < 0) return ZS_ERR_HPARAM;
  if (!(hp->beta1 >= 0 && hp->beta1 < 1) || !(hp->beta2 >= 0 && hp->beta2 < 1)) return ZS_ERR_HPARAM;
  if (hp->step < 1) return ZS_ERR_HPARAM;
  return ZS_OK;
}

zs_status check_rows(const void* const* rows, int32_t world, int32_t dtype, int64_t n) {
  if (world < 1 || world > ZS_MAX_WORLD) return ZS_ERR_WORLD;
  if (dtype != ZS_F32 && dtype != ZS_BF16) return ZS_ERR_DTYPE;
  if (n < 0) return ZS_ERR_SIZE;
  if (n == 0) return ZS_OK;  // nothing is read: rows (and their entries) may be NULL
  if (!rows) return ZS_ERR_NULL;
  for (int32_t q = 0; q < world; ++q) {
    if (!rows[q]) return ZS_ERR_NULL;
    if (!aligned(rows[q], (uintptr_t)elem_size(dtype))) return ZS_ERR_ALIGN;
  }
  return ZS_OK;
}

// Device work goes through launch(): a HIP error already pending on this thread
// (left by an earlier, unrelated call) is handed back as ZS_ERR_HIP before
// anything is enqueued, and stays pending for the caller; otherwise the status
// is that of this call's own launches.
template <typename F>
zs_status launch(F&& f) {
  if (hipPeekAtLastError() != hipSuccess) return ZS_ERR_HIP;
  return f() == hipSuccess ? ZS_OK : ZS_ERR_HIP;
}

// The sum of squares' workspace and result are written while the rows are read
// and `out` (n fp32) is written: none of them may share bytes.
zs_status check_sumsq_buffers(const void* const* rows, int32_t world, int32_t dtype, int64_t n,
                              const void* out, const void* sumsq, const void* ws, size_t ws_bytes) {
  const int64_t wb = (int64_t)ws_bytes;
  if (overlaps(sumsq, 8, ws, wb) || overlaps(sumsq, 8, out, n * 4) || overlaps(ws, wb, out, n * 4))
    return ZS_ERR_OVERLAP;
  for (int32_t q = 0; q < world && n > 0; ++q) {
    const int64_t rb = n * elem_size(dtype);
    if (overlaps(rows[q], rb, sumsq, 8) || overlaps(rows[q], rb, ws, wb)) return ZS_ERR_OVERLAP;
  }
  return ZS_OK;
}

// The gradient scale is read by every workgroup while the state is written.
bool scale_overlaps(const float* scale, const void* a, const void* b, const void* c, int64_t n,
                    const void* bf16_out) {
  return scale && (overlaps(scale, 4, a, n * 4) || overlaps(scale, 4, b, n * 4) ||
                   overlaps(scale, 4, c, n * 4) || (bf16_out && overlaps(scale, 4, bf16_out, n * 2)));
}

inline bool float_type(int32_t dtype) { return dtype == ZS_F32 || dtype == ZS_BF16; }
inline bool index_type_ok(int32_t t) { return t == ZS_I32 || t == ZS_I64; }
inline int64_t index_size(int32_t t) { return t == ZS_I32 ? 4 : 8; }

// Sizes of the embedding and layer norm calls: counts stay in 31 bits (sorted
// positions and keys are 32-bit), widths in 24 (columns are 32-bit, and the
// launches over columns stay within a dispatch's 32-bit work-item count).
constexpr int64_t kMaxCount = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxDim = (int64_t(1) << 24) - 1;
inline bool count_ok(int64_t n) { return n >= 0 && n <= kMaxCount; }
inline bool dim_ok(int64_t d) { return d >= 0 && d <= kMaxDim; }

// A row stride holds a row, and the last row's end (in bytes) stays in 63 bits.
inline bool stride_ok(int64_t rows, int64_t dim, int64_t ld) {
  return ld >= dim && ld <= (INT64_MAX / 8 - dim) / (rows > 0 ? rows : 1);
}

// Device memory of one argument, for the overlap checks. Rows that leave gaps
// between them count with their gaps.
struct Span {
  const void* p;
  int64_t bytes;
};
Span rows_span(const void* p, int64_t rows, int64_t dim, int64_t ld, int32_t dtype) {
  return Span{p, p && rows > 0 && dim > 0 ? ((rows - 1) * ld + dim) * elem_size(dtype) : 0};
}
bool any_overlap(const Span& a, const Span* b, int n) {
  for (int i = 0; i < n; ++i)
    if (overlaps(a.p, a.bytes, b[i].p, b[i].bytes)) return true;
  return false;
}

// Activations in 8 bits: a byte and a share of a scale for each element.
inline int64_t scale_blocks(int64_t dim) { return (dim + 127) / 128; }
Span codes_span(const void* p, int64_t rows, int64_t dim, int64_t ld) {
  return Span{p, p && rows > 0 && dim > 0 ? (rows - 1) * ld + dim : 0};
}
Span scales_span(const void* p, int64_t rows, int64_t dim, int64_t ld) {
  return rows_span(p, rows, scale_blocks(dim), ld, ZS_F32);
}
inline bool codes_size_ok(int64_t rows, int64_t dim, int64_t codes_ld, int64_t scales_ld) {
  return stride_ok(rows, dim, codes_ld) && stride_ok(rows, scale_blocks(dim), scales_ld);
}
// The residual stream has the type of what is added to it, or fp32.
inline bool stream_type_ok(int32_t dtype, int32_t stream) { return stream == ZS_F32 || (stream == ZS_BF16 && dtype == ZS_BF16); }

// Sizes of the loss over a vocabulary: 256 rows of three planes within 32 bits of
// offset, a grid of tiles within 31 bits.
inline bool head_size_ok(int64_t n, int64_t vocab, int64_t dim) {
  return count_ok(n) && count_ok(vocab) && dim >= 0 && dim <= (1 << 20) &&
         (vocab / 128 + 1) * (n / 128 + 1) <= INT32_MAX;
}

}  // namespace

extern "C" {

int32_t zs_version(void) { return 200; /* 0.2.0 */ }

const char* zs_status_string(zs_status s) {
  switch (s) {
    case ZS_OK: return "ZS_OK";
    case ZS_ERR_NULL: return "ZS_ERR_NULL";
    case ZS_ERR_SIZE: return "ZS_ERR_SIZE";
    case ZS_ERR_WORLD: return "ZS_ERR_WORLD";
    case ZS_ERR_RANK: return "ZS_ERR_RANK";
    case ZS_ERR_DTYPE: return "ZS_ERR_DTYPE";
    case ZS_ERR_HPARAM: return "ZS_ERR_HPARAM";
    case ZS_ERR_SHARD: return "ZS_ERR_SHARD";
    case ZS_ERR_WORKSPACE: return "ZS_ERR_WORKSPACE";
    case ZS_ERR_LAYOUT: return "ZS_ERR_LAYOUT";
    case ZS_ERR_ALIGN: return "ZS_ERR_ALIGN";
    case ZS_ERR_OVERLAP: return "ZS_ERR_OVERLAP";
    case ZS_ERR_HIP: return "ZS_ERR_HIP";
    default: return "ZS_ERR_UNKNOWN";
  }
}

// S of a unit of t elements over `world` ranks: ceil(t / world) rounded up to a
// multiple of `align`; ZS_ERR_SIZE when it or S * world overflows int64.
static zs_status shard_length(int64_t t, int32_t world, int64_t align, int64_t* s_out) {
  int64_t s = t / world + (t % world != 0);
  if (align > 1) {
    if (s > INT64_MAX - (align - 1)) return ZS_ERR_SIZE;
    s = (s + align - 1) / align * align;
  }
  if (s > INT64_MAX / world) return ZS_ERR_SIZE;
  *s_out = s;
  return ZS_OK;
}

zs_status zs_flat_layout(const int64_t* numels, int32_t nparams, int32_t world, int64_t align,
                         int64_t* offsets_out, int64_t* total_out, int64_t* padded_out,
                         int64_t* shard_out) {
  if (nparams < 0 || align < 1) return ZS_ERR_SIZE;
  if (world < 1) return ZS_ERR_WORLD;
  if (nparams > 0 && !numels) return ZS_ERR_NULL;
  int64_t t = 0;
  for (int32_t i = 0; i < nparams; ++i) {
    if (numels[i] < 0) return ZS_ERR_SIZE;
    if (numels[i] > INT64_MAX - t) return ZS_ERR_SIZE;
    t += numels[i];
  }
  int64_t s = 0;
  if (const zs_status st = shard_length(t, world, align, &s)) return st;
  if (offsets_out) {
    int64_t run = 0;
    for (int32_t i = 0; i < nparams; ++i) {
      offsets_out[i] = run;
      run += numels[i];
    }
  }
  if (total_out) *total_out = t;
  if (padded_out) *padded_out = s * world;
  if (shard_out) *shard_out = s;
  return ZS_OK;
}

zs_status zs_check_layout(const zs_param_desc* host_desc, int32_t nparams, int64_t total,
                          int32_t dtype) {
  if (dtype != ZS_F32 && dtype != ZS_BF16) return ZS_ERR_DTYPE;
  if (nparams < 0 || total < 0) return ZS_ERR_SIZE;
  if (nparams == 0) return total == 0 ? ZS_OK : ZS_ERR_LAYOUT;
  if (!host_desc) return ZS_ERR_NULL;
  int64_t run = 0;
  for (int32_t i = 0; i < nparams; ++i) {
    const zs_param_desc& d = host_desc[i];
    if (d.numel < 0) return ZS_ERR_SIZE;
    if (d.flat_offset != run) return ZS_ERR_LAYOUT;
    if (d.numel > 0 && !d.ptr) return ZS_ERR_NULL;
    if (d.numel > 0 && !aligned(d.ptr, (uintptr_t)elem_size(dtype))) return ZS_ERR_ALIGN;
    if (d.numel > INT64_MAX - run) return ZS_ERR_SIZE;
    run += d.numel;
  }
  return run == total ? ZS_OK : ZS_ERR_LAYOUT;
}

size_t zs_workspace_bytes(int64_t n) {
  if (n < 0) return 0;
  return (size_t)(zs::max_partials(n) + zs::kFinalizeBlocks) * sizeof(double);
}

zs_status zs_pack_shard(const zs_param_desc* d_desc, int32_t nparams, int64_t total_numel,
                        int32_t src_dtype, int32_t world, int32_t rank, int64_t align,
                        int64_t shard_numel, float* master, float* exp_avg, float* exp_avg_sq,
                        hipStream_t stream) {
  if (nparams < 0 || total_numel < 0 || shard_numel < 0 || align < 1) return ZS_ERR_SIZE;
  if (nparams == 0 && total_numel != 0) return ZS_ERR_SIZE;
  if (world < 1) return ZS_ERR_WORLD;
  if (rank < 0 || rank >= world) return ZS_ERR_RANK;
  if (src_dtype != ZS_F32 && src_dtype != ZS_BF16) return ZS_ERR_DTYPE;
  int64_t s = 0;
  if (const zs_status st = shard_length(total_numel, world, align, &s)) return st;
  if (shard_numel != s) return ZS_ERR_SHARD;
  if (shard_numel == 0) return ZS_OK;
  if (!master || (nparams > 0 && !d_desc)) return ZS_ERR_NULL;
  if (!aligned(master, 4) || (exp_avg && !aligned(exp_avg, 4)) ||
      (exp_avg_sq && !aligned(exp_avg_sq, 4)) || !aligned(d_desc, 8))
    return ZS_ERR_ALIGN;
  const int64_t b = shard_numel * 4;
  if (overlaps(master, b, exp_avg, exp_avg ? b : 0) ||
      overlaps(master, b, exp_avg_sq, exp_avg_sq ? b : 0) ||
      overlaps(exp_avg, exp_avg ? b : 0, exp_avg_sq, exp_avg_sq ? b : 0))
    return ZS_ERR_OVERLAP;
  return launch([&] { return zs::launch_pack(d_desc, nparams, total_numel, src_dtype,
                                    (int64_t)rank * shard_numel, shard_numel, master, exp_avg,
                                    exp_avg_sq, stream); });
}

zs_status zs_reduce_grads(const void* const* rows, int32_t world, int32_t dtype, int64_t n,
                          float* grad_out, double* sumsq_out, void* workspace,
                          size_t workspace_bytes, hipStream_t stream) {
  zs_status st = check_rows(rows, world, dtype, n);
  if (st != ZS_OK) return st;
  if (n > 0 && !grad_out) return ZS_ERR_NULL;
  if (grad_out && !aligned(grad_out, 4)) return ZS_ERR_ALIGN;
  if (sumsq_out) {
    if (!aligned(sumsq_out, 8)) return ZS_ERR_ALIGN;
    if (!workspace || workspace_bytes < zs_workspace_bytes(n)) return ZS_ERR_WORKSPACE;
    if (!aligned(workspace, 8)) return ZS_ERR_ALIGN;
    st = check_sumsq_buffers(rows, world, dtype, n, grad_out, sumsq_out, workspace, workspace_bytes);
    if (st != ZS_OK) return st;
  }
  if (n == 0) {
    if (!sumsq_out) return ZS_OK;
    // an empty shard's sum of squares is 0; written by the finalize kernel
    return launch([&] { return zs::launch_reduce(rows, world, dtype, 0, grad_out, sumsq_out,
                                        static_cast<double*>(workspace), stream); });
  }
  for (int32_t q = 0; q < world; ++q)
    if (overlaps(grad_out, n * 4, rows[q], n * elem_size(dtype))) return ZS_ERR_OVERLAP;
  return launch([&] { return zs::launch_reduce(rows, world, dtype, n, grad_out, sumsq_out,
                                      static_cast<double*>(workspace), stream); });
}

zs_status zs_reduce_grads_noalloc(const void* const* rows, int32_t world, int32_t dtype, int64_t n,
                                  float* grad_out, double* sumsq_out, hipStream_t stream) {
  zs_status st = check_rows(rows, world, dtype, n);
  if (st != ZS_OK) return st;
  if (n > 0 && !grad_out) return ZS_ERR_NULL;
  if (grad_out && !aligned(grad_out, 4)) return ZS_ERR_ALIGN;
  if (sumsq_out) {
    if (n > ZS_NOALLOC_MAX_N) return ZS_ERR_WORKSPACE;  // beyond the library's scratch
    if (!aligned(sumsq_out, 8)) return ZS_ERR_ALIGN;
    st = check_sumsq_buffers(rows, world, dtype, n, grad_out, sumsq_out, nullptr, 0);
    if (st != ZS_OK) return st;
  }
  if (n == 0 && !sumsq_out) return ZS_OK;
  for (int32_t q = 0; q < world && n > 0; ++q)
    if (overlaps(grad_out, n * 4, rows[q], n * elem_size(dtype))) return ZS_ERR_OVERLAP;
  return launch([&] {
    double* partials = nullptr;
    if (sumsq_out) {
      const hipError_t e = zs::static_partials(stream, &partials);
      if (e != hipSuccess) return e;
    }
    return zs::launch_reduce(rows, world, dtype, n, grad_out, sumsq_out, partials, stream);
  });
}

zs_status zs_adamw_step(float* master, float* exp_avg, float* exp_avg_sq, const float* grad,
                        int64_t n, const zs_adamw_hparams* hp, const float* grad_scale,
                        uint16_t* bf16_out, hipStream_t stream) {
  if (n < 0) return ZS_ERR_SIZE;
  zs_status st = check_hparams(hp);
  if (st != ZS_OK) return st;
  if (n == 0) return ZS_OK;
  if (!master || !exp_avg || !exp_avg_sq || !grad) return ZS_ERR_NULL;
  if (!aligned(master, 4) || !aligned(exp_avg, 4) || !aligned(exp_avg_sq, 4) ||
      !aligned(grad, 4) || (bf16_out && !aligned(bf16_out, 2)) ||
      (grad_scale && !aligned(grad_scale, 4)))
    return ZS_ERR_ALIGN;
  const int64_t b = n * 4;
  if (overlaps(master, b, exp_avg, b) || overlaps(master, b, exp_avg_sq, b) ||
      overlaps(exp_avg, b, exp_avg_sq, b) || overlaps(grad, b, master, b) ||
      overlaps(grad, b, exp_avg, b) || overlaps(grad, b, exp_avg_sq, b))
    return ZS_ERR_OVERLAP;
  if (bf16_out && (overlaps(bf16_out, n * 2, master, b) || overlaps(bf16_out, n * 2, exp_avg, b) ||
                   overlaps(bf16_out, n * 2, exp_avg_sq, b) || overlaps(bf16_out, n * 2, grad, b)))
    return ZS_ERR_OVERLAP;
  if (scale_overlaps(grad_scale, master, exp_avg, exp_avg_sq, n, bf16_out)) return ZS_ERR_OVERLAP;
  return launch([&] {
    return zs::launch_adamw(master, exp_avg, exp_avg_sq, grad, n, *hp, grad_scale, bf16_out, stream);
  });
}

zs_status zs_cast_for_gather(const float* master, int64_t n, uint16_t* gather_slot,
                             hipStream_t stream) {
  if (n < 0) return ZS_ERR_SIZE;
  if (n == 0) return ZS_OK;
  if (!master || !gather_slot) return ZS_ERR_NULL;
  if (!aligned(master, 4) || !aligned(gather_slot, 2)) return ZS_ERR_ALIGN;
  if (overlaps(master, n * 4, gather_slot, n * 2)) return ZS_ERR_OVERLAP;
  return launch([&] { return zs::launch_cast(master, n, gather_slot, stream); });
}

zs_status zs_copy_out(const uint16_t* gathered, int64_t gathered_numel, const zs_param_desc* d_desc,
                      int32_t nparams, int64_t total_numel, hipStream_t stream) {
  if (nparams < 0 || total_numel < 0 || gathered_numel < 0) return ZS_ERR_SIZE;
  if (total_numel > gathered_numel) return ZS_ERR_SIZE;
  if (nparams == 0 && total_numel != 0) return ZS_ERR_SIZE;
  if (total_numel == 0) return ZS_OK;
  if (!gathered || !d_desc) return ZS_ERR_NULL;
  if (!aligned(gathered, 2) || !aligned(d_desc, 8)) return ZS_ERR_ALIGN;
  return launch([&] { return zs::launch_copy_out(gathered, d_desc, nparams, total_numel, stream); });
}

zs_status zs_dim0_layout(const int64_t* dim0, const int64_t* rowsize, int32_t nparams, int32_t world,
                         int64_t* chunk_out, int64_t* local_offsets_out, int64_t* local_total_out) {
  if (nparams < 0) return ZS_ERR_SIZE;
  if (world < 1) return ZS_ERR_WORLD;
  if (nparams > 0 && (!dim0 || !rowsize)) return ZS_ERR_NULL;
  int64_t t = 0;
  for (int32_t i = 0; i < nparams; ++i) {
    if (dim0[i] < 0 || rowsize[i] < 0) return ZS_ERR_SIZE;
    const int64_t rows = dim0[i] / world + (dim0[i] % world != 0);
    if (rowsize[i] > 0 && rows > INT64_MAX / world / rowsize[i]) return ZS_ERR_SIZE;
    const int64_t c = rows * rowsize[i];
    if (c > INT64_MAX - t) return ZS_ERR_SIZE;
    if (chunk_out) chunk_out[i] = c;
    if (local_offsets_out) local_offsets_out[i] = t;
    t += c;
  }
  if (local_total_out) *local_total_out = t;
  return ZS_OK;
}

zs_status zs_check_dim0_layout(const zs_dim0_desc* host_desc, int32_t nparams, int32_t world,
                               int64_t total, int64_t local_total, int32_t dtype) {
  if (dtype != ZS_F32 && dtype != ZS_BF16) return ZS_ERR_DTYPE;
  if (nparams < 0 || total < 0 || local_total < 0) return ZS_ERR_SIZE;
  if (world < 1) return ZS_ERR_WORLD;
  if (nparams == 0) return total == 0 && local_total == 0 ? ZS_OK : ZS_ERR_LAYOUT;
  if (!host_desc) return ZS_ERR_NULL;
  int64_t run = 0, lrun = 0;
  for (int32_t i = 0; i < nparams; ++i) {
    const zs_dim0_desc& d = host_desc[i];
    if (d.numel < 0 || d.chunk < 0) return ZS_ERR_SIZE;
    if (d.flat_offset != run || d.local_offset != lrun) return ZS_ERR_LAYOUT;
    if (d.numel > 0 && !d.ptr) return ZS_ERR_NULL;
    if (d.numel > 0 && !aligned(d.ptr, (uintptr_t)elem_size(dtype))) return ZS_ERR_ALIGN;
    // the N chunks must cover the parameter: numel <= world * chunk
    if (d.chunk < d.numel / world + (d.numel % world != 0)) return ZS_ERR_LAYOUT;
    if (d.numel > INT64_MAX - run || d.chunk > INT64_MAX - lrun) return ZS_ERR_SIZE;
    run += d.numel;
    lrun += d.chunk;
  }
  if (lrun > INT64_MAX / world) return ZS_ERR_SIZE;
  return run == total && lrun == local_total ? ZS_OK : ZS_ERR_LAYOUT;
}

zs_status zs_pack_shard_dim0(const zs_dim0_desc* d_desc, int32_t nparams, int32_t src_dtype,
                             int32_t world, int32_t rank, int64_t local_total, float* master,
                             float* exp_avg, float* exp_avg_sq, hipStream_t stream) {
  if (nparams < 0 || local_total < 0) return ZS_ERR_SIZE;
  if (nparams == 0 && local_total != 0) return ZS_ERR_SIZE;
  if (world < 1) return ZS_ERR_WORLD;
  if (rank < 0 || rank >= world) return ZS_ERR_RANK;
  if (src_dtype != ZS_F32 && src_dtype != ZS_BF16) return ZS_ERR_DTYPE;
  if (local_total == 0) return ZS_OK;
  if (!master || !d_desc) return ZS_ERR_NULL;
  if (!aligned(master, 4) || (exp_avg && !aligned(exp_avg, 4)) ||
      (exp_avg_sq && !aligned(exp_avg_sq, 4)) || !aligned(d_desc, 8))
    return ZS_ERR_ALIGN;
  const int64_t b = local_total * 4;
  if (overlaps(master, b, exp_avg, exp_avg ? b : 0) ||
      overlaps(master, b, exp_avg_sq, exp_avg_sq ? b : 0) ||
      overlaps(exp_avg, exp_avg ? b : 0, exp_avg_sq, exp_avg_sq ? b : 0))
    return ZS_ERR_OVERLAP;
  return launch([&] { return zs::launch_pack_dim0(d_desc, nparams, src_dtype, rank, local_total, master,
                                         exp_avg, exp_avg_sq, stream); });
}

zs_status zs_copy_out_dim0(const uint16_t* gathered, int64_t gathered_numel,
                           const zs_dim0_desc* d_desc, int32_t nparams, int32_t world,
                           int64_t total, int64_t local_total, hipStream_t stream) {
  if (nparams < 0 || total < 0 || local_total < 0 || gathered_numel < 0) return ZS_ERR_SIZE;
  if (world < 1) return ZS_ERR_WORLD;
  if (nparams == 0 && (total != 0 || local_total != 0)) return ZS_ERR_SIZE;
  if (local_total > INT64_MAX / world || world * local_total > gathered_numel) return ZS_ERR_SIZE;
  if (total > world * local_total) return ZS_ERR_SIZE;
  if (total == 0) return ZS_OK;
  if (!gathered || !d_desc) return ZS_ERR_NULL;
  if (!aligned(gathered, 2) || !aligned(d_desc, 8)) return ZS_ERR_ALIGN;
  return launch([&] {
    return zs::launch_copy_out_dim0(gathered, d_desc, nparams, world, total, local_total, stream);
  });
}

zs_status zs_sharded_step(const void* const* rows, int32_t world, int32_t dtype, int64_t n,
                          float* master, float* exp_avg, float* exp_avg_sq,
                          const zs_adamw_hparams* hp, const float* grad_scale,
                          uint16_t* bf16_out, hipStream_t stream) {
  zs_status st = check_rows(rows, world, dtype, n);
  if (st != ZS_OK) return st;
  st = check_hparams(hp);
  if (st != ZS_OK) return st;
  if (n == 0) return ZS_OK;
  if (!master || !exp_avg || !exp_avg_sq) return ZS_ERR_NULL;
  if (!aligned(master, 4) || !aligned(exp_avg, 4) || !aligned(exp_avg_sq, 4) ||
      (bf16_out && !aligned(bf16_out, 2)) || (grad_scale && !aligned(grad_scale, 4)))
    return ZS_ERR_ALIGN;
  const int64_t b = n * 4;
  if (overlaps(master, b, exp_avg, b) || overlaps(master, b, exp_avg_sq, b) ||
      overlaps(exp_avg, b, exp_avg_sq, b))
    return ZS_ERR_OVERLAP;
  for (int32_t q = 0; q < world; ++q) {
    const int64_t rb = n * elem_size(dtype);
    if (overlaps(rows[q], rb, master, b) || overlaps(rows[q], rb, exp_avg, b) ||
        overlaps(rows[q], rb, exp_avg_sq, b) || (bf16_out && overlaps(rows[q], rb, bf16_out, n * 2)))
      return ZS_ERR_OVERLAP;
  }
  if (bf16_out && (overlaps(bf16_out, n * 2, master, b) || overlaps(bf16_out, n * 2, exp_avg, b) ||
                   overlaps(bf16_out, n * 2, exp_avg_sq, b)))
    return ZS_ERR_OVERLAP;
  if (scale_overlaps(grad_scale, master, exp_avg, exp_avg_sq, n, bf16_out)) return ZS_ERR_OVERLAP;
  return launch([&] { return zs::launch_fused(rows, world, dtype, n, master, exp_avg, exp_avg_sq, *hp,
                                     grad_scale, bf16_out, stream); });
}

zs_status zs_accumulate_grads(const void* const* rows, int32_t world, int32_t dtype, int64_t n,
                              float* acc, float scale, int32_t first, double* sumsq_out,
                              void* workspace, size_t workspace_bytes, hipStream_t stream) {
  zs_status st = check_rows(rows, world, dtype, n);
  if (st != ZS_OK) return st;
  if (!std::isfinite(scale)) return ZS_ERR_HPARAM;
  if (n > 0 && !acc) return ZS_ERR_NULL;
  if (acc && !aligned(acc, 4)) return ZS_ERR_ALIGN;
  if (sumsq_out) {
    if (!aligned(sumsq_out, 8)) return ZS_ERR_ALIGN;
    if (!workspace || workspace_bytes < zs_workspace_bytes(n)) return ZS_ERR_WORKSPACE;
    if (!aligned(workspace, 8)) return ZS_ERR_ALIGN;
    st = check_sumsq_buffers(rows, world, dtype, n, acc, sumsq_out, workspace, workspace_bytes);
    if (st != ZS_OK) return st;
  }
  if (n == 0 && !sumsq_out) return ZS_OK;
  for (int32_t q = 0; q < world && n > 0; ++q)
    if (overlaps(acc, n * 4, rows[q], n * elem_size(dtype))) return ZS_ERR_OVERLAP;
  return launch([&] { return zs::launch_accumulate(rows, world, dtype, n, acc, scale, first != 0, sumsq_out,
                                          static_cast<double*>(workspace), stream); });
}

zs_status zs_accumulate_local(const void* grad, int32_t dtype, int64_t n, float* acc,
                              int32_t first, hipStream_t stream) {
  if (dtype != ZS_F32 && dtype != ZS_BF16) return ZS_ERR_DTYPE;
  if (n < 0) return ZS_ERR_SIZE;
  if (n == 0) return ZS_OK;
  if (!grad || !acc) return ZS_ERR_NULL;
  if (!aligned(grad, (uintptr_t)elem_size(dtype)) || !aligned(acc, 4)) return ZS_ERR_ALIGN;
  if (overlaps(grad, n * elem_size(dtype), acc, n * 4)) return ZS_ERR_OVERLAP;
  return launch([&] { return zs::launch_accumulate_local(grad, dtype, n, acc, first != 0, stream); });
}

zs_status zs_clip_coefficient(const double* partials, int32_t count, double max_norm,
                              float* coef_out, double* norm_out, hipStream_t stream) {
  if (count < 1) return ZS_ERR_SIZE;
  if (!std::isfinite(max_norm) || !(max_norm > 0)) return ZS_ERR_HPARAM;
  if (!partials || !coef_out) return ZS_ERR_NULL;
  if (!aligned(partials, 8) || !aligned(coef_out, 4) || (norm_out && !aligned(norm_out, 8)))
    return ZS_ERR_ALIGN;
  return launch([&] { return zs::launch_clip(partials, count, max_norm, coef_out, norm_out, stream); });
}

zs_status zs_embed_forward(const void* table, int32_t dtype, int64_t vocab, int64_t dim,
                           int64_t table_ld, const void* pos_table, int64_t pos_rows, int64_t pos_ld,
                           const void* tokens, const void* positions, int32_t index_type, int64_t n,
                           float scale, void* out, int32_t out_dtype, int64_t out_ld,
                           hipStream_t stream) {
  if (!float_type(dtype) || !float_type(out_dtype) || !index_type_ok(index_type)) return ZS_ERR_DTYPE;
  if (!count_ok(n) || !count_ok(vocab) || !dim_ok(dim)) return ZS_ERR_SIZE;
  if (!stride_ok(vocab, dim, table_ld) || !stride_ok(n, dim, out_ld)) return ZS_ERR_SIZE;
  if (pos_table && (!count_ok(pos_rows) || !stride_ok(pos_rows, dim, pos_ld))) return ZS_ERR_SIZE;
  if (!std::isfinite(scale)) return ZS_ERR_HPARAM;
  if (n == 0 || dim == 0) return ZS_OK;
  if (!out || !tokens || (vocab > 0 && !table) || (pos_table && !positions)) return ZS_ERR_NULL;
  const uintptr_t es = (uintptr_t)elem_size(dtype), is = (uintptr_t)index_size(index_type);
  if (!aligned(table, es) || !aligned(pos_table, es) || !aligned(out, (uintptr_t)elem_size(out_dtype)) ||
      !aligned(tokens, is) || (pos_table && !aligned(positions, is)))
    return ZS_ERR_ALIGN;
  const Span in[4] = {rows_span(table, vocab, dim, table_ld, dtype),
                      rows_span(pos_table, pos_rows, dim, pos_ld, dtype),
                      {tokens, n * (int64_t)is},
                      {positions, pos_table ? n * (int64_t)is : 0}};
  if (any_overlap(rows_span(out, n, dim, out_ld, out_dtype), in, 4)) return ZS_ERR_OVERLAP;
  return launch([&] {
    return zs::launch_embed_forward(table, dtype, vocab, dim, table_ld, pos_table, pos_rows, pos_ld, tokens,
                                    positions, index_type, n, scale, out, out_dtype, out_ld, stream);
  });
}

size_t zs_embed_workspace_bytes(int64_t n, int64_t vocab, int64_t dim) {
  if (!count_ok(n) || !count_ok(vocab) || !dim_ok(dim)) return 0;
  return (size_t)zs::embed_plan(n, vocab, dim).bytes;
}

zs_status zs_embed_backward(const void* dout, int32_t dtype, int64_t dout_ld, const void* tokens,
                            int32_t index_type, int64_t n, int64_t vocab, int64_t dim,
                            int64_t padding_idx, float scale, void* grad, int32_t grad_dtype,
                            int64_t grad_ld, int32_t first, void* workspace, size_t workspace_bytes,
                            hipStream_t stream) {
  if (!float_type(dtype) || !float_type(grad_dtype) || !index_type_ok(index_type)) return ZS_ERR_DTYPE;
  if (!count_ok(n) || !count_ok(vocab) || !dim_ok(dim)) return ZS_ERR_SIZE;
  if (!stride_ok(n, dim, dout_ld) || !stride_ok(vocab, dim, grad_ld)) return ZS_ERR_SIZE;
  if (!std::isfinite(scale)) return ZS_ERR_HPARAM;
  if (vocab == 0 || dim == 0 || (n == 0 && !first)) return ZS_OK;
  if (!grad || (n > 0 && (!dout || !tokens))) return ZS_ERR_NULL;
  if (!aligned(grad, (uintptr_t)elem_size(grad_dtype)) ||
      (n > 0 && (!aligned(dout, (uintptr_t)elem_size(dtype)) || !aligned(tokens, (uintptr_t)index_size(index_type)))))
    return ZS_ERR_ALIGN;
  const size_t need = zs_embed_workspace_bytes(n, vocab, dim);
  if (!workspace || workspace_bytes < need) return ZS_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return ZS_ERR_ALIGN;
  const Span g = rows_span(grad, vocab, dim, grad_ld, grad_dtype), ws = {workspace, (int64_t)need};
  const Span in[2] = {rows_span(dout, n, dim, dout_ld, dtype), {tokens, n * index_size(index_type)}};
  if (any_overlap(g, in, 2) || any_overlap(ws, in, 2) || any_overlap(g, &ws, 1)) return ZS_ERR_OVERLAP;
  return launch([&] {
    return zs::launch_embed_backward(dout, dtype, dout_ld, tokens, index_type, n, vocab, dim, padding_idx, scale, grad,
                                     grad_dtype, grad_ld, first != 0, workspace, stream);
  });
}

zs_status zs_layer_norm_forward(const void* x, int32_t dtype, int64_t x_ld, const void* weight,
                                const void* bias, int32_t wdtype, int64_t rows, int64_t dim,
                                double eps, void* y, int64_t y_ld, float* mean, float* rstd,
                                hipStream_t stream) {
  if (!float_type(dtype) || !float_type(wdtype)) return ZS_ERR_DTYPE;
  if (!count_ok(rows) || !dim_ok(dim) || (rows > 0 && dim < 1)) return ZS_ERR_SIZE;
  if (!stride_ok(rows, dim, x_ld) || !stride_ok(rows, dim, y_ld)) return ZS_ERR_SIZE;
  if (!std::isfinite((float)eps) || eps < 0) return ZS_ERR_HPARAM;
  if (rows == 0) return ZS_OK;
  if (!x || !y) return ZS_ERR_NULL;
  const uintptr_t es = (uintptr_t)elem_size(dtype), wsz = (uintptr_t)elem_size(wdtype);
  if (!aligned(x, es) || !aligned(y, es) || !aligned(weight, wsz) || !aligned(bias, wsz) || !aligned(mean, 4) ||
      !aligned(rstd, 4))
    return ZS_ERR_ALIGN;
  const Span in[3] = {rows_span(x, rows, dim, x_ld, dtype), rows_span(weight, 1, dim, dim, wdtype),
                      rows_span(bias, 1, dim, dim, wdtype)};
  const Span out[3] = {rows_span(y, rows, dim, y_ld, dtype), {mean, mean ? rows * 4 : 0}, {rstd, rstd ? rows * 4 : 0}};
  for (int i = 0; i < 3; ++i)
    if (any_overlap(out[i], in, 3) || any_overlap(out[i], out, i)) return ZS_ERR_OVERLAP;
  return launch([&] {
    return zs::launch_layer_norm_forward(x, dtype, x_ld, weight, bias, wdtype, rows, dim, (float)eps, y, y_ld, mean,
                                         rstd, stream);
  });
}

size_t zs_layer_norm_workspace_bytes(int64_t rows, int64_t dim) {
  if (!count_ok(rows) || !dim_ok(dim)) return 0;
  const zs::LnPlan p = zs::ln_plan(rows, dim);
  return (size_t)(2 * p.parts * p.pitch) * sizeof(float);
}

zs_status zs_layer_norm_backward(const void* dy, int64_t dy_ld, const void* x, int64_t x_ld,
                                 int32_t dtype, const void* weight, int32_t wdtype, const float* mean,
                                 const float* rstd, int64_t rows, int64_t dim, void* dx, int64_t dx_ld,
                                 void* dweight, void* dbias, int32_t grad_dtype, int32_t first,
                                 void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (!float_type(dtype) || !float_type(wdtype) || !float_type(grad_dtype)) return ZS_ERR_DTYPE;
  if (!count_ok(rows) || !dim_ok(dim) || (rows > 0 && dim < 1)) return ZS_ERR_SIZE;
  if (!stride_ok(rows, dim, dy_ld) || !stride_ok(rows, dim, x_ld) || !stride_ok(rows, dim, dx_ld)) return ZS_ERR_SIZE;
  const bool grads = dweight || dbias;
  if (dim == 0 || (rows == 0 && (!grads || !first))) return ZS_OK;
  if (rows > 0 && (!dy || !x || !mean || !rstd || !dx)) return ZS_ERR_NULL;
  const uintptr_t es = (uintptr_t)elem_size(dtype), gs = (uintptr_t)elem_size(grad_dtype);
  if (rows > 0 && (!aligned(dy, es) || !aligned(x, es) || !aligned(dx, es) || !aligned(mean, 4) || !aligned(rstd, 4) ||
                   !aligned(weight, (uintptr_t)elem_size(wdtype))))
    return ZS_ERR_ALIGN;
  if (!aligned(dweight, gs) || !aligned(dbias, gs)) return ZS_ERR_ALIGN;
  const size_t need = grads ? zs_layer_norm_workspace_bytes(rows, dim) : 0;
  if (need > 0) {
    if (!workspace || workspace_bytes < need) return ZS_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return ZS_ERR_ALIGN;
  }
  const Span in[5] = {rows_span(dy, rows, dim, dy_ld, dtype), rows_span(x, rows, dim, x_ld, dtype),
                      rows_span(weight, rows > 0, dim, dim, wdtype), {mean, rows * 4}, {rstd, rows * 4}};
  const Span out[4] = {rows_span(dx, rows, dim, dx_ld, dtype), rows_span(dweight, 1, dim, dim, grad_dtype),
                       rows_span(dbias, 1, dim, dim, grad_dtype),
                       {workspace, (int64_t)need}};
  for (int i = 0; i < 4; ++i)
    if (any_overlap(out[i], in, 5) || any_overlap(out[i], out, i)) return ZS_ERR_OVERLAP;
  return launch([&] {
    return zs::launch_layer_norm_backward(dy, dy_ld, x, x_ld, dtype, weight, wdtype, mean, rstd, rows, dim, dx, dx_ld,
                                          dweight, dbias, grad_dtype, first != 0, workspace, stream);
  });
}

zs_status zs_activation_pack(const void* x, int32_t dtype, int64_t x_ld, int64_t rows, int64_t dim,
                             uint8_t* codes, int64_t codes_ld, float* scales, int64_t scales_ld,
                             hipStream_t stream) {
  if (!float_type(dtype)) return ZS_ERR_DTYPE;
  if (!count_ok(rows) || !dim_ok(dim)) return ZS_ERR_SIZE;
  if (!stride_ok(rows, dim, x_ld) || !codes_size_ok(rows, dim, codes_ld, scales_ld)) return ZS_ERR_SIZE;
  if (rows == 0 || dim == 0) return ZS_OK;
  if (!x || !codes || !scales) return ZS_ERR_NULL;
  if (!aligned(x, (uintptr_t)elem_size(dtype)) || !aligned(scales, 4)) return ZS_ERR_ALIGN;
  const Span in = rows_span(x, rows, dim, x_ld, dtype), c = codes_span(codes, rows, dim, codes_ld),
             sc = scales_span(scales, rows, dim, scales_ld);
  if (any_overlap(c, &in, 1) || any_overlap(sc, &in, 1) || any_overlap(sc, &c, 1)) return ZS_ERR_OVERLAP;
  return launch([&] {
    return zs::launch_activation_pack(x, dtype, x_ld, rows, dim, codes, codes_ld, scales, scales_ld, stream);
  });
}

zs_status zs_activation_unpack(const uint8_t* codes, int64_t codes_ld, const float* scales,
                               int64_t scales_ld, int64_t rows, int64_t dim, void* out, int32_t dtype,
                               int64_t out_ld, hipStream_t stream) {
  if (!float_type(dtype)) return ZS_ERR_DTYPE;
  if (!count_ok(rows) || !dim_ok(dim)) return ZS_ERR_SIZE;
  if (!stride_ok(rows, dim, out_ld) || !codes_size_ok(rows, dim, codes_ld, scales_ld)) return ZS_ERR_SIZE;
  if (rows == 0 || dim == 0) return ZS_OK;
  if (!codes || !scales || !out) return ZS_ERR_NULL;
  if (!aligned(out, (uintptr_t)elem_size(dtype)) || !aligned(scales, 4)) return ZS_ERR_ALIGN;
  const Span in[2] = {codes_span(codes, rows, dim, codes_ld), scales_span(scales, rows, dim, scales_ld)};
  if (any_overlap(rows_span(out, rows, dim, out_ld, dtype), in, 2)) return ZS_ERR_OVERLAP;
  return launch([&] {
    return zs::launch_activation_unpack(codes, codes_ld, scales, scales_ld, rows, dim, out, dtype, out_ld, stream);
  });
}

zs_status zs_rms_norm_forward(const void* x, int32_t dtype, int64_t x_ld, const void* residual,
                              int64_t residual_ld, void* sum, int64_t sum_ld, int32_t sum_dtype,
                              const void* weight, int32_t wdtype, int64_t rows, int64_t dim, double eps,
                              void* y, int64_t y_ld, uint8_t* codes, int64_t codes_ld, float* scales,
                              int64_t scales_ld, float* rstd, hipStream_t stream) {
  if (!float_type(dtype) || !float_type(wdtype) || (residual && !stream_type_ok(dtype, sum_dtype))) return ZS_ERR_DTYPE;
  if (!count_ok(rows) || !dim_ok(dim) || (rows > 0 && dim < 1)) return ZS_ERR_SIZE;
  if (!stride_ok(rows, dim, x_ld) || (residual && !stride_ok(rows, dim, residual_ld)) ||
      (sum && !stride_ok(rows, dim, sum_ld)) || (y && !stride_ok(rows, dim, y_ld)) ||
      (codes && !codes_size_ok(rows, dim, codes_ld, scales_ld)))
    return ZS_ERR_SIZE;
  if (!std::isfinite((float)eps) || eps < 0) return ZS_ERR_HPARAM;
  if (rows == 0) return ZS_OK;
  if (!x || (!y && !codes) || (sum && !residual) || (codes == nullptr) != (scales == nullptr)) return ZS_ERR_NULL;
  const uintptr_t es = (uintptr_t)elem_size(dtype), rs = (uintptr_t)elem_size(sum_dtype);
  if (!aligned(x, es) || !aligned(y, es) || !aligned(weight, (uintptr_t)elem_size(wdtype)) || !aligned(scales, 4) ||
      !aligned(rstd, 4) || (residual && (!aligned(residual, rs) || !aligned(sum, rs))))
    return ZS_ERR_ALIGN;
  const Span in[3] = {rows_span(x, rows, dim, x_ld, dtype), rows_span(residual, rows, dim, residual_ld, sum_dtype),
                      rows_span(weight, 1, dim, dim, wdtype)};
  const Span out[5] = {rows_span(sum, rows, dim, sum_ld, sum_dtype), rows_span(y, rows, dim, y_ld, dtype),
                       codes_span(codes, rows, dim, codes_ld), scales_span(scales, rows, dim, scales_ld),
                       {rstd, rstd ? rows * 4 : 0}};
  // the sum may take the place of what it is made from: each element is read by the lane that writes it
  const bool on_x = sum == x && sum_ld == x_ld && sum_dtype == dtype, on_residual = sum == residual && sum_ld == residual_ld;
  if ((!on_x && any_overlap(out[0], &in[0], 1)) || (!on_residual && any_overlap(out[0], &in[1], 1)) ||
      any_overlap(out[0], &in[2], 1))
    return ZS_ERR_OVERLAP;
  for (int i = 1; i < 5; ++i)
    if (any_overlap(out[i], in, 3) || any_overlap(out[i], out, i)) return ZS_ERR_OVERLAP;
  return launch([&] {
    return zs::launch_rms_norm_forward(x, dtype, x_ld, residual, residual_ld, sum, sum_ld, residual ? sum_dtype : dtype,
                                       weight, wdtype, rows, dim, (float)eps, y, y_ld, codes, codes_ld, scales,
                                       scales_ld, rstd, stream);
  });
}

size_t zs_rms_norm_workspace_bytes(int64_t rows, int64_t dim) {
  if (!count_ok(rows) || !dim_ok(dim)) return 0;
  const zs::RmsPlan p = zs::rms_plan(rows, dim);
  return (size_t)(p.parts * p.pitch) * sizeof(float);
}

zs_status zs_rms_norm_backward(const void* dy, int32_t dtype, int64_t dy_ld, const void* h,
                               int32_t h_dtype, int64_t h_ld, const float* scales, int64_t scales_ld,
                               const void* weight, int32_t wdtype, const float* rstd, const void* dres,
                               int64_t dres_ld, int64_t rows, int64_t dim, void* dh, int64_t dh_ld,
                               int32_t dh_dtype, void* dweight, int32_t grad_dtype, int32_t first,
                               void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const bool kept8 = h_dtype == ZS_E4M3;
  if (!float_type(dtype) || !float_type(wdtype) || !float_type(grad_dtype) || !stream_type_ok(dtype, dh_dtype) ||
      (!kept8 && h_dtype != dh_dtype))
    return ZS_ERR_DTYPE;
  if (!count_ok(rows) || !dim_ok(dim) || (rows > 0 && dim < 1)) return ZS_ERR_SIZE;
  if (!stride_ok(rows, dim, dy_ld) || !stride_ok(rows, dim, h_ld) || !stride_ok(rows, dim, dh_ld) ||
      (kept8 && !stride_ok(rows, scale_blocks(dim), scales_ld)) || (dres && !stride_ok(rows, dim, dres_ld)))
    return ZS_ERR_SIZE;
  if (dim == 0 || (rows == 0 && (!dweight || !first))) return ZS_OK;
  if (rows > 0 && (!dy || !h || !rstd || !dh || (kept8 && !scales))) return ZS_ERR_NULL;
  const uintptr_t es = (uintptr_t)elem_size(dtype), rs = (uintptr_t)elem_size(dh_dtype);
  if (rows > 0 && (!aligned(dy, es) || !aligned(h, kept8 ? 1 : rs) || !aligned(dh, rs) || !aligned(dres, rs) ||
                   !aligned(rstd, 4) || (kept8 && !aligned(scales, 4)) ||
                   !aligned(weight, (uintptr_t)elem_size(wdtype))))
    return ZS_ERR_ALIGN;
  if (!aligned(dweight, (uintptr_t)elem_size(grad_dtype))) return ZS_ERR_ALIGN;
  const size_t need = dweight ? zs_rms_norm_workspace_bytes(rows, dim) : 0;
  if (need > 0) {
    if (!workspace || workspace_bytes < need) return ZS_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return ZS_ERR_ALIGN;
  }
  const Span in[6] = {rows_span(dres, rows, dim, dres_ld, dh_dtype), rows_span(dy, rows, dim, dy_ld, dtype),
                      kept8 ? codes_span(h, rows, dim, h_ld) : rows_span(h, rows, dim, h_ld, dh_dtype),
                      scales_span(kept8 ? scales : nullptr, rows, dim, scales_ld),
                      rows_span(weight, rows > 0, dim, dim, wdtype), {rstd, rows * 4}};
  const Span out[3] = {rows_span(dh, rows, dim, dh_ld, dh_dtype), rows_span(dweight, 1, dim, dim, grad_dtype),
                       {workspace, (int64_t)need}};
  for (int i = 0; i < 3; ++i) {
    const int skip = i == 0 && dh == dres && dh_ld == dres_ld ? 1 : 0;  // in place: read by the lane that writes
    if (any_overlap(out[i], in + skip, 6 - skip) || any_overlap(out[i], out, i)) return ZS_ERR_OVERLAP;
  }
  return launch([&] {
    return zs::launch_rms_norm_backward(dy, dtype, dy_ld, h, h_dtype, h_ld, scales, scales_ld, weight, wdtype, rstd, dres,
                                        dres_ld, rows, dim, dh, dh_ld, dh_dtype, dweight, grad_dtype, first != 0,
                                        workspace, stream);
  });
}

size_t zs_linear_cross_entropy_workspace_bytes(int64_t n, int64_t vocab, int64_t dim, int32_t dtype,
                                               int32_t grad_dtype) {
  if (!float_type(dtype) || (grad_dtype != -1 && !float_type(grad_dtype)) || !head_size_ok(n, vocab, dim)) return 0;
  return (size_t)zs::head_plan(n, vocab, dim, dtype, grad_dtype).bytes;
}

zs_status zs_linear_cross_entropy_forward(const void* hidden, int64_t hidden_ld, int32_t dtype,
                                          const void* weight, int64_t weight_ld, const void* labels,
                                          int32_t index_type, int64_t n, int64_t vocab, int64_t dim,
                                          float* loss, float* lse, void* workspace,
                                          size_t workspace_bytes, hipStream_t stream) {
  if (!float_type(dtype) || !index_type_ok(index_type)) return ZS_ERR_DTYPE;
  if (!head_size_ok(n, vocab, dim) || (n > 0 && dim < 1)) return ZS_ERR_SIZE;
  if (!stride_ok(n, dim, hidden_ld) || !stride_ok(vocab, dim, weight_ld)) return ZS_ERR_SIZE;
  if (n == 0) return ZS_OK;
  if (!hidden || (vocab > 0 && !weight) || !labels || !loss) return ZS_ERR_NULL;
  const uintptr_t es = (uintptr_t)elem_size(dtype), is = (uintptr_t)index_size(index_type);
  if (!aligned(hidden, es) || !aligned(weight, es) || !aligned(labels, is) || !aligned(loss, 4) || !aligned(lse, 4))
    return ZS_ERR_ALIGN;
  const size_t need = zs_linear_cross_entropy_workspace_bytes(n, vocab, dim, dtype, -1);
  if (!workspace || workspace_bytes < need) return ZS_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return ZS_ERR_ALIGN;
  const Span in[3] = {rows_span(hidden, n, dim, hidden_ld, dtype), rows_span(weight, vocab, dim, weight_ld, dtype),
                      {labels, n * (int64_t)is}};
  const Span out[3] = {{loss, n * 4}, {lse, lse ? n * 4 : 0}, {workspace, (int64_t)need}};
  for (int i = 0; i < 3; ++i)
    if (any_overlap(out[i], in, 3) || any_overlap(out[i], out, i)) return ZS_ERR_OVERLAP;
  return launch([&] {
    return zs::launch_head_forward(hidden, hidden_ld, dtype, weight, weight_ld, labels, index_type, n, vocab, dim, loss,
                                   lse, workspace, stream);
  });
}

zs_status zs_linear_cross_entropy_backward(const void* hidden, int64_t hidden_ld, int32_t dtype,
                                           const void* weight, int64_t weight_ld, const void* labels,
                                           int32_t index_type, const float* lse, const float* dloss,
                                           float scale, int64_t n, int64_t vocab, int64_t dim,
                                           void* dhidden, int64_t dhidden_ld, void* dweight,
                                           int32_t grad_dtype, int64_t dweight_ld, int32_t first,
                                           void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (!float_type(dtype) || !float_type(grad_dtype) || !index_type_ok(index_type)) return ZS_ERR_DTYPE;
  if (!head_size_ok(n, vocab, dim) || (n > 0 && dim < 1)) return ZS_ERR_SIZE;
  if (!stride_ok(n, dim, hidden_ld) || !stride_ok(vocab, dim, weight_ld) || !stride_ok(n, dim, dhidden_ld) ||
      !stride_ok(vocab, dim, dweight_ld))
    return ZS_ERR_SIZE;
  if (!std::isfinite(scale)) return ZS_ERR_HPARAM;
  if (n == 0 && (!first || vocab == 0 || dim == 0)) return ZS_OK;
  if ((n > 0 && (!hidden || !labels || !lse || !dhidden)) || (vocab > 0 && (!weight || !dweight))) return ZS_ERR_NULL;
  const uintptr_t es = (uintptr_t)elem_size(dtype), is = (uintptr_t)index_size(index_type);
  if (!aligned(hidden, es) || !aligned(weight, es) || !aligned(dhidden, es) || !aligned(labels, is) ||
      !aligned(lse, 4) || !aligned(dloss, 4) || !aligned(dweight, (uintptr_t)elem_size(grad_dtype)))
    return ZS_ERR_ALIGN;
  const bool scratch = n > 0 && vocab > 0;  // otherwise zeros are written, and nothing else
  const size_t need = scratch ? zs_linear_cross_entropy_workspace_bytes(n, vocab, dim, dtype, grad_dtype) : 0;
  if (scratch && (!workspace || workspace_bytes < need)) return ZS_ERR_WORKSPACE;
  if (scratch && !aligned(workspace, 16)) return ZS_ERR_ALIGN;
  const Span in[5] = {rows_span(hidden, n, dim, hidden_ld, dtype), rows_span(weight, vocab, dim, weight_ld, dtype),
                      {labels, n * (int64_t)is}, {lse, n * 4}, {dloss, dloss ? n * 4 : 0}};
  const Span out[3] = {rows_span(dhidden, n, dim, dhidden_ld, dtype),
                       rows_span(dweight, vocab, dim, dweight_ld, grad_dtype), {workspace, (int64_t)need}};
  for (int i = 0; i < 3; ++i)
    if (any_overlap(out[i], in, 5) || any_overlap(out[i], out, i)) return ZS_ERR_OVERLAP;
  return launch([&] {
    return zs::launch_head_backward(hidden, hidden_ld, dtype, weight, weight_ld, labels, index_type, lse, dloss, scale,
                                    n, vocab, dim, dhidden, dhidden_ld, dweight, grad_dtype, dweight_ld, first != 0,
                                    workspace, stream);
  });
}

}  // extern "C"
