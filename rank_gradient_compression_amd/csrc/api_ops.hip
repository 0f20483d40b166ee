// C ABI entry points of the gradient clip and of the microscaled 4-bit
// operands.  Argument checks on the host, then launches on the caller's
// stream: no allocation on the device and no synchronisation.

#include <hip/hip_runtime.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>
#include <new>
#include <vector>

#include "psgd_clip.h"
#include "psgd_internal.h"
#include "psgd_kernels.h"
#include "psgd_mx.h"

namespace psgd {

static_assert(kF32 == PSGD_DTYPE_F32 && kBF16 == PSGD_DTYPE_BF16 && kF16 == PSGD_DTYPE_F16, "element types");

static bool known_dtype(int32_t d) { return d == kF32 || d == kBF16 || d == kF16; }
static bool misaligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) != 0; }

static psgd_status_t invalid(const char* fn, const char* what) {
  set_error("%s: %s", fn, what);
  return PSGD_ERR_INVALID_ARG;
}

static psgd_status_t launch_status(hipError_t e, const char* fn) {
  if (e == hipSuccess) return PSGD_OK;
  set_error("%s: %s", fn, hipGetErrorString(e));
  return PSGD_ERR_HIP;
}

// Byte ranges [p, p + n) of two buffers share a byte.
static bool overlap(const void* p, size_t n, const void* q, size_t m) {
  const uintptr_t a = (uintptr_t)p, b = (uintptr_t)q;
  return n && m && a < b + m && b < a + n;
}

static size_t strided_bytes(int64_t rows, int64_t cols, int64_t ld, int32_t dtype) {
  return rows && cols ? ((size_t)(rows - 1) * (size_t)ld + (size_t)cols) * dtype_bytes(dtype) : 0;
}

constexpr int64_t kMaxDim = INT32_MAX;
constexpr int64_t kMaxGrid = INT32_MAX;

static bool bad_dim(int64_t d) { return d < 0 || d > kMaxDim; }

static psgd_status_t check_operand(const char* fn, const uint8_t* codes, const uint8_t* scales, int64_t rows,
                                   int64_t cols) {
  if (rows == 0 || cols == 0) return PSGD_OK;
  if (!codes || !scales) return invalid(fn, "an operand's codes or scales are NULL");
  if (misaligned(codes, 16) || misaligned(scales, 16)) return invalid(fn, "codes and scales must be 16-byte aligned");
  return PSGD_OK;
}

static psgd_status_t check_strided(const char* fn, const void* p, int32_t dtype, int64_t rows, int64_t cols,
                                   int64_t ld) {
  if (!known_dtype(dtype)) return invalid(fn, "unknown element type");
  if (bad_dim(rows) || bad_dim(cols)) return invalid(fn, "a size is negative or above INT32_MAX");
  if (rows > 1 && (ld < cols || ld > kMaxDim)) return invalid(fn, "the row stride is smaller than the row or above INT32_MAX");
  if (rows && cols && !p) return invalid(fn, "a required buffer is NULL");
  if (misaligned(p, dtype_bytes(dtype))) return invalid(fn, "a buffer is not aligned to its element type");
  return PSGD_OK;
}

}  // namespace psgd

using namespace psgd;

// ---------------------------------------------------------------- the clip

extern "C" psgd_status_t psgd_clip_create(int32_t ntensors, const int64_t* numel, const int32_t* in_dtypes,
                                          const int32_t* out_dtypes, psgd_clip_t* out) {
  clear_error();
  const char* fn = "psgd_clip_create";
  if (!out) return invalid(fn, "out is NULL");
  *out = nullptr;
  if (ntensors < 0 || (ntensors > 0 && (!numel || !in_dtypes || !out_dtypes)))
    return invalid(fn, "negative tensor count or a NULL list");
  int64_t total = 0;
  for (int32_t t = 0; t < ntensors; ++t) {
    if (numel[t] < 0 || numel[t] > (int64_t(1) << 46)) return invalid(fn, "a tensor's size is negative or too large");
    if (!known_dtype(in_dtypes[t]) || !known_dtype(out_dtypes[t])) return invalid(fn, "unknown element type");
    total += numel[t];
    if (total > (int64_t(1) << 46)) return invalid(fn, "the set is too large");
  }
  psgd_clip* c = nullptr;
  try {
    c = new psgd_clip;
    c->tensors.resize((size_t)ntensors);
    int64_t nsums = 0, nchunks = 0, bytes_in = 0, bytes_out = 0;
    for (int32_t t = 0; t < ntensors; ++t) {
      const int64_t n = numel[t], chunks = (n + kClipChunk - 1) / kClipChunk;
      // its share of the norm's workgroups, by size
      const int64_t share = n == 0 ? 0 : (int64_t)((double)n / (double)total * kClipSumGroups) + 1;
      const int64_t groups = std::min(chunks, share);
      if (nchunks + chunks > kMaxGrid) {
        delete c;
        return invalid(fn, "the set is too large");
      }
      c->tensors[(size_t)t] = ClipTensor{nullptr,          nullptr,         n, in_dtypes[t], out_dtypes[t],
                                         (int32_t)nsums, (int32_t)groups, (int32_t)nchunks, 0};
      c->sum_map.insert(c->sum_map.end(), (size_t)groups, t);
      c->chunk_map.insert(c->chunk_map.end(), (size_t)chunks, t);
      nsums += groups;
      nchunks += chunks;
      bytes_in += n * dtype_bytes(in_dtypes[t]);
      bytes_out += n * dtype_bytes(out_dtypes[t]);
    }
    c->stream_in = bytes_in > kStreamHintBytes;
    c->stream_out = bytes_in + bytes_out > kClipCacheBytes;
    auto up = [](size_t b) { return (b + 255) / 256 * 256; };
    c->lay.sum_map_off = up(c->tensors.size() * sizeof(ClipTensor));
    c->lay.chunk_map_off = c->lay.sum_map_off + up(c->sum_map.size() * sizeof(int32_t));
    c->lay.sums_off = c->lay.chunk_map_off + up(c->chunk_map.size() * sizeof(int32_t));
    c->lay.bytes = std::max<size_t>(256, c->lay.sums_off + up(c->sum_map.size() * sizeof(double)));
    c->tables.assign(c->lay.sums_off, 0);
    auto put = [&](size_t off, const void* p, size_t n) {
      if (n) memcpy(c->tables.data() + off, p, n);
    };
    put(0, c->tensors.data(), c->tensors.size() * sizeof(ClipTensor));
    put(c->lay.sum_map_off, c->sum_map.data(), c->sum_map.size() * sizeof(int32_t));
    put(c->lay.chunk_map_off, c->chunk_map.data(), c->chunk_map.size() * sizeof(int32_t));
  } catch (const std::bad_alloc&) {
    delete c;
    return invalid(fn, "out of host memory");
  }
  *out = c;
  return PSGD_OK;
}

extern "C" void psgd_clip_destroy(psgd_clip_t c) { delete c; }

extern "C" psgd_status_t psgd_clip_workspace(psgd_clip_t c, size_t* bytes) {
  clear_error();
  if (!c || !bytes) return invalid("psgd_clip_workspace", "NULL argument");
  *bytes = c->lay.bytes;
  return PSGD_OK;
}

static psgd_status_t check_clip_ws(const char* fn, const psgd_clip* c, const void* ws, size_t bytes) {
  if (!c) return invalid(fn, "clip is NULL");
  if (!ws || misaligned(ws, 256) || bytes < c->lay.bytes) {
    set_error("%s: the workspace must be %zu bytes, 256-byte aligned", fn, c->lay.bytes);
    return PSGD_ERR_WORKSPACE;
  }
  return PSGD_OK;
}

extern "C" psgd_status_t psgd_clip_workspace_init(psgd_clip_t c, void* ws, size_t bytes, hipStream_t stream) {
  clear_error();
  const char* fn = "psgd_clip_workspace_init";
  if (psgd_status_t s = check_clip_ws(fn, c, ws, bytes)) return s;
  if (c->tables.empty()) return PSGD_OK;
  return launch_status(hipMemcpyAsync(ws, c->tables.data(), c->tables.size(), hipMemcpyHostToDevice, stream), fn);
}

extern "C" psgd_status_t psgd_clip_bind(psgd_clip_t c, const void* const* in, void* const* out, void* ws, size_t bytes,
                                        hipStream_t stream) {
  clear_error();
  const char* fn = "psgd_clip_bind";
  if (psgd_status_t s = check_clip_ws(fn, c, ws, bytes)) return s;
  const int n = (int)c->tensors.size();
  if (n > 0 && !in) return invalid(fn, "in is NULL");
  try {
    struct Range {
      uintptr_t b, e;
      int t;
    };
    std::vector<Range> outs;
    for (int t = 0; t < n; ++t) {
      const ClipTensor& d = c->tensors[(size_t)t];
      if (d.numel == 0) continue;
      if (!in[t] || misaligned(in[t], dtype_bytes(d.in_dtype)))
        return invalid(fn, "a gradient pointer is NULL or not aligned to its element type");
      if (!out) continue;
      if (!out[t] || misaligned(out[t], dtype_bytes(d.out_dtype)))
        return invalid(fn, "an output pointer is NULL or not aligned to its element type");
      const uintptr_t b = (uintptr_t)out[t];
      outs.push_back({b, b + (uintptr_t)d.numel * dtype_bytes(d.out_dtype), t});
    }
    std::sort(outs.begin(), outs.end(), [](const Range& x, const Range& y) { return x.b < y.b; });
    for (size_t i = 1; i < outs.size(); ++i)
      if (outs[i].b < outs[i - 1].e) return invalid(fn, "two outputs overlap");
    for (int t = 0; t < n && !outs.empty(); ++t) {
      const ClipTensor& d = c->tensors[(size_t)t];
      if (d.numel == 0) continue;
      const uintptr_t b = (uintptr_t)in[t], e = b + (uintptr_t)d.numel * dtype_bytes(d.in_dtype);
      // the outputs are disjoint and sorted: the first that ends after b
      auto it = std::upper_bound(outs.begin(), outs.end(), b, [](uintptr_t v, const Range& r) { return v < r.e; });
      for (; it != outs.end() && it->b < e; ++it)
        if (it->t != t || it->b != b || dtype_bytes(d.in_dtype) != dtype_bytes(d.out_dtype))
          return invalid(fn, "an output overlaps a gradient other than being its own gradient in place");
    }
  } catch (const std::bad_alloc&) {
    return invalid(fn, "out of host memory");
  }
  ClipTensor* dev = static_cast<ClipTensor*>(ws);
  for (int f = 0; f < n; f += kClipBindPairs) {
    const int m = std::min(kClipBindPairs, n - f);
    ClipPointers p{};
    for (int i = 0; i < m; ++i) {
      p.in[i] = in[f + i];
      p.out[i] = out ? out[f + i] : nullptr;
    }
    if (psgd_status_t s = launch_status(launch_clip_bind(dev, p, f, m, stream), fn)) return s;
  }
  return PSGD_OK;
}

static ClipArgs clip_args(const psgd_clip* c, void* ws, float scale, float max_norm, float* stats) {
  char* b = static_cast<char*>(ws);
  ClipArgs a{};
  a.tensors = reinterpret_cast<const ClipTensor*>(b);
  a.sum_map = reinterpret_cast<const int32_t*>(b + c->lay.sum_map_off);
  a.chunk_map = reinterpret_cast<const int32_t*>(b + c->lay.chunk_map_off);
  a.sums = reinterpret_cast<double*>(b + c->lay.sums_off);
  a.ntensors = (int32_t)c->tensors.size();
  a.nsums = (int32_t)c->sum_map.size();
  a.nchunks = (int32_t)c->chunk_map.size();
  a.stream_in = c->stream_in;
  a.stream_out = c->stream_out;
  a.scale = scale;
  a.max_norm = max_norm;
  a.stats = stats;
  return a;
}

static psgd_status_t check_clip_call(const char* fn, const psgd_clip* c, float max_norm, float scale, float* stats,
                                     const void* ws, size_t bytes) {
  if (psgd_status_t s = check_clip_ws(fn, c, ws, bytes)) return s;
  if (!stats || misaligned(stats, 4)) return invalid(fn, "stats is NULL or misaligned");
  if (!(scale - scale == 0.f)) return invalid(fn, "scale is not finite");
  if (!(max_norm >= 0.f)) return invalid(fn, "max_norm is negative or NaN");
  return PSGD_OK;
}

extern "C" psgd_status_t psgd_clip_norm(psgd_clip_t c, float max_norm, float scale, float* stats, void* ws,
                                        size_t bytes, hipStream_t stream) {
  clear_error();
  const char* fn = "psgd_clip_norm";
  if (psgd_status_t s = check_clip_call(fn, c, max_norm, scale, stats, ws, bytes)) return s;
  return launch_status(launch_clip_norm(clip_args(c, ws, scale, max_norm, stats), stream), fn);
}

extern "C" psgd_status_t psgd_clip_apply(psgd_clip_t c, float max_norm, float scale, float* stats, void* ws,
                                         size_t bytes, hipStream_t stream) {
  clear_error();
  const char* fn = "psgd_clip_apply";
  if (psgd_status_t s = check_clip_call(fn, c, max_norm, scale, stats, ws, bytes)) return s;
  const ClipArgs a = clip_args(c, ws, scale, max_norm, stats);
  return launch_status(launch_clip_apply(a, stream), fn);
}

// ------------------------------------------------ microscaled 4-bit operands

extern "C" psgd_status_t psgd_mx_sizes(int64_t rows, int64_t cols, size_t* code_bytes, size_t* scale_bytes) {
  clear_error();
  if (bad_dim(rows) || bad_dim(cols) || !code_bytes || !scale_bytes)
    return invalid("psgd_mx_sizes", "a size is negative or above INT32_MAX, or an output is NULL");
  *code_bytes = (size_t)(rows * mx_pitch(cols));
  *scale_bytes = (size_t)mx_scale_bytes(rows, cols);
  return PSGD_OK;
}

extern "C" psgd_status_t psgd_mx_quantize(const void* x, int32_t dtype, int64_t rows, int64_t cols, int64_t ld,
                                          const uint8_t* rand, uint8_t* row_codes, uint8_t* row_scales,
                                          uint8_t* col_codes, uint8_t* col_scales, void* values, int64_t ldv,
                                          hipStream_t stream) {
  clear_error();
  const char* fn = "psgd_mx_quantize";
  if (psgd_status_t s = check_strided(fn, x, dtype, rows, cols, ld)) return s;
  if ((row_codes != nullptr) != (row_scales != nullptr) || (col_codes != nullptr) != (col_scales != nullptr))
    return invalid(fn, "an operand's codes and scales must be given together");
  if (rows == 0 || cols == 0) return PSGD_OK;
  if (!row_codes && !col_codes && !values) return invalid(fn, "no output is wanted");
  if (row_codes)
    if (psgd_status_t s = check_operand(fn, row_codes, row_scales, rows, cols)) return s;
  if (col_codes)
    if (psgd_status_t s = check_operand(fn, col_codes, col_scales, cols, rows)) return s;
  const size_t xb = strided_bytes(rows, cols, ld, dtype);
  if (values) {
    if (psgd_status_t s = check_strided(fn, values, dtype, rows, cols, ldv)) return s;
    const bool in_place = values == x && (ldv == ld || rows == 1);
    if (!in_place && overlap(x, xb, values, strided_bytes(rows, cols, ldv, dtype)))
      return invalid(fn, "values overlaps x without being x in place");
    if (rand && overlap(rand, (size_t)(rows * cols), values, strided_bytes(rows, cols, ldv, dtype)))
      return invalid(fn, "values overlaps rand");
  }
  const void* outs[] = {row_codes, row_scales, col_codes, col_scales};
  const size_t sizes[] = {(size_t)(rows * mx_pitch(cols)), (size_t)mx_scale_bytes(rows, cols),
                          (size_t)(cols * mx_pitch(rows)), (size_t)mx_scale_bytes(cols, rows)};
  for (int i = 0; i < 4; ++i) {
    if (!outs[i]) continue;
    if (overlap(outs[i], sizes[i], x, xb) || (rand && overlap(outs[i], sizes[i], rand, (size_t)(rows * cols))) ||
        (values && overlap(outs[i], sizes[i], values, strided_bytes(rows, cols, ldv, dtype))))
      return invalid(fn, "codes or scales overlap another buffer");
    for (int j = 0; j < i; ++j)
      if (outs[j] && overlap(outs[i], sizes[i], outs[j], sizes[j])) return invalid(fn, "two outputs overlap");
  }
  if (((rows + 127) / 32) * (mx_chunks(cols) + 1) > kMaxGrid) return invalid(fn, "the matrix is too large");
  MxQuantArgs a{x, dtype, rows, cols, rows > 1 ? ld : cols, rand, row_codes, row_scales, col_codes, col_scales,
                values, rows > 1 ? ldv : cols};
  return launch_status(launch_mx_quantize(a, stream), fn);
}

extern "C" psgd_status_t psgd_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols,
                                            void* out, int32_t dtype, int64_t ld, hipStream_t stream) {
  clear_error();
  const char* fn = "psgd_mx_dequantize";
  if (psgd_status_t s = check_strided(fn, out, dtype, rows, cols, ld)) return s;
  if (psgd_status_t s = check_operand(fn, codes, scales, rows, cols)) return s;
  const size_t ob = strided_bytes(rows, cols, ld, dtype);
  if (overlap(out, ob, codes, (size_t)(rows * mx_pitch(cols))) ||
      overlap(out, ob, scales, (size_t)mx_scale_bytes(rows, cols)))
    return invalid(fn, "out overlaps the operand");
  if (((rows + 31) / 32) * mx_chunks(cols) > kMaxGrid) return invalid(fn, "the matrix is too large");
  return launch_status(launch_mx_dequantize(codes, scales, rows, cols, out, dtype, rows > 1 ? ld : cols, stream), fn);
}

static psgd_status_t check_product(const char* fn, int64_t m, int64_t n, int64_t k, const uint8_t* b_codes,
                                   const uint8_t* b_scales, const void* c, int32_t dtype, int64_t ldc) {
  if (bad_dim(k)) return invalid(fn, "a size is negative or above INT32_MAX");
  if (psgd_status_t s = check_strided(fn, c, dtype, m, n, ldc)) return s;
  if (m && psgd::check_operand(fn, b_codes, b_scales, n, k) != PSGD_OK) return PSGD_ERR_INVALID_ARG;
  const size_t cb = strided_bytes(m, n, ldc, dtype);
  if (overlap(c, cb, b_codes, (size_t)(n * mx_pitch(k))) || overlap(c, cb, b_scales, (size_t)mx_scale_bytes(n, k)))
    return invalid(fn, "the result overlaps an operand");
  if (((m + 31) / 32) * ((n + 31) / 32) > kMaxGrid / 4 || m * n / 256 > kMaxGrid / 2)
    return invalid(fn, "the product is too large");
  return PSGD_OK;
}

static psgd_status_t check_workspace(const char* fn, size_t need, const void* ws, size_t bytes) {
  if (need == 0) return PSGD_OK;
  if (!ws || misaligned(ws, 256) || bytes < need) {
    set_error("%s: the workspace must be %zu bytes, 256-byte aligned", fn, need);
    return PSGD_ERR_WORKSPACE;
  }
  return PSGD_OK;
}

extern "C" psgd_status_t psgd_mx_product(int64_t m, int64_t n, int64_t k, const uint8_t* a_codes,
                                         const uint8_t* a_scales, const uint8_t* b_codes, const uint8_t* b_scales,
                                         void* c, int32_t dtype, int64_t ldc, int32_t accumulate,
                                         hipStream_t stream) {
  clear_error();
  const char* fn = "psgd_mx_product";
  if (psgd_status_t s = check_product(fn, m, n, k, b_codes, b_scales, c, dtype, ldc)) return s;
  if (n)
    if (psgd_status_t s = check_operand(fn, a_codes, a_scales, m, k)) return s;
  const size_t cb = strided_bytes(m, n, ldc, dtype);
  if (overlap(c, cb, a_codes, (size_t)(m * mx_pitch(k))) || overlap(c, cb, a_scales, (size_t)mx_scale_bytes(m, k)))
    return invalid(fn, "the result overlaps an operand");
  const MxProductArgs p{m, n, k, {a_codes, a_scales}, {b_codes, b_scales}, c, dtype, m > 1 ? ldc : n, accumulate != 0};
  return launch_status(launch_mx_product(p, stream), fn);
}

// Operands in a workspace: codes, then scales, each from a multiple of 256 bytes on.
static size_t up256(size_t b) { return (b + 255) / 256 * 256; }
static size_t operand_bytes(int64_t rows, int64_t cols) {
  return up256((size_t)(rows * mx_pitch(cols))) + up256((size_t)mx_scale_bytes(rows, cols));
}
struct WsOperand {
  uint8_t *codes, *scales;
};
static WsOperand ws_operand(void* ws, size_t off, int64_t rows, int64_t cols) {
  uint8_t* codes = static_cast<uint8_t*>(ws) + off;
  return {codes, codes + up256((size_t)(rows * mx_pitch(cols)))};
}

static MxQuantArgs quant_args(const void* x, int32_t dtype, int64_t rows, int64_t cols, int64_t ld) {
  MxQuantArgs a{};
  a.x = x;
  a.dtype = dtype;
  a.rows = rows;
  a.cols = cols;
  a.ld = rows > 1 ? ld : cols;
  return a;
}

extern "C" psgd_status_t psgd_mx_linear_workspace(int64_t m, int64_t n, int64_t k, int32_t x_dtype, size_t* bytes) {
  clear_error();
  if (!known_dtype(x_dtype)) return invalid("psgd_mx_linear_workspace", "unknown element type");
  if (bad_dim(m) || bad_dim(n) || bad_dim(k) || !bytes)
    return invalid("psgd_mx_linear_workspace", "a size is negative or above INT32_MAX, or bytes is NULL");
  *bytes = mx_linear_fuses(m, n, k, x_dtype) ? 0 : operand_bytes(m, k);
  return PSGD_OK;
}

extern "C" psgd_status_t psgd_mx_linear(int64_t m, int64_t n, int64_t k, const void* x, int32_t x_dtype, int64_t ldx,
                                        const uint8_t* w_codes, const uint8_t* w_scales, void* y, int32_t y_dtype,
                                        int64_t ldy, void* ws, size_t bytes, hipStream_t stream) {
  clear_error();
  const char* fn = "psgd_mx_linear";
  if (psgd_status_t s = check_product(fn, m, n, k, w_codes, w_scales, y, y_dtype, ldy)) return s;
  if (psgd_status_t s = check_strided(fn, x, x_dtype, m, k, ldx)) return s;
  if (overlap(x, strided_bytes(m, k, ldx, x_dtype), y, strided_bytes(m, n, ldy, y_dtype)))
    return invalid(fn, "y overlaps x");
  MxProductArgs p{m, n, k, {nullptr, nullptr}, {w_codes, w_scales}, y, y_dtype, m > 1 ? ldy : n, false};
  if (mx_linear_fuses(m, n, k, x_dtype)) {
    if (m == 0 || n == 0) return PSGD_OK;
    return launch_status(launch_mx_linear_fused(p, x, x_dtype, m > 1 ? ldx : k, stream), fn);
  }
  const size_t need = operand_bytes(m, k);
  if (psgd_status_t s = check_workspace(fn, need, ws, bytes)) return s;
  if (overlap(ws, need, x, strided_bytes(m, k, ldx, x_dtype)) || overlap(ws, need, y, strided_bytes(m, n, ldy, y_dtype)) ||
      overlap(ws, need, w_codes, (size_t)(n * mx_pitch(k))) || overlap(ws, need, w_scales, (size_t)mx_scale_bytes(n, k)))
    return invalid(fn, "the workspace overlaps another buffer");
  if (m == 0 || n == 0) return PSGD_OK;
  const WsOperand q = ws_operand(ws, 0, m, k);
  MxQuantArgs a = quant_args(x, x_dtype, m, k, ldx);
  a.row_codes = q.codes;
  a.row_scales = q.scales;
  if (psgd_status_t s = launch_status(launch_mx_quantize(a, stream), fn)) return s;
  p.a = {q.codes, q.scales};
  return launch_status(launch_mx_product(p, stream), fn);
}

// -------------------------------------------------- the layer's training pass
extern "C" psgd_status_t psgd_mx_train_workspace(int64_t m, int64_t n, int64_t k, size_t* bytes) {
  clear_error();
  if (bad_dim(m) || bad_dim(n) || bad_dim(k) || !bytes)
    return invalid("psgd_mx_train_workspace", "a size is negative or above INT32_MAX, or bytes is NULL");
  *bytes = std::max(operand_bytes(m, k) + operand_bytes(n, k), operand_bytes(m, n) + operand_bytes(n, m));
  return PSGD_OK;
}

namespace {
struct Range {
  const void* p;
  size_t n;
};
Range codes_of(const uint8_t* codes, int64_t rows, int64_t cols) { return {codes, (size_t)(rows * mx_pitch(cols))}; }
Range scales_of(const uint8_t* scales, int64_t rows, int64_t cols) {
  return {scales, (size_t)mx_scale_bytes(rows, cols)};
}
// One of the first `nout` ranges shares a byte with another range.
template <int N>
bool outputs_overlap(const Range (&r)[N], int nout) {
  for (int i = 0; i < nout; ++i)
    for (int j = 0; j < N; ++j)
      if (i != j && r[i].p && r[j].p && overlap(r[i].p, r[i].n, r[j].p, r[j].n)) return true;
  return false;
}
}  // namespace

// Sizes whose tiles a launch can count, whichever of the three axes it spans.
static psgd_status_t check_train(const char* fn, int64_t m, int64_t n, int64_t k, const uint8_t* xt_codes,
                                 const uint8_t* xt_scales, const uint8_t* wt_codes, const uint8_t* wt_scales,
                                 const void* ws, size_t bytes) {
  if (bad_dim(m) || bad_dim(n) || bad_dim(k)) return invalid(fn, "a size is negative or above INT32_MAX");
  const int64_t sizes[3][2] = {{m, k}, {n, k}, {m, n}};
  for (const auto& s : sizes)
    if (((s[0] + 127) / 32) * ((s[1] + 127) / 32) > kMaxGrid / 4 || s[0] * s[1] / 256 > kMaxGrid / 2)
      return invalid(fn, "the layer is too large");
  if (m && k)
    if (psgd_status_t s = check_operand(fn, xt_codes, xt_scales, k, m)) return s;
  if (n && k)
    if (psgd_status_t s = check_operand(fn, wt_codes, wt_scales, k, n)) return s;
  size_t need;
  psgd_mx_train_workspace(m, n, k, &need);
  return check_workspace(fn, need, ws, bytes);
}

extern "C" psgd_status_t psgd_mx_train_forward(int64_t m, int64_t n, int64_t k, const void* x, int32_t x_dtype,
                                               int64_t ldx, const void* w, int32_t w_dtype, int64_t ldw,
                                               uint8_t* xt_codes, uint8_t* xt_scales, uint8_t* wt_codes,
                                               uint8_t* wt_scales, void* y, int32_t y_dtype, int64_t ldy, void* ws,
                                               size_t bytes, hipStream_t stream) {
  clear_error();
  const char* fn = "psgd_mx_train_forward";
  if (psgd_status_t s = check_train(fn, m, n, k, xt_codes, xt_scales, wt_codes, wt_scales, ws, bytes)) return s;
  if (psgd_status_t s = check_strided(fn, x, x_dtype, m, k, ldx)) return s;
  if (psgd_status_t s = check_strided(fn, w, w_dtype, n, k, ldw)) return s;
  if (psgd_status_t s = check_strided(fn, y, y_dtype, m, n, ldy)) return s;
  const Range r[] = {{y, strided_bytes(m, n, ldy, y_dtype)}, codes_of(xt_codes, k, m), scales_of(xt_scales, k, m),
                     codes_of(wt_codes, k, n),               scales_of(wt_scales, k, n), {ws, bytes},
                     {x, strided_bytes(m, k, ldx, x_dtype)}, {w, strided_bytes(n, k, ldw, w_dtype)}};
  if (outputs_overlap(r, 6)) return invalid(fn, "an output or the workspace overlaps another buffer");
  const WsOperand xr = ws_operand(ws, 0, m, k), wr = ws_operand(ws, operand_bytes(m, k), n, k);
  MxQuantArgs a = quant_args(x, x_dtype, m, k, ldx), b = quant_args(w, w_dtype, n, k, ldw);
  a.row_codes = xr.codes, a.row_scales = xr.scales, a.col_codes = xt_codes, a.col_scales = xt_scales;
  b.row_codes = wr.codes, b.row_scales = wr.scales, b.col_codes = wt_codes, b.col_scales = wt_scales;
  if (psgd_status_t s = launch_status(launch_mx_quantize_pair(a, b, stream), fn)) return s;
  const MxProductArgs p{m, n, k, {xr.codes, xr.scales}, {wr.codes, wr.scales}, y, y_dtype, m > 1 ? ldy : n, false};
  return launch_status(launch_mx_product(p, stream), fn);
}

extern "C" psgd_status_t psgd_mx_train_backward(int64_t m, int64_t n, int64_t k, const void* dy, int32_t dy_dtype,
                                                int64_t lddy, const uint8_t* rand, const uint8_t* xt_codes,
                                                const uint8_t* xt_scales, const uint8_t* wt_codes,
                                                const uint8_t* wt_scales, void* dx, int32_t dx_dtype, int64_t lddx,
                                                void* dw, int32_t dw_dtype, int64_t lddw, int32_t accumulate, void* ws,
                                                size_t bytes, hipStream_t stream) {
  clear_error();
  const char* fn = "psgd_mx_train_backward";
  if (psgd_status_t s = check_train(fn, m, n, k, xt_codes, xt_scales, wt_codes, wt_scales, ws, bytes)) return s;
  if (psgd_status_t s = check_strided(fn, dy, dy_dtype, m, n, lddy)) return s;
  if (dx)
    if (psgd_status_t s = check_strided(fn, dx, dx_dtype, m, k, lddx)) return s;
  if (dw)
    if (psgd_status_t s = check_strided(fn, dw, dw_dtype, n, k, lddw)) return s;
  const Range r[] = {{dx, strided_bytes(m, k, lddx, dx_dtype)},
                     {dw, strided_bytes(n, k, lddw, dw_dtype)},
                     {ws, bytes},
                     {dy, strided_bytes(m, n, lddy, dy_dtype)},
                     {rand, (size_t)(m * n)},
                     codes_of(xt_codes, k, m),
                     scales_of(xt_scales, k, m),
                     codes_of(wt_codes, k, n),
                     scales_of(wt_scales, k, n)};
  if (outputs_overlap(r, 3)) return invalid(fn, "an output or the workspace overlaps another buffer");
  if (!dx && !dw) return PSGD_OK;
  const WsOperand dr = ws_operand(ws, 0, m, n), dt = ws_operand(ws, operand_bytes(m, n), n, m);
  MxQuantArgs a = quant_args(dy, dy_dtype, m, n, lddy);
  a.rand = rand;
  if (dx) a.row_codes = dr.codes, a.row_scales = dr.scales;
  if (dw) a.col_codes = dt.codes, a.col_scales = dt.scales;
  if (psgd_status_t s = launch_status(launch_mx_quantize(a, stream), fn)) return s;
  if (dx) {
    const MxProductArgs p{m, k, n, {dr.codes, dr.scales}, {wt_codes, wt_scales}, dx, dx_dtype, m > 1 ? lddx : k, false};
    if (psgd_status_t s = launch_status(launch_mx_product(p, stream), fn)) return s;
  }
  if (!dw) return PSGD_OK;
  const MxProductArgs p{n, k, m, {dt.codes, dt.scales}, {xt_codes, xt_scales}, dw, dw_dtype, n > 1 ? lddw : k, accumulate != 0};
  return launch_status(launch_mx_product(p, stream), fn);
}
