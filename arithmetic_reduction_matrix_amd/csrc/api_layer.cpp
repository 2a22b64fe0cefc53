// The C entry points of the layer operators declared in include/armx.h: check
// arguments, make a plan, enqueue kernels on the caller's stream.  Nothing
// here allocates.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <initializer_list>

#include "armx.h"
#include "launch.h"
#include "layer.h"

namespace {

constexpr uint64_t kMaxElements = uint64_t(1) << 40;
constexpr uint64_t kMaxCols = uint64_t(1) << 30;     // exclusive: 32-bit byte offsets
constexpr uint64_t kMaxProductK = 131071;            // 131071 * 128 * 128 < 2^31
constexpr uint64_t kMaxProductLd = uint64_t(1) << 23;
constexpr uint64_t kMaxProductRows = uint64_t(1) << 30;
// tiles of 256 x 256, the largest, that a grid holds: threads are counted in 32 bits
constexpr uint64_t kMaxProductTiles = 0x7FFFFFFF / 1024;

bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

int hip_status(hipError_t e) { return e == hipSuccess ? ARMX_OK : ARMX_ERR_HIP; }

// Only the events of a configuration are used here.
int check_cfg(const armx_config* cfg) {
  if (!cfg) return ARMX_OK;
  return cfg->block_threads || cfg->chain_r || cfg->grid_blocks || cfg->flags ? ARMX_ERR_CONFIG
                                                                             : ARMX_OK;
}

// One rows x cols matrix: its pointer, the alignment of its rows (bytes and
// elements) and its extent.  `optional`: NULL is fine.
int check_matrix(const void* p, uint64_t rows, uint64_t cols, uint64_t ld, uintptr_t bytes,
                 uint64_t elements, bool optional = false) {
  if (!p) return optional || rows == 0 || cols == 0 ? ARMX_OK : ARMX_ERR_NULL;
  if (rows == 0 || cols == 0) return ARMX_OK;
  if (!aligned(p, bytes)) return ARMX_ERR_ALIGN;
  if (rows > 1) {
    if (ld < cols) return ARMX_ERR_SHAPE;
    if (ld % elements) return ARMX_ERR_ALIGN;
    if (ld > kMaxElements || rows - 1 > (kMaxElements - cols) / ld) return ARMX_ERR_SHAPE;
  }
  return ARMX_OK;
}

int check_sizes(uint64_t rows, uint64_t cols) {
  return rows > kMaxElements || cols >= kMaxCols ? ARMX_ERR_SHAPE : ARMX_OK;
}

int check_type(int type) {
  return type == ARMX_F16 || type == ARMX_BF16 ? ARMX_OK : ARMX_ERR_CONFIG;
}

int first_error(std::initializer_list<int> checks) {
  for (int st : checks)
    if (st != ARMX_OK) return st;
  return ARMX_OK;
}

bool log_enabled() {
  static const bool on = std::getenv("ARMX_LOG") != nullptr;
  return on;
}

void log_rows(const char* entry, uint64_t rows, uint64_t cols, int type) {
  if (!log_enabled()) return;
  const armx::RowShape s = armx::row_shape(cols);
  std::fprintf(stderr, "armx: %s rows=%llu cols=%llu type=%d threads=%d chunks=%d\n", entry,
               (unsigned long long)rows, (unsigned long long)cols, type, s.threads, s.chunks);
}

// The checks that the two norms and the quantiser share, and what they write
// for rows without values.  `done` is set when nothing is left to launch.
int prepare_norm(const armx::NormArgs& a, bool norm, const armx_config* cfg, hipStream_t stream,
                 bool* done) {
  *done = true;
  const bool codes = !a.out;
  int st = first_error(
      {check_type(a.type), check_cfg(cfg), norm && !(a.eps >= 0.0f) ? ARMX_ERR_CONFIG : ARMX_OK,
       check_sizes(a.rows, a.cols), check_matrix(a.x, a.rows, a.cols, a.ldx, 16, 8),
       check_matrix(a.residual, a.rows, a.cols, a.ldr, 16, 8, true),
       check_matrix(a.sum_out, a.rows, a.cols, a.lds, 16, 8, true)});
  if (st != ARMX_OK) return st;
  if (norm && a.rows && a.cols && !a.weight) return ARMX_ERR_NULL;
  if (norm && !aligned(a.weight, 16)) return ARMX_ERR_ALIGN;
  if (a.sum_out && !a.residual) return ARMX_ERR_CONFIG;
  if (a.sum_out && a.sum_out == a.out && a.rows && a.cols) return ARMX_ERR_CONFIG;
  if (!aligned(a.inv_rms, 4) || !aligned(a.scales, 4)) return ARMX_ERR_ALIGN;
  if (a.rows == 0) return ARMX_OK;
  if (codes && !a.scales) return ARMX_ERR_NULL;
  if (a.cols == 0) {
    float* zeros = codes ? a.scales : a.inv_rms;
    return zeros ? hip_status(armx::launch_zero(zeros, a.rows, stream)) : ARMX_OK;
  }
  *done = false;
  return ARMX_OK;
}

}  // namespace

extern "C" {

int rms_norm_rows(const void* x, size_t ldx, const void* residual, size_t ldr,
                  const void* weight, int type, size_t rows, size_t cols, float eps, void* out,
                  size_t ldo, void* sum_out, size_t lds, float* inv_rms,
                  const armx_config* cfg, void* stream) {
  armx::NormArgs a;
  a.x = static_cast<const uint16_t*>(x);
  a.residual = static_cast<const uint16_t*>(residual);
  a.weight = static_cast<const uint16_t*>(weight);
  a.out = static_cast<uint16_t*>(out);
  a.sum_out = static_cast<uint16_t*>(sum_out);
  a.inv_rms = inv_rms;
  a.rows = rows, a.cols = cols;
  a.ldx = ldx, a.ldr = ldr, a.ldo = ldo, a.lds = lds;
  a.eps = eps, a.type = type;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (rows && cols && !out) return ARMX_ERR_NULL;
  int st = check_matrix(out, rows, cols, ldo, 16, 8);
  if (st != ARMX_OK) return st;
  if (!a.out) a.out = reinterpret_cast<uint16_t*>(16);  // no values: never written
  bool done;
  st = prepare_norm(a, true, cfg, s, &done);
  if (st != ARMX_OK || done) return st;
  log_rows("rms_norm_rows", rows, cols, type);
  return hip_status(armx::launch_norm(a, cfg, s));
}

int rms_norm_rows_int8(const void* x, size_t ldx, const void* residual, size_t ldr,
                       const void* weight, int type, size_t rows, size_t cols, float eps,
                       int8_t* codes, size_t ldc, float* scales, void* sum_out, size_t lds,
                       const armx_config* cfg, void* stream) {
  armx::NormArgs a;
  a.x = static_cast<const uint16_t*>(x);
  a.residual = static_cast<const uint16_t*>(residual);
  a.weight = static_cast<const uint16_t*>(weight);
  a.codes = codes, a.scales = scales;
  a.sum_out = static_cast<uint16_t*>(sum_out);
  a.rows = rows, a.cols = cols;
  a.ldx = ldx, a.ldr = ldr, a.ldc = ldc, a.lds = lds;
  a.eps = eps, a.type = type;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  int st = check_matrix(codes, rows, cols, ldc, 16, 16);
  if (st != ARMX_OK) return st;
  bool done;
  st = prepare_norm(a, true, cfg, s, &done);
  if (st != ARMX_OK || done) return st;
  log_rows("rms_norm_rows_int8", rows, cols, type);
  return hip_status(armx::launch_norm(a, cfg, s));
}

int quantize_rows_int8(const void* x, size_t ldx, int type, size_t rows, size_t cols,
                       int8_t* codes, size_t ldc, float* scales, const armx_config* cfg,
                       void* stream) {
  armx::NormArgs a;
  a.x = static_cast<const uint16_t*>(x);
  a.codes = codes, a.scales = scales;
  a.rows = rows, a.cols = cols;
  a.ldx = ldx, a.ldc = ldc;
  a.type = type;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  int st = check_matrix(codes, rows, cols, ldc, 16, 16);
  if (st != ARMX_OK) return st;
  bool done;
  st = prepare_norm(a, false, cfg, s, &done);
  if (st != ARMX_OK || done) return st;
  log_rows("quantize_rows_int8", rows, cols, type);
  return hip_status(armx::launch_norm(a, cfg, s));
}

int rms_norm_rows_backward(const void* dy, size_t ldy, const void* h, size_t ldh,
                           const void* weight, const float* inv_rms, const void* dsum,
                           size_t ldd, int type, size_t rows, size_t cols, void* dx,
                           size_t ldx, float* dweight, void* ws, size_t ws_bytes,
                           const armx_config* cfg, void* stream) {
  int st = first_error(
      {check_type(type), check_cfg(cfg), check_sizes(rows, cols),
       cols > armx::kMaxBackwardCols ? ARMX_ERR_SHAPE : ARMX_OK,
       check_matrix(dy, rows, cols, ldy, 16, 8), check_matrix(h, rows, cols, ldh, 16, 8),
       check_matrix(dsum, rows, cols, ldd, 16, 8, true),
       check_matrix(dx, rows, cols, ldx, 16, 8)});
  if (st != ARMX_OK) return st;
  if (cols == 0) return ARMX_OK;
  if (!dweight) return ARMX_ERR_NULL;
  if (!aligned(dweight, 16)) return ARMX_ERR_ALIGN;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (rows == 0) return hip_status(armx::launch_zero(dweight, cols, s));
  if (!weight || !inv_rms) return ARMX_ERR_NULL;
  if (!aligned(weight, 16) || !aligned(inv_rms, 4)) return ARMX_ERR_ALIGN;
  const armx::NormBackwardPlan plan =
      armx::plan_norm_backward(rows, cols, armx::current_cu_count());
  if (plan.ws_bytes) {
    if (!ws) return ARMX_ERR_NULL;
    if (!aligned(ws, 256)) return ARMX_ERR_ALIGN;
    if (ws_bytes < plan.ws_bytes) return ARMX_ERR_WORKSPACE;
  }
  armx::NormBackwardArgs a;
  a.dy = static_cast<const uint16_t*>(dy);
  a.h = static_cast<const uint16_t*>(h);
  a.weight = static_cast<const uint16_t*>(weight);
  a.inv_rms = inv_rms;
  a.dsum = static_cast<const uint16_t*>(dsum);
  a.dx = static_cast<uint16_t*>(dx);
  a.dweight = dweight;
  a.partials = static_cast<float*>(ws);
  a.rows = rows, a.cols = cols;
  a.ldy = ldy, a.ldh = ldh, a.ldd = ldd, a.ldx = ldx;
  a.type = type;
  log_rows("rms_norm_rows_backward", rows, cols, type);
  return hip_status(armx::launch_norm_backward(a, plan, cfg, s));
}

int matmul_int8(const int8_t* a, size_t lda, const float* a_scales, const int8_t* b, size_t ldb,
                const float* b_scales, const void* bias, size_t m, size_t n, size_t k,
                void* out, size_t ldo, int out_type, const armx_config* cfg, void* stream) {
  if (out_type != ARMX_F16 && out_type != ARMX_BF16 && out_type != ARMX_F32)
    return ARMX_ERR_CONFIG;
  int st = check_cfg(cfg);
  if (st != ARMX_OK) return st;
  const uintptr_t size = out_type == ARMX_F32 ? 4 : 2;
  if (k > kMaxProductK || m > kMaxProductRows || n > kMaxProductRows) return ARMX_ERR_SHAPE;
  st = first_error({check_matrix(a, m, k, lda, 16, 16), check_matrix(b, n, k, ldb, 16, 16),
                    check_matrix(out, m, n, ldo, size, 1)});
  if (st != ARMX_OK) return st;
  if ((m > 1 && lda > kMaxProductLd) || (n > 1 && ldb > kMaxProductLd)) return ARMX_ERR_SHAPE;
  if ((m + 255) / 256 * ((n + 255) / 256) > kMaxProductTiles) return ARMX_ERR_SHAPE;
  if (m == 0 || n == 0) return ARMX_OK;
  if (!a_scales || !b_scales) return ARMX_ERR_NULL;
  if (!aligned(a_scales, 4) || !aligned(b_scales, 4) || !aligned(bias, size))
    return ARMX_ERR_ALIGN;
  armx::MatmulArgs p;
  p.a = a, p.b = b;
  p.a_scales = a_scales, p.b_scales = b_scales;
  p.bias = bias, p.out = out;
  p.m = m, p.n = n, p.k = k;
  // a single row's pitch is never used as one; keep it in range
  p.lda = m > 1 ? lda : 0, p.ldb = n > 1 ? ldb : 0, p.ldo = m > 1 ? ldo : n;
  p.out_type = out_type;
  const int cu_count = armx::current_cu_count();
  if (log_enabled()) {
    const armx::MatmulTile t = armx::choose_matmul_tile(p, cu_count);
    std::fprintf(stderr,
                 "armx: matmul_int8 m=%llu n=%llu k=%llu out_type=%d tile=%dx%d groups=%d "
                 "off_lines=%d\n",
                 (unsigned long long)m, (unsigned long long)n, (unsigned long long)k, out_type,
                 t.rows, t.cols, t.groups, int(t.off_lines));
  }
  return hip_status(
      armx::launch_matmul_int8(p, cu_count, cfg, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
