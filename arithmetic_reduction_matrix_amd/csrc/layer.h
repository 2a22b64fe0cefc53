// Arguments and launch shapes of the layer entry points (row norms, 8-bit
// codes, the product of codes), shared by their C entry points and launchers.
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

#include "armx.h"

namespace armx {

// 16-byte loads: 8 values of a 16-bit type.
constexpr uint32_t kRowVec = 8;

// How a row of `cols` values lies on threads: `threads` per row (8, 16, 32, or
// whole wavefronts), each with `chunks` 16-byte loads in registers (chunk j of
// thread t is the row's chunk j * threads + t).  chunks 0: the row does not fit,
// and is walked in a loop, twice.  A function of cols only, so a row's bits depend
// on nothing else.
struct RowShape {
  int threads;
  int chunks;
};

RowShape row_shape(uint64_t cols);
constexpr int kRowBlock = 256;  // threads per block of rows of at most a wavefront

// Results of at least this many values are written past the caches: 16-bit ones of
// 32 MiB, what the L2s hold together, and codes of half of that.  Written so they take
// less of HBM's time (MI355X, us, through the caches / past them: norm of 8192 x 4096
// 47.6 / 46.4, 16384 x 1024 24.7 / 21.0, 17000 x 1001 25.9 / 22.6; to codes 8192 x 4096
// 44.9 / 43.6, 17000 x 1001 22.7 / 21.8, 335544 x 100 70.3 / 59.4; gradients of 17000 x
// 1001 28.7 / 27.8), except on narrow rows, whose tails and neighbours complete the same
// lines (norm of 335544 x 100 78.2 / 79.0, 1016800 x 33 104.7 / 108.8).  What reads them
// next finds less in the caches: codes of a norm and their product with 256 rows, both
// calls, 8192 x 4096 57.2 / 61.7, 4096 x 8192 56.0 / 64.0, 17000 x 1001 33.6 / 34.0; a
// norm and its codes 16384 x 1024 37.5 / 34.7, 335544 x 100 101.9 / 107.3.
constexpr uint64_t kStreamValues = uint64_t(1) << 24;

struct NormArgs {
  const uint16_t* x = nullptr;
  const uint16_t* residual = nullptr;  // may be null
  const uint16_t* weight = nullptr;    // null: quantise only
  uint16_t* out = nullptr;             // 16-bit result, or
  int8_t* codes = nullptr;             // codes and scales
  float* scales = nullptr;
  uint16_t* sum_out = nullptr;  // may be null
  float* inv_rms = nullptr;     // may be null
  uint64_t rows = 0, cols = 0;
  uint64_t ldx = 0, ldr = 0, ldo = 0, lds = 0, ldc = 0;
  float eps = 0;
  int type = ARMX_F16;
};

struct NormBackwardArgs {
  const uint16_t* dy = nullptr;
  const uint16_t* h = nullptr;
  const uint16_t* weight = nullptr;
  const float* inv_rms = nullptr;
  const uint16_t* dsum = nullptr;  // may be null
  uint16_t* dx = nullptr;
  float* dweight = nullptr;
  float* partials = nullptr;  // blocks x pitch, when the plan has a workspace
  uint64_t rows = 0, cols = 0;
  uint64_t ldy = 0, ldh = 0, ldd = 0, ldx = 0;
  int type = ARMX_F16;
};

struct NormBackwardPlan {
  RowShape shape{};
  int block = 0;        // threads per block
  bool apart = false;   // some blocks sum dweight's columns, the others make dx
  uint64_t blocks = 0;  // otherwise each sums dweight over its own rows
  uint64_t pitch = 0;   // floats between the blocks' partial sums
  size_t ws_bytes = 0;
};

// Longest rows of the backward pass: their column blocks of 64 and a block for each of
// 2^20 rows fill the largest grid.
constexpr uint64_t kMaxBackwardCols = uint64_t(1) << 26;
NormBackwardPlan plan_norm_backward(uint64_t rows, uint64_t cols, int cu_count);

struct MatmulArgs {
  const int8_t* a = nullptr;
  const int8_t* b = nullptr;
  const float* a_scales = nullptr;
  const float* b_scales = nullptr;
  const void* bias = nullptr;  // may be null
  void* out = nullptr;
  uint64_t m = 0, n = 0, k = 0, lda = 0, ldb = 0, ldo = 0;
  int out_type = ARMX_F16;
};

// The tile of out that a block of the product makes, and over how many groups of its
// wavefronts k is split.
struct MatmulTile {
  int rows, cols, groups;
  bool off_lines;  // rows of codes do not all start on a 128-byte line
  int index;       // in its table
};
MatmulTile choose_matmul_tile(const MatmulArgs& args, int cu_count);

// Each launches on the current device and stream with the call's events.
hipError_t launch_norm(const NormArgs& args, const armx_config* cfg, hipStream_t stream);
hipError_t launch_norm_backward(const NormBackwardArgs& args, const NormBackwardPlan& plan,
                                const armx_config* cfg, hipStream_t stream);
hipError_t launch_matmul_int8(const MatmulArgs& args, int cu_count, const armx_config* cfg,
                              hipStream_t stream);

// Compute units of the current device (api.cpp).
int current_cu_count();

}  // namespace armx
