// Arguments and plans of the loss of rows against a vocabulary, shared by its C entry
// points and launchers.
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

#include "armx.h"

namespace armx {

struct CrossEntropyArgs {
  const uint16_t* x = nullptr;
  const uint16_t* weight = nullptr;
  const int64_t* targets = nullptr;
  uint64_t rows = 0, vocab = 0, cols = 0;
  uint64_t ldx = 0, ldw = 0;
  int64_t ignore = -100;
  int type = ARMX_F16;
};

// The products reach a tile's rows, at most 256 of them, by 32-bit byte offsets from its
// first: those of x and of the weight by a limit on their pitches, those made in the
// workspace by their plan (tile_reaches).
constexpr uint64_t kMaxTileLd = uint64_t(1) << 22, kMostTileRows = 256;
constexpr bool tile_reaches(uint64_t rows, uint64_t ld, uint64_t k) {
  // (whole steps of 64 values, 2 bytes each)
  return ((rows < kMostTileRows ? rows : kMostTileRows) - 1) * ld * 2 + (k + 63) / 64 * 128 <=
         0xFFFFFFF0u;
}
static_assert(tile_reaches(kMostTileRows, kMaxTileLd, kMaxTileLd), "pitches of x and the weight");

// The sums of a tile's 64 columns, a piece, stand apart until they are joined in order.
constexpr uint64_t kLossPiece = 64;

struct CrossEntropyPlan {
  uint64_t pieces = 0;
  size_t partials = 0, hits = 0;   // byte offsets in the workspace
  size_t ws_bytes = 0;
};

struct CrossEntropyGradPlan {
  uint64_t piece = 0;     // vocabulary rows at a time
  uint64_t ldz = 0;       // values between rows of dz (rows x piece)
  uint64_t terms = 0;     // 16-bit terms that stand for a value of dz's transpose
  uint64_t ldt = 0;       // values between rows of it and of x's transpose
  uint64_t splits = 0;    // parts of a piece whose products for dx stand apart
  int dx_tile = 0;        // and what they are made of
  uint64_t ldd = 0;       // floats between rows of those products
  // byte offsets in the workspace
  size_t top = 0, rows = 0, dz = 0, dzt = 0, xt = 0, dx = 0;
  size_t ws_bytes = 0;   // size_t(-1): sizes that the products do not reach
};

CrossEntropyPlan plan_cross_entropy(uint64_t rows, uint64_t vocab);
CrossEntropyGradPlan plan_cross_entropy_backward(uint64_t rows, uint64_t vocab, uint64_t cols,
                                                 bool dx, bool dweight, int cu_count);

hipError_t launch_cross_entropy(const CrossEntropyArgs& args, const CrossEntropyPlan& plan,
                                float* loss, float* lse, void* ws, int cu_count,
                                const armx_config* cfg, hipStream_t stream);
struct CrossEntropyGrads {
  const float* dloss = nullptr;
  const float* lse = nullptr;
  uint16_t* dx = nullptr;     // may be null, like
  void* dweight = nullptr;
  uint64_t lddx = 0, lddw = 0;
  int dweight_type = ARMX_F16;
};
hipError_t launch_cross_entropy_backward(const CrossEntropyArgs& args,
                                         const CrossEntropyGradPlan& plan,
                                         const CrossEntropyGrads& grads, void* ws, int cu_count,
                                         const armx_config* cfg, hipStream_t stream);

// Which of the tiles below a product of m x n over k takes.
int choose_tile16(uint64_t m, uint64_t n, uint64_t k, int cu_count);
// And with k in parts (powers of two up to `most`) whose products, in 32 bits, are joined.
struct Split16 {
  int tile = 0;
  uint64_t splits = 1;
};
Split16 choose_split16(uint64_t m, uint64_t n, uint64_t k, int cu_count, uint64_t most);
struct Tile16Size {
  int bm, bn;
};
Tile16Size tile16_size(int index);

}  // namespace armx
