// The softmax cross entropy of rows x (hidden states) against the rows of a weight (a
// vocabulary's output vectors): z = x w^T, lse = log sum over v of exp(z), loss =
// lse - z[target].  The logits z are made tile by tile in registers and never stored:
// of each row's 64 columns of a tile its largest z and its sum of exp(z - largest) are
// kept, and those are joined in order by a second kernel.
//
// Many rows are bound by the matrix units and the clock that their power leaves (8192 x
// 131072 x 4096 bf16 5.9 to 6.3 ms by card, 1390 to 1500 TFLOP/s, 97 to 99% of the rate of a
// library's product alone; units busy in 80% of cycles at 1.7 GHz), few by reading the weight
// (8 x 32768 x 1024 14.7 us, 12 of them at 5.4 TB/s).
//
// A row's sums do not depend on the tile that makes them: k runs in order in every
// tile, a wavefront has 64 columns, and their sum is one tree over them.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "cross_entropy.h"
#include "device_common.hpp"
#include "launch.h"
#include "tile16.hpp"
#include "tile16_choice.hpp"

namespace armx {
namespace {

constexpr float kLog2E = 1.44269504088896340736f;
constexpr float kMinusInf = -__builtin_inff();

__device__ __forceinline__ float exp_of(float v) { return __builtin_amdgcn_exp2f(v * kLog2E); }

__device__ __forceinline__ float max_xor16(float v) {
  auto p = __builtin_amdgcn_permlane16_swap(fbits(v), fbits(v), false, false);
  return __builtin_fmaxf(bitsf(int(p[0])), bitsf(int(p[1])));
}
__device__ __forceinline__ float max_xor32(float v) {
  auto p = __builtin_amdgcn_permlane32_swap(fbits(v), fbits(v), false, false);
  return __builtin_fmaxf(bitsf(int(p[0])), bitsf(int(p[1])));
}

struct Part {
  float top, sum;   // largest z, sum of exp(z - top)
};

// Where a row's part of a piece is: the parts of 8 rows lie together, by pieces, as one
// block joins them and as a lane with 8 rows has them.
constexpr uint64_t kJoinRows = 8;
__device__ __forceinline__ uint64_t part_of(uint64_t piece, uint64_t pieces, uint64_t row) {
  return (row / kJoinRows * pieces + piece) * kJoinRows + row % kJoinRows;
}

template <class T, int TYPE>
__global__ __launch_bounds__(T::kThreads, T::kPerSimd) void cross_entropy_kernel(
    Matrix16 x, Matrix16 w, uint32_t cols, const int64_t* targets, Part* parts, uint64_t pieces,
    float* hits, unsigned tiles_m, unsigned tiles_n) {
  static_assert(T::kNT == 4, "a wavefront's columns are one piece");
  __shared__ __attribute__((aligned(1024))) int8_t lds[T::kLdsBytes];
  unsigned ti, tj;
  tile_of<T>(unsigned(xcd_block_id()), tiles_m, tiles_n, ti, tj);
  const uint64_t i0 = uint64_t(ti) * T::kBM, j0 = uint64_t(tj) * T::kBN;
  floatx4 z[T::kMT][T::kNT];
  multiply_tile<T, TYPE>(x, w, cols, i0, j0, lds, z);
  const uint64_t col = j0 + wave_col<T>();
  // a wavefront whose columns are all past the vocabulary has nothing to add
  const uint64_t piece = col / kLossPiece;
  if (piece * kLossPiece >= w.rows) return;
  if (j0 + T::kBN > w.rows) {
#pragma unroll
    for (int y = 0; y < T::kNT; ++y)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (col + lane_column(4 * y + e) >= w.rows) {
#pragma unroll
          for (int i = 0; i < T::kMT; ++i) z[i][y][e] = kMinusInf;
        }
  }
  // the rows' targets in flight together, before the first store (which the compiler
  // keeps later loads behind)
  int64_t target[T::kMT];
#pragma unroll
  for (int i = 0; i < T::kMT; ++i) {
    const uint64_t row = i0 + lane_row<T>() + i;
    target[i] = targets[row < x.rows ? row : x.rows - 1];
  }
#pragma unroll
  for (int i = 0; i < T::kMT; ++i) {
    const uint64_t row = i0 + lane_row<T>() + i;
    float m = kMinusInf;
#pragma unroll
    for (int y = 0; y < T::kNT; ++y)
#pragma unroll
      for (int e = 0; e < 4; ++e) m = __builtin_fmaxf(m, z[i][y][e]);
    m = max_xor32(max_xor16(m));
    const float from = m == kMinusInf ? 0.0f : m;
    float s[4];
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      const floatx4 v = z[i][y];
      s[y] = (exp_of(v[0] - from) + exp_of(v[1] - from)) +
             (exp_of(v[2] - from) + exp_of(v[3] - from));
    }
    const float sum = add_xor32(add_xor16((s[0] + s[1]) + (s[2] + s[3])));
    if (row < x.rows) {
      if (lane_id() < 16) parts[part_of(piece, pieces, row)] = Part{m, sum};
      const uint32_t at = column_index(target[i] - int64_t(col));
      if (at < T::kCols && target[i] < int64_t(w.rows)) {
        float hit = 0.0f;
#pragma unroll
        for (int c = 0; c < T::kCols; ++c) hit = at == uint32_t(c) ? z[i][c / 4][c % 4] : hit;
        hits[row] = hit;
      }
    }
  }
}

// Parts joined to one, all to the largest's scale.  (One without a largest has a sum of 0,
// or of NaNs, which stay.)
template <int N>
__device__ __forceinline__ Part join(Part all, const Part (&v)[N]) {
  float m = all.top;
#pragma unroll
  for (int i = 0; i < N; ++i) m = __builtin_fmaxf(m, v[i].top);
  auto scaled = [&](Part p) ARMX_INLINE {
    return p.top == kMinusInf ? p.sum : p.sum * exp_of(p.top - m);
  };
  float s = scaled(all);
#pragma unroll
  for (int i = 0; i < N; ++i) s += scaled(v[i]);
  return Part{m, s};
}

// 8 rows a block: 64 threads take a row's pieces, number p of them p, p + 64, ..., eight at
// a time, and their sums are joined in order, 8 by 8.  (16 rows and 16 threads for each: the
// loss of 8 x 32768 x 1024 16.5 -> 14.7 us.)
constexpr int kJoinThreads = 64, kJoinFlight = 8;
__global__ __launch_bounds__(kJoinRows * kJoinThreads) void cross_entropy_join_kernel(
    const Part* parts, uint64_t pieces, const float* hits, const int64_t* targets, uint64_t rows,
    uint64_t vocab, int64_t ignore, float* loss, float* lse) {
  __shared__ Part of[kJoinThreads][kJoinRows];
  const uint32_t r = threadIdx.x % kJoinRows, p = threadIdx.x / kJoinRows;
  const uint64_t row = uint64_t(blockIdx.x) * kJoinRows + r;
  const uint64_t from = row < rows ? row : rows - 1;
  const int64_t t = targets[from];
  const bool in = t >= 0 && t < int64_t(vocab) && t != ignore;
  const float hit = in ? hits[from] : 0.0f;
  Part all = {kMinusInf, 0.0f};
  for (uint64_t q = p; q < pieces; q += kJoinThreads * kJoinFlight) {
    Part v[kJoinFlight];
#pragma unroll
    for (int i = 0; i < kJoinFlight; ++i) {
      const uint64_t qi = q + uint64_t(i) * kJoinThreads;
      v[i] = parts[part_of(qi < pieces ? qi : q, pieces, from)];
      if (qi >= pieces) v[i] = Part{kMinusInf, 0.0f};
    }
    all = join(all, v);
  }
  of[p][r] = all;
  __syncthreads();
  if (p >= kJoinThreads / kJoinFlight) return;
  Part v[kJoinFlight];
#pragma unroll
  for (int i = 0; i < kJoinFlight; ++i) v[i] = of[p * kJoinFlight + i][r];
  of[p * kJoinFlight][r] = join(Part{kMinusInf, 0.0f}, v);
  // (these threads are one wavefront's: its LDS writes are done before the reads behind)
  __builtin_amdgcn_wave_barrier();
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  if (p != 0 || row >= rows) return;
#pragma unroll
  for (int i = 0; i < kJoinFlight; ++i) v[i] = of[i * kJoinFlight][r];
  all = join(Part{kMinusInf, 0.0f}, v);
  const float m = all.top, s = all.sum;
  const float l = m + __builtin_logf(s);
  lse[row] = l;
  loss[row] = t == ignore ? 0.0f : in ? l - hit : __builtin_nanf("");
}

}  // namespace

Tile16Size tile16_size(int index) {
  Tile16Size s{0, 0};
#define ARMX_TILE_CASE(T) s = Tile16Size{T::kBM, T::kBN}
  ARMX_OF_TILE(index, ARMX_TILE_CASE);
#undef ARMX_TILE_CASE
  return s;
}

namespace {

// The estimated time of a product's tiles (us), each of `steps` steps of 64 values of k.  A
// compute unit that makes q tiles runs them in rounds of at most `resident` blocks; a round
// takes `fixed` (its first loads, its results) and, per step, `alone` or, with several blocks
// on the unit, `each` of them if that is more.
//
// The constants are fitted to times of each tile on MI355X over 335 products of 1 to 131072
// rows, 256 to 131072 columns and lengths of 16 to 32064 with 16-bit results; over those the
// tile that they choose is 2.3% behind the fastest on average, more than 20% at 7 and 30% at
// worst (8192 x 1000 x 384).  Each pays where it is chosen (us, it and the best of the
// others): 256 x 256 at 1024 x 32003 x 2056 130 (166); 192 x 256 at 384 x 32003 x 1000 35 (38);
// 256 x 128 at 777 x 8192 x 8192 105 (122); 128 x 128 at 2048 x 32003 x 128 34 (42); 64 x 128
// at 256 x 8192 x 4096 35 (41); 16 x 128 at 1000 x 1000 x 32 4.1 (4.3), and its times at larger
// ones are those of the best (16 x 131072 x 512 27 (27)); 16 x 64 at 16 x 4096 x 8192 29 (43).
// (One of 32 x 128 was chosen more often than it paid.)
double tile16_time(int index, uint64_t tiles, uint64_t k, int cu_count) {
  struct Time {
    int resident;
    float fixed, alone, each;
  };
  constexpr Time times[kTile16s] = {
      {1, 7.25f, 1.21f, 1.21f}, {1, 4.66f, 1.07f, 1.07f}, {1, 3.74f, 0.73f, 0.73f},
      {2, 2.66f, 0.36f, 0.52f}, {2, 1.81f, 0.31f, 0.37f}, {2, 1.16f, 0.28f, 0.24f},
      {3, 1.08f, 0.27f, 0.12f}};
  const Time t = times[index];
  const uint64_t per_cu = ceil_div(tiles, uint64_t(cu_count));
  const double steps = double(ceil_div(k, uint64_t(kStepValues)));
  auto round = [&](uint64_t blocks) {
    const double together = double(blocks) * t.each;
    return blocks == 0 ? 0.0 : t.fixed + steps * (together > t.alone ? together : t.alone);
  };
  return double(per_cu / t.resident) * round(t.resident) + round(per_cu % t.resident);
}

constexpr uint64_t kLeastSplit = 512;   // values of k in a part
constexpr double kJoinLaunch = 4;       // us

}  // namespace

int choose_tile16(uint64_t m, uint64_t n, uint64_t k, int cu_count) {
  return choose_split16(m, n, k, cu_count, 1).tile;
}

Split16 choose_split16(uint64_t m, uint64_t n, uint64_t k, int cu_count, uint64_t most) {
  Split16 best;
  double least = -1;
  for (int i = 0; i < kTile16s; ++i) {
    const Tile16Size s = tile16_size(i);
    const uint64_t tiles = ceil_div(m, uint64_t(s.bm)) * ceil_div(n, uint64_t(s.bn));
    for (uint64_t splits = 1; splits <= most; splits *= 2) {
      if (tiles * splits > 0x7FFFFFFFu / 1024) break;  // the grid's limit
      if (splits > 1 && k / splits < kLeastSplit) break;
      // (products are written and read again to be joined, at 4.9 TB/s, by another launch)
      const double join =
          splits > 1 ? kJoinLaunch + double(splits) * double(m) * double(n) * 8 / 4.9e6 : 0;
      const double t = tile16_time(i, tiles * splits, ceil_div(k, splits), cu_count) + join;
      if (least < 0 || t < least) best = Split16{i, splits}, least = t;
    }
  }
  return best;
}

namespace {

template <int TYPE>
hipError_t launch_loss(const CrossEntropyArgs& a, const CrossEntropyPlan& plan, float* loss,
                       float* lse, void* ws, int cu_count, const armx_config* cfg,
                       hipStream_t stream) {
  Matrix16 x{a.x, a.rows, a.rows > 1 ? a.ldx : 0}, w{a.weight, a.vocab, a.vocab > 1 ? a.ldw : 0};
  uint32_t cols = uint32_t(a.cols);
  const int64_t* targets = a.targets;
  Part* parts = reinterpret_cast<Part*>(static_cast<char*>(ws) + plan.partials);
  float* hits = reinterpret_cast<float*>(static_cast<char*>(ws) + plan.hits);
  unsigned tiles_m = 0, tiles_n = 0;
  uint64_t pieces = plan.pieces;
  void* args[] = {&x, &w, &cols, &targets, &parts, &pieces, &hits, &tiles_m, &tiles_n};
  hipError_t e = hipErrorInvalidValue;
#define ARMX_TILE_CASE(T)                                                                      \
  tiles_m = unsigned(ceil_div(a.rows, uint64_t(T::kBM)));                                      \
  tiles_n = unsigned(ceil_div(a.vocab, uint64_t(T::kBN)));                                     \
  e = launch_kernel(reinterpret_cast<const void*>(&cross_entropy_kernel<T, TYPE>),             \
                    dim3(tiles_m * tiles_n), dim3(T::kThreads), args, 0, stream,               \
                    cfg ? static_cast<hipEvent_t>(cfg->start_event) : nullptr, nullptr)
  ARMX_OF_TILE(choose_tile16(a.rows, a.vocab, a.cols, cu_count), ARMX_TILE_CASE);
#undef ARMX_TILE_CASE
  if (e != hipSuccess) return e;
  const Part* from = parts;
  uint64_t rows = a.rows, vocab = a.vocab;
  const float* found = hits;
  int64_t ignore = a.ignore;
  void* join[] = {&from, &pieces, &found, &targets, &rows, &vocab, &ignore, &loss, &lse};
  return launch_kernel(reinterpret_cast<const void*>(&cross_entropy_join_kernel),
                       dim3(unsigned(ceil_div(rows, kJoinRows))),
                       dim3(kJoinRows * kJoinThreads), join, 0, stream, nullptr,
                       cfg ? static_cast<hipEvent_t>(cfg->stop_event) : nullptr);
}

}  // namespace

CrossEntropyPlan plan_cross_entropy(uint64_t rows, uint64_t vocab) {
  CrossEntropyPlan p;
  p.pieces = ceil_div(vocab, kLossPiece);
  p.hits = size_t(p.pieces * ceil_div(rows, kJoinRows) * kJoinRows * sizeof(Part));
  p.ws_bytes = p.hits + size_t(rows * sizeof(float));
  return p;
}

hipError_t launch_cross_entropy(const CrossEntropyArgs& a, const CrossEntropyPlan& plan,
                                float* loss, float* lse, void* ws, int cu_count,
                                const armx_config* cfg, hipStream_t stream) {
  return a.type == ARMX_F16 ? launch_loss<ARMX_F16>(a, plan, loss, lse, ws, cu_count, cfg, stream)
                            : launch_loss<ARMX_BF16>(a, plan, loss, lse, ws, cu_count, cfg, stream);
}

}  // namespace armx
