// The gradients of the cross entropy of rows against a vocabulary:
//   dz = dloss (exp(z - lse) - onehot(target)),  dx = dz w,  dweight = dz^T x,
// for a piece of the vocabulary at a time: its logits z are made again, turned into dz
// in the product's registers and stored in 16 bits, once by rows and once by columns;
// the piece's part of dx and its rows of dweight are products of those with the
// transposes of w's piece and of x, which like all products here run along both
// operands' rows.
//
// dz is rounded to 16 bits twice, with a scale of its own each time:
// - for dx, a row is divided by 1 - exp(z[target] - lse), its target's magnitude, which
//   then is a whole power of two and is not rounded at all (it outweighs the others of
//   its row together), and the row of dx is multiplied by it and by dloss in 32 bits.  Of a
//   row surer of its target than the roundings of its logits (least_rest) it is rounded;
// - for dweight, by dloss over the largest |dloss|; of up to kTwoTerms rows the rest that
//   the rounding leaves is a second 16-bit term, multiplied by the same row of x.  Of more
//   rows a second term costs more than it gives: the roundings of a frequent word's rows
//   average out.  A word that one row alone matters to has that row's, 2^-11 or 2^-8 of it,
//   in full.
// Powers of two keep both in binary16's range: 2^14 for dx, 2^15 for dweight.
//
// Of 4096 x 131072 x 4096 bf16 (9.4 to 9.9 ms by card) a piece of 32768 takes 833 us for logits
// and dz, whose second copy is 2% of them, 794 for dx and 760 for dweight, where a library's
// products alone take 740, 680 and 718 with operands laid out for them: the matrix units are
// busy in 69, 73 and 78% of cycles, at a clock of 1.7 to 1.8 GHz.  Pieces of 2^24 to 2^28
// values take the same time.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "cross_entropy.h"
#include "device_common.hpp"
#include "launch.h"
#include "layer.h"
#include "row_pieces.hpp"
#include "tile16.hpp"
#include "tile16_choice.hpp"

namespace armx {
namespace {

constexpr float kLog2E = 1.44269504088896340736f;
constexpr float kRowScale = 0x1p14f, kTopScale = 0x1p15f;

__device__ __forceinline__ float exp_of(float v) { return __builtin_amdgcn_exp2f(v * kLog2E); }

typedef uint32_t u32x3 __attribute__((ext_vector_type(3), aligned(4)));

// What a row of dz is made with: by rows (exp(z - lse) - onehot) * scale, by columns
// (exp(z - lse) - onehot) * dloss * that of the largest |dloss|; the row of dx is what
// comes out times `back`.  A row that is ignored has zeros, and one whose target is not
// in the vocabulary NaNs.
struct RowScale {
  float scale, dloss, back;
  uint32_t skip;
};

// The scale of the largest |dloss| and what undoes it.  (Below 2^-105, whose scale
// would not be finite, a fixed one.)
__device__ __forceinline__ float top_scale(uint32_t top_bits) {
  const float top = __builtin_bit_cast(float, top_bits);
  return top < 0x1p-105f ? 0x1p120f : kTopScale / top;
}

// The least that a row's scale counts as 1 - p of its target, from sum |x w| over the target's
// logit.  Where p is near 1, lse is about that logit, and what it is off by, d, moves all of
// the row's p by a factor e^d: the others may then add up to e^d - p, above 1 - p by d.
// Scaled by 2^14 / rest, four times below binary16's largest value, they stay in its range
// while d is up to three times `rest`: 48 roundings of the magnitudes that were summed.  An
// lse of cross_entropy_rows, made of the logits as they are here, is off by two, and another
// sum in binary32 by fewer than that as well.  (Where p is below 2/3 no value of a row can
// leave the range.)
__device__ __forceinline__ float least_rest(float size) {
  return __builtin_fminf(__builtin_fmaxf(size * 0x1p-20f, 0x1p-14f), 1.0f);
}

// Scales of 16 rows by block `block`.  Their targets' logits are the diagonal of 16 rows of x
// times the targets' 16 rows of the weight, by the instructions of multiply_tile over the same
// values in the same order (products of zeros past the rows left out), and so with the bits
// that loss_grad_kernel's have: another sum of them may differ by more than the 1 - p that it
// is to scale.  Beside it, by the same on magnitudes, what is summed.
//
// The wavefronts' loads are in flight together; then each multiplies its own in its turn and
// hands the sum on (hand[0]).  Magnitudes are summed by each wavefront apart.  (16 rows by one
// wavefront: gradients of 515 x 32003 x 1000 6 us more, of 8 x 32768 x 4096 6.5.  With a sum
// of its own for each row, in any order, few wide rows were 3.5 us faster, 8 x 1000 x 16384
// 96.7 against 100.2, and narrow ones 3 us slower, 300 x 1000 x 64 22.1 against 18.8.)
constexpr int kScaleRows = 16;
template <int TYPE>
__device__ __forceinline__ void scale_rows(const CrossEntropyArgs& k, const float* dloss,
                                           const float* lse, RowScale* rows, uint64_t block,
                                           floatx4 (*hand)[64]) {
  constexpr uint32_t kHalf = kStepValues / 2;   // a product's values of k
  constexpr uint32_t kFlight = 8, kWaves = 4;
  const uint64_t row0 = block * kScaleRows;
  const uint32_t lane = lane_id(), wave = wave_id(), r = lane & 15, g = lane >> 4;
  const uint64_t row = row0 + r < k.rows ? row0 + r : k.rows - 1;
  const int64_t t = k.targets[row];
  const bool in = t >= 0 && t < int64_t(k.vocab);
  const uint16_t* xr = k.x + row * k.ldx;
  const uint16_t* wr = k.weight + uint64_t(in ? t : 0) * k.ldw;
  const uint32_t cols = uint32_t(k.cols), full = cols / kHalf, all = (cols + kHalf - 1) / kHalf;
  u32x4 a[kFlight], b[kFlight], cut_a, cut_b;   // (the last product's, cut)
  auto load = [&](uint32_t first) ARMX_INLINE {
    if (full) {
#pragma unroll
      for (uint32_t i = 0; i < kFlight; ++i) {
        const uint32_t h = first + i < full ? first + i : full - 1;
        a[i] = *reinterpret_cast<const u32x4*>(xr + h * kHalf + 8 * g);
        b[i] = *reinterpret_cast<const u32x4*>(wr + h * kHalf + 8 * g);
      }
    }
  };
  floatx4 size = {0.0f, 0.0f, 0.0f, 0.0f};
  auto add_size = [&](u32x4 x, u32x4 w) ARMX_INLINE {
    size = mfma16<TYPE>(w & 0x7FFF7FFFu, x & 0x7FFF7FFFu, size);
  };
  load(wave * kFlight);
  for (uint32_t h0 = 0; h0 < all; h0 += kWaves * kFlight) {
    const uint32_t first = h0 + wave * kFlight;
    const bool cut = full < all && first <= full && full - first < kFlight;
    if (cut) {
      cut_a = load8_masked(xr, full * kHalf + 8 * g, cols, 0);
      cut_b = load8_masked(wr, full * kHalf + 8 * g, cols, 0);
      add_size(cut_a, cut_b);
    }
#pragma unroll
    for (uint32_t i = 0; i < kFlight; ++i)
      if (first + i < full) add_size(a[i], b[i]);
    for (uint32_t w = 0; w < kWaves && h0 + w * kFlight < all; ++w) {
      if (wave == w) {
        floatx4 z = {0.0f, 0.0f, 0.0f, 0.0f};
        if (first) z = hand[0][lane];
#pragma unroll
        for (uint32_t i = 0; i < kFlight; ++i)
          if (first + i < full) z = mfma16<TYPE>(b[i], a[i], z);
        if (cut) z = mfma16<TYPE>(cut_b, cut_a, z);
        hand[0][lane] = z;
        if (first + kWaves * kFlight < all) load(first + kWaves * kFlight);
      }
      __syncthreads();
    }
  }
  hand[1 + wave][lane] = size;
  __syncthreads();
  // row r's is with lane r of 16 number r / 4, value r % 4
  if (wave != 0 || g != r / 4 || row0 + r >= k.rows) return;
  auto mine = [&](int i) ARMX_INLINE {
    return reinterpret_cast<const float*>(&hand[i][lane])[r % 4];
  };
  RowScale s = {0.0f, 0.0f, 0.0f, 1u};
  if (t != k.ignore) {
    s.skip = 0;
    s.dloss = dloss[row];
    if (in) {
      const float left = __builtin_fabsf(1.0f - exp_of(mine(0) - lse[row]));
      const float least = least_rest((mine(1) + mine(2)) + (mine(3) + mine(4)));
      const float rest = __builtin_fmaxf(left, least);
      s.scale = kRowScale / rest;
      // (an infinite dloss makes infinities of both signs in dz, whose sums are NaNs)
      s.back = s.dloss - s.dloss == 0.0f ? s.dloss * (rest / kRowScale) : __builtin_nanf("");
    } else {
      s.scale = s.dloss = s.back = __builtin_nanf("");
    }
  }
  rows[row] = s;
}

// The largest |dloss| of rows that count (its bits, NaNs largest), by one block: 8 rows a
// thread in flight, which for as many rows as a call has is far shorter than its products.
__device__ __forceinline__ void top_of_rows(const CrossEntropyArgs& k, const float* dloss,
                                            uint32_t* top, uint32_t* most) {
  constexpr int kFlight = 8;
  uint32_t largest = 0;
  for (uint64_t r0 = threadIdx.x; r0 < k.rows; r0 += 256 * kFlight) {
    int64_t t[kFlight];
    float d[kFlight];
#pragma unroll
    for (int i = 0; i < kFlight; ++i) {
      const uint64_t r = r0 + 256 * i, row = r < k.rows ? r : r0;
      t[i] = k.targets[row];
      d[i] = dloss[row];
    }
#pragma unroll
    for (int i = 0; i < kFlight; ++i) {
      const bool in = t[i] >= 0 && t[i] < int64_t(k.vocab);
      uint32_t size = in ? __builtin_bit_cast(uint32_t, d[i]) & 0x7FFFFFFFu : 0x7FC00000u;
      size = t[i] == k.ignore ? 0 : size;
      largest = size > largest ? size : largest;
    }
  }
  most[threadIdx.x] = largest;
  __syncthreads();
  if (threadIdx.x >= 64) return;
#pragma unroll
  for (int i = 64; i < 256; i += 64) {
    const uint32_t size = most[threadIdx.x + i];
    largest = size > largest ? size : largest;
  }
#pragma unroll
  for (int i = 32; i > 0; i /= 2) {
    const uint32_t size = uint32_t(__shfl_xor(int(largest), i));
    largest = size > largest ? size : largest;
  }
  if (threadIdx.x == 0) *top = largest;
}

// to[c][r] = from[r][c], r < rows, c < cols, for the 64 x 64 tile at (r0, c0): 16 bytes a
// thread on both sides, turned in LDS; zeros for rows that are ignored and up to the next
// multiple of 8.  Two copies stand side by side, without zeros behind them.
template <int COPIES>
__device__ __forceinline__ void transpose_tile(const CrossEntropyArgs& k, uint64_t r0, uint64_t c0,
                                               uint16_t* to, uint64_t ldt, uint32_t (*tile)[33]) {
  const uint64_t rows = k.rows, cols = k.cols;
  const uint32_t chunk = threadIdx.x % 8, line = threadIdx.x / 8;
  u32x4 v[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint64_t r = r0 + line + 32 * i;
    const bool in = r < rows && k.targets[r] != k.ignore;
    v[i] = in ? load8_masked(k.x + r * k.ldx, c0 + chunk * 8, cols, 0) : u32x4{0, 0, 0, 0};
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) tile[line + 32 * i][chunk * 4 + e] = v[i][e];
  __syncthreads();
  // (a row of LDS has 33 words, so the 8 rows and 8 pairs of columns of 64 lanes fall on
  // banks of their own)
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t j = line + 32 * i, r = chunk * 8;
    const uint64_t c = c0 + j;
    uint32_t h[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = tile[r + e][j / 2] >> (16 * (j % 2)) & 0xFFFFu;
    if (c >= cols || r0 + r >= rows) continue;
    if constexpr (COPIES == 1) {
      *reinterpret_cast<u32x4*>(to + c * ldt + r0 + r) =
          u32x4{h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16};
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (r0 + r + e < rows) {
          to[c * ldt + r0 + r + e] = uint16_t(h[e]);
          to[c * ldt + rows + r0 + r + e] = uint16_t(h[e]);
        }
    }
  }
}

// What the products need before the first of them, in one launch: rows' scales by the first
// `scales` blocks, and for dweight (xt not null) the largest |dloss| by the next one and x's
// transpose, a tile at a time, by the others.  (In launches of their own, with an atomic
// maximum, against one: gradients of 300 x 1000 x 64 27.3 us / 24.7, of 2046 x 1216 x 192 41.0 /
// 36.0.)
template <int TYPE, int COPIES>
__global__ __launch_bounds__(256) void loss_prepare_kernel(CrossEntropyArgs k, const float* dloss,
                                                           const float* lse, RowScale* rows,
                                                           uint32_t* top, uint16_t* xt,
                                                           uint64_t ldt, unsigned scales) {
  __shared__ __attribute__((aligned(16))) uint32_t tile[64][33];
  if (blockIdx.x < scales) {
    scale_rows<TYPE>(k, dloss, lse, rows, blockIdx.x, reinterpret_cast<floatx4(*)[64]>(tile));
  } else if (blockIdx.x == scales) {
    top_of_rows(k, dloss, top, tile[0]);
  } else {
    const uint64_t down = ceil_div(k.rows, 64), tiles = down * ceil_div(k.cols, 64);
    for (uint64_t t = blockIdx.x - scales - 1; t < tiles; t += gridDim.x - scales - 1) {
      transpose_tile<COPIES>(k, t % down * 64, t / down * 64, xt, ldt, tile);
      __syncthreads();
    }
  }
}

// dz of a piece of the vocabulary (w: its rows, the first of them number `first`), by
// rows in dz and by columns in dzt (either may be null).  Both have whole tiles of room
// for columns, and dzt with one term for rows too; what is past the piece is never used.
template <class T, int TYPE>
__global__ __launch_bounds__(T::kThreads, T::kPerSimd) void loss_grad_kernel(
    Matrix16 x, Matrix16 w, uint32_t cols, const int64_t* targets, int64_t first,
    const float* lse, const RowScale* rows, const uint32_t* top, uint16_t* dz, uint64_t ldz,
    uint16_t* dzt, uint64_t ldt, uint64_t terms, unsigned tiles_m, unsigned tiles_n) {
  __shared__ __attribute__((aligned(1024))) int8_t lds[T::kLdsBytes];
  unsigned ti, tj;
  tile_of<T>(unsigned(xcd_block_id()), tiles_m, tiles_n, ti, tj);
  const uint64_t i0 = uint64_t(ti) * T::kBM, j0 = uint64_t(tj) * T::kBN;
  const float all = top ? top_scale(*top) : 0.0f;
  floatx4 z[T::kMT][T::kNT];
  multiply_tile<T, TYPE>(x, w, cols, i0, j0, lds, z);
  const uint64_t row0 = i0 + lane_row<T>(), col = j0 + wave_col<T>();
  // the rows' values in flight together, before the first store (which the compiler
  // keeps later loads behind)
  RowScale row_scale[T::kMT];
  float row_lse[T::kMT];
  uint32_t row_at[T::kMT];
#pragma unroll
  for (int i = 0; i < T::kMT; ++i) {
    const uint64_t row = row0 + i < x.rows ? row0 + i : x.rows - 1;
    row_scale[i] = rows[row];
    row_lse[i] = lse[row];
    row_at[i] = column_index(targets[row] - first - int64_t(col));
  }
  float each[T::kMT];
#pragma unroll
  for (int i = 0; i < T::kMT; ++i) {
    const RowScale s = row_scale[i];
    const float l = row_lse[i];
    each[i] = s.dloss * all;
    // (the difference first, which is exact where p is near 1: a rounding of lse log2 e is
    // 2^-24 of lse in p, which counts in the p - 1 of a row nearly sure of its target)
#pragma unroll
    for (int c = 0; c < T::kCols; ++c)
      z[i][c / 4][c % 4] = exp_of(z[i][c / 4][c % 4] - l);
    // few wavefronts have a row's target among their columns, or an ignored row
    const uint32_t at = row_at[i];
    if (at < T::kCols) {
#pragma unroll
      for (int c = 0; c < T::kCols; ++c) z[i][c / 4][c % 4] -= at == uint32_t(c) ? 1.0f : 0.0f;
    }
    if (s.skip) {
#pragma unroll
      for (int c = 0; c < T::kCols; ++c) z[i][c / 4][c % 4] = 0.0f;
    }
    if (dz && row0 + i < x.rows) {
#pragma unroll
      for (int c = 0; c < T::kCols; c += 8) {
        u32x4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          v[e] = narrow2<TYPE>(z[i][c / 4 + e / 2][2 * (e % 2)] * s.scale,
                               z[i][c / 4 + e / 2][2 * (e % 2) + 1] * s.scale);
        *reinterpret_cast<u32x4*>(dz + (row0 + i) * ldz + col + lane_column(c)) = v;
      }
    }
  }
  if (!dzt) return;
  if (terms == 1) {
#pragma unroll
    for (int c = 0; c < T::kCols; ++c) {
      uint16_t* to = dzt + (col + lane_column(c)) * ldt + row0;
      if constexpr (T::kMT == 1) {
        *to = uint16_t(narrow2<TYPE>(z[0][c / 4][c % 4] * each[0], 0.0f));
      } else {
        uint32_t v[T::kMT / 2];
#pragma unroll
        for (int i = 0; i < T::kMT; i += 2)
          v[i / 2] = narrow2<TYPE>(z[i][c / 4][c % 4] * each[i],
                                   z[i + 1][c / 4][c % 4] * each[i + 1]);
        if constexpr (T::kMT == 2) *reinterpret_cast<uint32_t*>(to) = v[0];
        if constexpr (T::kMT == 4) *reinterpret_cast<u32x2*>(to) = u32x2{v[0], v[1]};
        if constexpr (T::kMT == 6) *reinterpret_cast<u32x3*>(to) = u32x3{v[0], v[1], v[2]};
        if constexpr (T::kMT == 8)
          *reinterpret_cast<u32x4*>(to) = u32x4{v[0], v[1], v[2], v[3]};
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < T::kMT; ++i) {
      if (row0 + i >= x.rows) continue;
#pragma unroll
      for (int c = 0; c < T::kCols; ++c) {
        const float v = z[i][c / 4][c % 4] * each[i];
        const uint32_t high = narrow2<TYPE>(v, 0.0f);
        float f[8];
        widen8<TYPE>(u32x4{high, 0, 0, 0}, f);
        uint16_t* to = dzt + (col + lane_column(c)) * ldt + row0 + i;
        to[0] = uint16_t(high);
        to[x.rows] = uint16_t(narrow2<TYPE>(v - f[0], 0.0f));
      }
    }
  }
}

// The part of dx that a piece of the vocabulary makes: dz (rows x k) times the piece's rows
// of w (k x cols), k in `splits` parts of `per` whose products stand apart; added to what
// is there after the first piece.  `to` has whole tiles of room for columns.  With `dx` the
// piece is the last and its only product the whole of it: dx itself, times the rows'
// factors, instead.  (By way of the sums and a join / so: gradients of 2046 x 1216 x 192 36.4 us
// / 31.9, of 4096 x 131072 x 4096 9663 / 9631.)
template <class T, int TYPE>
__global__ __launch_bounds__(T::kThreads, T::kPerSimd) void loss_dx_kernel(
    Matrix16 dz, Matrix16 w, uint64_t cols, uint32_t k, uint32_t per, float* to, uint64_t ldd,
    bool more, uint16_t* dx, uint64_t lddx, const RowScale* rows, unsigned tiles_m,
    unsigned tiles_n) {
  __shared__ __attribute__((aligned(1024))) int8_t lds[T::kLdsBytes];
  const unsigned id = unsigned(xcd_block_id()), split = id / (tiles_m * tiles_n);
  unsigned ti, tj;
  tile_of<T>(id % (tiles_m * tiles_n), tiles_m, tiles_n, ti, tj);
  const uint64_t i0 = uint64_t(ti) * T::kBM, j0 = uint64_t(tj) * T::kBN;
  const uint32_t k0 = split * per;
  const uint32_t part = k0 >= k ? 0 : k - k0 < per ? k - k0 : per;
  dz.p += k0;
  w.p += uint64_t(k0) * w.ld;
  w.rows = part;
  floatx4 acc[T::kMT][T::kNT];
  multiply_tile<T, TYPE>(dz, w, part, i0, j0, lds, acc, cols);
  const uint32_t q = lane_id() >> 4;
  const uint64_t row0 = i0 + lane_row<T>();
  auto at = [&](int i) ARMX_INLINE {
    const uint64_t row = row0 + i < dz.rows ? row0 + i : dz.rows - 1;
    return reinterpret_cast<floatx4*>(to + (split * dz.rows + row) * ldd + j0 + wave_col<T>()) + q;
  };
  constexpr int kTogether = T::kMT % 4 == 0 ? 4 : T::kMT % 2 == 0 ? 2 : 1;
#pragma unroll
  for (int i0 = 0; i0 < T::kMT; i0 += kTogether) {
    if (more) {
      floatx4 old[kTogether][T::kNT];
#pragma unroll
      for (int i = 0; i < kTogether; ++i)
#pragma unroll
        for (int y = 0; y < T::kNT; ++y) old[i][y] = at(i0 + i)[4 * y];
#pragma unroll
      for (int i = 0; i < kTogether; ++i)
#pragma unroll
        for (int y = 0; y < T::kNT; ++y) acc[i0 + i][y] += old[i][y];
    }
    float back[kTogether];
    uint32_t skip[kTogether];
    if (dx) {
#pragma unroll
      for (int i = 0; i < kTogether; ++i) {
        const RowScale& r = rows[row0 + i0 + i < dz.rows ? row0 + i0 + i : dz.rows - 1];
        back[i] = r.back;
        skip[i] = r.skip;
      }
    }
#pragma unroll
    for (int i = i0; i < i0 + kTogether; ++i) {
      if (row0 + i >= dz.rows) continue;
      if (!dx) {
#pragma unroll
        for (int y = 0; y < T::kNT; ++y) at(i)[4 * y] = acc[i][y];
        continue;
      }
      uint16_t* out = dx + (row0 + i) * lddx;
#pragma unroll
      for (int y = 0; y < T::kNT; ++y) {
        const uint64_t c = j0 + wave_col<T>() + 16 * y + 4 * q;
        const floatx4 v = acc[i][y] * back[i - i0];
        u32x2 h = {narrow2<TYPE>(v[0], v[1]), narrow2<TYPE>(v[2], v[3])};
        if (skip[i - i0]) h = u32x2{0, 0};
        if (c + 4 <= cols) {
          *reinterpret_cast<u32x2*>(out + c) = h;
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (c + e < cols) out[c + e] = uint16_t(h[e / 2] >> (16 * (e % 2)));
        }
      }
    }
  }
}

// dx = the splits' products added in order, times the rows' factors; 8 columns a thread,
// whose products of 4 splits are in flight at once.  (One block for all of a row / so: dx
// of 1 x 32768 x 1024 43.6 us / 37.8.)
constexpr int kJoinChunks = 64;
template <int TYPE>
__global__ __launch_bounds__(kJoinChunks) void loss_dx_join_kernel(
    const float* from, uint64_t ldd, uint64_t splits, const RowScale* rows, uint64_t count,
    uint64_t cols, uint16_t* dx, uint64_t lddx) {
  const uint32_t chunks = uint32_t((cols + 7) / 8);
  const uint32_t c = blockIdx.y * kJoinChunks + threadIdx.x;
  if (c >= chunks) return;
  for (uint64_t row = blockIdx.x; row < count; row += gridDim.x) {
    const float back = rows[row].back;
    const bool skip = rows[row].skip;
    floatx4 a = {0, 0, 0, 0}, b = {0, 0, 0, 0};
    auto at = [&](uint64_t s) ARMX_INLINE {
      return reinterpret_cast<const floatx4*>(from + (s * count + row) * ldd) + 2 * c;
    };
    for (uint64_t s = 0; s < splits; s += 4) {
      floatx4 v[4][2];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const floatx4* p = at(s + i < splits ? s + i : s);
        v[i][0] = p[0];
        v[i][1] = p[1];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (s + i < splits) {
          a += v[i][0];
          b += v[i][1];
        }
    }
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = skip ? 0.0f : (i < 4 ? a[i] : b[i - 4]) * back;
    store_chunk8<false>(dx + row * lddx, c, uint32_t(cols), narrow8<TYPE>(f));
  }
}

typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));

// A piece's rows of dweight: dzt (rows x k) times xt (cols x k), times what undoes the
// scale of the largest |dloss|.
template <class T, int TYPE, int OUT>
__global__ __launch_bounds__(T::kThreads, T::kPerSimd) void loss_dweight_kernel(
    Matrix16 dzt, Matrix16 xt, uint32_t k, const uint32_t* top, void* to, uint64_t ldo,
    unsigned tiles_m, unsigned tiles_n) {
  __shared__ __attribute__((aligned(1024))) int8_t lds[T::kLdsBytes];
  unsigned ti, tj;
  tile_of<T>(unsigned(xcd_block_id()), tiles_m, tiles_n, ti, tj);
  const uint64_t i0 = uint64_t(ti) * T::kBM, j0 = uint64_t(tj) * T::kBN;
  const float back = 1.0f / top_scale(*top);
  floatx4 acc[T::kMT][T::kNT];
  multiply_tile<T, TYPE>(dzt, xt, k, i0, j0, lds, acc);
  const uint64_t col = j0 + wave_col<T>();
#pragma unroll
  for (int i = 0; i < T::kMT; ++i) {
    const uint64_t row = i0 + lane_row<T>() + i;
    if (row >= dzt.rows) continue;
#pragma unroll
    for (int y = 0; y < T::kNT; ++y) acc[i][y] *= back;
    if constexpr (OUT == ARMX_F32) {
      float* o = static_cast<float*>(to) + row * ldo;
#pragma unroll
      for (int y = 0; y < T::kNT; ++y) {
        const uint64_t c = col + lane_column(4 * y);
        if (c + 4 <= xt.rows) {
          *reinterpret_cast<f32x4u*>(o + c) = acc[i][y];
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (c + e < xt.rows) o[c + e] = acc[i][y][e];
        }
      }
    } else {
      uint16_t* o = static_cast<uint16_t*>(to) + row * ldo;
#pragma unroll
      for (int h = 0; h < T::kCols; h += 8) {
        const uint64_t c = col + lane_column(h);
        u32x4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          v[e] = narrow2<OUT>(acc[i][h / 4 + e / 2][2 * (e % 2)],
                              acc[i][h / 4 + e / 2][2 * (e % 2) + 1]);
        if (c + 8 <= xt.rows) {
          *reinterpret_cast<u32x4*>(o + c) = v;
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (c + e < xt.rows) o[c + e] = uint16_t(v[e / 2] >> (16 * (e % 2)));
        }
      }
    }
  }
}

// dweight of no rows at all.
__global__ __launch_bounds__(256) void zero_rows_kernel(void* to, uint64_t row_bytes,
                                                        uint64_t pitch, uint64_t rows) {
  for (uint64_t row = blockIdx.x; row < rows; row += gridDim.x)
    for (uint64_t i = threadIdx.x * 2; i < row_bytes; i += 512)
      *reinterpret_cast<uint16_t*>(static_cast<char*>(to) + row * pitch + i) = 0;
}

// ---- launches -----------------------------------------------------------------------------

// Rows (k of dweight's products) up to which a value of dz is kept in two terms.  (Gradients
// against 131072 x 4096, us, one term / two: 16 rows 698 / 690, 64 698 / 789, 128 837 / 983,
// 256 1027 / 1433, 512 1593 / 2250, 2048 5170 / 7810; against 32003 x 1000: 64 60 / 65, 128
// 71 / 91, 256 96 / 123, 512 140 / 254, 2048 448 / 899.)
constexpr uint64_t kTwoTerms = 128;
// dz of a piece: at most this many values, but at least kLeastPiece vocabulary rows.
constexpr uint64_t kPieceValues = uint64_t(1) << 27;
constexpr uint64_t kLeastPiece = 1024;
constexpr uint64_t kMostSplits = 64;
constexpr uint64_t kRoom = kLargestTile;

uint64_t round_up(uint64_t v, uint64_t to) { return ceil_div(v, to) * to; }

class Steps {
 public:
  Steps(const armx_config* cfg, hipStream_t stream) : cfg_(cfg), stream_(stream) {}
  hipError_t run(const void* fn, dim3 grid, int threads, void** args, bool last = false) {
    const bool first = first_;
    first_ = false;
    return launch_kernel(fn, grid, dim3(unsigned(threads)), args, 0, stream_,
                         cfg_ && first ? static_cast<hipEvent_t>(cfg_->start_event) : nullptr,
                         cfg_ && last ? static_cast<hipEvent_t>(cfg_->stop_event) : nullptr);
  }

 private:
  const armx_config* cfg_;
  hipStream_t stream_;
  bool first_ = true;
};

template <int TYPE>
hipError_t launch_grads(const CrossEntropyArgs& a, const CrossEntropyGradPlan& plan,
                        const CrossEntropyGrads& grads, void* ws, int cu_count,
                        const armx_config* cfg, hipStream_t stream) {
  Steps steps(cfg, stream);
  char* base = static_cast<char*>(ws);
  uint32_t* top = reinterpret_cast<uint32_t*>(base + plan.top);
  RowScale* rows = reinterpret_cast<RowScale*>(base + plan.rows);
  uint16_t* dz = grads.dx ? reinterpret_cast<uint16_t*>(base + plan.dz) : nullptr;
  uint16_t* dzt = grads.dweight ? reinterpret_cast<uint16_t*>(base + plan.dzt) : nullptr;
  uint16_t* xt = reinterpret_cast<uint16_t*>(base + plan.xt);
  float* sums = reinterpret_cast<float*>(base + plan.dx);
  CrossEntropyArgs copy = a;
  const float *dloss = grads.dloss, *lse = grads.lse;
  hipError_t e;
  {
    unsigned scales = unsigned(ceil_div(a.rows, kScaleRows));
    uint64_t blocks = scales, ldt = plan.ldt;
    if (dzt) {
      const uint64_t tiles = ceil_div(a.rows, 64) * ceil_div(a.cols, 64);
      blocks += 1 + (tiles < kMaxGrid ? tiles : kMaxGrid);
    } else {
      top = nullptr;   // dweight's
    }
    void* args[] = {&copy, &dloss, &lse, &rows, &top, &xt, &ldt, &scales};
    e = steps.run(plan.terms == 1 ? reinterpret_cast<const void*>(&loss_prepare_kernel<TYPE, 1>)
                                  : reinterpret_cast<const void*>(&loss_prepare_kernel<TYPE, 2>),
                  dim3(unsigned(blocks)), 256, args);
    if (e != hipSuccess) return e;
  }
  uint32_t cols = uint32_t(a.cols);
  const int64_t* targets = a.targets;
  uint64_t ldz = plan.ldz, ldt = plan.ldt, terms = plan.terms, ldd = plan.ldd;
  for (uint64_t v0 = 0; v0 < a.vocab; v0 += plan.piece) {
    const uint64_t count = a.vocab - v0 < plan.piece ? a.vocab - v0 : plan.piece;
    const bool last = v0 + count == a.vocab;
    unsigned tiles_m = 0, tiles_n = 0;
    {
      Matrix16 x{a.x, a.rows, a.rows > 1 ? a.ldx : 0};
      Matrix16 w{a.weight + v0 * a.ldw, count, count > 1 ? a.ldw : 0};
      int64_t first = int64_t(v0);
      void* args[] = {&x, &w, &cols, &targets, &first, &lse, &rows, &top, &dz, &ldz, &dzt, &ldt,
                      &terms, &tiles_m, &tiles_n};
#define ARMX_TILE_CASE(T)                                                         \
  tiles_m = unsigned(ceil_div(a.rows, uint64_t(T::kBM)));                         \
  tiles_n = unsigned(ceil_div(count, uint64_t(T::kBN)));                          \
  e = steps.run(reinterpret_cast<const void*>(&loss_grad_kernel<T, TYPE>),        \
                dim3(tiles_m * tiles_n), T::kThreads, args, last && !dz && !dzt)
      ARMX_OF_TILE(choose_tile16(a.rows, count, a.cols, cu_count), ARMX_TILE_CASE);
#undef ARMX_TILE_CASE
      if (e != hipSuccess) return e;
    }
    if (dz) {
      Matrix16 mz{dz, a.rows, plan.ldz}, mw{a.weight + v0 * a.ldw, count, a.ldw};
      uint32_t k = uint32_t(count);
      uint64_t across = a.cols;
      uint32_t per = uint32_t(round_up(ceil_div(count, plan.splits), kStepValues));
      bool more = v0 != 0;
      uint16_t* out = last && plan.splits == 1 ? grads.dx : nullptr;
      uint64_t lddx = grads.lddx;
      void* args[] = {&mz, &mw, &across, &k, &per, &sums, &ldd, &more, &out, &lddx, &rows,
                      &tiles_m, &tiles_n};
#define ARMX_TILE_CASE(T)                                                      \
  tiles_m = unsigned(ceil_div(a.rows, uint64_t(T::kBM)));                      \
  tiles_n = unsigned(ceil_div(a.cols, uint64_t(T::kBN)));                      \
  e = steps.run(reinterpret_cast<const void*>(&loss_dx_kernel<T::Across, TYPE>), \
                dim3(tiles_m * tiles_n * unsigned(plan.splits)), T::kThreads, args,       \
                out && !dzt)
      ARMX_OF_TILE(plan.dx_tile, ARMX_TILE_CASE);
#undef ARMX_TILE_CASE
      if (e != hipSuccess) return e;
    }
    if (dzt) {
      Matrix16 mz{dzt, count, plan.ldt}, mx{xt, a.cols, plan.ldt};
      uint32_t k = uint32_t(a.rows * plan.terms);
      const uint64_t size = grads.dweight_type == ARMX_F32 ? 4 : 2;
      void* to = static_cast<char*>(grads.dweight) + v0 * grads.lddw * size;
      uint64_t ldo = grads.lddw;
      void* args[] = {&mz, &mx, &k, &top, &to, &ldo, &tiles_m, &tiles_n};
#define ARMX_TILE_CASE(T)                                                                   \
  tiles_m = unsigned(ceil_div(count, uint64_t(T::kBM)));                                    \
  tiles_n = unsigned(ceil_div(a.cols, uint64_t(T::kBN)));                                   \
  e = steps.run(grads.dweight_type == ARMX_F32                                              \
                    ? reinterpret_cast<const void*>(&loss_dweight_kernel<T, TYPE, ARMX_F32>) \
                    : reinterpret_cast<const void*>(&loss_dweight_kernel<T, TYPE, TYPE>),   \
                dim3(tiles_m * tiles_n), T::kThreads, args, last && !(dz && plan.splits > 1))
      ARMX_OF_TILE(choose_tile16(count, a.cols, k, cu_count), ARMX_TILE_CASE);
#undef ARMX_TILE_CASE
      if (e != hipSuccess) return e;
    }
  }
  if (!dz || plan.splits == 1) return hipSuccess;
  const float* from = sums;
  uint64_t splits = plan.splits, count = a.rows, all = a.cols, lddx = grads.lddx;
  const RowScale* scales = rows;
  uint16_t* dx = grads.dx;
  void* args[] = {&from, &ldd, &splits, &scales, &count, &all, &dx, &lddx};
  const uint64_t across = ceil_div(all, 8 * kJoinChunks);
  const uint64_t most = kMaxGrid * 1024 / kJoinChunks / across;
  return steps.run(reinterpret_cast<const void*>(&loss_dx_join_kernel<TYPE>),
                   dim3(unsigned(count < most ? count : most), unsigned(across)), kJoinChunks,
                   args, true);
}

}  // namespace

CrossEntropyGradPlan plan_cross_entropy_backward(uint64_t rows, uint64_t vocab, uint64_t cols,
                                                 bool dx, bool dweight, int cu_count) {
  CrossEntropyGradPlan p;
  if (rows == 0 || vocab == 0 || cols == 0) return p;
  p.piece = kPieceValues / rows / kRoom * kRoom;
  if (p.piece < kLeastPiece) p.piece = kLeastPiece;
  // (and the grids of its products and its transpose)
  const uint64_t most = (uint64_t(1) << 34) / round_up(cols, kRoom) / kRoom * kRoom;
  if (p.piece > most) p.piece = most;
  if (p.piece > round_up(vocab, kRoom)) p.piece = round_up(vocab, kRoom);
  // no larger than what the pieces share evenly
  p.piece = round_up(ceil_div(vocab, ceil_div(vocab, p.piece)), kRoom);
  // A line more than whole tiles: rows that lie a power of two apart are in few of the
  // caches' channels (4096 x 4096 x 32768 917 us, with a line more 767).
  p.ldz = p.piece + kStepValues;
  p.terms = rows <= kTwoTerms ? 2 : 1;
  // with one term a tile's rows past the last are written too
  p.ldt = round_up(p.terms == 2 ? 2 * rows : rows + kRoom - 1, kStepValues) + kStepValues;
  // (rows * piece is at most 2^27 values or a piece kLeastPiece, and ldt little more than the
  // rows: all sizes that the calls take hold this, which their products rest on)
  if (!tile_reaches(rows, p.ldz, p.piece) || !tile_reaches(p.piece, p.ldt, rows * p.terms) ||
      !tile_reaches(cols, p.ldt, rows * p.terms)) {
    p.ws_bytes = size_t(-1);
    return p;
  }
  p.ldd = round_up(cols, kRoom);
  // Of few tiles, parts of the piece in blocks of their own: tile and parts are chosen
  // together.  (Parts up to a block of 128 x 128 for every compute unit, and their tile after
  // that: dx of 256 x 131072 x 4096 666 us, now 530; of 1024 x 32768 x 4096 550, now 450.)
  const Split16 dx_of = choose_split16(rows, cols, p.piece, cu_count, kMostSplits);
  p.splits = dx_of.splits;
  p.dx_tile = dx_of.tile;
  size_t at = 0;
  auto take = [&](size_t& offset, uint64_t bytes) {
    offset = at;
    at += size_t(round_up(bytes, 256));
  };
  take(p.top, 4);
  take(p.rows, rows * sizeof(RowScale));
  if (dx) {
    take(p.dz, rows * p.ldz * 2);
    if (p.splits > 1 || p.piece < vocab) take(p.dx, p.splits * rows * p.ldd * 4);
  }
  if (dweight) {
    take(p.dzt, p.piece * p.ldt * 2);
    take(p.xt, cols * p.ldt * 2);
  }
  p.ws_bytes = at;
  return p;
}

hipError_t launch_cross_entropy_backward(const CrossEntropyArgs& a,
                                         const CrossEntropyGradPlan& plan,
                                         const CrossEntropyGrads& grads, void* ws, int cu_count,
                                         const armx_config* cfg, hipStream_t stream) {
  if (a.rows == 0) {
    if (!grads.dweight) return hipSuccess;
    const uint64_t size = grads.dweight_type == ARMX_F32 ? 4 : 2;
    void* to = grads.dweight;
    uint64_t bytes = a.cols * size, pitch = grads.lddw * size, rows = a.vocab;
    void* args[] = {&to, &bytes, &pitch, &rows};
    return Steps(cfg, stream).run(reinterpret_cast<const void*>(&zero_rows_kernel),
                                  dim3(unsigned(rows < kMaxGrid ? rows : kMaxGrid)), 256, args,
                                  true);
  }
  return a.type == ARMX_F16
             ? launch_grads<ARMX_F16>(a, plan, grads, ws, cu_count, cfg, stream)
             : launch_grads<ARMX_BF16>(a, plan, grads, ws, cu_count, cfg, stream);
}

}  // namespace armx
