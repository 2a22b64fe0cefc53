// Root-mean-square norm of rows with the residual's addition (16-bit or 8-bit
// result), rows as 8-bit codes, and the norm's backward pass.
//
// Every kernel reads and writes each value once: a row lies in the registers
// of the threads that share it (row_shape), the row's sum of squares and its
// largest magnitude are combined across lanes and wavefronts, and the result
// is formed from the registers.  The bound is HBM.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "device_common.hpp"
#include "launch.h"
#include "layer.h"

namespace armx {

// Whole wavefronts for rows of more than 64 chunks, no more of them than hold the
// row: idle ones keep loads from being in flight (codes of 13421 x 2500 on 512
// threads per row 31.2 us, on 320 25.0).
RowShape row_shape(uint64_t cols) {
  const uint64_t n = (cols + kRowVec - 1) / kRowVec;  // 16-byte chunks
  if (n <= 8) return {8, 1};
  if (n <= 16) return {16, 1};
  if (n <= 32) return {32, 1};
  if (n > 4096) return {1024, 0};
  const int chunks = n <= 512 ? 1 : n <= 1024 ? 2 : 4;
  return {int((n + 64 * chunks - 1) / (64 * chunks)) * 64, chunks};
}

namespace {

using namespace dev;

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float floatx2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// ---- the two 16-bit types -------------------------------------------------------

template <int TYPE>
__device__ __forceinline__ void widen8(u32x4 v, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (TYPE == ARMX_F16) {
      f[2 * i] = lo_f32(v[i]);
      f[2 * i + 1] = hi_f32(v[i]);
    } else {
      f[2 * i] = __builtin_bit_cast(float, v[i] << 16);
      f[2 * i + 1] = __builtin_bit_cast(float, v[i] & 0xFFFF0000u);
    }
  }
}

// two values rounded to nearest even, in one word
template <int TYPE>
__device__ __forceinline__ uint32_t narrow2(float a, float b) {
  if constexpr (TYPE == ARMX_F16) {
    return __builtin_bit_cast(uint32_t, half2v{_Float16(a), _Float16(b)});
  } else {
    return __builtin_bit_cast(uint32_t, bf16x2{__bf16(a), __bf16(b)});
  }
}

template <int TYPE>
__device__ __forceinline__ u32x4 narrow8(const float (&f)[8]) {
  u32x4 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = narrow2<TYPE>(f[2 * i], f[2 * i + 1]);
  return v;
}

// ---- row pieces -------------------------------------------------------------------

// Chunk `c` (8 values) of a row of `cols` values; values past the row are 0.
__device__ __forceinline__ u32x4 load_chunk8(const uint16_t* row, uint32_t c, uint32_t cols) {
  return load8_masked(row, uint64_t(c) * 8, cols, 0u);
}

// STREAM: past the caches (kStreamValues).  The chunk that the row ends in is
// written in a piece of 4, one of 2 and one of 1 values, as its length has them.
template <bool STREAM>
__device__ __forceinline__ void store_chunk8(uint16_t* row, uint32_t c, uint32_t cols, u32x4 v) {
  const uint64_t e = uint64_t(c) * 8;
  if (e + 8 <= cols) {
    if constexpr (STREAM)
      __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(row + e));
    else
      *reinterpret_cast<u32x4*>(row + e) = v;
  } else if (e < cols) {
    const uint32_t rem = cols % 8;   // the same for every row
    if (rem & 4) *reinterpret_cast<u32x2*>(row + e) = u32x2{v[0], v[1]};
    if (rem & 2) *reinterpret_cast<uint32_t*>(row + e + (rem & 4)) = rem & 4 ? v[2] : v[0];
    const uint32_t last = rem & 4 ? (rem & 2 ? v[3] : v[2]) : (rem & 2 ? v[1] : v[0]);
    if (rem & 1) row[e + (rem & 6)] = uint16_t(last);
  }
}

template <bool STREAM>
__device__ __forceinline__ void store_codes8(int8_t* row, uint32_t c, uint32_t cols, u32x2 v) {
  const uint64_t e = uint64_t(c) * 8;
  if (e + 8 <= cols) {
    if constexpr (STREAM)
      __builtin_nontemporal_store(v, reinterpret_cast<u32x2*>(row + e));
    else
      *reinterpret_cast<u32x2*>(row + e) = v;
  } else if (e < cols) {
    const uint32_t rem = cols % 8;
    const uint32_t rest = rem & 4 ? v[1] : v[0];
    if (rem & 4) *reinterpret_cast<uint32_t*>(row + e) = v[0];
    if (rem & 2) *reinterpret_cast<uint16_t*>(row + e + (rem & 4)) = uint16_t(rest);
    if (rem & 1) row[e + (rem & 6)] = int8_t(rem & 2 ? rest >> 16 : rest);
  }
}

// A wavefront's row as a range-checked buffer of the 32-bit words that hold its
// values: a load of a chunk past them returns zeros with no memory access, so the
// loads of a row's chunks stand in no branch and are all in flight together (a
// branch around a load makes the compiler wait where its paths join: 37 rows of
// 5001 values, norm to codes, 6.8 -> 6.6 us).  With an odd count the last word
// holds one value past the row (trim).
constexpr int kRawBuffer = 0x00020000;
struct RowWords {
  __amdgpu_buffer_rsrc_t rs;
  // `row` must be the same in all lanes of the wavefront; cols 0: nothing is read
  __device__ __forceinline__ RowWords(const uint16_t* row, uint32_t cols)
      : rs(__builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(row), 0,
                                             int((cols + 1) / 2 * 4), kRawBuffer)) {}
  __device__ __forceinline__ u32x4 load(uint32_t c) const {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, c * 16, 0, 0));
  }
};

// How a row lies on a block.  TPR > 0: TPR lanes of a wavefront share a row (8 to
// 64, one chunk each), a block of 256 threads has several rows.  TPR 0: the whole
// block shares one, C chunks a thread, at most MAXT threads.
template <int TPR, int MAXT, int C>
struct Lay {
  static constexpr int kTpr = TPR;
  static constexpr int kMax = TPR ? kRowBlock : MAXT;
  static constexpr int kRows = TPR ? kRowBlock / TPR : 1;   // rows at a time
  static constexpr int kChunks = C;
  __device__ __forceinline__ static uint32_t threads() { return TPR ? TPR : blockDim.x; }
  __device__ __forceinline__ static uint32_t lane() {
    return TPR ? threadIdx.x % (TPR ? TPR : 1) : threadIdx.x;
  }
  __device__ __forceinline__ static uint32_t row() {
    return TPR ? threadIdx.x / (TPR ? TPR : 1) : 0;
  }
};

// Clears what a load brought of values past the row.  Applied where the values are
// used: it waits for them, and at the loads it would hold up those behind (48643 x
// 313 backward, rows read ahead: 66 against 37 us).
template <class L, int C>
__device__ __forceinline__ void trim(uint32_t cols, u32x4 (&v)[C]) {
  // rows of one wavefront or more are cut at whole words by the range check
  if (cols % (L::kTpr && L::kTpr < 64 ? 8 : 2) == 0) return;
#pragma unroll
  for (int j = 0; j < C; ++j) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t e = (j * L::threads() + L::lane()) * 8 + 2 * i;   // the word's first value
      v[j][i] &= e >= cols ? 0u : e + 1 == cols ? 0xFFFFu : 0xFFFFFFFFu;
    }
  }
}

// ---- combines across the threads of a row ------------------------------------------

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t v) {
  return uint32_t(__builtin_amdgcn_update_dpp(0, int(v), CTRL, 0xF, 0xF, false));
}

__device__ __forceinline__ uint32_t max_u32(uint32_t a, uint32_t b) { return a > b ? a : b; }

// Largest of aligned lane groups of 2^levels, in every lane (lane_tree's moves).
__device__ __forceinline__ uint32_t lane_max(uint32_t v, int levels) {
  if (levels >= 1) v = max_u32(v, dpp_u32<kDppXor1>(v));
  if (levels >= 2) v = max_u32(v, dpp_u32<kDppXor2>(v));
  if (levels >= 3) v = max_u32(v, dpp_u32<kDppHalfMirror>(v));
  if (levels >= 4) v = max_u32(v, dpp_u32<kDppMirror>(v));
  if (levels >= 5) {
    auto p = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = max_u32(p[0], p[1]);
  }
  if (levels >= 6) {
    auto p = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = max_u32(p[0], p[1]);
  }
  return v;
}

constexpr int log2_of(int v) { return v <= 1 ? 0 : 1 + log2_of(v / 2); }

// The row's sum of squares and largest magnitude (bits), in each of its
// threads: across lanes, and for a row of several wavefronts through LDS, added in
// wavefront order by every thread alike.
template <class L>
struct RowCombine {
  static constexpr int kWaves = L::kTpr ? 1 : L::kMax / 64;
  struct Lds {
    float s[kWaves];
    uint32_t m[kWaves];
  };
  // `turn` alternates between the two halves of `lds` from row to row, so one
  // barrier per row is enough
  __device__ __forceinline__ static void run(float& s, uint32_t& m, Lds* lds, int turn) {
    constexpr int levels = log2_of(L::kTpr ? L::kTpr : 64);
    s = lane_tree(s, levels);
    m = lane_max(m, levels);
    if constexpr (L::kTpr == 0) {
      Lds& l = lds[turn];
      if (lane_id() == 0) {
        l.s[wave_id()] = s;
        l.m[wave_id()] = m;
      }
      __syncthreads();
      s = l.s[0];
      m = l.m[0];
      // (a lane per wavefront and a tree instead: norm to codes of 3728 x 9000 50.0 ->
      // 63.2 us)
      const int waves = num_waves();
#pragma unroll 4
      for (int w = 1; w < waves; ++w) {
        s += l.s[w];
        m = max_u32(m, l.m[w]);
      }
    }
  }
};

// ---- codes ----------------------------------------------------------------------------

constexpr uint32_t kInfBits = 0x7F800000u;

// What a row's codes are made with, from its largest |p|.
struct CodeScale {
  float up;       // exact power of two that keeps the quotients finite and p normal
  float top;      // largest |p| * up
  float inverse;  // 1 / top, and
  float factor;   // 127 / top; 0 for a row of zeros or one that is not finite
  bool finite;
  __device__ __forceinline__ explicit CodeScale(uint32_t top_bits) {
    const float t = __builtin_bit_cast(float, top_bits);
    finite = top_bits < kInfBits;
    up = t < 0x1p-64f ? 0x1p60f : t > 0x1p64f ? 0x1p-60f : 1.0f;
    top = t * up;
    const bool some = finite && t > 0.0f;
    inverse = some ? 1.0f / top : 0.0f;
    factor = some ? 127.0f / top : 0.0f;
  }
};

// Codes of 8 products: round half to even of 127 p / top, of the exact quotient
// v.  t = p * factor is off by less than 2^-23 |v| (the quotient and the product
// round by 2^-24 each); adding 1.5 2^23 rounds it to a whole number whose code is
// the sum's low byte.
//
// NARROW (p of at most 11 bits, a value of a 16-bit type): a v that is no half lies
// at least 2^-12 |v| / 127 from one (bfloat16's 8 bits: 2^-9), since 2 * 127 p and every
// odd multiple of top are whole multiples of the smaller's last bit; only true halves,
// which are common (one value in some tens where top has few bits), need care.  One
// correction, t + (127 p - t top) / top with the difference exact, gives them exactly and
// any other v to 2^-24 |v|.
//
// Otherwise t rounds as v does unless it is within 2^-14 of a half.  There 254 |p|
// is compared with the odd multiple m of top: hi + lo = m top and e = 254 |p| - hi
// are exact (fma; the difference loses its first 13 bits), so e against lo decides.
template <bool NARROW>
__device__ __forceinline__ u32x2 codes8(const float (&p)[8], const CodeScale& cs) {
  constexpr float kMagic = 12582912.0f;
  uint32_t q[8];
  if constexpr (NARROW) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float s = p[i] * cs.up, n = 127.0f * s;
      float t = s * cs.factor;
      t = __builtin_fmaf(__builtin_fmaf(-t, cs.top, n), cs.inverse, t);
      q[i] = __builtin_bit_cast(uint32_t, t + kMagic);
    }
  } else {
    bool near = false;
    float t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      t[i] = (p[i] * cs.up) * cs.factor;
      const float r = t[i] + kMagic;
      q[i] = __builtin_bit_cast(uint32_t, r);
      near |= __builtin_fabsf(t[i] - (r - kMagic)) > 0.5f - 0x1p-14f;
    }
    if (__builtin_expect(near, 0)) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float a = __builtin_fabsf(t[i]), k = __builtin_floorf(a);
        const float m = 2.0f * k + 1.0f, hi = m * cs.top;
        const float lo = __builtin_fmaf(m, cs.top, -hi);
        const float e = __builtin_fmaf(254.0f, __builtin_fabsf(p[i] * cs.up), -hi);
        if (__builtin_fabsf(a - k - 0.5f) <= 0x1p-14f) {
          int c = int(k);
          if (e > lo || (e == lo && (c & 1))) ++c;
          q[i] = uint32_t(t[i] < 0.0f ? -c : c);
        }
      }
    }
  }
  u32x2 v;
#pragma unroll
  for (int w = 0; w < 2; ++w)
    v[w] = (q[4 * w] & 255u) | (q[4 * w + 1] & 255u) << 8 | (q[4 * w + 2] & 255u) << 16 |
           q[4 * w + 3] << 24;
  if (!cs.finite) v = u32x2{0u, 0u};
  return v;
}

// (a row of zeros has an infinite inv where eps is 0; its scale is 0 all the same)
__device__ __forceinline__ float code_scale(uint32_t top_bits, float inv) {
  if (top_bits >= kInfBits) return __builtin_nanf("");
  if (top_bits == 0) return 0.0f;
  return __builtin_bit_cast(float, top_bits) * inv / 127.0f;
}

__device__ __forceinline__ float inv_rms_of(float sum, uint64_t cols, float eps) {
  return 1.0f / __builtin_sqrtf(sum / float(cols) + eps);
}

// ---- forward --------------------------------------------------------------------------

// OUT: what the kernel writes.
constexpr int kOut16 = 0;     // the norm in 16 bits
constexpr int kOutCodes = 1;  // the norm in codes
constexpr int kOutQuant = 2;  // the input in codes

// h = x + residual, as stored (one rounding)
template <int TYPE>
__device__ __forceinline__ u32x4 sum8(u32x4 x, u32x4 r) {
  float a[8], b[8];
  widen8<TYPE>(x, a);
  widen8<TYPE>(r, b);
#pragma unroll
  for (int i = 0; i < 8; ++i) a[i] += b[i];
  return narrow8<TYPE>(a);
}

template <int TYPE, bool RES>
__device__ __forceinline__ u32x4 load_sum(const uint16_t* xr, const uint16_t* rr, uint32_t c,
                                          uint32_t cols) {
  const u32x4 x = load_chunk8(xr, c, cols);
  if constexpr (!RES) return x;
  return sum8<TYPE>(x, load_chunk8(rr, c, cols));
}

// The chunks that a thread holds of its row, to be trimmed: p is the first row of
// the block's, ld their pitch (narrow rows: below kNarrowMaxLd), `rows` how many
// there are from it on.
template <class L, int C>
__device__ __forceinline__ void load_row(const uint16_t* p, uint64_t ld, uint64_t rows,
                                         uint32_t cols, u32x4 (&v)[C]) {
  const uint32_t t = L::lane();
  if constexpr (L::kTpr == 0 || L::kTpr == 64) {
    const uint64_t r = L::kTpr ? uint64_t(wave_id()) : 0;
    const bool live = r < rows;
    const RowWords row(p + (live ? r * ld : 0), live ? cols : 0);
#pragma unroll
    for (int j = 0; j < C; ++j) v[j] = row.load(j * L::threads() + t);
  } else {
    static_assert(C == 1, "a narrow row has a chunk per lane");
    constexpr uint32_t kRows = 64 / (L::kTpr ? L::kTpr : 1);   // a wavefront's
    const uint64_t first = uint64_t(wave_id()) * kRows;
    const uint64_t left = first < rows ? rows - first : 0;
    const uint32_t live = uint32_t(left < kRows ? left : kRows);
    const uint32_t rr = L::row() % kRows;
    const bool in = rr < live && t * 8 < cols;
    // the wavefront's rows as one range-checked buffer; what a chunk takes of the
    // pitch behind its row is trimmed
    const uint32_t bytes =
        live ? uint32_t((live - 1) * uint32_t(ld) * 2 + (cols + 1) / 2 * 4) : 0u;
    const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint16_t*>(p + (live ? first * ld : 0)), 0, int(bytes), kRawBuffer);
    const uint32_t off = in ? rr * uint32_t(ld) * 2 + t * 16 : 0xFFFFFFF0u;
    v[0] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, off, 0, 0));
  }
}

// The weight's chunks of a thread, to be trimmed.
template <class L, int C>
__device__ __forceinline__ void load_weight(const uint16_t* w, uint32_t cols, u32x4 (&v)[C]) {
  const RowWords row(w, cols);
#pragma unroll
  for (int j = 0; j < C; ++j) v[j] = row.load(j * L::threads() + L::lane());
}

// A chunk's share of the sum of squares and of the largest |p|.
template <int TYPE, int OUT>
__device__ __forceinline__ void measure_chunk(u32x4 h, u32x4 w, float& s, uint32_t& m) {
  float f[8];
  widen8<TYPE>(h, f);
  if constexpr (OUT != kOutQuant) {
    float a = 0.0f, b = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a = __builtin_fmaf(f[2 * i], f[2 * i], a);
      b = __builtin_fmaf(f[2 * i + 1], f[2 * i + 1], b);
    }
    s += a + b;
  }
  if constexpr (OUT == kOutCodes) {
    float g[8];
    widen8<TYPE>(w, g);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] *= g[i];
  }
  if constexpr (OUT != kOut16) {
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max_u32(m, __builtin_bit_cast(uint32_t, f[i]) & 0x7FFFFFFFu);
  }
}

template <int TYPE, int OUT, bool STREAM>
__device__ __forceinline__ void finish_chunk(const NormArgs& k, uint64_t row, uint32_t c, u32x4 h,
                                             u32x4 w, float inv, const CodeScale& cs) {
  float f[8], g[8];
  widen8<TYPE>(h, f);
  if constexpr (OUT != kOutQuant) widen8<TYPE>(w, g);
  const uint32_t cols = uint32_t(k.cols);
  if constexpr (OUT == kOut16) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = f[i] * inv * g[i];
    store_chunk8<STREAM>(k.out + row * k.ldo, c, cols, narrow8<TYPE>(f));
  } else {
    if constexpr (OUT == kOutCodes) {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] *= g[i];
    }
    store_codes8<STREAM>(k.codes + row * k.ldc, c, cols, codes8<OUT == kOutQuant>(f, cs));
  }
}

template <int OUT>
__device__ __forceinline__ void finish_row(const NormArgs& k, uint64_t row, float inv,
                                           uint32_t top) {
  if constexpr (OUT == kOut16) {
    if (k.inv_rms) k.inv_rms[row] = inv;
  } else {
    k.scales[row] = code_scale(top, inv);
  }
}

// Norm, norm to codes and codes of rows in registers (Lay): loads, the two row
// sums, results.  HBM bounds it where there are many rows (us and TB/s of what it
// reads and writes, on MI355X: the norm of 8192 x 4096 with its sum 46.1, 5.8; its
// codes of 8192 x 8192 79.3, 5.9; codes of 16384 x 8192 70.0, 5.8), and the chain of
// a load, a combine and a store where there are few (1 x 4096 2.5 us, 64 x 14336
// 4.8).  Odd and narrow rows pay for the lanes without a chunk and for lines shared
// by rows (335544 x 100 at a pitch of 104: norm 79 us, 3.4 TB/s).
template <int TYPE, int OUT, bool RES, bool STREAM, class L>
__global__ __launch_bounds__(L::kMax) void norm_kernel(NormArgs k) {
  constexpr int C = L::kChunks;
  __shared__ typename RowCombine<L>::Lds lds[2];
  const uint32_t cols = uint32_t(k.cols), chunks = (cols + 7) / 8;
  u32x4 w[C];
#pragma unroll
  for (int j = 0; j < C; ++j) w[j] = u32x4{0, 0, 0, 0};
  if constexpr (OUT != kOutQuant) load_weight<L>(k.weight, cols, w);
  int turn = 0;
  // every thread of a block makes the same number of rounds (barriers)
  for (uint64_t base = uint64_t(blockIdx.x) * L::kRows; base < k.rows;
       base += uint64_t(gridDim.x) * L::kRows, turn ^= 1) {
    const uint64_t row = base + L::row();
    const bool live = row < k.rows;
    u32x4 h[C];
    float s = 0.0f;
    uint32_t m = 0;
    load_row<L>(k.x + base * k.ldx, k.ldx, k.rows - base, cols, h);
    if constexpr (RES) {
      u32x4 res[C];
      load_row<L>(k.residual + base * k.ldr, k.ldr, k.rows - base, cols, res);
#pragma unroll
      for (int j = 0; j < C; ++j) h[j] = sum8<TYPE>(h[j], res[j]);
    }
    trim<L>(cols, h);
    if constexpr (OUT != kOutQuant) trim<L>(cols, w);
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const uint32_t c = j * L::threads() + L::lane();
      if (RES && k.sum_out && live && c < chunks)
        store_chunk8<STREAM>(k.sum_out + row * k.lds, c, cols, h[j]);
      measure_chunk<TYPE, OUT>(h[j], w[j], s, m);
    }
    RowCombine<L>::run(s, m, lds, turn);
    const float inv = OUT == kOutQuant ? 1.0f : inv_rms_of(s, k.cols, k.eps);
    const CodeScale cs(m);
    if (!live) continue;
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const uint32_t c = j * L::threads() + L::lane();
      if (c < chunks) finish_chunk<TYPE, OUT, STREAM>(k, row, c, h[j], w[j], inv, cs);
    }
    if (L::lane() == 0) finish_row<OUT>(k, row, inv, m);
  }
}

// Rows too long for the registers: one block per row, walked twice, the second time
// mostly from the caches (norm of 1016 x 33000 60 us, 4.5 TB/s of one read).  The
// second walk forms h again from what the first read, or reads it from
// sum_out (where each thread wrote its own chunks), so that outputs may stand
// where inputs did.
template <int TYPE, int OUT, bool RES>
__global__ __launch_bounds__(1024) void norm_loop_kernel(NormArgs k) {
  __shared__ typename RowCombine<Lay<0, 1024, 1>>::Lds lds[2];
  const uint32_t cols = uint32_t(k.cols), chunks = (cols + 7) / 8;
  int turn = 0;
  for (uint64_t row = blockIdx.x; row < k.rows; row += gridDim.x, turn ^= 1) {
    const uint16_t* xr = k.x + row * k.ldx;
    const uint16_t* rr = k.residual + row * k.ldr;
    float s = 0.0f;
    uint32_t m = 0;
    for (uint32_t c = threadIdx.x; c < chunks; c += 1024) {
      const u32x4 h = load_sum<TYPE, RES>(xr, rr, c, cols);
      if (RES && k.sum_out) store_chunk8<false>(k.sum_out + row * k.lds, c, cols, h);
      const u32x4 w = OUT == kOutCodes ? load_chunk8(k.weight, c, cols) : u32x4{0, 0, 0, 0};
      measure_chunk<TYPE, OUT>(h, w, s, m);
    }
    RowCombine<Lay<0, 1024, 1>>::run(s, m, lds, turn);
    const float inv = OUT == kOutQuant ? 1.0f : inv_rms_of(s, k.cols, k.eps);
    const CodeScale cs(m);
    for (uint32_t c = threadIdx.x; c < chunks; c += 1024) {
      const u32x4 h = RES && k.sum_out ? load_chunk8(k.sum_out + row * k.lds, c, cols)
                                       : load_sum<TYPE, RES>(xr, rr, c, cols);
      const u32x4 w = OUT != kOutQuant ? load_chunk8(k.weight, c, cols) : u32x4{0, 0, 0, 0};
      finish_chunk<TYPE, OUT, false>(k, row, c, h, w, inv, cs);
    }
    if (threadIdx.x == 0) finish_row<OUT>(k, row, inv, m);
  }
}

constexpr uint64_t kMaxGrid = 0x7FFFFFFF / 1024;  // the runtime counts threads in 32 bits

hipError_t launch_rows_kernel(const void* fn, uint64_t blocks, int threads, void** args,
                              const armx_config* cfg, hipStream_t stream, bool first = true,
                              bool last = true) {
  return launch_kernel(fn, dim3(unsigned(blocks)), dim3(unsigned(threads)), args, 0, stream,
                       cfg && first ? static_cast<hipEvent_t>(cfg->start_event) : nullptr,
                       cfg && last ? static_cast<hipEvent_t>(cfg->stop_event) : nullptr);
}

// Calls CASE(Lay) for the layout of shape `s`, if its rows lie in registers.
#define ARMX_OF_SHAPE(s, CASE)                                                       \
  do {                                                                               \
    if ((s).chunks == 1 && (s).threads == 8) CASE(ARMX_LAY(8, 0, 1));                \
    if ((s).chunks == 1 && (s).threads == 16) CASE(ARMX_LAY(16, 0, 1));              \
    if ((s).chunks == 1 && (s).threads == 32) CASE(ARMX_LAY(32, 0, 1));              \
    if ((s).chunks == 1 && (s).threads == 64) CASE(ARMX_LAY(64, 0, 1));              \
    if ((s).chunks == 1 && (s).threads > 64) CASE(ARMX_LAY(0, 512, 1));              \
    if ((s).chunks == 2) CASE(ARMX_LAY(0, 512, 2));                                  \
    if ((s).chunks == 4 && (s).threads <= 512) CASE(ARMX_LAY(0, 512, 4));            \
  } while (0)
#define ARMX_LAY(...) Lay<__VA_ARGS__>
typedef Lay<0, 1024, 4> WidestLay;

// Narrow rows of a larger pitch take a wavefront each: a wavefront's rows, at most
// 8, are reached by 32-bit offsets.  A row's bits stay the same, the lanes in front
// adding as before and the others 0.
constexpr uint64_t kNarrowMaxLd = uint64_t(1) << 27;
RowShape for_pitch(RowShape s, uint64_t ld) {
  if (s.threads < 64 && ld >= kNarrowMaxLd) s.threads = 64;
  return s;
}

bool is_widest(const RowShape& s) { return s.chunks == 4 && s.threads > 512; }

// Columns of a block that sums dweight apart from dx: 64, whole lines of a row, but 32
// on rows of up to 320 chunks, of which 64 would make few blocks (us, 64 / 32: 500 x 333
// 6.2 / 4.3, 515 x 2056 6.7 / 6.2; 1000 x 4096 9.9 / 11.2, 256 x 8192 6.0 / 7.1).
bool half_columns(const RowShape& s) { return s.chunks == 1 && s.threads <= 320; }
uint64_t column_blocks(const RowShape& s, uint64_t cols) {
  const uint64_t width = half_columns(s) ? 32 : 64;
  return (cols + width - 1) / width;
}

// Threads of a block and the rows it takes at a time.
int block_threads(const RowShape& s) { return s.threads > 64 ? s.threads : kRowBlock; }
uint64_t block_rows(const RowShape& s) { return s.threads > 64 ? 1 : kRowBlock / s.threads; }

template <int TYPE, int OUT, bool RES>
hipError_t launch_norm_typed(const NormArgs& a, const armx_config* cfg, hipStream_t stream) {
  const RowShape s = for_pitch(row_shape(a.cols), RES && a.ldr > a.ldx ? a.ldr : a.ldx);
  const bool stream_out = a.rows * a.cols >= kStreamValues;
  const void* fn = nullptr;
#define ARMX_NORM_CASE(...)                                                             \
  fn = stream_out ? reinterpret_cast<const void*>(&norm_kernel<TYPE, OUT, RES, true, __VA_ARGS__>) \
                  : reinterpret_cast<const void*>(&norm_kernel<TYPE, OUT, RES, false, __VA_ARGS__>)
  ARMX_OF_SHAPE(s, ARMX_NORM_CASE);
  if (is_widest(s)) ARMX_NORM_CASE(WidestLay);
#undef ARMX_NORM_CASE
  if (s.chunks == 0) fn = reinterpret_cast<const void*>(&norm_loop_kernel<TYPE, OUT, RES>);
  // One block per row group, the next blocks' loads hiding what one waits for.  Where
  // codes are all that is written, four times the blocks that fill the card, which
  // walk on (335544 x 100 27.0 -> 24.6 us, 13421 x 2500 25.0 -> 23.6; with a norm the
  // other way, its codes 64.6 -> 72.5 and its 16-bit values 79.6 -> 86.2; on longer
  // rows too, 16384 x 8192 70.1 -> 72.3).
  uint64_t blocks = (a.rows + block_rows(s) - 1) / block_rows(s);
  const uint64_t most = OUT == kOutQuant && s.chunks == 1
                            ? uint64_t(current_cu_count()) * 32 * 256 / block_threads(s)
                            : kMaxGrid;
  if (blocks > most) blocks = most;
  NormArgs copy = a;
  void* args[] = {&copy};
  return launch_rows_kernel(fn, blocks, block_threads(s), args, cfg, stream);
}

template <int TYPE>
hipError_t launch_norm_out(const NormArgs& a, const armx_config* cfg, hipStream_t stream) {
  if (!a.weight) return launch_norm_typed<TYPE, kOutQuant, false>(a, cfg, stream);
  if (a.codes)
    return a.residual ? launch_norm_typed<TYPE, kOutCodes, true>(a, cfg, stream)
                      : launch_norm_typed<TYPE, kOutCodes, false>(a, cfg, stream);
  return a.residual ? launch_norm_typed<TYPE, kOut16, true>(a, cfg, stream)
                    : launch_norm_typed<TYPE, kOut16, false>(a, cfg, stream);
}

// ---- backward ---------------------------------------------------------------------------

// One chunk's share of the row's sum of g h.
template <int TYPE>
__device__ __forceinline__ float dot_chunk(u32x4 dy, u32x4 h, u32x4 w, float dot) {
  float fy[8], fh[8], fw[8];
  widen8<TYPE>(dy, fy);
  widen8<TYPE>(h, fh);
  widen8<TYPE>(w, fw);
#pragma unroll
  for (int i = 0; i < 8; ++i) dot = __builtin_fmaf(fy[i] * fw[i], fh[i], dot);
  return dot;
}

// dx of a chunk; f = inv^2 mean(g h)
template <int TYPE, bool DSUM>
__device__ __forceinline__ u32x4 grad_chunk(u32x4 dy, u32x4 h, u32x4 w, u32x4 ds, float inv,
                                            float f) {
  float fy[8], fh[8], fw[8], fd[8];
  widen8<TYPE>(dy, fy);
  widen8<TYPE>(h, fh);
  widen8<TYPE>(w, fw);
  if constexpr (DSUM) widen8<TYPE>(ds, fd);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    fy[i] = inv * (fy[i] * fw[i] - fh[i] * f);
    if constexpr (DSUM) fy[i] += fd[i];
  }
  return narrow8<TYPE>(fy);
}

// dx of the chunks of a row that a thread holds.
template <int TYPE, bool DSUM, bool STREAM, class L, int C>
__device__ __forceinline__ void store_grads(const NormBackwardArgs& k, uint64_t row, float inv,
                                            float dot, const u32x4 (&dy)[C], const u32x4 (&h)[C],
                                            const u32x4 (&ds)[C], const u32x4 (&w)[C]) {
  const uint32_t cols = uint32_t(k.cols), chunks = (cols + 7) / 8;
  const float f = inv * inv * (dot / float(k.cols));
#pragma unroll
  for (int j = 0; j < C; ++j) {
    const uint32_t c = j * L::threads() + L::lane();
    if (c < chunks)
      store_chunk8<STREAM>(k.dx + row * k.ldx, c, cols,
                           grad_chunk<TYPE, DSUM>(dy[j], h[j], w[j], ds[j], inv, f));
  }
}

// HBM bounds it: 8192 x 4096 with dsum 47.9 us, and 4.7 for norm_join_kernel, against
// 51.8 for its bytes at a large copy's rate.
// Block b takes the row groups b, b + blocks, ...; every thread keeps the
// dweight sums of its own columns in registers over the block's rows.  A block
// of several rows at a time adds its row groups' sums through LDS, in order.
template <int TYPE, bool DSUM, bool STREAM, class L>
__global__ __launch_bounds__(L::kMax) void norm_backward_kernel(NormBackwardArgs k, float* dst,
                                                               uint64_t pitch) {
  constexpr int C = L::kChunks;
  __shared__ typename RowCombine<L>::Lds lds[2];
  __shared__ float part[L::kRows > 1 ? kRowBlock * 8 : 1];
  const uint32_t cols = uint32_t(k.cols);
  u32x4 w[C];
  float acc[C][8];
#pragma unroll
  for (int j = 0; j < C; ++j) {
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[j][i] = 0.0f;
  }
  load_weight<L>(k.weight, cols, w);
  // One row group's values; with kAhead the next group's are on their way while
  // this one's are combined (8192 x 4096 56.6 -> 54.3 us; at four chunks a thread,
  // where the registers no longer hold both, 62 -> 71).
  struct Rows {
    u32x4 dy[C], h[C], ds[C];
    float inv;
  };
  constexpr bool kAhead = C <= 2;
  auto load = [&](uint64_t base) __attribute__((always_inline)) {
    Rows v;
    const uint64_t row = base + L::row(), left = k.rows - base;
    v.inv = row < k.rows ? k.inv_rms[row] : 0.0f;
    load_row<L>(k.dy + base * k.ldy, k.ldy, left, cols, v.dy);
    load_row<L>(k.h + base * k.ldh, k.ldh, left, cols, v.h);
    if constexpr (DSUM) load_row<L>(k.dsum + base * k.ldd, k.ldd, left, cols, v.ds);
    return v;
  };
  int turn = 0;
  const uint64_t stride = uint64_t(gridDim.x) * L::kRows;
  Rows ahead;
  if constexpr (kAhead) ahead = load(uint64_t(blockIdx.x) * L::kRows);
  for (uint64_t base = uint64_t(blockIdx.x) * L::kRows; base < k.rows; base += stride, turn ^= 1) {
    const uint64_t row = base + L::row();
    const bool live = row < k.rows;
    Rows now;
    if constexpr (kAhead) {
      now = ahead;
      if (base + stride < k.rows) ahead = load(base + stride);
    } else {
      now = load(base);
    }
    trim<L>(cols, now.dy);
    trim<L>(cols, now.h);
    trim<L>(cols, w);
    float dot = 0.0f;
#pragma unroll
    for (int j = 0; j < C; ++j) {
      dot = dot_chunk<TYPE>(now.dy[j], now.h[j], w[j], dot);
      if (live) {
        float fy[8], fh[8];
        widen8<TYPE>(now.dy[j], fy);
        widen8<TYPE>(now.h[j], fh);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[j][i] = __builtin_fmaf(fy[i], fh[i] * now.inv, acc[j][i]);
      }
    }
    uint32_t unused = 0;
    RowCombine<L>::run(dot, unused, lds, turn);
    if (live)
      store_grads<TYPE, DSUM, STREAM, L>(k, row, now.inv, dot, now.dy, now.h, now.ds, w);
  }
  if constexpr (L::kRows > 1) {
    constexpr uint32_t kPitch = L::kTpr * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) part[L::row() * kPitch + L::lane() * 8 + i] = acc[0][i];
    __syncthreads();
    for (uint32_t e = threadIdx.x; e < cols; e += kRowBlock) {
      float v = part[e];
      for (int r = 1; r < L::kRows; ++r) v += part[r * kPitch + e];
      dst[uint64_t(blockIdx.x) * pitch + e] = v;
    }
  } else {
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const uint32_t c = j * L::threads() + L::lane();
      float* d = dst + uint64_t(blockIdx.x) * pitch + uint64_t(c) * 8;
      if (c * 8 + 8 <= cols) {
        reinterpret_cast<floatx4*>(d)[0] = floatx4{acc[j][0], acc[j][1], acc[j][2], acc[j][3]};
        reinterpret_cast<floatx4*>(d)[1] = floatx4{acc[j][4], acc[j][5], acc[j][6], acc[j][7]};
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (c * 8 + i < cols) d[i] = acc[j][i];
      }
    }
  }
}

// A chunk that starts at any value.
typedef u32x4 __attribute__((aligned(2))) u32x4_any;

// dweight over all rows for 8 LANES columns (number `block` of them), by a whole block:
// LANES lanes take a row's, rows in steps of the block's, FLIGHT in flight.  part: 64
// floats per wavefront.
template <int TYPE, int LANES, int FLIGHT>
__device__ __forceinline__ void sum_columns_in(const NormBackwardArgs& k, uint32_t block,
                                            float (*part)[64]) {
  const uint32_t cols = uint32_t(k.cols), chunks = (cols + 7) / 8;
  const uint32_t c = block * LANES + threadIdx.x % LANES;
  // The last chunk is read as the row's last 8 values, without a branch (a lane with
  // none too); those in front of the chunk are the lane's before it.
  const uint32_t e0 = c * 8 + 8 <= cols ? c * 8 : cols - 8;
  const uint32_t step = blockDim.x / LANES;
  float acc[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  for (uint64_t r = threadIdx.x / LANES; r < k.rows; r += FLIGHT * step) {
    u32x4 y[FLIGHT], x[FLIGHT];
    float inv[FLIGHT];
#pragma unroll
    for (int q = 0; q < FLIGHT; ++q) {
      // a row past the last is read as this thread's first, and not added
      const uint64_t rq = r + q * step < k.rows ? r + q * step : r;
      inv[q] = k.inv_rms[rq];
      if (cols >= 8) {
        y[q] = *reinterpret_cast<const u32x4_any*>(k.dy + rq * k.ldy + e0);
        x[q] = *reinterpret_cast<const u32x4_any*>(k.h + rq * k.ldh + e0);
      } else {
        y[q] = c == 0 ? load_chunk8(k.dy + rq * k.ldy, 0, cols) : u32x4{0, 0, 0, 0};
        x[q] = c == 0 ? load_chunk8(k.h + rq * k.ldh, 0, cols) : u32x4{0, 0, 0, 0};
      }
    }
#pragma unroll
    for (int q = 0; q < FLIGHT; ++q) {
      if (r + q * step >= k.rows) continue;
      float fy[8], fh[8];
      widen8<TYPE>(y[q], fy);
      widen8<TYPE>(x[q], fh);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = __builtin_fmaf(fy[i], fh[i] * inv[q], acc[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {   // over the wavefront's rows: lanes LANES and more apart
    float v = acc[i];
    if constexpr (LANES == 4) v += dpp<kDppRor4>(v);
    v += dpp<kDppRor8>(v);
    v = add_xor16(v);
    v = add_xor32(v);
    const uint32_t e = (cols >= 8 ? e0 : c * 8) + i;
    if (lane_id() < LANES && c < chunks && e >= c * 8)
      part[wave_id()][e - block * (8 * LANES)] = v;
  }
  __syncthreads();
  const uint32_t e = block * (8 * LANES) + threadIdx.x;
  if (threadIdx.x < 8 * LANES && e < cols) {
    float v = part[0][threadIdx.x];
    const int waves = num_waves();
    for (int q = 1; q < waves; ++q) v += part[q][threadIdx.x];
    k.dweight[e] = v;
  }
}

// Eight rows in flight where four would take a second round (us: 515 x 2056 7.1 -> 6.7,
// 300 x 16384 11.8 -> 11.1; with one round 64 x 4096 3.3 -> 3.8, and where the row
// blocks' registers fill the compute units 559 x 60001 90 -> 93).
template <int TYPE, bool LONG>
__device__ __forceinline__ void sum_columns(const NormBackwardArgs& k, uint32_t block,
                                            float (*part)[64], bool half) {
  const uint32_t lanes = half ? 4 : 8;
  const bool one_round = k.rows <= 4 * (blockDim.x / lanes);
  if constexpr (LONG) {
    sum_columns_in<TYPE, 8, 4>(k, block, part);
  } else if (half) {
    if (one_round)
      sum_columns_in<TYPE, 4, 4>(k, block, part);
    else
      sum_columns_in<TYPE, 4, 8>(k, block, part);
  } else {
    if (one_round)
      sum_columns_in<TYPE, 8, 4>(k, block, part);
    else
      sum_columns_in<TYPE, 8, 8>(k, block, part);
  }
}

// dx and dweight apart, in one launch without a workspace: the first `col_blocks`
// blocks each sum dweight over all rows for 64 or 32 columns (`half`), reading dy and
// h once more, and the others make the dx of their row groups.  With few rows (515 x
// 2056 6.2 us) the column blocks' rounds of loads bound it, with long ones the second
// read and, at 128 registers a thread, one block per compute unit (1024 x 32768 with
// dsum 94 us, 3.6 TB/s of one read).
template <int TYPE, bool DSUM, class L>
__global__ __launch_bounds__(L::kMax) void norm_backward_apart_kernel(NormBackwardArgs k,
                                                                     unsigned col_blocks,
                                                                     bool half) {
  constexpr int C = L::kChunks;
  __shared__ typename RowCombine<L>::Lds lds[2];
  __shared__ float part[L::kMax / 64][64];
  if (blockIdx.x < col_blocks) {
    sum_columns<TYPE, (L::kMax > 512)>(k, blockIdx.x, part, half);
    return;
  }
  const uint32_t cols = uint32_t(k.cols);
  u32x4 w[C];
  load_weight<L>(k.weight, cols, w);
  int turn = 0;
  const uint64_t stride = uint64_t(gridDim.x - col_blocks) * L::kRows;
  for (uint64_t base = uint64_t(blockIdx.x - col_blocks) * L::kRows; base < k.rows;
       base += stride, turn ^= 1) {
    const uint64_t row = base + L::row(), left = k.rows - base;
    const bool live = row < k.rows;
    u32x4 dy[C], h[C], ds[C];
    load_row<L>(k.dy + base * k.ldy, k.ldy, left, cols, dy);
    load_row<L>(k.h + base * k.ldh, k.ldh, left, cols, h);
    if constexpr (DSUM && C < 4) load_row<L>(k.dsum + base * k.ldd, k.ldd, left, cols, ds);
    const float inv = live ? k.inv_rms[row] : 0.0f;
    trim<L>(cols, dy);
    trim<L>(cols, h);
    trim<L>(cols, w);
    float dot = 0.0f;
#pragma unroll
    for (int j = 0; j < C; ++j) dot = dot_chunk<TYPE>(dy[j], h[j], w[j], dot);
    uint32_t unused = 0;
    // the registers do not hold dsum's four chunks during the sums above (16-bit dx of
    // 1677 x 20000 96.5 -> 92.7 us)
    if constexpr (DSUM && C == 4) load_row<L>(k.dsum + base * k.ldd, k.ldd, left, cols, ds);
    RowCombine<L>::run(dot, unused, lds, turn);
    if (live) store_grads<TYPE, DSUM, false, L>(k, row, inv, dot, dy, h, ds, w);
  }
}

// The same for rows too long for the registers, which are walked twice, four chunks
// a thread at a time.
template <int TYPE, bool DSUM>
__global__ __launch_bounds__(1024) void norm_backward_loop_kernel(NormBackwardArgs k,
                                                                  unsigned col_blocks,
                                                                  bool half) {
  typedef Lay<0, 1024, 4> L;
  __shared__ typename RowCombine<L>::Lds lds[2];
  __shared__ float part[16][64];
  if (blockIdx.x < col_blocks) {
    sum_columns<TYPE, true>(k, blockIdx.x, part, half);
    return;
  }
  const uint32_t cols = uint32_t(k.cols), chunks = (cols + 7) / 8;
  const RowWords wr(k.weight, cols);
  // a whole row's loads of one chunk; values past the row cleared
  auto cut = [&](u32x4 v, uint32_t c) __attribute__((always_inline)) {
    if (cols & 1) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c * 8 + 2 * i + 1 == cols) v[i] &= 0xFFFFu;
    }
    return v;
  };
  int turn = 0;
  for (uint64_t row = blockIdx.x - col_blocks; row < k.rows;
       row += gridDim.x - col_blocks, turn ^= 1) {
    const RowWords yr(k.dy + row * k.ldy, cols), hr(k.h + row * k.ldh, cols);
    const float inv = k.inv_rms[row];
    float dot = 0.0f;
    for (uint32_t c0 = threadIdx.x; c0 < chunks; c0 += 4096) {
      u32x4 y[4], h[4], w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        y[j] = yr.load(c0 + j * 1024);
        h[j] = hr.load(c0 + j * 1024);
        w[j] = wr.load(c0 + j * 1024);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t c = c0 + j * 1024;
        dot = dot_chunk<TYPE>(cut(y[j], c), cut(h[j], c), cut(w[j], c), dot);
      }
    }
    uint32_t unused = 0;
    RowCombine<L>::run(dot, unused, lds, turn);
    const float f = inv * inv * (dot / float(k.cols));
    const RowWords dr(DSUM ? k.dsum + row * k.ldd : nullptr, DSUM ? cols : 0);
    for (uint32_t c0 = threadIdx.x; c0 < chunks; c0 += 4096) {
      u32x4 y[4], h[4], w[4], d[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        y[j] = yr.load(c0 + j * 1024);
        h[j] = hr.load(c0 + j * 1024);
        w[j] = wr.load(c0 + j * 1024);
        if constexpr (DSUM) d[j] = dr.load(c0 + j * 1024);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t c = c0 + j * 1024;
        if (c < chunks)
          store_chunk8<false>(k.dx + row * k.ldx, c, cols,
                              grad_chunk<TYPE, DSUM>(y[j], h[j], w[j], d[j], inv, f));
      }
    }
  }
}

// dweight[c] = the sum of the blocks' partial sums: 4 consecutive columns per
// thread, kJoinParts threads of a block sharing the partial sums of its columns
// (part t takes t, t + kJoinParts, ..., eight loads in flight), whose sums are
// then added in order.
constexpr int kJoinCols = 32, kJoinParts = 32;
__global__ __launch_bounds__(kJoinCols / 4 * kJoinParts) void norm_join_kernel(
    const float* partials, uint64_t blocks, uint64_t pitch, uint64_t cols, float* dweight) {
  constexpr int kQuads = kJoinCols / 4;
  __shared__ floatx4 part[kJoinParts][kQuads];
  const uint32_t tc = threadIdx.x % kQuads, tp = threadIdx.x / kQuads;
  // the pitch is a multiple of 64, so a quad past the columns is still inside it
  const uint64_t c = uint64_t(blockIdx.x) * kJoinCols + tc * 4;
  const floatx4* src = reinterpret_cast<const floatx4*>(partials + c);
  floatx4 v = {0.0f, 0.0f, 0.0f, 0.0f};
  for (uint64_t b = tp; b < blocks; b += 8 * kJoinParts) {
    floatx4 t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint64_t bi = b + uint64_t(i) * kJoinParts;
      t[i] = src[(bi < blocks ? bi : b) * (pitch / 4)];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (b + uint64_t(i) * kJoinParts < blocks) v += t[i];
  }
  part[tp][tc] = v;
  __syncthreads();
  if (tp == 0) {
    const uint64_t last = blocks < kJoinParts ? blocks : kJoinParts;
    for (uint64_t t = 1; t < last; ++t) v += part[t][tc];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (c + i < cols) dweight[c + i] = v[i];
  }
}

// Whether two matrices of a call may share memory (their extents meet).
bool meet(const void* a, uint64_t lda, const void* b, uint64_t ldb, uint64_t rows, uint64_t cols) {
  const char* pa = static_cast<const char*>(a);
  const char* pb = static_cast<const char*>(b);
  return pa < pb + 2 * ((rows - 1) * ldb + cols) && pb < pa + 2 * ((rows - 1) * lda + cols);
}

RowShape backward_shape(const NormBackwardArgs& a, const NormBackwardPlan& plan) {
  uint64_t ld = a.ldy > a.ldh ? a.ldy : a.ldh;
  if (a.dsum && a.ldd > ld) ld = a.ldd;
  return for_pitch(plan.shape, ld);
}

template <int TYPE, bool DSUM>
hipError_t launch_backward_apart(const NormBackwardArgs& a, const NormBackwardPlan& plan,
                                 const armx_config* cfg, hipStream_t stream) {
  const RowShape s = backward_shape(a, plan);
  const void* fn = nullptr;
#define ARMX_NORM_CASE(...) \
  fn = reinterpret_cast<const void*>(&norm_backward_apart_kernel<TYPE, DSUM, __VA_ARGS__>)
  ARMX_OF_SHAPE(s, ARMX_NORM_CASE);
  if (is_widest(s)) ARMX_NORM_CASE(WidestLay);
#undef ARMX_NORM_CASE
  if (s.chunks == 0) fn = reinterpret_cast<const void*>(&norm_backward_loop_kernel<TYPE, DSUM>);
  NormBackwardArgs copy = a;
  unsigned col_blocks = unsigned(column_blocks(plan.shape, a.cols));
  bool half = half_columns(plan.shape);
  void* args[] = {&copy, &col_blocks, &half};
  const uint64_t row_blocks = plan.blocks - col_blocks;
  // dx where dy or h is: every column's sums before any row's gradient
  if (!meet(a.dx, a.ldx, a.dy, a.ldy, a.rows, a.cols) &&
      !meet(a.dx, a.ldx, a.h, a.ldh, a.rows, a.cols))
    return launch_rows_kernel(fn, plan.blocks, plan.block, args, cfg, stream);
  const hipError_t e =
      launch_rows_kernel(fn, col_blocks, plan.block, args, cfg, stream, true, false);
  if (e != hipSuccess) return e;
  col_blocks = 0;
  return launch_rows_kernel(fn, row_blocks, plan.block, args, cfg, stream, false, true);
}

template <int TYPE, bool DSUM>
hipError_t launch_backward_typed(const NormBackwardArgs& a, const NormBackwardPlan& plan,
                                 const armx_config* cfg, hipStream_t stream) {
  if (plan.apart) return launch_backward_apart<TYPE, DSUM>(a, plan, cfg, stream);
  const RowShape s = backward_shape(a, plan);
  const bool stream_out = a.rows * a.cols >= kStreamValues;
  const void* fn = nullptr;
#define ARMX_NORM_CASE(...)                                                                    \
  fn = stream_out                                                                              \
           ? reinterpret_cast<const void*>(&norm_backward_kernel<TYPE, DSUM, true, __VA_ARGS__>) \
           : reinterpret_cast<const void*>(&norm_backward_kernel<TYPE, DSUM, false, __VA_ARGS__>)
  ARMX_OF_SHAPE(s, ARMX_NORM_CASE);
#undef ARMX_NORM_CASE
  NormBackwardArgs copy = a;
  float* dst = a.partials;
  uint64_t pitch = plan.pitch;
  void* args[] = {&copy, &dst, &pitch};
  hipError_t e = launch_rows_kernel(fn, plan.blocks, plan.block, args, cfg, stream, true, false);
  if (e != hipSuccess) return e;
  const float* partials = a.partials;
  uint64_t blocks = plan.blocks, cols = a.cols;
  float* dweight = a.dweight;
  void* join_args[] = {&partials, &blocks, &pitch, &cols, &dweight};
  return launch_rows_kernel(reinterpret_cast<const void*>(&norm_join_kernel),
                            (cols + kJoinCols - 1) / kJoinCols, kJoinCols / 4 * kJoinParts,
                            join_args, cfg, stream, false, true);
}

}  // namespace

NormBackwardPlan plan_norm_backward(uint64_t rows, uint64_t cols, int cu_count) {
  NormBackwardPlan p;
  p.shape = row_shape(cols);
  p.block = block_threads(p.shape);
  if (rows == 0 || cols == 0) return p;
  const uint64_t groups = (rows + block_rows(p.shape) - 1) / block_rows(p.shape);
  // Few rows: the column blocks read them in a few rounds, from the caches (us,
  // partial sums / columns apart: 512 x 100 5.5 / 3.5, 1024 x 100 5.6 / 4.6, 1536 x 256
  // 6.0 / 5.8, 2048 x 256 5.9 / 7.0, 512 x 1024 7.3 / 4.8, 1024 x 1024 9.2 / 9.3, 1536 x
  // 1024 10.3 / 13.1, 1024 x 8192 17.9 / 14.0, 2048 x 4096 15.4 / 16.8).
  // Rows of more than 16384 values, however many: the registers do not hold the
  // partial sums too (512 x 32768 106 / 39, 559 x 60001 294 / 104).
  p.apart = (rows <= 1024 && rows * cols <= uint64_t(1) << 23) ||
            is_widest(p.shape) || p.shape.chunks == 0;
  if (p.apart) {
    p.blocks = column_blocks(p.shape, cols) + (groups < kMaxGrid / 2 ? groups : kMaxGrid / 2);
    return p;
  }
  // Every block's dweight sums are written and read again, so fewer blocks move
  // less, and too few leave loads unsent: about 8 wavefronts per compute unit.
  // Measured on MI355X at 4, 8 and 16 of them (us): 8192 x 4096 55.4, 54.3, 61.2;
  // 32768 x 128 11.6, 10.7, 11.7.
  const uint64_t most = uint64_t(cu_count) * ((511 + p.block) / p.block);
  p.blocks = groups < most ? groups : most;
  p.pitch = (cols + 63) / 64 * 64;
  p.ws_bytes = size_t(p.blocks * p.pitch * sizeof(float));
  return p;
}

hipError_t launch_norm(const NormArgs& args, const armx_config* cfg, hipStream_t stream) {
  return args.type == ARMX_F16 ? launch_norm_out<ARMX_F16>(args, cfg, stream)
                               : launch_norm_out<ARMX_BF16>(args, cfg, stream);
}

hipError_t launch_norm_backward(const NormBackwardArgs& a, const NormBackwardPlan& plan,
                                const armx_config* cfg, hipStream_t stream) {
  if (a.type == ARMX_F16)
    return a.dsum ? launch_backward_typed<ARMX_F16, true>(a, plan, cfg, stream)
                  : launch_backward_typed<ARMX_F16, false>(a, plan, cfg, stream);
  return a.dsum ? launch_backward_typed<ARMX_BF16, true>(a, plan, cfg, stream)
                : launch_backward_typed<ARMX_BF16, false>(a, plan, cfg, stream);
}

}  // namespace armx
