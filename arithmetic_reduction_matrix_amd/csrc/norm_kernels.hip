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

RowShape row_shape(uint64_t cols) {
  const uint64_t n = (cols + kRowVec - 1) / kRowVec;  // 16-byte chunks
  if (n <= 8) return {8, 1};
  if (n <= 16) return {16, 1};
  if (n <= 32) return {32, 1};
  if (n <= 64) return {64, 1};
  if (n <= 128) return {128, 1};
  if (n <= 256) return {256, 1};
  if (n <= 512) return {512, 1};
  if (n <= 1024) return {512, 2};
  if (n <= 2048) return {512, 4};
  if (n <= 4096) return {1024, 4};
  return {1024, 0};
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
// holds one value past the row; trim() clears it.
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

// Applied where the values are used: it waits for them, and at the loads it would
// hold up those behind (48643 x 313 backward, rows read ahead: 66 against 37 us).
template <int TPR, int C>
__device__ __forceinline__ void trim(uint32_t t, uint32_t cols, u32x4 (&v)[C]) {
  if (cols % 2 == 0) return;
#pragma unroll
  for (int j = 0; j < C; ++j) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if ((j * TPR + t) * 8 + 2 * i + 1 == cols) v[j][i] &= 0xFFFFu;
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
// threads.  TPR > 64: over the row's wavefronts through LDS, added in wavefront
// order by every thread alike; the block's ROWS rows each have a place.
template <int TPR, int ROWS>
struct RowCombine {
  static constexpr int kWaves = TPR > 64 ? TPR / 64 : 1;
  struct Lds {
    float s[ROWS][kWaves];
    uint32_t m[ROWS][kWaves];
  };
  // `turn` alternates between the two halves of `lds` from row to row, so one
  // barrier per row is enough
  __device__ __forceinline__ static void run(float& s, uint32_t& m, Lds* lds, int turn) {
    constexpr int levels = log2_of(TPR > 64 ? 64 : TPR);
    s = lane_tree(s, levels);
    m = lane_max(m, levels);
    if constexpr (TPR > 64) {
      Lds& l = lds[turn];
      const int row = wave_id() / kWaves;
      if (lane_id() == 0) {
        l.s[row][wave_id() % kWaves] = s;
        l.m[row][wave_id() % kWaves] = m;
      }
      __syncthreads();
      s = 0.0f;
      m = 0;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        s += l.s[row][w];
        m = max_u32(m, l.m[row][w]);
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
// at least 2^-9 |v| / 127 from one, since 2 * 127 p and every odd multiple of top
// are whole multiples of the smaller's last bit; only true halves, which are common
// (one value in some tens where top has few bits), need care.  One correction,
// t + (127 p - t top) / top with the difference exact, gives them exactly.
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

__device__ __forceinline__ float code_scale(uint32_t top_bits, float inv) {
  if (top_bits >= kInfBits) return __builtin_nanf("");
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

// Chunks t, t + TPR, ... of a row that TPR threads share, to be trimmed: p is the
// first row of the block's, ld its pitch, `live` whether this thread's row exists.
template <int TPR, int C>
__device__ __forceinline__ void load_row(const uint16_t* p, uint64_t ld, bool live, uint32_t t,
                                         uint32_t cols, u32x4 (&v)[C]) {
  if constexpr (TPR >= 64) {
    const uint64_t r = uint64_t(__builtin_amdgcn_readfirstlane(int(threadIdx.x / TPR)));
    const uint32_t count = __builtin_amdgcn_readfirstlane(live ? int(cols) : 0);
    const RowWords row(p + (count ? r * ld : 0), count);
#pragma unroll
    for (int j = 0; j < C; ++j) v[j] = row.load(j * TPR + t);
  } else {
    const uint32_t chunks = (cols + 7) / 8;
#pragma unroll
    for (int j = 0; j < C; ++j) {
      v[j] = u32x4{0, 0, 0, 0};
      if (live && j * TPR + t < chunks)
        v[j] = load_chunk8(p + (threadIdx.x / TPR) * ld, j * TPR + t, cols);
    }
  }
}

// The weight's chunks of a thread, to be trimmed.
template <int TPR, int C>
__device__ __forceinline__ void load_weight(const uint16_t* w, uint32_t t, uint32_t cols,
                                            u32x4 (&v)[C]) {
  const RowWords row(w, cols);
#pragma unroll
  for (int j = 0; j < C; ++j) v[j] = row.load(j * TPR + t);
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

// Rows in registers: TPR threads per row, C chunks each; a block of at least
// kRowBlock threads takes block / TPR rows at a time.
template <int TYPE, int OUT, bool RES, bool STREAM, int TPR, int C>
__global__ __launch_bounds__(TPR > kRowBlock ? TPR : kRowBlock) void norm_kernel(NormArgs k) {
  constexpr int kBlock = TPR > kRowBlock ? TPR : kRowBlock;
  constexpr int kRows = kBlock / TPR;
  __shared__ typename RowCombine<TPR, kRows>::Lds lds[2];
  const uint32_t t = threadIdx.x % TPR, cols = uint32_t(k.cols);
  const uint32_t chunks = (cols + 7) / 8;
  u32x4 w[C];
#pragma unroll
  for (int j = 0; j < C; ++j) w[j] = u32x4{0, 0, 0, 0};
  if constexpr (OUT != kOutQuant) load_weight<TPR>(k.weight, t, cols, w);
  int turn = 0;
  // every thread of a block makes the same number of rounds (barriers)
  for (uint64_t base = uint64_t(blockIdx.x) * kRows; base < k.rows;
       base += uint64_t(gridDim.x) * kRows, turn ^= 1) {
    const uint64_t row = base + threadIdx.x / TPR;
    const bool live = row < k.rows;
    u32x4 h[C];
    float s = 0.0f;
    uint32_t m = 0;
    load_row<TPR>(k.x + base * k.ldx, k.ldx, live, t, cols, h);
    if constexpr (RES) {
      u32x4 res[C];
      load_row<TPR>(k.residual + base * k.ldr, k.ldr, live, t, cols, res);
#pragma unroll
      for (int j = 0; j < C; ++j) h[j] = sum8<TYPE>(h[j], res[j]);
    }
    trim<TPR>(t, cols, h);
    if constexpr (OUT != kOutQuant) trim<TPR>(t, cols, w);
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const uint32_t c = j * TPR + t;
      if (RES && k.sum_out && live && c < chunks)
        store_chunk8<STREAM>(k.sum_out + row * k.lds, c, cols, h[j]);
      measure_chunk<TYPE, OUT>(h[j], w[j], s, m);
    }
    RowCombine<TPR, kRows>::run(s, m, lds, turn);
    const float inv = OUT == kOutQuant ? 1.0f : inv_rms_of(s, k.cols, k.eps);
    const CodeScale cs(m);
    if (!live) continue;
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const uint32_t c = j * TPR + t;
      if (c < chunks) finish_chunk<TYPE, OUT, STREAM>(k, row, c, h[j], w[j], inv, cs);
    }
    if (t == 0) finish_row<OUT>(k, row, inv, m);
  }
}

// Rows too long for the registers: one block per row, walked twice.  The
// second walk forms h again from what the first read, or reads it from
// sum_out (where each thread wrote its own chunks), so that outputs may stand
// where inputs did.
template <int TYPE, int OUT, bool RES>
__global__ __launch_bounds__(1024) void norm_loop_kernel(NormArgs k) {
  __shared__ typename RowCombine<1024, 1>::Lds lds[2];
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
    RowCombine<1024, 1>::run(s, m, lds, turn);
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

#define ARMX_EACH_SHAPE_BELOW_1024(CASE) \
  CASE(8, 1);                 \
  CASE(16, 1);                \
  CASE(32, 1);                \
  CASE(64, 1);                \
  CASE(128, 1);               \
  CASE(256, 1);               \
  CASE(512, 1);               \
  CASE(512, 2);               \
  CASE(512, 4)
#define ARMX_EACH_SHAPE(CASE)       \
  ARMX_EACH_SHAPE_BELOW_1024(CASE); \
  CASE(1024, 4)

template <int TYPE, int OUT, bool RES>
hipError_t launch_norm_typed(const NormArgs& a, const armx_config* cfg, hipStream_t stream) {
  const RowShape s = row_shape(a.cols);
  const bool stream_out = a.rows * a.cols >= kStreamValues;
  const void* fn = nullptr;
#define ARMX_NORM_CASE(T, C) \
  if (s.threads == T && s.chunks == C) \
    fn = stream_out ? reinterpret_cast<const void*>(&norm_kernel<TYPE, OUT, RES, true, T, C>) \
                    : reinterpret_cast<const void*>(&norm_kernel<TYPE, OUT, RES, false, T, C>)
  ARMX_EACH_SHAPE(ARMX_NORM_CASE);
#undef ARMX_NORM_CASE
  if (s.chunks == 0) fn = reinterpret_cast<const void*>(&norm_loop_kernel<TYPE, OUT, RES>);
  const int block = s.threads > kRowBlock ? s.threads : kRowBlock;
  const uint64_t per = uint64_t(block / s.threads);
  uint64_t blocks = (a.rows + per - 1) / per;
  if (blocks > kMaxGrid) blocks = kMaxGrid;
  NormArgs copy = a;
  void* args[] = {&copy};
  return launch_rows_kernel(fn, blocks, block, args, cfg, stream);
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

// dx of the chunks of a row that a thread holds.
template <int TYPE, bool DSUM, bool STREAM, int TPR, int C>
__device__ __forceinline__ void store_grads(const NormBackwardArgs& k, uint64_t row, uint32_t t,
                                            float inv, float dot, const u32x4 (&dy)[C],
                                            const u32x4 (&h)[C], const u32x4 (&ds)[C],
                                            const u32x4 (&w)[C]) {
  const uint32_t cols = uint32_t(k.cols), chunks = (cols + 7) / 8;
  const float f = inv * inv * (dot / float(k.cols));
#pragma unroll
  for (int j = 0; j < C; ++j) {
    const uint32_t c = j * TPR + t;
    if (c >= chunks) continue;
    float fy[8], fh[8], fw[8], fd[8];
    widen8<TYPE>(dy[j], fy);
    widen8<TYPE>(h[j], fh);
    widen8<TYPE>(w[j], fw);
    if constexpr (DSUM) widen8<TYPE>(ds[j], fd);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      fy[i] = inv * (fy[i] * fw[i] - fh[i] * f);
      if constexpr (DSUM) fy[i] += fd[i];
    }
    store_chunk8<STREAM>(k.dx + row * k.ldx, c, cols, narrow8<TYPE>(fy));
  }
}

// Block b takes the row groups b, b + blocks, ...; every thread keeps the
// dweight sums of its own columns in registers over the block's rows.  A block
// of several rows at a time adds its row groups' sums through LDS, in order.
template <int TYPE, bool DSUM, bool STREAM, int TPR, int C>
__global__ __launch_bounds__(TPR > kRowBlock ? TPR : kRowBlock) void norm_backward_kernel(
    NormBackwardArgs k, float* dst, uint64_t pitch) {
  constexpr int kBlock = TPR > kRowBlock ? TPR : kRowBlock;
  constexpr int kRows = kBlock / TPR;
  __shared__ typename RowCombine<TPR, kRows>::Lds lds[2];
  __shared__ float part[kRows > 1 ? kRows * TPR * C * 8 : 1];
  const uint32_t t = threadIdx.x % TPR, cols = uint32_t(k.cols);
  const uint32_t chunks = (cols + 7) / 8;
  u32x4 w[C];
  float acc[C][8];
#pragma unroll
  for (int j = 0; j < C; ++j) {
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[j][i] = 0.0f;
  }
  load_weight<TPR>(k.weight, t, cols, w);
  // One row group's values; with kAhead the next group's are on their way while
  // this one's are combined (8192 x 4096 56.6 -> 54.3 us; at 512 threads x 4, where
  // the registers no longer hold both, 62 -> 71).
  struct Rows {
    u32x4 dy[C], h[C], ds[C];
    float inv;
  };
  constexpr bool kAhead = TPR * C <= 1024;
  auto load = [&](uint64_t base) __attribute__((always_inline)) {
    Rows v;
    const uint64_t row = base + threadIdx.x / TPR;
    const bool live = row < k.rows;
    v.inv = live ? k.inv_rms[row] : 0.0f;
    load_row<TPR>(k.dy + base * k.ldy, k.ldy, live, t, cols, v.dy);
    load_row<TPR>(k.h + base * k.ldh, k.ldh, live, t, cols, v.h);
    if constexpr (DSUM) load_row<TPR>(k.dsum + base * k.ldd, k.ldd, live, t, cols, v.ds);
    return v;
  };
  int turn = 0;
  const uint64_t stride = uint64_t(gridDim.x) * kRows;
  Rows ahead;
  if constexpr (kAhead) ahead = load(uint64_t(blockIdx.x) * kRows);
  for (uint64_t base = uint64_t(blockIdx.x) * kRows; base < k.rows; base += stride, turn ^= 1) {
    const uint64_t row = base + threadIdx.x / TPR;
    const bool live = row < k.rows;
    Rows now;
    if constexpr (kAhead) {
      now = ahead;
      if (base + stride < k.rows) ahead = load(base + stride);
    } else {
      now = load(base);
    }
    trim<TPR>(t, cols, now.dy);
    trim<TPR>(t, cols, now.h);
    trim<TPR>(t, cols, w);
    const u32x4 (&dy)[C] = now.dy, (&h)[C] = now.h, (&ds)[C] = now.ds;
    const float inv = now.inv;
    float dot = 0.0f;
#pragma unroll
    for (int j = 0; j < C; ++j) {
      float fy[8], fh[8], fw[8];
      widen8<TYPE>(dy[j], fy);
      widen8<TYPE>(h[j], fh);
      widen8<TYPE>(w[j], fw);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        dot = __builtin_fmaf(fy[i] * fw[i], fh[i], dot);
        if (live) acc[j][i] = __builtin_fmaf(fy[i], fh[i] * inv, acc[j][i]);
      }
    }
    uint32_t unused = 0;
    RowCombine<TPR, kRows>::run(dot, unused, lds, turn);
    if (!live) continue;
    store_grads<TYPE, DSUM, STREAM, TPR>(k, row, t, inv, dot, dy, h, ds, w);
  }
  if constexpr (kRows > 1) {
#pragma unroll
    for (int j = 0; j < C; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        part[(threadIdx.x / TPR) * (TPR * C * 8) + (j * TPR + t) * 8 + i] = acc[j][i];
    __syncthreads();
    for (uint32_t e = threadIdx.x; e < cols; e += kBlock) {
      float v = part[e];
      for (int r = 1; r < kRows; ++r) v += part[r * (TPR * C * 8) + e];
      dst[uint64_t(blockIdx.x) * pitch + e] = v;
    }
  } else {
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const uint32_t c = j * TPR + t;
      float* d = dst + uint64_t(blockIdx.x) * pitch + c * 8;
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

// Rows too long for the registers: two walks per row, the block's dweight sums
// kept in its own row of `dst` (each thread reads and writes its own columns).
template <int TYPE, bool DSUM>
__global__ __launch_bounds__(1024) void norm_backward_loop_kernel(NormBackwardArgs k, float* dst,
                                                                  uint64_t pitch) {
  __shared__ typename RowCombine<1024, 1>::Lds lds[2];
  const uint32_t cols = uint32_t(k.cols), chunks = (cols + 7) / 8;
  float* sums = dst + uint64_t(blockIdx.x) * pitch;
  for (uint32_t c = threadIdx.x; c < chunks; c += 1024)
    for (uint32_t i = 0; i < 8; ++i)
      if (c * 8 + i < cols) sums[c * 8 + i] = 0.0f;
  int turn = 0;
  for (uint64_t row = blockIdx.x; row < k.rows; row += gridDim.x, turn ^= 1) {
    const uint16_t* yr = k.dy + row * k.ldy;
    const uint16_t* hr = k.h + row * k.ldh;
    const float inv = k.inv_rms[row];
    float dot = 0.0f;
    for (uint32_t c = threadIdx.x; c < chunks; c += 1024) {
      float fy[8], fh[8], fw[8];
      widen8<TYPE>(load_chunk8(yr, c, cols), fy);
      widen8<TYPE>(load_chunk8(hr, c, cols), fh);
      widen8<TYPE>(load_chunk8(k.weight, c, cols), fw);
#pragma unroll
      for (int i = 0; i < 8; ++i) dot = __builtin_fmaf(fy[i] * fw[i], fh[i], dot);
    }
    uint32_t unused = 0;
    RowCombine<1024, 1>::run(dot, unused, lds, turn);
    const float f = inv * inv * (dot / float(k.cols));
    for (uint32_t c = threadIdx.x; c < chunks; c += 1024) {
      float fy[8], fh[8], fw[8], fd[8];
      widen8<TYPE>(load_chunk8(yr, c, cols), fy);
      widen8<TYPE>(load_chunk8(hr, c, cols), fh);
      widen8<TYPE>(load_chunk8(k.weight, c, cols), fw);
      if constexpr (DSUM) widen8<TYPE>(load_chunk8(k.dsum + row * k.ldd, c, cols), fd);
      for (uint32_t i = 0; i < 8; ++i)
        if (c * 8 + i < cols) sums[c * 8 + i] = __builtin_fmaf(fy[i], fh[i] * inv, sums[c * 8 + i]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        fy[i] = inv * (fy[i] * fw[i] - fh[i] * f);
        if constexpr (DSUM) fy[i] += fd[i];
      }
      store_chunk8<false>(k.dx + row * k.ldx, c, cols, narrow8<TYPE>(fy));
    }
  }
}

// dx and dweight apart, in one launch without a workspace: the first `col_blocks`
// blocks each sum dweight over all rows for 64 columns, reading dy and h once more,
// and the others make the dx of their row groups.
template <int TYPE, bool DSUM, int TPR, int C>
__global__ __launch_bounds__(TPR > kRowBlock ? TPR : kRowBlock) void norm_backward_apart_kernel(
    NormBackwardArgs k, unsigned col_blocks) {
  constexpr int kBlock = TPR > kRowBlock ? TPR : kRowBlock;
  constexpr int kRows = kBlock / TPR;
  constexpr int kWaves = kBlock / 64;
  __shared__ typename RowCombine<TPR, kRows>::Lds lds[2];
  __shared__ float part[kWaves][64];
  const uint32_t cols = uint32_t(k.cols), chunks = (cols + 7) / 8;
  if (blockIdx.x >= col_blocks) {
    const uint32_t t = threadIdx.x % TPR;
    u32x4 w[C];
    load_weight<TPR>(k.weight, t, cols, w);
    int turn = 0;
    const uint64_t stride = uint64_t(gridDim.x - col_blocks) * kRows;
    for (uint64_t base = uint64_t(blockIdx.x - col_blocks) * kRows; base < k.rows;
         base += stride, turn ^= 1) {
      const uint64_t row = base + threadIdx.x / TPR;
      const bool live = row < k.rows;
      u32x4 dy[C], h[C], ds[C];
      load_row<TPR>(k.dy + base * k.ldy, k.ldy, live, t, cols, dy);
      load_row<TPR>(k.h + base * k.ldh, k.ldh, live, t, cols, h);
      if constexpr (DSUM) load_row<TPR>(k.dsum + base * k.ldd, k.ldd, live, t, cols, ds);
      const float inv = live ? k.inv_rms[row] : 0.0f;
      trim<TPR>(t, cols, dy);
      trim<TPR>(t, cols, h);
      trim<TPR>(t, cols, w);
      float dot = 0.0f;
#pragma unroll
      for (int j = 0; j < C; ++j) {
        float fy[8], fh[8], fw[8];
        widen8<TYPE>(dy[j], fy);
        widen8<TYPE>(h[j], fh);
        widen8<TYPE>(w[j], fw);
#pragma unroll
        for (int i = 0; i < 8; ++i) dot = __builtin_fmaf(fy[i] * fw[i], fh[i], dot);
      }
      uint32_t unused = 0;
      RowCombine<TPR, kRows>::run(dot, unused, lds, turn);
      if (live) store_grads<TYPE, DSUM, false, TPR>(k, row, t, inv, dot, dy, h, ds, w);
    }
    return;
  }
  // 8 lanes take a row's 64 columns, 8 rows to a wavefront; rows in steps of the
  // block's, four in flight
  const uint32_t c = blockIdx.x * 8 + (threadIdx.x & 7);
  const bool whole = (blockIdx.x + 1) * 64 <= cols;   // the same for the block
  constexpr uint32_t kStep = kBlock / 8;
  float acc[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  auto add = [&](u32x4 y, u32x4 x, float inv) __attribute__((always_inline)) {
    float fy[8], fh[8];
    widen8<TYPE>(y, fy);
    widen8<TYPE>(x, fh);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = __builtin_fmaf(fy[i], fh[i] * inv, acc[i]);
  };
  for (uint64_t r = threadIdx.x >> 3; r < k.rows; r += 4 * kStep) {
    u32x4 y[4], x[4];
    float inv[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      // a row past the last is read as this thread's first, and not added
      const uint64_t rq = r + q * kStep < k.rows ? r + q * kStep : r;
      inv[q] = k.inv_rms[rq];
      if (whole) {
        y[q] = *reinterpret_cast<const u32x4*>(k.dy + rq * k.ldy + uint64_t(c) * 8);
        x[q] = *reinterpret_cast<const u32x4*>(k.h + rq * k.ldh + uint64_t(c) * 8);
      } else {
        y[q] = c < chunks ? load_chunk8(k.dy + rq * k.ldy, c, cols) : u32x4{0, 0, 0, 0};
        x[q] = c < chunks ? load_chunk8(k.h + rq * k.ldh, c, cols) : u32x4{0, 0, 0, 0};
      }
    }
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (r + q * kStep < k.rows) add(y[q], x[q], inv[q]);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {   // over the wavefront's 8 rows: lanes 8, 16 and 32 apart
    float v = acc[i];
    v += dpp<kDppRor8>(v);
    v = add_xor16(v);
    v = add_xor32(v);
    if (lane_id() < 8) part[wave_id()][lane_id() * 8 + i] = v;
  }
  __syncthreads();
  const uint32_t e = blockIdx.x * 64 + threadIdx.x;
  if (threadIdx.x < 64 && e < cols) {
    float v = part[0][threadIdx.x];
#pragma unroll
    for (int q = 1; q < kWaves; ++q) v += part[q][threadIdx.x];
    k.dweight[e] = v;
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

template <int TYPE, bool DSUM>
hipError_t launch_backward_apart(const NormBackwardArgs& a, const NormBackwardPlan& plan,
                                 const armx_config* cfg, hipStream_t stream) {
  const RowShape s = plan.shape;
  const void* fn = nullptr;
#define ARMX_NORM_CASE(T, C)              \
  if (s.threads == T && s.chunks == C)    \
    fn = reinterpret_cast<const void*>(&norm_backward_apart_kernel<TYPE, DSUM, T, C>)
  ARMX_EACH_SHAPE(ARMX_NORM_CASE);
#undef ARMX_NORM_CASE
  NormBackwardArgs copy = a;
  unsigned col_blocks = unsigned((a.cols + 63) / 64);
  void* args[] = {&copy, &col_blocks};
  const uint64_t row_blocks = plan.blocks - col_blocks;
  // dx where dy is: every column's sums before any row's gradient
  if (!meet(a.dx, a.ldx, a.dy, a.ldy, a.rows, a.cols))
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
  const RowShape s = plan.shape;
  const bool stream_out = a.rows * a.cols >= kStreamValues;
  const void* fn = nullptr;
#define ARMX_NORM_CASE(T, C)                                                                   \
  if (s.threads == T && s.chunks == C)                                                         \
    fn = stream_out                                                                            \
             ? reinterpret_cast<const void*>(&norm_backward_kernel<TYPE, DSUM, true, T, C>)    \
             : reinterpret_cast<const void*>(&norm_backward_kernel<TYPE, DSUM, false, T, C>)
  ARMX_EACH_SHAPE_BELOW_1024(ARMX_NORM_CASE);
#undef ARMX_NORM_CASE
  if (s.chunks == 0) fn = reinterpret_cast<const void*>(&norm_backward_loop_kernel<TYPE, DSUM>);
  NormBackwardArgs copy = a;
  const bool join = plan.blocks > 1;
  float* dst = join ? a.partials : a.dweight;
  uint64_t pitch = join ? plan.pitch : 0;
  void* args[] = {&copy, &dst, &pitch};
  hipError_t e = launch_rows_kernel(fn, plan.blocks, plan.block, args, cfg, stream, true, !join);
  if (e != hipSuccess || !join) return e;
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
  p.block = p.shape.threads > kRowBlock ? p.shape.threads : kRowBlock;
  if (rows == 0 || cols == 0) return p;
  const uint64_t per = uint64_t(p.block / p.shape.threads);
  const uint64_t groups = (rows + per - 1) / per;
  // Few rows: the column blocks read them in at most four rounds, from the caches
  // (us, partial sums / columns apart: 512 x 1024 8.1 / 5.3, 1024 x 8192 17.9 / 15.9,
  // 2048 x 4096 16.9 / 16.8, 2048 x 1024 9.6 / 21.7, 1024 x 16384 36.3 / 36.5).
  // 1024 threads of four chunks each, of any number of rows: their registers do not
  // hold the partial sums too (512 x 32768 106 / 39).
  p.apart = (p.shape.chunks > 0 && rows <= 2 * uint64_t(p.block) &&
             rows * cols <= uint64_t(1) << 23) ||
            (p.shape.threads == 1024 && p.shape.chunks > 0);
  if (p.apart) {
    p.blocks = (cols + 63) / 64 + (groups < kMaxGrid / 2 ? groups : kMaxGrid / 2);
    return p;
  }
  // Every block's dweight sums are written and read again, so fewer blocks move
  // less, and too few leave loads unsent.  Measured on MI355X at 1, 2 and 4 blocks
  // of 256 threads per compute unit (us): 8192 x 4096 55.4, 54.3, 61.2; 4096 x 8192
  // 54.9, 58.9, 69.0; 32768 x 128 11.6, 10.7, 11.7.
  const uint64_t most = uint64_t(cu_count) * (cols <= 2048 ? 2 : 1);
  p.blocks = groups < most ? groups : most;
  p.pitch = (cols + 63) / 64 * 64;
  if (p.blocks > 1) p.ws_bytes = size_t(p.blocks * p.pitch * sizeof(float));
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
