// Rows of 16-bit values in the registers of the threads that share them: how a row
// lies on threads, its loads and stores, the two types, and the launches of such
// kernels.  Each source that includes it gets its own.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "device_common.hpp"
#include "launch.h"
#include "layer.h"

namespace armx {
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

constexpr int log2_of(int v) { return v <= 1 ? 0 : 1 + log2_of(v / 2); }

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

// A chunk that starts at any value.
typedef u32x4 __attribute__((aligned(2))) u32x4_any;

// Whether two matrices of a call may share memory (their extents meet).
bool meet(const void* a, uint64_t lda, const void* b, uint64_t ldb, uint64_t rows, uint64_t cols) {
  const char* pa = static_cast<const char*>(a);
  const char* pb = static_cast<const char*>(b);
  return pa < pb + 2 * ((rows - 1) * ldb + cols) && pb < pa + 2 * ((rows - 1) * lda + cols);
}

}  // namespace
}  // namespace armx
