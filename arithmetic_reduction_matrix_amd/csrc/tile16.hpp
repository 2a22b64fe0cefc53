// Tiles of products of 16-bit matrices whose rows both lie along the sum, by
// v_mfma_f32_16x16x32_{f16,bf16}, summed in binary32.  Each source that includes it
// gets its own.
//
// Operand layout: lane l of a wavefront supplies row l % 16 of its 16-row operand tile
// and the 8 consecutive values of k-group l / 16, one 16-byte piece.  The rows of b go
// in as the MFMA's first operand and those of a as its second, so that lane l ends with
// the product's row l % 16 and the 4 consecutive columns 4 (l / 16) .. + 3.
//
// Which rows of a and b make up an operand tile is free.  Row r of operand tile x of a
// wavefront's kMT is its row r kMT + x, and row 4 q + e of operand tile y of b's 4 is its
// column 32 (y / 2) + 8 q + 4 (y % 2) + e: lane (q, r) ends with kMT consecutive rows of
// two runs of 8 columns (lane_column), whole 16-byte pieces of either order of the product
// in 16 bits, of which 4 lanes write 64 bytes in a row at once.  (With one run of 16, whose
// halves they wrote in turn, 131072 x 4096 x 32 in tiles of 192 x 256 took 317 us, now 296.)
// Of products written in 32 bits (ACROSS) it is column 16 y + 4 q + e.
//
// Steps of 64 values of k (128 bytes, a line) go from memory straight to LDS
// (buffer_load ... lds) into rings of buffers, NS steps ahead of the one that is
// multiplied.  The half of a step (32 values) that is multiplied next is read from LDS
// under the products of the one before, so a step's buffers are free again in its middle;
// there a's loads of the step NS on are sent, and b's, whose ring has one buffer more,
// already under the first half: loads are spread over the whole step.
// (256 x 256, both operands' loads in the second half of a step: 4096 x 32768 x 4096 806
// us, 4096 x 4096 x 32768 763; spread 779 and 744; and with the two wavefronts of a SIMD
// taking turns, TURNS, 763 and 715.)
//
// LDS rows are in operand order, 8 slots of 16 bytes; row r of an operand tile keeps its
// piece c in slot c ^ swizzle(r), so that the 16 lanes of a 16-byte LDS read, whose rows are
// 128 bytes apart, meet no bank twice.  The load writes LDS in lane order, so the swizzle is
// made on the memory side: the lane that fills slot s of row r fetches piece s ^ swizzle(r).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "device_common.hpp"

namespace armx {
namespace {

using namespace dev;

#define ARMX_INLINE __attribute__((always_inline))

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

template <int TYPE>
__device__ __forceinline__ floatx4 mfma16(u32x4 x, u32x4 y, floatx4 acc) {
  if constexpr (TYPE == ARMX_F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8, x),
                                                  __builtin_bit_cast(half8, y), acc, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x),
                                                   __builtin_bit_cast(bf16x8, y), acc, 0, 0, 0);
}

// A matrix of 16-bit values, `k` of each row counting.  `ld` (values, a multiple of 8) lets
// a tile's rows be reached by 32-bit byte offsets (tile_reaches of cross_entropy.h).
struct Matrix16 {
  const uint16_t* p;
  uint64_t rows, ld;
};

// Rows from row0 on as a range-checked buffer that ends with the 32-bit word of the
// last row's last value: reads past it return zeros without a memory access.
constexpr int kTileBuffer = 0x00020000;
__device__ __forceinline__ __amdgpu_buffer_rsrc_t tile_rows(const Matrix16& m, uint64_t k,
                                                            uint64_t row0) {
  uint64_t left = row0 < m.rows ? (m.rows - 1 - row0) * m.ld * 2 + (k + 1) / 2 * 4 : 0;
  if (left > 0xFFFFFFF0u) left = 0xFFFFFFF0u;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(m.p + (left ? row0 * m.ld : 0)),
                                           0, int(uint32_t(left)), kTileBuffer);
}

// The first `keep` of a lane's 8 values (keep <= 0: none), the others zero.
__device__ __forceinline__ u32x4 keep_values(u32x4 v, int keep) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = keep - 2 * i;
    v[i] &= n >= 2 ? 0xFFFFFFFFu : n <= 0 ? 0u : 0xFFFFu;
  }
  return v;
}

__device__ __forceinline__ uint32_t swizzle(uint32_t r) { return (r >> 1) & 7; }

template <int N>
struct Int {
  static constexpr int value = N;
};
using Yes = Int<1>;
using No = Int<0>;

constexpr int kStepBytes = 128, kStepValues = 64;

// A block makes BM x BN of the product with WM x WN wavefronts.  NS steps of a have a
// buffer, and of b one step more, so that its loads need not wait for the middle of a step.
// ACROSS: b's rows lie across the sum, so that its transpose is multiplied.
template <int BM, int BN, int WM, int WN, int NS, bool TURNS = false, bool ACROSS = false>
struct Tile16 {
  typedef Tile16<BM, BN, WM, WN, NS, TURNS, true> Across;
  static constexpr int kBM = BM, kBN = BN, kWM = WM, kWN = WN, kNS = NS;
  static constexpr bool kTurns = TURNS, kAcross = ACROSS;
  static constexpr int kWaves = WM * WN, kThreads = 64 * kWaves;
  static constexpr unsigned kGroup = BM < 128 ? 4 : 1024 / BM;   // tile_of
  static constexpr int kMT = BM / WM / 16;  // 16-row operand tiles per wavefront
  static constexpr int kNT = BN / WN / 16;
  static constexpr int kRows = kMT, kCols = 4 * kNT;   // a lane's part of the product
  static constexpr int kLoadsA = BM / 8 / kWaves;  // wavefront loads per step
  static constexpr int kLoadsB = BN / 8 / kWaves;
  static constexpr int kStageA = BM * kStepBytes, kStageB = BN * kStepBytes;
  static constexpr int kNA = NS, kNB = NS + 1;
  static constexpr int kLdsBytes = kNA * kStageA + kNB * kStageB;
  // wavefronts per SIMD that the LDS leaves room for, at most 2 (of 256 registers)
  static constexpr int kResident = 160 * 1024 / kLdsBytes * kWaves / 4;
  static constexpr int kPerSimd = kResident < 1 ? 1 : kResident < 2 ? kResident : 2;
  static_assert(kLoadsA * 8 * kWaves == BM && kLoadsB * 8 * kWaves == BN, "whole loads");
  static_assert(kLdsBytes <= 160 * 1024, "a compute unit's LDS");
  static_assert(NS >= 2 && NS <= 4, "the last steps are written out");
  static constexpr int kRowB = 2 * BN;   // bytes of a row of b's step that lies across
  static_assert(kMT <= 16, "operand tiles");
  static_assert(kNT == 4, "lane_column");
  static_assert(BN == 256 || BN == 128 || BN == 64, "across_swizzle");
  static_assert(!TURNS || (kWaves == 8 && NS == 2), "two wavefronts a SIMD, in turns");
};

typedef __attribute__((address_space(3))) int8_t tile_lds_byte;
typedef short s16x4 __attribute__((ext_vector_type(4)));

// 16 bytes per lane from `rows` into LDS at `lds` + 16 lane.  Written as asm so that
// the compiler, which cannot tell the buffers apart, does not wait for these loads
// before every read of LDS; nothing comes back in registers, and wait_loads() and a
// barrier stand between these writes and their reads.  The load reads M0, which needs a
// wait state after its scalar write; the compiler puts none inside an asm string.  (M0
// is a reserved register, which a clobber list cannot name; the compiler uses it for
// nothing else here.)
__device__ __forceinline__ void lds_load16(__amdgpu_buffer_rsrc_t rows, uint32_t lds,
                                           uint32_t off) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :
               : "s"(lds), "v"(off), "s"(rows)
               : "memory");
}

__device__ __forceinline__ u32x4 lds_read16(uint32_t at) {
  return *reinterpret_cast<const u32x4 __attribute__((address_space(3)))*>(at);
}

// 16 lanes, each with the address of 4 values: lane 4 j + c of the 16 those of row j of
// column quad c, say; lane 4 c + e receives column e of quad c, rows 0 to 3.
__device__ __forceinline__ uint64_t lds_read_across(uint32_t at) {
  return __builtin_bit_cast(
      uint64_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    reinterpret_cast<s16x4 __attribute__((address_space(3)))*>(at)));
}

// Rows of b that lie across: 64 of a step, BN values each, pieces of 16 bytes.  A row keeps
// its piece p in slot p ^ across_swizzle(row).  A read of 4 values a lane serves 32 lanes at
// a time: 32 bytes each of 8 rows, 0 to 3 and 8 to 11 (or 16 and 8 on), which the rows'
// bits lead to different banks.
template <class T>
__device__ __forceinline__ uint32_t across_swizzle(uint32_t row) {
  const uint32_t third = (row >> 3) & 1;
  if constexpr (T::kBN == 64)   // two rows in 256 bytes
    return (((row >> 1) & 1) | third << 1) << 1;
  return ((row & 3) | third << 2) << 1;
}

// vmcnt(N): all but this wavefront's last N loads into LDS have landed
template <int N>
__device__ __forceinline__ void wait_loads() {
  static_assert(N < 64, "the count's six bits");
  __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | (N >> 4) << 14);
}

// Which tile a block makes: every XCD takes a contiguous range of ids, and ids run down
// kGroup rows of tiles before the next column, so that blocks running at the same time on
// one XCD share operand rows in its L2: 1024 rows of the product, or 4 of the small tiles.
// (Us, 4 rows of tiles / 1024 rows: 777 x 50001 x 2056 of 192 x 256 196 / 181, 131072 x 4096
// x 256 of 128 x 128 459 / 423, but logits and dz of 2046 x 1216 x 192, of 64 x 128, 9.3 /
// 12.0; 768, 1536, 2048 and 4096 rows over the shapes where each tile is chosen are 1% slower
// on average, 32768 x 4096 x 4096 of 256 x 256 727 with 1024 rows, 756 with 1536.)
template <class T>
__device__ __forceinline__ void tile_of(unsigned id, unsigned tiles_m, unsigned tiles_n,
                                        unsigned& ti, unsigned& tj) {
  const unsigned per = T::kGroup * tiles_n, grp = id / per, first = grp * T::kGroup;
  const unsigned rows = tiles_m - first < T::kGroup ? tiles_m - first : T::kGroup;
  const unsigned in = id - grp * per;
  ti = first + in % rows;
  tj = in / rows;
}

// acc = the tile at (i0, j0) of a b^T over k values, rows and columns past the
// matrices' undefined.  ACROSS: of a b over the rows of b, of which there are at least k
// or that end where zeros are to be read, and whose columns are `across`.  `lds`:
// T::kLdsBytes, at a multiple of 1024, free again after a barrier.  Every thread of the
// block takes part.
template <class T, int TYPE>
__device__ __forceinline__ void multiply_tile(const Matrix16& ma, const Matrix16& mb, uint32_t k,
                                              uint64_t i0, uint64_t j0, int8_t* lds,
                                              floatx4 (&acc)[T::kMT][T::kNT],
                                              uint64_t across = 0) {
  constexpr int kMT = T::kMT, kNT = T::kNT, NS = T::kNS;
  const int lane = lane_id(), w = wave_id();
  const uint32_t ring_a = uint32_t(reinterpret_cast<uintptr_t>((tile_lds_byte*)lds));
  const uint32_t ring_b = ring_a + T::kNA * T::kStageA;
  uint32_t base_a = ring_a, base_b = ring_b;
  auto after_a = [&](uint32_t at) ARMX_INLINE {
    return at == ring_a + (T::kNA - 1) * T::kStageA ? ring_a : at + T::kStageA;
  };
  auto after_b = [&](uint32_t at) ARMX_INLINE {
    return at == ring_b + (T::kNB - 1) * T::kStageB ? ring_b : at + T::kStageB;
  };
  const __amdgpu_buffer_rsrc_t a = tile_rows(ma, k, i0);
  const __amdgpu_buffer_rsrc_t b = T::kAcross ? a : tile_rows(mb, k, j0);
  // across: the next step's rows of b, whose steps are sent in order, and the bytes from
  // there on
  const uint16_t* next_b = mb.p + j0;
  const uint64_t step_b = uint64_t(kStepValues) * mb.ld * 2;
  uint64_t left_b =
      T::kAcross && mb.rows ? (mb.rows - 1) * mb.ld * 2 + (across - j0 + 1) / 2 * 4 : 0;
  __amdgpu_buffer_rsrc_t rows_b = b;
  auto take_b = [&]() ARMX_INLINE {
    rows_b = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint16_t*>(next_b), 0,
        int(uint32_t(left_b < 0xFFFFFFF0u ? left_b : 0xFFFFFFF0u)), kTileBuffer);
    next_b += step_b / 2;
    left_b = left_b > step_b ? left_b - step_b : 0;
  };
  // rows past the matrix are read from its last row
  const uint32_t last_a = uint32_t(ma.rows - 1 - i0 < T::kBM ? ma.rows - 1 - i0 : T::kBM - 1);
  const uint32_t last_b =
      T::kAcross ? 0u : uint32_t(mb.rows - 1 - j0 < T::kBN ? mb.rows - 1 - j0 : T::kBN - 1);
  // byte offsets of the pieces that this lane brings into its slots of LDS rows
  uint32_t off_a[T::kLoadsA], off_b[T::kLoadsB];
#pragma unroll
  for (int x = 0; x < T::kLoadsA; ++x) {
    const uint32_t slot = (w * T::kLoadsA + x) * 8 + (lane >> 3);
    const uint32_t in = slot % (16 * kMT), r = in % 16;
    const uint32_t row = slot / (16 * kMT) * (16 * kMT) + r * kMT + in / 16;
    off_a[x] = (row < last_a ? row : last_a) * uint32_t(ma.ld * 2) +
               ((uint32_t(lane) & 7) ^ swizzle(r)) * 16;
  }
#pragma unroll
  for (int x = 0; x < T::kLoadsB; ++x) {
    if constexpr (T::kAcross) {
      const uint32_t byte = (w * T::kLoadsB + x) * 1024 + lane * 16, row = byte / T::kRowB;
      off_b[x] = row * uint32_t(mb.ld * 2) +
                 (byte % T::kRowB / 16 ^ across_swizzle<T>(row)) * 16;
      continue;
    }
    const uint32_t slot = (w * T::kLoadsB + x) * 8 + (lane >> 3);
    const uint32_t in = slot % (16 * kNT), r = in % 16;
    const uint32_t row = slot / (16 * kNT) * (16 * kNT) + in / 32 * 32 + r / 4 * 8 +
                         in / 16 % 2 * 4 + r % 4;
    off_b[x] = (row < last_b ? row : last_b) * uint32_t(mb.ld * 2) +
               ((uint32_t(lane) & 7) ^ swizzle(r)) * 16;
  }
  // wavefront load x of an operand's step at byte k0, into the buffer at `to`
  auto send_a = [&](uint32_t to, uint32_t k0, int x) ARMX_INLINE {
    lds_load16(a, to + (w * T::kLoadsA + x) * 1024, off_a[x] + k0);
  };
  auto send_b = [&](uint32_t to, uint32_t k0, int x) ARMX_INLINE {
    if constexpr (T::kAcross) {
      if (x == 0) take_b();
      lds_load16(rows_b, to + (w * T::kLoadsB + x) * 1024, off_b[x]);
    } else {
      lds_load16(b, to + (w * T::kLoadsB + x) * 1024, off_b[x] + k0);
    }
  };
  constexpr int kLoads = T::kLoadsA + T::kLoadsB;
  auto stage = [&](uint32_t t) ARMX_INLINE {
#pragma unroll
    for (int x = 0; x < T::kLoadsA; ++x) send_a(ring_a + t * T::kStageA, t * kStepBytes, x);
#pragma unroll
    for (int x = 0; x < T::kLoadsB; ++x) send_b(ring_b + t * T::kStageB, t * kStepBytes, x);
  };
  // all but the wavefront's last `loads` loads have landed and all the block's reads are
  // done
  auto sync = [&](auto loads) ARMX_INLINE {
    wait_loads<decltype(loads)::value>();
    if constexpr (T::kWaves > 1)
      __syncthreads();
    else
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  };
  // operand registers of half a step (32 values of k): lane l reads row l % 16 of each
  // operand tile, piece 4 half + l / 16
  const uint32_t r = lane & 15, g = lane >> 4;
  uint32_t at_a[2], at_b[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t in = r * kStepBytes + ((4 * h + g) ^ swizzle(r)) * 16;
    at_a[h] = (w % T::kWM) * (kMT * 16 * kStepBytes) + in;
    at_b[h] = (w / T::kWM) * (kNT * 16 * kStepBytes) + in;
  }
  // across: lane 4 j + c of its 16 reads row 8 g + j (and 4 on), column quad c of tile y
  uint32_t at_across[kNT];
  if constexpr (T::kAcross) {
    const uint32_t j = r / 4, c = r % 4, row = 8 * g + j;
#pragma unroll
    for (int y = 0; y < kNT; ++y) {
      const uint32_t byte = (w / T::kWM) * (kNT * 32) + y * 32 + c * 8;
      at_across[y] = row * T::kRowB + (byte / 16 ^ across_swizzle<T>(row)) * 16 + byte % 16;
    }
  }
  auto read_b = [&](uint32_t from, int h, int y) ARMX_INLINE {
    if constexpr (T::kAcross) {
      const uint32_t at = from + at_across[y] + h * 32 * T::kRowB;
      const uint64_t low = lds_read_across(at), high = lds_read_across(at + 4 * T::kRowB);
      return u32x4{uint32_t(low), uint32_t(low >> 32), uint32_t(high), uint32_t(high >> 32)};
    } else {
      return lds_read16(from + y * 16 * kStepBytes);
    }
  };
#pragma unroll
  for (int x = 0; x < kMT; ++x)
#pragma unroll
    for (int y = 0; y < kNT; ++y) acc[x][y] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
  if (k == 0) return;
  const uint32_t steps = (k + kStepValues - 1) / kStepValues;
  const bool cut = k % kStepValues != 0;
  if constexpr (T::kTurns) {
    // The two wavefronts of a SIMD take turns: between two barriers one reads its
    // operands of half a step and sends loads, while the other multiplies, which it does
    // at a higher priority; the second group of four is a barrier behind the first.
    //
    // Reads of a step's buffers by both groups end a barrier after the first one's second
    // half, so from the next step on they may be filled again: a's loads of step u + 1 are
    // sent in the first half of step u (two buffers), b's of step u + 2 in its second
    // (three).  Every wavefront waits for its own loads before the barrier behind which
    // the first group reads step u + 1: all but b's of step u + 2.
    u32x4 fa[kMT], fb[kNT];
    const bool second = w >= T::kWaves / 2;
    auto barrier = [&]() ARMX_INLINE {
      __builtin_amdgcn_sched_barrier(0);
      asm volatile("s_barrier" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
    };
    auto read = [&](int h) ARMX_INLINE {
      // (opaque to the compiler, so that it keeps two addresses and puts the rest into the
      // reads' offsets)
      uint32_t from_a = base_a + at_a[h], from_b = base_b + (T::kAcross ? 0 : at_b[h]);
      asm("" : "+v"(from_a));
      asm("" : "+v"(from_b));
      // (a first: with ACROSS's reads of b, two for each of a's, in front dx's product of
      // 4096 x 4096 x 32768 was 2% slower; others do not tell)
#pragma unroll
      for (int x = 0; x < kMT; ++x) fa[x] = lds_read16(from_a + x * 16 * kStepBytes);
#pragma unroll
      for (int y = 0; y < kNT; ++y) fb[y] = read_b(from_b, h, y);
      __builtin_amdgcn_sched_barrier(0);
    };
    // the reads are done, and values past k cut from both operands (what stands there may
    // be a NaN; across, b has zeros there)
    auto have = [&](uint32_t u, int h) ARMX_INLINE {
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      if (cut && u + 1 == steps) {
        const int keep = int(k) - int(u * kStepValues + 32 * h + 8 * g);
#pragma unroll
        for (int x = 0; x < kMT; ++x) fa[x] = keep_values(fa[x], keep);
#pragma unroll
        for (int y = 0; y < kNT; ++y) fb[y] = T::kAcross ? fb[y] : keep_values(fb[y], keep);
      }
    };
    auto multiply = [&]() ARMX_INLINE {
      __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int x = 0; x < kMT; ++x)
#pragma unroll
        for (int y = 0; y < kNT; ++y) acc[x][y] = mfma16<TYPE>(fb[y], fa[x], acc[x][y]);
      __builtin_amdgcn_s_setprio(0);
    };
    auto landed = [&](uint32_t u) ARMX_INLINE {
      if (u + 2 < steps)
        wait_loads<T::kLoadsB>();
      else
        wait_loads<0>();
    };
#pragma unroll
    for (int x = 0; x < T::kLoadsA; ++x) send_a(ring_a, 0, x);
#pragma unroll
    for (int x = 0; x < T::kLoadsB; ++x) send_b(ring_b, 0, x);
    if (steps > 1) {
#pragma unroll
      for (int x = 0; x < T::kLoadsB; ++x) send_b(ring_b + T::kStageB, kStepBytes, x);
      wait_loads<T::kLoadsB>();
    } else {
      wait_loads<0>();
    }
    barrier();
    if (second) barrier();
    for (uint32_t u = 0; u < steps; ++u) {
      read(0);
      if (u + 1 < steps) {
        const uint32_t to = after_a(base_a);
#pragma unroll
        for (int x = 0; x < T::kLoadsA; ++x) send_a(to, (u + 1) * kStepBytes, x);
      }
      have(u, 0);
      barrier();
      multiply();
      barrier();
      read(1);
      if (u + 2 < steps) {
        const uint32_t to = after_b(after_b(base_b));
#pragma unroll
        for (int x = 0; x < T::kLoadsB; ++x) send_b(to, (u + 2) * kStepBytes, x);
      }
      have(u, 1);
      if (second) landed(u);
      barrier();
      multiply();
      if (!second) landed(u);
      barrier();
      base_a = after_a(base_a);
      base_b = after_b(base_b);
    }
    if (!second) barrier();
    return;
  }
  u32x4 fa[2][kMT], fb[2][kNT];
  constexpr int kReads = kMT + kNT;
  // Where this lane reads half h of the buffer at `from`; opaque to the compiler, so
  // that it keeps two addresses and puts the rest into the reads' offsets.
  struct Place {
    uint32_t a, b;
  };
  auto place = [&](uint32_t from_a, uint32_t from_b, int h) ARMX_INLINE {
    Place at = {from_a + at_a[h], from_b + (T::kAcross ? 0 : at_b[h])};
    asm("" : "+v"(at.a));
    asm("" : "+v"(at.b));
    return at;
  };
  // read j of half h, in the order in which its products need them
  auto fetch = [&](Place at, int h, int j) ARMX_INLINE {
    if (j < kNT)
      fb[h][j] = read_b(at.b, h, j);
    else
      fa[h][j - kNT] = lds_read16(at.a + (j - kNT) * 16 * kStepBytes);
  };
  auto fetch_half = [&](int h) ARMX_INLINE {
    const Place at = place(base_a, base_b, h);
#pragma unroll
    for (int j = 0; j < kReads; ++j) {
      fetch(at, h, j);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // values past k are cut from both operands (what stands there may be a NaN)
  auto mask_half = [&](uint32_t k0, int h) ARMX_INLINE {
    const int keep = int(k) - int(k0 + 32 * h + 8 * g);
#pragma unroll
    for (int x = 0; x < kMT; ++x) fa[h][x] = keep_values(fa[h][x], keep);
#pragma unroll
    for (int y = 0; y < kNT; ++y) fb[h][y] = T::kAcross ? fb[h][y] : keep_values(fb[h][y], keep);
  };
  auto multiply_row = [&](int h, int x) ARMX_INLINE {
#pragma unroll
    for (int y = 0; y < kNT; ++y) acc[x][y] = mfma16<TYPE>(fb[h][y], fa[h][x], acc[x][y]);
  };
  auto multiply = [&](int h) ARMX_INLINE {
#pragma unroll
    for (int x = 0; x < kMT; ++x) multiply_row(h, x);
  };
  // The products of one half, with the other's operands (h) read from `at` and COUNT
  // loads sent between them.
  auto multiply_and_fetch = [&](int h, Place at, auto count, auto send) ARMX_INLINE {
    constexpr int kCount = decltype(count)::value;
    constexpr int kPerR = (kReads + kMT - 1) / kMT;
#pragma unroll
    for (int i = 0; i < kMT; ++i) {
#pragma unroll
      for (int j = kCount * i / kMT; j < kCount * (i + 1) / kMT; ++j) send(j);
#pragma unroll
      for (int j = i * kPerR; j < (i + 1) * kPerR; ++j)
        if (j < kReads) fetch(at, h, j);
      __builtin_amdgcn_sched_barrier(0);
      multiply_row(1 - h, i);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // A step but the last (its first half's operands already in registers): the second
  // half's are read while the first is multiplied, and with SEND the step NS on is sent
  // for into b's spare buffer; then, after the barrier that ends all reading of this
  // step's buffers and finds the next one's filled (all but `out` loads), into a's of this
  // step, while the next step's first half is read under the second half's products.
  uint32_t spare_b = ring_b + (T::kNB - 1) * T::kStageB;
  auto step = [&](auto send, auto out, uint32_t s) ARMX_INLINE {
    constexpr bool kSend = decltype(send)::value;
    const uint32_t k0 = (s + NS) * kStepBytes;
    multiply_and_fetch(1, place(base_a, base_b, 1), Int<kSend ? T::kLoadsB : 0>{},
                       [&](int x) ARMX_INLINE { send_b(spare_b, k0, x); });
    sync(out);
    const uint32_t old_a = base_a, old_b = base_b;
    base_a = after_a(base_a);
    base_b = after_b(base_b);
    spare_b = old_b;
    multiply_and_fetch(0, place(base_a, base_b, 0), Int<kSend ? T::kLoadsA : 0>{},
                       [&](int x) ARMX_INLINE { send_a(old_a, k0, x); });
  };
  uint32_t s = 0;
  if (steps >= NS) {
#pragma unroll
    for (int t = 0; t < NS; ++t) stage(t);
    sync(Int<(NS - 1) * kLoads>{});
  } else {
    for (uint32_t t = 0; t < steps; ++t) stage(t);
    sync(No{});
  }
  fetch_half(0);
  for (; steps - s > NS; ++s) step(Yes{}, Int<(NS - 2) * kLoads + T::kLoadsB>{}, s);
  // the last steps; what is still out shrinks with them
  if constexpr (NS > 3)
    if (steps - s > 3) step(No{}, Int<2 * kLoads>{}, s), ++s;
  if constexpr (NS > 2)
    if (steps - s > 2) step(No{}, Int<kLoads>{}, s), ++s;
  if (steps - s > 1) step(No{}, No{}, s), ++s;
  // (one half after the other: the registers do not hold both beside the masks)
  if (cut) mask_half(s * kStepValues, 0);
  multiply(0);
  fetch_half(1);
  if (cut) mask_half(s * kStepValues, 1);
  multiply(1);
}

}  // namespace
}  // namespace armx
