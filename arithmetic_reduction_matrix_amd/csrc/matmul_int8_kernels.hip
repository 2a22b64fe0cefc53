// out = (a b^T) scaled by rows and columns: 8-bit codes multiplied by
// v_mfma_i32_16x16x64_i8 with exact 32-bit integer sums.
//
// Integer sums are exact, so any tile, any order and any split along k gives
// the same bits; the order of k inside an MFMA does not matter either, as long
// as both operands use the same one.
//
// Operand layout used throughout: lane l of a wavefront supplies row l % 16 of
// its 16-row operand tile and the 16 consecutive codes of k-group l / 16, one
// 16-byte load.  The rows of b go in as the MFMA's first operand and those of
// a as its second, so that lane l ends with out row l % 16 and the 4
// consecutive columns 4 (l / 16) .. + 3.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "device_common.hpp"
#include "launch.h"
#include "layer.h"

namespace armx {
namespace {

using namespace dev;

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ i32x4 mfma_i8(u32x4 x, u32x4 y, i32x4 acc) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, x),
                                               __builtin_bit_cast(i32x4, y), acc, 0, 0, 0);
}

// Rows [row0, row0 + ...) of a matrix of codes as a range-checked buffer: a
// read at or past the end (the last row's codes rounded up to 16) returns
// zeros without a memory access.  Offsets are 32-bit: a tile's rows span at
// most 255 * 2^23 + 2^17 bytes.
constexpr int kRawBuffer = 0x00020000;
struct CodeRows {
  __amdgpu_buffer_rsrc_t rs;
  __device__ __forceinline__ CodeRows(const int8_t* p, uint64_t rows, uint64_t ld, uint64_t k,
                                      uint64_t row0) {
    uint64_t left = 0;
    if (row0 < rows) left = (rows - 1 - row0) * ld + (k + 15) / 16 * 16;
    if (left > 0x7FFFFFFFu + 0x00100000ull) left = 0x7FFFFFFFu + 0x00100000ull;
    rs = __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t*>(p + (left ? row0 * ld : 0)), 0,
                                           int(uint32_t(left)), kRawBuffer);
  }
  __device__ __forceinline__ u32x4 load(uint32_t off) const {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, off, 0, 0));
  }
};

// The first `keep` of a lane's 16 codes (keep <= 0: none), the others zero.
__device__ __forceinline__ u32x4 keep_codes(u32x4 v, int keep) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = keep - 4 * i;
    v[i] &= n >= 4 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << (8 * n)) - 1u;
  }
  return v;
}

// ---- scales, bias, rounding ---------------------------------------------------

typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));
// whole stores into rows of out, which start at any value: 16-bit ones 16 bytes at a
// time instead of value by value, 4096 x 4100 x 5001 92 us instead of 136
typedef uint32_t u32x4h __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2h __attribute__((ext_vector_type(2), aligned(2)));

// The epilogue of one lane's C consecutive columns (a multiple of 4), whose
// scales and bias stay in registers while its rows pass.
template <int OUT, int C>
struct Columns {
  const MatmulArgs& p;
  uint64_t j;
  bool whole;  // all of the columns exist
  float scale[C], bias[C];

  __device__ __forceinline__ float bias_at(uint64_t c) const {
    if constexpr (OUT == ARMX_F32) return static_cast<const float*>(p.bias)[c];
    if constexpr (OUT == ARMX_F16) return float(static_cast<const _Float16*>(p.bias)[c]);
    return float(static_cast<const __bf16*>(p.bias)[c]);
  }

  __device__ __forceinline__ Columns(const MatmulArgs& args, uint64_t first)
      : p(args), j(first), whole(first + C <= args.n) {
#pragma unroll
    for (int c = 0; c < C; c += 4) {
      if (j + c + 4 <= p.n) {
        const f32x4u v = *reinterpret_cast<const f32x4u*>(p.b_scales + j + c);
#pragma unroll
        for (int e = 0; e < 4; ++e) scale[c + e] = v[e];
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) scale[c + e] = j + c + e < p.n ? p.b_scales[j + c + e] : 0.0f;
      }
    }
    if (p.bias) {
#pragma unroll
      for (int c = 0; c < C; ++c) bias[c] = j + c < p.n ? bias_at(j + c) : 0.0f;
    }
  }

  // Row i: float(sum) * (row scale * column scale) + bias, each step one
  // rounding, then one to the output's type.
  __device__ __forceinline__ void store(uint64_t i, const i32x4 (&sums)[C / 4]) const {
    if (i >= p.m) return;
    const float sa = p.a_scales[i];
    float y[C];
#pragma unroll
    for (int c = 0; c < C; ++c) y[c] = float(sums[c / 4][c % 4]) * (sa * scale[c]);
    if (p.bias) {
#pragma unroll
      for (int c = 0; c < C; ++c) y[c] += bias[c];
    }
    if constexpr (OUT == ARMX_F32) {
      float* o = static_cast<float*>(p.out) + i * p.ldo + j;
      if (whole) {
#pragma unroll
        for (int c = 0; c < C; c += 4)
          *reinterpret_cast<f32x4u*>(o + c) = f32x4u{y[c], y[c + 1], y[c + 2], y[c + 3]};
      } else {
#pragma unroll
        for (int c = 0; c < C; ++c)
          if (j + c < p.n) o[c] = y[c];
      }
    } else {
      uint32_t v[C / 2];
#pragma unroll
      for (int c = 0; c < C; c += 2) {
        if constexpr (OUT == ARMX_F16)
          v[c / 2] = __builtin_bit_cast(uint32_t, half2v{_Float16(y[c]), _Float16(y[c + 1])});
        else
          v[c / 2] = __builtin_bit_cast(uint32_t, bf16x2{__bf16(y[c]), __bf16(y[c + 1])});
      }
      uint16_t* o = static_cast<uint16_t*>(p.out) + i * p.ldo + j;
      if (whole) {
        if constexpr (C % 8 == 0) {
#pragma unroll
          for (int c = 0; c < C / 2; c += 4)
            *reinterpret_cast<u32x4h*>(o + 2 * c) = u32x4h{v[c], v[c + 1], v[c + 2], v[c + 3]};
        } else {
          static_assert(C == 4, "whole stores");
          *reinterpret_cast<u32x2h*>(o) = u32x2h{v[0], v[1]};
        }
      } else {
#pragma unroll
        for (int c = 0; c < C; ++c)
          if (j + c < p.n) o[c] = uint16_t(v[c / 2] >> (16 * (c % 2)));
      }
    }
  }
};

// ---- tiles staged through LDS -------------------------------------------------
//
// A block makes BM x BN outputs.  Its wavefronts form KS groups of WM x WN that
// share k: a group takes every KS-th step of 128 codes and sums over its own.
// A step's rows of a and b go from memory straight to LDS (buffer_load ... lds,
// 16 bytes per lane, 8 rows of 128 bytes per wavefront load) into one of the
// group's NS buffers, NS - 1 steps ahead of the one that is multiplied.  (Steps of
// 64 codes in four buffers, with rows of 64 bytes, measured slower, 8192^3 450 ->
// 715 us: memory moves lines of 128 bytes, and each was moved twice.)
//
// With SHIFT a step's window of a row starts at the last 128-byte line before the
// step, `phase` pieces early, so that a load takes whole lines and none is moved
// twice; a step of the row then lies in its window and the next one's, and what is
// read from LDS comes `phase` pieces further on.  (That brings rows of unlike phase to
// one bank, half of the reads by count; kept in the slots of the step's own pieces they
// never meet, but four lanes then load from both halves of a line: 1500 x 8192 x 4112
// at 128 x 128 64.3 against 67.4 us, and nothing gained elsewhere.)
//
// Row 4 q + e of a wavefront's operand tile y of b is its column 4 (q kNT + y) + e,
// so that the lanes of group q end with 4 kNT consecutive columns of a row over the
// tiles, which they store together.
//
// LDS rows are 128 bytes, 8 slots of 16; row r keeps its piece c in slot
// c ^ swizzle(r), taken of the row's place in its operand tile.  A 16-byte LDS read
// serves 16 lanes at a time (lanes 0-3, 12-15, 20-23 and 24-27 first, and so on)
// from 64 banks, that is from 16 slots: rows r and r + 1 lie in different halves of
// them, and the rows of one parity that are read together differ in swizzle (no bank
// conflicts, by count).  The load writes LDS in lane order, so the swizzle is made on
// the memory side: the lane that fills slot s of row r fetches piece s ^ swizzle(r).
//
// What bounds it on MI355X: at many full tiles the matrix units, busy in 68% of the
// cycles, and the clock, which falls under them (8192^3 420 us, 2.6e15 operations a
// second); at smaller tiles the L2, from which the compute units together take a step's
// rows at 15 to 20 TB/s (192 x 192 48 KB in 0.84 us each, 128 x 128 32 KB in 0.52, two
// 64 x 64 32 KB in 0.38; matrix units 41% busy at 777 x 4100 x 5001, 23.6 us); with few
// rows the reading of b and the way to the first product (48 x 8192 x 4096 8.8 us,
// 3.8 TB/s of b; 1 x 4096 x 4096 5.2).
__device__ __forceinline__ uint32_t swizzle(uint32_t r) { return (r >> 1) & 7; }

constexpr int kStepK = 128;
#define ARMX_INLINE __attribute__((always_inline))
template <int N>
struct Int {
  static constexpr int value = N;
};
using Yes = Int<1>;
using No = Int<0>;

template <int BM, int BN, int WM, int WN, int KS, int NS, bool SHIFT>
struct Tile {
  static constexpr int kGroup = WM * WN;  // wavefronts of a group
  static constexpr int kWaves = kGroup * KS;
  static constexpr int kMT = BM / WM / 16;  // 16-row operand tiles per wavefront
  static constexpr int kNT = BN / WN / 16;
  static constexpr int kLoadsA = BM / 8 / kGroup;  // wavefront loads per step
  static constexpr int kLoadsB = BN / 8 / kGroup;
  static constexpr int kStageBytes = (BM + BN) * kStepK;
  static constexpr int kSumBytes = KS > 1 ? KS * BM * BN * 4 : 0;
  static constexpr int kRingBytes = NS * kStageBytes;   // a group's buffers
  static constexpr int kLdsBytes = KS * kRingBytes > kSumBytes ? KS * kRingBytes : kSumBytes;
  static_assert(kLoadsA * 8 * kGroup == BM && kLoadsB * 8 * kGroup == BN, "whole loads");
  static_assert(kLdsBytes <= 160 * 1024, "a compute unit's LDS");
  // steps that are under way or sent for at a time: with shifted windows a step lies
  // in two buffers
  static constexpr int kDepth = SHIFT ? NS - 1 : NS;
  static_assert(kDepth >= 2 && kDepth <= 4, "the last steps are written out");
  static_assert(!SHIFT || KS == 1, "a group's windows follow one another");
};

typedef __attribute__((address_space(3))) int8_t lds_byte;

// 16 bytes per lane from `rows` into LDS at `lds` + 16 lane.  Written as asm so
// that the compiler, which cannot tell the two buffers apart, does not wait for
// these loads before every read of LDS; nothing comes back in registers, and
// wait_loads() and a barrier stand between these writes and their reads.  The load
// reads M0, which needs a wait state after its scalar write; the compiler puts none
// inside an asm string.  (M0 is a reserved register, which a clobber list cannot name;
// the compiler uses it for nothing else here.)
__device__ __forceinline__ void lds_load16(const CodeRows& rows, uint32_t lds, uint32_t off) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :
               : "s"(lds), "v"(off), "s"(rows.rs)
               : "memory");
}

__device__ __forceinline__ u32x4 lds_read16(uint32_t at) {
  return *reinterpret_cast<const u32x4 __attribute__((address_space(3)))*>(at);
}

// vmcnt(N): all but this wavefront's last N loads into LDS have landed
template <int N>
__device__ __forceinline__ void wait_loads() {
  static_assert(N < 64, "the count's six bits");
  __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | (N >> 4) << 14);
}

// Which tile a block makes: every XCD takes a contiguous range of ids, and ids
// run down 4 rows of tiles before the next column, so that blocks running at
// the same time on one XCD share operand rows in its L2.
constexpr unsigned kTileGroup = 4;
__device__ __forceinline__ void tile_of_block(unsigned tiles_m, unsigned tiles_n, unsigned& ti,
                                              unsigned& tj) {
  const unsigned id = unsigned(xcd_block_id());
  const unsigned per = kTileGroup * tiles_n, grp = id / per, first = grp * kTileGroup;
  const unsigned rows = tiles_m - first < kTileGroup ? tiles_m - first : kTileGroup;
  const unsigned in = id - grp * per;
  ti = first + in % rows;
  tj = in / rows;
}

template <int BM, int BN, int WM, int WN, int KS, int NS, bool SHIFT, int OUT>
__global__ __launch_bounds__(64 * WM * WN * KS, 2) void matmul_tiled_kernel(MatmulArgs p,
                                                                           unsigned tiles_m,
                                                                           unsigned tiles_n) {
  using T = Tile<BM, BN, WM, WN, KS, NS, SHIFT>;
  constexpr int kDepth = T::kDepth;
  __shared__ __attribute__((aligned(1024))) int8_t lds[T::kLdsBytes];
  const int lane = lane_id(), group = wave_id() / T::kGroup, w = wave_id() % T::kGroup;
  // the group's ring of buffers, and the one in use
  const uint32_t ring = uint32_t(reinterpret_cast<uintptr_t>((lds_byte*)lds)) +
                        uint32_t(group) * T::kRingBytes;
  uint32_t base = ring;
  auto next = [&](uint32_t at) ARMX_INLINE {
    return at == ring + (NS - 1) * T::kStageBytes ? ring : at + T::kStageBytes;
  };
  unsigned ti, tj;
  tile_of_block(tiles_m, tiles_n, ti, tj);
  const uint64_t i0 = uint64_t(ti) * BM, j0 = uint64_t(tj) * BN;
  const CodeRows a(p.a, p.m, p.lda, p.k, i0), b(p.b, p.n, p.ldb, p.k, j0);
  const uint32_t k = uint32_t(p.k);
  // rows past the matrix are read from its last row; their outputs are not stored
  uint32_t off_a[T::kLoadsA], off_b[T::kLoadsB];
  const uint32_t last_a = uint32_t(p.m - 1 - i0 < BM ? p.m - 1 - i0 : BM - 1);
  const uint32_t last_b = uint32_t(p.n - 1 - j0 < BN ? p.n - 1 - j0 : BN - 1);
  // pieces from a line's start to that of a tile's row (SHIFT)
  auto phase = [&](const int8_t* rows, uint32_t ld, uint32_t row) ARMX_INLINE {
    return SHIFT ? (uint32_t(reinterpret_cast<uintptr_t>(rows) >> 4) + row * (ld >> 4)) & 7 : 0u;
  };
  const int8_t* tile_a = p.a + i0 * p.lda;
  const int8_t* tile_b = p.b + j0 * p.ldb;
  // byte offset of the piece that this lane brings into its slot of tile row
  // `row`, which is row `at` of an operand tile; one in front of the tile (SHIFT)
  // wraps past the buffer's end
  auto source = [&](const int8_t* rows, uint32_t row, uint32_t at, uint32_t last, uint32_t ld)
      ARMX_INLINE {
    return (row < last ? row : last) * ld + ((uint32_t(lane) & 7) ^ swizzle(at)) * 16 -
           phase(rows, ld, row) * 16;
  };
#pragma unroll
  for (int x = 0; x < T::kLoadsA; ++x) {
    const uint32_t row = (w * T::kLoadsA + x) * 8 + (lane >> 3);
    off_a[x] = source(tile_a, row, row, last_a, uint32_t(p.lda));
  }
#pragma unroll
  for (int x = 0; x < T::kLoadsB; ++x) {
    const uint32_t row = (w * T::kLoadsB + x) * 8 + (lane >> 3);
    off_b[x] =
        source(tile_b, row, row / (4 * T::kNT) * 4 + row % 4, last_b, uint32_t(p.ldb));
  }
  // wavefront load x of the step at k0, into the buffer at `to`
  auto stage_one = [&](uint32_t to, uint32_t k0, int x) ARMX_INLINE {
    if (x < T::kLoadsA) {
      lds_load16(a, to + (w * T::kLoadsA + x) * 1024, off_a[x] + k0);
    } else {
      x -= T::kLoadsA;
      lds_load16(b, to + BM * kStepK + (w * T::kLoadsB + x) * 1024, off_b[x] + k0);
    }
  };
  constexpr int kLoads = T::kLoadsA + T::kLoadsB;
  auto stage = [&](uint32_t to, uint32_t k0) ARMX_INLINE {
#pragma unroll
    for (int x = 0; x < kLoads; ++x) stage_one(to, k0, x);
  };
  // all but the group's last `steps` steps of loads have landed and all its reads are
  // done; a group of one wavefront has only itself to wait for
  auto sync = [&](auto steps) ARMX_INLINE {
    wait_loads<decltype(steps)::value * kLoads>();
    if constexpr (T::kGroup > 1)
      __syncthreads();
    else
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  };
  // operand registers of half a step (64 codes of k): lane l reads row l % 16,
  // piece 4 half + l / 16, which with SHIFT lies its row's phase further on, perhaps
  // in the next buffer.  Rows 16 apart have one phase (pitches are multiples of 16),
  // and of those 4 apart every other one (kinds of b's tiles: even and odd).
  constexpr int kKinds = SHIFT ? 2 : 1;
  const uint32_t r = lane & 15, g = lane >> 4;
  uint32_t at_a[2], at_b[2][kKinds];
  bool far_a[2] = {false, false}, far_b[2][kKinds] = {};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t piece = 4 * h + g + phase(tile_a, uint32_t(p.lda), r);
    far_a[h] = SHIFT && piece >= 8;
    at_a[h] = ((w % WM) * (BM / WM) + r) * kStepK + ((piece & 7) ^ swizzle(r)) * 16;
#pragma unroll
    for (int q = 0; q < kKinds; ++q) {
      const uint32_t row = (w / WM) * (BN / WN) + r / 4 * (4 * T::kNT) + r % 4 + 4 * q;
      piece = 4 * h + g + phase(tile_b, uint32_t(p.ldb), row);
      far_b[h][q] = SHIFT && piece >= 8;
      at_b[h][q] = (BM + row - 4 * q) * kStepK + ((piece & 7) ^ swizzle(r)) * 16;
    }
  }
  u32x4 fa[2][T::kMT], fb[2][T::kNT];
  constexpr int kReads = T::kMT + T::kNT;
  // Where this lane reads half h of the buffer at `from`; opaque to the compiler, so
  // that it keeps two addresses and puts the rest into the reads' offsets (left to
  // itself it adds up an address for every read).
  struct Place {
    uint32_t a, b[kKinds];
  };
  auto place = [&](uint32_t from, int h) ARMX_INLINE {
    const uint32_t after = SHIFT ? next(from) : from;
    Place at;
    at.a = (far_a[h] ? after : from) + at_a[h];
    asm("" : "+v"(at.a));
#pragma unroll
    for (int q = 0; q < kKinds; ++q) {
      at.b[q] = (far_b[h][q] ? after : from) + at_b[h][q];
      asm("" : "+v"(at.b[q]));
    }
    return at;
  };
  // read j of half h, in the order in which its products need them
  auto fetch = [&](Place at, int h, int j) ARMX_INLINE {
    if (j < T::kNT)
      fb[h][j] = lds_read16(at.b[j % kKinds] + j * 4 * kStepK);
    else
      fa[h][j - T::kNT] = lds_read16(at.a + (j - T::kNT) * 16 * kStepK);
  };
  auto fetch_half = [&](uint32_t from, int h) ARMX_INLINE {
    const Place at = place(from, h);
#pragma unroll
    for (int j = 0; j < kReads; ++j) {
      fetch(at, h, j);
      // in this order: the wait at the loop's head is the stricter of the two
      // orders that reach it
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // codes past k are cut from a's operands
  auto mask_half = [&](uint32_t k0, int h) ARMX_INLINE {
    const int keep = int(k) - int(k0 + 64 * h + 16 * g);
#pragma unroll
    for (int x = 0; x < T::kMT; ++x) fa[h][x] = keep_codes(fa[h][x], keep);
  };
  i32x4 acc[T::kMT][T::kNT];
#pragma unroll
  for (int x = 0; x < T::kMT; ++x)
#pragma unroll
    for (int y = 0; y < T::kNT; ++y) acc[x][y] = i32x4{0, 0, 0, 0};
  auto multiply_row = [&](int h, int x) ARMX_INLINE {
#pragma unroll
    for (int y = 0; y < T::kNT; ++y) acc[x][y] = mfma_i8(fb[h][y], fa[h][x], acc[x][y]);
  };
  auto multiply = [&](int h) ARMX_INLINE {
#pragma unroll
    for (int x = 0; x < T::kMT; ++x) multiply_row(h, x);
  };
  // The products of one half, with the other's operands (h) read from `from`
  // and, with SEND, the loads of the step at k0 into `to` spread between them.
  auto multiply_and_fetch = [&](int h, uint32_t from, auto send, uint32_t to, uint32_t k0)
      ARMX_INLINE {
    constexpr int kPer = (kLoads + T::kMT - 1) / T::kMT;
    constexpr int kPerR = (kReads + T::kMT - 1) / T::kMT;
    const Place at = place(from, h);
#pragma unroll
    for (int i = 0; i < T::kMT; ++i) {
      if constexpr (send.value) {
#pragma unroll
        for (int j = i * kPer; j < (i + 1) * kPer; ++j)
          if (j < kLoads) stage_one(to, k0, j);
      }
#pragma unroll
      for (int j = i * kPerR; j < (i + 1) * kPerR; ++j)
        if (j < kReads) fetch(at, h, j);
      __builtin_amdgcn_sched_barrier(0);
      multiply_row(1 - h, i);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // A step but the last (its first half's operands already in registers): the
  // second half's are read while the first is multiplied; then, after the
  // barrier that ends all reading of this buffer and finds the next one filled
  // (`out`: steps sent for behind that one), the step NS on is sent for into it
  // (SEND) and the next step's first half read under the second half's products.
  constexpr uint32_t kStride = KS * kStepK;
  auto step = [&](auto send, auto out, uint32_t k0) ARMX_INLINE {
    multiply_and_fetch(1, base, No{}, 0, 0);
    sync(out);
    const uint32_t other = next(base);
    multiply_and_fetch(0, other, send, base, k0 + NS * kStride);
    base = other;
  };
  if (k > 0) {
    // every group makes the same number of steps, counted by `left`, so that all
    // meet at the barriers; one that lies past k loads nothing (the range check)
    // and is cut to zeros
    uint32_t k0 = uint32_t(group) * kStepK;
    uint32_t left = (k + kStride - 1) / kStride;
    if (left >= kDepth) {
#pragma unroll
      for (int t = 0; t < NS; ++t) stage(ring + t * T::kStageBytes, k0 + t * kStride);
      sync(Int<kDepth - 1>{});
    } else {
      for (uint32_t t = 0; t < left + (SHIFT ? 1 : 0); ++t)
        stage(ring + t * T::kStageBytes, k0 + t * kStride);
      sync(No{});
    }
    fetch_half(base, 0);
    for (; left > kDepth; --left, k0 += kStride) step(Yes{}, Int<kDepth - 2>{}, k0);
    // the last steps; what is still out shrinks with them
    if constexpr (kDepth > 3)
      if (left > 3) {
        step(No{}, Int<kDepth - 2>{}, k0);
        --left, k0 += kStride;
      }
    if constexpr (kDepth > 2)
      if (left > 2) {
        step(No{}, Int<1>{}, k0);
        --left, k0 += kStride;
      }
    if (left > 1) {
      step(No{}, No{}, k0);
      k0 += kStride;
    }
    fetch_half(base, 1);
    mask_half(k0, 0);
    multiply(0);
    mask_half(k0, 1);
    multiply(1);
  }
  constexpr int kCols = 4 * T::kNT;   // a lane's columns of a row
  auto columns = [&](int wave) ARMX_INLINE {
    return Columns<OUT, kCols>(p, j0 + (wave / WM) * (BN / WN) + kCols * g);
  };
  if constexpr (KS == 1) {
    const auto out = columns(w);
#pragma unroll
    for (int x = 0; x < T::kMT; ++x) out.store(i0 + (w % WM) * (BM / WM) + 16 * x + r, acc[x]);
  } else {
    // the groups' sums meet in LDS; 16 rows of a wavefront's tile at a time are
    // added and stored by one wavefront, dealt out over all of them
    constexpr int kRowUnits = T::kGroup * T::kMT;
    i32x4* sums = reinterpret_cast<i32x4*>(lds);
    __syncthreads();
#pragma unroll
    for (int x = 0; x < T::kMT; ++x)
#pragma unroll
      for (int y = 0; y < T::kNT; ++y)
        sums[(((group * T::kGroup + w) * T::kMT + x) * T::kNT + y) * 64 + lane] = acc[x][y];
    __syncthreads();
    for (int u = group * T::kGroup + w; u < kRowUnits; u += T::kWaves) {
      i32x4 v[T::kNT];
#pragma unroll
      for (int y = 0; y < T::kNT; ++y) {
        v[y] = sums[(u * T::kNT + y) * 64 + lane];
#pragma unroll
        for (int q = 1; q < KS; ++q) v[y] += sums[((q * kRowUnits + u) * T::kNT + y) * 64 + lane];
      }
      const int uw = u / T::kMT;
      columns(uw).store(i0 + (uw % WM) * (BM / WM) + 16 * (u % T::kMT) + r, v);
    }
  }
}

template <int OUT, int BM, int BN, int WM, int WN, int KS, int NS, bool SHIFT = false>
hipError_t launch_tiled(const MatmulArgs& p, const armx_config* cfg, hipStream_t stream) {
  MatmulArgs copy = p;
  unsigned tiles_m = unsigned((p.m + BM - 1) / BM), tiles_n = unsigned((p.n + BN - 1) / BN);
  void* args[] = {&copy, &tiles_m, &tiles_n};
  const auto fn = &matmul_tiled_kernel<BM, BN, WM, WN, KS, NS, SHIFT, OUT>;
  return launch_kernel(reinterpret_cast<const void*>(fn),
                       dim3(tiles_m * tiles_n), dim3(64 * WM * WN * KS), args, 0, stream,
                       cfg ? static_cast<hipEvent_t>(cfg->start_event) : nullptr,
                       cfg ? static_cast<hipEvent_t>(cfg->stop_event) : nullptr);
}

// ---- which tile ---------------------------------------------------------------
//
// The tile whose estimated time is least.  A compute unit that makes q tiles runs
// them in rounds of at most `resident` blocks; a round takes `fixed` (its first
// loads, its epilogue) and, per step of KS x 128 codes, `alone` or, with several
// blocks on the unit, `each` of them if that is more.  The constants (us) are
// fitted to times of each tile on MI355X over 192 shapes of 1 to 8192 rows, 128 to
// 28672 columns and lengths of 128 to 14336.  All eleven timed at 192 shapes of that
// range, the one they choose is 0.6% behind the fastest on average and 11% at worst.
// Each pays where it is chosen (us, it and the best of the others): 256 x 256 at
// 4096 x 4096 x 14336 175 (212); 192 x 192 at 2048 x 4100 x 5001 44.1 (56.5);
// 128 x 256 at 8192 x 1024 x 8192 61.4 (80.3); 192 x 128 at 1024 x 4100 x 5001 28.2
// (33.1); 128 x 128 at 1024 x 4096 x 14336 67.8 (78.0); 64 x 128 at 512 x 4096 x 14336
// 49.9 (58.6); 64 x 64 at 256 x 4096 x 14336 35.4 (44.8); 64 x 32 at
// 128 x 4096 x 14336 25.7 (34.9); 32 x 32 at 33 x 4096 x 14336 17.0 (22.3);
// 16 x 32 at 128 x 1024 x 8192 7.3 (8.3); 16 x 16 at 16 x 4096 x 14336 13.4 (18.2).
//
// Where rows do not all start on a 128-byte line, a step of a row lies in two lines,
// and each is moved twice; the tiles with SHIFT move it once (us, without and with it,
// at a pitch of k rounded up to 16: 128 x 128 at 777 x 4096 x 4112 24.2, 20.1;
// 192 x 128 at 1500 x 4096 x 14336 + 16 117, 84), and their times and those of the
// others at such rows are in a table of their own.  The tiles it chooses are 0.7%
// behind the fastest of the eleven on average and 24% at worst (1 x 12288 x 1024,
// 6.9 us; over the same shapes, at pitches off the lines).  256 x 256 has no room for a
// third buffer, and on 16 and 32 rows, whose lines stay in the first cache until their
// second use, the split along k pays more.
struct TileTime {
  int bm, bn, ks, resident;
  float fixed, alone, each;
};
constexpr TileTime kTiles[] = {
    {256, 256, 1, 1, 3.04f, 1.50f, 1.50f}, {192, 192, 1, 1, 4.80f, 0.84f, 0.84f},
    {128, 256, 1, 1, 3.46f, 0.86f, 0.86f}, {192, 128, 1, 1, 3.01f, 0.65f, 0.65f},
    {128, 128, 1, 1, 2.58f, 0.52f, 0.52f}, {64, 128, 1, 2, 2.22f, 0.11f, 0.33f},
    {64, 64, 1, 2, 1.93f, 0.09f, 0.19f},   {64, 32, 4, 1, 1.89f, 0.56f, 0.56f},
    {32, 32, 4, 1, 1.69f, 0.39f, 0.39f},   {16, 32, 8, 1, 1.42f, 0.70f, 0.70f},
    {16, 16, 8, 1, 1.28f, 0.46f, 0.46f},
};
constexpr TileTime kOffLineTiles[] = {
    {256, 256, 1, 1, 3.90f, 1.78f, 1.78f}, {192, 192, 1, 1, 5.59f, 0.97f, 0.97f},
    {128, 256, 1, 1, 2.34f, 1.15f, 1.15f}, {192, 128, 1, 1, 3.72f, 0.65f, 0.65f},
    {128, 128, 1, 1, 2.89f, 0.52f, 0.52f}, {128, 64, 1, 1, 2.11f, 0.36f, 0.36f},
    {64, 64, 1, 2, 1.95f, 0.22f, 0.20f},   {64, 32, 1, 2, 1.72f, 0.16f, 0.14f},
    {32, 32, 4, 1, 1.30f, 0.50f, 0.50f},   {16, 32, 8, 1, 0.81f, 0.94f, 0.94f},
    {16, 16, 8, 1, 0.89f, 0.63f, 0.63f},
};
static_assert(sizeof(kTiles) == sizeof(kOffLineTiles), "eleven each");

inline uint64_t ceil_div(uint64_t a, uint64_t b) { return (a + b - 1) / b; }

inline uint64_t tile_count(const TileTime& t, const MatmulArgs& p) {
  return ceil_div(p.m, uint64_t(t.bm)) * ceil_div(p.n, uint64_t(t.bn));
}

double tile_time(const TileTime& t, const MatmulArgs& p, int cu_count) {
  const uint64_t per_cu = ceil_div(tile_count(t, p), uint64_t(cu_count));
  const double steps = double(ceil_div(p.k, uint64_t(t.ks) * kStepK));
  auto round = [&](uint64_t blocks) {
    const double together = double(blocks) * t.each;
    return blocks == 0 ? 0.0 : t.fixed + steps * (together > t.alone ? together : t.alone);
  };
  return double(per_cu / t.resident) * round(t.resident) + round(per_cu % t.resident);
}

int choose_tile(const TileTime (&tiles)[11], const MatmulArgs& p, int cu_count) {
  int best = -1;
  for (int i = 0; i < 11; ++i) {
    if (tile_count(tiles[i], p) > 0x7FFFFFFFu / 1024) continue;  // the grid's limit
    if (best < 0 || tile_time(tiles[i], p, cu_count) < tile_time(tiles[best], p, cu_count))
      best = i;
  }
  return best;
}

template <int OUT>
hipError_t launch_typed(const MatmulArgs& p, int cu_count, const armx_config* cfg,
                        hipStream_t stream) {
  const MatmulTile tile = choose_matmul_tile(p, cu_count);
  if (!tile.off_lines) {
    switch (tile.index) {
      case 0: return launch_tiled<OUT, 256, 256, 2, 4, 1, 2>(p, cfg, stream);
      case 1: return launch_tiled<OUT, 192, 192, 4, 2, 1, 3>(p, cfg, stream);
      case 2: return launch_tiled<OUT, 128, 256, 2, 4, 1, 3>(p, cfg, stream);
      case 3: return launch_tiled<OUT, 192, 128, 4, 2, 1, 3>(p, cfg, stream);
      case 4: return launch_tiled<OUT, 128, 128, 2, 4, 1, 3>(p, cfg, stream);
      case 5: return launch_tiled<OUT, 64, 128, 2, 4, 1, 3>(p, cfg, stream);
      case 6: return launch_tiled<OUT, 64, 64, 2, 2, 1, 4>(p, cfg, stream);
      case 7: return launch_tiled<OUT, 64, 32, 1, 1, 4, 3>(p, cfg, stream);
      case 8: return launch_tiled<OUT, 32, 32, 1, 1, 4, 4>(p, cfg, stream);
      case 9: return launch_tiled<OUT, 16, 32, 1, 1, 8, 2>(p, cfg, stream);
      case 10: return launch_tiled<OUT, 16, 16, 1, 1, 8, 4>(p, cfg, stream);
    }
  } else {
    switch (tile.index) {
      case 0: return launch_tiled<OUT, 256, 256, 2, 4, 1, 2>(p, cfg, stream);
      case 1: return launch_tiled<OUT, 192, 192, 4, 2, 1, 3, true>(p, cfg, stream);
      case 2: return launch_tiled<OUT, 128, 256, 2, 4, 1, 3>(p, cfg, stream);
      case 3: return launch_tiled<OUT, 192, 128, 4, 2, 1, 4, true>(p, cfg, stream);
      case 4: return launch_tiled<OUT, 128, 128, 2, 4, 1, 4, true>(p, cfg, stream);
      case 5: return launch_tiled<OUT, 128, 64, 4, 2, 1, 4, true>(p, cfg, stream);
      case 6: return launch_tiled<OUT, 64, 64, 2, 2, 1, 5, true>(p, cfg, stream);
      case 7: return launch_tiled<OUT, 64, 32, 2, 2, 1, 5, true>(p, cfg, stream);
      case 8: return launch_tiled<OUT, 32, 32, 1, 1, 4, 4>(p, cfg, stream);
      case 9: return launch_tiled<OUT, 16, 32, 1, 1, 8, 2>(p, cfg, stream);
      case 10: return launch_tiled<OUT, 16, 16, 1, 1, 8, 4>(p, cfg, stream);
    }
  }
  return hipErrorInvalidValue;  // more tiles than the entry point lets through
}

}  // namespace

MatmulTile choose_matmul_tile(const MatmulArgs& p, int cu_count) {
  const uint64_t starts = reinterpret_cast<uintptr_t>(p.a) | reinterpret_cast<uintptr_t>(p.b) |
                          p.lda | p.ldb;
  const bool off = starts % 128 != 0;
  const TileTime(&tiles)[11] = off ? kOffLineTiles : kTiles;
  const int i = choose_tile(tiles, p, cu_count);
  if (i < 0) return {0, 0, 0, off, i};
  return {tiles[i].bm, tiles[i].bn, tiles[i].ks, off, i};
}

hipError_t launch_matmul_int8(const MatmulArgs& args, int cu_count, const armx_config* cfg,
                              hipStream_t stream) {
  switch (args.out_type) {
    case ARMX_F16: return launch_typed<ARMX_F16>(args, cu_count, cfg, stream);
    case ARMX_BF16: return launch_typed<ARMX_BF16>(args, cu_count, cfg, stream);
    default: return launch_typed<ARMX_F32>(args, cu_count, cfg, stream);
  }
}

}  // namespace armx
