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
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

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

// Scales, bias and rounding of 4 consecutive columns of one row, stored.
template <int OUT>
__device__ __forceinline__ void store_out4(const MatmulArgs& p, uint64_t i, uint64_t j, i32x4 acc,
                                           bool wide) {
  if (i >= p.m || j >= p.n) return;
  const float sa = p.a_scales[i];
  float y[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const uint64_t jc = j + c < p.n ? j + c : p.n - 1;
    y[c] = float(acc[c]) * (sa * p.b_scales[jc]);
    if (p.bias) {
      if constexpr (OUT == ARMX_F32)
        y[c] += static_cast<const float*>(p.bias)[jc];
      else if constexpr (OUT == ARMX_F16)
        y[c] += float(static_cast<const _Float16*>(p.bias)[jc]);
      else
        y[c] += float(static_cast<const __bf16*>(p.bias)[jc]);
    }
  }
  const bool full = wide && j + 4 <= p.n;
  if constexpr (OUT == ARMX_F32) {
    float* o = static_cast<float*>(p.out) + i * p.ldo + j;
    if (full) {
      *reinterpret_cast<floatx4*>(o) = floatx4{y[0], y[1], y[2], y[3]};
      return;
    }
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (j + c < p.n) o[c] = y[c];
  } else {
    u32x2 v;
    if constexpr (OUT == ARMX_F16) {
      v[0] = __builtin_bit_cast(uint32_t, half2v{_Float16(y[0]), _Float16(y[1])});
      v[1] = __builtin_bit_cast(uint32_t, half2v{_Float16(y[2]), _Float16(y[3])});
    } else {
      v[0] = __builtin_bit_cast(uint32_t, bf16x2{__bf16(y[0]), __bf16(y[1])});
      v[1] = __builtin_bit_cast(uint32_t, bf16x2{__bf16(y[2]), __bf16(y[3])});
    }
    uint16_t* o = static_cast<uint16_t*>(p.out) + i * p.ldo + j;
    if (full) {
      *reinterpret_cast<u32x2*>(o) = v;
      return;
    }
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (j + c < p.n) o[c] = uint16_t(v[c / 2] >> (16 * (c % 2)));
  }
}

// 64 x 64 outputs per block, 32 x 32 per wavefront, operands straight from
// memory to the MFMA's registers.
template <int OUT>
__global__ __launch_bounds__(256) void matmul_direct_kernel(MatmulArgs p, uint64_t tiles_n,
                                                            int wide) {
  const uint64_t ti = blockIdx.x / tiles_n, tj = blockIdx.x % tiles_n;
  const int lane = lane_id(), w = wave_id();
  const uint64_t i0 = ti * 64 + (w & 1) * 32, j0 = tj * 64 + (w >> 1) * 32;
  const CodeRows a(p.a, p.m, p.lda, p.k, i0), b(p.b, p.n, p.ldb, p.k, j0);
  const uint32_t r = lane & 15, g = uint32_t(lane >> 4) * 16;
  const uint32_t lda = uint32_t(p.lda), ldb = uint32_t(p.ldb), k = uint32_t(p.k);
  i32x4 acc[2][2];
#pragma unroll
  for (int x = 0; x < 2; ++x)
#pragma unroll
    for (int y = 0; y < 2; ++y) acc[x][y] = i32x4{0, 0, 0, 0};
  for (uint32_t t = 0; t < k; t += 64) {
    u32x4 va[2], vb[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      va[x] = keep_codes(a.load((r + 16 * x) * lda + t + g), int(k) - int(t + g));
      vb[x] = b.load((r + 16 * x) * ldb + t + g);
    }
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int y = 0; y < 2; ++y) acc[x][y] = mfma_i8(vb[y], va[x], acc[x][y]);
  }
#pragma unroll
  for (int x = 0; x < 2; ++x)
#pragma unroll
    for (int y = 0; y < 2; ++y)
      store_out4<OUT>(p, i0 + 16 * x + r, j0 + 16 * y + (lane >> 4) * 4, acc[x][y], wide != 0);
}

template <int OUT>
hipError_t launch_typed(const MatmulArgs& p, const armx_config* cfg, hipStream_t stream) {
  MatmulArgs copy = p;
  uint64_t tiles_n = (p.n + 63) / 64;
  const uint64_t blocks = (p.m + 63) / 64 * tiles_n;
  constexpr uint64_t quad = OUT == ARMX_F32 ? 16 : 8;
  int wide = p.ldo % 4 == 0 && reinterpret_cast<uintptr_t>(p.out) % quad == 0;
  void* args[] = {&copy, &tiles_n, &wide};
  return launch_kernel(reinterpret_cast<const void*>(&matmul_direct_kernel<OUT>),
                       dim3(unsigned(blocks)), dim3(256), args, 0, stream,
                       cfg ? static_cast<hipEvent_t>(cfg->start_event) : nullptr,
                       cfg ? static_cast<hipEvent_t>(cfg->stop_event) : nullptr);
}

}  // namespace

hipError_t launch_matmul_int8(const MatmulArgs& args, int cu_count, const armx_config* cfg,
                              hipStream_t stream) {
  (void)cu_count;
  switch (args.out_type) {
    case ARMX_F16: return launch_typed<ARMX_F16>(args, cfg, stream);
    case ARMX_BF16: return launch_typed<ARMX_BF16>(args, cfg, stream);
    default: return launch_typed<ARMX_F32>(args, cfg, stream);
  }
}

}  // namespace armx
