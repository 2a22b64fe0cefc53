// Dropout's random bits: the counter-based generator Philox4x32-10 (Salmon, Moraes,
// Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011), whose words
// are a function of a key and a counter, so that no mask is stored and the backward
// pass makes the same bits again.
//
// The key is the seed, the counter of row r's chunk c of 8 values (c, r, low and high
// word of offset + step).  Its 128 bits are 16 for each value: a value's are compared
// with limit = round(65536 p).  (With 32 bits a value there are two calls a chunk, of
// 20 products of 32 x 32 bits each at a quarter of the rate of an addition: the vector
// units would take as long as HBM does.)
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "layer.h"

namespace armx {
namespace {

struct Dropper {
  uint32_t key0, key1, c2, c3, first_row, limit;
  float scale;

  // (a wavefront's lanes all read the same step)
  __device__ __forceinline__ explicit Dropper(const DropoutArgs& d)
      : key0(d.key0), key1(d.key1), first_row(d.first_row), limit(d.limit), scale(d.scale) {
    const uint64_t place = d.offset + (d.step ? *d.step : 0);
    c2 = uint32_t(place);
    c3 = uint32_t(place >> 32);
  }

  // The 8 x 16 bits of chunk `c` of row `row` of the call's matrix.
  __device__ __forceinline__ void bits(uint32_t c, uint32_t row, uint32_t (&v)[4]) const {
    uint32_t x0 = c, x1 = first_row + row, x2 = c2, x3 = c3;
    uint32_t k0 = key0, k1 = key1;
#pragma unroll
    for (int round = 0; round < 10; ++round) {
      const uint64_t a = uint64_t(x0) * 0xD2511F53u, b = uint64_t(x2) * 0xCD9E8D57u;
      x0 = uint32_t(b >> 32) ^ x1 ^ k0;
      x1 = uint32_t(b);
      x2 = uint32_t(a >> 32) ^ x3 ^ k1;
      x3 = uint32_t(a);
      k0 += 0x9E3779B9u;
      k1 += 0xBB67AE85u;
    }
    v[0] = x0, v[1] = x1, v[2] = x2, v[3] = x3;
  }

  // The chunk's values times the scale, or 0 (whatever stood there) where dropped.
  __device__ __forceinline__ void apply(uint32_t c, uint32_t row, float (&f)[8]) const {
    uint32_t v[4];
    bits(c, row, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = (v[i] & 0xFFFFu) >= limit ? f[2 * i] * scale : 0.0f;
      f[2 * i + 1] = v[i] >> 16 >= limit ? f[2 * i + 1] * scale : 0.0f;
    }
  }
};

}  // namespace
}  // namespace armx
