// The tiles that the products of 16-bit matrices are made of, and launches of them.
#pragma once

#include "cross_entropy.h"
#include "launch.h"
#include "tile16.hpp"

namespace armx {
namespace {

typedef Tile16<256, 256, 2, 4, 2, true> Tile0;
typedef Tile16<192, 256, 2, 4, 2> Tile1;
typedef Tile16<256, 128, 4, 2, 3> Tile2;
typedef Tile16<128, 128, 2, 2, 2> Tile3;
typedef Tile16<64, 128, 2, 2, 2> Tile4;
typedef Tile16<16, 128, 1, 2, 3> Tile5;
typedef Tile16<16, 64, 1, 1, 4> Tile6;
constexpr int kTile16s = 7;
constexpr uint64_t kLargestTile = 256;   // rows and columns

// Calls CASE(T) for tile number `index`.
#define ARMX_OF_TILE(index, CASE) \
  do {                            \
    switch (index) {              \
      case 0: CASE(Tile0); break; \
      case 1: CASE(Tile1); break; \
      case 2: CASE(Tile2); break; \
      case 3: CASE(Tile3); break; \
      case 4: CASE(Tile4); break; \
      case 5: CASE(Tile5); break; \
      case 6: CASE(Tile6); break; \
    }                             \
  } while (0)

__host__ __device__ inline uint64_t ceil_div(uint64_t a, uint64_t b) { return (a + b - 1) / b; }

// The first row of the product that a lane of a wavefront holds, in its tile, and the first
// column of the wavefront.
template <class T>
__device__ __forceinline__ uint32_t lane_row() {
  return (wave_id() % T::kWM) * (T::kBM / T::kWM) + (lane_id() & 15) * T::kRows;
}
template <class T>
__device__ __forceinline__ uint32_t wave_col() {
  return (wave_id() / T::kWM) * (T::kBN / T::kWN);
}
// A lane's column c of 16 (value c % 4 of operand tile c / 4), in its wavefront's 64.
__device__ __forceinline__ uint32_t lane_column(uint32_t c) {
  return c / 8 * 32 + uint32_t(lane_id() >> 4) * 8 + c % 8;
}
// Which of a lane's columns is column `at` of its wavefront; 16 or more: none.
__device__ __forceinline__ uint32_t column_index(int64_t at) {
  const bool mine = at >= 0 && at < 64 && uint32_t(at) / 8 % 4 == uint32_t(lane_id() >> 4);
  return mine ? uint32_t(at) / 32 * 8 + uint32_t(at) % 8 : 16u;
}

}  // namespace
}  // namespace armx
