// The tiles that the products of 16-bit matrices are made of, and launches of them.
#pragma once

#include "cross_entropy.h"
#include "launch.h"
#include "tile16.hpp"

namespace armx {
namespace {

typedef Tile16<256, 256, 2, 4, 2, true, true> Tile0;
typedef Tile16<192, 256, 2, 4, 2> Tile1;
typedef Tile16<256, 128, 4, 2, 3> Tile2;
typedef Tile16<128, 128, 2, 2, 2> Tile3;
typedef Tile16<64, 128, 2, 2, 2> Tile4;
typedef Tile16<32, 128, 1, 2, 3> Tile5;
typedef Tile16<16, 128, 1, 2, 3> Tile6;
typedef Tile16<16, 64, 1, 1, 4> Tile7;
constexpr int kTile16s = 8;
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
      case 7: CASE(Tile7); break; \
    }                             \
  } while (0)

inline uint64_t ceil_div(uint64_t a, uint64_t b) { return (a + b - 1) / b; }

// The first row and column of the product that a lane of a wavefront holds, in its tile.
template <class T>
__device__ __forceinline__ uint32_t lane_row() {
  return (wave_id() % T::kWM) * (T::kBM / T::kWM) + (lane_id() & 15) * T::kRows;
}
template <class T>
__device__ __forceinline__ uint32_t lane_col() {
  return (wave_id() / T::kWM) * (T::kBN / T::kWN) + (lane_id() >> 4) * T::kCols;
}

}  // namespace
}  // namespace armx
