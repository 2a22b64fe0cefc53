// Layer norm of rows with the residual's addition and dropout, its gradients, and
// dropout by itself.
//
// As in the root-mean-square norm a row lies in the registers of the threads that
// share it and every value is read and written once: HBM is the bound.  (8192 x 4096 bf16
// with residual and dropout 47 us, 5.7 TB/s read and written; its gradients with all that
// flows 72, 4.7 TB/s, 5 of them the join of the blocks' sums; dropout of 16384 x 8192 87,
// 6.1 TB/s; a large copy reaches 4.9.  The bits of dropout cost 120 vector instructions for
// 8 values, which hide under the loads of other wavefronts.)
//
// Mean and squared deviations are taken by a wavefront of its own part of the row
// first: its mean m (to 16 bits: coarse), then the sum q of (h - m)^2 and the sum e of h - m, which
// is what m's rounding left, so that the part's mean is m + e / n and its squared deviations
// q - e^2 / n.  Parts are joined by
//   mean = sum n_w mean_w / n,   M = sum (M_w + n_w (mean_w - mean)^2),
// sums of numbers of one sign, with one barrier a row.  Nothing cancels, whatever the
// row's offset (sums of h and of h^2 lose mean^2 / variance of their 24 bits).
#include <hip/hip_runtime.h>

#include <cstdint>

#include "device_common.hpp"
#include "dropout.hpp"
#include "launch.h"
#include "layer.h"
#include "row_pieces.hpp"

namespace armx {
namespace {

// How a row lies on threads: as row_shape, but rows of more than `from` and up to 512
// chunks with two chunks a thread, so that half as many wavefronts take and join their
// parts (us, one / two: norm of 8192 x 4096 34 / 24, with residual and dropout 55 / 50,
// 16384 x 2048 30 / 23 and 51 / 47, but 32768 x 1024 28 / 57 on one wavefront a block;
// gradients of 9000 x 3728 with all 82 / 73, but 16384 x 2048 66 / 72).
RowShape two_chunks(uint64_t cols, uint64_t from) {
  const uint64_t n = (cols + kRowVec - 1) / kRowVec;
  if (n > from && n <= 512) return {int((n + 127) / 128) * 64, 2};
  return row_shape(cols);
}
RowShape norm_shape(uint64_t cols) { return two_chunks(cols, 128); }
RowShape grad_shape(uint64_t cols) { return two_chunks(cols, 256); }

// What reaches the norm.
constexpr int kPlain = 0;     // x
constexpr int kResidual = 1;  // x + residual
constexpr int kDropped = 2;   // dropout of x, + residual if there is one

// How many of chunk `c`'s 8 values are in a row of `cols` (0 or less: none).
__device__ __forceinline__ int in_chunk(uint32_t cols, uint32_t c) {
  return int(cols) - int(c * 8);
}

// h of a chunk, as stored (one rounding)
template <int TYPE>
__device__ __forceinline__ u32x4 drop_sum8(const Dropper& d, u32x4 x, u32x4 r, uint32_t c,
                                           uint32_t row) {
  float a[8], b[8];
  widen8<TYPE>(x, a);
  widen8<TYPE>(r, b);
  d.apply(c, row, a);
#pragma unroll
  for (int i = 0; i < 8; ++i) a[i] += b[i];
  return narrow8<TYPE>(a);
}

template <int TYPE>
__device__ __forceinline__ u32x4 add8(u32x4 x, u32x4 r) {
  float a[8], b[8];
  widen8<TYPE>(x, a);
  widen8<TYPE>(r, b);
#pragma unroll
  for (int i = 0; i < 8; ++i) a[i] += b[i];
  return narrow8<TYPE>(a);
}

// m to 16 significant bits: a 16-bit value's difference from it is exact unless the value is
// more than 2^8 times m, or less than 2^-13 of it, where it is rounded (from an m of 24 bits
// most are, a row's alike, and their sum is off by that many times the rounding).
__device__ __forceinline__ float coarse(float m) {
  return __builtin_bit_cast(float, (__builtin_bit_cast(uint32_t, m) + 0x80u) & 0xFFFFFF00u);
}

// The mean of a row.  Of one below a quarter of the deviations, many of whose differences are
// rounded, the values' own sum is the more exact, of others what is made of the deviations.
// (Off by, rms, rows of 4096 values around 0: 1.7e-8 without either, now 4.4e-10, for 4% of the
// time of a norm of 16384 x 2048.  The squared deviations take each difference's rounding as
// it comes, 2^-24 of it.)
__device__ __forceinline__ float mean_of(float mean, float m2, float sum, uint32_t cols,
                                         float inv_cols) {
  const float n = float(cols), m = sum * inv_cols;
  return m * m * (16.0f * n) < m2 ? __builtin_fmaf(__builtin_fmaf(-m, n, sum), inv_cols, m) : mean;
}

// Mean and sum of squared deviations of a row, in each of its threads.
template <class L>
struct Moments {
  static constexpr int kWaves = L::kTpr ? 1 : L::kMax / 64;
  static constexpr int kLevels = log2_of(L::kTpr ? L::kTpr : 64);
  struct Lds {
    float mean[kWaves], m2[kWaves], sum[kWaves];
  };
  // values of wavefront `w`'s part of the row
  __device__ __forceinline__ static float part(uint32_t cols, int w) {
    if constexpr (L::kTpr != 0) return float(cols);
    int n = 0;
#pragma unroll
    for (int j = 0; j < L::kChunks; ++j) {
      const int left = int(cols) - int((j * blockDim.x + 64 * w) * 8);
      n += left < 0 ? 0 : left < 512 ? left : 512;
    }
    return float(n);
  }
  template <int TYPE>
  __device__ __forceinline__ static void run(const u32x4 (&h)[L::kChunks], uint32_t cols,
                                             float inv_cols, Lds* lds, int turn, float& mean,
                                             float& m2) {
    constexpr int C = L::kChunks;
    const int wave = L::kTpr ? 0 : wave_id();
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < C; ++j) {
      float f[8];
      widen8<TYPE>(h[j], f);   // trimmed: zeros past the row
      s += ((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7]));
    }
    // (m is near the mean and no more, so the quick reciprocal does)
    const float n = part(cols, wave), each = __builtin_amdgcn_rcpf(n);
    s = lane_tree(s, kLevels);
    const float m = coarse(s * each);
    float q = 0.0f, e = 0.0f;
#pragma unroll
    for (int j = 0; j < C; ++j) {
      float f[8];
      widen8<TYPE>(h[j], f);
      const int in = in_chunk(cols, j * L::threads() + L::lane());
      if (cols % 8 == 0) {   // whole chunks: in one with no values all differences are 0
        const float from = in > 0 ? m : 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float d = f[i] - from;
          q = __builtin_fmaf(d, d, q);
          e += d;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float d = i < in ? f[i] - m : 0.0f;
          q = __builtin_fmaf(d, d, q);
          e += d;
        }
      }
    }
    q = lane_tree(q, kLevels);
    e = lane_tree(e, kLevels);
    mean = m + e * each;
    m2 = q - e * (e * each);
    if constexpr (L::kTpr == 0) {
      Lds& l = lds[turn];
      if (lane_id() == 0) {
        l.mean[wave] = mean;
        l.m2[wave] = m2;
        l.sum[wave] = s;
      }
      __syncthreads();
      const int waves = num_waves();
      const float first = l.mean[0];
      float off = 0.0f;
      s = l.sum[0];
#pragma unroll 4
      for (int w = 1; w < waves; ++w) {
        off = __builtin_fmaf(part(cols, w), l.mean[w] - first, off);
        s += l.sum[w];
      }
      mean = first + off * inv_cols;
      m2 = 0.0f;
#pragma unroll 4
      for (int w = 0; w < waves; ++w) {
        const float d = l.mean[w] - mean;
        m2 += __builtin_fmaf(part(cols, w) * d, d, l.m2[w]);
      }
    }
    mean = mean_of(mean, m2, s, cols, inv_cols);
  }
};

__device__ __forceinline__ float inv_std_of(float m2, float inv_cols, float eps) {
  // (a part's deviations may come out a rounding below 0 where they are none)
  const float v = m2 * inv_cols;
  return __builtin_amdgcn_rsqf((v < 0.0f ? 0.0f : v) + eps);
}

template <int TYPE>
__device__ __forceinline__ u32x4 normed8(u32x4 h, u32x4 w, u32x4 b, float mean, float inv) {
  float f[8], g[8], a[8];
  widen8<TYPE>(h, f);
  widen8<TYPE>(w, g);
  widen8<TYPE>(b, a);
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = __builtin_fmaf((f[i] - mean) * inv, g[i], a[i]);
  return narrow8<TYPE>(f);
}

// ---- forward --------------------------------------------------------------------------

// A row group's h, and its store where the caller wants it.
template <int TYPE, int IN, bool STREAM, class L, int C>
__device__ __forceinline__ void load_sums(const LayerNormArgs& k, const Dropper& d, uint64_t base,
                                          uint16_t* to, uint64_t ldt, u32x4 (&h)[C]) {
  const uint32_t cols = uint32_t(k.cols), chunks = (cols + 7) / 8;
  const uint64_t row = base + L::row(), left = k.rows - base;
  load_row<L>(k.x + base * k.ldx, k.ldx, left, cols, h);
  if constexpr (IN != kPlain) {
    u32x4 res[C];
    // without a residual no row of it is there, and zeros come without a read
    load_row<L>(k.residual + (k.residual ? base * k.ldr : 0), k.ldr, k.residual ? left : 0, cols,
                res);
#pragma unroll
    for (int j = 0; j < C; ++j) {
      if constexpr (IN == kDropped)
        h[j] = drop_sum8<TYPE>(d, h[j], res[j], j * L::threads() + L::lane(), uint32_t(row));
      else
        h[j] = add8<TYPE>(h[j], res[j]);
    }
  }
  trim<L>(cols, h);
  if (to && row < k.rows) {
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const uint32_t c = j * L::threads() + L::lane();
      if (c < chunks) store_chunk8<STREAM>(to + row * ldt, c, cols, h[j]);
    }
  }
}

template <int TYPE, int IN, bool STREAM, class L>
__global__ __launch_bounds__(L::kMax) void layer_norm_kernel(LayerNormArgs k) {
  constexpr int C = L::kChunks;
  __shared__ typename Moments<L>::Lds lds[2];
  const uint32_t cols = uint32_t(k.cols), chunks = (cols + 7) / 8;
  const Dropper drop(k.dropout);
  u32x4 w[C], b[C];
  // (the registers of 1024 threads do not hold them beside the row's sums)
  constexpr bool kEarly = L::kMax < 1024;
  if constexpr (kEarly) {
    load_weight<L>(k.weight, cols, w);
    load_weight<L>(k.bias, k.bias ? cols : 0, b);
  }
  int turn = 0;
  // every thread of a block makes the same number of rounds (barriers)
  for (uint64_t base = uint64_t(blockIdx.x) * L::kRows; base < k.rows;
       base += uint64_t(gridDim.x) * L::kRows, turn ^= 1) {
    const uint64_t row = base + L::row();
    u32x4 h[C];
    load_sums<TYPE, IN, STREAM, L>(k, drop, base, IN == kPlain ? nullptr : k.sum_out, k.lds, h);
    float mean, m2;
    Moments<L>::template run<TYPE>(h, cols, k.inv_cols, lds, turn, mean, m2);
    if (row >= k.rows) continue;
    const float inv = inv_std_of(m2, k.inv_cols, k.eps);
    if constexpr (!kEarly) {
      load_weight<L>(k.weight, cols, w);
      load_weight<L>(k.bias, k.bias ? cols : 0, b);
    }
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const uint32_t c = j * L::threads() + L::lane();
      if (c < chunks)
        store_chunk8<STREAM>(k.out + row * k.ldo, c, cols,
                             normed8<TYPE>(h[j], w[j], b[j], mean, inv));
    }
    if (L::lane() == 0) {
      if (k.mean) k.mean[row] = mean;
      if (k.inv_std) k.inv_std[row] = inv;
    }
  }
}

template <int TYPE, int IN, bool STREAM, class L>
__global__ __launch_bounds__(L::kMax) void dropout_kernel(LayerNormArgs k) {
  const Dropper drop(k.dropout);
  for (uint64_t base = uint64_t(blockIdx.x) * L::kRows; base < k.rows;
       base += uint64_t(gridDim.x) * L::kRows) {
    u32x4 h[L::kChunks];
    load_sums<TYPE, IN, STREAM, L>(k, drop, base, k.out, k.ldo, h);
  }
}

// One chunk of h of a row that is walked.
template <int TYPE, int IN>
__device__ __forceinline__ u32x4 load_sum_chunk(const LayerNormArgs& k, const Dropper& d,
                                                uint64_t row, uint32_t c) {
  const uint32_t cols = uint32_t(k.cols);
  const u32x4 x = load_chunk8(k.x + row * k.ldx, c, cols);
  if constexpr (IN == kPlain) return x;
  const u32x4 r = k.residual ? load_chunk8(k.residual + row * k.ldr, c, cols) : u32x4{0, 0, 0, 0};
  if constexpr (IN == kResidual) return add8<TYPE>(x, r);
  return drop_sum8<TYPE>(d, x, r, c, uint32_t(row));
}

// A block's sum of v, in every thread; `part` has a float per wavefront and is free
// again after the next barrier.
__device__ __forceinline__ float block_sum(float v, float* part) {
  v = lane_tree_full(v);
  if (lane_id() == 0) part[wave_id()] = v;
  __syncthreads();
  v = part[0];
  const int waves = num_waves();
  for (int w = 1; w < waves; ++w) v += part[w];
  return v;
}

// Rows too long for the registers: one block per row, walked twice.  A thread joins
// its chunks' means and deviations one by one, and the threads' are joined as the
// wavefronts' are above.
template <int TYPE, int IN>
__global__ __launch_bounds__(1024) void layer_norm_loop_kernel(LayerNormArgs k) {
  __shared__ float part[3][16];
  const uint32_t cols = uint32_t(k.cols), chunks = (cols + 7) / 8;
  const Dropper drop(k.dropout);
  for (uint64_t row = blockIdx.x; row < k.rows; row += gridDim.x) {
    float n = 0.0f, mean = 0.0f, m2 = 0.0f, sum = 0.0f;
    for (uint32_t c = threadIdx.x; c < chunks; c += 1024) {
      const u32x4 h = load_sum_chunk<TYPE, IN>(k, drop, row, c);
      if (IN != kPlain && k.sum_out) store_chunk8<false>(k.sum_out + row * k.lds, c, cols, h);
      float f[8];
      widen8<TYPE>(h, f);
      const int in = in_chunk(cols, c) < 8 ? in_chunk(cols, c) : 8;
      float s = 0.0f, q = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) s += i < in ? f[i] : 0.0f;
      const float m = s / float(in);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float d = i < in ? f[i] - m : 0.0f;
        q = __builtin_fmaf(d, d, q);
      }
      const float d = m - mean, all = n + float(in);
      m2 += __builtin_fmaf(d * d, n * (float(in) / all), q);
      mean = __builtin_fmaf(d, float(in) / all, mean);
      sum += s;
      n = all;
    }
    sum = block_sum(sum, part[0]);
    const float first = sum * k.inv_cols;
    const float d = mean - first;
    m2 = block_sum(__builtin_fmaf(n * d, d, m2), part[1]);
    // what the first mean's rounding left
    const float e = block_sum(n * d, part[2]);
    mean = first + e * k.inv_cols;
    m2 -= e * (e * k.inv_cols);
    mean = mean_of(mean, m2, sum, cols, k.inv_cols);
    const float inv = inv_std_of(m2, k.inv_cols, k.eps);
    for (uint32_t c = threadIdx.x; c < chunks; c += 1024) {
      // from sum_out (where this thread wrote it), so that outputs may stand where
      // inputs did
      const u32x4 h = IN != kPlain && k.sum_out ? load_chunk8(k.sum_out + row * k.lds, c, cols)
                                                : load_sum_chunk<TYPE, IN>(k, drop, row, c);
      const u32x4 w = load_chunk8(k.weight, c, cols);
      const u32x4 b = k.bias ? load_chunk8(k.bias, c, cols) : u32x4{0, 0, 0, 0};
      store_chunk8<false>(k.out + row * k.ldo, c, cols, normed8<TYPE>(h, w, b, mean, inv));
    }
    if (threadIdx.x == 0) {
      if (k.mean) k.mean[row] = mean;
      if (k.inv_std) k.inv_std[row] = inv;
    }
    __syncthreads();
  }
}

template <int TYPE, int IN>
__global__ __launch_bounds__(1024) void dropout_loop_kernel(LayerNormArgs k) {
  const uint32_t cols = uint32_t(k.cols), chunks = (cols + 7) / 8;
  const Dropper drop(k.dropout);
  for (uint64_t row = blockIdx.x; row < k.rows; row += gridDim.x)
    for (uint32_t c = threadIdx.x; c < chunks; c += 1024)
      store_chunk8<false>(k.out + row * k.ldo, c, cols, load_sum_chunk<TYPE, IN>(k, drop, row, c));
}

template <int TYPE, int IN, bool NORM>
hipError_t launch_typed(const LayerNormArgs& a, const armx_config* cfg, hipStream_t stream) {
  const RowShape s =
      for_pitch(NORM ? norm_shape(a.cols) : row_shape(a.cols),
                a.residual && a.ldr > a.ldx ? a.ldr : a.ldx);
  const bool stream_out = a.rows * a.cols >= kStreamValues;
  const void* fn = nullptr;
#define ARMX_ROWS_CASE(...)                                                                      \
  do {                                                                                           \
    if constexpr (NORM)                                                                          \
      fn = stream_out                                                                            \
               ? reinterpret_cast<const void*>(&layer_norm_kernel<TYPE, IN, true, __VA_ARGS__>)  \
               : reinterpret_cast<const void*>(&layer_norm_kernel<TYPE, IN, false, __VA_ARGS__>); \
    else                                                                                         \
      fn = stream_out                                                                            \
               ? reinterpret_cast<const void*>(&dropout_kernel<TYPE, IN, true, __VA_ARGS__>)     \
               : reinterpret_cast<const void*>(&dropout_kernel<TYPE, IN, false, __VA_ARGS__>);   \
  } while (0)
  ARMX_OF_SHAPE(s, ARMX_ROWS_CASE);
  if (is_widest(s)) ARMX_ROWS_CASE(WidestLay);
#undef ARMX_ROWS_CASE
  if (s.chunks == 0) {
    if constexpr (NORM)
      fn = reinterpret_cast<const void*>(&layer_norm_loop_kernel<TYPE, IN>);
    else
      fn = reinterpret_cast<const void*>(&dropout_loop_kernel<TYPE, IN>);
  }
  uint64_t blocks = (a.rows + block_rows(s) - 1) / block_rows(s);
  if (blocks > kMaxGrid) blocks = kMaxGrid;
  LayerNormArgs copy = a;
  void* args[] = {&copy};
  return launch_rows_kernel(fn, blocks, block_threads(s), args, cfg, stream);
}

// ---- backward ---------------------------------------------------------------------------

struct RowStats {
  float mean, inv;
};

// A block's row sums of two values, in each of the row's threads.
template <class L>
struct PairCombine {
  static constexpr int kWaves = L::kTpr ? 1 : L::kMax / 64;
  static constexpr int kLevels = log2_of(L::kTpr ? L::kTpr : 64);
  struct Lds {
    float a[kWaves], b[kWaves];
  };
  __device__ __forceinline__ static void run(float& a, float& b, Lds* lds, int turn) {
    a = lane_tree(a, kLevels);
    b = lane_tree(b, kLevels);
    if constexpr (L::kTpr == 0) {
      Lds& l = lds[turn];
      if (lane_id() == 0) {
        l.a[wave_id()] = a;
        l.b[wave_id()] = b;
      }
      __syncthreads();
      a = l.a[0];
      b = l.b[0];
      const int waves = num_waves();
#pragma unroll 4
      for (int w = 1; w < waves; ++w) {
        a += l.a[w];
        b += l.b[w];
      }
    }
  }
};

// One chunk's share of the row's sums of g and of g n, where g = dy weight and n is
// the normalised h.
template <int TYPE>
__device__ __forceinline__ void sums_chunk(u32x4 dy, u32x4 h, u32x4 w, RowStats r, float& a,
                                           float& b) {
  float fy[8], fh[8], fw[8];
  widen8<TYPE>(dy, fy);
  widen8<TYPE>(h, fh);
  widen8<TYPE>(w, fw);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float g = fy[i] * fw[i];
    a += g;
    b = __builtin_fmaf(g, (fh[i] - r.mean) * r.inv, b);
  }
}

// The gradient of h of a chunk; a, b: the means of g and of g n.
template <int TYPE>
__device__ __forceinline__ void grad_chunk(u32x4 dy, u32x4 h, u32x4 w, RowStats r, float a,
                                           float b, float (&f)[8]) {
  float fh[8], fw[8];
  widen8<TYPE>(dy, f);
  widen8<TYPE>(h, fh);
  widen8<TYPE>(w, fw);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float n = (fh[i] - r.mean) * r.inv;
    f[i] = r.inv * ((f[i] * fw[i] - a) - n * b);
  }
}

// GRAD: what else flows.
constexpr int kAlone = 0;    // nothing
constexpr int kJoined = 1;   // dsum
constexpr int kThrough = 2;  // dsum or not, and on through the dropout

// Stores the gradients of a chunk (ds: dsum's, zeros without one).
template <int TYPE, int GRAD, bool STREAM>
__device__ __forceinline__ void store_grad_chunk(const LayerNormBackwardArgs& k, const Dropper& d,
                                                 uint64_t row, uint32_t c, float (&f)[8],
                                                 u32x4 ds) {
  const uint32_t cols = uint32_t(k.cols);
  if constexpr (GRAD != kAlone) {
    float fd[8];
    widen8<TYPE>(ds, fd);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] += fd[i];
  }
  if constexpr (GRAD == kThrough) {
    if (k.dresidual)
      store_chunk8<STREAM>(k.dresidual + row * k.ldr, c, cols, narrow8<TYPE>(f));
    d.apply(c, uint32_t(row), f);
  }
  store_chunk8<STREAM>(k.dx + row * k.ldx, c, cols, narrow8<TYPE>(f));
}

template <int TYPE, int GRAD, bool STREAM, class L, int C>
__device__ __forceinline__ void store_grads(const LayerNormBackwardArgs& k, const Dropper& d,
                                            uint64_t row, RowStats r, float a, float b,
                                            const u32x4 (&dy)[C], const u32x4 (&h)[C],
                                            const u32x4 (&ds)[C], const u32x4 (&w)[C]) {
  const uint32_t cols = uint32_t(k.cols), chunks = (cols + 7) / 8;
  a *= k.inv_cols;
  b *= k.inv_cols;
#pragma unroll
  for (int j = 0; j < C; ++j) {
    const uint32_t c = j * L::threads() + L::lane();
    if (c < chunks) {
      float f[8];
      grad_chunk<TYPE>(dy[j], h[j], w[j], r, a, b, f);
      store_grad_chunk<TYPE, GRAD, STREAM>(k, d, row, c, f, ds[j]);
    }
  }
}

template <int GRAD, class L, int C>
__device__ __forceinline__ void load_dsum(const LayerNormBackwardArgs& k, uint64_t base,
                                          u32x4 (&ds)[C]) {
  if constexpr (GRAD != kAlone)
    load_row<L>(k.dsum + (k.dsum ? base * k.ldd : 0), k.ldd, k.dsum ? k.rows - base : 0,
                uint32_t(k.cols), ds);
}

// Block b takes the row groups b, b + blocks, ...; every thread keeps the sums for
// dweight and dbias of its own columns in registers over the block's rows.  A block of
// several rows at a time adds its row groups' sums through LDS, in order.
template <int TYPE, int GRAD, bool STREAM, class L>
__global__ __launch_bounds__(L::kMax) void layer_norm_backward_kernel(LayerNormBackwardArgs k,
                                                                     uint64_t pitch) {
  constexpr int C = L::kChunks;
  __shared__ typename PairCombine<L>::Lds lds[2];
  __shared__ float part[L::kRows > 1 ? kRowBlock * 8 : 1];
  const uint32_t cols = uint32_t(k.cols);
  const Dropper drop(k.dropout);
  u32x4 w[C];
  float dw[C][8], db[C][8];
#pragma unroll
  for (int j = 0; j < C; ++j) {
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[j][i] = db[j][i] = 0.0f;
  }
  load_weight<L>(k.weight, cols, w);
  // One row group's values; with kAhead the next group's are on their way while
  // this one's are combined.
  struct Rows {
    u32x4 dy[C], h[C], ds[C];
    RowStats r;
  };
  constexpr bool kAhead = C <= 2;
  auto load = [&](uint64_t base) __attribute__((always_inline)) {
    Rows v;
    const uint64_t row = base + L::row(), left = k.rows - base;
    v.r.mean = row < k.rows ? k.mean[row] : 0.0f;
    v.r.inv = row < k.rows ? k.inv_std[row] : 0.0f;
    load_row<L>(k.dy + base * k.ldy, k.ldy, left, cols, v.dy);
    load_row<L>(k.h + base * k.ldh, k.ldh, left, cols, v.h);
    load_dsum<GRAD, L>(k, base, v.ds);
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
    float a = 0.0f, b = 0.0f;
#pragma unroll
    for (int j = 0; j < C; ++j) {
      sums_chunk<TYPE>(now.dy[j], now.h[j], w[j], now.r, a, b);
      if (live) {
        float fy[8], fh[8];
        widen8<TYPE>(now.dy[j], fy);
        widen8<TYPE>(now.h[j], fh);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          dw[j][i] = __builtin_fmaf(fy[i], (fh[i] - now.r.mean) * now.r.inv, dw[j][i]);
          db[j][i] += fy[i];
        }
      }
    }
    PairCombine<L>::run(a, b, lds, turn);
    if (live)
      store_grads<TYPE, GRAD, STREAM, L>(k, drop, row, now.r, a, b, now.dy, now.h, now.ds, w);
  }
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    float* dst = k.partials + (uint64_t(blockIdx.x) * 2 + which) * pitch;
    auto& acc = which ? db : dw;
    if constexpr (L::kRows > 1) {
      constexpr uint32_t kPitch = L::kTpr * 8;
      if (which) __syncthreads();
#pragma unroll
      for (int i = 0; i < 8; ++i) part[L::row() * kPitch + L::lane() * 8 + i] = acc[0][i];
      __syncthreads();
      for (uint32_t e = threadIdx.x; e < cols; e += kRowBlock) {
        float v = part[e];
        for (int r = 1; r < L::kRows; ++r) v += part[r * kPitch + e];
        dst[e] = v;
      }
    } else {
#pragma unroll
      for (int j = 0; j < C; ++j) {
        const uint32_t c = j * L::threads() + L::lane();
        float* d = dst + uint64_t(c) * 8;
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
}

// dweight and dbias over all rows for 8 LANES columns (number `block` of them), by a
// whole block: LANES lanes take a row's, rows in steps of the block's, FLIGHT in
// flight.  part: two times 64 floats per wavefront.
template <int TYPE, int LANES, int FLIGHT>
__device__ __forceinline__ void sum_columns_in(const LayerNormBackwardArgs& k, uint32_t block,
                                               float (*part)[2][64]) {
  const uint32_t cols = uint32_t(k.cols), chunks = (cols + 7) / 8;
  const uint32_t c = block * LANES + threadIdx.x % LANES;
  // The last chunk is read as the row's last 8 values, without a branch (a lane with
  // none too); those in front of the chunk are the lane's before it.
  const uint32_t e0 = c * 8 + 8 <= cols ? c * 8 : cols - 8;
  const uint32_t step = blockDim.x / LANES;
  float dw[8] = {}, db[8] = {};
  for (uint64_t r = threadIdx.x / LANES; r < k.rows; r += FLIGHT * step) {
    u32x4 y[FLIGHT], x[FLIGHT];
    RowStats s[FLIGHT];
#pragma unroll
    for (int q = 0; q < FLIGHT; ++q) {
      // a row past the last is read as this thread's first, and not added
      const uint64_t rq = r + q * step < k.rows ? r + q * step : r;
      s[q] = {k.mean[rq], k.inv_std[rq]};
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
      for (int i = 0; i < 8; ++i) {
        dw[i] = __builtin_fmaf(fy[i], (fh[i] - s[q].mean) * s[q].inv, dw[i]);
        db[i] += fy[i];
      }
    }
  }
#pragma unroll
  for (int which = 0; which < 2; ++which) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {   // over the wavefront's rows: lanes LANES and more apart
      float v = which ? db[i] : dw[i];
      if constexpr (LANES == 4) v += dpp<kDppRor4>(v);
      v += dpp<kDppRor8>(v);
      v = add_xor16(v);
      v = add_xor32(v);
      const uint32_t e = (cols >= 8 ? e0 : c * 8) + i;
      if (lane_id() < LANES && c < chunks && e >= c * 8)
        part[wave_id()][which][e - block * (8 * LANES)] = v;
    }
  }
  __syncthreads();
  const uint32_t at = threadIdx.x % (8 * LANES), which = threadIdx.x / (8 * LANES);
  const uint32_t e = block * (8 * LANES) + at;
  if (which < 2 && e < cols) {
    float v = part[0][which][at];
    const int waves = num_waves();
    for (int q = 1; q < waves; ++q) v += part[q][which][at];
    (which ? k.dbias : k.dweight)[e] = v;
  }
}

// (eight rows in flight where four would take a second round, as in the
// root-mean-square norm's gradients)
template <int TYPE, bool LONG>
__device__ __forceinline__ void sum_columns(const LayerNormBackwardArgs& k, uint32_t block,
                                            float (*part)[2][64], bool half) {
  const bool one_round = k.rows <= 4 * (blockDim.x / (half ? 4 : 8));
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

// The rows' gradients and the sums over rows apart, in one launch without a workspace:
// the first `col_blocks` blocks each make dweight and dbias over all rows for 64 or 32
// columns (`half`), reading dy and h once more, and the others make the dx of their
// row groups.
template <int TYPE, int GRAD, class L>
__global__ __launch_bounds__(L::kMax) void layer_norm_backward_apart_kernel(
    LayerNormBackwardArgs k, unsigned col_blocks, bool half) {
  constexpr int C = L::kChunks;
  __shared__ typename PairCombine<L>::Lds lds[2];
  __shared__ float part[L::kMax / 64][2][64];
  if (blockIdx.x < col_blocks) {
    sum_columns<TYPE, (L::kMax > 512)>(k, blockIdx.x, part, half);
    return;
  }
  const uint32_t cols = uint32_t(k.cols);
  const Dropper drop(k.dropout);
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
    if constexpr (C < 4) load_dsum<GRAD, L>(k, base, ds);
    const RowStats r = {live ? k.mean[row] : 0.0f, live ? k.inv_std[row] : 0.0f};
    trim<L>(cols, dy);
    trim<L>(cols, h);
    trim<L>(cols, w);
    float a = 0.0f, b = 0.0f;
#pragma unroll
    for (int j = 0; j < C; ++j) sums_chunk<TYPE>(dy[j], h[j], w[j], r, a, b);
    // the registers do not hold dsum's four chunks during the sums above
    if constexpr (C == 4) load_dsum<GRAD, L>(k, base, ds);
    PairCombine<L>::run(a, b, lds, turn);
    if (live) store_grads<TYPE, GRAD, false, L>(k, drop, row, r, a, b, dy, h, ds, w);
  }
}

// The same for rows too long for the registers, which are walked twice, four chunks
// a thread at a time.
template <int TYPE, int GRAD>
__global__ __launch_bounds__(1024) void layer_norm_backward_loop_kernel(LayerNormBackwardArgs k,
                                                                        unsigned col_blocks,
                                                                        bool half) {
  typedef Lay<0, 1024, 4> L;
  __shared__ typename PairCombine<L>::Lds lds[2];
  __shared__ float part[16][2][64];
  if (blockIdx.x < col_blocks) {
    sum_columns<TYPE, true>(k, blockIdx.x, part, half);
    return;
  }
  const uint32_t cols = uint32_t(k.cols), chunks = (cols + 7) / 8;
  const Dropper drop(k.dropout);
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
    const RowStats r = {k.mean[row], k.inv_std[row]};
    float a = 0.0f, b = 0.0f;
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
        sums_chunk<TYPE>(cut(y[j], c), cut(h[j], c), cut(w[j], c), r, a, b);
      }
    }
    PairCombine<L>::run(a, b, lds, turn);
    a *= k.inv_cols;
    b *= k.inv_cols;
    const RowWords dr(k.dsum ? k.dsum + row * k.ldd : nullptr, GRAD != kAlone && k.dsum ? cols : 0);
    for (uint32_t c0 = threadIdx.x; c0 < chunks; c0 += 4096) {
      u32x4 y[4], h[4], w[4], d[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        y[j] = yr.load(c0 + j * 1024);
        h[j] = hr.load(c0 + j * 1024);
        w[j] = wr.load(c0 + j * 1024);
        if constexpr (GRAD != kAlone) d[j] = dr.load(c0 + j * 1024);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t c = c0 + j * 1024;
        if (c < chunks) {
          float f[8];
          grad_chunk<TYPE>(y[j], h[j], w[j], r, a, b, f);
          store_grad_chunk<TYPE, GRAD, false>(k, drop, row, c, f, d[j]);
        }
      }
    }
  }
}

// dweight and dbias from the blocks' partial sums (each 2 x pitch floats, dweight's in
// front): 4 consecutive columns per thread, kJoinParts threads of a block sharing the
// partial sums of its columns (part t takes t, t + kJoinParts, ..., eight loads in
// flight), whose sums are then added in order.
constexpr int kJoinCols = 32, kJoinParts = 32;
__global__ __launch_bounds__(kJoinCols / 4 * kJoinParts) void layer_norm_join_kernel(
    const float* partials, uint64_t blocks, uint64_t pitch, uint64_t cols, float* dweight,
    float* dbias) {
  constexpr int kQuads = kJoinCols / 4;
  __shared__ floatx4 part[kJoinParts][kQuads];
  const uint32_t tc = threadIdx.x % kQuads, tp = threadIdx.x / kQuads;
  // the pitch is a multiple of 64, so a quad past the columns is still inside it
  const uint64_t c = uint64_t(blockIdx.x) * kJoinCols + tc * 4;
  const floatx4* src =
      reinterpret_cast<const floatx4*>(partials + uint64_t(blockIdx.y) * pitch + c);
  floatx4 v = {0.0f, 0.0f, 0.0f, 0.0f};
  for (uint64_t b = tp; b < blocks; b += 8 * kJoinParts) {
    floatx4 t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint64_t bi = b + uint64_t(i) * kJoinParts;
      t[i] = src[(bi < blocks ? bi : b) * (pitch / 2)];
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
    float* to = blockIdx.y ? dbias : dweight;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (c + i < cols) to[c + i] = v[i];
  }
}

RowShape backward_shape(const LayerNormBackwardArgs& a, const NormBackwardPlan& plan) {
  uint64_t ld = a.ldy > a.ldh ? a.ldy : a.ldh;
  if (a.dsum && a.ldd > ld) ld = a.ldd;
  return for_pitch(plan.shape, ld);
}

template <int TYPE, int GRAD>
hipError_t launch_backward_apart(const LayerNormBackwardArgs& a, const NormBackwardPlan& plan,
                                 const armx_config* cfg, hipStream_t stream) {
  const RowShape s = backward_shape(a, plan);
  const void* fn = nullptr;
#define ARMX_ROWS_CASE(...) \
  fn = reinterpret_cast<const void*>(&layer_norm_backward_apart_kernel<TYPE, GRAD, __VA_ARGS__>)
  ARMX_OF_SHAPE(s, ARMX_ROWS_CASE);
  if (is_widest(s)) ARMX_ROWS_CASE(WidestLay);
#undef ARMX_ROWS_CASE
  if (s.chunks == 0)
    fn = reinterpret_cast<const void*>(&layer_norm_backward_loop_kernel<TYPE, GRAD>);
  LayerNormBackwardArgs copy = a;
  unsigned col_blocks = unsigned(column_blocks(plan.shape, a.cols));
  bool half = half_columns(plan.shape);
  void* args[] = {&copy, &col_blocks, &half};
  const uint64_t row_blocks = plan.blocks - col_blocks;
  // a result where dy or h is: every column's sums before any row's gradient
  auto over = [&](const void* p, uint64_t ld) {
    return p && (meet(p, ld, a.dy, a.ldy, a.rows, a.cols) ||
                 meet(p, ld, a.h, a.ldh, a.rows, a.cols));
  };
  if (!over(a.dx, a.ldx) && !over(a.dresidual, a.ldr))
    return launch_rows_kernel(fn, plan.blocks, plan.block, args, cfg, stream);
  const hipError_t e =
      launch_rows_kernel(fn, col_blocks, plan.block, args, cfg, stream, true, false);
  if (e != hipSuccess) return e;
  col_blocks = 0;
  return launch_rows_kernel(fn, row_blocks, plan.block, args, cfg, stream, false, true);
}

template <int TYPE, int GRAD>
hipError_t launch_backward_typed(const LayerNormBackwardArgs& a, const NormBackwardPlan& plan,
                                 const armx_config* cfg, hipStream_t stream) {
  if (plan.apart) return launch_backward_apart<TYPE, GRAD>(a, plan, cfg, stream);
  const RowShape s = backward_shape(a, plan);
  const bool stream_out = a.rows * a.cols >= kStreamValues;
  const void* fn = nullptr;
#define ARMX_ROWS_CASE(...)                                                                   \
  fn = stream_out ? reinterpret_cast<const void*>(                                            \
                        &layer_norm_backward_kernel<TYPE, GRAD, true, __VA_ARGS__>)           \
                  : reinterpret_cast<const void*>(                                            \
                        &layer_norm_backward_kernel<TYPE, GRAD, false, __VA_ARGS__>)
  ARMX_OF_SHAPE(s, ARMX_ROWS_CASE);
#undef ARMX_ROWS_CASE
  LayerNormBackwardArgs copy = a;
  uint64_t pitch = plan.pitch;
  void* args[] = {&copy, &pitch};
  hipError_t e = launch_rows_kernel(fn, plan.blocks, plan.block, args, cfg, stream, true, false);
  if (e != hipSuccess) return e;
  const float* partials = a.partials;
  uint64_t blocks = plan.blocks, cols = a.cols;
  float *dweight = a.dweight, *dbias = a.dbias;
  void* join_args[] = {&partials, &blocks, &pitch, &cols, &dweight, &dbias};
  return launch_kernel(reinterpret_cast<const void*>(&layer_norm_join_kernel),
                       dim3(unsigned((cols + kJoinCols - 1) / kJoinCols), 2),
                       dim3(kJoinCols / 4 * kJoinParts), join_args, 0, stream, nullptr,
                       cfg ? static_cast<hipEvent_t>(cfg->stop_event) : nullptr);
}

template <int TYPE, bool NORM>
hipError_t launch_in(const LayerNormArgs& a, const armx_config* cfg, hipStream_t stream) {
  if (a.drop) return launch_typed<TYPE, kDropped, NORM>(a, cfg, stream);
  if constexpr (!NORM) return hipErrorInvalidValue;   // a dropout always drops
  else
    return a.residual ? launch_typed<TYPE, kResidual, true>(a, cfg, stream)
                      : launch_typed<TYPE, kPlain, true>(a, cfg, stream);
}

template <int TYPE>
hipError_t launch_grad(const LayerNormBackwardArgs& a, const NormBackwardPlan& plan,
                       const armx_config* cfg, hipStream_t stream) {
  if (a.drop) return launch_backward_typed<TYPE, kThrough>(a, plan, cfg, stream);
  return a.dsum ? launch_backward_typed<TYPE, kJoined>(a, plan, cfg, stream)
                : launch_backward_typed<TYPE, kAlone>(a, plan, cfg, stream);
}

}  // namespace

NormBackwardPlan plan_layer_norm_backward(uint64_t rows, uint64_t cols, int cu_count) {
  NormBackwardPlan p = plan_norm_backward(rows, cols, cu_count);
  p.ws_bytes *= 2;
  const RowShape s = grad_shape(cols);
  if (p.apart || s.threads == p.shape.threads) return p;
  p.shape = s;
  p.block = block_threads(s);
  const uint64_t most = uint64_t(cu_count) * ((511 + p.block) / p.block);
  p.blocks = rows < most ? rows : most;   // a row at a time
  p.ws_bytes = size_t(2 * p.blocks * p.pitch * sizeof(float));
  return p;
}

hipError_t launch_layer_norm(const LayerNormArgs& a, const armx_config* cfg, hipStream_t stream) {
  if (a.weight)
    return a.type == ARMX_F16 ? launch_in<ARMX_F16, true>(a, cfg, stream)
                              : launch_in<ARMX_BF16, true>(a, cfg, stream);
  return a.type == ARMX_F16 ? launch_in<ARMX_F16, false>(a, cfg, stream)
                            : launch_in<ARMX_BF16, false>(a, cfg, stream);
}

hipError_t launch_layer_norm_backward(const LayerNormBackwardArgs& a,
                                      const NormBackwardPlan& plan, const armx_config* cfg,
                                      hipStream_t stream) {
  return a.type == ARMX_F16 ? launch_grad<ARMX_F16>(a, plan, cfg, stream)
                            : launch_grad<ARMX_BF16>(a, plan, cfg, stream);
}

}  // namespace armx
