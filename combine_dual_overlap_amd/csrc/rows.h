// Kernels that keep a row in registers (gfx950): a row of 16-byte chunks is held
// by W waves, CH chunks in each lane (chunk i of a lane is i * 64 W + its thread).
#pragma once

#include <type_traits>

#include "common.h"

namespace dbomoe {

// Threads of a workgroup: one wave per row packs four rows into it, more waves have it to themselves.
template <int W>
struct RowShape {
  static constexpr int THREADS = W == 1 ? 256 : 64 * W;
  static constexpr int ROWS = W == 1 ? 4 : 1;
};

// The values of a chunk as floats and back.
template <bool BF16>
struct Chunk {
  static constexpr int N = BF16 ? 8 : 4;
  static __device__ __forceinline__ void unpack(const u32x4_t& v, float* f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (BF16) {
        f[2 * i] = __uint_as_float(v[i] << 16);
        f[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
      } else {
        f[i] = __uint_as_float(v[i]);
      }
    }
  }
  static __device__ __forceinline__ u32x4_t pack(const float* f) {
    u32x4_t v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (BF16) {
        typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
        bf16x2 h;
        h[0] = static_cast<__bf16>(f[2 * i]);           // round to nearest even
        h[1] = static_cast<__bf16>(f[2 * i + 1]);
        v[i] = __builtin_bit_cast(uint32_t, h);
      } else {
        v[i] = __float_as_uint(f[i]);
      }
    }
    return v;
  }
};

// Sum (or maximum of bit patterns) over the W waves of a row, the same in every
// lane; always added in the same order.  s: W words of LDS that no earlier
// exchange still reads (two exchanges in a row need two arrays, or a barrier).
template <int W>
__device__ __forceinline__ float row_sum(float v, float* s) {
  v = wave_sum_f(v);
  if constexpr (W > 1) {
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
    __syncthreads();
    v = s[0];
#pragma unroll
    for (int w = 1; w < W; ++w) v += s[w];
  }
  return v;
}

template <int W>
__device__ __forceinline__ uint32_t row_max_bits(uint32_t v, uint32_t* s) {
#pragma unroll
  for (int d = kWave / 2; d > 0; d >>= 1) v = max(v, static_cast<uint32_t>(__shfl_xor(static_cast<int>(v), d, kWave)));
  if constexpr (W > 1) {
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
    __syncthreads();
    v = s[0];
#pragma unroll
    for (int w = 1; w < W; ++w) v = max(v, s[w]);
  }
  return v;
}

// Calls f(W, CH) with the shape for rows of rc chunks (at most kRowMaxChunks):
// one wave while that holds the row in four chunks per lane and there are rows
// enough to fill the GPU with one wave each, else four, else sixteen.
constexpr int kRowMaxChunks = 4096;
template <typename F>
inline void with_row_shape(int64_t rows, int rc, F f) {
  auto with_ch = [&](auto w) {
    constexpr int W = decltype(w)::value;
    const int ch = (rc + 64 * W - 1) / (64 * W);
    if (ch <= 1)
      f(w, std::integral_constant<int, 1>{});
    else if (ch <= 2)
      f(w, std::integral_constant<int, 2>{});
    else
      f(w, std::integral_constant<int, 4>{});
  };
  if (rc <= 64 || (rc <= 256 && rows >= 2048))
    with_ch(std::integral_constant<int, 1>{});
  else if (rc <= 1024)
    with_ch(std::integral_constant<int, 4>{});
  else
    with_ch(std::integral_constant<int, 16>{});
}

}  // namespace dbomoe
