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

// A chunk that the caches need not keep (STREAM), or as ever.
template <bool STREAM>
__device__ __forceinline__ u32x4_t load_chunk(const u32x4_t* p) {
  if constexpr (STREAM) return __builtin_nontemporal_load(p);
  return *p;
}

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

// Sum over a wave, the same in every lane, by cross-lane adds in registers (six
// dependent adds; through LDS permutes the same takes six round trips).
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_add(float v) {
  const int o = __builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, ROWS, 0xf, false);
  return v + __int_as_float(o);
}
__device__ __forceinline__ float wave_sum_dpp(float v) {
  v = dpp_add<0x111, 0xf>(v);          // row_shr 1, 2, 4, 8: lane 15 of each 16 has their sum
  v = dpp_add<0x112, 0xf>(v);
  v = dpp_add<0x114, 0xf>(v);
  v = dpp_add<0x118, 0xf>(v);
  v = dpp_add<0x142, 0xa>(v);          // lane 15 of a row to the next, lane 31 to the upper half
  v = dpp_add<0x143, 0xc>(v);
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

// Sum (or maximum of bit patterns) over the W waves of a row, the same in every
// lane; always added in the same order.  s: W words of LDS that no earlier
// exchange still reads (two exchanges in a row need two arrays, or a barrier).
template <int W>
__device__ __forceinline__ float row_sum(float v, float* s) {
  v = wave_sum_dpp(v);
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

// Calls f(W, CH) with the shape for rows of rc chunks (at most kRowMaxChunks): one
// wave for rows of up to `narrow` chunks (64, 128 or 256; short rows of few tokens
// excepted), else four, else sixteen.  Sixteen waves for a row of 256 chunks took
// twice the time of one or four in every kernel; of rows of 896 chunks they are on par
// with four, and with few rows, where a lane's one chunk leaves room for all the rows of
// a combine at once, faster: 256 x 7168 combined (k = 8) and normed 8.9 us against 11.4,
// normed 3.6 / 4.3, quantised 3.7 / 3.9; 512 rows 19.0 / 17.1, 5.2 / 4.9, 4.8 / 4.6.
constexpr int kRowMaxChunks = 4096;
template <typename F>
inline void with_row_shape(int64_t rows, int rc, int narrow, F f) {
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
  // (256 rows of 256 chunks: 5.5 us with four waves each, 9.9 us with one)
  if (rc <= 64 || (rc <= narrow && rows >= 2048))
    with_ch(std::integral_constant<int, 1>{});
  else if (rc <= 512 || (rc <= 1024 && rows > 256))
    with_ch(std::integral_constant<int, 4>{});
  else
    with_ch(std::integral_constant<int, 16>{});
}

}  // namespace dbomoe
