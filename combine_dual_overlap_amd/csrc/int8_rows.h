// Rows to 8-bit integers with a scale each: the arithmetic (gfx950).
// scale = amax * fp32(1 / 127), rounded to fp32, code = the integer nearest to x / scale,
// ties to even.  x times the rounded 1 / scale, added to 1.5 * 2^23 in one fma, leaves
// the nearest integer in the sum's low bits; it can only be wrong next to a half, which
// the exact remainder x - code * scale (one fma) shows, and is then put right.  So codes
// depend on the values alone, for six instructions each.  65536 x 2048 bf16: 67 us (5.9
// TB/s); with conversions and the comparisons in every one, 16 instructions, 85.  8192 x
// 2048 11.4 us; where a lane with a tie did all its chunks again, 15.4.
// A row that holds an infinity or NaN gets the scale NaN and codes 0: everything
// computed from it is NaN.
#pragma once

#include "rows.h"

namespace dbomoe {

struct RowQuant {
  float scale, up, s, inv, half;
  __device__ __forceinline__ explicit RowQuant(uint32_t amax_bits) {
    const float amax = __uint_as_float(amax_bits);
    if (amax_bits >= 0x7f800000u) {
      scale = __uint_as_float(0x7fc00000u);
      up = s = inv = half = 0.f;
      return;
    }
    scale = amax * (1.0f / 127.0f);
    up = amax < 1e-30f ? 0x1p100f : 1.0f;        // keeps 1 / scale and scale / 2 normal; exact
    s = scale * up;
    inv = s > 0.f ? 1.0f / s : 0.f;
    half = 0.5f * s;
  }
  __device__ __forceinline__ bool plain() const { return up == 1.0f && inv > 0.f; }
  // any row
  __device__ __forceinline__ int code(float x) const {
    x = inv > 0.f ? x * up : 0.f;
    float t = rintf(x * inv);
    const float d = fmaf(-t, s, x);              // exact: a multiple of the last bit, no larger than about half
    const bool odd = static_cast<int>(t) & 1;
    if (fabsf(d) > half || (fabsf(d) == half && odd)) t += copysignf(1.0f, d);
    return static_cast<int>(fminf(fmaxf(t, -127.0f), 127.0f));   // past 127 only where the scale is subnormal
  }
};

// A chunk's codes, four to a word, of any row.  A loop: it is not run often, and code
// that is read for the first time takes longer than what it does.
template <bool BF16>
__device__ __forceinline__ void codes_any(u32x4_t v, const RowQuant& rq, uint32_t (&w)[Chunk<BF16>::N / 4]) {
  uint64_t all = 0;
#pragma unroll 1
  for (int i = 0; i < 4; ++i) {
    const uint32_t x = v[0];
    if constexpr (BF16) {
      const uint32_t lo = rq.code(__uint_as_float(x << 16)) & 0xff, hi = rq.code(__uint_as_float(x & 0xffff0000u)) & 0xff;
      all = all >> 16 | static_cast<uint64_t>(lo | hi << 8) << 48;
    } else {
      all = all >> 8 | static_cast<uint64_t>(rq.code(__uint_as_float(x)) & 0xff) << 56;
    }
    v = u32x4_t{v[1], v[2], v[3], x};
  }
  if constexpr (BF16) w[0] = static_cast<uint32_t>(all);
  w[Chunk<BF16>::N / 4 - 1] = static_cast<uint32_t>(all >> 32);
}

// The same of a row whose scale is plain(); true where one is next to a half.
template <bool BF16>
__device__ __forceinline__ bool codes_plain(const u32x4_t& v, const RowQuant& rq, uint32_t (&w)[Chunk<BF16>::N / 4]) {
  constexpr int N = Chunk<BF16>::N;
  constexpr float kMagic = 12582912.0f;
  float f[N], most = 0.f;
  Chunk<BF16>::unpack(v, f);
  uint32_t y[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float t = fmaf(f[i], rq.inv, kMagic);
    y[i] = __float_as_uint(t);
    most = fmaxf(most, fabsf(fmaf(kMagic - t, rq.s, f[i])));
  }
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    const uint32_t lo = __builtin_amdgcn_perm(y[4 * i + 1], y[4 * i], 0x0c0c0400u);
    const uint32_t hi = __builtin_amdgcn_perm(y[4 * i + 3], y[4 * i + 2], 0x0c0c0400u);
    w[i] = lo | hi << 16;
  }
  return most >= rq.half;
}

// The same with those put right: the remainder is more than half the scale, or half
// and the code odd (as one comparison of bit patterns).
template <bool BF16>
__device__ __forceinline__ void codes_near(const u32x4_t& v, const RowQuant& rq, uint32_t (&w)[Chunk<BF16>::N / 4]) {
  constexpr int N = Chunk<BF16>::N;
  float f[N];
  Chunk<BF16>::unpack(v, f);
#pragma unroll
  for (int i = 0; i < N / 4; ++i) w[i] = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float t = fmaf(f[i], rq.inv, 12582912.0f);
    const int d = __float_as_int(fmaf(12582912.0f - t, rq.s, f[i]));
    uint32_t y = __float_as_uint(t);
    if ((d & 0x7fffffff) + static_cast<int>(y & 1) > __float_as_int(rq.half)) y += d >> 31 | 1;
    w[i / 4] |= (y & 0xff) << (8 * (i & 3));
  }
}

// Those of a lane's CH chunks.  Ties are common: a row of bf16 numbers as often as not
// holds half of its largest one, 63.5 times the scale.  Only the chunks that have one
// are done again.
template <bool BF16, int CH>
__device__ __forceinline__ void codes_of(const u32x4_t (&v)[CH], const RowQuant& rq, uint32_t (&w)[CH][Chunk<BF16>::N / 4]) {
  if (!rq.plain()) {                             // (the same in every lane of the row)
#pragma unroll
    for (int i = 0; i < CH; ++i) codes_any<BF16>(v[i], rq, w[i]);
    return;
  }
  uint32_t again = 0;
#pragma unroll
  for (int i = 0; i < CH; ++i) again |= static_cast<uint32_t>(codes_plain<BF16>(v[i], rq, w[i])) << i;
  if (again) {
#pragma unroll
    for (int i = 0; i < CH; ++i)
      if (again >> i & 1) codes_near<BF16>(v[i], rq, w[i]);
  }
}

template <bool BF16>
__device__ __forceinline__ void put_codes(int8_t* q, int c, const uint32_t (&w)[Chunk<BF16>::N / 4]) {
  if constexpr (BF16)
    *reinterpret_cast<uint2*>(q + static_cast<int64_t>(c) * 8) = make_uint2(w[0], w[1]);
  else
    *reinterpret_cast<uint32_t*>(q + static_cast<int64_t>(c) * 4) = w[0];
}

// The largest magnitude's bits, as those of an fp32 (bf16: two at a time).
template <bool BF16>
__device__ __forceinline__ uint32_t chunk_max_bits(const u32x4_t& v) {
  if constexpr (BF16) {
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    auto of = [&](int i) { return __builtin_bit_cast(u16x2, v[i] & 0x7fff7fffu); };
    const u16x2 m = __builtin_elementwise_max(__builtin_elementwise_max(of(0), of(1)), __builtin_elementwise_max(of(2), of(3)));
    return static_cast<uint32_t>(m[0] > m[1] ? m[0] : m[1]) << 16;
  } else {
    return max(max(v[0] & 0x7fffffffu, v[1] & 0x7fffffffu), max(v[2] & 0x7fffffffu, v[3] & 0x7fffffffu));
  }
}

}  // namespace dbomoe
