// AdamW over many tensors in few launches, for gfx950.
//   m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2,  g = grad * grad_scale
//   p = p (1 - lr wd) - lr / (1 - b1^t) * m / (sqrt(v / (1 - b2^t)) + eps)
// in fp32.  HBM-bound: every tensor is read
// once and written once.
//
// 8-bit states: blocks of 128 consecutive elements hold E4M3 codes and one
// E8M0 byte b (scale 2^(b-127), the smallest with max <= 448 * scale), as the
// fp8 rows of the dispatch do.  The second moment is stored as its square
// root, which halves its range in powers of two.  Codes are rounded
// stochastically: a step changes a state by less than half a code's distance
// for almost every element (b2 = 0.999 changes sqrt(v) by 0.05 %, a code is
// up to 12 % away), so rounding to nearest would hold it where it is.  A
// nonzero sqrt(v) never becomes code 0, or the next step would divide by eps
// alone.  bf16 parameters without an fp32 master are rounded stochastically
// for the same reason.  What is not finite becomes a NaN code and has no part in
// its block's scale.
//
// Random numbers: two 32-bit hashes of (seed, step, tensor, element), so the
// result depends on nothing else.  mix() is two rounds of xor-shift and
// multiplication, a bijection of 32-bit words, with the constants that C. Wellons
// found by search for a low bias ("Prospecting for Hash Functions", 2018);
// 0x9e3779b9 is 2^32 over the golden ratio, 0x85ebca77 an odd constant.
#include <math.h>
#include <string.h>

#include <algorithm>
#include <type_traits>

#include "common.h"

namespace dbomoe {

constexpr int kAdamTensors = 4096;    // tensors per launch at most (64 x 64: two ballots find one)
constexpr int kAdamGroup = 2048;      // elements a workgroup takes at a time (8 a thread)
constexpr uint32_t kAdamMagic = 0x41644d57;

struct AdamTensor {
  void* p;
  const void* g;
  void* m;
  void* v;
  uint8_t* ms;
  uint8_t* vs;
  float* master;
  int64_t n;
  uint32_t key;                       // 0x85ebca77 * the tensor's number
};

// The table: a header, the launches (tensors of one combination of types), the
// first workgroup of each tensor inside its launch, the tensors.  The host copy
// gives the launches, the device copy is what the kernels read.  (As a kernel
// argument the tensors sat in host memory, and a step of 24 small tensors
// waited 5 us for them.)
struct AdamLaunch {
  int32_t begin, count;               // tensors [begin, begin + count) of the table
  int32_t combo;                      // bit 0: 8-bit states, bit 1: bf16 gradients, then AdamParam
  int32_t groups;                     // groups of kAdamGroup elements per workgroup
  int32_t blocks, pad;
};

struct AdamHeader {
  uint32_t magic;
  int32_t launches, tensors;
  int32_t scales_in_params;           // nonzero: no step takes this table
};

struct AdamLayout {
  size_t launch, first, tensor, bytes;
  explicit AdamLayout(size_t n)
      : launch(align_up(sizeof(AdamHeader), 64)),
        first(align_up(launch + n * sizeof(AdamLaunch), 64)),
        tensor(align_up(first + n * sizeof(int32_t), 64)),
        bytes(align_up(tensor + n * sizeof(AdamTensor), 256)) {}
};

struct AdamArgs {
  const int32_t* first;
  const AdamTensor* t;
  int32_t count, groups;
  uint32_t seed;
  float b1, omb1, b2, omb2, eps, lr, lr_wd;
  float root_b2, root_omb2;           // sqrt(b2), sqrt(1 - b2), both times 2^120
  double log_b1, log_b2;
  const int32_t* step;
  const float* lr_scale;
  const float* grad_scale;
};

// One array of a tensor, in bytes.
struct AdamRange {
  uintptr_t begin, end;
};
static_assert(6 * sizeof(AdamRange) <= sizeof(AdamLaunch) + sizeof(int32_t) + sizeof(AdamTensor),
              "the table's bytes hold six ranges of each tensor while they are compared");

__device__ __forceinline__ uint32_t mix(uint32_t x) {
  x ^= x >> 16;
  x *= 0x7feb352du;
  x ^= x >> 15;
  x *= 0x846ca68bu;
  return x ^ (x >> 16);
}

__device__ __forceinline__ float pow2f(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }
// E8M0 byte -> scale; byte 0 is 2^-127, a denormal.
__device__ __forceinline__ float e8m0(uint8_t b) { return __uint_as_float(b ? static_cast<uint32_t>(b) << 23 : 0x400000u); }

// The square root instruction: off by at most one unit, and it takes a denormal
// for zero, so that a small argument is scaled out of that range (exactly).
__device__ __forceinline__ float root_f32(float v) {
  const bool small = v < 0x1p-100f;
  return __builtin_amdgcn_sqrtf(small ? v * 0x1p64f : v) * (small ? 0x1p-32f : 1.f);
}

// sqrt(b2 r^2 + (1 - b2) g^2) where that is below 2^-60: its square leaves
// fp32's normal range, or fp32.  A nonzero one does not become 0.
__device__ __forceinline__ float small_root(float r, float g, float root_b2, float root_omb2) {
  const float x = r * root_b2, y = g * root_omb2;           // times 2^120: below 2^60
  const float w = x * x + y * y;
  return w > 0.f ? fmaxf(__builtin_amdgcn_sqrtf(w) * 0x1p-120f, 0x1p-149f) : 0.f;
}

template <int N>
__device__ __forceinline__ float row_rotated(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x120 + N, 0xf, 0xf, true));
}

// max over the 16 lanes that share a block of 128 elements (one DPP row)
__device__ __forceinline__ float block_max(float v) {
  v = fmaxf(v, row_rotated<8>(v));
  v = fmaxf(v, row_rotated<4>(v));
  v = fmaxf(v, row_rotated<2>(v));
  return fmaxf(v, row_rotated<1>(v));
}

__device__ __forceinline__ int block_exponent(float top) {
  const uint32_t b = __float_as_uint(top);
  const int e = static_cast<int>(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  return e < -127 ? -127 : e;
}

// Eight values (in units of their block's scale) to E4M3 codes by stochastic
// rounding: floor(value / code step + r / 2^20) with r the upper 20 bits of a
// random word, which is what v_cvt_sr_fp8_f32 computes (compared with that
// definition over 2^24 values, denormal codes among them).
__device__ __forceinline__ uint64_t encode8(const float* y, const uint32_t* r) {
  int lo = 0, hi = 0;
  lo = __builtin_amdgcn_cvt_sr_fp8_f32(y[0], static_cast<int>(r[0]), lo, 0);
  lo = __builtin_amdgcn_cvt_sr_fp8_f32(y[1], static_cast<int>(r[1]), lo, 1);
  lo = __builtin_amdgcn_cvt_sr_fp8_f32(y[2], static_cast<int>(r[2]), lo, 2);
  lo = __builtin_amdgcn_cvt_sr_fp8_f32(y[3], static_cast<int>(r[3]), lo, 3);
  hi = __builtin_amdgcn_cvt_sr_fp8_f32(y[4], static_cast<int>(r[4]), hi, 0);
  hi = __builtin_amdgcn_cvt_sr_fp8_f32(y[5], static_cast<int>(r[5]), hi, 1);
  hi = __builtin_amdgcn_cvt_sr_fp8_f32(y[6], static_cast<int>(r[6]), hi, 2);
  hi = __builtin_amdgcn_cvt_sr_fp8_f32(y[7], static_cast<int>(r[7]), hi, 3);
  return static_cast<uint64_t>(static_cast<uint32_t>(hi)) << 32 | static_cast<uint32_t>(lo);
}

// STREAM: accesses that the caches need not keep.  With 8-bit states (a state
// byte is next used one step later) they took 42 M parameters from 91.7 to
// 86.7 us; with fp32 states the same hint cost 15 %.
template <bool STREAM, typename T>
__device__ __forceinline__ T read_as(const void* p) {
  if constexpr (STREAM) return __builtin_nontemporal_load(static_cast<const T*>(p));
  return *static_cast<const T*>(p);
}

// 8 elements from index i on; those behind n read as zero.  FULL: none is.
template <bool BF16, bool FULL, bool STREAM>
__device__ __forceinline__ void load8(const void* base, int64_t i, int64_t n, float* x) {
  if (FULL || i + 8 <= n) {
    if constexpr (BF16) {
      const u32x4_t v = read_as<STREAM, u32x4_t>(static_cast<const bf16_t*>(base) + i);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[2 * j] = __uint_as_float(v[j] << 16);
        x[2 * j + 1] = __uint_as_float(v[j] & 0xffff0000u);
      }
    } else {
      const float* s = static_cast<const float*>(base) + i;
      const f32x4_t a = read_as<STREAM, f32x4_t>(s), b = read_as<STREAM, f32x4_t>(s + 4);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[j] = a[j];
        x[4 + j] = b[j];
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      x[j] = 0.f;
      if (i + j < n) x[j] = BF16 ? bf16_to_f32(static_cast<const bf16_t*>(base)[i + j]) : static_cast<const float*>(base)[i + j];
    }
  }
}

template <bool FULL>
__device__ __forceinline__ void store8_f32(float* base, int64_t i, int64_t n, const float* x) {
  if (FULL || i + 8 <= n) {
    f32x4_t* d = reinterpret_cast<f32x4_t*>(base + i);
    d[0] = f32x4_t{x[0], x[1], x[2], x[3]};
    d[1] = f32x4_t{x[4], x[5], x[6], x[7]};
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i + j < n) base[i + j] = x[j];
  }
}

template <bool FULL>
__device__ __forceinline__ void store8_bf16(bf16_t* base, int64_t i, int64_t n, const uint32_t* h) {
  if (FULL || i + 8 <= n) {
    *reinterpret_cast<u32x4_t*>(base + i) =
        u32x4_t{h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16};
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i + j < n) base[i + j] = static_cast<bf16_t>(h[j]);
  }
}

template <bool FULL>
__device__ __forceinline__ uint64_t load8_codes(const uint8_t* base, int64_t i, int64_t n) {
  if (FULL || i + 8 <= n) return read_as<true, uint64_t>(base + i);
  uint64_t v = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (i + j < n) v |= static_cast<uint64_t>(base[i + j]) << (8 * j);
  return v;
}

template <bool FULL>
__device__ __forceinline__ void store8_codes(uint8_t* base, int64_t i, int64_t n, uint64_t q) {
  if (FULL || i + 8 <= n) {
    __builtin_nontemporal_store(q, reinterpret_cast<uint64_t*>(base + i));
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i + j < n) base[i + j] = static_cast<uint8_t>(q >> (8 * j));
  }
}

__device__ __forceinline__ void decode8(uint64_t q, float scale, float* x) {
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const int v = static_cast<int>(q >> (32 * w));
    const auto a = __builtin_amdgcn_cvt_pk_f32_fp8(v, false);
    const auto b = __builtin_amdgcn_cvt_pk_f32_fp8(v, true);
    x[4 * w] = a[0] * scale;
    x[4 * w + 1] = a[1] * scale;
    x[4 * w + 2] = b[0] * scale;
    x[4 * w + 3] = b[1] * scale;
  }
}

enum AdamParam { PARAM_F32 = 0, PARAM_BF16 = 1, PARAM_MASTER = 2 };

template <bool EIGHT, int PARAM, bool GRAD_BF16>
__global__ __launch_bounds__(256) void k_adamw(AdamArgs a) {
#pragma clang fp contract(off)
  // this workgroup's tensor: the last whose first workgroup is not behind it
  const int blk = blockIdx.x, lane = threadIdx.x & 63;
  int base = 0, span = a.count;
  if (a.count > 64) {
    span = (a.count + 63) / 64;
    const int at = lane * span < a.count ? a.first[lane * span] : 0x7fffffff;
    base = (__popcll(__ballot(at <= blk)) - 1) * span;
  }
  const int mine = lane < span && base + lane < a.count ? a.first[base + lane] : 0x7fffffff;
  const int q = __builtin_amdgcn_readfirstlane(__popcll(__ballot(mine <= blk)) - 1);
  const int first = __builtin_amdgcn_readlane(mine, q);
  // the table does not change while a step runs: scalar loads, kept across the stores
  typedef const __attribute__((address_space(4))) AdamTensor ConstTensor;
  const ConstTensor& t = ((ConstTensor*)(a.t))[__builtin_amdgcn_readfirstlane(base) + q];
  const int64_t n = t.n;
  const int step = max(*a.step, 1);
  const float gs = a.grad_scale ? *a.grad_scale : 1.f;
  const float ls = a.lr_scale ? *a.lr_scale : 1.f;
  // 1 - beta^t; an error of some 2^-24 in these factors moves p by that part of its update only
  const float step_size = a.lr * ls / -expm1f(static_cast<float>(step * a.log_b1));
  const float rbc2 = 1.f / sqrtf(-expm1f(static_cast<float>(step * a.log_b2)));
  const float decay = fmaf(-a.lr_wd, ls, 1.f);
  const uint32_t key0 = mix(mix(a.seed + 0x9e3779b9u * static_cast<uint32_t>(step)) + t.key);

  const int64_t begin = static_cast<int64_t>(blk - first) * a.groups * kAdamGroup + threadIdx.x * 8;
  auto group = [&](int64_t i, auto full) {
    constexpr bool FULL = decltype(full)::value;
    float g[8], m[8], v[8], p[8], root[8];
    load8<GRAD_BF16, FULL, EIGHT>(t.g, i, n, g);
    if constexpr (EIGHT) {
      const uint64_t qm = load8_codes<FULL>(static_cast<const uint8_t*>(t.m), i, n);
      const uint64_t qv = load8_codes<FULL>(static_cast<const uint8_t*>(t.v), i, n);
      decode8(qm, e8m0(t.ms[i >> 7]), m);
      decode8(qv, e8m0(t.vs[i >> 7]), root);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = root[j] * root[j];
    } else {
      load8<false, FULL, EIGHT>(t.m, i, n, m);
      load8<false, FULL, EIGHT>(t.v, i, n, v);
    }
    auto load_p = [&](int64_t at, float* x) {
      if constexpr (PARAM == PARAM_MASTER)
        load8<false, FULL, EIGHT>(t.master, at, n, x);
      else
        load8<PARAM == PARAM_BF16, FULL, EIGHT>(t.p, at, n, x);
    };
    auto updated = [&](float old, float mj, float rj) {      // (the reciprocal's argument is at least eps, a normal number)
      return old * decay - step_size * (mj * __builtin_amdgcn_rcpf(rj * rbc2 + a.eps));
    };
    auto moment2 = [&](float old, float gj) { return old * a.b2 + (gj * a.omb2) * gj; };
    // EARLY: the update before the branch for small roots, which then repeats its
    // elements' update.  44 M elements, 8-bit states, us: bf16 weights 95 to 98 (late
    // 98 to 101), where they are in fp32, or a master is, 137 and 152 (late 131 and 145).
    constexpr bool EARLY = EIGHT && PARAM == PARAM_BF16;
    load_p(i, p);
    float low = INFINITY;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float gj = g[j] * gs;
      m[j] = m[j] * a.b1 + gj * a.omb1;
      v[j] = moment2(v[j], gj);
      low = fminf(low, v[j]);
      root[j] = EIGHT ? __builtin_amdgcn_sqrtf(v[j]) : root_f32(v[j]);
      if constexpr (EARLY) p[j] = updated(p[j], m[j], root[j]);
    }
    if constexpr (EIGHT) {
      if (low < 0x1p-120f) {
        // Seldom, so a branch; what it needs is read again, which costs the rest
        // less than keeping registers for it.
        float r[8], h[8], old[8];
        int64_t at = i;
        asm volatile("" : "+v"(at));                         // (opaque, or the values above are kept)
        load8<GRAD_BF16, FULL, EIGHT>(t.g, at, n, h);
        decode8(load8_codes<FULL>(static_cast<const uint8_t*>(t.v), at, n), e8m0(t.vs[at >> 7]), r);
        if constexpr (EARLY) load_p(at, old);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float hj = h[j] * gs;
          if (moment2(r[j] * r[j], hj) < 0x1p-120f) {
            root[j] = small_root(r[j], hj, a.root_b2, a.root_omb2);
            if constexpr (EARLY) p[j] = updated(old[j], m[j], root[j]);
          }
        }
      }
    }
    if constexpr (!EARLY) {
#pragma unroll
      for (int j = 0; j < 8; ++j) p[j] = updated(p[j], m[j], root[j]);
    }
    uint32_t one[8], two[8];
    if constexpr (EIGHT || PARAM == PARAM_BF16) {
      const uint32_t key = key0 ^ (static_cast<uint32_t>(i >> 32) * 0x9e3779b9u);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        one[j] = mix(static_cast<uint32_t>(i + j) ^ key);
        two[j] = mix(one[j] + 0x9e3779b9u);
      }
    }
    if constexpr (EIGHT) {
      float tm = 0.f, tv = 0.f;                             // (fmaxf passes over NaN)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        tm = fmaxf(tm, fabsf(m[j]));
        tv = fmaxf(tv, root[j]);
      }
      if (fmaxf(tm, tv) == INFINITY) {
        tm = tv = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (fabsf(m[j]) < INFINITY)
            tm = fmaxf(tm, fabsf(m[j]));
          else
            m[j] = NAN;
          if (root[j] < INFINITY)
            tv = fmaxf(tv, root[j]);
          else
            root[j] = NAN;
        }
      }
      const int em = block_exponent(block_max(tm)), ev = block_exponent(block_max(tv));
      const float im = pow2f(-em), iv = pow2f(-ev);
      float ym[8], yv[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        ym[j] = m[j] * im;
        // a nonzero value below the smallest code (2^-9) becomes that code; NaN, whose
        // bits are above every number's, stays
        yv[j] = root[j] == 0.f ? 0.f : __uint_as_float(max(__float_as_uint(root[j] * iv), 0x3b000000u));
      }
      store8_codes<FULL>(static_cast<uint8_t*>(t.m), i, n, encode8(ym, one));
      store8_codes<FULL>(static_cast<uint8_t*>(t.v), i, n, encode8(yv, two));
      if ((threadIdx.x & 15) == 0) {
        t.ms[i >> 7] = static_cast<uint8_t>(em + 127);
        t.vs[i >> 7] = static_cast<uint8_t>(ev + 127);
      }
    } else {
      store8_f32<FULL>(static_cast<float*>(t.m), i, n, m);
      store8_f32<FULL>(static_cast<float*>(t.v), i, n, v);
    }
    if constexpr (PARAM == PARAM_F32) {
      store8_f32<FULL>(static_cast<float*>(t.p), i, n, p);
    } else {
      uint32_t h[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if constexpr (PARAM == PARAM_BF16) {
          const uint32_t u = __float_as_uint(p[j]);
          const uint32_t r = (one[j] & 0xfffu) << 4 | (two[j] & 0xfu);
          h[j] = (u & 0x7f800000u) == 0x7f800000u ? f32_to_bf16(p[j]) : (u + r) >> 16;
        } else {
          h[j] = f32_to_bf16(p[j]);
        }
      }
      store8_bf16<FULL>(static_cast<bf16_t*>(t.p), i, n, h);
      if constexpr (PARAM == PARAM_MASTER) store8_f32<FULL>(t.master, i, n, p);
    }
  };
  for (int it = 0; it < a.groups; ++it) {
    const int64_t i = begin + it * kAdamGroup;
    if (i - threadIdx.x * 8 + kAdamGroup <= n)                // the whole workgroup's elements exist
      group(i, std::integral_constant<bool, true>{});
    else if (i - (threadIdx.x & 15) * 8 < n)                  // the 16 lanes of a block of 128 meet in block_max
      group(i, std::integral_constant<bool, false>{});
  }
}

template <bool EIGHT, int PARAM>
static void adamw_launch(const AdamArgs& a, bool gbf16, unsigned blocks, hipStream_t s) {
  if (gbf16)
    hipLaunchKernelGGL((k_adamw<EIGHT, PARAM, true>), dim3(blocks), dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((k_adamw<EIGHT, PARAM, false>), dim3(blocks), dim3(256), 0, s, a);
}

}  // namespace dbomoe

using namespace dbomoe;

extern "C" size_t moe_adamw_table_size(int32_t n_tensors) {
  return n_tensors < 1 ? 0 : AdamLayout(n_tensors).bytes;
}

extern "C" moe_status moe_adamw_table_build(const moe_adamw_tensor* tensors, int32_t n_tensors, void* table,
                                            size_t bytes) {
  if (!tensors || !table || n_tensors < 1) return MOE_ERR_INVALID_ARG;
  if (!aligned16(table)) return MOE_ERR_MISALIGNED;
  const AdamLayout l(n_tensors);
  if (bytes < l.bytes) return MOE_ERR_WORKSPACE;
  int64_t total = 0;
  for (int i = 0; i < n_tensors; ++i) {
    const moe_adamw_tensor& t = tensors[i];
    if (t.n < 0) return MOE_ERR_INVALID_ARG;
    if ((t.param_dtype != MOE_F32 && t.param_dtype != MOE_BF16) ||
        (t.grad_dtype != MOE_F32 && t.grad_dtype != MOE_BF16) ||
        (t.state_dtype != MOE_F32 && t.state_dtype != MOE_FP8_E4M3FN) || t.n > (int64_t{1} << 36))
      return MOE_ERR_UNSUPPORTED;
    if (t.master && t.param_dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
    if (t.n == 0) continue;
    const bool eight = t.state_dtype == MOE_FP8_E4M3FN;
    if (!t.param || !t.grad || !t.m || !t.v || (eight != (t.m_scale != nullptr)) || (eight != (t.v_scale != nullptr)))
      return MOE_ERR_INVALID_ARG;
    if (t.param == t.grad || t.m == t.v || t.param == t.master) return MOE_ERR_INVALID_ARG;
    if (!aligned16(t.param) || !aligned16(t.grad) || !aligned16(t.m) || !aligned16(t.v) || !aligned16(t.master))
      return MOE_ERR_MISALIGNED;
    total += (t.n + kAdamGroup - 1) / kAdamGroup;
  }
  // Two workgroups must not update one element, and none what another reads:
  // the updated arrays are sorted, in the table's own bytes, and compared with
  // their neighbours and the gradients.
  auto* ranges = static_cast<AdamRange*>(table);
  size_t nr = 0;
  auto collect = [&](bool params, bool moments, bool scales) {
    nr = 0;
    for (int i = 0; i < n_tensors; ++i) {
      const moe_adamw_tensor& t = tensors[i];
      auto add = [&](const void* p, int64_t bytes) {
        const uintptr_t a = reinterpret_cast<uintptr_t>(p);
        if (p && t.n > 0) ranges[nr++] = AdamRange{a, a + static_cast<uintptr_t>(bytes)};
      };
      const int64_t state = t.state_dtype == MOE_F32 ? 4 : 1;
      if (params) add(t.param, t.n * static_cast<int64_t>(dtype_size(t.param_dtype)));
      if (moments) {
        add(t.m, t.n * state);
        add(t.v, t.n * state);
        add(t.master, t.n * 4);
      }
      if (scales) {
        add(t.m_scale, (t.n + 127) / 128);
        add(t.v_scale, (t.n + 127) / 128);
      }
    }
    std::sort(ranges, ranges + nr, [](const AdamRange& a, const AdamRange& b) { return a.begin < b.begin; });
  };
  auto overlap = [&] {
    for (size_t i = 1; i < nr; ++i)
      if (ranges[i].begin < ranges[i - 1].end) return true;
    return false;
  };
  auto meets_gradient = [&] {
    for (int i = 0; i < n_tensors; ++i) {
      const moe_adamw_tensor& t = tensors[i];
      if (t.n == 0) continue;
      const uintptr_t a = reinterpret_cast<uintptr_t>(t.grad);
      const uintptr_t z = a + static_cast<uintptr_t>(t.n * static_cast<int64_t>(dtype_size(t.grad_dtype)));
      const AdamRange* r = std::upper_bound(ranges, ranges + nr, a, [](uintptr_t v, const AdamRange& x) { return v < x.end; });
      if (r != ranges + nr && r->begin < z) return true;
    }
    return false;
  };
  collect(true, true, false);
  if (overlap() || meets_gradient()) return MOE_ERR_INVALID_ARG;
  collect(false, true, true);
  if (overlap() || meets_gradient()) return MOE_ERR_INVALID_ARG;
  // (A table whose only fault is a scale inside a param is built, and refused by
  // moe_adamw_table_check and by every step: callers rely on that status.)
  collect(true, false, true);
  const bool scales_in_params = overlap();
  auto* out = static_cast<uint8_t*>(table);
  memset(out, 0, l.bytes);
  auto* launch = reinterpret_cast<AdamLaunch*>(out + l.launch);
  auto* first = reinterpret_cast<int32_t*>(out + l.first);
  auto* entry = reinterpret_cast<AdamTensor*>(out + l.tensor);
  // four groups a workgroup where that leaves enough workgroups
  const int groups = total >= 8192 ? 4 : 1;
  const int64_t per = static_cast<int64_t>(groups) * kAdamGroup;
  int launches = 0, at = 0;
  for (int combo = 0; combo < 12; ++combo) {
    AdamLaunch* cur = nullptr;
    for (int i = 0; i < n_tensors; ++i) {
      const moe_adamw_tensor& t = tensors[i];
      const int kind = t.master ? PARAM_MASTER : t.param_dtype == MOE_BF16 ? PARAM_BF16 : PARAM_F32;
      const int mine = (t.state_dtype == MOE_FP8_E4M3FN ? 1 : 0) | (t.grad_dtype == MOE_BF16 ? 2 : 0) | kind << 2;
      if (t.n == 0 || mine != combo) continue;
      const int64_t nb = (t.n + per - 1) / per;
      // a grid holds fewer than 2^32 threads
      if (!cur || cur->count == kAdamTensors || cur->blocks + nb >= (1 << 24)) {
        if (nb >= (1 << 24)) return MOE_ERR_UNSUPPORTED;
        cur = &launch[launches++];
        *cur = AdamLaunch{at, 0, combo, groups, 0, 0};
      }
      first[at] = cur->blocks;
      entry[at] = AdamTensor{t.param, t.grad, t.m, t.v, t.m_scale, t.v_scale, t.master, t.n,
                             0x85ebca77u * static_cast<uint32_t>(i)};
      cur->blocks += static_cast<int32_t>(nb);
      ++cur->count;
      ++at;
    }
  }
  *reinterpret_cast<AdamHeader*>(out) = AdamHeader{kAdamMagic, launches, n_tensors, scales_in_params};
  return MOE_OK;
}

extern "C" moe_status moe_adamw_table_check(const void* table_host) {
  if (!table_host) return MOE_ERR_INVALID_ARG;
  if (!aligned16(table_host)) return MOE_ERR_MISALIGNED;
  const auto* head = static_cast<const AdamHeader*>(table_host);
  return head->magic != kAdamMagic || head->tensors < 1 || head->scales_in_params ? MOE_ERR_INVALID_ARG : MOE_OK;
}

extern "C" moe_status moe_adamw_step(const void* table_host, const void* table_dev, const moe_adamw_params* hp,
                                     const int32_t* step, const float* lr_scale, const float* grad_scale,
                                     void* stream) {
  if (!hp || !table_host || !table_dev || !step) return MOE_ERR_INVALID_ARG;
  if (!(hp->lr >= 0) || !(hp->beta1 >= 0 && hp->beta1 < 1) || !(hp->beta2 >= 0 && hp->beta2 < 1) ||
      !(hp->eps >= 1.2e-38) || !(hp->weight_decay >= 0) || !isfinite(hp->lr) || !isfinite(hp->eps) ||
      !isfinite(hp->weight_decay))
    return MOE_ERR_INVALID_ARG;
  if (!aligned16(table_host) || !aligned256(table_dev) || !aligned16(step) || !aligned16(lr_scale) ||
      !aligned16(grad_scale))
    return MOE_ERR_MISALIGNED;
  const auto* host = static_cast<const uint8_t*>(table_host);
  const auto* head = reinterpret_cast<const AdamHeader*>(host);
  if (moe_adamw_table_check(table_host) != MOE_OK) return MOE_ERR_INVALID_ARG;
  const AdamLayout l(head->tensors);
  const auto* launch = reinterpret_cast<const AdamLaunch*>(host + l.launch);
  const auto* dev = static_cast<const uint8_t*>(table_dev);
  AdamArgs a{};
  a.seed = hp->seed;
  a.b1 = static_cast<float>(hp->beta1);
  a.omb1 = static_cast<float>(1.0 - hp->beta1);
  a.b2 = static_cast<float>(hp->beta2);
  a.omb2 = static_cast<float>(1.0 - hp->beta2);
  a.eps = static_cast<float>(hp->eps);
  a.root_b2 = static_cast<float>(ldexp(sqrt(hp->beta2), 120));
  a.root_omb2 = static_cast<float>(ldexp(sqrt(1.0 - hp->beta2), 120));
  a.lr = static_cast<float>(hp->lr);
  a.lr_wd = static_cast<float>(hp->lr * hp->weight_decay);
  a.log_b1 = log(hp->beta1);
  a.log_b2 = log(hp->beta2);
  a.step = step;
  a.lr_scale = lr_scale;
  a.grad_scale = grad_scale;
  const hipStream_t s = as_stream(stream);
  for (int i = 0; i < head->launches; ++i) {
    const AdamLaunch& c = launch[i];
    a.first = reinterpret_cast<const int32_t*>(dev + l.first) + c.begin;
    a.t = reinterpret_cast<const AdamTensor*>(dev + l.tensor) + c.begin;
    a.count = c.count;
    a.groups = c.groups;
    const bool eight = c.combo & 1, gbf16 = c.combo & 2;
    const unsigned nb = static_cast<unsigned>(c.blocks);
    switch (c.combo >> 2) {
      case PARAM_F32:
        eight ? adamw_launch<true, PARAM_F32>(a, gbf16, nb, s) : adamw_launch<false, PARAM_F32>(a, gbf16, nb, s);
        break;
      case PARAM_BF16:
        eight ? adamw_launch<true, PARAM_BF16>(a, gbf16, nb, s) : adamw_launch<false, PARAM_BF16>(a, gbf16, nb, s);
        break;
      default:
        eight ? adamw_launch<true, PARAM_MASTER>(a, gbf16, nb, s) : adamw_launch<false, PARAM_MASTER>(a, gbf16, nb, s);
    }
    DBOMOE_CHECK_LAUNCH();
  }
  return MOE_OK;
}
