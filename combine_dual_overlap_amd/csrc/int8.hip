// Products of 8-bit integers grouped by expert, with a scale for each token (row
// of a) and each output channel (row of b), and the quantisation that feeds them,
// for gfx950.
//   C[r, n] = (sum_k A[r, k] B[e, n, k]) * as[r] * bs[e, n]     sums in int32: exact
// An LDS stage, a fragment and an MFMA (v_mfma_i32_16x16x64_i8) are those of the
// bf16 product with two integers in the place of one bf16: twice the operations
// for the same bytes.
#include "grouped_tile.h"
#include "rows.h"

namespace dbomoe {

typedef int i32x4_t __attribute__((ext_vector_type(4)));

// ---- rows to 8-bit integers ---------------------------------------------------
// scale = amax * fp32(1 / 127), rounded to fp32, code = the integer nearest to x / scale,
// ties to even: x / scale is found by a multiplication and put right by the exact
// remainder x - code * scale (one fma), so that codes depend on the values alone.
// A row that holds an infinity or NaN gets the scale NaN and codes 0: everything
// computed from it is NaN.
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
  __device__ __forceinline__ int code(float x) const {
    x = inv > 0.f ? x * up : 0.f;
    float t = rintf(x * inv);
    const float d = fmaf(-t, s, x);              // exact: a multiple of the last bit, no larger than about half
    const bool odd = static_cast<int>(t) & 1;
    if (fabsf(d) > half || (fabsf(d) == half && odd)) t += copysignf(1.0f, d);
    return static_cast<int>(fminf(fmaxf(t, -127.0f), 127.0f));   // past 127 only where the scale is subnormal
  }
};

template <bool BF16>
__device__ __forceinline__ void put_codes(int8_t* q, int c, const u32x4_t& v, const RowQuant& rq) {
  float f[Chunk<BF16>::N];
  Chunk<BF16>::unpack(v, f);
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < Chunk<BF16>::N; ++i) w[i / 4] |= static_cast<uint32_t>(rq.code(f[i]) & 0xff) << (8 * (i & 3));
  if constexpr (BF16)
    *reinterpret_cast<uint2*>(q + static_cast<int64_t>(c) * 8) = make_uint2(w[0], w[1]);
  else
    *reinterpret_cast<uint32_t*>(q + static_cast<int64_t>(c) * 4) = w[0];
}

template <bool BF16>
__device__ __forceinline__ uint32_t chunk_max_bits(const u32x4_t& v) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BF16) {
      m = max(m, (v[i] << 16) & 0x7fffffffu);
      m = max(m, v[i] & 0x7fff0000u);
    } else {
      m = max(m, v[i] & 0x7fffffffu);
    }
  }
  return m;
}

// W waves per row, CH chunks per lane held in registers (CH 0: rows of any
// length, read twice).  inv: row t's codes go to the rows inv[t k + j] >= 0; else
// to row t.  last: only rows from [0] up to [E] of these offsets hold anything.
template <bool BF16, int W, int CH>
__global__ __launch_bounds__(RowShape<W>::THREADS) void k_quant_int8(const u32x4_t* __restrict__ x, int64_t T, int rc,
                                                                     int k, const int32_t* __restrict__ inv,
                                                                     const int32_t* __restrict__ offsets, int E,
                                                                     int8_t* __restrict__ q, float* __restrict__ scale) {
  constexpr int ROWS = RowShape<W>::ROWS;
  __shared__ uint32_t s_max[W];
  const int lane = threadIdx.x & 63;
  const int l = W == 1 ? lane : threadIdx.x;
  const int64_t row_bytes = static_cast<int64_t>(rc) * Chunk<BF16>::N;
  int64_t lo = 0, hi = T;
  if (offsets) {
    lo = max(offsets[0], 0);
    hi = min(static_cast<int64_t>(offsets[E]), T);
  }
  const int64_t first = lo + static_cast<int64_t>(blockIdx.x) * ROWS + (W == 1 ? threadIdx.x >> 6 : 0);
  for (int64_t t = first; t < hi; t += static_cast<int64_t>(gridDim.x) * ROWS) {
    const int my_pos = inv && lane < k ? inv[t * k + lane] : -1;
    if (inv && __ballot(my_pos >= 0) == 0) continue;          // (the same in every wave of the row)
    const u32x4_t* src = x + t * rc;
    u32x4_t v[CH > 0 ? CH : 1];
    uint32_t m = 0;
    if constexpr (CH > 0) {
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int c = i * 64 * W + l;
        v[i] = c < rc ? src[c] : u32x4_t{0, 0, 0, 0};
      }
#pragma unroll
      for (int i = 0; i < CH; ++i) m = max(m, chunk_max_bits<BF16>(v[i]));
    } else {
      for (int c = l; c < rc; c += 64 * W) m = max(m, chunk_max_bits<BF16>(src[c]));
    }
    const RowQuant rq(row_max_bits<W>(m, s_max));
    const int n = inv ? k : 1;
    for (int j = 0; j < n; ++j) {
      const int64_t pos = inv ? static_cast<int64_t>(__shfl(my_pos, j, kWave)) : t;
      if (pos < 0) continue;
      int8_t* dst = q + pos * row_bytes;
      if constexpr (CH > 0) {
#pragma unroll
        for (int i = 0; i < CH; ++i) {
          const int c = i * 64 * W + l;
          if (c < rc) put_codes<BF16>(dst, c, v[i], rq);
        }
      } else {
        for (int c = l; c < rc; c += 64 * W) put_codes<BF16>(dst, c, src[c], rq);
      }
      if (l == 0) scale[pos] = rq.scale;
    }
    if constexpr (W > 1) __syncthreads();                     // s_max read by all before the next row's
  }
}

moe_status launch_quant_int8(const QuantInt8Args& a, hipStream_t s) {
  if (a.T == 0) return MOE_OK;
  const int rc = static_cast<int>(static_cast<int64_t>(a.K) * dtype_size(a.act) / 16);
  auto go = [&](auto kernel, int rows, int threads) {
    int64_t blocks = std::min<int64_t>((a.T + rows - 1) / rows, 1 << 20);
    if (a.max_blocks > 0 && blocks > a.max_blocks) blocks = a.max_blocks;
    hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(blocks)), dim3(threads), 0, s, static_cast<const u32x4_t*>(a.x),
                       a.T, rc, a.k, a.inv, a.offsets, a.E, a.q, a.scale);
  };
  auto pick = [&](auto bf16) {
    constexpr bool BF16 = decltype(bf16)::value;
    if (rc > kRowMaxChunks) {
      go(k_quant_int8<BF16, 16, 0>, 1, 1024);
      return;
    }
    with_row_shape(a.T, rc, [&](auto w, auto ch) {
      constexpr int W = decltype(w)::value;
      go(k_quant_int8<BF16, W, decltype(ch)::value>, RowShape<W>::ROWS, RowShape<W>::THREADS);
    });
  };
  if (a.act == MOE_BF16)
    pick(std::true_type{});
  else
    pick(std::false_type{});
  DBOMOE_CHECK_LAUNCH();
  return MOE_OK;
}

// ---- grouped products ---------------------------------------------------------

struct I8Params {
  GgParams g;          // K in pairs of integers
  const float* as;     // [cap]
  const float* bs;     // [E, N] (SwiGLU: [E, 2N])
};

// C = product (c_f32, or bf16), or with SwiGLU h = silu(gate) * up.  The tile of
// the bf16 product (grouped_gemm.hip) for one reduction part: BM x BN, BK pairs
// per stage, WAVES_M x WAVES_N (x WAVES_K halves of a stage) waves, a ring of
// NBUF stages.
template <int EPI, int BM, int BN, int BK, int WAVES_M, int WAVES_N, int WAVES_K, int NBUF, int TM>
__device__ __forceinline__ void i8_tile(const I8Params& ip, const GgTile& t, uint8_t* lds) {
  const GgParams& p = ip.g;
  constexpr int NW = WAVES_M * WAVES_N * WAVES_K;
  constexpr int WM = TM * 16, WN = BN / WAVES_N, TN = WN / 16;
  using OpA = Operand<true, BM, BK, NW, TM * 16 * WAVES_M>;
  using OpB = Operand<true, BN, BK, NW>;
  constexpr int NDMA = OpA::NQ + OpB::NQ, STAGE = OpA::BYTES + OpB::BYTES;
  static_assert((NBUF - 1) * NDMA < 64, "vmcnt");
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wk = wave / (WAVES_M * WAVES_N), wm = wave / WAVES_N % WAVES_M, wn = wave % WAVES_N;
  const int KT = (p.K + BK - 1) / BK;

  OpA a;
  OpB b;
  a.init(static_cast<const bf16_t*>(p.A) + (t.row0 + t.m_off) * p.K, p.K, 0, 0,
         [&](int r) { return min(r, t.rows - 1 - t.m_off); });
  const int brows = EPI == EPI_SWIGLU ? 2 * p.N : p.N;
  const bf16_t* B = static_cast<const bf16_t*>(p.B) + static_cast<int64_t>(t.e) * brows * p.K;
  if constexpr (EPI == EPI_SWIGLU)       // half a tile of gate rows, then the matching up rows
    b.init(B + static_cast<int64_t>(t.nt * (BN / 2)) * p.K, p.K, 0, 0, [&](int r) {
      return min(r % (BN / 2), p.N - 1 - t.nt * (BN / 2)) + (r < BN / 2 ? 0 : p.N);
    });
  else
    b.init(B + static_cast<int64_t>(t.nt * BN) * p.K, p.K, 0, 0, [&](int r) { return min(r, p.N - 1 - t.nt * BN); });
  const uint32_t lds0 = static_cast<uint32_t>(
      reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t*)(lds)));
  __builtin_amdgcn_s_waitcnt(0);           // from here on only counted DMAs are in flight
  auto issue = [&](int kt) {
    const uint32_t at = lds0 + (kt % NBUF) * STAGE;
    const int left = p.K - kt * BK;
    if (left >= BK) {
      a.issue(at, kt);
      b.issue(at + OpA::BYTES, kt);
    } else {
      a.issue_tail(at, kt, left);
      b.issue_tail(at + OpA::BYTES, kt, left);
    }
  };

  // Accumulators hold C transposed: lane l has row l & 15 and the four columns
  // 4 * (l >> 4) .. + 3 of each 16 x 16 tile.
  i32x4_t acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = i32x4_t{0, 0, 0, 0};
  auto b_pos = [&](int tn) {
    if constexpr (EPI == EPI_SWIGLU)
      return tn < TN / 2 ? wn * (WN / 2) + tn * 16 : BN / 2 + wn * (WN / 2) + (tn - TN / 2) * 16;
    else
      return wn * WN + tn * 16;
  };
  constexpr int KK = BK / 32 / WAVES_K;              // steps of a stage that this wave takes
  static_assert(KK % 2 == 0, "the second operand's sets in turn");
  i32x4_t af[TM], bfr[2][TN];
  auto at_a = [&](int kt) { return lds + (kt % NBUF) * STAGE; };
  auto read_a = [&](int kt, int kk, int i) {
    af[i] = __builtin_bit_cast(i32x4_t, OpA::frag(at_a(kt), wm * WM + i * 16, wk * KK + kk));
  };
  auto read_b = [&](int kt, int kk, int set) {
#pragma unroll
    for (int j = 0; j < TN; ++j)
      bfr[set][j] = __builtin_bit_cast(i32x4_t, OpB::frag(at_a(kt) + OpA::BYTES, b_pos(j), wk * KK + kk));
  };
  auto mfmas = [&](int i, int set) {
#pragma unroll
    for (int j = 0; j < TN; ++j)
      acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(bfr[set][j], af[i], acc[i][j], 0, 0, 0);
    __builtin_amdgcn_sched_barrier(0);
  };
  // (The last stage reads a stage that does not exist: bytes of the ring that
  // nothing uses.)
  auto stage = [&](int kt) {
#pragma unroll
    for (int kk = 0; kk < KK; ++kk) {
      const int set = kk & 1;
      if (kk + 1 < KK) {
        read_b(kt, kk + 1, set ^ 1);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < TM; ++i) {
          mfmas(i, set);
          read_a(kt, kk + 1, i);
        }
      } else {
#pragma unroll
        for (int i = 0; i < TM / 2; ++i) mfmas(i, set);
        // this wave's reads of the stage are done, and its DMAs of the next
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        wait_stages<NDMA, NBUF - 2>(min(KT - 1, kt + NBUF - 1) - (kt + 1));
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        if (kt + NBUF < KT) issue(kt + NBUF);
        read_b(kt + 1, 0, set ^ 1);
#pragma unroll
        for (int i = 0; i < TM / 2; ++i) read_a(kt + 1, 0, i);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = TM / 2; i < TM; ++i) {
          mfmas(i, set);
          read_a(kt + 1, 0, i);
        }
      }
    }
  };
  {
    const int pre = min(NBUF, KT);
    for (int s = 0; s < pre; ++s) issue(s);
    wait_stages<NDMA, NBUF - 1>(pre - 1);
    __syncthreads();
    read_b(0, 0, 0);
#pragma unroll
    for (int i = 0; i < TM; ++i) read_a(0, 0, i);
#pragma unroll 1
    for (int kt = 0; kt < KT; ++kt) stage(kt);
  }

  // Epilogue: the wave turns 16 rows at a time through LDS so that each lane has
  // eight columns of a row; the sums become fp32 there (a rounding of 2^-24) and
  // take the row's scale, then the channel's.
  constexpr int CH = WN / 4;                         // 16-byte chunks of a row
  constexpr int OUT = EPI == EPI_SWIGLU ? WN / 16 : WN / 8;   // lanes per row
  constexpr int HN = (16 * OUT + 63) / 64;           // passes of the wave over 16 rows
  const int q = lane % OUT;
  const int col = EPI == EPI_SWIGLU ? t.nt * (BN / 2) + wn * (WN / 2) + q * 8 : t.nt * BN + wn * WN + q * 8;
  const bool col_ok = col < p.N;
  f32x4_t s0{0.f, 0.f, 0.f, 0.f}, s1 = s0, u0 = s0, u1 = s0;
  if (col_ok) {
    const f32x4_t* bs = reinterpret_cast<const f32x4_t*>(ip.bs + static_cast<int64_t>(t.e) * brows + col);
    s0 = bs[0];
    s1 = bs[1];
    if constexpr (EPI == EPI_SWIGLU) {
      const f32x4_t* us = reinterpret_cast<const f32x4_t*>(ip.bs + static_cast<int64_t>(t.e) * brows + p.N + col);
      u0 = us[0];
      u1 = us[1];
    }
  }
  __syncthreads();                                   // the ring is free
  constexpr int JOIN = WAVES_K == 1 ? 0 : NW * TM * TN * 1024;
  static_assert(JOIN + NW * 16 * WN * 4 <= NBUF * STAGE, "epilogue scratch");
  auto mine = [&](int i) { return WAVES_K == 1 || (i & 1) == wk; };
  if constexpr (WAVES_K == 2) {
    i32x4_t* slot = reinterpret_cast<i32x4_t*>(lds);
#pragma unroll
    for (int i = 0; i < TM; ++i)
      if (!mine(i))
#pragma unroll
        for (int j = 0; j < TN; ++j) slot[((wave * TM + i) * TN + j) * 64 + lane] = acc[i][j];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < TM; ++i)
      if (mine(i))
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] += slot[(((wave ^ (NW / 2)) * TM + i) * TN + j) * 64 + lane];
  }
  float* turn = reinterpret_cast<float*>(lds + JOIN) + wave * 16 * WN;
  auto chunk = [&](int r, int c) { return reinterpret_cast<f32x4_t*>(turn + r * WN + ((c ^ (r & (CH - 1))) << 2)); };
  auto store8_f32 = [&](int64_t at, const f32x4_t& v0, const f32x4_t& v1) {
    f32x4_t* c = reinterpret_cast<f32x4_t*>(static_cast<float*>(p.C) + at);
    c[0] = v0;
    c[1] = v1;
  };
  auto store8_bf16 = [&](int64_t at, const f32x4_t& v0, const f32x4_t& v1) {
    *reinterpret_cast<u32x4_t*>(static_cast<bf16_t*>(p.C) + at) =
        u32x4_t{cvt_bf16x2(v0[0], v0[1]), cvt_bf16x2(v0[2], v0[3]), cvt_bf16x2(v1[0], v1[1]), cvt_bf16x2(v1[2], v1[3])};
  };
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    if (!mine(i)) continue;
#pragma unroll
    for (int j = 0; j < TN; ++j) *chunk(lane & 15, j * 4 + (lane >> 4)) = __builtin_convertvector(acc[i][j], f32x4_t);
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
    for (int h = 0; h < HN; ++h) {
      const int r = (h * 64 + lane) / OUT, in = wm * WM + i * 16 + r;
      if (r >= 16 || in >= t.m_n || !col_ok) continue;
      const int64_t row = t.row0 + t.m_off + in;
      const float as = ip.as[row];
      f32x4_t v0 = *chunk(r, 2 * q) * as * s0, v1 = *chunk(r, 2 * q + 1) * as * s1;
      if constexpr (EPI == EPI_SWIGLU) {
        const f32x4_t w0 = *chunk(r, CH / 2 + 2 * q) * as * u0, w1 = *chunk(r, CH / 2 + 2 * q + 1) * as * u1;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          v0[x] = silu_f32(v0[x]) * w0[x];
          v1[x] = silu_f32(v1[x]) * w1[x];
        }
      }
      const int64_t at = row * p.N + col;
      if (p.c_f32)
        store8_f32(at, v0, v1);
      else
        store8_bf16(at, v0, v1);
    }
    __builtin_amdgcn_wave_barrier();
  }
}

template <int EPI, int BM, int BN, int BK, int WAVES_M, int WAVES_N, int WAVES_K, int NBUF, int TM>
__device__ __forceinline__ void i8_tile_of(int tm, const I8Params& p, const GgTile& t, uint8_t* lds) {
  if constexpr (TM == 1) {
    i8_tile<EPI, BM, BN, BK, WAVES_M, WAVES_N, WAVES_K, NBUF, 1>(p, t, lds);
  } else {
    if (tm == TM)
      i8_tile<EPI, BM, BN, BK, WAVES_M, WAVES_N, WAVES_K, NBUF, TM>(p, t, lds);
    else
      i8_tile_of<EPI, BM, BN, BK, WAVES_M, WAVES_N, WAVES_K, NBUF, TM - 1>(tm, p, t, lds);
  }
}

template <int EPI, int BM, int BN, int BK, int WAVES_M, int WAVES_N, int WAVES_K, int NBUF>
__global__ __launch_bounds__(WAVES_M * WAVES_N * WAVES_K * 64, 2) void k_grouped_int8(I8Params p) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[NBUF * (BM + BN) * BK * 2];
  GgTile t;
  if (!gg_locate<MOE_GEMM_NT, BM>(p.g, reinterpret_cast<int*>(lds), t)) return;
  i8_tile_of<EPI, BM, BN, BK, WAVES_M, WAVES_N, WAVES_K, NBUF, BM / WAVES_M / 16>(
      (t.m_n + 16 * WAVES_M - 1) / (16 * WAVES_M), p, t, lds);
}

// ---- host -----------------------------------------------------------------------

template <int EPI>
static moe_status launch_int8(I8Params& p, hipStream_t s) {
  const int64_t cap = p.g.cap, rows = cap / p.g.E;
  const bool dense = !p.g.offsets;
  auto tiles = [&](int BM, int BN) {
    const int64_t width = EPI == EPI_SWIGLU ? BN / 2 : BN;
    return max_row_tiles(cap, p.g.E, BM, dense) * ((p.g.N + width - 1) / width);
  };
  int BM = 128, BN = 128;
  if (rows <= 32)
    BM = 32;
  else if (rows > 128 && tiles(256, 256) >= 256)
    BM = BN = 256;
  else if (tiles(64, 128) <= 128)
    BM = 64;
  const int width = EPI == EPI_SWIGLU ? BN / 2 : BN;
  p.g.n_tiles = (p.g.N + width - 1) / width;
  p.g.splits = 1;
  const int64_t n = gemm_grid(tiles(BM, BN));
  if (n >= (1 << 23)) return MOE_ERR_UNSUPPORTED;      // at most 512 threads each, 2^32 in a grid
  const dim3 grid(static_cast<unsigned>(n));
  if (BM == 256)
    hipLaunchKernelGGL((k_grouped_int8<EPI, 256, 256, 64, 2, 4, 1, 2>), grid, dim3(512), 0, s, p);
  else if (BM == 128)
    hipLaunchKernelGGL((k_grouped_int8<EPI, 128, 128, 64, 2, 2, 1, 2>), grid, dim3(256), 0, s, p);
  else if (BM == 64)
    hipLaunchKernelGGL((k_grouped_int8<EPI, 64, 128, 128, 2, 2, 2, 3>), grid, dim3(512), 0, s, p);
  else
    hipLaunchKernelGGL((k_grouped_int8<EPI, 32, 128, 64, 1, 4, 1, 3>), grid, dim3(256), 0, s, p);
  DBOMOE_CHECK_LAUNCH();
  return MOE_OK;
}

// What every product checks: sizes, then pointers.
static moe_status int8_check_sizes(bool dense, int32_t E_loc, int64_t cap, int32_t N, int32_t K) {
  if (E_loc < 1 || E_loc > 256 || cap < 0 || N < 1 || K < 1) return MOE_ERR_INVALID_ARG;
  if (dense && E_loc != 1) return MOE_ERR_INVALID_ARG;
  // 127^2 K stays below 2^31
  if (cap > (1 << 30) || N > (1 << 22) || K > (1 << 17)) return MOE_ERR_UNSUPPORTED;
  return N % 8 || K % 16 ? MOE_ERR_MISALIGNED : MOE_OK;
}

static moe_status int8_check(const int32_t* offsets, int32_t E_loc, int64_t cap, int32_t N, int32_t K) {
  const moe_status st = int8_check_sizes(!offsets, E_loc, cap, N, K);
  return st == MOE_OK && offsets && !aligned16(offsets) ? MOE_ERR_MISALIGNED : st;
}

static I8Params int8_params(const int8_t* a, const float* as, const int8_t* b, const float* bs, const int32_t* offsets,
                            int32_t E_loc, int64_t cap, int32_t N, int32_t K, void* c, bool f32) {
  I8Params p{};
  p.g.A = a;
  p.g.B = b;
  p.g.C = c;
  p.g.offsets = offsets;
  p.g.E = E_loc;
  p.g.cap = cap;
  p.g.N = N;
  p.g.K = K / 2;
  p.g.c_f32 = f32;
  p.as = as;
  p.bs = bs;
  return p;
}

struct FfnInt8Ws {
  size_t codes, scale, bytes;      // after h [cap, I] fp32
};

static FfnInt8Ws ffn_int8_ws(int64_t cap, int32_t I) {
  FfnInt8Ws w;
  w.codes = align_up(static_cast<size_t>(cap) * I * 4, 256);
  w.scale = w.codes + align_up(static_cast<size_t>(cap) * I, 256);
  w.bytes = w.scale + align_up(static_cast<size_t>(cap) * 4, 256);
  return w;
}

size_t ffn_int8_ws_bytes(int64_t cap, int32_t I) { return ffn_int8_ws(cap, I).bytes; }

moe_status check_ffn_int8_shapes(bool dense, int32_t E_loc, int64_t cap, int32_t H, int32_t I) {
  moe_status st = int8_check_sizes(dense, E_loc, cap, I, H);
  if (st == MOE_OK) st = int8_check_sizes(dense, E_loc, cap, H, I);
  if (st != MOE_OK) return st;
  // the up rows are addressed by 32-bit byte offsets from the gate rows
  return (static_cast<int64_t>(I) + 256) * H >= (int64_t{1} << 32) ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

// h stays in fp32 until it is quantised: in bf16 its own rounding would move
// every eighth code or so.
moe_status launch_ffn_int8(const FfnInt8Args& a, hipStream_t s) {
  if (a.cap_rows == 0) return MOE_OK;
  const FfnInt8Ws w = ffn_int8_ws(a.cap_rows, a.I);
  char* ws = static_cast<char*>(a.ws);
  int8_t* hq = reinterpret_cast<int8_t*>(ws + w.codes);
  float* hs = reinterpret_cast<float*>(ws + w.scale);
  if (a.t0 && hipEventRecord(a.t0, s) != hipSuccess) return MOE_ERR_HIP;
  I8Params p = int8_params(a.xq, a.xs, a.w13, a.s13, a.offsets, a.E_loc, a.cap_rows, a.I, a.H, ws, true);
  moe_status st = launch_int8<EPI_SWIGLU>(p, s);
  if (st != MOE_OK) return st;
  QuantInt8Args qa{};
  qa.x = ws;
  qa.act = MOE_F32;
  qa.T = a.cap_rows;
  qa.K = a.I;
  qa.offsets = a.offsets;
  qa.E = a.E_loc;
  qa.q = hq;
  qa.scale = hs;
  st = launch_quant_int8(qa, s);
  if (st != MOE_OK) return st;
  if (a.t1 && hipEventRecord(a.t1, s) != hipSuccess) return MOE_ERR_HIP;
  p = int8_params(hq, hs, a.w2, a.s2, a.offsets, a.E_loc, a.cap_rows, a.H, a.I, a.y, false);
  st = launch_int8<EPI_STORE>(p, s);
  if (st != MOE_OK) return st;
  if (a.t2 && hipEventRecord(a.t2, s) != hipSuccess) return MOE_ERR_HIP;
  return MOE_OK;
}

}  // namespace dbomoe

using namespace dbomoe;

extern "C" moe_status moe_quant_int8_rows(const void* x, moe_dtype act, int64_t n, int32_t K, int8_t* q, float* scale,
                                          void* stream) {
  if (n < 0 || K <= 0) return MOE_ERR_INVALID_ARG;
  if (act != MOE_F32 && act != MOE_BF16) return MOE_ERR_UNSUPPORTED;
  if (K % 16) return MOE_ERR_MISALIGNED;
  if (n == 0) return MOE_OK;
  if (!x || !q || !scale) return MOE_ERR_INVALID_ARG;
  if (x == q || x == scale || static_cast<void*>(q) == scale) return MOE_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(q) || !aligned16(scale)) return MOE_ERR_MISALIGNED;
  QuantInt8Args a{};
  a.x = x;
  a.act = act;
  a.T = n;
  a.K = K;
  a.q = q;
  a.scale = scale;
  return launch_quant_int8(a, as_stream(stream));
}

extern "C" moe_status moe_grouped_gemm_int8(const int8_t* a, const float* a_scale, const int8_t* b, const float* b_scale,
                                            const int32_t* offsets, int32_t E_loc, int64_t cap_rows, int32_t N,
                                            int32_t K, void* c, moe_dtype ct, void* stream) {
  const moe_status st = int8_check(offsets, E_loc, cap_rows, N, K);
  if (st != MOE_OK) return st;
  if (ct != MOE_F32 && ct != MOE_BF16) return MOE_ERR_UNSUPPORTED;
  if (cap_rows == 0) return MOE_OK;
  if (!a || !a_scale || !b || !b_scale || !c) return MOE_ERR_INVALID_ARG;
  if (c == a || c == b || c == a_scale || c == b_scale) return MOE_ERR_INVALID_ARG;
  if (!aligned16(a) || !aligned16(a_scale) || !aligned16(b) || !aligned16(b_scale) || !aligned16(c))
    return MOE_ERR_MISALIGNED;
  I8Params p = int8_params(a, a_scale, b, b_scale, offsets, E_loc, cap_rows, N, K, c, ct == MOE_F32);
  return launch_int8<EPI_STORE>(p, as_stream(stream));
}

extern "C" moe_status moe_grouped_swiglu_int8(const int8_t* xq, const float* xq_scale, const int8_t* w13,
                                              const float* w13_scale, const int32_t* offsets, int32_t E_loc,
                                              int64_t cap_rows, int32_t H, int32_t I, void* h, moe_dtype ht,
                                              void* stream) {
  const moe_status st = int8_check(offsets, E_loc, cap_rows, I, H);
  if (st != MOE_OK) return st;
  if (ht != MOE_F32 && ht != MOE_BF16) return MOE_ERR_UNSUPPORTED;
  if ((static_cast<int64_t>(I) + 256) * H >= (int64_t{1} << 32)) return MOE_ERR_UNSUPPORTED;
  if (cap_rows == 0) return MOE_OK;
  if (!xq || !xq_scale || !w13 || !w13_scale || !h) return MOE_ERR_INVALID_ARG;
  if (h == xq || h == w13 || h == xq_scale || h == w13_scale) return MOE_ERR_INVALID_ARG;
  if (!aligned16(xq) || !aligned16(xq_scale) || !aligned16(w13) || !aligned16(w13_scale) || !aligned16(h))
    return MOE_ERR_MISALIGNED;
  I8Params p = int8_params(xq, xq_scale, w13, w13_scale, offsets, E_loc, cap_rows, I, H, h, ht == MOE_F32);
  return launch_int8<EPI_SWIGLU>(p, as_stream(stream));
}

extern "C" size_t moe_ffn_int8_workspace_size(int64_t cap_rows, int32_t I) {
  if (cap_rows <= 0 || I <= 0) return 0;
  return ffn_int8_ws_bytes(cap_rows, I);
}

extern "C" moe_status moe_grouped_ffn_int8(const int8_t* xq, const float* xq_scale, int32_t H, int32_t I,
                                           const int32_t* offsets, int32_t E_loc, int64_t cap_rows, const int8_t* w13,
                                           const int8_t* w2, const float* w13_scale, const float* w2_scale, void* y,
                                           void* ws, size_t ws_bytes, void* stream) {
  const moe_status st = check_ffn_int8_shapes(!offsets, E_loc, cap_rows, H, I);
  if (st != MOE_OK) return st;
  if (offsets && !aligned16(offsets)) return MOE_ERR_MISALIGNED;
  if (cap_rows == 0) return MOE_OK;
  if (!xq || !xq_scale || !w13 || !w13_scale || !w2 || !w2_scale || !y || !ws) return MOE_ERR_INVALID_ARG;
  if (y == xq || y == xq_scale || y == w13 || y == w2 || y == w13_scale || y == w2_scale || y == ws)
    return MOE_ERR_INVALID_ARG;
  if (!aligned16(xq) || !aligned16(xq_scale) || !aligned16(w13) || !aligned16(w13_scale) || !aligned16(w2) ||
      !aligned16(w2_scale) || !aligned16(y) || !aligned256(ws))
    return MOE_ERR_MISALIGNED;
  if (ws_bytes < ffn_int8_ws_bytes(cap_rows, I)) return MOE_ERR_WORKSPACE;
  FfnInt8Args a{xq, xq_scale, H, I, offsets, E_loc, cap_rows, w13, w2, w13_scale, w2_scale, y, ws};
  return launch_ffn_int8(a, as_stream(stream));
}
