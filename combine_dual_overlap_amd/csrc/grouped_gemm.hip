// Matrix products grouped by expert with ragged row counts, for gfx950: the
// forward product, the input gradient and the weight gradient of an expert's
// linear layer, with SwiGLU (forward and derivative) as optional epilogues.
// Expert e owns rows [offsets[e], offsets[e+1]) of the row operands.
//   NT  C[r, n]    = sum_k A[r, k] B[e, n, k]     A [rows, K], B [E, N, K]
//   NN  C[r, n]    = sum_k A[r, k] B[e, k, n]     A [rows, K], B [E, K, N]
//   TN  C[e, n, k] = sum_r A[r, n] B[r, k]        A [rows, N], B [rows, K]
// Every sum is kept in fp32 and rounded once, to C's type.
#include "gemm_mfma.h"

namespace dbomoe {

enum GgEpi { EPI_STORE = 0, EPI_SWIGLU = 1, EPI_SWIGLU_BWD = 2 };

// Sizes in terms of one output tile: m and n are its two axes, r the reduction.
struct GgParams {
  const void* A;
  const void* B;
  void* C;                 // NT/NN [cap, N]; TN [E, N, K]; SwiGLU: h [cap, N]; its backward: dgu [cap, 2N]
  const void* gu;          // SwiGLU backward: pre-activations [cap, 2N]
  void* gu_out;            // SwiGLU: pre-activations out or NULL
  float* part;             // split reduction: fp32 partial outputs [splits][...], or NULL
  int64_t part_stride;     // elements of one partial output
  const int32_t* offsets;  // [E+1] or NULL (one group of cap rows)
  int E;
  int64_t cap;
  int N, K;
  int n_tiles;             // tiles along the second output axis
  int m_tiles;             // TN: tiles along the first
  int splits;
  int c_f32, accumulate;
};

struct GgTile {
  int e, m_off, nt, split;
  int rows;                // the expert's rows
  int64_t row0;            // its first row
};

static __device__ __attribute__((aligned(16))) uint32_t g_zero16[4];   // source of the zeros behind a reduction's end

// Rows of expert e, kept inside the row operands whatever the offsets hold.
__device__ __forceinline__ void gg_rows(const GgParams& p, int e, int& o, int& n) {
  const int cap = static_cast<int>(p.cap);
  o = 0;
  n = cap;
  if (p.offsets) {
    o = min(max(p.offsets[e], 0), cap);
    n = max(min(p.offsets[e + 1], cap) - o, 0);
  }
}

// This workgroup's tile.  Workgroup b runs on XCD b % 8: each XCD walks a
// contiguous run of tiles, so that tiles sharing operands share its L2.
// NT/NN: every workgroup rebuilds the tile map from the device offsets with
// one wave scan; the host launches the worst-case grid.
template <int KIND, int BM>
__device__ __forceinline__ bool gg_locate(const GgParams& p, int* s_loc, GgTile& t) {
  const int b = blockIdx.x;
  if constexpr (KIND == MOE_GEMM_TN) {
    const int per_e = p.m_tiles * p.n_tiles;
    const int64_t R = static_cast<int64_t>(p.E) * per_e;
    const int64_t per = (R + 7) / 8;
    const int64_t L = (b & 7) * per + (b >> 3);
    if ((b >> 3) >= per || L >= R) return false;
    t.e = static_cast<int>(L / per_e);
    const int l = static_cast<int>(L % per_e);
    t.m_off = (l % p.m_tiles) * BM;
    t.nt = l / p.m_tiles;
    int o, n;
    gg_rows(p, t.e, o, n);
    t.row0 = o;
    t.rows = n;
  } else {
    if (threadIdx.x < kWave) {
      const int lane = threadIdx.x;
      int t4[4], o4[4], n4[4], sum = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int ex = lane * 4 + i;
        o4[i] = n4[i] = 0;
        if (ex < p.E) gg_rows(p, ex, o4[i], n4[i]);
        t4[i] = (n4[i] + BM - 1) / BM;
        sum += t4[i];
      }
      const int incl = wave_incl_scan(sum);
      const int R = __shfl(incl, 63, kWave) * p.n_tiles;
      const int per = (R + 7) / 8;
      const int L = (b & 7) * per + (b >> 3);
      const bool valid = (b >> 3) < per && L < R;
      if (lane == 0) s_loc[0] = valid;
      int acc = incl - sum;
      if (valid && L >= acc * p.n_tiles && L < incl * p.n_tiles) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (L >= acc * p.n_tiles && L < (acc + t4[i]) * p.n_tiles) {
            const int l = L - acc * p.n_tiles;
            s_loc[1] = lane * 4 + i;
            s_loc[2] = l % t4[i];
            s_loc[3] = l / t4[i];
            s_loc[4] = o4[i];
            s_loc[5] = n4[i];
          }
          acc += t4[i];
        }
      }
    }
    __syncthreads();
    if (!s_loc[0]) return false;
    t.e = s_loc[1];
    t.m_off = s_loc[2] * BM;
    t.nt = s_loc[3];
    t.row0 = s_loc[4];
    t.rows = s_loc[5];
    __syncthreads();                // read by all before the scratch is reused
  }
  t.split = blockIdx.y;
  return true;
}

// ---- epilogues: four consecutive output columns of one row ------------------

__device__ __forceinline__ uint64_t pack4(const f32x4_t& v) {
  return static_cast<uint64_t>(cvt_bf16x2(v[0], v[1])) | (static_cast<uint64_t>(cvt_bf16x2(v[2], v[3])) << 32);
}

__device__ __forceinline__ f32x4_t unpack4(uint64_t v) {
  return f32x4_t{bf16_to_f32(static_cast<bf16_t>(v)), bf16_to_f32(static_cast<bf16_t>(v >> 16)),
                 bf16_to_f32(static_cast<bf16_t>(v >> 32)), bf16_to_f32(static_cast<bf16_t>(v >> 48))};
}

template <bool F32>
__device__ __forceinline__ f32x4_t load4(const void* base, int64_t i) {
  if constexpr (F32)
    return *reinterpret_cast<const f32x4_t*>(static_cast<const float*>(base) + i);
  else
    return unpack4(*reinterpret_cast<const uint64_t*>(static_cast<const bf16_t*>(base) + i));
}

template <bool F32>
__device__ __forceinline__ void store4(void* base, int64_t i, const f32x4_t& v) {
  if constexpr (F32)
    *reinterpret_cast<f32x4_t*>(static_cast<float*>(base) + i) = v;
  else
    *reinterpret_cast<uint64_t*>(static_cast<bf16_t*>(base) + i) = pack4(v);
}

__device__ __forceinline__ void store_c(const GgParams& p, int64_t i, f32x4_t v) {
  if (p.part) {
    store4<true>(p.part + static_cast<int64_t>(blockIdx.y) * p.part_stride, i, v);
  } else if (p.c_f32) {
    if (p.accumulate) v += load4<true>(p.C, i);
    store4<true>(p.C, i, v);
  } else {
    if (p.accumulate) v += load4<false>(p.C, i);
    store4<false>(p.C, i, v);
  }
}

template <bool F32>
__device__ __forceinline__ void store_swiglu(const GgParams& p, int64_t row, int col, const f32x4_t& g,
                                             const f32x4_t& u) {
  f32x4_t h;
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = silu_f32(g[i]) * u[i];
  store4<F32>(p.C, row * p.N + col, h);
  if (p.gu_out) {
    store4<F32>(p.gu_out, row * 2 * p.N + col, g);
    store4<F32>(p.gu_out, row * 2 * p.N + p.N + col, u);
  }
}

// d silu(g)/dg = s (1 + g (1 - s)), s the sigmoid of g
template <bool F32>
__device__ __forceinline__ void store_swiglu_bwd(const GgParams& p, int64_t row, int col, const f32x4_t& dh) {
  const int64_t gi = row * 2 * p.N + col;
  const f32x4_t g = load4<F32>(p.gu, gi), u = load4<F32>(p.gu, gi + p.N);
  f32x4_t dg, du;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float s = 1.0f / (1.0f + __expf(-g[i]));
    dg[i] = dh[i] * u[i] * (s * (1.0f + g[i] * (1.0f - s)));
    du[i] = dh[i] * (g[i] * s);
  }
  store4<F32>(p.C, gi, dg);
  store4<F32>(p.C, gi + p.N, du);
}

// ---- bf16 -------------------------------------------------------------------

typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef short s16x8_t __attribute__((ext_vector_type(8)));

// One operand's tile of BT output-axis positions x BK of the reduction, staged
// by LDS DMA.  RCONT: the reduction axis is the contiguous one in memory; LDS
// rows are the output-axis positions, BK elements each, and a fragment is one
// 16-byte read.  Otherwise LDS rows are reduction steps, BT elements each, and
// a fragment is two transposing reads (ds_read_b64_tr_b16: 16 lanes read a
// 4 x 16 block and each gets the four reduction steps of one column).
// Swizzles, so that the addresses of one read spread over the banks: RCONT
// XORs the 16-byte chunk with the row; the other XORs the 32-byte chunk with
// (step & 3) + 4 * (step >> 3 & 1), the eight steps that half a wave reads.
template <bool RCONT, int BT, int BK, int NW>
struct Operand {
  static constexpr int ROWS = RCONT ? BT : BK, COLS = RCONT ? BK : BT;
  static constexpr int CPR = COLS / 8, RPD = 64 / CPR;     // 16-byte chunks per row, rows per DMA
  static constexpr int NQ = ROWS / RPD / NW;               // DMAs per wave and stage
  static constexpr int BYTES = BT * BK * 2;
  static_assert(NQ >= 1 && NQ * NW * RPD == ROWS, "DMA split");
  static_assert(RCONT || COLS >= 128, "transposing reads: 8 chunks of 32 bytes");

  const bf16_t* src[NQ];
  int step[NQ];             // reduction step of this lane's chunk inside the stage
  int64_t advance;          // elements per stage

  // base: element (0, 0) of the tile's matrix; t0: first output-axis position;
  // row(i): matrix row of output-axis position i (RCONT); limit: valid
  // positions on the output axis (positions behind it read a valid one: their
  // outputs are not stored).
  template <typename RowOf>
  __device__ __forceinline__ void init(const bf16_t* base, int64_t ld, int t0, int limit, RowOf row) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int lr = lane / CPR, pos = lane % CPR;
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      const int R = RPD * (wave * NQ + i) + lr;
      if constexpr (RCONT) {
        const int c = pos ^ (R & 7);
        step[i] = c * 8;
        src[i] = base + static_cast<int64_t>(row(R)) * ld + c * 8;
      } else {
        const int key = (R & 3) | ((R >> 3 & 1) << 2);
        int col = t0 + (((pos >> 1) ^ key) << 4) + (pos & 1) * 8;
        col = min(col, limit - 8);
        step[i] = R;
        src[i] = base + static_cast<int64_t>(R) * ld + col;
      }
    }
    advance = RCONT ? BK : static_cast<int64_t>(BK) * ld;
  }

  __device__ __forceinline__ void issue(uint32_t lds, int ks) const {
    const int wave = threadIdx.x >> 6;
    const int64_t off = ks * advance;
#pragma unroll
    for (int i = 0; i < NQ; ++i) lds_dma16(lds + (wave * NQ + i) * 1024, src[i] + off);
  }

  // the stage that holds the reduction's end: `left` of its steps exist
  __device__ __forceinline__ void issue_tail(uint32_t lds, int ks, int left) const {
    const int wave = threadIdx.x >> 6;
    const int64_t off = ks * advance;
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      const void* ptr = step[i] < left ? static_cast<const void*>(src[i] + off) : g_zero16;
      lds_dma16(lds + (wave * NQ + i) * 1024, ptr);
    }
  }

  // the fragment of 16 positions from `pos` on, 32 reduction steps from kk * 32 on
  static __device__ __forceinline__ bf16x8_t frag(const uint8_t* tile, int pos, int kk) {
    const int lane = threadIdx.x & 63;
    const bf16_t* T = reinterpret_cast<const bf16_t*>(tile);
    if constexpr (RCONT) {
      return *reinterpret_cast<const bf16x8_t*>(&T[lds_off_k<BK>(pos + (lane & 15), kk * 4 + (lane >> 4))]);
    } else {
      const int g = lane >> 4, L = lane & 15;
      const int key = (L >> 2) | ((g & 1) << 2);
      const int r = kk * 32 + g * 8 + (L >> 2);
      const bf16_t* a = T + r * COLS + (((pos >> 4) ^ key) << 4) + (L & 3) * 4;
      typedef __attribute__((address_space(3))) s16x4_t* lds4;
      const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(a));
      const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(a + 4 * COLS));
      return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
  }
};

// Tile BM x BN, BK reduction steps per stage, WM x WN waves, a ring of NBUF
// stages (stage s in buffer s % NBUF, issued NBUF - 1 stages ahead).
template <int KIND, int EPI, int BM, int BN, int BK, int WAVES_M, int WAVES_N, int NBUF, int MINW>
__global__ __launch_bounds__(WAVES_M * WAVES_N * 64, MINW) void k_grouped_gemm(GgParams p) {
  constexpr int NW = WAVES_M * WAVES_N;
  constexpr int WM = BM / WAVES_M, WN = BN / WAVES_N, TM = WM / 16, TN = WN / 16;
  using OpA = Operand<KIND != MOE_GEMM_TN, BM, BK, NW>;
  using OpB = Operand<KIND == MOE_GEMM_NT, BN, BK, NW>;
  constexpr int NDMA = OpA::NQ + OpB::NQ, STAGE = OpA::BYTES + OpB::BYTES;
  static_assert((NBUF - 2) * NDMA < 64, "vmcnt");
  __shared__ __attribute__((aligned(16))) uint8_t lds[NBUF * STAGE];

  GgTile t;
  if (!gg_locate<KIND, BM>(p, reinterpret_cast<int*>(lds), t)) return;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WAVES_N, wn = wave % WAVES_N;
  const int nout = KIND == MOE_GEMM_TN ? p.K : p.N;              // positions on the second output axis
  const int red = KIND == MOE_GEMM_TN ? t.rows : p.K;            // reduction length
  const int KT_all = (red + BK - 1) / BK;
  // split reduction: stages [kt0, kt0 + KT)
  const int per_split = (KT_all + p.splits - 1) / p.splits;
  const int kt0 = min(t.split * per_split, KT_all);
  const int KT = min(per_split, KT_all - kt0);

  OpA a;
  OpB b;
  if constexpr (KIND == MOE_GEMM_TN) {
    a.init(static_cast<const bf16_t*>(p.A) + t.row0 * p.N, p.N, t.m_off, p.N, [](int) { return 0; });
    b.init(static_cast<const bf16_t*>(p.B) + t.row0 * p.K, p.K, t.nt * BN, p.K, [](int) { return 0; });
  } else {
    a.init(static_cast<const bf16_t*>(p.A) + t.row0 * p.K, p.K, 0, 0,
           [&](int r) { return min(t.m_off + r, t.rows - 1); });
    const int brows = EPI == EPI_SWIGLU ? 2 * p.N : p.N;
    const bf16_t* B = static_cast<const bf16_t*>(p.B) + static_cast<int64_t>(t.e) * brows * p.K;
    if constexpr (KIND == MOE_GEMM_NN)
      b.init(B, p.N, t.nt * BN, p.N, [](int) { return 0; });
    else if constexpr (EPI == EPI_SWIGLU)       // half a tile of gate rows, then the matching up rows
      b.init(B, p.K, 0, 0, [&](int r) {
        return min(t.nt * (BN / 2) + r % (BN / 2), p.N - 1) + (r < BN / 2 ? 0 : p.N);
      });
    else
      b.init(B, p.K, 0, 0, [&](int r) { return min(t.nt * BN + r, p.N - 1); });
  }
  const uint32_t lds0 = static_cast<uint32_t>(
      reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t*)(lds)));
  __builtin_amdgcn_s_waitcnt(0);           // from here on only counted DMAs are in flight
  auto issue = [&](int kt) {
    const uint32_t at = lds0 + (kt % NBUF) * STAGE;
    const int ks = kt0 + kt, left = red - ks * BK;
    if (left >= BK) {
      a.issue(at, ks);
      b.issue(at + OpA::BYTES, ks);
    } else {
      a.issue_tail(at, ks, left);
      b.issue_tail(at + OpA::BYTES, ks, left);
    }
  };

  // Accumulators hold C transposed (the second operand is the MFMA's first):
  // lane l has row l & 15 and the four columns 4 * (l >> 4) .. + 3 of each
  // 16 x 16 tile, so that it stores whole pieces of a row.
  f32x4_t acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  auto b_pos = [&](int tn) {
    if constexpr (EPI == EPI_SWIGLU)
      return tn < TN / 2 ? wn * (WN / 2) + tn * 16 : BN / 2 + wn * (WN / 2) + (tn - TN / 2) * 16;
    else
      return wn * WN + tn * 16;
  };
  auto compute = [&](int kt) {
    const uint8_t* sA = lds + (kt % NBUF) * STAGE;
    const uint8_t* sB = sA + OpA::BYTES;
#pragma unroll
    for (int kk = 0; kk < BK / 32; ++kk) {
      bf16x8_t af[TM], bfr[TN];
#pragma unroll
      for (int i = 0; i < TM; ++i) af[i] = OpA::frag(sA, wm * WM + i * 16, kk);
#pragma unroll
      for (int j = 0; j < TN; ++j) bfr[j] = OpB::frag(sB, b_pos(j), kk);
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bfr[j], af[i], acc[i][j], 0, 0, 0);
    }
  };

  const int pre = min(NBUF - 1, KT);
  for (int s = 0; s < pre; ++s) issue(s);
  wait_stages<NDMA, NBUF - 2>(pre - 1);
  __syncthreads();
  for (int kt = 0; kt < KT; ++kt) {
    if (kt + NBUF - 1 < KT) issue(kt + NBUF - 1);
    compute(kt);
    wait_stages<NDMA, NBUF - 2>(min(KT - 1, kt + NBUF - 1) - (kt + 1));
    __syncthreads();
  }

  const int m_lim = KIND == MOE_GEMM_TN ? p.N : t.rows;
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int m = t.m_off + wm * WM + i * 16 + (lane & 15);
    if (m >= m_lim) continue;
    if constexpr (EPI == EPI_SWIGLU) {
#pragma unroll
      for (int j = 0; j < TN / 2; ++j) {
        const int col = t.nt * (BN / 2) + wn * (WN / 2) + j * 16 + (lane >> 4) * 4;
        if (col < nout) store_swiglu<false>(p, t.row0 + m, col, acc[i][j], acc[i][j + TN / 2]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        const int col = t.nt * BN + wn * WN + j * 16 + (lane >> 4) * 4;
        if (col >= nout) continue;
        if constexpr (EPI == EPI_SWIGLU_BWD)
          store_swiglu_bwd<false>(p, t.row0 + m, col, acc[i][j]);
        else if constexpr (KIND == MOE_GEMM_TN)
          store_c(p, (static_cast<int64_t>(t.e) * p.N + m) * p.K + col, acc[i][j]);
        else
          store_c(p, (t.row0 + m) * p.N + col, acc[i][j]);
      }
    }
  }
}

// ---- fp32 -------------------------------------------------------------------

// 64 x 64 tiles, 16 reduction steps per stage, 2 x 2 waves of 2 x 2 MFMA tiles
// (v_mfma_f32_16x16x4_f32).  LDS rows are reduction steps, 80 floats apart (16
// banks), so the four steps of a fragment read fall into different banks.
template <int KIND, int EPI>
__global__ __launch_bounds__(256) void k_grouped_gemm_f32(GgParams p) {
  constexpr int BM = 64, BN = 64, BK = 16, LD = 80;
  __shared__ float sA[BK][LD];
  __shared__ float sB[BK][LD];
  __shared__ int s_loc[8];
  GgTile t;
  if (!gg_locate<KIND, BM>(p, s_loc, t)) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave >> 1, wn = wave & 1;
  const int nout = KIND == MOE_GEMM_TN ? p.K : p.N;
  const int red = KIND == MOE_GEMM_TN ? t.rows : p.K;
  const int KT_all = (red + BK - 1) / BK;
  const int per_split = (KT_all + p.splits - 1) / p.splits;
  const int kt0 = min(t.split * per_split, KT_all);
  const int kt1 = min(kt0 + per_split, KT_all);

  // This thread's four consecutive floats of each operand's stage: along the
  // reduction (4 chunks x 64 positions) or along the output axis (16 x 16).
  constexpr bool AR = KIND != MOE_GEMM_TN, BR = KIND == MOE_GEMM_NT;
  const int ra_step = AR ? (tid & 3) * 4 : tid >> 4, ra_pos = AR ? tid >> 2 : (tid & 15) * 4;
  const int rb_step = BR ? (tid & 3) * 4 : tid >> 4, rb_pos = BR ? tid >> 2 : (tid & 15) * 4;
  const float* asrc;
  const float* bsrc;
  int64_t astep, bstep;
  if constexpr (AR) {
    asrc = static_cast<const float*>(p.A) + (t.row0 + min(t.m_off + ra_pos, t.rows - 1)) * p.K + ra_step;
    astep = BK;
  } else {
    asrc = static_cast<const float*>(p.A) + (t.row0 + ra_step) * p.N + min(t.m_off + ra_pos, p.N - 4);
    astep = static_cast<int64_t>(BK) * p.N;
  }
  if constexpr (KIND == MOE_GEMM_TN) {
    bsrc = static_cast<const float*>(p.B) + (t.row0 + rb_step) * p.K + min(t.nt * BN + rb_pos, p.K - 4);
    bstep = static_cast<int64_t>(BK) * p.K;
  } else {
    const int brows = EPI == EPI_SWIGLU ? 2 * p.N : p.N;
    const float* B = static_cast<const float*>(p.B) + static_cast<int64_t>(t.e) * brows * p.K;
    if constexpr (KIND == MOE_GEMM_NN) {
      bsrc = B + static_cast<int64_t>(rb_step) * p.N + min(t.nt * BN + rb_pos, p.N - 4);
      bstep = static_cast<int64_t>(BK) * p.N;
    } else {
      const int r = EPI == EPI_SWIGLU ? min(t.nt * (BN / 2) + rb_pos % (BN / 2), p.N - 1) + (rb_pos < BN / 2 ? 0 : p.N)
                                      : min(t.nt * BN + rb_pos, p.N - 1);
      bsrc = B + static_cast<int64_t>(r) * p.K + rb_step;
      bstep = BK;
    }
  }
  const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
  auto load = [&](int kt, f32x4_t& ra, f32x4_t& rb) {
    const int left = red - kt * BK;            // a multiple of 4 where the reduction is the contiguous axis
    ra = ra_step < left ? *reinterpret_cast<const f32x4_t*>(asrc + kt * astep) : zero;
    rb = rb_step < left ? *reinterpret_cast<const f32x4_t*>(bsrc + kt * bstep) : zero;
  };
  auto put = [&](float (*s)[LD], bool along_r, int step, int pos, const f32x4_t& v) {
    if (along_r) {
#pragma unroll
      for (int i = 0; i < 4; ++i) s[step + i][pos] = v[i];
    } else {
      *reinterpret_cast<f32x4_t*>(&s[step][pos]) = v;
    }
  };
  auto b_pos = [&](int j) { return EPI == EPI_SWIGLU ? j * 32 + wn * 16 : wn * 32 + j * 16; };
  f32x4_t acc[2][2] = {{zero, zero}, {zero, zero}};
  f32x4_t ra = zero, rb = zero;
  if (kt0 < kt1) load(kt0, ra, rb);
  for (int kt = kt0; kt < kt1; ++kt) {
    __syncthreads();
    put(sA, AR, ra_step, ra_pos, ra);
    put(sB, BR, rb_step, rb_pos, rb);
    __syncthreads();
    if (kt + 1 < kt1) load(kt + 1, ra, rb);
#pragma unroll
    for (int k4 = 0; k4 < BK; k4 += 4) {
      float af[2], bfr[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) af[i] = sA[k4 + (lane >> 4)][wm * 32 + i * 16 + (lane & 15)];
#pragma unroll
      for (int j = 0; j < 2; ++j) bfr[j] = sB[k4 + (lane >> 4)][b_pos(j) + (lane & 15)];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(bfr[j], af[i], acc[i][j], 0, 0, 0);
    }
  }

  const int m_lim = KIND == MOE_GEMM_TN ? p.N : t.rows;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int m = t.m_off + wm * 32 + i * 16 + (lane & 15);
    if (m >= m_lim) continue;
    if constexpr (EPI == EPI_SWIGLU) {
      const int col = t.nt * (BN / 2) + wn * 16 + (lane >> 4) * 4;
      if (col < nout) store_swiglu<true>(p, t.row0 + m, col, acc[i][0], acc[i][1]);
    } else {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int col = t.nt * BN + wn * 32 + j * 16 + (lane >> 4) * 4;
        if (col >= nout) continue;
        if constexpr (EPI == EPI_SWIGLU_BWD)
          store_swiglu_bwd<true>(p, t.row0 + m, col, acc[i][j]);
        else if constexpr (KIND == MOE_GEMM_TN)
          store_c(p, (static_cast<int64_t>(t.e) * p.N + m) * p.K + col, acc[i][j]);
        else
          store_c(p, (t.row0 + m) * p.N + col, acc[i][j]);
      }
    }
  }
}

// Sums the partial outputs of a split reduction in split order (so the result
// does not depend on timing) and stores C.  NT/NN: only the rows of experts.
__global__ __launch_bounds__(256) void k_join_splits(GgParams p, int64_t quads, int row_quads) {
  int64_t lo = 0, lim = quads;
  if (row_quads && p.offsets) {
    lo = min(static_cast<int64_t>(max(p.offsets[0], 0)), p.cap) * row_quads;
    lim = min(static_cast<int64_t>(max(p.offsets[p.E], 0)), p.cap) * row_quads;
  }
  const float* part = p.part;
  GgParams q = p;
  q.part = nullptr;
  for (int64_t i = lo + static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < lim;
       i += static_cast<int64_t>(gridDim.x) * 256) {
    f32x4_t v = load4<true>(part, i * 4);
    for (int s = 1; s < p.splits; ++s) v += load4<true>(part + s * p.part_stride, i * 4);
    store_c(q, i * 4, v);
  }
}

// ---- host -------------------------------------------------------------------

// Parts the reduction is cut into: doubled while the grid has fewer than 256
// workgroups and each part keeps at least 256 steps, at most 16.
static int gg_splits(int kind, int E, int64_t cap, int N, int K, int BM, int BN) {
  int64_t tiles, red;
  if (kind == MOE_GEMM_TN) {
    tiles = static_cast<int64_t>(E) * ((N + BM - 1) / BM) * ((K + BN - 1) / BN);
    red = cap / E;
  } else {
    tiles = (cap + BM - 1) / BM * ((N + BN - 1) / BN);
    red = K;
  }
  int S = 1;
  while (S < 16 && tiles * S < 256 && red / (2 * S) >= 256) S *= 2;
  return S;
}

struct GgTileShape { int BM, BN; };
static GgTileShape gg_shape(int kind, bool f32, int64_t cap, int E) {
  if (f32) return {64, 64};
  if (kind == MOE_GEMM_TN) return {128, 128};
  return {cap / E <= 32 ? 32 : 128, 128};
}

template <int KIND, int EPI>
static moe_status gg_launch(GgParams& p, bool f32, hipStream_t s) {
  const GgTileShape ts = gg_shape(KIND, f32, p.cap, p.E);
  const int cols = KIND == MOE_GEMM_TN ? p.K : EPI == EPI_SWIGLU ? 2 * p.N : p.N;
  // a SwiGLU tile holds BN / 2 gate columns and the matching up columns
  p.n_tiles = EPI == EPI_SWIGLU ? (p.N + ts.BN / 2 - 1) / (ts.BN / 2) : (cols + ts.BN - 1) / ts.BN;
  p.m_tiles = (p.N + ts.BM - 1) / ts.BM;
  const int64_t tiles = KIND == MOE_GEMM_TN ? static_cast<int64_t>(p.E) * p.m_tiles * p.n_tiles
                                            : max_row_tiles(p.cap, p.E, ts.BM, p.offsets == nullptr) * p.n_tiles;
  if (gemm_grid(tiles) >= (1 << 24)) return MOE_ERR_UNSUPPORTED;      // 256 threads each, 2^32 in a grid
  const dim3 grid(static_cast<unsigned>(gemm_grid(tiles)), p.splits);
  if (f32) {
    hipLaunchKernelGGL((k_grouped_gemm_f32<KIND, EPI>), grid, dim3(256), 0, s, p);
  } else if (ts.BM == 32) {
    if constexpr (KIND != MOE_GEMM_TN)
      hipLaunchKernelGGL((k_grouped_gemm<KIND, EPI, 32, 128, 64, 1, 4, 3, 2>), grid, dim3(256), 0, s, p);
  } else {
    hipLaunchKernelGGL((k_grouped_gemm<KIND, EPI, 128, 128, 64, 2, 2, 2, 2>), grid, dim3(256), 0, s, p);
  }
  DBOMOE_CHECK_LAUNCH();
  if (p.splits > 1) {
    const int64_t elems = KIND == MOE_GEMM_TN ? static_cast<int64_t>(p.E) * p.N * p.K : p.cap * p.N;
    const int64_t blocks = (elems / 4 + 255) / 256;
    hipLaunchKernelGGL(k_join_splits, dim3(static_cast<unsigned>(blocks < 4096 ? blocks : 4096)), dim3(256), 0, s, p,
                       elems / 4, KIND == MOE_GEMM_TN ? 0 : p.N / 4);
    DBOMOE_CHECK_LAUNCH();
  }
  return MOE_OK;
}

// Checks that every grouped product shares.  E_loc, sizes and types only.
static moe_status gg_check(moe_dtype ab, const int32_t* offsets, int32_t E_loc, int64_t cap_rows, int32_t N, int32_t K) {
  if (E_loc < 1 || E_loc > 256 || cap_rows < 0 || N < 1 || K < 1) return MOE_ERR_INVALID_ARG;
  if (!offsets && E_loc != 1) return MOE_ERR_INVALID_ARG;
  if (ab != MOE_F32 && ab != MOE_BF16) return MOE_ERR_UNSUPPORTED;
  if (cap_rows > (1 << 30) || N > (1 << 24) || K > (1 << 24)) return MOE_ERR_UNSUPPORTED;
  const int q = ab == MOE_F32 ? 4 : 8;        // rows start on 16 bytes
  if (N % q || K % q) return MOE_ERR_MISALIGNED;
  if (offsets && !aligned16(offsets)) return MOE_ERR_MISALIGNED;
  return MOE_OK;
}

static int gg_call_splits(int kind, moe_dtype ab, int32_t E_loc, int64_t cap_rows, int32_t N, int32_t K) {
  const GgTileShape ts = gg_shape(kind, ab == MOE_F32, cap_rows, E_loc);
  return gg_splits(kind, E_loc, cap_rows, N, K, ts.BM, ts.BN);
}

}  // namespace dbomoe

using namespace dbomoe;

extern "C" size_t moe_grouped_gemm_workspace_size(moe_gemm_kind kind, moe_dtype ab, int32_t E_loc, int64_t cap_rows,
                                                  int32_t N, int32_t K) {
  if (kind != MOE_GEMM_NT && kind != MOE_GEMM_NN && kind != MOE_GEMM_TN) return 0;
  if (E_loc < 1 || E_loc > 256 || cap_rows < 1 || N < 1 || K < 1) return 0;
  const int S = gg_call_splits(kind, ab, E_loc, cap_rows, N, K);
  if (S == 1) return 0;
  const size_t out = kind == MOE_GEMM_TN ? static_cast<size_t>(E_loc) * N * K : static_cast<size_t>(cap_rows) * N;
  return align_up(out * 4 * S, 256);
}

extern "C" moe_status moe_grouped_gemm(moe_gemm_kind kind, const void* a, const void* b, moe_dtype ab,
                                       const int32_t* offsets, int32_t E_loc, int64_t cap_rows, int32_t N, int32_t K,
                                       void* c, moe_dtype ct, int32_t accumulate, void* ws, size_t ws_bytes,
                                       void* stream) {
  if (kind != MOE_GEMM_NT && kind != MOE_GEMM_NN && kind != MOE_GEMM_TN) return MOE_ERR_INVALID_ARG;
  const moe_status st = gg_check(ab, offsets, E_loc, cap_rows, N, K);
  if (st != MOE_OK) return st;
  if (accumulate != 0 && accumulate != 1) return MOE_ERR_INVALID_ARG;
  if (ct != MOE_F32 && !(ct == MOE_BF16 && ab == MOE_BF16)) return MOE_ERR_UNSUPPORTED;
  const bool tn = kind == MOE_GEMM_TN;
  if (cap_rows == 0 && !tn) return MOE_OK;
  if (!c || (!b && !(tn && cap_rows == 0)) || (!a && cap_rows > 0)) return MOE_ERR_INVALID_ARG;
  if (c == a || c == b) return MOE_ERR_INVALID_ARG;
  if (!aligned16(a) || !aligned16(b) || !aligned16(c)) return MOE_ERR_MISALIGNED;
  GgParams p{};
  p.A = a;
  p.B = b;
  p.C = c;
  p.offsets = offsets;
  p.E = E_loc;
  p.cap = cap_rows;
  p.N = N;
  p.K = K;
  p.c_f32 = ct == MOE_F32;
  p.accumulate = accumulate;
  p.splits = gg_call_splits(kind, ab, E_loc, cap_rows, N, K);
  if (p.splits > 1) {
    if (!ws) return MOE_ERR_INVALID_ARG;
    if (!aligned256(ws)) return MOE_ERR_MISALIGNED;
    if (ws_bytes < moe_grouped_gemm_workspace_size(kind, ab, E_loc, cap_rows, N, K)) return MOE_ERR_WORKSPACE;
    p.part = static_cast<float*>(ws);
    p.part_stride = tn ? static_cast<int64_t>(E_loc) * N * K : cap_rows * N;
  }
  const bool f32 = ab == MOE_F32;
  const hipStream_t s = as_stream(stream);
  if (kind == MOE_GEMM_NT) return gg_launch<MOE_GEMM_NT, EPI_STORE>(p, f32, s);
  if (kind == MOE_GEMM_NN) return gg_launch<MOE_GEMM_NN, EPI_STORE>(p, f32, s);
  return gg_launch<MOE_GEMM_TN, EPI_STORE>(p, f32, s);
}

extern "C" moe_status moe_grouped_swiglu(const void* x_perm, const void* w13, moe_dtype act, const int32_t* offsets,
                                         int32_t E_loc, int64_t cap_rows, int32_t H, int32_t I, void* gu, void* h,
                                         void* stream) {
  const moe_status st = gg_check(act, offsets, E_loc, cap_rows, I, H);
  if (st != MOE_OK) return st;
  if (cap_rows == 0) return MOE_OK;
  if (!x_perm || !w13 || !h) return MOE_ERR_INVALID_ARG;
  if (h == x_perm || h == w13 || h == gu || (gu && (gu == x_perm || gu == w13))) return MOE_ERR_INVALID_ARG;
  if (!aligned16(x_perm) || !aligned16(w13) || !aligned16(h) || (gu && !aligned16(gu))) return MOE_ERR_MISALIGNED;
  GgParams p{};
  p.A = x_perm;
  p.B = w13;
  p.C = h;
  p.gu_out = gu;
  p.offsets = offsets;
  p.E = E_loc;
  p.cap = cap_rows;
  p.N = I;
  p.K = H;
  p.splits = 1;
  return gg_launch<MOE_GEMM_NT, EPI_SWIGLU>(p, act == MOE_F32, as_stream(stream));
}

extern "C" moe_status moe_grouped_swiglu_backward(const void* dy_perm, const void* w2, const void* gu, moe_dtype act,
                                                  const int32_t* offsets, int32_t E_loc, int64_t cap_rows, int32_t H,
                                                  int32_t I, void* dgu, void* stream) {
  const moe_status st = gg_check(act, offsets, E_loc, cap_rows, I, H);
  if (st != MOE_OK) return st;
  if (cap_rows == 0) return MOE_OK;
  if (!dy_perm || !w2 || !gu || !dgu) return MOE_ERR_INVALID_ARG;
  if (dgu == dy_perm || dgu == w2) return MOE_ERR_INVALID_ARG;
  if (!aligned16(dy_perm) || !aligned16(w2) || !aligned16(gu) || !aligned16(dgu)) return MOE_ERR_MISALIGNED;
  GgParams p{};
  p.A = dy_perm;
  p.B = w2;
  p.C = dgu;
  p.gu = gu;
  p.offsets = offsets;
  p.E = E_loc;
  p.cap = cap_rows;
  p.N = I;
  p.K = H;
  p.splits = 1;
  return gg_launch<MOE_GEMM_NN, EPI_SWIGLU_BWD>(p, act == MOE_F32, as_stream(stream));
}
