// Matrix products grouped by expert with ragged row counts, for gfx950: the
// forward product, the input gradient and the weight gradient of an expert's
// linear layer, with SwiGLU (forward and derivative) as optional epilogues.
// Expert e owns rows [offsets[e], offsets[e+1]) of the row operands.
//   NT  C[r, n]    = sum_k A[r, k] B[e, n, k]     A [rows, K], B [E, N, K]
//   NN  C[r, n]    = sum_k A[r, k] B[e, k, n]     A [rows, K], B [E, K, N]
//   TN  C[e, n, k] = sum_r A[r, n] B[r, k]        A [rows, N], B [rows, K]
// Every sum is kept in fp32 and rounded once, to C's type.
//
// What bounds them (MI355X, bf16, 256 x 256 tiles): a dense product of 8192^3 runs
// at 1.33 to 1.39 PFLOP/s (the library's 1.50).  A stage of 64 reduction steps
// takes 3040 clocks at 2.07 GHz, 2048 of them the matrix pipes'; without its loads
// into LDS 2420, so that traffic from L2 (64 KB a stage and compute unit, 11 TB/s in
// all) costs the most.  LDS reads cost 4 % and show no bank conflicts.  Rings of
// smaller stages, loads spread between the MFMAs, other barrier positions,
// staggered starts and persistent workgroups gain nothing.  A grouped product also
// reads its weights cold from HBM: 36006 Zipf-distributed rows x 2048 x 1408 of 64
// experts take 246 us (0.84 PFLOP/s, 686 MB read, 147 MB written).
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
  int m_n;                 // positions of the tile on the first axis
  int rows;                // the expert's rows
  int64_t row0;            // its first row
};

static __device__ __attribute__((aligned(16))) uint32_t g_zero16[4];   // source of the zeros behind a reduction's end

// The lane number, opaque to the compiler: what is computed from it inside a
// loop stays there instead of occupying registers around the main loop.
__device__ __forceinline__ int fresh_lane() {
  int lane = threadIdx.x & 63;
  asm volatile("" : "+v"(lane));
  return lane;
}

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
    // Every expert's tiles are spread over the XCDs, the experts of most rows
    // first (in classes of a factor of two), so that no XCD is left with a
    // large expert at the end: with Zipf-distributed rows (largest expert 29 %
    // of them) a contiguous run of experts per XCD took 3.5 times as long.
    const int per_e = p.m_tiles * p.n_tiles, per_x = (per_e + 7) / 8;
    int k = (b >> 3) / per_x;                         // the expert's place in that order
    if (k >= p.E) return false;
    const int l = ((b + k) & 7) * per_x + (b >> 3) % per_x;
    if (l >= per_e) return false;
    const int lane = threadIdx.x & 63;
    int cls[4], o4[4], n4[4], top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o4[i] = n4[i] = 0;
      if (lane * 4 + i < p.E) gg_rows(p, lane * 4 + i, o4[i], n4[i]);
      cls[i] = lane * 4 + i >= p.E ? -1 : n4[i] == 0 ? 0 : 32 - __clz((n4[i] + 31) / 32);
      top = max(top, cls[i]);
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) top = max(top, __shfl_xor(top, d, kWave));
    int e = 0;
    for (int c = __builtin_amdgcn_readfirstlane(top); c >= 0; --c) {
      bool found = false;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint64_t has = __ballot(cls[i] == c);
        const int count = __popcll(has);
        if (!found && k < count) {
          const bool mine = cls[i] == c && __popcll(has & lanemask_lt()) == k;
          const int src = __builtin_amdgcn_readfirstlane(__ffsll(static_cast<unsigned long long>(__ballot(mine))) - 1);
          e = src * 4 + i;
          t.row0 = __builtin_amdgcn_readlane(o4[i], src);
          t.rows = __builtin_amdgcn_readlane(n4[i], src);
          found = true;
        }
        if (!found) k -= count;
      }
      if (found) break;
    }
    t.e = e;
    // bands of four tiles along the first axis: an XCD's share is compact
    const int band = l / (4 * p.n_tiles), r = l - band * 4 * p.n_tiles;
    const int high = min(4, p.m_tiles - 4 * band);
    t.m_off = (4 * band + r % high) * BM;
    t.m_n = min(BM, p.N - t.m_off);
    t.nt = r / high;
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
            // bands of eight row tiles: what runs together on an XCD is about
            // as high as wide
            const int band = l / (8 * p.n_tiles), r = l - band * 8 * p.n_tiles;
            const int high = min(8, t4[i] - 8 * band);
            // the expert's rows in tiles of equal height (a multiple of 32
            // where tiles are higher than that)
            const int height = BM <= 32 ? BM : ((n4[i] + t4[i] - 1) / t4[i] + 31) / 32 * 32;
            s_loc[2] = (8 * band + r % high) * height;
            s_loc[3] = r / high;
            s_loc[6] = min(height, n4[i] - s_loc[2]);
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
    t.m_off = s_loc[2];
    t.m_n = s_loc[6];
    t.nt = s_loc[3];
    t.row0 = s_loc[4];
    t.rows = s_loc[5];
    __syncthreads();                // read by all before the scratch is reused
  }
  t.e = __builtin_amdgcn_readfirstlane(t.e);
  t.m_off = __builtin_amdgcn_readfirstlane(t.m_off);
  t.m_n = __builtin_amdgcn_readfirstlane(t.m_n);
  t.nt = __builtin_amdgcn_readfirstlane(t.nt);
  t.rows = __builtin_amdgcn_readfirstlane(t.rows);
  t.row0 = __builtin_amdgcn_readfirstlane(static_cast<int>(t.row0));
  t.split = blockIdx.y;
  return true;
}

// TN that adds to C leaves an expert without rows as it is: nothing is read or
// written (a whole workgroup returns; k_join_splits skips the expert too).  64
// experts, 8 of them with 64 rows, 2816 x 2048 fp32: 537 -> 146 us.  In the bf16
// kernel it stands before the epilogue: at the start it cost 1 % where nobody is idle.
template <int KIND>
__device__ __forceinline__ bool gg_idle(const GgParams& p, const GgTile& t) {
  return KIND == MOE_GEMM_TN && p.accumulate && t.rows == 0;
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
__device__ __forceinline__ void swiglu_bwd(const f32x4_t& dh, const f32x4_t& g, const f32x4_t& u, f32x4_t& dg,
                                           f32x4_t& du) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float s = 1.0f / (1.0f + __expf(-g[i]));
    dg[i] = dh[i] * u[i] * (s * (1.0f + g[i] * (1.0f - s)));
    du[i] = dh[i] * (g[i] * s);
  }
}

template <bool F32>
__device__ __forceinline__ void store_swiglu_bwd(const GgParams& p, int64_t row, int col, const f32x4_t& dh) {
  const int64_t gi = row * 2 * p.N + col;
  const f32x4_t g = load4<F32>(p.gu, gi), u = load4<F32>(p.gu, gi + p.N);
  f32x4_t dg, du;
  swiglu_bwd(dh, g, u, dg, du);
  store4<F32>(p.C, gi, dg);
  store4<F32>(p.C, gi + p.N, du);
}

// Eight columns of a row.  STREAM (weight gradients, which the optimizer reads
// much later, and the SwiGLU backward's dgu): a store that the caches need not
// keep; the skewed layer's gate/up gradient 557 -> 528 us, dgu of 32768 rows 2 to
// 4 %.  (The same for gate/up outputs cost 2 %.)
template <bool STREAM, typename T>
__device__ __forceinline__ void write_as(void* p, const T& v) {
  if constexpr (STREAM)
    __builtin_nontemporal_store(v, static_cast<T*>(p));
  else
    *static_cast<T*>(p) = v;
}

// Likewise for what an epilogue reads once: gu, and the bf16 C that TN adds to
// (64 rows an expert 475 -> 443 us; fp32 C gained nothing).
template <bool STREAM>
__device__ __forceinline__ u32x4_t read_as(const u32x4_t* p) {
  if constexpr (STREAM) return __builtin_nontemporal_load(p);
  return *p;
}

template <bool STREAM = false>
__device__ __forceinline__ void store8(void* base, int64_t i, const f32x4_t& a, const f32x4_t& b) {
  write_as<STREAM>(static_cast<bf16_t*>(base) + i, u32x4_t{cvt_bf16x2(a[0], a[1]), cvt_bf16x2(a[2], a[3]),
                                                           cvt_bf16x2(b[0], b[1]), cvt_bf16x2(b[2], b[3])});
}

__device__ __forceinline__ void unpack8(const u32x4_t& v, f32x4_t& a, f32x4_t& b) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    a[2 * k] = __uint_as_float(v[k] << 16);
    a[2 * k + 1] = __uint_as_float(v[k] & 0xffff0000u);
    b[2 * k] = __uint_as_float(v[2 + k] << 16);
    b[2 * k + 1] = __uint_as_float(v[2 + k] & 0xffff0000u);
  }
}

__device__ __forceinline__ void store_swiglu8(const GgParams& p, int64_t row, int col, const f32x4_t& g0,
                                              const f32x4_t& g1, const f32x4_t& u0, const f32x4_t& u1) {
  f32x4_t a, b;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    a[i] = silu_f32(g0[i]) * u0[i];
    b[i] = silu_f32(g1[i]) * u1[i];
  }
  store8(p.C, row * p.N + col, a, b);
  if (p.gu_out) {
    store8(p.gu_out, row * 2 * p.N + col, g0, g1);
    store8(p.gu_out, row * 2 * p.N + p.N + col, u0, u1);
  }
}

__device__ __forceinline__ void store_swiglu_bwd8(const GgParams& p, int64_t row, int col, const f32x4_t& d0,
                                                  const f32x4_t& d1, const u32x4_t& gate, const u32x4_t& up) {
  const int64_t gi = row * 2 * p.N + col;
  f32x4_t g[2], u[2], dg[2], du[2];
  unpack8(gate, g[0], g[1]);
  unpack8(up, u[0], u[1]);
#pragma unroll
  for (int k = 0; k < 2; ++k) swiglu_bwd(k ? d1 : d0, g[k], u[k], dg[k], du[k]);
  store8<true>(p.C, gi, dg[0], dg[1]);
  store8<true>(p.C, gi + p.N, du[0], du[1]);
}

// ---- bf16 -------------------------------------------------------------------

typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef short s16x8_t __attribute__((ext_vector_type(8)));

// LDS DMA from a uniform base plus a 32-bit byte offset per lane (see lds_dma16).
__device__ __forceinline__ void lds_dma16_at(uint32_t lds_addr, const void* base, uint32_t off) {
  const uint32_t a = __builtin_amdgcn_readfirstlane(lds_addr);
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(a), "v"(off), "s"(base)
               : "memory");
}

__device__ __forceinline__ int64_t uniform64(int64_t v) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v >> 32));
  return static_cast<int64_t>(static_cast<uint64_t>(hi) << 32 | lo);
}

// One operand's tile of BT output-axis positions x BK of the reduction, staged
// by LDS DMA.  RCONT: the reduction axis is the contiguous one in memory; LDS
// rows are the output-axis positions, BK elements each, and a fragment is one
// 16-byte read.  Otherwise LDS rows are reduction steps, BT elements each, and
// a fragment is two transposing reads (ds_read_b64_tr_b16: 16 lanes read a
// 4 x 16 block and each gets the four reduction steps of one column).
// Swizzles, so that the addresses of one read spread over the banks: RCONT
// XORs the 16-byte chunk with the row; the other XORs the 32-byte chunk with
// (step & 3) + 4 * (step >> 3 & 1), the eight steps that half a wave reads
// (64 positions: two steps share a 256-byte row of banks, see key32).
// USED: positions that hold anything (RCONT only: the others are not loaded).
template <bool RCONT, int BT, int BK, int NW, int USED = BT>
struct Operand {
  static constexpr int ROWS = RCONT ? USED : BK, COLS = RCONT ? BK : BT;
  static constexpr int CPR = COLS / 8, RPD = 64 / CPR;     // 16-byte chunks per row, rows per DMA
  static constexpr int NQ = (ROWS + RPD * NW - 1) / (RPD * NW);   // DMAs per wave and stage
  static constexpr int BYTES = BT * BK * 2;
  static_assert(NQ * NW * RPD <= (RCONT ? BT : BK), "DMA split");
  static_assert(RCONT || COLS >= 64, "transposing reads: at least 4 chunks of 32 bytes");

  // the XOR that row r (a reduction step) puts on its 32-byte chunks
  static __device__ __forceinline__ int key32(int r) {
    return COLS == 64 ? (r >> 1 & 1) | ((r >> 3 & 1) << 1) : (r & 3) | ((r >> 3 & 1) << 2);
  }
  // RCONT: the XOR that row r puts on its 16-byte chunks
  static __device__ __forceinline__ int swz(int r) { return r & (BK == 128 ? 15 : 7); }

  const bf16_t* base;       // uniform
  uint32_t off[NQ];         // this lane's chunks: byte offsets from the stage's base
  int64_t advance;          // elements per stage

  // base: element (0, 0) of the tile's matrix; t0: first output-axis position;
  // row(i): matrix row of output-axis position i (RCONT); limit: valid
  // positions on the output axis (positions behind it read a valid one: their
  // outputs are not stored).
  template <typename RowOf>
  __device__ __forceinline__ void init(const bf16_t* first, int64_t ld, int t0, int limit, RowOf row) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int lr = lane / CPR, pos = lane % CPR;
    base = first;
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      const int R = RPD * (i * NW + wave) + lr;
      if constexpr (RCONT) {
        off[i] = (static_cast<uint32_t>(row(R)) * static_cast<uint32_t>(ld) + (pos ^ swz(R)) * 8) * 2;
      } else {
        int col = t0 + (((pos >> 1) ^ key32(R)) << 4) + (pos & 1) * 8;
        col = min(col, limit - 8);
        off[i] = (static_cast<uint32_t>(R) * static_cast<uint32_t>(ld) + col) * 2;
      }
    }
    advance = RCONT ? BK : static_cast<int64_t>(BK) * ld;
  }

  __device__ __forceinline__ void issue(uint32_t lds, int ks) const {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const bf16_t* at = base + ks * advance;
#pragma unroll
    for (int i = 0; i < NQ; ++i) lds_dma16_at(lds + (i * NW + wave) * 1024, at, off[i]);
  }

  // the stage that holds the reduction's end: `left` of its steps exist, the rest are zeros
  __device__ __forceinline__ void issue_tail(uint32_t lds, int ks, int left) const {
    const int lane = fresh_lane();
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint8_t* at = reinterpret_cast<const uint8_t*>(base + ks * advance);
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      const int R = RPD * (i * NW + wave) + lane / CPR;
      const int step = RCONT ? ((lane % CPR) ^ swz(R)) * 8 : R;
      lds_dma16(lds + (i * NW + wave) * 1024, step < left ? static_cast<const void*>(at + off[i]) : g_zero16);
    }
  }

  // the fragment of 16 positions from `pos` on, 32 reduction steps from kk * 32 on
  static __device__ __forceinline__ bf16x8_t frag(const uint8_t* tile, int pos, int kk) {
    const int lane = threadIdx.x & 63;
    const bf16_t* T = reinterpret_cast<const bf16_t*>(tile);
    if constexpr (RCONT) {
      const int r = pos + (lane & 15);
      return *reinterpret_cast<const bf16x8_t*>(&T[r * BK + (((kk * 4 + (lane >> 4)) ^ swz(r)) << 3)]);
    } else {
      const int g = lane >> 4, L = lane & 15;
      const int r = kk * 32 + g * 8 + (L >> 2);
      // (the step four further on has the same key; the key does not depend on kk)
      const bf16_t* a = T + r * COLS + (((pos >> 4) ^ key32(g * 8 + (L >> 2))) << 4) + (L & 3) * 4;
      typedef __attribute__((address_space(3))) s16x4_t* lds4;
      const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(a));
      const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(a + 4 * COLS));
      return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
  }
};

// Tile BM x BN, BK reduction steps per stage, WAVES_M x WAVES_N waves, a ring
// of NBUF stages (stage s in buffer s % NBUF).  TM: 16-position subtiles of
// the first axis per wave that hold anything.  WAVES_K = 2: twice the waves;
// each half takes half of every stage's steps, and the halves' sums are joined
// through LDS (subtile i by half i & 1).
template <int KIND, int EPI, int BM, int BN, int BK, int WAVES_M, int WAVES_N, int WAVES_K, int NBUF, int TM>
__device__ __forceinline__ void gg_tile(const GgParams& p, const GgTile& t, uint8_t* lds) {
  constexpr int NW = WAVES_M * WAVES_N * WAVES_K;
  constexpr int WM = TM * 16, WN = BN / WAVES_N, TN = WN / 16;
  using OpA = Operand<KIND != MOE_GEMM_TN, BM, BK, NW, TM * 16 * WAVES_M>;
  using OpB = Operand<KIND == MOE_GEMM_NT, BN, BK, NW>;
  constexpr int NDMA = OpA::NQ + OpB::NQ, STAGE = OpA::BYTES + OpB::BYTES;
  static_assert((NBUF - 1) * NDMA < 64, "vmcnt");
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wk = wave / (WAVES_M * WAVES_N), wm = wave / WAVES_N % WAVES_M, wn = wave % WAVES_N;
  const int nout = KIND == MOE_GEMM_TN ? p.K : p.N;              // positions on the second output axis
  const int red = KIND == MOE_GEMM_TN ? t.rows : p.K;            // reduction length
  const int KT_all = (red + BK - 1) / BK;
  // split reduction: stages [kt0, kt0 + KT)
  const int per_split = (KT_all + p.splits - 1) / p.splits;
  const int kt0 = min(t.split * per_split, KT_all);
  const int end = min(red, (kt0 + per_split) * BK);              // reduction steps behind it are zeros
  const int KT = min(per_split, KT_all - kt0);

  OpA a;
  OpB b;
  if constexpr (KIND == MOE_GEMM_TN) {
    a.init(static_cast<const bf16_t*>(p.A) + t.row0 * p.N, p.N, t.m_off, p.N, [](int) { return 0; });
    b.init(static_cast<const bf16_t*>(p.B) + t.row0 * p.K, p.K, t.nt * BN, p.K, [](int) { return 0; });
  } else {
    a.init(static_cast<const bf16_t*>(p.A) + (t.row0 + t.m_off) * p.K, p.K, 0, 0,
           [&](int r) { return min(r, t.rows - 1 - t.m_off); });
    const int brows = EPI == EPI_SWIGLU ? 2 * p.N : p.N;
    const bf16_t* B = static_cast<const bf16_t*>(p.B) + static_cast<int64_t>(t.e) * brows * p.K;
    if constexpr (KIND == MOE_GEMM_NN)
      b.init(B, p.N, t.nt * BN, p.N, [](int) { return 0; });
    else if constexpr (EPI == EPI_SWIGLU)       // half a tile of gate rows, then the matching up rows
      b.init(B + static_cast<int64_t>(t.nt * (BN / 2)) * p.K, p.K, 0, 0, [&](int r) {
        return min(r % (BN / 2), p.N - 1 - t.nt * (BN / 2)) + (r < BN / 2 ? 0 : p.N);
      });
    else
      b.init(B + static_cast<int64_t>(t.nt * BN) * p.K, p.K, 0, 0, [&](int r) { return min(r, p.N - 1 - t.nt * BN); });
  }
  const uint32_t lds0 = static_cast<uint32_t>(
      reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t*)(lds)));
  __builtin_amdgcn_s_waitcnt(0);           // from here on only counted DMAs are in flight
  auto issue = [&](int kt) {
    const uint32_t at = lds0 + (kt % NBUF) * STAGE;
    const int ks = kt0 + kt, left = end - ks * BK;
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
  // The reduction advances in steps of 32.  The first operand's fragment of
  // subtile i is read again, for the next step, as soon as this step's MFMAs
  // have taken it, and the second operand's fragments of the next step are
  // read ahead into a second set: LDS reads are spread between the MFMAs and
  // 192 registers hold a 128 x 64 wave tile.  In a stage's last step half of
  // the MFMAs run before the barrier that hands the stage's buffer back.
  constexpr int KK = BK / 32 / WAVES_K;              // steps of a stage that this wave takes
  static_assert(KK % 2 == 0, "the second operand's sets in turn");
  bf16x8_t af[TM], bfr[2][TN];
  auto at_a = [&](int kt) { return lds + (kt % NBUF) * STAGE; };
  auto read_a = [&](int kt, int kk, int i) { af[i] = OpA::frag(at_a(kt), wm * WM + i * 16, wk * KK + kk); };
  auto read_b = [&](int kt, int kk, int set) {
#pragma unroll
    for (int j = 0; j < TN; ++j) bfr[set][j] = OpB::frag(at_a(kt) + OpA::BYTES, b_pos(j), wk * KK + kk);
  };
  auto mfmas = [&](int i, int set) {
#pragma unroll
    for (int j = 0; j < TN; ++j)
      acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bfr[set][j], af[i], acc[i][j], 0, 0, 0);
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
  if (KT > 0) {
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

  // Epilogue.  An accumulator lane holds four columns of one of 16 rows, 32
  // bytes of a bf16 row; the wave turns 16 rows at a time through LDS (16-byte
  // chunks XORed with the row) so that each lane has eight columns and eight
  // neighbouring lanes fill a 128-byte line.  What the epilogue reads (gu, or
  // C to add to) is loaded four groups of rows ahead.
  constexpr int CH = WN / 4;                         // 16-byte chunks of a row
  constexpr int OUT = EPI == EPI_SWIGLU ? WN / 16 : WN / 8;   // lanes per row
  constexpr int HN = (16 * OUT + 63) / 64;           // passes of the wave over 16 rows
  constexpr int AHEAD = TM < 4 ? TM : 4;
  const bool reads = EPI == EPI_SWIGLU_BWD || (EPI == EPI_STORE && p.accumulate && !p.part);
  if (gg_idle<KIND>(p, t)) return;
  u32x4_t old[AHEAD][HN][2];
  struct At { int in, q; int64_t row; int col; bool ok; };
  auto at = [&](int i, int h) {
    At x;
    const int r = (h * 64 + lane) / OUT;
    x.q = lane % OUT;
    x.in = r;
    const int in = wm * WM + i * 16 + r;
    x.row = KIND == MOE_GEMM_TN ? static_cast<int64_t>(t.e) * p.N + t.m_off + in : t.row0 + t.m_off + in;
    x.col = EPI == EPI_SWIGLU ? t.nt * (BN / 2) + wn * (WN / 2) + x.q * 8 : t.nt * BN + wn * WN + x.q * 8;
    x.ok = r < 16 && in < t.m_n && x.col < nout;
    return x;
  };
  auto read_old = [&](int i) {
#pragma unroll
    for (int h = 0; h < HN; ++h) {
      const At x = at(i, h);
      if (!x.ok) continue;
      if constexpr (EPI == EPI_SWIGLU_BWD) {
        const bf16_t* g = static_cast<const bf16_t*>(p.gu) + x.row * 2 * p.N + x.col;
        old[i % AHEAD][h][0] = read_as<true>(reinterpret_cast<const u32x4_t*>(g));
        old[i % AHEAD][h][1] = read_as<true>(reinterpret_cast<const u32x4_t*>(g + p.N));
      } else if (p.c_f32) {
        const u32x4_t* c = reinterpret_cast<const u32x4_t*>(static_cast<const float*>(p.C) + x.row * nout + x.col);
        old[i % AHEAD][h][0] = c[0];
        old[i % AHEAD][h][1] = c[1];
      } else {
        old[i % AHEAD][h][0] = read_as<KIND == MOE_GEMM_TN>(
            reinterpret_cast<const u32x4_t*>(static_cast<const bf16_t*>(p.C) + x.row * nout + x.col));
      }
    }
  };
  auto mine = [&](int i) { return WAVES_K == 1 || (i & 1) == wk; };
  if (reads) {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
      if (mine(i)) read_old(i);
  }
  __syncthreads();                                   // the ring is free
  constexpr int JOIN = WAVES_K == 1 ? 0 : NW * TM * TN * 1024;
  static_assert(JOIN + NW * 16 * WN * 4 <= NBUF * STAGE, "epilogue scratch");
  if constexpr (WAVES_K == 2) {
    f32x4_t* slot = reinterpret_cast<f32x4_t*>(lds);
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
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    if (!mine(i)) continue;
#pragma unroll
    for (int j = 0; j < TN; ++j) *chunk(lane & 15, j * 4 + (lane >> 4)) = acc[i][j];
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
    for (int h = 0; h < HN; ++h) {
      const At x = at(i, h);
      if (!x.ok) continue;
      f32x4_t v0 = *chunk(x.in, 2 * x.q), v1 = *chunk(x.in, 2 * x.q + 1);
      const u32x4_t* o = old[i % AHEAD][h];
      if constexpr (EPI == EPI_SWIGLU) {
        const f32x4_t u0 = *chunk(x.in, CH / 2 + 2 * x.q), u1 = *chunk(x.in, CH / 2 + 2 * x.q + 1);
        store_swiglu8(p, x.row, x.col, v0, v1, u0, u1);
      } else if constexpr (EPI == EPI_SWIGLU_BWD) {
        store_swiglu_bwd8(p, x.row, x.col, v0, v1, o[0], o[1]);
      } else {
        const int64_t at_c = x.row * nout + x.col;
        if (p.part) {
          float* part = p.part + static_cast<int64_t>(blockIdx.y) * p.part_stride;
          store4<true>(part, at_c, v0);
          store4<true>(part, at_c + 4, v1);
        } else if (p.c_f32) {
          if (reads) {
            v0 += __builtin_bit_cast(f32x4_t, o[0]);
            v1 += __builtin_bit_cast(f32x4_t, o[1]);
          }
          write_as<KIND == MOE_GEMM_TN>(static_cast<float*>(p.C) + at_c, v0);
          write_as<KIND == MOE_GEMM_TN>(static_cast<float*>(p.C) + at_c + 4, v1);
        } else {
          if (reads) {
            f32x4_t c0, c1;
            unpack8(o[0], c0, c1);
            v0 += c0;
            v1 += c1;
          }
          store8<KIND == MOE_GEMM_TN>(p.C, at_c, v0, v1);
        }
      }
    }
    if (reads && i + AHEAD < TM) read_old(i + AHEAD);   // (two halves: AHEAD is all of them)
    __builtin_amdgcn_wave_barrier();
  }
}

template <int KIND, int EPI, int BM, int BN, int BK, int WAVES_M, int WAVES_N, int WAVES_K, int NBUF, int TM>
__device__ __forceinline__ void gg_tile_of(int tm, const GgParams& p, const GgTile& t, uint8_t* lds) {
  if constexpr (TM == 1) {
    gg_tile<KIND, EPI, BM, BN, BK, WAVES_M, WAVES_N, WAVES_K, NBUF, 1>(p, t, lds);
  } else {
    if (tm == TM)
      gg_tile<KIND, EPI, BM, BN, BK, WAVES_M, WAVES_N, WAVES_K, NBUF, TM>(p, t, lds);
    else
      gg_tile_of<KIND, EPI, BM, BN, BK, WAVES_M, WAVES_N, WAVES_K, NBUF, TM - 1>(tm, p, t, lds);
  }
}

template <int KIND, int EPI, int BM, int BN, int BK, int WAVES_M, int WAVES_N, int WAVES_K, int NBUF>
__global__ __launch_bounds__(WAVES_M * WAVES_N * WAVES_K * 64, 2) void k_grouped_gemm(GgParams p) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[NBUF * (BM + BN) * BK * 2];
  GgTile t;
  if (!gg_locate<KIND, BM>(p, reinterpret_cast<int*>(lds), t)) return;
  constexpr int TM = BM / WAVES_M / 16;
  if constexpr (KIND == MOE_GEMM_TN)
    gg_tile<KIND, EPI, BM, BN, BK, WAVES_M, WAVES_N, WAVES_K, NBUF, TM>(p, t, lds);
  else
    gg_tile_of<KIND, EPI, BM, BN, BK, WAVES_M, WAVES_N, WAVES_K, NBUF, TM>((t.m_n + 16 * WAVES_M - 1) / (16 * WAVES_M),
                                                                          p, t, lds);
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
  if (gg_idle<KIND>(p, t)) return;
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

#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int in = wm * 32 + i * 16 + (lane & 15), m = t.m_off + in;
    if (in >= t.m_n) continue;
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

// Few fp32 tiles: one workgroup per 32 x 32 outputs (SwiGLU: 16 gate and 16 up
// columns), its four waves each with every fourth 16 steps of the reduction,
// fragments loaded straight from memory eight chunks at a time, the four sums
// joined through LDS in wave order.  Without the barriers of the tiled kernel
// a short call is one or two memory round trips: 128 rows of 8 experts,
// 128 x 512: 13.3 us tiled.
template <int KIND, int EPI>
__global__ __launch_bounds__(256) void k_grouped_gemm_f32_few(GgParams p) {
  static_assert(KIND != MOE_GEMM_TN, "a row product");
  constexpr int BM = 32, AHEAD = 4;
  __shared__ f32x4_t red[4][4][64];
  __shared__ int s_loc[8];
  GgTile t;
  if (!gg_locate<KIND, BM>(p, s_loc, t)) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int l15 = lane & 15, g4 = (lane >> 4) * 4;       // fragment: position l15, steps g4 .. g4 + 3
  const int c0 = t.nt * (EPI == EPI_SWIGLU ? 16 : 32);
  const float* a[2];
  const float* b[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    a[i] = static_cast<const float*>(p.A) + (t.row0 + t.m_off + min(i * 16 + l15, t.m_n - 1)) * p.K + g4;
    const int brows = EPI == EPI_SWIGLU ? 2 * p.N : p.N;
    const float* B = static_cast<const float*>(p.B) + static_cast<int64_t>(t.e) * brows * p.K;
    const int col = EPI == EPI_SWIGLU ? min(c0 + l15, p.N - 1) + i * p.N : min(c0 + i * 16 + l15, p.N - 1);
    b[i] = KIND == MOE_GEMM_NT ? B + static_cast<int64_t>(col) * p.K + g4 : B + static_cast<int64_t>(g4) * p.N + col;
  }
  const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
  f32x4_t acc[2][2] = {{zero, zero}, {zero, zero}};
  const int chunks = (p.K + 15) / 16;
  for (int c = wave; c < chunks; c += 4 * AHEAD) {
    f32x4_t av[AHEAD][2], bv[AHEAD][2];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      const int k = (c + 4 * u) * 16;
      const bool in = k + g4 < p.K;                      // K is a multiple of 4: four steps or none
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        av[u][i] = in ? *reinterpret_cast<const f32x4_t*>(a[i] + k) : zero;
        if constexpr (KIND == MOE_GEMM_NT) {
          bv[u][i] = in ? *reinterpret_cast<const f32x4_t*>(b[i] + k) : zero;
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q) bv[u][i][q] = in ? b[i][static_cast<int64_t>(k + q) * p.N] : 0.f;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < AHEAD; ++u)
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(bv[u][j][q], av[u][i][q], acc[i][j], 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) red[wave][i * 2 + j][lane] = acc[i][j];
  __syncthreads();
  // wave w finishes subtile (w >> 1, w & 1)
  auto sum = [&](int q) {
    f32x4_t v = red[0][q][lane];
#pragma unroll
    for (int w = 1; w < 4; ++w) v += red[w][q][lane];
    return v;
  };
  const int i = wave >> 1, j = wave & 1, in = i * 16 + l15;
  if (in >= t.m_n) return;
  const int64_t row = t.row0 + t.m_off + in;
  if constexpr (EPI == EPI_SWIGLU) {
    const int col = c0 + g4;
    if (j == 0 && col < p.N) store_swiglu<true>(p, row, col, sum(i * 2), sum(i * 2 + 1));
  } else {
    const int col = c0 + j * 16 + g4;
    if (col >= p.N) return;
    if constexpr (EPI == EPI_SWIGLU_BWD)
      store_swiglu_bwd<true>(p, row, col, sum(wave));
    else
      store_c(p, row * p.N + col, sum(wave));
  }
}

// Sums the partial outputs of a split reduction in split order (so the result
// does not depend on timing) and stores C.  NT/NN (row_quads: a row's, else 0):
// only the rows of experts.  TN (expert_quads: an expert's) that adds to C: only
// the experts that have rows, the others made no parts.
__global__ __launch_bounds__(256) void k_join_splits(GgParams p, int64_t quads, int row_quads, uint32_t expert_quads) {
  int64_t lo = 0, lim = quads;
  if (row_quads && p.offsets) {
    lo = min(static_cast<int64_t>(max(p.offsets[0], 0)), p.cap) * row_quads;
    lim = min(static_cast<int64_t>(max(p.offsets[p.E], 0)), p.cap) * row_quads;
  }
  const float* part = p.part;
  GgParams q = p;
  q.part = nullptr;
  const bool skips = p.offsets && !row_quads && p.accumulate;
  for (int64_t i = lo + static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < lim;
       i += static_cast<int64_t>(gridDim.x) * 256) {
    if (skips) {
      int o, n;
      gg_rows(p, static_cast<uint32_t>(i) / expert_quads, o, n);     // (a split C has fewer than 2^23 elements)
      if (n == 0) continue;
    }
    f32x4_t v = load4<true>(part, i * 4);
    for (int s = 1; s < p.splits; ++s) v += load4<true>(part + s * p.part_stride, i * 4);
    store_c(q, i * 4, v);
  }
}

// ---- host -------------------------------------------------------------------

// Tile and reduction parts of a call, from its sizes alone.  (The workspace
// query makes the same choice; adds, the one argument it does not have, decides
// between two shapes that are never split.)  Measured on both sides of each border, 64
// experts, us with uniform / Zipf-distributed (1.2) rows:
//   32 x 128 against 128 x 128, by rows of an average expert (2048 x 1408): the
//   SwiGLU backward with 24 rows 76 / 77 against 82 / 87, with 32 rows 83 / 87
//   against 87 / 90; NT with 32 rows 74 / 84 against 72 / 85, with 48 rows 95
//   against 78 (uniform).
//   256 x 256 against 128 x 128: NT with 96 rows 93 against 90 (uniform), with 128
//   rows 98 / 121 against 108 / 109, with 192 rows 108 / 124 against 129 / 132; TN
//   with 32 to 256 rows 107 to 174 against 124 to 187 (uniform).
//   Where the epilogue reads as much as it writes and the reduction is short, two
//   workgroups of 128 x 128 on a compute unit overlap one's epilogue with the
//   other's MFMAs.  SwiGLU backward, 512 rows an expert x 1408, against 256 x 256:
//   H = 512 153 / 135 against 172 / 157, 1024 197 / 188 against 209 / 204, 2048
//   302 / 303 against 307 / 305, 4096 520 / 528 against 501 / 521; 768 wide (128
//   experts), H = 2048 334 / 332 against 326 / 325.  TN that adds to C, 2816 x
//   2048 fp32 (uniform): 64 rows 541 against 614, 256 rows 662 against 720, 512
//   rows 841 against 864, 1024 rows 1183 against 1136.
//   64 x 128 (the reduction split inside the workgroup) up to 128 tiles, against
//   128 x 128: TN 8192 rows 128 x 2048 19 against 23, NN 661 rows of 8 experts
//   760 x 104 7.0 against 10.0; with more tiles its traffic from L2 (12 TB/s)
//   bounds it: TN 4096 rows 256 x 7168 44 against 34.
//   fp32: 32 x 32 while 64 x 64 would give fewer than 256 tiles: NN 128 rows of 8
//   experts 128 x 512 6.9 against 13.3.
struct GgPlan { int BM, BN, splits; int64_t tiles; };

static int64_t gg_tiles(int kind, int epi, int E, int64_t cap, bool dense, int N, int K, int BM, int BN) {
  const int64_t mt = (N + BM - 1) / BM, nt = kind == MOE_GEMM_TN ? (K + BN - 1) / BN
                                           : epi == EPI_SWIGLU   ? (N + BN / 2 - 1) / (BN / 2)
                                                                 : (N + BN - 1) / BN;
  if (kind == MOE_GEMM_TN) return E * ((mt * nt + 7) / 8 * 8);      // each XCD's share of an expert is rounded up
  return max_row_tiles(cap, E, BM, dense) * nt;
}

static GgPlan gg_plan(int kind, int epi, bool f32, int E, int64_t cap, bool dense, int N, int K, bool adds = false) {
  const int64_t rows = cap / E;                     // of an average expert
  const int cols = kind == MOE_GEMM_TN ? K : epi == EPI_SWIGLU ? 2 * N : N;
  GgPlan q{128, 128, 1, 0};
  if (f32)
    q.BM = q.BN = kind != MOE_GEMM_TN && gg_tiles(kind, epi, E, cap, dense, N, K, 64, 64) < 256 ? 32 : 64;
  else if (kind != MOE_GEMM_TN && rows <= 32)
    q.BM = 32;
  else if (cols > 128 && (kind == MOE_GEMM_TN ? N > 128 : rows > 128) &&
           !(epi == EPI_SWIGLU_BWD && K < 2048) && !(kind == MOE_GEMM_TN && adds && rows <= 512) &&
           gg_tiles(kind, epi, E, cap, dense, N, K, 256, 256) >= 256)
    q.BM = q.BN = 256;
  else if (gg_tiles(kind, epi, E, cap, dense, N, K, 64, 128) <= 128)
    q.BM = 64;
  q.tiles = gg_tiles(kind, epi, E, cap, dense, N, K, q.BM, q.BN);
  // The reduction is cut into parts, doubled while the grid has fewer than 256
  // workgroups (64-row tiles, one a compute unit: as long as it stays within
  // 256) and each part keeps at least 256 steps, at most 16.
  const int64_t red = kind == MOE_GEMM_TN ? rows : K, limit = q.BM == 64 && !f32 ? 129 : 256;
  if (epi == EPI_STORE && !(f32 && q.BM == 32))
    while (q.splits < 16 && q.tiles * q.splits < limit && red / (2 * q.splits) >= 256) q.splits *= 2;
  return q;
}

template <int KIND, int EPI>
static moe_status gg_launch(GgParams& p, const GgPlan& q, bool f32, hipStream_t s) {
  const int cols = KIND == MOE_GEMM_TN ? p.K : p.N, width = EPI == EPI_SWIGLU ? q.BN / 2 : q.BN;
  p.n_tiles = (cols + width - 1) / width;
  p.m_tiles = (p.N + q.BM - 1) / q.BM;
  p.splits = q.splits;
  if (gemm_grid(q.tiles) >= (1 << 23)) return MOE_ERR_UNSUPPORTED;      // at most 512 threads each, 2^32 in a grid
  const dim3 grid(static_cast<unsigned>(gemm_grid(q.tiles)), q.splits);
  if (f32 && q.BM == 64) {
    hipLaunchKernelGGL((k_grouped_gemm_f32<KIND, EPI>), grid, dim3(256), 0, s, p);
  } else if (f32) {
    if constexpr (KIND != MOE_GEMM_TN)
      hipLaunchKernelGGL((k_grouped_gemm_f32_few<KIND, EPI>), grid, dim3(256), 0, s, p);
  } else if (q.BM == 256) {
    hipLaunchKernelGGL((k_grouped_gemm<KIND, EPI, 256, 256, 64, 2, 4, 1, 2>), grid, dim3(512), 0, s, p);
  } else if (q.BM == 128) {
    hipLaunchKernelGGL((k_grouped_gemm<KIND, EPI, 128, 128, 64, 2, 2, 1, 2>), grid, dim3(256), 0, s, p);
  } else if (q.BM == 64) {
    hipLaunchKernelGGL((k_grouped_gemm<KIND, EPI, 64, 128, 128, 2, 2, 2, 3>), grid, dim3(512), 0, s, p);
  } else if constexpr (KIND != MOE_GEMM_TN) {
    hipLaunchKernelGGL((k_grouped_gemm<KIND, EPI, 32, 128, 64, 1, 4, 1, 3>), grid, dim3(256), 0, s, p);
  }
  DBOMOE_CHECK_LAUNCH();
  if (q.splits > 1) {
    const int64_t elems = KIND == MOE_GEMM_TN ? static_cast<int64_t>(p.E) * p.N * p.K : p.cap * p.N;
    const int64_t blocks = (elems / 4 + 255) / 256;
    hipLaunchKernelGGL(k_join_splits, dim3(static_cast<unsigned>(blocks < 4096 ? blocks : 4096)), dim3(256), 0, s, p,
                       elems / 4, KIND == MOE_GEMM_TN ? 0 : p.N / 4,
                       static_cast<uint32_t>(static_cast<int64_t>(p.N) * p.K / 4));
    DBOMOE_CHECK_LAUNCH();
  }
  return MOE_OK;
}

// Checks that every grouped product shares.  E_loc, sizes and types only.
static moe_status gg_check_sizes(moe_dtype ab, bool dense, int32_t E_loc, int64_t cap_rows, int32_t N, int32_t K) {
  if (E_loc < 1 || E_loc > 256 || cap_rows < 0 || N < 1 || K < 1) return MOE_ERR_INVALID_ARG;
  if (dense && E_loc != 1) return MOE_ERR_INVALID_ARG;
  if (ab != MOE_F32 && ab != MOE_BF16) return MOE_ERR_UNSUPPORTED;
  if (cap_rows > (1 << 30) || N > (1 << 22) || K > (1 << 22)) return MOE_ERR_UNSUPPORTED;
  const int q = ab == MOE_F32 ? 4 : 8;        // rows start on 16 bytes
  if (N % q || K % q) return MOE_ERR_MISALIGNED;
  return MOE_OK;
}

static moe_status gg_check(moe_dtype ab, const int32_t* offsets, int32_t E_loc, int64_t cap_rows, int32_t N, int32_t K) {
  const moe_status st = gg_check_sizes(ab, !offsets, E_loc, cap_rows, N, K);
  if (st != MOE_OK) return st;
  return offsets && !aligned16(offsets) ? MOE_ERR_MISALIGNED : MOE_OK;
}

}  // namespace dbomoe

using namespace dbomoe;

extern "C" size_t moe_grouped_gemm_workspace_size(moe_gemm_kind kind, moe_dtype ab, int32_t dense, int32_t E_loc,
                                                  int64_t cap_rows, int32_t N, int32_t K) {
  if (kind != MOE_GEMM_NT && kind != MOE_GEMM_NN && kind != MOE_GEMM_TN) return 0;
  if (cap_rows < 1 || gg_check_sizes(ab, dense != 0, E_loc, cap_rows, N, K) != MOE_OK) return 0;
  const int S = gg_plan(kind, EPI_STORE, ab == MOE_F32, E_loc, cap_rows, dense != 0, N, K).splits;
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
  const bool f32 = ab == MOE_F32;
  const GgPlan q = gg_plan(kind, EPI_STORE, f32, E_loc, cap_rows, !offsets, N, K, accumulate != 0);
  if (q.splits > 1) {
    if (!ws) return MOE_ERR_INVALID_ARG;
    if (!aligned256(ws)) return MOE_ERR_MISALIGNED;
    if (ws_bytes < moe_grouped_gemm_workspace_size(kind, ab, !offsets, E_loc, cap_rows, N, K)) return MOE_ERR_WORKSPACE;
    p.part = static_cast<float*>(ws);
    p.part_stride = tn ? static_cast<int64_t>(E_loc) * N * K : cap_rows * N;
  }
  const hipStream_t s = as_stream(stream);
  if (kind == MOE_GEMM_NT) return gg_launch<MOE_GEMM_NT, EPI_STORE>(p, q, f32, s);
  if (kind == MOE_GEMM_NN) return gg_launch<MOE_GEMM_NN, EPI_STORE>(p, q, f32, s);
  return gg_launch<MOE_GEMM_TN, EPI_STORE>(p, q, f32, s);
}

extern "C" moe_status moe_grouped_swiglu(const void* x_perm, const void* w13, moe_dtype act, const int32_t* offsets,
                                         int32_t E_loc, int64_t cap_rows, int32_t H, int32_t I, void* gu, void* h,
                                         void* stream) {
  const moe_status st = gg_check(act, offsets, E_loc, cap_rows, I, H);
  if (st != MOE_OK) return st;
  if (cap_rows == 0) return MOE_OK;
  if (!x_perm || !w13 || !h) return MOE_ERR_INVALID_ARG;
  // the up rows are addressed by 32-bit byte offsets from the gate rows
  if ((static_cast<int64_t>(I) + 256) * H * 2 >= (int64_t{1} << 32)) return MOE_ERR_UNSUPPORTED;
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
  const GgPlan q = gg_plan(MOE_GEMM_NT, EPI_SWIGLU, act == MOE_F32, E_loc, cap_rows, !offsets, I, H);
  return gg_launch<MOE_GEMM_NT, EPI_SWIGLU>(p, q, act == MOE_F32, as_stream(stream));
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
  const GgPlan q = gg_plan(MOE_GEMM_NN, EPI_SWIGLU_BWD, act == MOE_F32, E_loc, cap_rows, !offsets, I, H);
  return gg_launch<MOE_GEMM_NN, EPI_SWIGLU_BWD>(p, q, act == MOE_F32, as_stream(stream));
}
