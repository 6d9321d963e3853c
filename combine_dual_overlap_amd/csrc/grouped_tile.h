// Tiles of the products grouped by expert (gfx950): where a workgroup's tile lies,
// and one operand's tile staged into LDS.  An element is 16 bits here; two 8-bit
// integers of one row count as one.
#pragma once

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

}  // namespace dbomoe
