// Products of 8-bit integers grouped by expert, with a scale for each token (row
// of a) and each output channel (row of b), and the quantisation that feeds them,
// for gfx950.
//   C[r, n] = (sum_k A[r, k] B[e, n, k]) * as[r] * bs[e, n]     sums in int32: exact
// An LDS stage, a fragment and an MFMA (v_mfma_i32_16x16x64_i8) are those of the
// bf16 product with two integers in the place of one bf16: twice the operations
// for the same bytes.
// Few rows an expert: HBM-bound, 193 MB of weights in 40 us (4.8 TB/s).  Many: bound by
// the matrix pipes at the clock that random integers leave (2.0 - 2.1 GHz): 8192^3 2040
// TOP/s, 2780 with zeros; 65536 rows of 128 experts, 2048 -> 2 x 768 with SwiGLU 272 us
// (1515 TOP/s), 768 -> 2048 165 us, 50 of these its stores, which all workgroups make at
// about the same time.  LDS bank conflicts by the counters: 12 to 25 thousand cycles a call on all
// compute units together, less than one in a thousand.
#include "grouped_tile.h"
#include "int8_rows.h"

namespace dbomoe {

typedef int i32x4_t __attribute__((ext_vector_type(4)));

// ---- rows to 8-bit integers ---------------------------------------------------
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
    uint32_t w[CH > 0 ? CH : 1][Chunk<BF16>::N / 4];
    if constexpr (CH > 0) codes_of<BF16>(v, rq, w);
    const int n = inv ? k : 1;
    for (int j = 0; j < n; ++j) {
      const int64_t pos = inv ? static_cast<int64_t>(__shfl(my_pos, j, kWave)) : t;
      if (pos < 0) continue;
      int8_t* dst = q + pos * row_bytes;
      if constexpr (CH > 0) {
#pragma unroll
        for (int i = 0; i < CH; ++i) {
          const int c = i * 64 * W + l;
          if (c < rc) put_codes<BF16>(dst, c, w[i]);
        }
      } else {
        for (int c = l; c < rc; c += 64 * W) {
          codes_any<BF16>(src[c], rq, w[0]);
          put_codes<BF16>(dst, c, w[0]);
        }
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
    // (65536 rows of 256 bf16 chunks: 85 us with one wave each, 104 with four)
    with_row_shape(a.T, rc, 256, [&](auto w, auto ch) {
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

// C = product (c_f32, or bf16), or with SwiGLU h = silu(gate) * up.
//
// A workgroup walks tiles BM x BN of its XCD's contiguous run of them, BK pairs of
// integers per stage, in a ring of NBUF stages that runs on from one tile into the
// next: the next tile's first stages are on their way while this one's results are
// scaled and stored.
//  - Every wave keeps the whole tile map (experts' rows and first tiles) in LDS.
//  - The tile's scales come to LDS as its first stage does.
//  - Of eight waves four load, one on each SIMD: while a stage's DMAs queue up (64 of
//    16 clocks), the SIMD's other wave goes on with its MFMAs.  All eight loading
//    against four: prefill gate/up 284 / 266 us (with a shorter SwiGLU), down 170 / 165, 8192^3 of zeros 423 /
//    395 (of random integers 545 / 538: the clock gives way to the power).
//  - The second operand's rows are dealt to the MFMA's positions so that a lane ends
//    up with 16 bytes of consecutive columns of its row and stores them as they are
//    (64 bytes of a row by four lanes): position q of TG neighbouring subtiles is row
//    (q / 4) 4 TG + 4 j + q % 4 of theirs, TG = 1 for fp32 and 2 for bf16.
template <int EPI, bool F32, int BM, int BN, int WAVES_M, int WAVES_N, int NBUF>
struct I8Shape {
  static constexpr int BK = 64;                                 // pairs: 128 bytes of a row
  static constexpr int NW = WAVES_M * WAVES_N;
  static constexpr int WM = BM / WAVES_M, WN = BN / WAVES_N, TM = WM / 16, TN = WN / 16;
  static constexpr int TH = EPI == EPI_SWIGLU ? TN / 2 : TN;    // subtiles of output columns
  static constexpr int TG = F32 || TH == 1 ? 1 : 2;
  static constexpr int STAGE = (BM + BN) * BK * 2;
  static constexpr int NI = NW == 8 ? 4 : NW;                   // waves that load
  static constexpr int NQA = BM / (8 * NI), NQB = BN / (8 * NI);  // their DMAs per stage: 8 rows each
  static constexpr int NDMA = NQB + 1;                          // at least: rows of a that do not exist are not loaded
  static constexpr int SLOTS = 4;                               // tiles whose scales are in LDS: NBUF + 1 at most
  static_assert(NQA * 8 * NI == BM && NQB * 8 * NI == BN && NI % 4 == 0, "DMA split");
  static_assert((BM + 63) / 64 + BN / 64 <= NW && NBUF < SLOTS && (NBUF - 1) * (NQA + NQB) < 64, "scales, ring, vmcnt");
  // the XORs that rows put on their 16-byte chunks: the eight lanes that read together
  // hit rows of both parities and four keys
  static __device__ __forceinline__ int key_a(int r) { return r & 7; }
  static __device__ __forceinline__ int key_b(int r) { return (r >> 1 & 1) | (r / (4 * TG) & 3) << 1; }
};

// The quotient of the hardware's reciprocal is put right by its exact remainder, so h is what fp32
// arithmetic makes it, and its codes with it; the fixup gives what is infinite or NaN its value.
// (With that reciprocal alone and the hardware's exponential, three of ten h were off in the last
// places, and one code in thousands: the prefill experts in 525 us, not 540; with an IEEE division
// 562.)  From 1 + e^-g = 2^126 on, g < -87, the reciprocal and h are 0.
__device__ __forceinline__ float silu(float g) {
  const float d = 1.0f + expf(-g);
  const float r = __builtin_amdgcn_rcpf(d), q = g * r;
  return __builtin_amdgcn_div_fixupf(fmaf(fmaf(-d, q, g), r, q), d, g);
}

struct I8Tile {
  int e, m_n, nt, tm;
  int64_t row;             // first row of the tile
};

template <int EPI, bool F32, int BM, int BN, int WAVES_M, int WAVES_N, int NBUF>
__global__ __launch_bounds__(WAVES_M * WAVES_N * 64, 2) void k_grouped_int8(I8Params ip) {
  using S = I8Shape<EPI, F32, BM, BN, WAVES_M, WAVES_N, NBUF>;
  constexpr int BK = S::BK, NW = S::NW, NI = S::NI, WN = S::WN, TM = S::TM, TN = S::TN, TH = S::TH, TG = S::TG;
  __shared__ __attribute__((aligned(1024))) uint8_t ring[NBUF * S::STAGE];
  __shared__ float s_scale[S::SLOTS][BM + BN];
  __shared__ __attribute__((aligned(16))) int s_first[256];     // the expert's first tile
  __shared__ int s_row0[256], s_rows[256];
  const GgParams& p = ip.g;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WAVES_N, wn = wave % WAVES_N;

  if (threadIdx.x < kWave) {
    int t4[4], sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      int o = 0, n = 0;
      if (lane * 4 + i < p.E) gg_rows(p, lane * 4 + i, o, n);
      s_row0[lane * 4 + i] = o;
      s_rows[lane * 4 + i] = n;
      t4[i] = (n + BM - 1) / BM * p.n_tiles;
      sum += t4[i];
    }
    int at = wave_incl_scan(sum) - sum;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s_first[lane * 4 + i] = at;
      at += t4[i];
    }
    if (lane == 63) s_scale[0][0] = __int_as_float(at);         // all tiles
  }
  __syncthreads();
  const int R = __builtin_amdgcn_readfirstlane(__float_as_int(s_scale[0][0]));
  __syncthreads();
  // Workgroup b runs on XCD b % 8, which walks a contiguous run of tiles.
  const int per = (R + 7) / 8, xcd = blockIdx.x & 7, stride = gridDim.x >> 3;
  const int stop = min((xcd + 1) * per, R);
  const int L0 = xcd * per + (blockIdx.x >> 3);
  if (L0 >= stop) return;
  auto locate = [&](int L) {
    const int4 f = reinterpret_cast<const int4*>(s_first)[lane];
    const int e = __popcll(__ballot(f.x <= L)) + __popcll(__ballot(f.y <= L)) + __popcll(__ballot(f.z <= L)) +
                  __popcll(__ballot(f.w <= L)) - 1;             // the last expert that starts at L or before
    const int rows = __builtin_amdgcn_readfirstlane(s_rows[e]);
    const int l = L - __builtin_amdgcn_readfirstlane(s_first[e]);
    const int tiles = (rows + BM - 1) / BM;
    // bands of eight row tiles: what runs together on an XCD is about as high as wide
    const int band = l / (8 * p.n_tiles), r = l - band * 8 * p.n_tiles, high = min(8, tiles - 8 * band);
    // the expert's rows in tiles of equal height (a multiple of 32 where tiles are higher than that)
    const int height = BM <= 32 ? BM : ((rows + tiles - 1) / tiles + 31) / 32 * 32;
    const int m_off = (8 * band + r % high) * height;
    I8Tile t;
    t.e = __builtin_amdgcn_readfirstlane(e);
    t.nt = __builtin_amdgcn_readfirstlane(r / high);
    t.m_n = __builtin_amdgcn_readfirstlane(min(height, rows - m_off));
    t.row = __builtin_amdgcn_readfirstlane(s_row0[e] + m_off);
    // subtiles of 16 rows go to the waves in turn: a tile that is not full keeps them all busy
    t.tm = __builtin_amdgcn_readfirstlane(((t.m_n + 15) / 16 - wm + WAVES_M - 1) / WAVES_M);
    return t;
  };

  // ---- loads: the tile whose stages are being asked for runs ahead of the one computed
  const int KT = (p.K + BK - 1) / BK;
  const int brows = EPI == EPI_SWIGLU ? 2 * p.N : p.N;
  const uint32_t lds0 = static_cast<uint32_t>(
      reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t*)(ring)));
  const uint32_t lds_scale = static_cast<uint32_t>(
      reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) float*)(&s_scale[0][0])));
  const int64_t row_bytes = static_cast<int64_t>(p.K) * 2;
  const uint8_t *a_base, *b_base;                    // uniform
  int a_dmas = 0;                                    // of this wave and stage: those with rows of the tile
  uint32_t a_last, b_most;                           // the lane's chunk of the last of them; the last columns' rows
  int L_in = L0, kt_in = 0, issued = 0, tile_in = 0;
  // A DMA takes eight rows: lane l the row l / 8 of them and chunk (l % 8) ^ key, a key
  // that does not depend on which of the wave's DMAs it is.  So a lane's offsets are the
  // same in all of them, from bases that stay in scalar registers, but for the last rows
  // of a.
  const int lr = lane >> 3, pos = lane & 7;
  const int chunk_a = pos ^ S::key_a(lr), chunk_b = pos ^ S::key_b(8 * wave + lr);
  const uint32_t step8 = static_cast<uint32_t>(row_bytes) * 8, step = step8 * NI;
  const uint32_t a_off = (8 * wave + lr) * static_cast<uint32_t>(row_bytes) + chunk_a * 16;
  const uint32_t b_off = lr * static_cast<uint32_t>(row_bytes) + chunk_b * 16;
  auto open_tile = [&](int L) {
    const I8Tile t = locate(L);
    a_base = static_cast<const uint8_t*>(p.A) + t.row * row_bytes;
    const int m_last = t.m_n - 1;                    // rows and columns behind the last are its copies
    a_dmas = (t.m_n + 8 * NI - 1) / (8 * NI);
    a_last = min(8 * ((a_dmas - 1) * NI + wave) + lr, m_last) * static_cast<uint32_t>(row_bytes) + chunk_a * 16;
    const int col0 = t.nt * (EPI == EPI_SWIGLU ? BN / 2 : BN);
    const int n_last = p.N - 1 - col0;
    // row of b of row x of the tile (SwiGLU: half a tile of gate rows, then the matching up rows)
    auto row_of = [&](int x) {
      return EPI == EPI_SWIGLU ? min(x & (BN / 2 - 1), n_last) + (x < BN / 2 ? 0 : p.N) : min(x, n_last);
    };
    b_most = (min(n_last, BN - 1) - 7) * static_cast<uint32_t>(row_bytes);   // (columns come in eights)
    b_base = static_cast<const uint8_t*>(p.B) + (static_cast<int64_t>(t.e) * brows + col0) * row_bytes;
    // the scales: 64 rows or columns by each wave
    constexpr int WA = (BM + 63) / 64;
    const uint32_t at = lds_scale + (tile_in % S::SLOTS) * (BM + BN) * 4;
    if (wave < WA) {
      const int r = wave * 64 + lane;
      if (r < BM) lds_dma4(at + wave * 256, ip.as + t.row + min(r, m_last));
    } else if (wave < WA + BN / 64) {
      const int c = (wave - WA) * 64;
      lds_dma4(at + BM * 4 + c * 4, ip.bs + static_cast<int64_t>(t.e) * brows + col0 + row_of(c + lane));
    }
  };
  auto issue = [&]() {
    if (kt_in == KT) {
      L_in += stride;
      kt_in = 0;
      ++tile_in;
    }
    if (L_in >= stop) return;
    if (kt_in == 0) open_tile(L_in);
    const uint32_t at = lds0 + (issued % NBUF) * S::STAGE + wave * 1024;
    const int left = p.K - kt_in * BK;
    const uint8_t *as = a_base + kt_in * (BK * 2), *bs = b_base + kt_in * (BK * 2);
    if (NI == NW || wave < NI) {
      // rows of b of DMA i (SwiGLU: gate rows, then up rows)
      constexpr int HALF = EPI == EPI_SWIGLU ? S::NQB / 2 : S::NQB;
      auto b_at = [&](int i) {
        const uint32_t up = i < HALF ? 0 : static_cast<uint32_t>(p.N) * static_cast<uint32_t>(row_bytes);
        return bs + min(wave * step8 + i % HALF * step, b_most) + up;
      };
      if (left >= BK) {
#pragma unroll
        for (int i = 0; i < S::NQA; ++i) {
          if (i < a_dmas - 1)
            lds_dma16_at(at + i * NI * 1024, as + i * step, a_off);
          else if (i == a_dmas - 1)
            lds_dma16_at(at + i * NI * 1024, as, a_last);
        }
#pragma unroll
        for (int i = 0; i < S::NQB; ++i) lds_dma16_at(at + BM * 128 + i * NI * 1024, b_at(i), b_off);
      } else {                                       // the reduction ends inside the stage: zeros behind it
#pragma unroll
        for (int i = 0; i < S::NQA; ++i) {
          const uint8_t* src = as + (i < a_dmas - 1 ? i * step + a_off : a_last);
          if (i < a_dmas) lds_dma16(at + i * NI * 1024, chunk_a * 8 < left ? static_cast<const void*>(src) : g_zero16);
        }
#pragma unroll
        for (int i = 0; i < S::NQB; ++i)
          lds_dma16(at + BM * 128 + i * NI * 1024, chunk_b * 8 < left ? static_cast<const void*>(b_at(i) + b_off) : g_zero16);
      }
    }
    ++kt_in;
    ++issued;
  };

  // ---- products.  Accumulators hold C transposed: lane l has row l & 15 and four
  // positions 4 (l >> 4) .. + 3 of each 16 x 16 subtile.
  i32x4_t acc[TM][TN], af[TM], bfr[2][TN];
  const int l15 = lane & 15, g = lane >> 4;
  const int rb = (l15 >> 2) * (4 * TG) + (l15 & 3);
  // first column of subtile j in the lane's own of the wave's, but for the lane's place among them
  auto sub = [](int j) { return j / TG * (16 * TG) + j % TG * 4; };
  auto frag = [&](const uint8_t* tile, int r, int key, int kk) {
    return *reinterpret_cast<const i32x4_t*>(tile + r * (BK * 2) + (((kk * 4 + g) ^ key) << 4));
  };
  auto read_a = [&](int s, int kk, int i) {
    const int r = (i * WAVES_M + wm) * 16 + l15;
    af[i] = frag(ring + (s % NBUF) * S::STAGE, r, S::key_a(r), kk);
  };
  auto read_b = [&](int s, int kk, int set) {
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const int r = EPI == EPI_SWIGLU ? (j / TH) * (BN / 2) + wn * (WN / 2) + rb + sub(j % TH) : wn * WN + rb + sub(j);
      bfr[set][j] = frag(ring + (s % NBUF) * S::STAGE + BM * BK * 2, r, S::key_b(r), kk);
    }
  };
  int tm = TM;
  auto mfmas = [&](int i, int set) {
    if (i < tm) {
#pragma unroll
      for (int j = 0; j < TN; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(bfr[set][j], af[i], acc[i][j], 0, 0, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  // The reduction advances in two steps of 32 pairs a stage.  A fragment of the first
  // operand is read again, for the next step, as soon as this step's MFMAs have taken
  // it, and the second operand's of the next step are read ahead into a second set.
  // Half of the second step's MFMAs run before the barrier that hands the stage's
  // buffer back; the DMAs that fill it again follow at once.  (Spread between the MFMAs
  // behind it, they come late: 4 % slower.  After the last stage of all, bytes are read
  // that nothing uses.)
  auto stage = [&](int s) {
    read_b(s, 1, 1);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      mfmas(i, 0);
      read_a(s, 1, i);
    }
#pragma unroll
    for (int i = 0; i < TM / 2; ++i) mfmas(i, 1);
    // this wave's reads of the stage are done, and its DMAs of the next
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    wait_stages<S::NDMA, NBUF - 2>(issued - s - 2);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    issue();
    read_b(s + 1, 0, 0);
#pragma unroll
    for (int i = 0; i < TM / 2; ++i) read_a(s + 1, 0, i);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = TM / 2; i < TM; ++i) {
      mfmas(i, 1);
      read_a(s + 1, 0, i);
    }
  };

  __builtin_amdgcn_s_waitcnt(0);           // from here on only counted DMAs are in flight (and stores, which are younger)
  for (int s = 0; s < NBUF; ++s) issue();
  wait_stages<S::NDMA, NBUF - 1>(issued - 1);
  __syncthreads();
  read_b(0, 0, 0);
#pragma unroll
  for (int i = 0; i < TM; ++i) read_a(0, 0, i);
  int s = 0, tile = 0;
#pragma unroll 1
  for (int L = L0; L < stop; L += stride, ++tile) {
    const I8Tile t = locate(L);
    tm = t.tm;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = i32x4_t{0, 0, 0, 0};
#pragma unroll 1
    for (int kt = 0; kt < KT; ++kt, ++s) stage(s);

    // The sums become fp32 (a rounding of 2^-24), times the row's scale, times the channel's.
    const float* sc = s_scale[tile % S::SLOTS];
    const int c0 = (EPI == EPI_SWIGLU ? wn * (WN / 2) : wn * WN) + g * (4 * TG);
    const int col = t.nt * (EPI == EPI_SWIGLU ? BN / 2 : BN) + c0;
    f32x4_t bs[TN];
#pragma unroll
    for (int j = 0; j < TN; ++j)
      bs[j] = *reinterpret_cast<const f32x4_t*>(sc + BM + c0 + (EPI == EPI_SWIGLU ? (j / TH) * (BN / 2) : 0) + sub(j % TH));
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      if (i >= tm) break;
      const int in = (i * WAVES_M + wm) * 16 + l15;
      if (in >= t.m_n) continue;
      const float as = sc[in];
      f32x4_t v[TN];
#pragma unroll
      for (int j = 0; j < TN; ++j) v[j] = __builtin_convertvector(acc[i][j], f32x4_t) * as * bs[j];
      if constexpr (EPI == EPI_SWIGLU) {
#pragma unroll
        for (int j = 0; j < TH; ++j)
#pragma unroll
          for (int x = 0; x < 4; ++x) v[j][x] = silu(v[j][x]) * v[j + TH][x];
      }
      const int64_t at = (t.row + in) * p.N + col;
      if constexpr (F32) {
#pragma unroll
        for (int j = 0; j < TH; ++j)
          if (col + sub(j) < p.N) *reinterpret_cast<f32x4_t*>(static_cast<float*>(p.C) + at + sub(j)) = v[j];
      } else if constexpr (TG == 1) {
        if (col < p.N)
          *reinterpret_cast<uint2*>(static_cast<bf16_t*>(p.C) + at) = make_uint2(cvt_bf16x2(v[0][0], v[0][1]), cvt_bf16x2(v[0][2], v[0][3]));
      } else {
#pragma unroll
        for (int j = 0; j < TH; j += 2)
          if (col + sub(j) < p.N)
            *reinterpret_cast<u32x4_t*>(static_cast<bf16_t*>(p.C) + at + sub(j)) =
                u32x4_t{cvt_bf16x2(v[j][0], v[j][1]), cvt_bf16x2(v[j][2], v[j][3]), cvt_bf16x2(v[j + 1][0], v[j + 1][1]),
                        cvt_bf16x2(v[j + 1][2], v[j + 1][3])};
      }
    }
  }
}

// Few tiles: one workgroup per 32 x 32 outputs (SwiGLU: 16 gate and 16 up columns), its
// eight waves each with every eighth 128 bytes of the reduction, fragments loaded straight
// from memory, the eight sums joined through LDS.  No barrier until then: where the tiled
// kernel takes 0.42 us a stage whatever is in it, a short call is two or three memory
// round trips.  One row x 2048 x 2048 9.2 -> 5.2 us, x 1024 x 7168 23 -> 10; 64 rows of 4
// experts x 2048 x 1408 7.9 -> 5.9.  (256 bytes or more at a time: 3 to 30 % slower.)
template <int EPI, bool F32>
__global__ __launch_bounds__(512) void k_grouped_int8_few(I8Params ip) {
  constexpr int BM = 32, NW = 8;
  __shared__ i32x4_t red[NW][4][64];
  __shared__ int s_loc[8];
  const GgParams& p = ip.g;
  GgTile t;
  if (!gg_locate<MOE_GEMM_NT, BM>(p, s_loc, t)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l15 = lane & 15, g = lane >> 4;                   // fragment: position l15, bytes 16 g .. 16 g + 15 of 64
  const int c0 = t.nt * (EPI == EPI_SWIGLU ? 16 : 32);
  const int brows = EPI == EPI_SWIGLU ? 2 * p.N : p.N;
  const int64_t row_bytes = static_cast<int64_t>(p.K) * 2;
  const int64_t row0 = t.row0 + t.m_off;
  const bool two = t.m_n > 16;
  const uint8_t *a[2], *b[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    a[i] = static_cast<const uint8_t*>(p.A) + (row0 + min(i * 16 + l15, t.m_n - 1)) * row_bytes + g * 16;
    const int col = EPI == EPI_SWIGLU ? min(c0 + l15, p.N - 1) + i * p.N : min(c0 + i * 16 + l15, p.N - 1);
    b[i] = static_cast<const uint8_t*>(p.B) + (static_cast<int64_t>(t.e) * brows + col) * row_bytes + g * 16;
  }
  // the scales of what this wave will finish: subtile (wave >> 1, wave & 1)
  const int fi = wave >> 1 & 1, fj = wave & 1, in = fi * 16 + l15;
  const int col = c0 + (EPI == EPI_SWIGLU ? 0 : fj * 16) + g * 4;
  const float as = ip.as[row0 + min(in, t.m_n - 1)];
  const float* bs = ip.bs + static_cast<int64_t>(t.e) * brows + min(col, p.N - 4);
  const f32x4_t bs0 = *reinterpret_cast<const f32x4_t*>(bs);
  const f32x4_t bs1 = EPI == EPI_SWIGLU ? *reinterpret_cast<const f32x4_t*>(bs + p.N) : bs0;
  const i32x4_t zero = {0, 0, 0, 0};
  i32x4_t acc[2][2] = {{zero, zero}, {zero, zero}};
  const int lines = (static_cast<int>(row_bytes) + 127) / 128;
  for (int c = wave; c < lines; c += NW) {
    i32x4_t av[2][2], bv[2][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = c * 128 + h * 64;
      const bool there = k + g * 16 < row_bytes;              // K is a multiple of 16: a chunk or none
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        av[h][i] = there && (i == 0 || two) ? *reinterpret_cast<const i32x4_t*>(a[i] + k) : zero;
        bv[h][i] = there ? *reinterpret_cast<const i32x4_t*>(b[i] + k) : zero;
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          if (i == 0 || two) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(bv[h][j], av[h][i], acc[i][j], 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) red[wave][i * 2 + j][lane] = acc[i][j];
  __syncthreads();
  auto sum = [&](int q) {
    i32x4_t v = red[0][q][lane];
#pragma unroll
    for (int w = 1; w < NW; ++w) v += red[w][q][lane];
    return __builtin_convertvector(v, f32x4_t);
  };
  if (wave >= 4 || in >= t.m_n || col >= p.N) return;
  f32x4_t v;
  if constexpr (EPI == EPI_SWIGLU) {
    if (fj) return;
    const f32x4_t gate = sum(fi * 2) * as * bs0, up = sum(fi * 2 + 1) * as * bs1;
#pragma unroll
    for (int x = 0; x < 4; ++x) v[x] = silu(gate[x]) * up[x];
  } else {
    v = sum(wave) * as * bs0;
  }
  const int64_t at = (row0 + in) * p.N + col;
  if constexpr (F32)
    *reinterpret_cast<f32x4_t*>(static_cast<float*>(p.C) + at) = v;
  else
    *reinterpret_cast<uint2*>(static_cast<bf16_t*>(p.C) + at) = make_uint2(cvt_bf16x2(v[0], v[1]), cvt_bf16x2(v[2], v[3]));
}

// ---- host -----------------------------------------------------------------------

// Tiles, from the sizes alone; us on both sides of each border (N x K, uniform rows):
//   32 x 32 outputs a workgroup up to 384 of them: 8 rows of 4 experts, 2048 -> 2 x 1408
//   (352) 8.7 against 9.6, 128 dense rows x 2048 x 2048 (256) 7.0 / 9.8; 192 rows (384)
//   10.6 / 9.9, 256 rows (512) 10.7 / 10.0, 400 rows 17.9 / 10.1.
//   32 x 128 for up to 32 rows an expert, and while their grid is no more than what
//   runs at once: 512 rows x 2048 x 2048 9.8 against 14.9 with 128 x 128, 1024 rows
//   12.7 / 15.5, 2048 rows 22.4 / 16.8; 451 rows of 8 experts x 784 x 1504 8.4 / 12.0.
//   256 x 256 where there are more than 192 of them, from 129 rows an expert on: 64
//   experts x 2048 x 1408, 136 rows each 48 against 53, 192 rows 52 / 56, 256 rows 62 / 72,
//   290 rows 90 / 94, 512 rows 116 / 150; of 128 rows 46 / 41.  With rows drawn at random,
//   so that half of the experts need a second, short tile, 256 rows 78 / 81; Zipf (1.2)
//   256 rows 91 / 81, 562 rows 154 / 170.  Dense, 2048 wide: 192 tiles 35 / 35, 196 tiles
//   35 / 40, 112 tiles 33 / 25.
//   (64 x 128 lies between its neighbours; 256 x 256 and 128 x 128 in four half stages
//   are 5 to 15 % slower: rows of 64 bytes come to LDS at 15 TB/s, of 128 at 25.)
template <int EPI>
static moe_status launch_int8(I8Params& p, hipStream_t s) {
  const int64_t cap = p.g.cap, rows = cap / p.g.E;
  const bool dense = !p.g.offsets;
  auto tiles = [&](int BM, int BN) {                 // at most, whatever the experts' rows
    const int64_t width = EPI == EPI_SWIGLU ? BN / 2 : BN;
    const int64_t some = dense ? 0 : std::min<int64_t>(p.g.E, cap);    // experts with rows, at most
    return (some + (cap - some + (dense ? BM - 1 : 0)) / BM) * ((p.g.N + width - 1) / width);
  };
  int BM = 128, BN = 128;
  if (tiles(32, 32) <= 384)
    BM = BN = 32;
  else if (rows <= 32 || tiles(32, 128) <= 512)
    BM = 32;
  else if (rows > 128 && tiles(256, 256) > 192)
    BM = BN = 256;
  const int width = EPI == EPI_SWIGLU ? BN / 2 : BN;
  p.g.n_tiles = (p.g.N + width - 1) / width;
  p.g.splits = 1;
  const int64_t n = gemm_grid(tiles(BM, BN));
  if (n >= (1 << 23)) return MOE_ERR_UNSUPPORTED;      // at most 512 threads each, 2^32 in a grid
  const dim3 grid(static_cast<unsigned>(n));
  auto go = [&](auto kernel, int threads, int per_cu) {
    const int64_t most = 256 * per_cu;               // what runs at once
    hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(n < most ? n : most)), dim3(threads), 0, s, p);
  };
  auto pick = [&](auto f32) {
    constexpr bool F32 = decltype(f32)::value;
    if (BM == 256)
      go(k_grouped_int8<EPI, F32, 256, 256, 2, 4, 2>, 512, 1);
    else if (BN == 32)
      go(k_grouped_int8_few<EPI, F32>, 512, 1 << 20);
    else if (BM == 128)
      go(k_grouped_int8<EPI, F32, 128, 128, 2, 2, 2>, 256, 2);
    else
      go(k_grouped_int8<EPI, F32, 32, 128, 1, 4, 3>, 256, 2);
  };
  if (p.g.c_f32)
    pick(std::true_type{});
  else
    pick(std::false_type{});
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
