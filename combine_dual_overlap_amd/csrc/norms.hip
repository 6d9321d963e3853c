// Norms before and after the layer, with its gate, scale and residual, and their
// gradients, for gfx950.
//   r(v) = 1 / sqrt(mean(v^2) + eps)
//   before   n   = x r(x) w
//   after    out = res + scale * g * (y r(y) w_post)      and, in the same pass, the
//            next layer's n = out r(out) w_next
// y is a tensor, or the combine's weighted sum of expert rows, which then never
// leaves the registers (unless the backward pass needs it).  Everything is fp32
// between loading a row and the one rounding of each output; out's rounding is not
// in what follows from it in the same pass.
// HBM-bound: each row is read once into registers and written once.  8192 tokens x 8
// rows of 2048 bf16 combined, normed and normed again 67 us (5.5 TB/s); gradients of
// 8192 x 2048 22 us (4.7 TB/s) and 3 for the columns' sums, of 2047 x 7168 25 and 4.
#include "rows.h"

namespace dbomoe {

static_assert(kRowMaxBytes <= kRowMaxChunks * 16, "rows in registers");

struct NormOutParams {
  const u32x4_t* y;            // [T] rows, or the dispatched rows (GATHER)
  const int32_t* inv;          // GATHER: [T k]
  const float* topk_w;         // GATHER: [T, k]
  const u32x4_t* shared;       // GATHER: n_shared slabs of [T] rows, weight 1, or NULL
  int k, n_shared;
  int64_t T;
  int rc;                      // 16-byte chunks of a row
  float inv_h, eps, scale;
  const u32x4_t* res;          // NULL: no residual
  const u32x4_t* post_w;       // NULL: no norm
  const void* gate;
  int gate_kind;
  const u32x4_t* next_w;       // NULL: no next norm
  u32x4_t* out;
  u32x4_t* y_out;              // GATHER: y rounded, or NULL
  float* rstd;
  u32x4_t* next_n;
  float* next_rstd;
};

// The sum of a token's expert rows and shared rows, four rows' loads in flight.
template <bool BF16, int W, int CH, bool STREAM>
__device__ __forceinline__ void gather_sum(const NormOutParams& p, int64_t t, int l,
                                           float (&v)[CH][Chunk<BF16>::N]) {
  constexpr int N = Chunk<BF16>::N, G = CH == 1 ? 8 : 4;
  const int lane = threadIdx.x & 63;
  const int my_pos = lane < p.k ? p.inv[t * p.k + lane] : -1;
  const float my_w = lane < p.k ? p.topk_w[t * p.k + lane] : 0.f;
#pragma unroll
  for (int i = 0; i < CH; ++i)
#pragma unroll
    for (int e = 0; e < N; ++e) v[i][e] = 0.f;
  const int rows = p.k + p.n_shared;
  for (int j0 = 0; j0 < rows; j0 += G) {
    u32x4_t c[G][CH];
    float w[G];
    unsigned used = 0;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int j = j0 + g;
      const int pos = __builtin_amdgcn_readfirstlane(__shfl(my_pos, j < p.k ? j : 0, kWave));
      w[g] = __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(__shfl(my_w, j < p.k ? j : 0, kWave))));
      const u32x4_t* src = nullptr;
      if (j < p.k) {
        if (pos >= 0) src = p.y + static_cast<int64_t>(pos) * p.rc;
      } else if (j < rows) {
        src = p.shared + (static_cast<int64_t>(j - p.k) * p.T + t) * p.rc;
        w[g] = 1.f;
      }
      if (src) {
        used |= 1u << g;
#pragma unroll
        for (int i = 0; i < CH; ++i)
          if (i * 64 * W + l < p.rc) c[g][i] = load_chunk<STREAM>(src + i * 64 * W + l);
      }
    }
#pragma unroll
    for (int g = 0; g < G; ++g) {
      if (!(used & (1u << g))) continue;
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        if (i * 64 * W + l >= p.rc) continue;
        float f[N];
        Chunk<BF16>::unpack(c[g][i], f);
#pragma unroll
        for (int e = 0; e < N; ++e) v[i][e] += w[g] * f[e];
      }
    }
  }
}

template <bool BF16, int W, int CH, bool GATHER, bool STREAM>
__global__ __launch_bounds__(RowShape<W>::THREADS) void k_norm_out(NormOutParams p) {
  constexpr int N = Chunk<BF16>::N;
  using C = Chunk<BF16>;
  __shared__ float s_one[W], s_two[W];
  const int l = W == 1 ? threadIdx.x & 63 : threadIdx.x;
  auto at = [&](int i) { return i * 64 * W + l; };
  const int64_t first = static_cast<int64_t>(blockIdx.x) * RowShape<W>::ROWS + (W == 1 ? threadIdx.x >> 6 : 0);
  for (int64_t t = first; t < p.T; t += static_cast<int64_t>(gridDim.x) * RowShape<W>::ROWS) {
    float v[CH][N];
    if constexpr (GATHER) {
      gather_sum<BF16, W, CH, STREAM>(p, t, l, v);
    } else {
#pragma unroll
      for (int i = 0; i < CH; ++i)
        C::unpack(at(i) < p.rc ? load_chunk<STREAM>(p.y + t * p.rc + at(i)) : u32x4_t{0, 0, 0, 0}, v[i]);
    }
    if constexpr (GATHER) {
      if (p.y_out)
#pragma unroll
        for (int i = 0; i < CH; ++i)
          if (at(i) < p.rc) p.y_out[t * p.rc + at(i)] = C::pack(v[i]);
    }
    // what the outputs need besides y, asked for before the sum over the row
    u32x4_t res[CH], pw[CH], gt[CH], nw[CH];
    const u32x4_t* gate = static_cast<const u32x4_t*>(p.gate);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      if (at(i) >= p.rc) continue;
      if (p.res) res[i] = load_chunk<STREAM>(p.res + t * p.rc + at(i));
      if (p.post_w) pw[i] = p.post_w[at(i)];
      if (p.gate_kind == MOE_GATE_CHANNEL) gt[i] = gate[at(i)];
      if (p.gate_kind == MOE_GATE_FULL) gt[i] = gate[t * p.rc + at(i)];
      if (p.next_w) nw[i] = p.next_w[at(i)];
    }
    float a = p.scale;
    if (p.gate_kind == MOE_GATE_TOKEN) a *= static_cast<const float*>(p.gate)[t];
    if (p.post_w) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < CH; ++i)
#pragma unroll
        for (int e = 0; e < N; ++e) ss = fmaf(v[i][e], v[i][e], ss);
      const float r = 1.0f / sqrtf(row_sum<W>(ss, s_one) * p.inv_h + p.eps);
      if (p.rstd && l == 0) p.rstd[t] = r;
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        if (at(i) >= p.rc) continue;
        float w[N];
        C::unpack(pw[i], w);
#pragma unroll
        for (int e = 0; e < N; ++e) v[i][e] = v[i][e] * r * w[e];
      }
    }
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      if (at(i) >= p.rc) continue;
      if (p.gate_kind == MOE_GATE_CHANNEL || p.gate_kind == MOE_GATE_FULL) {
        float g[N];
        C::unpack(gt[i], g);
#pragma unroll
        for (int e = 0; e < N; ++e) v[i][e] *= g[e];
      }
      float f[N];
      if (p.res) {
        C::unpack(res[i], f);
      } else {
#pragma unroll
        for (int e = 0; e < N; ++e) f[e] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < N; ++e) {
        v[i][e] = fmaf(a, v[i][e], f[e]);
        ss = fmaf(v[i][e], v[i][e], ss);
      }
      if (p.out) p.out[t * p.rc + at(i)] = C::pack(v[i]);
    }
    if (p.next_w) {
      const float r = 1.0f / sqrtf(row_sum<W>(ss, s_two) * p.inv_h + p.eps);
      if (p.next_rstd && l == 0) p.next_rstd[t] = r;
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        if (at(i) >= p.rc) continue;
        float w[N];
        C::unpack(nw[i], w);
#pragma unroll
        for (int e = 0; e < N; ++e) w[e] *= v[i][e] * r;
        p.next_n[t * p.rc + at(i)] = C::pack(w);
      }
    }
    if constexpr (W > 1) __syncthreads();                     // the exchanges read by all before the next row's
  }
}

// Rows are read past the caches where there are more than kStreamBytes of them: k = 8,
// 8192 x 2048 76 -> 70 us, 2048 x 7168 80 -> 65; 2048 x 2048 (67 MB) 19 either way.
constexpr int64_t kStreamBytes = int64_t{64} << 20;

// Rows of 256 chunks are spread over four waves: 8192 x 2048, k = 8, with one wave
// (217 registers) 89 us, with four 76; without a combine 31 and 26.  Rows of 128 the
// other way round: 4096 x 1024, k = 8, 18 and 21.
static moe_status launch_norm_out(const NormOutParams& p, bool bf16, bool gather, hipStream_t s, int max_blocks = 0) {
  if (p.T == 0) return MOE_OK;
  const bool stream = p.T * (gather ? p.k + p.n_shared : 1) * p.rc * 16 > kStreamBytes;
  with_row_shape(p.T, p.rc, 128, [&](auto w, auto ch) {
    constexpr int W = decltype(w)::value, CH = decltype(ch)::value;
    int64_t blocks = (p.T + RowShape<W>::ROWS - 1) / RowShape<W>::ROWS;
    if (max_blocks > 0 && blocks > max_blocks) blocks = max_blocks;
    const dim3 grid(static_cast<unsigned>(blocks));
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(RowShape<W>::THREADS), 0, s, p); };
    auto of = [&](auto b, auto g) {
      constexpr bool B = decltype(b)::value, G = decltype(g)::value;
      stream ? go(k_norm_out<B, W, CH, G, true>) : go(k_norm_out<B, W, CH, G, false>);
    };
    if (bf16)
      gather ? of(std::true_type{}, std::true_type{}) : of(std::true_type{}, std::false_type{});
    else
      gather ? of(std::false_type{}, std::true_type{}) : of(std::false_type{}, std::false_type{});
  });
  DBOMOE_CHECK_LAUNCH();
  return MOE_OK;
}

// ---- gradients --------------------------------------------------------------------
// With yh = y r and the incoming gradient d (post: a = scale * dout, else a = d):
//   q  = a g w                      the gradient of yh
//   dy = r (q - yh mean(q yh)) + dres
//   dw = sum_t a g yh,  dg = a yh w (summed over what the gate is shared by)
// Without a norm w is 1, r is 1 and the mean is left out.  A gate per channel
// leaves one column sum for both: S_h = sum_t a yh, dw = g S, dg = w S.
// A workgroup walks rows gridDim.x apart with the column sums of its lanes in
// registers, leaves one row of partial sums, and k_norm_cols adds these in order.
struct NormBwdParams {
  const u32x4_t* d;
  const u32x4_t* y;
  int64_t T;
  int rc;
  float inv_h, scale;
  const float* rstd;           // NULL: no norm
  const u32x4_t* w;            // NULL: no norm
  const void* gate;
  int gate_kind;
  const u32x4_t* dres;         // or NULL
  u32x4_t* dy;
  void* dgate;                 // token: fp32 [T]; full: [T] rows; (channel: k_norm_cols)
  float* part;                 // [gridDim.x][H] or NULL
};

// Rows and weights stay packed as they were loaded and are taken apart twice (for
// the sums over the row, then for dy): fp32 copies of them would leave two waves to a
// SIMD.
template <bool BF16, int W, int CH, int GATE, bool STREAM>
__global__ __launch_bounds__(RowShape<W>::THREADS) void k_norm_bwd(NormBwdParams p) {
  constexpr int N = Chunk<BF16>::N, ROWS = RowShape<W>::ROWS;
  using C = Chunk<BF16>;
  __shared__ float s_one[W], s_two[W];
  __shared__ float s_col[W == 1 ? 4 * 64 * N : 1];
  const int l = W == 1 ? threadIdx.x & 63 : threadIdx.x;
  const int sub = W == 1 ? threadIdx.x >> 6 : 0;
  auto at = [&](int i) { return i * 64 * W + l; };
  const u32x4_t* gate = static_cast<const u32x4_t*>(p.gate);
  const uint32_t one = BF16 ? 0x3f803f80u : 0x3f800000u;
  u32x4_t w[CH], g[GATE == MOE_GATE_CHANNEL ? CH : 1];
  float col[CH][N];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const bool in = at(i) < p.rc;
    w[i] = in && p.w ? p.w[at(i)] : u32x4_t{one, one, one, one};
    if constexpr (GATE == MOE_GATE_CHANNEL) g[i] = in ? gate[at(i)] : u32x4_t{0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < N; ++e) col[i][e] = 0.f;
  }
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * ROWS + sub; t < p.T; t += static_cast<int64_t>(gridDim.x) * ROWS) {
    u32x4_t dv[CH], yv[CH], rv[CH], gv[GATE == MOE_GATE_FULL ? CH : 1];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      dv[i] = yv[i] = rv[i] = u32x4_t{0, 0, 0, 0};
      if constexpr (GATE == MOE_GATE_FULL) gv[i] = u32x4_t{0, 0, 0, 0};
      if (at(i) >= p.rc) continue;
      dv[i] = load_chunk<STREAM>(p.d + t * p.rc + at(i));
      yv[i] = load_chunk<STREAM>(p.y + t * p.rc + at(i));
      if (p.dres) rv[i] = load_chunk<STREAM>(p.dres + t * p.rc + at(i));
      if constexpr (GATE == MOE_GATE_FULL) gv[i] = gate[t * p.rc + at(i)];
    }
    const float r = p.rstd ? p.rstd[t] : 1.f;
    const float gt = GATE == MOE_GATE_TOKEN ? static_cast<const float*>(p.gate)[t] : 1.f;
    // of chunk i: a = scale d, yh, the weights and the gate
    auto take = [&](int i, float (&a)[N], float (&yh)[N], float (&wf)[N], float (&gf)[N]) {
      C::unpack(dv[i], a);
      C::unpack(yv[i], yh);
      C::unpack(w[i], wf);
      if constexpr (GATE == MOE_GATE_CHANNEL) C::unpack(g[i], gf);
      if constexpr (GATE == MOE_GATE_FULL) C::unpack(gv[i], gf);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        a[e] *= p.scale;
        yh[e] *= r;
        if constexpr (GATE == MOE_GATE_NONE || GATE == MOE_GATE_TOKEN) gf[e] = gt;
      }
    };
    float dot = 0.f, tok = 0.f;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      float a[N], yh[N], wf[N], gf[N];
      take(i, a, yh, wf, gf);
      if constexpr (GATE == MOE_GATE_FULL) {
        float dg[N];
#pragma unroll
        for (int e = 0; e < N; ++e) dg[e] = a[e] * yh[e] * wf[e];
        if (p.dgate && at(i) < p.rc) static_cast<u32x4_t*>(p.dgate)[t * p.rc + at(i)] = C::pack(dg);
      }
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float ay = a[e] * yh[e];
        // the column sums leave a channel's gate out
        col[i][e] = GATE == MOE_GATE_CHANNEL || GATE == MOE_GATE_NONE ? col[i][e] + ay : fmaf(gf[e], ay, col[i][e]);
        if constexpr (GATE == MOE_GATE_TOKEN) tok = fmaf(ay, wf[e], tok);
        dot = fmaf(ay, gf[e] * wf[e], dot);
      }
    }
    if constexpr (GATE == MOE_GATE_TOKEN) {
      tok = row_sum<W>(tok, s_one);
      if (p.dgate && l == 0) static_cast<float*>(p.dgate)[t] = tok;
    }
    float mean = 0.f;
    if (p.rstd) mean = row_sum<W>(dot, s_two) * p.inv_h;
    // (nothing that was taken apart above is kept)
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      asm volatile("" : "+v"(dv[i]), "+v"(yv[i]), "+v"(w[i]));
      if constexpr (GATE == MOE_GATE_CHANNEL) asm volatile("" : "+v"(g[i]));
      if constexpr (GATE == MOE_GATE_FULL) asm volatile("" : "+v"(gv[i]));
    }
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      if (at(i) >= p.rc) continue;
      float a[N], yh[N], wf[N], gf[N], f[N];
      take(i, a, yh, wf, gf);
      C::unpack(rv[i], f);
#pragma unroll
      for (int e = 0; e < N; ++e) f[e] = fmaf(r, a[e] * gf[e] * wf[e] - yh[e] * mean, f[e]);
      p.dy[t * p.rc + at(i)] = C::pack(f);
    }
    if constexpr (W > 1) __syncthreads();                   // the exchanges read by all before the next row's
  }
  if (!p.part) return;
  float* mine = p.part + static_cast<int64_t>(blockIdx.x) * p.rc * N;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    if constexpr (W == 1) {                                 // the four rows' lanes hold the same columns
#pragma unroll
      for (int e = 0; e < N; ++e) s_col[(sub * 64 + l) * N + e] = col[i][e];
      __syncthreads();
      for (int x = threadIdx.x; x < 64 * N; x += 256) {
        const int c = i * 64 * N + x;
        if (c < p.rc * N) mine[c] = ((s_col[x] + s_col[64 * N + x]) + s_col[128 * N + x]) + s_col[192 * N + x];
      }
      __syncthreads();
    } else if (at(i) < p.rc) {
#pragma unroll
      for (int e = 0; e < N; ++e) mine[at(i) * N + e] = col[i][e];
    }
  }
}

// Column sums of the partial rows: S_h; dw = S g (g per channel, else 1), dgate = S w.
// 32 columns by 32 parts of the rows in a workgroup, eight rows' loads in flight (16 by 64:
// 2047 x 7168 31.3 us in all, not 29.1).
constexpr int kColWidth = 32, kColParts = 32;
template <bool BF16>
__global__ __launch_bounds__(kColWidth * kColParts) void k_norm_cols(const float* __restrict__ part, int rows, int H,
                                                                     const void* __restrict__ w,
                                                                     const void* __restrict__ gate,
                                                                     float* __restrict__ dw, float* __restrict__ dgate,
                                                                     int accumulate) {
  __shared__ float s[kColParts][kColWidth + 1];
  const int x = threadIdx.x % kColWidth, y = threadIdx.x / kColWidth, h = blockIdx.x * kColWidth + x;
  float v = 0.f;
  if (h < H) {
    for (int r0 = y; r0 < rows; r0 += 8 * kColParts) {
      float f[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int r = r0 + u * kColParts;
        f[u] = r < rows ? part[static_cast<int64_t>(r) * H + h] : 0.f;
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) v += f[u];
    }
  }
  s[y][x] = v;
  __syncthreads();
  for (int n = kColParts / 2; n > 0; n /= 2) {
    if (y < n) s[y][x] += s[y + n][x];
    __syncthreads();
  }
  if (y != 0 || h >= H) return;
  v = s[0][x];
  auto get = [&](const void* p) {
    return p == nullptr ? 1.f : BF16 ? bf16_to_f32(static_cast<const bf16_t*>(p)[h]) : static_cast<const float*>(p)[h];
  };
  if (dw) dw[h] = (accumulate ? dw[h] : 0.f) + v * get(gate);
  if (dgate) dgate[h] = (accumulate ? dgate[h] : 0.f) + v * get(w);
}

// A workgroup is one row of parts.  Few rows have a workgroup each (64 x 7168 11.9 -> 7.4 us,
// 256 x 2048 7.4 -> 6.2), up to 256; 512 x 7168 with 128, 256 and 512: 16.0, 14.6 and 16.7.
static int64_t norm_bwd_blocks(int64_t T) {
  return std::max<int64_t>(std::min<int64_t>((T + 3) / 4, 512), std::min<int64_t>(T, 256));
}

static moe_status launch_norm_bwd(NormBwdParams& p, bool bf16, int32_t H, float* dw, float* dgate_cols, bool accumulate,
                                  void* ws, hipStream_t s) {
  const bool cols = dw || dgate_cols;
  const int blocks = static_cast<int>(cols ? norm_bwd_blocks(p.T) : std::min<int64_t>(p.T, 512));
  p.part = cols ? static_cast<float*>(ws) : nullptr;
  if (p.T > 0) {
    // past the caches (see kStreamBytes) from 24 MB an operand on: 16384 x 2048 41 -> 37 us,
    // 2047 x 7168 with a residual 26.9 -> 24.7; 4096 x 2048 (17 MB) 13.5 -> 14.0
    const bool stream = p.T * p.rc * 16 > (int64_t{24} << 20);
    // (8192 rows of 256 chunks: 22.5 us with one wave each, 27.6 with four)
    with_row_shape(p.T, p.rc, 256, [&](auto w, auto ch) {
      constexpr int W = decltype(w)::value, CH = decltype(ch)::value;
      auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3(blocks), dim3(RowShape<W>::THREADS), 0, s, p); };
      auto of_gate = [&](auto gate) {
        constexpr int GATE = decltype(gate)::value;
        if (bf16)
          stream ? go(k_norm_bwd<true, W, CH, GATE, true>) : go(k_norm_bwd<true, W, CH, GATE, false>);
        else
          stream ? go(k_norm_bwd<false, W, CH, GATE, true>) : go(k_norm_bwd<false, W, CH, GATE, false>);
      };
      switch (p.gate_kind) {
        case MOE_GATE_CHANNEL: of_gate(std::integral_constant<int, MOE_GATE_CHANNEL>{}); break;
        case MOE_GATE_TOKEN: of_gate(std::integral_constant<int, MOE_GATE_TOKEN>{}); break;
        case MOE_GATE_FULL: of_gate(std::integral_constant<int, MOE_GATE_FULL>{}); break;
        default: of_gate(std::integral_constant<int, MOE_GATE_NONE>{});
      }
    });
    DBOMOE_CHECK_LAUNCH();
  }
  if (cols && !(p.T == 0 && accumulate)) {
    const void* gate = p.gate_kind == MOE_GATE_CHANNEL ? p.gate : nullptr;
    auto go = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>((H + kColWidth - 1) / kColWidth)),
                         dim3(kColWidth * kColParts), 0, s, p.part,
                         p.T > 0 ? blocks : 0, H, static_cast<const void*>(p.w), gate, dw, dgate_cols, accumulate ? 1 : 0);
    };
    bf16 ? go(k_norm_cols<true>) : go(k_norm_cols<false>);
    DBOMOE_CHECK_LAUNCH();
  }
  return MOE_OK;
}

// ---- checks -----------------------------------------------------------------------

static moe_status norm_check_sizes(moe_dtype act, int64_t T, int32_t H) {
  if (T < 0 || H <= 0) return MOE_ERR_INVALID_ARG;
  if (act != MOE_F32 && act != MOE_BF16) return MOE_ERR_UNSUPPORTED;
  const int64_t bytes = static_cast<int64_t>(H) * dtype_size(act);
  if (bytes % 16) return MOE_ERR_MISALIGNED;
  if (bytes > kRowMaxBytes) return MOE_ERR_UNSUPPORTED;
  if (T >= (int64_t{1} << 22)) return MOE_ERR_UNSUPPORTED;          // 1024 threads a row, 2^32 in a grid
  return MOE_OK;
}

moe_status check_post_norm(const moe_post_norm_params* q) {
  if (!q) return MOE_ERR_INVALID_ARG;
  if (q->gate_kind < MOE_GATE_NONE || q->gate_kind > MOE_GATE_FULL) return MOE_ERR_INVALID_ARG;
  if ((q->gate_kind == MOE_GATE_NONE) != (q->gate == nullptr)) return MOE_ERR_INVALID_ARG;
  if (!(q->eps > 0.f) || !(q->eps <= 3.4e38f) || !(q->scale >= -3.4e38f && q->scale <= 3.4e38f)) return MOE_ERR_INVALID_ARG;
  if (!aligned16(q->post_w) || !aligned16(q->gate) || !aligned16(q->next_w)) return MOE_ERR_MISALIGNED;
  return MOE_OK;
}

static NormOutParams norm_out_params(const moe_post_norm_params& q, int64_t T, int32_t H, moe_dtype act) {
  NormOutParams p{};
  p.T = T;
  p.rc = static_cast<int>(static_cast<int64_t>(H) * dtype_size(act) / 16);
  p.inv_h = 1.0f / static_cast<float>(H);
  p.eps = q.eps;
  p.scale = q.scale;
  p.post_w = static_cast<const u32x4_t*>(q.post_w);
  p.gate = q.gate;
  p.gate_kind = q.gate_kind;
  p.next_w = static_cast<const u32x4_t*>(q.next_w);
  return p;
}

moe_status launch_pre_norm(const void* x, moe_dtype act, int64_t T, int32_t H, const void* w, float eps, void* n,
                           float* rstd, hipStream_t s) {
  // n = x r(x) w: what follows the residual sum, with x as that sum
  moe_post_norm_params q{};
  q.eps = eps;
  q.scale = 1.f;
  q.next_w = w;
  NormOutParams p = norm_out_params(q, T, H, act);
  p.y = static_cast<const u32x4_t*>(x);
  p.next_n = static_cast<u32x4_t*>(n);
  p.next_rstd = rstd;
  return launch_norm_out(p, act == MOE_BF16, false, s);
}

moe_status launch_combine_post_norm(const CombineArgs& a, const void* res, const moe_post_norm_params& q, void* y_out,
                                    float* rstd, void* next_n, float* next_rstd, hipStream_t s) {
  NormOutParams p = norm_out_params(q, a.T, a.H, a.act);
  p.y = static_cast<const u32x4_t*>(a.y);
  p.inv = a.inv;
  p.topk_w = a.w;
  p.shared = static_cast<const u32x4_t*>(a.shared);
  p.k = a.k;
  p.n_shared = a.shared ? std::max(a.n_shared, 1) : 0;
  p.res = static_cast<const u32x4_t*>(res);
  p.out = static_cast<u32x4_t*>(a.out);
  p.y_out = static_cast<u32x4_t*>(y_out);
  p.rstd = rstd;
  p.next_n = static_cast<u32x4_t*>(next_n);
  p.next_rstd = next_rstd;
  return launch_norm_out(p, a.act == MOE_BF16, true, s, a.max_blocks);
}

}  // namespace dbomoe

using namespace dbomoe;

extern "C" moe_status moe_pre_norm(const void* x, moe_dtype act, int64_t T, int32_t H, const void* w, float eps, void* n,
                                   float* rstd, void* stream) {
  const moe_status st = norm_check_sizes(act, T, H);
  if (st != MOE_OK) return st;
  if (!(eps > 0.f) || !(eps <= 3.4e38f)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!x || !w || !n || n == w) return MOE_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(w) || !aligned16(n) || !aligned16(rstd)) return MOE_ERR_MISALIGNED;
  return launch_pre_norm(x, act, T, H, w, eps, n, rstd, as_stream(stream));
}

// What moe_post_norm and moe_combine_post_norm share.
static moe_status post_norm_check(const void* y, moe_dtype act, int64_t T, int32_t H, const void* res,
                                  const moe_post_norm_params* q, const void* out, const void* next_n, const float* rstd,
                                  const float* next_rstd) {
  moe_status st = norm_check_sizes(act, T, H);
  if (st != MOE_OK) return st;
  st = check_post_norm(q);
  if (st != MOE_OK) return st;
  if ((q->next_w == nullptr) != (next_n == nullptr)) return MOE_ERR_INVALID_ARG;
  if ((rstd && !q->post_w) || (next_rstd && !q->next_w)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!y || !out) return MOE_ERR_INVALID_ARG;
  if (out == y || out == q->gate || out == q->post_w || out == q->next_w || out == next_n) return MOE_ERR_INVALID_ARG;
  if (next_n && (next_n == y || next_n == res || next_n == q->gate || next_n == q->post_w || next_n == q->next_w))
    return MOE_ERR_INVALID_ARG;
  if (!aligned16(y) || !aligned16(res) || !aligned16(out) || !aligned16(next_n) || !aligned16(rstd) ||
      !aligned16(next_rstd))
    return MOE_ERR_MISALIGNED;
  return MOE_OK;
}

extern "C" moe_status moe_post_norm(const void* y, moe_dtype act, int64_t T, int32_t H, const void* res,
                                    const moe_post_norm_params* params, void* out, float* rstd, void* next_n,
                                    float* next_rstd, void* stream) {
  const moe_status st = post_norm_check(y, act, T, H, res, params, out, next_n, rstd, next_rstd);
  if (st != MOE_OK || T == 0) return st;
  NormOutParams p = norm_out_params(*params, T, H, act);
  p.y = static_cast<const u32x4_t*>(y);
  p.res = static_cast<const u32x4_t*>(res);
  p.out = static_cast<u32x4_t*>(out);
  p.rstd = rstd;
  p.next_n = static_cast<u32x4_t*>(next_n);
  p.next_rstd = next_rstd;
  return launch_norm_out(p, act == MOE_BF16, false, as_stream(stream));
}

extern "C" moe_status moe_combine_post_norm(const void* y_perm, moe_dtype act, int64_t T, int32_t H, int32_t k,
                                            const int32_t* inv, const float* topk_w, const void* shared_out,
                                            const void* res, const moe_post_norm_params* params, void* out, void* y_out,
                                            float* rstd, void* next_n, float* next_rstd, void* stream) {
  if (k < 1 || k > 16) return MOE_ERR_INVALID_ARG;
  const moe_status st = post_norm_check(y_perm, act, T, H, res, params, out, next_n, rstd, next_rstd);
  if (st != MOE_OK || T == 0) return st;
  if (!inv || !topk_w) return MOE_ERR_INVALID_ARG;
  if (shared_out && (out == shared_out || next_n == shared_out)) return MOE_ERR_INVALID_ARG;
  if (y_out && (y_out == y_perm || y_out == shared_out || y_out == res || y_out == out || y_out == next_n ||
                y_out == params->gate || y_out == params->post_w || y_out == params->next_w))
    return MOE_ERR_INVALID_ARG;
  if (!aligned16(inv) || !aligned16(topk_w) || !aligned16(shared_out) || !aligned16(y_out)) return MOE_ERR_MISALIGNED;
  CombineArgs a{y_perm, act, T, H, k, inv, topk_w, shared_out, out, 0, shared_out ? 1 : 0};
  return launch_combine_post_norm(a, res, *params, y_out, rstd, next_n, next_rstd, as_stream(stream));
}

extern "C" size_t moe_norm_backward_workspace_size(int64_t T, int32_t H) {
  if (T <= 0 || H <= 0) return 0;
  return align_up(static_cast<size_t>(norm_bwd_blocks(T)) * H * sizeof(float), 256);
}

extern "C" moe_status moe_pre_norm_backward(const void* dn, const void* x, moe_dtype act, int64_t T, int32_t H,
                                            const float* rstd, const void* w, const void* dres, void* dx, float* dw,
                                            int32_t accumulate, void* ws, size_t ws_bytes, void* stream) {
  const moe_status st = norm_check_sizes(act, T, H);
  if (st != MOE_OK) return st;
  if (accumulate != 0 && accumulate != 1) return MOE_ERR_INVALID_ARG;
  if (!w) return MOE_ERR_INVALID_ARG;
  if (T > 0 && (!dn || !x || !rstd || !dx)) return MOE_ERR_INVALID_ARG;
  if (T > 0 && (dx == x || dx == w || static_cast<const void*>(rstd) == dx || static_cast<void*>(dw) == dx))
    return MOE_ERR_INVALID_ARG;
  if (dw && (dw == w || dw == rstd || dw == dn || dw == x || dw == dres || dw == ws)) return MOE_ERR_INVALID_ARG;
  if (!aligned16(dn) || !aligned16(x) || !aligned16(rstd) || !aligned16(w) || !aligned16(dres) || !aligned16(dx) ||
      !aligned16(dw) || !aligned256(ws))
    return MOE_ERR_MISALIGNED;
  if (dw && T > 0 && !ws) return MOE_ERR_INVALID_ARG;
  if (dw && ws_bytes < moe_norm_backward_workspace_size(T, H)) return MOE_ERR_WORKSPACE;
  NormBwdParams p{};
  p.d = static_cast<const u32x4_t*>(dn);
  p.y = static_cast<const u32x4_t*>(x);
  p.T = T;
  p.rc = static_cast<int>(static_cast<int64_t>(H) * dtype_size(act) / 16);
  p.inv_h = 1.0f / static_cast<float>(H);
  p.scale = 1.f;
  p.rstd = rstd;
  p.w = static_cast<const u32x4_t*>(w);
  p.dres = static_cast<const u32x4_t*>(dres);
  p.dy = static_cast<u32x4_t*>(dx);
  return launch_norm_bwd(p, act == MOE_BF16, H, dw, nullptr, accumulate != 0, ws, as_stream(stream));
}

extern "C" moe_status moe_post_norm_backward(const void* dout, const void* y, moe_dtype act, int64_t T, int32_t H,
                                             const float* rstd, const moe_post_norm_params* params, void* dy,
                                             float* dpost_w, void* dgate, int32_t accumulate, void* ws, size_t ws_bytes,
                                             void* stream) {
  moe_status st = norm_check_sizes(act, T, H);
  if (st != MOE_OK) return st;
  st = check_post_norm(params);
  if (st != MOE_OK) return st;
  if (accumulate != 0 && accumulate != 1) return MOE_ERR_INVALID_ARG;
  if ((dpost_w && !params->post_w) || (dgate && !params->gate)) return MOE_ERR_INVALID_ARG;
  if (T > 0 && (!dout || !y || !dy || (params->post_w == nullptr) != (rstd == nullptr))) return MOE_ERR_INVALID_ARG;
  if (T > 0 && (dy == y || dy == params->post_w || dy == params->gate || static_cast<const void*>(rstd) == dy ||
                static_cast<void*>(dpost_w) == dy || dgate == dy))
    return MOE_ERR_INVALID_ARG;
  for (void* o : {static_cast<void*>(dpost_w), dgate})
    if (o && (o == params->post_w || o == params->gate || o == rstd || o == dout || o == y || o == ws))
      return MOE_ERR_INVALID_ARG;
  if (dgate && dgate == static_cast<void*>(dpost_w)) return MOE_ERR_INVALID_ARG;
  if (!aligned16(dout) || !aligned16(y) || !aligned16(rstd) || !aligned16(dy) || !aligned16(dpost_w) ||
      !aligned16(dgate) || !aligned256(ws))
    return MOE_ERR_MISALIGNED;
  const bool cols = dpost_w || (dgate && params->gate_kind == MOE_GATE_CHANNEL);
  if (cols && T > 0 && !ws) return MOE_ERR_INVALID_ARG;
  if (cols && ws_bytes < moe_norm_backward_workspace_size(T, H)) return MOE_ERR_WORKSPACE;
  NormBwdParams p{};
  p.d = static_cast<const u32x4_t*>(dout);
  p.y = static_cast<const u32x4_t*>(y);
  p.T = T;
  p.rc = static_cast<int>(static_cast<int64_t>(H) * dtype_size(act) / 16);
  p.inv_h = 1.0f / static_cast<float>(H);
  p.scale = params->scale;
  p.rstd = rstd;
  p.w = static_cast<const u32x4_t*>(params->post_w);
  p.gate = params->gate;
  p.gate_kind = params->gate_kind;
  p.dy = static_cast<u32x4_t*>(dy);
  const bool channel = params->gate_kind == MOE_GATE_CHANNEL;
  p.dgate = channel ? nullptr : dgate;
  return launch_norm_bwd(p, act == MOE_BF16, H, dpost_w, channel ? static_cast<float*>(dgate) : nullptr,
                         accumulate != 0, ws, as_stream(stream));
}
