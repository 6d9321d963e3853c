// Gradients of the combine and of the router's gate, for gfx950.
#include "common.h"

namespace dbomoe {

// ---- combine ----------------------------------------------------------------
// out[t] = sum_j w[t, j] y[inv[t, j]], so
//   dy[inv[t, j]] = w[t, j] dout[t]         (one rounding to act)
//   dw[t, j]      = <dout[t], y[inv[t, j]]>  (fp32; 0 for a pair without a row)
// HBM-bound: every dispatched row is read once and written once; dout rows are
// read by the waves of one token at about the same time, through L2.
// One wave per (token, slot) pair.  STREAM: rows that the caches need not keep
// (more of them than L2 holds): 8192 x 8 rows of 4 KB 120 -> 113 us (5.1 TB/s),
// 4096 x 1 rows of 14 KB 40 -> 34 us.
template <bool BF16, bool STREAM>
__global__ __launch_bounds__(256) void k_combine_bwd(const u32x4_t* __restrict__ dout, const u32x4_t* __restrict__ y,
                                                     int64_t pairs, int64_t cap, int rc, int k,
                                                     const int32_t* __restrict__ inv, const float* __restrict__ w,
                                                     u32x4_t* __restrict__ dy, float* __restrict__ dw) {
  const int lane = threadIdx.x & 63;
  const int64_t pr = static_cast<int64_t>(blockIdx.x) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (pr >= pairs) return;
  const int64_t pos = inv[pr];
  if (pos < 0 || pos >= cap) {
    if (lane == 0) dw[pr] = 0.f;
    return;
  }
  const float wj = w[pr];
  const u32x4_t* d = dout + pr / k * rc;
  const u32x4_t* yr = y + pos * rc;
  u32x4_t* o = dy + pos * rc;
  float s0 = 0.f, s1 = 0.f;
#pragma unroll 4
  for (int c = lane; c < rc; c += 64) {
    const u32x4_t a = d[c], b = STREAM ? __builtin_nontemporal_load(yr + c) : yr[c];
    u32x4_t r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (BF16) {
        const float a0 = __uint_as_float(a[i] << 16), a1 = __uint_as_float(a[i] & 0xffff0000u);
        s0 = fmaf(a0, __uint_as_float(b[i] << 16), s0);
        s1 = fmaf(a1, __uint_as_float(b[i] & 0xffff0000u), s1);
        r[i] = pack_bf16x2(wj * a0, wj * a1);
      } else {
        const float a0 = __uint_as_float(a[i]);
        s0 = fmaf(a0, __uint_as_float(b[i]), s0);
        r[i] = __float_as_uint(wj * a0);
      }
    }
    if constexpr (STREAM)
      __builtin_nontemporal_store(r, o + c);
    else
      o[c] = r;
  }
  const float s = wave_sum_f(s0 + s1);
  if (lane == 0) dw[pr] = s;
}

// ---- router gate --------------------------------------------------------------
// With d_j = routed_scale * dw[t, j] and p the scores (softmax over all E, or
// sigmoid), w_j = p[id_j], or p[id_j] / sum_i p[id_i] when renormalised:
//   softmax                dl_e = p_e (sum_{j: id_j = e} d_j - sum_j p[id_j] d_j)
//   softmax, renormalised  dl_e = sum_{j: id_j = e} w_j (d_j - sum_i w_i d_i)
//                          (the softmax's own sum cancels; only chosen experts)
//   sigmoid                dl_e = sum_{j: id_j = e} p (1 - p) d_j
//   sigmoid, renormalised  dl_e = sum_{j: id_j = e} (1 - p) w_j (d_j - sum_i w_i d_i)
// The selection itself has no gradient.  p is computed as the forward routing
// computes it; 1 - p is the sigmoid of -l, so it does not cancel.
// One wave per token; lane l holds experts l, l + 64, ..; slot j lives in lane j.
template <typename Out>
__global__ __launch_bounds__(256) void k_route_bwd(const float* __restrict__ logits, int64_t T,
                                                   const int32_t* __restrict__ ids, const float* __restrict__ dw,
                                                   moe_route_params rp, Out* __restrict__ dl) {
  const int lane = threadIdx.x & 63;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (t >= T) return;
  const int E = rp.E, k = rp.k;
  const float* row = logits + t * E;
  int id = -1;
  float d = 0.f;
  if (lane < k) {
    id = ids[t * k + lane];
    if (id < 0 || id >= E) id = -1;          // such a slot's weight is the constant 0
    if (id >= 0) d = dw[t * k + lane] * rp.routed_scale;
  }
  const float mine = id >= 0 ? row[id] : -INFINITY;
  const bool softmax = rp.score == MOE_SCORE_SOFTMAX;
  float p4[4] = {0.f, 0.f, 0.f, 0.f};
  float p = 0.f, slope = 1.f;               // the slot's score; for sigmoid its 1 - p
  bool dead = false;                        // no expert has a finite logit
  if (softmax) {
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = lane + 64 * i < E ? row[lane + 64 * i] : -INFINITY;
    const float lmax = wave_max_f(fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])));
    dead = lmax == -INFINITY;
    float denom = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      p4[i] = lane + 64 * i < E ? expf(v[i] - lmax) : 0.f;
      denom += p4[i];
    }
    denom = wave_sum_f(denom);
#pragma unroll
    for (int i = 0; i < 4; ++i) p4[i] /= denom;
    if (id >= 0) p = expf(mine - lmax) / denom;
  } else if (id >= 0) {
    p = 1.0f / (1.0f + expf(-mine));
    slope = 1.0f / (1.0f + expf(mine));
  }
  const float wsum = wave_sum_f(lane < k ? p : 0.f);
  const bool renorm = rp.renormalize != 0 && wsum > 0.f;
  const float w = renorm ? p / wsum : p;
  const float dot = wave_sum_f(lane < k && id >= 0 ? w * d : 0.f);
  // c: what the slot adds to its expert's gradient (softmax: before the factor p_e)
  float c;
  if (renorm)
    c = w * (d - dot) * slope;
  else
    c = softmax ? d : p * slope * d;
  if (id < 0) c = 0.f;
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
  for (int j = 0; j < k; ++j) {
    const int ej = __shfl(id, j, kWave);
    const float cj = __shfl(c, j, kWave);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (ej == lane + 64 * i) acc[i] += cj;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = lane + 64 * i;
    if (e >= E) continue;
    float g = acc[i];
    if (softmax && !renorm) g = p4[i] * (acc[i] - dot);
    if (dead) g = 0.f;
    if constexpr (sizeof(Out) == 2)
      dl[t * E + e] = f32_to_bf16(g);
    else
      dl[t * E + e] = g;
  }
}

}  // namespace dbomoe

using namespace dbomoe;

extern "C" moe_status moe_combine_backward(const void* dout, const void* y_perm, moe_dtype act, int64_t T, int32_t H,
                                           int32_t k, int64_t cap_rows, const int32_t* inv, const float* topk_w,
                                           void* dy_perm, float* dtopk_w, void* stream) {
  if (T < 0 || H <= 0 || k < 1 || k > 16 || cap_rows < 0) return MOE_ERR_INVALID_ARG;
  if (act != MOE_F32 && act != MOE_BF16) return MOE_ERR_UNSUPPORTED;
  if (T >= (int64_t{1} << 26) / k) return MOE_ERR_UNSUPPORTED;      // 64 threads a pair, 2^32 in a grid
  if (T == 0) return MOE_OK;
  if (!dout || !inv || !topk_w || !dtopk_w || (cap_rows > 0 && (!y_perm || !dy_perm))) return MOE_ERR_INVALID_ARG;
  if (cap_rows > 0 && (dy_perm == y_perm || dy_perm == dout)) return MOE_ERR_INVALID_ARG;
  if (dtopk_w == topk_w) return MOE_ERR_INVALID_ARG;
  if ((static_cast<int64_t>(H) * dtype_size(act)) % 16) return MOE_ERR_MISALIGNED;
  if (!aligned16(dout) || !aligned16(y_perm) || !aligned16(inv) || !aligned16(topk_w) || !aligned16(dy_perm) ||
      !aligned16(dtopk_w))
    return MOE_ERR_MISALIGNED;
  const int rc = static_cast<int>(static_cast<int64_t>(H) * dtype_size(act) / 16);
  const dim3 grid(static_cast<unsigned>((T * k + 3) / 4));
  const auto* d = static_cast<const u32x4_t*>(dout);
  const auto* y = static_cast<const u32x4_t*>(y_perm);
  auto* dy = static_cast<u32x4_t*>(dy_perm);
  const bool stream_rows = T * k * rc * 16 > (int64_t{32} << 20);        // L2 of the eight XCDs: 32 MB
  auto launch = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, as_stream(stream), d, y, T * k, cap_rows, rc, k, inv, topk_w, dy, dtopk_w);
  };
  if (act == MOE_BF16)
    stream_rows ? launch(k_combine_bwd<true, true>) : launch(k_combine_bwd<true, false>);
  else
    stream_rows ? launch(k_combine_bwd<false, true>) : launch(k_combine_bwd<false, false>);
  DBOMOE_CHECK_LAUNCH();
  return MOE_OK;
}

extern "C" moe_status moe_route_backward(const float* logits, int64_t T, const int32_t* topk_ids,
                                         const float* dtopk_w, const moe_route_params* params, void* dlogits,
                                         moe_dtype dl, void* stream) {
  const moe_status st = check_route_params(params);
  if (st != MOE_OK) return st;
  if (T < 0) return MOE_ERR_INVALID_ARG;
  if (dl != MOE_F32 && dl != MOE_BF16) return MOE_ERR_UNSUPPORTED;
  if (T >= (int64_t{1} << 26)) return MOE_ERR_UNSUPPORTED;          // 64 threads a token, 2^32 in a grid
  if (T == 0) return MOE_OK;
  if (!logits || !topk_ids || !dtopk_w || !dlogits) return MOE_ERR_INVALID_ARG;
  if (static_cast<const void*>(logits) == dlogits) return MOE_ERR_INVALID_ARG;
  if (!aligned16(logits) || !aligned16(topk_ids) || !aligned16(dtopk_w) || !aligned16(dlogits))
    return MOE_ERR_MISALIGNED;
  const dim3 grid(static_cast<unsigned>((T + 3) / 4));
  if (dl == MOE_BF16)
    hipLaunchKernelGGL(k_route_bwd<bf16_t>, grid, dim3(256), 0, as_stream(stream), logits, T, topk_ids, dtopk_w,
                       *params, static_cast<bf16_t*>(dlogits));
  else
    hipLaunchKernelGGL(k_route_bwd<float>, grid, dim3(256), 0, as_stream(stream), logits, T, topk_ids, dtopk_w,
                       *params, static_cast<float*>(dlogits));
  DBOMOE_CHECK_LAUNCH();
  return MOE_OK;
}
