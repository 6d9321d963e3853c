// Routing that keeps the experts balanced, for gfx950: selection with a bias that
// the weights do not see, the bias's update from the experts' load, and the
// balance loss with its gradient.
#include "gemm_mfma.h"

namespace dbomoe {

// ---- selection ------------------------------------------------------------------
// With p the scores (softmax over all experts, or sigmoid, of the logits) and b the
// bias: experts are chosen by p + b (groups by the sum of their group_topn best),
// and weighted by p alone.  Scores and sums are kept in 64 bits: the bias brings
// experts close to each other on purpose, and what is chosen must not hang on the
// rounding of a score.  (Logits that the caller already has: 4096 x 256 of them
// are 4 MB, under 1 us of HBM time; the steps of the selection bound it.)
// An expert whose logit is -inf or NaN has score 0 and is chosen only when no
// other is left; a logit of +inf counts as the largest finite one.
struct SelectParams {
  const float* part;       // [S][T][E] partial logits (S == 1: the logits)
  int S;
  int64_t T;
  const float* logit_bias;
  const float* bias;       // selection bias or NULL
  moe_route_params rp;
  float* logits;
  int32_t* ids;
  float* w;
  int32_t* load;           // [E] or NULL: what each expert got is added
};

__device__ __forceinline__ double wave_sum_d(double v) {
#pragma unroll
  for (int d = kWave / 2; d > 0; d >>= 1) v += __shfl_xor(v, d, kWave);
  return v;
}

// (value descending, index ascending): the best of the wave, in every lane.
__device__ __forceinline__ void wave_best(double& v, int& e) {
#pragma unroll
  for (int d = kWave / 2; d > 0; d >>= 1) {
    const double ov = __shfl_xor(v, d, kWave);
    const int oe = __shfl_xor(e, d, kWave);
    if (ov > v || (ov == v && oe < e)) {
      v = ov;
      e = oe;
    }
  }
}

constexpr int kSelTokens = 4;      // tokens of a workgroup, one wave each

__global__ __launch_bounds__(64 * kSelTokens) void k_select(SelectParams p) {
  __shared__ double s_key[kSelTokens][256];
  __shared__ int s_load[256];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int E = p.rp.E, k = p.rp.k;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kSelTokens + wave;
  if (p.load) {
    for (int e = threadIdx.x; e < E; e += blockDim.x) s_load[e] = 0;
    __syncthreads();
  }
  if (t < p.T) {
    float l[4];
    unsigned cand = 0;                         // bit i: expert lane + 64 i may be chosen
    float lmax = -INFINITY;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = lane + 64 * i;
      l[i] = -INFINITY;
      if (e >= E) continue;
      float s = 0.f;
      for (int s0 = 0; s0 < p.S; ++s0) s += p.part[(s0 * p.T + t) * E + e];     // in split order
      if (p.logit_bias) s += p.logit_bias[e];
      if (p.logits) p.logits[t * E + e] = s;
      if (s > -INFINITY) {
        l[i] = fminf(s, 3.402823466e38f);
        cand |= 1u << i;
        lmax = fmaxf(lmax, l[i]);
      }
    }
    const bool softmax = p.rp.score == MOE_SCORE_SOFTMAX;
    double pr[4], key[4];
    if (softmax) {
      lmax = wave_max_f(lmax);
      double sum = 0.0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        pr[i] = (cand >> i) & 1u ? exp(static_cast<double>(l[i]) - static_cast<double>(lmax)) : 0.0;
        sum += pr[i];
      }
      sum = wave_sum_d(sum);
#pragma unroll
      for (int i = 0; i < 4; ++i) pr[i] = (cand >> i) & 1u ? pr[i] / sum : 0.0;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) pr[i] = (cand >> i) & 1u ? 1.0 / (1.0 + exp(-static_cast<double>(l[i]))) : 0.0;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      key[i] = pr[i] + (p.bias && lane + 64 * i < E ? static_cast<double>(p.bias[lane + 64 * i]) : 0.0);
    const double NEG = -INFINITY;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (!(key[i] > NEG)) cand &= ~(1u << i);         // a bias of -inf or NaN masks too
    if (p.rp.n_groups > 1) {
      const int G = p.rp.n_groups, per = E / G, n = p.rp.group_topn;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (lane + 64 * i < E) s_key[wave][lane + 64 * i] = (cand >> i) & 1u ? key[i] : NEG;
      __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
      __builtin_amdgcn_wave_barrier();
      double gs = NEG;
      if (lane < G) {
        double top[4] = {NEG, NEG, NEG, NEG};
        for (int j = 0; j < per; ++j) {
          double x = s_key[wave][lane * per + j];
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (q < n && x > top[q]) {
              const double tmp = top[q];
              top[q] = x;
              x = tmp;
            }
        }
        gs = top[0];
#pragma unroll
        for (int q = 1; q < 4; ++q)
          if (q < n && top[q] > NEG) gs += top[q];
      }
      uint64_t kept = 0;
      for (int r = 0; r < p.rp.topk_groups; ++r) {
        const bool open = lane < G && !((kept >> lane) & 1ull);
        double bv = open ? gs : NEG;
        int be = open ? lane : 1 << 30;
        wave_best(bv, be);
        kept |= 1ull << be;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int e = lane + 64 * i;
        if (e < E && !((kept >> (e / per)) & 1ull)) cand &= ~(1u << i);
      }
    }

    unsigned left = 0;                         // not chosen yet
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (lane + 64 * i < E) left |= 1u << i;
    int my_e = 0;
    double my_p = 0.0, sum = 0.0;
#pragma unroll 1
    for (int j = 0; j < k; ++j) {
      double bv = NEG;
      int be = 1 << 30;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int e = lane + 64 * i;
        if (((cand >> i) & 1u) && (key[i] > bv || be == 1 << 30)) {
          bv = key[i];
          be = e;
        }
      }
      wave_best(bv, be);
      bool real = be < E;
      if (!real) {                             // no candidate is left: the first expert not chosen, weight 0
        bv = 0.0;
        be = 1 << 30;
#pragma unroll
        for (int i = 3; i >= 0; --i)
          if ((left >> i) & 1u) be = lane + 64 * i;
        wave_best(bv, be);
      }
      const int i = be >> 6;
      if ((be & 63) == lane) {
        cand &= ~(1u << i);
        left &= ~(1u << i);
      }
      const double mine = i == 0 ? pr[0] : i == 1 ? pr[1] : i == 2 ? pr[2] : pr[3];
      const double pj = real ? __shfl(mine, be & 63, kWave) : 0.0;
      sum += pj;
      if (lane == j) {
        my_e = be;
        my_p = pj;
        if (p.load && real) atomicAdd(&s_load[be], 1);
      }
    }
    if (lane < k) {
      const double w = p.rp.renormalize && sum > 0.0 ? my_p / sum : my_p;
      p.ids[t * k + lane] = my_e;
      p.w[t * k + lane] = static_cast<float>(w * static_cast<double>(p.rp.routed_scale));
    }
  }
  if (p.load) {
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += blockDim.x)
      if (s_load[e]) atomicAdd(&p.load[e], s_load[e]);        // whole numbers: any order
  }
}

moe_status launch_select(const SelectParams& p, hipStream_t s) {
  if (p.T == 0) return MOE_OK;
  hipLaunchKernelGGL(k_select, dim3(static_cast<unsigned>((p.T + kSelTokens - 1) / kSelTokens)), dim3(64 * kSelTokens), 0,
                     s, p);
  DBOMOE_CHECK_LAUNCH();
  return MOE_OK;
}

moe_status launch_route_balanced(const RouteArgs& a, const float* select_bias, int32_t* load, hipStream_t s) {
  if (a.T == 0) return MOE_OK;
  const moe_status st = launch_route_logits(a, s);
  if (st != MOE_OK) return st;
  SelectParams p{a.part, route_splits(a.T, a.H, a.p.E), a.T, a.bias, select_bias, a.p, a.logits, a.ids, a.w, load};
  return launch_select(p, s);
}

// ---- the bias's update ------------------------------------------------------------
// b_e += rate * sign(mean load - load_e), compared as E * load_e against the sum, in
// 64 bits; the load starts again from zero.
__global__ __launch_bounds__(256) void k_bias_update(float* __restrict__ bias, int32_t* __restrict__ load, int E,
                                                     float rate) {
  __shared__ long long s_sum[4];
  const int e = threadIdx.x;
  const long long mine = e < E ? load[e] : 0;
  long long sum = mine;
#pragma unroll
  for (int d = kWave / 2; d > 0; d >>= 1) sum += __shfl_xor(sum, d, kWave);
  if ((e & 63) == 0) s_sum[e >> 6] = sum;
  __syncthreads();
  sum = s_sum[0] + s_sum[1] + s_sum[2] + s_sum[3];
  if (e >= E) return;
  const long long own = mine * E;
  if (own != sum) bias[e] += own < sum ? rate : -rate;
  load[e] = 0;
}

// ---- the balance loss ---------------------------------------------------------------
// f_e = E load_e / sum load and q_te = p_te (softmax) or p_te / sum_e p_te (sigmoid):
//   loss = coef / T sum_t sum_e f_e q_te
//   dl_te = coef / T q_te (f_e - sum_j f_j q_tj)     (sigmoid: times 1 - p_te)
// The loads are counts and have no gradient.  f - 1 takes the place of f in the
// difference: the q of a token sum to 1, and f is near 1 where the experts are
// balanced.  One wave per token; each workgroup leaves the sum of its tokens'
// inner sums, and k_loss_sum adds these in order.
constexpr int kLossBlocks = 1024;      // at most; four waves each

template <typename Out, bool ADD>
__global__ __launch_bounds__(256) void k_balance_loss(const float* __restrict__ logits, int64_t T,
                                                      const int32_t* __restrict__ load, int E, int softmax, float scale,
                                                      Out* __restrict__ dl, double* __restrict__ part) {
  __shared__ double s_part[4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  float f1[4];                          // f - 1
  long long n[4], sum = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    n[i] = lane + 64 * i < E ? load[lane + 64 * i] : 0;
    sum += n[i];
  }
#pragma unroll
  for (int d = kWave / 2; d > 0; d >>= 1) sum += __shfl_xor(sum, d, kWave);
  const float none = sum > 0 ? 0.f : -1.f;        // no load: f = 0, no loss
#pragma unroll
  for (int i = 0; i < 4; ++i)
    f1[i] = sum > 0 ? static_cast<float>(static_cast<double>(n[i] * E - sum) / static_cast<double>(sum)) : 0.f;
  double total = 0.0;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * 4 + wave; t < T; t += static_cast<int64_t>(gridDim.x) * 4) {
    const float* row = logits + t * E;
    float l[4], q[4], c[4] = {1.f, 1.f, 1.f, 1.f};
    bool in[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float v = lane + 64 * i < E ? row[lane + 64 * i] : -INFINITY;
      in[i] = v > -INFINITY;                      // masked experts (-inf, NaN): q = 0, no gradient
      l[i] = in[i] ? fminf(v, 3.402823466e38f) : -INFINITY;
    }
    float norm = 0.f;
    if (softmax) {
      const float lmax = wave_max_f(fmaxf(fmaxf(l[0], l[1]), fmaxf(l[2], l[3])));
#pragma unroll
      for (int i = 0; i < 4; ++i) q[i] = in[i] ? expf(l[i] - lmax) : 0.f;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        q[i] = in[i] ? 1.0f / (1.0f + expf(-l[i])) : 0.f;
        c[i] = in[i] ? 1.0f / (1.0f + expf(l[i])) : 0.f;      // 1 - p, without cancellation
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) norm += q[i];
    norm = wave_sum_f(norm);
    const float inv = norm > 0.f ? 1.0f / norm : 0.f;
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      q[i] *= inv;
      dot += q[i] * f1[i];
    }
    dot = wave_sum_f(dot);
    if (norm > 0.f) total += static_cast<double>(dot) + 1.0 + none;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = lane + 64 * i;
      if (e >= E) continue;
      float g = scale * (q[i] * c[i]) * (f1[i] - dot);
      Out* at = dl + t * E + e;
      if constexpr (sizeof(Out) == 2) {
        if (ADD) g += bf16_to_f32(*at);
        *at = f32_to_bf16(g);
      } else {
        if (ADD) g += *at;
        *at = g;
      }
    }
  }
  if (lane == 0) s_part[wave] = total;
  __syncthreads();
  if (threadIdx.x == 0) part[blockIdx.x] = ((s_part[0] + s_part[1]) + s_part[2]) + s_part[3];
}

__global__ __launch_bounds__(256) void k_loss_sum(const double* __restrict__ part, int n, double scale,
                                                  float* __restrict__ loss) {
  __shared__ double s_part[4];
  double v = 0.0;
  for (int i = threadIdx.x; i < n; i += 256) v += part[i];
  v = wave_sum_d(v);
  if ((threadIdx.x & 63) == 0) s_part[threadIdx.x >> 6] = v;
  __syncthreads();
  if (threadIdx.x == 0) *loss = static_cast<float>(scale * (((s_part[0] + s_part[1]) + s_part[2]) + s_part[3]));
}

static int64_t loss_blocks(int64_t T) { return std::min<int64_t>((T + 3) / 4, kLossBlocks); }

}  // namespace dbomoe

using namespace dbomoe;

extern "C" moe_status moe_route_select(const float* logits, int64_t T, const float* select_bias,
                                       const moe_route_params* params, int32_t* topk_ids, float* topk_w, int32_t* load,
                                       void* stream) {
  const moe_status st = check_route_params(params);
  if (st != MOE_OK) return st;
  if (T < 0) return MOE_ERR_INVALID_ARG;
  if (T >= (int64_t{1} << 26)) return MOE_ERR_UNSUPPORTED;          // 64 threads a token, 2^32 in a grid
  if (T == 0) return MOE_OK;
  if (!logits || !topk_ids || !topk_w) return MOE_ERR_INVALID_ARG;
  if (static_cast<const void*>(topk_w) == logits || static_cast<const void*>(topk_ids) == logits ||
      static_cast<const void*>(topk_ids) == topk_w || (load && (load == topk_ids || static_cast<const void*>(load) == logits)))
    return MOE_ERR_INVALID_ARG;
  if (!aligned16(logits) || (select_bias && !aligned16(select_bias)) || !aligned16(topk_ids) || !aligned16(topk_w) ||
      (load && !aligned16(load)))
    return MOE_ERR_MISALIGNED;
  SelectParams p{logits, 1, T, nullptr, select_bias, *params, nullptr, topk_ids, topk_w, load};
  return launch_select(p, as_stream(stream));
}

extern "C" moe_status moe_route_balanced(const void* x, moe_dtype act, int64_t T, int32_t H, const void* w_router,
                                         const float* logit_bias, const float* select_bias,
                                         const moe_route_params* params, float* logits_out, int32_t* topk_ids,
                                         float* topk_w, int32_t* load, void* ws, size_t ws_bytes, void* stream) {
  const moe_status st = check_route_params(params);
  if (st != MOE_OK) return st;
  if (T < 0 || H <= 0) return MOE_ERR_INVALID_ARG;
  if (act != MOE_F32 && act != MOE_BF16) return MOE_ERR_UNSUPPORTED;
  if (H % 128) return MOE_ERR_UNSUPPORTED;
  if (T >= (int64_t{1} << 26)) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!x || !w_router || !topk_ids || !topk_w || !ws) return MOE_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(w_router) || !aligned16(topk_ids) || !aligned16(topk_w) ||
      (logit_bias && !aligned16(logit_bias)) || (select_bias && !aligned16(select_bias)) ||
      (logits_out && !aligned16(logits_out)) || (load && !aligned16(load)) || !aligned256(ws))
    return MOE_ERR_MISALIGNED;
  if (ws_bytes < route_ws_bytes(T, H, params->E)) return MOE_ERR_WORKSPACE;
  RouteArgs a{x, act, T, H, w_router, logit_bias, nullptr, *params, logits_out, topk_ids, topk_w, static_cast<float*>(ws)};
  return launch_route_balanced(a, select_bias, load, as_stream(stream));
}

extern "C" moe_status moe_route_bias_update(float* bias, int32_t* load, int32_t E, float rate, void* stream) {
  if (E < 1 || E > 256) return MOE_ERR_INVALID_ARG;
  if (!(rate >= 0.f) || rate > 3.4e38f) return MOE_ERR_INVALID_ARG;
  if (!bias || !load || static_cast<void*>(bias) == load) return MOE_ERR_INVALID_ARG;
  if (!aligned16(bias) || !aligned16(load)) return MOE_ERR_MISALIGNED;
  hipLaunchKernelGGL(k_bias_update, dim3(1), dim3(256), 0, as_stream(stream), bias, load, E, rate);
  DBOMOE_CHECK_LAUNCH();
  return MOE_OK;
}

extern "C" size_t moe_route_balance_loss_workspace_size(int64_t T, int32_t E) {
  if (T <= 0 || E < 1 || E > 256) return 0;
  return align_up(static_cast<size_t>(loss_blocks(T)) * sizeof(double), 256);
}

extern "C" moe_status moe_route_balance_loss(const float* logits, int64_t T, const int32_t* load,
                                             const moe_route_params* params, float coef, float* loss, void* dlogits,
                                             moe_dtype dl, int32_t accumulate, void* ws, size_t ws_bytes, void* stream) {
  const moe_status st = check_route_params(params);
  if (st != MOE_OK) return st;
  if (T < 0 || (accumulate != 0 && accumulate != 1)) return MOE_ERR_INVALID_ARG;
  if (!(coef >= 0.f) || coef > 3.4e38f) return MOE_ERR_INVALID_ARG;
  if (dl != MOE_F32 && dl != MOE_BF16) return MOE_ERR_UNSUPPORTED;
  if (T >= (int64_t{1} << 26)) return MOE_ERR_UNSUPPORTED;
  if (!loss) return MOE_ERR_INVALID_ARG;
  if (!aligned16(loss)) return MOE_ERR_MISALIGNED;
  const hipStream_t s = as_stream(stream);
  if (T == 0) {                          // no tokens: no loss
    hipLaunchKernelGGL(k_loss_sum, dim3(1), dim3(256), 0, s, nullptr, 0, 0.0, loss);
    DBOMOE_CHECK_LAUNCH();
    return MOE_OK;
  }
  if (!logits || !load || !dlogits || !ws) return MOE_ERR_INVALID_ARG;
  if (static_cast<const void*>(logits) == dlogits || static_cast<const void*>(load) == dlogits ||
      static_cast<const void*>(loss) == dlogits || static_cast<const void*>(loss) == logits ||
      static_cast<const void*>(loss) == load || static_cast<const void*>(ws) == dlogits)
    return MOE_ERR_INVALID_ARG;
  if (!aligned16(logits) || !aligned16(load) || !aligned16(dlogits) || !aligned256(ws)) return MOE_ERR_MISALIGNED;
  if (ws_bytes < moe_route_balance_loss_workspace_size(T, params->E)) return MOE_ERR_WORKSPACE;
  const int blocks = static_cast<int>(loss_blocks(T));
  const double over_t = static_cast<double>(coef) / static_cast<double>(T);
  double* part = static_cast<double*>(ws);
  const int softmax = params->score == MOE_SCORE_SOFTMAX;
  auto go = [&](auto kernel, auto* out) {
    hipLaunchKernelGGL(kernel, dim3(blocks), dim3(256), 0, s, logits, T, load, params->E, softmax,
                       static_cast<float>(over_t), out, part);
  };
  if (dl == MOE_BF16)
    accumulate ? go(k_balance_loss<bf16_t, true>, static_cast<bf16_t*>(dlogits))
               : go(k_balance_loss<bf16_t, false>, static_cast<bf16_t*>(dlogits));
  else
    accumulate ? go(k_balance_loss<float, true>, static_cast<float*>(dlogits))
               : go(k_balance_loss<float, false>, static_cast<float*>(dlogits));
  DBOMOE_CHECK_LAUNCH();
  hipLaunchKernelGGL(k_loss_sum, dim3(1), dim3(256), 0, s, part, blocks, over_t, loss);
  DBOMOE_CHECK_LAUNCH();
  return MOE_OK;
}
