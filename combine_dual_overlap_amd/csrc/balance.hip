// Routing that keeps the experts balanced, for gfx950: selection with a bias that
// the weights do not see, the bias's update from the experts' load, and the
// balance loss with its gradient.
#include "gemm_mfma.h"
#include "rows.h"

namespace dbomoe {

// ---- selection ------------------------------------------------------------------
// With p the scores (softmax over all experts, or sigmoid, of the logits) and b the
// bias: experts are chosen by p + b (groups by the sum of their group_topn best),
// and weighted by p alone.  Scores and sums are kept in 64 bits: the bias brings
// experts close to each other on purpose, and what is chosen must not hang on the
// rounding of a score.  4096 x 256 logits are 4 MB, under 1 us of HBM time: the steps
// of the selection bound it.  One wave takes a token, so that a maximum is six DPP
// instructions; 256 tokens x 6 of 64 3.4 us (4.6 with the load), 4096 x 8 of 256 in 4 of 8
// groups 9.6 (11.8; a lane has neighbouring experts, so that a group is a team of lanes; by way of
// LDS two more).
// An expert whose logit is -inf or NaN has score 0 and is chosen only when no
// candidate is left; a logit of +inf counts as the largest finite one.
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
  int count_here;          // k_select adds it all; else only takes off what k_count will add too much
};

// Cross-lane moves in registers (the lane permutes through LDS that __shfl makes are
// a round trip each, and the steps here depend on one another).
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp_move(uint32_t v) {
  return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, ROWS, 0xf, false));
}

template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ double dpp_d(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint64_t lo = dpp_move<CTRL, ROWS>(static_cast<uint32_t>(b)), hi = dpp_move<CTRL, ROWS>(static_cast<uint32_t>(b >> 32));
  return __builtin_bit_cast(double, hi << 32 | lo);
}

template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_add_d(double v) { return v + dpp_d<CTRL, ROWS>(v); }

__device__ __forceinline__ double lane_of(double v, int lane) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint64_t lo = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(b), lane));
  const uint64_t hi = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(b >> 32), lane));
  return __builtin_bit_cast(double, hi << 32 | lo);
}

// Sum of the first 16 lanes, of the wave; the largest of the wave: the same in every lane.
__device__ __forceinline__ double row_sum_d(double v) {
  v = dpp_add_d<0x111, 0xf>(v);          // row_shr 1, 2, 4, 8: lane 15 of each 16 has their sum
  v = dpp_add_d<0x112, 0xf>(v);
  v = dpp_add_d<0x114, 0xf>(v);
  v = dpp_add_d<0x118, 0xf>(v);
  return v;
}

__device__ __forceinline__ double wave_sum_d(double v) {
  v = row_sum_d(v);
  v = dpp_add_d<0x142, 0xa>(v);          // lane 15 of a row to the next, lane 31 to the upper half
  v = dpp_add_d<0x143, 0xc>(v);
  return lane_of(v, 63);
}

__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
  v = max(v, dpp_move<0x111, 0xf>(v));
  v = max(v, dpp_move<0x112, 0xf>(v));
  v = max(v, dpp_move<0x114, 0xf>(v));
  v = max(v, dpp_move<0x118, 0xf>(v));
  v = max(v, dpp_move<0x142, 0xa>(v));
  v = max(v, dpp_move<0x143, 0xc>(v));
  return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), 63));
}

// Bits whose order as whole numbers is that of the floats; 0 is below all of them.
__device__ __forceinline__ uint32_t ordered(float f) {
  const uint32_t u = __float_as_uint(f);
  return u ^ (u >> 31 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t u) {
  return __uint_as_float(u ^ (u >> 31 ? 0x80000000u : 0xffffffffu));
}

// e^x for x <= 0, and 1 / x for x >= 1, to a few units in the last place of 64 bits:
// x = n ln 2 + r with |r| <= ln 2 / 2, the Taylor sum of e^r to r^13 (the next term is
// below 2^-57), times 2^n; Newton steps from the hardware's reciprocal.  (The general
// functions are several times as long, and what a token's wave waits for here is
// instructions.)
__device__ __forceinline__ double exp_neg(double x) {
  x = fmax(x, -800.0);                                   // e^-800 is 0
  const double n = rint(x * 1.4426950408889634);
  double r = fma(n, -0x1.62e42fefa0000p-1, x);           // ln 2 in two parts, the first exact times n
  r = fma(n, -0x1.cf79abc9e3b3ap-40, r);
  double s = 1.0 / 6227020800.0;
  s = fma(s, r, 1.0 / 479001600.0);
  s = fma(s, r, 1.0 / 39916800.0);
  s = fma(s, r, 1.0 / 3628800.0);
  s = fma(s, r, 1.0 / 362880.0);
  s = fma(s, r, 1.0 / 40320.0);
  s = fma(s, r, 1.0 / 5040.0);
  s = fma(s, r, 1.0 / 720.0);
  s = fma(s, r, 1.0 / 120.0);
  s = fma(s, r, 1.0 / 24.0);
  s = fma(s, r, 1.0 / 6.0);
  s = fma(s, r, 0.5);
  s = fma(s, r, 1.0);
  s = fma(s, r, 1.0);
  return __builtin_amdgcn_ldexp(s, static_cast<int>(n));
}

__device__ __forceinline__ double inverse(double x) {
  double r = __builtin_amdgcn_rcp(x);
  r = fma(fma(-x, r, 1.0), r, r);
  return fma(fma(-x, r, 1.0), r, r);
}

constexpr int kSelTokens = 4;      // tokens of a workgroup, one wave each

// One wave per token, NE neighbouring experts in a lane.
// A slot's expert is found by the keys rounded to fp32 (which keeps their order):
// the wave's largest, then a ballot for who has it; only where several do, the keys
// themselves are compared.
template <int NE>
__global__ __launch_bounds__(64 * kSelTokens) void k_select(SelectParams p) {
  __shared__ double s_val[kSelTokens][64 * NE];
  __shared__ int s_load[64 * NE];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int E = p.rp.E, k = p.rp.k;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kSelTokens + wave;
  if (p.load) {
    for (int e = threadIdx.x; e < E; e += blockDim.x) s_load[e] = 0;
    __syncthreads();
  }
  if (t < p.T) {
    const double NEG = -INFINITY;
    double* val = s_val[wave];
    // Lane l has experts l NE .. l NE + NE - 1.
    typedef float some_t __attribute__((ext_vector_type(NE), aligned(4)));
    const int e0 = lane * NE, have = min(max(E - e0, 0), NE);
    auto get = [&](const float* row) {
      some_t v = 0.f;
      if (have == NE) {
        v = *reinterpret_cast<const some_t*>(row + e0);
      } else {
#pragma unroll
        for (int i = 0; i < NE; ++i)
          if (i < have) v[i] = row[e0 + i];
      }
      return v;
    };
    float l[NE];
    bool cand[NE];                             // may be chosen
    some_t sum_l = 0.f, bias = 0.f;
    if (p.bias) bias = get(p.bias);
    for (int s0 = 0; s0 < p.S; ++s0) sum_l += get(p.part + (s0 * p.T + t) * E);      // in split order
    if (p.logit_bias) sum_l += get(p.logit_bias);
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      if (p.logits && i < have) p.logits[t * E + e0 + i] = sum_l[i];
      l[i] = i < have && sum_l[i] > -INFINITY ? fminf(sum_l[i], 3.402823466e38f) : -INFINITY;
    }
    double pr[NE], key[NE];
    if (p.rp.score == MOE_SCORE_SOFTMAX) {
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < NE; ++i) top = max(top, ordered(l[i]));
      const double lmax = unordered(wave_max_u32(top));
      double sum = 0.0;
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        pr[i] = l[i] > -INFINITY ? exp_neg(static_cast<double>(l[i]) - lmax) : 0.0;
        sum += pr[i];
      }
      sum = wave_sum_d(sum);
      const double inv = sum > 0.0 ? inverse(sum) : 0.0;     // (a sum is at least 1)
#pragma unroll
      for (int i = 0; i < NE; ++i) pr[i] *= inv;
    } else {
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        const double e = exp_neg(-fabs(static_cast<double>(l[i])));      // (0 for a masked one)
        pr[i] = (l[i] < 0.f ? e : 1.0) * inverse(1.0 + e);
        if (!(l[i] > -INFINITY)) pr[i] = 0.0;
      }
    }
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      key[i] = l[i] > -INFINITY ? pr[i] + static_cast<double>(bias[i]) : NEG;
      cand[i] = key[i] > NEG;                  // (a bias of -inf or NaN, which has no place here, masks too)
    }

    if (p.rp.n_groups > 1) {
      // A group's members are with a team of lanes: those that have them, or, where a
      // group is not a power of two of lanes, as many as fit into the wave, through LDS.
      // Each keeps its group_topn best in order, and the team's lists are merged.
      const int G = p.rp.n_groups, per = E / G, n = p.rp.group_topn;
      const bool own = per % NE == 0 && (per / NE & (per / NE - 1)) == 0;
      const int team = own ? per / NE : 64 >> (32 - __clz(G - 1));     // a power of two
      const int grp = lane / team, at = lane & (team - 1);
      auto score_of = [&](auto length) {                 // lists of two or four, at least n
        constexpr int N = decltype(length)::value;
        double best[N];
#pragma unroll
        for (int q = 0; q < N; ++q) best[q] = NEG;
        auto insert = [&](double x) {
#pragma unroll
          for (int q = 0; q < N; ++q) {
            const double was = best[q];
            const bool more = x > was;
            best[q] = more ? x : was;
            x = more ? was : x;
          }
        };
        if (own) {
#pragma unroll
          for (int i = 0; i < NE; ++i) insert(cand[i] ? key[i] : NEG);
        } else if (grp < G) {
          for (int j0 = at; j0 < per; j0 += 4 * team) {  // four reads in flight
            double x[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) x[q] = j0 + q * team < per ? val[grp * per + j0 + q * team] : NEG;
#pragma unroll
            for (int q = 0; q < 4; ++q) insert(x[q]);
          }
        }
        auto merge = [&](auto from) {
          double other[N];
#pragma unroll
          for (int q = 0; q < N; ++q) other[q] = from(best[q]);
#pragma unroll
          for (int q = 0; q < N; ++q) insert(other[q]);
        };
        // with the neighbour, the other pair, the other four, the other eight (whose
        // lanes all have the same list, so that a mirror will do)
        if (team > 1) merge([](double x) { return dpp_d<0xb1>(x); });
        if (team > 2) merge([](double x) { return dpp_d<0x4e>(x); });
        if (team > 4) merge([](double x) { return dpp_d<0x141>(x); });
        if (team > 8) merge([](double x) { return dpp_d<0x140>(x); });
        for (int d = 16; d < team; d <<= 1) merge([d](double x) { return __shfl_xor(x, d, kWave); });
        double sum = best[0];
#pragma unroll
        for (int q = 1; q < N; ++q)
          if (q < n && best[q] > NEG) sum += best[q];
        return sum;
      };
      if (!own) {
#pragma unroll
        for (int i = 0; i < NE; ++i)
          if (i < have) val[e0 + i] = cand[i] ? key[i] : NEG;
        __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
        __builtin_amdgcn_wave_barrier();
      }
      const double score = n <= 2 ? score_of(std::integral_constant<int, 2>{}) : score_of(std::integral_constant<int, 4>{});
      __builtin_amdgcn_wave_barrier();                   // val is read by all before it is written again
      // its place among the groups
      int place = 0;
      for (int o = 0; o < G; ++o) {
        const double so = lane_of(score, o * team);
        place += so > score || (so == score && o < grp);
      }
      const uint64_t kept = __ballot(grp < G && place < p.rp.topk_groups);
#pragma unroll
      for (int i = 0; i < NE; ++i) cand[i] = cand[i] && (kept >> ((own ? grp : (e0 + i) / per) * team) & 1ull);
    }

    uint32_t u[NE];
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      u[i] = cand[i] ? ordered(static_cast<float>(key[i])) : 0;
      if (i < have) val[e0 + i] = pr[i];
    }
    __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
    __builtin_amdgcn_wave_barrier();
    int my_e = 0, real = 0;                    // slot j is kept by lane j
#pragma unroll 1
    for (; real < k; ++real) {
      uint32_t m = u[0];
#pragma unroll
      for (int i = 1; i < NE; ++i) m = max(m, u[i]);
      m = wave_max_u32(m);
      if (m == 0) break;                       // no candidate is left
      uint64_t who[NE];
      int many = 0;
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        who[i] = __ballot(u[i] == m);
        many += __popcll(who[i]);
      }
      auto lowest = [&](double& its) {         // the lowest expert of who, and its key
        uint64_t any = 0;
#pragma unroll
        for (int i = 0; i < NE; ++i) any |= who[i];
        const int src = __ffsll(static_cast<unsigned long long>(any)) - 1;
        int be = 0;
#pragma unroll
        for (int i = NE - 1; i >= 0; --i)
          if (who[i] >> src & 1) {
            be = src * NE + i;
            its = lane_of(key[i], src);
          }
        return be;
      };
      int be = 0;
      if (many == 1) {
        uint64_t it = 0;
#pragma unroll
        for (int i = 0; i < NE; ++i) {
          it |= who[i];
          if (who[i]) be = i;
        }
        be += (__ffsll(static_cast<unsigned long long>(it)) - 1) * NE;
      } else {
        // those above the lowest one's key, until there are none
        bool more = true;
        while (more) {
          double its = 0.0;
          be = lowest(its);
          more = false;
          uint64_t above[NE];
#pragma unroll
          for (int i = 0; i < NE; ++i) {
            above[i] = __ballot(u[i] == m && key[i] > its);
            more |= above[i] != 0;
          }
          if (more)
#pragma unroll
            for (int i = 0; i < NE; ++i) who[i] = above[i];
        }
      }
#pragma unroll
      for (int i = 0; i < NE; ++i)
        if (e0 + i == be) u[i] = 0;
      if (lane == real) my_e = be;
    }
    // The slots without a candidate: the first masked experts, weight 0.  There are enough, since
    // the kept groups have k experts or more.  (Not the others of groups that were dropped: their
    // score is not 0, and the gradient of the weights would count them.)
    if (real < k) {
      uint64_t masked[NE];
#pragma unroll
      for (int i = 0; i < NE; ++i) masked[i] = __ballot(i < have && !(key[i] > NEG));
      for (int j = real; j < k; ++j) {
        uint64_t any = 0;
#pragma unroll
        for (int i = 0; i < NE; ++i) any |= masked[i];
        const int src = __ffsll(static_cast<unsigned long long>(any)) - 1;
        int e = 0;
#pragma unroll
        for (int i = NE - 1; i >= 0; --i)
          if (masked[i] >> src & 1) e = src * NE + i;
#pragma unroll
        for (int i = 0; i < NE; ++i)
          if (src * NE + i == e) masked[i] &= ~(1ull << src);
        if (lane == j) my_e = e;
      }
    }
    const double my_p = lane < real ? val[my_e] : 0.0;
    const double sum = lane_of(row_sum_d(my_p), 15);     // (at most 16 slots)
    if (lane < k) {
      const double w = p.rp.renormalize && sum > 0.0 ? my_p / sum : my_p;
      p.ids[t * k + lane] = my_e;
      p.w[t * k + lane] = static_cast<float>(w * static_cast<double>(p.rp.routed_scale));
      if (p.load && (lane < real) == (p.count_here != 0)) atomicAdd(&s_load[my_e], 1);
    }
  }
  if (p.load) {
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += blockDim.x)
      if (s_load[e]) atomicAdd(&p.load[e], p.count_here ? s_load[e] : -s_load[e]);      // whole numbers: any order
  }
}

// Up to this many tokens k_select adds up the load itself.  512 tokens x 8 of 256: 1.3 us
// for it, where k_count takes 3.5; 4096 x 8: 13 us, and k_count 4.
constexpr int64_t kCountHere = 512;

// load[e] += how often e is among the n ids.  Few workgroups: it is the additions to the
// same few cache lines from all over the GPU that take the time.
__global__ __launch_bounds__(1024) void k_count(const int32_t* __restrict__ ids, int64_t n, int E,
                                                int32_t* __restrict__ load) {
  __shared__ int s_load[4][256];
  s_load[threadIdx.x >> 8][threadIdx.x & 255] = 0;
  __syncthreads();
  int* mine = s_load[threadIdx.x & 3];
  const int4* ids4 = reinterpret_cast<const int4*>(ids);
  const int64_t n4 = n / 4, stride = static_cast<int64_t>(gridDim.x) * 1024;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 1024 + threadIdx.x; i < n4; i += stride) {
    const int4 v = ids4[i];
    atomicAdd(&mine[v.x], 1);
    atomicAdd(&mine[v.y], 1);
    atomicAdd(&mine[v.z], 1);
    atomicAdd(&mine[v.w], 1);
  }
  if (blockIdx.x == 0 && threadIdx.x < (n & 3)) atomicAdd(&mine[ids[n4 * 4 + threadIdx.x]], 1);
  __syncthreads();
  const int e = threadIdx.x;
  if (e >= E) return;
  const int sum = s_load[0][e] + s_load[1][e] + s_load[2][e] + s_load[3][e];
  if (sum) atomicAdd(&load[e], sum);
}

moe_status launch_select(SelectParams p, hipStream_t s) {
  if (p.T == 0) return MOE_OK;
  const int64_t n = p.T * p.rp.k;
  p.count_here = p.T <= kCountHere;
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>((p.T + kSelTokens - 1) / kSelTokens)), dim3(64 * kSelTokens), 0,
                       s, p);
  };
  p.rp.E <= 64 ? go(k_select<1>) : p.rp.E <= 128 ? go(k_select<2>) : go(k_select<4>);
  DBOMOE_CHECK_LAUNCH();
  if (p.load && !p.count_here) {
    const int64_t blocks = std::min<int64_t>(std::max<int64_t>(n / 2048, 1), 16);
    hipLaunchKernelGGL(k_count, dim3(static_cast<unsigned>(blocks)), dim3(1024), 0, s, p.ids, n, p.rp.E, p.load);
    DBOMOE_CHECK_LAUNCH();
  }
  return MOE_OK;
}

moe_status launch_route_balanced(const RouteArgs& a, const float* select_bias, int32_t* load, hipStream_t s) {
  if (a.T == 0) return MOE_OK;
  const moe_status st = launch_route_logits(a, s);
  if (st != MOE_OK) return st;
  SelectParams p{a.part, route_splits(a.T, a.H, a.p.E), a.T, a.bias, select_bias, a.p, a.logits, a.ids, a.w, load, 0};
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

template <typename Out, bool ADD, int NE>
__global__ __launch_bounds__(256) void k_balance_loss(const float* __restrict__ logits, int64_t T,
                                                      const int32_t* __restrict__ load, int E, int softmax, float scale,
                                                      Out* __restrict__ dl, double* __restrict__ part) {
  __shared__ double s_part[4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  float f1[NE];                         // f - 1
  double n[NE], sum = 0.0;              // (whole numbers below 2^53: exact)
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    n[i] = lane + 64 * i < E ? load[lane + 64 * i] : 0;
    sum += n[i];
  }
  sum = wave_sum_d(sum);
  const bool any = sum > 0.0;           // no load: f = 0, no loss
#pragma unroll
  for (int i = 0; i < NE; ++i) f1[i] = any ? static_cast<float>((n[i] * E - sum) / sum) : 0.f;
  double total = 0.0;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * 4 + wave; t < T; t += static_cast<int64_t>(gridDim.x) * 4) {
    const float* row = logits + t * E;
    float l[NE], q[NE], c[NE], was[NE];
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const int e = lane + 64 * i;
      l[i] = -INFINITY;
      was[i] = 0.f;
      if (e >= E) continue;
      if constexpr (ADD && sizeof(Out) == 2) was[i] = bf16_to_f32(dl[t * E + e]);
      if constexpr (ADD && sizeof(Out) == 4) was[i] = dl[t * E + e];
      const float v = row[e];
      if (v > -INFINITY) l[i] = fminf(v, 3.402823466e38f);       // masked experts (-inf, NaN): q = 0, no gradient
    }
    float norm = 0.f;
    if (softmax) {
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < NE; ++i) top = max(top, ordered(l[i]));
      const float lmax = unordered(wave_max_u32(top));
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        q[i] = l[i] > -INFINITY ? expf(l[i] - lmax) : 0.f;
        c[i] = 1.f;
      }
    } else {
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        const float e = expf(-fabsf(l[i])), r = 1.0f / (1.0f + e);
        const bool in = l[i] > -INFINITY;
        q[i] = in ? (l[i] < 0.f ? e * r : r) : 0.f;
        c[i] = l[i] < 0.f ? r : e * r;                           // 1 - p, without cancellation
      }
    }
#pragma unroll
    for (int i = 0; i < NE; ++i) norm += q[i];
    norm = wave_sum_dpp(norm);
    // Sigmoid scores that fp32 hardly holds, or not at all: relative to the largest (the sum is
    // then 1 at least; 1 + e^l is 1 here).  Above that, what fp32 loses of a score is 2^-66 of the sum.
    if (!softmax && norm < 0x1p-60f) {
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < NE; ++i) top = max(top, ordered(l[i]));
      const float lmax = unordered(wave_max_u32(top));
      norm = 0.f;
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        q[i] = l[i] > -INFINITY ? expf(l[i] - lmax) : 0.f;
        norm += q[i];
      }
      norm = wave_sum_dpp(norm);
    }
    const float inv = norm > 0.f ? 1.0f / norm : 0.f;
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      q[i] *= inv;
      dot += q[i] * f1[i];
    }
    dot = wave_sum_dpp(dot);
    if (norm > 0.f && any) total += static_cast<double>(dot) + 1.0;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const int e = lane + 64 * i;
      if (e >= E) continue;
      const float g = was[i] + scale * (q[i] * c[i]) * (f1[i] - dot);
      if constexpr (sizeof(Out) == 2)
        dl[t * E + e] = f32_to_bf16(g);
      else
        dl[t * E + e] = g;
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
      static_cast<const void*>(topk_ids) == topk_w ||
      (load && (load == topk_ids || static_cast<const void*>(load) == topk_w || static_cast<const void*>(load) == logits)))
    return MOE_ERR_INVALID_ARG;
  if (select_bias && (select_bias == topk_w || static_cast<const void*>(select_bias) == topk_ids ||
                      static_cast<const void*>(select_bias) == load))
    return MOE_ERR_INVALID_ARG;
  if (!aligned16(logits) || (select_bias && !aligned16(select_bias)) || !aligned16(topk_ids) || !aligned16(topk_w) ||
      (load && !aligned16(load)))
    return MOE_ERR_MISALIGNED;
  SelectParams p{logits, 1, T, nullptr, select_bias, *params, nullptr, topk_ids, topk_w, load, 0};
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
  const void* outs[] = {topk_ids, topk_w, ws, logits_out, load};
  const void* ins[] = {x, w_router, logit_bias, select_bias};
  for (int i = 0; i < 5; ++i) {
    if (!outs[i]) continue;
    for (int j = 0; j < i; ++j)
      if (outs[i] == outs[j]) return MOE_ERR_INVALID_ARG;
    for (const void* in : ins)
      if (outs[i] == in) return MOE_ERR_INVALID_ARG;
  }
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
      static_cast<const void*>(loss) == load || static_cast<const void*>(ws) == dlogits || ws == logits || ws == load ||
      ws == loss)
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
  auto of = [&](auto ne) {
    constexpr int NE = decltype(ne)::value;
    if (dl == MOE_BF16)
      accumulate ? go(k_balance_loss<bf16_t, true, NE>, static_cast<bf16_t*>(dlogits))
                 : go(k_balance_loss<bf16_t, false, NE>, static_cast<bf16_t*>(dlogits));
    else
      accumulate ? go(k_balance_loss<float, true, NE>, static_cast<float*>(dlogits))
                 : go(k_balance_loss<float, false, NE>, static_cast<float*>(dlogits));
  };
  if (params->E <= 64)
    of(std::integral_constant<int, 1>{});
  else if (params->E <= 128)
    of(std::integral_constant<int, 2>{});
  else
    of(std::integral_constant<int, 4>{});
  DBOMOE_CHECK_LAUNCH();
  hipLaunchKernelGGL(k_loss_sum, dim3(1), dim3(256), 0, s, part, blocks, over_t, loss);
  DBOMOE_CHECK_LAUNCH();
  return MOE_OK;
}
