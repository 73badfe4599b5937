// The MoE router: from a token's logits l its top_k experts, their weights, the
// routing tables that the MoE folds take, the balance loss, and the gradient.
//
//   p_te = exp(l_te - max_t) / sum_e exp(l_te - max_t)
//   experts of t: the top_k largest l_te, the lower index first among equals
//   w_tj = p_te, or p_te / (sum of the chosen p_te) with norm_topk
//   loss = E / (top_k N^2) * sum_e c_e S_e,  c_e = rows of expert e,
//          S_e = sum_t p_te,  N = tokens that route
//
// The choice compares logits, not probabilities, so that it is exact.  A group
// of LPT lanes serves one token, VPT logits a lane, in registers from the load
// to the last use.  Probabilities, weights and sums are fp32; all sums run in
// a fixed order (per lane over its tokens, over the lanes and waves of a
// block, over the blocks), so results do not change from run to run.
//
// Three launches: route (choices, and per block of 64 tokens the counts and
// probability sums of every expert), scan (per expert, over the blocks) and
// place (each row's place in the expert-sorted order).  A block keeps one
// 64-bit mask per expert of its tokens that chose it: the set bits below a
// token's own are its rank there, whatever order the lanes arrive in.
#include "rld_device.hpp"
#include "rld_internal.hpp"

namespace rld {

constexpr uint32_t kRouteTokens = 64;  // tokens of a block (bits of a mask)
constexpr uint32_t kMaxExperts = 1024;
constexpr uint32_t kMaxTopK = 32;

struct RouterArgs {
  uint64_t logits_, mask_, indices_, weights_;
  uint64_t counts_, offsets_, tokens_, rows_, loss_;
  uint64_t cnt_, psum_;      // [E + 1][nblk]: counts (then their prefix sums), sums of p
  uint64_t total_, ptotal_;  // [E + 1], [E]
  uint32_t ls, T, E, k, nblk, norm;
};

template <int LPT>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int o = 1; o < LPT; o <<= 1) v = fmaxf(v, __shfl_xor(v, o));
  return v;
}

template <int LPT>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = 1; o < LPT; o <<= 1) v += __shfl_xor(v, o);
  return v;
}

// This lane's logits of a token: experts l, l + LPT, ... ; -Inf past E.
template <bool F32, int LPT, int VPT>
__device__ __forceinline__ void load_logits(uint64_t base, uint64_t at, uint32_t E, int l,
                                            float (&v)[VPT]) {
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const uint32_t e = l + LPT * i;
    v[i] = -__builtin_inff();
    if (e < E)
      v[i] = F32 ? gp<const float>(base)[at + e] : bf16_to_f32(gp<const uint16_t>(base)[at + e]);
  }
}

// State of a token: routes (finite largest logit), empty (masked, or nothing
// but -Inf), or bad (a NaN or +Inf among the logits).
enum TokenState { kEmpty, kRoutes, kBad };

template <int LPT, int VPT>
__device__ __forceinline__ TokenState token_state(bool on, const float (&v)[VPT], float& top) {
  float m = -__builtin_inff(), nan = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    m = fmaxf(m, v[i]);
    nan = (v[i] != v[i]) ? 1.f : nan;
  }
  top = group_max<LPT>(m);
  const bool bad = group_max<LPT>(nan) != 0.f || top == __builtin_inff();
  if (!on) return kEmpty;
  if (bad) return kBad;
  return top == -__builtin_inff() ? kEmpty : kRoutes;
}

template <bool F32, int LPT, int VPT>
__global__ void __launch_bounds__(256) route_kernel(RouterArgs a) {
  constexpr int kTokensPerWave = 64 / LPT;
  __shared__ uint64_t chose[kMaxExperts];
  __shared__ float psum[4][LPT * VPT];
  __shared__ int live_s;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int l = lane % LPT, grp = lane / LPT;
  const uint32_t t0 = blockIdx.x * kRouteTokens;
  for (uint32_t e = threadIdx.x; e < a.E; e += 256) chose[e] = 0ull;
  if (threadIdx.x == 0) live_s = 0;
  __syncthreads();

  float sum_p[VPT] = {};
  int live = 0;
  for (uint32_t q = wave * kTokensPerWave + grp; q < kRouteTokens; q += 4 * kTokensPerWave) {
    const uint32_t t = t0 + q;
    const bool on = t < a.T && (a.mask_ == 0 || gp<const int32_t>(a.mask_)[t] != 0);
    float v[VPT], p[VPT], top;
    load_logits<F32, LPT, VPT>(a.logits_, (uint64_t)min(t, a.T - 1) * a.ls, a.E, l, v);
    const TokenState state = token_state<LPT, VPT>(on, v, top);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      p[i] = expf(v[i] - top);
      s += p[i];
    }
    s = group_sum<LPT>(s);
    const float nan = __builtin_nanf("");
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      p[i] = p[i] / s;
      sum_p[i] += state == kRoutes ? p[i] : state == kBad ? nan : 0.f;
    }
    live += state != kEmpty && l == 0;

    // top_k rounds: the lane's best unused logit, then the group's
    float chosen_sum = 0.f, mine_w[(kMaxTopK + LPT - 1) / LPT];
    int mine_e[(kMaxTopK + LPT - 1) / LPT];
    uint32_t used = 0;
#pragma unroll
    for (int i = 0; i < (int)((kMaxTopK + LPT - 1) / LPT); ++i) {
      mine_e[i] = -1;
      mine_w[i] = state == kBad ? nan : 0.f;
    }
    for (uint32_t j = 0; j < a.k; ++j) {
      float best = -__builtin_inff(), bp = 0.f;
      uint32_t at = 0x7fffffffu;
#pragma unroll
      for (int i = 0; i < VPT; ++i)
        if (!((used >> i) & 1) && v[i] > best) {
          best = v[i];
          bp = p[i];
          at = l + LPT * i;
        }
#pragma unroll
      for (int o = 1; o < LPT; o <<= 1) {
        const float ob = __shfl_xor(best, o), op = __shfl_xor(bp, o);
        const uint32_t oa = __shfl_xor(at, o);
        if (ob > best || (ob == best && oa < at)) {
          best = ob;
          bp = op;
          at = oa;
        }
      }
      if (at != 0x7fffffffu && at % LPT == (uint32_t)l) used |= 1u << (at / LPT);
      const bool ok = state == kRoutes && at != 0x7fffffffu;
      if (ok) {
        chosen_sum += bp;
        if (l == 0) atomicOr((unsigned long long*)&chose[at], 1ull << q);
      }
#pragma unroll
      for (int i = 0; i < (int)((kMaxTopK + LPT - 1) / LPT); ++i)
        if (ok && j == (uint32_t)(l + LPT * i)) {
          mine_e[i] = (int)at;
          mine_w[i] = bp;
        }
    }
    if (t < a.T) {
#pragma unroll
      for (int i = 0; i < (int)((kMaxTopK + LPT - 1) / LPT); ++i) {
        const uint32_t j = l + LPT * i;
        if (j < a.k) {
          const float w = (a.norm && mine_e[i] >= 0) ? mine_w[i] / chosen_sum : mine_w[i];
          gp<int32_t>(a.indices_)[(uint64_t)t * a.k + j] = mine_e[i];
          gp<float>(a.weights_)[(uint64_t)t * a.k + j] = w;
        }
      }
    }
  }
  // over the wave's groups, then (below) over the waves
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    float s = sum_p[i];
#pragma unroll
    for (int o = LPT; o < 64; o <<= 1) s += __shfl_xor(s, o);
    if (grp == 0) psum[wave][l + LPT * i] = s;
  }
  if (live) atomicAdd(&live_s, live);
  __syncthreads();
  for (uint32_t e = threadIdx.x; e < a.E; e += 256) {
    gp<int32_t>(a.cnt_)[(uint64_t)e * a.nblk + blockIdx.x] = __popcll(chose[e]);
    gp<float>(a.psum_)[(uint64_t)e * a.nblk + blockIdx.x] =
        (psum[0][e] + psum[1][e]) + (psum[2][e] + psum[3][e]);
  }
  if (threadIdx.x == 0) gp<int32_t>(a.cnt_)[(uint64_t)a.E * a.nblk + blockIdx.x] = live_s;
}

// One block per expert (and one for the routing tokens): its counts become
// the exclusive prefix sums over the blocks of tokens.
__global__ void __launch_bounds__(256) router_scan_kernel(RouterArgs a) {
  __shared__ int wsum[4];
  __shared__ float fsum[4];
  const uint32_t e = blockIdx.x;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  RLD_GLOBAL int32_t* cnt = gp<int32_t>(a.cnt_) + (uint64_t)e * a.nblk;
  int before = 0;
  float ps = 0.f;
  for (uint32_t b0 = 0; b0 < a.nblk; b0 += 256) {
    const uint32_t b = b0 + threadIdx.x;
    const int c = b < a.nblk ? cnt[b] : 0;
    if (b < a.nblk && e < a.E) ps += gp<const float>(a.psum_)[(uint64_t)e * a.nblk + b];
    int inc = c;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int u = __shfl_up(inc, o);
      if (lane >= o) inc += u;
    }
    if (lane == 63) wsum[wave] = inc;
    __syncthreads();
    int off = before, tot = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      off += w < wave ? wsum[w] : 0;
      tot += wsum[w];
    }
    if (b < a.nblk) cnt[b] = off + inc - c;
    before += tot;
    __syncthreads();
  }
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) ps += __shfl_xor(ps, o);
  if (lane == 0) fsum[wave] = ps;
  __syncthreads();
  if (threadIdx.x == 0) {
    gp<int32_t>(a.total_)[e] = before;
    if (e < a.E) gp<float>(a.ptotal_)[e] = (fsum[0] + fsum[1]) + (fsum[2] + fsum[3]);
  }
}

// One block per 64 tokens: the rows' places.  Every block adds up the experts'
// totals itself; block 0 also writes the tables and the loss.
__global__ void __launch_bounds__(256) router_place_kernel(RouterArgs a) {
  __shared__ uint64_t chose[kMaxExperts];
  __shared__ int off[kMaxExperts];
  __shared__ int wsum[4];
  __shared__ double dsum[4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint32_t t0 = blockIdx.x * kRouteTokens;
  // four consecutive experts a thread
  int c[4], sum = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t e = threadIdx.x * 4 + i;
    c[i] = e < a.E ? gp<const int32_t>(a.total_)[e] : 0;
    sum += c[i];
    if (e < a.E) chose[e] = 0ull;
  }
  int inc = sum;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(inc, o);
    if (lane >= o) inc += u;
  }
  if (lane == 63) wsum[wave] = inc;
  __syncthreads();
  int at = inc - sum, total = 0;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    at += w < wave ? wsum[w] : 0;
    total += wsum[w];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t e = threadIdx.x * 4 + i;
    if (e < a.E) off[e] = at;
    at += c[i];
  }
  __syncthreads();

  if (blockIdx.x == 0) {
    double d = 0.0;
    for (uint32_t e = threadIdx.x; e < a.E; e += 256) {
      const int n = gp<const int32_t>(a.total_)[e];
      if (a.counts_) gp<int32_t>(a.counts_)[e] = n;
      if (a.offsets_) gp<int32_t>(a.offsets_)[e] = off[e];
      d += (double)n * (double)gp<const float>(a.ptotal_)[e];
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) d += __shfl_xor(d, o);
    if (lane == 0) dsum[wave] = d;
    __syncthreads();
    if (threadIdx.x == 0) {
      const int n = gp<const int32_t>(a.total_)[a.E];
      if (a.counts_) gp<int32_t>(a.counts_)[a.E] = n;
      if (a.offsets_) gp<int32_t>(a.offsets_)[a.E] = total;
      if (a.loss_) {
        const double s = (dsum[0] + dsum[1]) + (dsum[2] + dsum[3]);
        gp<float>(a.loss_)[0] =
            n ? (float)(s * (double)a.E / ((double)a.k * (double)n * (double)n)) : 0.f;
      }
    }
  }
  if (!a.tokens_ && !a.rows_) return;

  const uint32_t nt = min(kRouteTokens, a.T - t0);
  const uint64_t r0 = (uint64_t)t0 * a.k;
  const uint32_t nr = nt * a.k;
  for (uint32_t i = threadIdx.x; i < nr; i += 256) {
    const int e = gp<const int32_t>(a.indices_)[r0 + i];
    if (e >= 0) atomicOr((unsigned long long*)&chose[e], 1ull << (i / a.k));
  }
  __syncthreads();
  for (uint32_t i = threadIdx.x; i < nr; i += 256) {
    const int e = gp<const int32_t>(a.indices_)[r0 + i];
    if (e >= 0) {
      const uint32_t q = i / a.k;
      const uint64_t dst = (uint64_t)off[e] +
                           gp<const int32_t>(a.cnt_)[(uint64_t)e * a.nblk + blockIdx.x] +
                           __popcll(chose[e] & ((1ull << q) - 1));
      if (a.tokens_) gp<int32_t>(a.tokens_)[dst] = (int)(t0 + q);
      if (a.rows_) gp<int32_t>(a.rows_)[dst] = (int)(r0 + i);
    }
    if (r0 + i >= (uint64_t)total) {  // no row of the order lies here
      if (a.tokens_) gp<int32_t>(a.tokens_)[r0 + i] = -1;
      if (a.rows_) gp<int32_t>(a.rows_)[r0 + i] = -1;
    }
  }
}

// ------------------------------------------------------------------- grad ----

struct RouterGradArgs {
  uint64_t logits_, mask_, indices_, counts_, dw_, dloss_, out_;
  uint32_t ls, os, T, E, k, norm;
};

// With h_e = dloss E c_e / (top_k N^2) (c_e has no gradient):
//   dl = p (h - p.h), and for the weights
//   norm_topk:  w (dw - w.dw) at the chosen experts (w is their softmax);
//   otherwise:  p (D - p.D), D = dw at the chosen experts, 0 elsewhere.
template <bool F32, int LPT, int VPT>
__global__ void __launch_bounds__(256) router_grad_kernel(RouterGradArgs a) {
  constexpr int KPL = (kMaxTopK + LPT - 1) / LPT;
  constexpr uint32_t kTokens = 256 / LPT;
  const int lane = threadIdx.x & 63;
  const int l = lane % LPT;
  const uint32_t t = blockIdx.x * kTokens + threadIdx.x / LPT;
  const uint32_t tc = min(t, a.T - 1);
  const bool on = t < a.T && (a.mask_ == 0 || gp<const int32_t>(a.mask_)[tc] != 0);
  float v[VPT], d[VPT], top;
  load_logits<F32, LPT, VPT>(a.logits_, (uint64_t)tc * a.ls, a.E, l, v);
  const TokenState state = token_state<LPT, VPT>(on, v, top);
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    v[i] = expf(v[i] - top);
    s += v[i];
  }
  s = group_sum<LPT>(s);
#pragma unroll
  for (int i = 0; i < VPT; ++i) v[i] = v[i] / s;  // p

  float coef = 0.f;
  if (a.dloss_) {
    const float n = (float)gp<const int32_t>(a.counts_)[a.E];
    coef = n > 0.f ? gp<const float>(a.dloss_)[0] * ((float)a.E / (float)a.k) / n / n : 0.f;
  }
  float dot = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const uint32_t e = l + LPT * i;
    d[i] = (a.dloss_ && e < a.E) ? coef * (float)gp<const int32_t>(a.counts_)[e] : 0.f;
    dot += v[i] * d[i];
  }
  dot = group_sum<LPT>(dot);
#pragma unroll
  for (int i = 0; i < VPT; ++i) d[i] = v[i] * (d[i] - dot);

  if (a.dw_) {
    // lane j of the group (and j + LPT, ...) takes chosen expert j
    int at[KPL];
    float w[KPL], dw[KPL], wsum = 0.f;
#pragma unroll
    for (int i = 0; i < KPL; ++i) {
      const uint32_t j = l + LPT * i;
      at[i] = -1;
      w[i] = 0.f;
      dw[i] = 0.f;
      if (j < a.k) {
        const int e = gp<const int32_t>(a.indices_)[(uint64_t)tc * a.k + j];
        if (e >= 0 && (uint32_t)e < a.E) {
          const uint64_t le = (uint64_t)tc * a.ls + e;
          const float lv = F32 ? gp<const float>(a.logits_)[le]
                               : bf16_to_f32(gp<const uint16_t>(a.logits_)[le]);
          at[i] = e;
          w[i] = expf(lv - top) / s;
          dw[i] = gp<const float>(a.dw_)[(uint64_t)tc * a.k + j];
        }
      }
      wsum += w[i];
    }
    wsum = group_sum<LPT>(wsum);
    float wd = 0.f;
#pragma unroll
    for (int i = 0; i < KPL; ++i) {
      if (a.norm && at[i] >= 0) w[i] /= wsum;
      wd += w[i] * dw[i];
    }
    wd = group_sum<LPT>(wd);
#pragma unroll
    for (int i = 0; i < KPL; ++i) w[i] *= a.norm ? dw[i] - wd : dw[i];
    if (!a.norm) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) d[i] -= v[i] * wd;
    }
#pragma unroll
    for (int i = 0; i < KPL; ++i) {
      for (uint32_t j = 0; j < (uint32_t)LPT && j + LPT * i < a.k; ++j) {
        const int e = __shfl(at[i], (int)j, LPT);
        const float add = __shfl(w[i], (int)j, LPT);
#pragma unroll
        for (int q = 0; q < VPT; ++q)
          if (e == l + LPT * q) d[q] += add;
      }
    }
  }
  if (t >= a.T) return;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const uint32_t e = l + LPT * i;
    if (e >= a.E) continue;
    const float r = state == kRoutes ? d[i] : state == kBad ? __builtin_nanf("") : 0.f;
    const uint64_t o = (uint64_t)t * a.os + e;
    if (F32) gp<float>(a.out_)[o] = r;
    else gp<uint16_t>(a.out_)[o] = (uint16_t)f32_to_bf16(r);
  }
}

// ------------------------------------------------------------------- host ----

static int check_router(const void* logits, int f32, uint32_t ls, uint32_t T, uint32_t E,
                        uint32_t k) {
  if (E == 0 || k == 0 || k > E) return RLD_EINVAL;
  if (E > kMaxExperts || k > kMaxTopK) return RLD_EUNSUPPORTED;
  if ((uint64_t)T * k >= (1ull << 31) || (uint64_t)T * 64 >= (1ull << 32))
    return RLD_EUNSUPPORTED;
  if (T == 0) return RLD_OK;
  if (!logits || ls < E) return RLD_EINVAL;
  if ((uintptr_t)logits & (f32 ? 3u : 1u)) return RLD_EALIGN;
  return RLD_OK;
}

static bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }

// Lanes of a token by the number of experts: eight logits a lane (16 above 512).
template <template <bool, int, int> class K, class A>
static void by_experts(bool f32, uint32_t E, const A& a, hipStream_t st) {
  if (E <= 64) f32 ? K<true, 8, 8>::go(a, st) : K<false, 8, 8>::go(a, st);
  else if (E <= 128) f32 ? K<true, 16, 8>::go(a, st) : K<false, 16, 8>::go(a, st);
  else if (E <= 256) f32 ? K<true, 32, 8>::go(a, st) : K<false, 32, 8>::go(a, st);
  else if (E <= 512) f32 ? K<true, 64, 8>::go(a, st) : K<false, 64, 8>::go(a, st);
  else f32 ? K<true, 64, 16>::go(a, st) : K<false, 64, 16>::go(a, st);
}

template <bool F32, int LPT, int VPT>
struct Route {
  static void go(const RouterArgs& a, hipStream_t st) {
    route_kernel<F32, LPT, VPT><<<a.nblk, 256, 0, st>>>(a);
  }
};

template <bool F32, int LPT, int VPT>
struct RouterGrad {
  static void go(const RouterGradArgs& a, hipStream_t st) {
    router_grad_kernel<F32, LPT, VPT><<<div_ceil(a.T, 256u / LPT), 256, 0, st>>>(a);
  }
};

// An empty batch: no counts, offsets of zero, a loss of zero.
__global__ void router_empty_kernel(RouterArgs a) {
  for (uint32_t e = threadIdx.x; e <= a.E; e += blockDim.x) {
    if (a.counts_) gp<int32_t>(a.counts_)[e] = 0;
    if (a.offsets_) gp<int32_t>(a.offsets_)[e] = 0;
  }
  if (threadIdx.x == 0 && a.loss_) gp<float>(a.loss_)[0] = 0.f;
}

}  // namespace rld

using namespace rld;

extern "C" size_t rld_moe_router_workspace_bytes(uint32_t num_tokens, uint32_t num_experts,
                                                 uint32_t top_k) {
  if (num_tokens == 0 || num_experts == 0 || top_k == 0) return 0;
  const size_t nblk = div_ceil(num_tokens, kRouteTokens);
  return ((size_t)(num_experts + 1) * nblk * 8 + (size_t)(num_experts + 1) * 8 + 15) & ~(size_t)15;
}

extern "C" int rld_moe_router(const void* logits, int logits_f32, uint32_t logits_row_stride,
                              const int32_t* token_mask, uint32_t num_tokens,
                              uint32_t num_experts, uint32_t top_k, int norm_topk,
                              int32_t* indices, float* weights, int32_t* counts,
                              int32_t* expert_offsets, int32_t* sorted_token_ids,
                              int32_t* sorted_rows, float* loss, void* workspace,
                              size_t workspace_bytes, void* stream) {
  const int e = check_router(logits, logits_f32, logits_row_stride, num_tokens, num_experts,
                             top_k);
  if (e) return e;
  if (!aligned4(token_mask) || !aligned4(indices) || !aligned4(weights) || !aligned4(counts) ||
      !aligned4(expert_offsets) || !aligned4(sorted_token_ids) || !aligned4(sorted_rows) ||
      !aligned4(loss))
    return RLD_EALIGN;
  RouterArgs a;
  a.counts_ = (uint64_t)counts;
  a.offsets_ = (uint64_t)expert_offsets;
  a.loss_ = (uint64_t)loss;
  a.T = num_tokens;
  a.E = num_experts;
  const hipStream_t st = (hipStream_t)stream;
  if (num_tokens == 0) {
    if (!counts && !expert_offsets && !loss) return RLD_OK;
    router_empty_kernel<<<1, 256, 0, st>>>(a);
    return launch_status();
  }
  if (!indices || !weights || !workspace) return RLD_EINVAL;
  if (!aligned16(workspace)) return RLD_EALIGN;
  if (workspace_bytes < rld_moe_router_workspace_bytes(num_tokens, num_experts, top_k))
    return RLD_ENOSPACE;
  a.logits_ = (uint64_t)logits;
  a.mask_ = (uint64_t)token_mask;
  a.indices_ = (uint64_t)indices;
  a.weights_ = (uint64_t)weights;
  a.tokens_ = (uint64_t)sorted_token_ids;
  a.rows_ = (uint64_t)sorted_rows;
  a.ls = logits_row_stride;
  a.k = top_k;
  a.norm = norm_topk ? 1u : 0u;
  a.nblk = div_ceil(num_tokens, kRouteTokens);
  const uint64_t cells = (uint64_t)(num_experts + 1) * a.nblk;
  a.cnt_ = (uint64_t)workspace;
  a.psum_ = a.cnt_ + cells * 4;
  a.total_ = a.psum_ + cells * 4;
  a.ptotal_ = a.total_ + (uint64_t)(num_experts + 1) * 4;
  by_experts<Route>(logits_f32 != 0, num_experts, a, st);
  int r = launch_status();
  if (r) return r;
  if (!counts && !expert_offsets && !sorted_token_ids && !sorted_rows && !loss) return RLD_OK;
  router_scan_kernel<<<num_experts + 1, 256, 0, st>>>(a);
  if ((r = launch_status())) return r;
  router_place_kernel<<<a.nblk, 256, 0, st>>>(a);
  return launch_status();
}

extern "C" int rld_moe_router_grad(const void* logits, int logits_f32,
                                   uint32_t logits_row_stride, const int32_t* token_mask,
                                   uint32_t num_tokens, uint32_t num_experts, uint32_t top_k,
                                   int norm_topk, const int32_t* indices, const int32_t* counts,
                                   const float* dweights, const float* dloss, void* dlogits,
                                   uint32_t dlogits_row_stride, void* stream) {
  const int e = check_router(logits, logits_f32, logits_row_stride, num_tokens, num_experts,
                             top_k);
  if (e) return e;
  if (!dweights && !dloss) return RLD_EINVAL;
  if (num_tokens == 0) return RLD_OK;
  if (!dlogits || dlogits_row_stride < num_experts || (dweights && !indices) ||
      (dloss && !counts))
    return RLD_EINVAL;
  if (!aligned4(token_mask) || !aligned4(indices) || !aligned4(counts) || !aligned4(dweights) ||
      !aligned4(dloss) || ((uintptr_t)dlogits & (logits_f32 ? 3u : 1u)))
    return RLD_EALIGN;
  RouterGradArgs a;
  a.logits_ = (uint64_t)logits;
  a.mask_ = (uint64_t)token_mask;
  a.indices_ = (uint64_t)indices;
  a.counts_ = (uint64_t)counts;
  a.dw_ = (uint64_t)dweights;
  a.dloss_ = (uint64_t)dloss;
  a.out_ = (uint64_t)dlogits;
  a.ls = logits_row_stride;
  a.os = dlogits_row_stride;
  a.T = num_tokens;
  a.E = num_experts;
  a.k = top_k;
  a.norm = norm_topk ? 1u : 0u;
  by_experts<RouterGrad>(logits_f32 != 0, num_experts, a, (hipStream_t)stream);
  return launch_status();
}
