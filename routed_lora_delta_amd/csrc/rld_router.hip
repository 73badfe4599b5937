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
// to the last use.  Probabilities, weights and a block's sums of probabilities (at
// most 23 additions) are fp32, the sums over the blocks are 64 bits wide; all sums
// run in a fixed order (per lane over its tokens, over the lanes and waves of a
// block, over the blocks), so results do not change from run to run.
//
// One launch for up to 64 tokens, two otherwise: route (choices, and per block
// of 32 to 128 tokens the counts and probability sums of every expert) and
// place (each row's place in the expert-sorted order, from the counts of all
// blocks); past 32 blocks a scan in between turns the counts into prefix
// sums, so that no place block reads them all (8192 tokens in 64 blocks: 23.6 us
// with the scan, 24.7 without; 32768 in 256: 27.2 and 39.6).  A block keeps 128
// bits per expert of its tokens that chose it: the set bits below a token's
// own are its rank there, whatever order the lanes arrive in.
#include <algorithm>
#include <type_traits>

#include "rld_device.hpp"
#include "rld_internal.hpp"

namespace rld {

constexpr uint32_t kOneBlock = 64;       // tokens up to which one block does everything
constexpr uint32_t kRouteTokens = 128;   // tokens of a block, at most
constexpr uint32_t kPlaceThreads = 1024;
constexpr uint32_t kPlaceWaves = kPlaceThreads / 64;
constexpr uint32_t kScanBlocks = 32;    // token blocks above which the scan is worth a launch
constexpr uint32_t kMaxExperts = 1024;
constexpr uint32_t kMaxTokens = (1u << 26) - 4;
constexpr uint32_t kMaxTopK = 32;

struct RouterArgs {
  uint64_t logits_, mask_, indices_, weights_;
  uint64_t counts_, offsets_, tokens_, rows_, loss_;
  uint64_t cnt_, psum_;      // [nblk][E + 1]: counts (after the scan their prefix sums), [nblk][E]:
                             // sums of p
  uint64_t total_, ptotal_;  // [E + 1], [E]: of the scan
  uint32_t ls, T, E, k, nblk, tokens, norm, scanned;  // tokens: of a block
};

// A value of another lane of the row of 16, in the vector pipe.
template <int CTRL>
__device__ __forceinline__ int dpp(int v) {
  return __builtin_amdgcn_mov_dpp(v, CTRL, 0xf, 0xf, true);
}

// x of the lane that a group's exchange STEP pairs with this one: the lanes 1 and
// 2 away, the mirrored eight and sixteen, the lanes 16 and 32 away.
template <int STEP, class T>
__device__ __forceinline__ T exchange(T x) {
  if constexpr (STEP >= 4) {
    return __shfl_xor(x, 1 << STEP);
  } else {
    constexpr int C = STEP == 0 ? 0xB1 : STEP == 1 ? 0x4E : STEP == 2 ? 0x141 : 0x140;
    if constexpr (sizeof(T) == 8) {
      const uint64_t u = __builtin_bit_cast(uint64_t, x);
      return __builtin_bit_cast(T, (uint64_t)(uint32_t)dpp<C>((int)(uint32_t)u) |
                                       (uint64_t)(uint32_t)dpp<C>((int)(uint32_t)(u >> 32)) << 32);
    } else {
      return __builtin_bit_cast(T, dpp<C>(__builtin_bit_cast(int, x)));
    }
  }
}

// v combined over the LPT lanes of a group, the same bits in each.
template <int LPT, int STEP = 0, class T, class F>
__device__ __forceinline__ T group_all(T v, F f) {
  if constexpr (1 << STEP < LPT) return group_all<LPT, STEP + 1>(f(v, exchange<STEP>(v)), f);
  else return v;
}

template <int LPT>
__device__ __forceinline__ float group_max(float v) {
  return group_all<LPT>(v, [](float x, float y) { return fmaxf(x, y); });
}

template <int LPT>
__device__ __forceinline__ float group_sum(float v) {
  return group_all<LPT>(v, [](float x, float y) { return x + y; });
}

template <int LPT>
__device__ __forceinline__ uint32_t group_umax(uint32_t v) {
  return group_all<LPT>(v, [](uint32_t x, uint32_t y) { return x > y ? x : y; });
}

// exp(d), d <= 0 (NaN as -150, exp of which is 0): 2^n times 2^f with n the
// whole part of d log2(e) and f, within a half, from the product's two parts.
__device__ __forceinline__ float exp_le0(float d) {
  d = fmaxf(d, -150.f);
  const float hi = 1.44269502f, lo = 1.92596299e-8f;  // log2(e)
  const float n = __builtin_rintf(d * hi);
  const float f = __builtin_fmaf(d, lo, __builtin_fmaf(d, hi, -n));
  return __builtin_amdgcn_ldexpf(__builtin_amdgcn_exp2f(f), (int)n);
}

// Keys that order the logits of a token, the lower expert first among equals,
// all different.  BF16: the ordered bits (negative numbers complemented) and
// the expert's complement below them.  fp32: the value as a double, whose
// significand has 29 bits to spare, with the expert (or its complement, where
// more is larger) in the last ten.  -Inf has keys as well, below those of all
// finite values; none() lies below every key.
struct KeyBf16 {
  using T = uint32_t;
  static __device__ __forceinline__ T none() { return 0u; }
  static __device__ __forceinline__ T make(float v, uint32_t e) {
    const uint32_t u = __float_as_uint(v + 0.f);  // -0 as +0
    const uint32_t flip = (uint32_t)((int)u >> 31) | 0x80000000u;
    return ((u ^ flip) & 0xffff0000u) | (0xffffu - e);
  }
  static __device__ __forceinline__ bool finite(T k) { return k > 0x007fffffu; }
  static __device__ __forceinline__ T max(T x, T y) { return x > y ? x : y; }
  static __device__ __forceinline__ T min(T x, T y) { return x > y ? y : x; }
  static __device__ __forceinline__ uint32_t expert(T k) { return 0xffffu - (k & 0xffffu); }
  static __device__ __forceinline__ float value(T k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7fff0000u : ~(k | 0xffffu));
  }
};

struct KeyF32 {
  using T = double;
  static __device__ __forceinline__ T none() { return -__builtin_inf(); }
  static __device__ __forceinline__ T make(float v, uint32_t e) {
    const float z = v + 0.f;  // -0 as +0
    // -Inf as a number below fp32's: its bits with an expert in them are a NaN's
    const uint64_t u = __builtin_bit_cast(uint64_t, max((double)z, -0x1p130));
    const uint32_t flip = (uint32_t)((int)(uint32_t)(u >> 32) >> 31);
    return __builtin_bit_cast(double, u | ((flip ^ (1023u - e)) & 1023u));
  }
  static __device__ __forceinline__ bool finite(T k) { return k > -0x1p129; }
  // (written out: no operand is a NaN that would have to be made quiet first)
  static __device__ __forceinline__ T max(T x, T y) {
    T r;
    asm("v_max_f64 %0, %1, %2" : "=v"(r) : "v"(x), "v"(y));
    return r;
  }
  static __device__ __forceinline__ T min(T x, T y) {
    T r;
    asm("v_min_f64 %0, %1, %2" : "=v"(r) : "v"(x), "v"(y));
    return r;
  }
  static __device__ __forceinline__ uint32_t expert(T k) {
    const uint32_t e = (uint32_t)__builtin_bit_cast(uint64_t, k) & 1023u;
    return k < 0.0 ? e : 1023u - e;
  }
  static __device__ __forceinline__ float value(T k) {
    return (float)__builtin_bit_cast(double, __builtin_bit_cast(uint64_t, k) & ~1023ull);
  }
};

// Sorts N keys, the largest first (odd-even merge sort: 19 exchanges for 8).
template <class K, int N>
__device__ __forceinline__ void sort_keys(typename K::T (&k)[N]) {
#pragma unroll
  for (int p = 1; p < N; p <<= 1)
#pragma unroll
    for (int q = p; q >= 1; q >>= 1)
#pragma unroll
      for (int j = q % p; j + q < N; j += 2 * q)
#pragma unroll
        for (int i = 0; i < q; ++i)
          if (i + j + q < N && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
            const typename K::T x = k[i + j], y = k[i + j + q];
            k[i + j] = K::max(x, y);
            k[i + j + q] = K::min(x, y);
          }
}

// The N largest keys of a group, sorted, in every lane, from each lane's sorted
// keys: at each exchange the larger of one list's and the other's reversed are
// the N largest of both, rising and then falling, which log2(N) rounds sort.
template <class K, int LPT, int N, int STEP = 0>
__device__ __forceinline__ void merge_keys(typename K::T (&k)[N]) {
  if constexpr (1 << STEP < LPT) {
    typename K::T o[N];
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = exchange<STEP>(k[i]);
#pragma unroll
    for (int i = 0; i < N; ++i) k[i] = K::max(k[i], o[N - 1 - i]);
#pragma unroll
    for (int q = N / 2; q >= 1; q >>= 1)
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (!(i & q)) {
          const typename K::T x = k[i], y = k[i + q];
          k[i] = K::max(x, y);
          k[i + q] = K::min(x, y);
        }
    merge_keys<K, LPT, N, STEP + 1>(k);
  }
}

// mine[i]: the group's choice l + LPT i, of the k <= N largest.
template <class K, int LPT, int N, int VPT, int KPL>
__device__ __forceinline__ void choose(const typename K::T (&key)[VPT], int l, uint32_t k,
                                       typename K::T (&mine)[KPL]) {
  typename K::T top[N];
#pragma unroll
  for (int i = 0; i < N; ++i) top[i] = key[i];
  merge_keys<K, LPT, N>(top);
#pragma unroll
  for (int i = 0; i < N; ++i) mine[0] = ((uint32_t)i < k && i == l) ? top[i] : mine[0];
}

// This lane's logits of a token: experts l, l + LPT, ... ; -Inf past E.
template <bool F32, int LPT, int VPT>
__device__ __forceinline__ void load_logits(uint64_t base, uint64_t at, uint32_t E, int l,
                                            float (&v)[VPT]) {
  auto load = [&](uint32_t e) {
    return F32 ? gp<const float>(base)[at + e] : bf16_to_f32(gp<const uint16_t>(base)[at + e]);
  };
  if (E == LPT * VPT) {  // one address, no lane left out
#pragma unroll
    for (int i = 0; i < VPT; ++i) v[i] = load(l + LPT * i);
  } else {
#pragma unroll
    for (int i = 0; i < VPT; ++i) v[i] = load(min((uint32_t)(l + LPT * i), E - 1));
#pragma unroll
    for (int i = 0; i < VPT; ++i) v[i] = l + LPT * i < E ? v[i] : -__builtin_inff();
  }
}

// State of a token: routes (finite largest logit), empty (masked, or nothing
// but -Inf), or bad (a NaN or +Inf among the logits).
enum TokenState { kEmpty, kRoutes, kBad };

template <int LPT, int VPT>
__device__ __forceinline__ TokenState token_state(bool on, const float (&v)[VPT], float& top) {
  float m = -__builtin_inff();
  uint32_t nan = 0;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    m = fmaxf(m, v[i]);
    nan = (v[i] != v[i]) ? 1u : nan;
  }
  top = group_max<LPT>(m);
  const bool bad = group_umax<LPT>(nan) != 0 || top == __builtin_inff();
  if (!on) return kEmpty;
  if (bad) return kBad;
  return top == -__builtin_inff() ? kEmpty : kRoutes;
}

struct PlaceSmem {
  uint64_t chose[2][kMaxExperts];  // tokens 0-63 and 64-127 of the block
  int off[kMaxExperts];            // the place of the block's first row of an expert
  int wsum[kPlaceWaves];
  double dsum[kPlaceWaves];
};

// Sum over the block before this thread, and the block's sum.
__device__ __forceinline__ int block_prefix(int v, int* wsum, int& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int inc = v;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(inc, o);
    if (lane >= o) inc += u;
  }
  if (lane == 63) wsum[wave] = inc;
  __syncthreads();
  int at = inc - v;
  total = 0;
#pragma unroll
  for (uint32_t w = 0; w < kPlaceWaves; ++w) {
    at += w < (uint32_t)wave ? wsum[w] : 0;
    total += wsum[w];
  }
  __syncthreads();
  return at;
}

// The block's rows to their places; block 0 also writes the tables and the
// loss.  total(e), ptotal(e): rows and probability sum of expert e over all
// tokens (total(E): tokens that route); before(e): its rows in earlier blocks;
// index(i): the expert of the block's row i.  `chose` is filled.
template <class Total, class PTotal, class Before, class Index>
__device__ __forceinline__ void place_rows(const RouterArgs& a, uint32_t blk, PlaceSmem& sm,
                                           Total total, PTotal ptotal, Before before,
                                           Index index) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  static_assert(kMaxExperts <= kPlaceThreads, "one expert a thread");
  const uint32_t e1 = threadIdx.x;
  const int c = e1 < a.E ? total(e1) : 0;
  int rows;
  const int at = block_prefix(c, sm.wsum, rows);
  if (e1 < a.E) sm.off[e1] = at + before(e1);
  __syncthreads();
  if (blk == 0) {
    double d = 0.0;
    if (e1 < a.E) {
      if (a.counts_) gp<int32_t>(a.counts_)[e1] = c;
      if (a.offsets_) gp<int32_t>(a.offsets_)[e1] = at;
      d = (double)c * (double)ptotal(e1);
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) d += __shfl_xor(d, o);
    if (lane == 0) sm.dsum[wave] = d;
    __syncthreads();
    if (threadIdx.x == 0) {
      const int n = total(a.E);
      if (a.counts_) gp<int32_t>(a.counts_)[a.E] = n;
      if (a.offsets_) gp<int32_t>(a.offsets_)[a.E] = rows;
      if (a.loss_) {
        double s = 0.0;
        for (uint32_t w = 0; w < kPlaceWaves; ++w) s += sm.dsum[w];
        gp<float>(a.loss_)[0] =
            n ? (float)(s * (double)a.E / ((double)a.k * (double)n * (double)n)) : 0.f;
      }
    }
  }
  if (!a.tokens_ && !a.rows_) return;
  const uint32_t t0 = blk * a.tokens;
  const uint64_t r0 = (uint64_t)t0 * a.k;
  const uint32_t nr = min(a.tokens, a.T - t0) * a.k;
  for (uint32_t i = threadIdx.x; i < nr; i += kPlaceThreads) {
    const int e = index(i);
    if (e >= 0) {
      const uint32_t q = i / a.k;
      const uint64_t m0 = sm.chose[0][e], m1 = sm.chose[1][e];
      const uint32_t rank = q < 64 ? __popcll(m0 & ((1ull << q) - 1))
                                   : __popcll(m0) + __popcll(m1 & ((1ull << (q - 64)) - 1));
      const uint32_t dst = (uint32_t)sm.off[e] + rank;
      if (a.tokens_) gp<int32_t>(a.tokens_)[dst] = (int)(t0 + q);
      if (a.rows_) gp<int32_t>(a.rows_)[dst] = (int)(r0 + i);
    }
    if (r0 + i >= (uint64_t)rows) {  // no row of the order lies here
      if (a.tokens_) gp<int32_t>(a.tokens_)[r0 + i] = -1;
      if (a.rows_) gp<int32_t>(a.rows_)[r0 + i] = -1;
    }
  }
}

// Bound by the issue of vector instructions, some 700 for the tokens that a wave
// takes at once (four of 128 experts), not by memory: 32771 tokens of 128 fp32 logits,
// k 8, in 14.8 us (1.1 TB/s).  512 threads, so that two blocks fit a CU (the call with
// 257 blocks of 128 tokens: 26.9 us against 28.1 of 1024 threads); one block alone
// takes the 1024 of place.  (Loading the next tokens' logits ahead: no gain.)
template <bool F32, int LPT, int VPT, uint32_t THREADS>
__global__ void __launch_bounds__(THREADS) route_kernel(RouterArgs a) {
  constexpr uint32_t kWaves = THREADS / 64;
  constexpr uint32_t kTokensPerWave = 64 / LPT;
  constexpr int KPL = (kMaxTopK + LPT - 1) / LPT;
  __shared__ PlaceSmem sm;
  __shared__ float psum[kWaves][LPT * VPT];
  __shared__ int16_t index[kOneBlock * kMaxTopK];  // of a batch of one block
  __shared__ int live_s;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int l = lane % LPT, grp = lane / LPT;
  const uint32_t t0 = blockIdx.x * a.tokens;
  for (uint32_t e = threadIdx.x; e < a.E; e += THREADS)
    sm.chose[0][e] = sm.chose[1][e] = 0ull;
  if (threadIdx.x == 0) live_s = 0;
  __syncthreads();

  float sum_p[VPT] = {};
  int live = 0;
  const uint32_t here = min(a.tokens, a.T - t0);
  // (a wave stays together: the exchanges take every lane)
  for (uint32_t q0 = wave * kTokensPerWave; q0 < here; q0 += kWaves * kTokensPerWave) {
    const uint32_t q = q0 + grp, t = t0 + q;
    const bool on = q < here && (a.mask_ == 0 || gp<const int32_t>(a.mask_)[min(t, a.T - 1)] != 0);
    float v[VPT], top;
    load_logits<F32, LPT, VPT>(a.logits_, (uint64_t)min(t, a.T - 1) * a.ls, a.E, l, v);
    const TokenState state = token_state<LPT, VPT>(on, v, top);
    float s = 0.f, p[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      p[i] = exp_le0(v[i] - top);
      s += p[i];
    }
    s = group_sum<LPT>(s);
    const float nan = __builtin_nanf(""), inv = 1.f / s;
    // (every p is finite, also of a token that does not route)
    const float share = state == kRoutes ? inv : state == kBad ? nan : 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) sum_p[i] = __builtin_fmaf(p[i], share, sum_p[i]);
    live += state != kEmpty && l == 0;

    // Every lane sorts its keys once.  Up to eight choices the group's lists are
    // merged (32768 tokens, k 8 of 128: fp32 25.2 us against 27.2 by rounds, bf16 the
    // same); for more, a round for each choice takes the largest of their heads.
    // Lane j of the group (and j + LPT, ...) keeps choice j.
    using Key = std::conditional_t<F32, KeyF32, KeyBf16>;
    typename Key::T key[VPT], mine[KPL];
#pragma unroll
    for (int i = 0; i < VPT; ++i) key[i] = Key::make(v[i], l + LPT * i);
    sort_keys<Key>(key);
#pragma unroll
    for (int i = 0; i < KPL; ++i) mine[i] = Key::none();
    if (a.k <= 2) choose<Key, LPT, 2>(key, l, a.k, mine);
    else if (a.k <= 4) choose<Key, LPT, 4>(key, l, a.k, mine);
    else if (a.k <= 8) choose<Key, LPT, 8>(key, l, a.k, mine);
    else
      for (uint32_t j = 0; j < a.k; ++j) {
        const typename Key::T best =
            group_all<LPT>(key[0], [](auto x, auto y) { return Key::max(x, y); });
        const bool own = key[0] == best;
        typename Key::T next[VPT];
#pragma unroll
        for (int i = 0; i + 1 < VPT; ++i) next[i] = key[i + 1];
        next[VPT - 1] = Key::none();
#pragma unroll
        for (int i = 0; i < VPT; ++i) key[i] = own ? next[i] : key[i];
#pragma unroll
        for (int i = 0; i < KPL; ++i) mine[i] = j == (uint32_t)(l + LPT * i) ? best : mine[i];
      }
    int mine_e[KPL];
    float w[KPL], chosen = 0.f;
#pragma unroll
    for (int i = 0; i < KPL; ++i) {
      const bool ok = state == kRoutes && Key::finite(mine[i]);
      mine_e[i] = ok ? (int)Key::expert(mine[i]) : -1;
      w[i] = ok ? exp_le0(Key::value(mine[i]) - top) * inv : 0.f;
      chosen += w[i];
    }
    chosen = group_sum<LPT>(chosen);
    if (q < here) {
#pragma unroll
      for (int i = 0; i < KPL; ++i) {
        const uint32_t j = l + LPT * i;
        if (j >= a.k) continue;
        if (mine_e[i] >= 0) {
          atomicOr((unsigned long long*)&sm.chose[q >> 6][mine_e[i]], 1ull << (q & 63));
          if (a.norm) w[i] /= chosen;
        }
        if (state == kBad) w[i] = nan;
        if (THREADS == kPlaceThreads) index[q * a.k + j] = (int16_t)mine_e[i];
        gp<int32_t>(a.indices_)[(uint64_t)t * a.k + j] = mine_e[i];
        gp<float>(a.weights_)[(uint64_t)t * a.k + j] = w[i];
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
  auto block_psum = [&](uint32_t e) {
    float s = psum[0][e];
    for (uint32_t w = 1; w < kWaves; ++w) s += psum[w][e];
    return s;
  };
  auto block_count = [&](uint32_t e) {
    return e == a.E ? live_s : (int)(__popcll(sm.chose[0][e]) + __popcll(sm.chose[1][e]));
  };
  if constexpr (THREADS < kPlaceThreads) {
    for (uint32_t e = threadIdx.x; e <= a.E; e += THREADS) {
      gp<int32_t>(a.cnt_)[(uint64_t)blockIdx.x * (a.E + 1) + e] = block_count(e);
      if (e < a.E) gp<float>(a.psum_)[(uint64_t)blockIdx.x * a.E + e] = block_psum(e);
    }
  } else {
    place_rows(a, 0, sm, block_count, block_psum, [](uint32_t) { return 0; },
               [&](uint32_t i) { return (int)index[i]; });
  }
}

// 16 experts a block (and the tokens that route): the counts become the
// exclusive prefix sums over the blocks of tokens, in 64 runs of blocks.  6 us for
// 257 blocks and 128 experts, of latency.
__global__ void __launch_bounds__(1024) router_scan_kernel(RouterArgs a) {
  __shared__ int run[64][16];
  __shared__ double fsum[16][16];  // of a wave's four runs (fp32 would drift: a run may
                                   // have 2^13 blocks)
  const int l = threadIdx.x & 15, part = threadIdx.x >> 4;
  const uint32_t e = blockIdx.x * 16 + l, w = a.E + 1;
  const uint32_t per = (a.nblk + 63) / 64, b0 = min(part * per, a.nblk), b1 = min(b0 + per, a.nblk);
  RLD_GLOBAL int32_t* cnt = gp<int32_t>(a.cnt_);
  int n = 0;
  double ps = 0.0;
#pragma unroll 8
  for (uint32_t b = b0; b < b1; ++b) {
    n += e < w ? cnt[(uint64_t)b * w + e] : 0;
    ps += (double)(e < a.E ? gp<const float>(a.psum_)[(uint64_t)b * a.E + e] : 0.f);
  }
  run[part][l] = n;
#pragma unroll
  for (int o = 16; o < 64; o <<= 1) ps += __shfl_xor(ps, o);
  if ((part & 3) == 0) fsum[part >> 2][l] = ps;
  __syncthreads();
  if (e >= w) return;
  int at = 0, total = 0;
#pragma unroll 16
  for (int i = 0; i < 64; ++i) {
    at += i < part ? run[i][l] : 0;
    total += run[i][l];
  }
  for (uint32_t b = b0; b < b1; b += 8) {
    int c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = b + i < b1 ? cnt[(uint64_t)(b + i) * w + e] : 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (b + i < b1) {
        cnt[(uint64_t)(b + i) * w + e] = at;
        at += c[i];
      }
  }
  if (part == 0) {
    gp<int32_t>(a.total_)[e] = total;
    double ptotal = 0.0;
#pragma unroll
    for (int i = 0; i < 16; ++i) ptotal += fsum[i][l];
    if (e < a.E) gp<float>(a.ptotal_)[e] = (float)ptotal;  // one rounding
  }
}

// One block per block of tokens; 7 us for 32771 tokens of 8 rows, whose places are
// scattered stores of 4 bytes.  Without the scan the block adds up all blocks'
// counts itself, and block 0 the probability sums (experts over the lanes, every
// `parts`-th block of tokens a thread; the threads' sums in order).
__global__ void __launch_bounds__(kPlaceThreads) router_place_kernel(RouterArgs a) {
  __shared__ PlaceSmem sm;
  __shared__ int all[kMaxExperts + 1], early[kMaxExperts + 1];
  __shared__ double ps[kPlaceThreads];
  const uint32_t w = a.E + 1, blk = blockIdx.x;
  for (uint32_t e = threadIdx.x; e < w; e += kPlaceThreads) {
    all[e] = early[e] = 0;
    if (e < a.E) sm.chose[0][e] = sm.chose[1][e] = 0ull;
  }
  __syncthreads();
  const RLD_GLOBAL int32_t* cnt = gp<const int32_t>(a.cnt_);
  const uint32_t parts = kPlaceThreads / a.E, part = threadIdx.x / a.E, e1 = threadIdx.x % a.E;
  if (a.scanned) {
    for (uint32_t e = threadIdx.x; e < w; e += kPlaceThreads) {
      all[e] = gp<const int32_t>(a.total_)[e];
      early[e] = cnt[(uint64_t)blk * w + e];
    }
  } else {
    if (part < parts) {
      int n = 0, m = 0;
      double p = 0.0;
#pragma unroll 16
      for (uint32_t b = part; b < a.nblk; b += parts) {
        const int c = cnt[(uint64_t)b * w + e1];
        n += c;
        m += b < blk ? c : 0;
      }
      if (blk == 0) {
#pragma unroll 16
        for (uint32_t b = part; b < a.nblk; b += parts)
          p += (double)gp<const float>(a.psum_)[(uint64_t)b * a.E + e1];
      }
      ps[threadIdx.x] = p;
      atomicAdd(&all[e1], n);  // whole numbers: any order gives the same sum
      atomicAdd(&early[e1], m);
    }
    if (blk == 0) {
      int n = 0;
      for (uint32_t b = threadIdx.x; b < a.nblk; b += kPlaceThreads) n += cnt[(uint64_t)b * w + a.E];
      if (n) atomicAdd(&all[a.E], n);
    }
  }
  const uint32_t t0 = blk * a.tokens;
  const uint64_t r0 = (uint64_t)t0 * a.k;
  const uint32_t nr = min(a.tokens, a.T - t0) * a.k;
  for (uint32_t i = threadIdx.x; i < nr; i += kPlaceThreads) {
    const int e = gp<const int32_t>(a.indices_)[r0 + i];
    const uint32_t q = i / a.k;
    if (e >= 0) atomicOr((unsigned long long*)&sm.chose[q >> 6][e], 1ull << (q & 63));
  }
  __syncthreads();
  place_rows(
      a, blk, sm, [&](uint32_t e) { return all[e]; },
      [&](uint32_t e) {
        if (a.scanned) return (double)gp<const float>(a.ptotal_)[e];
        double p = ps[e];
        for (uint32_t i = 1; i < parts; ++i) p += ps[i * a.E + e];
        return p;
      },
      [&](uint32_t e) { return early[e]; },
      [&](uint32_t i) { return gp<const int32_t>(a.indices_)[r0 + i]; });
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
// One pass, bound by memory once tokens are many: 32771 tokens of 128 fp32 logits in
// 9.8 us, 36 MB at 3.7 TB/s; 4096 of bf16 take 5.3 us a call, most of it the launch's.
template <bool F32, int LPT, int VPT>
__global__ void __launch_bounds__(256) router_grad_kernel(RouterGradArgs a) {
  constexpr int KPL = (kMaxTopK + LPT - 1) / LPT;
  constexpr uint32_t kTokens = 256 / LPT;
  __shared__ float spread[kTokens][LPT * VPT];
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
    v[i] = exp_le0(v[i] - top);
    s += v[i];
  }
  const float inv = 1.f / group_sum<LPT>(s);
#pragma unroll
  for (int i = 0; i < VPT; ++i) v[i] *= inv;  // p

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
    // lane j of the group (and j + LPT, ...) takes chosen expert j and adds its
    // gradient at that expert's place in LDS, which the expert's lane reads
    float* const add = spread[threadIdx.x / LPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) add[l + LPT * i] = 0.f;
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
          w[i] = exp_le0(lv - top) * inv;
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
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < KPL; ++i)
      if (at[i] >= 0) atomicAdd(&add[at[i]], w[i] * (a.norm ? dw[i] - wd : dw[i]));
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      if (!a.norm) d[i] -= v[i] * wd;
      d[i] += add[l + LPT * i];
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
  // a grid holds fewer than 2^32 threads: at most 64 a token, in blocks of 256
  if ((uint64_t)T * k >= (1ull << 31) || T > kMaxTokens) return RLD_EUNSUPPORTED;
  if (T == 0) return RLD_OK;
  if (!logits || ls < E) return RLD_EINVAL;
  if ((uintptr_t)logits & (f32 ? 3u : 1u)) return RLD_EALIGN;
  return RLD_OK;
}

// Tokens of a block: as few as keep the blocks within one for each CU, since a
// CU takes 2 to 3 us for 32 of them (k = 8 of 128 experts, us with blocks of 128
// against these: 256 tokens 16.4 and 11.1, 4096 19.3 and 15.9, 16384 22.0 and 19.5).
static uint32_t block_tokens(uint32_t T) {
  if (T <= kOneBlock) return kOneBlock;
  uint32_t n = kRouteTokens;
  while (n > 32 && div_ceil(T, n / 2) <= 256) n /= 2;
  return n;
}

static size_t router_bytes(size_t blocks, size_t experts) {
  return ((experts + 1) * blocks * 8 + (experts + 1) * 8 + 15) & ~(size_t)15;
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
    if (a.nblk > 1) route_kernel<F32, LPT, VPT, 512><<<a.nblk, 512, 0, st>>>(a);
    else route_kernel<F32, LPT, VPT, kPlaceThreads><<<1, kPlaceThreads, 0, st>>>(a);
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
  // a call of fewer tokens may have up to 256 blocks of 32
  const uint32_t blocks = div_ceil(num_tokens, block_tokens(num_tokens));
  return router_bytes(std::max(blocks, std::min(div_ceil(num_tokens, 32u), 256u)), num_experts);
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
  if (workspace_bytes < router_bytes(div_ceil(num_tokens, block_tokens(num_tokens)), num_experts))
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
  a.tokens = block_tokens(num_tokens);
  a.nblk = div_ceil(num_tokens, a.tokens);
  a.scanned = a.nblk > kScanBlocks ? 1u : 0u;
  const uint64_t cells = (uint64_t)(num_experts + 1) * a.nblk;
  a.cnt_ = (uint64_t)workspace;
  a.psum_ = a.cnt_ + cells * 4;
  a.total_ = a.psum_ + cells * 4;
  a.ptotal_ = a.total_ + (uint64_t)(num_experts + 1) * 4;
  by_experts<Route>(logits_f32 != 0, num_experts, a, st);
  int r = launch_status();
  if (r) return r;
  if (!counts && !expert_offsets && !sorted_token_ids && !sorted_rows && !loss) return RLD_OK;
  if (a.nblk == 1) return RLD_OK;  // placed in the first launch
  if (a.scanned) {
    router_scan_kernel<<<div_ceil(num_experts + 1, 16), 1024, 0, st>>>(a);
    if ((r = launch_status())) return r;
  }
  router_place_kernel<<<a.nblk, kPlaceThreads, 0, st>>>(a);
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
