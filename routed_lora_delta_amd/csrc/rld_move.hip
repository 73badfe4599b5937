// MoE token movement: tokens to the experts' order and back, and the gradients.
//
// A flat row f = t * top_k + j is choice j of token t.  The router's sorted_rows
// names the flat row of each expert-sorted row p; places is its inverse, written
// by the dispatch.  Row p belongs to f where places[f] = p and sorted_rows[p] = f,
// and only there: an entry of places that no dispatch wrote may hold anything and
// finds no row.
//
//   dispatch       rows[p] = x[f / top_k]
//   combine        out[t] = sum_j w[t, j] rows[p(t, j)] + add[t]
//   dispatch_grad  the same sum without weights
//   combine_grad   drows[p(t, j)] = w[t, j] dout[t],  dw[t, j] = rows[p(t, j)] . dout[t]
//
// All of them are bound by memory.  A lane holds 16 bytes of a row (a unit): a
// wave's access is 1 KB of one row, contiguous, or 512 bytes of each of two where a row
// has up to 32 units, 256 of each of four where it has up to 16.  (us so and with a wave
// for each row: 128 MB of 8 rows of 64 BF16 a token, combine 29 and 60, its gradient 56
// and 131, dispatch 37 and 46; 200 MB of 2 rows of 192 64 and 87, 92 and 147, 60 and 80;
// of 8 rows of 256 41 and 41, 76 and 78, 41 and 41.)  What is read once and what is
// written passes the caches by (load_once, store_once), which costs a reader of the
// result nothing and still finds what a writer before left in them: dispatch of 4096
// tokens to 8 rows of 2048 BF16 each and a pass over the rows take 65.3 us so, 68.9
// otherwise; of 16384 237 and 286; a copy into 64 MB of rows and their combine 36.8 and
// 37.8.
#include "rld_device.hpp"
#include "rld_internal.hpp"

namespace rld {

constexpr uint32_t kMaxMoveTopK = 32;
constexpr uint32_t kMaxMoveWidth = 1u << 21;  // a row's bytes fit 32 bits

// What 16 bytes hold: 8 BF16 or 4 fp32.
template <bool F32>
struct Unit {
  static constexpr int N = F32 ? 4 : 8;
  static __device__ __forceinline__ void open(const u32x4& u, float* v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (F32) {
        v[i] = __uint_as_float(u[i]);
      } else {
        v[2 * i] = __uint_as_float(u[i] << 16);
        v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
      }
    }
  }
  static __device__ __forceinline__ u32x4 close(const float* v) {
    u32x4 u;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      u[i] = F32 ? __float_as_uint(v[i]) : pack_bf16x2(v[2 * i], v[2 * i + 1]);
    return u;
  }
};

// A group of G lanes works on one token (or row): the whole wave, or 16 or 32 lanes of
// it.
// What the group has in common is in scalar registers if it is the wave.  Branches
// around from() and vote() are the same for a whole group.
template <int G>
struct Group {
  uint32_t base, lane;  // the group's first lane; this lane within it
  __device__ __forceinline__ Group() {
    const uint32_t l = threadIdx.x & 63;
    base = G == 64 ? 0u : l & ~(uint32_t)(G - 1);
    lane = l - base;
  }
  __device__ __forceinline__ uint32_t same(uint32_t v) const { return G == 64 ? uniform(v) : v; }
  template <class T>
  __device__ __forceinline__ T from(T v, int lane) const {
    return G == 64 ? from_lane(v, lane) : __shfl(v, base + lane);
  }
  // the group's bits of a vote
  __device__ __forceinline__ uint64_t vote(bool v) const {
    const uint64_t m = __ballot(v);
    return G == 64 ? m : m >> base & ((1ull << (G & 63)) - 1);
  }
};

// Threads of a block in groups: the number of this thread's.
template <int G>
__device__ __forceinline__ uint32_t group_number() {
  return (blockIdx.x * blockDim.x + threadIdx.x) / G;
}

// ---------------------------------------------------------------- dispatch ----

struct DispatchArgs {
  uint64_t x_, sorted_, rows_, places_;
  uint64_t xs, rs;  // bytes of a row
  uint32_t T, n, k, units, slices;
};

// A group copies kRowUnits units a lane of one sorted row.
constexpr int kRowUnits = 2;

template <int G>
__global__ void __launch_bounds__(256) dispatch_rows_kernel(DispatchArgs a) {
  const Group<G> g;
  const uint32_t item = g.same(group_number<G>());
  const uint32_t p = G < 64 ? item : item / a.slices, slice = G < 64 ? 0 : item - p * a.slices;
  if (p >= a.n) return;
  const uint32_t f = g.same((uint32_t)gp<const int32_t>(a.sorted_)[p]);
  if (f >= a.n) return;
  if (slice == 0 && g.lane == 0) gp<int32_t>(a.places_)[f] = (int32_t)p;
  const uint32_t u0 = slice * (64u * kRowUnits) + g.lane;
  const uint64_t from = a.x_ + (f / a.k) * a.xs, to = a.rows_ + p * a.rs;
  u32x4 v[kRowUnits];
#pragma unroll
  for (int i = 0; i < kRowUnits; ++i)
    if (u0 + G * i < a.units) v[i] = load_unit(from, (u0 + G * i) * 16u);
#pragma unroll
  for (int i = 0; i < kRowUnits; ++i)
    if (u0 + G * i < a.units) store_once(to, (u0 + G * i) * 16u, v[i]);
}

__global__ void __launch_bounds__(256) dispatch_places_kernel(DispatchArgs a) {
  const uint32_t p = blockIdx.x * 256u + threadIdx.x;
  if (p >= a.n) return;
  const uint32_t f = (uint32_t)gp<const int32_t>(a.sorted_)[p];
  if (f < a.n) gp<int32_t>(a.places_)[f] = (int32_t)p;
}

// The second launch of large calls: a group reads G units of a token once and writes
// them to each of its rows.
template <int G>
__global__ void __launch_bounds__(256) dispatch_tokens_kernel(DispatchArgs a) {
  const Group<G> g;
  const uint32_t item = g.same(group_number<G>());
  const uint32_t t = G < 64 ? item : item / a.slices, slice = G < 64 ? 0 : item - t * a.slices;
  if (t >= a.T) return;
  const uint32_t u = slice * 64u + g.lane;
  const uint32_t at = min(u, a.units - 1u) * 16u;
  const u32x4 v = load_unit(a.x_ + t * a.xs, at);
  for (uint32_t j0 = 0; j0 < a.k; j0 += G) {
    const bool in = j0 + g.lane < a.k;
    const uint32_t f = t * a.k + (in ? j0 + g.lane : j0);
    uint32_t p = (uint32_t)gp<const int32_t>(a.places_)[f];
    const bool have = in && p < a.n;
    p = have ? p : 0u;
    uint64_t own = g.vote(have && (uint32_t)gp<const int32_t>(a.sorted_)[p] == f);
    while (own) {
      const int j = __builtin_ctzll(own);
      own &= own - 1;
      const uint64_t row = a.rows_ + g.from(p, j) * a.rs;
      if (u < a.units) store_once(row, at, v);
    }
  }
}

// ----------------------------------------------------------------- combine ----

struct CombineArgs {
  uint64_t rows_, indices_, sorted_, places_, weights_, add_, out_;
  uint64_t rs, as, os;  // bytes of a row
  uint32_t T, n, k, units, slices;
};

// The rows of a token's choices j0 .. j0 + KB - 1: lane j of the group holds choice
// j0 + j.  `have` has a bit for each row that can be read; own() one for each of them
// that belongs to its choice, which takes one load more.  The sums call it once the
// rows' loads are out; combine's gradient, whose stores need it, before them, and waits
// for it by itself.
template <int G>
struct Choices {
  uint32_t row, back, f;
  uint64_t have;
  __device__ __forceinline__ uint64_t own(const Group<G>& g) {
    asm volatile("" : "+v"(back) : : "memory");  // the comparison stays behind those loads
    return have & g.vote(back == f);
  }
};

// Loads without a branch, from clamped places.
template <bool SORTED, int KB, int G, class A>
__device__ __forceinline__ Choices<G> find_choices(const A& a, const Group<G>& g, uint32_t t,
                                                   uint32_t j0) {
  const bool in = g.lane < KB && j0 + g.lane < a.k;
  Choices<G> c;
  c.f = t * a.k + (in ? j0 + g.lane : j0);
  c.row = c.back = c.f;
  bool have = in;
  if (SORTED) {
    const uint32_t p = (uint32_t)gp<const int32_t>(a.places_)[c.f];
    have = in && p < a.n;
    c.row = have ? p : 0u;
    c.back = (uint32_t)gp<const int32_t>(a.sorted_)[c.row];
  } else if (a.indices_) {
    const int32_t e = gp<const int32_t>(a.indices_)[c.f];
    have = in && e >= 0;
  }
  c.have = g.vote(have);
  return c;
}

// A group adds up one slice of G units of a token's rows, in fp32, j ascending: eight
// rows' loads at a time, the places before them, the check and the weights beside
// them.  32771 tokens of 8 rows of 2048 BF16, onto a residual: 209 us, 5.9 TB/s.
template <bool F32, bool SORTED, int G>
__global__ void __launch_bounds__(256) combine_kernel(CombineArgs a) {
  constexpr int N = Unit<F32>::N;
  const Group<G> g;
  const uint32_t item = g.same(group_number<G>());
  const uint32_t t = G < 64 ? item : item / a.slices, slice = G < 64 ? 0 : item - t * a.slices;
  if (t >= a.T) return;
  const uint32_t u = slice * 64u + g.lane;
  const uint32_t at = min(u, a.units - 1u) * 16u;  // lanes past the row load its last unit
  u32x4 last = {0u, 0u, 0u, 0u};
  if (a.add_) last = load_once(a.add_ + t * a.as, at);
  float acc[N];
#pragma unroll
  for (int i = 0; i < N; ++i) acc[i] = 0.f;
#pragma nounroll
  for (uint32_t j0 = 0; j0 < a.k; j0 += 8) {
    Choices<G> c = find_choices<SORTED, 8>(a, g, t, j0);
    float w = 1.f;
    if (a.weights_) w = gp<const float>(a.weights_)[c.f];
    u32x4 r[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      r[j] = u32x4{0u, 0u, 0u, 0u};
      if ((c.have >> j) & 1u) r[j] = load_once(a.rows_ + g.from(c.row, j) * a.rs, at);
    }
    const uint64_t own = c.own(g);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if ((own >> j) & 1u) {
        const float wj = g.from(w, j);
        float v[N];
        Unit<F32>::open(r[j], v);
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] += wj * v[i];
      }
    }
  }
  float v[N];
  Unit<F32>::open(last, v);
#pragma unroll
  for (int i = 0; i < N; ++i) acc[i] += v[i];
  if (u < a.units) store_once(a.out_ + t * a.os, at, Unit<F32>::close(acc));
}

// ------------------------------------------------------------ combine grad ----

struct CombineGradArgs {
  uint64_t rows_, indices_, sorted_, places_, weights_, dout_, drows_, dweights_;
  uint64_t rs, ds, os;  // bytes of a row of rows, dout, drows
  uint32_t T, n, k, units, waves;
};

// Sums of KB values over a group: each of the first exchanges halves the values that
// a lane holds (10 exchanges for eight over a wave).  Lane G / KB * i of the group
// gets the sum of v[i].
template <int KB, int G>
__device__ __forceinline__ float sum_each(float* v, uint32_t lane) {
  int m = G / 2;
#pragma unroll
  for (int half = KB / 2; half >= 1; half >>= 1, m >>= 1) {
    const bool up = (lane & m) != 0;
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const float keep = up ? v[i + half] : v[i];
      const float give = up ? v[i] : v[i + half];
      v[i] = keep + __shfl_xor(give, m);
    }
  }
  float s = v[0];
#pragma unroll
  for (; m >= 1; m >>= 1) s += __shfl_xor(s, m);
  return s;
}

// Units of a row that a lane of combine_grad takes at a time, by the rows it takes: 62500
// tokens of one row of 2048 BF16 118 us with two, 123 with one or four.  Two rows are
// within 10 percent either way (us with two and one: 31250 tokens of 2048 BF16 104 and
// 102, 64000 of 1000 121 and 113, 123076 of 520 129 and 133, 61538 of 520 fp32 115 and
// 133).
__host__ __device__ constexpr uint32_t units_per_lane(uint32_t rows) { return rows > 2 ? 1 : 2; }

// `waves` groups share a token's columns (one, if groups are narrow).  A group takes KB
// of its rows and UPL units a lane of each at a time.  A row's unit is read before the
// same thread writes it, so drows may be rows.  16387 tokens of 8 rows of 2048 BF16: 204
// us, 5.05 TB/s, where a copy reaches 5.2 (more waves a CU, by fewer registers, spill).
template <bool F32, bool SORTED, int KB, int G>
__global__ void __launch_bounds__(1024) combine_grad_kernel(CombineGradArgs a) {
  constexpr int N = Unit<F32>::N, UPL = units_per_lane(KB);
  __shared__ float part[16][KB];
  const Group<G> g;
  const uint32_t waves = G < 64 ? 1u : a.waves;
  const uint32_t wave = uniform(threadIdx.x >> 6), w0 = wave & (waves - 1u), first = wave - w0;
  const uint32_t t = g.same(group_number<G>()) / waves;
  const bool on = t < a.T;
#pragma nounroll
  for (uint32_t j0 = 0; j0 < a.k; j0 += KB) {
    float dot[KB];
#pragma unroll
    for (int j = 0; j < KB; ++j) dot[j] = 0.f;
    uint64_t own = 0;
    if (on) {
      Choices<G> c = find_choices<SORTED, KB>(a, g, t, j0);
      float w = 0.f;
      if (a.drows_) w = gp<const float>(a.weights_)[c.f];
      own = c.own(g);
      // a wave's lanes past the row leave the loop; a narrow group stays together, once
      for (uint32_t u0 = w0 * (G * UPL) + g.lane; G < 64 ? u0 == g.lane : u0 < a.units;
           u0 += G * UPL * waves) {
        const auto in = [&](int q) { return (G == 64 && q == 0) || u0 + G * q < a.units; };
        u32x4 dv[UPL], r[UPL][KB];
        // zeros past the row, as r has there: infinity times 0 is NaN (loads under a branch
        // instead take 60 us, not 49, for 20833 tokens of 4 rows of 768 BF16)
#pragma unroll
        for (int q = 0; q < UPL; ++q) {
          dv[q] = load_once(a.dout_ + t * a.ds, min(u0 + G * q, a.units - 1u) * 16u);
          if (!in(q)) dv[q] = u32x4{0u, 0u, 0u, 0u};
        }
        if (a.dweights_) {
#pragma unroll
          for (int j = 0; j < KB; ++j) {
#pragma unroll
            for (int q = 0; q < UPL; ++q) r[q][j] = u32x4{0u, 0u, 0u, 0u};
            if ((c.have >> j) & 1u) {
              const uint64_t row = a.rows_ + g.from(c.row, j) * a.rs;
#pragma unroll
              for (int q = 0; q < UPL; ++q)
                if (in(q)) r[q][j] = load_once(row, (u0 + G * q) * 16u);
            }
          }
        }
#pragma unroll
        for (int q = 0; q < UPL; ++q) {
          float d[N];
          Unit<F32>::open(dv[q], d);
          if (a.dweights_) {
#pragma unroll
            for (int j = 0; j < KB; ++j) {
              float v[N];
              Unit<F32>::open(r[q][j], v);
#pragma unroll
              for (int i = 0; i < N; ++i) dot[j] += d[i] * v[i];
            }
          }
          if (a.drows_) {
#pragma unroll
            for (int j = 0; j < KB; ++j) {
              if ((own >> j) & 1u) {
                const float wj = g.from(w, j);
                const uint64_t row = a.drows_ + g.from(c.row, j) * a.os;
                float v[N];
#pragma unroll
                for (int i = 0; i < N; ++i) v[i] = wj * d[i];
                if (in(q)) store_once(row, (u0 + G * q) * 16u, Unit<F32>::close(v));
              }
            }
          }
        }
      }
    }
    if (!a.dweights_) continue;
    float s = sum_each<KB, G>(dot, g.lane);
    const uint32_t j = g.lane / (G / KB);
    const bool mine = g.lane % (G / KB) == 0;
    if (waves > 1) {
      if (j0) __syncthreads();
      if (mine) part[wave][j] = s;
      __syncthreads();
      s = part[first][j];
      for (uint32_t v = 1; v < waves; ++v) s += part[first + v][j];
    }
    if (on && w0 == 0 && mine && j0 + j < a.k)
      gp<float>(a.dweights_)[(uint64_t)t * a.k + j0 + j] = ((own >> j) & 1u) ? s : 0.f;
  }
}

// -------------------------------------------------------------------- host ----

static bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }

static int check_move(uint32_t T, uint32_t k, uint32_t width) {
  if (k == 0 || width == 0) return RLD_EINVAL;
  if (k > kMaxMoveTopK || width > kMaxMoveWidth || (uint64_t)T * k >= (1ull << 31))
    return RLD_EUNSUPPORTED;
  if (!mult8(width)) return RLD_EALIGN;
  return RLD_OK;
}

static uint32_t units_of(uint32_t width, int f32) { return width / (f32 ? 4u : 8u); }

// One wave for each item, in a grid of fewer than 2^32 threads.
static bool too_many(uint64_t items) { return items > (1ull << 26) - 4; }

// Lanes of a group by a row's units, and a launch by them.
template <int G>
struct Lanes {
  static constexpr int N = G;
};

template <class F>
static void by_lanes(uint32_t units, F launch) {
  if (units <= 16) launch(Lanes<16>());
  else if (units <= 32) launch(Lanes<32>());
  else launch(Lanes<64>());
}

// Where the rows of the choices are: both tables, or neither (flat order).
static int check_tables(const int32_t* indices, const int32_t* sorted_rows,
                        const int32_t* places) {
  if ((sorted_rows == nullptr) != (places == nullptr)) return RLD_EINVAL;
  return aligned4(indices) && aligned4(sorted_rows) && aligned4(places) ? RLD_OK : RLD_EALIGN;
}

// Blocks of one wave, but of four where rows share cache lines, which the waves of one
// block then find in their CU (us with one and four, rows of 2048 BF16, top_k 8: 32771
// tokens in whole lines 209 and 214, 256 MB of rows 16 bytes apart 58 and 54; of 768 66
// and 56).
template <bool F32, bool SORTED>
static void launch_combine(const CombineArgs& a, hipStream_t s) {
  const uint32_t threads = ((a.rows_ | a.rs) & 127u) == 0 ? 64 : 256;
  by_lanes(a.units, [&](auto lanes) {
    constexpr int G = decltype(lanes)::N;
    const uint32_t blocks = div_ceil(a.T * (G < 64 ? 1 : a.slices), threads / G);
    combine_kernel<F32, SORTED, G><<<blocks, threads, 0, s>>>(a);
  });
}

static int combine(const void* rows, int f32, uint32_t rs, const int32_t* indices,
                   const int32_t* sorted_rows, const int32_t* places, const float* weights,
                   uint32_t T, uint32_t k, uint32_t width, const void* add, uint32_t as,
                   void* out, uint32_t os, void* stream) {
  int st = check_move(T, k, width);
  if (st || T == 0) return st;
  if ((st = check_rows(rows, rs, width))) return st;
  if ((st = check_rows(out, os, width))) return st;
  if (add && (st = check_rows(add, as, width))) return st;
  if ((st = check_tables(indices, sorted_rows, places))) return st;
  if (!aligned4(weights)) return RLD_EALIGN;
  const uint64_t size = f32 ? 4 : 2;
  CombineArgs a;
  a.rows_ = (uint64_t)rows;
  a.indices_ = (uint64_t)indices;
  a.sorted_ = (uint64_t)sorted_rows;
  a.places_ = (uint64_t)places;
  a.weights_ = (uint64_t)weights;
  a.add_ = (uint64_t)add;
  a.out_ = (uint64_t)out;
  a.rs = rs * size;
  a.as = as * size;
  a.os = os * size;
  a.T = T;
  a.n = T * k;
  a.k = k;
  a.units = units_of(width, f32);
  a.slices = div_ceil(a.units, 64);
  if (too_many((uint64_t)T * a.slices)) return RLD_EUNSUPPORTED;
  hipStream_t s = (hipStream_t)stream;
  if (f32)
    places ? launch_combine<true, true>(a, s) : launch_combine<true, false>(a, s);
  else
    places ? launch_combine<false, true>(a, s) : launch_combine<false, false>(a, s);
  return launch_status();
}

template <bool F32, bool SORTED, int KB>
static void launch_combine_grad(const CombineGradArgs& a, hipStream_t s) {
  by_lanes(a.units, [&](auto lanes) {
    constexpr int G = decltype(lanes)::N;
    const uint32_t group = G < 64 ? G : 64 * a.waves, threads = group > 256 ? group : 256;
    combine_grad_kernel<F32, SORTED, KB, G>
        <<<div_ceil(a.T, threads / group), threads, 0, s>>>(a);
  });
}

// Waves of a token: as many as take its columns at once, up to 8; 16 where 8 would take
// more than twice as long.  (us with 4, 8 and 16, 256 MB of 8 rows a token: 4096 BF16
// 91, 88 and 89, 8192 BF16 97, 93 and 97, 8192 fp32 98, 94 and 92; of 7 tokens of 8192
// BF16 9.0, 7.5 and 7.6, of 3 of fp32 17.7, 11.9 and 9.9.)
template <bool F32, bool SORTED>
static void launch_combine_grad(CombineGradArgs a, hipStream_t s) {
  const uint32_t units = 64 * units_per_lane(a.k);
  a.waves = 1;
  while (a.waves < 8 && a.waves * units < a.units) a.waves *= 2;
  if (2 * 8 * units < a.units) a.waves = 16;
  while (too_many((uint64_t)a.T * a.waves)) a.waves /= 2;
  if (a.k > 4) launch_combine_grad<F32, SORTED, 8>(a, s);
  else if (a.k > 2) launch_combine_grad<F32, SORTED, 4>(a, s);
  else if (a.k > 1) launch_combine_grad<F32, SORTED, 2>(a, s);
  else launch_combine_grad<F32, SORTED, 1>(a, s);
}

}  // namespace rld

using namespace rld;

extern "C" int rld_moe_dispatch(const void* x, int rows_f32, uint32_t x_row_stride,
                                uint32_t num_tokens, uint32_t top_k, uint32_t width,
                                const int32_t* sorted_rows, void* rows, uint32_t rows_row_stride,
                                int32_t* places, void* stream) {
  int st = check_move(num_tokens, top_k, width);
  if (st || num_tokens == 0) return st;
  if ((st = check_rows(x, x_row_stride, width))) return st;
  if ((st = check_rows(rows, rows_row_stride, width))) return st;
  if (!sorted_rows || !places) return RLD_EINVAL;
  if (!aligned4(sorted_rows) || !aligned4(places)) return RLD_EALIGN;
  const uint64_t size = rows_f32 ? 4 : 2;
  DispatchArgs a;
  a.x_ = (uint64_t)x;
  a.sorted_ = (uint64_t)sorted_rows;
  a.rows_ = (uint64_t)rows;
  a.places_ = (uint64_t)places;
  a.xs = x_row_stride * size;
  a.rs = rows_row_stride * size;
  a.T = num_tokens;
  a.n = num_tokens * top_k;
  a.k = top_k;
  a.units = units_of(width, rows_f32);
  a.slices = div_ceil(a.units, 64);
  if (too_many((uint64_t)a.n * a.slices)) return RLD_EUNSUPPORTED;
  hipStream_t s = (hipStream_t)stream;
  // Reading a token once saves top_k - 1 reads of it, from the caches mostly, and
  // costs a launch: us with one launch and with two, 2048 BF16 a row, top_k 8: 512
  // tokens 5.2 and 6.4, 1024 (29 MB saved) 9.0 and 9.1, 4096 33.3 and 27.2, 16384 136
  // and 98; rows of 4096, top_k 2: 1024 6.1 and 6.8, 4096 (34 MB) 18.9 and 18.1.  Rows
  // that share cache lines are better written in order, so that their parts meet: 1000
  // BF16, top_k 6, 106 MB saved 34.7 and 35.8, 333 MB 110 and 105; 264, top_k 8, 147 MB
  // 59.5 and 57.0, top_k 2, 131 and 105; but 2056, top_k 8, 46 and 51.  Of up to 32 units,
  // which share a wave, they always are: 200, top_k 8, 147 MB saved 53 and 64, 315 MB 115
  // and 132, top_k 2, 147 MB 111 and 118; 136, top_k 8, 57 and 74; 72, 350 MB 169 and 254.
  const uint64_t saved = (uint64_t)(a.n - a.T) * width * size;
  const bool lines = ((a.rows_ | a.rs | width * size) & 127u) == 0;
  const bool twice = lines ? saved >= (32u << 20) : a.units > 32 && saved >= (128u << 20);
  if (twice) dispatch_places_kernel<<<div_ceil(a.n, 256), 256, 0, s>>>(a);
  else a.slices = div_ceil(a.units, 64u * kRowUnits);
  by_lanes(a.units, [&](auto lanes) {
    constexpr int G = decltype(lanes)::N;
    const uint32_t blocks = div_ceil((twice ? a.T : a.n) * a.slices, 256 / G);
    if (twice) dispatch_tokens_kernel<G><<<blocks, 256, 0, s>>>(a);
    else dispatch_rows_kernel<G><<<blocks, 256, 0, s>>>(a);
  });
  return launch_status();
}

extern "C" int rld_moe_dispatch_grad(const void* drows, int rows_f32, uint32_t drows_row_stride,
                                     const int32_t* sorted_rows, const int32_t* places,
                                     uint32_t num_tokens, uint32_t top_k, uint32_t width,
                                     const void* add, uint32_t add_row_stride, void* dx,
                                     uint32_t dx_row_stride, void* stream) {
  if (num_tokens && (!sorted_rows || !places)) return RLD_EINVAL;
  return combine(drows, rows_f32, drows_row_stride, nullptr, sorted_rows, places, nullptr,
                 num_tokens, top_k, width, add, add_row_stride, dx, dx_row_stride, stream);
}

extern "C" int rld_moe_combine(const void* rows, int rows_f32, uint32_t rows_row_stride,
                               const int32_t* indices, const int32_t* sorted_rows,
                               const int32_t* places, const float* weights, uint32_t num_tokens,
                               uint32_t top_k, uint32_t width, const void* add,
                               uint32_t add_row_stride, void* out, uint32_t out_row_stride,
                               void* stream) {
  if (num_tokens && !weights) return RLD_EINVAL;
  return combine(rows, rows_f32, rows_row_stride, indices, sorted_rows, places, weights,
                 num_tokens, top_k, width, add, add_row_stride, out, out_row_stride, stream);
}

extern "C" int rld_moe_combine_grad(const void* rows, int rows_f32, uint32_t rows_row_stride,
                                    const int32_t* indices, const int32_t* sorted_rows,
                                    const int32_t* places, const float* weights, const void* dout,
                                    uint32_t dout_row_stride, uint32_t num_tokens, uint32_t top_k,
                                    uint32_t width, void* drows, uint32_t drows_row_stride,
                                    float* dweights, void* stream) {
  int st = check_move(num_tokens, top_k, width);
  if (st) return st;
  if (!drows && !dweights) return RLD_EINVAL;
  if (num_tokens == 0) return RLD_OK;
  if ((st = check_rows(dout, dout_row_stride, width))) return st;
  if (dweights && (st = check_rows(rows, rows_row_stride, width))) return st;
  if (drows && (st = check_rows(drows, drows_row_stride, width))) return st;
  if (drows && !weights) return RLD_EINVAL;
  if ((st = check_tables(indices, sorted_rows, places))) return st;
  if (!aligned4(weights) || !aligned4(dweights)) return RLD_EALIGN;
  const uint64_t size = rows_f32 ? 4 : 2;
  CombineGradArgs a;
  a.rows_ = (uint64_t)rows;
  a.indices_ = (uint64_t)indices;
  a.sorted_ = (uint64_t)sorted_rows;
  a.places_ = (uint64_t)places;
  a.weights_ = (uint64_t)weights;
  a.dout_ = (uint64_t)dout;
  a.drows_ = (uint64_t)drows;
  a.dweights_ = (uint64_t)dweights;
  a.rs = rows_row_stride * size;
  a.ds = dout_row_stride * size;
  a.os = drows_row_stride * size;
  a.T = num_tokens;
  a.n = num_tokens * top_k;
  a.k = top_k;
  a.units = units_of(width, rows_f32);
  if (too_many(num_tokens)) return RLD_EUNSUPPORTED;
  hipStream_t s = (hipStream_t)stream;
  if (rows_f32)
    places ? launch_combine_grad<true, true>(a, s) : launch_combine_grad<true, false>(a, s);
  else
    places ? launch_combine_grad<false, true>(a, s) : launch_combine_grad<false, false>(a, s);
  return launch_status();
}
