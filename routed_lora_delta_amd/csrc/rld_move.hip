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
// wave's access is 1 KB of one row, contiguous.  What is read once and what is written
// passes the caches by (load_once, store_once), which also serves who reads the result
// next: dispatch of 4096 tokens to 8 rows of 2048 BF16 each and a pass over the rows
// take 65.3 us so, 68.9 otherwise; of 16384 237 and 286.
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

// ---------------------------------------------------------------- dispatch ----

struct DispatchArgs {
  uint64_t x_, sorted_, rows_, places_;
  uint64_t xs, rs;  // bytes of a row
  uint32_t T, n, k, units, slices;
};

// A wave copies kRowUnits units a lane of one sorted row.
constexpr int kRowUnits = 2;

__global__ void __launch_bounds__(256) dispatch_rows_kernel(DispatchArgs a) {
  const uint32_t lane = threadIdx.x & 63;
  const uint32_t item = uniform(blockIdx.x * 4u + (threadIdx.x >> 6));
  const uint32_t p = item / a.slices, slice = item - p * a.slices;
  if (p >= a.n) return;
  const uint32_t f = uniform((uint32_t)gp<const int32_t>(a.sorted_)[p]);
  if (f >= a.n) return;
  if (slice == 0 && lane == 0) gp<int32_t>(a.places_)[f] = (int32_t)p;
  const uint32_t u0 = slice * (64u * kRowUnits) + lane;
  const uint64_t from = a.x_ + (f / a.k) * a.xs, to = a.rows_ + p * a.rs;
  u32x4 v[kRowUnits];
#pragma unroll
  for (int i = 0; i < kRowUnits; ++i)
    if (u0 + 64u * i < a.units) v[i] = load_unit(from, (u0 + 64u * i) * 16u);
#pragma unroll
  for (int i = 0; i < kRowUnits; ++i)
    if (u0 + 64u * i < a.units) store_once(to, (u0 + 64u * i) * 16u, v[i]);
}

__global__ void __launch_bounds__(256) dispatch_places_kernel(DispatchArgs a) {
  const uint32_t p = blockIdx.x * 256u + threadIdx.x;
  if (p >= a.n) return;
  const uint32_t f = (uint32_t)gp<const int32_t>(a.sorted_)[p];
  if (f < a.n) gp<int32_t>(a.places_)[f] = (int32_t)p;
}

// The second launch of large calls: a wave reads 64 units of a token once and writes
// them to each of its rows.
__global__ void __launch_bounds__(256) dispatch_tokens_kernel(DispatchArgs a) {
  const uint32_t lane = threadIdx.x & 63;
  const uint32_t item = uniform(blockIdx.x * 4u + (threadIdx.x >> 6));
  const uint32_t t = item / a.slices, slice = item - t * a.slices;
  if (t >= a.T) return;
  const uint32_t u = slice * 64u + lane;
  const uint32_t at = min(u, a.units - 1u) * 16u;
  const u32x4 v = load_unit(a.x_ + t * a.xs, at);
  const uint32_t f = t * a.k + min(lane, a.k - 1u);
  uint32_t p = (uint32_t)gp<const int32_t>(a.places_)[f];
  const bool have = lane < a.k && p < a.n;
  p = have ? p : 0u;
  uint64_t own = __ballot(have && (uint32_t)gp<const int32_t>(a.sorted_)[p] == f);
  while (own) {
    const int j = __builtin_ctzll(own);
    own &= own - 1;
    if (u < a.units) store_once(a.rows_ + from_lane(p, j) * a.rs, at, v);
  }
}

// ----------------------------------------------------------------- combine ----

struct CombineArgs {
  uint64_t rows_, indices_, sorted_, places_, weights_, add_, out_;
  uint64_t rs, as, os;  // bytes of a row
  uint32_t T, n, k, units, slices;
};

// The rows of a token's choices j0 .. j0 + 7: lane j holds choice j0 + j.  `have`
// has a bit for each row that can be read; own() one for each of them that belongs
// to its choice, which takes one load more: called once the rows' loads are out.
struct Choices {
  uint32_t row, back, f;
  uint64_t have;
  __device__ __forceinline__ uint64_t own() {
    asm volatile("" : "+v"(back) : : "memory");  // the comparison stays behind those loads
    return have & __ballot(back == f);
  }
};

// Loads without a branch, from clamped places.
template <bool SORTED, class A>
__device__ __forceinline__ Choices find_choices(const A& a, uint32_t t, uint32_t j0,
                                                uint32_t lane) {
  const bool in = lane < 8u && j0 + lane < a.k;
  Choices c;
  c.f = t * a.k + (in ? j0 + lane : j0);
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
  c.have = __ballot(have);
  return c;
}

// A wave adds up one slice of 64 units of a token's rows, in fp32, j ascending: eight
// rows' loads at a time, the places before them, the check and the weights beside
// them.  32771 tokens of 8 rows of 2048 BF16, onto a residual: 209 us, 5.9 TB/s, in
// blocks of one wave (214 in blocks of four).
template <bool F32, bool SORTED>
__global__ void __launch_bounds__(64) combine_kernel(CombineArgs a) {
  constexpr int N = Unit<F32>::N;
  const uint32_t lane = threadIdx.x;
  const uint32_t t = blockIdx.x / a.slices, slice = blockIdx.x - t * a.slices;
  const uint32_t u = slice * 64u + lane;
  const uint32_t at = min(u, a.units - 1u) * 16u;  // lanes past the row load its last unit
  u32x4 last = {0u, 0u, 0u, 0u};
  if (a.add_) last = load_once(a.add_ + t * a.as, at);
  float acc[N];
#pragma unroll
  for (int i = 0; i < N; ++i) acc[i] = 0.f;
#pragma nounroll
  for (uint32_t j0 = 0; j0 < a.k; j0 += 8) {
    Choices c = find_choices<SORTED>(a, t, j0, lane);
    float w = 1.f;
    if (a.weights_) w = gp<const float>(a.weights_)[c.f];
    u32x4 r[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      r[j] = u32x4{0u, 0u, 0u, 0u};
      if ((c.have >> j) & 1u) r[j] = load_once(a.rows_ + from_lane(c.row, j) * a.rs, at);
    }
    const uint64_t own = c.own();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if ((own >> j) & 1u) {
        const float wj = from_lane(w, j);
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
  uint32_t T, n, k, units;
};

// Sums of eight values over a wave, for ten exchanges: each of the first three
// halves the values that a lane holds.  Lane 8 i gets the sum of v[i].
__device__ __forceinline__ float sum8(float* v, uint32_t lane) {
#pragma unroll
  for (int half = 4, m = 32; half >= 1; half >>= 1, m >>= 1) {
    const bool up = (lane & m) != 0;
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const float keep = up ? v[i + half] : v[i];
      const float give = up ? v[i] : v[i + half];
      v[i] = keep + __shfl_xor(give, m);
    }
  }
  float s = v[0];
  s += __shfl_xor(s, 4);
  s += __shfl_xor(s, 2);
  s += __shfl_xor(s, 1);
  return s;
}

// WPT waves share a token's columns; 256 / (64 WPT) tokens a block.  A row's unit
// is read before the same thread writes it, so drows may be rows.  16387 tokens of 8
// rows of 2048 BF16: 204 us, 5.05 TB/s, where a copy reaches 5.2 (212 with two waves a
// token, 222 with one; more waves a CU, by fewer registers, spill).
template <bool F32, bool SORTED, int WPT>
__global__ void __launch_bounds__(256) combine_grad_kernel(CombineGradArgs a) {
  constexpr int N = Unit<F32>::N;
  __shared__ float part[4][8];
  const uint32_t lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const uint32_t w0 = wave % WPT;
  const uint32_t t = blockIdx.x * (4u / WPT) + wave / WPT;
  const bool on = t < a.T;
#pragma nounroll
  for (uint32_t j0 = 0; j0 < a.k; j0 += 8) {
    float dot[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) dot[j] = 0.f;
    uint64_t own = 0;
    if (on) {
      Choices c = find_choices<SORTED>(a, t, j0, lane);
      float w = 0.f;
      if (a.drows_) w = gp<const float>(a.weights_)[c.f];
      own = c.own();
      for (uint32_t u = w0 * 64u + lane; u < a.units; u += 64u * WPT) {
        const uint32_t at = u * 16u;
        float d[N];
        u32x4 r[8];
        const u32x4 dv = load_once(a.dout_ + t * a.ds, at);
        if (a.dweights_) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            r[j] = u32x4{0u, 0u, 0u, 0u};
            if ((c.have >> j) & 1u) r[j] = load_once(a.rows_ + from_lane(c.row, j) * a.rs, at);
          }
        }
        Unit<F32>::open(dv, d);
        if (a.dweights_) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            float v[N];
            Unit<F32>::open(r[j], v);
#pragma unroll
            for (int i = 0; i < N; ++i) dot[j] += d[i] * v[i];
          }
        }
        if (a.drows_) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if ((own >> j) & 1u) {
              const float wj = from_lane(w, j);
              float v[N];
#pragma unroll
              for (int i = 0; i < N; ++i) v[i] = wj * d[i];
              store_once(a.drows_ + from_lane(c.row, j) * a.os, at, Unit<F32>::close(v));
            }
          }
        }
      }
    }
    if (!a.dweights_) continue;
    float s = sum8(dot, lane);
    const uint32_t j = lane >> 3;
    if (WPT > 1) {
      if (j0) __syncthreads();
      if ((lane & 7u) == 0) part[wave][j] = s;
      __syncthreads();
      s = part[wave - w0][j];
#pragma unroll
      for (int v = 1; v < WPT; ++v) s += part[wave - w0 + v][j];
    }
    if (on && w0 == 0 && (lane & 7u) == 0 && j0 + j < a.k)
      gp<float>(a.dweights_)[(uint64_t)t * a.k + j0 + j] = ((own >> j) & 1u) ? s : 0.f;
  }
}

// -------------------------------------------------------------------- host ----

static bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }

static int check_move(uint32_t T, uint32_t k, uint32_t width) {
  if (k == 0 || width == 0) return RLD_EINVAL;
  if (k > kMaxMoveTopK || width > kMaxMoveWidth || (uint64_t)T * k >= (1ull << 31)) return RLD_EUNSUPPORTED;
  if (!mult8(width)) return RLD_EALIGN;
  return RLD_OK;
}

static uint32_t units_of(uint32_t width, int f32) { return width / (f32 ? 4u : 8u); }

// One wave for each item, in a grid of fewer than 2^32 threads.
static bool too_many(uint64_t items) { return items > (1ull << 26) - 4; }

// Where the rows of the choices are: both tables, or neither (flat order).
static int check_tables(const int32_t* indices, const int32_t* sorted_rows,
                        const int32_t* places) {
  if ((sorted_rows == nullptr) != (places == nullptr)) return RLD_EINVAL;
  return aligned4(indices) && aligned4(sorted_rows) && aligned4(places) ? RLD_OK : RLD_EALIGN;
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
  const uint32_t blocks = T * a.slices;
  hipStream_t s = (hipStream_t)stream;
  if (a.places_) f32 ? combine_kernel<true, true><<<blocks, 64, 0, s>>>(a)
                     : combine_kernel<false, true><<<blocks, 64, 0, s>>>(a);
  else f32 ? combine_kernel<true, false><<<blocks, 64, 0, s>>>(a)
           : combine_kernel<false, false><<<blocks, 64, 0, s>>>(a);
  return launch_status();
}

template <bool F32, bool SORTED>
static void launch_combine_grad(const CombineGradArgs& a, hipStream_t s) {
  if (a.units <= 64) combine_grad_kernel<F32, SORTED, 1><<<div_ceil(a.T, 4), 256, 0, s>>>(a);
  else if (a.units <= 128) combine_grad_kernel<F32, SORTED, 2><<<div_ceil(a.T, 2), 256, 0, s>>>(a);
  else combine_grad_kernel<F32, SORTED, 4><<<a.T, 256, 0, s>>>(a);
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
  // and 98; rows of 4096, top_k 2: 1024 6.1 and 6.8, 4096 (34 MB) 18.9 and 18.1.
  if ((uint64_t)(a.n - a.T) * width * size < (32u << 20)) {
    a.slices = div_ceil(a.units, 64u * kRowUnits);
    dispatch_rows_kernel<<<div_ceil(a.n * a.slices, 4), 256, 0, s>>>(a);
  } else {
    dispatch_places_kernel<<<div_ceil(a.n, 256), 256, 0, s>>>(a);
    dispatch_tokens_kernel<<<div_ceil(a.T * a.slices, 4), 256, 0, s>>>(a);
  }
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
  // blocks of 256 threads, as many as tokens at most
  if (num_tokens >= (1u << 24)) return RLD_EUNSUPPORTED;
  hipStream_t s = (hipStream_t)stream;
  if (places) rows_f32 ? launch_combine_grad<true, true>(a, s) : launch_combine_grad<false, true>(a, s);
  else rows_f32 ? launch_combine_grad<true, false>(a, s) : launch_combine_grad<false, false>(a, s);
  return launch_status();
}
