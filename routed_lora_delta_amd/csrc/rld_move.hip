// MoE token movement: tokens to the experts' order and back, and the gradients.
//
// A flat row f = t * top_k + j is choice j of token t.  The router's sorted_rows
// names the flat row of each expert-sorted row p; places is its inverse, written
// by the dispatch.  Row p belongs to f where places[f] = p and sorted_rows[p] = f,
// and only there: an entry of places that no dispatch wrote may hold anything and
// finds no row.
//
//   dispatch       rows[p] = x[f / top_k]
//   combine        out[t] = add[t] + sum_j w[t, j] rows[p(t, j)]
//   dispatch_grad  the same sum without weights
//   combine_grad   drows[p(t, j)] = w[t, j] dout[t],  dw[t, j] = rows[p(t, j)] . dout[t]
//
// All of them are bound by memory.  A lane holds 16 bytes of a row (a unit): a
// wave's access is 1 KB of one row, contiguous.
#include "rld_device.hpp"
#include "rld_internal.hpp"

namespace rld {

constexpr uint32_t kMaxMoveTopK = 32;

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
  uint32_t n, k, units, slices;
};

// A wave copies up to kDispatchUnits units of a lane of one sorted row.
constexpr int kDispatchUnits = 4;

__global__ void __launch_bounds__(256) dispatch_kernel(DispatchArgs a) {
  const uint32_t lane = threadIdx.x & 63;
  const uint32_t item = uniform(blockIdx.x * 4u + (threadIdx.x >> 6));
  const uint32_t p = item / a.slices, slice = item - p * a.slices;
  if (p >= a.n) return;
  const uint32_t f = uniform((uint32_t)gp<const int32_t>(a.sorted_)[p]);
  if (f >= a.n) return;
  if (slice == 0 && lane == 0) gp<int32_t>(a.places_)[f] = (int32_t)p;
  const uint32_t u0 = slice * (64u * kDispatchUnits) + lane;
  const uint64_t from = a.x_ + (uint64_t)(f / a.k) * a.xs, to = a.rows_ + (uint64_t)p * a.rs;
  u32x4 v[kDispatchUnits];
#pragma unroll
  for (int i = 0; i < kDispatchUnits; ++i)
    if (u0 + 64u * i < a.units) v[i] = load_unit(from + (u0 + 64u * i) * 16ull);
#pragma unroll
  for (int i = 0; i < kDispatchUnits; ++i)
    if (u0 + 64u * i < a.units) store_unit(to + (u0 + 64u * i) * 16ull, v[i]);
}

// ----------------------------------------------------------------- combine ----

struct CombineArgs {
  uint64_t rows_, indices_, sorted_, places_, weights_, add_, out_;
  uint64_t rs, as, os;  // bytes of a row
  uint32_t T, n, k, units, slices;
};

// The rows of a token's choices j0 .. j0 + 7: lane j holds choice j0 + j.  `have`
// tells which rows can be read, `own` which of them belong to the choice (the
// same ones, in the flat order); `own` is known one load later.
struct Choices {
  uint32_t row;
  uint64_t have;
  bool own;
};

template <class A>
__device__ __forceinline__ Choices find_choices(const A& a, uint32_t t, uint32_t j0, uint32_t lane) {
  const uint32_t j = j0 + lane;
  const bool in = lane < 8u && j < a.k;
  const uint32_t f = in ? t * a.k + j : 0u;
  Choices c;
  c.row = f;
  bool have = in;
  if (a.places_) {
    c.row = in ? (uint32_t)gp<const int32_t>(a.places_)[f] : 0u;
    have = in && c.row < a.n;
    c.own = have && (uint32_t)gp<const int32_t>(a.sorted_)[have ? c.row : 0u] == f;
  } else {
    if (a.indices_) have = in && gp<const int32_t>(a.indices_)[f] >= 0;
    c.own = have;
  }
  c.have = __ballot(have);
  return c;
}

// A wave adds up one slice of 64 units of a token's rows, in fp32, j ascending.
template <bool F32>
__global__ void __launch_bounds__(256) combine_kernel(CombineArgs a) {
  constexpr int N = Unit<F32>::N;
  const uint32_t lane = threadIdx.x & 63;
  const uint32_t item = uniform(blockIdx.x * 4u + (threadIdx.x >> 6));
  const uint32_t t = item / a.slices, slice = item - t * a.slices;
  if (t >= a.T) return;
  const uint32_t u = slice * 64u + lane;
  const uint64_t at = u * 16ull;
  const bool in = u < a.units;
  float acc[N];
#pragma unroll
  for (int i = 0; i < N; ++i) acc[i] = 0.f;
  if (a.add_ && in) Unit<F32>::open(load_unit(a.add_ + t * a.as + at), acc);
  for (uint32_t j0 = 0; j0 < a.k; j0 += 8) {
    const Choices c = find_choices(a, t, j0, lane);
    u32x4 r[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      r[j] = u32x4{0u, 0u, 0u, 0u};
      if ((c.have >> j) & 1u) {
        const uint64_t row = a.rows_ + (uint64_t)__builtin_amdgcn_readlane(c.row, j) * a.rs;
        if (in) r[j] = load_unit(row + at);
      }
    }
    float w = 1.f;
    if (a.weights_ && c.own) w = gp<const float>(a.weights_)[t * a.k + j0 + lane];
    const uint64_t own = __ballot(c.own);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if ((own >> j) & 1u) {
        const float wj = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(w), j));
        float v[N];
        Unit<F32>::open(r[j], v);
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] += wj * v[i];
      }
    }
  }
  if (in) store_unit(a.out_ + t * a.os + at, Unit<F32>::close(acc));
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
// is read before the same thread writes it, so drows may be rows.
template <bool F32, int WPT>
__global__ void __launch_bounds__(256) combine_grad_kernel(CombineGradArgs a) {
  constexpr int N = Unit<F32>::N;
  __shared__ float part[4][8];
  const uint32_t lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const uint32_t w0 = wave % WPT;
  const uint32_t t = blockIdx.x * (4u / WPT) + wave / WPT;
  const bool on = t < a.T;
  for (uint32_t j0 = 0; j0 < a.k; j0 += 8) {
    float dot[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) dot[j] = 0.f;
    uint64_t own = 0;
    if (on) {
      const Choices c = find_choices(a, t, j0, lane);
      own = __ballot(c.own);
      float w = 0.f;
      if (a.drows_ && c.own) w = gp<const float>(a.weights_)[t * a.k + j0 + lane];
      for (uint32_t u = w0 * 64u + lane; u < a.units; u += 64u * WPT) {
        const uint64_t at = u * 16ull;
        float d[N];
        u32x4 r[8];
        const u32x4 dv = load_unit(a.dout_ + t * a.ds + at);
        if (a.dweights_) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            r[j] = u32x4{0u, 0u, 0u, 0u};
            if ((c.have >> j) & 1u)
              r[j] = load_unit(a.rows_ + (uint64_t)__builtin_amdgcn_readlane(c.row, j) * a.rs + at);
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
              const float wj = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(w), j));
              float v[N];
#pragma unroll
              for (int i = 0; i < N; ++i) v[i] = wj * d[i];
              store_unit(a.drows_ + (uint64_t)__builtin_amdgcn_readlane(c.row, j) * a.os + at,
                         Unit<F32>::close(v));
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
  if (k > kMaxMoveTopK || (uint64_t)T * k >= (1ull << 31)) return RLD_EUNSUPPORTED;
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
  const uint32_t blocks = div_ceil(T * a.slices, 4);
  hipStream_t s = (hipStream_t)stream;
  if (f32) combine_kernel<true><<<blocks, 256, 0, s>>>(a);
  else combine_kernel<false><<<blocks, 256, 0, s>>>(a);
  return launch_status();
}

template <bool F32>
static void launch_combine_grad(const CombineGradArgs& a, hipStream_t s) {
  if (a.units <= 64) combine_grad_kernel<F32, 1><<<div_ceil(a.T, 4), 256, 0, s>>>(a);
  else if (a.units <= 128) combine_grad_kernel<F32, 2><<<div_ceil(a.T, 2), 256, 0, s>>>(a);
  else combine_grad_kernel<F32, 4><<<a.T, 256, 0, s>>>(a);
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
  a.n = num_tokens * top_k;
  a.k = top_k;
  a.units = units_of(width, rows_f32);
  a.slices = div_ceil(a.units, 64u * kDispatchUnits);
  if (too_many((uint64_t)a.n * a.slices)) return RLD_EUNSUPPORTED;
  dispatch_kernel<<<div_ceil(a.n * a.slices, 4), 256, 0, (hipStream_t)stream>>>(a);
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
  if (num_tokens > (1u << 24) - 1u) return RLD_EUNSUPPORTED;
  if (rows_f32) launch_combine_grad<true>(a, (hipStream_t)stream);
  else launch_combine_grad<false>(a, (hipStream_t)stream);
  return launch_status();
}
