// The norm of each group of gradients, and clipping by it.
//
//   norm_g = sqrt(sum of x^2 over the group's gradients),  x <- x min(1, limit_g / (norm_g + 1e-6))
//
// The list is made on the host once (rld_grad_pack): chunks of up to kGradChunk
// bytes, the chunks of a group together.  A wave takes a run of consecutive chunks.
// Squares are formed and added in 64 bits, where the square of an fp32 number is
// exact and neither overflows nor vanishes: a norm is off by its last rounding.
// Memory bounds it all: 785 MB of fp32 in 128 us, 6.1 TB/s of the 6.7 that 4 GB reach
// (the second launch takes 5 of them); from the caches it does 23 TB/s of fp32 and 16
// of BF16, which is what the 64-bit arithmetic allows.
#include "rld_device.hpp"
#include "rld_internal.hpp"

namespace rld {

constexpr uint32_t kGradWaves = 4096;  // of a launch at most: all of them run at once

// Clipping walks each run backwards, so it begins with what the norm read last: the
// last kKeep chunks of a run, 256 MB over all waves, are read through the 256 MB
// cache behind the L2s and found there.  The rest passes it by.  Norm and clipping of
// 311 MB, out of place, with kKeep 0 / 4 / 8 / 12: 175, 162, 151 and 156 us; the norm
// alone of 785 MB 124.5, 125.3, 128.5 and 131.3.
constexpr uint32_t kKeep = 8;
constexpr float kClipEps = 1e-6f;

struct GradArgs {
  uint64_t chunks_, starts_, partial_, norms_, squares_, limits_;
  uint32_t num_chunks, num_groups, waves;
};

// Wave v takes the chunks [first_chunk(v), first_chunk(v + 1)).
__host__ __device__ inline uint32_t first_chunk(uint32_t v, uint32_t chunks, uint32_t waves) {
  return (uint32_t)((uint64_t)v * chunks / waves);
}

// The wave that takes chunk c.
__host__ __device__ inline uint32_t wave_of(uint32_t c, uint32_t chunks, uint32_t waves) {
  return (uint32_t)((((uint64_t)c + 1) * waves - 1) / chunks);
}

struct Chunk {
  uint64_t at, to;
  uint32_t count, bf16, group;
};

// Lane l of a wave holds chunk c0 + l of its run; chunk(i) is the i-th of them in
// scalar registers.
struct ChunkRun {
  u32x4 lo, hi;
  __device__ __forceinline__ ChunkRun(uint64_t chunks, uint32_t c, uint32_t end) {
    lo = hi = u32x4{0u, 0u, 0u, 0u};
    if (c < end) {
      const auto at = gp<const u32x4>(chunks + (uint64_t)c * sizeof(rld_grad_chunk));
      lo = at[0];
      hi = at[1];
    }
  }
  __device__ __forceinline__ Chunk chunk(int i) const {
    Chunk c;
    c.at = (uint64_t)from_lane(lo[1], i) << 32 | from_lane(lo[0], i);
    c.to = (uint64_t)from_lane(lo[3], i) << 32 | from_lane(lo[2], i);
    c.count = from_lane(hi[0], i);
    c.group = from_lane(hi[1], i);
    c.bf16 = from_lane(hi[2], i);
    return c;
  }
};

// Two loads that differ in this alone would be merged by the compiler if they were
// the two sides of a branch: callers keep them in loops of their own.
template <bool ONCE>
__device__ __forceinline__ u32x4 load_grad(uint64_t at, uint32_t offset) {
  return ONCE ? load_once(at, offset) : load_unit(at, offset);
}

__device__ __forceinline__ void add_squares(const u32x4& v, bool bf16, double& s0, double& s1) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (bf16) {
      const double a = __uint_as_float(v[i] << 16), b = __uint_as_float(v[i] & 0xffff0000u);
      s0 += a * a;
      s1 += b * b;
    } else {
      const double a = __uint_as_float(v[i]);
      if (i & 1) s1 += a * a;
      else s0 += a * a;
    }
  }
}

__device__ __forceinline__ float element(uint64_t at, uint32_t i, bool bf16) {
  return bf16 ? bf16_to_f32(gp<const uint16_t>(at)[i]) : gp<const float>(at)[i];
}

constexpr int kGradUnits = kGradChunk / 1024;  // 16-byte units of a lane in a whole chunk

template <bool BF16, bool ONCE>
__device__ __forceinline__ double chunk_squares(const Chunk& c, uint32_t lane) {
  constexpr uint32_t N = BF16 ? 8 : 4;
  const uint32_t units = c.count / N;
  double s0 = 0., s1 = 0.;
  if (units == 64u * kGradUnits) {
    u32x4 v[kGradUnits];
#pragma unroll
    for (int i = 0; i < kGradUnits; ++i) v[i] = load_grad<ONCE>(c.at, (lane + 64u * i) * 16u);
#pragma unroll
    for (int i = 0; i < kGradUnits; ++i) add_squares(v[i], BF16, s0, s1);
  } else {
    for (uint32_t u = lane; u < units; u += 64)
      add_squares(load_grad<ONCE>(c.at, u * 16u), BF16, s0, s1);
    const uint32_t e = units * N + lane;
    if (e < c.count) {
      const double a = element(c.at, e, BF16);
      s0 += a * a;
    }
  }
  return s0 + s1;
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m);
  return v;
}

// A wave's sum of the group that it is in.  Each wave leaves one sum for each group
// it meets, at place wave + group: groups ascend with the chunks, so no two sums
// share a place and a group's lie together.
struct GroupSum {
  double sum;
  uint32_t group;
  __device__ __forceinline__ void leave(const GradArgs& a, uint32_t w, uint32_t lane) {
    if (group < a.num_groups) {
      sum = wave_sum(sum);
      if (lane == 0) gp<double>(a.partial_)[(uint64_t)w + group] = sum;
    }
  }
  template <bool ONCE>
  __device__ __forceinline__ void add(const GradArgs& a, const ChunkRun& run, int from, int to,
                                      uint32_t w, uint32_t lane) {
#pragma nounroll
    for (int i = from; i < to; ++i) {
      const Chunk c = run.chunk(i);
      if (c.group != group) {
        leave(a, w, lane);
        sum = 0.;
        group = c.group;
      }
      sum += c.bf16 ? chunk_squares<true, ONCE>(c, lane) : chunk_squares<false, ONCE>(c, lane);
    }
  }
};

__global__ void __launch_bounds__(256) grad_squares_kernel(GradArgs a) {
  const uint32_t lane = threadIdx.x & 63;
  const uint32_t w = uniform(blockIdx.x * 4u + (threadIdx.x >> 6));
  if (w >= a.waves) return;
  const uint32_t end = first_chunk(w + 1, a.num_chunks, a.waves);
  GroupSum s = {0., ~0u};
  for (uint32_t c0 = first_chunk(w, a.num_chunks, a.waves); c0 < end; c0 += 64) {
    const ChunkRun run(a.chunks_, c0 + lane, end);
    const int n = min(64u, end - c0), once = min((uint32_t)n, end - c0 - min(kKeep, end - c0));
    s.add<true>(a, run, 0, once, w, lane);
    s.add<false>(a, run, once, n, w, lane);
  }
  s.leave(a, w, lane);
}

// One block a group adds its waves' sums, in a fixed order.  (Of 256 threads: 0.9 us
// more for 1024 sums a group, 0.1 less for 64.)
constexpr uint32_t kNormThreads = 512;

__global__ void __launch_bounds__(kNormThreads) grad_norms_kernel(GradArgs a) {
  __shared__ double part[kNormThreads / 64];
  const uint32_t g = blockIdx.x;
  const uint32_t c0 = gp<const uint32_t>(a.starts_)[g], c1 = gp<const uint32_t>(a.starts_)[g + 1];
  double s = 0.;
  if (c0 < c1 && c1 <= a.num_chunks) {
    const uint64_t p1 = wave_of(c1 - 1, a.num_chunks, a.waves) + (uint64_t)g;
    for (uint64_t p = wave_of(c0, a.num_chunks, a.waves) + (uint64_t)g + threadIdx.x; p <= p1;
         p += kNormThreads)
      s += gp<const double>(a.partial_)[p];
  }
  s = wave_sum(s);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x != 0) return;
  s = 0.;
#pragma unroll
  for (uint32_t i = 0; i < kNormThreads / 64; ++i) s += part[i];
  gp<float>(a.norms_)[g] = (float)sqrt(s);
  if (a.squares_) gp<double>(a.squares_)[g] = s;
}

template <bool BF16>
__device__ __forceinline__ u32x4 scaled(const u32x4& v, float f) {
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    r[i] = BF16 ? pack_bf16x2(__uint_as_float(v[i] << 16) * f,
                              __uint_as_float(v[i] & 0xffff0000u) * f)
                : __float_as_uint(__uint_as_float(v[i]) * f);
  return r;
}

template <bool BF16, bool ONCE>
__device__ __forceinline__ void chunk_scale(const Chunk& c, float f, uint32_t lane) {
  constexpr uint32_t N = BF16 ? 8 : 4;
  const uint32_t units = c.count / N;
  if (units == 64u * kGradUnits) {
    u32x4 v[kGradUnits];
#pragma unroll
    for (int i = 0; i < kGradUnits; ++i) v[i] = load_grad<ONCE>(c.at, (lane + 64u * i) * 16u);
#pragma unroll
    for (int i = 0; i < kGradUnits; ++i)
      store_once(c.to, (lane + 64u * i) * 16u, scaled<BF16>(v[i], f));
  } else {
    for (uint32_t u = lane; u < units; u += 64)
      store_once(c.to, u * 16u, scaled<BF16>(load_grad<ONCE>(c.at, u * 16u), f));
    const uint32_t e = units * N + lane;
    if (e < c.count) {
      const float v = element(c.at, e, BF16) * f;
      if (BF16) gp<uint16_t>(c.to)[e] = (uint16_t)f32_to_bf16(v);
      else gp<float>(c.to)[e] = v;
    }
  }
}

// The chunks [from, to) of a run, backwards; lane l holds the factor of its chunk l.
template <bool ONCE>
__device__ __forceinline__ void clip_chunks(const ChunkRun& run, int from, int to, float factor,
                                            uint32_t lane) {
#pragma nounroll
  for (int i = to - 1; i >= from; --i) {
    const Chunk c = run.chunk(i);
    const float f = from_lane(factor, i);
    if (f == 1.f && c.to == c.at) continue;
    if (c.bf16) chunk_scale<true, ONCE>(c, f, lane);
    else chunk_scale<false, ONCE>(c, f, lane);
  }
}

__global__ void __launch_bounds__(256) grad_clip_kernel(GradArgs a) {
  const uint32_t lane = threadIdx.x & 63;
  const uint32_t w = uniform(blockIdx.x * 4u + (threadIdx.x >> 6));
  if (w >= a.waves) return;
  const uint32_t begin = first_chunk(w, a.num_chunks, a.waves);
  const uint32_t end = first_chunk(w + 1, a.num_chunks, a.waves);
  for (uint32_t c1 = end; c1 > begin;) {
    const uint32_t c0 = c1 - min(64u, c1 - begin);
    const ChunkRun run(a.chunks_, c0 + lane, c1);
    float factor = 1.f;
    if (run.hi[1] < a.num_groups) {
      const float limit = gp<const float>(a.limits_)[run.hi[1]];
      const float f = limit / (gp<const float>(a.norms_)[run.hi[1]] + kClipEps);
      if (limit >= 0.f && limit < __builtin_inff() && !(f >= 1.f)) factor = f;
    }
    const int n = c1 - c0, once = min((uint32_t)n, end - c0 - min(kKeep, end - c0));
    clip_chunks<false>(run, once, n, factor, lane);
    clip_chunks<true>(run, 0, once, factor, lane);
    c1 = c0;
  }
}

// -------------------------------------------------------------------- host ----

static int check_list(const rld_grad_list* l) {
  if (!l) return RLD_EINVAL;
  if (l->num_groups > kMaxGradGroups || l->num_chunks > kMaxGradChunks) return RLD_EUNSUPPORTED;
  if (l->num_groups == 0) return l->num_chunks ? RLD_EINVAL : RLD_OK;
  if (!l->group_starts || (l->num_chunks && !l->chunks)) return RLD_EINVAL;
  if (!aligned16(l->chunks) || ((uintptr_t)l->group_starts & 3u)) return RLD_EALIGN;
  return RLD_OK;
}

static GradArgs grad_args(const rld_grad_list* l) {
  GradArgs a = {};
  a.chunks_ = (uint64_t)l->chunks;
  a.starts_ = (uint64_t)l->group_starts;
  a.num_chunks = l->num_chunks;
  a.num_groups = l->num_groups;
  a.waves = l->num_chunks < kGradWaves ? l->num_chunks : kGradWaves;
  return a;
}

}  // namespace rld

using namespace rld;

extern "C" size_t rld_grad_norm_workspace_bytes(const rld_grad_list* list) {
  if (check_list(list) || list->num_groups == 0) return 0;
  return ((size_t)grad_args(list).waves + list->num_groups + 1) / 2 * 16;
}

extern "C" int rld_grad_norm(const rld_grad_list* list, float* norms, double* squares,
                             void* workspace, size_t workspace_bytes, void* stream) {
  const int st = check_list(list);
  if (st || list->num_groups == 0) return st;
  if (!norms || !workspace) return RLD_EINVAL;
  if (((uintptr_t)norms & 3u) || ((uintptr_t)squares & 7u) || !aligned16(workspace))
    return RLD_EALIGN;
  if (workspace_bytes < rld_grad_norm_workspace_bytes(list)) return RLD_ENOSPACE;
  GradArgs a = grad_args(list);
  a.partial_ = (uint64_t)workspace;
  a.norms_ = (uint64_t)norms;
  a.squares_ = (uint64_t)squares;
  if (a.waves) grad_squares_kernel<<<div_ceil(a.waves, 4), 256, 0, (hipStream_t)stream>>>(a);
  grad_norms_kernel<<<a.num_groups, kNormThreads, 0, (hipStream_t)stream>>>(a);
  return launch_status();
}

extern "C" int rld_grad_clip(const rld_grad_list* list, const float* norms, const float* limits,
                             void* stream) {
  const int st = check_list(list);
  if (st || list->num_groups == 0 || list->num_chunks == 0) return st;
  if (!norms || !limits) return RLD_EINVAL;
  if (((uintptr_t)norms & 3u) || ((uintptr_t)limits & 3u)) return RLD_EALIGN;
  GradArgs a = grad_args(list);
  a.norms_ = (uint64_t)norms;
  a.limits_ = (uint64_t)limits;
  grad_clip_kernel<<<div_ceil(a.waves, 4), 256, 0, (hipStream_t)stream>>>(a);
  return launch_status();
}
