// The shared projection beside its routed adapters, and its gradient:
//
//   y_i  = x_i W^T + u_i B_s^T,   u_i = scale_s x_i A_s^T        (s = seq_slot[i])
//   dx_i = dy_i W  + g_i A_s,     g_i = scale_s dy_i B_s
//   dA_s = sum_{i in s} g_i^T x_i,   dB_s = sum_{i in s} dy_i^T u_i
//
// (W frozen).  Kernels:
//   sort     the rows by slot (stable; base rows last), so that a tile's rows name
//            few slots and a slot's rows lie together.  The kernels below work on
//            sorted positions and reach x, dy and the outputs through the order.
//   low      the low-rank products u and g of every routed row, as fp32 partial
//            sums of k chunks; low_reduce adds the chunks and applies the scale.
//   big_tile one 256 x 256 output tile of x W^T (or dy W) with the low rows times
//            the slots' second matrices added into the same accumulators, so the
//            output is rounded once and written once.
//   part     for calls with too few such tiles: smaller tiles over a split of K, as
//            fp32 sums.  The low products and, where they do not need it, the sort
//            are other blocks of the same launch (start).
//   finish   adds the splits and the low rows times the second matrices, and rounds.
//   wgrad    dA and dB: the products over a slot's rows, in one launch with the
//            finish of dx (end); wgrad_sum where the positions are split.
//
// u and g stay in fp32 (bf16 copies would add a rounding of 2^-9 to every
// term).  The matrix cores take bf16, so a low value enters as the sum of two
// bf16 parts where the result is rounded to bf16 (16 significand bits, an
// error of 2^-17) and of three where it is fp32 (24 bits: all of it).
#include <algorithm>
#include <type_traits>

#include "rld_device.hpp"
#include "rld_internal.hpp"

namespace rld {

typedef short s16x4 __attribute__((ext_vector_type(4)));
#define RLD_LDS __attribute__((address_space(3)))
#define RLD_CONST __attribute__((address_space(4)))

constexpr uint32_t kFinishRows = 64;  // positions of a finish block of a large call
constexpr uint32_t kLowRows = 64;    // rows of a low item
constexpr uint32_t kLowChunk = 512;  // k elements of a low item, at least
constexpr uint32_t kMaxStride = 1u << 21;
// 256 x 256 tiles from which a grid of them pays (us against smaller split ones,
// 96 tiles, 4096 -> 4096: 99.1 and 95.2; 128: 99 and 99; 144: 100 and 133; 144,
// 12288 -> 4096: 261 and 358).
constexpr uint32_t kBigTiles = 128;

// 16 bytes of zeros per device: where a lane's source is outside the operand.
__device__ uint4 g_zero16[1];

// ------------------------------------------------------------- bf16 parts ----

// v as the sum of two bf16 values, the larger first, to 2^-17.  Rounding to nearest
// makes the remainder exact in fp32 (it fits the 24 - 8 bits left).  The first part is
// kept finite (a value above 1.996 2^127 would round to infinity, and one infinity
// less another is a NaN); an infinity is the second part.
__device__ __forceinline__ float first_part(float v) {
  const float top = __uint_as_float(0x7f7f0000u);  // the largest bf16
  return __builtin_amdgcn_fmed3f(v, -top, top);
}

__device__ __forceinline__ void bf16_parts(const float (&v)[8], uint4 (&out)[2]) {
  uint32_t w[4], r[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    w[e] = pack_bf16x2(first_part(v[2 * e]), first_part(v[2 * e + 1]));
    r[e] = pack_bf16x2(v[2 * e] - bf16_to_f32(w[e] & 0xffffu),
                       v[2 * e + 1] - bf16_to_f32(w[e] >> 16));
  }
  out[0] = make_uint4(w[0], w[1], w[2], w[3]);
  out[1] = make_uint4(r[0], r[1], r[2], r[3]);
}

// ------------------------------------------------------------------- sort ----

struct SortArgs {
  uint64_t seq_, atab_, btab_;
  uint64_t order_, skey_;  // [n]: the row at a sorted position; its slot, -1 for base rows
  uint64_t rkey_, rpos_;   // [n]: by row, the same slot and the row's position
  uint64_t span_;          // [max_loras][2]: a slot's first position and rows
  uint32_t n, max_loras;
};

constexpr uint32_t kSortBatch = 4096;  // rows of a pass: 16 a thread

typedef int i32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));

// Keys of this thread's 16 consecutive rows of a batch; past n: INT_MIN.
__device__ __forceinline__ void sort_keys(const SortArgs& a, uint32_t r0, int (&key)[16]) {
  const RLD_GLOBAL int32_t* seq = gp<const int32_t>(a.seq_);
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    if (r0 + 4 * v + 4 <= a.n) {
      const i32x4_a4 k = *reinterpret_cast<const RLD_GLOBAL i32x4_a4*>(seq + r0 + 4 * v);
#pragma unroll
      for (int e = 0; e < 4; ++e) key[4 * v + e] = k[e];
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        key[4 * v + e] = r0 + 4 * v + e < a.n ? seq[r0 + 4 * v + e] : (int)0x80000000;
    }
    // ids that name no slot sort as max_loras
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (key[4 * v + e] < 0 || (uint32_t)key[4 * v + e] >= a.max_loras)
        key[4 * v + e] = r0 + 4 * v + e < a.n ? (int)a.max_loras : 0x7fffffff;
  }
}

// Sum over the block before this thread, and the block's sum.
__device__ __forceinline__ uint32_t block_prefix(uint32_t v, uint32_t* wsum, uint32_t& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t inc = v;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint32_t u = __shfl_up(inc, o);
    if (lane >= o) inc += u;
  }
  __syncthreads();
  if (lane == 63) wsum[wave] = inc;
  __syncthreads();
  uint32_t at = inc - v;
  total = 0;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    at += w < wave ? wsum[w] : 0;
    total += wsum[w];
  }
  return at;
}

// One block per slot, and one for the base rows: its rows in ascending order,
// behind those of the slots below it, which the block counts itself (no block
// waits for another).  Bound by the latency of two passes over the ids while slots are
// few: 4.7 us for 1237 rows and 16 slots, 7 us for 4096 rows.  With thousands of slots
// and rows the slots times the rows count, some 3 10^11 a second (a projection of
// 4096 rows 4096 -> 1024 at rank 16 with 16, 1000, 4096 and 16384 slots: 67, 140, 258
// and 346 us; of 16384 rows with 16384 slots 1.1 ms, 0.15 of them with 16).
__device__ __forceinline__ void sort_item(const SortArgs& a, uint32_t item, uint32_t* wsum) {
  const int s = (int)item;
  const bool base = (uint32_t)s == a.max_loras;
  const bool active =
      !base && gp<const uint64_t>(a.atab_)[s] != 0ull && gp<const uint64_t>(a.btab_)[s] != 0ull;
  int key[16];
  uint32_t below = 0, own = 0, first, cnt = 0;
  for (uint32_t b0 = 0; b0 < a.n; b0 += kSortBatch) {
    sort_keys(a, b0 + threadIdx.x * 16, key);
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      below += key[e] < s;
      own += key[e] == s;
    }
  }
  // one batch: both sums, of at most 2^12, in one pass of a word
  const bool one = a.n <= kSortBatch;
  uint32_t before = block_prefix(one ? below << 16 | own : below, wsum, first);
  const uint32_t both = first;
  if (one) first >>= 16;
  for (uint32_t b0 = 0; b0 < a.n; b0 += kSortBatch) {
    const uint32_t r0 = b0 + threadIdx.x * 16;
    uint32_t tot = both & 0xffffu;
    before &= 0xffffu;
    if (!one) {
      sort_keys(a, r0, key);
      own = 0;
#pragma unroll
      for (int e = 0; e < 16; ++e) own += key[e] == s;
      before = block_prefix(own, wsum, tot);
    }
    uint32_t at = first + cnt + before;
#pragma unroll
    for (int e = 0; e < 16; ++e)
      if (key[e] == s) {
        gp<int32_t>(a.order_)[at] = (int)(r0 + e);
        gp<int32_t>(a.skey_)[at] = active ? s : -1;
        gp<int32_t>(a.rkey_)[r0 + e] = active ? s : -1;
        gp<int32_t>(a.rpos_)[r0 + e] = (int)at;
        ++at;
      }
    cnt += tot;
  }
  if (!base && threadIdx.x == 0) {
    gp<uint32_t>(a.span_)[2 * s] = first;
    gp<uint32_t>(a.span_)[2 * s + 1] = active ? cnt : 0u;
  }
}

__global__ void __launch_bounds__(256) sort_kernel(SortArgs a) {
  __shared__ uint32_t wsum[4];
  sort_item(a, blockIdx.x, wsum);
}

// ------------------------------------------------------- memory to LDS ----

// Until at most N of this wave's loads and stores are in flight.
template <int N>
__device__ __forceinline__ void wait_vm() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// The block meets: every wave's LDS reads so far have their data, so what they read may
// be loaded over behind this, and of its loads from memory at most N are in flight.
// (The barrier itself waits for nothing, and the compiler may leave a wait for an LDS
// read, with the matrix instruction that needs it, behind the barrier.)
template <int N>
__device__ __forceinline__ void meet() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

typedef int rsrc_t __attribute__((ext_vector_type(4)));

// The size of the largest buffer, and so an offset behind every buffer.
constexpr uint32_t kBufferEnd = 0x7ffffff0u;
// Operands of a tile's product span at most 2^30 + 2^26 bytes from their base
// (rows are kept in their own order where a batch spans more): an offset that is
// behind them, also with the offset of a k step or another such offset added.
constexpr uint32_t kOutside = 0x60000000u;
constexpr uint64_t kGatherSpan = 1ull << 30;

// A raw buffer of `bytes` at `base`, uniform over the wave:
// a lane whose offset lies past it reads zeros.
__device__ __forceinline__ rsrc_t buffer(uint64_t base, uint64_t bytes) {
  return rsrc_t{(int)(uint32_t)base, (int)(uint32_t)(base >> 32),
                (int)min(bytes, (uint64_t)kBufferEnd), 0x00027000};
}

// 16 bytes a lane from buffer offset voff + soff to LDS byte `to` + 16 * lane.
// The builtin for this makes the compiler wait for every load in flight before
// the next LDS read; written out, the kernel's own vmcnt waits count.  (No
// output registers: nothing for the compiler to reuse while the load flies.)
__device__ __forceinline__ void dma16(const rsrc_t& r, uint32_t to, uint32_t voff, uint32_t soff) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "buffer_load_dwordx4 %1, %2, %3 offen lds"
      :
      : "s"(to), "v"(voff), "s"(r), "s"(soff)
      : "m0", "memory");
}

// The same from a 64-bit address of each lane.
__device__ __forceinline__ void dma16(uint64_t from, uint32_t to) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %1, off"
      :
      : "s"(to), "v"(from)
      : "m0", "memory");
}

__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return (uint32_t)(uintptr_t)(RLD_LDS const void*)p;
}

__device__ __forceinline__ RLD_LDS unsigned char* lds_at(uint32_t a) {
  return (RLD_LDS unsigned char*)(uintptr_t)a;
}

__device__ __forceinline__ uint4 lds16(const RLD_LDS unsigned char* p) {
  const u32x4 v = *reinterpret_cast<const RLD_LDS u32x4*>(p);
  return make_uint4(v.x, v.y, v.z, v.w);
}

// A fragment from a tile whose rows are k: eight k (rows r, r + 1 .. r + 3 and
// the four behind them, `skip` bytes on) of one column.  The lanes of a group
// of 16 address four columns of four rows each and get a column of four rows.
__device__ __forceinline__ uint4 lds_tr16(RLD_LDS unsigned char* p, int skip) {
  const uint2 lo = __builtin_bit_cast(
      uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((RLD_LDS s16x4*)p));
  const uint2 hi = __builtin_bit_cast(
      uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((RLD_LDS s16x4*)(p + skip)));
  return make_uint4(lo.x, lo.y, hi.x, hi.y);
}

// What the 32-byte column pairs of row k are swapped by, where a row of such a tile
// has PAIRS of them: half a wave reads rows 0 .. 3 of two neighbouring eights at a
// time, whose eight places should lie on all of the 256 bytes of banks.  (Rows of
// 128 bytes take turns in its halves by themselves, rows of 64 in its quarters.)
template <int PAIRS>
__device__ __forceinline__ uint32_t tr_swap(uint32_t k) {
  const uint32_t eight = (k >> 3) & 1;
  return PAIRS >= 8 ? (k & 3) | eight << 2
         : PAIRS == 4 ? ((k >> 1) & 1) | eight << 1
         : PAIRS == 2 ? eight : 0;
}

// Buffer accesses that need no branch: lanes past the end read zeros and store
// nothing.
__device__ __forceinline__ uint4 buffer_load16(uint64_t base, uint64_t bytes, uint32_t off) {
  const auto r = __builtin_amdgcn_make_buffer_rsrc(
      (void*)base, 0, (int)min(bytes, (uint64_t)kBufferEnd), 0x00027000);
  const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0);
  return make_uint4(v.x, v.y, v.z, v.w);
}

__device__ __forceinline__ void buffer_store8(uint64_t base, uint64_t bytes, uint32_t off,
                                              const uint2v& v) {
  const auto r = __builtin_amdgcn_make_buffer_rsrc(
      (void*)base, 0, (int)min(bytes, (uint64_t)kBufferEnd), 0x00027000);
  __builtin_amdgcn_raw_buffer_store_b64(v, r, off, 0, 0);
}

__device__ __forceinline__ uint32_t buffer_load2(uint64_t base, uint64_t bytes, uint32_t off) {
  const auto r = __builtin_amdgcn_make_buffer_rsrc(
      (void*)base, 0, (int)min(bytes, (uint64_t)kBufferEnd), 0x00027000);
  return (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, off, 0, 0);
}

// A value that is the same in every lane, in scalar registers.
__device__ __forceinline__ uint64_t uniform64(uint64_t v) {
  return (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)v) |
         (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(v >> 32)) << 32;
}

// -------------------------------------------------------------------- low ----

struct LowArgs {
  uint64_t x_, mtab_, otab_, stab_, partial_;
  uint64_t order_;  // sorted positions' rows, or 0: positions are rows
  uint64_t key_;    // slots by position
  // the values' bf16 parts, [n][np][R]: up to two copies (0: not wanted), and
  // where a position goes in either (0: the same place)
  uint64_t parts_[2], at_[2];
  uint32_t xs, n, max_loras, K, R, np, kc, nch, nz, tiles;
};

// Four columns of a low row, scaled, to where they are wanted.
__device__ __forceinline__ void store_low(const LowArgs& a, uint32_t from, uint32_t col,
                                          floatx4 v) {
  uint2v part[3];
#pragma unroll
  for (int p = 0; p < 3; ++p) {
    const floatx4 f = p ? v
                        : floatx4{first_part(v[0]), first_part(v[1]), first_part(v[2]),
                                  first_part(v[3])};
    part[p] = uint2v{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3])};
    const floatx4 is = {bf16_to_f32(part[p].x & 0xffffu), bf16_to_f32(part[p].x >> 16),
                        bf16_to_f32(part[p].y & 0xffffu), bf16_to_f32(part[p].y >> 16)};
#pragma unroll
    for (int i = 0; i < 4; ++i)  // of an infinite second part nothing remains
      v[i] = p == 1 && v[i] == is[i] ? 0.f : v[i] - is[i];
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (!a.parts_[i]) continue;
    const uint32_t pos = a.at_[i] ? (uint32_t)gp<const int32_t>(a.at_[i])[from] : from;
    RLD_GLOBAL uint16_t* q = gp<uint16_t>(a.parts_[i]) + (size_t)pos * a.np * a.R + col;
    *reinterpret_cast<RLD_GLOBAL uint2v*>(q) = part[0];
    *reinterpret_cast<RLD_GLOBAL uint2v*>(q + a.R) = part[1];
    if (a.np > 2) *reinterpret_cast<RLD_GLOBAL uint2v*>(q + 2 * a.R) = part[2];
  }
}

// A slot's two table entries, of which `mine` is the matrix of the product at
// hand.  Up to 64 slots the wave loads the whole tables, one slot a lane, while
// the rows' slot ids are still on their way.
struct SlotTables {
  uint64_t mine, other;  // this lane's slot
  uint64_t mtab, otab;
  bool held;
  __device__ __forceinline__ SlotTables(uint64_t m, uint64_t o, uint32_t max_loras)
      : mtab(m), otab(o), held(max_loras <= 64) {
    const uint32_t lane = threadIdx.x & 63;
    mine = other = 0;
    if (held && lane < max_loras) {
      mine = gp<const uint64_t>(m)[lane];
      other = gp<const uint64_t>(o)[lane];
    }
  }
  // of a slot that is the same in the whole wave; 0: not adapted
  __device__ __forceinline__ uint64_t at(int s) const {
    uint64_t a, b;
    if (held) {
      a = lane64(mine, s);
      b = lane64(other, s);
    } else {
      a = uniform64(gp<const uint64_t>(mtab)[s]);
      b = uniform64(gp<const uint64_t>(otab)[s]);
    }
    return a != 0ull && b != 0ull ? a : 0ull;
  }
  static __device__ __forceinline__ uint64_t lane64(uint64_t v, int l) {
    return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, l) |
           (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), l) << 32;
  }
};

// The r-th set bit of m (r below their number).
__device__ __forceinline__ uint32_t nth_bit(uint64_t m, uint32_t r) {
  uint32_t at = 0;
#pragma unroll
  for (int w = 32; w; w >>= 1) {
    const uint32_t c = __popcll(m & ((1ull << w) - 1));
    const bool up = r >= c;
    r -= up ? c : 0u;
    at += up ? w : 0;
    m = up ? m >> w : m;
  }
  return at;
}

constexpr int kLowStages = 4;
constexpr int kLowLds = kLowStages * 128 * 128;

// One item: 64 positions, one k chunk, every nz-th of the distinct slots that
// they name, one after another: that slot's positions, close together (the
// places behind them hold zeros), times 64 columns of its matrix at a time.
// x and the matrix go by in 64-wide k steps through LDS, in whole 128-byte
// pieces; four waves of 32 x 32.
// TRANS: the matrix is [K][R] (B_s) instead of [R][K] (A_s).
// Bound by reading x: u of 4096 rows of 12288 and g of 4096 in 34.5 us, 134 MB at
// 3.9 TB/s (a large copy reaches 4.7).
template <bool TRANS>
__device__ __forceinline__ void low_item(const LowArgs& a, uint32_t item, unsigned char* lds) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, c = lane & 15;
  const int wr = wave >> 1, wc = wave & 1;
  const uint32_t tile = item % a.tiles, ch = item / a.tiles % a.nch;
  const uint32_t z = item / (a.tiles * a.nch);
  const uint32_t pos0 = tile * kLowRows;
  const uint32_t kb = ch * a.kc, ke = min(kb + a.kc, a.K), nk = (ke - kb + 63) / 64;
  const uint32_t lds0 = lds_addr(lds);
  const uint64_t zeros = (uint64_t)&g_zero16[0];

  const SlotTables tables(a.mtab_, a.otab_, a.max_loras);
  const int key = pos0 + lane < a.n ? gp<const int32_t>(a.key_)[pos0 + lane] : -1;
  const int row_of = (a.order_ && pos0 + lane < a.n) ? gp<const int32_t>(a.order_)[pos0 + lane]
                                                     : (int)(pos0 + lane);
  uint64_t left = __ballot(key >= 0 && (uint32_t)key < a.max_loras);
  for (uint32_t idx = 0; left; ++idx) {
    const int s = __builtin_amdgcn_readlane(key, __builtin_ctzll(left));
    const uint64_t mine = __ballot(key == s);
    left &= ~mine;
    if (idx % a.nz != z) continue;
    const uint64_t mt = tables.at(s);
    if (mt == 0ull) continue;
    const uint32_t cnt = __popcll(mine);

    // this wave's loads of a stage: two of eight rows of x, two of the matrix
    uint64_t px[2];
    uint32_t kx[2], km[2], vm[2];
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const uint32_t r = (wave + 4 * p) * 8 + (lane >> 3);
      const uint32_t q = (lane & 7) ^ ((r >> 1) & 7);
      const uint32_t row = (uint32_t)__shfl(row_of, (int)nth_bit(mine, min(r, cnt - 1)));
      px[p] = a.x_ + ((uint64_t)row * a.xs + kb + q * 8) * 2;
      kx[p] = r < cnt ? kb + q * 8 : 0xff000000u;
    }
    for (uint32_t j0 = 0; j0 < a.R; j0 += 64) {
      const uint32_t ranks = min(64u, a.R - j0);
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const uint32_t r = (wave + 4 * p) * 8 + (lane >> 3);
        if constexpr (!TRANS) {
          const uint32_t q = (lane & 7) ^ ((r >> 1) & 7);
          vm[p] = r * a.K * 2 + q * 16;
          km[p] = r < ranks ? kb + q * 8 : 0xff000000u;
        } else {
          const uint32_t h = tr_swap<4>(r);
          const uint32_t col = (((lane & 7) >> 1 ^ h) * 2 + (lane & 1)) * 8;
          vm[p] = (r * a.R + col) * 2;
          km[p] = col < ranks ? kb + r : 0xff000000u;
        }
      }
      const rsrc_t rm =
          TRANS ? buffer(mt + ((uint64_t)kb * a.R + j0) * 2, ((uint64_t)(ke - kb) * a.R - j0) * 2)
                : buffer(mt + ((uint64_t)j0 * a.K + kb) * 2,
                         ((uint64_t)(ranks - 1) * a.K + ke - kb) * 2);
      auto issue = [&](uint32_t t) {
        const uint32_t st = lds0 + (t % kLowStages) * 16384 + wave * 1024;
#pragma unroll
        for (int p = 0; p < 2; ++p)
          dma16(kx[p] + t * 64 < ke ? px[p] + t * 128 : zeros, st + p * 4096);
        const uint32_t at = TRANS ? t * 128 * a.R : t * 128;
#pragma unroll
        for (int p = 0; p < 2; ++p)
          dma16(rm, st + 8192 + p * 4096, km[p] + t * 64 < ke ? vm[p] + at : kOutside, 0);
      };
      floatx4 acc[2][2] = {};
#pragma unroll
      for (int t = 0; t < kLowStages - 1; ++t) issue(t);
      for (uint32_t t = 0; t < nk; ++t) {
        meet<(kLowStages - 2) * 4>();
        issue(t + kLowStages - 1);
        const uint32_t st = lds0 + (t % kLowStages) * 16384;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          const uint32_t sw = ((ks * 4 + g) ^ (c >> 1)) * 16;
          uint4 xf[2], mf[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            xf[i] = lds16(lds_at(st + (wr * 32 + i * 16 + c) * 128 + sw));
            if constexpr (!TRANS) {
              mf[i] = lds16(lds_at(st + 8192 + (wc * 32 + i * 16 + c) * 128 + sw));
            } else {
              const int h = tr_swap<4>(8 * g + (c >> 2));
              mf[i] = lds_tr16(lds_at(st + 8192 + (ks * 32 + 8 * g + (c >> 2)) * 128 +
                                      ((wc * 2 + i) ^ h) * 32 + (c & 3) * 8),
                               4 * 128);
            }
          }
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i)
              acc[j][i] = mfma_bf16_16x16x32(mf[j], xf[i], acc[j][i]);
        }
      }
      meet<0>();  // the loads past the end too, of zeros: the places may be loaded again
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t r = wr * 32 + i * 16 + c;
        const uint32_t pos = pos0 + nth_bit(mine, min(r, cnt - 1));
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t col = j0 + wc * 32 + j * 16 + 4 * g;
          if (r >= cnt || col >= a.R) continue;
          if (a.partial_)
            *gp<floatx4>(a.partial_ + (((size_t)ch * a.n + pos) * a.R + col) * 4) = acc[j][i];
          else
            store_low(a, pos, col, acc[j][i] * gp<const float>(a.stab_)[s]);
        }
      }
    }
  }
}

__global__ void __launch_bounds__(256) low_kernel(LowArgs a) {
  __shared__ __attribute__((aligned(1024))) unsigned char lds[kLowLds];
  low_item<false>(a, blockIdx.x, lds);
}

// u = x A^T and g = dy B in one launch: the first `items` blocks make u.
__global__ void __launch_bounds__(256) low_pair_kernel(LowArgs u, LowArgs gr, uint32_t items) {
  __shared__ __attribute__((aligned(1024))) unsigned char lds[kLowLds];
  if (blockIdx.x < items) low_item<false>(u, blockIdx.x, lds);
  else low_item<true>(gr, blockIdx.x - items, lds);
}

// low[p] = scale_s * (the chunks' sums in chunk order), routed rows only.
__device__ __forceinline__ void low_sum(const LowArgs& a, uint32_t block) {
  const uint32_t q = a.R / 4;
  const uint64_t t = (uint64_t)block * 256 + threadIdx.x;
  if (t >= (uint64_t)a.n * q) return;
  const uint32_t pos = (uint32_t)(t / q);
  const int s = gp<const int32_t>(a.key_)[pos];
  if (s < 0 || (uint32_t)s >= a.max_loras) return;
  floatx4 sum = {};
#pragma unroll 8
  for (uint32_t ch = 0; ch < a.nch; ++ch)
    sum += gp<const floatx4>(a.partial_)[(size_t)ch * a.n * q + t];
  store_low(a, pos, (uint32_t)(t % q) * 4, sum * gp<const float>(a.stab_)[s]);
}

__global__ void __launch_bounds__(256) low_reduce_kernel(LowArgs u, LowArgs gr, uint32_t blocks) {
  if (blockIdx.x < blocks) low_sum(u, blockIdx.x);
  else low_sum(gr, blockIdx.x - blocks);
}

// ------------------------------------------------------------------- tile ----

struct TileArgs {
  uint64_t x_, w_, out_, parts_, etab_;
  uint64_t order_;  // sorted positions' rows, or 0: rows in their own order, their
                    // offsets taken from a tile's first row
  uint64_t skey_;   // slots by position
  uint32_t xs, ws, os, n, K, N, R, np, tiles_m, tiles_n;
};

// The row at position p, less the row that offsets are taken from.
__device__ __forceinline__ uint32_t tile_row(const TileArgs& a, uint32_t p, uint32_t first) {
  return (a.order_ ? (uint32_t)gp<const int32_t>(a.order_)[p] : p) - first;
}

// The last K - k0 < 64 of the product, from global memory (zeros past K).
template <int MI, int NI, bool TRANS>
__device__ __forceinline__ void k_tail(const TileArgs& a, uint32_t k0, floatx4 (&acc)[NI][MI],
                                       uint32_t row0, uint32_t col0,
                                       const uint32_t (&rows_at)[MI],
                                       const uint32_t (&cols_at)[NI]) {
  const int lane = threadIdx.x & 63;
  const uint32_t rows = a.n - row0, cols = a.N - col0;
  const uint32_t first = a.order_ ? 0u : row0;
  const uint64_t x = a.x_ + (uint64_t)first * a.xs * 2;
  for (; k0 < a.K; k0 += 32) {
    int tl = lane;  // offsets are computed here, not before the loop and held
    asm volatile("" : "+v"(tl));
    const int g = tl >> 4, c = tl & 15;
    const uint32_t k = k0 + 8 * g;
    uint4 wf[NI];
#pragma unroll
    for (int ni = 0; ni < NI; ++ni) {
      const uint32_t col = cols_at[ni] + c;
      const bool in = k < a.K && col < cols;
      if constexpr (!TRANS) {
        wf[ni] = buffer_load16(a.w_ + (uint64_t)col0 * a.ws * 2, kBufferEnd,
                               in ? (col * a.ws + k) * 2 : kBufferEnd);
      } else {
        uint32_t e[8];
#pragma unroll
        for (int q = 0; q < 8; ++q)
          e[q] = buffer_load2(a.w_ + ((uint64_t)(k0 + q) * a.ws + col0) * 2, kBufferEnd,
                              in ? 16 * g * a.ws + col * 2 : kBufferEnd);
        wf[ni] = make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16,
                            e[6] | e[7] << 16);
      }
    }
#pragma unroll
    for (int mi = 0; mi < MI; ++mi) {
      const uint32_t r = rows_at[mi] + c;
      const uint32_t o = tile_row(a, row0 + min(r, rows - 1), first);
      const uint4 xf = buffer_load16(x, kBufferEnd,
                                     (k < a.K && r < rows) ? (o * a.xs + k) * 2 : kBufferEnd);
#pragma unroll
      for (int ni = 0; ni < NI; ++ni) acc[ni][mi] = mfma_bf16_16x16x32(wf[ni], xf, acc[ni][mi]);
      if (mi % 4 == 3) issue_point();
    }
  }
}

// acc[ni][mi] of a wave holds the 16 x 16 block of positions row0 + rows_at[mi] ..
// and columns col0 + cols_at[ni] .. , transposed: lane (g, c) has columns
// 4g .. 4g + 3 of position c.

// The rounded outputs to their rows.
template <int MI, int NI>
__device__ __forceinline__ void store_tile(const TileArgs& a, const floatx4 (&acc)[NI][MI],
                                           uint32_t row0, uint32_t col0,
                                           const uint32_t (&rows_at)[MI],
                                           const uint32_t (&cols_at)[NI]) {
  const int lane = threadIdx.x & 63;
  const uint32_t rows = a.n - row0, cols = a.N - col0;
  const uint32_t first = a.order_ ? 0u : row0;
  const uint64_t out = a.out_ + ((uint64_t)first * a.os + col0) * 2;
  uint32_t at[MI];
#pragma unroll
  for (int mi = 0; mi < MI; ++mi) {
    const uint32_t r = rows_at[mi] + (lane & 15);
    at[mi] = tile_row(a, row0 + min(r, rows - 1), first);
  }
#pragma unroll
  for (int mi = 0; mi < MI; ++mi) {
    int tl = lane;  // offsets are computed here, not ahead and held
    asm volatile("" : "+v"(tl));
    const uint32_t r = rows_at[mi] + (tl & 15);
#pragma unroll
    for (int ni = 0; ni < NI; ++ni) {
      const uint32_t col = cols_at[ni] + 4 * (tl >> 4);
      const floatx4 v = acc[ni][mi];
      buffer_store8(out, kBufferEnd,
                    (r < rows && col < cols) ? (at[mi] * a.os + col) * 2 : kBufferEnd,
                    uint2v{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])});
    }
    issue_point();
  }
}

// ------------------------------------------------------------------- part ----

struct PartArgs {
  uint64_t x_, w_, sum_;  // sum_: fp32 [splits][n][N]
  uint32_t xs, ws, n, K, N;
  uint32_t tiles_m, tiles_n, splits, steps;  // steps of 64 of K in a split
};

// A BM x BN tile of x W^T over one split of K, for calls too small to fill the
// chip with large tiles: K is split until a grid does, and finish adds the
// splits.  Four waves (WR x WC); K goes by in steps of 64 through STAGES LDS
// buffers that buffer loads fill directly, 16 bytes a lane in whole 128-byte
// pieces of a row (lanes past the operand's end get zeros).  Chunk q of row r
// lies at q ^ (r/2 % 8), so that the 16 rows of a fragment read fall on all
// banks.  TRANS: W is [K][N]; its tile keeps that order, 32-byte column pairs
// swizzled by the row, and transposing LDS reads make the fragments.
// The product is computed transposed (W as the first operand), so a lane
// holds four consecutive output columns of one row.
// Bound by reading W where rows are few (64 rows 4096 -> 4096 with their low rows in
// 9.5 us, 36 MB at 3.8 TB/s; 256 rows 4096 -> 12288 in 43.4 us, 144 MB of W, 31 slots' A,
// x and the sums at 3.3 TB/s, of which the counters see 190 MB, 4.4 TB/s), else by
// how far the two blocks of a CU overlap their LDS and matrix work: 1792 rows 4096 ->
// 4096 in 67 us, 900 TFLOP/s, and no faster where all loads hit the cache; 450 with
// one block a CU (1237 rows 4096 -> 1024 in 23 us).  Three stages, so one block a CU,
// take 25 to 40% longer, tiles of 64 columns 5 to 10%.
template <int BM, int BN, int WR, int WC, int STAGES, bool TRANS>
__device__ __forceinline__ void part_item(const PartArgs& a, uint32_t item, unsigned char* lds) {
  constexpr int MI = BM / (16 * WR), NI = BN / (16 * WC);
  constexpr int LA = BM / 8, LB = BN / 8;       // 1 KB loads of a stage
  constexpr int PL = (LA + LB + 3) / 4;         // of a wave
  constexpr int kStageB = (BM + BN) * 128;
  constexpr int kPairs = BN / 16;
  static_assert(WR * WC == 4, "four waves");
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, c = lane & 15;
  const int wr = wave / WC, wc = wave % WC;
  const uint32_t tiles = a.tiles_m * a.tiles_n;
  // Runs of items on one XCD (blocks go to the 8 in turn), in patches four tiles
  // high: neighbours read their slabs of x and W through one L2 (1237 ragged
  // rows 33.3 us against 34.6 in the grid's order, 256 decode rows 76.8 and 78.4).
  const uint32_t xcd = item & 7, all = tiles * a.splits;
  const uint32_t id = xcd * (all >> 3) + min(xcd, all & 7) + (item >> 3);
  const uint32_t split = id / tiles, tile = id % tiles;
  const uint32_t patch = tile / (4 * a.tiles_n), in = tile % (4 * a.tiles_n);
  const uint32_t high = min(4u, a.tiles_m - patch * 4);
  const uint32_t row0 = (patch * 4 + in % high) * BM, col0 = in / high * BN;
  const uint32_t rows = min((uint32_t)BM, a.n - row0), cols = min((uint32_t)BN, a.N - col0);
  const uint32_t kt0 = split * a.steps;
  const uint32_t nk = min(a.steps, (a.K + 63) / 64 - kt0);

  const rsrc_t rx =
      buffer(a.x_ + (uint64_t)row0 * a.xs * 2, ((uint64_t)(rows - 1) * a.xs + a.K) * 2);
  const rsrc_t rw0 =
      buffer(a.w_ + (uint64_t)col0 * a.ws * 2, ((uint64_t)(cols - 1) * a.ws + a.K) * 2);
  // Load j of this wave is load wave + 4 j of the stage (the last again where
  // there is none: every wave counts the same number of loads).
  uint32_t off[PL], kq[PL], to[PL];
  bool is_x[PL];
#pragma unroll
  for (int j = 0; j < PL; ++j) {
    const int i = min(wave + 4 * j, LA + LB - 1);
    is_x[j] = i < LA;
    to[j] = i * 1024;
    const uint32_t r = (is_x[j] ? i : i - LA) * 8 + (lane >> 3);
    const uint32_t q = (lane & 7) ^ ((r >> 1) & 7);
    kq[j] = q * 8;
    off[j] = r * (is_x[j] ? a.xs : a.ws) * 2 + q * 16;
    if (TRANS && !is_x[j]) {
      constexpr int CPR = BN / 8;  // chunks of a row
      const uint32_t k = (i - LA) * (64 / CPR) + lane / CPR;
      const uint32_t slot = lane % CPR;
      const uint32_t h = tr_swap<kPairs>(k);
      off[j] = k * a.ws * 2 + (((slot >> 1) ^ h) * 2 + (slot & 1)) * 16;
      kq[j] = 0;
    }
  }
  const uint32_t lds0 = lds_addr(lds);
  auto issue = [&](uint32_t kt) {
    const uint32_t st = lds0 + (kt % STAGES) * kStageB;
    const uint32_t k0 = (kt0 + kt) * 64;
    const bool in = kt < nk;
    rsrc_t rw = rw0;
    if constexpr (TRANS)
      rw = buffer(a.w_ + ((uint64_t)(in ? k0 : 0) * a.ws + col0) * 2,
                  in ? ((uint64_t)(a.K - k0 - 1) * a.ws + a.N - col0) * 2 : 0);
#pragma unroll
    for (int j = 0; j < PL; ++j) {
      uint32_t v = off[j];
      if (k0 + 64 > a.K && k0 + kq[j] >= a.K && (is_x[j] || !TRANS)) v = kOutside;
      const bool rows_of_k = !is_x[j] && TRANS;
      const uint32_t at = rows_of_k ? 0u : in ? k0 * 2 : kOutside;
      dma16(is_x[j] ? rx : rw, st + to[j], v, at);
    }
  };

  floatx4 acc[NI][MI];
#pragma unroll
  for (int ni = 0; ni < NI; ++ni)
#pragma unroll
    for (int mi = 0; mi < MI; ++mi) acc[ni][mi] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int t = 0; t < STAGES - 1; ++t) issue(t);

  for (uint32_t kt = 0; kt < nk; ++kt) {
    meet<(STAGES - 2) * PL>();
    issue(kt + STAGES - 1);
    const uint32_t st = lds0 + (kt % STAGES) * kStageB;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      uint4 xf[MI], wf[NI];
      const uint32_t sw = ((ks * 4 + g) ^ (c >> 1)) * 16;
#pragma unroll
      for (int mi = 0; mi < MI; ++mi)
        xf[mi] = lds16(lds_at(st + (wr * MI * 16 + c) * 128 + sw) + mi * 2048);
#pragma unroll
      for (int ni = 0; ni < NI; ++ni) {
        if constexpr (!TRANS) {
          wf[ni] = lds16(lds_at(st + BM * 128 + (wc * NI * 16 + c) * 128 + sw) + ni * 2048);
        } else {
          const int h = tr_swap<kPairs>(8 * g + (c >> 2));
          wf[ni] = lds_tr16(lds_at(st + BM * 128 + (ks * 32 + 8 * g + (c >> 2)) * (BN * 2) +
                                   ((wc * NI + ni) ^ h) * 32 + (c & 3) * 8),
                            4 * BN * 2);
        }
      }
      // matrix work before the other block's reads, where both compute much (dy W of
      // 1536 rows 4096 -> 4096: the call 92 us against 100; x W^T the same, small
      // tiles 2% slower)
      if constexpr (TRANS && BM == 128) __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int ni = 0; ni < NI; ++ni)
#pragma unroll
        for (int mi = 0; mi < MI; ++mi)
          acc[ni][mi] = mfma_bf16_16x16x32(wf[ni], xf[mi], acc[ni][mi]);
      if constexpr (TRANS && BM == 128) __builtin_amdgcn_s_setprio(0);
    }
  }
  wait_vm<0>();  // the loads past the end, of zeros

#pragma unroll
  for (int mi = 0; mi < MI; ++mi) {
    const uint32_t r = (wr * MI + mi) * 16 + c;
    if (r >= rows) continue;
#pragma unroll
    for (int ni = 0; ni < NI; ++ni) {
      const uint32_t col = col0 + (wc * NI + ni) * 16 + 4 * g;
      if (col < a.N)
        *gp<floatx4>(a.sum_ + (((uint64_t)split * a.n + row0 + r) * a.N + col) * 4) = acc[ni][mi];
    }
  }
}

// ----------------------------------------------------------------- finish ----

struct FinishArgs {
  uint64_t sum_, out_;     // fp32 [splits][n][N]; the output
  uint64_t order_;         // sorted positions' rows, or 0: positions are rows
  uint64_t key_;           // slots by position (raw ids if order_ is 0)
  uint64_t etab_, otab_, stab_;
  uint64_t parts_;         // bf16 [n][np][R], or 0: from
  uint64_t partial_;       // fp32 [nch][n][R]; by row, or by position with low_sorted
  uint32_t os, n, N, R, splits, nch, max_loras, tiles;  // tiles: of 64 columns
  uint32_t low_sorted, np;
};

// 16 * MI positions x 64 columns, 16 columns a wave: the splits of the product,
// in order, plus the low rows times their slots' second matrices.  A slot's
// product is made apart and added to its own rows alone (a NaN or infinity of
// its matrix would survive zeros in the others).  KS: 32-wide steps of rank.
// TRANS: the matrices are [R][N]; their 64 columns go through LDS (32 KB) and
// transposing reads.
// Bound by reading the sums and the slots' matrices: 256 rows of 31 slots of rank
// 64, 12288 columns in 22 us, 80 MB at 3.7 TB/s; 5 us of a single row are latency.
template <int KS, int MI, bool TRANS>
__device__ __forceinline__ void finish_item(const FinishArgs& a, uint32_t item,
                                            unsigned char* lds) {
  constexpr int SB = KS == 1 ? 8 : KS == 2 ? 4 : 2;  // slots whose matrices are loaded at once
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, c = lane & 15;
  const uint32_t tile0 = item % a.tiles * 64, col0 = tile0 + wave * 16;
  const uint32_t pos0 = item / a.tiles * (16 * MI);
  const SlotTables tables(a.etab_, a.otab_, a.max_loras);
  const uint32_t col = col0 + 4 * g;
  const bool in_col = col < a.N;
  int key[MI], left[MI];
  uint32_t row[MI];
#pragma unroll
  for (int mi = 0; mi < MI; ++mi) {
    const uint32_t pos = pos0 + mi * 16 + c, at = min(pos, a.n - 1);
    key[mi] = gp<const int32_t>(a.key_)[at];
    row[mi] = a.order_ ? (uint32_t)gp<const int32_t>(a.order_)[at] : at;
    if (pos >= a.n || key[mi] < 0 || (uint32_t)key[mi] >= a.max_loras) key[mi] = -1;
    left[mi] = key[mi];
  }

  floatx4 acc[MI];
#pragma unroll
  for (int mi = 0; mi < MI; ++mi) acc[mi] = floatx4{0.f, 0.f, 0.f, 0.f};
  constexpr int SP = MI == 1 ? 4 : 2;  // splits loaded at once
  for (uint32_t sp = 0; sp < a.splits; sp += SP) {
    floatx4 v[SP][MI];
#pragma unroll
    for (int i = 0; i < SP; ++i) {
      const uint64_t at =
          a.sum_ + ((uint64_t)min(sp + i, a.splits - 1) * a.n * a.N + (in_col ? col : 0u)) * 4;
#pragma unroll
      for (int mi = 0; mi < MI; ++mi)
        v[i][mi] = *gp<const floatx4>(at + (uint64_t)row[mi] * a.N * 4);
    }
#pragma unroll
    for (int i = 0; i < SP; ++i)
#pragma unroll
      for (int mi = 0; mi < MI; ++mi)
        if (sp + i < a.splits) acc[mi] += v[i][mi];
  }

  auto next_slot = [&]() {
    int first = -1;
#pragma unroll
    for (int mi = 0; mi < MI; ++mi) first = first < 0 ? left[mi] : first;
    const uint64_t m = __ballot(first >= 0);
    if (!m) return -1;
    const int s = __builtin_amdgcn_readlane(first, __builtin_ctzll(m));
#pragma unroll
    for (int mi = 0; mi < MI; ++mi) left[mi] = left[mi] == s ? -1 : left[mi];
    return s;
  };
  int s = next_slot();
  [[maybe_unused]] const uint32_t lds0 = lds_addr(lds);
  if (s >= 0) {
    uint4 hi[MI][KS], lo[MI][KS];
#pragma unroll
    for (int mi = 0; mi < MI; ++mi) {
      const uint32_t at = a.low_sorted ? pos0 + mi * 16 + c : row[mi];
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const uint32_t k = ks * 32 + 8 * g;
        hi[mi][ks] = lo[mi][ks] = zero16();
        if (key[mi] >= 0 && k < a.R) {
          if (a.parts_) {
            const RLD_GLOBAL uint16_t* p = gp<const uint16_t>(a.parts_) + (size_t)at * a.np * a.R + k;
            hi[mi][ks] = load16(p);
            lo[mi][ks] = load16(p + a.R);
          } else {
            floatx4 u = {}, v = {};
#pragma unroll 8
            for (uint32_t ch = 0; ch < a.nch; ++ch) {
              const RLD_GLOBAL floatx4* p =
                  gp<const floatx4>(a.partial_ + (((size_t)ch * a.n + at) * a.R + k) * 4);
              u += p[0];
              v += p[1];
            }
            const float sc = gp<const float>(a.stab_)[key[mi]];
            float f[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              f[i] = u[i] * sc;
              f[4 + i] = v[i] * sc;
            }
            uint4 two[2];
            bf16_parts(f, two);
            hi[mi][ks] = two[0];
            lo[mi][ks] = two[1];
          }
        }
      }
    }
    while (s >= 0) {
      int of[SB];  // the slots of this turn; -1: none, or not adapted
      uint4 ef[SB][KS];
#pragma unroll
      for (int b = 0; b < SB; ++b) {
        of[b] = s;
        if (s >= 0) {
          const uint64_t eb = tables.at(s);
          if (eb == 0ull) of[b] = -1;
          s = next_slot();
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            if constexpr (!TRANS) {
              const uint32_t k = ks * 32 + 8 * g;
              ef[b][ks] = buffer_load16(
                  eb + (uint64_t)col0 * a.R * 2, eb != 0ull ? kBufferEnd : 0u,
                  (k < a.R && col0 + c < a.N) ? (c * a.R + k) * 2 : kBufferEnd);
            } else {
              const uint32_t r = ks * 32 + wave * 8 + (lane >> 3);
              const uint32_t h = tr_swap<4>(r);
              const uint32_t cc = (((lane & 7) >> 1 ^ h) * 2 + (lane & 1)) * 8;
              const rsrc_t re = buffer(eb + (uint64_t)tile0 * 2,
                                       eb != 0ull ? ((uint64_t)a.R * a.N - tile0) * 2 : 0u);
              dma16(re, lds0 + (b * KS + ks) * 4096 + wave * 1024,
                    (r < a.R && tile0 + cc < a.N) ? (r * a.N + cc) * 2 : kOutside, 0);
            }
          }
        }
      }
      if constexpr (TRANS) {
        meet<0>();
      }
#pragma unroll
      for (int b = 0; b < SB; ++b) {
        if (of[b] < 0) continue;
        if constexpr (TRANS) {
          const int h = tr_swap<4>(8 * g + (c >> 2));
#pragma unroll
          for (int ks = 0; ks < KS; ++ks)
            ef[b][ks] = lds_tr16(lds_at(lds0 + (b * KS + ks) * 4096 + (8 * g + (c >> 2)) * 128 +
                                        (wave ^ h) * 32 + (c & 3) * 8),
                                 4 * 128);
        }
#pragma unroll
        for (int mi = 0; mi < MI; ++mi) {
          floatx4 t = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            t = mfma_bf16_16x16x32(ef[b][ks], lo[mi][ks], t);
            t = mfma_bf16_16x16x32(ef[b][ks], hi[mi][ks], t);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[mi][i] += key[mi] == of[b] ? t[i] : 0.f;
        }
      }
      if constexpr (TRANS) {
        meet<0>();  // the next slots may come
      }
    }
  }
#pragma unroll
  for (int mi = 0; mi < MI; ++mi)
    if (pos0 + mi * 16 + c < a.n && in_col)
      *gp<uint2v>(a.out_ + ((size_t)row[mi] * a.os + col) * 2) =
          uint2v{pack_bf16x2(acc[mi][0], acc[mi][1]), pack_bf16x2(acc[mi][2], acc[mi][3])};
}

// Work on a product that no other work of the call waits for goes out together:
// first the product's tiles, then the low rows (u, g), then the sort.
struct StartArgs {
  PartArgs part;
  LowArgs u, g;
  SortArgs sort;
  uint32_t parts, us, gs, sorts;  // blocks of each
};

template <int BM, int BN, int WR, int WC, int STAGES, bool TRANS>
__device__ __forceinline__ void start_body(const StartArgs& a) {
  constexpr int kTile = STAGES * (BM + BN) * 128;
  __shared__ __attribute__((aligned(1024))) unsigned char lds[kTile > kLowLds ? kTile : kLowLds];
  uint32_t b = blockIdx.x;
  if (b < a.parts) return part_item<BM, BN, WR, WC, STAGES, TRANS>(a.part, b, lds);
  b -= a.parts;
  if (b < a.us) return low_item<false>(a.u, b, lds);
  b -= a.us;
  if (TRANS && b < a.gs) return low_item<true>(a.g, b, lds);
  b -= a.gs;
  sort_item(a.sort, b, reinterpret_cast<uint32_t*>(lds));
}

template <int BM, int BN, int WR, int WC, int STAGES, bool TRANS>
__global__ void __launch_bounds__(256, 2) start_kernel(StartArgs a) {
  start_body<BM, BN, WR, WC, STAGES, TRANS>(a);
}

// ------------------------------------------------------------- large tiles ----

// A 256 x 256 tile by 2 x 4 waves of 128 x 64, for grids that fill the chip.
//
// The tile's k steps of 64 are cut into half operands (128 rows, 16 KB): X0, X1
// and W0, W1, two of each in LDS.  A step has four phases, each of one half of
// the rows against one half of the columns (16 matrix instructions a wave):
//   phase    multiplies    reads from LDS      loads into the place just read
//     0      X0 W0         X0 of this step     W0 of the step after next
//     1      X0 W1         W1                  X0
//     2      X1 W1         X1                  W1
//     3      X1 W0         W0 of the next step X1
// so that twelve loads of each wave stay in flight all the time, one and a half
// steps ahead.  Waves 4-7 run one barrier behind waves 0-3 (each SIMD has one
// of either): while one half multiplies, the other reads.
//
// Bound by the matrix cores' rate under these loads: 4096 x 12288 x 4096 with 64
// ranks of low rows 310-340 us, 1.23 PFLOP/s (a library's product without them: 270);
// dy W 320-345 (310).  The whole call took 495 us with 128 x 128 tiles of four waves, now 345.
//
// What makes it safe.  Every phase is
//   reads, loads, wait (reads done; all but 12 loads landed), barrier,
//   matrix instructions, barrier.
// A half operand is read at the earliest one phase, hence two barriers, after
// each wave waited for its loads of it (they are the oldest 2 of 14), of which
// the shift of one barrier leaves one.  A place is loaded again one phase
// after its read, and a wave's reads are done before the barrier in between.
template <bool TRANS>
__device__ __forceinline__ void big_tile_body(const TileArgs& a) {
  __shared__ __attribute__((aligned(1024))) unsigned char lds[2 * 65536];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, c = lane & 15;
  const int wr = wave >> 2, wc = wave & 3;
  // Runs of tiles on one XCD, in patches four tiles high: the 32 tiles that an
  // XCD works on at once share 4 row and 8 column slabs through its L2.
  const uint32_t total = a.tiles_m * a.tiles_n;
  const uint32_t pid = xcd_work_item(total);
  if (pid >= total) return;
  const uint32_t patch = pid / (4 * a.tiles_n), in = pid % (4 * a.tiles_n);
  const uint32_t high = min(4u, a.tiles_m - patch * 4);
  const uint32_t row0 = (patch * 4 + in % high) * 256, col0 = in / high * 256;

  const uint32_t rows = min(256u, a.n - row0), cols = min(256u, a.N - col0);
  const uint32_t first = a.order_ ? 0u : row0;
  const rsrc_t rx = buffer(a.x_ + (uint64_t)first * a.xs * 2,
                           ((uint64_t)((a.order_ ? a.n : rows) - 1) * a.xs + a.K) * 2);
  const rsrc_t rw0 =
      buffer(a.w_ + (uint64_t)col0 * a.ws * 2, ((uint64_t)(cols - 1) * a.ws + a.K) * 2);
  // The slot of the first row: its low rows and second matrix are loaded as if
  // they were steps behind K (a scalar load, the same for the whole block).
  const int slot0 = *(const RLD_CONST int*)(a.skey_ + (uint64_t)row0 * 4);
  uint64_t e0 = 0;
  if (slot0 >= 0) e0 = *(const RLD_CONST uint64_t*)(a.etab_ + (uint64_t)slot0 * 8);

  uint32_t vx[2][2], vw[2][2];  // [half][load]
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const uint32_t r = (wave * 2 + p) * 8 + (lane >> 3);
    const uint32_t q = (lane & 7) ^ ((r >> 1) & 7);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t hr = h * 128 + r;
      const uint32_t o = tile_row(a, row0 + min(hr, rows - 1), first);
      vx[h][p] = hr < rows ? o * a.xs * 2 + q * 16 : kOutside;
      if constexpr (!TRANS) {
        vw[h][p] = (h * 128 + r) * a.ws * 2 + q * 16;
      } else {
        const uint32_t k = (wave * 2 + p) * 4 + (lane >> 4);
        const uint32_t slot = lane & 15;
        const uint32_t sw = ((k & 3) | ((k >> 3) & 3) << 2) & 7;
        vw[h][p] = k * a.ws * 2 + h * 256 + (((slot >> 1) ^ sw) * 2 + (slot & 1)) * 16;
      }
    }
  }
  // Whole steps; the last K % 64 are added from global memory after the loop.
  // Steps go in pairs: with an odd number, step 0 has operands of zeros.
  const uint32_t nk = a.K / 64, odd = nk & 1, steps = nk + odd;
  const uint32_t lds0 = lds_addr(lds);
  const uint32_t put = lds0 + wave * 2048;
  // places of the halves in a step's 64 KB: X0, X1, W0, W1
  auto load_x = [&](int h, uint32_t t, int buf) {
    const uint32_t at = t < odd ? kOutside : (t - odd) * 128;
#pragma unroll
    for (int p = 0; p < 2; ++p)
      dma16(rx, put + buf * 65536 + h * 16384 + p * 1024, vx[h][p], at);
  };
  auto load_w = [&](int h, uint32_t t, int buf) {
    const uint32_t to = put + buf * 65536 + 32768 + h * 16384;
    if constexpr (TRANS) {
      const uint32_t k0 = t < odd ? 0 : (t - odd) * 64;
      const rsrc_t rw =
          buffer(a.w_ + ((uint64_t)k0 * a.ws + col0) * 2,
                 t < odd ? 0 : ((uint64_t)(a.K - k0 - 1) * a.ws + a.N - col0) * 2);
#pragma unroll
      for (int p = 0; p < 2; ++p) dma16(rw, to + p * 1024, vw[h][p], 0);
    } else {
      const uint32_t at = t < odd ? kOutside : (t - odd) * 128;
#pragma unroll
      for (int p = 0; p < 2; ++p) dma16(rw0, to + p * 1024, vw[h][p], at);
    }
  };
  // Low operands, 64 of rank from k0: half h of the rows' part `lo` (0 or 1) into
  // the X places, half h of a slot's second matrix into the W places.
  const uint32_t lrow = a.np * a.R * 2;  // bytes of a row's parts
  const rsrc_t rlow = buffer(a.parts_ + (uint64_t)row0 * lrow, (uint64_t)rows * lrow);
  auto load_low = [&](int h, int lo, uint32_t k0, int buf) {
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const uint32_t r = (wave * 2 + p) * 8 + (lane >> 3);
      const uint32_t k = k0 + ((lane & 7) ^ ((r >> 1) & 7)) * 8;
      dma16(rlow, put + buf * 65536 + h * 16384 + p * 1024,
            k < a.R ? (h * 128 + r) * lrow + (lo * a.R + k) * 2 : kOutside, 0);
    }
  };
  auto load_e = [&](int h, uint64_t e, uint32_t k0, int buf) {
    const uint32_t to = put + buf * 65536 + 32768 + h * 16384;
    if constexpr (TRANS) {
      const rsrc_t re =
          buffer(e + ((uint64_t)k0 * a.N + col0) * 2,
                 e == 0 || k0 >= a.R ? 0 : ((uint64_t)(a.R - k0 - 1) * a.N + a.N - col0) * 2);
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const uint32_t k = (wave * 2 + p) * 4 + (lane >> 4);
        const uint32_t sw = ((k & 3) | ((k >> 3) & 3) << 2) & 7;
        const uint32_t slot = lane & 15;
        dma16(re, to + p * 1024,
              k0 + k < a.R ? k * a.N * 2 + h * 256 + (((slot >> 1) ^ sw) * 2 + (slot & 1)) * 16
                           : kOutside, 0);
      }
    } else {
      const rsrc_t re = buffer(e + (uint64_t)col0 * a.R * 2,
                               e == 0 ? 0 : (uint64_t)cols * a.R * 2);
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const uint32_t r = (wave * 2 + p) * 8 + (lane >> 3);
        const uint32_t k = k0 + ((lane & 7) ^ ((r >> 1) & 7)) * 8;
        dma16(re, to + p * 1024, k < a.R ? (h * 128 + r) * a.R * 2 + k * 2 : kOutside, 0);
      }
    }
  };

  uint4 xf[2][4], wf[2][2][2], w0n[2][2];  // xf[ks][mi], wf[half][ks][ni]
  const uint32_t gx = lds0 + (wr * 64 + c) * 128 + (g ^ (c >> 1)) * 16;
  const uint32_t gw = lds0 + 32768 + (wc * 32 + c) * 128 + (g ^ (c >> 1)) * 16;
  const uint32_t tw = lds0 + 32768 + (8 * g + (c >> 2)) * 256 + (c & 3) * 8;
  const int tsw = ((c >> 2) | g << 2) & 7;
  auto read_x = [&](int h, int buf) {
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      const RLD_LDS unsigned char* st =
          lds_at((gx ^ (ks * 64)) + buf * 65536);
#pragma unroll
      for (int mi = 0; mi < 4; ++mi) xf[ks][mi] = lds16(st + h * 16384 + mi * 2048);
    }
  };
  auto read_w = [&](int h, int buf, uint4 (&f)[2][2]) {
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
#pragma unroll
      for (int ni = 0; ni < 2; ++ni) {
        if constexpr (!TRANS) {
          const RLD_LDS unsigned char* st =
              lds_at((gw ^ (ks * 64)) + buf * 65536);
          f[ks][ni] = lds16(st + h * 16384 + ni * 2048);
        } else {
          RLD_LDS unsigned char* st =
              lds_at(tw + ((wc * 2 + ni) ^ tsw) * 32 + buf * 65536);
          f[ks][ni] = lds_tr16(st + h * 16384 + ks * 8192, 1024);
        }
      }
  };

  floatx4 acc[4][8];
#pragma unroll
  for (int ni = 0; ni < 4; ++ni)
#pragma unroll
    for (int mi = 0; mi < 8; ++mi) acc[ni][mi] = floatx4{0.f, 0.f, 0.f, 0.f};
  auto multiply = [&](int xh, int wh, const uint4 (&f)[2][2]) {
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
#pragma unroll
      for (int ni = 0; ni < 2; ++ni)
#pragma unroll
        for (int mi = 0; mi < 4; ++mi)
          acc[wh * 2 + ni][xh * 4 + mi] =
              mfma_bf16_16x16x32(f[ks][ni], xf[ks][mi], acc[wh * 2 + ni][xh * 4 + mi]);
  };
  auto settle = [&]() {  // reads done, loads of the next phase's reads landed
    asm volatile("s_waitcnt vmcnt(12) lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_setprio(1);
  };
  auto next_phase = [&]() {
    __builtin_amdgcn_s_setprio(0);
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };
  // One step from buffer `buf`: w0 holds W0 of this step, w0next gets the next's.
  // LAST: behind this step come no more of K; the loads are the low operands.
  auto step = [&](auto last, uint32_t t, int buf, uint4 (&w0)[2][2], uint4 (&w0next)[2][2]) {
    constexpr bool LAST = decltype(last)::value;
    read_x(0, buf);
    LAST ? load_e(0, e0, 0, buf) : load_w(0, t + 2, buf);
    settle();
    multiply(0, 0, w0);
    next_phase();
    read_w(1, buf, wf[1]);
    LAST ? load_low(0, buf, 0, buf) : load_x(0, t + 2, buf);
    settle();
    multiply(0, 1, wf[1]);
    next_phase();
    read_x(1, buf);
    LAST ? load_e(1, e0, 0, buf) : load_w(1, t + 2, buf);
    settle();
    multiply(1, 1, wf[1]);
    next_phase();
    read_w(0, buf ^ 1, w0next);
    LAST ? load_low(1, buf, 0, buf) : load_x(1, t + 2, buf);
    settle();
    multiply(1, 0, w0);
    next_phase();
  };

  if (steps) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      load_w(0, t, t);
      load_x(0, t, t);
      load_w(1, t, t);
      load_x(1, t, t);
    }
    asm volatile("s_waitcnt vmcnt(12)" ::: "memory");  // W0 and X0 of step 0
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    read_w(0, 0, wf[0]);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    if (wave >= 4) __builtin_amdgcn_s_barrier();  // half a phase behind
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    uint32_t t = 0;
    for (; t + 2 < steps; t += 2) {
      step(std::false_type{}, t, 0, wf[0], w0n);
      step(std::false_type{}, t + 1, 1, w0n, wf[0]);
    }
    step(std::true_type{}, t, 0, wf[0], w0n);
    step(std::true_type{}, t + 1, 1, w0n, wf[0]);
    if (wave < 4) __builtin_amdgcn_s_barrier();  // as many barriers as the others
  } else {
    load_e(0, e0, 0, 0);
    load_e(1, e0, 0, 0);
#pragma unroll
    for (int lo = 0; lo < 2; ++lo) {
      load_low(0, lo, 0, lo);
      load_low(1, lo, 0, lo);
    }
  }

  uint32_t rows_at[8], cols_at[4];
#pragma unroll
  for (int mi = 0; mi < 8; ++mi)
    rows_at[mi] = (mi >> 2) * 128 + wr * 64 + (mi & 3) * 16;
#pragma unroll
  for (int ni = 0; ni < 4; ++ni)
    cols_at[ni] = (ni >> 1) * 128 + wc * 32 + (ni & 1) * 16;
  k_tail<8, 4, TRANS>(a, nk * 64, acc, row0, col0, rows_at, cols_at);

  // The low-rank part.  The rows' first parts lie in the X places of buffer 0,
  // their second parts in buffer 1's; the slots' matrices take turns in the two
  // W places.  A slot's product is made apart and added to its own rows alone
  // (a NaN or infinity of its matrix would survive zeros in the others).
  int key[8], left[4];
#pragma unroll
  for (int mi = 0; mi < 8; ++mi) {
    const uint32_t r = rows_at[mi] + c;
    key[mi] = r < rows ? gp<const int32_t>(a.skey_)[row0 + r] : -1;
  }
  auto all_rows = [&]() {  // the tile's slots, in every wave alike
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t r = j * 64 + lane;
      left[j] = r < rows ? gp<const int32_t>(a.skey_)[row0 + r] : -1;
    }
  };
  auto next_slot = [&]() {
    int s = -1;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint64_t m = __ballot(left[j] >= 0);
      const int first_j = __builtin_amdgcn_readlane(left[j], m ? __builtin_ctzll(m) : 0);
      s = (s < 0 && m) ? first_j : s;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) left[j] = left[j] == s ? -1 : left[j];
    return s;
  };
  for (uint32_t k0 = 0; k0 < a.R; k0 += 64) {
    all_rows();
    int s = next_slot();
    if (s < 0) break;
    if (k0 != 0) {
      meet<0>();  // everyone has read what is overwritten
#pragma unroll
      for (int lo = 0; lo < 2; ++lo) {
        load_low(0, lo, k0, lo);
        load_low(1, lo, k0, lo);
      }
    }
    if (k0 != 0 || s != slot0) {  // not loaded behind K
      const uint64_t e = uniform64(gp<const uint64_t>(a.etab_)[s]);
      if (k0 == 0) meet<0>();  // what was loaded there has landed
      load_e(0, e, k0, 0);
      load_e(1, e, k0, 0);
    }
    meet<0>();
    for (int buf = 0; s >= 0; buf ^= 1) {
      const int following = next_slot();
      if (following >= 0) {
        const uint64_t e = uniform64(gp<const uint64_t>(a.etab_)[following]);
        load_e(0, e, k0, buf ^ 1);
        load_e(1, e, k0, buf ^ 1);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        bool any = false;
#pragma unroll
        for (int mi = 0; mi < 4; ++mi) any |= key[h * 4 + mi] == s;
        if (__ballot(any) == 0) continue;
#pragma unroll
        for (int wh = 0; wh < 2; ++wh) {
          uint4 ef[2][2];
          read_w(wh, buf, ef);
          floatx4 t[2][4];
#pragma unroll
          for (int ni = 0; ni < 2; ++ni)
#pragma unroll
            for (int mi = 0; mi < 4; ++mi) t[ni][mi] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int lo = 1; lo >= 0; --lo) {
            read_x(h, lo);
#pragma unroll
            for (int ks = 0; ks < 2; ++ks)
#pragma unroll
              for (int ni = 0; ni < 2; ++ni)
#pragma unroll
                for (int mi = 0; mi < 4; ++mi)
                  t[ni][mi] = mfma_bf16_16x16x32(ef[ks][ni], xf[ks][mi], t[ni][mi]);
          }
#pragma unroll
          for (int ni = 0; ni < 2; ++ni)
#pragma unroll
            for (int mi = 0; mi < 4; ++mi)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                acc[wh * 2 + ni][h * 4 + mi][i] += key[h * 4 + mi] == s ? t[ni][mi][i] : 0.f;
        }
      }
      s = following;
      meet<0>();
    }
  }
  wait_vm<0>();
  store_tile<8, 4>(a, acc, row0, col0, rows_at, cols_at);
}

template <bool TRANS>
__global__ void __launch_bounds__(512) big_tile_kernel(TileArgs a) {
  big_tile_body<TRANS>(a);
}

// ------------------------------------------------------------------ wgrad ----

struct WgradArgs {
  uint64_t v_, parts_, order_, span_, dtab_;  // parts_: bf16 [n][3][R] by position
  uint32_t vs, width, R, tiles, accumulate;
  uint64_t sum_;  // fp32 [splits][slots] results of a split, added up afterwards
  uint32_t splits, slots;
};

// The shape of a block for ranks up to 16 * RT: 128 columns of the wide operand,
// its waves over the ranks (WR) and the columns.  A stage holds kStep positions of
// both operands: 32 where that lets more blocks into a CU and they pay, two for one
// above rank 64 (4096 rows 4096 -> 4096, rank 128: dA and dB 91 us against 107) and
// five for two, mostly of finish, up to 32 (2050 rows 2048 -> 768: the call 43.7 us
// against 45.5); up to 16 and 64, 64 (with 32: 23.3 for 22.9 us of 333 rows 4096 ->
// 1024, and 452 for 450 of 4096 rows 12288 -> 4096).
template <int RT>
struct WgradShape {
  static constexpr int RP = 16 * RT;              // ranks of a row in LDS
  static constexpr int WR = RT >= 4 ? 2 : 1, WC = 4 / WR;
  static constexpr int MT = RT / WR, NT = 8 / WC;  // 16 x 16 blocks of a wave
  static constexpr int kStep = RT == 2 || RT == 8 ? 32 : 64;
  static constexpr int kWide = kStep * 256, kLow = kStep * RP * 2;
  static constexpr int kStage = kWide + 3 * kLow;
  static constexpr int kLds = 2 * kStage > 32768 ? 2 * kStage : 32768;  // finish: 32 KB
};

// Slot s, 128 columns of the wide operand (x for dA, dy for dB): the sum over
// the slot's positions of low[pos][r] * wide[row][col], kStep positions a step,
// two steps in LDS.  Both operands lie by position, as their rows do in memory,
// and are read transposed.  The low values come in three bf16 parts, which
// hold all 24 bits.  DB: the result is [col][R] instead of [R][col].  With few
// slots and columns the positions are split as well (wgrad_splits).
// Bound by the latency of a step's loads beside three times the matrix work: 4096
// rows in four slots, 12288 and 4096 columns, rank 64, 55 to 60 us, 134 MB at 2.3 TB/s
// and 440 TFLOP/s of bf16 parts.  (Rows' numbers in scalar registers, which spares waits,
// or a third stage in one block a CU: 15% longer.)
template <int RT, bool DB>
__device__ __forceinline__ void wgrad_item(const WgradArgs& a, uint32_t item, unsigned char* lds) {
  using S = WgradShape<RT>;
  constexpr int kPairs = S::RP / 16;
  constexpr int LL = S::kLow / 1024, LP = (3 * LL + 3) / 4;  // 1 KB loads of a part; a wave's
  constexpr int WL = S::kStep / 16;                          // and of the wide operand
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, c = lane & 15;
  const int wr = wave / S::WC, wc = wave % S::WC;
  const uint32_t part = item / a.tiles, split = part / a.slots, s = part % a.slots;
  const uint32_t col0 = item % a.tiles * 128;
  const uint64_t table = gp<const uint64_t>(a.dtab_)[s];
  if (table == 0ull) return;
  const bool whole = a.splits == 1;
  const uint64_t dst = whole ? table : a.sum_ + (uint64_t)part * a.width * a.R * 4;
  const uint32_t all = gp<const uint32_t>(a.span_)[2 * s + 1];
  const uint32_t per = ((all + 63) / 64 + a.splits - 1) / a.splits * 64, skip = min(split * per, all);
  const uint32_t begin = gp<const uint32_t>(a.span_)[2 * s] + skip, cnt = min(per, all - skip);
  const RLD_GLOBAL int32_t* order = gp<const int32_t>(a.order_) + begin;
  const uint64_t zeros = (uint64_t)&g_zero16[0];
  const uint32_t lds0 = lds_addr(lds);
  const uint32_t lrow = 3 * a.R * 2;
  const uint64_t parts = uniform64(a.parts_ + (uint64_t)begin * lrow);

  // this lane's rows (WL of a step) and column of the wide operand
  uint32_t rw[WL];
  uint64_t vcol[WL];
#pragma unroll
  for (int p = 0; p < WL; ++p) {
    rw[p] = (wave * WL + p) * 4 + (lane >> 4);
    const uint32_t h = tr_swap<8>(rw[p]);
    const uint32_t slot = lane & 15;
    const uint32_t col = col0 + (((slot >> 1) ^ h) * 2 + (slot & 1)) * 8;
    vcol[p] = col < a.width ? a.v_ + (uint64_t)col * 2 : 0ull;
  }
  // and of the low parts: load j is load wave + 4 j of the 3 * LL
  uint32_t vl[LP];
#pragma unroll
  for (int j = 0; j < LP; ++j) {
    const int i = min(wave + 4 * j, 3 * LL - 1);
    constexpr int CPR = S::RP / 8;  // chunks of a row
    const uint32_t k = (i % LL) * (64 / CPR) + lane / CPR;
    const uint32_t slot = lane % CPR;
    const uint32_t h = tr_swap<kPairs>(k);
    const uint32_t r = (((slot >> 1) ^ h) * 2 + (slot & 1)) * 8;
    vl[j] = r < a.R ? k * lrow + ((i / LL) * a.R + r) * 2 : kOutside;
  }
  uint32_t row[WL];
  auto rows_of = [&](uint32_t i0) {
#pragma unroll
    for (int p = 0; p < WL; ++p) {
      const uint32_t i = i0 + rw[p];
      row[p] = i < cnt ? (uint32_t)order[i] : 0xffffffffu;
    }
  };
  auto issue = [&](uint32_t i0) {  // row: of these positions
    const uint32_t st = lds0 + (i0 / S::kStep & 1) * S::kStage;
#pragma unroll
    for (int p = 0; p < WL; ++p)
      dma16((row[p] != 0xffffffffu && vcol[p]) ? vcol[p] + (uint64_t)row[p] * a.vs * 2 : zeros,
            st + (wave * WL + p) * 1024);
    const rsrc_t rl = buffer(parts + (uint64_t)i0 * lrow,
                             i0 < cnt ? (uint64_t)min(cnt - i0, (uint32_t)S::kStep) * lrow : 0);
#pragma unroll
    for (int j = 0; j < LP; ++j)
      dma16(rl, st + S::kWide + min(wave + 4 * j, 3 * LL - 1) * 1024, vl[j], 0);
  };

  floatx4 acc[S::MT][S::NT];
#pragma unroll
  for (int mt = 0; mt < S::MT; ++mt)
#pragma unroll
    for (int nt = 0; nt < S::NT; ++nt) acc[mt][nt] = floatx4{0.f, 0.f, 0.f, 0.f};

  rows_of(0);
  issue(0);
  rows_of(S::kStep);
  for (uint32_t i0 = 0; i0 < cnt; i0 += S::kStep) {
    meet<0>();
    issue(i0 + S::kStep);
    rows_of(i0 + 2 * S::kStep);
    const uint32_t st = lds0 + (i0 / S::kStep & 1) * S::kStage;
#pragma unroll
    for (int ks = 0; ks < S::kStep / 32; ++ks) {
      const uint32_t k = ks * 32 + 8 * g + (c >> 2);
      const int hw = tr_swap<8>(8 * g + (c >> 2)), hl = tr_swap<kPairs>(8 * g + (c >> 2));
      uint4 vf[S::NT];
#pragma unroll
      for (int nt = 0; nt < S::NT; ++nt)
        vf[nt] = lds_tr16(
            lds_at(st + k * 256 + ((wc * S::NT + nt) ^ hw) * 32 + (c & 3) * 8), 4 * 256);
#pragma unroll
      for (int p = 2; p >= 0; --p)
#pragma unroll
        for (int mt = 0; mt < S::MT; ++mt) {
          const uint4 lf = lds_tr16(
              lds_at(st + S::kWide + p * S::kLow + k * (S::RP * 2) +
                     ((wr * S::MT + mt) ^ hl) * 32 + (c & 3) * 8),
              4 * S::RP * 2);
#pragma unroll
          for (int nt = 0; nt < S::NT; ++nt)
            acc[mt][nt] = DB ? mfma_bf16_16x16x32(lf, vf[nt], acc[mt][nt])
                             : mfma_bf16_16x16x32(vf[nt], lf, acc[mt][nt]);
        }
    }
  }
  wait_vm<0>();  // the loads past the end, of zeros

#pragma unroll
  for (int mt = 0; mt < S::MT; ++mt)
#pragma unroll
    for (int nt = 0; nt < S::NT; ++nt) {
      // first operand: index 4g + i, four consecutive per lane; second: index c
      const uint32_t col = col0 + (wc * S::NT + nt) * 16 + (DB ? c : 4 * g);
      const uint32_t rank = (wr * S::MT + mt) * 16 + (DB ? 4 * g : c);
      if (col >= a.width || rank >= a.R) continue;
      const uint64_t at = DB ? (uint64_t)col * a.R + rank : (uint64_t)rank * a.width + col;
      RLD_GLOBAL floatx4* o = gp<floatx4>(dst + at * 4);
      *o = whole && a.accumulate ? *o + acc[mt][nt] : acc[mt][nt];
    }
}

// dA, dB and, behind them, the last part of dx in one launch: the first `ia`
// blocks make dA, the next `ib` dB.
template <int RT>
__global__ void __launch_bounds__(256, 2) end_kernel(WgradArgs da, WgradArgs db, FinishArgs fin,
                                                  uint32_t ia, uint32_t ib) {
  __shared__ __attribute__((aligned(1024))) unsigned char lds[WgradShape<RT>::kLds];
  constexpr int KS = RT < 2 ? 1 : RT / 2;
  if (blockIdx.x < ia) wgrad_item<RT, false>(da, blockIdx.x, lds);
  else if (blockIdx.x < ia + ib) wgrad_item<RT, true>(db, blockIdx.x - ia, lds);
  else finish_item<KS, kFinishRows / 16, true>(fin, blockIdx.x - ia - ib, lds);
}

template <int KS, int MI>
__global__ void __launch_bounds__(256) finish_kernel(FinishArgs a) {
  finish_item<KS, MI, false>(a, blockIdx.x, nullptr);
}

// The splits of dA and dB added up in their order, four values a thread.
__global__ void __launch_bounds__(256) wgrad_sum_kernel(WgradArgs da, WgradArgs db, uint32_t blocks) {
  const bool second = blockIdx.x >= blocks;
  const WgradArgs& a = second ? db : da;
  const uint32_t quads = a.width * (a.R / 4);
  const uint32_t i = (blockIdx.x - (second ? blocks : 0u)) * 256 + threadIdx.x;
  if (i >= a.slots * quads) return;
  const uint64_t table = gp<const uint64_t>(a.dtab_)[i / quads];
  if (table == 0ull) return;
  floatx4 v = floatx4{0.f, 0.f, 0.f, 0.f};
  for (uint32_t sp = 0; sp < a.splits; ++sp)
    v += *gp<const floatx4>(a.sum_ + ((uint64_t)sp * a.slots * quads + i) * 16);
  RLD_GLOBAL floatx4* o = gp<floatx4>(table + (uint64_t)(i % quads) * 16);
  *o = a.accumulate ? *o + v : v;
}

// ------------------------------------------------------------------- host ----

static inline size_t round16(size_t v) { return (v + 15) & ~(size_t)15; }

struct LowPlan {
  uint32_t kc, nch;
  size_t low, partial;  // bytes
};

static LowPlan low_plan(uint32_t n, uint32_t K, uint32_t R, uint32_t np) {
  LowPlan p;
  // Longer chunks once they make some 256 items: each loads its slots' tables and
  // starts its pipeline anew (4096 rows, K 4096: 13.6 us against 17.8 with 512
  // items).  Half as long for one tile of rows, whose call waits for little else.
  const uint64_t items = (uint64_t)div_ceil(n, kLowRows) * div_ceil(K, kLowChunk);
  p.kc = n <= kLowRows ? kLowChunk / 2
         : kLowChunk * (items < 512 ? 1u : items >= 256 * 16 ? 16u : (uint32_t)(items / 256));
  p.nch = div_ceil(K, p.kc);
  p.low = round16((size_t)n * R * np * 2);
  p.partial = round16((size_t)p.nch * n * R * 4);
  return p;
}

// How a product of n rows, K and N columns is cut.
struct TilePlan {
  bool big;         // 256 x 256 tiles, which also finish their outputs
  uint32_t bm, bn;  // otherwise: tiles of a part,
  uint32_t tiles_m, tiles_n, splits, steps;  // and its splits of `steps` x 64 of K
  size_t sums;      // bytes of the splits' sums
};

static TilePlan tile_plan(uint32_t n, uint32_t K, uint32_t N) {
  TilePlan p = {};
  const uint64_t big = (uint64_t)div_ceil(n, 256) * div_ceil(N, 256);
  p.big = big >= kBigTiles && N > 128;
  if (p.big) {
    p.tiles_m = div_ceil(n, 256);
    p.tiles_n = div_ceil(N, 256);
    return p;
  }
  p.bm = n <= 16 ? 16 : n <= 32 ? 32 : n <= 128 ? 64 : 128;
  p.bn = n <= 128 ? 64 : 128;
  p.tiles_m = div_ceil(n, p.bm);
  p.tiles_n = div_ceil(N, p.bn);
  // One block a CU, or two where one would leave CUs idle; of at least four
  // steps each.  (us, splits for 256 blocks against 512: 64 rows 16.1 against
  // 20.5, 1237 ragged rows 35.8 against 44.3; 192 tiles whole 91, halved 80.)
  const uint32_t tiles = p.tiles_m * p.tiles_n, steps = div_ceil(K, 64);
  uint32_t s = tiles <= 128 ? 256 / tiles : tiles <= 256 ? 2 : 1;
  if (s > steps / 4) s = steps / 4;
  if (s > 16) s = 16;
  if (s < 1) s = 1;
  p.steps = div_ceil(steps, s);
  p.splits = div_ceil(steps, p.steps);
  p.sums = round16((size_t)p.splits * n * N * 4);
  return p;
}

// How often dA's and dB's positions are split: until some 512 blocks are busy, of
// at least 256 positions each if the slots have equally many.  (us of dA and dB
// whole against split, one slot of rank 16, 4096 -> 4096: 4096 rows 69 and 48,
// 16384 rows 251 and 138, where x and dy are read twice in 113.)
static uint32_t wgrad_splits(uint32_t n, uint32_t K, uint32_t N, uint32_t slots) {
  const uint64_t items = (uint64_t)slots * (div_ceil(K, 128) + div_ceil(N, 128));
  const uint64_t s = std::min<uint64_t>(512 / items, n / ((uint64_t)slots * 256));
  return s < 1 ? 1u : s > 16 ? 16u : (uint32_t)s;
}

static size_t wgrad_bytes(uint32_t n, uint32_t K, uint32_t N, uint32_t R, uint32_t slots) {
  const uint32_t s = wgrad_splits(n, K, N, slots);
  return s == 1 ? 0 : (size_t)s * slots * R * ((size_t)K + N) * 4;
}

static size_t sort_bytes(uint32_t n, uint32_t max_loras) {
  return 4 * round16((size_t)n * 4) + round16((size_t)max_loras * 8);
}

static size_t proj_bytes(uint32_t n, uint32_t K, uint32_t N, uint32_t R, uint32_t slots) {
  const LowPlan p = low_plan(n, K, R, 2);
  return sort_bytes(n, slots) + p.low + p.partial + tile_plan(n, K, N).sums;
}

static size_t grad_bytes(uint32_t n, uint32_t K, uint32_t N, uint32_t R, uint32_t slots) {
  const LowPlan u = low_plan(n, K, R, 3), g = low_plan(n, N, R, 3);
  return sort_bytes(n, slots) + u.low + u.partial + 2 * g.low + g.partial +
         (n ? tile_plan(n, N, K).sums : 0) + wgrad_bytes(n, K, N, R, slots);
}

// The most that a call of up to n rows takes.  The plans are fixed between 16, 32
// and multiples of 64 rows, and from 2^18 rows on, so the bytes grow there.
template <class F>
static size_t most_bytes(uint32_t n, F bytes) {
  size_t most = bytes(n);
  for (uint32_t rows = 16; rows < n && rows <= 1u << 18; rows += rows < 64 ? rows : 64)
    most = std::max(most, bytes(rows));
  return most;
}

static SortArgs sort_args(const rld_route* r, const int32_t* seq, uint32_t n,
                          uint64_t workspace) {
  SortArgs a;
  a.seq_ = (uint64_t)seq;
  a.atab_ = (uint64_t)r->a_table;
  a.btab_ = (uint64_t)r->b_table;
  a.order_ = workspace;
  a.skey_ = a.order_ + round16((size_t)n * 4);
  a.rkey_ = a.skey_ + round16((size_t)n * 4);
  a.rpos_ = a.rkey_ + round16((size_t)n * 4);
  a.span_ = a.rpos_ + round16((size_t)n * 4);
  a.n = n;
  a.max_loras = r->max_loras;
  return a;
}

// order 0: low rows by row, key slots by row.
static LowArgs low_args(const rld_route* r, bool trans, const void* x, uint32_t xs, uint32_t n,
                        uint64_t order, uint64_t key, uint32_t np, uint64_t parts,
                        uint64_t partial) {
  LowArgs a;
  a.x_ = (uint64_t)x;
  a.mtab_ = (uint64_t)(trans ? r->b_table : r->a_table);
  a.otab_ = (uint64_t)(trans ? r->a_table : r->b_table);
  a.stab_ = (uint64_t)r->scale_table;
  a.partial_ = partial;
  a.order_ = order;
  a.key_ = key;
  a.np = np;
  a.parts_[0] = parts;
  a.parts_[1] = a.at_[0] = a.at_[1] = 0;
  a.xs = xs;
  a.n = n;
  a.max_loras = r->max_loras;
  a.K = trans ? r->n_out : r->k_in;
  a.R = r->max_rank;
  const LowPlan p = low_plan(n, a.K, a.R, np);
  a.kc = p.kc;
  a.nch = p.nch;
  a.tiles = div_ceil(n, kLowRows);
  // Unsorted rows: a tile's slots are items too, and up to four chunks make one where
  // they come to some 200 all the same (16 slots of rank 16, us with chunks of 512
  // against these: 256 rows 4096 -> 4096 29.3 and 27.1, 384 rows 39.4 and 36.4; of 4
  // slots, which stay, 256 rows 4096 -> 1024 22.3, and 24.8 with two in one).
  const uint64_t pieces = (uint64_t)a.tiles * a.nch * std::min(r->max_loras, kLowRows);
  if (!order && n > kLowRows && a.kc == kLowChunk && pieces >= 2 * 192) {
    a.kc *= (uint32_t)std::min<uint64_t>(4, pieces / 192);
    a.nch = div_ceil(a.K, a.kc);
  }
  // few items: the slots of a tile go to several blocks
  const uint32_t items = a.tiles * a.nch;
  a.nz = items >= 1024u ? 1u : div_ceil(1024u, items ? items : 1u);
  if (a.nz > r->max_loras) a.nz = r->max_loras;
  if (a.nz > n) a.nz = n;
  if (a.nz > kLowRows) a.nz = kLowRows;
  // sorted rows: the slots of a tile, if they have equally many rows (192 shuffled
  // rows, us with at most two against these: 64 slots, 4096 -> 4096, 63 and 36; 200
  // slots, 4096 -> 1024, 99 and 37)
  const uint32_t named = n ? 1 + div_ceil(std::min(r->max_loras, n) * kLowRows, n) : 1u;
  if (order && a.nz > named) a.nz = named;
  return a;
}

static uint32_t low_items(const LowArgs& a) { return a.tiles * a.nch * a.nz; }
static uint32_t sum_blocks(const LowArgs& a) {
  return (uint32_t)(((uint64_t)a.n * (a.R / 4) + 255) / 256);
}

// Whether the low products (of K columns in all) are worth waiting for the sort.
// Unsorted, every 64 rows may name every slot and take its matrix by itself; the
// sort takes 5 us, in which some 1000 pieces of 512 columns are multiplied so.  (us
// unsorted against sorted, 16 slots of rank 16, 4096 -> 4096, slots shuffled: 512
// rows 43.8 and 42.0, 768 rows 55.9 and 51.3, 1024 rows 73.0 and 60.4; 1237 rows
// 4096 -> 1024 in runs of one slot, the other way: 33.4 and 35.7.)
static bool sort_first(const rld_route* r, uint32_t n, uint64_t K) {
  const uint64_t slots = r->max_loras < kLowRows ? r->max_loras : kLowRows;
  return div_ceil(n, kLowRows) * slots * ((K + kLowChunk - 1) / kLowChunk) > 1024;
}

template <bool TRANS>
static int launch_start(const TilePlan& p, const StartArgs& a, hipStream_t st) {
  const uint32_t grid = a.parts + a.us + a.gs + a.sorts;
  if (p.bm == 16) start_kernel<16, 64, 1, 4, 4, TRANS><<<grid, 256, 0, st>>>(a);
  else if (p.bm == 32) start_kernel<32, 64, 1, 4, 4, TRANS><<<grid, 256, 0, st>>>(a);
  else if (p.bm == 64) start_kernel<64, 64, 2, 2, 4, TRANS><<<grid, 256, 0, st>>>(a);
  else start_kernel<128, 128, 2, 2, 2, TRANS><<<grid, 256, 0, st>>>(a);
  return launch_status();
}

template <bool TRANS>
static PartArgs part_args(const TilePlan& p, const void* w, uint32_t ws, const void* x,
                          uint32_t xs, uint32_t n, uint32_t K, uint32_t N, uint64_t sums) {
  PartArgs a;
  a.x_ = (uint64_t)x;
  a.w_ = (uint64_t)w;
  a.sum_ = sums;
  a.xs = xs;
  a.ws = ws;
  a.n = n;
  a.K = K;
  a.N = N;
  a.tiles_m = p.tiles_m;
  a.tiles_n = p.tiles_n;
  a.splits = p.splits;
  a.steps = p.steps;
  return a;
}

static FinishArgs finish_args(const rld_route* r, bool trans, const TilePlan& p, uint64_t sums,
                              uint64_t order, uint64_t key, uint64_t parts, uint64_t partial,
                              uint32_t nch, bool low_sorted, void* out, uint32_t os, uint32_t n) {
  FinishArgs a;
  a.sum_ = sums;
  a.out_ = (uint64_t)out;
  a.order_ = order;
  a.key_ = key;
  a.etab_ = (uint64_t)(trans ? r->a_table : r->b_table);
  a.otab_ = (uint64_t)(trans ? r->b_table : r->a_table);
  a.stab_ = (uint64_t)r->scale_table;
  a.parts_ = parts;
  a.partial_ = partial;
  a.os = os;
  a.n = n;
  a.N = trans ? r->k_in : r->n_out;
  a.R = r->max_rank;
  a.splits = p.splits;
  a.nch = nch;
  a.max_loras = r->max_loras;
  a.tiles = div_ceil(a.N, 64);
  a.low_sorted = low_sorted ? 1u : 0u;
  a.np = trans ? 3 : 2;
  return a;
}

template <int MI>
static int launch_finish(const FinishArgs& f, uint32_t rows, hipStream_t st) {
  const uint32_t grid = f.tiles * div_ceil(f.n, rows);
  if (f.R <= 32) finish_kernel<1, MI><<<grid, 256, 0, st>>>(f);
  else if (f.R <= 64) finish_kernel<2, MI><<<grid, 256, 0, st>>>(f);
  else finish_kernel<4, MI><<<grid, 256, 0, st>>>(f);
  return launch_status();
}

template <bool TRANS>
static int launch_big(const rld_route* r, const TilePlan& p, const void* w, uint32_t ws,
                      const void* x, uint32_t xs, uint64_t order, uint64_t key, uint32_t n,
                      uint64_t parts, void* out, uint32_t os, hipStream_t st) {
  TileArgs a;
  a.x_ = (uint64_t)x;
  a.w_ = (uint64_t)w;
  a.out_ = (uint64_t)out;
  a.parts_ = parts;
  a.etab_ = (uint64_t)(TRANS ? r->a_table : r->b_table);
  a.order_ = order;
  a.skey_ = key;
  a.xs = xs;
  a.ws = ws;
  a.os = os;
  a.n = n;
  a.K = TRANS ? r->n_out : r->k_in;
  a.N = TRANS ? r->k_in : r->n_out;
  a.R = r->max_rank;
  a.np = TRANS ? 3 : 2;
  a.tiles_m = p.tiles_m;
  a.tiles_n = p.tiles_n;
  big_tile_kernel<TRANS><<<xcd_grid(a.tiles_m * a.tiles_n), 512, 0, st>>>(a);
  return launch_status();
}

// Rows that large tiles cannot reach in any order through 32-bit offsets.
static bool too_far(uint32_t n, uint32_t stride) { return (uint64_t)n * stride * 2 > kGatherSpan; }

static int check_wide(uint32_t stride) { return stride > kMaxStride ? RLD_EUNSUPPORTED : RLD_OK; }

// A grid holds fewer than 2^32 threads of at most 256 a block.
static int check_items(const rld_route* r, uint32_t n) {
  const uint64_t k = r->k_in > r->n_out ? r->k_in : r->n_out;
  const uint64_t tiles = (k + 63) / 64;
  if (n > (1u << 26) || k > kMaxStride || div_ceil(n, 64) * tiles >= (1u << 23) ||
      r->max_loras * tiles >= (1u << 21) || (uint64_t)n * (r->max_rank / 4) >= (1u << 30))
    return RLD_EUNSUPPORTED;
  // the sort reads every id for every slot: a second at most
  if ((uint64_t)n * r->max_loras >= (1ull << 38)) return RLD_EUNSUPPORTED;
  return RLD_OK;
}

}  // namespace rld

using namespace rld;

extern "C" size_t rld_proj_workspace_bytes(uint32_t n, uint32_t k_in, uint32_t n_out,
                                           uint32_t max_rank, uint32_t max_loras) {
  if (n == 0 || k_in == 0 || n_out == 0 || max_rank == 0 || max_loras == 0) return 0;
  return most_bytes(n, [=](uint32_t rows) {
    return proj_bytes(rows, k_in, n_out, max_rank, max_loras);
  });
}

extern "C" int rld_proj(const rld_route* route, const void* w, uint32_t w_row_stride,
                        const void* x, uint32_t x_row_stride, const int32_t* seq_slot,
                        uint32_t n, void* out, uint32_t out_row_stride, void* workspace,
                        size_t workspace_bytes, void* stream) {
  int e = check_route(route);
  if (e) return e;
  if (n == 0) return RLD_OK;
  if (!seq_slot || !workspace) return RLD_EINVAL;
  if ((e = check_rows(w, w_row_stride, route->k_in))) return e;
  if ((e = check_rows(x, x_row_stride, route->k_in))) return e;
  if ((e = check_rows(out, out_row_stride, route->n_out))) return e;
  if (!aligned16(workspace)) return RLD_EALIGN;
  if ((e = check_wide(w_row_stride)) || (e = check_wide(x_row_stride)) ||
      (e = check_wide(out_row_stride)))
    return e;
  if ((e = check_items(route, n))) return e;
  const uint32_t K = route->k_in, N = route->n_out, R = route->max_rank;
  if (workspace_bytes < proj_bytes(n, K, N, R, route->max_loras))
    return RLD_ENOSPACE;
  const LowPlan p = low_plan(n, K, R, 2);
  const TilePlan t = tile_plan(n, K, N);
  const uint64_t parts = (uint64_t)workspace + sort_bytes(n, route->max_loras);
  const uint64_t partial = parts + p.low;
  const uint64_t sums = partial + p.partial;
  const uint64_t seq = (uint64_t)seq_slot;
  const hipStream_t st = (hipStream_t)stream;
  const SortArgs sort = sort_args(route, seq_slot, n, (uint64_t)workspace);

  if (t.big) {
    sort_kernel<<<route->max_loras + 1, 256, 0, st>>>(sort);
    if ((e = launch_status())) return e;
    const bool keep = too_far(n, x_row_stride) || too_far(n, out_row_stride);
    const uint64_t order = keep ? 0 : sort.order_, key = keep ? sort.rkey_ : sort.skey_;
    const LowArgs l = low_args(route, false, x, x_row_stride, n, order, key, 2, parts,
                               p.nch == 1 ? 0 : partial);
    low_kernel<<<low_items(l), 256, 0, st>>>(l);
    if ((e = launch_status())) return e;
    if (p.nch > 1) {
      low_reduce_kernel<<<sum_blocks(l), 256, 0, st>>>(l, l, sum_blocks(l));
      if ((e = launch_status())) return e;
    }
    return launch_big<false>(route, t, w, w_row_stride, x, x_row_stride, order, key, n, parts, out,
                             out_row_stride, st);
  }

  // up to 64 rows no sort: a block of finish has 16 rows' slots at most
  const bool sorted = n > 64, first = sorted && sort_first(route, n, K);
  if (first) {
    sort_kernel<<<route->max_loras + 1, 256, 0, st>>>(sort);
    if ((e = launch_status())) return e;
  }
  const LowArgs l = low_args(route, false, x, x_row_stride, n, first ? sort.order_ : 0,
                             first ? sort.skey_ : seq, 2, parts, partial);
  // finish adds up the low rows' chunks itself while they are few: each of its
  // tiles of 64 columns reads them (4096 -> 1024 at rank 16, itself against summed
  // first: 1237 rows, 10 MB read so, 35.7 us and 37.6; 2048 rows, 17 MB, 48.2 and 44.5)
  const uint64_t again = (uint64_t)div_ceil(N, 64) * n * R * 4 * l.nch;
  const bool sum = again > (12ull << 20);
  StartArgs s;
  s.part = part_args<false>(t, w, w_row_stride, x, x_row_stride, n, K, N, sums);
  s.u = l;
  s.g = l;
  s.sort = sort;
  s.sorts = sorted && !first ? route->max_loras + 1 : 0u;
  s.parts = t.tiles_m * t.tiles_n * t.splits;
  s.us = low_items(l);
  s.gs = 0;
  if ((e = launch_start<false>(t, s, st))) return e;
  if (sum) {
    low_reduce_kernel<<<sum_blocks(l), 256, 0, st>>>(l, l, sum_blocks(l));
    if ((e = launch_status())) return e;
  }
  const FinishArgs f =
      finish_args(route, false, t, sums, sorted ? sort.order_ : 0, sorted ? sort.skey_ : seq,
                  sum ? parts : 0, partial, l.nch, first, out, out_row_stride, n);
  // 64 positions a block where the low rows are summed already (adding up their
  // chunks takes longer for more rows a wave: 17 us against 10 for 1237 rows)
  return sum ? launch_finish<4>(f, 64, st) : launch_finish<1>(f, 16, st);
}

extern "C" size_t rld_proj_grad_workspace_bytes(uint32_t n, uint32_t k_in, uint32_t n_out,
                                                uint32_t max_rank, uint32_t max_loras) {
  if (k_in == 0 || n_out == 0 || max_rank == 0 || max_loras == 0) return 0;
  return most_bytes(n, [=](uint32_t rows) {
    return grad_bytes(rows, k_in, n_out, max_rank, max_loras);
  });
}

extern "C" int rld_proj_grad(const rld_route* route, const void* w, uint32_t w_row_stride,
                             const void* x, uint32_t x_row_stride, const void* dy,
                             uint32_t dy_row_stride, const int32_t* seq_slot, uint32_t n,
                             void* dx, uint32_t dx_row_stride, const uint64_t* da_table,
                             const uint64_t* db_table, int accumulate, void* workspace,
                             size_t workspace_bytes, void* stream) {
  int e = check_route(route);
  if (e) return e;
  const bool adapters = da_table || db_table;
  if (!dx && !adapters) return RLD_EINVAL;
  if (!workspace) return RLD_EINVAL;
  if (!aligned16(workspace) || ((uintptr_t)da_table & 7u) || ((uintptr_t)db_table & 7u))
    return RLD_EALIGN;
  if (n != 0) {
    if (!seq_slot) return RLD_EINVAL;
    if ((e = check_rows(dy, dy_row_stride, route->n_out))) return e;
    if ((e = check_wide(dy_row_stride))) return e;
    if (dx) {
      if ((e = check_rows(w, w_row_stride, route->k_in))) return e;
      if ((e = check_wide(w_row_stride))) return e;
      if ((e = check_rows(dx, dx_row_stride, route->k_in))) return e;
      if ((e = check_wide(dx_row_stride))) return e;
    }
    if (adapters) {
      if ((e = check_rows(x, x_row_stride, route->k_in))) return e;
    }
  }
  if ((e = check_items(route, n))) return e;
  const uint32_t K = route->k_in, N = route->n_out, R = route->max_rank;
  if (workspace_bytes < grad_bytes(n, K, N, R, route->max_loras))
    return RLD_ENOSPACE;
  if (n == 0 && !adapters) return RLD_OK;
  const LowPlan pu = low_plan(n, K, R, 3), pg = low_plan(n, N, R, 3);
  const uint64_t uparts = (uint64_t)workspace + sort_bytes(n, route->max_loras);
  const uint64_t usum = uparts + pu.low;
  const uint64_t gparts = usum + pu.partial;  // by position
  const uint64_t grows = gparts + pg.low;     // by row, for rows in their own order
  const uint64_t gsum = grows + pg.low;
  const uint64_t sums = gsum + pg.partial;
  const hipStream_t st = (hipStream_t)stream;
  const SortArgs sort = sort_args(route, seq_slot, n, (uint64_t)workspace);
  const TilePlan t = n ? tile_plan(n, N, K) : TilePlan{};
  const bool want_u = n && db_table, want_g = n && (dx || da_table);
  const bool part = n && dx && !t.big;
  // the sort first where the low products gain from it, or nothing else starts with it
  const bool first = !part || sort_first(route, n, (uint64_t)K + N);
  // low rows by sorted position, if they are sorted first and the large tiles
  // can reach the rows so
  const bool keep =
      n && dx && t.big && (too_far(n, dy_row_stride) || too_far(n, dx_row_stride));
  const bool by_pos = first && !keep;
  const uint64_t order = by_pos ? sort.order_ : 0;
  const uint64_t key = by_pos ? sort.skey_ : keep ? sort.rkey_ : (uint64_t)seq_slot;
  // u for dB; g for dx and dA: by position, and by row too where dx takes it so
  LowArgs u = low_args(route, false, x, x_row_stride, n, order, key, 3, uparts, usum);
  LowArgs g = low_args(route, true, dy, dy_row_stride, n, order, key, 3, gparts, gsum);
  if (!by_pos) u.at_[0] = g.at_[0] = sort.rpos_;
  if (keep) g.parts_[1] = grows;
  const uint32_t iu = want_u ? low_items(u) : 0u, ig = want_g ? low_items(g) : 0u;
  if (first) {
    sort_kernel<<<route->max_loras + 1, 256, 0, st>>>(sort);
    if ((e = launch_status())) return e;
  }
  if (part) {
    StartArgs s;
    s.part = part_args<true>(t, w, w_row_stride, dy, dy_row_stride, n, N, K, sums);
    s.u = u;
    s.g = g;
    s.sort = sort;
    s.sorts = first ? 0u : route->max_loras + 1;
    s.parts = t.tiles_m * t.tiles_n * t.splits;
    s.us = iu;
    s.gs = ig;
    if ((e = launch_start<true>(t, s, st))) return e;
  } else if (iu + ig) {
    low_pair_kernel<<<iu + ig, 256, 0, st>>>(u, g, iu);
    if ((e = launch_status())) return e;
  }
  if (iu + ig) {
    const uint32_t bu = want_u ? sum_blocks(u) : 0u, bg = want_g ? sum_blocks(g) : 0u;
    low_reduce_kernel<<<bu + bg, 256, 0, st>>>(u, g, bu);
    if ((e = launch_status())) return e;
  }
  if (n && dx && t.big &&
      (e = launch_big<true>(route, t, w, w_row_stride, dy, dy_row_stride, order, key, n,
                            keep ? grows : gparts, dx, dx_row_stride, st)))
    return e;
  WgradArgs a, b;
  a.v_ = (uint64_t)x;
  b.v_ = (uint64_t)dy;
  a.vs = x_row_stride;
  b.vs = dy_row_stride;
  a.parts_ = gparts;
  b.parts_ = uparts;
  a.dtab_ = (uint64_t)da_table;
  b.dtab_ = (uint64_t)db_table;
  a.width = K;
  b.width = N;
  a.order_ = b.order_ = sort.order_;
  a.span_ = b.span_ = sort.span_;
  a.R = b.R = R;
  a.accumulate = b.accumulate = accumulate ? 1u : 0u;
  a.tiles = div_ceil(a.width, 128);
  b.tiles = div_ceil(b.width, 128);
  a.slots = b.slots = route->max_loras;
  a.splits = b.splits = wgrad_splits(n, K, N, route->max_loras);
  a.sum_ = sums + t.sums;
  b.sum_ = a.sum_ + (uint64_t)a.splits * a.slots * R * K * 4;
  const uint32_t ia = da_table ? a.tiles * a.slots * a.splits : 0u;
  const uint32_t ib = db_table ? b.tiles * b.slots * b.splits : 0u;
  const FinishArgs f = finish_args(route, true, t, sums, sort.order_, sort.skey_, gparts, 0, 0, true, dx,
                                   dx_row_stride, n);
  const uint32_t grid = ia + ib + (part ? f.tiles * div_ceil(n, kFinishRows) : 0u);
  if (grid == 0) return RLD_OK;
  if (R <= 16) end_kernel<1><<<grid, 256, 0, st>>>(a, b, f, ia, ib);
  else if (R <= 32) end_kernel<2><<<grid, 256, 0, st>>>(a, b, f, ia, ib);
  else if (R <= 64) end_kernel<4><<<grid, 256, 0, st>>>(a, b, f, ia, ib);
  else end_kernel<8><<<grid, 256, 0, st>>>(a, b, f, ia, ib);
  if (a.splits > 1 && adapters) {
    if ((e = launch_status())) return e;
    const uint32_t ba = da_table ? div_ceil(a.slots * K * (R / 4), 256u) : 0u;
    const uint32_t bb = db_table ? div_ceil(b.slots * N * (R / 4), 256u) : 0u;
    wgrad_sum_kernel<<<ba + bb, 256, 0, st>>>(a, b, ba);
  }
  return launch_status();
}
