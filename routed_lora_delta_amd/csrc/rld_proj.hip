// The shared projection beside its routed adapters, and its gradient:
//
//   y_i  = x_i W^T + u_i B_s^T,   u_i = scale_s x_i A_s^T        (s = seq_slot[i])
//   dx_i = dy_i W  + g_i A_s,     g_i = scale_s dy_i B_s
//   dA_s = sum_{i in s} g_i^T x_i,   dB_s = sum_{i in s} dy_i^T u_i
//
// (W frozen).  Four kernels:
//   low      the low-rank products u and g of every routed row, as fp32 partial
//            sums of k chunks; low_reduce adds the chunks and applies the scale.
//   tile     one output tile of x W^T (or dy W) on the matrix cores, with the
//            low rows times the slots' second matrices added into the same
//            accumulators, so the output is rounded once and written once.
//   lists    each slot's rows in ascending order.
//   wgrad    dA or dB: the products over a slot's rows.
//
// u and g stay in fp32 (bf16 copies would add a rounding of 2^-9 to every
// term).  The matrix cores take bf16, so a low value enters as the sum of two
// bf16 parts where the result is rounded to bf16 (16 significand bits, an
// error of 2^-17) and of three where it is fp32 (24 bits: all of it).
#include "rld_device.hpp"
#include "rld_internal.hpp"

namespace rld {

typedef short s16x4 __attribute__((ext_vector_type(4)));
#define RLD_LDS __attribute__((address_space(3)))

constexpr uint32_t kLowRows = 64;    // rows of a low item
constexpr uint32_t kLowChunk = 512;  // k elements of a low item
constexpr uint32_t kMaxStride = 1u << 21;
constexpr uint32_t kBigTiles = 160;  // 256 x 256 tiles from which a grid of them pays

// 16 bytes of zeros per device: where a lane's source is outside the operand.
__device__ uint4 g_zero16[1];

// ------------------------------------------------------------- bf16 parts ----

// v as the sum of NP bf16 values, the largest first.  Rounding to nearest
// makes each remainder exact in fp32 (it fits the 24 - 8 bits left).
template <int NP>
__device__ __forceinline__ void bf16_parts(const float (&v)[8], uint4 (&out)[NP]) {
  float r[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) r[e] = v[e];
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      w[e] = pack_bf16x2(r[2 * e], r[2 * e + 1]);
      r[2 * e] -= bf16_to_f32(w[e] & 0xffffu);
      r[2 * e + 1] -= bf16_to_f32(w[e] >> 16);
    }
    out[p] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// -------------------------------------------------------------------- low ----

struct LowArgs {
  uint64_t x_, seq_, mtab_, otab_, stab_, partial_;
  uint64_t low_;    // fp32 [n][R], or 0: not wanted
  uint64_t parts_;  // bf16 [n][2][R]: the value's two parts, or 0
  uint32_t xs, n, max_loras, K, R, nch, nz;
};

// Four columns of a low row, scaled, to where they are wanted.
__device__ __forceinline__ void store_low(const LowArgs& a, uint32_t row, uint32_t col,
                                          const floatx4& v) {
  if (a.low_) *gp<floatx4>(a.low_ + ((size_t)row * a.R + col) * 4) = v;
  if (a.parts_) {
    const uint2v hi = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    const uint2v lo = {
        pack_bf16x2(v[0] - bf16_to_f32(hi.x & 0xffffu), v[1] - bf16_to_f32(hi.x >> 16)),
        pack_bf16x2(v[2] - bf16_to_f32(hi.y & 0xffffu), v[3] - bf16_to_f32(hi.y >> 16))};
    RLD_GLOBAL uint16_t* p = gp<uint16_t>(a.parts_) + (size_t)row * 2 * a.R + col;
    *reinterpret_cast<RLD_GLOBAL uint2v*>(p) = hi;
    *reinterpret_cast<RLD_GLOBAL uint2v*>(p + a.R) = lo;
  }
}

// One block: 64 rows, one k chunk, every nz-th of the distinct slots that the
// rows name.  The x fragments stay in registers over the slots; each wave
// contracts every fourth 32-wide step and the four sums meet in LDS.
// TRANS: the matrix is [K][R] (B_s) instead of [R][K] (A_s).
template <bool TRANS>
__global__ void __launch_bounds__(256) low_kernel(LowArgs a) {
  __shared__ floatx4 red[2][4][4][kWave];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int g = lane >> 4, c = lane & 15;
  const uint32_t tiles = div_ceil_dev(a.n, kLowRows);
  const uint32_t tile = blockIdx.x % tiles, ch = blockIdx.x / tiles % a.nch;
  const uint32_t z = blockIdx.x / (tiles * a.nch);
  const uint32_t row0 = tile * kLowRows;
  const uint32_t kb = ch * kLowChunk, ke = min(kb + kLowChunk, a.K);

  const RLD_GLOBAL int32_t* seq = gp<const int32_t>(a.seq_);
  const uint32_t myrow = row0 + lane;
  const int key = myrow < a.n ? seq[myrow] : -1;
  uint64_t left = __ballot(key >= 0 && (uint32_t)key < a.max_loras);
  if (!left) return;

  uint4 xf[4][4];
#pragma unroll
  for (int mi = 0; mi < 4; ++mi) {
    const uint32_t row = row0 + mi * 16 + c;
    const RLD_GLOBAL uint16_t* xr = gp<const uint16_t>(a.x_) + (size_t)min(row, a.n - 1) * a.xs;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t k = kb + (wave + 4 * i) * 32 + g * 8;
      xf[mi][i] = (row < a.n && k < ke) ? load16(xr + k) : zero16();
    }
  }

  int buf = 0;
  for (uint32_t idx = 0; left; ++idx) {
    const int s = __builtin_amdgcn_readlane(key, __builtin_ctzll(left));
    const uint64_t mine = __ballot(key == s);
    left &= ~mine;
    if (idx % a.nz != z) continue;
    const uint64_t mt = gp<const uint64_t>(a.mtab_)[s], ot = gp<const uint64_t>(a.otab_)[s];
    if (mt == 0ull || ot == 0ull) continue;
    const RLD_GLOBAL uint16_t* M = gp<const uint16_t>(mt);
    for (uint32_t j0 = 0; j0 < a.R; j0 += 16) {
      const uint32_t j = j0 + c;
      floatx4 acc[4] = {};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t k = kb + (wave + 4 * i) * 32 + g * 8;
        uint4 m = zero16();
        if (j < a.R && k < ke) {
          if constexpr (!TRANS) {
            m = load16(M + (size_t)j * a.K + k);
          } else {
            uint32_t e[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) e[q] = M[(size_t)(k + q) * a.R + j];
            m = make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16,
                           e[6] | e[7] << 16);
          }
        }
#pragma unroll
        for (int mi = 0; mi < 4; ++mi) acc[mi] = mfma_bf16_16x16x32(m, xf[mi][i], acc[mi]);
      }
#pragma unroll
      for (int mi = 0; mi < 4; ++mi) red[buf][wave][mi][lane] = acc[mi];
      __syncthreads();
      // wave w finishes rows 16w .. 16w+15: lane (g, c) holds columns 4g.. of row c
      floatx4 sum = red[buf][0][wave][lane];
#pragma unroll
      for (int v = 1; v < 4; ++v) sum += red[buf][v][wave][lane];
      buf ^= 1;
      const int lr = wave * 16 + c;
      const uint32_t col = j0 + 4 * g;
      if (((mine >> lr) & 1) && col < a.R) {
        if (a.nch == 1)
          store_low(a, row0 + lr, col, sum * gp<const float>(a.stab_)[s]);
        else
          *gp<floatx4>(a.partial_ + (((size_t)ch * a.n + row0 + lr) * a.R + col) * 4) = sum;
      }
    }
  }
}

__device__ __forceinline__ bool low_active(const LowArgs& a, int s) {
  if (s < 0 || (uint32_t)s >= a.max_loras) return false;
  const uint64_t t = gp<const uint64_t>(a.mtab_)[s], o = gp<const uint64_t>(a.otab_)[s];
  return t != 0ull && o != 0ull;
}

// low[i] = scale_s * (the chunks' sums in chunk order), routed rows only.
__global__ void __launch_bounds__(256) low_reduce_kernel(LowArgs a) {
  const uint32_t q = a.R / 4;
  const uint64_t t = (uint64_t)blockIdx.x * 256 + threadIdx.x;
  if (t >= (uint64_t)a.n * q) return;
  const uint32_t row = (uint32_t)(t / q);
  const int s = gp<const int32_t>(a.seq_)[row];
  if (!low_active(a, s)) return;
  floatx4 sum = {};
  for (uint32_t ch = 0; ch < a.nch; ++ch)
    sum += gp<const floatx4>(a.partial_)[(size_t)ch * a.n * q + t];
  store_low(a, row, (uint32_t)(t % q) * 4, sum * gp<const float>(a.stab_)[s]);
}

// ------------------------------------------------------------------- tile ----

struct TileArgs {
  uint64_t x_, w_, out_, seq_, parts_, etab_, otab_;
  uint32_t xs, ws, os, n, K, N, R, max_loras, tiles_m, tiles_n;
};

// Until at most N of this wave's loads and stores are in flight.
template <int N>
__device__ __forceinline__ void wait_vm() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

typedef int rsrc_t __attribute__((ext_vector_type(4)));

// The size of the largest buffer, and so an offset behind every buffer.
constexpr uint32_t kBufferEnd = 0x7ffffff0u;

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
      : "memory");
}

__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return (uint32_t)(uintptr_t)(RLD_LDS const void*)p;
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

// The last K - k0 < 64 of the product, from global memory (zeros past K).
template <int MI, int NI, bool TRANS>
__device__ __forceinline__ void k_tail(const TileArgs& a, uint32_t k0, floatx4 (&acc)[NI][MI],
                                       uint32_t row0, uint32_t col0,
                                       const uint32_t (&rows_at)[MI],
                                       const uint32_t (&cols_at)[NI]) {
  const int lane = threadIdx.x & 63;
  const uint32_t rows = a.n - row0, cols = a.N - col0;
  const uint64_t x = a.x_ + (uint64_t)row0 * a.xs * 2;
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
      const uint4 xf = buffer_load16(x, kBufferEnd,
                                     (k < a.K && r < rows) ? (r * a.xs + k) * 2 : kBufferEnd);
#pragma unroll
      for (int ni = 0; ni < NI; ++ni) acc[ni][mi] = mfma_bf16_16x16x32(wf[ni], xf, acc[ni][mi]);
      if (mi % 4 == 3) issue_point();
    }
  }
}

// A value that is the same in every lane, in scalar registers.
__device__ __forceinline__ uint64_t uniform64(uint64_t v) {
  return (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)v) |
         (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(v >> 32)) << 32;
}

// What follows a tile's main product: the low-rank part and the store.
// acc[ni][mi] holds the 16 x 16 block of rows row0 + rows_at[mi] .. and columns
// col0 + cols_at[ni] .. , transposed: lane (g, c) has columns 4g .. 4g + 3 of
// row c.  No branch touches the accumulators (they fill the registers): every
// slot of the wave's rows goes through all row blocks, with zeros for the rows
// of other slots, which then leave its product out (a NaN or infinity of its
// matrix would survive the zeros).
template <int MI, int NI, bool TRANS>
__device__ __forceinline__ void finish_tile(const TileArgs& a, floatx4 (&acc)[NI][MI],
                                            uint32_t row0, uint32_t col0,
                                            const uint32_t (&rows_at)[MI],
                                            const uint32_t (&cols_at)[NI]) {
  constexpr int MH = MI < 4 ? MI : 4;  // row blocks whose low rows are held at once
  const int lane = threadIdx.x & 63;
  const int g = lane >> 4, c = lane & 15;
  const uint32_t rows = a.n - row0, cols = a.N - col0;  // at least one tile's, or up to the end

  int key[MI];  // the slot of a routed row, -1 for base rows and rows done
#pragma unroll
  for (int mi = 0; mi < MI; ++mi) {
    const uint32_t r = rows_at[mi] + c;
    int k = r < rows ? gp<const int32_t>(a.seq_)[row0 + r] : -1;
    if (k < 0 || (uint32_t)k >= a.max_loras) k = -1;
    const uint64_t e = gp<const uint64_t>(a.etab_)[k < 0 ? 0 : k];
    const uint64_t o = gp<const uint64_t>(a.otab_)[k < 0 ? 0 : k];
    key[mi] = (e != 0ull && o != 0ull) ? k : -1;
  }
  const uint64_t low = a.parts_ + (uint64_t)row0 * a.R * 4;
  const uint32_t R = a.R;
  int s = -1;
  uint64_t et = 0;
  for (uint32_t k0 = R;; k0 += 32) {
    if (k0 >= R) {  // on to the first slot that is left
      int first = -1;
#pragma unroll
      for (int mi = 0; mi < MI; ++mi) {
        key[mi] = key[mi] == s ? -1 : key[mi];
        first = first < 0 ? key[mi] : first;
      }
      const uint64_t m = __ballot(first >= 0);
      if (!m) break;
      s = __builtin_amdgcn_readlane(first, __builtin_ctzll(m));
      et = uniform64(gp<const uint64_t>(a.etab_)[s]);
      k0 = 0;
    }
    // the lane through an empty asm: offsets are computed here, not before the
    // loop and held
    int tl = lane;
    asm volatile("" : "+v"(tl));
    const int g = tl >> 4, c = tl & 15;
    const uint32_t k = k0 + 8 * g;
    uint4 ef[NI];
#pragma unroll
    for (int ni = 0; ni < NI; ++ni) {
      const uint32_t col = cols_at[ni] + c;
      const bool in = k < R && col < cols;
      if constexpr (!TRANS) {
        ef[ni] = buffer_load16(et + (uint64_t)col0 * R * 2, kBufferEnd,
                               in ? (col * R + k) * 2 : kBufferEnd);
      } else {
        uint32_t e[8];
#pragma unroll
        for (int q = 0; q < 8; ++q)
          e[q] = buffer_load2(et + ((uint64_t)(k0 + q) * a.N + col0) * 2, kBufferEnd,
                              in ? 16 * g * a.N + col * 2 : kBufferEnd);
        ef[ni] = make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16,
                            e[6] | e[7] << 16);
      }
    }
#pragma unroll
    for (int h = 0; h < MI; h += MH) {
      uint4 hi[MH], lo[MH];
#pragma unroll
      for (int mi = 0; mi < MH; ++mi) {
        const uint32_t at = (rows_at[h + mi] + c) * R * 4 + k * 2;
        const uint32_t off = (key[h + mi] == s && k < R) ? at : kBufferEnd;
        hi[mi] = buffer_load16(low, kBufferEnd, off);
        lo[mi] = buffer_load16(low + R * 2, kBufferEnd, off);
      }
#pragma unroll
      for (int mi = 0; mi < MH; ++mi) {
        const bool mine = key[h + mi] == s;
#pragma unroll
        for (int ni = 0; ni < NI; ++ni) {
          floatx4 t = mfma_bf16_16x16x32(ef[ni], lo[mi], floatx4{0.f, 0.f, 0.f, 0.f});
          t = mfma_bf16_16x16x32(ef[ni], hi[mi], t);
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[ni][h + mi][i] += mine ? t[i] : 0.f;
        }
      }
      issue_point();
    }
  }

  const uint64_t out = a.out_ + ((uint64_t)row0 * a.os + col0) * 2;
#pragma unroll
  for (int mi = 0; mi < MI; ++mi) {
    int tl = lane;
    asm volatile("" : "+v"(tl));
    const int g = tl >> 4, c = tl & 15;
    const uint32_t r = rows_at[mi] + c;
    const uint32_t at = r * a.os * 2;
#pragma unroll
    for (int ni = 0; ni < NI; ++ni) {
      const uint32_t col = cols_at[ni] + 4 * g;
      const floatx4 v = acc[ni][mi];
      buffer_store8(out, kBufferEnd, (r < rows && col < cols) ? at + col * 2 : kBufferEnd,
                    uint2v{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])});
    }
    issue_point();
  }
}

// A BM x BN output tile by WR x WC waves.  K goes by in steps of 64 through
// STAGES LDS buffers that buffer loads fill directly (16 bytes a lane; lanes
// past the operand's end get zeros).  Rows of 128 bytes are swizzled: chunk q
// of row r lies at q ^ (r/2 % 8), so that the 16 rows of a fragment read fall
// on all banks.  TRANS: W is [K][N]; its tile keeps that order, 32-byte
// column pairs swizzled by the row, and transposing LDS reads make the
// fragments.
// The product is computed transposed (W as the first operand), so a lane
// holds four consecutive output columns of one row.
template <int BM, int BN, int WR, int WC, int STAGES, bool TRANS>
__device__ __forceinline__ void tile_body(const TileArgs& a) {
  constexpr int NW = WR * WC;
  constexpr int MI = BM / (16 * WR), NI = BN / (16 * WC);
  constexpr int PA = BM / (8 * NW), PB = BN / (8 * NW);
  constexpr int kStageB = (BM + BN) * 128;
  constexpr int kPairs = BN / 16;
  __shared__ __attribute__((aligned(1024))) unsigned char lds[STAGES * kStageB];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, c = lane & 15;
  const int wr = wave / WC, wc = wave % WC;
  const uint32_t tm = blockIdx.x % a.tiles_m, tn = blockIdx.x / a.tiles_m;
  const uint32_t row0 = tm * BM, col0 = tn * BN;
  const uint32_t rows = min((uint32_t)BM, a.n - row0);

  const rsrc_t rx = buffer(a.x_ + (uint64_t)row0 * a.xs * 2,
                           ((uint64_t)(rows - 1) * a.xs + a.K) * 2);
  const uint32_t wrows = min((uint32_t)BN, a.N - col0);
  const rsrc_t rw0 = buffer(a.w_ + (uint64_t)col0 * a.ws * 2,
                            ((uint64_t)(wrows - 1) * a.ws + a.K) * 2);

  uint32_t va[PA], vb[PB];
#pragma unroll
  for (int p = 0; p < PA; ++p) {
    const uint32_t r = (wave * PA + p) * 8 + (lane >> 3);
    va[p] = r * a.xs * 2 + (((lane & 7) ^ ((r >> 1) & 7)) * 16);
  }
#pragma unroll
  for (int p = 0; p < PB; ++p) {
    if constexpr (!TRANS) {
      const uint32_t r = (wave * PB + p) * 8 + (lane >> 3);
      vb[p] = r * a.ws * 2 + (((lane & 7) ^ ((r >> 1) & 7)) * 16);
    } else {
      constexpr int CPR = BN / 8;  // chunks of a row
      const uint32_t k = (wave * PB + p) * (64 / CPR) + lane / CPR;
      const uint32_t slot = lane % CPR;
      const uint32_t h = ((k & 3) | ((k >> 3) & 3) << 2) & (kPairs - 1);
      vb[p] = k * a.ws * 2 + (((slot >> 1) ^ h) * 2 + (slot & 1)) * 16;
    }
  }
  const uint32_t nk = (a.K + 63) / 64;
  const uint32_t lds0 = lds_addr(lds);
  auto issue = [&](uint32_t kt) {
    const uint32_t st = __builtin_amdgcn_readfirstlane(lds0 + (kt % STAGES) * kStageB);
    const uint32_t k0 = kt * 64;
    const bool tail = k0 + 64 > a.K;
#pragma unroll
    for (int p = 0; p < PA; ++p) {
      uint32_t v = va[p];
      if (tail) {
        const uint32_t r = (wave * PA + p) * 8 + (lane >> 3);
        const uint32_t k = k0 + (((lane & 7) ^ ((r >> 1) & 7)) * 8);
        if (k >= a.K) v = kBufferEnd;
      }
      dma16(rx, st + (wave * PA + p) * 1024, v, k0 * 2);
    }
    if constexpr (!TRANS) {
#pragma unroll
      for (int p = 0; p < PB; ++p) {
        uint32_t v = vb[p];
        if (tail) {
          const uint32_t r = (wave * PB + p) * 8 + (lane >> 3);
          const uint32_t k = k0 + (((lane & 7) ^ ((r >> 1) & 7)) * 8);
          if (k >= a.K) v = kBufferEnd;
        }
        dma16(rw0, st + BM * 128 + (wave * PB + p) * 1024, v, k0 * 2);
      }
    } else {
      const bool in = k0 < a.K;
      const rsrc_t rw = buffer(a.w_ + ((uint64_t)(in ? k0 : 0) * a.ws + col0) * 2,
                               in ? ((uint64_t)(a.K - k0 - 1) * a.ws + a.N - col0) * 2 : 0);
#pragma unroll
      for (int p = 0; p < PB; ++p)
        dma16(rw, st + BM * 128 + (wave * PB + p) * 1024, vb[p], 0);
    }
  };

  floatx4 acc[NI][MI];
#pragma unroll
  for (int ni = 0; ni < NI; ++ni)
#pragma unroll
    for (int mi = 0; mi < MI; ++mi) acc[ni][mi] = floatx4{0.f, 0.f, 0.f, 0.f};

#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s) issue(s);

  for (uint32_t kt = 0; kt < nk; ++kt) {
    wait_vm<(STAGES - 2) * (PA + PB)>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    issue(kt + STAGES - 1);
    const unsigned char* st = lds + (kt % STAGES) * kStageB;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      uint4 xf[MI], wf[NI];
#pragma unroll
      for (int mi = 0; mi < MI; ++mi)
        xf[mi] = *reinterpret_cast<const uint4*>(st + ((wr * MI + mi) * 16 + c) * 128 +
                                                 ((ks * 4 + g) ^ (c >> 1)) * 16);
#pragma unroll
      for (int ni = 0; ni < NI; ++ni) {
        if constexpr (!TRANS) {
          wf[ni] = *reinterpret_cast<const uint4*>(st + BM * 128 +
                                                   ((wc * NI + ni) * 16 + c) * 128 +
                                                   ((ks * 4 + g) ^ (c >> 1)) * 16);
        } else {
          const int h = ((c >> 2) | g << 2) & (kPairs - 1);
          const unsigned char* p = st + BM * 128 + (ks * 32 + 8 * g + (c >> 2)) * (BN * 2) +
                                   ((wc * NI + ni) ^ h) * 32 + (c & 3) * 8;
          const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((RLD_LDS s16x4*)p);
          const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
              (RLD_LDS s16x4*)(p + 4 * BN * 2));
          const uint2 l2 = __builtin_bit_cast(uint2, lo), h2 = __builtin_bit_cast(uint2, hi);
          wf[ni] = make_uint4(l2.x, l2.y, h2.x, h2.y);
        }
      }
#pragma unroll
      for (int ni = 0; ni < NI; ++ni)
#pragma unroll
        for (int mi = 0; mi < MI; ++mi)
          acc[ni][mi] = mfma_bf16_16x16x32(wf[ni], xf[mi], acc[ni][mi]);
    }
  }

  wait_vm<0>();  // the loads past K, of zeros

  uint32_t rows_at[MI], cols_at[NI];
#pragma unroll
  for (int mi = 0; mi < MI; ++mi) rows_at[mi] = (wr * MI + mi) * 16;
#pragma unroll
  for (int ni = 0; ni < NI; ++ni) cols_at[ni] = (wc * NI + ni) * 16;
  finish_tile<MI, NI, TRANS>(a, acc, row0, col0, rows_at, cols_at);
}

template <int BM, int BN, int WR, int WC, int STAGES, bool TRANS>
__global__ void __launch_bounds__(64 * WR * WC) tile_kernel(TileArgs a) {
  tile_body<BM, BN, WR, WC, STAGES, TRANS>(a);
}

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
  const rsrc_t rx =
      buffer(a.x_ + (uint64_t)row0 * a.xs * 2, ((uint64_t)(rows - 1) * a.xs + a.K) * 2);
  const rsrc_t rw0 =
      buffer(a.w_ + (uint64_t)col0 * a.ws * 2, ((uint64_t)(cols - 1) * a.ws + a.K) * 2);
  uint32_t vx[2][2], vw[2][2];  // [half][load]
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const uint32_t r = (wave * 2 + p) * 8 + (lane >> 3);
    const uint32_t q = (lane & 7) ^ ((r >> 1) & 7);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      vx[h][p] = (h * 128 + r) * a.xs * 2 + q * 16;
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
  // Loads of steps past the end are sent behind the buffers' ends.
  const uint32_t nk = a.K / 64;
  const uint32_t lds0 = lds_addr(lds);
  const uint32_t put = lds0 + wave * 2048;
  // places of the halves in a step's 64 KB: X0, X1, W0, W1
  auto load_x = [&](int h, uint32_t kt, int buf) {
    const uint32_t at = kt < nk ? kt * 128 : 0x7f000000u;
#pragma unroll
    for (int p = 0; p < 2; ++p)
      dma16(rx, put + buf * 65536 + h * 16384 + p * 1024, vx[h][p], at);
  };
  auto load_w = [&](int h, uint32_t kt, int buf) {
    const uint32_t to = put + buf * 65536 + 32768 + h * 16384;
    if constexpr (TRANS) {
      const uint32_t k0 = kt < nk ? kt * 64 : 0;
      const rsrc_t rw =
          buffer(a.w_ + ((uint64_t)k0 * a.ws + col0) * 2,
                 kt < nk ? ((uint64_t)(a.K - k0 - 1) * a.ws + a.N - col0) * 2 : 0);
#pragma unroll
      for (int p = 0; p < 2; ++p) dma16(rw, to + p * 1024, vw[h][p], 0);
    } else {
      const uint32_t at = kt < nk ? kt * 128 : 0x7f000000u;
#pragma unroll
      for (int p = 0; p < 2; ++p) dma16(rw0, to + p * 1024, vw[h][p], at);
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
          (const RLD_LDS unsigned char*)((gx ^ (ks * 64)) + buf * 65536);
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
              (const RLD_LDS unsigned char*)((gw ^ (ks * 64)) + buf * 65536);
          f[ks][ni] = lds16(st + h * 16384 + ni * 2048);
        } else {
          RLD_LDS unsigned char* st =
              (RLD_LDS unsigned char*)(tw + ((wc * 2 + ni) ^ tsw) * 32 + buf * 65536);
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
  auto meet = [&]() {
    __builtin_amdgcn_s_setprio(0);
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };
  // One step from buffer `buf`: w0 holds W0 of this step, w0next gets the next's.
  auto step = [&](uint32_t kt, int buf, uint4 (&w0)[2][2], uint4 (&w0next)[2][2]) {
    read_x(0, buf);
    load_w(0, kt + 2, buf);
    settle();
    multiply(0, 0, w0);
    meet();
    read_w(1, buf, wf[1]);
    load_x(0, kt + 2, buf);
    settle();
    multiply(0, 1, wf[1]);
    meet();
    read_x(1, buf);
    load_w(1, kt + 2, buf);
    settle();
    multiply(1, 1, wf[1]);
    meet();
    read_w(0, buf ^ 1, w0next);
    load_x(1, kt + 2, buf);
    settle();
    multiply(1, 0, w0);
    meet();
  };

#pragma unroll
  for (int kt = 0; kt < 2; ++kt) {
    load_w(0, kt, kt);
    load_x(0, kt, kt);
    load_w(1, kt, kt);
    load_x(1, kt, kt);
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
  // steps in pairs; past the last the operands are zeros
  for (uint32_t kt = 0; kt < nk; kt += 2) {
    step(kt, 0, wf[0], w0n);
    step(kt + 1, 1, w0n, wf[0]);
  }
  if (wave < 4) __builtin_amdgcn_s_barrier();  // as many barriers as the others
  wait_vm<0>();

  uint32_t rows_at[8], cols_at[4];
#pragma unroll
  for (int mi = 0; mi < 8; ++mi)
    rows_at[mi] = (mi >> 2) * 128 + wr * 64 + (mi & 3) * 16;
#pragma unroll
  for (int ni = 0; ni < 4; ++ni)
    cols_at[ni] = (ni >> 1) * 128 + wc * 32 + (ni & 1) * 16;
  k_tail<8, 4, TRANS>(a, nk * 64, acc, row0, col0, rows_at, cols_at);
  finish_tile<8, 4, TRANS>(a, acc, row0, col0, rows_at, cols_at);
}

template <bool TRANS>
__global__ void __launch_bounds__(512) big_tile_kernel(TileArgs a) {
  big_tile_body<TRANS>(a);
}

// ------------------------------------------------------------------ lists ----

struct ListArgs {
  uint64_t seq_, atab_, btab_, order_, span_;
  uint32_t n, max_loras;
};

// One wave per slot: its rows in ascending order at order[span[2s]] ..,
// span[2s+1] of them.  A slot's rows begin behind those of the slots below
// it, which the wave counts itself (no wave waits for another).
__global__ void __launch_bounds__(64) lists_kernel(ListArgs a) {
  const int s = blockIdx.x, lane = threadIdx.x;
  const RLD_GLOBAL int32_t* seq = gp<const int32_t>(a.seq_);
  uint32_t below = 0, cnt = 0;
  for (uint32_t r0 = 0; r0 < a.n; r0 += 64) {
    const int key = r0 + lane < a.n ? seq[r0 + lane] : -1;
    below += __popcll(__ballot(key >= 0 && key < s));
  }
  if (gp<const uint64_t>(a.atab_)[s] != 0ull && gp<const uint64_t>(a.btab_)[s] != 0ull) {
    RLD_GLOBAL int32_t* order = gp<int32_t>(a.order_);
    for (uint32_t r0 = 0; r0 < a.n; r0 += 64) {
      const bool hit = r0 + lane < a.n && seq[r0 + lane] == s;
      const uint64_t m = __ballot(hit);
      if (hit) order[below + cnt + __popcll(m & lanemask_lt(lane))] = (int)(r0 + lane);
      cnt += __popcll(m);
    }
  }
  if (lane == 0) {
    gp<uint32_t>(a.span_)[2 * s] = below;
    gp<uint32_t>(a.span_)[2 * s + 1] = cnt;
  }
}

// ------------------------------------------------------------------ wgrad ----

struct WgradArgs {
  uint64_t v_, low_, order_, span_, dtab_;
  uint32_t vs, width, R, tiles, accumulate;
};

// Slot s, 64 columns of the wide operand (x for dA, dy for dB): the sum over
// the slot's rows of low[row][r] * wide[row][col].  Each of four waves takes
// every fourth 32-row group, staged in LDS of its own (no barrier in the
// loop) and read transposed; the waves' sums meet in LDS at the end.
// DB: the result is [col][R] instead of [R][col].
template <int RT, bool DB>
__global__ void __launch_bounds__(256) wgrad_kernel(WgradArgs a) {
  __shared__ __attribute__((aligned(1024))) unsigned char stage[4][4096];
  __shared__ floatx4 red[4][4][kWave];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, c = lane & 15;
  const int s = blockIdx.x / a.tiles;
  const uint32_t col0 = blockIdx.x % a.tiles * 64;
  const uint64_t dst = gp<const uint64_t>(a.dtab_)[s];
  if (dst == 0ull) return;
  const uint32_t begin = gp<const uint32_t>(a.span_)[2 * s];
  const uint32_t cnt = gp<const uint32_t>(a.span_)[2 * s + 1];
  const RLD_GLOBAL int32_t* order = gp<const int32_t>(a.order_) + begin;
  const RLD_GLOBAL float* low = gp<const float>(a.low_);

  floatx4 acc[RT][4];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int ni = 0; ni < 4; ++ni) acc[rt][ni] = floatx4{0.f, 0.f, 0.f, 0.f};

  for (uint32_t i0 = wave * 32; i0 < cnt; i0 += 128) {
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const uint32_t k = p * 8 + (lane >> 3);
      const uint32_t h = ((k >> 1) & 1) | ((k >> 3) & 1) << 1;
      const uint32_t col = col0 + ((((lane & 7) >> 1) ^ h) * 2 + (lane & 1)) * 8;
      const bool in = i0 + k < cnt && col < a.width;
      const uint64_t src =
          a.v_ + ((uint64_t)(in ? order[i0 + k] : 0) * a.vs + (in ? col : 0)) * 2;
      __builtin_amdgcn_global_load_lds((const void*)(in ? src : (uint64_t)&g_zero16[0]),
                                       (RLD_LDS void*)(&stage[wave][p * 1024]), 16, 0, 0);
    }
    uint32_t row[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t i = i0 + 8 * g + e;
      row[e] = i < cnt ? (uint32_t)order[i] : 0xffffffffu;
    }
    uint4 lf[RT][3];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const uint32_t r = rt * 16 + c;
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e)
        v[e] = (row[e] != 0xffffffffu && r < a.R) ? low[(size_t)row[e] * a.R + r] : 0.f;
      bf16_parts<3>(v, lf[rt]);
    }
    wait_vm<0>();
#pragma unroll
    for (int ni = 0; ni < 4; ++ni) {
      const int h = ((c >> 3) & 1) | (g & 1) << 1;
      const unsigned char* p =
          &stage[wave][(8 * g + (c >> 2)) * 128 + (ni ^ h) * 32 + (c & 3) * 8];
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((RLD_LDS s16x4*)p);
      // rows 4 further on: (k >> 1) & 1 and (k >> 3) & 1 are the same
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((RLD_LDS s16x4*)(p + 4 * 128));
      const uint2 l2 = __builtin_bit_cast(uint2, lo), h2 = __builtin_bit_cast(uint2, hi);
      const uint4 vf = make_uint4(l2.x, l2.y, h2.x, h2.y);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int p3 = 2; p3 >= 0; --p3)
          acc[rt][ni] = DB ? mfma_bf16_16x16x32(lf[rt][p3], vf, acc[rt][ni])
                           : mfma_bf16_16x16x32(vf, lf[rt][p3], acc[rt][ni]);
    }
    // the next group's loads overwrite what the reads above still fetch
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }

#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    __syncthreads();
#pragma unroll
    for (int ni = 0; ni < 4; ++ni) red[wave][ni][lane] = acc[rt][ni];
    __syncthreads();
    floatx4 sum = red[0][wave][lane];
#pragma unroll
    for (int v = 1; v < 4; ++v) sum += red[v][wave][lane];
    // first operand: index 4g + i, four consecutive per lane; second: index c
    const uint32_t col = col0 + wave * 16 + (DB ? c : 4 * g);
    const uint32_t r = rt * 16 + (DB ? 4 * g : c);
    if (col < a.width && r < a.R) {
      const uint64_t at = DB ? (uint64_t)col * a.R + r : (uint64_t)r * a.width + col;
      RLD_GLOBAL floatx4* p = gp<floatx4>(dst + at * 4);
      *p = a.accumulate ? *p + sum : sum;
    }
  }
}

// ------------------------------------------------------------------- host ----

static inline size_t round16(size_t v) { return (v + 15) & ~(size_t)15; }

struct LowPlan {
  uint32_t nch;
  size_t low, partial;  // bytes
};

static LowPlan low_plan(uint32_t n, uint32_t K, uint32_t R) {
  LowPlan p;
  p.nch = div_ceil(K, kLowChunk);
  p.low = (size_t)n * R * 4;
  p.partial = p.nch == 1 ? 0 : (size_t)p.nch * n * R * 4;
  return p;
}

static int launch_low(const rld_route* r, bool trans, const void* x, uint32_t xs,
                      const int32_t* seq, uint32_t n, uint64_t low, uint64_t parts,
                      uint64_t partial, hipStream_t st) {
  LowArgs a;
  a.x_ = (uint64_t)x;
  a.seq_ = (uint64_t)seq;
  a.mtab_ = (uint64_t)(trans ? r->b_table : r->a_table);
  a.otab_ = (uint64_t)(trans ? r->a_table : r->b_table);
  a.stab_ = (uint64_t)r->scale_table;
  a.low_ = low;
  a.parts_ = parts;
  a.partial_ = partial;
  a.xs = xs;
  a.n = n;
  a.max_loras = r->max_loras;
  a.K = trans ? r->n_out : r->k_in;
  a.R = r->max_rank;
  a.nch = div_ceil(a.K, kLowChunk);
  const uint32_t items = div_ceil(n, kLowRows) * a.nch;
  // few items: the slots of a tile go to several blocks
  a.nz = items >= 1024u ? 1u : div_ceil(1024u, items);
  if (a.nz > r->max_loras) a.nz = r->max_loras;
  if (a.nz > n) a.nz = n;
  if (a.nz > kLowRows) a.nz = kLowRows;
  if (trans) low_kernel<true><<<items * a.nz, 256, 0, st>>>(a);
  else low_kernel<false><<<items * a.nz, 256, 0, st>>>(a);
  const int e = launch_status();
  if (e || a.nch == 1) return e;
  const uint64_t thr = (uint64_t)n * (a.R / 4);
  low_reduce_kernel<<<(uint32_t)((thr + 255) / 256), 256, 0, st>>>(a);
  return launch_status();
}

template <bool TRANS>
static int launch_tiles(const rld_route* r, const void* w, uint32_t ws, const void* x,
                        uint32_t xs, const int32_t* seq, uint32_t n, uint64_t parts, void* out,
                        uint32_t os, hipStream_t st) {
  TileArgs a;
  a.x_ = (uint64_t)x;
  a.w_ = (uint64_t)w;
  a.out_ = (uint64_t)out;
  a.seq_ = (uint64_t)seq;
  a.parts_ = parts;
  a.etab_ = (uint64_t)(TRANS ? r->a_table : r->b_table);
  a.otab_ = (uint64_t)(TRANS ? r->b_table : r->a_table);
  a.xs = xs;
  a.ws = ws;
  a.os = os;
  a.n = n;
  a.K = TRANS ? r->n_out : r->k_in;
  a.N = TRANS ? r->k_in : r->n_out;
  a.R = r->max_rank;
  a.max_loras = r->max_loras;
  const uint32_t big = div_ceil(n, 256) * div_ceil(a.N, 256);
  if (big >= kBigTiles) {
    a.tiles_m = div_ceil(n, 256);
    a.tiles_n = div_ceil(a.N, 256);
    big_tile_kernel<TRANS><<<xcd_grid(big), 512, 0, st>>>(a);
  } else if (n > 128) {
    a.tiles_m = div_ceil(n, 128);
    a.tiles_n = div_ceil(a.N, 128);
    tile_kernel<128, 128, 2, 2, 2, TRANS><<<a.tiles_m * a.tiles_n, 256, 0, st>>>(a);
  } else {
    a.tiles_m = div_ceil(n, 64);
    a.tiles_n = div_ceil(a.N, 64);
    tile_kernel<64, 64, 2, 2, 4, TRANS><<<a.tiles_m * a.tiles_n, 256, 0, st>>>(a);
  }
  return launch_status();
}

template <bool DB>
static int launch_wgrad(const rld_route* r, const void* v, uint32_t vs, uint64_t low,
                        uint64_t order, uint64_t span, const uint64_t* dtab, int accumulate,
                        hipStream_t st) {
  WgradArgs a;
  a.v_ = (uint64_t)v;
  a.low_ = low;
  a.order_ = order;
  a.span_ = span;
  a.dtab_ = (uint64_t)dtab;
  a.vs = vs;
  a.width = DB ? r->n_out : r->k_in;
  a.R = r->max_rank;
  a.tiles = div_ceil(a.width, 64);
  a.accumulate = accumulate ? 1u : 0u;
  const uint32_t grid = a.tiles * r->max_loras;
  if (a.R <= 16) wgrad_kernel<1, DB><<<grid, 256, 0, st>>>(a);
  else if (a.R <= 32) wgrad_kernel<2, DB><<<grid, 256, 0, st>>>(a);
  else if (a.R <= 64) wgrad_kernel<4, DB><<<grid, 256, 0, st>>>(a);
  else wgrad_kernel<8, DB><<<grid, 256, 0, st>>>(a);
  return launch_status();
}

static int check_wide(uint32_t stride) { return stride > kMaxStride ? RLD_EUNSUPPORTED : RLD_OK; }

// A grid holds fewer than 2^32 threads of at most 256 a block.
static int check_items(const rld_route* r, uint32_t n) {
  const uint64_t k = r->k_in > r->n_out ? r->k_in : r->n_out;
  const uint64_t tiles = (k + 63) / 64;
  if (k > (1u << 24) || div_ceil(n, 64) * tiles >= (1u << 23) ||
      r->max_loras * tiles >= (1u << 23) || (uint64_t)n * (r->max_rank / 4) >= (1u << 31))
    return RLD_EUNSUPPORTED;
  return RLD_OK;
}

}  // namespace rld

using namespace rld;

extern "C" size_t rld_proj_workspace_bytes(uint32_t n, uint32_t k_in, uint32_t max_rank) {
  if (n == 0 || k_in == 0 || max_rank == 0) return 0;
  const LowPlan p = low_plan(n, k_in, max_rank);
  return round16(p.low) + p.partial;
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
  if (workspace_bytes < rld_proj_workspace_bytes(n, route->k_in, route->max_rank))
    return RLD_ENOSPACE;
  const LowPlan p = low_plan(n, route->k_in, route->max_rank);
  const uint64_t low = (uint64_t)workspace;
  const hipStream_t st = (hipStream_t)stream;
  e = launch_low(route, false, x, x_row_stride, seq_slot, n, 0, low, low + round16(p.low), st);
  if (e) return e;
  return launch_tiles<false>(route, w, w_row_stride, x, x_row_stride, seq_slot, n, low, out,
                             out_row_stride, st);
}

extern "C" size_t rld_proj_grad_workspace_bytes(uint32_t n, uint32_t k_in, uint32_t n_out,
                                                uint32_t max_rank, uint32_t max_loras) {
  if (k_in == 0 || n_out == 0 || max_rank == 0 || max_loras == 0) return 0;
  const LowPlan u = low_plan(n, k_in, max_rank), g = low_plan(n, n_out, max_rank);
  return round16(u.low) + u.partial + 2 * round16(g.low) + g.partial + round16((size_t)n * 4) +
         round16((size_t)max_loras * 8);
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
  if (workspace_bytes < rld_proj_grad_workspace_bytes(n, route->k_in, route->n_out,
                                                      route->max_rank, route->max_loras))
    return RLD_ENOSPACE;
  const LowPlan pu = low_plan(n, route->k_in, route->max_rank);
  const LowPlan pg = low_plan(n, route->n_out, route->max_rank);
  const uint64_t u = (uint64_t)workspace;
  const uint64_t up = u + round16(pu.low);
  const uint64_t gl = up + pu.partial;
  const uint64_t gparts = gl + round16(pg.low);
  const uint64_t gpart = gparts + round16(pg.low);
  const uint64_t order = gpart + pg.partial;
  const uint64_t span = order + round16((size_t)n * 4);
  const hipStream_t st = (hipStream_t)stream;
  if (n != 0) {
    if (db_table && (e = launch_low(route, false, x, x_row_stride, seq_slot, n, u, 0, up, st)))
      return e;
    if ((dx || da_table) &&
        (e = launch_low(route, true, dy, dy_row_stride, seq_slot, n, da_table ? gl : 0,
                        dx ? gparts : 0, gpart, st)))
      return e;
    if (dx && (e = launch_tiles<true>(route, w, w_row_stride, dy, dy_row_stride, seq_slot, n,
                                      gparts, dx, dx_row_stride, st)))
      return e;
  }
  if (!adapters) return RLD_OK;
  ListArgs l;
  l.seq_ = (uint64_t)seq_slot;
  l.atab_ = (uint64_t)route->a_table;
  l.btab_ = (uint64_t)route->b_table;
  l.order_ = order;
  l.span_ = span;
  l.n = n;
  l.max_loras = route->max_loras;
  lists_kernel<<<route->max_loras, 64, 0, st>>>(l);
  if ((e = launch_status())) return e;
  if (da_table && (e = launch_wgrad<false>(route, x, x_row_stride, gl, order, span, da_table,
                                           accumulate, st)))
    return e;
  if (db_table && (e = launch_wgrad<true>(route, dy, dy_row_stride, u, order, span, db_table,
                                          accumulate, st)))
    return e;
  return RLD_OK;
}
