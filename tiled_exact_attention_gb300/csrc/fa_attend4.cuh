// Attention of one or a few query tokens per sequence over a paged 4-bit cache.
//
// Mathematics.  With k = min_k + s_k c (c = 0..15) the score of a key is
//   scale (s_k sum_d q_d c_d + min_k sum_d q_d)     per group of dims, summed,
// so the codes enter the products as they are: an fp16 whose bits are 0x000c is the
// subnormal c 2^-24, and one whose bits are 0x00c0 is 16 c 2^-24, exactly, so a
// 32-bit word of eight codes becomes four operand registers of m16n8k16 MMAs in
// five integer instructions, with no conversion.  The factor 2^-24 goes into the
// score's scale, the factor 16 into Q (exactly: powers of two).  O is likewise
//   sum_j (p_j s_vj) (c_j - 8) + sum_j p_j (min_vj + 8 s_vj),
// the weights p s_v rounded to fp16 for the MMA and 8 times their sum as rounded taken
// off in fp32, so the rounding multiplies only the centred part of V.  Scores, the
// running maximum and sum, and O are fp32.
//
// Layout of the work.  K (keys x dims) and V^T (dims x keys) are the A operands, 16
// rows an MMA; the rows of queries (query tokens x the g query heads that share the
// KV head) are the 8-wide N side, so few query rows waste little.  S^T leaves its MMA
// with keys along lanes / 4 and becomes the B operand of the second product by a
// transposing register move (movmatrix).  Each warp is a stream of its own: lane 0
// copies whole units of the cache (K, V and their parameters are adjacent: one bulk
// copy of some 4-10 KB) into the warp's ring in shared memory, and no barrier joins
// the warps until the end of a (sequence, KV head, row tile).
//
// Split.  The blocks of all items (sequence, KV head, row tile) form one line that is
// cut evenly over the grid, whatever the lengths; they are read on the device, so a
// captured call follows them.  An item that crosses a cut is merged from fp32
// partials by the last of its CTAs to finish.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fa_kv4.h"
#include "ptx.cuh"

namespace fa {
namespace attend4 {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kMinBlocks = kWarps;  // blocks a CTA takes at least: one for each warp
constexpr float kLn2 = 0.69314718055994530942f;

enum : int { kSiteFull = 48 };

template <int D, int NG, int NT>
struct Cfg {
#ifndef A4_UNITS
#define A4_UNITS (D == 64 ? 2 : 1)
#endif
#ifndef A4_STAGES
#define A4_STAGES (D == 256 ? 2 : 3)
#endif
#ifndef A4_CTAS
#define A4_CTAS (SMEM <= 74 * 1024 ? 3 : (SMEM <= 112 * 1024 ? 2 : 1))
#endif
  static constexpr int UNITS = A4_UNITS;  // units per block (a block lies in one page)
  static constexpr int BK = UNITS * kKv4Unit;    // keys per block
  static constexpr int UB = kv4_unit_bytes(D, NG);
  static constexpr int STAGE = UNITS * UB;
  static constexpr int STAGES = A4_STAGES;
  static constexpr int ROWS = 8 * NT;
  static constexpr int OP = D + 4;  // pitch of a row of the merge buffers (floats)
  static constexpr int RING = kWarps * STAGES * STAGE;
  static constexpr int SMEM = RING + ROWS * OP * 4 + kWarps * ROWS * 8 + kWarps * STAGES * 8 + 64;
  static constexpr int CTAS = A4_CTAS;  // per SM
  static constexpr bool ONES = NG <= 2;
};

template <bool BF16>
__device__ __forceinline__ float widen(uint32_t h) {
  if constexpr (BF16) return __uint_as_float(h << 16);
  return __half2float(__ushort_as_half(static_cast<unsigned short>(h)));
}

template <bool BF16>
__device__ __forceinline__ float widen_hi(uint32_t w) {
  if constexpr (BF16) return __uint_as_float(w & 0xffff0000u);
  return __half2float(__ushort_as_half(static_cast<unsigned short>(w >> 16)));
}

__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  const __half2 x = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&x);
}

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// N consecutive 32-bit words of shared memory, N = 1, 2, 4 or 8.
template <int N>
__device__ __forceinline__ void lds_words(const uint8_t* p, uint32_t (&w)[N]) {
  if constexpr (N == 1) {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (N == 2) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    w[0] = u.x;
    w[1] = u.y;
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint4 u = *reinterpret_cast<const uint4*>(p + 16 * i);
      w[4 * i] = u.x;
      w[4 * i + 1] = u.y;
      w[4 * i + 2] = u.z;
      w[4 * i + 3] = u.w;
    }
  }
}

// Keys of a sequence; one that outruns its block-table row has none (and is reported).
__device__ __forceinline__ int seq_len(const Attend4Params& p, int seq) {
  const int n = p.seqlens[seq];
  if (n > p.bt_stride * p.page_size) {
    record_error(p.status, kErrDeviceArg);
    return 0;
  }
  return n > 0 ? n : 0;
}

// Keys [lo, hi) that the rows of a tile see, all in all.
__device__ __forceinline__ void tile_range(const Attend4Params& p, int len, int rows, int tile, int* lo, int* hi) {
  const int r1 = min(p.sq * p.g, (tile + 1) * rows) - 1;
  const int first = len - p.sq + tile * rows / p.g, last = len - p.sq + r1 / p.g;
  *hi = max(last + 1, 0);
  *lo = p.window_left >= 0 ? max(0, first - p.window_left) : 0;
}

// One item: a row tile of one KV head of one sequence, n blocks from blo on (one,
// with nothing in it, where no row sees a key).
template <int BK, int ROWS>
struct Item {
  int seq, kvh, tile, len, lo, hi, blo, n;
  __device__ __forceinline__ void range(const Attend4Params& p) {
    tile_range(p, len, ROWS, tile, &lo, &hi);
    blo = lo / BK;
    n = hi > lo ? (hi + BK - 1) / BK - blo : 1;
  }
  __device__ __forceinline__ void next(const Attend4Params& p) {
    if (++tile == p.ntiles) {
      tile = 0;
      if (++kvh == p.hkv) {
        kvh = 0;
        len = seq_len(p, ++seq);
      }
    }
    range(p);
  }
};

// A CTA's stretch of the line, item by item: blocks [u0, ue) of the current one.
template <int BK, int ROWS>
struct Walk {
  Item<BK, ROWS> it;
  int u0, ue;
  int left;  // blocks of the CTA from u0 on
  __device__ __forceinline__ void enter() { ue = min(it.n, u0 + left); }
  __device__ __forceinline__ bool next(const Attend4Params& p) {  // false: nothing is left
    left -= ue - u0;
    if (left <= 0) return false;
    it.next(p);
    u0 = 0;
    enter();
    return true;
  }
};

// Blocks of one sequence (all its KV heads and tiles).
template <int BK, int ROWS>
__device__ __forceinline__ int64_t seq_blocks(const Attend4Params& p, int seq) {
  Item<BK, ROWS> it;
  it.len = seq_len(p, seq);
  int64_t n = 0;
  for (it.tile = 0; it.tile < p.ntiles; ++it.tile) {
    it.range(p);
    n += it.n;
  }
  return n * p.hkv;
}

template <int D, int NG, bool BF16, int NT>
__global__ void __launch_bounds__(kThreads, Cfg<D, NG, NT>::CTAS) attend4_kernel(const __grid_constant__ Attend4Params p) {
  using C = Cfg<D, NG, NT>;
  constexpr int J = kv4_j(D), NC = D / 32 / J, NW = D / 32, GW = NW / NG;
  constexpr int BK = C::BK, ROWS = C::ROWS;
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t* ring = smem + static_cast<int>(threadIdx.x >> 5) * C::STAGES * C::STAGE;
  float* obuf = reinterpret_cast<float*>(smem + C::RING);                    // [ROWS][OP]
  float2* ml = reinterpret_cast<float2*>(obuf + ROWS * C::OP);           // [kWarps][ROWS]
  uint64_t* full = reinterpret_cast<uint64_t*>(ml + kWarps * ROWS) + (threadIdx.x >> 5) * C::STAGES;
  int64_t* sh = reinterpret_cast<int64_t*>(reinterpret_cast<uint64_t*>(ml + kWarps * ROWS) + kWarps * C::STAGES);
  const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), g = lane >> 2, t = lane & 3;

  if (lane == 0) {
    for (int s = 0; s < C::STAGES; ++s) mbar_init(&full[s], 1);
    fence_mbar_init();
  }
  // ---- the CTA's stretch of the line of blocks: total, then the sequence where it starts
  int64_t total = 0;
  for (int s = threadIdx.x; s < p.b; s += kThreads) total += seq_blocks<BK, ROWS>(p, s);
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) total += __shfl_xor_sync(0xffffffffu, total, x);
  if (lane == 0) sh[warp] = total;
  __syncthreads();
  total = sh[0] + sh[1] + sh[2] + sh[3];
  int64_t share64 = (total + gridDim.x - 1) / gridDim.x;
  if (share64 < kMinBlocks) share64 = kMinBlocks;
  const int share = static_cast<int>(share64);
  const int64_t begin = static_cast<int64_t>(blockIdx.x) * share;
  if (begin >= total) return;
  __syncthreads();
  if (warp == 0) {
    int64_t before = 0;
    for (int s0 = 0; s0 < p.b; s0 += 32) {
      const int64_t n = s0 + lane < p.b ? seq_blocks<BK, ROWS>(p, s0 + lane) : 0;
      int64_t incl = n;
#pragma unroll
      for (int x = 1; x < 32; x <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, incl, x);
        if (lane >= x) incl += y;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, begin < before + incl);
      if (hit != 0) {
        if (lane == __ffs(hit) - 1) {
          sh[4] = s0 + lane;
          sh[5] = begin - (before + incl - n);
        }
        break;
      }
      before += __shfl_sync(0xffffffffu, incl, 31);
    }
  }
  __syncthreads();
  Walk<BK, ROWS> cw;
  cw.left = static_cast<int>(min(total - begin, static_cast<int64_t>(share)));
  cw.it.seq = static_cast<int>(sh[4]);
  cw.it.len = seq_len(p, cw.it.seq);
  {
    int64_t rem = sh[5];
    const int64_t per_head = seq_blocks<BK, ROWS>(p, cw.it.seq) / p.hkv;
    cw.it.kvh = static_cast<int>(rem / per_head);
    rem %= per_head;
    cw.it.tile = 0;
    cw.it.range(p);
    while (rem >= cw.it.n) {
      rem -= cw.it.n;
      ++cw.it.tile;
      cw.it.range(p);
    }
    cw.u0 = static_cast<int>(rem);
    cw.enter();
  }
  const int64_t item0 = begin - cw.u0;  // where the first item starts on the line

  // ---- the warp's stream of blocks: `pw` runs ahead of the consumer
  Walk<BK, ROWS> pw = cw;
  int pu = pw.u0 + warp, prow = 0;  // the next block, and its row in its page
  const int* ptable = nullptr;      // ... whose table entry this is
  const uint8_t* src = nullptr;     // the next block to copy (null: none)
  auto place = [&]() {
    const int key = (pw.it.blo + pu) * BK, page = key / p.page_size;
    prow = key - page * p.page_size;
    ptable = p.block_table + pw.it.seq * p.bt_stride + page;
  };
  auto seek = [&](bool fresh) {
    bool more = true;
    while (more && (pu >= pw.ue || pw.it.hi <= pw.it.lo)) {
      more = pw.next(p);
      pu = pw.u0 + warp;
      fresh = true;
    }
    src = nullptr;
    if (more) {
      if (fresh) place();
      int page = *ptable;
      if (page < 0 || page >= p.num_pages) {
        record_error(p.status, kErrDeviceArg);
        page = 0;
      }
      src = p.cache + page * p.c_st[0] + pw.it.kvh * p.c_st[1] + (prow / kKv4Unit) * C::UB;
      pu += kWarps;
      prow += kWarps * BK;
      while (prow >= p.page_size) {
        prow -= p.page_size;
        ++ptable;
      }
    }
  };
  auto issue = [&](int slot) {
    if (src != nullptr) {
      if (lane == 0) {
        mbar_arrive_expect_tx(&full[slot], C::STAGE);
        bulk_load(ring + slot * C::STAGE, src, C::STAGE, &full[slot]);
      }
      seek(false);
    }
  };
  seek(true);
#pragma unroll
  for (int s = 0; s < C::STAGES; ++s) issue(s);
  int slot = 0;
  uint32_t phase = 0;

  int64_t item_at = item0;
  for (bool live = true; live;) {
    const auto& it = cw.it;
    const int R = p.sq * p.g;
    // ---- Q of the tile's rows as B operands; its row scales and group sums
    uint32_t qf[NW][2][NT][2];
    float qs[NG][NT][2], rs[NT][2], m[NT][2], l[NT][2], tv[NG][NT][2], o[NW][2][NT][4], ones[C::ONES ? NG : 1][NT][4];
    float cap_rs[NT][2];
    int row_hi[NT][2], row_lo[NT][2];
    const bool capped = p.sc_b > 0.f;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = it.tile * ROWS + nt * 8 + g;
      uint4 u[NW];
#pragma unroll
      for (int j = 0; j < NW; ++j) {
        u[j] = make_uint4(0u, 0u, 0u, 0u);
        if (r < R)
          u[j] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + it.seq * p.q_st[0] +
                                                 (r / p.g) * p.q_st[1] + (it.kvh * p.g + r % p.g) * p.q_st[2] +
                                                 32 * j + 8 * t);
      }
      // the row is scaled by a power of two so that its largest value lies in [2^14, 2^15)
      float top = 0.f;
#pragma unroll
      for (int j = 0; j < NW; ++j) {
        const uint32_t w[4] = {u[j].x, u[j].y, u[j].z, u[j].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) top = fmaxf(top, fmaxf(fabsf(widen<BF16>(w[e] & 0xffffu)), fabsf(widen_hi<BF16>(w[e]))));
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const uint32_t ex = max(__float_as_uint(top) >> 23, 15u);
      const float up = __uint_as_float((268u - ex) << 23), down = __uint_as_float((ex - 14u) << 23);  // 1 / up
      float sum[NG];
#pragma unroll
      for (int j = 0; j < NW; ++j) {
        const uint32_t w[4] = {u[j].x, u[j].y, u[j].z, u[j].w};
        float x[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[2 * e] = widen<BF16>(w[e] & 0xffffu) * up;
          x[2 * e + 1] = widen_hi<BF16>(w[e]) * up;
        }
        const float s8 = ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
        sum[j / GW] = j % GW == 0 ? s8 : sum[j / GW] + s8;
        qf[j][0][nt][0] = pack_f16(x[0], x[4]);
        qf[j][0][nt][1] = pack_f16(x[2], x[6]);
        qf[j][1][nt][0] = pack_f16(x[1] * 0.0625f, x[5] * 0.0625f);
        qf[j][1][nt][1] = pack_f16(x[3] * 0.0625f, x[7] * 0.0625f);
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int from = 4 * (2 * t + c);
        const float scale = __shfl_sync(0xffffffffu, down, from) * 0x1p24f * p.scale_log2;
        cap_rs[nt][c] = scale;
        rs[nt][c] = capped ? 1.f : scale;
        const int rc = it.tile * ROWS + nt * 8 + 2 * t + c, pos = it.len - p.sq + rc / p.g;
        row_hi[nt][c] = rc < R ? pos : -1;
        row_lo[nt][c] = p.window_left >= 0 ? pos - p.window_left : 0;
        m[nt][c] = -INFINITY;
        l[nt][c] = 0.f;
      }
#pragma unroll
      for (int q = 0; q < NG; ++q) {
        sum[q] += __shfl_xor_sync(0xffffffffu, sum[q], 1);
        sum[q] += __shfl_xor_sync(0xffffffffu, sum[q], 2);
        sum[q] *= 0x1p-24f;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          qs[q][nt][c] = __shfl_sync(0xffffffffu, sum[q], 4 * (2 * t + c));
          tv[q][nt][c] = 0.f;
        }
        if (C::ONES) {
#pragma unroll
          for (int e = 0; e < 4; ++e) ones[q][nt][e] = 0.f;
        }
      }
#pragma unroll
      for (int j = 0; j < NW; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[j][0][nt][e] = o[j][1][nt][e] = 0.f;
    }
    // keys that every row of the tile sees: no mask there
    const int all_hi = it.len - p.sq + it.tile * ROWS / p.g;
    const int all_lo = p.window_left >= 0
                           ? max(0, it.len - p.sq + (min(R, (it.tile + 1) * ROWS) - 1) / p.g - p.window_left) : 0;
    float vscale = 0.f;  // V's weights are held times this power of two (0: not chosen yet)

    if (it.hi > it.lo)
      for (int u = cw.u0 + warp; u < cw.ue; u += kWarps) {
        mbar_wait(&full[slot], phase, p.status, kSiteFull);
        const uint8_t* st = ring + slot * C::STAGE;
        const int key0 = (it.blo + u) * BK;
        const bool edge = key0 + BK - 1 > all_hi || key0 < all_lo;
        // ---- scores
        float s[2 * C::UNITS][NT][4];
#pragma unroll
        for (int mt = 0; mt < 2 * C::UNITS; ++mt) {
          const uint8_t* unit = st + (mt / 2) * C::UB;
          const int r = 16 * (mt % 2) + g;
          uint32_t pa[NG], pb[NG];
          lds_words<NG>(unit + 32 * D + r * NG * 4, pa);
          lds_words<NG>(unit + 32 * D + (r + 8) * NG * 4, pb);
          float acc[NT][4];
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            uint32_t wa[J], wb[J];
            lds_words<J>(unit + ((32 * c + r) * 4 + t) * J * 4, wa);
            lds_words<J>(unit + ((32 * c + r + 8) * 4 + t) * J * 4, wb);
#pragma unroll
            for (int j = 0; j < J; ++j) {
              const int w = c * J + j;
              if (w % GW == 0) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                  for (int e = 0; e < 4; ++e) acc[nt][e] = 0.f;
              }
              const uint32_t ha = wa[j] >> 8, hb = wb[j] >> 8;
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                mma16816(acc[nt], wa[j] & 0x000f000fu, wb[j] & 0x000f000fu, ha & 0x000f000fu, hb & 0x000f000fu,
                         qf[w][0][nt][0], qf[w][0][nt][1]);
                mma16816(acc[nt], wa[j] & 0x00f000f0u, wb[j] & 0x00f000f0u, ha & 0x00f000f0u, hb & 0x00f000f0u,
                         qf[w][1][nt][0], qf[w][1][nt][1]);
              }
              if (w % GW == GW - 1) {
                const int q = w / GW;
                const float sa = widen<BF16>(pa[q] & 0xffffu), na = widen_hi<BF16>(pa[q]);
                const float sb = widen<BF16>(pb[q] & 0xffffu), nb = widen_hi<BF16>(pb[q]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                  for (int e = 0; e < 4; ++e) {
                    const float prod = (e < 2 ? na : nb) * qs[q][nt][e & 1];
                    const float rest = q == 0 ? prod : s[mt][nt][e] + prod;
                    s[mt][nt][e] = fmaf(e < 2 ? sa : sb, acc[nt][e], rest);
                  }
              }
            }
          }
        }
        if (capped) {  // (from here on the scores are final: rs is 1)
#pragma unroll
          for (int mt = 0; mt < 2 * C::UNITS; ++mt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                s[mt][nt][e] = p.sc_b * tanh_from_exp2_arg(p.sc_k * (s[mt][nt][e] * cap_rs[nt][e & 1]));
        }
        if (edge) {
#pragma unroll
          for (int mt = 0; mt < 2 * C::UNITS; ++mt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int key = key0 + 16 * mt + g + 8 * (e >> 1);
                if (key > row_hi[nt][e & 1] || key < row_lo[nt][e & 1]) s[mt][nt][e] = -INFINITY;
              }
        }
        // ---- running maximum; O, l and the rest follow it when it grows
        bool grown = false;
        float mn[NT][2], ref[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float x = fmaxf(s[0][nt][c], s[0][nt][c + 2]);
#pragma unroll
            for (int mt = 1; mt < 2 * C::UNITS; ++mt) x = fmaxf(x, fmaxf(s[mt][nt][c], s[mt][nt][c + 2]));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
            mn[nt][c] = fmaxf(m[nt][c], x * rs[nt][c]);
            grown = grown || mn[nt][c] > m[nt][c];
          }
        if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const float a = m[nt][c] == -INFINITY ? 0.f : ex2_approx(m[nt][c] - mn[nt][c]);
              m[nt][c] = mn[nt][c];
              l[nt][c] *= a;
#pragma unroll
              for (int q = 0; q < NG; ++q) {
                tv[q][nt][c] *= a;
                if (C::ONES) ones[q][nt][c] *= a;
              }
#pragma unroll
              for (int j = 0; j < NW; ++j) {
                o[j][0][nt][c] *= a;
                o[j][0][nt][c + 2] *= a;
                o[j][1][nt][c] *= a;
                o[j][1][nt][c + 2] *= a;
              }
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) ref[nt][c] = m[nt][c] == -INFINITY ? 0.f : m[nt][c];
        // ---- V's weights stay in fp16's normal range: times a power of two that puts the
        // first block's largest scale at 2^7..2^8 and is lowered when one passes 2^15
        {
          float top = 0.f;
#pragma unroll
          for (int un = 0; un < C::UNITS; ++un) {
            uint32_t w[NG];
            lds_words<NG>(st + un * C::UB + 32 * D + 128 * NG + lane * NG * 4, w);
            const int key = key0 + 32 * un + lane;
            if (key >= it.lo && key < it.hi) {
#pragma unroll
              for (int q = 0; q < NG; ++q) top = fmaxf(top, widen<BF16>(w[q] & 0xffffu));
            }
          }
          top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
          if (top > 0.f && (vscale == 0.f || top * vscale > 0x1p15f)) {
            const float now = __uint_as_float((261u - (__float_as_uint(top) >> 23)) << 23);
            if (vscale > 0.f) {
              const float a = now / vscale;
              if (C::ONES) {
#pragma unroll
                for (int q = 0; q < NG; ++q)
#pragma unroll
                  for (int nt = 0; nt < NT; ++nt) {
                    ones[q][nt][0] *= a;
                    ones[q][nt][1] *= a;
                  }
              }
#pragma unroll
              for (int j = 0; j < NW; ++j)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                  for (int e = 0; e < 4; ++e) {
                    o[j][0][nt][e] *= a;
                    o[j][1][nt][e] *= a;
                  }
            }
            vscale = now;
          }
        }
        const float off8 = vscale > 0.f ? -8.f / vscale : 0.f;
        // ---- probabilities and O
#pragma unroll
        for (int mt = 0; mt < 2 * C::UNITS; ++mt) {
          const uint8_t* unit = st + (mt / 2) * C::UB;
          const int r = 16 * (mt % 2) + g;
          uint32_t pa[NG], pb[NG];
          lds_words<NG>(unit + 32 * D + 128 * NG + r * NG * 4, pa);
          lds_words<NG>(unit + 32 * D + 128 * NG + (r + 8) * NG * 4, pb);
          if (edge) {
            const int key = key0 + 16 * mt + g;
#pragma unroll
            for (int q = 0; q < NG; ++q) {
              if (key < it.lo || key >= it.hi) pa[q] = 0;
              if (key + 8 < it.lo || key + 8 >= it.hi) pb[q] = 0;
            }
          }
          float pr[NT][4];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              pr[nt][e] = ex2_approx(fmaf(s[mt][nt][e], rs[nt][e & 1], -ref[nt][e & 1]));
              l[nt][e & 1] += pr[nt][e];
            }
          uint32_t bw[NG][NT][2];
#pragma unroll
          for (int q = 0; q < NG; ++q) {
            const float sa = widen<BF16>(pa[q] & 0xffffu), na = fmaf(8.f, sa, widen_hi<BF16>(pa[q]));
            const float sb = widen<BF16>(pb[q] & 0xffffu), nb = fmaf(8.f, sb, widen_hi<BF16>(pb[q]));
            const float va = sa * vscale, vb = sb * vscale;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const uint32_t ha = pack_f16(pr[nt][0] * va, pr[nt][1] * va);
              const uint32_t hb = pack_f16(pr[nt][2] * vb, pr[nt][3] * vb);
              tv[q][nt][0] = fmaf(pr[nt][0], na, fmaf(pr[nt][2], nb, tv[q][nt][0]));
              tv[q][nt][1] = fmaf(pr[nt][1], na, fmaf(pr[nt][3], nb, tv[q][nt][1]));
              if (!C::ONES) {
                const float2 fa = __half22float2(*reinterpret_cast<const __half2*>(&ha));
                const float2 fb = __half22float2(*reinterpret_cast<const __half2*>(&hb));
                tv[q][nt][0] = fmaf(fa.x + fb.x, off8, tv[q][nt][0]);
                tv[q][nt][1] = fmaf(fa.y + fb.y, off8, tv[q][nt][1]);
              }
              bw[q][nt][0] = transpose8(ha);
              bw[q][nt][1] = transpose8(hb);
              if (C::ONES)  // the sum of the weights as rounded, in units of 2^-24
                mma16816(ones[q][nt], 0x00010001u, 0u, 0x00010001u, 0u, bw[q][nt][0], bw[q][nt][1]);
            }
          }
          const uint8_t* vu = unit + 16 * D;
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            uint32_t wa[J], wb[J];
            lds_words<J>(vu + (((2 * (mt % 2) * NC + c) * 8 + g) * 4 + t) * J * 4, wa);
            lds_words<J>(vu + ((((2 * (mt % 2) + 1) * NC + c) * 8 + g) * 4 + t) * J * 4, wb);
#pragma unroll
            for (int j = 0; j < J; ++j) {
              const int w = c * J + j, q = w / GW;
              const uint32_t ha = wa[j] >> 8, hb = wb[j] >> 8;
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                mma16816(o[w][0][nt], wa[j] & 0x000f000fu, wa[j] & 0x00f000f0u, wb[j] & 0x000f000fu,
                         wb[j] & 0x00f000f0u, bw[q][nt][0], bw[q][nt][1]);
                mma16816(o[w][1][nt], ha & 0x000f000fu, ha & 0x00f000f0u, hb & 0x000f000fu, hb & 0x00f000f0u,
                         bw[q][nt][0], bw[q][nt][1]);
              }
            }
          }
        }
        __syncwarp();  // every lane has read the stage
        issue(slot);
        if (++slot == C::STAGES) {
          slot = 0;
          phase ^= 1u;
        }
      }

    // ---- the warps' shares of the segment: common maximum, then O warp by warp into one buffer
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) {
          l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], x);
#pragma unroll
          for (int q = 0; q < NG; ++q) tv[q][nt][c] += __shfl_xor_sync(0xffffffffu, tv[q][nt][c], x);
        }
    if (g == 0) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) ml[warp * ROWS + nt * 8 + 2 * t + c] = make_float2(m[nt][c], l[nt][c]);
    }
    __syncthreads();
    const float unscale = vscale > 0.f ? 0x1p24f / vscale : 0.f;
#pragma unroll 1
    for (int turn = 0; turn < kWarps; ++turn) {
      if (warp == turn) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int r = nt * 8 + 2 * t + c;
            float M = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, ml[w * ROWS + r].x);
            const float a = m[nt][c] == -INFINITY ? 0.f : ex2_approx(m[nt][c] - M), au = a * unscale;
#pragma unroll
            for (int j = 0; j < NW; ++j) {
              float add = a * tv[j / GW][nt][c];
              if (C::ONES) add = fmaf(ones[j / GW][nt][c], -8.f * au, add);
              float4 x = make_float4(fmaf(o[j][0][nt][c], au, add), fmaf(o[j][0][nt][c + 2], au * 0.0625f, add),
                                     fmaf(o[j][1][nt][c], au, add), fmaf(o[j][1][nt][c + 2], au * 0.0625f, add));
              float4* dst = reinterpret_cast<float4*>(obuf + r * C::OP + 32 * j + 4 * g);
              if (turn > 0) {
                const float4 y = *dst;
                x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
              }
              *dst = x;
            }
          }
      }
      __syncthreads();
    }

    // ---- out: the whole item, or a partial of it
    const int64_t c0 = item_at / share, c1 = (item_at + it.n - 1) / share;  // the CTAs that hold the item
    const bool whole = c0 == c1;
    const int64_t cta = blockIdx.x;
    const int my = static_cast<int>(2 * cta + (cta == c0 && item_at > c0 * share ? 1 : 0));
    constexpr int PER = D / 4;  // float4 of a row
    bool merge = false;
    if (!whole) {
      for (int x = threadIdx.x; x < ROWS * PER; x += kThreads) {
        const int r = x / PER, e = x % PER;
        reinterpret_cast<float4*>(p.part_o)[(static_cast<int64_t>(my) * ROWS + r) * PER + e] =
            *reinterpret_cast<const float4*>(obuf + r * C::OP + 4 * e);
      }
      if (threadIdx.x < ROWS) {
        float M = -INFINITY, L = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, ml[w * ROWS + threadIdx.x].x);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float2 x = ml[w * ROWS + threadIdx.x];
          if (x.x != -INFINITY) L = fmaf(x.y, ex2_approx(x.x - M), L);
        }
        p.part_ml[static_cast<int64_t>(my) * ROWS + threadIdx.x] = make_float2(M, L);
      }
      __threadfence();
      __syncthreads();
      if (threadIdx.x == 0) sh[0] = atomicAdd(p.counters + c0, 1) == static_cast<int>(c1 - c0);
      __syncthreads();
      merge = sh[0] != 0;
      if (merge) __threadfence();
    }
    if (whole || merge) {
      for (int x = threadIdx.x; x < ROWS * (D / 8); x += kThreads) {
        const int r = x / (D / 8), e = x % (D / 8), row = it.tile * ROWS + r;
        if (row >= R) continue;
        float f[8], M = -INFINITY, L = 0.f;
        if (whole) {
#pragma unroll
          for (int w = 0; w < kWarps; ++w) M = fmaxf(M, ml[w * ROWS + r].x);
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            const float2 y = ml[w * ROWS + r];
            if (y.x != -INFINITY) L = fmaf(y.y, ex2_approx(y.x - M), L);
          }
#pragma unroll
          for (int k = 0; k < 8; ++k) f[k] = obuf[r * C::OP + 8 * e + k];
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k) f[k] = 0.f;
          const int s0 = static_cast<int>(2 * c0 + (item_at > c0 * share ? 1 : 0));
          for (int64_t c = c0; c <= c1; ++c)
            M = fmaxf(M, __ldcg(&p.part_ml[(c == c0 ? s0 : 2 * c) * ROWS + r]).x);
#pragma unroll 4
          for (int64_t c = c0; c <= c1; ++c) {
            const int64_t at = (c == c0 ? s0 : 2 * c) * ROWS + r;
            const float2 y = __ldcg(&p.part_ml[at]);
            const float4 a = __ldcg(reinterpret_cast<const float4*>(p.part_o) + at * PER + 2 * e);
            const float4 b = __ldcg(reinterpret_cast<const float4*>(p.part_o) + at * PER + 2 * e + 1);
            const float w = y.x == -INFINITY ? 0.f : ex2_approx(y.x - M);
            L = fmaf(y.y, w, L);
            f[0] = fmaf(a.x, w, f[0]);
            f[1] = fmaf(a.y, w, f[1]);
            f[2] = fmaf(a.z, w, f[2]);
            f[3] = fmaf(a.w, w, f[3]);
            f[4] = fmaf(b.x, w, f[4]);
            f[5] = fmaf(b.y, w, f[5]);
            f[6] = fmaf(b.z, w, f[6]);
            f[7] = fmaf(b.w, w, f[7]);
          }
        }
        const float inv = L > 0.f ? 1.f / L : 0.f;
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float a = f[2 * k] * inv, b = f[2 * k + 1] * inv;
          if constexpr (BF16) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
            w[k] = *reinterpret_cast<const uint32_t*>(&h);
          } else {
            w[k] = pack_f16(a, b);
          }
        }
        const int qi = row / p.g, h = it.kvh * p.g + row % p.g;
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) + it.seq * p.o_st[0] + qi * p.o_st[1] + h * p.o_st[2] +
                                  8 * e) = make_uint4(w[0], w[1], w[2], w[3]);
        if (e == 0)
          p.lse[(static_cast<int64_t>(it.seq) * p.hq + h) * p.sq + qi] =
              L > 0.f ? (M + lg2_approx(L)) * kLn2 : -INFINITY;
      }
    }
    item_at += it.n;
    live = cw.next(p);
    if (live) __syncthreads();  // the buffers are free again
  }
}

// CTAs of a full grid, and the bytes of its partials.
template <int D, int NG, int NT>
constexpr int ctas_per_sm() {
  return Cfg<D, NG, NT>::CTAS;
}

template <int D, int NG, bool BF16, int NT>
cudaError_t launch_one(const Attend4Params& p, int grid, cudaStream_t stream) {
  using C = Cfg<D, NG, NT>;
  auto* k = attend4_kernel<D, NG, BF16, NT>;
  static_assert(C::SMEM <= 227 * 1024, "shared memory");
  const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  k<<<grid, kThreads, C::SMEM, stream>>>(p);
  return cudaGetLastError();
}

template <int D, int NG, int NT>
cudaError_t launch_dtype(const Attend4Params& p, int dtype, int sms, Attend4Plan* plan, cudaStream_t stream) {
  using C = Cfg<D, NG, NT>;
  if (plan != nullptr) {
    plan->rows = C::ROWS;
    plan->block = C::BK;
    plan->max_ctas = sms * C::CTAS;
    return cudaSuccess;
  }
  return dtype == 0 ? launch_one<D, NG, true, NT>(p, p.grid, stream) : launch_one<D, NG, false, NT>(p, p.grid, stream);
}

// Up to eight query rows of a KV head per pass, or sixteen.
template <int D, int NG>
cudaError_t launch_rows(const Attend4Params& p, int dtype, int sms, Attend4Plan* plan, cudaStream_t stream) {
  return p.sq * p.g <= 8 ? launch_dtype<D, NG, 1>(p, dtype, sms, plan, stream)
                         : launch_dtype<D, NG, 2>(p, dtype, sms, plan, stream);
}

}  // namespace attend4
}  // namespace fa
