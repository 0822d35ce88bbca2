// Attention of one or a few query tokens per sequence over a paged 4-bit cache.
//
// Mathematics.  With k = min_k + s_k c (c = 0..15) the score of a key is
//   scale (s_k sum_d q_d c_d + min_k sum_d q_d)     per group of dims, summed,
// so the codes enter the products as they are: an fp16 whose bits are 0x000c is the
// subnormal c 2^-24, and one whose bits are 0x00c0 is 16 c 2^-24, exactly, so a
// 32-bit word of eight codes becomes four operand registers of m16n8k16 MMAs in
// five integer instructions, with no conversion.  The factor 2^-24 goes into the
// score's scale, the factor 16 into Q (exactly: powers of two) or, for V, whose factor
// is a row's, into O at the end.  O is likewise
//   sum_j (p_j s_vj) (c_j - 8) + sum_j p_j (min_vj + 8 s_vj),
// the weights p s_v rounded to fp16 for the MMA, so the rounding multiplies only the
// centred part of V; the 8 is taken off in fp32 at the end.  (The ones that sum the
// weights are the fp16 1.0: products of the subnormal 2^-24 lose their low bits in the
// tensor core when larger ones stand beside them, which cost 3.3e-3 of O at 32768 keys.)
// Scores, the running maximum and sum, and O are fp32.
//
// Layout of the work.  K (keys x dims) and V^T (dims x keys) are the A operands, 16
// rows an MMA; the rows of queries (query tokens x the g query heads that share the
// KV head) are the 8-wide N side, so few query rows waste little.  S^T leaves its MMA
// with keys along lanes / 4 and becomes the B operand of the second product by a
// transposing register move (movmatrix).  Each warp is a stream of its own: whole units
// of the cache (K, V and their parameters are adjacent: one bulk copy of 5-10 KB) go to
// the warp's ring in shared memory, each copied by the lane that looked its page up, and
// no barrier joins the warps until the end of a (sequence, KV head, row tile).
//
// Split.  The blocks of all items (sequence, KV head, row tile) form one line that is
// cut evenly over the grid, whatever the lengths; they are read on the device, so a
// captured call follows them.  An item that crosses a cut is merged from fp32
// partials by the last of its CTAs to finish.
//
// Bound: HBM while it streams (8 x 32768 keys of 8 heads, d = 128, groups of 128: 285 MB
// in 46 us, 6.2 TB/s); with the start (launch, page lookup, first copies: 5 us) and the
// joining of shares and parts at the end (5 us) the call takes 56.2 us, 5.07 TB/s, 75% of
// the measured copy rate.  Groups of 32 cost four scales a key and need 1390 instructions
// a block of 64 keys against 800, and are bound by their issue (48 uneven sequences: 139
// MB in 42 us).  tcgen05 is not used: its operands come from shared memory, so the codes
// would have to be widened into it, at four times the cache's bytes.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>

#include "fa_kv4.h"
#include "ptx.cuh"

namespace fa {
namespace attend4 {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
// The line of blocks (see the top).  Measured (us; 777 keys / 8 x 32768 / 48 uneven with
// groups of 32 / drafted d = 64 / windowed d = 256): gap 8: 10.0 56.7 40.4 17.4 19.3; 12:
// 9.6 56.5 41.2 16.3 19.2; 16: 9.9 56.2 41.3; items of up to 8 uncut: 11.3 56.5 40.7, of
// up to 24: 9.9 56.4 42.5.
constexpr int kGap = 12;            // what an item costs besides its blocks, in blocks
constexpr int kMinShare = 4 + kGap;  // a CTA's stretch of the line at least ...
constexpr int kUncut = 16;          // ... and items of up to so many blocks are never cut
constexpr int kMostParts = 32;  // CTAs that share an item at most
constexpr float kLn2 = 0.69314718055994530942f;

enum : int { kSiteFull = 48 };

// fp16 pairs of -8 2^-24 and -128 2^-24: what takes 8 off a code, in its row's factor.
constexpr uint32_t kLess8 = 0x80088008u, kLess128 = 0x80808080u;

template <int D, int NG, int NT>
struct Cfg {
  static constexpr int UNITS = D == 256 ? 1 : 2;  // units per block (a block lies in one page)
  static constexpr int BK = UNITS * kKv4Unit;     // keys per block
  static constexpr int UB = kv4_unit_bytes(D, NG);
  static constexpr int STAGE = UNITS * UB;
  static constexpr int STAGES = 2;
  static constexpr int ROWS = 8 * NT;
  static constexpr int DP = D < 128 ? D : 128;  // dims of O that the warps exchange at a time
  static constexpr int OP = DP + 4;             // pitch of a row there (floats)
  static constexpr int RING = kWarps * STAGES * STAGE;
  static constexpr int SMEM = RING + kMostParts * ROWS * 4 + kWarps * ROWS * 8 + kWarps * STAGES * 8 + kWarps * 4 + 16;
  static constexpr int FIT = 227 * 1024 / (SMEM + 1024);
  static constexpr int WANT = NT == 1 && D == 64 ? 3 : 2;
  static constexpr int CTAS = FIT < WANT ? FIT : WANT;  // per SM
  // How 8 is taken off the codes of V: by the sum of the weights from one more MMA a
  // group, with ones, where there are registers for it, else by a second MMA per word
  // with a constant A (8 x 32768 keys, d = 128: 56.4 against 61.0 us; 6 windows of 4096
  // keys, d = 256: 19.4 against 20.1).
  static constexpr bool ONES = NG * NT <= 4;
  static_assert(ROWS * OP * 4 <= STAGE, "a warp's share of O fits the stage that it read last");
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

// c += a b, or c = a b where `first` (a constant).
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1, bool first = false) {
  if (first) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
  } else {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  }
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

// Keys of a sequence; one that outruns its block-table row, or 2^30, has none (and is
// reported).
__device__ __forceinline__ int seq_len(const Attend4Params& p, int seq) {
  const int n = p.seqlens[seq];
  if (n > p.bt_width * p.page_size || n > (1 << 30)) {
    record_error(p.status, kErrDeviceArg);
    return 0;
  }
  return n > 0 ? n : 0;
}

// Rows to query tokens.
__device__ __forceinline__ int over_g(const Attend4Params& p, int rows) {
  return p.g_shift >= 0 ? rows >> p.g_shift : rows / p.g;
}

// One item: a row tile of one KV head of one sequence, keys [lo, hi) all in all, n
// blocks from blo on (one, with nothing in it, where no row sees a key).
template <int BK, int ROWS>
struct Item {
  int seq, kvh, tile, len, lo, hi, blo, n;
  __device__ __forceinline__ void range(const Attend4Params& p) {
    int first = len - p.sq, last = first;  // positions of the tile's first and last row
    if (p.sq > 1) {
      first += over_g(p, tile * ROWS);
      last += over_g(p, min(p.sq * p.g, (tile + 1) * ROWS) - 1);
    }
    hi = max(last + 1, 0);
    lo = p.window_left >= 0 ? max(0, first - p.window_left) : 0;
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

// A CTA's stretch of the line, item by item: blocks [u0, ue) of the current one.  On
// the line every item's blocks follow a gap of kGap positions, so that a CTA that ends
// one item and begins the next gets less of both.  An item of few blocks belongs to
// the CTA in whose stretch its first block lies.
template <int BK, int ROWS>
struct Walk {
  Item<BK, ROWS> it;
  int u0, ue;
  int left;  // blocks from u0 to the end of the stretch
  __device__ __forceinline__ void enter() { ue = it.n <= kUncut ? it.n : min(it.n, u0 + left); }
  __device__ __forceinline__ bool next(const Attend4Params& p) {  // false: nothing is left
    left -= ue - u0 + kGap;
    if (left <= 0) return false;
    it.next(p);
    u0 = 0;
    enter();
    return true;
  }
};

// Line positions of one KV head of a sequence, all tiles; `most`: blocks of its largest item.
template <int BK, int ROWS>
__device__ __forceinline__ int head_blocks(const Attend4Params& p, int seq, int* most) {
  Item<BK, ROWS> it;
  it.len = seq_len(p, seq);
  it.tile = p.ntiles - 1;
  it.range(p);
  int n = it.n + kGap;
  *most = it.n;
  if (p.sq == 1) return n * p.ntiles;  // every tile sees the same keys
  for (it.tile = 0; it.tile < p.ntiles - 1; ++it.tile) {
    it.range(p);
    n += it.n + kGap;
    *most = max(*most, it.n);
  }
  return n;
}

// Eight dims of a finished row, times inv, and its LSE (M, L: log2 maximum and sum).
template <int D, bool BF16>
__device__ __forceinline__ void store_row(const Attend4Params& p, int seq, int kvh, int row, int dim, const float* f,
                                          float inv) {
  const int qi = p.sq > 1 ? over_g(p, row) : 0, h = kvh * p.g + row - qi * p.g;
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if constexpr (BF16) {
      const __nv_bfloat162 x = __floats2bfloat162_rn(f[2 * k] * inv, f[2 * k + 1] * inv);
      w[k] = *reinterpret_cast<const uint32_t*>(&x);
    } else {
      w[k] = pack_f16(f[2 * k] * inv, f[2 * k + 1] * inv);
    }
  }
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) + seq * p.o_st[0] + qi * p.o_st[1] + h * p.o_st[2] + dim) =
      make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void store_lse(const Attend4Params& p, int seq, int kvh, int row, float M, float L) {
  const int qi = p.sq > 1 ? over_g(p, row) : 0, h = kvh * p.g + row - qi * p.g;
  p.lse[(static_cast<int64_t>(seq) * p.hq + h) * p.sq + qi] = L > 0.f ? (M + lg2_approx(L)) * kLn2 : -INFINITY;
}

__device__ __forceinline__ int count_in(int* counter) {
  int old;
  asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(old) : "l"(counter) : "memory");
  return old;
}

template <int D, int NG, bool BF16, int NT>
__global__ void __launch_bounds__(kThreads, Cfg<D, NG, NT>::CTAS) attend4_kernel(const __grid_constant__ Attend4Params p) {
  using C = Cfg<D, NG, NT>;
  constexpr int J = kv4_j(D), NC = D / 32 / J, NW = D / 32, GW = NW / NG;
  constexpr int BK = C::BK, ROWS = C::ROWS;
  // The eleven bits of an fp16 q times a code in a subnormal's lowest four bits are more
  // than the tensor core keeps beside a larger product: LSE was off by up to 2.8e-6 of its
  // size (in fp32).  So for fp16 all codes of K go to bits 4..7, at two more shifts a word
  // (48 sequences, groups of 32: 41.2 to 42.3 us), which leaves 2.4e-7; bf16's eight bits
  // lose 1.4e-6 at most and are left alone.
  constexpr bool HIGH = !BF16;
  constexpr float low = HIGH ? 0.0625f : 1.f;
  extern __shared__ __align__(128) uint8_t smem[];
  const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), g = lane >> 2, t = lane & 3;
  uint8_t* ring = smem + warp * C::STAGES * C::STAGE;
  float* wbuf = reinterpret_cast<float*>(smem + C::RING);                // [kMostParts][ROWS]
  float2* ml = reinterpret_cast<float2*>(wbuf + kMostParts * ROWS);      // [kWarps][ROWS]
  uint64_t* bars = reinterpret_cast<uint64_t*>(ml + kWarps * ROWS);
  uint64_t* full = bars + warp * C::STAGES;
  int* held = reinterpret_cast<int*>(bars + kWarps * C::STAGES);  // [kWarps]: the stage with the warp's share of O
  int* last_in = held + kWarps;

  if (lane == 0) {
    for (int s = 0; s < C::STAGES; ++s) mbar_init(&full[s], 1);
    fence_mbar_init();
  }
  __syncwarp();
  // ---- the CTA's stretch of the line of blocks, found by every warp for itself: the
  // total, the share of a CTA, the sequence where this one's stretch begins
  Walk<BK, ROWS> cw;
  int share, item_at;  // where the current item's blocks start on the line
  {
    int mine = 0, head = 0, most = 0;
    for (int s = lane; s < p.b; s += 32) {
      int m1;
      head = head_blocks<BK, ROWS>(p, s, &m1);
      mine += head * p.hkv;
      most = max(most, m1);
    }
    const int total = __reduce_add_sync(0xffffffffu, mine);
    most = __reduce_max_sync(0xffffffffu, most);
    share = static_cast<int>((static_cast<unsigned>(total) + gridDim.x - 1) / gridDim.x);
    share = max(max(share, kMinShare), (most + kMostParts - 2) / (kMostParts - 1));
    if (static_cast<int64_t>(blockIdx.x) * share >= total) return;
    const int begin = static_cast<int>(blockIdx.x) * share;
    int before = 0, rem = 0;
    for (int s0 = 0; s0 < p.b; s0 += 32) {
      if (p.b > 32) {
        int m1;
        head = s0 + lane < p.b ? head_blocks<BK, ROWS>(p, s0 + lane, &m1) : 0;
        mine = head * p.hkv;
      }
      int incl = mine;
#pragma unroll
      for (int x = 1; x < 32; x <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, x);
        if (lane >= x) incl += y;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, begin < before + incl);
      if (hit != 0) {
        const int at = __ffs(hit) - 1;
        cw.it.seq = s0 + at;
        rem = begin - before - __shfl_sync(0xffffffffu, incl - mine, at);
        head = __shfl_sync(0xffffffffu, head, at);
        break;
      }
      before += __shfl_sync(0xffffffffu, incl, 31);
    }
    cw.left = min(total - begin, share);
    cw.it.len = seq_len(p, cw.it.seq);
    // (a quotient below 2^16: off by one at most)
    cw.it.kvh = static_cast<int>(__fdividef(static_cast<float>(rem), static_cast<float>(head)));
    if (cw.it.kvh * head > rem) --cw.it.kvh;
    if ((cw.it.kvh + 1) * head <= rem) ++cw.it.kvh;
    int u = rem - cw.it.kvh * head - kGap;  // (negative: in the gap)
    cw.it.tile = 0;
    cw.it.range(p);
    while (u >= cw.it.n) {
      u -= cw.it.n + kGap;
      ++cw.it.tile;
      cw.it.range(p);
    }
    item_at = begin - u;
    if (u < 0) {
      cw.left += u;
      if (cw.left <= 0) return;
    }
    cw.u0 = max(u, 0);
    cw.enter();
    if (u > 0 && cw.it.n <= kUncut) {  // an earlier CTA has this one whole
      item_at += cw.it.n + kGap;
      if (!cw.next(p)) return;
    }
  }
  const int R = p.sq * p.g;

  // ---- Q of a tile's rows, as stored (row 8 nt + g, dims 32 j + 8 t ..): loaded ahead
  uint4 qraw[NT][NW];
  auto load_q = [&]() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = cw.it.tile * ROWS + nt * 8 + g;
      const int qi = p.sq > 1 ? over_g(p, r) : 0, h = r - qi * p.g;
      const uint16_t* at = static_cast<const uint16_t*>(p.q) + cw.it.seq * p.q_st[0] + qi * p.q_st[1] +
                           (cw.it.kvh * p.g + h) * p.q_st[2] + 8 * t;
#pragma unroll
      for (int j = 0; j < NW; ++j)
        qraw[nt][j] = r < R ? *reinterpret_cast<const uint4*>(at + 32 * j) : make_uint4(0u, 0u, 0u, 0u);
    }
  };
  load_q();

  // ---- the warp's stream of blocks: `pw` runs ahead of the consumer by batches of up
  // to 32 blocks of an item.  Lane i holds where block i of the batch lies and copies it.
  Walk<BK, ROWS> pw = cw;
  int pu = pw.u0 + warp, batch = 0, next = 0;  // the batch after this one; blocks in it; the next to copy
  int page = 0, flying = 0;  // copies that have not been waited for
  int64_t off = 0;
  bool more = true;
  auto refill = [&]() {
    while (more && (pu >= pw.ue || pw.it.hi <= pw.it.lo)) {
      more = pw.next(p);
      pu = pw.u0 + warp;
    }
    next = batch = 0;
    if (more) {
      batch = min(32, (pw.ue - pu + kWarps - 1) / kWarps);
      const int key = (pw.it.blo + pu + lane * kWarps) * BK;
      const int at = p.page_shift >= 0 ? key >> p.page_shift : key / p.page_size;
      if (lane < batch) page = p.block_table[pw.it.seq * p.bt_stride + at];
      off = pw.it.kvh * p.c_st[1] + static_cast<int64_t>((key - at * p.page_size) / kKv4Unit) * C::UB;
      pu += 32 * kWarps;
    }
  };
  auto copy_next = [&](int slot) {
    if (batch == 0) return;
    ++flying;
    if (lane == next) {
      if (page < 0 || page >= p.num_pages) {
        record_error(p.status, kErrDeviceArg);
        page = 0;
      }
      mbar_arrive_expect_tx(&full[slot], C::STAGE);
      bulk_load(ring + slot * C::STAGE, p.cache + page * p.c_st[0] + off, C::STAGE, &full[slot]);
    }
    if (++next == batch) refill();
  };
  refill();
#pragma unroll 1
  for (int s = 0; s < C::STAGES; ++s) copy_next(s);
  int slot = 0;
  uint32_t phase = 0;
  bool dead = false;  // a wait gave up

  for (bool live = true; live;) {
    const Item<BK, ROWS> it = cw.it;
    // ---- Q of the tile's rows as B operands; its row scales and group sums
    uint32_t qf[NW][2][NT][2];
    float qs[NG][NT][2], rs[NT][2], m[NT][2], l[NT][2], tv[NG][NT][2], o[NW][2][NT][4], ones[C::ONES ? NG : 1][NT][4];
    float cap_rs[NT][2];
    int row_hi[NT][2], row_lo[NT][2];
    const bool capped = p.sc_b > 0.f;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const uint4(&u)[NW] = qraw[nt];
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
        qf[j][0][nt][0] = pack_f16(x[0] * low, x[4] * low);
        qf[j][0][nt][1] = pack_f16(x[2] * low, x[6] * low);
        qf[j][1][nt][0] = pack_f16(x[1] * 0.0625f, x[5] * 0.0625f);
        qf[j][1][nt][1] = pack_f16(x[3] * 0.0625f, x[7] * 0.0625f);
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int from = 4 * (2 * t + c);
        const float scale = __shfl_sync(0xffffffffu, down, from) * 0x1p24f * p.scale_log2;
        cap_rs[nt][c] = scale;
        rs[nt][c] = capped ? 1.f : scale;
        const int rc = it.tile * ROWS + nt * 8 + 2 * t + c;
        const int pos = it.len - p.sq + (p.sq > 1 ? over_g(p, rc) : 0);
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
        if constexpr (C::ONES) {
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
    int all_hi = it.len - p.sq, all_lo = it.hi - 1 - p.window_left;
    if (p.sq > 1) all_hi += over_g(p, it.tile * ROWS);
    if (p.window_left < 0) all_lo = 0;
    int hold = -1;
    float vscale = 0.f;  // V's weights are held times this power of two (0: not chosen yet)

    if (it.hi > it.lo && !dead)
      for (int u = cw.u0 + warp; u < cw.ue; u += kWarps) {
        if (!__all_sync(0xffffffffu, mbar_wait(&full[slot], phase, p.status, kSiteFull))) {
          // the wait gave up (and said so): this warp reads no more, and its copies land
          // before it leaves
          for (; flying > 0; --flying) {
            mbar_wait(&full[slot], phase, p.status, kSiteFull, true);
            if (++slot == C::STAGES) {
              slot = 0;
              phase ^= 1u;
            }
          }
          batch = 0;
          dead = true;
          break;
        }
        --flying;
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
              // nibbles 0, 4 (and 2, 6 through ha, hb) for the first MMA, 1, 5 (3, 7) for the second
              const uint32_t ha = wa[j] >> 8, hb = wb[j] >> 8;
              uint32_t e0 = wa[j] & 0x000f000fu, e1 = wb[j] & 0x000f000fu, e2 = ha & 0x000f000fu, e3 = hb & 0x000f000fu;
              if constexpr (HIGH) {
                e0 = (wa[j] << 4) & 0x00f000f0u;
                e1 = (wb[j] << 4) & 0x00f000f0u;
                e2 = (wa[j] >> 4) & 0x00f000f0u;
                e3 = (wb[j] >> 4) & 0x00f000f0u;
              }
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                mma16816(acc[nt], e0, e1, e2, e3, qf[w][0][nt][0], qf[w][0][nt][1], w % GW == 0);
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
                if constexpr (C::ONES) ones[q][nt][c] *= a;
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
            const float now = __uint_as_float((261u - max(__float_as_uint(top) >> 23, 8u)) << 23);
            if (vscale > 0.f) {
              const float a = now / vscale;
              if constexpr (C::ONES) {
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
              bw[q][nt][0] = transpose8(ha);
              bw[q][nt][1] = transpose8(hb);
              if constexpr (C::ONES) mma16816(ones[q][nt], 0x3c003c00u, 0u, 0x3c003c00u, 0u, bw[q][nt][0], bw[q][nt][1]);
            }
          }
          if constexpr (!C::ONES) {
#pragma unroll
            for (int w = 0; w < NW; ++w)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                mma16816(o[w][0][nt], kLess8, kLess128, kLess8, kLess128, bw[w / GW][nt][0], bw[w / GW][nt][1]);
                mma16816(o[w][1][nt], kLess8, kLess128, kLess8, kLess128, bw[w / GW][nt][0], bw[w / GW][nt][1]);
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
        if (u + kWarps < cw.ue) copy_next(slot);
        else hold = slot;  // (the last stage read carries the warp's share of O first)
        if (++slot == C::STAGES) {
          slot = 0;
          phase ^= 1u;
        }
      }

    // ---- the next item is found and its Q loaded while this one's shares are joined
    const int at = item_at;
    item_at += it.n + kGap;
    live = cw.next(p);
    if (live) load_q();

    // ---- the warps' shares: each row's maximum, sum and O (as of the warp's maximum)
    // through shared memory, dims [128 ps, 128 ps + DP) at a time
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
    if (lane == 0) held[warp] = hold;
    if (g == 0) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) ml[warp * ROWS + nt * 8 + 2 * t + c] = make_float2(m[nt][c], l[nt][c]);
    }
    const float unscale = vscale > 0.f ? 0x1p24f / vscale : 0.f;
    const int cta = blockIdx.x;
    int c0 = cta, c1 = cta;  // the CTAs that hold the item
    if (it.n > kUncut) {
      c0 = at / share;
      c1 = (at + it.n - 1) / share;
    }
    const bool whole = c0 == c1;
    const int s0 = 2 * c0 + (at > c0 * share ? 1 : 0);  // the first part's slot
    const int my = cta == c0 ? s0 : 2 * cta;
    constexpr int PER = C::DP / 8;  // threads of a row
#pragma unroll
    for (int ps = 0; ps < D / C::DP; ++ps) {
      if (ps > 0) __syncthreads();
      if (hold >= 0) {
        float* mine = reinterpret_cast<float*>(ring + hold * C::STAGE);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int j = 0; j < C::DP / 32; ++j) {
              const int w = ps * (C::DP / 32) + j;
              float add = tv[w / GW][nt][c];
              if constexpr (C::ONES) add = fmaf(ones[w / GW][nt][c], -0x1p-21f * unscale, add);
              *reinterpret_cast<float4*>(mine + (nt * 8 + 2 * t + c) * C::OP + 32 * j + 4 * g) =
                  make_float4(fmaf(o[w][0][nt][c], unscale, add), fmaf(o[w][0][nt][c + 2], unscale * 0.0625f, add),
                              fmaf(o[w][1][nt][c], unscale, add), fmaf(o[w][1][nt][c + 2], unscale * 0.0625f, add));
            }
        fence_proxy_async_smem();  // (the stage's next copy comes after these stores)
      }
      __syncthreads();
      for (int x = threadIdx.x; x < ROWS * PER; x += kThreads) {
        const int r = x / PER, e = x % PER, row = it.tile * ROWS + r;
        float M = -INFINITY, L = 0.f, f[8];
        float2 y[kWarps];
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          y[w] = ml[w * ROWS + r];
          M = fmaxf(M, y[w].x);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          if (y[w].x == -INFINITY) continue;  // (a warp without a block has no share)
          const float a = ex2_approx(y[w].x - M);
          const float4* from = reinterpret_cast<const float4*>(smem + (w * C::STAGES + held[w]) * C::STAGE) + (r * C::OP) / 4 + 2 * e;
          const float4 u = from[0], v = from[1];
          L = fmaf(y[w].y, a, L);
          f[0] = fmaf(u.x, a, f[0]);
          f[1] = fmaf(u.y, a, f[1]);
          f[2] = fmaf(u.z, a, f[2]);
          f[3] = fmaf(u.w, a, f[3]);
          f[4] = fmaf(v.x, a, f[4]);
          f[5] = fmaf(v.y, a, f[5]);
          f[6] = fmaf(v.z, a, f[6]);
          f[7] = fmaf(v.w, a, f[7]);
        }
        if (whole) {
          if (row < R) store_row<D, BF16>(p, it.seq, it.kvh, row, ps * C::DP + 8 * e, f, L > 0.f ? 1.f / L : 0.f);
          if (row < R && e == 0 && ps == 0) store_lse(p, it.seq, it.kvh, row, M, L);
        } else {
          float4* to = reinterpret_cast<float4*>(p.part_o + (static_cast<int64_t>(my) * ROWS + r) * D + ps * C::DP + 8 * e);
          to[0] = make_float4(f[0], f[1], f[2], f[3]);
          to[1] = make_float4(f[4], f[5], f[6], f[7]);
          if (e == 0 && ps == 0) p.part_ml[static_cast<int64_t>(my) * ROWS + r] = make_float2(M, L);
        }
      }
    }
    if (!whole) {
      // the last of the item's CTAs to get here joins the parts (the barrier puts the
      // CTA's stores before thread 0's releasing and acquiring count)
      __syncthreads();
      asm volatile("griddepcontrol.wait;" ::: "memory");  // the counters are zeroed by the grid before
      if (threadIdx.x == 0) *last_in = count_in(p.counters + c0) == c1 - c0;
      __syncthreads();
      if (*last_in) {
        constexpr int TPR = kThreads / ROWS;  // threads of a row for the weights
        const int parts = c1 - c0 + 1;
        {
          const int r = threadIdx.x / TPR, k = threadIdx.x % TPR, row = it.tile * ROWS + r;
          float M = -INFINITY, L = 0.f;
          for (int s = k; s < parts; s += TPR) {
            const float2 y = __ldcg(&p.part_ml[static_cast<int64_t>(s == 0 ? s0 : 2 * (c0 + s)) * ROWS + r]);
            const float n = fmaxf(M, y.x);
            if (n != -INFINITY) L = L * ex2_approx(M - n) + (y.x == -INFINITY ? 0.f : y.y * ex2_approx(y.x - n));
            M = n;
            wbuf[s * ROWS + r] = y.x;
          }
#pragma unroll
          for (int x = 1; x < TPR; x <<= 1) {
            const float m2 = __shfl_xor_sync(0xffffffffu, M, x), l2 = __shfl_xor_sync(0xffffffffu, L, x);
            const float n = fmaxf(M, m2);
            if (n != -INFINITY) L = L * ex2_approx(M - n) + l2 * ex2_approx(m2 - n);
            M = n;
          }
          const float inv = L > 0.f ? 1.f / L : 0.f;
          for (int s = k; s < parts; s += TPR)
            wbuf[s * ROWS + r] = M == -INFINITY ? 0.f : ex2_approx(wbuf[s * ROWS + r] - M) * inv;
          if (k == 0 && row < R) store_lse(p, it.seq, it.kvh, row, M, L);
        }
        __syncthreads();
        for (int x = threadIdx.x; x < ROWS * (D / 8); x += kThreads) {
          const int r = x / (D / 8), e = x % (D / 8), row = it.tile * ROWS + r;
          float f[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) f[k] = 0.f;
#pragma unroll 8
          for (int s = 0; s < parts; ++s) {
            const float4* from = reinterpret_cast<const float4*>(
                p.part_o + (static_cast<int64_t>(s == 0 ? s0 : 2 * (c0 + s)) * ROWS + r) * D + 8 * e);
            const float4 u = __ldcg(from), v = __ldcg(from + 1);
            const float a = wbuf[s * ROWS + r];
            f[0] = fmaf(u.x, a, f[0]);
            f[1] = fmaf(u.y, a, f[1]);
            f[2] = fmaf(u.z, a, f[2]);
            f[3] = fmaf(u.w, a, f[3]);
            f[4] = fmaf(v.x, a, f[4]);
            f[5] = fmaf(v.y, a, f[5]);
            f[6] = fmaf(v.z, a, f[6]);
            f[7] = fmaf(v.w, a, f[7]);
          }
          if (row < R) store_row<D, BF16>(p, it.seq, it.kvh, row, 8 * e, f, 1.f);
        }
      }
    }
    if (live) {
      __syncthreads();  // the buffers are free again
      if (hold >= 0) copy_next(hold);
    }
  }
  // (block 0 always has a stretch.)  This grid ends after the one that zeroes the counters
  // even where no item is cut, so nothing of the call touches the workspace behind it.
  if (blockIdx.x == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
}

static __global__ void zero_counters_kernel(int* counters, int n) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  for (int i = threadIdx.x; i < n; i += blockDim.x) counters[i] = 0;
}

template <int D, int NG, bool BF16, int NT>
cudaError_t launch_one(const Attend4Params& p, int grid, cudaStream_t stream) {
  using C = Cfg<D, NG, NT>;
  auto* k = attend4_kernel<D, NG, BF16, NT>;
  static_assert(C::SMEM <= 227 * 1024, "shared memory");
  static std::atomic<uint64_t> ready{0};  // devices whose kernel may use that much shared memory
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = static_cast<uint64_t>(1) << (dev & 63);
  if ((ready.load(std::memory_order_relaxed) & bit) == 0) {
    e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_relaxed);
  }
  if (!p.cuts) {
    k<<<grid, kThreads, C::SMEM, stream>>>(p);
    return cudaGetLastError();
  }
  // the kernel starts beside the one that zeroes its counters and waits for it only
  // before it counts
  zero_counters_kernel<<<1, 512, 0, stream>>>(p.counters, grid);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, p);
}

template <int D, int NG, int NT>
cudaError_t launch_dtype(const Attend4Params& p, int dtype, int sms, Attend4Plan* plan, cudaStream_t stream) {
  using C = Cfg<D, NG, NT>;
  if (plan != nullptr) {
    plan->rows = C::ROWS;
    plan->block = C::BK;
    plan->gap = kGap;
    plan->uncut = kUncut;
    plan->max_ctas = sms * C::CTAS;
    return cudaSuccess;
  }
  return dtype == 0 ? launch_one<D, NG, true, NT>(p, p.grid, stream) : launch_one<D, NG, false, NT>(p, p.grid, stream);
}

// Up to eight query rows of a KV head per reading of the cache, or sixteen.  Sixteen of
// 256 dims do not fit the registers: two readings measured 21.6 against 39.6 us there (4
// x 8192 keys, two tokens of eight heads a KV head), while at d = 128 one reading takes
// 82 against 100 us (8 x 32768 keys, 16 heads a KV head).
template <int D, int NG>
cudaError_t launch_rows(const Attend4Params& p, int dtype, int sms, Attend4Plan* plan, cudaStream_t stream) {
  if constexpr (D <= 128) {
    if (p.sq * p.g > 8) return launch_dtype<D, NG, 2>(p, dtype, sms, plan, stream);
  }
  return launch_dtype<D, NG, 1>(p, dtype, sms, plan, stream);
}

}  // namespace attend4
}  // namespace fa
