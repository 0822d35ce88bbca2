// Filling a paged cache: the rotary rotation of new queries and keys, the store of
// new keys and values into their pages (16-bit rows, or 4-bit codes with group
// scales), and the gather of 4-bit pages back into 16-bit rows.
//
// All of it is bound by HBM traffic for prompts and by latency for single tokens.  A
// lane keeps sixteen dims of one token, d / 16 lanes a token, and walks over the
// token's heads: the rotation's cosines and sines are read once per token and stay in
// registers, as does the token's place in the cache.  Several heads' rows are loaded
// before the first is used.  The heads of a token are dealt to as many warps as
// suit the GPU: one head each for a few tokens, all heads to a warp for long prompts.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>

#include "fa_kv4.h"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kThreads = 128;
constexpr int kAppendCtas = 7, kGatherCtas = 10;  // CTAs an SM holds
constexpr int kFlight = 2;                        // rows of the append that a warp has in flight

// ---- two fp32 values in one 64-bit register, for the packed operations
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t x;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a), "f"(b));
  return x;
}

__device__ __forceinline__ float2 unpack2(uint64_t x) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(x));
  return f;
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t x;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(x) : "l"(a), "l"(b));
  return x;
}

__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t x;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(x) : "l"(a), "l"(b));
  return x;
}

__device__ __forceinline__ uint64_t sub2(uint64_t a, uint64_t b) {
  uint64_t x;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(x) : "l"(a), "l"(b));
  return x;
}

__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t x;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(x) : "l"(a), "l"(b), "l"(c));
  return x;
}

// ---- 16-bit pairs <-> fp32 pairs
template <bool BF16>
__device__ __forceinline__ uint64_t widen2(uint32_t w) {
  if constexpr (BF16) return pack2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&w));
  return pack2(x.x, x.y);
}

template <bool BF16>
__device__ __forceinline__ uint32_t narrow2(float a, float b) {
  if constexpr (BF16) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&x);
  } else {
    const __half2 x = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&x);
  }
}

template <bool BF16>
__device__ __forceinline__ float widen1(uint32_t h) {
  if constexpr (BF16) return __uint_as_float(h << 16);
  return __half2float(__ushort_as_half(static_cast<unsigned short>(h)));
}

template <bool BF16>
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  if constexpr (BF16) {
    const __nv_bfloat162 x = __hmin2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&x);
  } else {
    const __half2 x = __hmin2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&x);
  }
}

template <bool BF16>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  if constexpr (BF16) {
    const __nv_bfloat162 x = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&x);
  } else {
    const __half2 x = __hmax2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&x);
  }
}

// Eight 16-bit dims of a row.
struct Chunk {
  uint32_t w[4];
};

__device__ __forceinline__ Chunk load_chunk(const uint16_t* p) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  return Chunk{{u.x, u.y, u.z, u.w}};
}

__device__ __forceinline__ void store_chunk(uint16_t* p, const Chunk& c) {
  *reinterpret_cast<uint4*>(p) = make_uint4(c.w[0], c.w[1], c.w[2], c.w[3]);
}

// The two chunks of a row (of D / 8) that lane k of its D / 16 lanes holds, in the
// order of the 4-bit cache: its codes of K are one 64-bit word, those of V two.
__device__ __forceinline__ int cache_chunk(int k, int which) { return 8 * (k / 4) + k % 4 + 4 * which; }

// A token's place: sequence, position, page and row.  ok = false: it has none (a row
// of no sequence, a padding token, or an argument that fails its check).
struct Slot {
  bool ok;
  int pos, page, row;
};

// The places of a warp's tokens, one a lane.  The sequence of a row of the packed
// tensors is the number of sequences that end at or before it: 32 of the prefix sums
// (all of them, for up to 32 sequences) are compared at once, then a binary search
// ends among the rest.
template <int LPT>
__device__ __forceinline__ Slot find_slot(const int* cu, int b, int total, const int* seqlens, const int* table,
                                          int64_t bt_stride, int64_t bt_width, int page_size, int num_pages,
                                          int max_positions, int tok,
                                          int* status) {
  Slot s{false, 0, 0, 0};
  const int lane = threadIdx.x & 31;
  const bool live = tok < total;
  int seq = 0, first = 0, n = 0;
  if (cu == nullptr) {
    n = total / b;
    seq = live ? tok / n : 0;
    first = seq * n;
  } else {
    const int stride = (b + 31) / 32;
    const int v = cu[min(b, (lane + 1) * stride)];
    int count = 0;
#pragma unroll
    for (int j = 0; j < 32 / LPT; ++j) {
      const int other = __shfl_sync(0xffffffffu, tok, j * LPT);
      const int c = __popc(__ballot_sync(0xffffffffu, v <= other && (lane + 1) * stride <= b));
      if (lane / LPT == j) count = c;
    }
    int lo = min(count * stride, b - 1), hi = min(lo + stride, b);
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (cu[mid] <= tok) lo = mid; else hi = mid;
    }
    seq = lo;
    first = cu[lo];
    n = cu[lo + 1] - first;
  }
  if (!live || first > tok || tok - first >= n) return s;
  const int64_t pos = static_cast<int64_t>(seqlens[seq]) - n + (tok - first);
  if (pos < 0) return s;  // padding before the sequence's first key
  if (pos >= bt_width * page_size || (max_positions > 0 && pos >= max_positions)) {
    record_error(status, kErrDeviceArg);
    return s;
  }
  s.pos = static_cast<int>(pos);
  const int at = s.pos / page_size;
  s.page = table[seq * bt_stride + at];
  s.row = s.pos - at * page_size;
  s.ok = s.page >= 0 && s.page < num_pages;
  if (!s.ok) record_error(status, kErrDeviceArg);
  return s;
}

// The prefix sums are checked once per launch, by the first block.
__device__ __forceinline__ void check_prefix(const int* cu, int b, int total, int* status) {
  if (cu == nullptr || blockIdx.x != 0) return;
  bool ok = cu[0] >= 0 && cu[b] <= total;
  for (int i = threadIdx.x; i < b; i += blockDim.x) ok = ok && cu[i] <= cu[i + 1];
  if (!ok) record_error(status, kErrDeviceArg);
}

// The rotation of a lane's two chunks.  Half-split: dims [8 c, 8 c + 8) turn with dims
// R / 2 further on, and the lane holds both chunks, so no row is read twice and the
// eight cosines and sines serve both.  Interleaved: a chunk holds four pairs that turn
// in themselves.  Products and sums are rounded one by one, as in the plain formula.
struct Turn {
  float c[8], s[8];  // half-split: of the eight angles; interleaved: of the chunks' four each
  bool on[2];
  bool split;
};

template <bool BF16>
__device__ __forceinline__ void turn(Chunk (&x)[2], const Turn& t) {
  if (t.split) {
    if (!t.on[0]) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint64_t a = widen2<BF16>(x[0].w[i]), b = widen2<BF16>(x[1].w[i]);
      const uint64_t c = pack2(t.c[2 * i], t.c[2 * i + 1]), s = pack2(t.s[2 * i], t.s[2 * i + 1]);
      const float2 ya = unpack2(sub2(mul2(a, c), mul2(b, s))), yb = unpack2(add2(mul2(b, c), mul2(a, s)));
      x[0].w[i] = narrow2<BF16>(ya.x, ya.y);
      x[1].w[i] = narrow2<BF16>(yb.x, yb.y);
    }
    return;
  }
#pragma unroll
  for (int q = 0; q < 2; ++q)
    if (t.on[q]) {
#pragma unroll
      for (int i = 0; i < 4; i += 2) {  // two pairs: their first dims and their second ones
        const float2 v = unpack2(widen2<BF16>(x[q].w[i])), u = unpack2(widen2<BF16>(x[q].w[i + 1]));
        const uint64_t a = pack2(v.x, u.x), b = pack2(v.y, u.y);
        const uint64_t c = pack2(t.c[4 * q + i], t.c[4 * q + i + 1]), s = pack2(t.s[4 * q + i], t.s[4 * q + i + 1]);
        const float2 ya = unpack2(sub2(mul2(a, c), mul2(b, s))), yb = unpack2(add2(mul2(b, c), mul2(a, s)));
        x[q].w[i] = narrow2<BF16>(ya.x, yb.x);
        x[q].w[i + 1] = narrow2<BF16>(ya.y, yb.y);
      }
    }
}

// The smallest value of one or both chunks, and of their negatives, in one word.
template <bool BF16>
__device__ __forceinline__ uint32_t extremes(const Chunk* x, int n) {
  uint32_t mn = x[0].w[0], mx = x[0].w[0];
#pragma unroll
  for (int i = 1; i < 4 * n; ++i) {
    mn = min2<BF16>(mn, x[i / 4].w[i % 4]);
    mx = max2<BF16>(mx, x[i / 4].w[i % 4]);
  }
  mx ^= 0x80008000u;
  return min2<BF16>(__byte_perm(mn, mx, 0x5410), __byte_perm(mn, mx, 0x7632));
}

// The levels of a group from its extremes: the (scale, min) pair as stored, and what
// the codes are computed with.  The minimum is exact in the rows' type; the scale
// (max - min) / 15 is rounded to it (halved first, so that it cannot overflow).
struct Levels {
  uint32_t pair;
  float low, s, r;
};

template <bool BF16>
__device__ __forceinline__ Levels levels(uint32_t both) {
  Levels v;
  v.low = widen1<BF16>(both & 0xffffu);
  const float half_range = __fsub_rn(-0.5f * widen1<BF16>(both >> 16), 0.5f * v.low);
  const float by = 0x1.111112p-3f;  // 1 / 7.5 to nearest; the quotient is corrected as below
  float q = __fmul_rn(half_range, by);
  q = __fmaf_rn(__fmaf_rn(-7.5f, q, half_range), by, q);
  v.pair = narrow2<BF16>(q, v.low);
  v.s = widen1<BF16>(v.pair & 0xffffu);
  if (v.s < 0x1p-100f) {
    v.s = 0.f;
    v.pair &= 0xffff0000u;
  }
  v.r = v.s > 0.f ? rcp_approx(v.s) : 0.f;
  return v;
}

// The codes of a chunk, value i in nibble i.  Many 16-bit values lie exactly between
// two levels, so where (x - min) / scale is a number with a half it has to come out
// exactly: x times the reciprocal, then one correction by its exact remainder
// (Markstein's), which leaves less than 2^-44 of an error before the last rounding.  The
// nearest integer is in the low bits of the quotient's sum with 1.5 * 2^23.  CLAMP: a
// subnormal fp16 scale may be far below (max - min) / 15.
template <bool BF16, bool CLAMP>
__device__ __forceinline__ uint32_t quantise(const Chunk& x, const Levels& v) {
  const uint64_t r2 = pack2(v.r, v.r), s2 = pack2(-v.s, -v.s), m2 = pack2(-v.low, -v.low);
  const uint64_t magic = pack2(12582912.f, 12582912.f);
  uint32_t word = 0;
#pragma unroll
  for (int i = 3; i >= 0; --i) {
    const uint64_t a = add2(widen2<BF16>(x.w[i]), m2);
    uint64_t y = mul2(a, r2);
    y = fma2(fma2(s2, y, a), r2, y);
    if (CLAMP) {
      const float2 f = unpack2(y);
      y = pack2(fminf(f.x, 15.f), fminf(f.y, 15.f));
    }
    const float2 z = unpack2(add2(y, magic));  // bits 0x4b400000 + code
    word = (word << 4) + __float_as_uint(z.y);
    word = (word << 4) + __float_as_uint(z.x);
  }
  return word - 0x3f400000u;  // the sum of 0x4b400000 << 4 i, i = 0..7
}

// Both chunks of a lane (in the cache's order) quantised in groups of `group` dims; the
// four or eight lanes of a group take part.  pair[1] is the second chunk's.
template <bool BF16>
__device__ __forceinline__ void quantise_row(const Chunk (&x)[2], int group, uint32_t (&codes)[2], uint32_t (&pair)[2]) {
  Levels v0, v1;
  if (group == 32) {
    uint32_t e0 = extremes<BF16>(x, 1), e1 = extremes<BF16>(x + 1, 1);
#pragma unroll
    for (int s = 1; s < 4; s *= 2) {
      e0 = min2<BF16>(e0, __shfl_xor_sync(0xffffffffu, e0, s));
      e1 = min2<BF16>(e1, __shfl_xor_sync(0xffffffffu, e1, s));
    }
    v0 = levels<BF16>(e0);
    v1 = levels<BF16>(e1);
  } else {
    uint32_t e = extremes<BF16>(x, 2);
    for (int s = 1; s < group / 16; s *= 2) e = min2<BF16>(e, __shfl_xor_sync(0xffffffffu, e, s));
    v0 = v1 = levels<BF16>(e);
  }
  if (!BF16 && __any_sync(0xffffffffu, fminf(v0.s, v1.s) < 0x1p-14f)) {
    codes[0] = quantise<BF16, true>(x[0], v0);
    codes[1] = quantise<BF16, true>(x[1], v1);
  } else {
    codes[0] = quantise<BF16, false>(x[0], v0);
    codes[1] = quantise<BF16, false>(x[1], v1);
  }
  pair[0] = v0.pair;
  pair[1] = v1.pair;
}

// Two rows in flight a lane and 28 warps an SM: 16-bit, four prompts of 4096: 62.5 us, 6.6
// TB/s of traffic.  Other choices, before the rows were dealt as they are now (63.6 us then,
// 26.6 for uneven chunks at d = 256, 80.2 for the prompts at 4 bits with the gather): 32
// warps, which spill, 63.9, 27.5 and 83.2; four rows and 24 or 20 warps 63.0, 27.4 and 88.2;
// one row and 40 or 36 warps 66.0, 28.0 and 86.5.  A queue of single rows ahead of the one
// at work was slower (69 to 80 us): loads and stores alternate then.
template <int D, bool BF16, bool INT4>
__global__ void __launch_bounds__(kThreads, kAppendCtas) kv_append_kernel(const __grid_constant__ KvAppendParams p) {
  constexpr int LPT = D / 16, TPW = 32 / LPT;  // lanes of a token, tokens of a warp
  constexpr int U = kFlight;
  check_prefix(p.cu, p.b, p.total, p.status);
  const int lane = threadIdx.x & 31, k = lane % LPT;
  const unsigned w = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int parts = p.parts, part = static_cast<int>(w % parts);  // this warp's rows: part, part + parts, ...
  const unsigned tok_u = (w / parts) * TPW + lane / LPT;
  const int tok = static_cast<int>(min(tok_u, 0x7fffffffu));
  const bool live = tok < p.total;

  // ---- the lane's chunks of rows that turn: the cache's, or a chunk and its partner
  Turn t;
  t.split = p.rot > 0 && !p.interleaved;
  int ca = cache_chunk(k, 0), cb = cache_chunk(k, 1);
  int from[2], slot[2];  // half-split: the lane, and which of its chunks, that has the cache's chunk
  if (t.split) {
    const int nr = p.rot / 16;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int want = cache_chunk(k, c);
      from[c] = want < nr ? want : (want < 2 * nr ? want - nr : nr + (want - 2 * nr) / 2);
      slot[c] = want < nr ? 0 : (want < 2 * nr ? 1 : want % 2);
      from[c] += lane - k;
    }
    ca = k < nr ? k : 2 * k;
    cb = k < nr ? k + nr : 2 * k + 1;
    t.on[0] = t.on[1] = k < nr;
  } else {
    t.on[0] = 8 * ca < p.rot;
    t.on[1] = 8 * cb < p.rot;
  }

  // Rows h = part, part + parts, ... of one tensor, U at a time; the first are loaded
  // before the token's place is known.
  auto load_rows = [&](Chunk (&x)[U][2], const uint16_t* base, int64_t step, int h0, int n, int c0, int c1) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u * parts;
      if (live && h < n) {
        x[u][0] = load_chunk(base + h * step + 8 * c0);
        x[u][1] = load_chunk(base + h * step + 8 * c1);
      } else {
        x[u][0] = x[u][1] = Chunk{{0u, 0u, 0u, 0u}};
      }
    }
  };
  const uint16_t* q_at = static_cast<const uint16_t*>(p.q) + tok * p.q_st[0];
  const uint16_t* k_at = static_cast<const uint16_t*>(p.k) + tok * p.k_st[0];
  const uint16_t* v_at = static_cast<const uint16_t*>(p.v) + tok * p.v_st[0];
  const int k_first = (part + parts - p.hq % parts) % parts;              // rows are dealt over q, k and v in turn
  const int v_first = (part + parts - (p.hq + p.hkv) % parts) % parts;
  Chunk x[U][2];
  if (part < p.hq) load_rows(x, q_at, p.q_st[1], part, p.hq, ca, cb);
  const Slot s = find_slot<LPT>(p.cu, p.b, p.total, p.seqlens, p.block_table, p.bt_stride, p.bt_width, p.page_size, p.num_pages,
                                p.rot > 0 ? p.max_positions : 0, tok, p.status);
#pragma unroll
  for (int i = 0; i < 8; ++i) t.c[i] = t.s[i] = 0.f;
  if (s.ok) {
    const float* cs = p.cos_sin + static_cast<int64_t>(s.pos) * p.rot;
    const int half = p.rot / 2;
#pragma unroll
    for (int q = 0; q < 2; ++q)
      if (t.on[q]) {
        const int a = t.split ? 8 * ca + 4 * q : 4 * (q == 0 ? ca : cb);
        const float2 c0 = *reinterpret_cast<const float2*>(cs + a), c1 = *reinterpret_cast<const float2*>(cs + a + 2);
        const float2 s0 = *reinterpret_cast<const float2*>(cs + half + a);
        const float2 s1 = *reinterpret_cast<const float2*>(cs + half + a + 2);
        t.c[4 * q] = c0.x, t.c[4 * q + 1] = c0.y, t.c[4 * q + 2] = c1.x, t.c[4 * q + 3] = c1.y;
        t.s[4 * q] = s0.x, t.s[4 * q + 1] = s0.y, t.s[4 * q + 2] = s1.x, t.s[4 * q + 3] = s1.y;
      }
  }

  // ---- queries
  uint16_t* qo_at = static_cast<uint16_t*>(p.q_out) + tok * p.qo_st[0];
  for (int h0 = part; h0 < p.hq; h0 += U * parts) {
    if (h0 != part) load_rows(x, q_at, p.q_st[1], h0, p.hq, ca, cb);
    __syncwarp();  // (q_out may be q: a row is read before any lane writes it)
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u * parts;
      if (h < p.hq && s.ok) {
        turn<BF16>(x[u], t);
        store_chunk(qo_at + h * p.qo_st[1] + 8 * ca, x[u][0]);
        store_chunk(qo_at + h * p.qo_st[1] + 8 * cb, x[u][1]);
      }
    }
  }

  if constexpr (!INT4) {
    uint16_t* kc_at = static_cast<uint16_t*>(p.k_cache) + s.page * p.kc_st[0] + s.row * p.kc_st[1];
    for (int h0 = k_first; h0 < p.hkv; h0 += U * parts) {
      load_rows(x, k_at, p.k_st[1], h0, p.hkv, ca, cb);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = h0 + u * parts;
        if (h < p.hkv && s.ok) {
          turn<BF16>(x[u], t);
          store_chunk(kc_at + h * p.kc_st[2] + 8 * ca, x[u][0]);
          store_chunk(kc_at + h * p.kc_st[2] + 8 * cb, x[u][1]);
        }
      }
    }
    uint16_t* vc_at = static_cast<uint16_t*>(p.v_cache) + s.page * p.vc_st[0] + s.row * p.vc_st[1];
    for (int h0 = v_first; h0 < p.hkv; h0 += U * parts) {
      load_rows(x, v_at, p.v_st[1], h0, p.hkv, 2 * k, 2 * k + 1);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = h0 + u * parts;
        if (h < p.hkv && s.ok) {
          store_chunk(vc_at + h * p.vc_st[2] + 16 * k, x[u][0]);
          store_chunk(vc_at + h * p.vc_st[2] + 16 * k + 8, x[u][1]);
        }
      }
    }
  } else {
    const int ng = D / p.group, r = s.row % kKv4Unit;
    const int g0 = 8 * cache_chunk(k, 0) / p.group, g1 = 8 * cache_chunk(k, 1) / p.group;
    const bool tells = k % 4 == 0 && (p.group < 128 || k % 8 == 0);  // this lane stores its groups' pairs
    uint8_t* unit0 = p.cache + s.page * p.c_st[0] + static_cast<int64_t>(s.row / kKv4Unit) * kv4_unit_bytes(D, ng);
    auto store_pairs = [&](uint8_t* unit, bool of_v, const uint32_t (&pair)[2]) {
      if (s.ok && tells) {
        uint32_t* at = reinterpret_cast<uint32_t*>(unit + 32 * D) + (of_v ? 32 * ng : 0) + r * ng;
        at[g0] = pair[0];
        if (g1 != g0) at[g1] = pair[1];
      }
    };
    for (int h0 = k_first; h0 < p.hkv; h0 += U * parts) {
      load_rows(x, k_at, p.k_st[1], h0, p.hkv, ca, cb);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = h0 + u * parts;
        if (h >= p.hkv) break;
        turn<BF16>(x[u], t);
        if (t.split) {  // to the cache's order
          Chunk y[2];
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t a = __shfl_sync(0xffffffffu, x[u][0].w[i], from[c]), b = __shfl_sync(0xffffffffu, x[u][1].w[i], from[c]);
              y[c].w[i] = slot[c] ? b : a;
            }
          x[u][0] = y[0];
          x[u][1] = y[1];
        }
        uint32_t codes[2], pair[2];
        quantise_row<BF16>(x[u], p.group, codes, pair);
        uint8_t* unit = unit0 + h * p.c_st[1];
        if (s.ok)
          *reinterpret_cast<uint2*>(reinterpret_cast<uint32_t*>(unit) + kv4_k_word(D, r, cache_chunk(k, 0))) =
              make_uint2(codes[0], codes[1]);
        store_pairs(unit, false, pair);
      }
    }
    // a token and the one after it, both in this warp, share V's words if they are an
    // even and an odd key of one page
    const int np = __shfl_down_sync(0xffffffffu, s.ok ? s.page : -1, LPT), nr = __shfl_down_sync(0xffffffffu, s.row, LPT);
    const bool with_next = s.ok && lane < 32 - LPT && s.row % 2 == 0 && np == s.page && nr == s.row + 1;
    const int up = __shfl_up_sync(0xffffffffu, with_next ? 1 : 0, LPT);
    const bool with_prev = lane >= LPT && up != 0;
    const int quad = 2 * cache_chunk(k, 0);  // V's quads of the first chunk: this one and the next
    for (int h0 = v_first; h0 < p.hkv; h0 += U * parts) {
      load_rows(x, v_at, p.v_st[1], h0, p.hkv, cache_chunk(k, 0), cache_chunk(k, 1));
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = h0 + u * parts;
        if (h >= p.hkv) break;
        uint32_t codes[2], pair[2];
        quantise_row<BF16>(x[u], p.group, codes, pair);
        uint8_t* unit = unit0 + h * p.c_st[1];
        const uint32_t n0 = __shfl_down_sync(0xffffffffu, codes[0], LPT), n1 = __shfl_down_sync(0xffffffffu, codes[1], LPT);
        uint16_t* vh = reinterpret_cast<uint16_t*>(unit + 16 * D);
        if (with_next) {  // (the words of the second chunk follow those of the first)
          uint32_t* vw = reinterpret_cast<uint32_t*>(vh);
          *reinterpret_cast<uint2*>(vw + kv4_v_half(D, r, quad) / 2) =
              make_uint2(__byte_perm(codes[0], n0, 0x5410), __byte_perm(codes[1], n1, 0x5410));
          *reinterpret_cast<uint2*>(vw + kv4_v_half(D, r, quad + 1) / 2) =
              make_uint2(__byte_perm(codes[0], n0, 0x7632), __byte_perm(codes[1], n1, 0x7632));
        } else if (s.ok && !with_prev) {
          vh[kv4_v_half(D, r, quad)] = static_cast<uint16_t>(codes[0]);
          vh[kv4_v_half(D, r, quad + 1)] = static_cast<uint16_t>(codes[0] >> 16);
          vh[kv4_v_half(D, r, quad) + 2] = static_cast<uint16_t>(codes[1]);
          vh[kv4_v_half(D, r, quad + 1) + 2] = static_cast<uint16_t>(codes[1] >> 16);
        }
        store_pairs(unit, true, pair);
      }
    }
  }
}

// One head of a token at a time (two or four in flight measured no faster).  40 warps an
// SM: four sequences of 4096 keys of eight heads, d = 128, 18.6 us, 10000 keys 12.7; 48
// warps 19.6 and 14.3; 32 warps 18.5 and 13.7.
template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads, kGatherCtas) kv_gather4_kernel(const __grid_constant__ KvGatherParams p) {
  constexpr int LPT = D / 16, TPW = 32 / LPT;
  check_prefix(p.cu, p.b, p.total, p.status);
  const int lane = threadIdx.x & 31, k = lane % LPT;
  const unsigned w = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int parts = p.parts, part = static_cast<int>(w % parts);
  const unsigned tok_u = (w / parts) * TPW + lane / LPT;
  const int tok = static_cast<int>(min(tok_u, 0x7fffffffu));
  const Slot s = find_slot<LPT>(p.cu, p.b, p.total, p.seqlens, p.block_table, p.bt_stride, p.bt_width, p.page_size, p.num_pages, 0,
                                tok, p.status);
  if (!s.ok) return;
  const int ng = D / p.group, r = s.row % kKv4Unit, chunk = cache_chunk(k, 0);
  const int g0 = 8 * chunk / p.group, g1 = (8 * chunk + 32) / p.group;
  const uint8_t* base = p.cache + s.page * p.c_st[0] + static_cast<int64_t>(s.row / kKv4Unit) * kv4_unit_bytes(D, ng);
  const uint32_t mine = r % 2 != 0 ? 0x7632u : 0x5410u;  // the key's half of two words of V
  uint16_t* to[2] = {static_cast<uint16_t*>(p.k) + tok * p.k_st[0] + 8 * chunk,
                     static_cast<uint16_t*>(p.v) + tok * p.v_st[0] + 8 * chunk};
  for (int h = part; h < p.hkv; h += parts) {
    const uint8_t* unit = base + h * p.c_st[1];
    const uint32_t* vw = reinterpret_cast<const uint32_t*>(unit + 16 * D);
    const uint32_t* par = reinterpret_cast<const uint32_t*>(unit + 32 * D) + r * ng;
    const uint2 kw = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint32_t*>(unit) + kv4_k_word(D, r, chunk));
    const uint2 v0 = *reinterpret_cast<const uint2*>(vw + kv4_v_half(D, r, 2 * chunk) / 2);
    const uint2 v1 = *reinterpret_cast<const uint2*>(vw + kv4_v_half(D, r, 2 * chunk + 1) / 2);
    const uint32_t pair[2][2] = {{par[g0], par[g1]}, {par[32 * ng + g0], par[32 * ng + g1]}};
    const uint32_t codes[2][2] = {{kw.x, kw.y}, {__byte_perm(v0.x, v1.x, mine), __byte_perm(v0.y, v1.y, mine)}};
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      uint16_t* dst = to[kv] + h * (kv == 0 ? p.k_st[1] : p.v_st[1]);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float sc = widen1<BF16>(pair[kv][c] & 0xffffu), mn = widen1<BF16>(pair[kv][c] >> 16);
        const uint64_t s2 = pack2(sc, sc), m2 = pack2(mn, mn), off = pack2(-1024.f, -1024.f);
        // nibbles i and i + 4 of a word as the fp16 pair 1024 + code, then fp32; scale * code
        // is exact, so the fused sum is min + scale * code rounded once
        float f[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t two = ((codes[kv][c] >> (4 * i)) & 0x000f000fu) | 0x64006400u;
          const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&two));
          const float2 y = unpack2(fma2(s2, add2(pack2(x.x, x.y), off), m2));
          f[i] = y.x;
          f[i + 4] = y.y;
        }
        store_chunk(dst + 32 * c, Chunk{{narrow2<BF16>(f[0], f[1]), narrow2<BF16>(f[2], f[3]), narrow2<BF16>(f[4], f[5]),
                                         narrow2<BF16>(f[6], f[7])}});
      }
    }
  }
}

// Warps that share a token's rows (hq of one tensor, hkv of two more, `flight` at a time),
// and the blocks of the launch.  With n warps a token the launch takes
//   ceil(groups n / resident) + 0.25   waves of warps (the rest: its start and end)
//   of as many rows as a warp goes through, in whole flights, + 1.3 (the token's place and
//   angles) each;
// the n with the least of it is taken.  Measured at 500 to 45000 tokens with 1 to 48 warps a
// token, in three head layouts: 1 to 3% slower on average than the best n of each, where 32
// warps an SM whatever the tokens (the n that makes them) lose 8 to 15%.  32 / 8 heads of
// 128, 16-bit and 4-bit with the gather, us, that and this: 1000 tokens 7.0 and 6.0, 12.4
// and 10.6; 10000: 48.4 and 41.8, 61.7 and 54.5; four prompts of 4096: 65.3 and 62.5, 80.3
// and 79.6.
unsigned deal(int64_t total, int d, int hq, int hkv, int flight, int resident, int* parts) {
  const int64_t groups = (total * (d / 16) + 31) / 32;  // warps that hold the tokens once
  const int rows = hq + 2 * hkv;
  int64_t n = rows;
  if (groups * rows > resident) {
    const int64_t most = 5 * (resident / groups) + 5;  // (past five waves there is nothing to win)
    float best = INFINITY;
    for (int64_t k = 1; k <= most && k <= rows; ++k) {
      const int64_t waves = (groups * k + resident - 1) / resident, per = k * flight;
      const int64_t flights = (hq + per - 1) / per + 2 * ((hkv + per - 1) / per);
      const float cost = (static_cast<float>(waves) + 0.25f) * (static_cast<float>(flights * flight) + 1.3f);
      if (cost < best) {
        best = cost;
        n = k;
      }
    }
  }
  *parts = static_cast<int>(n);
  return static_cast<unsigned>((groups * n * 32 + kThreads - 1) / kThreads);
}

template <int D>
void launch_append_d(const KvAppendParams& p, int dtype, unsigned grid, cudaStream_t stream) {
  const bool i4 = p.group > 0;
  if (dtype == 0) {
    if (i4) kv_append_kernel<D, true, true><<<grid, kThreads, 0, stream>>>(p);
    else kv_append_kernel<D, true, false><<<grid, kThreads, 0, stream>>>(p);
  } else {
    if (i4) kv_append_kernel<D, false, true><<<grid, kThreads, 0, stream>>>(p);
    else kv_append_kernel<D, false, false><<<grid, kThreads, 0, stream>>>(p);
  }
}

}  // namespace

cudaError_t launch_kv_append(KvAppendParams& p, int dtype, int sms, cudaStream_t stream) {
  const unsigned grid = deal(p.total, p.d, p.hq, p.hkv, kFlight, kThreads / 32 * kAppendCtas * sms, &p.parts);
  if (p.d == 64) launch_append_d<64>(p, dtype, grid, stream);
  else if (p.d == 128) launch_append_d<128>(p, dtype, grid, stream);
  else launch_append_d<256>(p, dtype, grid, stream);
  return cudaGetLastError();
}

cudaError_t launch_kv_gather4(KvGatherParams& p, int dtype, int sms, cudaStream_t stream) {
  const unsigned grid = deal(p.total, p.d, p.hkv, 0, 1, kThreads / 32 * kGatherCtas * sms, &p.parts);
  if (dtype == 0) {
    if (p.d == 64) kv_gather4_kernel<64, true><<<grid, kThreads, 0, stream>>>(p);
    else if (p.d == 128) kv_gather4_kernel<128, true><<<grid, kThreads, 0, stream>>>(p);
    else kv_gather4_kernel<256, true><<<grid, kThreads, 0, stream>>>(p);
  } else {
    if (p.d == 64) kv_gather4_kernel<64, false><<<grid, kThreads, 0, stream>>>(p);
    else if (p.d == 128) kv_gather4_kernel<128, false><<<grid, kThreads, 0, stream>>>(p);
    else kv_gather4_kernel<256, false><<<grid, kThreads, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace fa
