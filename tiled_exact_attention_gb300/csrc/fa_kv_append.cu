// Filling a paged cache: the rotary rotation of new queries and keys, the store of
// new keys and values into their pages (16-bit rows, or 4-bit codes with group
// scales), and the gather of 4-bit pages back into 16-bit rows.
//
// All of it is bound by HBM traffic for prompts and by latency for single tokens.  A
// lane keeps sixteen dims of one token, d / 16 lanes a token, and walks over the
// token's heads: the rotation's cosines and sines are read once per token and stay in
// registers, as does the token's place in the cache.  Several heads' rows are loaded
// before the first is used.  The heads of a token are dealt to as many warps as it
// takes to fill the GPU: one head each for a few tokens, all heads to a warp for
// prompts.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fa_kv4.h"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kThreads = 128;

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

// Sixteen dims of a row.
struct Row16 {
  uint4 a, b;
  __device__ __forceinline__ uint32_t word(int i) const {  // (i is a constant once unrolled)
    switch (i) {
      case 0: return a.x;
      case 1: return a.y;
      case 2: return a.z;
      case 3: return a.w;
      case 4: return b.x;
      case 5: return b.y;
      case 6: return b.z;
      default: return b.w;
    }
  }
};

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
                                          int64_t bt_stride, int page_size, int num_pages, int max_positions, int tok,
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
  if (pos >= bt_stride * page_size || (max_positions > 0 && pos >= max_positions)) {
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

// The rotation of a lane's sixteen dims (two chunks of eight).  Every pair of
// neighbouring dims becomes x * c + o * s with the dims o that they turn with (those of
// the chunk R / 2 away, or, interleaved, the same two exchanged) and the sign in s:
// each product and the sum rounded once (no contraction), as in the plain formula.
struct Turn {
  uint64_t c[8], s[8];
  bool on[2];     // the chunk is rotated
  int other[2];   // half-split: first dim of the chunk it turns with
};

template <bool BF16>
__device__ __forceinline__ Row16 turn(const Row16& x, const Row16& o, const Turn& t, bool interleaved) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    w[i] = x.word(i);
    if (t.on[i / 4]) {
      const uint64_t v = widen2<BF16>(w[i]);
      const float2 p = unpack2(v);
      const uint64_t u = interleaved ? pack2(p.y, p.x) : widen2<BF16>(o.word(i));
      const float2 y = unpack2(add2(mul2(v, t.c[i]), mul2(u, t.s[i])));
      w[i] = narrow2<BF16>(y.x, y.y);
    }
  }
  return Row16{make_uint4(w[0], w[1], w[2], w[3]), make_uint4(w[4], w[5], w[6], w[7])};
}

// Sixteen 16-bit values quantised with the other lanes of their group (group / 16
// lanes): codes (nibble i of a word: value i) and the (scale, min) pair as stored.
// The minimum is exact in the rows' type; the scale (max - min) / 15 is rounded to it
// (halved first, so that it cannot overflow).  Many 16-bit values lie exactly between
// two levels, so the quotient (x - min) / scale has to be the correctly rounded one:
// x times the reciprocal, then one correction by its exact remainder (Markstein).
// Codes are taken from the sum with 1.5 * 2^23, whose low bits are the nearest integer.
template <bool BF16>
__device__ __forceinline__ void quantise16(const Row16& x, int lanes, uint32_t (&codes)[2], uint32_t* pair) {
  // minimum of the values and of their negatives, two and two, then both in one word
  uint32_t mn = x.word(0), mx = x.word(0) ^ 0x80008000u;
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    mn = min2<BF16>(mn, x.word(i));
    mx = min2<BF16>(mx, x.word(i) ^ 0x80008000u);
  }
  uint32_t both = min2<BF16>(__byte_perm(mn, mx, 0x5410), __byte_perm(mn, mx, 0x7632));
  for (int s = 1; s < lanes; s *= 2) both = min2<BF16>(both, __shfl_xor_sync(0xffffffffu, both, s));
  const float low = widen1<BF16>(both & 0xffffu), neg_high = widen1<BF16>(both >> 16);
  const float half_range = __fsub_rn(-0.5f * neg_high, 0.5f * low);
  const float by = 0x1.111112p-3f;  // 1 / 7.5 to nearest
  float q = __fmul_rn(half_range, by);
  q = __fmaf_rn(__fmaf_rn(-7.5f, q, half_range), by, q);
  uint32_t sm = narrow2<BF16>(q, low);
  float s = widen1<BF16>(sm & 0xffffu);
  if (s < 0x1p-100f) {
    s = 0.f;
    sm &= 0xffff0000u;
  }
  *pair = sm;
  const float r = s > 0.f ? __frcp_rn(s) : 0.f;
  const uint64_t r2 = pack2(r, r), s2 = pack2(-s, -s), m2 = pack2(-low, -low);
  const uint64_t magic = pack2(12582912.f, 12582912.f);
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    uint32_t word = 0;
#pragma unroll
    for (int i = 3; i >= 0; --i) {
      const uint64_t a = add2(widen2<BF16>(x.word(4 * c + i)), m2);
      uint64_t y = mul2(a, r2);
      y = fma2(fma2(s2, y, a), r2, y);
      if (!BF16 && s < 0x1p-14f) {  // a subnormal scale may be far too small
        const float2 f = unpack2(y);
        y = pack2(fminf(f.x, 15.f), fminf(f.y, 15.f));
      }
      const float2 z = unpack2(add2(y, magic));  // bits 0x4b400000 + code
      word = (word << 4) + __float_as_uint(z.y);
      word = (word << 4) + __float_as_uint(z.x);
    }
    codes[c] = word - 0x3f400000u;  // the sum of 0x4b400000 << 4 i, i = 0..7
  }
}

template <int D, bool BF16, bool INT4>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const __grid_constant__ KvAppendParams p) {
  constexpr int LPT = D / 16, TPW = 32 / LPT;  // lanes of a token, tokens of a warp
  constexpr int U = 2;                         // rows in flight
  check_prefix(p.cu, p.b, p.total, p.status);
  const int lane = threadIdx.x & 31, k = lane % LPT;
  const unsigned w = (blockIdx.x * kThreads + threadIdx.x) >> 5;
  const int part = static_cast<int>(w % p.parts);  // this warp's heads: part, part + parts, ...
  const unsigned tok_u = (w / p.parts) * TPW + lane / LPT;
  const int tok = static_cast<int>(min(tok_u, 0x7fffffffu));
  const bool live = tok < p.total;
  const int heads = p.hq + 2 * p.hkv, turned = p.hq + p.hkv;

  auto row_of = [&](int h) {
    const uint16_t* x;
    if (h < p.hq) x = static_cast<const uint16_t*>(p.q) + tok * p.q_st[0] + h * p.q_st[1];
    else if (h < turned) x = static_cast<const uint16_t*>(p.k) + tok * p.k_st[0] + (h - p.hq) * p.k_st[1];
    else x = static_cast<const uint16_t*>(p.v) + tok * p.v_st[0] + (h - turned) * p.v_st[1];
    return x;
  };
  auto load16 = [&](const uint16_t* x) {
    return Row16{*reinterpret_cast<const uint4*>(x), *reinterpret_cast<const uint4*>(x + 8)};
  };

  // ---- what the chunks turn with (known before the place is)
  Turn t;
  const int half = p.rot / 2;
  const bool split = p.rot > 0 && !p.interleaved;
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int dim = 16 * k + 8 * c;
    t.on[c] = dim < p.rot;
    t.other[c] = !t.on[c] || !split ? dim : (dim < half ? dim + half : dim - half);
  }
  Row16 x[U], o[U];
  auto load_rows = [&](int h0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u * p.parts;
      if (live && h < heads) {
        const uint16_t* row = row_of(h);
        x[u] = load16(row + 16 * k);
        if (split && h < turned)
          o[u] = Row16{*reinterpret_cast<const uint4*>(row + t.other[0]), *reinterpret_cast<const uint4*>(row + t.other[1])};
      } else {
        x[u] = o[u] = Row16{make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
      }
    }
  };
  load_rows(part);
  const Slot s = find_slot<LPT>(p.cu, p.b, p.total, p.seqlens, p.block_table, p.bt_stride, p.page_size, p.num_pages,
                                p.rot > 0 ? p.max_positions : 0, tok, p.status);
  {
    const float* cs = p.cos_sin + static_cast<int64_t>(s.pos) * p.rot;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      t.c[i] = t.s[i] = 0;
      if (s.ok && t.on[i / 4]) {
        if (p.interleaved) {
          const int a = 8 * k + i;
          const float co = cs[a], si = cs[half + a];
          t.c[i] = pack2(co, co);
          t.s[i] = pack2(-si, si);
        } else {
          const int dim = 16 * k + 2 * i;
          const bool low = dim < half;
          const int a = low ? dim : dim - half;
          const float2 co = *reinterpret_cast<const float2*>(cs + a), si = *reinterpret_cast<const float2*>(cs + half + a);
          t.c[i] = pack2(co.x, co.y);
          t.s[i] = low ? pack2(-si.x, -si.y) : pack2(si.x, si.y);
        }
      }
    }
  }
  const int ng = INT4 ? D / p.group : 1;
  // 4-bit: a token and the one after it, both in this warp, share V's words if they
  // are an even and an odd key of one sequence's page
  const int r = s.row % kKv4Unit;
  bool with_next = false, with_prev = false;
  if constexpr (INT4) {
    const int np = __shfl_down_sync(0xffffffffu, s.ok ? s.page : -1, LPT), nr = __shfl_down_sync(0xffffffffu, s.row, LPT);
    with_next = s.ok && lane < 32 - LPT && s.row % 2 == 0 && np == s.page && nr == s.row + 1;
    const int up = __shfl_up_sync(0xffffffffu, with_next ? 1 : 0, LPT);
    with_prev = lane >= LPT && up != 0;
  }

  for (int h0 = part; h0 < heads; h0 += U * p.parts) {
    if (h0 != part) load_rows(h0);
    __syncwarp();  // (q_out may be q: a row is read before any lane writes it)
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u * p.parts;
      if (h >= heads) break;
      const bool is_q = h < p.hq, is_k = !is_q && h < turned;
      const Row16 y = (is_q || is_k) && p.rot > 0 ? turn<BF16>(x[u], o[u], t, p.interleaved != 0) : x[u];
      if (is_q) {
        if (s.ok) {
          uint16_t* dst = static_cast<uint16_t*>(p.q_out) + tok * p.qo_st[0] + h * p.qo_st[1] + 16 * k;
          *reinterpret_cast<uint4*>(dst) = y.a;
          *reinterpret_cast<uint4*>(dst + 8) = y.b;
        }
        continue;
      }
      const int kvh = is_k ? h - p.hq : h - turned;
      if constexpr (!INT4) {
        if (s.ok) {
          uint16_t* dst = is_k ? static_cast<uint16_t*>(p.k_cache) + s.page * p.kc_st[0] + s.row * p.kc_st[1] + kvh * p.kc_st[2]
                               : static_cast<uint16_t*>(p.v_cache) + s.page * p.vc_st[0] + s.row * p.vc_st[1] + kvh * p.vc_st[2];
          *reinterpret_cast<uint4*>(dst + 16 * k) = y.a;
          *reinterpret_cast<uint4*>(dst + 16 * k + 8) = y.b;
        }
      } else {
        uint32_t codes[2], pair;
        quantise16<BF16>(y, p.group / 16, codes, &pair);
        uint8_t* unit = p.cache + s.page * p.c_st[0] + kvh * p.c_st[1] +
                        static_cast<int64_t>(s.row / kKv4Unit) * kv4_unit_bytes(D, ng);
        if (is_k) {
          if (s.ok) {
            uint32_t* kw = reinterpret_cast<uint32_t*>(unit);
            kw[kv4_k_word(D, r, 2 * k)] = codes[0];
            kw[kv4_k_word(D, r, 2 * k + 1)] = codes[1];
          }
        } else {
          const uint32_t n0 = __shfl_down_sync(0xffffffffu, codes[0], LPT), n1 = __shfl_down_sync(0xffffffffu, codes[1], LPT);
          uint16_t* vh = reinterpret_cast<uint16_t*>(unit + 16 * D);
          if (with_next) {
            uint32_t* vw = reinterpret_cast<uint32_t*>(vh);
            vw[kv4_v_half(D, r, 4 * k) / 2] = __byte_perm(codes[0], n0, 0x5410);
            vw[kv4_v_half(D, r, 4 * k + 1) / 2] = __byte_perm(codes[0], n0, 0x7632);
            vw[kv4_v_half(D, r, 4 * k + 2) / 2] = __byte_perm(codes[1], n1, 0x5410);
            vw[kv4_v_half(D, r, 4 * k + 3) / 2] = __byte_perm(codes[1], n1, 0x7632);
          } else if (s.ok && !with_prev) {
            vh[kv4_v_half(D, r, 4 * k)] = static_cast<uint16_t>(codes[0]);
            vh[kv4_v_half(D, r, 4 * k + 1)] = static_cast<uint16_t>(codes[0] >> 16);
            vh[kv4_v_half(D, r, 4 * k + 2)] = static_cast<uint16_t>(codes[1]);
            vh[kv4_v_half(D, r, 4 * k + 3)] = static_cast<uint16_t>(codes[1] >> 16);
          }
        }
        if (s.ok && k % (p.group / 16) == 0)
          reinterpret_cast<uint32_t*>(unit + 32 * D)[(is_k ? 0 : 32 * ng) + r * ng + 16 * k / p.group] = pair;
      }
    }
  }
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads) kv_gather4_kernel(const __grid_constant__ KvGatherParams p) {
  constexpr int LPT = D / 16, TPW = 32 / LPT;
  constexpr int U = 2;
  check_prefix(p.cu, p.b, p.total, p.status);
  const int lane = threadIdx.x & 31, k = lane % LPT;
  const unsigned w = (blockIdx.x * kThreads + threadIdx.x) >> 5;
  const int part = static_cast<int>(w % p.parts);
  const unsigned tok_u = (w / p.parts) * TPW + lane / LPT;
  const int tok = static_cast<int>(min(tok_u, 0x7fffffffu));
  const Slot s = find_slot<LPT>(p.cu, p.b, p.total, p.seqlens, p.block_table, p.bt_stride, p.page_size, p.num_pages, 0,
                                tok, p.status);
  if (!s.ok) return;
  const int ng = D / p.group, r = s.row % kKv4Unit;
  const uint8_t* base = p.cache + s.page * p.c_st[0] + static_cast<int64_t>(s.row / kKv4Unit) * kv4_unit_bytes(D, ng);
  const uint32_t high = r % 2 != 0 ? 0x7632u : 0x5410u;  // the key's half of two words of V
  for (int h0 = part; h0 < p.hkv; h0 += U * p.parts) {
    uint32_t codes[U][2][2], pair[U][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u * p.parts;
      if (h >= p.hkv) break;
      const uint8_t* unit = base + h * p.c_st[1];
      const uint32_t* kw = reinterpret_cast<const uint32_t*>(unit);
      const uint32_t* vw = reinterpret_cast<const uint32_t*>(unit + 16 * D);
      const uint32_t* par = reinterpret_cast<const uint32_t*>(unit + 32 * D) + r * ng + 16 * k / p.group;
      codes[u][0][0] = kw[kv4_k_word(D, r, 2 * k)];
      codes[u][0][1] = kw[kv4_k_word(D, r, 2 * k + 1)];
      pair[u][0] = par[0];
      pair[u][1] = par[32 * ng];
#pragma unroll
      for (int c = 0; c < 2; ++c)
        codes[u][1][c] = __byte_perm(vw[kv4_v_half(D, r, 4 * k + 2 * c) / 2], vw[kv4_v_half(D, r, 4 * k + 2 * c + 1) / 2], high);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u * p.parts;
      if (h >= p.hkv) break;
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const float sc = widen1<BF16>(pair[u][kv] & 0xffffu), mn = widen1<BF16>(pair[u][kv] >> 16);
        uint32_t out[8];
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            // (scale * code is exact, so the fused sum is min + scale * code rounded once)
            const uint32_t two = codes[u][kv][c] >> (8 * i);
            const float a = static_cast<float>(two & 15u), b = static_cast<float>((two >> 4) & 15u);
            out[4 * c + i] = narrow2<BF16>(__fmaf_rn(sc, a, mn), __fmaf_rn(sc, b, mn));
          }
        uint16_t* dst = (kv == 0 ? static_cast<uint16_t*>(p.k) + tok * p.k_st[0] + h * p.k_st[1]
                                 : static_cast<uint16_t*>(p.v) + tok * p.v_st[0] + h * p.v_st[1]) + 16 * k;
        *reinterpret_cast<uint4*>(dst) = make_uint4(out[0], out[1], out[2], out[3]);
        *reinterpret_cast<uint4*>(dst + 8) = make_uint4(out[4], out[5], out[6], out[7]);
      }
    }
  }
}

// Warps that share a token's rows, and the blocks of the launch: as many warps as keep
// every SM busy (32 each), at least two rows a warp where there are that many tokens.
unsigned deal(int64_t total, int rows, int d, int sms, int* parts) {
  const int64_t groups = (total * (d / 16) + 31) / 32;  // warps that hold the tokens once
  int64_t n = (static_cast<int64_t>(sms) * 32 + groups - 1) / groups;
  if (n > rows) n = rows;
  if (n < 1) n = 1;
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
  const unsigned grid = deal(p.total, p.hq + 2 * p.hkv, p.d, sms, &p.parts);
  if (p.d == 64) launch_append_d<64>(p, dtype, grid, stream);
  else if (p.d == 128) launch_append_d<128>(p, dtype, grid, stream);
  else launch_append_d<256>(p, dtype, grid, stream);
  return cudaGetLastError();
}

cudaError_t launch_kv_gather4(KvGatherParams& p, int dtype, int sms, cudaStream_t stream) {
  const unsigned grid = deal(p.total, p.hkv, p.d, sms, &p.parts);
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
