// Filling a paged cache: the rotary rotation of new queries and keys, the store of
// new keys and values into their pages (16-bit rows, or 4-bit codes with group
// scales), and the gather of 4-bit pages back into 16-bit rows.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fa_kv4.h"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kThreads = 256;

// Eight 16-bit values <-> fp32.
template <bool BF16>
__device__ __forceinline__ void widen8(const uint4& u, float* f) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BF16) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    } else {
      const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      f[2 * i] = x.x;
      f[2 * i + 1] = x.y;
    }
  }
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
__device__ __forceinline__ uint4 narrow8(const float* f) {
  return make_uint4(narrow2<BF16>(f[0], f[1]), narrow2<BF16>(f[2], f[3]), narrow2<BF16>(f[4], f[5]),
                    narrow2<BF16>(f[6], f[7]));
}

// One 16-bit value to fp32.
template <bool BF16>
__device__ __forceinline__ float widen1(uint32_t h) {
  if constexpr (BF16) return __uint_as_float(h << 16);
  return __half2float(__ushort_as_half(static_cast<unsigned short>(h)));
}

// Where new token `tok` goes: its sequence, position, page and row.
struct Slot {
  int seq, pos, page, row;
};

// False: the token has no place (a padding token, or an argument that fails its check).
__device__ __forceinline__ bool find_slot(const int* cu, int b, int total, const int* seqlens, const int* table,
                                          int64_t bt_stride, int page_size, int num_pages, int max_positions, int tok,
                                          int* status, Slot* s) {
  int seq, first, n;
  if (cu == nullptr) {
    n = total / b;
    seq = tok / n;
    first = seq * n;
  } else {
    int lo = 0, hi = b;  // the last sequence that starts at or before tok
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (cu[mid] <= tok) lo = mid; else hi = mid;
    }
    seq = lo;
    first = cu[lo];
    const int end = cu[lo + 1];
    if (first > tok || end <= tok) return false;  // a row of no sequence
    n = end - first;
  }
  const int64_t pos = static_cast<int64_t>(seqlens[seq]) - n + (tok - first);
  if (pos < 0) return false;  // padding before the sequence's first key
  if (pos >= bt_stride * page_size || (max_positions > 0 && pos >= max_positions)) {
    record_error(status, kErrDeviceArg);
    return false;
  }
  s->seq = seq;
  s->pos = static_cast<int>(pos);
  s->page = table[seq * bt_stride + pos / page_size];
  s->row = static_cast<int>(pos % page_size);
  if (s->page < 0 || s->page >= num_pages) {
    record_error(status, kErrDeviceArg);
    return false;
  }
  return true;
}

// The prefix sums are checked once per launch, by the first block.
__device__ __forceinline__ void check_prefix(const int* cu, int b, int total, int* status) {
  if (cu == nullptr || blockIdx.x != 0) return;
  bool ok = cu[0] >= 0 && cu[b] <= total;
  for (int i = threadIdx.x; i < b; i += blockDim.x) ok = ok && cu[i] <= cu[i + 1];
  if (!ok) record_error(status, kErrDeviceArg);
}

// Rotation of the eight dims [8 c, 8 c + 8) of a row at x, products and sums rounded
// one by one in fp32 (no contraction, so that the result does not depend on how it
// is compiled), then once to the row's type.
template <bool BF16>
__device__ __forceinline__ uint4 rotate8(const uint16_t* x, int c, const float* cs, int rot, int interleaved) {
  const uint4 own = *reinterpret_cast<const uint4*>(x + 8 * c);
  if (8 * c >= rot) return own;
  float f[8], y[8];
  widen8<BF16>(own, f);
  const int half = rot / 2;
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float co = cs[4 * c + i], si = cs[half + 4 * c + i];
      y[2 * i] = __fsub_rn(__fmul_rn(f[2 * i], co), __fmul_rn(f[2 * i + 1], si));
      y[2 * i + 1] = __fadd_rn(__fmul_rn(f[2 * i + 1], co), __fmul_rn(f[2 * i], si));
    }
  } else {
    const bool low = 8 * c < half;
    const int a = low ? 8 * c : 8 * c - half;  // angle of the first dim
    float o[8];
    widen8<BF16>(*reinterpret_cast<const uint4*>(x + (low ? 8 * c + half : 8 * c - half)), o);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float co = cs[a + i], si = cs[half + a + i];
      y[i] = low ? __fsub_rn(__fmul_rn(f[i], co), __fmul_rn(o[i], si))
                 : __fadd_rn(__fmul_rn(f[i], co), __fmul_rn(o[i], si));
    }
  }
  return narrow8<BF16>(y);
}

// Eight 16-bit values of a row quantised with the other lanes of their group: the
// codes (nibble i = value i) and the (scale, min) pair as stored.  The rows' minimum
// is exact in their type; the scale (max - min) / 15 is rounded to it (halved first,
// so that it cannot overflow); a code is the nearest level, the quotient being the
// IEEE one (many 16-bit values lie exactly between two levels).
template <bool BF16>
__device__ __forceinline__ uint32_t quantise8(const uint4& u, int group_lanes, uint32_t* pair) {
  float f[8];
  widen8<BF16>(u, f);
  float mn = f[0], mx = f[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    mn = fminf(mn, f[i]);
    mx = fmaxf(mx, f[i]);
  }
  for (int x = 1; x < group_lanes; x *= 2) {
    mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, x));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
  }
  const uint32_t sm = narrow2<BF16>(__fdiv_rn(__fsub_rn(0.5f * mx, 0.5f * mn), 7.5f), mn);
  float s = widen1<BF16>(sm & 0xffffu);
  if (s < 0x1p-100f) s = 0.f;
  *pair = s > 0.f ? sm : sm & 0xffff0000u;
  uint32_t codes = 0;
  if (s > 0.f) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      codes |= static_cast<uint32_t>(fminf(rintf(__fdiv_rn(__fsub_rn(f[i], mn), s)), 15.f)) << (4 * i);
  }
  return codes;
}

// One thread per (token, head row, eight dims); consecutive lanes hold a row.
template <bool BF16, bool INT4>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const __grid_constant__ KvAppendParams p) {
  check_prefix(p.cu, p.b, p.total, p.status);
  const int lpr = p.d / 8, heads = p.hq + 2 * p.hkv;
  const int64_t idx = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t row = idx / lpr;
  const int c = static_cast<int>(idx % lpr);
  const bool live = row < static_cast<int64_t>(p.total) * heads;
  const int tok = live ? static_cast<int>(row / heads) : 0, h = live ? static_cast<int>(row % heads) : 0;
  Slot s;
  const bool ok = live && find_slot(p.cu, p.b, p.total, p.seqlens, p.block_table, p.bt_stride, p.page_size,
                                    p.num_pages, p.rot > 0 ? p.max_positions : 0, tok, p.status, &s);
  const bool is_q = h < p.hq, is_k = !is_q && h < p.hq + p.hkv;
  const int kvh = is_q ? 0 : (is_k ? h - p.hq : h - p.hq - p.hkv);
  uint4 x = make_uint4(0u, 0u, 0u, 0u);
  if (ok) {
    if (is_q || is_k) {
      const uint16_t* src = is_q ? static_cast<const uint16_t*>(p.q) + tok * p.q_st[0] + h * p.q_st[1]
                                 : static_cast<const uint16_t*>(p.k) + tok * p.k_st[0] + kvh * p.k_st[1];
      x = rotate8<BF16>(src, c, p.cos_sin + static_cast<int64_t>(s.pos) * p.rot, p.rot, p.interleaved);
    } else {
      x = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.v) + tok * p.v_st[0] + kvh * p.v_st[1] +
                                          8 * c);
    }
  }
  __syncwarp();  // (q_out may be q: a row's lanes have read it before any of them writes it)
  uint32_t codes = 0, pair = 0;
  if constexpr (INT4) codes = quantise8<BF16>(x, p.group / 8, &pair);
  if (!ok) return;
  if (is_q) {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.q_out) + tok * p.qo_st[0] + h * p.qo_st[1] + 8 * c) = x;
  } else if constexpr (!INT4) {
    uint16_t* dst = is_k ? static_cast<uint16_t*>(p.k_cache) + s.page * p.kc_st[0] + s.row * p.kc_st[1] + kvh * p.kc_st[2]
                         : static_cast<uint16_t*>(p.v_cache) + s.page * p.vc_st[0] + s.row * p.vc_st[1] + kvh * p.vc_st[2];
    *reinterpret_cast<uint4*>(dst + 8 * c) = x;
  } else {
    const int ng = p.d / p.group, r = s.row % kKv4Unit;
    uint8_t* unit = p.cache + s.page * p.c_st[0] + kvh * p.c_st[1] +
                    static_cast<int64_t>(s.row / kKv4Unit) * kv4_unit_bytes(p.d, ng);
    if (is_k) {
      reinterpret_cast<uint32_t*>(unit)[kv4_k_word(p.d, r, c)] = codes;
    } else {
      uint16_t* vh = reinterpret_cast<uint16_t*>(unit + 16 * p.d);
      vh[kv4_v_half(p.d, r, 2 * c)] = static_cast<uint16_t>(codes);
      vh[kv4_v_half(p.d, r, 2 * c + 1)] = static_cast<uint16_t>(codes >> 16);
    }
    if (c % (p.group / 8) == 0)
      reinterpret_cast<uint32_t*>(unit + 32 * p.d)[(is_k ? 0 : 32 * ng) + r * ng + 8 * c / p.group] = pair;
  }
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads) kv_gather4_kernel(const __grid_constant__ KvGatherParams p) {
  check_prefix(p.cu, p.b, p.total, p.status);
  const int lpr = p.d / 8, ng = p.d / p.group;
  const int64_t idx = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t row = idx / lpr;
  const int c = static_cast<int>(idx % lpr);
  if (row >= static_cast<int64_t>(p.total) * p.hkv) return;
  const int tok = static_cast<int>(row / p.hkv), h = static_cast<int>(row % p.hkv);
  Slot s;
  if (!find_slot(p.cu, p.b, p.total, p.seqlens, p.block_table, p.bt_stride, p.page_size, p.num_pages, 0, tok, p.status,
                 &s))
    return;
  const int r = s.row % kKv4Unit;
  const uint8_t* unit = p.cache + s.page * p.c_st[0] + h * p.c_st[1] +
                        static_cast<int64_t>(s.row / kKv4Unit) * kv4_unit_bytes(p.d, ng);
  const uint16_t* vh = reinterpret_cast<const uint16_t*>(unit + 16 * p.d);
  const uint32_t codes[2] = {reinterpret_cast<const uint32_t*>(unit)[kv4_k_word(p.d, r, c)],
                             static_cast<uint32_t>(vh[kv4_v_half(p.d, r, 2 * c)]) |
                                 static_cast<uint32_t>(vh[kv4_v_half(p.d, r, 2 * c + 1)]) << 16};
  const uint32_t* par = reinterpret_cast<const uint32_t*>(unit + 32 * p.d) + r * ng + 8 * c / p.group;
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    const uint32_t sm = par[kv * 32 * ng];
    const float sc = widen1<BF16>(sm & 0xffffu), mn = widen1<BF16>(sm >> 16);
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      f[i] = __fadd_rn(mn, __fmul_rn(sc, static_cast<float>((codes[kv] >> (4 * i)) & 15u)));
    uint16_t* dst = kv == 0 ? static_cast<uint16_t*>(p.k) + tok * p.k_st[0] + h * p.k_st[1]
                            : static_cast<uint16_t*>(p.v) + tok * p.v_st[0] + h * p.v_st[1];
    *reinterpret_cast<uint4*>(dst + 8 * c) = narrow8<BF16>(f);
  }
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendParams& p, int dtype, cudaStream_t stream) {
  const int64_t threads = static_cast<int64_t>(p.total) * (p.hq + 2 * p.hkv) * (p.d / 8);
  const unsigned grid = static_cast<unsigned>((threads + kThreads - 1) / kThreads);
  const bool i4 = p.group > 0;
  if (dtype == 0) {
    if (i4) kv_append_kernel<true, true><<<grid, kThreads, 0, stream>>>(p);
    else kv_append_kernel<true, false><<<grid, kThreads, 0, stream>>>(p);
  } else {
    if (i4) kv_append_kernel<false, true><<<grid, kThreads, 0, stream>>>(p);
    else kv_append_kernel<false, false><<<grid, kThreads, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

cudaError_t launch_kv_gather4(const KvGatherParams& p, int dtype, cudaStream_t stream) {
  const int64_t threads = static_cast<int64_t>(p.total) * p.hkv * (p.d / 8);
  const unsigned grid = static_cast<unsigned>((threads + kThreads - 1) / kThreads);
  if (dtype == 0) kv_gather4_kernel<true><<<grid, kThreads, 0, stream>>>(p);
  else kv_gather4_kernel<false><<<grid, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace fa
