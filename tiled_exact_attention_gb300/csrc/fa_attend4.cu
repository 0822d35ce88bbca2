// Attention of one or a few query tokens per sequence over a paged 4-bit cache.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fa_kv4.h"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kWarps = 4;
constexpr float kLn2f = 0.69314718055994530942f;

template <bool BF16>
__device__ __forceinline__ float widen(uint32_t h) {
  if constexpr (BF16) return __uint_as_float(h << 16);
  return __half2float(__ushort_as_half(static_cast<unsigned short>(h)));
}

// One block per (query head, query token, sequence); d / 8 lanes take one key at a
// time, each eight dims, and keep a running (m, l, o) merged at the end.
template <int D, bool BF16>
__global__ void __launch_bounds__(kWarps * 32) attend4_kernel(const __grid_constant__ Attend4Params p) {
  constexpr int LPR = D / 8, RPW = 32 / LPR, ROWS = kWarps * RPW;
  __shared__ float sm_m[ROWS], sm_l[ROWS], sm_o[ROWS][D];
  const int h = blockIdx.x, i = blockIdx.y, bi = blockIdx.z, kvh = h / p.g;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = lane % LPR, sub = warp * RPW + lane / LPR;
  const int ng = D / p.group, unit_bytes = kv4_unit_bytes(D, ng);
  int64_t len = p.seqlens[bi];
  if (len > p.bt_stride * p.page_size) {
    if (threadIdx.x == 0 && h == 0 && i == 0) record_error(p.status, kErrDeviceArg);
    len = 0;
  }
  const int64_t at = len - p.sq + i;  // the query's position
  const int64_t first = p.window_left >= 0 && at > p.window_left ? at - p.window_left : 0;
  float q[8], o[8], m = -INFINITY, l = 0.f;
  const uint16_t* qp = static_cast<const uint16_t*>(p.q) + bi * p.q_st[0] + i * p.q_st[1] + h * p.q_st[2] + 8 * c;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    q[e] = widen<BF16>(qp[e]);
    o[e] = 0.f;
  }
  for (int64_t base = first; base <= at; base += ROWS) {
    const int64_t key = base + sub;
    bool ok = key <= at;
    int page = 0;
    if (ok) {
      page = p.block_table[bi * p.bt_stride + key / p.page_size];
      if (page < 0 || page >= p.num_pages) {
        record_error(p.status, kErrDeviceArg);
        ok = false;
      }
    }
    float s = 0.f, v[8];
    if (ok) {
      const int row = static_cast<int>(key % p.page_size), r = row % kKv4Unit;
      const uint8_t* unit = p.cache + page * p.c_st[0] + kvh * p.c_st[1] + static_cast<int64_t>(row / kKv4Unit) * unit_bytes;
      const uint16_t* vh = reinterpret_cast<const uint16_t*>(unit + 16 * D);
      const uint32_t* par = reinterpret_cast<const uint32_t*>(unit + 32 * D) + r * ng + 8 * c / p.group;
      const uint32_t kw = reinterpret_cast<const uint32_t*>(unit)[kv4_k_word(D, r, c)];
      const uint32_t vw = static_cast<uint32_t>(vh[kv4_v_half(D, r, 2 * c)]) |
                          static_cast<uint32_t>(vh[kv4_v_half(D, r, 2 * c + 1)]) << 16;
      const uint32_t kp = par[0], vp = par[32 * ng];
      const float ks = widen<BF16>(kp & 0xffffu), km = widen<BF16>(kp >> 16);
      const float vs = widen<BF16>(vp & 0xffffu), vm = widen<BF16>(vp >> 16);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        s = fmaf(q[e], fmaf(ks, static_cast<float>((kw >> (4 * e)) & 15u), km), s);
        v[e] = fmaf(vs, static_cast<float>((vw >> (4 * e)) & 15u), vm);
      }
    }
#pragma unroll
    for (int x = 1; x < LPR; x *= 2) s += __shfl_xor_sync(0xffffffffu, s, x);
    if (ok) {
      s *= p.scale_log2;
      if (p.sc_b > 0.f) s = p.sc_b * tanh_from_exp2_arg(p.sc_k * s);
      const float mn = fmaxf(m, s), a = ex2_approx(m - mn), w = ex2_approx(s - mn);
      l = fmaf(l, a, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = fmaf(o[e], a, w * v[e]);
      m = mn;
    }
  }
  if (c == 0) {
    sm_m[sub] = m;
    sm_l[sub] = l;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) sm_o[sub][8 * c + e] = o[e];
  __syncthreads();
  float M = -INFINITY, L = 0.f;
  for (int r = 0; r < ROWS; ++r) M = fmaxf(M, sm_m[r]);
  for (int r = 0; r < ROWS; ++r) L += sm_l[r] > 0.f ? sm_l[r] * ex2_approx(sm_m[r] - M) : 0.f;
  const float inv = L > 0.f ? 1.f / L : 0.f;
  uint16_t* op = static_cast<uint16_t*>(p.o) + bi * p.o_st[0] + i * p.o_st[1] + h * p.o_st[2];
  for (int e = threadIdx.x; e < D; e += kWarps * 32) {
    float x = 0.f;
    for (int r = 0; r < ROWS; ++r)
      if (sm_l[r] > 0.f) x = fmaf(sm_o[r][e], ex2_approx(sm_m[r] - M), x);
    x *= inv;
    if constexpr (BF16) op[e] = __bfloat16_as_ushort(__float2bfloat16_rn(x));
    else op[e] = __half_as_ushort(__float2half_rn(x));
  }
  if (threadIdx.x == 0)
    p.lse[(static_cast<int64_t>(bi) * p.hq + h) * p.sq + i] = L > 0.f ? (M + lg2_approx(L)) * kLn2f : -INFINITY;
}

template <bool BF16>
void launch_d(const Attend4Params& p, cudaStream_t stream) {
  const dim3 grid(p.hq, p.sq, p.b);
  if (p.d == 64) attend4_kernel<64, BF16><<<grid, kWarps * 32, 0, stream>>>(p);
  else if (p.d == 128) attend4_kernel<128, BF16><<<grid, kWarps * 32, 0, stream>>>(p);
  else attend4_kernel<256, BF16><<<grid, kWarps * 32, 0, stream>>>(p);
}

}  // namespace

cudaError_t launch_attend4(const Attend4Params& p, int dtype, cudaStream_t stream) {
  if (dtype == 0) launch_d<true>(p, stream);
  else launch_d<false>(p, stream);
  return cudaGetLastError();
}

}  // namespace fa
