// Host side of the paged cache's entry points (include/fa.h): argument validation
// and launches.  Nothing is allocated here.
#include <cmath>
#include <cstdint>
#include <cstring>

#include "fa.h"
#include "fa_kv4.h"

namespace fa {
namespace {

bool is_aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// Strides in elements of a 16-bit tensor: positive multiples of 8.
bool strides8(const int64_t* s, int n) {
  for (int i = 0; i < n; ++i)
    if (s[i] <= 0 || s[i] % 8 != 0 || s[i] >= (static_cast<int64_t>(1) << 39)) return false;
  return true;
}

bool strides16b(const int64_t* s, int n) {
  for (int i = 0; i < n; ++i)
    if (s[i] <= 0 || s[i] % 16 != 0 || s[i] >= (static_cast<int64_t>(1) << 40)) return false;
  return true;
}

bool head_dim_ok(int d) { return d == 64 || d == 128 || d == 256; }
bool group_ok(int group, int d) { return (group == 32 || group == 64 || group == 128) && group <= d; }

// The block table and lengths of a paged cache.
fa_status validate_pages(int num_pages, int page_size, const int32_t* table, int table_stride, int table_width,
                         const int32_t* seqlens) {
  if (num_pages < 1 || page_size < 1 || table == nullptr || seqlens == nullptr || table_stride < 0 || table_width < 1)
    return FA_ERR_INVALID_ARG;
  if (page_size % 64 != 0) return FA_ERR_UNSUPPORTED;
  if (!is_aligned(table, 4) || !is_aligned(seqlens, 4)) return FA_ERR_INVALID_ARG;
  return FA_OK;
}

fa_status validate_cache4(const void* cache, const int64_t strides[2], int page_size, int d, int group) {
  if (!group_ok(group, d)) return FA_ERR_UNSUPPORTED;
  if (cache == nullptr || !is_aligned(cache, 16) || !strides16b(strides, 2)) return FA_ERR_INVALID_ARG;
  if (strides[1] < static_cast<int64_t>(page_size / kKv4Unit) * kv4_unit_bytes(d, d / group))
    return FA_ERR_INVALID_ARG;
  return FA_OK;
}

fa_status validate_append(const fa_kv_append_args* a, bool int4) {
  if (a == nullptr) return FA_ERR_INVALID_ARG;
  if (a->dtype != FA_BF16 && a->dtype != FA_FP16) return FA_ERR_INVALID_ARG;
  if (a->b < 1 || a->total < 0 || a->hq < 0 || a->hkv < 1) return FA_ERR_INVALID_ARG;
  if (a->interleaved != 0 && a->interleaved != 1) return FA_ERR_INVALID_ARG;
  if (!head_dim_ok(a->d)) return FA_ERR_UNSUPPORTED;
  if (a->total > (1 << 30) || a->hq > (1 << 16) || a->hkv > (1 << 16)) return FA_ERR_UNSUPPORTED;
  if (a->rotary_dim < 0 || a->rotary_dim > a->d) return FA_ERR_INVALID_ARG;
  if (a->rotary_dim > 0) {
    // whole eight-dim chunks: of both halves, or of pairs
    if (a->rotary_dim % (a->interleaved ? 8 : 16) != 0) return FA_ERR_UNSUPPORTED;
    if (a->cos_sin == nullptr || !is_aligned(a->cos_sin, 16) || a->max_positions < 1) return FA_ERR_INVALID_ARG;
  }
  const fa_status v = validate_pages(a->num_pages, a->page_size, a->block_table, a->block_table_stride, a->block_table_width,
                                     a->seqlens_k);
  if (v != FA_OK) return v;
  if (a->cu_seqlens == nullptr ? a->total % a->b != 0 : !is_aligned(a->cu_seqlens, 4)) return FA_ERR_INVALID_ARG;
  if (int4) {
    const fa_status c = validate_cache4(a->cache, a->cache_strides, a->page_size, a->d, a->group);
    if (c != FA_OK) return c;
  } else {
    if (a->k_cache == nullptr || a->v_cache == nullptr || !is_aligned(a->k_cache, 16) || !is_aligned(a->v_cache, 16))
      return FA_ERR_INVALID_ARG;
    if (!strides8(a->k_cache_strides, 3) || !strides8(a->v_cache_strides, 3)) return FA_ERR_INVALID_ARG;
  }
  if (a->total == 0) return FA_OK;
  if (a->k == nullptr || a->v == nullptr || !is_aligned(a->k, 16) || !is_aligned(a->v, 16)) return FA_ERR_INVALID_ARG;
  if (!strides8(a->k_strides, 2) || !strides8(a->v_strides, 2)) return FA_ERR_INVALID_ARG;
  if (a->hq > 0) {
    if (a->q == nullptr || a->q_out == nullptr || !is_aligned(a->q, 16) || !is_aligned(a->q_out, 16))
      return FA_ERR_INVALID_ARG;
    if (!strides8(a->q_strides, 2) || !strides8(a->q_out_strides, 2)) return FA_ERR_INVALID_ARG;
  }
  return FA_OK;
}

fa_status append(const fa_kv_append_args* a, bool int4, void* stream) {
  const fa_status v = validate_append(a, int4);
  if (v != FA_OK || a->total == 0) return v;
  KvAppendParams p;
  std::memset(&p, 0, sizeof(p));
  int sms = 0;
  if (!current_device_info(&p.status, &sms)) return FA_ERR_CUDA;
  p.q = a->q;
  p.q_out = a->q_out;
  p.k = a->k;
  p.v = a->v;
  for (int i = 0; i < 2; ++i) {
    p.q_st[i] = a->q_strides[i];
    p.qo_st[i] = a->q_out_strides[i];
    p.k_st[i] = a->k_strides[i];
    p.v_st[i] = a->v_strides[i];
    p.c_st[i] = a->cache_strides[i];
  }
  for (int i = 0; i < 3; ++i) {
    p.kc_st[i] = a->k_cache_strides[i];
    p.vc_st[i] = a->v_cache_strides[i];
  }
  p.b = a->b;
  p.total = a->total;
  p.hq = a->hq;
  p.hkv = a->hkv;
  p.d = a->d;
  p.cu = a->cu_seqlens;
  p.seqlens = a->seqlens_k;
  p.cos_sin = a->cos_sin;
  p.rot = a->rotary_dim;
  p.max_positions = a->max_positions;
  p.interleaved = a->interleaved;
  p.k_cache = a->k_cache;
  p.v_cache = a->v_cache;
  p.cache = static_cast<uint8_t*>(a->cache);
  p.group = int4 ? a->group : 0;
  p.num_pages = a->num_pages;
  p.page_size = a->page_size;
  p.block_table = a->block_table;
  p.bt_stride = a->block_table_stride;
  p.bt_width = a->block_table_width;
  return launch_kv_append(p, a->dtype, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status validate_attend(const fa_kvcache_int4_args* a) {
  if (a == nullptr) return FA_ERR_INVALID_ARG;
  if (a->dtype != FA_BF16 && a->dtype != FA_FP16) return FA_ERR_INVALID_ARG;
  if (a->b < 1 || a->sq < 0 || a->hq < 1 || a->hkv < 1 || a->hq % a->hkv != 0) return FA_ERR_INVALID_ARG;
  if (!(a->scale > 0.f) || !std::isfinite(a->scale)) return FA_ERR_INVALID_ARG;
  if (!(a->softcap == 0.f || (a->softcap > 0.f && std::isfinite(a->softcap)))) return FA_ERR_INVALID_ARG;
  if ((a->local != 0 && a->local != 1) || (a->local && a->window_left < -1)) return FA_ERR_INVALID_ARG;
  if (!head_dim_ok(a->d)) return FA_ERR_UNSUPPORTED;
  if (a->b > 65535 || static_cast<int64_t>(a->sq) * (a->hq / a->hkv) > 65536) return FA_ERR_UNSUPPORTED;
  const fa_status v = validate_pages(a->num_pages, a->page_size, a->block_table, a->block_table_stride, a->block_table_width,
                                     a->seqlens_k);
  if (v != FA_OK) return v;
  const fa_status c = validate_cache4(a->cache, a->cache_strides, a->page_size, a->d, a->group);
  if (c != FA_OK) return c;
  if (a->sq == 0) return FA_OK;
  if (a->q == nullptr || a->o == nullptr || a->lse == nullptr) return FA_ERR_INVALID_ARG;
  if (!is_aligned(a->q, 16) || !is_aligned(a->o, 16) || !is_aligned(a->lse, 4)) return FA_ERR_INVALID_ARG;
  if (!strides8(a->q_strides, 3) || !strides8(a->o_strides, 3)) return FA_ERR_INVALID_ARG;
  return FA_OK;
}

cudaError_t attend(const Attend4Params& p, int dtype, int sms, Attend4Plan* plan, cudaStream_t stream) {
  if (p.d == 64) return attend4_d64(p, dtype, sms, plan, stream);
  if (p.d == 128) return attend4_d128(p, dtype, sms, plan, stream);
  return attend4_d256(p, dtype, sms, plan, stream);
}

// log2 of a power of two, -1 of another number.
int shift_of(int x) {
  for (int i = 0; i < 31; ++i)
    if (x == 1 << i) return i;
  return -1;
}

size_t round256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// The kernel for a call, its grid and the sizes of its workspace's three parts.
struct AttendWork {
  Attend4Plan plan;
  int ntiles, grid;
  size_t o_bytes, ml_bytes, bytes;
};

bool plan_attend(const fa_kvcache_int4_args* a, int sms, AttendWork* w) {
  Attend4Params p;
  std::memset(&p, 0, sizeof(p));
  p.d = a->d;
  p.group = a->group;
  p.sq = a->sq;
  p.g = a->hq / a->hkv;
  if (attend(p, a->dtype, sms, &w->plan, nullptr) != cudaSuccess) return false;
  const int64_t rows = static_cast<int64_t>(a->sq) * p.g;
  w->ntiles = static_cast<int>((rows + w->plan.rows - 1) / w->plan.rows);
  // no more CTAs than blocks there could be (a block table's row is the longest sequence)
  const double blocks = static_cast<double>(a->b) * a->hkv * w->ntiles *
                        (static_cast<double>(a->block_table_width) * a->page_size / w->plan.block + 1.0 + w->plan.gap);
  w->grid = blocks < w->plan.max_ctas ? static_cast<int>(blocks) : w->plan.max_ctas;
  if (w->grid < 1) w->grid = 1;
  if (blocks > 2e9) return false;  // (counted in 32 bits: 2^36 keys over all KV heads and row tiles)
  w->o_bytes = round256(static_cast<size_t>(2) * w->grid * w->plan.rows * a->d * sizeof(float));
  w->ml_bytes = round256(static_cast<size_t>(2) * w->grid * w->plan.rows * sizeof(float2));
  w->bytes = w->o_bytes + w->ml_bytes + round256(static_cast<size_t>(w->grid) * sizeof(int));
  return true;
}

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" {

size_t fa_kvcache_int4_page_bytes(int32_t page_size, int32_t d, int32_t group) {
  if (page_size < 64 || page_size % 64 != 0 || !head_dim_ok(d) || !group_ok(group, d)) return 0;
  return static_cast<size_t>(page_size / kKv4Unit) * kv4_unit_bytes(d, d / group);
}

fa_status fa_kv_append(const fa_kv_append_args* a, void* stream) { return append(a, false, stream); }

fa_status fa_kv_append_int4(const fa_kv_append_args* a, void* stream) { return append(a, true, stream); }

fa_status fa_kv_gather_int4(const fa_kv_gather_int4_args* a, void* stream) {
  if (a == nullptr) return FA_ERR_INVALID_ARG;
  if (a->dtype != FA_BF16 && a->dtype != FA_FP16) return FA_ERR_INVALID_ARG;
  if (a->b < 1 || a->total < 0 || a->hkv < 1) return FA_ERR_INVALID_ARG;
  if (!head_dim_ok(a->d)) return FA_ERR_UNSUPPORTED;
  if (a->total > (1 << 30) || a->hkv > (1 << 16)) return FA_ERR_UNSUPPORTED;
  const fa_status v = validate_pages(a->num_pages, a->page_size, a->block_table, a->block_table_stride, a->block_table_width,
                                     a->seqlens_k);
  if (v != FA_OK) return v;
  const fa_status c = validate_cache4(a->cache, a->cache_strides, a->page_size, a->d, a->group);
  if (c != FA_OK) return c;
  if (a->cu_seqlens == nullptr ? a->total % a->b != 0 : !is_aligned(a->cu_seqlens, 4)) return FA_ERR_INVALID_ARG;
  if (a->total == 0) return FA_OK;
  if (a->k == nullptr || a->v == nullptr || !is_aligned(a->k, 16) || !is_aligned(a->v, 16)) return FA_ERR_INVALID_ARG;
  if (!strides8(a->k_strides, 2) || !strides8(a->v_strides, 2)) return FA_ERR_INVALID_ARG;
  KvGatherParams p;
  std::memset(&p, 0, sizeof(p));
  int sms = 0;
  if (!current_device_info(&p.status, &sms)) return FA_ERR_CUDA;
  p.cache = static_cast<const uint8_t*>(a->cache);
  for (int i = 0; i < 2; ++i) {
    p.c_st[i] = a->cache_strides[i];
    p.k_st[i] = a->k_strides[i];
    p.v_st[i] = a->v_strides[i];
  }
  p.b = a->b;
  p.total = a->total;
  p.hkv = a->hkv;
  p.d = a->d;
  p.group = a->group;
  p.num_pages = a->num_pages;
  p.page_size = a->page_size;
  p.block_table = a->block_table;
  p.bt_stride = a->block_table_stride;
  p.bt_width = a->block_table_width;
  p.seqlens = a->seqlens_k;
  p.cu = a->cu_seqlens;
  p.k = a->k;
  p.v = a->v;
  return launch_kv_gather4(p, a->dtype, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

size_t fa_kvcache_int4_workspace_size(const fa_kvcache_int4_args* a) {
  if (validate_attend(a) != FA_OK) return 0;
  if (a->sq == 0) return 256;
  int* status = nullptr;
  int sms = 0;
  AttendWork w;
  if (!current_device_info(&status, &sms) || !plan_attend(a, sms, &w)) return 0;
  return w.bytes;
}

fa_status fa_fwd_kvcache_int4(const fa_kvcache_int4_args* a, void* workspace, size_t workspace_bytes, void* stream) {
  const fa_status v = validate_attend(a);
  if (v != FA_OK || a->sq == 0) return v;
  Attend4Params p;
  std::memset(&p, 0, sizeof(p));
  int sms = 0;
  AttendWork w;
  if (!current_device_info(&p.status, &sms)) return FA_ERR_CUDA;
  if (!plan_attend(a, sms, &w)) return FA_ERR_UNSUPPORTED;
  if (workspace == nullptr || workspace_bytes < w.bytes || !is_aligned(workspace, 256)) return FA_ERR_INVALID_ARG;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.part_o = reinterpret_cast<float*>(ws);
  p.part_ml = reinterpret_cast<float2*>(ws + w.o_bytes);
  p.counters = reinterpret_cast<int*>(ws + w.o_bytes + w.ml_bytes);
  p.ntiles = w.ntiles;
  p.g_shift = shift_of(a->hq / a->hkv);
  p.page_shift = shift_of(a->page_size);
  p.grid = w.grid;
  p.q = a->q;
  p.o = a->o;
  p.lse = a->lse;
  for (int i = 0; i < 3; ++i) {
    p.q_st[i] = a->q_strides[i];
    p.o_st[i] = a->o_strides[i];
  }
  p.b = a->b;
  p.sq = a->sq;
  p.hq = a->hq;
  p.hkv = a->hkv;
  p.g = a->hq / a->hkv;
  p.d = a->d;
  p.group = a->group;
  p.cache = static_cast<const uint8_t*>(a->cache);
  p.c_st[0] = a->cache_strides[0];
  p.c_st[1] = a->cache_strides[1];
  p.num_pages = a->num_pages;
  p.page_size = a->page_size;
  p.block_table = a->block_table;
  p.bt_stride = a->block_table_stride;
  p.bt_width = a->block_table_width;
  p.seqlens = a->seqlens_k;
  // (no sequence has more than 2^30 keys)
  p.window_left = !a->local ? -1 : a->window_left < (1 << 30) ? a->window_left : 1 << 30;
  p.scale_log2 = static_cast<float>(static_cast<double>(a->scale) * 1.4426950408889634);
  if (a->softcap > 0.f) {
    // scores arrive times scale log2(e): tanh(s / c) = 1 - 2 / (2^(sc_k x) + 1), sc_b = c log2(e)
    p.sc_k = static_cast<float>(2.0 / static_cast<double>(a->softcap));
    p.sc_b = static_cast<float>(static_cast<double>(a->softcap) * 1.4426950408889634);
  }
  p.cuts = static_cast<int64_t>(a->block_table_width) * a->page_size > static_cast<int64_t>(w.plan.uncut) * w.plan.block;
  return attend(p, a->dtype, sms, nullptr, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // extern "C"
