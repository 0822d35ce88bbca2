// Internal declarations of the paged cache's operators: the rotary append, the
// 4-bit cache's layout, its gather and the attention over it.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace fa {

// Status word and SM count of the current device (defined in fa_api.cu).
bool current_device_info(int** status, int* sms);

// ---------------------------------------------------------------------------
// The 4-bit cache.  Per page and KV head: page_size / 32 units of 32 keys, each
// unit  [K codes 16 d][V codes 16 d][K parameters][V parameters]  bytes, the
// parameters 32 x ng pairs (scale, min) of the cache's 16-bit type, ng = d / group.
// A 32-bit word holds eight codes.  The orders below are the ones in which the
// lanes of a warp hold the A operand of an m16n8k16 MMA (lane = 4 g + t), so that
// the attention kernel's shared-memory reads are contiguous over a warp:
//   K: a word is eight consecutive dims of one key: dim = 32 (J c + j) + 8 t + n,
//      nibble n, at word ((32 c + key) * 4 + t) * J + j;
//   V: a word is four consecutive dims of two consecutive keys (low half: the even
//      one): dim = 32 (J c + j) + 4 g + n, key = 16 a + 8 h + 2 t + parity, at word
//      ((((2 a + h) * C + c) * 8 + g) * 4 + t) * J + j.
// J = min(d / 32, 4) words of a lane per read, C = d / (32 J).
// ---------------------------------------------------------------------------
constexpr int kKv4Unit = 32;  // keys per unit

__host__ __device__ constexpr int kv4_j(int d) { return d >= 128 ? 4 : d / 32; }
__host__ __device__ constexpr int kv4_unit_bytes(int d, int ng) { return kKv4Unit * (d + 8 * ng); }

// Word of K dims [8 chunk, 8 chunk + 8) of key r (< 32).
__host__ __device__ constexpr int kv4_k_word(int d, int r, int chunk) {
  const int j = chunk / 4, t = chunk % 4, J = kv4_j(d);
  return ((32 * (j / J) + r) * 4 + t) * J + j % J;
}

// Half word (16 bits) of V dims [4 quad, 4 quad + 4) of key r (< 32).
__host__ __device__ constexpr int kv4_v_half(int d, int r, int quad) {
  const int i = quad / 8, g = quad % 8, J = kv4_j(d), C = d / 32 / J;
  const int word = ((((r / 8) * C + i / J) * 8 + g) * 4 + (r % 8) / 2) * J + i % J;
  return 2 * word + r % 2;
}

// New tokens into a paged cache (16-bit: group = 0, k_cache / v_cache; 4-bit: cache).
struct KvAppendParams {
  const void* q;  // [total][hq][d] (hq = 0: none), strides (row, head) in elements
  void* q_out;
  const void* k;
  const void* v;
  int64_t q_st[2], qo_st[2], k_st[2], v_st[2];
  int b, total, hq, hkv, d;
  int parts;          // warps that share a token's rows
  const int* cu;      // [b + 1], or null: total / b tokens each
  const int* seqlens;  // [b] keys after the append
  const float* cos_sin;  // [max_positions][rot]: rot / 2 cosines, rot / 2 sines
  int rot, max_positions, interleaved;
  void* k_cache;
  void* v_cache;
  int64_t kc_st[3], vc_st[3];  // (page, row, head) in elements
  uint8_t* cache;
  int64_t c_st[2];  // (page, head) in bytes
  int group;
  int num_pages, page_size;
  const int* block_table;
  int64_t bt_stride, bt_width;
  int* status;
};

// The last n_b positions of each sequence of a 4-bit cache, as 16-bit rows.
struct KvGatherParams {
  const uint8_t* cache;
  int64_t c_st[2];
  int b, total, hkv, d, group, num_pages, page_size;
  int parts;  // warps that share a token's heads
  const int* block_table;
  int64_t bt_stride, bt_width;
  const int* seqlens;
  const int* cu;
  void* k;
  void* v;
  int64_t k_st[2], v_st[2];
  int* status;
};

// sq query tokens per sequence against a 4-bit cache.
struct Attend4Params {
  const void* q;  // [b][sq][hq][d]
  void* o;
  float* lse;     // [b][hq][sq]
  int64_t q_st[3], o_st[3];  // (batch, row, head) in elements
  int b, sq, hq, hkv, g, d, group;
  int g_shift, page_shift;  // log2 of g and of page_size, -1 where they are no powers of two
  int ntiles;     // row tiles of a KV head: ceil(sq * g / rows of a tile)
  int grid;       // CTAs
  int cuts;       // 0: no item can be long enough to be cut
  const uint8_t* cache;
  int64_t c_st[2];
  int num_pages, page_size;
  const int* block_table;
  int64_t bt_stride, bt_width;
  const int* seqlens;
  int window_left;   // -1: no left edge
  float scale_log2;  // scale * log2(e)
  float sc_k, sc_b;  // softcap as in DecodeParams (sc_b = 0: off)
  // Partials of items that several CTAs share, two slots a CTA: O before the division
  // [2 grid][rows][d], its maximum and sum [2 grid][rows]; counters [grid], zeroed by
  // the launch, one for the item that starts in a CTA's stretch and leaves it.
  float* part_o;
  float2* part_ml;
  int* counters;
  int* status;
};

// The kernel a call takes: query rows of a tile, keys of a block, blocks that an item costs
// besides its own, blocks of an item that is never cut, CTAs of a full grid.
struct Attend4Plan {
  int rows, block, gap, uncut, max_ctas;
};

// dtype 0 = bf16, 1 = fp16.
cudaError_t launch_kv_append(KvAppendParams& p, int dtype, int sms, cudaStream_t stream);  // (sets p.parts)
cudaError_t launch_kv_gather4(KvGatherParams& p, int dtype, int sms, cudaStream_t stream);
// With a plan: fill it from p.group, p.sq and p.g and launch nothing.
cudaError_t attend4_d64(const Attend4Params& p, int dtype, int sms, Attend4Plan* plan, cudaStream_t stream);
cudaError_t attend4_d128(const Attend4Params& p, int dtype, int sms, Attend4Plan* plan, cudaStream_t stream);
cudaError_t attend4_d256(const Attend4Params& p, int dtype, int sms, Attend4Plan* plan, cudaStream_t stream);

}  // namespace fa
