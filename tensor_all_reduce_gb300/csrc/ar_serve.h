// Kernel parameters and entries of the attention block's operators (paged plan, per-head norm
// with rotation, paged attention), shared by their kernels and the C ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "ar.h"

namespace ar {

constexpr int kStatusBadIndex = 2;  // status word: an index in device memory was out of range

// Division by an invariant d of numerators below 2^31 (T. Granlund and P. Montgomery, "Division by
// invariant integers using multiplication", PLDI 1994): n / d = (hi(n m) + n) >> s.
struct FastDiv {
  uint32_t d, m;
  int s;
};

inline FastDiv fast_div(uint32_t d) {
  FastDiv f;
  f.d = d;
  f.s = 0;
  while (((uint64_t)1 << f.s) < d) ++f.s;
  f.m = (uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << f.s) - d)) / d + 1);
  return f;
}

struct PlanParams {
  int requests, page;
  int64_t max_tokens, free_capacity, table_cols, table_stride;
  const int32_t* cached;
  const int32_t* fresh;
  const int32_t* free_blocks;
  const int32_t* free_count;
  int32_t* table;
  int32_t* cu_q;
  int32_t* seq_lens;
  int64_t* slots;
  int32_t* positions;
  int32_t* free_count_out;
  int32_t* info;
  int* status;
};

struct HeadRows {  // [tokens, heads, head_dim] with unit last stride
  const void* in;
  void* out;  // NULL: not stored
  int64_t in_ts, in_hs, out_ts, out_hs;
  const void* weight;  // NULL: no norm
  int heads;
};

struct RopeParams {
  int64_t tokens;
  int head_dim;
  HeadRows q, k;
  const void* v;
  int64_t v_ts, v_hs;
  float eps, inv_dim;
  int gemma, half, pairs, axes, dealt;  // half: frequencies, rot_dim / 2
  FastDiv half_div;
  int sections[AR_MAX_ROPE_AXES];
  const int32_t* positions;
  int64_t pos_stride;
  const float* inv_freq;
  void* k_cache;
  void* v_cache;
  int64_t kc_bs, kc_ps, kc_hs, vc_bs, vc_ps, vc_hs;  // strides: block, token of a block, head
  int64_t num_slots;
  int page;
  const int64_t* slots;
  int* status;
  int stall;  // test hook: the first copy of the vector form is not issued, so that its wait runs out
  long long wait_cycles;
};

// Scales of a cache of E4M3 codes, one a block and head.
struct Scales {
  float* p;
  int64_t bs, hs;  // strides: block, head
};

// Scales outside this range count as its nearer end, NaN as the lower one.
constexpr float kScaleLow = 0x1p-32f, kScaleHigh = 0x1p32f;

struct AppendParams {
  int64_t tokens;
  int requests, heads, head_dim;
  const void* k;
  const void* v;
  int64_t k_ts, k_hs, v_ts, v_hs;
  const void* weight;  // of k; NULL: no norm
  float eps;
  int gemma, half, pairs, axes, dealt;  // half: frequencies, rot_dim / 2
  FastDiv half_div;
  int sections[AR_MAX_ROPE_AXES];
  const int32_t* positions;  // NULL: the token's place in its request
  int64_t pos_stride;
  const float* inv_freq;
  uint8_t* k_cache;
  uint8_t* v_cache;
  int64_t kc_bs, kc_ps, kc_hs, vc_bs, vc_ps, vc_hs;  // strides: block, token of a block, head
  int64_t num_blocks;
  FastDiv page;
  Scales k_scale, v_scale;
  const int32_t* table;
  int64_t table_stride;
  int max_len;  // tokens that a table row can name, at most 2^30
  const int32_t* cu_q;
  const int32_t* seq_lens;
  int* status;
};

struct AttnParams {
  int64_t tokens;
  int requests, q_heads, kv_heads, head_dim;
  FastDiv group;  // q heads of a key head
  const void* q;
  void* out;
  int64_t q_ts, q_hs, o_ts, o_hs;
  float* lse;
  const void* k;
  const void* v;
  int64_t k_bs, k_ps, k_hs, v_bs, v_ps, v_hs;
  Scales k_scale, v_scale;  // of a cache in 8 bits
  int64_t num_blocks;
  FastDiv page;
  const int32_t* table;
  int64_t table_stride;
  int max_len;  // keys that a table row can name, at most 2^30
  const int32_t* cu_q;
  const int32_t* seq_lens;
  float scale_log2;  // scale * log2(e)
  float cap_log2;    // cap * log2(e), 0: no cap
  float cap_inv;     // 1 / cap_log2
  float cap_twice;   // exponent (to the base 2) of e^2x, x = scale q.k / cap, a unit of q.k
  int causal, window;
  const float* slopes;
  const int32_t* prefix;
  int vec;  // 16-byte loads of q and the cache, 16-byte stores of out
  int wide;  // 32-byte stores of out and of partial rows (the tensor-core form)
  // workspace: the partial results of the spans that begin or end inside an item
  int spans, tile_rows, part_dim;  // CTAs, rows of an item, floats of a partial row
  int* headers;
  float* part_o;
  float* part_ml;
  int* status;
  // the tensor-core form
  int box_rows;  // keys of one copy: the largest power of two, at most 128, that divides the page
  int stall;     // test hook: the first copy is not issued, so that its wait runs out
  long long wait_cycles;
};

const void* plan_kernel();
struct RopePlan {  // how the vector form divides its work
  int step, split, per, heads;  // tokens of a unit; units that share a token's heads; heads of a unit, in all
  int pitch;                    // floats between the tokens of a unit's cosines and sines
  int row_bytes, stage_bytes;   // a unit's rows; with its angles
  FastDiv heads_div;            // by `per`
  int64_t units;
  unsigned ctas;
};

const void* rope_scalar_kernel(bool bf16);
const void* rope_vec_kernel(bool bf16, int head_dim, int half, bool pairs);
RopePlan rope_plan(const RopeParams& p, int sm_count);
size_t rope_smem(const RopePlan& plan);
size_t rope_smem_most();
struct AppendPlan {  // how the vector form divides its work
  int warps;         // of a task: the new keys or values of a head in a block
  int parts;         // units that share a block's heads
  int round_tokens;  // tokens whose angles are held at once
  int pitch;         // floats between their cosines
  unsigned ctas;
};

const void* append_scalar_kernel(bool bf16);
const void* append_vec_kernel(bool bf16, int head_dim, bool halves);  // halves: of a multiple of 4 (else adjacent pairs, or no rotation)
AppendPlan append_plan(const AppendParams& p, int sm_count);
size_t append_smem(const AppendPlan& plan);
size_t append_smem_most();
const void* attn_mma_kernel(bool bf16, int padded_dim, bool fp8 = false);  // fp8: a cache in 8 bits
const void* attn_combine_kernel(bool bf16);

// Dynamic shared memory of the general attention kernel: 64 query rows, keys and values each,
// padded by 16 bytes.
inline size_t attn_mma_smem(int padded_dim) { return (size_t)3 * 64 * (padded_dim + 8) * 2; }

const void* attn_tma_kernel(bool bf16, int padded_dim, float cap, bool bias);  // cap 0: none; bias: also a scale that is not positive
size_t attn_tma_smem(int padded_dim);
int attn_tma_rows(int padded_dim);  // query rows of an item

constexpr int kAttn8FewRows = 16, kAttn8FewThreads = 256;  // most rows of an item; two CTAs an SM
const void* attn8_few_kernel(bool bf16, int padded_dim, int rows);  // for few rows a request: items of 8 or 16
size_t attn8_few_smem(int padded_dim, int rows);
constexpr int kAttn8Threads = 512;  // the kernel's division of registers waits for as many
const void* attn8_tma_kernel(bool bf16, int padded_dim, bool few, float cap, bool bias);  // over a cache in 8 bits; few: items of 128 rows
size_t attn8_tma_smem();

// Tensor map of a cache [blocks, page, heads, dim] (strides in elements) with boxes of box_rows
// tokens by 128 bytes; `encode` is the driver's cuTensorMapEncodeTiled.
enum class CacheType { kF16, kBF16, kE4M3 };
bool attn_tensor_map(void* encode, CUtensorMap* map, const void* base, CacheType type, int64_t dim, int64_t page, int64_t heads, int64_t blocks,
                     int64_t page_stride, int64_t head_stride, int64_t block_stride, int box_rows);

// Function attributes, module loading and occupancies for all of the above, once per context.
cudaError_t serve_prepare(ar_ctx* ctx);

}  // namespace ar
