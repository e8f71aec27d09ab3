// C ABI of the attention block's operators: argument validation, choice of the kernel, launch.
//
// As in ar_api.cu, validation precedes any use of the context, and nothing here allocates or
// synchronises.
#include <math.h>
#include <string.h>

#include "ar.h"
#include "ar_common.cuh"
#include "ar_ctx.h"
#include "ar_launch.h"
#include "ar_serve.h"

namespace {

constexpr int64_t kMaxRows = (int64_t)1 << 30;

// A strided array: runs of `run` bytes in up to three dimensions, `stride` bytes apart.
struct Extent {
  const void* p;
  int64_t run;
  int64_t stride[3], count[3];
  bool empty() const { return !p || run <= 0 || count[0] <= 0 || count[1] <= 0 || count[2] <= 0; }
  // Bytes from the first to the last one of the dimensions that are not whole multiples of s apart (s 0: of all).
  int64_t bytes(int64_t s = 0) const {
    int64_t n = run;
    for (int i = 0; i < 3; ++i)
      if (count[i] > 1 && (s == 0 || stride[i] % s)) n += (count[i] - 1) * stride[i];
    return n;
  }
};

Extent flat(const void* p, int64_t bytes) { return {p, bytes, {0, 0, 0}, {1, 1, 1}}; }

Extent table(const void* p, int64_t run, int64_t stride, int64_t rows) { return {p, run, {0, 0, stride}, {1, 1, rows}}; }

// Whether two arrays share a byte.  They may lie between each other's runs (q, k and v of a packed projection,
// side by side in a token or in a head; k and v of one cache tensor, side by side in a block, a token or a
// head): that is so where, modulo one of the strides, the two keep to parts that do not meet.
bool overlap(const Extent& a, const Extent& b) {
  if (a.empty() || b.empty()) return false;
  if (!overlaps(a.p, a.bytes(), b.p, b.bytes())) return false;
  for (int i = 0; i < 6; ++i) {
    const Extent& e = i < 3 ? a : b;
    const int64_t s = e.stride[i % 3];
    if (e.count[i % 3] < 2 || s <= 0) continue;
    int64_t d = (int64_t)(addr(b.p) - addr(a.p)) % s;  // b's start after a's
    if (d < 0) d += s;
    if (d >= a.bytes(s) && d + b.bytes(s) <= s) return false;
  }
  return true;
}

struct Operands {
  Extent in[24], out[8];
  int ni = 0, no = 0;
  void read(const Extent& e) { if (!e.empty()) in[ni++] = e; }
  void write(const Extent& e) { if (!e.empty()) out[no++] = e; }
  // `alias[o]`: index + 1 of the input that output o is exactly
  bool ok(const int* alias = nullptr) const {
    for (int o = 0; o < no; ++o) {
      for (int i = 0; i < ni; ++i)
        if (!(alias && alias[o] == i + 1) && overlap(out[o], in[i])) return false;
      for (int q = o + 1; q < no; ++q)
        if (overlap(out[o], out[q])) return false;
    }
    return true;
  }
};

// Non-negative strides of [outer, inner, dim] that keep rows and heads apart.
bool strides_ok(int64_t outer, int64_t os, int64_t inner, int64_t is, int64_t dim) {
  constexpr int64_t most = (int64_t)1 << 40;
  if (os < 0 || is < 0 || os > most || is > most) return false;
  if (inner > 1 && is < dim) return false;
  if (outer > 1 && os < dim) return false;
  return true;
}

// Steps of whole eights of elements (or other units); a single one has no step.
bool eights(int64_t stride, int64_t count, int unit = 8) { return count < 2 || stride % unit == 0; }

Extent cache_extent(const void* p, int64_t d, int64_t heads, int64_t hs, int64_t page, int64_t ps, int64_t blocks, int64_t bs) {
  return {p, d * 2, {hs * 2, ps * 2, bs * 2}, {heads, page, blocks}};
}

}  // namespace

extern "C" {

ar_status ar_paged_plan(ar_ctx* ctx, const ar_paged_plan_args* a, void* stream) {
  if (!a) return AR_ERR_INVALID_ARG;
  const int64_t i31 = 0x7fffffff;
  if (a->requests < 0 || a->requests > AR_MAX_REQUESTS || a->page_size < 1 || a->page_size > 65536 || a->max_tokens < 0 ||
      a->max_tokens > kMaxRows || a->free_capacity < 0 || a->free_capacity > i31 || a->table_cols < 0 || a->table_cols > i31 ||
      a->table_stride < 0 || (a->table_stride && a->table_stride < a->table_cols) || a->table_stride > ((int64_t)1 << 40))
    return AR_ERR_INVALID_ARG;
  const int64_t ts = a->table_stride ? a->table_stride : a->table_cols;
  const int64_t r = a->requests;
  if (!a->cu_q || !a->free_count || !a->free_count_out || !a->info || (a->free_capacity && !a->free_blocks) ||
      (a->max_tokens && (!a->slots || !a->positions)) ||
      (r && (!a->cached_lens || !a->new_lens || !a->seq_lens || (a->table_cols && !a->block_table))))
    return AR_ERR_INVALID_ARG;
  if (!aligned(a->cached_lens, 4) || !aligned(a->new_lens, 4) || !aligned(a->free_blocks, 4) || !aligned(a->free_count, 4) ||
      !aligned(a->block_table, 4) || !aligned(a->cu_q, 4) || !aligned(a->seq_lens, 4) || !aligned(a->slots, 8) ||
      !aligned(a->positions, 4) || !aligned(a->free_count_out, 4) || !aligned(a->info, 4))
    return AR_ERR_ALIGNMENT;
  Operands c;
  c.read(flat(a->cached_lens, r * 4));
  c.read(flat(a->new_lens, r * 4));
  c.read(flat(a->free_blocks, a->free_capacity * 4));
  c.read(flat(a->free_count, 4));
  c.write(table(a->block_table, a->table_cols * 4, ts * 4, r));
  c.write(flat(a->cu_q, (r + 1) * 4));
  c.write(flat(a->seq_lens, r * 4));
  c.write(flat(a->slots, a->max_tokens * 8));
  c.write(flat(a->positions, a->max_tokens * 4));
  c.write(flat(a->free_count_out, 4));
  c.write(flat(a->info, 16));
  if (!c.ok()) return AR_ERR_OVERLAP;
  if (!ctx) return AR_ERR_NOT_INITIALIZED;
  if (ctx->serve_error) return fail_cuda(ctx, ctx->serve_error, "the attention block's kernels");

  ar::PlanParams p;
  p.requests = a->requests;
  p.page = a->page_size;
  p.max_tokens = a->max_tokens;
  p.free_capacity = a->free_capacity;
  p.table_cols = a->table_cols;
  p.table_stride = ts;
  p.cached = a->cached_lens;
  p.fresh = a->new_lens;
  p.free_blocks = a->free_blocks;
  p.free_count = a->free_count;
  p.table = a->block_table;
  p.cu_q = a->cu_q;
  p.seq_lens = a->seq_lens;
  p.slots = a->slots;
  p.positions = a->positions;
  p.free_count_out = a->free_count_out;
  p.info = a->info;
  p.status = ctx->d_status;
  // a CTA for every 512 tokens, one an SM at most
  int64_t grid = (a->max_tokens + 511) / 512;
  if (grid > ctx->sm_count) grid = ctx->sm_count;
  if (grid < 1) grid = 1;
  DeviceGuard g(ctx->device);
  void* args[1] = {&p};
  const ar_status st = launch(ctx, ar::plan_kernel(), (unsigned)grid, 512, 1, args, (size_t)(r ? r : 1) * 8, stream);
  if (st == AR_OK) ctx->last_variant = "paged_plan";
  return st;
}

ar_status ar_qk_norm_rope(ar_ctx* ctx, const ar_qk_norm_rope_args* a, void* stream) {
  if (!a) return AR_ERR_INVALID_ARG;
  const bool cache = a->k_cache || a->v_cache;
  if (a->tokens < 0 || a->q_heads < 0 || a->kv_heads < 0 || a->q_heads + (int64_t)a->kv_heads < 1 || a->q_heads > 65536 ||
      a->kv_heads > 65536 || a->head_dim < 1 || a->head_dim > AR_MAX_HEAD_DIM || a->tokens > kMaxRows ||
      (a->dtype != AR_DTYPE_BF16 && a->dtype != AR_DTYPE_F16))
    return AR_ERR_INVALID_ARG;
  if (!(a->eps >= 0.0f) || isinf(a->eps)) return AR_ERR_INVALID_ARG;
  if (a->rot_dim < 0 || a->rot_dim > a->head_dim || (a->rot_dim & 1)) return AR_ERR_INVALID_ARG;
  const int half = a->rot_dim / 2;
  if (half) {
    if (a->axes < 1 || a->axes > AR_MAX_ROPE_AXES || a->position_stride < 0 ||
        (a->position_stride && a->axes > 1 && a->position_stride < a->tokens) || a->position_stride > ((int64_t)1 << 40))
      return AR_ERR_INVALID_ARG;
    if (a->axes > 1) {
      int sum = 0;
      for (int i = 0; i < a->axes; ++i) {
        if (a->sections[i] < 0 || a->sections[i] > half) return AR_ERR_INVALID_ARG;
        sum += a->sections[i];
      }
      if (sum != half) return AR_ERR_INVALID_ARG;
    }
  }
  const int64_t n = a->tokens, d = a->head_dim, hq = a->q_heads, hk = a->kv_heads;
  if (cache && (!a->k_cache || !a->v_cache || !hk || a->num_blocks < 0 || a->page_size < 1 || a->page_size > 65536 ||
                a->num_blocks > ((int64_t)1 << 40) / a->page_size))
    return AR_ERR_INVALID_ARG;
  if (n == 0) {
    if (!ctx) return AR_ERR_NOT_INITIALIZED;
    ctx->last_variant = "none";
    return AR_OK;
  }
  if ((hq && (!a->q || !a->q_out)) || (hk && (!a->k || (!a->k_out && !cache))) || (half && (!a->positions || !a->inv_freq)) ||
      (cache && (!a->v || !a->slots)))
    return AR_ERR_INVALID_ARG;
  const bool k_out = hk && a->k_out;
  if ((hq && (!strides_ok(n, a->q_token_stride, hq, a->q_head_stride, d) || !strides_ok(n, a->q_out_token_stride, hq, a->q_out_head_stride, d))) ||
      (hk && !strides_ok(n, a->k_token_stride, hk, a->k_head_stride, d)) ||
      (k_out && !strides_ok(n, a->k_out_token_stride, hk, a->k_out_head_stride, d)) ||
      (cache && (!strides_ok(n, a->v_token_stride, hk, a->v_head_stride, d) ||
                 !strides_ok(a->num_blocks, a->k_block_stride, a->page_size, a->k_page_stride, d) ||
                 !strides_ok(a->num_blocks, a->v_block_stride, a->page_size, a->v_page_stride, d) ||
                 !strides_ok(1, 0, hk, a->k_cache_head_stride, d) || !strides_ok(1, 0, hk, a->v_cache_head_stride, d))))
    return AR_ERR_INVALID_ARG;
  const void* two[] = {hq ? a->q : nullptr, hq ? a->q_out : nullptr, hk ? a->k : nullptr, k_out ? a->k_out : nullptr, a->q_weight, a->k_weight,
                       cache ? a->v : nullptr, a->k_cache, a->v_cache};
  for (const void* x : two)
    if (!aligned(x, 2)) return AR_ERR_ALIGNMENT;
  if ((half && (!aligned(a->positions, 4) || !aligned(a->inv_freq, 4))) || (cache && !aligned(a->slots, 8))) return AR_ERR_ALIGNMENT;

  Operands c;
  int alias[4] = {0, 0, 0, 0};
  auto heads = [&](const void* p, int64_t ts, int64_t h, int64_t hs) { return Extent{p, d * 2, {hs * 2, 0, ts * 2}, {h, 1, n}}; };
  if (hq) c.read(heads(a->q, a->q_token_stride, hq, a->q_head_stride));
  const int qi = c.ni;
  if (hk) c.read(heads(a->k, a->k_token_stride, hk, a->k_head_stride));
  const int ki = c.ni;
  if (cache) c.read(heads(a->v, a->v_token_stride, hk, a->v_head_stride));
  if (hq) c.read(flat(a->q_weight, d * 2));
  if (hk) c.read(flat(a->k_weight, d * 2));
  if (half) {
    const int64_t ps = a->position_stride ? a->position_stride : n;
    c.read(table(a->positions, n * 4, ps * 4, a->axes));
    c.read(flat(a->inv_freq, half * 4));
  }
  if (cache) c.read(flat(a->slots, n * 8));
  if (hq) {
    if (a->q_out == a->q && a->q_out_token_stride == a->q_token_stride && a->q_out_head_stride == a->q_head_stride) alias[c.no] = qi;
    c.write(heads(a->q_out, a->q_out_token_stride, hq, a->q_out_head_stride));
  }
  if (k_out) {
    if (a->k_out == a->k && a->k_out_token_stride == a->k_token_stride && a->k_out_head_stride == a->k_head_stride) alias[c.no] = ki;
    c.write(heads(a->k_out, a->k_out_token_stride, hk, a->k_out_head_stride));
  }
  if (cache && a->num_blocks) {
    const int64_t pg = a->page_size;
    c.write(cache_extent(a->k_cache, d, hk, a->k_cache_head_stride, pg, a->k_page_stride, a->num_blocks, a->k_block_stride));
    c.write(cache_extent(a->v_cache, d, hk, a->v_cache_head_stride, pg, a->v_page_stride, a->num_blocks, a->v_block_stride));
  }
  if (!c.ok(alias)) return AR_ERR_OVERLAP;
  if (!ctx) return AR_ERR_NOT_INITIALIZED;
  if (ctx->serve_error) return fail_cuda(ctx, ctx->serve_error, "the attention block's kernels");

  ar::RopeParams p;
  memset(&p, 0, sizeof(p));
  p.tokens = n;
  p.head_dim = a->head_dim;
  p.q = {a->q, hq ? a->q_out : nullptr, a->q_token_stride, a->q_head_stride, a->q_out_token_stride, a->q_out_head_stride, a->q_weight, a->q_heads};
  p.k = {a->k, k_out ? a->k_out : nullptr, a->k_token_stride, a->k_head_stride, a->k_out_token_stride, a->k_out_head_stride, a->k_weight, a->kv_heads};
  p.v = a->v;
  p.v_ts = a->v_token_stride;
  p.v_hs = a->v_head_stride;
  p.eps = a->eps;
  p.inv_dim = (float)(1.0 / (double)d);
  p.gemma = a->gemma != 0;
  p.half = half;
  p.half_div = ar::fast_div(half ? (uint32_t)half : 1);
  p.pairs = a->pairs != 0;
  p.axes = half ? a->axes : 1;
  p.dealt = a->dealt != 0;
  for (int i = 0; i < AR_MAX_ROPE_AXES; ++i) p.sections[i] = i < p.axes ? a->sections[i] : 0;
  p.positions = a->positions;
  p.pos_stride = a->position_stride ? a->position_stride : n;
  p.inv_freq = a->inv_freq;
  p.k_cache = a->k_cache;
  p.v_cache = a->v_cache;
  p.kc_bs = a->k_block_stride;
  p.kc_ps = a->k_page_stride;
  p.kc_hs = a->k_cache_head_stride;
  p.vc_bs = a->v_block_stride;
  p.vc_ps = a->v_page_stride;
  p.vc_hs = a->v_cache_head_stride;
  p.page = cache ? a->page_size : 1;
  p.num_slots = cache ? a->num_blocks * a->page_size : 0;
  p.slots = a->slots;
  p.status = ctx->d_status;
  p.stall = ctx->test_stall;
  p.wait_cycles = ctx->wait_cycles ? ctx->wait_cycles : 2000000000LL;
  // the vector form: every row on a 16-byte boundary
  auto row = [&](const void* q, int64_t ts, int64_t heads, int64_t hs) { return aligned(q, 16) && eights(ts, n) && eights(hs, heads); };
  bool vec = d % 8 == 0 && ctx->force_variant != 4;
  if (hq)
    vec = vec && row(a->q, a->q_token_stride, hq, a->q_head_stride) && row(a->q_out, a->q_out_token_stride, hq, a->q_out_head_stride) &&
          aligned(a->q_weight, 16);
  if (hk) vec = vec && row(a->k, a->k_token_stride, hk, a->k_head_stride) && aligned(a->k_weight, 16);
  if (k_out) vec = vec && row(a->k_out, a->k_out_token_stride, hk, a->k_out_head_stride);
  if (cache)
    vec = vec && row(a->v, a->v_token_stride, hk, a->v_head_stride) && aligned(a->k_cache, 16) && aligned(a->v_cache, 16) &&
          eights(a->k_block_stride, a->num_blocks) && eights(a->v_block_stride, a->num_blocks) && eights(a->k_page_stride, a->page_size) &&
          eights(a->v_page_stride, a->page_size) && eights(a->k_cache_head_stride, hk) && eights(a->v_cache_head_stride, hk);
  const bool bf16 = a->dtype == AR_DTYPE_BF16;
  DeviceGuard g(ctx->device);
  ar_status st;
  if (vec) {
    ar::RopePlan plan = ar::rope_plan(p, ctx->sm_count);
    void* args[2] = {&p, &plan};
    st = launch(ctx, ar::rope_vec_kernel(bf16, p.head_dim, half, p.pairs), plan.ctas, 320, 1, args, ar::rope_smem(plan), stream);
  } else {
    const int64_t warps = n * (hq + hk * (cache ? 2 : 1));
    int64_t grid = (warps + 7) / 8;
    if (grid > ctx->sm_count * 8) grid = ctx->sm_count * 8;
    void* args[1] = {&p};
    st = launch(ctx, ar::rope_scalar_kernel(bf16), (unsigned)grid, 256, 1, args, 0, stream);
  }
  if (st == AR_OK) ctx->last_variant = vec ? "qk_norm_rope_vec" : "qk_norm_rope_scalar";
  return st;
}

}  // extern "C"

namespace {

int padded_dim(int d) { return d <= 64 ? 64 : d <= 128 ? 128 : 256; }

constexpr int kMmaRows = 64;

struct Workspace {
  int64_t ml, o, bytes;  // offsets of the statistics and the sums behind the headers
};

Workspace workspace_of(int64_t spans, int64_t rows, int64_t part_dim) {
  auto up = [](int64_t x) { return (x + 255) / 256 * 256; };
  Workspace w;
  w.ml = up(spans * 8 * 4);
  w.o = w.ml + up(spans * 2 * rows * 8);
  w.bytes = w.o + up(spans * 2 * rows * part_dim * 4);
  return w;
}

int mma_spans(const ar_ctx* ctx, bool bf16, int dp) {
  return ctx->sm_count * ctx->attn_mma_per_sm[bf16][dp == 64 ? 0 : dp == 128 ? 1 : 2];
}

int part_dim(int d) { return (d + 3) / 4 * 4; }

int64_t workspace_need(const ar_ctx* ctx, bool bf16, int d) {
  const int64_t general = workspace_of(mma_spans(ctx, bf16, padded_dim(d)), kMmaRows, part_dim(d)).bytes;
  const int64_t tma = workspace_of(ctx->sm_count, ar::attn_tma_rows(padded_dim(d)), part_dim(d)).bytes;
  return tma > general ? tma : general;
}

}  // namespace

extern "C" {

ar_status ar_paged_attention_workspace(ar_ctx* ctx, const ar_paged_attention_args* a, size_t* bytes) {
  if (!a || !bytes || a->head_dim < 1 || a->head_dim > AR_MAX_HEAD_DIM || (a->dtype != AR_DTYPE_BF16 && a->dtype != AR_DTYPE_F16))
    return AR_ERR_INVALID_ARG;
  if (!ctx) return AR_ERR_NOT_INITIALIZED;
  if (ctx->serve_error) return fail_cuda(ctx, ctx->serve_error, "the attention block's kernels");
  *bytes = (size_t)workspace_need(ctx, a->dtype == AR_DTYPE_BF16, a->head_dim);
  return AR_OK;
}

ar_status ar_paged_attention(ar_ctx* ctx, const ar_paged_attention_args* a, void* stream) {
  if (!a) return AR_ERR_INVALID_ARG;
  if (a->tokens < 0 || a->requests < 0 || a->requests > AR_MAX_REQUESTS || a->q_heads < 1 || a->kv_heads < 1 || a->q_heads % a->kv_heads ||
      a->q_heads > 65536 || a->head_dim < 1 || a->head_dim > AR_MAX_HEAD_DIM || (a->dtype != AR_DTYPE_BF16 && a->dtype != AR_DTYPE_F16))
    return AR_ERR_INVALID_ARG;
  if (!isfinite(a->scale) || !isfinite(a->softcap) || a->softcap < 0.0f || a->window < 0) return AR_ERR_INVALID_ARG;
  if (a->page_size < 1 || a->page_size > 65536 || a->num_blocks < 0 || a->num_blocks > ((int64_t)1 << 40) / a->page_size || a->table_cols < 0 ||
      a->table_cols > 0x7fffffff || a->table_stride < 0 || (a->table_stride && a->table_stride < a->table_cols) ||
      a->table_stride > ((int64_t)1 << 40))
    return AR_ERR_INVALID_ARG;
  const int64_t n = a->tokens, d = a->head_dim, hq = a->q_heads, hk = a->kv_heads, r = a->requests, pg = a->page_size;
  if (n > kMaxRows || n * (hq / hk) > kMaxRows) return AR_ERR_UNSUPPORTED;
  // the key tiles of one query tile and all heads are counted in 32 bits
  const int64_t room = a->table_cols * pg < kMaxRows ? a->table_cols * pg : kMaxRows;
  if (room * hk > (int64_t)1 << 36) return AR_ERR_UNSUPPORTED;
  if (n == 0 || r == 0) {
    if (!ctx) return AR_ERR_NOT_INITIALIZED;
    ctx->last_variant = "none";
    return AR_OK;
  }
  if (!a->q || !a->out || !a->cu_q || !a->seq_lens || (a->table_cols && !a->block_table) || (a->num_blocks && (!a->k_cache || !a->v_cache)) ||
      !a->workspace)
    return AR_ERR_INVALID_ARG;
  if (!strides_ok(n, a->q_token_stride, hq, a->q_head_stride, d) || !strides_ok(n, a->out_token_stride, hq, a->out_head_stride, d) ||
      !strides_ok(a->num_blocks, a->k_block_stride, pg, a->k_page_stride, d) || !strides_ok(a->num_blocks, a->v_block_stride, pg, a->v_page_stride, d) ||
      !strides_ok(1, 0, hk, a->k_head_stride, d) || !strides_ok(1, 0, hk, a->v_head_stride, d))
    return AR_ERR_INVALID_ARG;
  if (!aligned(a->q, 2) || !aligned(a->out, 2) || !aligned(a->lse, 4) || !aligned(a->k_cache, 2) || !aligned(a->v_cache, 2) ||
      !aligned(a->block_table, 4) || !aligned(a->cu_q, 4) || !aligned(a->seq_lens, 4) || !aligned(a->slopes, 4) ||
      !aligned(a->prefix_lens, 4) || !aligned(a->workspace, 16))
    return AR_ERR_ALIGNMENT;
  const int64_t ts = a->table_stride ? a->table_stride : a->table_cols;
  Operands c;
  c.read({a->q, d * 2, {a->q_head_stride * 2, 0, a->q_token_stride * 2}, {hq, 1, n}});
  c.read(cache_extent(a->k_cache, d, hk, a->k_head_stride, pg, a->k_page_stride, a->num_blocks, a->k_block_stride));
  c.read(cache_extent(a->v_cache, d, hk, a->v_head_stride, pg, a->v_page_stride, a->num_blocks, a->v_block_stride));
  c.read(table(a->block_table, a->table_cols * 4, ts * 4, r));
  c.read(flat(a->cu_q, (r + 1) * 4));
  c.read(flat(a->seq_lens, r * 4));
  c.read(flat(a->slopes, hq * 4));
  c.read(flat(a->prefix_lens, r * 4));
  c.write({a->out, d * 2, {a->out_head_stride * 2, 0, a->out_token_stride * 2}, {hq, 1, n}});
  c.write(flat(a->lse, n * hq * 4));
  c.write(flat(a->workspace, (int64_t)a->workspace_bytes));
  if (!c.ok()) return AR_ERR_OVERLAP;
  if (!ctx) return AR_ERR_NOT_INITIALIZED;
  if (ctx->serve_error) return fail_cuda(ctx, ctx->serve_error, "the attention block's kernels");
  const bool bf16 = a->dtype == AR_DTYPE_BF16;
  if ((int64_t)a->workspace_bytes < workspace_need(ctx, bf16, a->head_dim)) return AR_ERR_INVALID_ARG;

  ar::AttnParams p;
  memset(&p, 0, sizeof(p));
  p.tokens = n;
  p.requests = a->requests;
  p.q_heads = a->q_heads;
  p.kv_heads = a->kv_heads;
  p.group = ar::fast_div((uint32_t)(a->q_heads / a->kv_heads));
  p.head_dim = a->head_dim;
  p.q = a->q;
  p.out = a->out;
  p.q_ts = a->q_token_stride;
  p.q_hs = a->q_head_stride;
  p.o_ts = a->out_token_stride;
  p.o_hs = a->out_head_stride;
  p.lse = a->lse;
  p.k = a->k_cache;
  p.v = a->v_cache;
  p.k_bs = a->k_block_stride;
  p.k_ps = a->k_page_stride;
  p.k_hs = a->k_head_stride;
  p.v_bs = a->v_block_stride;
  p.v_ps = a->v_page_stride;
  p.v_hs = a->v_head_stride;
  p.num_blocks = a->num_blocks;
  p.page = ar::fast_div((uint32_t)pg);
  p.table = a->block_table;
  p.table_stride = ts;
  p.max_len = (int)room;
  p.cu_q = a->cu_q;
  p.seq_lens = a->seq_lens;
  p.causal = a->causal != 0;
  p.window = a->window >= kMaxRows ? 0 : a->window;  // no length reaches it
  const double log2e = 1.4426950408889634;
  // Factors that a type of 32 bits does not hold are cut to its largest (half of it for the cap, which is
  // doubled), so that a product of 0 stays 0.
  auto cut = [](double x, double most) { return (float)(x > most ? most : x < -most ? -most : x); };
  constexpr double most = 3.4028234663852886e38;
  p.scale_log2 = cut(a->scale * log2e, most);
  if (a->softcap > 0.0f) {
    p.cap_log2 = cut(a->softcap * log2e, most / 2);
    p.cap_inv = cut(1.0 / (a->softcap * log2e), most);
    p.cap_twice = cut(2.0 * log2e * a->scale / a->softcap, most);
  }
  p.slopes = a->slopes;
  p.prefix = a->prefix_lens;
  p.vec = d % 8 == 0 && eights(a->q_token_stride, n) && eights(a->q_head_stride, hq) && eights(a->out_token_stride, n) &&
          eights(a->out_head_stride, hq) && eights(a->k_block_stride, a->num_blocks) && eights(a->k_page_stride, pg) && eights(a->k_head_stride, hk) &&
          eights(a->v_block_stride, a->num_blocks) && eights(a->v_page_stride, pg) && eights(a->v_head_stride, hk) && aligned(a->q, 16) &&
          aligned(a->out, 16) && aligned(a->k_cache, 16) && aligned(a->v_cache, 16) && ctx->force_variant != 4;
  p.status = ctx->d_status;
  p.wait_cycles = ctx->wait_cycles ? ctx->wait_cycles : 2000000000LL;

  // The tensor-core form takes aligned rows and pages that whole groups of
  // 8 keys (the swizzle's period) fill; the general form the rest.
  const int dp = padded_dim(a->head_dim);
  int box = 1;
  while (box < 128 && pg % (box * 2) == 0) box *= 2;
  bool tma = p.vec && box >= 8 && a->num_blocks > 0 && a->num_blocks < 0x7fffffff && ctx->encode_tensor_map;
  CUtensorMap kmap, vmap;
  if (tma) {
    p.box_rows = box;
    p.stall = ctx->test_stall;
    tma = ar::attn_tensor_map(ctx->encode_tensor_map, &kmap, a->k_cache, bf16, d, pg, hk, a->num_blocks, a->k_page_stride, a->k_head_stride,
                              a->k_block_stride, box) &&
          ar::attn_tensor_map(ctx->encode_tensor_map, &vmap, a->v_cache, bf16, d, pg, hk, a->num_blocks, a->v_page_stride, a->v_head_stride,
                              a->v_block_stride, box);
  }
  p.spans = tma ? ctx->sm_count : mma_spans(ctx, bf16, dp);
  p.tile_rows = tma ? ar::attn_tma_rows(dp) : kMmaRows;
  p.part_dim = part_dim(a->head_dim);
  const Workspace w = workspace_of(p.spans, p.tile_rows, p.part_dim);
  char* base = static_cast<char*>(a->workspace);
  p.headers = reinterpret_cast<int*>(base);
  p.part_ml = reinterpret_cast<float*>(base + w.ml);
  p.part_o = reinterpret_cast<float*>(base + w.o);
  p.wide = d % 16 == 0 && eights(a->out_token_stride, n, 16) && eights(a->out_head_stride, hq, 16) && aligned(a->out, 32) && aligned(base, 32);
  DeviceGuard g(ctx->device);
  void* args[3] = {&p, &kmap, &vmap};
  const bool bias = a->slopes || !(a->scale > 0.0f);
  ar_status st = tma ? launch(ctx, ar::attn_tma_kernel(bf16, dp, a->softcap, bias), (unsigned)p.spans, 384, 1, args, ar::attn_tma_smem(dp), stream)
                     : launch(ctx, ar::attn_mma_kernel(bf16, dp), (unsigned)p.spans, 128, 1, args, ar::attn_mma_smem(dp), stream);
  if (st != AR_OK) return st;
  // Blocks that may join the rows of one item: 4 where a request has few rows, else 16 (us with
  // 4, 8, 16, 32: one token 10.9, 11.0, 12.3, 15.0; 128 tokens over 3000: 54.5, 40.4, 32.7, 31.8).
  const unsigned joiners = n * (hq / hk) > 64 * r ? 16 : 4;
  st = launch(ctx, ar::attn_combine_kernel(bf16), dim3((unsigned)p.spans, joiners), 256, 1, args, 0, stream);
  if (st == AR_OK) ctx->last_variant = tma ? "paged_attention_tma" : "paged_attention_mma";
  return st;
}

}  // extern "C"

namespace ar {

cudaError_t serve_prepare(ar_ctx* ctx) {
  cudaError_t e = cudaSuccess;
  cudaFuncAttributes fa;
  auto keep = [&](cudaError_t x) {
    if (e == cudaSuccess) e = x;
  };
  keep(cudaFuncGetAttributes(&fa, plan_kernel()));
  keep(cudaFuncSetAttribute(plan_kernel(), cudaFuncAttributeMaxDynamicSharedMemorySize, AR_MAX_REQUESTS * 8));
  for (int b = 0; b < 2; ++b) {
    keep(cudaFuncGetAttributes(&fa, rope_scalar_kernel(b)));
    for (int d : {64, 80, 96, 128, 256, 72})
      for (int mode = 0; mode < 3; ++mode)
        keep(cudaFuncSetAttribute(rope_vec_kernel(b, d, mode == 1 ? 8 : 4, mode == 0), cudaFuncAttributeMaxDynamicSharedMemorySize, (int)rope_smem_most()));
    keep(cudaFuncGetAttributes(&fa, attn_combine_kernel(b)));
    for (int i = 0; i < 3; ++i)
      for (int ext = 0; ext < 6; ++ext)  // no cap, a cap, a wide one
        keep(cudaFuncSetAttribute(attn_tma_kernel(b, 64 << i, (float)(ext >> 1) * 50.0f, ext & 1), cudaFuncAttributeMaxDynamicSharedMemorySize, (int)attn_tma_smem(64 << i)));
    for (int i = 0; i < 3; ++i) {
      const int dp = 64 << i;
      const void* f = attn_mma_kernel(b, dp);
      keep(cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)attn_mma_smem(dp)));
      keep(cudaOccupancyMaxActiveBlocksPerMultiprocessor(&ctx->attn_mma_per_sm[b][i], f, 128, attn_mma_smem(dp)));
      if (ctx->attn_mma_per_sm[b][i] < 1) ctx->attn_mma_per_sm[b][i] = 1;
    }
  }
  cudaDriverEntryPointQueryResult found = cudaDriverEntryPointSymbolNotFound;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ctx->encode_tensor_map, 12000, cudaEnableDefault, &found) != cudaSuccess ||
      found != cudaDriverEntryPointSuccess)
    ctx->encode_tensor_map = nullptr;
  return e;
}

}  // namespace ar
