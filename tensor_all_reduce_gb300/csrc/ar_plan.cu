// Paged plan: block tables and slot maps of one step from its request lengths.
//
// Two prefix sums over the requests (new tokens, blocks needed) decide everything: token t
// belongs to the request that holds it in the first sum, block b of the step to the one that
// holds it in the second.  The sums are tiny (at most 8192 requests), so every CTA computes
// them for itself into shared memory and then fills its part of the tokens: one launch, no
// exchange between CTAs.  Nothing a CTA reads is written by another: the table's entries in
// front of the cached tokens' end stay, and a new block's number is taken from the free list.
//
// Bound: latency.  A step's bytes (12 a token, 4 a block) take well under a microsecond; what is
// left is the chain of dependent loads (lengths, then table) around one block-wide scan.  On GB300
// a step of 8 requests takes 4.8 us, of 256 5.5 us, of 1024 prompts (160,000 tokens) 8.2 us.
#include "ar_common.cuh"
#include "ar_serve.h"

namespace ar {
namespace {

constexpr int kPlanThreads = 512;
constexpr int kPerThread = AR_MAX_REQUESTS / kPlanThreads;

struct Pair {
  long long a, b;
};

// Exclusive prefix of v over the block's threads; `total` is the sum over all.
__device__ Pair block_scan(Pair v, Pair* warp_sums, Pair& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Pair s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long a = __shfl_up_sync(0xffffffffu, s.a, o), b = __shfl_up_sync(0xffffffffu, s.b, o);
    if (lane >= o) {
      s.a += a;
      s.b += b;
    }
  }
  if (lane == 31) warp_sums[warp] = s;
  __syncthreads();
  Pair base = {0, 0};
  total = {0, 0};
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    const Pair t = warp_sums[w];
    if (w < warp) {
      base.a += t.a;
      base.b += t.b;
    }
    total.a += t.a;
    total.b += t.b;
  }
  return {base.a + s.a - v.a, base.b + s.b - v.b};
}

// The last r in [0, n) with start[r] <= x (start[0] = 0 <= x, not decreasing): the owner of x
// when x is below the sum, because requests that own nothing start where the next one does.
__device__ __forceinline__ int owner(const int* start, int n, int x) {
  int lo = 0, hi = n;  // start[lo] <= x; start[hi] > x or hi == n
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kPlanThreads) plan(const __grid_constant__ PlanParams p) {
  extern __shared__ int sm[];  // first token, then first block, of each request
  __shared__ Pair warp_sums[kPlanThreads / 32];
  pdl_wait_and_release();
  int* first_token = sm;
  int* first_block = sm + p.requests;
  const int per = (p.requests + kPlanThreads - 1) / kPlanThreads;  // consecutive requests of a thread
  const int r0 = threadIdx.x * per;

  int code = AR_PLAN_OK;
  Pair mine = {0, 0};
  int tok[kPerThread], blk[kPerThread];
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    tok[i] = blk[i] = 0;
    if (i >= per || r0 + i >= p.requests) continue;
    const long long c = p.cached[r0 + i], n = p.fresh[r0 + i];
    if (c < 0 || n < 0 || c + n > 0x7fffffffLL) {
      code = AR_PLAN_BAD_LENGTH;
      continue;
    }
    const long long have = (c + p.page - 1) / p.page, last = (c + n + p.page - 1) / p.page;
    if (last > p.table_cols && code < AR_PLAN_TABLE_FULL) code = AR_PLAN_TABLE_FULL;
    tok[i] = (int)n;
    blk[i] = (int)(last - have);
    mine.a += tok[i];
    mine.b += blk[i];
  }
  Pair total;
  Pair at = block_scan(mine, warp_sums, total);
  const int count = *p.free_count;
  if (count < 0 || count > p.free_capacity) code = AR_PLAN_BAD_LENGTH;
  if (total.a > p.max_tokens && code < AR_PLAN_TOO_MANY_TOKENS) code = AR_PLAN_TOO_MANY_TOKENS;
  if (total.b > count && code < AR_PLAN_NO_BLOCKS) code = AR_PLAN_NO_BLOCKS;
  // the largest code of the block's threads, a bit for each
  const int bits = (__syncthreads_or(code == 1) ? 2 : 0) | (__syncthreads_or(code == 2) ? 4 : 0) |
                   (__syncthreads_or(code == 3) ? 8 : 0) | (__syncthreads_or(code == 4) ? 16 : 0);
  const int refusal = bits ? 31 - __clz(bits) : 0;
  const bool ok = refusal == 0;

#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int r = r0 + i;
    if (i >= per || r >= p.requests) continue;
    if (ok) {  // below max_tokens and the free count: 32 bits hold them
      first_token[r] = (int)at.a;
      first_block[r] = (int)at.b;
    }
    if (blockIdx.x == 0) {
      const int c = p.cached[r];
      p.cu_q[r] = ok ? (int)at.a : 0;
      p.seq_lens[r] = ok ? c + tok[i] : (c < 0 ? 0 : c);
    }
    at.a += tok[i];
    at.b += blk[i];
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    p.cu_q[p.requests] = ok ? (int)total.a : 0;
    *p.free_count_out = ok ? count - (int)total.b : count;
    p.info[0] = ok ? (int)total.a : 0;
    p.info[1] = ok ? (int)total.b : 0;
    p.info[2] = refusal;
    p.info[3] = total.b > 0x7fffffffLL ? 0x7fffffff : (int)total.b;
  }
  __syncthreads();

  const int64_t step = (int64_t)gridDim.x * kPlanThreads;
  const int64_t me = (int64_t)blockIdx.x * kPlanThreads + threadIdx.x;
  const int64_t tokens = ok ? total.a : 0;
  for (int64_t t = me; t < p.max_tokens; t += step) {
    int64_t slot = -1;
    int pos = 0;
    if (t < tokens) {
      const int r = owner(first_token, p.requests, (int)t);
      const int c = p.cached[r];
      pos = c + (int)t - first_token[r];
      const int j = pos / p.page, have = (int)(((long long)c + p.page - 1) / p.page);
      const int block = j < have ? p.table[(int64_t)r * p.table_stride + j]
                                 : p.free_blocks[count - 1 - first_block[r] - (j - have)];
      slot = (int64_t)block * p.page + (pos - j * p.page);
      if (block < 0) {  // no block: not a slot, and not the -1 of a row without a token
        slot = -2;
        *p.status = kStatusBadIndex;
      }
    }
    p.slots[t] = slot;
    p.positions[t] = pos;
  }
  if (!ok) return;
  for (int64_t b = me; b < total.b; b += step) {
    const int r = owner(first_block, p.requests, (int)b);
    const int have = (int)(((long long)p.cached[r] + p.page - 1) / p.page);
    p.table[(int64_t)r * p.table_stride + have + ((int)b - first_block[r])] = p.free_blocks[count - 1 - b];
  }
}

}  // namespace

const void* plan_kernel() { return reinterpret_cast<const void*>(&plan); }

}  // namespace ar
