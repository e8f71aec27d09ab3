// Walk of the append to an 8-bit cache over the blocks that its tokens go to.
//
// A unit is a block of a request that gets tokens in this call.  The units of all requests stand in one
// sequence, and every CTA takes an equal, contiguous span of it; a block belongs to one CTA (or, split by
// heads, to CTAs with different heads), so scales are found and codes rewritten without atomics.
#pragma once

#include "ar_common.cuh"
#include "ar_e4m3.cuh"
#include "ar_fastdiv.cuh"
#include "ar_serve.h"

namespace ar {

struct AppendRequest {
  int q0, place, end;  // row of its first new token; that token's place, and the place behind the last one
  int first;           // its first block
  int blocks;          // blocks that get tokens
};

__device__ __forceinline__ AppendRequest append_request(const AppendParams& p, int r) {
  const int a = p.cu_q[r], b = p.cu_q[r + 1], len = p.seq_lens[r];
  const int most = (int)p.tokens;
  AppendRequest q;
  q.q0 = min(max(a, 0), most);
  const int n = min(max(b, q.q0), most) - q.q0;
  bool bad = a < 0 || b < a || b > most;
  q.place = len - n;
  q.end = min(len, p.max_len);
  q.first = q.blocks = 0;
  if (len < n) {
    bad = true;
  } else if (n > 0) {
    bad = bad || q.end < len;
    if (q.place < q.end) {
      q.first = q.place / p.page;
      q.blocks = (q.end - 1) / p.page - q.first + 1;
    }
  }
  if (bad) *p.status = kStatusBadIndex;
  return q;
}

// One unit as a CTA works on it.
struct AppendUnit {
  int64_t block;  // -1: outside the cache
  int held;       // tokens that the block holds already
  int row;        // first new token: its row,
  int place;      // its place in the request,
  int n;          // and how many there are
  int part;       // which share of the heads
};

struct AppendShared {
  long long warp_sum[32];
  int r, block, part;  // where the span starts
  long long units;     // and its length
};

// The CTA's span; `parts`: units that share a block.  All threads take part.
template <int THREADS>
__device__ void append_span(const AppendParams& p, int parts, AppendShared& sh) {
  constexpr int WARPS = THREADS / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int blocks = 0;
  long long before = 0, excl = 0;
  auto scan = [&](int base) {
    const int r = base + (int)threadIdx.x;
    blocks = r < p.requests ? append_request(p, r).blocks : 0;
    long long s = blocks;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += u;
    }
    if (lane == 31) sh.warp_sum[warp] = s;
    __syncthreads();
    excl = before + s - blocks;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      const long long u = sh.warp_sum[w];
      if (w < warp) excl += u;
      before += u;
    }
  };
  const bool one = p.requests <= THREADS;
  for (int base = 0; base < p.requests; base += THREADS) {
    if (base) __syncthreads();
    scan(base);
  }
  const long long total = before * parts, each = total / gridDim.x, more = total - each * gridDim.x;
  const long long b = blockIdx.x, s0 = each * b + (b < more ? b : more), units = each + (b < more ? 1 : 0);
  const long long at = s0 / parts;
  if (threadIdx.x == 0) {
    sh.units = units;
    sh.part = (int)(s0 - at * parts);
  }
  before = 0;
  for (int base = 0; base < p.requests; base += THREADS) {
    if (!one) {
      __syncthreads();
      scan(base);
    }
    if (units > 0 && excl <= at && at < excl + blocks) {
      sh.r = base + (int)threadIdx.x;
      sh.block = (int)(at - excl);
    }
  }
  __syncthreads();
}

// Every thread walks for itself.
struct AppendWalk {
  AppendRequest q;
  int r, block, part, parts;
  long long left;

  __device__ __forceinline__ void start(const AppendParams& p, const AppendShared& sh, int n) {
    left = sh.units;
    parts = n;
    if (left <= 0) return;
    r = sh.r;
    block = sh.block;
    part = sh.part;
    q = append_request(p, r);
  }

  __device__ __forceinline__ bool next(const AppendParams& p, AppendUnit& u) {
    if (left <= 0) return false;
    --left;
    const int j = q.first + block, page = (int)p.page.d;
    const int64_t low = (int64_t)j * page;  // below 2^30
    const int first = max((int)low, q.place), end = (int)min(low + page, (int64_t)q.end);
    u.held = first - (int)low;
    u.row = q.q0 + first - q.place;
    u.place = first;
    u.n = end - first;
    u.part = part;
    const int b = p.table[(int64_t)r * p.table_stride + j];
    u.block = b;
    if (b < 0 || b >= p.num_blocks) {
      u.block = -1;
      if (threadIdx.x == 0) *p.status = kStatusBadIndex;
    }
    if (++part == parts) {
      part = 0;
      if (++block == q.blocks) {
        block = 0;
        q.blocks = 0;
        if (left > 0)
          while (q.blocks == 0 && ++r < p.requests) q = append_request(p, r);
      }
    }
    return true;
  }
};

}  // namespace ar
