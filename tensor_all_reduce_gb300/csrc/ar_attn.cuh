// Work division of the paged attention kernels.
//
// An item is a tile of ROWS consecutive query rows of one request and one key head (rows are
// the request's new tokens times the q heads that share the key head, token-major), with the
// tiles of KT keys that some row of it can see.  All (item, key tile) pairs of the call stand in
// one sequence, request by request, query tile by query tile, head by head, and every CTA of a
// resident grid takes an equal, contiguous span of it.  So one rule serves single tokens over
// long caches, chunks, and both in one batch, and the lengths may stay in device memory.
//
// A CTA that covers an item's tiles whole writes the output.  Otherwise it leaves the unnormalised
// sum, maximum and weight sum of its part in the workspace: a CTA's span touches at most one
// item that began before it (slot 0) and one that ends after it (slot 1).  A second small
// kernel joins the parts in a fixed order, so results do not depend on timing.
//
// An item of many rows costs more than its tiles: its queries arrive, its first scores and its last
// sum stand alone, its rows are written.  So it counts kItemCost tiles more, in front of its own.
// (Measured on GB300 with 20 q heads, 4 key heads of 128, causal, us with 0, 2, 4, 6 tiles: 5 requests
// of 983 tokens 94, 61, 58, 61; 12 q heads, 300 tokens over 10000: 43, 41, 38, 38.)
//
// Storing and joining its parts takes as long as about kSplitCost tiles.  So one of no more tiles
// than that and a span together is not split, as long as it is short (up to kWholeMost tiles; long
// ones would leave SMs idle): a span that would begin or end inside it is moved to its nearer end
// (both neighbours decide alike).  (12 q heads, 2 key heads of 128, us with 12, 8, 6, 4: 512 tokens
// over 1000 32.1, 34.2, 26.9, 26.9; 1024 over none 25.9, 25.9, 26.0, 27.3; without the rule, on an
// earlier form that took 34 and 29 us with it, 44 and 36.)
#pragma once

#include "ar_common.cuh"
#include "ar_fastdiv.cuh"
#include "ar_serve.h"

namespace ar {

// What a CTA says of the item that begins in its span and does not end there: the CTA where it
// ends (0: there is no such item), first row of the request, rows of the request, query tile, head.
constexpr int kHeaderInts = 8;

constexpr int kItemCost = 4, kSplitCost = 6, kWholeMost = 24;
constexpr int kFewRows = 64;  // items of no more rows are split at any length, and count their tiles alone: their parts are small

struct Request {
  int q0, n, len, prefix;  // first row of q, new tokens, keys, keys that every row sees
};

__device__ __forceinline__ Request load_request(const AttnParams& p, int r) {
  Request q;
  const int a = p.cu_q[r], b = p.cu_q[r + 1];
  const int most = (int)p.tokens;
  q.q0 = min(max(a, 0), most);
  q.n = min(max(b, q.q0), most) - q.q0;
  const int len = p.seq_lens[r];
  q.len = min(max(len, 0), p.max_len);
  q.prefix = p.prefix ? min(max(p.prefix[r], 0), q.len) : 0;
  if (a < 0 || b < a || b > most || q.len != len) *p.status = kStatusBadIndex;
  return q;
}

// Keys [low, high) that some of a request's new tokens [t0, t1) sees besides the prefix: their windows, of
// neighbouring positions, leave no gap.
struct KeyRange {
  int low, high;
  __device__ __forceinline__ bool sees(const Request& q, int key) const { return key < q.prefix || (key < high && key >= low); }
};

__device__ __forceinline__ KeyRange key_range(const AttnParams& p, const Request& q, int t0, int t1) {
  const int p0 = q.len - q.n + t0, p1 = q.len - q.n + t1;  // positions; may be negative: rows that see no key
  // |p0| and window are at most 2^30
  return {p.window ? max(p0 - p.window + 1, 0) : 0, p.causal ? min(max(p1, 0), q.len) : q.len};
}

// Key tiles of a query tile: [0, pre), then [lo, hi).
struct TileRange {
  int pre, lo, hi;
  __device__ __forceinline__ int count() const { return max(pre + max(hi - lo, 0), 1); }  // an empty row is one masked tile
  __device__ __forceinline__ int tile(int i) const { return i < pre ? i : lo + (i - pre); }
};

template <int ROWS, int KT>
__device__ __forceinline__ TileRange tile_range(const AttnParams& p, const Request& q, int qt) {
  const int row0 = qt * ROWS, rows = q.n * (int)p.group.d;  // at most 2^30
  const KeyRange k = key_range(p, q, row0 / p.group, (min(row0 + ROWS, rows) - 1) / p.group + 1);
  TileRange t;
  t.pre = (q.prefix + KT - 1) / KT;
  t.lo = max(k.low / KT, t.pre);
  t.hi = (k.high + KT - 1) / KT;
  return t;
}

// Tiles that an item of so many rows counts besides its own, in front of them.
template <int ROWS>
__device__ __forceinline__ int extra_tiles(const AttnParams& p, const Request& q, int qt) {
  return q.n * (int)p.group.d - qt * ROWS > kFewRows ? kItemCost : 0;
}

struct Cursor {  // a place in the sequence
  int r, qt, h, tile;  // tile: extra ones first
};

// One item as a CTA walks over it.
struct Item {
  Request q;
  int rows;  // rows of the request (new tokens times group)
  int r, qt, h;
  TileRange range;
  int begin, end;  // tiles of this CTA's part
  bool first, last;  // the part holds the item's first, last tile
};

struct SpanShared {
  long long warp_sum[32];
  Cursor at;
  Request q;        // of request at.r
  long long tiles;  // tiles of this CTA's span
  long long end, each, longer;  // where it ends; the first `longer` spans have each + 1 tiles
};

// The CTA's span: where it starts and how many tiles it has.  All threads take part, a thread a
// request: the scan over the requests is redone by every CTA, which costs about a microsecond and
// saves a launch that would do it once.
template <int ROWS, int KT, int THREADS>
__device__ void find_span(const AttnParams& p, SpanShared& sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int WARPS = THREADS / 32;
  Request q = {0, 0, 0, 0};
  long long before = 0, mine = 0, excl = 0;
  auto query_tiles = [&](int n) { return (int)((n * p.group.d + ROWS - 1) / ROWS); };
  auto weight_of = [&](const Request& o, int qt) { return tile_range<ROWS, KT>(p, o, qt).count() + extra_tiles<ROWS>(p, o, qt); };
  auto share = [&](int src) {  // a lane's request, to its warp
    Request o;
    o.q0 = 0;
    o.n = __shfl_sync(0xffffffffu, q.n, src);
    o.len = __shfl_sync(0xffffffffu, q.len, src);
    o.prefix = __shfl_sync(0xffffffffu, q.prefix, src);
    return o;
  };
  auto scan = [&](int base) {  // `mine`: tiles of the thread's request; `excl`: of those before it; `before`: of all so far
    const int r = base + (int)threadIdx.x;
    q.n = 0;
    if (r < p.requests) q = load_request(p, r);
    const int nqt = query_tiles(q.n);
    mine = nqt == 1 ? weight_of(q, 0) : 0;
    for (unsigned many = __ballot_sync(0xffffffffu, nqt > 1); many; many &= many - 1) {  // the warp together
      const int src = __ffs(many) - 1;
      const Request o = share(src);
      const int m = query_tiles(o.n);
      long long s = 0;
      for (int t = lane; t < m; t += 32) s += weight_of(o, t);
#pragma unroll
      for (int k = 16; k > 0; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
      if (lane == src) mine = s;
    }
    mine *= p.kv_heads;
    long long s = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += u;
    }
    if (lane == 31) sh.warp_sum[warp] = s;
    __syncthreads();
    excl = before + s - mine;
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
  // equal spans, the first ones a tile longer; with fewer tiles than CTAs the first ones have
  // one each, so that spans with tiles stand side by side
  const long long total = before;
  const unsigned grid = gridDim.x, b = blockIdx.x;
  const long long each = total < 0x7fffffffLL ? (unsigned)total / grid : total / grid;
  const long long more = total - each * grid;
  const long long s0 = each * b + (b < more ? b : more), tiles = each + (b < more ? 1 : 0);
  if (threadIdx.x == 0) {
    sh.tiles = tiles;
    sh.end = s0 + tiles;
    sh.each = each;
    sh.longer = more;
  }
  before = 0;
  for (int base = 0; base < p.requests; base += THREADS) {
    if (!one) {
      __syncthreads();
      scan(base);
    }
    const unsigned owner = __ballot_sync(0xffffffffu, tiles > 0 && mine > 0 && excl <= s0 && s0 < excl + mine);
    if (!owner) continue;
    const int src = __ffs(owner) - 1;  // this warp has the span's first request: find the query tile, head and key tile
    if (lane == src) {
      sh.at.r = base + (int)threadIdx.x;
      sh.q = q;
    }
    const Request o = share(src);
    long long left = s0 - __shfl_sync(0xffffffffu, excl, src);
    const int m = query_tiles(o.n);
    for (int first = 0; first < m; first += 32) {
      const int t = first + lane;
      const int n = t < m ? weight_of(o, t) : 0;
      const long long own = (long long)n * p.kv_heads;
      long long s = own;
#pragma unroll
      for (int k = 1; k < 32; k <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, s, k);
        if (lane >= k) s += u;
      }
      const unsigned over = __ballot_sync(0xffffffffu, s > left);
      if (over) {
        if (lane == __ffs(over) - 1) {
          const long long in = left - (s - own);  // below 2^31: heads times tiles of one query tile
          sh.at.qt = t;
          sh.at.h = (int)((unsigned)in / (unsigned)n);
          sh.at.tile = (int)in - sh.at.h * n;
        }
        break;
      }
      left -= __shfl_sync(0xffffffffu, s, 31);
    }
  }
  __syncthreads();
}

// Walks the items of a span; every role of a CTA walks for itself.
template <int ROWS, int KT>
struct Walk {
  Cursor at;
  long long left;
  Request q;
  int whole;  // tiles up to which an item of many rows is not split

  __device__ __forceinline__ void start(const SpanShared& sh) {
    at = sh.at;
    left = sh.tiles;
    q = sh.q;
    whole = (int)min(sh.each + kSplitCost, (long long)kWholeMost);
  }

  __device__ __forceinline__ bool next(const AttnParams& p, Item& it) {
    while (left > 0) {
      const int rows = q.n * (int)p.group.d;
      it.q = q;
      it.rows = rows;
      it.r = at.r;
      it.qt = at.qt;
      it.h = at.h;
      it.range = tile_range<ROWS, KT>(p, q, at.qt);
      const int n = it.range.count(), extra = extra_tiles<ROWS>(p, q, at.qt);
      int begin = at.tile, end = (int)min((long long)(n + extra), at.tile + left);
      left -= end - begin;
      if (n <= whole && rows - it.qt * ROWS > kFewRows) {  // whole or not at all
        begin = begin * 2 < n + extra ? 0 : n;
        end = end * 2 < n + extra ? 0 : n;
      } else {
        begin = max(begin - extra, 0);
        end = max(end - extra, 0);
      }
      it.begin = begin;
      it.end = end;
      it.first = begin == 0;
      it.last = end == n;
      at.tile = 0;
      if (++at.h == p.kv_heads) {
        at.h = 0;
        if (++at.qt * ROWS >= rows) {
          at.qt = 0;
          if (left > 0) {  // a request with rows follows
            q.n = 0;
            while (q.n == 0 && ++at.r < p.requests) q = load_request(p, at.r);
            if (q.n == 0) left = 0;
          }
        }
      }
      if (begin < end) return true;
    }
    return false;
  }
};

// What a row of the item sees and how its scores are bent.
struct RowView {
  int pos;     // position of the query
  int see_lo;  // keys [see_lo, see_hi) besides the prefix
  int see_hi;
  float slope;  // slope * log2(e)
};

__device__ __forceinline__ RowView row_view(const AttnParams& p, const Item& it, int row) {
  RowView v;
  const int t = row / p.group, g = row - t * (int)p.group.d;
  v.pos = it.q.len - it.q.n + t;
  v.see_hi = p.causal ? min(v.pos + 1, it.q.len) : it.q.len;
  v.see_lo = p.window ? v.pos - p.window + 1 : 0;
  v.slope = p.slopes && row < it.rows ? p.slopes[it.h * (int)p.group.d + g] * 1.4426950408889634f : 0.0f;
  if (row >= it.rows) v.see_hi = 0;
  return v;
}

// (row, key) visible: rows behind the item's end have see_hi 0 and no outputs.
__device__ __forceinline__ bool visible(const Item& it, const RowView& v, int key) {
  return key < it.q.prefix || (key < v.see_hi && key >= v.see_lo);
}

// Score in log2 units from the raw product.
__device__ __forceinline__ float bend(const AttnParams& p, const RowView& v, float dot, int key) {
  float s = dot * p.scale_log2;
  if (p.cap_log2 > 0.0f) {
    const float x = s * p.cap_inv, bent = p.cap_log2 * tanhf(x);
    s = fabsf(x) < 0x1p-13f ? s : bent;  // there tanh(x) is x to 2^-27, and x may be subnormal
  }
  if (p.slopes) s -= v.slope * (float)abs(v.pos - key);
  return s;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Block and place in it of a key; -1 for a block number outside the cache, which is an error only
// where a row of the request sees the key (blocks behind a window may be gone).
__device__ __forceinline__ int64_t block_of(const AttnParams& p, const Item& it, int key, int& in_page) {
  const int j = key / p.page;
  in_page = key - j * (int)p.page.d;
  const int b = p.table[(int64_t)it.r * p.table_stride + j];
  if (b < 0 || b >= p.num_blocks) {
    if (key_range(p, it.q, 0, it.q.n).sees(it.q, key)) *p.status = kStatusBadIndex;
    return -1;
  }
  return b;
}

// Header of the item that begins in this span and goes on; it = NULL: there is none.
__device__ __forceinline__ void write_header(const AttnParams& p, const SpanShared& sh, const Item* it) {
  int* h = p.headers + (int64_t)blockIdx.x * kHeaderInts;
  int end = 0;
  if (it) {
    // the span that holds the item's last tile (this one ends at the item's tile it->end)
    const long long last = sh.end + (it->range.count() - it->end) - 1, long_part = sh.longer * (sh.each + 1);
    end = (int)(last < long_part ? last / (sh.each + 1) : sh.longer + (last - long_part) / sh.each);
    h[1] = it->q.q0;
    h[2] = it->rows;
    h[3] = it->qt;
    h[4] = it->h;
  }
  h[0] = end;
}

}  // namespace ar
