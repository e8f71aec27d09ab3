// What the attention kernels on the fifth-generation tensor cores share: tensor memory, matrix descriptors,
// waits, the shape of scores.
#pragma once

#include <cuda.h>

#include "ar_attn.cuh"
#include "ar_staged.cuh"

namespace ar {

constexpr int kKeys = 128;  // keys of a tile

// ---- tcgen05 ----------------------------------------------------------------

__device__ __forceinline__ void tmem_ld32(uint32_t (&r)[32], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
        "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}

__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};"
      ::"r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// After tmem_wait_ld: keeps the uses of loaded registers behind the wait.
__device__ __forceinline__ void settle(uint32_t (&r)[32]) {
  asm volatile("" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31]));
}

__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Arrives on `bar` when every matrix instruction this thread has issued is done.
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// Shared-memory matrix descriptor, 128-byte swizzle: rows of 128 bytes in groups of eight
// (1024 bytes apart).  `lead`: bytes between column blocks, for operands whose rows run along
// the reduction (values: a row is a key).
__device__ __forceinline__ uint64_t matrix_desc(uint32_t addr, uint32_t lead) {
  return (uint64_t)((addr >> 4) & 0x3fff) | ((uint64_t)(lead >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

__device__ __forceinline__ void tma_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_addr(bar))
      : "memory");
}

__device__ __forceinline__ void st_v8(void* dst, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]),
               "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// ---- waits --------------------------------------------------------------------

// Until the phase with `parity` completes; false when the wait ran out here or in another role.
// (B: the barriers of a kernel, with its `stop`.)
template <class B>
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, B& b, const AttnParams& p) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity)) {
    if (*reinterpret_cast<volatile int*>(&b.stop)) return false;
    if (clock64() - t0 > p.wait_cycles) {
      *reinterpret_cast<volatile int*>(&b.stop) = 1;
      *p.status = 1;
      return false;
    }
  }
  return true;
}

// Block numbers outside the cache are an error where a row of the request sees one of the block's keys
// (those behind a window may be gone).  A warp whose copies are issued looks for them, request by request,
// many CTAs a request where there are few: between the copies, which wide heads wait for, the test cost
// 2 x 1024 tokens over 8000 (heads of 256) 4 to 10 us of 162.
static __device__ void check_blocks(const AttnParams& p) {
  const int lane = threadIdx.x & 31, grid = (int)gridDim.x;
  const int parts = max(grid / p.requests, 1), part = (int)blockIdx.x % parts;
  for (int r = (int)blockIdx.x / parts; r < p.requests; r += grid / parts) {
    const Request q = load_request(p, r);
    const KeyRange range = key_range(p, q, 0, q.n);
    const int32_t* row = p.table + (int64_t)r * p.table_stride;
    const int pre = (q.prefix + (int)p.page.d - 1) / p.page, end = (range.high + (int)p.page.d - 1) / p.page;
    const int first = max(range.low / p.page, pre), blocks = q.n ? pre + max(end - first, 0) : 0;
    for (int i = part * 32 + lane; i < blocks; i += parts * 32)
      if ((unsigned)row[i < pre ? i : first + (i - pre)] >= (unsigned)p.num_blocks) *p.status = kStatusBadIndex;
  }
}

// How scores are bent, a bit each: kCap (tanh), kBias (distance; also any scale that is not positive,
// since the plain form scales after the maximum), kWide (a wide cap, always with the other two: a kernel of its
// own, since a branch in the others cost a mixed batch with a cap of 30 6 %).
enum { kCap = 1, kBias = 2, kWide = 4 };

inline int score_forms(float cap, bool bias) { return cap > 64.0f ? kCap | kBias | kWide : (cap > 0.0f ? kCap : 0) | (bias ? kBias : 0); }

__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A row's products with the N keys from key0 on to scores: in log2 units where they are bent, else
// as they are (the caller scales); masked where `edge` says that some row of the warp does not see all.
template <int EXT, int N>
__device__ __forceinline__ void shape_scores(const AttnParams& p, int prefix, const RowView& v, int key0, bool edge, float (&s)[N]) {
  if constexpr (EXT & kCap) {
    // c tanh(x) = c - 2 c / (1 + e^2x): one exponential and one reciprocal an element; an exponential that
    // overflows gives c.  The difference leaves an absolute error of 2^-22 c, whatever the score: 2^-16 at
    // most for caps of up to 64, far below the weights' rounding.  With wider caps, where usual scores are a
    // small part of c, |x| < 1/2 takes the score times tanh(x) / x, a polynomial in x^2 (interpolation at the
    // Chebyshev points of [0, 1/4], relative error 2^-24): the error is then 2^-21 of the score itself.
    const float twice = p.cap_twice, c = p.cap_log2;
    if constexpr (EXT & kWide) {
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float t = s[j] * p.scale_log2, x = t * p.cap_inv, u = x * x;
        const float far = fmaf(-2.0f * c, rcp(1.0f + ex2(s[j] * twice)), c);
        const float near = t * fmaf(fmaf(fmaf(fmaf(0.0171313444f, u, -0.0529842388f), u, 0.133247505f), u, -0.333330679f), u, 1.0f);
        s[j] = u < 0.25f ? near : far;
      }
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j) s[j] = fmaf(-2.0f * c, rcp(1.0f + ex2(s[j] * twice)), c);
    }
  }
  if constexpr (EXT & kBias) {
    const float scale = EXT & kCap ? 1.0f : p.scale_log2;
    const float far = (float)(v.pos - key0);
#pragma unroll
    for (int j = 0; j < N; ++j) s[j] = fmaf(-v.slope, fabsf(far - (float)j), s[j] * scale);
  }
  if (!edge) return;
  const int hi = v.see_hi - key0, lo = v.see_lo - key0, pre = prefix - key0;
#pragma unroll
  for (int j = 0; j < N; ++j)
    if (!(j < pre || (j < hi && j >= lo))) s[j] = -INFINITY;
}

// 64 columns of scores.
__device__ __forceinline__ void load_scores(uint32_t addr, float (&s)[64]) {
  uint32_t a[32], b[32];
  tmem_ld32(a, addr);
  tmem_ld32(b, addr + 32);
  tmem_wait_ld();
  settle(a);
  settle(b);
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    s[j] = __uint_as_float(a[j]);
    s[32 + j] = __uint_as_float(b[j]);
  }
}

}  // namespace ar
