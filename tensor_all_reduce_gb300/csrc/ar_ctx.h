// The context and the host helpers that every file of the C ABI shares.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>
#include <stdio.h>

#include "ar.h"

struct ar_ctx {
  int device;
  int sm_count;
  int64_t l2_bytes;
  int max_cluster;       // largest cluster the fused kernel can be launched with
  int max_dyn_smem;      // opt-in dynamic shared memory per block (bytes)
  int* d_status;         // device status word of the staged kernel (0 = no timeout)
  // overrides (0 = automatic)
  int force_variant;
  int cluster_size;
  int ppt;
  int reduce_unroll;
  int stages;
  int pdl;               // launch with programmatic stream serialisation
  long long wait_cycles; // bound of one staged-kernel wait (0: about a second)
  int test_stall;        // test hook: make the staged kernel's first waits run out
  int prefetch;          // warm L2 with the first inputs before the grid-dependency wait
  int attn_mma_per_sm[2][3];  // resident CTAs of the general attention kernel: fp16/bf16, heads of 64/128/256
  int attn8_mma_per_sm[2][3]; // the same over a cache in 8 bits
  void* encode_tensor_map;    // the driver's cuTensorMapEncodeTiled; NULL: the driver has none, the general form serves
  cudaError_t serve_error;    // why the attention block's kernels could not be prepared
  const char* last_variant;
  char last_error[256];
};

namespace {

// Switch to the context's device for the duration of a call, restoring the caller's.
struct DeviceGuard {
  int prev = -1;
  bool changed = false;
  explicit DeviceGuard(int dev) {
    if (cudaGetDevice(&prev) == cudaSuccess && prev != dev) changed = cudaSetDevice(dev) == cudaSuccess;
  }
  ~DeviceGuard() {
    if (changed) cudaSetDevice(prev);
  }
};

inline int elem_size(ar_dtype d) { return d == AR_DTYPE_F32 ? 4 : 2; }

inline bool dtype_ok(int d) { return d == AR_DTYPE_F32 || d == AR_DTYPE_F16 || d == AR_DTYPE_BF16; }

inline uintptr_t addr(const void* p) { return reinterpret_cast<uintptr_t>(p); }

inline bool overlaps(const void* a, int64_t an, const void* b, int64_t bn) {
  if (an <= 0 || bn <= 0) return false;
  return addr(a) < addr(b) + (uintptr_t)bn && addr(b) < addr(a) + (uintptr_t)an;
}

inline bool aligned(const void* p, int bytes) { return (addr(p) % (uintptr_t)bytes) == 0; }

inline ar_status fail_cuda(ar_ctx* ctx, cudaError_t e, const char* what) {
  if (ctx) snprintf(ctx->last_error, sizeof(ctx->last_error), "%s: %s", what, cudaGetErrorString(e));
  return AR_ERR_CUDA;
}

inline ar_status launch(ar_ctx* ctx, const void* fn, dim3 grid, unsigned block, int csize, void** args,
                 size_t dyn_smem, void* stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block, 1, 1);
  cfg.dynamicSmemBytes = dyn_smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  unsigned na = 0;
  if (csize > 1) {
    attr[na].id = cudaLaunchAttributeClusterDimension;
    attr[na].val.clusterDim.x = (unsigned)csize;
    attr[na].val.clusterDim.y = 1;
    attr[na].val.clusterDim.z = 1;
    ++na;
  }
  if (ctx->pdl) {
    attr[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[na].val.programmaticStreamSerializationAllowed = 1;
    ++na;
  }
  cfg.attrs = na ? attr : nullptr;
  cfg.numAttrs = na;
  cudaError_t e = cudaLaunchKernelExC(&cfg, fn, args);
  if (e != cudaSuccess) return fail_cuda(ctx, e, "kernel launch");
  return AR_OK;
}

}  // namespace
