"""Fused N-way partial reduce + residual add + RMSNorm (+ per-token FP8 E4M3) on GB300.

A thin ctypes binding over ``libar.so`` (see ``include/ar.h``).  The functions named like
the C ABI (``ar_init``, ``ar_reduce_sum``, ``ar_fused_reduce_rmsnorm``,
``ar_fused_reduce_rmsnorm_batch``, ``ar_fused_reduce_rmsnorm_host``,
``ar_fused_reduce_rmsnorm_noalloc``, ``ar_destroy`` ...) take raw pointers and sizes exactly
as the C functions do; the ``Context`` methods (``reduce_sum``, ``fused_reduce_rmsnorm``,
``fused_reduce_rmsnorm_batch``, ``fused_reduce_rmsnorm_host``) marshal torch tensors into
those calls.  The attention block between two fused calls is ``ar_paged_plan``,
``ar_qk_norm_rope`` and ``ar_paged_attention`` (methods ``paged_plan``, ``qk_norm_rope``,
``paged_attention``), over a cache held in 8 bits ``ar_paged_append_fp8`` and
``ar_paged_attention_fp8`` (``paged_append_fp8``, ``paged_attention_fp8``).  Every step of the computation runs in the library's CUDA kernels: there is no
Python or PyTorch compute path, and using the package without a built ``libar.so`` raises.
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import NamedTuple, Optional, Sequence

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libar.so")

# ---- mirrors of include/ar.h ----------------------------------------------
AR_OK = 0
AR_ERR_INVALID_ARG = 1
AR_ERR_UNSUPPORTED = 2
AR_ERR_ALIGNMENT = 3
AR_ERR_CUDA = 4
AR_ERR_NOT_INITIALIZED = 5
AR_ERR_OVERLAP = 6

AR_DTYPE_F32 = 0
AR_DTYPE_F16 = 1
AR_DTYPE_BF16 = 2
AR_MAX_PARTIALS = 8
AR_MAX_BATCH = 16
AR_QUANT_NONE = 0
AR_QUANT_FP8_E4M3_PER_TOKEN = 1
AR_QUANT_FP8_E4M3_PER_GROUP = 2

AR_OPT_FORCE_VARIANT = 0
AR_OPT_CLUSTER_SIZE = 1
AR_OPT_PACKS_PER_THREAD = 2
AR_OPT_REDUCE_UNROLL = 3
AR_OPT_STAGES = 4
AR_OPT_PDL = 5
AR_OPT_WAIT_CYCLES = 6
AR_OPT_TEST_STALL = 7
AR_OPT_L2_PREFETCH = 8
VARIANT_AUTO, VARIANT_ROW, VARIANT_CLUSTER, VARIANT_STAGED, VARIANT_SCALAR = 0, 1, 2, 3, 4

AR_INFO_SM_COUNT = 0
AR_INFO_L2_BYTES = 1
AR_INFO_REDUCE_TILE_PACKS = 2
AR_INFO_DEVICE = 3

AR_MAX_REQUESTS = 8192
AR_MAX_ROPE_AXES = 4
AR_MAX_HEAD_DIM = 256
AR_PLAN_OK = 0
AR_PLAN_NO_BLOCKS = 1
AR_PLAN_TABLE_FULL = 2
AR_PLAN_TOO_MANY_TOKENS = 3
AR_PLAN_BAD_LENGTH = 4


class ArFusedArgs(ctypes.Structure):
    _fields_ = [
        ("n", ctypes.c_int),
        ("partials", ctypes.c_void_p * AR_MAX_PARTIALS),
        ("residual_in", ctypes.c_void_p),
        ("residual_out", ctypes.c_void_p),
        ("weight", ctypes.c_void_p),
        ("out", ctypes.c_void_p),
        ("eps", ctypes.c_float),
        ("gemma", ctypes.c_int),
        ("quant", ctypes.c_int),
        ("q_out", ctypes.c_void_p),
        ("scale_out", ctypes.c_void_p),
        ("m", ctypes.c_int64),
        ("h", ctypes.c_int64),
        ("dtype", ctypes.c_int),
        ("skip_norm", ctypes.c_int),
        ("out_fp32", ctypes.c_int),
        ("group_size", ctypes.c_int),
        ("ld_in", ctypes.c_int64),
        ("ld_out", ctypes.c_int64),
    ]


def _fields(text):
    """ctypes fields from "type name name ..." lines: i int, l int64, f float, z size_t, p pointer."""
    kinds = {"i": ctypes.c_int, "l": ctypes.c_int64, "f": ctypes.c_float, "z": ctypes.c_size_t, "p": ctypes.c_void_p}
    return [(name, kinds[kind]) for kind, *names in map(str.split, text.strip().splitlines()) for name in names]


class ArPagedPlanArgs(ctypes.Structure):
    _fields_ = _fields("""
        i requests page_size
        l max_tokens free_capacity table_cols table_stride
        p cached_lens new_lens free_blocks free_count block_table cu_q seq_lens slots positions free_count_out info
    """)


class ArQkNormRopeArgs(ctypes.Structure):
    _fields_ = _fields("""
        l tokens
        i q_heads kv_heads head_dim dtype
        p q k v
        l q_token_stride q_head_stride k_token_stride k_head_stride v_token_stride v_head_stride
        p q_out k_out
        l q_out_token_stride q_out_head_stride k_out_token_stride k_out_head_stride
        p q_weight k_weight
        f eps
        i gemma rot_dim pairs axes
    """) + [("sections", ctypes.c_int * AR_MAX_ROPE_AXES)] + _fields("""
        i dealt
        p positions
        l position_stride
        p inv_freq k_cache v_cache
        l k_block_stride k_page_stride k_cache_head_stride v_block_stride v_page_stride v_cache_head_stride num_blocks
        i page_size
        p slots
    """)


class ArPagedAttentionArgs(ctypes.Structure):
    _fields_ = _fields("""
        l tokens
        i requests q_heads kv_heads head_dim dtype
        p q out
        l q_token_stride q_head_stride out_token_stride out_head_stride
        p lse k_cache v_cache
        l k_block_stride k_page_stride k_head_stride v_block_stride v_page_stride v_head_stride num_blocks
        i page_size
        p block_table
        l table_cols table_stride
        p cu_q seq_lens
        f scale
        i causal window
        f softcap
        p slopes prefix_lens workspace
        z workspace_bytes
    """)


class ArPagedAppendFp8Args(ctypes.Structure):
    _fields_ = _fields("""
        l tokens
        i requests kv_heads head_dim dtype
        p k v
        l k_token_stride k_head_stride v_token_stride v_head_stride
        p k_weight
        f eps
        i gemma rot_dim pairs axes
    """) + [("sections", ctypes.c_int * AR_MAX_ROPE_AXES)] + _fields("""
        i dealt
        p positions
        l position_stride
        p inv_freq k_cache v_cache
        l k_block_stride k_page_stride k_cache_head_stride v_block_stride v_page_stride v_cache_head_stride num_blocks
        i page_size
        p k_scale v_scale
        l k_scale_block_stride k_scale_head_stride v_scale_block_stride v_scale_head_stride
        p block_table
        l table_cols table_stride
        p cu_q seq_lens
    """)


class ArPagedAttentionFp8Args(ctypes.Structure):
    _fields_ = [("base", ArPagedAttentionArgs)] + _fields("""
        p k_scale v_scale
        l k_scale_block_stride k_scale_head_stride v_scale_block_stride v_scale_head_stride
    """)


def _packer(args):
    """pack(*values) of an argument structure's fields, as bytes that the C functions take for it
    (a third of the time of building the ctypes structure)."""
    codes = {ctypes.c_int: "i", ctypes.c_int64: "q", ctypes.c_float: "f", ctypes.c_size_t: "N", ctypes.c_void_p: "P",
             ctypes.c_int * AR_MAX_ROPE_AXES: f"{AR_MAX_ROPE_AXES}i"}

    def of(fields):
        return "".join(codes[kind] if kind in codes else of(kind._fields_) for _, kind in fields)

    return struct.Struct("@" + of(args._fields_)).pack


_pack_plan, _pack_rope, _pack_attention = map(_packer, (ArPagedPlanArgs, ArQkNormRopeArgs, ArPagedAttentionArgs))
_pack_append_fp8, _pack_attention_fp8 = map(_packer, (ArPagedAppendFp8Args, ArPagedAttentionFp8Args))
_NO_SECTIONS = (0,) * AR_MAX_ROPE_AXES
_NO_CACHES = (0, 0, 0, 0, 0, 0, 0, 0, 0, 1)
_KEPT_WORKSPACES = 8  # streams that a context keeps a workspace for


class PagedPlan(NamedTuple):
    """One step's plan (see ar_paged_plan): device tensors."""
    block_table: object
    cu_q: object
    seq_lens: object
    slots: object
    positions: object
    free_count: object
    info: object


class ArError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str = ""):
        self.status = status
        msg = f"{where}: {status_string(status)} ({status})"
        if detail:
            msg += f": {detail}"
        super().__init__(msg)


_lib: Optional[ctypes.CDLL] = None
_packed = {}  # C functions that take their arguments as packed bytes


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libar.so once.  Raises if it has not been built (no fallback exists)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it first (python -c 'import __graft_entry__ as g; g.build()')")
    lib = ctypes.CDLL(path)
    vp, i64, c_int = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    lib.ar_init.argtypes = [ctypes.POINTER(vp), c_int, ctypes.c_uint]
    lib.ar_destroy.argtypes = [vp]
    lib.ar_reduce_sum.argtypes = [vp, vp, ctypes.POINTER(vp), c_int, i64, c_int, vp]
    lib.ar_fused_reduce_rmsnorm.argtypes = [vp, ctypes.POINTER(ArFusedArgs), vp]
    lib.ar_fused_reduce_rmsnorm_host.argtypes = [vp, ctypes.POINTER(ArFusedArgs), vp]
    lib.ar_fused_reduce_rmsnorm_noalloc.argtypes = [ctypes.POINTER(ArFusedArgs), vp]
    lib.ar_status_string.argtypes = [c_int]
    lib.ar_status_string.restype = ctypes.c_char_p
    lib.ar_last_error.argtypes = [vp]
    lib.ar_last_error.restype = ctypes.c_char_p
    lib.ar_last_variant.argtypes = [vp]
    lib.ar_last_variant.restype = ctypes.c_char_p
    lib.ar_set_option.argtypes = [vp, c_int, i64]
    lib.ar_get_info.argtypes = [vp, c_int, ctypes.POINTER(i64)]
    lib.ar_device_status.argtypes = [vp, ctypes.POINTER(c_int)]
    lib.ar_fused_reduce_rmsnorm_batch.argtypes = [vp, ctypes.POINTER(ArFusedArgs), c_int, vp]
    lib.ar_paged_plan.argtypes = [vp, ctypes.POINTER(ArPagedPlanArgs), vp]
    lib.ar_qk_norm_rope.argtypes = [vp, ctypes.POINTER(ArQkNormRopeArgs), vp]
    lib.ar_paged_attention.argtypes = [vp, ctypes.POINTER(ArPagedAttentionArgs), vp]
    lib.ar_paged_attention_workspace.argtypes = [vp, ctypes.POINTER(ArPagedAttentionArgs),
                                                 ctypes.POINTER(ctypes.c_size_t)]
    lib.ar_paged_append_fp8.argtypes = [vp, ctypes.POINTER(ArPagedAppendFp8Args), vp]
    lib.ar_paged_attention_fp8.argtypes = [vp, ctypes.POINTER(ArPagedAttentionFp8Args), vp]
    for f in ("ar_paged_plan", "ar_qk_norm_rope", "ar_paged_attention", "ar_paged_attention_workspace",
              "ar_paged_append_fp8", "ar_paged_attention_fp8",
              "ar_init", "ar_destroy", "ar_reduce_sum", "ar_fused_reduce_rmsnorm", "ar_set_option",
              "ar_get_info", "ar_device_status", "ar_fused_reduce_rmsnorm_batch", "ar_fused_reduce_rmsnorm_host",
              "ar_fused_reduce_rmsnorm_noalloc"):
        getattr(lib, f).restype = c_int
    for f in ("ar_paged_plan", "ar_qk_norm_rope", "ar_paged_attention", "ar_paged_append_fp8", "ar_paged_attention_fp8"):
        _packed[f] = fn = lib[f]  # a function object of its own
        fn.argtypes, fn.restype = [vp, ctypes.c_char_p, vp], c_int
    _lib = lib
    return lib


def ar_status_string(status: int) -> str:
    return load_library().ar_status_string(int(status)).decode()


status_string = ar_status_string


# ---- the C ABI, one Python function per entry point -------------------------

def ar_init(device: int = 0, flags: int = 0) -> int:
    """Create a context; returns its opaque handle (an int)."""
    lib = load_library()
    h = ctypes.c_void_p()
    st = lib.ar_init(ctypes.byref(h), int(device), int(flags))
    if st != AR_OK:
        raise ArError(st, "ar_init")
    return h.value


def ar_destroy(ctx: Optional[int]) -> None:
    st = load_library().ar_destroy(ctx)
    if st != AR_OK:
        raise ArError(st, "ar_destroy")


def ar_last_variant(ctx: int) -> str:
    return load_library().ar_last_variant(ctx).decode()


def ar_last_error(ctx: int) -> str:
    return load_library().ar_last_error(ctx).decode()


def ar_set_option(ctx: int, opt: int, value: int) -> None:
    st = load_library().ar_set_option(ctx, int(opt), int(value))
    if st != AR_OK:
        raise ArError(st, "ar_set_option")


def ar_get_info(ctx: int, key: int) -> int:
    v = ctypes.c_int64()
    st = load_library().ar_get_info(ctx, int(key), ctypes.byref(v))
    if st != AR_OK:
        raise ArError(st, "ar_get_info")
    return v.value


def ar_device_status(ctx: int) -> int:
    """Read and clear the context's device status word (0: no bounded wait ran out)."""
    v = ctypes.c_int()
    st = load_library().ar_device_status(ctx, ctypes.byref(v))
    if st != AR_OK:
        raise ArError(st, "ar_device_status")
    return v.value


def _check(ctx, st, where):
    if st != AR_OK:
        raise ArError(st, where, ar_last_error(ctx) if (ctx and st == AR_ERR_CUDA) else "")


def ar_reduce_sum(ctx: int, out: int, partials: Sequence[int], numel: int, dtype: int,
                  stream: Optional[int] = None, raise_on_error: bool = True) -> int:
    """out[i] = round_T(sum_r partials[r][i]).  Pointers are device addresses (ints)."""
    n = len(partials)
    arr = (ctypes.c_void_p * max(n, 1))(*partials)
    st = load_library().ar_reduce_sum(ctx, out, arr, n, int(numel), int(dtype), stream)
    if raise_on_error:
        _check(ctx, st, "ar_reduce_sum")
    return st


def ar_fused_reduce_rmsnorm(ctx: int, args: ArFusedArgs, stream: Optional[int] = None,
                            raise_on_error: bool = True) -> int:
    st = load_library().ar_fused_reduce_rmsnorm(ctx, ctypes.byref(args), stream)
    if raise_on_error:
        _check(ctx, st, "ar_fused_reduce_rmsnorm")
    return st


def ar_fused_reduce_rmsnorm_host(ctx: int, args: ArFusedArgs, stream: Optional[int] = None,
                                 raise_on_error: bool = True) -> int:
    st = load_library().ar_fused_reduce_rmsnorm_host(ctx, ctypes.byref(args), stream)
    if raise_on_error:
        _check(ctx, st, "ar_fused_reduce_rmsnorm_host")
    return st


def ar_fused_reduce_rmsnorm_noalloc(args: ArFusedArgs, stream: Optional[int] = None,
                                    raise_on_error: bool = True) -> int:
    """The allocation-free form (no context; the calling thread's current device)."""
    st = load_library().ar_fused_reduce_rmsnorm_noalloc(ctypes.byref(args), stream)
    if raise_on_error:
        _check(None, st, "ar_fused_reduce_rmsnorm_noalloc")
    return st


def ar_fused_reduce_rmsnorm_batch(ctx: int, calls: Sequence[ArFusedArgs], stream: Optional[int] = None,
                                  raise_on_error: bool = True) -> int:
    arr = (ArFusedArgs * max(len(calls), 1))(*calls)
    st = load_library().ar_fused_reduce_rmsnorm_batch(ctx, arr, len(calls), stream)
    if raise_on_error:
        _check(ctx, st, "ar_fused_reduce_rmsnorm_batch")
    return st


def ar_paged_plan(ctx: int, args: ArPagedPlanArgs, stream: Optional[int] = None, raise_on_error: bool = True) -> int:
    st = (_lib or load_library()).ar_paged_plan(ctx, ctypes.byref(args), stream)
    if st != AR_OK and raise_on_error:
        _check(ctx, st, "ar_paged_plan")
    return st


def ar_qk_norm_rope(ctx: int, args: ArQkNormRopeArgs, stream: Optional[int] = None, raise_on_error: bool = True) -> int:
    st = (_lib or load_library()).ar_qk_norm_rope(ctx, ctypes.byref(args), stream)
    if st != AR_OK and raise_on_error:
        _check(ctx, st, "ar_qk_norm_rope")
    return st


def ar_paged_attention(ctx: int, args: ArPagedAttentionArgs, stream: Optional[int] = None,
                       raise_on_error: bool = True) -> int:
    st = (_lib or load_library()).ar_paged_attention(ctx, ctypes.byref(args), stream)
    if st != AR_OK and raise_on_error:
        _check(ctx, st, "ar_paged_attention")
    return st


def ar_paged_append_fp8(ctx: int, args: ArPagedAppendFp8Args, stream: Optional[int] = None,
                        raise_on_error: bool = True) -> int:
    st = (_lib or load_library()).ar_paged_append_fp8(ctx, ctypes.byref(args), stream)
    if st != AR_OK and raise_on_error:
        _check(ctx, st, "ar_paged_append_fp8")
    return st


def ar_paged_attention_fp8(ctx: int, args: ArPagedAttentionFp8Args, stream: Optional[int] = None,
                           raise_on_error: bool = True) -> int:
    st = (_lib or load_library()).ar_paged_attention_fp8(ctx, ctypes.byref(args), stream)
    if st != AR_OK and raise_on_error:
        _check(ctx, st, "ar_paged_attention_fp8")
    return st


def ar_paged_attention_workspace(ctx: int, args: ArPagedAttentionArgs) -> int:
    """Bytes of workspace for calls with the head size and element type of `args`."""
    n = ctypes.c_size_t()
    st = load_library().ar_paged_attention_workspace(ctx, ctypes.byref(args), ctypes.byref(n))
    if st != AR_OK:
        raise ArError(st, "ar_paged_attention_workspace")
    return n.value


def make_fused_args(partials: Sequence[int], residual_in: Optional[int], residual_out: Optional[int],
                    weight: Optional[int], out: Optional[int], eps: float, gemma: bool, quant: bool,
                    q_out: Optional[int], scale_out: Optional[int], m: int, h: int, dtype: int,
                    skip_norm: bool = False, out_fp32: bool = False, group_size: int = 0,
                    ld_in: int = 0, ld_out: int = 0) -> ArFusedArgs:
    a = ArFusedArgs()
    a.n = len(partials)
    for i, p in enumerate(partials):
        a.partials[i] = p
    a.residual_in = residual_in
    a.residual_out = residual_out
    a.weight = weight
    a.out = out
    a.eps = eps
    a.gemma = int(bool(gemma))
    a.quant = (AR_QUANT_FP8_E4M3_PER_GROUP if group_size else AR_QUANT_FP8_E4M3_PER_TOKEN) if quant else AR_QUANT_NONE
    a.group_size = int(group_size)
    a.ld_in = int(ld_in)
    a.ld_out = int(ld_out)
    a.q_out = q_out
    a.scale_out = scale_out
    a.m = m
    a.h = h
    a.dtype = dtype
    a.skip_norm = int(bool(skip_norm))
    a.out_fp32 = int(bool(out_fp32))
    return a


# ---- torch marshalling -----------------------------------------------------

def _torch_dtype_code(t) -> int:
    import torch
    return {torch.float32: AR_DTYPE_F32, torch.float16: AR_DTYPE_F16, torch.bfloat16: AR_DTYPE_BF16}[t.dtype]


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream) -> int:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _row_stride(tensors, m, h, dtype, what, host: bool = False) -> int:
    """The common row stride (in elements) of [m, h] CUDA tensors (with `host`, CUDA or
    pinned host tensors) with unit column stride."""
    ld = None
    for t in tensors:
        if t is None:
            continue
        placed = t.is_cuda or (host and t.is_pinned())
        if t.shape != (m, h) or not placed or (dtype is not None and t.dtype != dtype) or \
                (h > 1 and t.stride(1) != 1) or (m > 1 and t.stride(0) < h):
            kind = "CUDA or pinned host" if host else "CUDA"
            raise ValueError(f"{what} must be [m, h] {kind} tensors with unit column stride")
        s = t.stride(0) if m > 1 else h
        if ld is not None and s != ld:
            raise ValueError(f"{what} must share one row stride")
        ld = s
    return h if ld is None else ld


# What the attention block's methods need of torch, bound at the first use (importing this
# package does not import torch).
class _Torch:
    def __init__(self):
        import torch
        self.i32, self.i64, self.f32, self.u8 = torch.int32, torch.int64, torch.float32, torch.uint8
        self.codes = {torch.bfloat16: AR_DTYPE_BF16, torch.float16: AR_DTYPE_F16}
        self.e4m3 = (torch.float8_e4m3fn, torch.uint8)
        self.empty, self.device, self.use_stream = torch.empty, torch.device, torch.cuda.stream
        self.raw_stream = torch._C._cuda_getCurrentRawStream
        self.capturing = torch.cuda.is_current_stream_capturing


_torch: Optional[_Torch] = None


def _bind_torch() -> _Torch:
    global _torch
    if _torch is None:
        _torch = _Torch()
    return _torch


def _flat(t, dtype, n, device, what) -> int:
    """Address (0 for None) of a contiguous CUDA tensor of `n` elements (None: any number) on `device`."""
    if t is None:
        return 0
    if t.dtype is not dtype or t.get_device() != device or not t.is_contiguous() or (n is not None and t.numel() != n):
        raise ValueError(f"{what} must be a contiguous {dtype} tensor on cuda:{device}"
                         + ("" if n is None else f" with {n} elements"))
    return t.data_ptr()


def _heads(t, shape, dtype, device, what):
    """(address, token stride, head stride) of a [tokens, heads, dim] tensor with unit last stride."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != device:
        raise ValueError(f"{what} must be a {list(shape)} {dtype} tensor on cuda:{device}")
    ts, hs, one = t.stride()
    if one != 1 and shape[2] > 1:
        raise ValueError(f"{what} must have unit stride in its last dimension")
    return t.data_ptr(), ts, hs


def _caches(k, v, heads, dim, dtype, device):
    """(k address, v address, k's block, token and head strides, v's, blocks, page) of two
    [blocks, page, heads, dim] caches."""
    shape = k.shape
    if len(shape) != 4 or shape[2] != heads or shape[3] != dim or v.shape != shape or k.dtype is not dtype or \
            v.dtype is not dtype or k.get_device() != device or v.get_device() != device:
        raise ValueError(f"k_cache and v_cache must be [blocks, page, {heads}, {dim}] {dtype} tensors on cuda:{device}")
    kb, kp, kh, one = k.stride()
    vb, vp, vh, one_v = v.stride()
    if (one != 1 or one_v != 1) and dim > 1:
        raise ValueError("k_cache and v_cache must have unit stride in their last dimension")
    return k.data_ptr(), v.data_ptr(), kb, kp, kh, vb, vp, vh, shape[0], shape[1]


def _caches_fp8(k, v, heads, dim, device):
    """_caches of two caches of E4M3 codes (float8_e4m3fn or uint8)."""
    if k.dtype not in _torch.e4m3 or v.dtype not in _torch.e4m3:
        raise ValueError("k_cache and v_cache must be float8_e4m3fn (or uint8) tensors")
    if k.dtype is not v.dtype:
        k, v = k.view(_torch.u8), v.view(_torch.u8)
    return _caches(k, v, heads, dim, k.dtype, device)


def _scales(k, v, blocks, heads, device):
    """(k address, v address, k's block and head strides, v's) of two [blocks, heads] fp32 tensors."""
    shape = (blocks, heads)
    for t in (k, v):
        if t.shape != shape or t.dtype is not _torch.f32 or t.get_device() != device:
            raise ValueError(f"k_scale and v_scale must be {list(shape)} float32 tensors on cuda:{device}")
    return (k.data_ptr(), v.data_ptr(), *k.stride(), *v.stride())


def _table(t, requests, device):
    """(address, columns, row stride) of a [requests, columns] int32 block table."""
    shape = t.shape
    if len(shape) != 2 or shape[0] != requests or t.dtype is not _torch.i32 or t.get_device() != device:
        raise ValueError(f"block_table must be a [{requests}, columns] int32 tensor on cuda:{device}")
    rows, one = t.stride()
    if (shape[1] > 1 and one != 1) or (requests > 1 and rows < shape[1]):
        raise ValueError("block_table must have unit stride in its rows, and rows that do not overlap")
    return t.data_ptr(), shape[1], rows if requests > 1 else 0


class Context:
    """Owns one ar_ctx for a device; torch-tensor front end of the C ABI."""

    def __init__(self, device: int = 0):
        self.device = device
        self.handle = ar_init(device)
        self._workspace_bytes = {}
        self._torch_device = None
        self._workspaces = {}

    def close(self):
        if self.handle:
            ar_destroy(self.handle)
            self.handle = None
            self._workspaces = {}

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def last_variant(self) -> str:
        return ar_last_variant(self.handle)

    def set_option(self, opt: int, value: int):
        ar_set_option(self.handle, opt, value)

    def info(self, key: int) -> int:
        return ar_get_info(self.handle, key)

    def device_status(self) -> int:
        return ar_device_status(self.handle)

    def reduce_sum(self, partials, out=None, stream=None):
        """Sum contiguous same-shaped device tensors in rank order; returns `out`."""
        import torch
        x0 = partials[0]
        for p in partials:
            if p.shape != x0.shape or p.dtype != x0.dtype or not p.is_contiguous() or not p.is_cuda:
                raise ValueError("partials must be contiguous CUDA tensors of one shape and dtype")
        if out is None:
            out = torch.empty_like(x0)
        ar_reduce_sum(self.handle, out.data_ptr(), [p.data_ptr() for p in partials], x0.numel(),
                      _torch_dtype_code(x0), _stream(stream))
        return out

    def fused_reduce_rmsnorm(self, partials, residual, weight, eps: float = 1e-6, gemma: bool = False,
                             quant: bool = False, out=None, residual_out=None, q_out=None, scale_out=None,
                             want_out: bool = True, want_residual_out: bool = True, stream=None,
                             skip_norm: bool = False, out_fp32: bool = False, group_size: int = 0):
        """Returns (out, residual_out, q_out, scale_out); absent outputs are None.  With
        skip_norm there is no RMSNorm (weight may be None); with out_fp32 `out` is float32.
        Inputs (and given outputs) may have padded rows: unit column stride, one row stride
        for the inputs and one for the outputs; allocated outputs are contiguous."""
        return self._fused(False, partials, residual, weight, eps, gemma, quant, out, residual_out, q_out,
                           scale_out, want_out, want_residual_out, stream, skip_norm, out_fp32, group_size)

    def fused_reduce_rmsnorm_host(self, partials, residual, weight, eps: float = 1e-6, gemma: bool = False,
                                  quant: bool = False, out=None, residual_out=None, q_out=None, scale_out=None,
                                  want_out: bool = True, want_residual_out: bool = True, stream=None,
                                  skip_norm: bool = False, out_fp32: bool = False, group_size: int = 0):
        """fused_reduce_rmsnorm where tensors may be pinned host tensors (or CUDA tensors of
        this device): the kernel reads and writes host memory directly.  Outputs it allocates
        are pinned host tensors.  Asynchronous: synchronise `stream` before reading them."""
        return self._fused(True, partials, residual, weight, eps, gemma, quant, out, residual_out, q_out,
                           scale_out, want_out, want_residual_out, stream, skip_norm, out_fp32, group_size)

    def _fused(self, host, partials, residual, weight, eps, gemma, quant, out, residual_out, q_out, scale_out,
               want_out, want_residual_out, stream, skip_norm, out_fp32, group_size):
        import torch
        x0 = partials[0]
        m, h = x0.shape

        def alloc(shape, dtype):
            if host:
                return torch.empty(shape, dtype=dtype, pin_memory=True)
            return torch.empty(shape, dtype=dtype, device=x0.device)

        ld_in = _row_stride([*partials, residual], m, h, x0.dtype, "partials and residual", host)
        given = [t for t in (out, residual_out, q_out) if t is not None]
        ld_out = _row_stride(given, m, h, None, "outputs", host) if given else h
        if ld_out != h and ((out is None and (want_out or not quant)) or (residual_out is None and want_residual_out)
                            or (quant and q_out is None)):
            raise ValueError("with padded outputs every output must be given")
        if out is None and (want_out or not quant):
            out = alloc((m, h), torch.float32 if out_fp32 else x0.dtype)
        if residual_out is None and want_residual_out:
            residual_out = alloc((m, h), x0.dtype)
        if quant:
            if q_out is None:
                q_out = alloc((m, h), torch.uint8)
            if scale_out is None:
                scale_out = alloc((m, h // group_size) if group_size else (m,), torch.float32)
        args = make_fused_args([p.data_ptr() for p in partials], _ptr(residual), _ptr(residual_out),
                               _ptr(weight), _ptr(out), eps, gemma, quant, _ptr(q_out), _ptr(scale_out),
                               m, h, _torch_dtype_code(x0), skip_norm=skip_norm, out_fp32=out_fp32,
                               group_size=group_size, ld_in=ld_in, ld_out=ld_out)
        (ar_fused_reduce_rmsnorm_host if host else ar_fused_reduce_rmsnorm)(self.handle, args, _stream(stream))
        return out, residual_out, q_out, scale_out

    def fused_reduce_rmsnorm_batch(self, calls, stream=None):
        """Several independent fused calls in one launch.  `calls` is a list of dicts with the
        keyword arguments of fused_reduce_rmsnorm (partials, residual, weight, eps, gemma,
        quant, out, residual_out, q_out, scale_out, skip_norm, out_fp32); missing outputs are
        allocated.  Returns a list of (out, residual_out, q_out, scale_out)."""
        import torch
        results, args = [], []
        for c in calls:
            x0 = c["partials"][0]
            m, h = x0.shape
            quant, out_fp32 = c.get("quant", False), c.get("out_fp32", False)
            out = c.get("out")
            if out is None and (c.get("want_out", True) or not quant):
                out = torch.empty((m, h), dtype=torch.float32 if out_fp32 else x0.dtype, device=x0.device)
            ro = c.get("residual_out")
            if ro is None and c.get("want_residual_out", True):
                ro = torch.empty_like(x0)
            q = c.get("q_out")
            sc = c.get("scale_out")
            g = c.get("group_size", 0)
            if quant:
                q = q if q is not None else torch.empty((m, h), dtype=torch.uint8, device=x0.device)
                sc = sc if sc is not None else torch.empty((m, h // g) if g else (m,), dtype=torch.float32,
                                                           device=x0.device)
            ld_in = _row_stride([*c["partials"], c.get("residual")], m, h, x0.dtype, "partials and residual")
            outs = [t for t in (out, ro, q) if t is not None]
            ld_out = _row_stride(outs, m, h, None, "outputs") if outs else h
            args.append(make_fused_args([p.data_ptr() for p in c["partials"]], _ptr(c.get("residual")), _ptr(ro),
                                        _ptr(c.get("weight")), _ptr(out), c.get("eps", 1e-6), c.get("gemma", False),
                                        quant, _ptr(q), _ptr(sc), m, h, _torch_dtype_code(x0),
                                        skip_norm=c.get("skip_norm", False), out_fp32=out_fp32, group_size=g,
                                        ld_in=ld_in, ld_out=ld_out))
            results.append((out, ro, q, sc))
        ar_fused_reduce_rmsnorm_batch(self.handle, args, _stream(stream))
        return results

    # ---- the attention block ------------------------------------------------

    def _raw_stream(self, stream) -> int:
        if stream is None:
            return _torch.raw_stream(self.device)
        if stream.device.index != self.device:
            raise ValueError(f"the stream belongs to another device than cuda:{self.device}")
        return stream.cuda_stream

    def _empty(self, shape, dtype, stream):
        """An output on this device that belongs to `stream` (None: the current one)."""
        t = _bind_torch()
        if stream is None:
            return t.empty(shape, dtype=dtype, device=self._torch_device or self._make_torch_device())
        with t.use_stream(stream):
            return t.empty(shape, dtype=dtype, device=self._torch_device or self._make_torch_device())

    def _call(self, name, packed, stream):
        st = _packed[name](self.handle, packed, self._raw_stream(stream))
        if st != AR_OK:
            _check(self.handle, st, name)

    def _make_torch_device(self):
        self._torch_device = _torch.device("cuda", self.device)
        return self._torch_device

    def paged_plan(self, cached_lens, new_lens, free_blocks, free_count, block_table, page_size: int,
                   max_tokens: Optional[int] = None, cu_q=None, seq_lens=None, slots=None, positions=None,
                   free_count_out=None, info=None, stream=None) -> PagedPlan:
        """Block tables and slot maps of one step from int32 length tensors (see ar_paged_plan).
        `block_table` [requests, columns] is updated in place; the others are returned, allocated
        where not given.  `max_tokens` is the length of slots and positions (needed unless one of
        them is given); free_count_out must not be free_count itself."""
        t = _torch or _bind_torch()
        dev, i32, r = self.device, t.i32, cached_lens.numel()
        if max_tokens is None:
            given = slots if slots is not None else positions
            if given is None:
                raise ValueError("max_tokens, slots or positions must be given")
            max_tokens = given.numel()
        if cu_q is None:
            cu_q = self._empty((r + 1,), i32, stream)
        if seq_lens is None:
            seq_lens = self._empty((r,), i32, stream)
        if slots is None:
            slots = self._empty((max_tokens,), t.i64, stream)
        if positions is None:
            positions = self._empty((max_tokens,), i32, stream)
        if free_count_out is None:
            free_count_out = self._empty((1,), i32, stream)
        if info is None:
            info = self._empty((4,), i32, stream)
        table, cols, stride = _table(block_table, r, dev)
        args = _pack_plan(
            r, page_size, max_tokens, free_blocks.numel(), cols, stride,
            _flat(cached_lens, i32, r, dev, "cached_lens"), _flat(new_lens, i32, r, dev, "new_lens"),
            _flat(free_blocks, i32, None, dev, "free_blocks"), _flat(free_count, i32, 1, dev, "free_count"),
            table, _flat(cu_q, i32, r + 1, dev, "cu_q"), _flat(seq_lens, i32, r, dev, "seq_lens"),
            _flat(slots, t.i64, max_tokens, dev, "slots"), _flat(positions, i32, max_tokens, dev, "positions"),
            _flat(free_count_out, i32, 1, dev, "free_count_out"), _flat(info, i32, 4, dev, "info"))
        self._call("ar_paged_plan", args, stream)
        return PagedPlan(block_table, cu_q, seq_lens, slots, positions, free_count_out, info)

    def _rotation(self, positions, inv_freq, sections, n, where):
        """(frequencies, axes, sections, address and row stride of positions, address of inv_freq)."""
        t, dev = _torch, self.device
        half, axes, pos, pos_stride, freq = 0, 1, 0, 0, 0
        sec = _NO_SECTIONS
        if inv_freq is not None:
            half = inv_freq.numel()
            freq = _flat(inv_freq, t.f32, half, dev, "inv_freq")
        if half and positions is not None:
            shape = positions.shape
            if positions.dtype is not t.i32 or positions.get_device() != dev or len(shape) not in (1, 2) or \
                    shape[-1] != n or (n > 1 and positions.stride(-1) != 1):
                raise ValueError(f"positions must be a [{n}] or [axes, {n}] int32 tensor on cuda:{dev}, unit stride")
            pos = positions.data_ptr()
            if len(shape) == 2:
                axes = shape[0]
                if axes > 1:
                    pos_stride = positions.stride(0)
                    if axes > AR_MAX_ROPE_AXES:
                        raise ValueError(f"positions must have 1 to {AR_MAX_ROPE_AXES} axes")
                    if sections is None or len(sections) != axes:
                        raise ValueError("sections must name the frequencies of each position axis")
                    if pos_stride:
                        sec = (*sections, *_NO_SECTIONS[axes:])
                    else:  # one row for all axes (an expanded view) is the rotation by one axis; the C call takes 0 for `tokens`
                        if sum(sections) != half or min(sections) < 0:
                            raise ArError(AR_ERR_INVALID_ARG, where, "sections must add up to the frequencies")
                        axes = 1
                elif axes < 1:
                    raise ValueError(f"positions must have 1 to {AR_MAX_ROPE_AXES} axes")
        return half, axes, sec, pos, pos_stride, freq

    def qk_norm_rope(self, q, k, v, positions, inv_freq, q_weight=None, k_weight=None, eps: float = 1e-6,
                     gemma: bool = False, pairs: bool = False, sections: Optional[Sequence[int]] = None,
                     dealt: bool = False, k_cache=None, v_cache=None, slots=None, q_out=None, k_out=None,
                     want_k_out: bool = True, stream=None):
        """RMSNorm of each q and k head (where its weight is given), rotation by `positions`
        ([tokens] or [axes, tokens] int32) with the fp32 frequencies `inv_freq` (None: none), and
        the write of k and v to the paged cache at `slots` (see ar_qk_norm_rope).  q, k, v are
        [tokens, heads, head_dim] and may be views of one packed projection; q or k may be None.
        Positions that all axes share may be an expanded row.
        Returns (q_out, k_out); with a cache, want_k_out=False leaves k_out out (None)."""
        t = _torch or _bind_torch()
        dev = self.device
        x0 = q if q is not None else k
        if x0 is None:
            raise ValueError("q or k must be given")
        n, heads, d = x0.shape
        dt = x0.dtype
        code = t.codes.get(dt)
        if code is None:
            raise ValueError("q, k and v must be bfloat16 or float16")
        hq, hk = (0 if q is None else heads), (0 if k is None else k.shape[1])
        qp = kp = vp = qop = kop = slot = 0
        qt = qh = kt = kh = vt = vh = qot = qoh = kot = koh = 0
        if hq:
            shape = (n, hq, d)
            qp, qt, qh = _heads(q, shape, dt, dev, "q")
            if q_out is None:
                q_out = self._empty(shape, dt, stream)
            qop, qot, qoh = _heads(q_out, shape, dt, dev, "q_out")
        caches = _NO_CACHES
        if (k_cache is None) != (v_cache is None):
            raise ValueError("k_cache and v_cache are given together")
        if hk:
            shape = (n, hk, d)
            kp, kt, kh = _heads(k, shape, dt, dev, "k")
            if k_out is None and (want_k_out or k_cache is None):
                k_out = self._empty(shape, dt, stream)
            if k_out is not None:
                kop, kot, koh = _heads(k_out, shape, dt, dev, "k_out")
        if k_cache is not None:
            if not hk or v is None or slots is None:
                raise ValueError("a cache needs k, v and slots")
            vp, vt, vh = _heads(v, shape, dt, dev, "v")
            caches = _caches(k_cache, v_cache, hk, d, dt, dev)
            slot = _flat(slots, t.i64, n, dev, "slots")
        half, axes, sec, pos, pos_stride, freq = self._rotation(positions, inv_freq, sections, n, "ar_qk_norm_rope")
        args = _pack_rope(
            n, hq, hk, d, code, qp, kp, vp, qt, qh, kt, kh, vt, vh, qop, kop, qot, qoh, kot, koh,
            0 if q_weight is None else _flat(q_weight, dt, d, dev, "q_weight"),
            0 if k_weight is None else _flat(k_weight, dt, d, dev, "k_weight"),
            eps, gemma, 2 * half, pairs, axes, *sec, dealt, pos, pos_stride, freq, *caches, slot)
        self._call("ar_qk_norm_rope", args, stream)
        return q_out, k_out

    def paged_attention(self, q, k_cache, v_cache, block_table, cu_q, seq_lens, scale: Optional[float] = None,
                        causal: bool = True, window: int = 0, softcap: float = 0.0, slopes=None, prefix_lens=None,
                        out=None, lse=None, want_lse: bool = False, workspace=None, stream=None):
        """Attention of the requests' new tokens q [tokens, q_heads, head_dim] over the paged
        cache [blocks, page, kv_heads, head_dim] (see ar_paged_attention); scale defaults to
        head_dim ** -0.5.  Returns (out, lse); lse [tokens, q_heads] fp32 is None unless given or
        wanted.  Rows of no request are not written.  `workspace` is a uint8 tensor from
        paged_attention_workspace; calls that may run at the same time need one each.  Where it is not
        given the context keeps one (up to 40 MB) for each of the last eight streams that called, until
        release_workspaces or close, and a captured call allocates its own."""
        return self._attention(None, q, k_cache, v_cache, block_table, cu_q, seq_lens, scale, causal, window, softcap,
                               slopes, prefix_lens, out, lse, want_lse, workspace, stream)

    def paged_attention_fp8(self, q, k_cache, v_cache, k_scale, v_scale, block_table, cu_q, seq_lens,
                            scale: Optional[float] = None, causal: bool = True, window: int = 0, softcap: float = 0.0,
                            slopes=None, prefix_lens=None, out=None, lse=None, want_lse: bool = False, workspace=None,
                            stream=None):
        """paged_attention over a cache of E4M3 codes (float8_e4m3fn or uint8) with one fp32 scale a block
        and head, k_scale and v_scale [blocks, kv_heads] (see ar_paged_attention_fp8)."""
        return self._attention((k_scale, v_scale), q, k_cache, v_cache, block_table, cu_q, seq_lens, scale, causal, window,
                               softcap, slopes, prefix_lens, out, lse, want_lse, workspace, stream)

    def _attention(self, scales, q, k_cache, v_cache, block_table, cu_q, seq_lens, scale, causal, window, softcap, slopes,
                   prefix_lens, out, lse, want_lse, workspace, stream):
        t = _torch or _bind_torch()
        dev = self.device
        shape = q.shape
        n, hq, d = shape
        dt = q.dtype
        code = t.codes.get(dt)
        if code is None:
            raise ValueError("q must be bfloat16 or float16")
        r, hk = seq_lens.numel(), k_cache.shape[2]
        if hk < 1 or hq % hk:
            raise ValueError("q_heads must be a multiple of kv_heads")
        if out is None:
            out = self._empty(shape, dt, stream)
        if lse is None and want_lse:
            lse = self._empty((n, hq), t.f32, stream)
        if workspace is None:
            size = self._attention_workspace(d, code)
            workspace = self._own_workspace(size, stream)
            work = workspace.data_ptr()
        else:
            work, size = _flat(workspace, t.u8, None, dev, "workspace"), workspace.numel()
        qp, qt, qh = _heads(q, shape, dt, dev, "q")
        op, ot, oh = _heads(out, shape, dt, dev, "out")
        kp, vp, kb, kt, kh, vb, vt, vh, blocks, page = \
            _caches(k_cache, v_cache, hk, d, dt, dev) if scales is None else _caches_fp8(k_cache, v_cache, hk, d, dev)
        table, cols, stride = _table(block_table, r, dev)
        args = (
            n, r, hq, hk, d, code, qp, op, qt, qh, ot, oh,
            0 if lse is None else _flat(lse, t.f32, n * hq, dev, "lse"), kp, vp, kb, kt, kh, vb, vt, vh, blocks, page,
            table, cols, stride, _flat(cu_q, t.i32, r + 1, dev, "cu_q"), _flat(seq_lens, t.i32, r, dev, "seq_lens"),
            d ** -0.5 if scale is None else scale, causal, window, softcap,
            0 if slopes is None else _flat(slopes, t.f32, hq, dev, "slopes"),
            0 if prefix_lens is None else _flat(prefix_lens, t.i32, r, dev, "prefix_lens"), work, size)
        if scales is None:
            self._call("ar_paged_attention", _pack_attention(*args), stream)
        else:
            self._call("ar_paged_attention_fp8", _pack_attention_fp8(*args, *_scales(*scales, blocks, hk, dev)), stream)
        return out, lse

    def paged_append_fp8(self, k, v, k_cache, v_cache, k_scale, v_scale, block_table, cu_q, seq_lens, positions=None,
                         inv_freq=None, k_weight=None, eps: float = 1e-6, gemma: bool = False, pairs: bool = False,
                         sections: Optional[Sequence[int]] = None, dealt: bool = False, stream=None) -> None:
        """Appends the requests' new tokens k and v [tokens, kv_heads, head_dim] to a paged cache of E4M3 codes
        (float8_e4m3fn or uint8) with one fp32 scale a block and head, k_scale and v_scale [blocks, kv_heads], all
        updated in place (see ar_paged_append_fp8).  k gets RMSNorm (where k_weight is given) and the rotation of
        qk_norm_rope (where inv_freq is given) on the way; positions default to each token's place in its
        request.  q's norm and rotation are qk_norm_rope's, with k None."""
        t = _torch or _bind_torch()
        dev = self.device
        n, hk, d = shape = k.shape
        dt = k.dtype
        code = t.codes.get(dt)
        if code is None:
            raise ValueError("k and v must be bfloat16 or float16")
        r = seq_lens.numel()
        kp, kt, kh = _heads(k, shape, dt, dev, "k")
        vp, vt, vh = _heads(v, shape, dt, dev, "v")
        caches = _caches_fp8(k_cache, v_cache, hk, d, dev)
        if positions is None and sections is not None and len(sections) > 1:
            raise ValueError("several position axes need positions")
        half, axes, sec, pos, pos_stride, freq = self._rotation(positions, inv_freq, sections, n, "ar_paged_append_fp8")
        table, cols, stride = _table(block_table, r, dev)
        args = _pack_append_fp8(
            n, r, hk, d, code, kp, vp, kt, kh, vt, vh, 0 if k_weight is None else _flat(k_weight, dt, d, dev, "k_weight"),
            eps, gemma, 2 * half, pairs, axes, *sec, dealt, pos, pos_stride, freq, *caches,
            *_scales(k_scale, v_scale, caches[8], hk, dev), table, cols, stride,
            _flat(cu_q, t.i32, r + 1, dev, "cu_q"), _flat(seq_lens, t.i32, r, dev, "seq_lens"))
        self._call("ar_paged_append_fp8", args, stream)

    def _own_workspace(self, size: int, stream):
        """`size` bytes for one call on `stream`: kept for the calls behind it on that stream, which
        cannot overlap it; a captured call gets its own, which belongs to its graph."""
        if stream is not None:
            with _torch.use_stream(stream):
                return self._own_workspace(size, None)
        if _torch.capturing():
            return self._empty(size, _torch.u8, None)
        key = _torch.raw_stream(self.device)
        kept = self._workspaces.pop(key, None)
        if kept is None or kept.numel() < size:
            kept = self._empty(size, _torch.u8, None)
        self._workspaces[key] = kept  # the last used one stands last
        if len(self._workspaces) > _KEPT_WORKSPACES:
            # back to torch's allocator, which hands it out on its own stream only, behind the calls that use it
            del self._workspaces[next(iter(self._workspaces))]
        return kept

    def release_workspaces(self):
        """Gives the workspaces kept for paged_attention and paged_attention_fp8 back to torch's allocator."""
        self._workspaces.clear()

    def _attention_workspace(self, head_dim: int, code: int) -> int:
        n = self._workspace_bytes.get((head_dim, code))
        if n is None:
            n = self._workspace_bytes[head_dim, code] = ar_paged_attention_workspace(
                self.handle, ArPagedAttentionArgs(head_dim=head_dim, dtype=code))
        return n

    def paged_attention_workspace(self, head_dim: int, dtype):
        """A workspace for paged_attention and paged_attention_fp8 calls with this head size and element type, of any lengths."""
        t = _bind_torch()
        return self._empty(self._attention_workspace(head_dim, t.codes[dtype]), t.u8, None)
