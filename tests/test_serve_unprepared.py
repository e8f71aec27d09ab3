"""A context whose attention block could not be prepared, without a GPU: a block of zeros laid out as the context by
the C++ compiler, with the error set.  The attention block's calls say so before they touch the device; the others
do not ask."""
import ctypes
import os
import shutil
import subprocess

import pytest

import tensor_all_reduce_gb300 as tar
import test_serve_host as host

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def unprepared(tmp_path_factory):
    from tensor_all_reduce_gb300 import _build
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if shutil.which("g++") is None or not os.path.exists(nvcc):
        pytest.skip("no compiler")
    _build.build()
    tmp = tmp_path_factory.mktemp("ctx")
    src = tmp / "layout.cpp"
    src.write_text('#include <stddef.h>\n#include "ar_ctx.h"\nint main() {\n'
                   'printf("%zu %zu %zu", sizeof(ar_ctx), offsetof(ar_ctx, serve_error), offsetof(ar_ctx, last_variant)); }\n')
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")
    subprocess.run(["g++", "-std=c++17", "-w", "-c", "-I", os.path.join(ROOT, "include"), "-I", os.path.join(ROOT, "tensor_all_reduce_gb300", "csrc"),
                    "-I", include, str(src), "-o", str(tmp / "layout.o")], check=True)
    subprocess.run(["g++", "-Wl,--unresolved-symbols=ignore-all", str(tmp / "layout.o"), "-o", str(tmp / "layout")], check=True)
    size, error, variant = map(int, subprocess.run([str(tmp / "layout")], capture_output=True, text=True, check=True, timeout=60).stdout.split())
    block = ctypes.create_string_buffer(size)
    ctypes.c_int.from_buffer(block, error).value = 999  # cudaErrorUnknown
    none = ctypes.create_string_buffer(b"none")
    ctypes.c_void_p.from_buffer(block, variant).value = ctypes.addressof(none)
    block.keep = none
    return block


@pytest.mark.parametrize("call, valid", [(tar.ar_paged_plan, "plan"), (tar.ar_qk_norm_rope, "rope"), (tar.ar_paged_attention, "attention")])
@pytest.mark.parametrize("empty", [False, True])
def test_the_calls_say_so(unprepared, monkeypatch, call, valid, empty):
    ctx = ctypes.addressof(unprepared)
    monkeypatch.setattr(tar, call.__name__, lambda _, args, stream, raise_on_error: call(ctx, args, stream, raise_on_error=raise_on_error))
    kw = dict(tokens=0) if empty and valid != "plan" else {}
    st = getattr(host, valid)(**kw)
    if kw:
        assert st == tar.AR_OK  # nothing to launch
        return
    assert st == tar.AR_ERR_CUDA
    assert "attention block" in tar.ar_last_error(ctx)


def test_the_others_do_not_ask(unprepared):
    ctx = ctypes.addressof(unprepared)
    n = ctypes.c_size_t()
    lib = tar.load_library()
    assert lib.ar_paged_attention_workspace(ctx, ctypes.byref(tar.ArPagedAttentionArgs(head_dim=64, dtype=tar.AR_DTYPE_BF16)), ctypes.byref(n)) == tar.AR_ERR_CUDA
    assert tar.ar_reduce_sum(ctx, 0, [0, 0], 0, tar.AR_DTYPE_BF16) == tar.AR_OK
    lib.ar_set_option(ctx, tar.AR_OPT_STAGES, 2)
    assert tar.ar_last_variant(ctx) == "none"
