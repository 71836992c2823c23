"""The C entry points of the 4-bit products (coli_linear.h) and of 8-bit caches (coli_attn.h) refuse what they do not take before they
touch a GPU.  CPU only."""
import ctypes
import os
import re
import shutil

import pytest
import torch

from int4_routed_expert_quantize_gb300 import _build, attn, coli, linear


@pytest.fixture(scope="module", autouse=True)
def built():
    if shutil.which("nvcc") is None:
        pytest.skip("nvcc not available")
    if _build.is_stale():
        _build.build()
        coli._lib = None
    return linear.lib()


def create(**kw):
    base = dict(rows=16, cols=256, group=64, dtype=0, max_tokens=4)
    base.update(kw)
    cfg = linear.LinearConfig(*[base[f] for f, _ in linear.LinearConfig._fields_])
    h = ctypes.c_void_p(1)
    rc = linear.lib().coli_linear_create(ctypes.byref(cfg), ctypes.byref(h))
    if rc == 0:
        linear.lib().coli_linear_destroy(h)
        return 0, None
    return rc, h.value


@pytest.mark.parametrize("kw,expect", [
    (dict(rows=0), -1), (dict(rows=2 ** 24 + 1), -1), (dict(cols=0), -1), (dict(cols=96), -1), (dict(group=0), -1),
    (dict(max_tokens=0), -1), (dict(max_tokens=1000001), -1), (dict(group=16), -6), (dict(group=256), -6), (dict(dtype=2), -6),
    (dict(cols=32832), -6)])
def test_create_rejects(kw, expect):
    assert create(**kw) == (expect, None)


def test_create_without_gpu_reports_cuda_error():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert create() == (-4, None)


def test_null_arguments():
    L, h = linear.lib(), ctypes.c_void_p()
    assert L.coli_linear_create(None, ctypes.byref(h)) == -1 and L.coli_linear_create(None, None) == -1
    assert L.coli_linear_load(None, 16, 16, None) == -1 and L.coli_linear_status(None, None) == -1
    assert L.coli_linear_forward(None, 16, 256, 1, 16, 16, None) == -1
    L.coli_linear_destroy(None)
    out = ctypes.c_void_p(1)
    assert L.coli_attn_qcache_bind(None, ctypes.byref(attn.AttnQCache()), ctypes.byref(out)) == -1 and out.value is None
    assert L.coli_attn_qcache_bind(None, None, None) == -1


@pytest.mark.parametrize("args,expect", [
    ((None, 4, 128, 64, 0, 16, 16), -1), ((16, 4, 128, 64, 0, None, 16), -1), ((16, 4, 128, 64, 0, 16, None), -1),
    ((16, -1, 128, 64, 0, 16, 16), -1), ((16, 4, 0, 64, 0, 16, 16), -1), ((16, 4, 100, 64, 0, 16, 16), -1),
    ((16, 4, 128, 0, 0, 16, 16), -1), ((18, 4, 128, 64, 0, 16, 16), -1), ((16, 4, 128, 64, 0, 16, 17), -1),
    ((16, 4, 128, 16, 0, 16, 16), -6), ((16, 4, 128, 64, 2, 16, 16), -6), ((16, 0, 128, 64, 0, 16, 16), 0)])
def test_quantize_rejects(args, expect):
    assert linear.lib().coli_linear_quantize(*args, None) == expect


def test_constants_match_the_header():
    text = open(os.path.join(_build.INCLUDE, "coli_attn.h")).read()
    defs = {m.group(1): int(m.group(2)) for m in re.finditer(r"#define\s+(COLI_ATTN_\w+)\s+(\d+)", text)}
    assert attn.CODES == {torch.int8: defs["COLI_ATTN_CODE_INT8"], torch.float8_e4m3fn: defs["COLI_ATTN_CODE_E4M3"]}
