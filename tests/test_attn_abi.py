"""The C entry points of the paged-cache attention (coli_attn.h) refuse what they do not take before they touch a GPU.
CPU only."""
import ctypes
import math
import shutil

import pytest

from int4_routed_expert_quantize_gb300 import _build, attn, coli


@pytest.fixture(scope="module", autouse=True)
def built():
    if shutil.which("nvcc") is None:
        pytest.skip("nvcc not available")
    if _build.is_stale():
        _build.build()
        coli._lib = None
    return attn.lib()


def create(freq=None, **kw):
    base = dict(n_q=8, n_kv=2, head_dim=64, page=16, dtype=0, max_tokens=16, max_seqs=4, rot_dim=64, rot_interleaved=0,
                rope_base=10000.0)
    base.update(kw)
    cfg = attn.AttnConfig(*[base[f] for f, _ in attn.AttnConfig._fields_[:-1]], freq)
    h = ctypes.c_void_p(1)
    rc = attn.lib().coli_attn_create(ctypes.byref(cfg), ctypes.byref(h))
    if rc == 0:
        attn.lib().coli_attn_destroy(h)
        return 0, None
    return rc, h.value


@pytest.mark.parametrize("kw,expect", [
    (dict(n_kv=0), -1), (dict(n_q=7), -1), (dict(n_q=0), -1), (dict(n_kv=257, n_q=257), -1), (dict(max_tokens=0), -1),
    (dict(max_tokens=2 ** 22 + 1), -1), (dict(max_seqs=0), -1), (dict(max_seqs=4097), -1), (dict(rot_dim=-16), -1),
    (dict(rot_interleaved=2), -1), (dict(rope_base=0.0), -1), (dict(rope_base=math.inf), -1), (dict(rope_base=math.nan), -1),
    (dict(page=0), -1), (dict(head_dim=0), -1),
    (dict(head_dim=96), -6), (dict(head_dim=256), -6), (dict(page=8), -6), (dict(page=24), -6), (dict(page=512), -6),
    (dict(page=2 ** 31 - 1), -6), (dict(dtype=2), -6), (dict(n_q=130, n_kv=2), -6), (dict(rot_dim=24), -6),
    (dict(rot_dim=128), -6)])
def test_create_rejects(kw, expect):
    assert create(**kw) == (expect, None)


def test_create_rejects_frequencies_that_are_not_finite():
    freq = (ctypes.c_double * 32)(*([1.0] * 31 + [math.inf]))
    assert create(freq=freq) == (-1, None)


def test_null_arguments():
    L = attn.lib()
    h, batch = ctypes.c_void_p(), attn.AttnBatch()
    assert L.coli_attn_create(None, None) == -1 and L.coli_attn_create(None, ctypes.byref(h)) == -1
    assert L.coli_attn_cache_bind(None, None, None) == -1
    assert L.coli_attn_append(None, None, ctypes.addressof(batch), None, 0, None, 0, None, 0, None, 0, None, None) == -1
    assert L.coli_attn_window(None, None, None, None, 0, 0, 0, 1.0, None, 0, None, None) == -1
    assert L.coli_attn_prefix(None, None, None, None, 0, None, None, 0, 1.0, None, 0, None, None) == -1
    assert L.coli_attn_status(None, None) == -1 and L.coli_attn_launches(None, 0, 1) == -1
    L.coli_attn_destroy(None)
    L.coli_attn_cache_release(None)


def test_create_without_gpu_reports_cuda_error():
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert create() == (-4, None)


def test_constants_match_the_header():
    import os
    import re
    text = open(os.path.join(_build.INCLUDE, "coli_attn.h")).read()
    defs = {m.group(1): int(m.group(2)) for m in re.finditer(r"#define\s+(COLI_ATTN_\w+)\s+(\d+)", text)}
    import torch
    assert attn.DTYPES == {torch.bfloat16: defs["COLI_ATTN_BF16"], torch.float16: defs["COLI_ATTN_FP16"]}
