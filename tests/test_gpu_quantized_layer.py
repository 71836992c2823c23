"""4-bit projections, append and window over an 8-bit cache together, as a decoder layer uses them: prompts, then single tokens
from a captured graph, each operator against its definition in 64 bits on what the one before it gave."""
import os
import runpy

import pytest
import torch

from int4_routed_expert_quantize_gb300 import attn, linear

from .test_gpu_attn_q8 import BF, E4, HF, I8, Setup, close, i32, positions, rotated, stored
from .test_gpu_linear import check, expanded

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "quantized_decode.py")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)


@pytest.mark.parametrize("n_q,n_kv,D,dt,kind,group", [(8, 2, 64, BF, I8, 64), (6, 1, 128, HF, E4, 128)])
def test_layer_prompt_then_steps(n_q, n_kv, D, dt, kind, group):
    d, page, news, steps = 384, 16, [21, 1, 70], 9
    torch.manual_seed(3)
    s = Setup(news, news, n_q, n_kv, D, page, dt, kind)
    width = -(-(max(news) + steps) // page)
    s.table = torch.randperm(3 * width, device="cuda").int().view(3, width)
    s.kc, s.vc = (torch.full((3 * width, n_kv, page, D), 255, dtype=torch.uint8, device="cuda").view(kind) for _ in range(2))
    s.ks, s.vs = (torch.full((3 * width, n_kv, page), float("nan"), device="cuda") for _ in range(2))
    s.cache = s.eng.bind_cache(s.kc, s.vc, s.ks, s.vs)
    parts = []
    for rows, cols in (((n_q + 2 * n_kv) * D, d), (d, n_q * D)):
        packed, scales = linear.quantize(torch.randn((rows, cols), device="cuda") * cols ** -0.5, group, dt)
        parts.append((linear.Int4Linear(packed, scales, max_tokens=s.T), expanded(packed, scales)))
    (qkv_l, qkv_w), (out_l, out_w) = parts

    def forward(x):
        qkv = qkv_l.forward(x)
        raw = qkv.clone()
        q, k, v = qkv.view(x.shape[0], -1, D).split([n_q, n_kv, n_kv], 1)
        s.q = s.eng.append(s.cache, s.batch, k, v, q, q_out=q)
        o = s.eng.window(s.cache, s.batch, s.q, window=40, sinks=3)
        return raw, qkv, o, out_l.forward(o.view(x.shape[0], -1))

    def verify(x, raw, qkv, o, y):
        check(raw, x, qkv_w, group, dt)
        was, now = (t.view(x.shape[0], -1, D) for t in (raw, qkv))
        k, v = was[:, n_q:n_q + n_kv], was[:, n_q + n_kv:]
        pos = positions(s)[1]
        ref = rotated(was[:, :n_q].double(), pos, D, False, 10000.0)
        u = torch.finfo(dt).eps / 2
        assert ((now[:, :n_q].double() - ref).abs() <= u * ref.abs() + 2.0 ** -19 * ref.abs().amax(-1, keepdim=True)).all()
        assert torch.equal(now[:, n_q:], was[:, n_q:])
        (kc, ks), (vc, vs) = stored(s)
        close(kc, ks, rotated(k.double(), pos, D, False, 10000.0), kind)
        close(vc, vs, v.double(), kind)
        s.q = now[:, :n_q]
        s.check(o, None, s.reference(window=40, sinks=3))
        check(y, o.view(x.shape[0], -1), out_w, group, dt)

    s.batch = attn.Batch(i32(s.start), i32(s.lens), s.table, n_tokens=s.T, max_q=max(news))
    x = torch.randn((s.T, d), device="cuda").to(dt)
    verify(x, *forward(x))
    lens, before = i32(s.lens), s.lens
    s.news, s.T, s.start = [1] * 3, 3, list(range(4))
    s.batch = attn.Batch(i32(s.start), lens, s.table, n_tokens=3, max_q=1)
    x, g = torch.empty((3, d), dtype=dt, device="cuda"), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lens += 1
        got = forward(x)
    for step in range(steps):
        x.copy_(torch.randn((3, d), device="cuda"))
        s.lens = [m + step + 1 for m in before]
        g.replay()
        verify(x, *got)
    assert s.eng.status() == qkv_l.status() == out_l.status() == 0


@pytest.mark.parametrize("cache", ["int8", "e4m3"])
def test_example_runs(cache):
    """the example's captured steps are the eager calls' bits"""
    ex = runpy.run_path(PATH)
    users, prompt, steps = 3, 37, 4
    layer, first, outs = ex["run"](users, prompt, steps, cache, seed=4)
    assert first.shape == (users * prompt, layer.d) and len(outs) == steps
    lens = i32([prompt] * users)
    tables = torch.arange(layer.k.shape[0], dtype=torch.int32, device="cuda").view(users, -1)
    batch, x = attn.Batch(i32(list(range(users + 1))), lens, tables, n_tokens=users, max_q=1), first[prompt - 1::prompt].clone()
    for out in outs:  # the same slots are written again, with the same values
        lens += 1
        x = layer.forward(x, batch)
        assert torch.isfinite(x).all() and torch.equal(x, out)
