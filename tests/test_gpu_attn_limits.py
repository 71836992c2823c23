"""The edges of what the attention calls accept (coli_attn.h): outputs on 16-byte boundaries, page
tables of several strides, tensors of another device, cache
strides, offsets that are not what the header asks for, the smallest and largest scales, new outputs on another stream."""
import ctypes
import math

import pytest
import torch

from int4_routed_expert_quantize_gb300 import attn, coli

from .test_gpu_attn import BF, HF, Setup

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)


def padded(s, before, after):
    """an output view `before` values into its buffer, with rows of `after` more values than it needs"""
    wide = torch.full((before + s.T * (s.n_q * s.D + after),), 7.0, dtype=s.dt, device="cuda")
    return wide, wide[before:].view(s.T, -1)[:, :s.n_q * s.D].view(s.T, s.n_q, s.D)


@pytest.mark.parametrize("before,after", [(8, 0), (0, 8), (8, 8), (24, 40), (16, 16)])
@pytest.mark.parametrize("D,dt,news,lens", [
    (128, BF, [40, 300], [40, 900]), (64, HF, [100, 7], [333, 7]), (64, BF, [1, 4], [70, 90]), (128, HF, [1], [2000])])
def test_outputs_on_16_byte_boundaries(before, after, D, dt, news, lens):
    """bases and strides of 8 values: whole units, cut ones, and the prefix call's; nothing between the rows is written"""
    s = Setup(news, lens, 6, 2, D, 16, dt)
    want = s.window(window=200, sinks=3)
    wide, out = padded(s, before, after)
    assert s.eng.window(s.cache, s.batch, s.q, window=200, sinks=3, out=out) is out
    assert torch.equal(out, want)
    assert not (wide[:before] != 7).any() and not (wide[before:].view(s.T, -1)[:, s.n_q * s.D:] != 7).any()
    p = Setup([1, 2, 1], [9, 70, 3], 6, 2, D, 16, dt, prefix=333)
    want = p.shared()
    wide, out = padded(p, before, after)
    p.eng.prefix(p.cache, p.batch, p.prefix_table, p.prefix_len, p.q, out=out)
    assert torch.equal(out, want)
    assert not (wide[:before] != 7).any() and not (wide[before:].view(p.T, -1)[:, p.n_q * p.D:] != 7).any()
    assert s.eng.status() == 0 and p.eng.status() == 0


@pytest.mark.parametrize("news", [[1, 1, 1], [40, 1, 60]])
def test_expanded_page_table(news):
    """several sequences with one row of pages: what a copy of the row for each gives"""
    s = Setup(news, [300] * 3, 6, 2, 64, 16, BF, prefix=50)
    row = s.table[1:2].expand(3, -1)
    assert row.stride(0) == 0
    b = s.batch
    one, each = (attn.Batch(b.q_start, b.kv_len, t, n_tokens=s.T, max_q=b.max_q) for t in (row, row.contiguous()))
    want = s.eng.window(s.cache, each, s.q, window=100, sinks=5)
    assert torch.equal(s.eng.window(s.cache, one, s.q, window=100, sinks=5), want)
    if s.T <= 8 * len(news):
        want = s.eng.prefix(s.cache, each, s.prefix_table, s.prefix_len, s.q)
        assert torch.equal(s.eng.prefix(s.cache, one, s.prefix_table, s.prefix_len, s.q), want)
    assert s.eng.status() == 0
    with pytest.raises(ValueError):  # rows that overlap
        attn.Batch(b.q_start, b.kv_len, torch.as_strided(s.table, (3, 10), (4, 1)), n_tokens=s.T, max_q=b.max_q)


def test_tensors_of_another_device_are_refused():
    """by their device's number, so that one GPU is enough to see it"""
    s = Setup([1, 1], [40, 40], 4, 2, 64, 16, BF, junk=0.0, prefix=20)
    k = torch.zeros((2, 2, 64), dtype=BF, device="cuda")
    s.batch.c.device = s.eng.device + 1
    for call in (lambda: s.eng.window(s.cache, s.batch, s.q), lambda: s.eng.append(s.cache, s.batch, k, k),
                 lambda: s.eng.prefix(s.cache, s.batch, s.prefix_table, s.prefix_len, s.q)):
        with pytest.raises(ValueError):
            call()
    s.batch.c.device = s.eng.device
    s.shared()
    b = s.batch
    with pytest.raises(ValueError):  # not all on one device
        attn.Batch(b.q_start.cpu(), b.kv_len, s.table, n_tokens=2, max_q=1)
    s.eng.device += 1
    with pytest.raises(ValueError):
        s.eng.bind_cache(s.kc, s.vc)


def bind(strides, n_pages=3, n_kv=2, page=16, D=64):
    """the status of binding a cache whose K has these strides, and of one whose V has"""
    eng = attn.PagedAttention(2 * n_kv, n_kv, D, page, 4, 4)
    mem, good, out = torch.zeros(1 << 16, dtype=BF, device="cuda"), (n_kv * page * D, page * D, D), []
    for k, v in ((strides, good), (good, strides)):
        c, h = attn.AttnCache(mem.data_ptr(), mem.data_ptr() + mem.numel(), n_pages, *k, *v), ctypes.c_void_p()
        out.append(attn.lib().coli_attn_cache_bind(eng.h, ctypes.byref(c), ctypes.byref(h)))
        attn.lib().coli_attn_cache_release(h)
    return out


@pytest.mark.parametrize("strides", [(64, 64, 64), (2048, 64, 64), (64, 1024, 64), (2048, 1016, 64), (2040, 1024, 64),
                                     (2048, 64, 120), (1024, 2048, 64), (2 ** 37, 2 ** 37, 64)])
def test_cache_strides_that_let_tokens_overlap_are_refused(strides):
    assert bind(strides) == [-1, -1]


@pytest.mark.parametrize("strides,kw", [
    ((2048, 1024, 64), {}), ((2048, 64, 128), {}), ((64, 3072, 192), {}), ((2048, 64, 64), dict(n_kv=1)),
    ((64, 1024, 64), dict(n_pages=1)), ((2040, 1016, 64), dict(n_pages=1, n_kv=1)), ((3000, 1400, 72), {})])
def test_cache_strides_in_any_order(strides, kw):
    """pages, heads and slots nested in any order, padded, or of one entry"""
    assert bind(strides, **kw) == [0, 0]


@pytest.mark.parametrize("seqs", [3, 45])
@pytest.mark.parametrize("prefix", [0, 20])
def test_offsets_that_end_early_are_reported(seqs, prefix):
    """the last tokens belong to no sequence; the sequences' rows are within their bound all the same (a shorter list is cut
    elsewhere, so not the same bits)"""
    news = ([2, 3, 1] * seqs)[:seqs]
    s = Setup(news, [40 + i for i in range(seqs)], 4, 2, 64, 16, BF, prefix=prefix)
    call = s.shared if prefix else s.window
    want, n = call(), s.T - news[-1]
    s.batch.q_start[-1] -= news[-1]
    got = s.eng.prefix(s.cache, s.batch, s.prefix_table, s.prefix_len, s.q) if prefix else s.eng.window(s.cache, s.batch, s.q)
    assert s.eng.status() == -1 and s.eng.status() == 0
    assert (s.off(got[:n], [x[:n] for x in s.reference()]) <= 1).all()
    s.batch.q_start[-1] += news[-1]
    assert torch.equal(call(), want)


@pytest.mark.parametrize("news,lens", [([1], [300]), ([60], [900]), ([300, 1], [700, 50])])
@pytest.mark.parametrize("scale", [1e-38, 3e-39, 1e-44])
def test_scales_near_zero(news, lens, scale):
    """all weights alike, whichever kernel takes the batch; whole units and cut ones"""
    Setup(news, lens, 8, 2, 64, 16, BF).window(scale=scale)
    Setup([1, 4, 2], [30, 90, 7], 8, 2, 64, 16, BF, prefix=700).shared(scale=scale)


def test_scales_past_the_range_are_refused():
    """finite, but not times log2(e), which is what the kernels multiply by"""
    s = Setup([1], [30], 8, 2, 64, 16, BF, prefix=20)
    for call in (lambda: s.eng.window(s.cache, s.batch, s.q, scale=3e38),
                 lambda: s.eng.prefix(s.cache, s.batch, s.prefix_table, s.prefix_len, s.q, scale=3e38)):
        with pytest.raises(coli.ColiError) as e:
            call()
        assert e.value.status == -1


def test_append_with_offsets_that_do_not_ascend():
    """reported, and nothing is stored behind a sequence's cached tokens"""
    s = Setup([1, 1, 1], [40, 40, 40], 4, 2, 64, 16, BF, junk=0.0)
    eng = attn.PagedAttention(4, 2, 64, 16, 16, 4, rot_dim=0)
    kc, vc = s.kc.clone(), s.vc.clone()
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    b = attn.Batch(i32(0, 10, 2, 3), i32(20, 20, 20), s.table, n_tokens=10, max_q=10)
    k = torch.ones((10, 2, 64), dtype=BF, device="cuda")
    eng.append(eng.bind_cache(kc, vc), b, k, k)
    assert eng.status() == -1
    pages = s.table.long()
    for got, old in ((kc, s.kc), (vc, s.vc)):
        got, old = (x[pages].transpose(2, 3).reshape(3, -1, 2, 64)[:, 20:] for x in (got, old))
        assert torch.equal(got, old)


@pytest.mark.parametrize("n_q", [4, 64])
def test_spoilt_rows_with_offsets_that_do_not_ascend(n_q):
    """rows to compute again whose sequence, looked up by the offsets, is another one: reported, read nowhere, forgotten"""
    s = Setup([10, 1, 1], [48, 48, 48], n_q, 2, 64, 16, BF, junk=0.0)  # full page tables
    want = s.window(window=-1)
    b, pg = s.batch, int(s.table[0, 2])
    keep = s.vc[pg, :, 12].clone()
    s.vc[pg, :, 12] = math.nan  # token 44 of 48: the queries 0..5 do not see it
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    # tokens 3.. fall to sequence 2 (its one token is number 2) by the ends at or before them
    s.eng.window(s.cache, attn.Batch(i32(0, 12, 2, 3), b.kv_len, s.table, n_tokens=12, max_q=12), s.q)
    assert s.eng.status() == -1
    s.vc[pg, :, 12] = keep
    assert torch.equal(s.eng.window(s.cache, b, s.q), want) and s.eng.status() == 0


@pytest.mark.parametrize("seqs,T,pages", [(4096, 65536, 128), (4096, 65536, 256), (32, 65536, 8192), (4096, 32768, 128)])
def test_offsets_that_overlap_until_the_list_is_full(seqs, T, pages):
    """every other sequence claims all tokens: more key tiles than the list has places.  Reported, and the next call is right"""
    n_q, n_kv, D, page = 64, 8, 64, 256
    eng = attn.PagedAttention(n_q, n_kv, D, page, T, seqs)
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    kc, vc = (torch.randn((2, n_kv, page, D), generator=g, device="cuda").to(BF) for _ in range(2))
    cache, q = eng.bind_cache(kc, vc), torch.randn((T, n_q, D), generator=g, device="cuda").to(BF)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    small = attn.Batch(i32(0, 1, 3), i32(300, 5), i32(0, 1, 1, 0).view(2, 2), n_tokens=3, max_q=2)
    lse, out = torch.zeros((T, n_q), device="cuda"), torch.zeros_like(q)
    bad = attn.Batch(i32(*[0 if b % 2 == 0 else T for b in range(seqs)], T),
                     torch.full((seqs,), pages * page, dtype=torch.int32, device="cuda"),
                     torch.zeros((1, pages), dtype=torch.int32, device="cuda").expand(seqs, -1), n_tokens=T, max_q=T)
    calls = [lambda b, n: eng.window(cache, b, q[:n], out=out[:n], lse=lse[:n])]
    if T <= 8 * seqs:
        calls.append(lambda b, n: eng.prefix(cache, b, i32(1), i32(200), q[:n], out=out[:n], lse=lse[:n]))
    for call in calls:
        want = call(small, 3).clone()
        assert eng.status() == 0
        call(bad, T)
        assert eng.status() == -1
        assert torch.equal(call(small, 3), want) and eng.status() == 0


@pytest.mark.parametrize("op", ["append", "window", "prefix"])
@pytest.mark.parametrize("handle", [False, True])
def test_new_outputs_on_another_stream(op, handle):
    """their memory is not what the current stream still has work queued on, nor is it given to their stream again while
    the current one reads it"""
    s = Setup([3, 5], [70, 300], 6, 2, 128, 64, BF, prefix=30)
    k = torch.randn((s.T, 2, 128), device="cuda").to(BF)
    call = {"append": lambda **kw: s.eng.append(s.cache, s.batch, k, k, s.q, **kw),
            "window": lambda **kw: s.eng.window(s.cache, s.batch, s.q, **kw),
            "prefix": lambda **kw: s.eng.prefix(s.cache, s.batch, s.prefix_table, s.prefix_len, s.q, **kw)}[op]
    want, side = call(), torch.cuda.Stream()
    torch.cuda.synchronize()
    old = torch.empty_like(want)
    at = old.data_ptr()
    torch.cuda._sleep(200_000_000)
    old.fill_(5)
    del old  # its memory is free for the current stream's next tensor, and the fill is yet to come
    got = call(stream=side.cuda_stream if handle else side)
    assert got.data_ptr() != at
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    torch.cuda._sleep(200_000_000)
    copy = got.clone()
    del got
    with torch.cuda.stream(side):
        other = torch.empty_like(want).fill_(9)
    torch.cuda.synchronize()
    assert torch.equal(copy, want) and (other == 9).all()


@pytest.mark.parametrize("n_q,n_kv,D,dt", [(48, 8, 128, BF), (32, 8, 64, HF)])
def test_prefix_of_one_long_sequence_among_many(n_q, n_kv, D, dt):
    """own keys and prefix in launches of their own, a sequence of many blocks of the first; with and without values that
    only some of its rows see"""
    news = [1] * 20 + [230] + [2] * 30
    s = Setup(news, [60 + n for n in news], n_q, n_kv, D, 32, dt, prefix=150)
    assert s.eng.launches("prefix", len(news)) == 3 and s.T <= 8 * len(news)
    want = s.shared()
    j, ref = 200, s.reference()  # of 290 tokens; the queries are 60..289
    pg = int(s.table[20, j // 32])
    keep = s.vc[pg, :, j % 32].clone()
    s.vc[pg, :, j % 32] = math.nan
    out = s.eng.prefix(s.cache, s.batch, s.prefix_table, s.prefix_len, s.q)
    hit = torch.zeros(s.T, dtype=torch.bool, device="cuda")
    hit[20 + j - 60:250] = True
    assert (s.off(out, ref)[~hit] <= 1).all() and torch.isnan(out[hit]).all()
    s.vc[pg, :, j % 32] = keep
    assert torch.equal(s.eng.prefix(s.cache, s.batch, s.prefix_table, s.prefix_len, s.q), want)
