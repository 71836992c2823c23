"""Append and window over an 8-bit cache (coli_attn_qcache_bind) against their definitions in 64 bits.

Bounds, derived from the formats.  Codes multiply exactly.  A weight, in units of the largest |scale| of a value that
the row has seen, is rounded to fp16: 2^-11 of it, at least 2^-25 (the row's largest weight is 1 or more there), which a
code of at most `top` multiplies; the output is rounded once, u of it; scores and exponentials are fp32, under 2e-4 of a weight
for the inputs here (as over a 16-bit cache).  So |o - o*| <= (2^-11 + 2e-4) sum_j p_j |v_j| + u |o*| + n 2^-25 top max|vs|.
A stored value: top x / m is off by fp32 roundings of the rotation and of m, 16 * 2^-24 of top each, and by half a step."""
import math

import pytest
import torch

from int4_routed_expert_quantize_gb300 import attn, coli

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
U = {BF: 2.0 ** -8, HF: 2.0 ** -11}
I8, E4 = torch.int8, torch.float8_e4m3fn
TOP = {I8: 127.0, E4: 448.0}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def quantised(x, kind):
    """[..., D] in 64 bits -> codes, scales by the definition"""
    m = x.abs().amax(-1, keepdim=True)
    y = TOP[kind] * x / torch.where(m == 0, 1.0, m)
    return (torch.round(y) if kind is I8 else y.float()).to(kind), (m / TOP[kind]).float().squeeze(-1)


class Setup:
    """a ragged batch over an 8-bit cache of randomly ordered pages; unused slots hold codes of all ones and NaN scales"""

    def __init__(self, news, lens, n_q, n_kv, D, page, dt, kind, layout="head", seed=0, junk=math.nan, **kw):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.news, self.lens, self.n_q, self.n_kv, self.D, self.page, self.dt, self.kind = news, lens, n_q, n_kv, D, page, dt, kind
        need = [-(-m // page) for m in lens]
        n = sum(need) + 2
        order = torch.randperm(n, generator=g, device="cuda")
        codes = lambda *s: torch.full(s, 255, dtype=torch.uint8, device="cuda").view(kind)  # noqa: E731
        scale = lambda *s: torch.full(s, junk, device="cuda")  # noqa: E731
        if layout == "head":
            self.kc, self.vc = codes(n, n_kv, page, D), codes(n, n_kv, page, D)
            self.ks, self.vs = scale(n, n_kv, page), scale(n, n_kv, page)
        elif layout == "slot":  # codes by [page, slot, head], scales by [head, page, slot]
            self.kc, self.vc = codes(n, page, n_kv, D).transpose(1, 2), codes(n, page, n_kv, D).transpose(1, 2)
            self.ks, self.vs = scale(n_kv, n, page).transpose(0, 1), scale(n_kv, n, page).transpose(0, 1)
        else:  # K and V of a page next to each other, wider rows
            both, sc = codes(n, 2, n_kv, page, D + 16), scale(n, 2, n_kv, page + 4)
            self.kc, self.vc = both[:, 0, ..., :D], both[:, 1, ..., :D]
            self.ks, self.vs = sc[:, 0, ..., :page], sc[:, 1, ..., :page]
        width = max(need + [1])
        self.table = torch.full((len(news), width + 1), -1, dtype=torch.int32, device="cuda")[:, :width]
        at = 0
        for b, (m, c) in enumerate(zip(lens, need)):
            self.table[b, :c] = order[at:at + c].int()
            pos = torch.arange(m, device="cuda")
            pg, sl = order[at:at + c][pos // page], pos % page
            for cache, scales in ((self.kc, self.ks), (self.vc, self.vs)):
                x = torch.randn((m, n_kv, D), generator=g, device="cuda")
                x = x * torch.exp(0.5 * torch.randn((m, n_kv, 1), generator=g, device="cuda"))
                q, d = quantised(x.double(), kind)
                cache.view(torch.uint8)[pg, :, sl] = q.view(torch.uint8)
                scales[pg, :, sl] = d
            at += c
        self.T = sum(news)
        self.q = torch.randn((self.T, n_q, D), generator=g, device="cuda").to(dt)
        self.start = [sum(news[:i]) for i in range(len(news) + 1)]
        self.eng = attn.PagedAttention(n_q, n_kv, D, page, max_tokens=max(self.T, 1), max_seqs=len(news), dtype=dt, **kw)
        self.cache = self.eng.bind_cache(self.kc, self.vc, self.ks, self.vs)
        self.batch = attn.Batch(i32(self.start), i32(lens), self.table, n_tokens=self.T, max_q=max(news + [1]))

    def held(self, b, m):
        """sequence b's first m keys and values [n_kv, m, D] and the values' scales [n_kv, m], in 64 bits"""
        pos = torch.arange(m, device="cuda")
        pg, sl = self.table[b].long()[pos // self.page], pos % self.page
        out = []
        for cache, scales in ((self.kc, self.ks), (self.vc, self.vs)):
            c = cache.view(torch.uint8)[pg, :, sl].view(self.kind).float().double()
            out.append((c * scales[pg, :, sl].double()[..., None]).transpose(0, 1))
        return out[0], out[1], self.vs[pg, :, sl].double().transpose(0, 1)

    def reference(self, window=-1, sinks=0, scale=None):
        """-> (o, bound, lse) in 64 bits; rows without keys: 0, 0, -inf"""
        G, scale = self.n_q // self.n_kv, scale or 1 / math.sqrt(self.D)
        o = torch.zeros((self.T, self.n_q, self.D), dtype=torch.float64, device="cuda")
        bound, lse = torch.zeros_like(o), torch.full(o.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
        for b, (n, m) in enumerate(zip(self.news, self.lens)):
            k, v, vs = self.held(b, m)
            for i in range(n):
                p = m - n + i
                j = torch.arange(m, device="cuda")
                see = j <= p
                if window >= 0:
                    see &= (p - j < window) | (j < sinks)
                if not see.any():
                    continue
                t = self.start[b] + i
                s = self.q[t].double().view(self.n_kv, G, self.D) @ k[:, see].transpose(1, 2) * scale
                w = torch.softmax(s, -1)
                o[t] = (w @ v[:, see]).reshape(self.n_q, self.D)
                a = (w @ v[:, see].abs()).reshape(self.n_q, self.D)
                low = see.sum() * 2.0 ** -25 * TOP[self.kind] * vs[:, see].abs().amax(1)
                bound[t] = (2.0 ** -11 + 2e-4) * a + U[self.dt] * o[t].abs() + low.repeat_interleave(G)[:, None]
                lse[t] = torch.logsumexp(s, -1).reshape(self.n_q)
        return o, bound, lse

    def check(self, out, lse, ref, rows=slice(None)):
        o, bound, l = (x[rows] for x in ref)
        out = out[rows]
        assert torch.isfinite(out).all()
        worst = ((out.double() - o).abs() / (bound + 1e-30)).max() if out.numel() else 0.0
        assert worst <= 1, float(worst)
        if lse is not None:
            lse = lse[rows]
            assert torch.equal(torch.isinf(lse), torch.isinf(l))
            f = torch.isfinite(l)
            assert ((lse.double() - l)[f].abs() <= 2e-4).all()

    def window(self, **kw):
        lse = torch.full((self.T, self.n_q), 7.0, device="cuda")
        out = torch.full((self.T, self.n_q, self.D), 7.0, dtype=self.dt, device="cuda")
        self.eng.window(self.cache, self.batch, self.q, out=out, lse=lse, **kw)
        self.check(out, lse, self.reference(**kw))
        assert self.eng.status() == 0
        return out


# ---- window ----

@pytest.mark.parametrize("kind", [I8, E4])
@pytest.mark.parametrize("news,lens", [
    ([1], [1]), ([1], [65]), ([1], [2049]), ([1, 1, 1], [1, 700, 63]), ([5, 5, 5], [5, 333, 1000]),
    ([300], [300]), ([257], [1000]), ([1, 129, 1, 40], [900, 400, 1, 40]), ([0, 3, 0], [7, 9, 0]),
    ([1] * 70, list(range(1, 71)))])
@pytest.mark.parametrize("window,sinks", [(-1, 0), (100, 4), (0, 3), (128, 130)])
def test_window_lengths(news, lens, window, sinks, kind):
    Setup(news, lens, 6, 2, 128, 16, BF, kind).window(window=window, sinks=sinks)


@pytest.mark.parametrize("n_q,n_kv,D,page,dt,kind,layout", [
    (1, 1, 64, 16, HF, I8, "head"), (8, 1, 128, 32, BF, E4, "slot"), (16, 1, 64, 64, BF, I8, "both"),
    (17, 1, 128, 128, HF, E4, "head"), (64, 1, 64, 256, HF, I8, "slot"), (33, 1, 128, 16, BF, E4, "both"),
    (15, 5, 64, 16, BF, E4, "head"), (4, 4, 128, 256, HF, I8, "both")])
@pytest.mark.parametrize("news,lens", [([1, 1], [500, 33]), ([7, 2], [300, 2]), ([150, 70], [400, 70])])
def test_window_heads_pages_layouts(n_q, n_kv, D, page, dt, kind, layout, news, lens):
    s = Setup(news, lens, n_q, n_kv, D, page, dt, kind, layout)
    s.window(window=-1)
    s.window(window=77, sinks=20)


@pytest.mark.parametrize("kind", [I8, E4])
@pytest.mark.parametrize("news,lens,window,sinks", [
    ([3], [0], -1, 0), ([5, 2], [2, 9], -1, 0), ([2, 1], [50, 60], 0, 0), ([200], [90], 16, 0)])
def test_window_rows_that_see_nothing(news, lens, window, sinks, kind):
    """an empty cache, more queries than cached tokens, a window of 0: zeros and -inf"""
    Setup(news, lens, 8, 2, 64, 16, BF, kind).window(window=window, sinks=sinks)


@pytest.mark.parametrize("kind", [I8, E4])
@pytest.mark.parametrize("news", [1, 6, 300])
def test_window_ignores_what_a_row_does_not_see(news, kind):
    """scales of NaN, infinity and 2^100 at later tokens and at those that left the window"""
    s = Setup([news], [400], 8, 2, 128, 32, BF, kind)
    W, p = 64, torch.arange(400 - news, 400, device="cuda")
    ref = s.reference(window=W, sinks=3)
    for j in (399, 400 - news - W, 5):
        pg, sl = int(s.table[0, j // 32]), j % 32
        keep = s.ks[pg, :, sl].clone(), s.vs[pg, :, sl].clone()
        blind = ~((j <= p) & ((p - j < W) | (j < 3)))
        for bad in (math.nan, math.inf, 2.0 ** 100):
            s.ks[pg, :, sl], s.vs[pg, :, sl] = bad, bad
            out = s.eng.window(s.cache, s.batch, s.q, window=W, sinks=3)
            s.check(out, None, ref, blind)
            if bad != 2.0 ** 100:
                assert not torch.isfinite(out[~blind]).any()
        s.ks[pg, :, sl], s.vs[pg, :, sl] = keep


@pytest.mark.parametrize("kind", [I8, E4])
@pytest.mark.parametrize("news", [1, 40])
def test_window_scales_of_every_size(news, kind):
    """values whose scales differ by 2^20, heads of zeros, keys and queries far from 1"""
    s = Setup([news], [300], 8, 2, 64, 16, BF, kind, seed=4)
    s.vs *= torch.exp2(torch.randint(-20, 1, s.vs.shape, device="cuda").float())
    s.vs[:, :, 3] = 0
    s.ks[:, :, 7] = 0
    s.window()
    s.ks *= 2.0 ** 70
    s.q = (s.q.float() * 2.0 ** -70).to(BF)
    s.window()
    s.ks *= 2.0 ** -135
    s.vs *= 2.0 ** -60
    s.q = (s.q.double() * 2.0 ** 130).to(BF)
    s.window(scale=0.3)


@pytest.mark.parametrize("news", [[1, 1, 1], [3, 1, 20]])
def test_window_strides_streams_and_graphs(news):
    s = Setup(news, [70, 300, 20], 6, 2, 128, 64, BF, I8, "slot")
    want = s.window(window=90, sinks=2)
    wide = torch.zeros((s.T, 10, 128), dtype=BF, device="cuda")
    wide[:, 2:8] = s.q
    out = torch.zeros((s.T, 9, 128), dtype=BF, device="cuda")
    s.eng.window(s.cache, s.batch, wide[:, 2:8], window=90, sinks=2, out=out[:, 1:7])
    assert torch.equal(out[:, 1:7], want) and not out[:, 0].any() and not out[:, 7:].any()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = s.eng.window(s.cache, s.batch, s.q, window=90, sinks=2, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    g, buf = torch.cuda.CUDAGraph(), torch.empty_like(want)
    with torch.cuda.graph(g):
        s.eng.window(s.cache, s.batch, s.q, window=90, sinks=2, out=buf)
    for lens in ([70, 300, 20], [40, 64, 20]):  # lengths change on the device between replays
        s.batch.kv_len.copy_(i32(lens))
        s.lens = lens
        g.replay()
        s.check(buf, None, s.reference(window=90, sinks=2))
    assert s.eng.status() == 0


@pytest.mark.parametrize("many", [False, True])
def test_window_many_sequences(many):
    """more than 32 sequences, empty ones between; long ones among them"""
    r = torch.Generator().manual_seed(5)
    lens = torch.randint(1, 400, (90,), generator=r).tolist()
    news = [0 if i % 7 == 3 else 1 for i in range(90)]
    if many:
        news = [min(m, 120) if i % 10 == 4 else n for i, (n, m) in enumerate(zip(news, lens))]
    Setup(news, lens, 8, 2, 64, 16, HF, E4).window(window=150, sinks=5)


@pytest.mark.parametrize("news", [[1] * 9, [60, 1, 2, 33, 5, 6, 7, 8, 9]])
def test_window_repeats_bit_for_bit(news):
    s = Setup(news, [4000, 1, 2, 900, 901, 77, 65, 64, 63], 48, 8, 128, 64, BF, I8)
    want = s.eng.window(s.cache, s.batch, s.q, window=2000, sinks=4)
    for _ in range(3):
        assert torch.equal(s.eng.window(s.cache, s.batch, s.q, window=2000, sinks=4), want)


@pytest.mark.parametrize("news", [[1, 1], [1, 70]])
def test_pages_out_of_range_read_as_zeros(news):
    """they are reported; the other sequences' rows are right"""
    s = Setup(news, [100, 200], 8, 2, 64, 32, BF, I8)
    s.window()
    s.table[0, 1] = 10 ** 6
    out = s.eng.window(s.cache, s.batch, s.q)
    assert s.eng.status() == -1 and s.eng.status() == 0
    s.table[0, 1] = 0
    keep = s.kc[0].clone(), s.vc[0].clone(), s.ks[0].clone(), s.vs[0].clone()
    s.kc[0], s.vc[0], s.ks[0], s.vs[0] = 0, 0, 0, 0
    other = set(s.table[1].tolist())
    if 0 not in other:
        s.check(out, None, s.reference())
    s.kc[0], s.vc[0], s.ks[0], s.vs[0] = keep


def test_offsets_past_32_bits():
    """a cache of more than 2^32 codes each: pages at its end"""
    n, page, D = 2 ** 16 + 40, 256, 128
    kc, vc = (torch.zeros((n, 2, page, D), dtype=I8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros((n, 2, page), device="cuda") for _ in range(2))
    s = Setup([1, 90], [300, 400], 6, 2, D, page, BF, I8, junk=0.0, rot_dim=0)
    cache = s.eng.bind_cache(kc, vc, ks, vs)
    far = torch.arange(n - 1, n - 1 - s.kc.shape[0], -1, device="cuda")
    kc[far], vc[far], ks[far], vs[far] = s.kc, s.vc, s.ks, s.vs
    batch = attn.Batch(s.batch.q_start, s.batch.kv_len, far[s.table.long()].int(), n_tokens=91, max_q=90)
    assert torch.equal(s.eng.window(cache, batch, s.q, window=200, sinks=3), s.window(window=200, sinks=3))
    k = torch.randn((91, 2, D), device="cuda").to(BF)
    s.eng.append(cache, batch, k, 2 * k)
    s.eng.append(s.cache, s.batch, k, 2 * k)
    for a, b in ((kc, s.kc), (vc, s.vc), (ks, s.ks), (vs, s.vs)):
        assert torch.equal(a[far], b)
    assert s.eng.status() == 0


# ---- append ----

def rotated(x, pos, rot, inter, base):
    x = x.double()
    if not rot:
        return x
    f = base ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    a = (pos.double()[:, None] * f)[:, None]
    u, v = (x[..., 0:rot:2], x[..., 1:rot:2]) if inter else (x[..., :rot // 2], x[..., rot // 2:rot])
    p, q = u * a.cos() - v * a.sin(), v * a.cos() + u * a.sin()
    y = torch.stack((p, q), -1).flatten(-2) if inter else torch.cat((p, q), -1)
    return torch.cat((y, x[..., rot:]), -1)


def positions(s):
    seq = torch.cat([torch.full((n,), b) for b, n in enumerate(s.news)]).cuda()
    pos = torch.cat([torch.arange(m - n, m) for n, m in zip(s.news, s.lens)]).cuda()
    return seq, pos


def stored(s):
    """codes (as values) and scales of the batch's new tokens: K, V"""
    seq, pos = positions(s)
    pg, sl = s.table.long()[seq, pos.clamp(min=0) // s.page], pos % s.page
    return [(c.view(torch.uint8)[pg, :, sl].view(s.kind).float(), d[pg, :, sl]) for c, d in ((s.kc, s.ks), (s.vc, s.vs))]


def close(codes, scales, x, kind):
    """codes within half a step of the definition, scales to fp32"""
    m = x.abs().amax(-1)
    assert ((scales.double() - m / TOP[kind]).abs() <= 16 * 2.0 ** -24 * scales + 1e-40).all()
    y = TOP[kind] * x / m[..., None].clamp(min=1e-300)
    half = 0.5 if kind is I8 else torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6)))) * 2.0 ** -4
    assert ((codes.double() - y).abs() <= half + TOP[kind] * 2.0 ** -19).all()


@pytest.mark.parametrize("kind", [I8, E4])
@pytest.mark.parametrize("n_q,n_kv,D,page,dt,layout,rot,inter", [
    (8, 2, 128, 16, BF, "head", 128, False), (6, 3, 64, 32, HF, "slot", 64, True), (5, 5, 128, 64, HF, "both", 64, False),
    (28, 4, 64, 256, BF, "slot", 32, True), (7, 1, 128, 128, BF, "head", 0, False), (1, 1, 64, 16, HF, "both", 16, False)])
def test_append(n_q, n_kv, D, page, dt, layout, rot, inter, kind):
    s = Setup([1, 40, 0, 7], [300, 40, 9, 9000], n_q, n_kv, D, page, dt, kind, layout, rot_dim=rot, interleaved=inter)
    wide = torch.randn((s.T, n_q + 2 * n_kv, D), device="cuda").to(dt)
    wide[3] = 0
    q, k, v = wide[:, :n_q], wide[:, n_q:n_q + n_kv], wide[:, n_q + n_kv:]
    seq, pos = positions(s)
    fresh = torch.zeros(s.ks.shape, dtype=torch.bool, device="cuda")
    fresh[s.table.long()[seq, pos // page], :, pos % page] = True
    before = [t.clone() for t in (s.kc, s.vc, s.ks, s.vs)]
    got = s.eng.append(s.cache, s.batch, k, v, q)
    for a, b in zip((s.kc, s.vc, s.ks, s.vs), before):  # the other slots are as they were
        a, b = (x.view(torch.uint8) if x.element_size() == 1 else x.view(torch.int32) for x in (a.contiguous(), b.contiguous()))
        assert torch.equal(a[~fresh], b[~fresh])
    base = s.eng.append(s.eng.bind_cache(*(torch.zeros((s.kc.shape[0], n_kv, page, D), dtype=dt, device="cuda") for _ in "kv")),
                        s.batch, k, v, q)
    assert torch.equal(got, base)
    (kc, kd), (vc, vd) = stored(s)
    close(kc, kd, rotated(k, pos, rot, inter, 10000.0), kind)
    codes, scales = quantised(v.double(), kind)  # nothing is rounded before: equal, the borders between codes too
    assert torch.equal(vc, codes.float()) and torch.equal(vd, scales)
    if not rot:
        codes, scales = quantised(k.double(), kind)
        assert torch.equal(kc, codes.float()) and torch.equal(kd, scales)
    assert s.eng.status() == 0


@pytest.mark.parametrize("kind", [I8, E4])
@pytest.mark.parametrize("dt", [BF, HF])
def test_append_borders_and_extremes(dt, kind):
    """values half way between two codes; the largest and smallest of the type; infinity and NaN"""
    s = Setup([64], [64], 2, 2, 64, 16, dt, kind, rot_dim=0)
    v = torch.zeros((64, 2, 64), dtype=dt, device="cuda")
    n = torch.arange(64, device="cuda")
    v[:, 0] = ((n[:, None] + 1) * (n[None] - 31.5) / 32).to(dt)
    v[:, 1] = (torch.randint(-255, 256, (64, 64), device="cuda").float() / 2).to(dt)
    v[:, 1, 0] = 127
    big, small = torch.finfo(dt).max, torch.finfo(dt).smallest_normal * torch.finfo(dt).eps
    v[7, 0], v[8, 0] = big * torch.linspace(-1, 1, 64, device="cuda"), small * torch.arange(64, device="cuda")
    v[9, 0], v[10, 0] = 0, -big
    s.eng.append(s.cache, s.batch, v, v)
    codes, scales = quantised(v.double(), kind)
    for c, d in stored(s):
        assert torch.equal(c, codes.float())
        assert ((d.double() - scales.double()).abs() <= 2.0 ** -149).all()
    for bad in (math.inf, -math.inf, math.nan):
        w = v.clone()
        w[11, 1, 5] = bad
        s.eng.append(s.cache, s.batch, w, w)
        for c, d in stored(s):
            assert torch.isnan(d[11, 1]) and not c[11, 1].any()
            keep = torch.ones_like(d, dtype=torch.bool)
            keep[11, 1] = False
            assert torch.equal(c[keep], codes.float()[keep]) and torch.isfinite(d[keep]).all()
    out = s.eng.window(s.cache, s.batch, torch.ones((64, 2, 64), dtype=dt, device="cuda"), scale=1e-3)
    assert torch.isnan(out[11:, 1]).all() and torch.isfinite(out[:11]).all() and torch.isfinite(out[:, 0]).all()
    assert s.eng.status() == 0


def test_append_positions_and_pages_out_of_range():
    """more new tokens than cached ones: the first are not stored; a page out of range is reported and not written"""
    s = Setup([9, 3], [4, 3], 4, 2, 64, 16, BF, I8, rot_dim=0)
    k = torch.randn((12, 2, 64), device="cuda").to(BF)
    before = s.kc.clone()
    s.eng.append(s.cache, s.batch, k, k)
    assert s.eng.status() == 0
    pg = s.table.long()[0, 0]
    codes, _ = quantised(k.double(), I8)
    assert torch.equal(s.kc[pg, :, :4].transpose(0, 1), codes[5:9])
    assert torch.equal(s.kc[pg, :, 4:], before[pg, :, 4:])
    s.table[1, 0] = s.kc.shape[0]
    before = s.kc.clone()
    s.eng.append(s.cache, s.batch, k, k)
    assert s.eng.status() == -1 and torch.equal(s.kc, before)


# ---- together ----

@pytest.mark.parametrize("kind", [I8, E4])
def test_decode_steps_in_a_graph(kind):
    """a prompt, then single tokens: append and window captured once and replayed, against the definition each step"""
    T = 4
    s = Setup([30] * T, [30] * T, 8, 2, 64, 16, BF, kind, seed=2)
    table = torch.arange(T * 4, dtype=torch.int32, device="cuda").view(T, 4)
    n = T * 4
    s.kc, s.vc = (torch.full((n, 2, 16, 64), 255, dtype=torch.uint8, device="cuda").view(kind) for _ in range(2))
    s.ks, s.vs = (torch.full((n, 2, 16), math.nan, device="cuda") for _ in range(2))
    s.cache, s.table = s.eng.bind_cache(s.kc, s.vc, s.ks, s.vs), table
    r = lambda t, h: torch.randn((t, h, 64), device="cuda").to(BF)  # noqa: E731
    s.batch = attn.Batch(s.batch.q_start, s.batch.kv_len, table, n_tokens=s.T, max_q=30)
    s.q = s.eng.append(s.cache, s.batch, r(s.T, 2), r(s.T, 2), r(s.T, 8))
    s.window(window=20, sinks=2)
    s.news, s.T, s.start = [1] * T, T, list(range(T + 1))
    lens = i32([31] * T)
    s.batch = attn.Batch(i32(s.start), lens, table, n_tokens=T, max_q=1)
    q, k, v, out = r(T, 8), r(T, 2), r(T, 2), torch.empty((T, 8, 64), dtype=BF, device="cuda")
    s.q, g = torch.empty_like(q), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.eng.append(s.cache, s.batch, k, v, q, q_out=s.q)
        s.eng.window(s.cache, s.batch, s.q, window=20, sinks=2, out=out)
    for step in range(20):
        q.copy_(r(T, 8)), k.copy_(r(T, 2)), v.copy_(r(T, 2))
        s.lens = [31 + step] * T
        lens.copy_(i32(s.lens))
        g.replay()
        s.check(out, None, s.reference(window=20, sinks=2))
    assert s.eng.status() == 0


# ---- refusals ----

def test_refusals():
    s = Setup([1], [20], 4, 2, 64, 16, BF, I8)
    with pytest.raises(coli.ColiError) as e:  # a shared prefix is a 16-bit cache's
        s.eng.prefix(s.cache, s.batch, s.table[0], i32([16]), s.q)
    assert e.value.status == -6
    kc, vc, ks, vs = s.kc, s.vc, s.ks, s.vs
    for bad in ((kc, vc, ks, None), (kc, vc, None, vs), (kc.float(), vc.float(), ks, vs), (kc, vc.view(E4), ks, vs),
                (kc, vc, ks.double(), vs), (kc, vc, ks[:, :1], vs), (kc[:-1], vc, ks, vs), (kc.cpu(), vc, ks, vs),
                (kc, vc, ks.cpu(), vs), (kc, vc)):
        with pytest.raises(ValueError):
            s.eng.bind_cache(*bad)
    wide = torch.zeros((3, 2, 16, 72), dtype=I8, device="cuda")  # rows of 72 bytes
    sc = torch.zeros((3, 2, 16), device="cuda")
    odd = torch.zeros((3, 2, 18), device="cuda")[..., :16]  # scales every 18 floats
    off = torch.zeros(3 * 2 * 16 + 4, device="cuda")[1:97].view(3, 2, 16)
    same = torch.zeros((3, 1, 16), device="cuda").expand(-1, 2, -1)
    good = torch.zeros((3, 2, 16, 64), dtype=I8, device="cuda")
    for bad in ((wide[..., :64], good, sc, sc), (good, good, odd, sc), (good, good, sc, off), (good, good, same, sc)):
        with pytest.raises(coli.ColiError) as e:
            s.eng.bind_cache(*bad)
        assert e.value.status == -1
