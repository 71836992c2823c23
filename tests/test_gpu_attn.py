"""The paged-cache attention (coli_attn.h) against its definition in 64 bits: ragged batches of queries,
windows and sinks, rows that see nothing, pages of every size, strided caches and queries, infinities
and NaN in places that a row does not see, shared prefixes, the append's rotation at large positions.

Bounds, derived from the formats.  With u the unit roundoff of the type (2^-8 bf16, 2^-11 fp16), the
weights are rounded once before they multiply V and the output once: |o - o*| <= u * (sum_j p_j |v_j| +
|o*|), both with the normalised weights p.  Scores are fp32 sums of D products with an error of at most
D * 2^-24 * scale * sum|q_i k_i|, under 1e-4 for the inputs here, which moves every weight by as much
relatively; exp2 and the sums add less.  fp16 weights below 2^-14 lose bits: 2^-25 each, times the number of
keys and the largest |v|."""
import math

import pytest
import torch

from int4_routed_expert_quantize_gb300 import attn, coli

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)


class Setup:
    """a ragged batch over a cache of randomly ordered pages; unused slots and pages hold `junk`"""

    def __init__(self, news, lens, n_q, n_kv, D, page, dt, layout="head", prefix=0, junk=float("nan"), seed=0,
                 **kw):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        r = lambda *s: torch.randn(s, generator=g, device="cuda").to(dt)  # noqa: E731
        self.news, self.lens, self.n_q, self.n_kv, self.D, self.page, self.dt = news, lens, n_q, n_kv, D, page, dt
        self.prefix = prefix
        need = [-(-m // page) for m in lens]
        shared = -(-prefix // page)
        n = sum(need) + shared + 2
        order = torch.randperm(n, generator=g, device="cuda")
        if layout == "head":
            self.kc, self.vc = (torch.full((n, n_kv, page, D), junk, dtype=dt, device="cuda") for _ in range(2))
        elif layout == "slot":  # [page, slot, head, value]
            self.kc, self.vc = (torch.full((n, page, n_kv, D), junk, dtype=dt, device="cuda").transpose(1, 2)
                                for _ in range(2))
        else:  # K and V of a page next to each other, wider rows
            both = torch.full((n, 2, n_kv, page, D + 8), junk, dtype=dt, device="cuda")
            self.kc, self.vc = both[:, 0, ..., :D], both[:, 1, ..., :D]
        width = max(need + [1])
        self.table = torch.full((len(news), width + 1), -1, dtype=torch.int32, device="cuda")[:, :width]
        self.keys, self.vals, at = [], [], 0

        def fill(pages, m):
            k, v = r(n_kv, m, D), r(n_kv, m, D)
            pos = torch.arange(m, device="cuda")
            pg, sl = pages[pos // page], pos % page
            self.kc[pg, :, sl] = k.transpose(0, 1)
            self.vc[pg, :, sl] = v.transpose(0, 1)
            return k.double(), v.double()

        for b, (m, c) in enumerate(zip(lens, need)):
            self.table[b, :c] = order[at:at + c].int()
            k, v = fill(order[at:at + c], m)
            self.keys.append(k), self.vals.append(v)
            at += c
        self.prefix_table = order[at:at + max(shared, 1)].int()
        self.prefix_len = torch.tensor([prefix], dtype=torch.int32, device="cuda")
        self.pk, self.pv = fill(order[at:at + shared], prefix) if prefix else (None, None)
        self.T = sum(news)
        self.q = r(self.T, n_q, D)
        start = [sum(news[:i]) for i in range(len(news) + 1)]
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        self.start = start
        self.eng = attn.PagedAttention(n_q, n_kv, D, page, max_tokens=max(self.T, 1), max_seqs=len(news), dtype=dt, **kw)
        self.cache = self.eng.bind_cache(self.kc, self.vc)
        self.batch = attn.Batch(i32(start), i32(lens), self.table, n_tokens=self.T, max_q=max(news + [1]))

    def reference(self, window=-1, sinks=0, scale=None):
        """-> (o, sum_j p_j |v_j|, lse, keys) in 64 bits; rows without keys: 0, 0, -inf"""
        G, scale = self.n_q // self.n_kv, scale or 1 / math.sqrt(self.D)
        o = torch.zeros((self.T, self.n_q, self.D), dtype=torch.float64, device="cuda")
        a, lse = torch.zeros_like(o), torch.full(o.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
        for b, (n, m) in enumerate(zip(self.news, self.lens)):
            for i in range(n):
                p = m - n + i
                j = torch.arange(m, device="cuda")
                see = j <= p
                if window >= 0:
                    see &= (p - j < window) | (j < sinks)
                k, v = self.keys[b][:, see], self.vals[b][:, see]
                if self.prefix:
                    k, v = torch.cat((self.pk, k), 1), torch.cat((self.pv, v), 1)
                if k.shape[1] == 0:
                    continue
                t = self.start[b] + i
                q = self.q[t].double().view(self.n_kv, G, self.D)
                s = q @ k.transpose(1, 2) * scale
                w = torch.softmax(s, -1)
                o[t] = (w @ v).reshape(self.n_q, self.D)
                a[t] = (w @ v.abs()).reshape(self.n_q, self.D)
                lse[t] = torch.logsumexp(s, -1).reshape(self.n_q)
        return o, a, lse

    def off(self, out, ref):
        """each value's error as a share of its bound"""
        o, a, _ = ref
        bound = U[self.dt] * (a + o.abs()) + 2e-4 * a + 1e-30
        if self.dt is HF:
            bound = bound + (max(self.lens) + self.prefix) * 2.0 ** -25 * 6
        return (out.double() - o).abs() / bound

    def check(self, out, lse, ref):
        l = ref[2]
        assert torch.isfinite(out).all()
        worst = self.off(out, ref).max() if out.numel() else 0.0
        assert worst <= 1, float(worst)
        if lse is not None:
            assert torch.equal(torch.isinf(lse), torch.isinf(l))
            f = torch.isfinite(l)
            assert ((lse.double() - l)[f].abs() <= 2e-4).all()
        assert self.eng.status() == 0

    def window(self, **kw):
        lse = torch.full((self.T, self.n_q), 7.0, device="cuda")
        out = torch.full((self.T, self.n_q, self.D), 7.0, dtype=self.dt, device="cuda")
        self.eng.window(self.cache, self.batch, self.q, out=out, lse=lse, **kw)
        self.check(out, lse, self.reference(**kw))
        return out

    def shared(self, **kw):
        lse = torch.full((self.T, self.n_q), 7.0, device="cuda")
        out = torch.full((self.T, self.n_q, self.D), 7.0, dtype=self.dt, device="cuda")
        self.eng.prefix(self.cache, self.batch, self.prefix_table, self.prefix_len, self.q, out=out, lse=lse, **kw)
        self.check(out, lse, self.reference(**kw))
        return out


# ---- window ----

@pytest.mark.parametrize("news,lens", [
    ([1], [1]), ([1], [64]), ([1], [65]), ([1], [2049]), ([1, 1, 1], [1, 700, 63]), ([5, 5, 5], [5, 333, 1000]),
    ([300], [300]), ([257], [1000]), ([1, 129, 1, 40], [900, 400, 1, 40]), ([0, 3, 0], [7, 9, 0]),
    ([1] * 70, list(range(1, 71)))])
@pytest.mark.parametrize("window,sinks", [(-1, 0), (100, 4), (1, 0), (0, 3), (128, 130)])
def test_window_lengths(news, lens, window, sinks):
    Setup(news, lens, 6, 2, 128, 16, BF).window(window=window, sinks=sinks)


@pytest.mark.parametrize("n_q,n_kv,D,page,dt,layout", [
    (1, 1, 64, 16, HF, "head"), (8, 1, 128, 32, BF, "slot"), (16, 1, 64, 64, BF, "both"), (17, 1, 128, 128, HF, "head"),
    (64, 1, 64, 256, HF, "slot"), (33, 1, 128, 16, BF, "both"), (15, 5, 64, 16, BF, "head"), (4, 4, 128, 256, HF, "both")])
@pytest.mark.parametrize("news,lens", [([1, 1], [500, 33]), ([7, 2], [300, 2]), ([150, 70], [400, 70])])
def test_window_heads_pages_layouts(n_q, n_kv, D, page, dt, layout, news, lens):
    s = Setup(news, lens, n_q, n_kv, D, page, dt, layout)
    s.window(window=-1)
    s.window(window=77, sinks=20)


@pytest.mark.parametrize("news,lens,window,sinks", [
    ([3], [0], -1, 0), ([5, 2], [2, 9], -1, 0), ([2, 1], [50, 60], 0, 0), ([200], [90], 16, 0)])
def test_window_rows_that_see_nothing(news, lens, window, sinks):
    """an empty cache, more queries than cached tokens, a window of 0: zeros and -inf"""
    Setup(news, lens, 8, 2, 64, 16, BF).window(window=window, sinks=sinks)


def test_window_ignores_what_a_row_does_not_see():
    """inf and NaN in later tokens' keys and values and in those that left the window"""
    for news, lens in (([1], [400]), ([6], [400]), ([300], [400])):
        s = Setup(news, lens, 8, 2, 128, 32, BF)
        W = 64
        s.window(window=W, sinks=3)
        ref = s.reference(window=W, sinks=3)
        last, first = lens[0] - 1, lens[0] - news[0] - W  # the last token; the last one that no query sees
        for j, bad in ((last, math.nan), (last, math.inf), (first, math.nan), (5, -math.inf)):
            pg, sl = int(s.table[0, j // 32]), j % 32
            keep = s.kc[pg, :, sl].clone(), s.vc[pg, :, sl].clone()
            s.kc[pg, :, sl], s.vc[pg, :, sl] = bad, bad
            out = s.eng.window(s.cache, s.batch, s.q, window=W, sinks=3)
            p = torch.arange(lens[0] - news[0], lens[0], device="cuda")
            blind = ~((j <= p) & ((p - j < W) | (j < 3)))
            assert blind.any() or news == [1]
            assert (s.off(out, ref)[blind] <= 1).all(), (news, j, bad)
            assert not torch.isfinite(out[~blind]).any(), (news, j, bad)
            s.kc[pg, :, sl], s.vc[pg, :, sl] = keep


def test_window_visible_values_that_are_not_finite():
    """a single infinite value that some of a call's rows see reaches those rows' column alone"""
    for news in (1, 9, 140):
        s = Setup([news], [200], 8, 2, 64, 16, HF, seed=3)
        s.window(window=-1)
        ref = s.reference(window=-1)
        j = 199 - news // 2
        s.vc[int(s.table[0, j // 16]), 1, j % 16, 9] = math.inf
        out = s.eng.window(s.cache, s.batch, s.q, window=-1)
        p = torch.arange(200 - news, 200, device="cuda")
        hit = torch.zeros_like(out, dtype=torch.bool)
        hit[p >= j, 4:, 9] = True
        assert (s.off(out, ref)[~hit] <= 1).all()
        assert (out[hit] == math.inf).all()


def test_window_strides_streams_and_graphs():
    s = Setup([3, 1, 20], [70, 300, 20], 6, 2, 128, 64, BF, "slot")
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
        s.batch.kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
        s.lens = lens
        s.keys = [k[:, :m] for k, m in zip(s.keys, lens)]
        s.vals = [v[:, :m] for v, m in zip(s.vals, lens)]
        g.replay()
        s.check(buf, None, s.reference(window=90, sinks=2))


def test_window_many_sequences():
    """more than 32 sequences are placed through shared memory; long and short ones in one batch, empty ones between"""
    r = torch.Generator().manual_seed(5)
    lens = torch.randint(1, 400, (90,), generator=r).tolist()
    news = [0 if i % 7 == 3 else 1 for i in range(90)]
    Setup(news, lens, 8, 2, 64, 16, HF).window(window=150, sinks=5)
    news = [min(m, 120) if i % 10 == 4 else n for i, (n, m) in enumerate(zip(news, lens))]
    Setup(news, lens, 8, 2, 64, 16, HF).window(window=150, sinks=5)


def test_window_offsets_past_32_bits():
    """a cache whose elements do not fit 32-bit offsets: pages at its end"""
    n, page, D = 2 ** 15 + 40, 256, 128  # 2 heads: 2^31 elements and more, 4.3 GB each
    kc, vc = (torch.zeros((n, 2, page, D), dtype=BF, device="cuda") for _ in range(2))
    s = Setup([1, 90], [300, 400], 6, 2, D, page, BF, junk=0.0)
    eng = attn.PagedAttention(6, 2, D, page, max_tokens=91, max_seqs=2, rot_dim=0)
    cache = eng.bind_cache(kc, vc)
    far = torch.arange(n - 1, n - 1 - s.kc.shape[0], -1, device="cuda")
    kc[far], vc[far] = s.kc, s.vc
    batch = attn.Batch(s.batch.q_start, s.batch.kv_len, far[s.table.long()].int(), n_tokens=91, max_q=90)
    assert torch.equal(eng.window(cache, batch, s.q, window=200, sinks=3), s.window(window=200, sinks=3))
    k = torch.randn((91, 2, D), device="cuda").to(BF)
    eng.append(cache, batch, k, k)
    s.eng.append(s.cache, s.batch, k, k)
    assert torch.equal(vc[far], s.vc) and eng.status() == 0


def test_window_repeats_bit_for_bit():
    s = Setup([1] * 9, [4000, 1, 2, 900, 901, 77, 65, 64, 63], 48, 8, 128, 64, BF)
    a = s.window(window=2000, sinks=4)
    for _ in range(5):
        assert torch.equal(s.eng.window(s.cache, s.batch, s.q, window=2000, sinks=4), a)


def test_window_many_calls_in_a_row():
    """hundreds of long-row calls that nothing waits between: none of their bounded waits gives up"""
    s = Setup([1500], [2600], 8, 2, 128, 64, BF)
    a = s.window(window=-1)
    for _ in range(300):
        b = s.eng.window(s.cache, s.batch, s.q, window=-1)
    assert torch.equal(a, b) and s.eng.status() == 0


# ---- prefix ----

@pytest.mark.parametrize("n_q,n_kv,D,page,dt,layout", [
    (6, 2, 128, 64, BF, "head"), (15, 15, 64, 16, HF, "slot"), (20, 1, 64, 32, BF, "both"), (64, 1, 128, 128, HF, "head")])
@pytest.mark.parametrize("news,lens,prefix", [
    ([1], [1], 1), ([1, 1, 1], [5, 1, 200], 64), ([1, 2, 1, 4], [0, 2, 70, 9], 1000), ([1] * 40, list(range(40)), 129),
    ([1, 1], [3, 4], 0), ([2, 1], [0, 0], 0), ([3] * 30, [30] * 30, 2500)])
def test_prefix(n_q, n_kv, D, page, dt, layout, news, lens, prefix):
    s = Setup(news, lens, n_q, n_kv, D, page, dt, layout, prefix=prefix)
    a = s.shared()
    assert torch.equal(s.eng.prefix(s.cache, s.batch, s.prefix_table, s.prefix_len, s.q), a)


@pytest.mark.parametrize("n_q,n_kv", [(4, 2), (32, 1)])
def test_prefix_ignores_what_a_row_does_not_see(n_q, n_kv):
    """infinities and NaN in a later token's key and value, behind the suffix and behind the prefix"""
    for bad in (math.nan, math.inf):
        s = Setup([3, 2, 1], [40, 7, 90], n_q, n_kv, 64, 16, BF, prefix=70)
        s.shared()
        ref = s.reference()
        j = 39  # the last token of the first sequence: its two earlier queries do not see it
        pg = int(s.table[0, j // 16])
        s.kc[pg, :, j % 16], s.vc[pg, :, j % 16] = bad, bad
        out = s.eng.prefix(s.cache, s.batch, s.prefix_table, s.prefix_len, s.q)
        keep = torch.ones(6, dtype=torch.bool, device="cuda")
        keep[2] = False
        assert (s.off(out, ref)[keep] <= 1).all() and not torch.isfinite(out[2]).any()
        # the flags of that call are gone: the next one is clean again
        s.kc[pg, :, j % 16], s.vc[pg, :, j % 16] = s.keys[0][:, j].to(BF), s.vals[0][:, j].to(BF)
        s.shared()


@pytest.mark.parametrize("n_q,n_kv,D,page,dt,seqs,news", [
    (16, 16, 128, 16, BF, 20, [1, 3, 0, 2]), (48, 8, 128, 64, BF, 70, [1]), (64, 8, 64, 32, HF, 45, [1, 5, 2]),
    (256, 8, 64, 128, BF, 40, [1, 2]), (10, 5, 128, 256, HF, 150, [4, 1])])
@pytest.mark.parametrize("prefix", [0, 1, 70, 1500])
def test_prefix_many_sequences(n_q, n_kv, D, page, dt, seqs, news, prefix):
    """more than two blocks of own keys an SM: sequences and prefix in launches of their own; equal calls give equal bits"""
    news = (news * seqs)[:seqs]
    s = Setup(news, [n + 37 * i % 150 for i, n in enumerate(news)], n_q, n_kv, D, page, dt, prefix=prefix)
    assert s.eng.launches("prefix", seqs) == 3
    a = s.shared()
    for _ in range(20):
        assert torch.equal(s.eng.prefix(s.cache, s.batch, s.prefix_table, s.prefix_len, s.q), a)
    assert s.eng.status() == 0


def test_prefix_many_sequences_ignore_what_a_row_does_not_see():
    """the rows that see NaN, and only they, have it; the call after it is clean again"""
    s = Setup([2] * 160, [20 + i for i in range(160)], 8, 2, 64, 16, BF, prefix=300)
    a = s.shared()
    j = s.lens[7] - 1  # the last token of sequence 7: the query before it does not see it
    pg = int(s.table[7, j // 16])
    s.kc[pg, :, j % 16], s.vc[pg, :, j % 16] = math.nan, math.nan
    out = s.eng.prefix(s.cache, s.batch, s.prefix_table, s.prefix_len, s.q)
    keep = torch.ones(s.T, dtype=torch.bool, device="cuda")
    keep[15] = False
    assert (s.off(out, s.reference())[keep] <= 1).all() and not torch.isfinite(out[15]).any()
    s.kc[pg, :, j % 16], s.vc[pg, :, j % 16] = s.keys[7][:, j].to(BF), s.vals[7][:, j].to(BF)
    assert torch.equal(s.eng.prefix(s.cache, s.batch, s.prefix_table, s.prefix_len, s.q), a)


# ---- append ----

def rotated(x, pos, freq, rot, interleaved):
    x = x.double()
    u, v = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    c, s = torch.cos(pos[:, None, None] * freq), torch.sin(pos[:, None, None] * freq)
    a, b = u * c - v * s, v * c + u * s
    y = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((y, x[..., rot:]), -1)


@pytest.mark.parametrize("n_q,n_kv,D,page,dt,layout,rot,inter", [
    (6, 2, 128, 16, BF, "head", 128, False), (3, 3, 64, 64, HF, "slot", 32, True), (8, 1, 128, 256, BF, "both", 64, False),
    (5, 1, 64, 32, HF, "head", 64, True), (2, 2, 128, 16, BF, "slot", 0, False), (48, 8, 128, 64, HF, "both", 16, True)])
@pytest.mark.parametrize("news,lens", [([1], [1]), ([1, 1, 1], [64, 1, 1000]), ([0, 17, 3, 0], [5, 17, 200, 0]),
                                       ([400], [800]), ([4, 2], [1, 2])])
def test_append(n_q, n_kv, D, page, dt, layout, rot, inter, news, lens):
    """cache slots of the new tokens hold the rotated keys and the values, all others what they held"""
    s = Setup(news, lens, n_q, n_kv, D, page, dt, layout, junk=3.0, rot_dim=rot, interleaved=inter, rope_base=5e5)
    qkv = torch.randn((s.T, n_q + 2 * n_kv, D), device="cuda").to(dt)
    q, k, v = qkv[:, :n_q], qkv[:, n_q:n_q + n_kv], qkv[:, n_q + n_kv:]
    kc, vc = s.kc.clone(), s.vc.clone()
    base = torch.tensor([100000], dtype=torch.int32, device="cuda")
    for off in (None, base):
        got = s.eng.append(s.cache, s.batch, k, v, q, pos_base=off)
        pos = torch.cat([torch.arange(m - n, m) for n, m in zip(news, lens)]).cuda()
        freq = torch.tensor([5e5 ** (-2 * i / max(rot, 1)) for i in range(rot // 2)], dtype=torch.float64, device="cuda")
        at = pos.double() + (0 if off is None else 100000)
        rq, rk = rotated(q, at, freq, rot, inter), rotated(k, at, freq, rot, inter)
        # one rounding to the type; sines and cosines of fp32 (2 ulp) and two fp32 products
        tol = lambda r: U[dt] * r.abs() + 1e-6 * 6 + 2.0 ** -25  # noqa: E731
        assert ((got.double() - rq).abs() <= tol(rq)).all()
        ek, ev = kc.double(), vc.clone()
        for t, (p, b) in enumerate(zip(pos.tolist(), [b for b, n in enumerate(news) for _ in range(n)])):
            if p >= 0:
                pg = int(s.table[b, p // page])
                ek[pg, :, p % page], ev[pg, :, p % page] = rk[t], v[t]
        assert ((s.kc.double() - ek).abs() <= tol(ek)).all()
        assert torch.equal(s.vc, ev)
    inplace = q.clone()
    assert torch.equal(s.eng.append(s.cache, s.batch, k, v, inplace, q_out=inplace, pos_base=base), got)
    assert torch.equal(inplace, got)
    before = s.kc.clone()
    assert s.eng.append(s.cache, s.batch, k, v, pos_base=base) is None  # keys and values alone
    assert torch.equal(s.kc, before)
    assert s.eng.status() == 0


def test_append_large_positions():
    """the angle's error does not grow with the position; a table of frequencies replaces the base"""
    freq = [1.0, 0.5, 0.1, 1e-3, 1e-6, 7.0, 0.3, 0.01]
    s = Setup([2], [40], 2, 1, 64, 16, HF, rot_dim=16, inv_freq=freq, junk=0.0)
    q = torch.randn((2, 2, 64), device="cuda").half()
    k, v = q[:, :1].contiguous(), q[:, 1:].contiguous()
    for far in (10 ** 6, 2 ** 31 - 50, -(10 ** 6)):
        off = torch.tensor([far], dtype=torch.int32, device="cuda")
        got = s.eng.append(s.cache, s.batch, k, v, q, pos_base=off)
        pos = torch.tensor([far + 38, far + 39], dtype=torch.float64, device="cuda")
        # the reference's own angle in 64 bits is off by 2^31 * 7 * 2^-53 = 1.7e-6
        want = rotated(q, pos, torch.tensor(freq, dtype=torch.float64, device="cuda"), 16, False)
        assert ((got.double() - want).abs() <= 2.0 ** -11 * want.abs() + 2e-5).all()


# ---- refusals ----

def test_lengths_and_pages_out_of_range_are_reported():
    """clamped or read as zeros, never out of bounds; the status word says so once"""
    s = Setup([1, 1], [40, 40], 4, 2, 64, 16, BF, junk=0.0)
    s.batch.kv_len.copy_(torch.tensor([1000, -5], dtype=torch.int32))  # past the table; negative
    s.eng.window(s.cache, s.batch, s.q)
    assert s.eng.status() == -1 and s.eng.status() == 0
    s.batch.kv_len.copy_(torch.tensor([40, 40], dtype=torch.int32))
    s.table[0, 1], s.table[1, 2] = 10 ** 6, -3
    out = s.eng.window(s.cache, s.batch, s.q)
    assert torch.isfinite(out).all() and s.eng.status() == -1
    kc = s.kc.clone()
    k = torch.ones((2, 2, 64), dtype=BF, device="cuda")
    s.batch.kv_len.copy_(torch.tensor([20, 40], dtype=torch.int32))  # both new tokens in such pages
    s.eng.append(s.cache, s.batch, k, k)
    assert torch.equal(s.kc, kc) and s.eng.status() == -1


def test_more_new_tokens_than_announced_is_reported():
    s = Setup([1, 3], [40, 40], 4, 2, 64, 16, BF, junk=0.0, prefix=50)
    a = s.eng.window(s.cache, s.batch, s.q)
    right = s.batch
    s.batch = attn.Batch(right.q_start, right.kv_len, s.table, n_tokens=4, max_q=2)
    s.eng.window(s.cache, s.batch, s.q)
    assert s.eng.status() == -1
    s.eng.prefix(s.cache, s.batch, s.prefix_table, s.prefix_len, s.q)
    assert s.eng.status() == -1
    s.batch = right
    assert torch.equal(s.eng.window(s.cache, s.batch, s.q), a)
    s.shared()


def test_lists_that_do_not_fit_are_refused():
    """tables so wide that the positions of the work list could pass 32 bits: refused before anything is launched"""
    z = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    wide = z(1, 2 ** 22)  # 2^30 tokens: 2^24 tiles of 64 or 2^23 of 128
    for n_kv, news, group in ((130, 1, 1), (256, 8, 8)):
        eng = attn.PagedAttention(n_kv * group, n_kv, 64, 256, news, 1)
        cache = eng.bind_cache(*[torch.zeros((1, n_kv, 256, 64), dtype=BF, device="cuda") for _ in range(2)])
        q = torch.zeros((news, n_kv * group, 64), dtype=BF, device="cuda")
        start, length = torch.tensor([0, news], dtype=torch.int32, device="cuda"), torch.tensor([news], dtype=torch.int32, device="cuda")
        narrow = attn.Batch(start, length, z(1, 1), n_tokens=news, max_q=news)
        calls = [lambda: eng.window(cache, attn.Batch(start, length, wide, n_tokens=news, max_q=news), q),
                 lambda: eng.prefix(cache, narrow, wide[0], z(1), q)]
        for call in calls:
            before = eng.window(cache, narrow, q)
            with pytest.raises(coli.ColiError) as e:
                call()
            assert e.value.status == -6  # COLI_EUNSUPPORTED
            assert torch.equal(eng.window(cache, narrow, q), before) and eng.status() == 0


def test_refusals():
    s = Setup([1, 1], [40, 40], 4, 2, 64, 16, BF, junk=0.0)
    E = coli.ColiError
    for kw in (dict(sinks=-1), dict(scale=0.0), dict(scale=-1.0), dict(scale=math.inf), dict(scale=math.nan),
               dict(out=s.q)):
        with pytest.raises(E) as e:
            s.eng.window(s.cache, s.batch, s.q, **kw)
        assert e.value.status == -1
    both = torch.zeros((2, 12, 64), dtype=BF, device="cuda")  # queries and outputs between one another, then overlapping
    s.eng.window(s.cache, s.batch, both[:, :4], out=both[:, 4:8])
    for a, b in ((slice(0, 4), slice(2, 6)), (slice(4, 8), slice(1, 5))):
        with pytest.raises(E):
            s.eng.window(s.cache, s.batch, both[:, a], out=both[:, b])
    with pytest.raises(E):  # rotated queries over the keys
        s.eng.append(s.cache, s.batch, both[:, 4:6], both[:, 6:8], both[:, :4], q_out=both[:, 3:7])
    page256 = attn.PagedAttention(4, 2, 64, 256, 4, 4)
    pages = [torch.zeros((1, 2, 256, 64), dtype=BF, device="cuda") for _ in range(2)]
    wide = torch.zeros((2, 2 ** 22 + 1), dtype=torch.int32, device="cuda")
    with pytest.raises(E):  # a table that could hold more than 2^30 tokens
        page256.window(page256.bind_cache(*pages), attn.Batch(s.batch.q_start, s.batch.kv_len, wide, n_tokens=2, max_q=1), s.q)
    odd = torch.zeros(2 * 4 * 64 + 1, dtype=BF, device="cuda")[1:].view(2, 4, 64)
    with pytest.raises(E):
        s.eng.window(s.cache, s.batch, odd)
    with pytest.raises(ValueError):
        s.eng.window(s.cache, s.batch, s.q.half())
    with pytest.raises(ValueError):
        s.eng.window(s.cache, s.batch, s.q[:1])
    with pytest.raises(ValueError):
        s.eng.bind_cache(s.kc[:, :1], s.vc[:, :1])
    many = attn.Batch(torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda"),
                      torch.zeros((3, 1), dtype=torch.int32, device="cuda"), n_tokens=2, max_q=1)
    with pytest.raises(E):  # more sequences than the handle takes
        s.eng.window(s.cache, many, s.q)
    other = attn.PagedAttention(4, 2, 128, 16, 4, 4)
    with pytest.raises(E):  # a cache bound for other shapes
        other.window(s.cache, s.batch, torch.zeros((2, 4, 128), dtype=BF, device="cuda"))
    none = attn.Batch(torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda"),
                      torch.zeros((0, 1), dtype=torch.int32, device="cuda"), n_tokens=0, max_q=1)
    assert s.eng.window(s.cache, none, s.q[:0]).shape == (0, 4, 64)
    torch.cuda.synchronize()
    assert s.eng.status() == 0
