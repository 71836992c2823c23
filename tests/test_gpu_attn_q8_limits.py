"""Window over an 8-bit cache where rows meet what is not theirs: bits that depend on other rows, scales that are not finite one at
a time, queries with an outlier, pages out of range.  Bounds are those of test_gpu_attn_q8.py."""
import math

import pytest
import torch

from .test_gpu_attn_q8 import BF, E4, HF, I8, Setup

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)


def call(s, **kw):
    lse = torch.empty((s.T, s.n_q), device="cuda")
    out = s.eng.window(s.cache, s.batch, s.q, lse=lse, **kw)
    return out, lse


def place(s, b, j):
    return int(s.table[b, j // s.page]), j % s.page


def one_bad_scale(s, scales):
    """rows that see a scale that is not finite are NaN, the others are right"""
    new, W = s.T, 64
    p = torch.arange(400 - new, 400, device="cuda")
    ref = s.reference(window=W, sinks=3)
    for j in (398, 399 - W // 2, 1):
        pg, sl = place(s, 0, j)
        keep = scales[pg, :, sl].clone()
        blind = ~((j <= p) & ((p - j < W) | (j < 3)))
        for bad in (math.inf, -math.inf, math.nan):
            scales[pg, :, sl] = bad
            out, lse = call(s, window=W, sinks=3)
            s.check(out, lse, ref, blind)
            assert torch.isnan(out[~blind]).all() and torch.isnan(lse[~blind]).all()
        scales[pg, :, sl] = keep
    assert s.eng.status() == 0


@pytest.mark.parametrize("kind", [I8, E4])
@pytest.mark.parametrize("n_q,n_kv,D,page,new,length", [
    (5, 1, 64, 64, 5, 300), (40, 8, 64, 64, 5, 2999), (6, 1, 128, 64, 1, 700), (3, 1, 128, 128, 3, 200), (1, 1, 64, 16, 40, 300)])
def test_bits_do_not_come_from_unused_slots(n_q, n_kv, D, page, new, length, kind):
    """a block has more rows than the sequence has tokens: what those would see does not move the others' roundings"""
    s = Setup([new], [length], n_q, n_kv, D, page, HF, kind, junk=0.0)
    want = call(s)
    used = torch.arange(page, device="cuda") < (length - 1) % page + 1
    pg = place(s, 0, length - 1)[0]
    for junk in (1.0, 2.0 ** 40, math.inf, math.nan):
        s.ks[pg][:, ~used] = junk
        s.vs[pg][:, ~used] = junk
        got = call(s)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert s.eng.status() == 0


@pytest.mark.parametrize("kind", [I8, E4])
@pytest.mark.parametrize("new", [3, 40])
def test_bits_do_not_come_from_other_rows(new, kind):
    s = Setup([new], [900], 4, 1, 64, 16, HF, kind)
    want = call(s)
    for factor in (0.0, 64.0, math.nan):  # the last token's scores move much more often, or not at all
        s.q[-1] *= factor
        got = call(s)
        assert torch.equal(got[0][:-1], want[0][:-1]) and torch.equal(got[1][:-1], want[1][:-1])
        s.q[-1] = torch.randn_like(s.q[-1])


@pytest.mark.parametrize("kind", [I8, E4])
@pytest.mark.parametrize("new", [1, 6, 300])
def test_a_key_scale_that_is_not_finite(new, kind):
    """whatever the sign of the row's product with the key"""
    s = Setup([new], [400], 8, 2, 128, 32, BF, kind)
    one_bad_scale(s, s.ks)


@pytest.mark.parametrize("kind", [I8, E4])
@pytest.mark.parametrize("new", [1, 6, 300])
def test_a_value_scale_that_is_not_finite(new, kind):
    s = Setup([new], [400], 8, 2, 128, 32, BF, kind)
    one_bad_scale(s, s.vs)


@pytest.mark.parametrize("kind", [I8, E4])
@pytest.mark.parametrize("new,sinks", [(1, 0), (40, 0)])
def test_a_scale_that_is_not_finite_at_keys_of_no_weight(new, sinks, kind):
    """a whole part of the keys has scores 1000 below the others': its NaN is the row's all the same"""
    s = Setup([new], [6000], 4, 1, 64, 64, BF, kind)
    s.q = torch.ones_like(s.q)
    pages = s.table[0, :32].long()  # 2048 keys
    s.kc.view(torch.uint8)[pages] = torch.full((1, 64), -100.0 if kind is I8 else -448.0, device="cuda").to(kind).view(torch.uint8)
    s.ks[pages] = 1.0
    for scales in (s.vs, s.ks):
        for bad in (math.nan, math.inf):
            pg, sl = place(s, 0, 70)
            keep = scales[pg, :, sl].clone()
            scales[pg, :, sl] = bad
            out, lse = call(s)
            assert torch.isnan(out).all() and torch.isnan(lse).all()
            scales[pg, :, sl] = keep
    out, lse = call(s)
    s.check(out, lse, s.reference())


@pytest.mark.parametrize("kind", [I8, E4])
@pytest.mark.parametrize("n_q,n_kv,D,new", [(6, 1, 128, 1), (4, 2, 64, 5), (17, 1, 64, 1), (8, 2, 64, 60)])
def test_queries_multiply_exactly(n_q, n_kv, D, new, kind):
    """a query value 2^41 times the others', whose codes are 0, leaves the scores of the others alone"""
    s = Setup([new], [500], n_q, n_kv, D, 16, BF, kind)
    s.kc.view(torch.uint8)[..., 5] = 0
    s.q[..., 5] = 2.0 ** 41
    out, lse = call(s)
    s.check(out, lse, s.reference())


@pytest.mark.parametrize("kind", [I8, E4])
@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("new", [1, 40])
def test_every_code_is_exact(new, dt, kind):
    """one key and one-hot queries: the log-sum-exp is the key's value, for each of the 256 codes, a code of the value is the
    output.  (e4m3's 0x7F and 0xFF count as 480 and -480.)  The score is one fp32 product; log2(e) and ln 2 in fp32 and the sum of m and
    log2(1) round it by no more than 2^-22 of itself."""
    D, n = 64, 4
    s = Setup([new] * n, [new] * n, D, 1, D, 64, dt, kind, junk=1.0)
    codes = torch.arange(256, dtype=torch.uint8, device="cuda").view(n, D)
    value = codes.view(kind).float()
    if kind is E4:
        value = torch.where(codes == 127, 480.0, torch.where(codes == 255, -480.0, value))
    for b in range(n):
        pg = int(s.table[b, 0])
        s.kc.view(torch.uint8)[pg], s.vc.view(torch.uint8)[pg] = codes[b], codes[b]
    s.ks.fill_(1.0), s.vs.fill_(1.0)
    s.q = torch.eye(D, device="cuda").to(dt).repeat(s.T, 1, 1)
    out, lse = call(s, scale=1.0)
    m = value.repeat_interleave(new, 0).double()
    own = math.log(1.0)
    count = torch.arange(1, new + 1, device="cuda").repeat(n).double()  # a token sees as many equal keys
    ref = m + torch.log(count)[:, None] + own
    assert ((lse.double() - ref).abs() <= 2.0 ** -22 * (ref.abs() + m.abs()) + 2.0 ** -22).all()
    u = 2.0 ** -8 if dt is BF else 2.0 ** -11
    # equal weights: their fp16 roundings and the sum's cancel to within 2^-11 + 2^-20
    assert ((out.double() - m[:, None]).abs() <= (u + 2.0 ** -11 + 2.0 ** -20) * m[:, None].abs()).all()
    assert s.eng.status() == 0


@pytest.mark.parametrize("kind", [I8, E4])
@pytest.mark.parametrize("news", [[1, 1], [1, 70]])
@pytest.mark.parametrize("bad", [-1, 10 ** 6])
def test_a_page_out_of_range_reads_as_zeros(bad, news, kind):
    """a spare page of zeros, which is in no table, stands in for it in the reference"""
    s = Setup(news, [100, 200], 8, 2, 64, 32, BF, kind)
    spare = (set(range(s.kc.shape[0])) - {int(x) for x in s.table.flatten() if x >= 0}).pop()
    s.kc.view(torch.uint8)[spare], s.vc.view(torch.uint8)[spare], s.ks[spare], s.vs[spare] = 0, 0, 0, 0
    whole = s.reference()
    for b, page in ((0, 1), (1, 0), (1, 3)):
        keep = int(s.table[b, page])
        s.table[b, page] = bad
        out, lse = call(s)
        assert s.eng.status() == -1 and s.eng.status() == 0
        s.table[b, page] = spare
        ref = s.reference()
        s.check(out, lse, ref)
        other = slice(s.start[1 - b], s.start[2 - b])  # the other sequence's rows are those of before
        assert torch.equal(ref[0][other], whole[0][other])
        s.table[b, page] = keep


@pytest.mark.parametrize("kind", [I8, E4])
@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("new", [1, 5, 40])
@pytest.mark.parametrize("far", [20, 60])
def test_values_of_no_weight_cost_no_bits(new, far, dt, kind):
    """values 2^far times the others', at keys whose scores are 1000 below: what is lost of a weight is relative to the largest product of a
    weight and its scale, so the third term of the bound has that in the place of the largest scale"""
    s = Setup([new], [500], 4, 2, 64, 16, dt, kind)
    s.q = s.q.abs() + 1
    for j in (3, 200, 401, 455):  # the last ones in the tiles that only some of 40 rows see whole
        pg, sl = place(s, 0, j)
        s.kc.view(torch.uint8)[pg, :, sl] = torch.full((64,), -100.0 if kind is I8 else -448.0, device="cuda").to(kind).view(torch.uint8)
        s.ks[pg, :, sl] = 2.0
        s.vs[pg, :, sl] = 2.0 ** far
    out, lse = call(s)
    o, bound, ref_lse = s.reference()
    for j in (3, 200, 401, 455):
        pg, sl = place(s, 0, j)
        s.vs[pg, :, sl] = 0.0
    o2, bound2, _ = s.reference()
    assert torch.equal(o, o2)  # no weight, in 64 bits too
    s.check(out, lse, (o, bound2, ref_lse))
