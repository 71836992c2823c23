"""The 4-bit products with group scales (coli_linear.h) against their definition in 64 bits.

Bound: codes and x multiply exactly; a sum of `group` products, of cols / group scaled groups, of up to 16 warps and 8 CTAs is
rounded to fp32 at each addition, by at most 2^-23 of the sum of the magnitudes a = sum |s c x|; the output once, by u of it:
|y - y*| <= (group + cols / group + 24) 2^-23 a + u |y*|, and half of the type's smallest step."""
import math

import pytest
import torch

from int4_routed_expert_quantize_gb300 import coli, linear

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
U = {BF: 2.0 ** -8, HF: 2.0 ** -11}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)


def weights(rows, cols, group, dt, seed=0):
    """codes -8..7 in every place, scales of different sizes"""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    packed = torch.randint(0, 256, (rows, cols // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.exp(0.5 * torch.randn((rows, cols // group), generator=g, device="cuda")) * cols ** -0.5 / 4
    return packed, scales.to(dt)


def expanded(packed, scales):
    """the weights in 64 bits"""
    b = packed.to(torch.int16)
    c = torch.stack((b & 15, b >> 4), -1).flatten(1)
    c = torch.where(c > 7, c - 16, c)
    return c.double() * scales.double().repeat_interleave(2 * packed.shape[1] // scales.shape[1], 1)


def check(y, x, w, group, dt, rows=slice(None)):
    x, y = x.double()[rows], y[rows]
    ref, a = x @ w.T, x.abs() @ w.abs().T
    cols = w.shape[1]
    tiny = torch.finfo(dt).smallest_normal * torch.finfo(dt).eps
    bound = (group + cols / group + 24) * 2.0 ** -23 * a + U[dt] * ref.abs() + tiny
    assert torch.isfinite(y).all()
    worst = ((y.double() - ref).abs() / bound).max()
    assert worst <= 1, float(worst)


SHAPES = [(1, 32, 32), (7, 64, 64), (9, 128, 128), (1111, 1184, 32), (640, 448, 64), (33, 384, 128), (200, 6144, 128),
          (8192, 640, 128), (1000, 6272, 64), (77, 8192, 32), (5000, 2048, 32), (40, 12160, 64), (24, 32768, 128), (16, 32736, 32)]


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("rows,cols,group", SHAPES)
def test_shapes(rows, cols, group, dt):
    packed, scales = weights(rows, cols, group, dt)
    w = expanded(packed, scales)
    lin = linear.Int4Linear(packed, scales, max_tokens=64)
    packed.fill_(0), scales.fill_(math.nan)  # the handle has its own copy
    for tokens in (1, 2, 7, 8, 9, 13, 16, 17, 40, 64):
        x = torch.randn((tokens, cols), device="cuda").to(dt)
        y = torch.full((tokens, rows), math.nan, dtype=dt, device="cuda")
        assert lin.forward(x, out=y) is y
        check(y, x, w, group, dt)
        assert torch.equal(lin.forward(x), y)
    assert lin.status() == 0


def test_many_tokens():
    packed, scales = weights(300, 512, 64, BF)
    lin = linear.Int4Linear(packed, scales, max_tokens=5000)
    x = torch.randn((5000, 512), device="cuda").to(BF)
    check(lin.forward(x), x, expanded(packed, scales), 64, BF)
    assert lin.forward(x[:0]).shape == (0, 300) and lin.status() == 0


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("rows,cols", [(40000, 640), (19460, 1536), (50001, 128)])
def test_tokens_and_rows_of_several_passes(rows, cols, dt):
    packed, scales = weights(rows, cols, 128, dt)
    w = expanded(packed, scales)
    lin = linear.Int4Linear(packed, scales, max_tokens=200)
    wide = torch.randn((200, cols + 8), device="cuda").to(dt)
    for tokens in (17, 32, 33, 64, 65, 100, 200):
        y = torch.full((tokens, rows + 3), 7.0, dtype=dt, device="cuda")
        lin.forward(wide[:tokens, 8:], out=y[:, 1:rows + 1])
        check(y[:, 1:rows + 1], wide[:tokens, 8:], w, 128, dt)
        assert not (y[:, :1] != 7).any() and not (y[:, rows + 1:] != 7).any()
        assert torch.equal(y[:17, 1:rows + 1], lin.forward(wide[:17, 8:]))  # a token's sums do not depend on the others
    assert lin.status() == 0


@pytest.mark.parametrize("cols,tokens", [(32, 600001), (24704, 524291)])
def test_more_tokens_than_one_launch_takes(cols, tokens):
    packed, scales = weights(3, cols, 32, HF)
    lin = linear.Int4Linear(packed, scales, max_tokens=1000000)
    x = torch.zeros((tokens, cols), dtype=HF, device="cuda")
    some = torch.cat((torch.arange(9), torch.arange(524270, 524291), torch.arange(tokens - 9, tokens))).cuda()
    x[some] = torch.randn((len(some), cols), device="cuda").to(HF)
    y = lin.forward(x)
    check(y[some], x[some], expanded(packed, scales), 32, HF)
    assert torch.equal(y[some[:9]], lin.forward(x[:17])[:9]) and lin.status() == 0  # a call's sums have one order


def test_store_past_32_bits():
    """weights of more than 2^32 bytes: the first and the last rows"""
    rows, cols = 1500000, 6144
    packed, scales = weights(rows, cols, 128, BF)
    lin = linear.Int4Linear(packed, scales, max_tokens=2)
    x = torch.randn((2, cols), device="cuda").to(BF)
    y = lin.forward(x)
    for r in (slice(0, 100), slice(rows // 2, rows // 2 + 100), slice(rows - 100, rows)):
        check(y[:, r].contiguous(), x, expanded(packed[r], scales[r]), 128, BF)
    assert lin.status() == 0


@pytest.mark.parametrize("tokens", [3, 12, 30])
def test_strides_streams_and_graphs(tokens):
    packed, scales = weights(133, 1024, 128, HF)
    w = expanded(packed, scales)
    lin = linear.Int4Linear(packed, scales, max_tokens=tokens)
    wide = torch.randn((tokens, 1024 + 40), device="cuda").to(HF)
    x = wide[:, 16:1040]
    want = lin.forward(x)
    check(want, x, w, 128, HF)
    out = torch.full((tokens, 201), 7.0, dtype=HF, device="cuda")  # odd rows: outputs on 2-byte boundaries
    assert torch.equal(lin.forward(x, out=out[:, 5:138]), want)
    assert not (out[:, :5] != 7).any() and not (out[:, 138:] != 7).any()
    both = torch.zeros((tokens, 1024 + 136), dtype=HF, device="cuda")  # x and y in one wider row
    both[:, :1024] = x
    assert torch.equal(lin.forward(both[:, :1024], out=both[:, 1024:1157]), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = lin.forward(x, stream=side)
    same = lin.forward(x)  # one handle on two streams at once
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want) and torch.equal(same, want)
    g, buf, xs = torch.cuda.CUDAGraph(), torch.empty_like(want), x.clone()
    with torch.cuda.graph(g):
        lin.forward(xs, out=buf)
        lin.forward(xs, out=buf)
    for _ in range(3):
        xs.copy_(torch.randn(xs.shape, device="cuda"))
        g.replay()
        check(buf, xs, w, 128, HF)
    assert lin.status() == 0


@pytest.mark.parametrize("cols", [1024, 16384])
@pytest.mark.parametrize("tokens", [5, 11, 33])
def test_tokens_do_not_meet(tokens, cols):
    """a token's output does not depend on the others of calls of its kind, infinities and NaN among them"""
    packed, scales = weights(64, cols, 64, BF)
    lin = linear.Int4Linear(packed, scales, max_tokens=64)
    x = torch.randn((tokens, cols), device="cuda").to(BF)
    want = lin.forward(x)
    x[1], x[3, 5] = math.nan, math.inf
    y = lin.forward(x)
    keep = [t for t in range(tokens) if t not in (1, 3)]
    assert torch.equal(y[keep], want[keep]) and torch.isnan(y[1]).all()


def test_extremes():
    """scales of 0, the largest codes and values"""
    packed = torch.full((16, 128), 0x88, dtype=torch.uint8, device="cuda")  # -8
    scales = torch.ones((16, 2), dtype=BF, device="cuda")
    scales[3] = 0
    scales[4] = 2.0 ** -100
    lin = linear.Int4Linear(packed, scales, max_tokens=4)
    x = torch.ones((3, 256), dtype=BF, device="cuda")
    x[1] = 2.0 ** 100
    x[2] = -0.5
    y = lin.forward(x)
    check(y, x, expanded(packed, scales), 128, BF)
    assert (y[:, 3] == 0).all() and y[0, 0] == -2048 and y[1, 4] == -2048


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("rows,cols,group", [(1, 32, 32), (77, 1280, 64), (300, 6144, 128)])
def test_quantize(rows, cols, group, dt):
    w = torch.randn((rows, cols), device="cuda") * torch.exp(torch.randn((rows, 1), device="cuda"))
    w[0, :group] = 0
    packed, scales = linear.quantize(w, group, dt)
    seven = torch.full((1,), 7.0, device="cuda")  # (a tensor over a number is multiplied by the number's rounded inverse)
    d = (w.view(rows, -1, group).abs().amax(-1) / seven).to(dt)
    assert torch.equal(scales, d)
    q = w.view(rows, -1, group) / d.float()[..., None]
    c = torch.where(d[..., None] == 0, 0, torch.sign(q) * torch.floor(q.abs() + 0.5)).clamp(-7, 7).view(rows, cols)
    got = expanded(packed, torch.ones_like(scales))
    assert torch.equal(got, torch.nan_to_num(c).double())
    lin = linear.Int4Linear(packed, scales, max_tokens=4)
    x = torch.randn((4, cols), device="cuda").to(dt)
    check(lin.forward(x), x, expanded(packed, scales), group, dt)


def test_refusals():
    packed, scales = weights(16, 256, 64, BF)
    lin = linear.Int4Linear(packed, scales, max_tokens=4)
    x = torch.zeros((4, 256), dtype=BF, device="cuda")
    for bad in (x.half(), x[:, :128], x.cpu(), x[0], torch.zeros((4, 512), dtype=BF, device="cuda")[:, ::2], "x"):
        with pytest.raises(ValueError):
            lin.forward(bad)
    for out in (torch.zeros((4, 15), dtype=BF, device="cuda"), torch.zeros((3, 16), dtype=BF, device="cuda"),
                torch.zeros((4, 16), device="cuda")):
        with pytest.raises(ValueError):
            lin.forward(x, out=out)
    flat = torch.zeros(4 * 264 + 8, dtype=BF, device="cuda")
    for bad, out in ((torch.zeros((5, 256), dtype=BF, device="cuda"), None),  # more than max_tokens
                     (flat[1:1 + 4 * 264].view(4, 264)[:, :256], None),  # x on a 2-byte boundary
                     (torch.zeros((4, 257), dtype=BF, device="cuda")[:, :256], None),  # rows of 257
                     (x, x[:, 100:116])):  # y within x
        with pytest.raises(coli.ColiError) as e:
            lin.forward(bad, out=out)
        assert e.value.status == -1
    for p, s in ((packed.int(), scales), (packed, scales.float()), (packed, scales[:8]), (packed[:, ::2], scales),
                 (packed.cpu(), scales), (packed, scales[:, :3])):
        with pytest.raises(ValueError):
            linear.Int4Linear(p, s, max_tokens=4)
    for p, s, status in ((packed, scales[:, :1].contiguous(), -6), (packed, scales.repeat(1, 4), -6)):  # groups of 256 and 16
        with pytest.raises(coli.ColiError) as e:
            linear.Int4Linear(p, s, max_tokens=4)
        assert e.value.status == status
    w = torch.zeros((4, 96), device="cuda")
    for a in ((w.half(), 32, BF), (w, 64, BF), (w, 32, torch.float32), (w.cpu(), 32, BF), (w[:, ::3], 32, BF)):
        with pytest.raises(ValueError):
            linear.quantize(*a)
