"""The 4-bit products where the inputs' sizes differ by more than fp32 holds, and quantize on another stream.  Bounds are those of
test_gpu_linear.py: every product counts with its own size, so what is multiplied by 0 counts nothing."""
import pytest
import torch

from int4_routed_expert_quantize_gb300 import linear

from .test_gpu_linear import BF, HF, check, expanded, weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)


def microseconds(rows, cols, tokens, handles=6, calls=60):
    """a call among others, with weights that are not in the L2"""
    lins = [linear.Int4Linear(*weights(rows, cols, 128, BF, i), max_tokens=tokens) for i in range(handles)]
    x = torch.randn((tokens, cols), device="cuda").to(BF)
    y = torch.empty((tokens, rows), dtype=BF, device="cuda")
    times = []
    for _ in range(6):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for i in range(calls):
            lins[i % handles].forward(x, out=y)
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b) / calls * 1e3)
    return min(times[1:])


@pytest.mark.parametrize("tokens", [1, 8, 12, 16, 20, 40])
@pytest.mark.parametrize("rows,cols,group", [(33, 384, 128), (40, 640, 64), (9, 1184, 32), (200, 6144, 128), (24, 16384, 64)])
def test_outlier_at_codes_of_zero(rows, cols, group, tokens):
    """one value 2^41 and one 2^100 times the others, in columns whose codes are 0"""
    packed, scales = weights(rows, cols, group, BF)
    packed[:, 3], packed[:, cols // 4] = 0, 0  # columns 6, 7 and two in the middle
    lin = linear.Int4Linear(packed, scales, max_tokens=tokens)
    x = torch.randn((tokens, cols), device="cuda").to(BF)
    x[:, 6], x[:, cols // 2] = 2.0 ** 41, -2.0 ** 100
    check(lin.forward(x), x, expanded(packed, scales), group, BF)
    x[:, 6], x[:, cols // 2] = 2.0 ** -100, 0
    x[0] *= 2.0 ** -90
    check(lin.forward(x), x, expanded(packed, scales), group, BF)
    assert lin.status() == 0


@pytest.mark.parametrize("tokens", [1, 12, 20])
@pytest.mark.parametrize("rows,cols,group", [(33, 384, 128), (40, 640, 64), (9, 1184, 32), (200, 6144, 128)])
def test_groups_of_different_sizes(rows, cols, group, tokens):
    """a group of values 2^45 times the others', with scales 2^45 below"""
    packed, scales = weights(rows, cols, group, BF)
    scales[:, 1] *= 2.0 ** -45
    lin = linear.Int4Linear(packed, scales, max_tokens=tokens)
    x = torch.randn((tokens, cols), device="cuda").to(BF)
    x[:, group:2 * group] *= 2.0 ** 45
    check(lin.forward(x), x, expanded(packed, scales), group, BF)
    assert lin.status() == 0


def test_clusters_run_at_once():
    """columns that take clusters of three CTAs cost their bytes, 1.33 times those of two, and not a second round of clusters (2.2
    times; 1.4 without one)"""
    assert microseconds(8192, 8192, 16) < 1.8 * microseconds(8192, 6144, 16)


@pytest.mark.parametrize("handle", [False, True])
def test_quantize_on_another_stream(handle):
    """its outputs' memory is not what the current stream still has work queued on, nor is it given to their stream again while
    the current one reads it"""
    w = torch.randn((512, 512), device="cuda")
    want, side = linear.quantize(w, 64, HF), torch.cuda.Stream()
    assert all(torch.equal(a, b) for a, b in zip(linear.quantize(w, 64, HF, stream=0), want))
    torch.cuda.synchronize()
    old = [torch.empty_like(t) for t in want]
    at = [t.data_ptr() for t in old]
    torch.cuda._sleep(200_000_000)
    for t in old:
        t.fill_(5)
    del old, t  # free for the current stream's next tensors, and the fills are yet to come
    got = linear.quantize(w, 64, HF, stream=side.cuda_stream if handle else side)
    assert not {t.data_ptr() for t in got} & set(at)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    torch.cuda._sleep(200_000_000)
    copy = [t.clone() for t in got]
    del got
    with torch.cuda.stream(side):
        other = [torch.empty_like(t).fill_(9) for t in want]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(copy, want)) and all((t == 9).all() for t in other)


@pytest.mark.parametrize("rest", [1, 17, 40])
def test_a_short_last_launch(rest):
    """more tokens than one grid takes, with groups of 128: the last launch has few"""
    packed, scales = weights(19, 256, 128, BF)
    first = 8 * 65535
    lin = linear.Int4Linear(packed, scales, max_tokens=1000000)
    x = torch.randn((first + rest, 256), device="cuda").to(BF)
    y = lin.forward(x)
    check(y, x, expanded(packed, scales), 128, BF)
    assert torch.equal(lin.forward(x[-17:]), y[-17:]) and lin.status() == 0
