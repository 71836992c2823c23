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
