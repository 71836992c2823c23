"""The decoder-layer example: users behind one shared prompt get what one sequence alone gets."""
import os
import runpy

import pytest
import torch

from int4_routed_expert_quantize_gb300 import attn

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "shared_prompt_decode.py")


def test_shared_prompt_decode_equals_one_sequence():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ex = runpy.run_path(PATH)
    users, prompt, steps = 3, 53, 5
    first, outs = ex["run"](users, prompt, steps, seed=4)
    # the same, each user on a cache that holds the prompt and the user's own tokens: window over all keys
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    x0 = torch.randn((prompt, first.shape[1]), generator=g, device="cuda")
    xs = torch.randn((users, first.shape[1]), generator=g, device="cuda")
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    for u in range(users):
        layer = ex["DecoderLayer"](5, max_tokens=prompt, max_seqs=1, seed=4)
        table, n = torch.arange(5, dtype=torch.int32, device="cuda")[None], i32([prompt])
        alone = layer.prompt(x0, attn.Batch(i32([0, prompt]), n, table, n_tokens=prompt, max_q=prompt))
        assert torch.equal(alone, first)
        x, batch = xs[u:u + 1], attn.Batch(i32([0, 1]), n, table, n_tokens=1, max_q=1)
        for t in range(steps):
            n += 1
            x = layer.prompt(x, batch)
            # bf16 attention outputs (2^-8 each way) through products and experts whose int8 codes may step: 2 %
            # of the residual stream's size per step
            assert (x - outs[t][u:u + 1]).abs().max() <= 0.02 * (t + 1) * outs[t].abs().max()
