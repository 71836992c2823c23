"""One decoder layer in few bits: 4-bit projections, an 8-bit key/value cache, int4 experts.

    python examples/quantized_decode.py [--users 4] [--prompt 100] [--steps 8] [--cache int8|e4m3]

The users' prompts pass through the layer together, then every user's new token goes step by step, each step one replay
of a captured graph: the projection to queries, keys and values, append and window over the cache, the output projection,
the experts.  Weights and inputs are random: the layer is the small synthetic one of gen/workloads.py with 8 query heads of 64 over
2 key heads.
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

from gen import workloads  # noqa: E402
from int4_routed_expert_quantize_gb300 import attn, linear, synthetic  # noqa: E402

N_Q, N_KV, DIM, PAGE = 8, 2, 64, 16
CACHES = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


def norm(x):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)


class DecoderLayer:
    """x <- x + W_o attention(norm(x)); x <- x + experts(norm(x)), over a paged cache of `pages` pages in 8 bits"""

    def __init__(self, pages, max_tokens, max_seqs, cache="int8", seed=0):
        wl = workloads.WORKLOADS["tiny_t1"]
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.d = wl.d

        def project(rows, cols):
            w = torch.randn((rows, cols), generator=g, device="cuda") * cols ** -0.5
            return linear.Int4Linear(*linear.quantize(w, group=64), max_tokens=max_tokens)

        self.w_qkv, self.w_o = project((N_Q + 2 * N_KV) * DIM, wl.d), project(wl.d, N_Q * DIM)
        self.experts = synthetic.build_layer(wl, max_tokens=max_tokens)
        self.attn = attn.PagedAttention(N_Q, N_KV, DIM, PAGE, max_tokens=max_tokens, max_seqs=max_seqs)
        self.k, self.v = (torch.zeros((pages, N_KV, PAGE, DIM), dtype=torch.uint8, device="cuda").view(CACHES[cache]) for _ in range(2))
        self.ks, self.vs = (torch.zeros((pages, N_KV, PAGE), device="cuda") for _ in range(2))
        self.cache = self.attn.bind_cache(self.k, self.v, self.ks, self.vs)

    def forward(self, x, batch):
        qkv = self.w_qkv.forward(norm(x).to(torch.bfloat16)).view(-1, N_Q + 2 * N_KV, DIM)
        q, k, v = qkv[:, :N_Q], qkv[:, N_Q:N_Q + N_KV], qkv[:, N_Q + N_KV:]  # slices; nothing is copied
        q = self.attn.append(self.cache, batch, k, v, q, q_out=q)  # in place
        o = self.attn.window(self.cache, batch, q)
        x = x + self.w_o.forward(o.view(-1, N_Q * DIM)).float()
        return x + self.experts.forward(norm(x))

    def status(self):
        return [s.status() for s in (self.w_qkv, self.w_o, self.attn, self.experts)]


def run(users=4, prompt=100, steps=8, cache="int8", seed=0):
    """-> the layer, the prompts' outputs and the outputs of every step"""
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    own = -(-(prompt + steps) // PAGE)
    layer = DecoderLayer(users * own, max_tokens=users * prompt, max_seqs=users, cache=cache, seed=seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    tables = torch.arange(users * own, dtype=torch.int32, device="cuda").view(users, own)
    lens = i32([prompt] * users)
    batch = attn.Batch(i32([prompt * u for u in range(users + 1)]), lens, tables, n_tokens=users * prompt, max_q=prompt)
    first = layer.forward(torch.randn((users * prompt, layer.d), generator=g, device="cuda"), batch)
    batch = attn.Batch(i32(list(range(users + 1))), lens, tables, n_tokens=users, max_q=1)
    x, outs, graph = first[prompt - 1::prompt].clone(), [], torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):  # records the step, runs nothing yet
        lens += 1  # the batch reads its lengths on the device
        x.copy_(layer.forward(x, batch))
    for _ in range(steps):
        graph.replay()
        outs.append(x.clone())
    assert layer.status() == [0] * 4
    return layer, first, outs


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    for name, n in (("users", 4), ("prompt", 100), ("steps", 8)):
        ap.add_argument("--" + name, type=int, default=n)
    ap.add_argument("--cache", choices=sorted(CACHES), default="int8")
    a = ap.parse_args()
    _, first, outs = run(a.users, a.prompt, a.steps, a.cache)
    print(f"prompts {tuple(first.shape)}, {len(outs)} steps of {tuple(outs[0].shape)}, "
          f"mean |x| {first.abs().mean():.3f} -> {outs[-1].abs().mean():.3f}")
