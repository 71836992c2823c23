"""One decoder layer, attention and routed experts, answering several users behind one shared prompt.

    python examples/shared_prompt_decode.py [--users 4] [--prompt 100] [--steps 8]

The prompt's keys and values are appended to a paged cache once, its tokens attend to one another with the window
operator, and every user's new token then attends to the shared pages and to its own ones with the prefix
operator; the layer's int4 experts follow.  Weights and inputs are random: the layer is the small synthetic one of
gen/workloads.py with 8 query heads of 64 over 2 key heads.  The projections are plain matrix products.
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

from gen import workloads  # noqa: E402
from int4_routed_expert_quantize_gb300 import attn, synthetic  # noqa: E402

N_Q, N_KV, DIM, PAGE = 8, 2, 64, 16


def norm(x):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)


class DecoderLayer:
    """x <- x + W_o attention(norm(x)); x <- x + experts(norm(x)), over a paged cache of `pages` pages"""

    def __init__(self, pages, max_tokens, max_seqs, seed=0):
        wl = workloads.WORKLOADS["tiny_t1"]
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        w = lambda *s: (torch.randn(s, generator=g, device="cuda") * s[0] ** -0.5).to(torch.bfloat16)  # noqa: E731
        self.d = wl.d
        self.w_qkv, self.w_o = w(wl.d, (N_Q + 2 * N_KV) * DIM), w(N_Q * DIM, wl.d)
        self.experts = synthetic.build_layer(wl, max_tokens=max_tokens)
        self.attn = attn.PagedAttention(N_Q, N_KV, DIM, PAGE, max_tokens=max_tokens, max_seqs=max_seqs)
        self.k, self.v = (torch.zeros((pages, N_KV, PAGE, DIM), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.cache = self.attn.bind_cache(self.k, self.v)

    def heads(self, x):
        qkv = (norm(x).to(torch.bfloat16) @ self.w_qkv).view(x.shape[0], N_Q + 2 * N_KV, DIM)
        return qkv[:, :N_Q], qkv[:, N_Q:N_Q + N_KV], qkv[:, N_Q + N_KV:]  # slices; nothing is copied

    def finish(self, x, o):
        x = x + (o.reshape(x.shape[0], -1) @ self.w_o).float()
        return x + self.experts.forward(norm(x))

    def prompt(self, x, batch):
        q, k, v = self.heads(x)
        q = self.attn.append(self.cache, batch, k, v, q)
        return self.finish(x, self.attn.window(self.cache, batch, q))

    def decode(self, x, batch, prefix_table, prefix_len):
        q, k, v = self.heads(x)
        q = self.attn.append(self.cache, batch, k, v, q, pos_base=prefix_len)  # positions go on from the prompt's end
        return self.finish(x, self.attn.prefix(self.cache, batch, prefix_table, prefix_len, q))


def run(users=4, prompt=100, steps=8, seed=0):
    """-> the prompt's outputs and the users' outputs of every step"""
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    shared, own = -(-prompt // PAGE), -(-steps // PAGE)
    layer = DecoderLayer(shared + users * own, max_tokens=max(prompt, users), max_seqs=users, seed=seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    prefix_table, prefix_len = torch.arange(shared, dtype=torch.int32, device="cuda"), i32([prompt])
    tables = shared + torch.arange(users * own, dtype=torch.int32, device="cuda").view(users, own)
    first = layer.prompt(torch.randn((prompt, layer.d), generator=g, device="cuda"),
                         attn.Batch(i32([0, prompt]), prefix_len, prefix_table[None], n_tokens=prompt, max_q=prompt))
    lens = i32([0] * users)
    batch = attn.Batch(torch.arange(users + 1, dtype=torch.int32, device="cuda"), lens, tables, n_tokens=users, max_q=1)
    x, outs = torch.randn((users, layer.d), generator=g, device="cuda"), []
    for _ in range(steps):
        lens += 1  # the batch reads its lengths on the device
        x = layer.decode(x, batch, prefix_table, prefix_len)
        outs.append(x)
    assert layer.attn.status() == 0 and layer.experts.status() == 0
    return first, outs


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    for name, n in (("users", 4), ("prompt", 100), ("steps", 8)):
        ap.add_argument("--" + name, type=int, default=n)
    a = ap.parse_args()
    first, outs = run(a.users, a.prompt, a.steps)
    print(f"prompt {tuple(first.shape)}, {len(outs)} steps of {tuple(outs[0].shape)}, "
          f"mean |x| {first.abs().mean():.3f} -> {outs[-1].abs().mean():.3f}")
