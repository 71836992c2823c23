"""The attention operators of the paged key/value cache: what is measured, and their plain forms.

Three operators that serve a decoder layer next to its routed experts:

  append  new keys and values go into the paged cache, keys (and queries) rotated on the way
  window  causal attention over the cache: the last `window` keys and the first `sinks` ones
  prefix  attention of a batch whose sequences share one long prefix and have their own suffixes

A batch is ragged: sequence b has the query tokens q_start[b] .. q_start[b+1]-1, which are the last
of its kv_len[b] cached tokens, and its token j sits in slot j % page of page table[b, j // page].
With `own` false, run() computes them in elementary torch operations in 32 bits; with `own` true it
makes the calls a user makes.  Head counts: 48 query heads of 128 are the width 6144 of the expert
layers here; the others are generic.
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}

# one new token for each of 16 running sequences: a decode step's append, where latency counts
A1 = dict(name="append_decode_16", op="append", dtype="bf16", n_q=48, n_kv=8, dim=128, page=64,
          seqs=16, new=1, mix=0, ctx=8192, ragged=1, rot=128, inter=0, base=10000.0)
# ragged prompt chunks, interleaved pairs, half of the width rotated, an odd head group, small pages
A2 = dict(name="append_ragged_chunks", op="append", dtype="fp16", n_q=28, n_kv=4, dim=128, page=16,
          seqs=7, new=331, mix=0, ctx=2600, ragged=2, rot=64, inter=1, base=500000.0)
# a long prompt in one call
A3 = dict(name="append_prompt_16k", op="append", dtype="bf16", n_q=48, n_kv=8, dim=128, page=64,
          seqs=1, new=16384, mix=0, ctx=16384, ragged=3, rot=128, inter=0, base=1000000.0)
# one user, one token, a short context: the smallest call
W1 = dict(name="window_decode_1", op="window", dtype="bf16", n_q=48, n_kv=8, dim=128, page=64,
          seqs=1, new=1, mix=0, ctx=700, ragged=4, window=512, sinks=4)
# a decode step of 64 users with long contexts, of which the window keeps 4096 keys
W2 = dict(name="window_decode_64", op="window", dtype="bf16", n_q=48, n_kv=8, dim=128, page=64,
          seqs=64, new=1, mix=0, ctx=16384, ragged=5, window=4096, sinks=4)
# speculative verification of 5 tokens for each of 13 users; odd window, odd head group, small heads
W3 = dict(name="window_verify_13", op="window", dtype="fp16", n_q=40, n_kv=8, dim=64, page=16,
          seqs=13, new=5, mix=0, ctx=2999, ragged=6, window=1001, sinks=7)
# continuous batching: some users' prompt chunks beside the others' single tokens
W4 = dict(name="window_mixed_16", op="window", dtype="bf16", n_q=48, n_kv=8, dim=128, page=32,
          seqs=16, new=500, mix=1, ctx=4096, ragged=7, window=2048, sinks=16)
# a whole prompt, the window half as long: the largest
W5 = dict(name="window_prompt_8k", op="window", dtype="bf16", n_q=48, n_kv=8, dim=128, page=64,
          seqs=1, new=8192, mix=0, ctx=8192, ragged=8, window=4096, sinks=4)
# four answers drawn from one short prompt
P1 = dict(name="prefix_sample_4", op="prefix", dtype="bf16", n_q=48, n_kv=8, dim=128, page=64,
          seqs=4, new=1, mix=0, prefix=1000, ctx=33, ragged=9)
# 32 users behind one system prompt
P2 = dict(name="prefix_chat_32", op="prefix", dtype="bf16", n_q=48, n_kv=8, dim=128, page=64,
          seqs=32, new=1, mix=0, prefix=8192, ctx=512, ragged=10)
# 2 new tokens for each of 13 sequences, one head per key head, the prefix ends inside a page
P3 = dict(name="prefix_odd_13", op="prefix", dtype="fp16", n_q=15, n_kv=15, dim=64, page=16,
          seqs=13, new=2, mix=0, prefix=4099, ctx=77, ragged=11)
# a large batch behind a long document
P4 = dict(name="prefix_document_256", op="prefix", dtype="bf16", n_q=48, n_kv=8, dim=128, page=64,
          seqs=256, new=1, mix=0, prefix=32768, ctx=1024, ragged=12)


def listed():
    return [dict(c) for c in (A1, A2, A3, W1, W2, W3, W4, W5, P1, P2, P3, P4)]


HEADS = [(48, 8, 128), (32, 8, 128), (28, 4, 128), (40, 8, 64), (14, 14, 64), (15, 5, 64), (8, 1, 128),
         (20, 4, 128), (64, 8, 64), (12, 12, 128)]


def _log(rng, lo, hi):
    """a whole number of lo .. hi, spread over its logarithm; never the width 3072"""
    n = min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))
    return n + 1 if n == 3072 else n


def draw(rng):
    n_q, n_kv, dim = rng.choice(HEADS)
    case = dict(op=rng.choice(["append", "window", "prefix"]), dtype=rng.choice(["bf16", "fp16"]),
                n_q=n_q, n_kv=n_kv, dim=dim, page=rng.choice([16, 32, 64, 128]), mix=0,
                ragged=rng.randrange(1 << 20))
    if case["op"] == "append":
        seqs = _log(rng, 1, 64)
        new = rng.choice([1, _log(rng, 2, max(2, 8192 // seqs))])
        case.update(seqs=seqs, new=new, ctx=max(new, _log(rng, 64, 8192)),
                    rot=rng.choice([dim, dim // 2]), inter=rng.randrange(2),
                    base=rng.choice([10000.0, 500000.0]))
    elif case["op"] == "window":
        kind = rng.choice(["decode", "verify", "mixed", "prompt"])
        window = rng.choice([-1, _log(rng, 1, 4096), _log(rng, 64, 4096)])
        sinks = rng.choice([0, 4, _log(rng, 1, 200)])
        if kind == "prompt":
            n = _log(rng, 33, 4096)
            case.update(seqs=1, new=n, ctx=n + rng.choice([0, _log(rng, 1, 2048)]))
        elif kind == "mixed":
            case.update(seqs=_log(rng, 2, 16), new=_log(rng, 20, 400), ctx=_log(rng, 500, 4096), mix=1)
        else:
            new = 1 if kind == "decode" else rng.randint(2, 8)
            case.update(seqs=_log(rng, 1, 64), new=new, ctx=_log(rng, 64, 4096 if window < 0 else 12000))
        case.update(window=window, sinks=sinks)
    else:
        case.update(seqs=_log(rng, 2, 200), new=rng.choice([1, 1, rng.randint(2, 4)]),
                    prefix=_log(rng, 100, 16384), ctx=_log(rng, 8, 700))
    return case


def _lens(case):
    """new and cached tokens of every sequence (cached counts the new ones)"""
    r = random.Random(case["ragged"])
    news, lens = [], []
    for b in range(case["seqs"]):
        n = case["new"]
        if case["mix"]:
            n = r.randint((n + 1) // 2, n) if r.random() < 0.3 or b == 0 else 1
        elif n > 8 and case["seqs"] > 1:
            n = r.randint((n + 1) // 2, n)
        news.append(n)
        lens.append(max(n, r.randint((case["ctx"] + 3) // 4, case["ctx"]) if case["seqs"] > 1 else case["ctx"]))
    return news, lens


def _visible(case, n, length):
    """(query, key) pairs that see each other, and keys some query sees, of one sequence's own cache"""
    w, s = case.get("window", -1), case.get("sinks", 0)
    pairs = 0
    for p in range(length - n, length):
        lo = 0 if w < 0 else max(0, p - w + 1)
        pairs += p + 1 - lo + min(s, lo)
    lo = 0 if w < 0 else max(0, length - n - w + 1)
    return pairs, length - lo + min(s, lo)


def work(case):
    news, lens = _lens(case)
    T, kv, row = sum(news), 2 * case["n_kv"] * case["dim"], 2 * case["dim"]
    if case["op"] == "append":  # q, k and v read; rotated q and the cache slots written
        return {"bytes": 2 * T * (case["n_q"] + 2 * case["n_kv"]) * row, "flops": 3 * T * (case["n_q"] + case["n_kv"]) * case["rot"]}
    seen = [_visible(case, n, m) for n, m in zip(news, lens)]
    pairs, keys = sum(p for p, _ in seen), sum(k for _, k in seen)
    if case["op"] == "prefix":
        pairs, keys = pairs + T * case["prefix"], keys + case["prefix"]
    return {"bytes": 2 * T * case["n_q"] * row + keys * kv * 2, "flops": 4 * pairs * case["n_q"] * case["dim"]}


def _make(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    news, lens = _lens(case)
    dt, page, D = DT[case["dtype"]], case["page"], case["dim"]
    normal = lambda *shape: torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dt)  # noqa: E731
    T = sum(news)
    need = [-(-m // page) for m in lens]
    shared = -(-case["prefix"] // page) if case["op"] == "prefix" else 0
    n_pages = sum(need) + shared + 3
    order = torch.randperm(n_pages, generator=g, device="cuda", dtype=torch.int64).to(torch.int32)
    table = torch.zeros((case["seqs"], max(need)), dtype=torch.int32)
    at = 0
    rows = torch.arange(n_pages, dtype=torch.int32)
    for b, n in enumerate(need):
        table[b, :n] = rows[at:at + n]
        at += n
    s = dict(case=dict(case), T=T, max_q=max(news),
             q_start=torch.tensor([sum(news[:b]) for b in range(len(news) + 1)], dtype=torch.int32, device="cuda"),
             kv_len=torch.tensor(lens, dtype=torch.int32, device="cuda"),
             table=order[table.to("cuda").long()].contiguous(),
             k_cache=normal(n_pages, case["n_kv"], page, D), v_cache=normal(n_pages, case["n_kv"], page, D))
    if shared:
        s["prefix_table"] = order[at:at + shared].contiguous()
        s["prefix_len"] = torch.tensor([case["prefix"]], dtype=torch.int32, device="cuda")
    if case["op"] == "append":  # slices of the fused projection's rows, as a layer has them
        qkv = normal(T, (case["n_q"] + 2 * case["n_kv"]) * D)
        a, b = case["n_q"] * D, (case["n_q"] + case["n_kv"]) * D
        s["q"] = qkv[:, :a].view(T, case["n_q"], D)
        s["k"] = qkv[:, a:b].view(T, case["n_kv"], D)
        s["v"] = qkv[:, b:].view(T, case["n_kv"], D)
    else:
        s["q"] = normal(T, case["n_q"], D)
    return s


def prepare(case, seed):
    s = _make(case, seed)
    if own:  # the handles a serving program makes once, next to its cache and its batch
        from int4_routed_expert_quantize_gb300 import attn
        s["attn"] = attn.PagedAttention(case["n_q"], case["n_kv"], case["dim"], case["page"], max_tokens=s["T"],
                                        max_seqs=case["seqs"], dtype=DT[case["dtype"]],
                                        rot_dim=case.get("rot", 0), interleaved=bool(case.get("inter", 0)),
                                        rope_base=case.get("base", 10000.0))
        s["cache"] = s["attn"].bind_cache(s["k_cache"], s["v_cache"])
        s["batch"] = attn.Batch(s["q_start"], s["kv_len"], s["table"], n_tokens=s["T"], max_q=s["max_q"])
    return s


def run(s):
    c = s["case"]
    if own:
        if c["op"] == "append":
            q = s["attn"].append(s["cache"], s["batch"], s["k"], s["v"], s["q"])
            return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
        if c["op"] == "window":
            return s["attn"].window(s["cache"], s["batch"], s["q"], window=c["window"], sinks=c["sinks"])
        return s["attn"].prefix(s["cache"], s["batch"], s["prefix_table"], s["prefix_len"], s["q"])
    if c["op"] == "append":
        return _plain_append(s)
    return _plain_window(s) if c["op"] == "window" else _plain_prefix(s)


# ---- the plain forms ----

def _where_is(s):
    """each token's sequence, its index among the sequence's new tokens, and its position"""
    t = torch.arange(s["T"], device="cuda")
    start = s["q_start"].long()
    b = torch.searchsorted(start, t, right=True) - 1
    i = t - start[b]
    return b, i, s["kv_len"].long()[b] - (start[b + 1] - start[b]) + i


def _rotate(x, pos, c):
    """x [T, heads, dim]: the first `rot` values of a head rotated in pairs by pos * base^(-2i/rot)"""
    rot = c["rot"]
    f = c["base"] ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float32) / rot)
    a = pos.to(torch.float32)[:, None] * f
    cos, sin = torch.cos(a)[:, None], torch.sin(a)[:, None]
    x = x.to(torch.float32)
    r = x[..., :rot]
    u, v = (r[..., 0::2], r[..., 1::2]) if c["inter"] else (r[..., :rot // 2], r[..., rot // 2:])
    p, q = u * cos - v * sin, v * cos + u * sin
    y = torch.stack((p, q), -1).flatten(-2) if c["inter"] else torch.cat((p, q), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _plain_append(s):
    c = s["case"]
    b, _, pos = _where_is(s)
    page = s["table"].long()[b, pos // c["page"]]
    slot = pos % c["page"]
    dt = s["k_cache"].dtype
    s["k_cache"][page, :, slot] = _rotate(s["k"], pos, c).to(dt)
    s["v_cache"][page, :, slot] = s["v"]
    return {"q": _rotate(s["q"], pos, c).to(dt), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _padded(s):
    """q as [seqs, n_kv, max_q * group, dim] in 32 bits, scaled"""
    c = s["case"]
    at = (s["q_start"].long()[:-1, None] + torch.arange(s["max_q"], device="cuda")).clamp(max=s["T"] - 1)
    q = s["q"].to(torch.float32)[at] * (1.0 / math.sqrt(c["dim"]))
    q = q.view(c["seqs"], s["max_q"], c["n_kv"], c["n_q"] // c["n_kv"], c["dim"])
    return q.permute(0, 2, 1, 3, 4).reshape(c["seqs"], c["n_kv"], -1, c["dim"])


def _gathered(cache, table):
    """a page table's [..., pages] keys or values in order: [..., n_kv, pages * page, dim] in 32 bits"""
    x = cache[table.long()].to(torch.float32)
    return x.transpose(-4, -3).flatten(-3, -2)


def _own_scores(s, q):
    """scores of the padded queries with their own cache, -inf where a key is not visible"""
    c = s["case"]
    k = _gathered(s["k_cache"], s["table"])
    scores = (q @ k.transpose(-1, -2)).view(c["seqs"], c["n_kv"], s["max_q"], -1, k.shape[-2])
    new = (s["q_start"][1:] - s["q_start"][:-1]).long()
    pos = (s["kv_len"].long() - new)[:, None] + torch.arange(s["max_q"], device="cuda")
    j = torch.arange(k.shape[-2], device="cuda")
    seen = j <= pos[..., None]
    if c.get("window", -1) >= 0:
        seen = seen & ((pos[..., None] - j < c["window"]) | (j < c["sinks"]))
    return torch.where(seen[:, None, :, None], scores, -math.inf).flatten(2, 3)


def _tokens(s, o):
    """[seqs, n_kv, max_q * group, dim] back to [T, n_q, dim] of the inputs' type"""
    c = s["case"]
    b, i, _ = _where_is(s)
    o = o.view(c["seqs"], c["n_kv"], s["max_q"], -1, c["dim"])[b, :, i]
    return o.reshape(s["T"], c["n_q"], c["dim"]).to(s["q"].dtype)


def _plain_window(s):
    x = _own_scores(s, _padded(s))
    top = x.amax(-1, keepdim=True)
    x = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    total = x.sum(-1, keepdim=True)
    o = (x @ _gathered(s["v_cache"], s["table"])) / torch.where(total == 0, 1.0, total)
    return _tokens(s, o)


def _plain_prefix(s):
    c = s["case"]
    q = _padded(s)
    x = _own_scores(s, q)
    n = c["prefix"]
    flat = q.transpose(0, 1).flatten(1, 2)  # [n_kv, seqs * max_q * group, dim]: one product for all
    y = flat @ _gathered(s["k_cache"], s["prefix_table"])[:, :n].transpose(-1, -2)
    y = y.view(c["n_kv"], c["seqs"], -1, n).transpose(0, 1)
    top = torch.maximum(x.amax(-1, keepdim=True), y.amax(-1, keepdim=True))
    x, y = torch.exp(x - top), torch.exp(y - top)
    total = x.sum(-1, keepdim=True) + y.sum(-1, keepdim=True)
    o = x @ _gathered(s["v_cache"], s["table"])
    far = y.transpose(0, 1).flatten(1, 2) @ _gathered(s["v_cache"], s["prefix_table"])[:, :n]
    return _tokens(s, (o + far.view(c["n_kv"], c["seqs"], -1, c["dim"]).transpose(0, 1)) / total)


# ---- the definition in 64 bits: one sequence and one key head after the other ----

def exact(case, seed):
    s = _make(case, seed)
    news, lens = _lens(case)
    if case["op"] == "append":
        return _exact_append(case, s, news, lens)
    G, page, D = case["n_q"] // case["n_kv"], case["page"], case["dim"]
    out = torch.zeros((s["T"], case["n_q"], D), dtype=torch.float64, device="cuda")
    pool = {"k": s["k_cache"], "v": s["v_cache"]}
    first = 0
    for b, (n, m) in enumerate(zip(news, lens)):
        pages = s["table"][b, : -(-m // page)].long()
        p = torch.arange(m - n, m, device="cuda")[:, None]
        j = torch.arange(m, device="cuda")[None, :]
        hidden = j > p
        if case.get("window", -1) >= 0:
            hidden = hidden | ((j <= p - case["window"]) & (j >= case["sinks"]))
        for h in range(case["n_kv"]):
            both = {}
            for name, pages_of in pool.items():
                x = pages_of[pages, h].reshape(-1, D)[:m].double()
                if case["op"] == "prefix":
                    shared = pages_of[s["prefix_table"].long(), h].reshape(-1, D)[: case["prefix"]].double()
                    x = torch.cat((shared, x))
                both[name] = x
            mask = hidden
            if case["op"] == "prefix":
                mask = torch.cat((torch.zeros((n, case["prefix"]), dtype=torch.bool, device="cuda"), hidden), 1)
            for g in range(G):
                for r in range(0, n, 2048):
                    at = slice(first + r, first + min(n, r + 2048))
                    q = s["q"][at, h * G + g].double()
                    x = (q @ both["k"].T) / math.sqrt(D)
                    x = x.masked_fill(mask[r:r + 2048], -math.inf)
                    out[at, h * G + g] = torch.nan_to_num(torch.softmax(x, -1)) @ both["v"]
        first += n
    return out


def _exact_append(case, s, news, lens):
    rot, half = case["rot"], case["rot"] // 2
    k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
    pos = torch.cat([torch.arange(m - n, m) for n, m in zip(news, lens)]).cuda()
    seq = torch.cat([torch.full((n,), b) for b, n in enumerate(news)]).cuda()
    turn = pos.double()[:, None, None] * torch.tensor([case["base"] ** (-2.0 * i / rot) for i in range(half)],
                                                      dtype=torch.float64, device="cuda")
    unit = torch.polar(torch.ones_like(turn), turn)

    def rotated(x):
        x = x.double()
        z = x[..., :rot]
        z = z.unflatten(-1, (half, 2)) if case["inter"] else z.unflatten(-1, (2, half)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * unit)
        z = z if case["inter"] else z.transpose(-1, -2)
        return torch.cat((z.flatten(-2), x[..., rot:]), -1)

    at = s["table"].long()[seq, pos // case["page"]]
    k_cache[at, :, pos % case["page"]] = rotated(s["k"])
    v_cache[at, :, pos % case["page"]] = s["v"].double()
    return {"q": rotated(s["q"]), "k_cache": k_cache, "v_cache": v_cache}
