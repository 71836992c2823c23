"""The operators of a quantised decoder step: what is measured, and their plain forms.

Three operators beside the paged attention and the routed experts, for a layer whose cache is held in
8 bits and whose projections are held in 4:

  append  new keys and values go into the paged cache as 8-bit codes with a scale for each token and
          key head, keys (and queries) rotated on the way
  window  causal attention over such a cache: the last `window` keys and the first `sinks` ones
  linear  y = W x for few tokens, W in 4-bit codes with a scale for each group of a row

Codes are int8 (value = code * scale, scale = max|x| / 127) or e4m3 (scale = max|x| / 448); a row's
4-bit codes are two's complement, the even column in the low half of a byte.  A batch is ragged:
sequence b has the query tokens q_start[b] .. q_start[b+1]-1, which are the last of its kv_len[b] cached
tokens, and its token j sits in slot j % page of page table[b, j // page].  With `own` false, run()
computes them in elementary torch operations in 32 bits (rotation and quantisation in 64, for far
positions and values next to a border); with `own` true it makes the calls a user makes.  48 query heads
of 128 are the width 6144 of the expert layers here; the other sizes are generic.
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
CODE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
TOP = {"int8": 127.0, "e4m3": 448.0}

# one new token for each of 16 running sequences: a decode step's append, where latency counts
A1 = dict(name="append_decode_16", op="append", dtype="bf16", code="e4m3", n_q=48, n_kv=8, dim=128, page=64,
          seqs=16, new=1, mix=0, ctx=8192, ragged=1, rot=128, inter=0, base=10000.0)
# ragged prompt chunks of a model without rotation in its attention, an odd head group, small pages
A2 = dict(name="append_ragged_chunks", op="append", dtype="fp16", code="int8", n_q=28, n_kv=4, dim=128, page=16,
          seqs=7, new=331, mix=0, ctx=2600, ragged=2, rot=0, inter=0, base=10000.0)
# a long prompt in one call
A3 = dict(name="append_prompt_16k", op="append", dtype="bf16", code="e4m3", n_q=48, n_kv=8, dim=128, page=64,
          seqs=1, new=16384, mix=0, ctx=16384, ragged=3, rot=128, inter=0, base=1000000.0)
# one user, one token, a short context: the smallest call
W1 = dict(name="window_decode_1", op="window", dtype="bf16", code="int8", n_q=48, n_kv=8, dim=128, page=64,
          seqs=1, new=1, mix=0, ctx=700, ragged=4, window=512, sinks=4)
# a decode step of 64 users with long contexts, of which the window keeps 4096 keys
W2 = dict(name="window_decode_64", op="window", dtype="bf16", code="int8", n_q=48, n_kv=8, dim=128, page=64,
          seqs=64, new=1, mix=0, ctx=16384, ragged=5, window=4096, sinks=4)
# speculative verification of 5 tokens for each of 13 users; odd window, odd head group, small heads
W3 = dict(name="window_verify_13", op="window", dtype="fp16", code="e4m3", n_q=40, n_kv=8, dim=64, page=16,
          seqs=13, new=5, mix=0, ctx=2999, ragged=6, window=1001, sinks=7)
# continuous batching: some users' prompt chunks beside the others' single tokens
W4 = dict(name="window_mixed_16", op="window", dtype="bf16", code="e4m3", n_q=48, n_kv=8, dim=128, page=32,
          seqs=16, new=500, mix=1, ctx=4096, ragged=7, window=2048, sinks=16)
# a whole prompt, the window half as long: the largest
W5 = dict(name="window_prompt_8k", op="window", dtype="bf16", code="int8", n_q=48, n_kv=8, dim=128, page=64,
          seqs=1, new=8192, mix=0, ctx=8192, ragged=8, window=4096, sinks=4)
# the fused query, key and value projection of one token, where latency counts
L1 = dict(name="linear_qkv_1", op="linear", dtype="bf16", tokens=1, rows=8192, cols=6144, group=128, ragged=9)
# the output projection when 5 tokens of a user are verified
L2 = dict(name="linear_out_5", op="linear", dtype="fp16", tokens=5, rows=6144, cols=6144, group=64, ragged=10)
# a small odd layer: the narrowest groups, rows and columns that no tile divides
L3 = dict(name="linear_odd_13", op="linear", dtype="fp16", tokens=13, rows=1111, cols=1184, group=32, ragged=11)
# the logits of 16 users over a large vocabulary: the largest weights
L4 = dict(name="linear_head_16", op="linear", dtype="bf16", tokens=16, rows=100000, cols=6144, group=128, ragged=12)


def listed():
    return [dict(c) for c in (A1, A2, A3, W1, W2, W3, W4, W5, L1, L2, L3, L4)]


HEADS = [(48, 8, 128), (32, 8, 128), (28, 4, 128), (40, 8, 64), (14, 14, 64), (15, 5, 64), (8, 1, 128),
         (20, 4, 128), (64, 8, 64), (12, 12, 128)]


def _log(rng, lo, hi):
    """a whole number of lo .. hi, spread over its logarithm"""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op, dtype, ragged = rng.choice(["append", "window", "linear"]), rng.choice(["bf16", "fp16"]), rng.randrange(1 << 20)
    if op == "linear":
        group = rng.choice([32, 64, 128])
        cols = group * max(1, _log(rng, 256, 16384) // group)
        tokens = _log(rng, 1, 64)
        rows = _log(rng, 32, min(60000, L4["rows"] * L4["cols"] * L4["tokens"] // (cols * max(16, tokens))))
        return dict(op=op, dtype=dtype, tokens=tokens, rows=rows, cols=cols, group=group, ragged=ragged)
    n_q, n_kv, dim = rng.choice(HEADS)
    code = rng.choice(["int8", "e4m3"])
    case = dict(op=op, dtype=dtype, code=code, n_q=n_q, n_kv=n_kv, dim=dim, page=rng.choice([16, 32, 64, 128]),
                mix=0, ragged=ragged)
    if op == "append":  # int8 codes are whole numbers, which a rotated key that lies on a border may round either way
        seqs = _log(rng, 1, 64)
        new = rng.choice([1, _log(rng, 2, max(2, 8192 // seqs))])
        case.update(seqs=seqs, new=new, ctx=max(new, _log(rng, 64, 8192)),
                    rot=0 if code == "int8" else rng.choice([dim, dim // 2]), inter=rng.randrange(2),
                    base=rng.choice([10000.0, 500000.0]))
        return case
    kind = rng.choice(["decode", "verify", "mixed", "prompt", "long"])
    window = rng.choice([-1, _log(rng, 1, 4096), _log(rng, 64, 4096)])
    sinks = rng.choice([0, 4, _log(rng, 1, 200)])
    if kind == "prompt":
        n = _log(rng, 33, 4096)
        case.update(seqs=1, new=n, ctx=n + rng.choice([0, _log(rng, 1, 2048)]))
    elif kind == "mixed":
        case.update(seqs=_log(rng, 2, 16), new=_log(rng, 20, 400), ctx=_log(rng, 500, 4096), mix=1)
    elif kind == "long":
        case.update(seqs=rng.randint(1, 2), new=rng.choice([1, 1, 4]), ctx=_log(rng, 16384, 131072))
    else:
        new = 1 if kind == "decode" else rng.randint(2, 8)
        case.update(seqs=_log(rng, 1, 64), new=new, ctx=_log(rng, 64, 4096 if window < 0 else 12000))
    case.update(window=window, sinks=sinks)
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
    """(query, key) pairs that see each other, and keys some query sees, of one sequence"""
    w, s = case["window"], case["sinks"]
    pairs = 0
    for p in range(length - n, length):
        lo = 0 if w < 0 else max(0, p - w + 1)
        pairs += p + 1 - lo + min(s, lo)
    lo = 0 if w < 0 else max(0, length - n - w + 1)
    return pairs, length - lo + min(s, lo)


def work(case):
    if case["op"] == "linear":  # codes, group scales, x and y, once each
        t, n, k = case["tokens"], case["rows"], case["cols"]
        return {"bytes": n * k // 2 + 2 * n * (k // case["group"]) + 2 * t * (k + n), "flops": 2 * t * n * k}
    news, lens = _lens(case)
    T, row = sum(news), 2 * case["dim"]
    held = 2 * case["n_kv"] * (case["dim"] + 4)  # a token's codes and scales
    if case["op"] == "append":  # q, k and v read (no queries without a rotation); rotated q, codes and scales written
        q = case["n_q"] if case["rot"] else 0
        return {"bytes": T * ((2 * q + 2 * case["n_kv"]) * row + held),
                "flops": T * (3 * (q + case["n_kv"]) * case["rot"] + 4 * case["n_kv"] * case["dim"])}
    seen = [_visible(case, n, m) for n, m in zip(news, lens)]
    pairs, keys = sum(p for p, _ in seen), sum(k for _, k in seen)
    return {"bytes": 2 * T * case["n_q"] * row + keys * held, "flops": 4 * pairs * case["n_q"] * case["dim"]}


def _codes(x, kind):
    """x [..., dim] in 32 bits -> codes and scales, a scale for each row; as an earlier call has left them"""
    top = x.abs().amax(-1, keepdim=True)
    y = x * (TOP[kind] / top)
    return (y.round().to(torch.int8) if kind == "int8" else y.to(torch.float8_e4m3fn)), (top / TOP[kind]).squeeze(-1)


def _make(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DT[case["dtype"]]
    normal = lambda *shape: torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)  # noqa: E731
    s = dict(case=dict(case))
    if case["op"] == "linear":
        n, k, group = case["rows"], case["cols"], case["group"]
        s["packed"] = torch.empty((n, k // 2), dtype=torch.uint8, device="cuda")
        s["scales"] = torch.empty((n, k // group), dtype=dt, device="cuda")
        step = max(1, (1 << 26) // k)
        for r in range(0, n, step):
            w = normal(min(step, n - r), k // group, group) * k ** -0.5
            d = (w.abs().amax(-1) / 7).to(dt)
            c = (w / d.to(torch.float32)[..., None]).round().clamp(-7, 7).to(torch.int32).view(-1, k // 2, 2)
            s["packed"][r:r + step] = ((c[..., 0] & 15) | ((c[..., 1] & 15) << 4)).to(torch.uint8)
            s["scales"][r:r + step] = d
        s["x"] = normal(case["tokens"], k).to(dt)
        return s
    news, lens = _lens(case)
    page, D, kind = case["page"], case["dim"], case["code"]
    T = sum(news)
    need = [-(-m // page) for m in lens]
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, generator=g, device="cuda", dtype=torch.int64).to(torch.int32)
    table = torch.zeros((case["seqs"], max(need)), dtype=torch.int32)
    at = 0
    rows = torch.arange(n_pages, dtype=torch.int32)
    for b, n in enumerate(need):
        table[b, :n] = rows[at:at + n]
        at += n
    s.update(T=T, max_q=max(news),
             q_start=torch.tensor([sum(news[:b]) for b in range(len(news) + 1)], dtype=torch.int32, device="cuda"),
             kv_len=torch.tensor(lens, dtype=torch.int32, device="cuda"),
             table=order[table.to("cuda").long()].contiguous())
    for name in ("k", "v"):  # tokens differ in size
        s[name + "_cache"] = torch.empty((n_pages, case["n_kv"], page, D), dtype=CODE[kind], device="cuda")
        s[name + "_scale"] = torch.empty((n_pages, case["n_kv"], page), dtype=torch.float32, device="cuda")
        step = max(1, (1 << 26) // (case["n_kv"] * page * D))
        for r in range(0, n_pages, step):
            x = normal(min(step, n_pages - r), case["n_kv"], page, D)
            c, d = _codes(x * torch.exp(0.3 * normal(*x.shape[:-1], 1)), kind)
            s[name + "_cache"][r:r + step], s[name + "_scale"][r:r + step] = c, d
    if case["op"] == "append":  # slices of the fused projection's rows, as a layer has them
        qkv = normal(T, (case["n_q"] + 2 * case["n_kv"]) * D).to(dt)
        a, b = case["n_q"] * D, (case["n_q"] + case["n_kv"]) * D
        s["q"] = qkv[:, :a].view(T, case["n_q"], D) if case["rot"] else None
        s["k"] = qkv[:, a:b].view(T, case["n_kv"], D)
        s["v"] = qkv[:, b:].view(T, case["n_kv"], D)
    else:
        s["q"] = normal(T, case["n_q"], D).to(dt)
    return s


def prepare(case, seed):
    s = _make(case, seed)
    if own:  # the handles a serving program makes once, next to its weights, its cache and its batch
        if case["op"] == "linear":
            from int4_routed_expert_quantize_gb300 import linear
            s["linear"] = linear.Int4Linear(s["packed"], s["scales"], max_tokens=case["tokens"])
            return s
        from int4_routed_expert_quantize_gb300 import attn
        s["attn"] = attn.PagedAttention(case["n_q"], case["n_kv"], case["dim"], case["page"], max_tokens=s["T"],
                                        max_seqs=case["seqs"], dtype=DT[case["dtype"]],
                                        rot_dim=case.get("rot", 0), interleaved=bool(case.get("inter", 0)),
                                        rope_base=case.get("base", 10000.0))
        s["cache"] = s["attn"].bind_cache(s["k_cache"], s["v_cache"], k_scale=s["k_scale"], v_scale=s["v_scale"])
        s["batch"] = attn.Batch(s["q_start"], s["kv_len"], s["table"], n_tokens=s["T"], max_q=s["max_q"])
    return s


def run(s):
    c = s["case"]
    if own:
        if c["op"] == "linear":
            return s["linear"].forward(s["x"])
        if c["op"] == "append":
            q = s["attn"].append(s["cache"], s["batch"], s["k"], s["v"], s["q"])
            return _held(s, q)
        return s["attn"].window(s["cache"], s["batch"], s["q"], window=c["window"], sinks=c["sinks"])
    if c["op"] == "linear":
        return _plain_linear(s)
    return _plain_append(s) if c["op"] == "append" else _plain_window(s)


def _held(s, q):
    """an append's outputs: the rotated queries, and the cache as it is held"""
    out = {"k_codes": s["k_cache"], "v_codes": s["v_cache"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    return out if q is None else {"q": q, **out}


# ---- the plain forms ----

def _plain_linear(s):
    c = s["case"]
    b = s["packed"].to(torch.int32)
    codes = torch.stack((b & 15, b >> 4), -1)
    codes = torch.where(codes > 7, codes - 16, codes).to(torch.float32)
    w = codes.view(c["rows"], -1, c["group"]) * s["scales"].to(torch.float32)[..., None]
    return (s["x"].to(torch.float32) @ w.view(c["rows"], c["cols"]).T).to(s["x"].dtype)


def _where_is(s):
    """each token's sequence, its index among the sequence's new tokens, and its position"""
    t = torch.arange(s["T"], device="cuda")
    start = s["q_start"].long()
    b = torch.searchsorted(start, t, right=True) - 1
    i = t - start[b]
    return b, i, s["kv_len"].long()[b] - (start[b + 1] - start[b]) + i


def _rotate(x, pos, c):
    """x [T, heads, dim] in 64 bits: the first `rot` values of a head rotated in pairs by pos * base^(-2i/rot)"""
    rot = c["rot"]
    x = x.to(torch.float64)
    if rot == 0:
        return x
    f = c["base"] ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    a = pos.to(torch.float64)[:, None] * f
    cos, sin = torch.cos(a)[:, None], torch.sin(a)[:, None]
    r = x[..., :rot]
    u, v = (r[..., 0::2], r[..., 1::2]) if c["inter"] else (r[..., :rot // 2], r[..., rot // 2:])
    p, q = u * cos - v * sin, v * cos + u * sin
    y = torch.stack((p, q), -1).flatten(-2) if c["inter"] else torch.cat((p, q), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _quantised(x, kind):
    """[..., dim] in 64 bits -> codes and scales: code = TOP x / max|x| rounded to the nearest, ties to even"""
    top = x.abs().amax(-1, keepdim=True)
    y = TOP[kind] * x / torch.where(top == 0, 1.0, top)
    return (torch.round(y).to(torch.int8) if kind == "int8" else y.to(torch.float32).to(torch.float8_e4m3fn),
            (top / TOP[kind]).to(torch.float32).squeeze(-1))


def _plain_append(s):
    c = s["case"]
    b, _, pos = _where_is(s)
    page = s["table"].long()[b, pos // c["page"]]
    slot = pos % c["page"]
    for name, x in (("k", _rotate(s["k"], pos, c)), ("v", s["v"].to(torch.float64))):
        codes, scale = _quantised(x, c["code"])
        s[name + "_cache"].view(torch.uint8)[page, :, slot] = codes.view(torch.uint8)
        s[name + "_scale"][page, :, slot] = scale
    return _held(s, None if s["q"] is None else _rotate(s["q"], pos, c).to(s["q"].dtype))


def _values(codes, scale, table):
    """a page table's [..., pages] keys or values in order: [..., n_kv, pages * page, dim] in 32 bits"""
    t = table.long()
    x = codes.view(torch.uint8)[t].view(codes.dtype).to(torch.float32) * scale[t][..., None]
    return x.transpose(-4, -3).flatten(-3, -2)


def _plain_window(s):
    c = s["case"]
    at = (s["q_start"].long()[:-1, None] + torch.arange(s["max_q"], device="cuda")).clamp(max=s["T"] - 1)
    q = s["q"].to(torch.float32)[at] * (1.0 / math.sqrt(c["dim"]))
    q = q.view(c["seqs"], s["max_q"], c["n_kv"], c["n_q"] // c["n_kv"], c["dim"])
    q = q.permute(0, 2, 1, 3, 4).reshape(c["seqs"], c["n_kv"], -1, c["dim"])
    k = _values(s["k_cache"], s["k_scale"], s["table"])
    x = (q @ k.transpose(-1, -2)).view(c["seqs"], c["n_kv"], s["max_q"], -1, k.shape[-2])
    new = (s["q_start"][1:] - s["q_start"][:-1]).long()
    pos = (s["kv_len"].long() - new)[:, None] + torch.arange(s["max_q"], device="cuda")
    j = torch.arange(k.shape[-2], device="cuda")
    seen = j <= pos[..., None]
    if c["window"] >= 0:
        seen = seen & ((pos[..., None] - j < c["window"]) | (j < c["sinks"]))
    x = torch.where(seen[:, None, :, None], x, -math.inf).flatten(2, 3)
    top = x.amax(-1, keepdim=True)
    x = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    total = x.sum(-1, keepdim=True)
    o = (x @ _values(s["v_cache"], s["v_scale"], s["table"])) / torch.where(total == 0, 1.0, total)
    b, i, _ = _where_is(s)  # [seqs, n_kv, max_q * group, dim] back to [T, n_q, dim]
    o = o.view(c["seqs"], c["n_kv"], s["max_q"], -1, c["dim"])[b, :, i]
    return o.reshape(s["T"], c["n_q"], c["dim"]).to(s["q"].dtype)


# ---- the definitions in 64 bits ----

def exact(case, seed):
    s = _make(case, seed)
    return {"linear": _exact_linear, "append": _exact_append, "window": _exact_window}[case["op"]](case, s)


def _exact_linear(case, s):
    """a block of rows after the other"""
    x, out = s["x"].double(), []
    for r in range(0, case["rows"], 4096):
        p = s["packed"][r:r + 4096].long()
        nib = torch.stack((p % 16, p // 16), 2).flatten(1)
        w = ((nib + 8) % 16 - 8).double() * s["scales"][r:r + 4096].double().repeat_interleave(case["group"], 1)
        out.append(torch.einsum("tk,rk->tr", x, w))
    return torch.cat(out, 1)


def _exact_append(case, s):
    news, lens = _lens(case)
    rot, half = case["rot"], case["rot"] // 2
    pos = torch.cat([torch.arange(m - n, m) for n, m in zip(news, lens)]).cuda()
    seq = torch.cat([torch.full((n,), b) for b, n in enumerate(news)]).cuda()

    def rotated(x):
        x = x.double()
        if not rot:
            return x
        turn = pos.double()[:, None, None] * torch.tensor([case["base"] ** (-2.0 * i / rot) for i in range(half)],
                                                          dtype=torch.float64, device="cuda")
        z = x[..., :rot]
        z = z.unflatten(-1, (half, 2)) if case["inter"] else z.unflatten(-1, (2, half)).transpose(-1, -2)
        z = torch.view_as_complex(z.contiguous()) * torch.polar(torch.ones_like(turn), turn)
        z = torch.view_as_real(z)
        z = z if case["inter"] else z.transpose(-1, -2)
        return torch.cat((z.flatten(-2), x[..., rot:]), -1)

    at, slot, kind = s["table"].long()[seq, pos // case["page"]], pos % case["page"], case["code"]
    out = {} if s["q"] is None else {"q": rotated(s["q"])}
    held = {}
    for name, x in (("k", rotated(s["k"])), ("v", s["v"].double())):
        codes, scale = s[name + "_cache"], s[name + "_scale"].double()
        limit = torch.linalg.vector_norm(x, ord=math.inf, dim=-1)
        scale[at, :, slot] = limit / TOP[kind]
        y = (x * TOP[kind] / limit[..., None]).nan_to_num(0.0)
        if kind == "int8":  # whole numbers: they have to be equal
            codes = codes.clone()
            codes[at, :, slot] = torch.special.round(y).to(torch.int8)
        else:  # e4m3 from its definition: 4 significant bits down to 2^-6, steps of 2^-9 below
            codes = codes.to(torch.float32).double()
            step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
            codes[at, :, slot] = torch.round(y / step) * step
        held[name] = codes, scale
    return {**out, "k_codes": held["k"][0], "v_codes": held["v"][0], "k_scale": held["k"][1], "v_scale": held["v"][1]}


def _exact_window(case, s):
    """one sequence and one key head after the other"""
    news, lens = _lens(case)
    G, page, D = case["n_q"] // case["n_kv"], case["page"], case["dim"]
    out = torch.zeros((s["T"], case["n_q"], D), dtype=torch.float64, device="cuda")
    first = 0
    for b, (n, m) in enumerate(zip(news, lens)):
        pages = s["table"][b, : -(-m // page)].long()
        j = torch.arange(m, device="cuda")[None, :]
        for h in range(case["n_kv"]):
            both = {}
            for name in ("k", "v"):
                codes = s[name + "_cache"][:, h].view(torch.uint8)[pages].view(s[name + "_cache"].dtype)
                x = codes.to(torch.float32).double() * s[name + "_scale"][:, h][pages].double()[..., None]
                both[name] = x.reshape(-1, D)[:m]
            for r in range(0, n, 2048):
                e = min(n, r + 2048)
                p = torch.arange(m - n + r, m - n + e, device="cuda")[:, None]
                hidden = j > p
                if case["window"] >= 0:
                    hidden = hidden | ((j <= p - case["window"]) & (j >= case["sinks"]))
                for g in range(G):
                    x = (s["q"][first + r:first + e, h * G + g].double() @ both["k"].T) / math.sqrt(D)
                    x = torch.softmax(x.masked_fill(hidden, -math.inf), -1)
                    out[first + r:first + e, h * G + g] = torch.nan_to_num(x) @ both["v"]
        first += n
    return out
