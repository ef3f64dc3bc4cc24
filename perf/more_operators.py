"""Workloads of further language-model operators, each in a plain torch form and through the library.

head       log probabilities of given tokens from the last hidden rows and the head's weights, without the logits
head_grad  the gradient of those with respect to the hidden rows and the weights
append     keys and values put into a paged cache, queries and keys normed per head and rotated on the way
norm       queries and keys of a training step normed and rotated, and the gradients of that
prefix     attention of one new token per sequence, groups of sequences sharing a long prefix in the cache

With ``own`` false :func:`run` computes the plain form (32 bits throughout, rounded once at the
end); with ``own`` true it makes the library's calls on the same inputs.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
EPS = 1e-6
HEAD_WORK = 4096 * 128000 * 4096        # multiply-adds of the largest head cases' logits
TOKEN_ELEMENTS = 8191 * 80 * 96         # of the largest append case
NORM_ELEMENTS = 16384 * 40 * 128        # of the largest norm case
PREFIX_WORK = 128 * 32 * 128 * 65536    # multiply-adds of the largest prefix case's scores


def listed():
    return [
        # greedy decoding of four sequences of a small model: latency is all there is
        {"name": "head_step", "op": "head", "rows": 4, "vocab": 4099, "hidden": 512, "ranks": 2, "dtype": "bf16",
         "temperature": 1.0, "padded": False},
        # one step of a rollout batch on eight ranks: the weights are read once
        {"name": "head_rollout", "op": "head", "rows": 128, "vocab": 131072, "hidden": 4096, "ranks": 8, "dtype": "bf16",
         "temperature": 0.7, "padded": False},
        # log probabilities of a training batch, as a policy-gradient step takes them
        {"name": "head_train", "op": "head", "rows": 4096, "vocab": 128000, "hidden": 4096, "ranks": 1, "dtype": "bf16",
         "temperature": 1.0, "padded": False},
        # the gradient for a short batch in half precision, an odd vocabulary in uneven shards, an odd hidden size
        {"name": "head_grad_odd", "op": "head_grad", "rows": 509, "vocab": 50021, "hidden": 1000, "ranks": 3, "dtype": "f16",
         "temperature": 0.8, "padded": False},
        # the gradient of a training batch, eight ranks with padded shards
        {"name": "head_grad_train", "op": "head_grad", "rows": 4096, "vocab": 127900, "hidden": 4096, "ranks": 8,
         "dtype": "bf16", "temperature": 1.0, "padded": True},
        # the new tokens of 64 sequences in a decoding step
        {"name": "append_step", "op": "append", "seqs": 64, "tokens": 64, "q_heads": 32, "kv_heads": 8, "dim": 128,
         "rotary": 128, "interleaved": False, "page": 64, "dtype": "bf16", "length": 4000},
        # five prompts, heads of 80 of which 32 are rotated in neighbouring pairs
        {"name": "append_prompt", "op": "append", "seqs": 5, "tokens": 8191, "q_heads": 32, "kv_heads": 32, "dim": 80,
         "rotary": 32, "interleaved": True, "page": 16, "dtype": "f16", "length": 2000},
        # a short odd training batch in 32 bits, heads of 64
        {"name": "norm_odd", "op": "norm", "tokens": 517, "q_heads": 12, "kv_heads": 12, "dim": 64, "rotary": 64,
         "interleaved": True, "dtype": "f32", "length": 2048},
        # a training batch of shared key heads
        {"name": "norm_train", "op": "norm", "tokens": 16384, "q_heads": 32, "kv_heads": 8, "dim": 128, "rotary": 128,
         "interleaved": False, "dtype": "bf16", "length": 4096},
        # eight samples of a short odd prompt on one rank of eight
        {"name": "prefix_small", "op": "prefix", "prefixes": 1, "each": 8, "prefix": 1025, "own": 130, "q_heads": 8, "kv_heads": 1,
         "dim": 128, "page": 16, "dtype": "bf16"},
        # four prompts with samples of their own each, heads of 64, pages of an odd size
        {"name": "prefix_groups", "op": "prefix", "prefixes": 4, "each": 16, "prefix": 7001, "own": 500, "q_heads": 12,
         "kv_heads": 12, "dim": 64, "page": 24, "dtype": "f16"},
        # a serving batch behind one long document
        {"name": "prefix_long", "op": "prefix", "prefixes": 1, "each": 128, "prefix": 65536, "own": 1024, "q_heads": 32,
         "kv_heads": 8, "dim": 128, "page": 64, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["head", "head_grad", "append", "norm", "prefix"])
    if op in ("head", "head_grad"):
        vocab, hidden = _log(rng, 1000, 200000), 8 * _log(rng, 32, 1024)
        return {"op": op, "rows": _log(rng, 1, max(1, min(4096, HEAD_WORK // (vocab * hidden)))), "vocab": vocab,
                "hidden": hidden, "ranks": rng.choice([1, 1, 2, 3, 4, 8]), "dtype": rng.choice(["bf16", "bf16", "f16"]),
                "temperature": rng.choice([1.0, 1.0, 0.7, 1.3]), "padded": rng.random() < 0.3}
    kv_heads = rng.choice([1, 2, 4, 8, 12])
    c = {"op": op, "kv_heads": kv_heads, "q_heads": kv_heads * rng.choice([1, 2, 3, 4, 8, 16]),
         "dim": rng.choice([64, 96, 128, 128, 192, 256]), "dtype": rng.choice(["bf16", "bf16", "f16"])}
    if op == "prefix":
        c |= {"page": rng.choice([1, 16, 24, 64, 128]), "prefixes": rng.choice([1, 1, 1, 2, 4, 5]), "each": _log(rng, 1, 128),
              "own": _log(rng, 1, 2000)}
        c["each"] = max(1, min(c["each"], 160 // c["prefixes"]))
        per = c["prefixes"] * c["each"] * c["q_heads"] * c["dim"]
        cached = c["prefixes"] * kv_heads * c["dim"]
        c["prefix"] = _log(rng, 1, max(1, min(131072, PREFIX_WORK // per - c["own"], 65536 * 8 * 128 // cached)))
        return c
    c |= {"rotary": rng.choice([c["dim"], c["dim"], 32]), "interleaved": rng.random() < 0.5}
    if op == "norm":
        c["dtype"] = rng.choice(["bf16", "bf16", "f16", "f32"])
        per = c["dim"] * (c["q_heads"] + kv_heads) * BYTES[c["dtype"]] // 2
        c |= {"tokens": _log(rng, 1, min(16384, NORM_ELEMENTS // per)), "length": 4096}
        return c
    c["page"] = rng.choice([1, 16, 24, 64, 128])
    if rng.random() < 0.5:
        seqs = _log(rng, 1, 256)
        tokens = seqs
    else:
        seqs = rng.randint(1, 8)
        tokens = _log(rng, max(8, seqs), 8192)
    held = max(1, (1 << 27) // (seqs * kv_heads * c["dim"]))
    per = c["dim"] * (c["q_heads"] + 2 * kv_heads)
    c |= {"seqs": seqs, "tokens": max(seqs, min(tokens, TOKEN_ELEMENTS // per)), "length": _log(rng, 1, min(8000, held))}
    return c


def _widths(case):
    """Columns of the vocabulary that each rank holds, padding included."""
    v, p = case["vocab"], case["ranks"]
    if case["padded"]:
        return [(-(-v // p) + 63) // 64 * 64] * p
    return [v // p + (1 if r < v % p else 0) for r in range(p)]


def _new_tokens(case):
    """(sequence, position) of every appended token."""
    n, tokens = case["seqs"], case["tokens"]
    rng = random.Random(n * 1000003 + tokens)
    had = [rng.randint(0, case["length"]) for _ in range(n)]
    new = [tokens // n + (1 if b < tokens % n else 0) for b in range(n)]
    if tokens > n:  # prompts of uneven lengths
        for b in range(0, n - 1, 2):
            moved = rng.randint(0, new[b] // 2)
            new[b] -= moved
            new[b + 1] += moved
    return [(b, had[b] + i) for b in range(n) for i in range(new[b])]


def _prefix_lengths(case):
    """Cached tokens of every prefix and of every sequence behind it: the same for every seed."""
    p, n = case["prefixes"], case["prefixes"] * case["each"]
    rng = random.Random(case["prefix"] * 1000003 + n)
    prefix = [case["prefix"]] + [rng.randint(1, case["prefix"]) for _ in range(p - 1)]
    own_tokens = [case["own"]] + [rng.randint(0, case["own"]) for _ in range(n - 1)]
    if n >= 8:
        own_tokens[3], own_tokens[5] = 0, 1
    return prefix, own_tokens


def _tables(lengths, page, spare, gen, dev):
    """Page numbers of every row of tokens, -1 past its end, from one shuffled pool; and the number of pages."""
    need = [-(-n // page) for n in lengths]
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=gen, device=dev, dtype=torch.int64).to(torch.int32)
    width = max(1, max(need))
    first = torch.tensor([sum(need[:b]) for b in range(len(need))], device=dev)
    col = torch.arange(width, device=dev)
    at = (first[:, None] + col[None]).clamp(max=pages - 1)
    held = col[None] < torch.tensor(need, device=dev)[:, None]
    return torch.where(held, order[at], -1).contiguous(), pages


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32).to(dt)

    s = {"case": case}
    if case["op"] in ("head", "head_grad"):
        n, v, h = case["rows"], case["vocab"], case["hidden"]
        # a head whose logits are a few units wide, and rows that point to one token more than to the others
        weights = [torch.randn(w, h, generator=gen, device=dev).mul_(2.5 * h ** -0.5).to(dt) for w in _widths(case)]
        whole = torch.cat(weights, 0)[:v]
        tokens = torch.randint(0, v, (n,), generator=gen, device=dev)
        ahead = torch.rand(n, 1, generator=gen, device=dev) * 2
        x = torch.randn(n, h, generator=gen, device=dev) + ahead * whole[tokens].float()
        other = torch.randint(0, v, (n,), generator=gen, device=dev)
        tokens = torch.where(torch.rand(n, generator=gen, device=dev) < 0.7, tokens, other)
        s |= {"hidden": x.to(dt), "weights": weights, "tokens": tokens}
        f32 = {"device": dev, "dtype": torch.float32}
        if case["op"] == "head":
            s |= {"logprobs": torch.empty(n, **f32), "entropy": torch.empty(n, **f32), "lse": torch.empty(n, **f32)}
        else:
            lse, ent = [], []
            wf = whole.float()
            for at in range(0, n, 1024):
                z = torch.matmul(s["hidden"][at:at + 1024].float(), wf.t()) * (1.0 / case["temperature"])
                lse.append(torch.logsumexp(z, 1))
                z = z - lse[-1][:, None]
                ent.append(-(z.exp() * z).sum(1))
            s |= {"lse": torch.cat(lse), "entropy": torch.cat(ent)}
            s["grad_logprobs"] = torch.randn(n, generator=gen, **f32)
            s["grad_entropy"] = torch.randn(n, generator=gen, **f32) * 0.1
            # a fifth of the tokens belong to the prompt and carry no log probability
            s["tokens"] = torch.where(torch.rand(n, generator=gen, device=dev) < 0.2, -100, s["tokens"])
            s["grad_hidden"] = torch.empty_like(s["hidden"])
            s["grad_weights"] = [torch.empty_like(w) for w in weights]
        if own:  # the library's workspace, kept by the caller from call to call
            import reduce_copy_rank_gb300 as dc

            s["workspace"] = dc.linear_logprobs_workspace(n, h, sum(_widths(case)), backward=case["op"] == "head_grad")
        return s
    hq, hk, d = case["q_heads"], case["kv_heads"], case["dim"]
    if case["op"] in ("append", "norm"):
        rot = case["rotary"]
        if case["op"] == "append":
            where = _new_tokens(case)
            places = 1 + max(p for _, p in where)
            s["positions"] = torch.tensor([p for _, p in where], device=dev, dtype=torch.int32)
        else:  # packed sequences of a training batch
            where = range(case["tokens"])
            places = min(case["length"], case["tokens"])
            s["positions"] = (torch.arange(case["tokens"], device=dev) % case["length"]).to(torch.int32)
        t = len(where)
        both = normal(t, hq + 2 * hk, d) * 3  # the projection's output: queries, keys and values side by side
        angle = torch.arange(places, device=dev, dtype=torch.float64)[:, None] * \
            (10000.0 ** (-torch.arange(0, rot, 2, device=dev, dtype=torch.float64) / rot))[None]
        # norm weights as training leaves them: near one, in 32 bits while it trains
        weights = [1 + 0.3 * torch.randn(d, generator=gen, device=dev) for _ in range(2)]
        s |= {"q": both[:, :hq], "k": both[:, hq:hq + hk], "v": both[:, hq + hk:],
              "cos_sin": torch.cat([angle.cos(), angle.sin()], 1).to(torch.float32),
              "q_out": torch.empty(t, hq, d, device=dev, dtype=dt)}
        if case["op"] == "append":
            held = [max((p + 1 for b, p in where if b == i), default=0) for i in range(case["seqs"])]
            s["table"], pages = _tables(held, case["page"], 3, gen, dev)
            s |= {"q_norm": weights[0].to(dt), "k_norm": weights[1].to(dt),
                  "seqs": torch.tensor([b for b, _ in where], device=dev, dtype=torch.int32),
                  "k_cache": normal(pages, case["page"], hk, d), "v_cache": normal(pages, case["page"], hk, d)}
            return s
        s |= {"q_norm": weights[0], "k_norm": weights[1], "k_out": torch.empty(t, hk, d, device=dev, dtype=dt),
              "grad_q_out": normal(t, hq, d), "grad_k_out": normal(t, hk, d),
              "grad_q": torch.empty(t, hq, d, device=dev, dtype=dt), "grad_k": torch.empty(t, hk, d, device=dev, dtype=dt),
              "grad_q_norm": torch.empty(d, device=dev), "grad_k_norm": torch.empty(d, device=dev)}
        if own:
            import reduce_copy_rank_gb300 as dc

            s["workspace"] = dc.qk_norm_workspace(t, hq, hk, d)
        return s
    prefix, own_tokens = _prefix_lengths(case)
    n, page = len(own_tokens), case["page"]
    table, pages = _tables(prefix + own_tokens, page, 1, gen, dev)
    rows = [max(1, max(-(-x // page) for x in part)) for part in (prefix, own_tokens)]
    s |= {"q": normal(n, hq, d), "k_cache": normal(pages, page, hk, d), "v_cache": normal(pages, page, hk, d),
          "prefix_table": table[:len(prefix), :rows[0]].contiguous(), "table": table[len(prefix):, :rows[1]].contiguous(),
          "prefix_lengths": torch.tensor(prefix, device=dev, dtype=torch.int32),
          "lengths": torch.tensor(own_tokens, device=dev, dtype=torch.int32),
          "out": torch.empty(n, hq, d, device=dev, dtype=dt), "lse": torch.empty(n, hq, device=dev, dtype=torch.float32)}
    if own:
        import reduce_copy_rank_gb300 as dc

        s["workspace"] = dc.prefix_attention_workspace(n, len(prefix), hq, hk, d, rows[0] * page, rows[1] * page)
    return s


def run(state):
    op = state["case"]["op"]
    if own:
        return {"head": _own_head, "head_grad": _own_head_grad, "append": _own_append, "norm": _own_norm,
                "prefix": _own_prefix}[op](state)
    return {"head": _plain_head, "head_grad": _plain_head_grad, "append": _plain_append, "norm": _plain_norm,
            "prefix": _plain_prefix}[op](state)


# ---------------------------------------------------------------- the library
def _own_head(s):
    import reduce_copy_rank_gb300 as dc

    c = s["case"]
    dc.linear_logprobs(s["hidden"], s["weights"], s["tokens"], s["logprobs"], s["workspace"], entropy=s["entropy"],
                       lse=s["lse"], vocab=c["vocab"], temperature=c["temperature"])
    return {"logprobs": s["logprobs"], "entropy": s["entropy"], "lse": s["lse"]}


def _own_head_grad(s):
    import reduce_copy_rank_gb300 as dc

    c = s["case"]
    dc.linear_logprobs_backward(s["hidden"], s["weights"], s["tokens"], s["lse"], s["grad_logprobs"], s["grad_hidden"],
                                s["grad_weights"], s["workspace"], entropy=s["entropy"], grad_entropy=s["grad_entropy"],
                                vocab=c["vocab"], temperature=c["temperature"])
    return {"hidden": s["grad_hidden"], "weights": s["grad_weights"]}


def _own_append(s):
    import reduce_copy_rank_gb300 as dc

    dc.kv_append(s["k"], s["v"], s["positions"], s["seqs"], s["table"], s["k_cache"], s["v_cache"], q=s["q"],
                 q_out=s["q_out"], cos_sin=s["cos_sin"], interleaved=s["case"]["interleaved"], q_norm=s["q_norm"],
                 k_norm=s["k_norm"], eps=EPS)
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_norm(s):
    import reduce_copy_rank_gb300 as dc

    turned = s["case"]["interleaved"]
    dc.qk_norm_rotate(s["q"], s["k"], s["positions"], s["cos_sin"], s["q_norm"], s["k_norm"], s["q_out"], s["k_out"],
                      eps=EPS, interleaved=turned)
    dc.qk_norm_rotate_backward(s["q"], s["k"], s["positions"], s["cos_sin"], s["q_norm"], s["k_norm"], s["grad_q_out"],
                               s["grad_k_out"], s["grad_q"], s["grad_k"], s["grad_q_norm"], s["grad_k_norm"],
                               s["workspace"], eps=EPS, interleaved=turned)
    return {name: s[name] for name in ("q_out", "k_out", "grad_q", "grad_k", "grad_q_norm", "grad_k_norm")}


def _own_prefix(s):
    import reduce_copy_rank_gb300 as dc

    dc.prefix_attention(s["q"], s["k_cache"], s["v_cache"], s["prefix_table"], s["prefix_lengths"], s["table"],
                        s["lengths"], s["out"], s["workspace"], lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


# ------------------------------------------------------------ the plain forms
def _plain_logits(s):
    c = s["case"]
    w = torch.cat(s["weights"], 0)[:c["vocab"]].float()
    x = s["hidden"].float()
    return torch.matmul(x, w.t()) * (1.0 / c["temperature"]), x, w


def _plain_head(s):
    z = _plain_logits(s)[0]
    m = z.max(1, keepdim=True).values
    z = z - m
    e = z.exp()
    total = e.sum(1)
    log_total = total.log()
    return {"logprobs": z.gather(1, s["tokens"][:, None])[:, 0] - log_total,
            "entropy": log_total - (e * z).sum(1) / total, "lse": m[:, 0] + log_total}


def _plain_head_grad(s):
    c = s["case"]
    dt = DTYPES[c["dtype"]]
    logp, x, w = _plain_logits(s)
    logp = logp - s["lse"][:, None]
    kept = s["tokens"] >= 0
    g = torch.where(kept, s["grad_logprobs"], 0.0)[:, None]
    d = -logp.exp() * (g + s["grad_entropy"][:, None] * (logp + s["entropy"][:, None]))
    d = d.scatter_add(1, s["tokens"].clamp(min=0)[:, None], g) * (1.0 / c["temperature"])
    widths = [t.shape[0] for t in s["weights"]]
    grad_w = torch.matmul(d.t(), x)
    grad_w = torch.nn.functional.pad(grad_w, (0, 0, 0, sum(widths) - c["vocab"])).to(dt)
    return {"hidden": torch.matmul(d, w).to(dt), "weights": list(torch.split(grad_w, widths, dim=0))}


def _pairs(x, rot, interleaved):
    return (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])


def _join(a, b, rest, interleaved):
    both = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([both, rest], -1)


def _plain_normed(x, w, cos, sin, rot, interleaved):
    """Normed and rotated heads in 32 bits."""
    x = x.float()
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
    a, b = _pairs(y, rot, interleaved)
    return _join(a * cos - b * sin, b * cos + a * sin, y[..., rot:], interleaved)


def _plain_normed_grad(x, w, cos, sin, rot, interleaved, dy):
    x, dy, w = x.float(), dy.float(), w.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    a, b = _pairs(dy, rot, interleaved)
    g = _join(a * cos + b * sin, b * cos - a * sin, dy[..., rot:], interleaved)
    n = x * r
    gw = g * w
    return r * (gw - n * (gw * n).mean(-1, keepdim=True)), (g * n).sum((0, 1))


def _angles(s):
    c = s["case"]
    cs = s["cos_sin"][s["positions"].long()]
    half = c["rotary"] // 2
    return cs[:, None, :half], cs[:, None, half:], c["rotary"], c["interleaved"]


def _plain_append(s):
    c = s["case"]
    dt = DTYPES[c["dtype"]]
    how = _angles(s)
    q = _plain_normed(s["q"], s["q_norm"], *how).to(dt)
    k = _plain_normed(s["k"], s["k_norm"], *how).to(dt)
    pos = s["positions"].long()
    page = s["table"][s["seqs"].long(), pos // c["page"]].long()
    s["k_cache"][page, pos % c["page"]] = k
    s["v_cache"][page, pos % c["page"]] = s["v"]
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_norm(s):
    dt = DTYPES[s["case"]["dtype"]]
    how = _angles(s)
    found = {}
    for name in ("q", "k"):
        found[f"{name}_out"] = _plain_normed(s[name], s[f"{name}_norm"], *how).to(dt)
        dx, dw = _plain_normed_grad(s[name], s[f"{name}_norm"], *how, s[f"grad_{name}_out"])
        found[f"grad_{name}"], found[f"grad_{name}_norm"] = dx.to(dt), dw
    return {name: found[name] for name in ("q_out", "k_out", "grad_q", "grad_k", "grad_q_norm", "grad_k_norm")}


def _plain_prefix(s):
    c = s["case"]
    n, hq, d = s["q"].shape
    p, each, hk, group = c["prefixes"], c["each"], c["kv_heads"], hq // c["kv_heads"]
    q = s["q"].float() * (1.0 / math.sqrt(d))

    def cached(cache, table):
        return cache[table.long()].float().flatten(1, 2)  # [rows, tokens, heads, dim]

    def masked(score, lengths):  # [rows, heads, queries, tokens]
        held = torch.arange(score.shape[-1], device=score.device)[None] < lengths.long()[:, None]
        return torch.where(held[:, None, None], score, -math.inf)

    shared = q.reshape(p, each, hk, group, d).permute(0, 2, 1, 3, 4).reshape(p, hk, each * group, d)
    a = torch.matmul(shared, cached(s["k_cache"], s["prefix_table"]).permute(0, 2, 3, 1))
    a = masked(a, s["prefix_lengths"])
    b = torch.matmul(q.reshape(n, hk, group, d), cached(s["k_cache"], s["table"]).permute(0, 2, 3, 1))
    b = masked(b, s["lengths"])

    def sequences(x):  # [prefixes, heads, sequences of one x group, .] as [sequences, heads, group, .]
        return x.reshape(p, hk, each, group, -1).permute(0, 2, 1, 3, 4).reshape(n, hk, group, -1)

    m = torch.maximum(sequences(a.max(-1, keepdim=True).values), b.max(-1, keepdim=True).values).clamp(min=-1e30)
    a = (a - m.reshape(p, each, hk, group, 1).permute(0, 2, 1, 3, 4).reshape(p, hk, each * group, 1)).exp()
    b = (b - m).exp()
    total = sequences(a.sum(-1, keepdim=True)) + b.sum(-1, keepdim=True)
    out = sequences(torch.matmul(a, cached(s["v_cache"], s["prefix_table"]).permute(0, 2, 1, 3)))
    out = (out + torch.matmul(b, cached(s["v_cache"], s["table"]).permute(0, 2, 1, 3))) / total.clamp(min=1e-30)
    lse = torch.where(total > 0, m + total.log(), -math.inf)
    return {"out": out.to(s["q"].dtype).reshape(n, hq, d), "lse": lse.reshape(n, hq)}


# ------------------------------------------------------------- work and truth
def work(case):
    es = BYTES[case["dtype"]]
    if case["op"] in ("head", "head_grad"):
        n, v, h = case["rows"], case["vocab"], case["hidden"]
        if case["op"] == "head":
            return {"bytes": (n + v) * h * es + n * 20, "flops": 2 * n * v * h}
        return {"bytes": (2 * n + v + sum(_widths(case))) * h * es + n * 24, "flops": 6 * n * v * h}
    hq, hk, d = case["q_heads"], case["kv_heads"], case["dim"]
    if case["op"] == "append":
        t = case["tokens"]
        return {"bytes": t * ((hq + 2 * hk) * d * es * 2 + 12 + 4 * case["rotary"]),
                "flops": t * (hq + hk) * (4 * d + 3 * case["rotary"])}
    if case["op"] == "norm":
        t = case["tokens"]
        return {"bytes": t * ((hq + hk) * d * es * 4 + 4) + min(t, case["length"]) * 4 * case["rotary"],
                "flops": t * (hq + hk) * (13 * d + 6 * case["rotary"])}
    prefix, own_tokens = _prefix_lengths(case)
    n = len(own_tokens)
    pairs = sum(prefix) * case["each"] + sum(own_tokens)
    return {"bytes": 2 * (sum(prefix) + sum(own_tokens)) * hk * d * es + n * hq * (2 * d * es + 4), "flops": 4 * pairs * hq * d}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("head", "head_grad"):
        return _exact_head(case, s)
    f = torch.float64
    if case["op"] in ("append", "norm"):
        half = case["rotary"] // 2
        pos = s["positions"].long()
        cs = s["cos_sin"].to(f).index_select(0, pos)
        # each pair as a complex number, turned by its angle
        turn = torch.complex(cs[:, :half], cs[:, half:])[:, None]
        first = torch.arange(half, device=pos.device) * (2 if case["interleaved"] else 1)
        second = first + (1 if case["interleaved"] else half)

        def turned(x, w):
            y = x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * w
            z = torch.complex(y[..., first], y[..., second]) * turn
            return y.index_copy(2, first, z.real).index_copy(2, second, z.imag)

        if case["op"] == "append":
            k_cache, v_cache = s["k_cache"].to(f), s["v_cache"].to(f)
            slot = s["table"].long()[s["seqs"].long(), pos // case["page"]] * case["page"] + pos % case["page"]
            k_cache.view(-1, *k_cache.shape[2:]).index_copy_(0, slot, turned(s["k"].to(f), s["k_norm"].to(f)))
            v_cache.view(-1, *v_cache.shape[2:]).index_copy_(0, slot, s["v"].to(f))
            return {"q": turned(s["q"].to(f), s["q_norm"].to(f)), "k_cache": k_cache, "v_cache": v_cache}
        leaves = [s[name].to(f).requires_grad_() for name in ("q", "k", "q_norm", "k_norm")]
        outs = turned(leaves[0], leaves[2]), turned(leaves[1], leaves[3])
        grads = torch.autograd.grad(outs, leaves, (s["grad_q_out"].to(f), s["grad_k_out"].to(f)))
        return dict(zip(("q_out", "k_out", "grad_q", "grad_k", "grad_q_norm", "grad_k_norm"),
                        [o.detach() for o in outs] + list(grads)))
    hk, group = case["kv_heads"], case["q_heads"] // case["kv_heads"]
    prefix, own_tokens = _prefix_lengths(case)
    outs, lses = [], []
    for b, n in enumerate(own_tokens):
        p = b // case["each"]
        rows = []
        for table, length in ((s["prefix_table"][p], prefix[p]), (s["table"][b], n)):
            at = torch.arange(length, device=table.device)
            rows.append((table.long()[at // case["page"]], at % case["page"]))
        page, slot = (torch.cat(x) for x in zip(*rows))
        q = s["q"][b].to(f).view(hk, group, -1)
        score = torch.matmul(q, s["k_cache"][page, slot].to(f).permute(1, 2, 0)) / math.sqrt(case["dim"])
        lse = torch.logsumexp(score, -1)
        outs.append(torch.matmul(torch.exp(score - lse[..., None]), s["v_cache"][page, slot].to(f).transpose(0, 1)).flatten(0, 1))
        lses.append(lse.flatten())
    return {"out": torch.stack(outs), "lse": torch.stack(lses)}


def _exact_head(case, s):
    """Scores and gradients in 64 bits, a block of rows at a time."""
    inv = float(torch.tensor(1.0 / case["temperature"], dtype=torch.float32))
    n, v = case["rows"], case["vocab"]
    w = torch.cat(s["weights"], 0).to(torch.float64)
    grad = case["op"] == "head_grad"
    grad_w = torch.zeros_like(w) if grad else None
    found = [[] for _ in range(3)]
    for at in range(0, n, 512):
        part = slice(at, min(n, at + 512))
        x, token = s["hidden"][part].to(torch.float64), s["tokens"][part]
        z = torch.mm(x, w[:v].t()).mul_(inv)
        if not grad:
            logp = torch.log_softmax(z, 1)
            found[0].append(logp.gather(1, token[:, None])[:, 0])
            found[1].append(-(logp.exp() * logp).sum(1))
            found[2].append(torch.logsumexp(z, 1))
            continue
        logp = z.sub_(s["lse"][part].double()[:, None])
        p = logp.exp()
        kept = token >= 0
        g = s["grad_logprobs"][part].double() * kept
        d = -p * (g[:, None] + s["grad_entropy"][part].double()[:, None] * (logp + s["entropy"][part].double()[:, None]))
        d[torch.arange(len(token), device=p.device)[kept], token[kept]] += g[kept]
        d *= inv
        found[0].append(torch.mm(d, w[:v]))
        grad_w[:v].addmm_(d.t(), x)
    if grad:
        return {"hidden": torch.cat(found[0]), "weights": list(torch.split(grad_w, _widths(case), 0))}
    return {"logprobs": torch.cat(found[0]), "entropy": torch.cat(found[1]), "lse": torch.cat(found[2])}
