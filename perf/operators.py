"""Workloads of the language-model operators, each in a plain torch form and through the library.

score   log probabilities of given tokens over vocabulary shards, with entropy and top alternatives
grad    the gradient of those log probabilities and entropies with respect to the logits
append  keys and values put into a paged cache, queries and keys rotated to their positions on the way
attend  attention of one new token per sequence over the paged cache

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
LARGEST = 8192 * 128000  # logits of the largest scoring and gradient cases
TOKENS = 64 * 8192       # cached tokens of the largest attention case, at 8 heads of 128


def listed():
    return [
        # greedy decoding of four sequences, the head split over two ranks: latency is all there is
        {"name": "score_step", "op": "score", "rows": 4, "vocab": 32768, "ranks": 2, "dtype": "bf16", "top": 1,
         "temperature": 1.0, "padded": False},
        # one step of a rollout batch on eight ranks, with the alternatives that a distillation or an API keeps
        {"name": "score_rollout", "op": "score", "rows": 128, "vocab": 131072, "ranks": 8, "dtype": "bf16", "top": 20,
         "temperature": 0.7, "padded": False},
        # 32-bit logits of an odd vocabulary in uneven shards: rows that start at every alignment
        {"name": "score_odd", "op": "score", "rows": 1021, "vocab": 50021, "ranks": 3, "dtype": "f32", "top": 5,
         "temperature": 1.0, "padded": False},
        # log probabilities of a training batch, as a policy-gradient step takes them
        {"name": "score_train", "op": "score", "rows": 8192, "vocab": 128000, "ranks": 1, "dtype": "bf16", "top": 0,
         "temperature": 1.0, "padded": False},
        # the gradient for a short batch of half-precision logits of an odd vocabulary
        {"name": "grad_odd", "op": "grad", "rows": 509, "vocab": 50021, "ranks": 1, "dtype": "f16",
         "temperature": 0.8, "padded": False},
        # the gradient of a training batch, eight ranks with padded shards
        {"name": "grad_train", "op": "grad", "rows": 8192, "vocab": 127900, "ranks": 8, "dtype": "bf16",
         "temperature": 1.0, "padded": True},
        # the new tokens of 64 sequences in a decoding step
        {"name": "append_step", "op": "append", "seqs": 64, "tokens": 64, "q_heads": 32, "kv_heads": 8, "dim": 128,
         "rotary": 128, "interleaved": False, "page": 64, "dtype": "bf16", "length": 4000},
        # five prompts, heads of 80 of which 32 are rotated in neighbouring pairs
        {"name": "append_prompt", "op": "append", "seqs": 5, "tokens": 8191, "q_heads": 32, "kv_heads": 32, "dim": 80,
         "rotary": 32, "interleaved": True, "page": 16, "dtype": "f16", "length": 2000},
        # one rank of eight decoding one sequence: one key head, a short odd cache
        {"name": "attend_one", "op": "attend", "seqs": 1, "length": 1025, "q_heads": 8, "kv_heads": 1, "dim": 128,
         "page": 16, "window": 0, "dtype": "bf16"},
        # one long context on its own: the cache has to be split to use the machine
        {"name": "attend_long", "op": "attend", "seqs": 1, "length": 131072, "q_heads": 64, "kv_heads": 8, "dim": 128,
         "page": 64, "window": 0, "dtype": "bf16"},
        # a ragged serving batch, some sequences empty or one token long
        {"name": "attend_batch", "op": "attend", "seqs": 128, "length": 8192, "q_heads": 32, "kv_heads": 8, "dim": 128,
         "page": 64, "window": 0, "dtype": "bf16"},
        # a head of 64 for every query head, attending to a window of an odd batch
        {"name": "attend_window", "op": "attend", "seqs": 19, "length": 5000, "q_heads": 12, "kv_heads": 12, "dim": 64,
         "page": 16, "window": 1500, "dtype": "f16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["score", "grad", "append", "attend"])
    if op in ("score", "grad"):
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        vocab = _log(rng, 1000, 200000)
        rows = _log(rng, 1, min(8192, LARGEST * 2 // (vocab * BYTES[dtype])))
        c = {"op": op, "rows": rows, "vocab": vocab, "ranks": rng.choice([1, 1, 2, 3, 4, 8]), "dtype": dtype,
             "temperature": rng.choice([1.0, 1.0, 0.7, 1.3]), "padded": rng.random() < 0.3}
        if op == "score":
            # the alternatives' plain form sorts whole rows: fewer rows with them
            c["top"] = rng.choice([0, 1, 5, 20, 32]) if rows * vocab < 1 << 27 else 0
        return c
    kv_heads = rng.choice([1, 2, 4, 8, 12])
    c = {"op": op, "kv_heads": kv_heads, "q_heads": kv_heads * rng.choice([1, 2, 3, 4, 8, 16]),
         "dim": rng.choice([64, 96, 128, 128, 256]), "page": rng.choice([1, 16, 24, 64, 128]),
         "dtype": rng.choice(["bf16", "bf16", "f16"])}
    if op == "append":
        if rng.random() < 0.5:
            seqs = _log(rng, 1, 256)
            tokens = seqs
        else:
            seqs = rng.randint(1, 8)
            tokens = _log(rng, max(8, seqs), 8192)
        held = max(1, (1 << 27) // (seqs * kv_heads * c["dim"]))
        c |= {"seqs": seqs, "tokens": tokens, "length": _log(rng, 1, min(8000, held)), "rotary": rng.choice([c["dim"], c["dim"], 32]),
              "interleaved": rng.random() < 0.5}
        per = c["dim"] * (c["q_heads"] + 2 * kv_heads)
        c["tokens"] = max(seqs, min(tokens, 8191 * 80 * 96 // per))
    else:
        room = TOKENS * 8 * 128 // (kv_heads * c["dim"])
        seqs = _log(rng, 1, 256)
        length = _log(rng, 1, min(131072, max(1, room // seqs)))
        c |= {"seqs": seqs, "length": length, "window": rng.choice([0, 0, 0, _log(rng, 1, 4096)])}
    return c


def _lengths(case):
    """Cached tokens of each sequence: the same for every seed, the longest is `length`."""
    n, top = case["seqs"], case["length"]
    rng = random.Random(n * 1000003 + top)
    got = [top] + [rng.randint(1, top) for _ in range(n - 1)]
    if n >= 8:
        got[3], got[5] = 0, 1
    return got


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


def _widths(case):
    v, p = case["vocab"], case["ranks"]
    if case["padded"]:
        return [(-(-v // p) + 63) // 64 * 64] * p
    return [v // p + (1 if r < v % p else 0) for r in range(p)]


def _page_table(lengths, page, spare, gen, dev):
    """A table over shuffled pages, -1 past each sequence's end, and the number of pages."""
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
    if case["op"] in ("score", "grad"):
        n, v = case["rows"], case["vocab"]
        # logits as a trained head gives them: a few units wide, a few tokens far ahead, one in a hundred masked
        shards = []
        for w in _widths(case):
            x = torch.randn(n, w, generator=gen, device=dev, dtype=torch.float32).mul_(2.5)
            hot = torch.randint(0, w, (n, 4), generator=gen, device=dev)
            x.scatter_add_(1, hot, torch.rand(n, 4, generator=gen, device=dev) * 12)
            off = torch.randint(0, w, (n, max(1, w // 100)), generator=gen, device=dev)
            x.scatter_(1, off, -math.inf)
            shards.append(x.to(dt))
            del x
        whole = torch.cat(shards, 1)[:, :v]
        best = whole.argmax(1)
        guess = torch.randint(0, v, (n,), generator=gen, device=dev)
        tokens = torch.where(torch.rand(n, generator=gen, device=dev) < 0.7, best, guess)
        tokens = torch.where(torch.isinf(whole.gather(1, tokens[:, None])[:, 0]), best, tokens)
        s |= {"shards": shards, "tokens": tokens}
        f32 = {"device": dev, "dtype": torch.float32}
        if case["op"] == "score":
            k = case["top"]
            s |= {"logprobs": torch.empty(n, **f32), "entropy": torch.empty(n, **f32), "lse": torch.empty(n, **f32)}
            s["top_logprobs"] = torch.empty(n, k, **f32) if k else None
            s["top_tokens"] = torch.empty(n, k, device=dev, dtype=torch.int64) if k else None
        else:
            lse, ent = [], []
            for at in range(0, n, 1024):
                logp = torch.log_softmax(whole[at:at + 1024].float() * (1.0 / case["temperature"]), 1)
                first = whole[at:at + 1024, :].float().mul_(1.0 / case["temperature"])
                lse.append(torch.logsumexp(first, 1))
                ent.append(-(logp.exp() * logp.clamp(min=-1e30)).sum(1))
                del logp, first
            s |= {"lse": torch.cat(lse), "entropy": torch.cat(ent)}
            s["grad_logprobs"] = torch.randn(n, generator=gen, **f32)
            s["grad_entropy"] = torch.randn(n, generator=gen, **f32) * 0.1
            # a fifth of the tokens belong to the prompt and carry no log probability
            s["tokens"] = torch.where(torch.rand(n, generator=gen, device=dev) < 0.2, -100, tokens)
            s["grads"] = [torch.empty_like(x) for x in shards]
        return s
    hq, hk, d, page = case["q_heads"], case["kv_heads"], case["dim"], case["page"]
    if case["op"] == "append":
        where = _new_tokens(case)
        held = [max((p + 1 for b, p in where if b == i), default=0) for i in range(case["seqs"])]
        table, pages = _page_table(held, page, 3, gen, dev)
        t = len(where)
        both = normal(t, hq + 2 * hk, d)  # the projection's output: queries, keys and values side by side
        rot = case["rotary"]
        angle = torch.arange(max(held), device=dev, dtype=torch.float64)[:, None] * \
            (10000.0 ** (-torch.arange(0, rot, 2, device=dev, dtype=torch.float64) / rot))[None]
        s |= {"q": both[:, :hq], "k": both[:, hq:hq + hk], "v": both[:, hq + hk:],
              "seqs": torch.tensor([b for b, _ in where], device=dev, dtype=torch.int32),
              "positions": torch.tensor([p for _, p in where], device=dev, dtype=torch.int32),
              "table": table, "cos_sin": torch.cat([angle.cos(), angle.sin()], 1).to(torch.float32),
              "k_cache": normal(pages, page, hk, d), "v_cache": normal(pages, page, hk, d),
              "q_out": torch.empty(t, hq, d, device=dev, dtype=dt)}
        return s
    lengths = _lengths(case)
    table, pages = _page_table(lengths, page, 1, gen, dev)
    s |= {"q": normal(case["seqs"], hq, d), "k_cache": normal(pages, page, hk, d), "v_cache": normal(pages, page, hk, d),
          "table": table, "lengths": torch.tensor(lengths, device=dev, dtype=torch.int32),
          "out": torch.empty(case["seqs"], hq, d, device=dev, dtype=dt),
          "lse": torch.empty(case["seqs"], hq, device=dev, dtype=torch.float32)}
    if own:  # the library's workspace, kept by the caller from call to call
        import reduce_copy_rank_gb300 as dc

        s["workspace"] = dc.attention_workspace(case["seqs"], hq, hk, d, table.shape[1] * page)
    return s


def run(state):
    op = state["case"]["op"]
    if own:
        return {"score": _own_score, "grad": _own_grad, "append": _own_append, "attend": _own_attend}[op](state)
    return {"score": _plain_score, "grad": _plain_grad, "append": _plain_append, "attend": _plain_attend}[op](state)


# ---------------------------------------------------------------- the library
def _own_score(s):
    import reduce_copy_rank_gb300 as dc

    c = s["case"]
    dc.token_logprobs(s["shards"], s["tokens"], s["logprobs"], entropy=s["entropy"], lse=s["lse"],
                      top_logprobs=s["top_logprobs"], top_tokens=s["top_tokens"], vocab=c["vocab"],
                      temperature=c["temperature"])
    return _scores(s["logprobs"], s["entropy"], s["lse"], s["top_logprobs"], s["top_tokens"])


def _own_grad(s):
    import reduce_copy_rank_gb300 as dc

    c = s["case"]
    return dc.token_logprobs_backward(s["shards"], s["tokens"], s["lse"], s["grad_logprobs"], s["grads"],
                                      entropy=s["entropy"], grad_entropy=s["grad_entropy"], vocab=c["vocab"],
                                      temperature=c["temperature"])


def _own_append(s):
    import reduce_copy_rank_gb300 as dc

    dc.kv_append(s["k"], s["v"], s["positions"], s["seqs"], s["table"], s["k_cache"], s["v_cache"], q=s["q"],
                 q_out=s["q_out"], cos_sin=s["cos_sin"], interleaved=s["case"]["interleaved"])
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_attend(s):
    import reduce_copy_rank_gb300 as dc

    dc.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lengths"], s["out"], s["workspace"],
                       window=s["case"]["window"], lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


# ------------------------------------------------------------ the plain forms
def _scores(logprobs, entropy, lse, top_logprobs, top_tokens):
    r = {"logprobs": logprobs, "entropy": entropy, "lse": lse}
    if top_tokens is not None:
        r |= {"top_logprobs": top_logprobs, "top_tokens": top_tokens}
    return r


def _plain_score(s):
    c = s["case"]
    x = torch.cat(s["shards"], 1)[:, :c["vocab"]].float()
    z = x * (1.0 / c["temperature"])
    m = z.max(1, keepdim=True).values
    z = z - m
    e = z.exp()
    total = e.sum(1)
    log_total = total.log()
    entropy = log_total - (e * z.clamp(min=-1e4)).sum(1) / total
    logprobs = z.gather(1, s["tokens"][:, None])[:, 0] - log_total
    top = top_logprobs = None
    if c["top"]:
        top = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :c["top"]].contiguous()
        top_logprobs = z.gather(1, top) - log_total[:, None]
    return _scores(logprobs, entropy, m[:, 0] + log_total, top_logprobs, top)


def _plain_grad(s):
    c = s["case"]
    x = torch.cat(s["shards"], 1)[:, :c["vocab"]].float()
    logp = (x * (1.0 / c["temperature"]) - s["lse"][:, None]).clamp(min=-1e4)
    kept = s["tokens"] >= 0
    g = torch.where(kept, s["grad_logprobs"], 0.0)[:, None]
    d = -logp.exp() * (g + s["grad_entropy"][:, None] * (logp + s["entropy"][:, None]))
    d = d.scatter_add(1, s["tokens"].clamp(min=0)[:, None], g) * (1.0 / c["temperature"])
    widths = [t.shape[1] for t in s["shards"]]
    d = torch.nn.functional.pad(d, (0, sum(widths) - c["vocab"])).to(DTYPES[c["dtype"]])
    return list(torch.split(d, widths, dim=1))


def _rotate(x, cos, sin, rot, interleaved):
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
    ra, rb = a * cos - b * sin, b * cos + a * sin
    both = torch.stack([ra, rb], -1).flatten(-2) if interleaved else torch.cat([ra, rb], -1)
    return torch.cat([both, x[..., rot:]], -1)


def _plain_append(s):
    c = s["case"]
    rot, dt = c["rotary"], DTYPES[c["dtype"]]
    pos = s["positions"].long()
    cs = s["cos_sin"][pos]
    cos, sin = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
    q = _rotate(s["q"].float(), cos, sin, rot, c["interleaved"]).to(dt)
    k = _rotate(s["k"].float(), cos, sin, rot, c["interleaved"]).to(dt)
    page = s["table"][s["seqs"].long(), pos // c["page"]].long()
    s["k_cache"][page, pos % c["page"]] = k
    s["v_cache"][page, pos % c["page"]] = s["v"]
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_attend(s):
    c = s["case"]
    b, hq, d = s["q"].shape
    hk = c["kv_heads"]
    table = s["table"].long()
    k = s["k_cache"][table].float().view(b, -1, hk, d).permute(0, 2, 3, 1)
    score = torch.matmul(s["q"].float().view(b, hk, hq // hk, d), k) * (1.0 / math.sqrt(d))
    at = torch.arange(score.shape[-1], device=score.device)[None]
    length = s["lengths"].long()[:, None]
    held = at < length
    if c["window"]:
        held &= at >= length - c["window"]
    score = torch.where(held[:, None, None], score, -math.inf)
    m = score.max(-1, keepdim=True).values.clamp(min=-1e30)
    e = (score - m).exp()
    total = e.sum(-1, keepdim=True)
    v = s["v_cache"][table].float().view(b, -1, hk, d).permute(0, 2, 1, 3)
    out = torch.matmul(e, v) / total.clamp(min=1e-30)
    lse = torch.where(total > 0, m + total.log(), -math.inf)
    return {"out": out.to(s["q"].dtype).view(b, hq, d), "lse": lse.view(b, hq)}


# ------------------------------------------------------------- work and truth
def work(case):
    es = BYTES[case["dtype"]]
    if case["op"] in ("score", "grad"):
        n, v = case["rows"], case["vocab"]
        if case["op"] == "score":
            return {"bytes": n * (v * es + 8 + 12 + 12 * case["top"]), "flops": 6 * n * v}
        return {"bytes": n * ((v + sum(_widths(case))) * es + 8 + 16), "flops": 7 * n * v}
    hq, hk, d = case["q_heads"], case["kv_heads"], case["dim"]
    if case["op"] == "append":
        t = case["tokens"]
        return {"bytes": t * ((hq + 2 * hk) * d * es * 2 + 12 + 4 * case["rotary"]),
                "flops": 3 * t * (hq + hk) * case["rotary"]}
    tokens = sum(min(n, case["window"] or n) for n in _lengths(case))
    return {"bytes": 2 * tokens * hk * d * es + case["seqs"] * hq * (2 * d * es + 4), "flops": 4 * tokens * hq * d}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("score", "grad"):
        return _exact_logits(case, s)
    f = torch.float64
    if case["op"] == "append":
        k_cache, v_cache = s["k_cache"].to(f), s["v_cache"].to(f)
        pos, seq = s["positions"].long(), s["seqs"].long()
        cs = s["cos_sin"].to(f).index_select(0, pos)
        half = case["rotary"] // 2
        # each pair as a complex number, turned by its angle
        turn = torch.complex(cs[:, :half], cs[:, half:])[:, None]
        turned = []
        for x in (s["q"].to(f), s["k"].to(f)):
            if case["interleaved"]:
                first, second = torch.arange(half) * 2, torch.arange(half) * 2 + 1
            else:
                first, second = torch.arange(half), torch.arange(half) + half
            z = torch.complex(x[..., first], x[..., second]) * turn
            x = x.clone()
            x[..., first], x[..., second] = z.real, z.imag
            turned.append(x)
        slot = s["table"].long()[seq, pos // case["page"]] * case["page"] + pos % case["page"]
        k_cache.view(-1, *k_cache.shape[2:]).index_copy_(0, slot, turned[1])
        v_cache.view(-1, *v_cache.shape[2:]).index_copy_(0, slot, s["v"].to(f))
        return {"q": turned[0], "k_cache": k_cache, "v_cache": v_cache}
    hk, group = case["kv_heads"], case["q_heads"] // case["kv_heads"]
    outs, lses = [], []
    for b, n in enumerate(_lengths(case)):
        start = max(0, n - case["window"]) if case["window"] else 0
        at = torch.arange(start, n, device=s["table"].device)
        rows = s["table"][b].long()[at // case["page"]], at % case["page"]
        q = s["q"][b].to(f).view(hk, group, -1)
        score = torch.einsum("hgd,nhd->hgn", q, s["k_cache"][rows].to(f)) / math.sqrt(case["dim"])
        lse = torch.logsumexp(score, -1)
        outs.append(torch.einsum("hgn,nhd->hgd", torch.exp(score - lse[..., None]), s["v_cache"][rows].to(f)).flatten(0, 1))
        lses.append(lse.flatten())
    return {"out": torch.stack(outs), "lse": torch.stack(lses)}


def _exact_logits(case, s):
    """Scores and gradients in 64 bits, a block of rows at a time."""
    inv = float(torch.tensor(1.0 / case["temperature"], dtype=torch.float32))
    n, v, k = case["rows"], case["vocab"], case.get("top", 0)
    widths = _widths(case)
    found = [[] for _ in (widths if case["op"] == "grad" else range(5))]
    for at in range(0, n, 512):
        part = slice(at, min(n, at + 512))
        x = torch.cat([t[part] for t in s["shards"]], 1)[:, :v].to(torch.float64)
        token = s["tokens"][part]
        if case["op"] == "score":
            logp = torch.log_softmax(x * inv, 1)
            found[0].append(logp.gather(1, token[:, None])[:, 0])
            found[1].append(-torch.where(logp == -math.inf, 0.0, logp.exp() * logp).sum(1))
            found[2].append(torch.logsumexp(x * inv, 1))
            if k:
                # the k largest, ties to the lowest index: by hand, largest first
                left = x.clone()
                ids = []
                for _ in range(k):
                    best = left.max(1, keepdim=True).values
                    here = torch.where(left == best, torch.arange(v, device=x.device)[None], v).min(1, keepdim=True).values
                    left.scatter_(1, here, math.nan)
                    left = torch.where(torch.isnan(left), -math.inf, left)
                    ids.append(here)
                found[4].append(torch.cat(ids, 1))
                found[3].append(logp.gather(1, found[4][-1]))
        else:
            logp = x * inv - s["lse"][part].double()[:, None]
            p = logp.exp()
            hot = torch.zeros_like(p)
            kept = token >= 0
            hot[torch.arange(len(token), device=p.device)[kept], token[kept]] = 1.0
            g = s["grad_logprobs"][part].double() * kept
            spread = torch.where(p > 0, p * (logp + s["entropy"][part].double()[:, None]), 0.0)
            d = inv * (g[:, None] * (hot - p) - s["grad_entropy"][part].double()[:, None] * spread)
            d = torch.cat([d, torch.zeros(len(d), sum(widths) - v, dtype=d.dtype, device=d.device)], 1)
            for r, piece in enumerate(torch.split(d, widths, 1)):
                found[r].append(piece)
    if case["op"] == "grad":
        return [torch.cat(f) for f in found]
    r = {"logprobs": torch.cat(found[0]), "entropy": torch.cat(found[1]), "lse": torch.cat(found[2])}
    if k:
        r |= {"top_logprobs": torch.cat(found[3]), "top_tokens": None}
    return r
