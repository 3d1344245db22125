"""Measured cases of the serving operators around the verify step.

One speculative decoding step of a paged server is: sample the draft tokens
(`sample`), give every request the cache pages of its new tokens and map each
token to its slot (`slots`), write the new keys and values there (`append`),
attend from every new token over the request's pages (`attention`), and verify.
A case names the operator in "op" and its sizes; the ragged lengths of a case
belong to the case, all data come from the seed.

`own` false: `run` computes the operators in plain torch, in 32 bits, rounded
once at the end.  `own` true: it calls the library.
"""

import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one request's next token: latency
        dict(name="sample_b1", op="sample", rows=1, vocab=151936, dtype="bf16", kind="peaked",
             filters="topk_topp"),
        # a drafter's step at concurrency 32, every request with its own settings
        dict(name="sample_b32_mixed", op="sample", rows=32, vocab=151936, dtype="bf16",
             kind="peaked", filters="mixed"),
        # every drafted position of a large batch, flat rows: kept sets of
        # thousands of tokens under top-p alone
        dict(name="sample_flat_topp", op="sample", rows=96, vocab=129280, dtype="fp32",
             kind="flat", filters="topp"),
        # the largest: 512 rows of the largest vocabulary, top-k 20 and top-p 0.95
        dict(name="sample_b512", op="sample", rows=512, vocab=262144, dtype="bf16",
             kind="peaked", filters="topk_topp"),
        # a step of 32 requests with a block of up to 16 tokens each
        dict(name="slots_b32", op="slots", batch=32, new=16, ctx_lo=64, ctx_hi=32768, page=16,
             lens=1),
        # a full server: 1,024 requests with chunks of up to 256 tokens
        dict(name="slots_b1024", op="slots", batch=1024, new=256, ctx_lo=16, ctx_hi=16384,
             page=32, lens=2),
        # new keys and values of a verify step, slices of a fused projection
        dict(name="append_b32", op="append", rows=512, kv_heads=8, dim=128, page=16),
        # the same of long prompt chunks
        dict(name="append_prompt", op="append", rows=16384, kv_heads=8, dim=128, page=64),
        # one request's verify step: a block of 16 over a short context, latency
        dict(name="attn_b1", op="attention", batch=1, new=16, ragged=False, ctx_lo=4000,
             ctx_hi=4000, heads=32, kv_heads=8, dim=128, page=16, window=0, lens=3),
        # the verify step at concurrency 32, blocks of 16, mixed contexts
        dict(name="attn_b32_l16", op="attention", batch=32, new=16, ragged=False, ctx_lo=512,
             ctx_hi=32768, heads=32, kv_heads=8, dim=128, page=16, window=0, lens=4),
        # plain decoding: single tokens, wide groups, long contexts
        dict(name="attn_single_b48", op="attention", batch=48, new=1, ragged=False, ctx_lo=1024,
             ctx_hi=32768, heads=64, kv_heads=8, dim=128, page=64, window=0, lens=5),
        # prompt chunks behind cached prefixes: the matrix products bound it
        dict(name="attn_chunk", op="attention", batch=2, new=4096, ragged=False, ctx_lo=2000,
             ctx_hi=16000, heads=32, kv_heads=8, dim=128, page=64, window=0, lens=6),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sample", "sample", "slots", "append", "attention", "attention",
                     "attention"])
    if op == "sample":
        while True:
            c = dict(op=op, rows=_logint(rng, 1, 512), vocab=_logint(rng, 1000, 262144),
                     dtype=rng.choice(["bf16", "bf16", "fp32"]),
                     kind=rng.choice(["peaked", "peaked", "flat"]),
                     filters=rng.choice(["none", "topk_topp", "topp", "minp", "mixed"]))
            if work(c)["bytes"] <= 512 * 262144 * 2 // (4 if c["kind"] == "flat" else 1):
                return c
    if op == "slots":
        return dict(op=op, batch=_logint(rng, 1, 1024), new=_logint(rng, 1, 256), ctx_lo=16,
                    ctx_hi=_logint(rng, 64, 32768 if rng.random() < 0.5 else 4096),
                    page=rng.choice([16, 32, 64, 128]), lens=rng.randrange(1 << 20))
    if op == "append":
        return dict(op=op, rows=_logint(rng, 1, 16384), kv_heads=rng.choice([1, 2, 4, 8]),
                    dim=rng.choice([64, 128]), page=rng.choice([16, 32, 64, 128]))
    while True:
        chunk = rng.random() < 0.3
        new = _logint(rng, 17, 4096) if chunk else rng.choice([1, 1, 2, 4, 5, 8, 16, 16])
        lo = _logint(rng, 1, 8192)
        c = dict(op=op, batch=_logint(rng, 1, 16 if chunk else 256), new=new,
                 ragged=rng.random() < 0.5, ctx_lo=lo,
                 ctx_hi=min(65536, lo * rng.choice([1, 2, 8, 16])),
                 kv_heads=rng.choice([1, 2, 4, 8]), dim=rng.choice([64, 128, 128]),
                 page=rng.choice([16, 32, 64, 128]),
                 window=rng.choice([0, 0, 0, 0, 0, rng.randrange(100, 4096)]),
                 lens=rng.randrange(1 << 20))
        c["heads"] = c["kv_heads"] * rng.choice([1, 2, 4, 5, 8, 16])
        ctx, new_lens = lengths(c)
        S, B = max(a + b for a, b in zip(ctx, new_lens)), c["batch"]
        plain = 8 * B * S * c["kv_heads"] * c["dim"] + 12 * B * c["heads"] * max(new_lens) * S
        w = work(c)
        if w["bytes"] <= 1.5e9 and w["flops"] <= 1.2e12 and plain <= 60e9:
            return c


def lengths(case):
    """Cached tokens and new tokens of every request: the case's own."""
    r = random.Random(case["lens"])
    ctx, new = [], []
    for _ in range(case["batch"]):
        ctx.append(_logint(r, case["ctx_lo"], case["ctx_hi"]))
        new.append(r.randint(1, case["new"]) if case.get("ragged", True) else case["new"])
    return ctx, new


def work(case):
    op = case["op"]
    if op == "sample":  # every logit read once, five settings in and two results out per row
        es = 2 if case["dtype"] == "bf16" else 4
        n = case["rows"] * case["vocab"]
        return {"bytes": n * es + case["rows"] * 28, "flops": 3 * n}
    if op == "slots":  # per request its lengths and counts in and out; per token its position
        # and slot; per page taken the list entry read and the table entry written
        ctx, new = lengths(case)
        return {"bytes": 28 * case["batch"] + 12 * sum(new)
                + 8 * sum(-(-n // case["page"]) for n in new), "flops": 0}
    if op == "append":
        return {"bytes": case["rows"] * (8 + 8 * case["kv_heads"] * case["dim"]), "flops": 0}
    ctx, new = lengths(case)
    W, keys, pairs = case["window"], 0, 0
    for c, n in zip(ctx, new):
        first = max(0, c - W + 1) if W else 0
        keys += c + n - first
        at = np.arange(c, c + n, dtype=np.int64) + 1
        pairs += int(np.minimum(at, W).sum() if W else at.sum())
    row = case["heads"] * case["dim"]
    return {"bytes": 4 * keys * case["kv_heads"] * case["dim"]
            + sum(new) * (4 * row + 4 * case["heads"]),
            "flops": 4 * pairs * row}


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return {"sample": _prepare_sample, "slots": _prepare_slots, "append": _prepare_append,
            "attention": _prepare_attention}[case["op"]](case, seed, g)


def _logits(case, g):
    N, V = case["rows"], case["vocab"]
    if case["kind"] == "flat":  # wide rows: N(0, 3^2) with one raised id
        x = torch.randn(N, V, device=DEV, generator=g) * 3
        x[torch.arange(N, device=DEV),
          torch.randint(0, V, (N,), device=DEV, generator=g)] += 8
    else:  # a language model's rows: a few hundred likely tokens over a broad tail
        x = torch.randn(N, V, device=DEV, generator=g) * 2
        n = min(200, V)
        step = 1 + (torch.rand(N, 1, device=DEV, generator=g) * (V // n - 1)).long()
        ids = torch.randint(0, V, (N, 1), device=DEV, generator=g)
        ids = (ids + step * torch.arange(n, device=DEV)) % V  # no id twice
        rank = torch.log1p(torch.arange(n, device=DEV, dtype=torch.float32))
        x.scatter_(1, ids, 17 - 1.3 * rank + 0.7 * torch.randn(N, n, device=DEV, generator=g))
    return x.to(torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)


def _prepare_sample(case, seed, g):
    """Settings as served (temperature 0.6 to 1.3, top-k 20 or more, top-p 0.8
    to 0.95, min-p 0.05).  Tokens are whole numbers and have to come out equal,
    so no draw and no cut is left to a rounding: each row's top-p and min-p are
    moved to the middle of the step that they cut at, and its random number to
    the middle of the interval of a likely token."""
    N, V = case["rows"], case["vocab"]
    x = _logits(case, g)
    r = random.Random(seed)
    T, K, P, M = [], [], [], []
    for i in range(N):
        f = case["filters"]
        if f == "mixed":
            f = r.choice(["greedy", "none", "topk_topp", "topp", "minp", "topk", "all"])
        T.append(0.0 if f == "greedy" else r.choice([0.6, 0.8, 1.0, 1.0, 1.3]))
        K.append({"topk_topp": 20, "topk": r.choice([1, 5, 50, 300, 1000]),
                  "all": r.choice([20, 64, 100])}.get(f, 0))
        P.append({"topk_topp": 0.95, "topp": r.choice([0.8, 0.9, 0.95]),
                  "all": 0.9}.get(f, 1.0))
        M.append({"minp": 0.05, "all": 0.02}.get(f, 0.0))
    f32 = dict(device=DEV, dtype=torch.float32)
    T, P, M = torch.tensor(T, **f32), torch.tensor(P, **f32), torch.tensor(M, **f32)
    K = torch.tensor(K, device=DEV, dtype=torch.int32)
    u = torch.rand(N, device=DEV, generator=g)
    for a in range(0, N, 64):  # blocks of rows, for memory
        s = slice(a, min(N, a + 64))
        z, order = torch.sort(x[s].double() / torch.where(T[s] > 0, T[s], 1.0).double()[:, None],
                              dim=1, descending=True, stable=True)
        w = torch.exp(z - z[:, :1])
        rank = torch.arange(V, device=DEV)[None]
        k = torch.where((K[s] > 0) & (K[s] < V), K[s], V)[:, None]
        w = torch.where(rank < k, w, 0.0)
        c = torch.cumsum(w, 1)
        n = ((c - w) < P[s, None].double() * c[:, -1:]).sum(1, keepdim=True)
        mid = ((c - w / 2).gather(1, n - 1) / c[:, -1:])[:, 0]
        P[s] = torch.where(P[s] < 1, mid.float(), P[s])
        m = (w >= M[s, None].double()).sum(1, keepdim=True)
        edge = (w.gather(1, m - 1) * w.gather(1, m.clamp(max=V - 1))).sqrt()[:, 0]
        M[s] = torch.where((M[s] > 0) & (m[:, 0] < k[:, 0]), edge.float(), M[s])
        w = torch.where(rank < torch.minimum(n, m), w, 0.0)
        p = torch.zeros_like(w).scatter_(1, order, w)  # by id
        p /= p.sum(1, keepdim=True)
        likely = torch.where(p >= torch.clamp(p.max(1, keepdim=True).values, max=1 / 1024), p, 0.0)
        q = torch.cumsum(likely, 1)
        t = (q <= u[s, None] * q[:, -1:]).sum(1, keepdim=True).clamp(max=V - 1)
        u[s] = (torch.cumsum(p, 1) - p / 2).gather(1, t)[:, 0].float()
    return dict(case=case, logits=x, temperature=T, top_k=K, top_p=P, min_p=M, uniforms=u,
                tokens=torch.empty(N, dtype=torch.int32, device=DEV),
                probs=torch.empty(N, **f32),
                dev_error=torch.zeros(1, dtype=torch.int32, device=DEV))


def _prepare_slots(case, seed, g):
    """A server in mid-flight: tables of the pages held so far (some requests
    hold more than they now need: rejected drafts), a free list in random order."""
    B, page = case["batch"], case["page"]
    ctx, new = lengths(case)
    r = np.random.default_rng(seed)
    ctx, new = np.array(ctx), np.array(new)
    need, most = -(-(ctx + new) // page), -(-ctx // page) + 1 + 16 // page
    held = most - (r.random(B) < 0.8) * (1 + 16 // page)
    width = int(np.maximum(need, most).max()) + 3
    ids = r.permutation(int(most.sum()) + int(need.sum()) + 64).astype(np.int32)
    table = np.zeros((B, width), np.int32)
    table[np.arange(width)[None] < held[:, None]] = ids[:held.sum()]
    free = np.zeros(len(ids), np.int32)
    left = ids[held.sum():]
    free[:len(left)] = left
    n = int(new.sum()) + 5  # a few rows of padding, as a captured step has
    dev = lambda a: torch.tensor(np.asarray(a, np.int32), device=DEV)  # noqa: E731
    i32 = dict(device=DEV, dtype=torch.int32)
    return dict(case=case, ctx=dev(ctx), new=dev(new), table=dev(table), held=dev(held),
                free=dev(free), count=dev([len(left)]), rows=n,
                row_offsets=torch.empty(B + 1, **i32), seq_lens=torch.empty(B, **i32),
                positions=torch.empty(n, **i32),
                slots=torch.empty(n, device=DEV, dtype=torch.int64),
                held_out=torch.empty(B, **i32), count_out=torch.empty(1, **i32),
                dev_error=torch.zeros(1, **i32))


def _prepare_append(case, seed, g):
    """Keys and values as slices of one fused projection's output, and pages
    scattered over the cache; every 37th row is padding (slot -1)."""
    N, H, D, page = case["rows"], case["kv_heads"], case["dim"], case["page"]
    qkv = torch.randn(N, 6 * H * D, device=DEV, generator=g).to(torch.bfloat16)
    k = qkv[:, 4 * H * D:5 * H * D].view(N, H, D)
    v = qkv[:, 5 * H * D:].view(N, H, D)
    blocks = 2 * (-(-N // page)) + 8
    caches = [torch.randn(blocks, page, H, D, device=DEV, generator=g).to(torch.bfloat16)
              for _ in range(2)]
    at = torch.randperm(blocks, device=DEV, generator=g)
    i = torch.arange(N, device=DEV) + page // 3
    slots = at[i // page] * page + i % page
    slots[36::37] = -1
    return dict(case=case, k=k, v=v, k_cache=caches[0], v_cache=caches[1], slots=slots,
                dev_error=torch.zeros(1, dtype=torch.int32, device=DEV))


def _prepare_attention(case, seed, g):
    """A cache whose pages lie in random order.  Queries are scaled so that the
    scores have a standard deviation of 2.5."""
    B, Hq, Hk, D, page = (case[k] for k in ("batch", "heads", "kv_heads", "dim", "page"))
    ctx, new = lengths(case)
    seq = [a + b for a, b in zip(ctx, new)]
    need = [-(-s // page) for s in seq]
    width, blocks = max(need), sum(need) + 3
    r = np.random.default_rng(seed)
    ids = r.permutation(blocks).astype(np.int32)
    table = np.zeros((B, width), np.int32)
    table[np.arange(width)[None] < np.array(need)[:, None]] = ids[:sum(need)]
    bf = lambda *s: torch.randn(*s, device=DEV, generator=g).to(torch.bfloat16)  # noqa: E731
    N = sum(new)
    dev = lambda a: torch.tensor(np.asarray(a, np.int32), device=DEV)  # noqa: E731
    return dict(case=case, q=bf(N, Hq, D).mul_(2.5), k_cache=bf(blocks, page, Hk, D),
                v_cache=bf(blocks, page, Hk, D), table=dev(table), seq_lens=dev(seq),
                row_offsets=dev(np.concatenate([[0], np.cumsum(new)])), max_new=max(new),
                out=torch.empty(N, Hq, D, dtype=torch.bfloat16, device=DEV),
                lse=torch.empty(N, Hq, device=DEV),
                dev_error=torch.zeros(1, dtype=torch.int32, device=DEV))


# ---------------------------------------------------------------- one pass

def run(s):
    return (_own if own else _plain)[s["case"]["op"]](s)


def _own_sample(s):
    from speculative_decoding_verification_16_gb300 import binding
    binding.spec_verify_sample(s["logits"], s["uniforms"], temperature=s["temperature"],
                               top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"],
                               out_tokens=s["tokens"], out_probs=s["probs"],
                               dev_error=s["dev_error"])
    return {"tokens": s["tokens"], "probs": s["probs"]}


def _own_slots(s):
    from speculative_decoding_verification_16_gb300 import binding
    binding.spec_verify_slots(s["ctx"], s["new"], s["table"], s["held"], s["free"], s["count"],
                              page_size=s["case"]["page"], row_offsets=s["row_offsets"],
                              seq_lens=s["seq_lens"], positions=s["positions"], slots=s["slots"],
                              held_out=s["held_out"], free_count_out=s["count_out"],
                              dev_error=s["dev_error"])
    return {k: s[k] for k in ("table", "free", "row_offsets", "seq_lens", "positions", "slots",
                              "held_out", "count_out")}


def _own_append(s):
    from speculative_decoding_verification_16_gb300 import binding
    binding.spec_verify_append(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"],
                               dev_error=s["dev_error"])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_attention(s):
    from speculative_decoding_verification_16_gb300 import binding
    if "workspace" not in s:  # allocated once and kept, as a server does
        s["workspace"] = binding.alloc_attention_workspace(s["q"])
    binding.spec_verify_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["seq_lens"],
                                  s["row_offsets"], max_len=s["max_new"],
                                  window=s["case"]["window"], out=s["out"], lse=s["lse"],
                                  workspace=s["workspace"], dev_error=s["dev_error"])
    return {"out": s["out"], "lse": s["lse"]}


def _plain_sample(s):
    x, T, V = s["logits"].float(), s["temperature"], s["case"]["vocab"]
    z, order = torch.sort(x / torch.where(T > 0, T, 1.0)[:, None], dim=1, descending=True,
                          stable=True)
    w = torch.exp(z - z[:, :1])
    rank = torch.arange(V, device=x.device)[None]
    k = torch.where((s["top_k"] > 0) & (s["top_k"] < V), s["top_k"], V)[:, None]
    w = torch.where(rank < k, w, 0.0)
    c = torch.cumsum(w, 1)
    top_p = s["top_p"][:, None]
    w = torch.where(((c - w) < top_p * c[:, -1:]) | (top_p >= 1), w, 0.0)
    w = torch.where(w >= s["min_p"][:, None] * w[:, :1], w, 0.0)
    w = torch.where((T > 0)[:, None] | (rank == 0), w, 0.0)
    p = torch.zeros_like(w).scatter_(1, order, w)
    c = torch.cumsum(p, 1)
    t = (c <= s["uniforms"][:, None] * c[:, -1:]).sum(1, keepdim=True).clamp(max=V - 1)
    return {"tokens": t[:, 0].int(), "probs": (p.gather(1, t) / p.sum(1, keepdim=True))[:, 0]}


def _plain_slots(s):
    page, ctx, new, held = s["case"]["page"], s["ctx"].long(), s["new"].long(), s["held"].long()
    table, free = s["table"], s["free"]
    B, width = table.shape
    seq = ctx + new
    need = (seq + page - 1) // page
    col = torch.arange(width, device=table.device)[None]
    back = table[(col >= need[:, None]) & (col < held[:, None])]  # pages given back
    n = s["count"].long()
    free[n + torch.arange(back.numel(), device=table.device)] = back
    n = n + back.numel()
    take = (need - held).clamp(min=0)
    last = torch.cumsum(take, 0)
    k = (last - take)[:, None] + col - held[:, None]
    wanted = (col >= held[:, None]) & (col < need[:, None])
    table.copy_(torch.where(wanted, free[(n - 1 - k).clamp(0, free.numel() - 1)], table))
    offs = torch.cat([torch.zeros_like(new[:1]), torch.cumsum(new, 0)])
    i = torch.arange(s["rows"], device=table.device)
    r = torch.searchsorted(offs, i, right=True) - 1
    pad = r >= B
    r = r.clamp(max=B - 1)
    pos = torch.where(pad, 0, ctx[r] + i - offs[r])
    slots = torch.where(pad, -1, table[r, pos // page].long() * page + pos % page)
    return {"table": table, "free": free, "row_offsets": offs.int(), "seq_lens": seq.int(),
            "positions": pos.int(), "slots": slots, "held_out": need.int(),
            "count_out": (n - last[-1:]).int()}


def _plain_append(s):
    keep = torch.nonzero(s["slots"] >= 0)[:, 0]
    at = s["slots"][keep]
    s["k_cache"].flatten(0, 1)[at] = s["k"][keep]
    s["v_cache"].flatten(0, 1)[at] = s["v"][keep]
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_attention(s):
    q, c = s["q"].float(), s["case"]
    Hq, Hk, D, L, W = c["heads"], c["kv_heads"], c["dim"], s["max_new"], c["window"]
    offs, seq = s["row_offsets"].long(), s["seq_lens"].long()
    new = offs[1:] - offs[:-1]
    B, S = new.numel(), s["table"].shape[1] * c["page"]
    k = s["k_cache"][s["table"].long()].float().view(B, S, Hk, D)
    v = s["v_cache"][s["table"].long()].float().view(B, S, Hk, D)
    j = torch.arange(L, device=q.device)[None]
    row = (offs[:-1, None] + j).clamp(max=q.shape[0] - 1)  # padded to the longest
    pos = seq[:, None] - new[:, None] + j
    t = torch.arange(S, device=q.device)
    seen = (t <= pos[..., None]) & (t < seq[:, None, None])
    if W:
        seen &= t > pos[..., None] - W
    qp = q[row].view(B, L, Hk, Hq // Hk, D)
    x = torch.einsum("blhgd,bthd->bhglt", qp, k) / math.sqrt(D)
    x.masked_fill_(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    x.sub_(m).exp_()
    z = x.sum(-1, keepdim=True)
    o = torch.einsum("bhglt,bthd->blhgd", x, v.masked_fill((t >= seq[:, None])[..., None, None], 0.0))
    o = (o / z[..., 0].permute(0, 3, 1, 2)[..., None]).reshape(B, L, Hq, D)
    lse = (m + torch.log(z))[..., 0].permute(0, 3, 1, 2).reshape(B, L, Hq)
    real = j < new[:, None]
    return {"out": o[real].to(torch.bfloat16), "lse": lse[real]}


_own = {"sample": _own_sample, "slots": _own_slots, "append": _own_append,
        "attention": _own_attention}
_plain = {"sample": _plain_sample, "slots": _plain_slots, "append": _plain_append,
          "attention": _plain_attention}


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "sample":
        return _exact_sample(s)
    if case["op"] == "attention":
        return _exact_attention(s)
    return None  # whole numbers and copies


def _exact_sample(s):
    """Row by row, on the distinct logit values and their counts."""
    tokens, probs = [], []
    for i in range(s["case"]["rows"]):
        x = s["logits"][i].double()
        T, K, P, M, u = (float(s[k][i]) for k in ("temperature", "top_k", "top_p", "min_p",
                                                  "uniforms"))
        if T == 0:
            tokens.append(torch.argmax(x))
            probs.append(torch.ones((), dtype=torch.float64, device=x.device))
            continue
        val, inv, cnt = torch.unique(x, return_inverse=True, return_counts=True)
        val, cnt = val.flip(0), cnt.flip(0).double()  # best first
        inv = val.numel() - 1 - inv
        each = torch.exp((val - val[0]) / T)
        left = float(K) if 0 < K < x.numel() else float(x.numel())
        before = torch.cumsum(cnt, 0) - cnt
        cnt = torch.minimum(cnt, (left - before).clamp(min=0))  # after top-k
        mass = cnt * each
        if P < 1:
            short = P * mass.sum() - (torch.cumsum(mass, 0) - mass)
            cnt = torch.minimum(cnt, torch.ceil(short / each).clamp(min=0))
        cnt = torch.where(each >= M, cnt, 0.0)
        last = int((cnt > 0).sum()) - 1
        keep = inv < last
        ties = torch.nonzero(inv == last)[:int(cnt[last]), 0]
        keep[ties] = True
        w = torch.where(keep, torch.exp((x - val[0]) / T), 0.0)
        c = torch.cumsum(w, 0)
        t = torch.searchsorted(c, (u * c[-1]).reshape(1), right=True)[0]
        tokens.append(t)
        probs.append(w[t] / w.sum())
    return {"tokens": torch.stack(tokens).int(), "probs": torch.stack(probs)}


def _exact_attention(s):
    """Request by request, on the keys that its last row can see."""
    c = s["case"]
    Hk, D, page = c["kv_heads"], c["dim"], c["page"]
    G = c["heads"] // Hk
    offs, seq = s["row_offsets"].tolist(), s["seq_lens"].tolist()
    outs, lses = [], []
    for b, n in enumerate(seq):
        at = torch.arange(n, device=DEV)
        rows = s["table"][b].long()[at // page] * page + at % page
        k = s["k_cache"].flatten(0, 1)[rows].double().transpose(0, 1)  # [Hk, n, D]
        v = s["v_cache"].flatten(0, 1)[rows].double().transpose(0, 1)
        l = offs[b + 1] - offs[b]
        o = torch.empty(l, Hk, G, D, dtype=torch.float64, device=DEV)
        lse = torch.empty(l, Hk, G, dtype=torch.float64, device=DEV)
        for a in range(0, l, 512):  # for memory
            e = min(l, a + 512)
            q = s["q"][offs[b] + a:offs[b] + e].double().view(e - a, Hk, G, D)
            x = torch.matmul(q.permute(1, 2, 0, 3).reshape(Hk, G * (e - a), D),
                             k.transpose(1, 2)).view(Hk, G, e - a, n) / math.sqrt(D)
            far = (n - l + torch.arange(a, e, device=DEV))[:, None] - at[None]
            hide = far < 0
            if c["window"]:
                hide |= far >= c["window"]
            x = x.masked_fill(hide, -math.inf)
            top = torch.logsumexp(x, -1)
            p = torch.exp(x - top[..., None]).view(Hk, G * (e - a), n)
            o[a:e] = torch.matmul(p, v).view(Hk, G, e - a, D).permute(2, 0, 1, 3)
            lse[a:e] = top.permute(2, 0, 1)
        outs.append(o.reshape(l, Hk * G, D))
        lses.append(lse.reshape(l, Hk * G))
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}
