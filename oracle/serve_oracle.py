"""Plain fp64 / integer restatement of the paged serving operators: sampling
with per-row filters, block tables and slot maps, and attention of a chunk of
new tokens over a paged cache.  One row or request at a time; shares no code
with the kernels."""

from __future__ import annotations

import numpy as np


def _draw(ids, w, u, eps):
    """Tokens that an inverse CDF over ascending ids may give when running
    masses are off by up to eps, with their probabilities."""
    order = np.argsort(ids, kind="stable")
    ids, w = ids[order], w[order]
    p = w / w.sum()
    c = np.cumsum(p)
    hit = (c > u - eps) & (c - p <= u + eps) & (p > 0)
    return {int(i): float(q) for i, q in zip(ids[hit], p[hit])}


def sample_row(x, T=1.0, top_k=0, top_p=1.0, min_p=0.0, u=0.5, eps=1e-6):
    """{token: [its probabilities]} of the tokens that the row may give: one,
    unless a top-p cut, a min-p cut or the draw lies within eps of a tie."""
    x = np.asarray(x, np.float64) + 0.0  # -0 becomes +0
    if T == 0:
        return {int(np.argmax(x)): [1.0]}
    order = np.lexsort((np.arange(x.size), -x))
    w = np.exp((x[order] - x[order[0]]) / T)
    if 0 < top_k < x.size:
        order, w = order[:top_k], w[:top_k]
    sizes = {w.size}
    if top_p < 1:
        c = np.cumsum(w) / w.sum()
        sizes = {int(np.searchsorted(c, top_p + d, side="left")) + 1 for d in (-eps, 0.0, eps)}
        sizes = {min(n, w.size) for n in sizes}
    out = {}
    for n in sizes:
        for d in (-eps, 0.0, eps):
            m = max(1, min(n, int((w >= min_p + (d if min_p > 0 else 0.0)).sum())))
            for t, p in _draw(order[:m], w[:m], u, eps).items():
                out.setdefault(t, []).append(p)
    return out


def slots(ctx, new, table, held, free, count, page, n_rows):
    """The state after a step: dict of table, free, held, count, row_offsets,
    seq_lens, positions, slots and errors ('len', 'blocks')."""
    B, width = table.shape
    table, free, err = table.copy(), list(free[:count]), set()
    new = list(new)
    need = []
    for r in range(B):
        ok = 0 <= new[r] <= n_rows
        if not ok:
            new[r] = 0
        n = -(-(int(ctx[r]) + int(new[r])) // page)
        ok = ok and ctx[r] >= 0 and 0 <= held[r] <= width and n <= width
        if not ok:
            err.add("len")
        need.append(n if ok else None)
    for r in range(B):
        if need[r] is not None:
            free += [int(table[r, c]) for c in range(need[r], held[r])]
    stack = list(free)  # the list's memory: pops leave the ids in place
    held_out, short = [int(h) for h in held], False
    for r in range(B):
        if need[r] is None:
            continue
        take = max(need[r] - held[r], 0)
        if take and (short or take > len(free)):
            short = True
            err.add("blocks")
            continue
        for c in range(held[r], held[r] + take):
            table[r, c] = free.pop()
        held_out[r] = need[r]
    offs = np.concatenate([[0], np.cumsum(new)])
    pos, slot = np.zeros(n_rows, np.int64), np.full(n_rows, -1, np.int64)
    for r in range(B):
        if need[r] is None:
            continue
        for i in range(int(new[r])):
            p = int(ctx[r]) + i
            pos[offs[r] + i] = p
            if p // page < held_out[r]:
                slot[offs[r] + i] = int(table[r, p // page]) * page + p % page
    # no length for a request whose pages do not hold its tokens
    seq = [int(ctx[r]) + int(new[r]) if need[r] is not None and held_out[r] == need[r] else -1
           for r in range(B)]
    return dict(table=table, stack=stack, count=len(free), held=held_out, row_offsets=offs,
                seq_lens=seq, positions=pos, slots=slot, errors=err)


def attention_request(q, k, v, scale, window=0):
    """One request: q [l, Hq, D] are the last l of n tokens, k and v [n, Hk, D].
    Returns out [l, Hq, D], lse [l, Hq] and mag [l, Hq, D] = sum p |v|, what the
    roundings of the weights scale with."""
    l, Hq, D = q.shape
    n, Hk, _ = k.shape
    out, mag = np.zeros((l, Hq, D)), np.zeros((l, Hq, D))
    lse = np.full((l, Hq), -np.inf)
    for j in range(l):
        p = n - l + j
        lo = max(0, p - window + 1) if window > 0 else 0
        if p < lo:
            continue
        for h in range(Hk):
            g = slice(h * Hq // Hk, (h + 1) * Hq // Hk)
            s = scale * (q[j, g] @ k[lo:p + 1, h].T)
            m = s.max(1, keepdims=True)
            e = np.exp(s - m)
            z = e.sum(1, keepdims=True)
            out[j, g] = e @ v[lo:p + 1, h] / z
            mag[j, g] = e @ np.abs(v[lo:p + 1, h]) / z
            lse[j, g] = (m + np.log(z))[:, 0]
    return out, lse, mag
