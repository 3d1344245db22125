"""GPU parity of rotary positions, 8-bit caches and trees at the sizes, magnitudes and
paths where they can go wrong."""

import math

import numpy as np
import pytest
import torch

from oracle import tree_oracle as T
from test_gpu_tree import BF, DEV, E4, F32, dev_error, i32, np64, pack, random_tree

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- attention over given numbers

def paged(rng, rows, page, K, D, dtype):
    """Rows of every request, [n, K, D] as they shall lie in the cache (bf16, fp32, or the
    codes' numbers), and their exponents [n, K] or None, into pages in random order:
    cache, exponents, table."""
    need = [-(-len(x) // page) for x, _ in rows]
    ids = rng.permutation(sum(need) + 1)
    table, at = np.zeros((len(rows), max(need) + 1), np.int64), 0
    cache = torch.zeros(len(ids) * page, K, D, dtype=dtype if dtype != E4 else F32)
    exps = torch.zeros(len(ids) * page, K, dtype=torch.int8)
    for r, (x, e) in enumerate(rows):
        table[r, :need[r]] = ids[at:at + need[r]]
        at += need[r]
        t = np.arange(len(x))
        slot = torch.tensor(table[r, t // page] * page + t % page)
        cache[slot] = torch.tensor(np.asarray(x), dtype=cache.dtype)
        if e is not None:
            exps[slot] = torch.tensor(np.asarray(e), dtype=torch.int8)
    cache = cache.view(len(ids), page, K, D).to(DEV).to(dtype)
    return cache, exps.view(len(ids), page, K).to(DEV) if dtype == E4 else None, table


def check_numbers(lib, dtype, lens, q, keys, vals, page, scale, tree=False, window=0, seed=0, slack=0.0,
                  lse_slack=0.0):
    """q [N, Hq, D] and per request keys and values ([n, K, D] numbers or codes, [n, K]
    exponents or None; dtype E4 for codes) against the oracle.  Tolerances: what the
    callers give, beside 2^-7 sum p |v| (fp32 2^-12).  Over codes a small weight in fp16
    loses up to 2^-25 where the row's largest w is 2^7 or more, w a key's weight p times
    2^e, e the largest exponent of its tile's values; operands are at most 448 2^e, so a key
    loses at most 2^-32 448 max w."""
    rng = np.random.default_rng(seed)
    K, D = keys[0][0].shape[1:]
    G = q.shape[1] // K
    kc, ke, table = paged(np.random.default_rng(seed), keys, page, K, D, dtype)
    vc, ve, _ = paged(np.random.default_rng(seed), vals, page, K, D, dtype)
    seq, new = [n for n, _ in lens], [l for _, l in lens]
    seen, sets = [], []
    for n, l in lens:
        s = np.tril(np.ones((l, n), bool), n - l)
        if window:
            s &= ~np.tril(np.ones((l, n), bool), n - l - window)
        if tree:
            anc = T.ancestors(random_tree(rng, l)) if l else []
            s = np.zeros((l, n), bool)
            s[:, :n - l] = True
            for i in range(l):
                s[i, [n - l + j for j in anc[i]]] = True
            sets += anc
        seen.append(s)
    mask = pack(sets, (max(new) + 31) // 32) if tree else None
    err = dev_error()
    out, lse = lib.spec_verify_attention(q, kc, vc, i32(table), i32(seq), i32(np.concatenate([[0], np.cumsum(new)])),
                                         max_len=max(new), window=window, scale=scale, want_lse=True, key_exps=ke,
                                         value_exps=ve, tree_mask=mask, dev_error=err)
    assert err.item() == 0
    o, x, qn, at = np64(out), np64(lse), np64(q), 0
    for r, (n, l) in enumerate(lens):
        k, v = (np.asarray(a[r][0], np.float64) * (1.0 if a[r][1] is None else np.exp2(np.asarray(a[r][1], np.float64))[..., None])
                for a in (keys, vals))
        want, wl, mag = T.attention(qn[at:at + l], k, v, scale, seen[r])
        tol = mag * ((2.0 ** -12 if dtype == F32 else 2.0 ** -7) + slack) + 1e-30
        if dtype == E4:
            e = np.asarray(vals[r][1], np.float64)
            most = np.stack([e[t // 64 * 64:t // 64 * 64 + 64].max(0) for t in range(n)])
            for j in range(l):
                t = np.flatnonzero(seen[r][j])
                for h in range(K * G):
                    p = np.exp(scale * (k[t, h // G] @ qn[at + j, h]) - wl[j, h])
                    tol[j, h] += 2.0 ** -32 * 448 * len(t) * np.max(p * np.exp2(most[t, h // G]), initial=0.0)
        got, gl = o[at:at + l], x[at:at + l]
        assert np.isfinite(got).all(), (r, n, l, "not finite")
        assert (np.abs(got - want) <= tol).all(), (r, n, l, np.max(np.abs(got - want) / tol))
        assert (np.abs(gl - wl) <= 2.0 ** -12 + 2.0 ** -21 * np.abs(wl) + lse_slack).all(), \
            (r, n, l, np.max(np.abs(gl - wl)))
        at += l
    return out, lse


def some_codes(rng, *shape, most=192.0):
    """Numbers that codes hold, from -most to most, evenly over their exponents."""
    m = rng.integers(8, 16, shape) / 8.0
    return np.minimum(np.exp2(rng.integers(-3, int(math.log2(most)) + 1, shape)) * m, most) * rng.choice([-1, 1], shape)


# Value exponents in steps from tile to tile.  The sum of weights holds the keys of all
# tiles alike, however small their values are: lse is as exact as ever (2^-12), and the
# output is off by 2^-7 sum p |v|.
STEPS = {"rising": [-100, -20, 45, 60, 110], "falling": [110, 60, 45, -20, -100], "up and down": [60, -100, 60, -100],
         "down and up": [-100, 60], "zeros first": [None, 60], "zeros last": [60, None], "zeros between": [30, None, 100]}


@pytest.mark.parametrize("steps", list(STEPS))
@pytest.mark.parametrize("D,G,tree", [(64, 1, False), (128, 4, False), (256, 2, False), (128, 4, True), (64, 40, False)])
def test_codes_of_tiles_far_apart(cuda_lib, steps, D, G, tree):
    """Tiles of 64 tokens whose values differ by up to 2^210, in any order, within a
    worker's run and across the cut between two."""
    rng = np.random.default_rng(len(steps) + D)
    K, page, pattern = 2, 16, STEPS[steps]
    lens = [(64 * len(pattern), 2), (128, 3), (3000, 4), (9001, 1)]
    q = torch.tensor(rng.standard_normal((sum(l for _, l in lens), K * G, D)), device=DEV).to(BF)
    keys, vals = [], []
    for n, _ in lens:
        keys.append((some_codes(rng, n, K, D, most=2.0), np.zeros((n, K), int)))
        e = [pattern[t // 64 % len(pattern)] for t in range(n)]
        v = some_codes(rng, n, K, D)
        v[[x is None for x in e]] = 0
        vals.append((v, np.repeat(np.array([-100 if x is None else x for x in e])[:, None], K, 1)))
    check_numbers(cuda_lib, E4, lens, q, keys, vals, page, D ** -0.5, tree=tree)
    if not tree:
        check_numbers(cuda_lib, E4, lens, q, keys, vals, page, D ** -0.5, window=100)
