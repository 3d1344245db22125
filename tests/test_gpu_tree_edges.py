"""GPU parity of rotary positions, 8-bit caches and trees at the sizes, magnitudes and
paths where they can go wrong."""

import math

import numpy as np
import pytest
import torch

from oracle import tree_oracle as T
from test_gpu_tree import (BF, DEV, E4, F32, check_attention, check_rope_append, close, copy_state, dev_error, heads_of,
                           i32, make_caches, np64, pack, random_tree, some_freqs, tree_state, tree_step, values)

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


@pytest.mark.parametrize("D,G,tree", [(64, 1, False), (128, 4, False), (128, 4, True), (256, 2, True)])
def test_codes_of_tiles_far_apart_that_rows_do_not_see(cuda_lib, D, G, tree):
    """Rows that see nothing of a tile whose values are far smaller, or larger, than those
    that they see."""
    rng = np.random.default_rng(D + G)
    lens = [(70, 55), (130, 100), (200, 140), (65, 65)]
    for pattern in ([105, -100], [-100, 105], [100, -90, 100, -90], [-90, 60, -90, 60]):
        q = torch.tensor(rng.standard_normal((sum(l for _, l in lens), 2 * G, D)), device=DEV).to(BF)
        keys, vals = [], []
        for n, _ in lens:
            keys.append((some_codes(rng, n, 2, D, most=2.0), np.zeros((n, 2), int)))
            e = np.array([pattern[t // 64 % len(pattern)] for t in range(n)])
            vals.append((some_codes(rng, n, 2, D), np.repeat(e[:, None], 2, 1)))
        check_numbers(cuda_lib, E4, lens, q, keys, vals, 16, D ** -0.5, tree=tree)
        if not tree:
            check_numbers(cuda_lib, E4, lens, q, keys, vals, 16, D ** -0.5, window=20)


# Scores 2^17 + d of one unit each, exact in every type and in 32 bits: q k is 2^8 2^9 and
# a product of small whole numbers d.  Their differences are exact too, so weights are as
# far off as at any scale.  Over 16- and 32-bit caches scores are scaled before they are
# subtracted while |score| log2 e is below 2^20: three roundings to 2^-24 of it.
def counted(rng, lens, K, G, D, dtype):
    N = sum(l for _, l in lens)
    q = torch.zeros(N, K * G, D, device=DEV, dtype=dtype if dtype != E4 else BF)
    q[..., 0] = 256.0
    q[..., D - 1] = torch.tensor(rng.choice([1.0, 2.0, -1.0], (N, K * G)), device=DEV).to(q.dtype)
    keys, vals = [], []
    for n, _ in lens:
        e = rng.integers(1, 5, (n, K))
        k = np.zeros((n, K, D))
        k[..., 0], k[..., D - 1] = 512.0, rng.integers(0, 8, (n, K))
        v = some_codes(rng, n, K, D)
        if dtype == E4:
            tiles = rng.integers(-9, 9, (-(-n // 64), K))
            keys.append((k / np.exp2(e)[..., None], e))
            vals.append((v, tiles[np.arange(n) // 64] + rng.integers(-3, 1, (n, K))))
        else:
            keys.append((k, None))
            vals.append((v, None))
    return q, keys, vals


LARGE = [[(300, 2), (40, 3), (3000, 5), (64, 64)], [(9001, 1), (700, 1)], [(700, 70), (90, 33)]]


@pytest.mark.parametrize("scale", [0.5, -0.5, 40.0, 2.0 ** 11, -2.0 ** 13, 1e9, 1e30, -1e30])
@pytest.mark.parametrize("D,G", [(64, 1), (128, 4), (256, 2)])
def test_codes_of_large_scores(cuda_lib, scale, D, G):
    """The best keys of scores up to 10^35 share a row's weight, across tiles whose powers
    of two differ, rescalings and the join of parts."""
    rng = np.random.default_rng(D)
    for i, lens in enumerate(LARGE):
        q, keys, vals = counted(rng, lens, 2, G, D, E4)
        check_numbers(cuda_lib, E4, lens, q, keys, vals, 16, scale, tree=False, seed=i)
        check_numbers(cuda_lib, E4, lens, q, keys, vals, 16, scale, tree=True, seed=i)


@pytest.mark.parametrize("size", [2e4, 7e5, 3e7, 7e8, 3e10, 1e20])
def test_codes_of_large_mixed_scores(cuda_lib, size):
    """Random products at scales where a row's scores reach `size`.  A score is off by at
    most D 2^-24 sum |q k| |scale|; where the best key leads by 64 of those and 64 more, the
    output is its value."""
    rng = np.random.default_rng(7)
    n, l, K, G, D = 3001, 5, 2, 4, 64
    scale = size / 40.0
    q = torch.tensor(rng.standard_normal((l, K * G, D)), device=DEV).to(BF)
    k, ke = some_codes(rng, n, K, D, most=4.0), np.zeros((n, K), int)
    v, ve = some_codes(rng, n, K, D), np.repeat(rng.integers(-9, 9, (47, K)), 64, 0)[:n]
    kc, e0, table = paged(np.random.default_rng(1), [(k, ke)], 16, K, D, E4)
    vc, e1, _ = paged(np.random.default_rng(1), [(v, ve)], 16, K, D, E4)
    out, lse = cuda_lib.spec_verify_attention(q, kc, vc, i32(table), i32([n]), i32([0, l]), max_len=l, scale=scale,
                                              key_exps=e0, value_exps=e1, want_lse=True)
    assert bool(out.isfinite().all()) and bool(lse.isfinite().all())
    clear, qn = 0, np64(q)
    for j in range(l):
        for h in range(K * G):
            m = n - l + j + 1
            s = scale * (k[:m, h // G] @ qn[j, h])
            off = D * 2.0 ** -24 * scale * (np.abs(k[:m, h // G]) @ np.abs(qn[j, h])).max()
            best = int(s.argmax())
            s[best], top = -np.inf, s[best]
            assert abs(lse[j, h].item() - top) <= 2 * off + 2.0 ** -22 * abs(top) + 9
            if top - s.max() > 64 * off + 64:
                clear += 1
                want = v[best, h // G] * 2.0 ** float(ve[best, h // G])
                assert (np.abs(np64(out[j, h]) - want) <= 2.0 ** -8 * np.abs(want)).all()
    assert clear >= 20


def test_codes_infinite_scores_and_the_ends_of_the_scales(cuda_lib):
    """Scores far apart, the largest finite scales, whose scores leave fp32, and scale 0
    under products of any size."""
    n, D, page = 300, 64, 16
    rng = np.random.default_rng(2)
    v, ve = some_codes(rng, n, 1, D), rng.integers(-9, 9, (n, 1))
    vc, e1, table = paged(np.random.default_rng(1), [(v, ve)], page, 1, D, E4)
    a = (i32(table), i32([n]), i32([0, 2]))
    q = torch.zeros(2, 1, D, device=DEV, dtype=BF)
    value = v[:, 0] * np.exp2(ve.astype(np.float64))

    def call(k, ke, scale):
        kc, e0, _ = paged(np.random.default_rng(1), [(k, ke)], page, 1, D, E4)
        out, lse = cuda_lib.spec_verify_attention(q, kc, vc, *a, max_len=2, scale=scale, key_exps=e0, value_exps=e1,
                                                  want_lse=True)
        return np64(out)[:, 0], np64(lse)[:, 0]
    k, ke = np.zeros((n, 1, D)), np.zeros((n, 1), int)
    # products up to 1e31
    q[:, 0, 0] = 1.0
    k[:, 0, 0], ke[:] = 8.0 + np.arange(n) % 8, np.minimum(np.arange(n) // 8, 30)[:, None] + 70
    out, lse = call(k, ke, 1.0)
    best = 247  # the largest product, first of those that repeat
    top = k[:, 0, 0] * np.exp2(ke[:, 0].astype(np.float64))
    for j in range(2):
        ties = np.flatnonzero(top[:n - 1 + j] == top[best])
        want, mag = value[ties].mean(0), np.abs(value[ties]).mean(0)
        assert (np.abs(out[j] - want) <= 2.0 ** -7 * mag).all()
        assert abs(lse[j] - top[best]) <= 2.0 ** -21 * top[best]
    # scale 0: all keys alike
    out, lse = call(k, ke, 0.0)
    for j in range(2):
        want, mag = value[:n - 1 + j].mean(0), np.abs(value[:n - 1 + j]).mean(0)
        assert (np.abs(out[j] - want) <= 2.0 ** -7 * mag).all()
        assert abs(lse[j] - math.log(n - 1 + j)) <= 2.0 ** -12
    # scales whose product with log2 e leaves fp32: products of 0 and of 1, and of 0, 1 and 4
    for scale in (3e38, -3e38):
        q[:, 0, 0] = math.copysign(1.0, scale)
        for more in (False, True):
            k[:], ke[:] = 0, 0
            k[120, 0, 0] = 1.0
            best = 120
            if more:
                k[40, 0, 0], best = 4.0, 40
            out, _ = call(k, ke, scale)
            assert (out == np64(torch.tensor(value[best]).to(BF))).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("scale", [0.5, -0.5, 40.0, 2.0 ** 11, 1e9, -1e30])
@pytest.mark.parametrize("D,G", [(64, 1), (128, 4), (256, 2)])
def test_trees_of_large_scores(cuda_lib, dtype, scale, D, G):
    rng = np.random.default_rng(D)
    for i, lens in enumerate(LARGE):
        q, keys, vals = counted(rng, lens, 2, G, D, dtype)
        # three roundings of the score, twice in a weight and twice in the sum
        e = 2.0 ** 17 * abs(scale) * 2.0 ** -24 * 3 if abs(scale) < 40 else 0.0
        check_numbers(cuda_lib, dtype, lens, q, keys, vals, 16, scale, tree=True, seed=i, slack=4 * e, lse_slack=2 * e)


# ---------------------------------------------------------------- paths and moves

@pytest.mark.parametrize("dtype", [BF, E4])
def test_tree_move_leaves_row_0(cuda_lib, dtype):
    """Rows 1 .. accept_len are moved to; a path that starts behind row 0 leaves the last
    accepted token's keys and values as they are."""
    L, page, K, D, l = 3, 4, 2, 32, 7
    g = torch.Generator(device=DEV).manual_seed(1)
    c = [torch.randint(0, 120, (L, 4, page, K, D), device=DEV, generator=g, dtype=torch.uint8).view(E4) if dtype == E4
         else torch.randn(L, 4, page, K, D, device=DEV, generator=g).to(dtype) for _ in range(2)]
    e = [torch.randint(-9, 9, (L, 4, page, K), device=DEV, generator=g, dtype=torch.int8) if dtype == E4 else None
         for _ in range(2)]
    slots = torch.tensor([9, 3, 12, 0, 7, 15, 5, 1, 2], device=DEV)
    path, n, offs = [2, 4, 5, -1, -1, -1, -1, 1, -1], [2, 0], [0, l, 9]
    raw = [x.view(torch.uint8) if dtype == E4 else x for x in c] + [x for x in e if x is not None]
    want = [x.clone() for x in raw]
    for x, w in zip(raw, want):
        for j in (1, 2):
            s, d = int(slots[path[j]]), int(slots[j])
            w[:, d // page, d % page] = x[:, s // page, s % page]
    err = dev_error()
    cuda_lib.spec_verify_tree_move(i32(path), i32(n), i32(offs), slots, *c, max_len=8, key_exps=e[0], value_exps=e[1],
                                   dev_error=err)
    assert err.item() == 0
    for x, w in zip(raw, want):
        assert torch.equal(x, w)


def test_tree_move_of_a_request_without_rows(cuda_lib):
    """Without rows the length is -1; any other is out of range."""
    c = torch.zeros(2, 4, 1, 8, device=DEV)
    for n, flag in ((-1, 0), (0, cuda_lib.SV_DEVERR_LEN), (1, cuda_lib.SV_DEVERR_LEN)):
        err = dev_error()
        cuda_lib.spec_verify_tree_move(i32([0, -1]), i32([n, 0]), i32([0, 0, 2]), torch.arange(2, device=DEV), c,
                                       c.clone(), max_len=4, dev_error=err)
        assert err.item() == flag, n


def test_tree_accept_stops_where_no_token_was_sampled(cuda_lib):
    """A row whose token could not be sampled (-1) is followed by no row, one of a drafter
    that failed too among them."""
    tokens, nxt = [5, -1, 3, 4, 5, 6], [-1, 3, 4, 7, 6, -1]
    parents, offs = [-1, 0, 1, 2, -1, 0], [0, 4, 6]
    out, path, n = cuda_lib.spec_verify_tree_accept(i32(tokens), i32(nxt), i32(parents), i32(offs), max_len=4)
    assert n.tolist() == [0, 1]
    assert path.tolist() == [0, -1, -1, -1, 0, 1] and out.tolist() == [-1] * 4 + [6, -1]


# ---------------------------------------------------------------- rotary positions of many rows

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("D,R", [(64, 64), (128, 128), (256, 64), (80, 40), (128, 24), (96, 0)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_append_of_many_rows(cuda_lib, dtype, quant, D, R, interleaved):
    """Rows enough for a warp each, and heads enough for several rounds of a warp's loads."""
    check_rope_append(cuda_lib, dtype, quant, 1300, 21, 9, D, R, 16, "heads" if interleaved else "tokens", False, D + R,
                      interleaved=interleaved)


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("n,H,K,page,strided", [(1300, 0, 3, 7, True), (1501, 5, 1, 1, True), (1216, 17, 5, 64, False)])
def test_rope_append_of_many_rows_of_any_layout(cuda_lib, quant, n, H, K, page, strided):
    for dtype, D, R, layout in ((BF, 128, 64, "heads"), (F32, 64, 64, "tokens"), (BF, 72, 24, "tokens")):
        check_rope_append(cuda_lib, dtype, quant, n, H, K, D, R, page, layout, strided, n + D)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D,R", [(128, 128), (64, 24), (256, 256)])
def test_rope_of_many_rows_and_heads(cuda_lib, dtype, D, R):
    rng = np.random.default_rng(D)
    g = torch.Generator(device=DEV).manual_seed(D)
    for interleaved in (False, True):
        x = heads_of(g, 2500, 37, D, dtype, interleaved)
        f, pos = some_freqs(rng, R // 2), rng.integers(0, 100000, 2500)
        kw = dict(interleaved=interleaved, amplitude=1.25)
        freqs = torch.tensor(f.view(np.int64), device=DEV)
        out = cuda_lib.spec_verify_rope(x, i32(pos), freqs, **kw)
        close(out, *T.rope(np64(x), pos, f, interleaved, 1.25), dtype)
        cuda_lib.spec_verify_rope(x, i32(pos), freqs, out=x, **kw)  # in place
        assert torch.equal(x, out)


@pytest.mark.parametrize("quant", [False, True])
def test_rope_append_of_many_rows_skips_slots(cuda_lib, quant):
    """Slots below 0 and past the cache leave it as it is, among rows of all others."""
    n, K, D, page, blocks = 4000, 2, 64, 16, 200
    rng = np.random.default_rng(3)
    k = torch.randn(n, K, D, device=DEV, generator=torch.Generator(device=DEV).manual_seed(3)).to(BF)
    slots = np.full(n, -1)
    slots[1::2] = blocks * page + rng.integers(0, 2 ** 40, n // 2)
    on = rng.permutation(n)[:1500]
    slots[on] = rng.permutation(blocks * page)[:1500]
    kc = torch.full((blocks, page, K, D), 3.0, device=DEV).to(E4 if quant else BF)
    vc = kc.clone() if not quant else kc.view(torch.uint8).clone().view(E4)
    e = [torch.full((blocks, page, K), 9, dtype=torch.int8, device=DEV) if quant else None for _ in range(2)]
    err = dev_error()
    cuda_lib.spec_verify_append(k, -k, torch.tensor(slots, device=DEV), kc, vc, key_exps=e[0], value_exps=e[1],
                                dev_error=err) if quant else \
        cuda_lib.spec_verify_rope_append(None, k, -k, None, None, torch.tensor(slots, device=DEV), kc, vc, dev_error=err)
    assert err.item() == cuda_lib.SV_DEVERR_PAGE
    b, t = slots[on] // page, slots[on] % page
    off = torch.ones(blocks, page, dtype=torch.bool, device=DEV)
    off[torch.tensor(b, device=DEV), torch.tensor(t, device=DEV)] = False
    for c, x, s in ((kc, e[0], 1.0), (vc, e[1], -1.0)):
        assert bool((c.to(F32)[off] == 3).all()) and (x is None or bool((x[off] == 9).all()))
        got, want = values(c, x)[b, t], s * np64(k)[on]
        tol = 0 * want if not quant else np.maximum(
            2.0 ** -4 * np.abs(want), 2.0 ** -10 * np.exp2(x.cpu().numpy().astype(np.float64))[b, t][..., None])
        assert (np.abs(got - want) <= tol * (1 + 1e-9)).all()


# ---------------------------------------------------------------- one stream of rows

@pytest.mark.parametrize("codes,tree", [(True, False), (True, True), (False, True)])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [1, 5, 8, 24, 64, 192])
def test_pages_of_one_stream(cuda_lib, page, D, codes, tree):
    """At most 128 rows an item, contexts of many turns of the ring, items that are cut."""
    check_attention(cuda_lib, BF, codes, tree, [(5001, 16), (777, 9), (64, 1), (2600, 5), (16, 16)], 2, 5, D, page,
                    layout="heads" if page % 2 else "tokens", seed=page)
    check_attention(cuda_lib, BF, codes, tree, [(3000, 1), (9001, 1), (130, 1)], 1, 8, D, page, seed=page + 1)


# ---------------------------------------------------------------- together

def test_a_tree_step_s_attention_against_the_oracle(cuda_lib):
    """Slots, masks, rotated queries and an 8-bit cache: what each row of the step's trees
    attends to."""
    st = tree_state(cuda_lib, 8)
    n, B, K, G, D, new, ctx, par = st["nums"]
    err = st["err"]
    plan = cuda_lib.spec_verify_slots(st["ctx"], st["new"], st["table"], st["held"], st["free"], st["count"],
                                      page_size=16, n_rows=st["rows"], dev_error=err)
    pos, mask = cuda_lib.spec_verify_tree(st["parents"], plan.seq_lens, plan.row_offsets, max_len=64, dev_error=err)
    offs = np.concatenate([[0], np.cumsum(new)])
    for window in (0, 50):
        q = cuda_lib.spec_verify_rope_append(st["q"][0], st["k"][0], st["v"][0], pos, st["freqs"], plan.slots,
                                             st["kc"][0], st["vc"][0], key_exps=st["ke"][0], value_exps=st["ve"][0],
                                             dev_error=err)
        out, _ = cuda_lib.spec_verify_attention(q, st["kc"][0], st["vc"][0], st["table"], plan.seq_lens,
                                                plan.row_offsets, max_len=64, key_exps=st["ke"][0],
                                                value_exps=st["ve"][0], tree_mask=mask, positions=pos, window=window,
                                                dev_error=err)
        assert int(err) == 0
        keys, vals = values(st["kc"][0], st["ke"][0]), values(st["vc"][0], st["ve"][0])
        table, qn, o = st["table"].cpu().numpy(), np64(q), np64(out)
        for r in range(B):
            l, c = int(new[r]), int(ctx[r])
            t = np.arange(c + l)
            k, v = (x[table[r, t // 16], t % 16] for x in (keys, vals))
            anc = T.ancestors([int(p) for p in par[offs[r]:offs[r + 1]]])
            seen = np.zeros((l, c + l), bool)
            for i in range(l):
                seen[i, max(0, c + len(anc[i]) - window) if window else 0:c] = True
                seen[i, [c + j for j in anc[i]]] = True
            want, _, mag = T.attention(qn[offs[r]:offs[r + 1]], k, v, D ** -0.5, seen)
            tol = 2.0 ** -7 * mag + np.repeat(2.0 ** -32 * np.abs(v).sum(0), G, 0) + 1e-30
            assert (np.abs(o[offs[r]:offs[r + 1]] - want) <= tol).all()


def test_a_tree_step_over_memory_in_any_state(cuda_lib):
    """What the step's calls allocate may hold anything before; rows behind the last request
    keep it."""
    first = tree_state(cuda_lib, 11)
    rows = int(first["nums"][5].sum())
    stream, want = torch.cuda.Stream(), None
    for i, x in enumerate((0.0, float("nan"), 3e38, float("nan"))):
        st = copy_state(first)
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            for size in (1 << 10, 1 << 14, 1 << 18, 1 << 20, 1 << 22):
                waste = [torch.full((size,), x, device=DEV) for _ in range(8)]
                del waste
        got = tree_step(cuda_lib, st, stream) if i != 1 else tree_step(cuda_lib, st)
        torch.cuda.synchronize()
        assert int(st["err"]) == 0
        got = [y[:rows] for y in got[:2]] + got[2:]
        want = want or [y.clone() for y in got]
        for a, b in zip(got, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("codes,tree", [(True, False), (True, True), (False, True)])
@pytest.mark.parametrize("G,l,D", [(8, 1, 128), (4, 16, 128), (4, 64, 64)])
def test_calls_repeat_bit_by_bit(cuda_lib, codes, tree, G, l, D):
    """Whatever the workspace and the chip's memories held before."""
    g, rng = torch.Generator(device=DEV).manual_seed(l), np.random.default_rng(l)
    lens = [int(n) for n in rng.integers(l, 6000, 9)]
    need = [-(-n // 16) for n in lens]
    caches, exps = make_caches(g, rng, sum(need), 16, 2, D, BF, codes, "tokens")
    table = np.zeros((9, max(need)), np.int64)
    ids = np.split(rng.permutation(sum(need)), np.cumsum(need)[:-1])
    for r in range(9):
        table[r, :need[r]] = ids[r]
    q = torch.randn(9 * l, 2 * G, D, device=DEV, generator=g).to(BF)
    mask = pack([a for _ in range(9) for a in T.ancestors(random_tree(rng, l))], (l + 31) // 32) if tree else None
    args = (*caches, i32(table), i32(lens), i32(np.arange(10) * l))
    ws = cuda_lib.alloc_attention_workspace(q)
    kw = dict(max_len=l, key_exps=exps[0], value_exps=exps[1], tree_mask=mask, want_lse=True, workspace=ws)
    want = None
    for i in range(12):
        ws.copy_(torch.randint(0, 256, ws.shape, device=DEV, generator=g, dtype=torch.uint8) if i % 3 else
                 torch.full_like(ws, 255))
        if i % 2:  # operands of NaN and infinities stay behind
            cuda_lib.spec_verify_attention(q * float("nan") if i % 4 == 1 else q * 1e38 * 10, *args, **{**kw, "workspace": None})
        got = cuda_lib.spec_verify_attention(q, *args, **kw)
        if want is None:
            want = got
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), i
