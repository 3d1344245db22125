"""GPU parity of the paged serving operators (sampling, slot maps, cache
writes, chunk attention) with their fp64 oracle."""

import numpy as np
import pytest
import torch

from oracle import serve_oracle as S

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def dev_error():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def i32(a):
    return torch.tensor(np.asarray(a, np.int64), dtype=torch.int32, device=DEV)


def f32(a):
    return torch.tensor(np.asarray(a, np.float64), dtype=F32, device=DEV)


# ---------------------------------------------------------------- sampling
# Tolerances.  A weight is 2^y with y = (x - max) log2(e) / T formed in three
# roundings, so its relative error is about |y| 2^-22 and below 2e-6 where it
# matters; masses add rounding of the same order.  Draws and cuts within 1e-6
# of a tie admit either side; a probability is within 1e-5 of the oracle's.

def check_sample(lib, x, u, T=None, k=None, p=None, m=None, stride=None):
    N, V = x.shape
    if stride is not None:
        store = torch.full((N, stride), float("nan"), dtype=x.dtype, device=DEV)
        store[:, :V] = x
        x = store[:, :V]
    err = dev_error()
    opt = lambda a, f: None if a is None else f(a)  # noqa: E731
    tok, prob = lib.spec_verify_sample(x, f32(u), temperature=opt(T, f32), top_k=opt(k, i32),
                                       top_p=opt(p, f32), min_p=opt(m, f32), want_probs=True,
                                       dev_error=err)
    tok2, prob2 = lib.spec_verify_sample(x, f32(u), temperature=opt(T, f32), top_k=opt(k, i32),
                                         top_p=opt(p, f32), min_p=opt(m, f32), want_probs=True)
    assert torch.equal(tok, tok2) and torch.equal(prob, prob2)
    assert err.item() == 0
    xs, tok, prob = x.float().cpu().numpy(), tok.cpu().numpy(), prob.cpu().numpy()
    g = lambda a, i, d: d if a is None else float(np.float32(a[i]))  # noqa: E731
    for i in range(N):
        want = S.sample_row(xs[i], g(T, i, 1.0), int(g(k, i, 0)), g(p, i, 1.0), g(m, i, 0.0),
                            g(u, i, 0.0))
        assert int(tok[i]) in want, (i, tok[i], want)
        assert min(abs(prob[i] - q) for q in want[int(tok[i])]) <= 1e-5 * prob[i] + 1e-9


def settings(rng, N, V):
    """Every mixture of filters over the rows, greedy rows among them."""
    T = rng.choice([0.0, 0.3, 0.7, 1.0, 1.0, 1.7, 5.0], N)
    k = rng.choice([0, 0, 1, 2, 20, 64, 65, 300, 1000, V - 1, V, V + 7], N)
    p = rng.choice([1.0, 1.0, 0.999999, 0.95, 0.5, 0.1, 1e-6], N)
    m = rng.choice([0.0, 0.0, 0.0, 0.01, 0.3, 1.0], N)
    return T, k, p, m


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [1, 2, 3, 7, 17, 255, 1000, 4097, 20011, 40961, 151936])
def test_sample_mixed_settings(cuda_lib, dtype, V):
    rng = np.random.default_rng(V)
    N = 40 if V < 30000 else 16
    for spread, stride in ((3.0, None), (0.5, V + 3), (12.0, V + 64)):
        x = torch.tensor(rng.normal(0, spread, (N, V)), dtype=dtype, device=DEV)
        T, k, p, m = settings(rng, N, V)
        check_sample(cuda_lib, x, rng.random(N), T, k, p, m, stride)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [64, 3000, 65536])
def test_sample_ties_zeros_and_masks(cuda_lib, dtype, V):
    """Cuts inside classes of equal logits, zeros of both signs, rows that are
    mostly -inf, one finite token."""
    rng = np.random.default_rng(V + 1)
    N = 24
    x = rng.integers(-2, 3, (N, V)).astype(np.float64)
    x[4:8] = np.where(rng.random((4, V)) < 0.5, 0.0, -0.0)
    x[8:12] = 1.25
    x[12:16][rng.random((4, V)) < 0.9] = -np.inf
    x[16:20] = -np.inf
    x[np.arange(16, 20), rng.integers(0, V, 4)] = rng.normal(0, 50, 4)
    x[20:24] = -np.inf
    x[20:24, -5:] = 2.0
    x[:16, V // 2] = 2.0
    xt = torch.tensor(x, dtype=dtype, device=DEV)
    for k, p, m in ((0, 1, 0), (7, 1, 0), (0, 0.37, 0), (V // 2, 0.6, 0), (V // 3, 1, 0.9),
                    (0, 1, 0.5), (V - 1, 0.99, 0.1)):
        check_sample(cuda_lib, xt, rng.random(N), None, [k] * N, [p] * N, [m] * N)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [0.05, 1.3, 60.0])
@pytest.mark.parametrize("V", [5001, 60000])
def test_sample_flat_rows(cuda_lib, dtype, T, V):
    """Cuts far down flat rows: among few and among thousands of tokens of about one
    weight, the row longer than a CTA's part by a few tokens."""
    rng = np.random.default_rng(V)
    N = 72
    x = torch.tensor(rng.normal(0, 3, (N, V)), dtype=dtype, device=DEV)
    p = rng.uniform(0.3, 0.995, N)
    k = np.where(np.arange(N) % 3 == 0, rng.integers(200, V, N), 0)
    check_sample(cuda_lib, x, rng.random(N), [T] * N, k, np.where(np.arange(N) % 6 == 0, 1.0, p),
                 np.where(np.arange(N) % 4 == 0, 0.001, 0.0), V + 7)


def test_sample_without_settings_and_extremes(cuda_lib):
    rng = np.random.default_rng(3)
    x = torch.tensor(rng.normal(0, 2, (5, 5003)), dtype=F32, device=DEV)
    check_sample(cuda_lib, x, [0.0, 0.25, 0.5, 0.75, 1 - 2.0 ** -24])
    check_sample(cuda_lib, x, [0.0, 0.1, 0.5, 0.9, 1 - 2.0 ** -24], k=[3] * 5)
    # magnitudes at which x / T leaves the type: the best token has all the mass
    for scale, T in ((1e38, 1.0), (1e30, 1e-20), (1.0, 1e-30), (1e-30, 1e-38)):
        y = torch.arange(100, device=DEV, dtype=F32)[None].repeat(3, 1) * (scale / 100)
        tok, prob = cuda_lib.spec_verify_sample(y, f32([0.1, 0.5, 0.9]), temperature=f32([T] * 3),
                                                want_probs=True)
        assert tok.tolist() == [99] * 3 and prob.tolist() == [1.0] * 3
    assert cuda_lib.spec_verify_sample(x[:0], f32([]))[0].numel() == 0


def test_sample_large_rows(cuda_lib):
    """The largest vocabularies of the single row limit, peaked and flat."""
    rng = np.random.default_rng(5)
    for dtype, V in ((BF, 262144), (F32, 262144), (BF, 786432), (F32, 393216)):
        x = rng.normal(0, 2, (6, V))
        x[:3, rng.integers(0, V, 50)] += 12
        check_sample(cuda_lib, torch.tensor(x, dtype=dtype, device=DEV), rng.random(6), None,
                     [0, 50, 5000, 0, 50, 5000], [0.9, 0.95, 0.99, 0.9, 1, 0.5],
                     [0, 0, 0.001, 0, 0, 0])


def test_sample_flags_bad_rows_alone(cuda_lib):
    x = torch.zeros(8, 999, device=DEV)
    x[1, 500] = float("nan")
    x[2, 0] = float("inf")
    x[3] = -float("inf")
    for setting, bad in ((dict(), None), (dict(temperature=[1, 1, 1, 1, -1, float("nan"), 1, 1]), 4),
                         (dict(top_p=[1, 1, 1, 1, 0, 1.5, 1, 1]), 4),
                         (dict(min_p=[0, 0, 0, 0, -0.1, 1.1, 0, 0]), 4)):
        err = dev_error()
        tok, prob = cuda_lib.spec_verify_sample(
            x, f32([0.5] * 8), want_probs=True, dev_error=err,
            **{n: f32(v) for n, v in setting.items()})
        flags = cuda_lib.SV_DEVERR_NAN | (cuda_lib.SV_DEVERR_PARAM if bad else 0)
        assert err.item() == flags
        wrong = {1, 2, 3} | ({4, 5} if bad else set())
        for i in range(8):
            assert (tok[i].item() == -1) == (i in wrong) and (prob[i].item() == 0) == (i in wrong)
    err = dev_error()
    tok, _ = cuda_lib.spec_verify_sample(x[:1].repeat(3, 1), f32([1.0, -0.1, 0.3]), dev_error=err)
    assert err.item() == cuda_lib.SV_DEVERR_PARAM and tok.tolist()[:2] == [-1, -1]


def test_sample_follows_the_distribution(cuda_lib):
    """20,000 draws of one filtered row, within five standard deviations."""
    p = np.array([0.02, 0.3, 0.08, 0.25, 0.15, 0.2])
    N = 20000
    x = f32(np.log(p))[None].repeat(N, 1)
    u = np.random.default_rng(1).random(N)
    tok, _ = cuda_lib.spec_verify_sample(x, f32(u), top_k=i32([4] * N))
    kept = np.where(p >= 0.15, p, 0) / 0.9
    seen = np.bincount(tok.cpu().numpy(), minlength=6) / N
    assert np.all(np.abs(seen - kept) <= 5 * np.sqrt(kept * (1 - kept) / N) + 1e-12)


# ---------------------------------------------------------------- slots

def run_slots(lib, ctx, new, table, held, free, count, page, n_rows):
    t, f, err = i32(table), i32(free), dev_error()
    a = (i32(ctx), i32(new), t, i32(held), f, i32([count]))
    for _ in range(2):  # the counts are inputs: a second call does the same
        out = lib.spec_verify_slots(*a, page_size=page, n_rows=n_rows, dev_error=err)
    return out, t, f, err.item()


def check_slots(lib, ctx, new, table, held, free, count, page, n_rows, flags=0):
    want = S.slots(ctx, new, np.array(table), held, np.array(free), count, page, n_rows)
    out, t, f, err = run_slots(lib, ctx, new, table, held, free, count, page, n_rows)
    assert err == flags
    assert t.cpu().tolist() == want["table"].tolist()
    assert f.cpu().tolist()[:len(want["stack"])] == want["stack"]
    assert out.free_count.item() == want["count"]
    for name in ("row_offsets", "seq_lens", "positions", "slots"):
        assert getattr(out, name).cpu().tolist() == list(want[name]), name
    assert out.held.cpu().tolist() == list(want["held"])


@pytest.mark.parametrize("B", [1, 2, 31, 33, 512, 513, 1500])
@pytest.mark.parametrize("page", [1, 7, 16, 128])
def test_slots_random(cuda_lib, B, page):
    rng = np.random.default_rng(B * 131 + page)
    ctx = rng.integers(0, 40 * page, B)
    new = np.where(rng.random(B) < 0.2, 0, rng.integers(0, 2 * page + 3, B))
    ctx[rng.random(B) < 0.1] = 0
    need = -(-(ctx + new) // page)
    held = np.maximum(0, need + rng.integers(-2, 3, B))
    width = int(max(need.max(), held.max())) + 2
    ids = rng.permutation(B * width * 2 + 8)
    table = ids[:B * width].reshape(B, width)
    free = ids[B * width:]
    count = len(free) - int(held.sum())
    check_slots(cuda_lib, ctx, new, table, held, list(free), count, page, int(new.sum()) + 3)


def test_slots_takes_pages_returned_in_the_same_call(cuda_lib):
    # five pages come back; the second request takes them, the third finds none
    args = ([0, 0, 9], [0, 20, 8], [[5, 6, 7, 8, 9], [0] * 5, [3, 1, 0, 0, 0]], [5, 0, 2])
    check_slots(cuda_lib, *args, [0] * 8, 0, 4, 28, flags=cuda_lib.SV_DEVERR_BLOCKS)
    check_slots(cuda_lib, *args, [20, 21, 22] + [0] * 5, 3, 4, 28)


def test_slots_shortage_and_bad_lengths(cuda_lib):
    lib = cuda_lib
    check_slots(lib, [4, 0, 3, 0], [1, 9, 1, 4], np.arange(16).reshape(4, 4), [1, 0, 1, 1],
                [90, 91, 92], 3, 4, 15, flags=lib.SV_DEVERR_BLOCKS)
    check_slots(lib, [-1, 5, 3, 2], [2, 20, 1, -4], np.arange(16).reshape(4, 4), [1, 2, 1, 9],
                [90, 91, 92], 3, 4, 30, flags=lib.SV_DEVERR_LEN)
    # more new tokens than rows: flagged, nothing past the rows is written
    out, _, _, err = run_slots(lib, [0, 0], [5, 5], [[0, 0], [0, 0]], [0, 0], [7, 8, 9, 6], 4, 4, 6)
    assert err & lib.SV_DEVERR_LEN and out.slots.numel() == 6


def test_slots_refusals(cuda_lib):
    a = dict(page_size=4, n_rows=4)
    t, h = i32(np.zeros((2, 3))), i32([0, 0])
    with pytest.raises(cuda_lib.SpecVerifyError):
        cuda_lib.spec_verify_slots(i32([1, 1]), i32([1, 1]), t, h, i32([1]), i32([1]), held_out=h, **a)
    with pytest.raises(TypeError):
        cuda_lib.spec_verify_slots(i32([1, 1]).long(), i32([1, 1]), t, h, i32([1]), i32([1]), **a)
    with pytest.raises(ValueError):
        cuda_lib.spec_verify_slots(i32([1]), i32([1, 1]), t, h, i32([1]), i32([1]), **a)
    with pytest.raises(ValueError):
        cuda_lib.spec_verify_slots(i32([1, 1]), i32([1, 1]), t.T, h, i32([1]), i32([1]), **a)


# ---------------------------------------------------------------- append

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,H,D,page", [(1, 1, 1, 1), (3, 2, 24, 16), (5, 3, 7, 3),
                                           (400, 8, 128, 16), (1025, 4, 64, 64), (37, 1, 256, 5)])
@pytest.mark.parametrize("layout", ["tokens", "heads"])
def test_append(cuda_lib, dtype, rows, H, D, page, layout):
    g = torch.Generator(device=DEV).manual_seed(rows)
    blocks = -(-rows // page) + 4
    shape = (blocks, page, H, D) if layout == "tokens" else (blocks, H, page, D)
    caches = [torch.randn(shape, device=DEV, generator=g).to(dtype) for _ in range(2)]
    views = [c if layout == "tokens" else c.transpose(1, 2) for c in caches]
    fused = torch.randn(rows, 3 * H * D + 1, device=DEV, generator=g).to(dtype)
    k = fused[:, :H * D].unflatten(1, (H, D))
    v = fused[:, 2 * H * D + 1:].unflatten(1, (H, D))
    slots = torch.randperm(blocks * page, device=DEV, generator=g)[:rows]
    slots[::3] = -1
    want = [c.clone() for c in views]
    for w, x in zip(want, (k, v)):
        for i, s in enumerate(slots.tolist()):
            if s >= 0:
                w[s // page, s % page] = x[i]
    err = dev_error()
    cuda_lib.spec_verify_append(k, v, slots, *views, dev_error=err)
    assert err.item() == 0
    for w, c in zip(want, views):
        assert torch.equal(w, c)


def test_append_skips_slots_past_the_cache(cuda_lib):
    kc, vc = torch.zeros(2, 4, 1, 8, device=DEV), torch.zeros(2, 4, 1, 8, device=DEV)
    k = torch.ones(3, 1, 8, device=DEV)
    err = dev_error()
    cuda_lib.spec_verify_append(k, 2 * k, torch.tensor([8, 7, 1 << 40], device=DEV), kc, vc,
                                dev_error=err)
    assert err.item() == cuda_lib.SV_DEVERR_PAGE
    assert kc.sum().item() == 8 and kc[1, 3].sum().item() == 8 and vc.sum().item() == 16


def test_append_refusals(cuda_lib):
    kc = torch.zeros(2, 4, 2, 8, device=DEV)
    k, s = torch.ones(3, 2, 8, device=DEV), torch.zeros(3, dtype=torch.int64, device=DEV)
    for bad in (dict(key=k.bfloat16()), dict(slots=s.int()), dict(key=k[:2]), dict(key=k.cpu()),
                dict(value_cache=kc[:, :, :1]), dict(key_cache=kc.double()),
                dict(value_cache=torch.zeros(2, 2, 4, 8, device=DEV).transpose(1, 2))):
        a = {**dict(key=k, value=k, slots=s, key_cache=kc, value_cache=kc.clone()), **bad}
        with pytest.raises((TypeError, ValueError)):
            cuda_lib.spec_verify_append(*a.values())


# ---------------------------------------------------------------- attention
# Tolerances, for mag = sum p |v| >= |out|.  bf16 keeps 8 significant bits, so one
# rounding is off by at most 2^-8 (1 + 2^-8 lies halfway between 1 and its
# successor 1 + 2^-7): 2^-8 |out| for the output and 2^-8 mag for the weights,
# which are rounded for the tensor cores.  A score of
# magnitude up to 2^5 carries 2^-19 absolute error, far below.  fp32: scores are
# sums of up to 256 products, off by at most 2^-24 * 256 * sum |q k| scale
# (< 2^-12), typically 2^-18.  lse carries the scores' error.

def check_attention(lib, dtype, lens, Hk, G, D, page, window=0, layout="tokens", strided=False,
                    scale=None, seed=0, poison=True):
    """lens: (seq, new) of every request."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    rng = np.random.default_rng(seed)
    seq, new = [n for n, _ in lens], [l for _, l in lens]
    need = [-(-n // page) for n in seq]
    blocks, width, N, Hq = sum(need) + 2, max(need) + 1, sum(new), Hk * G
    ids = rng.permutation(blocks)
    table = np.full((len(lens), width), 2 ** 30)  # past the last page: never read
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = ids[at:at + n]
        at += n
    shape = (blocks, page, Hk, D) if layout == "tokens" else (blocks, Hk, page, D)
    caches = []
    for _ in range(2):
        c = torch.randn(shape, device=DEV, generator=g).to(dtype)
        caches.append(c if layout == "tokens" else c.transpose(1, 2))
    flat = [[c[torch.tensor(table[r, :need[r]], device=DEV)].flatten(0, 1)[:n] for c in caches]
            for r, n in enumerate(seq)]
    flat = [[x.double().cpu().numpy() for x in kv] for kv in flat]
    if poison:  # page tails and unused pages hold NaN and infinities
        for c in caches:
            keep = torch.zeros(blocks, page, dtype=torch.bool, device=DEV)
            for r, n in enumerate(seq):
                for j in range(need[r]):
                    keep[table[r, j], :min(page, n - j * page)] = True
            c[~keep] = torch.where(torch.rand(c[~keep].shape, device=DEV, generator=g) < 0.5,
                                   float("nan"), float("inf")).to(dtype)
    if strided:
        q = torch.randn(N, 2 * Hq + 1, D + 8, device=DEV, generator=g).to(dtype)[:, 1:2 * Hq:2, :D]
        out = torch.zeros(N, Hq + 1, 2 * D, device=DEV, dtype=dtype)[:, 1:, D:]
    else:
        q = torch.randn(N, Hq, D, device=DEV, generator=g).to(dtype)
        out = torch.full((N, Hq, D), float("nan"), dtype=dtype, device=DEV)
    q = q * 2 if not strided else q.mul_(2)
    err = dev_error()
    ws = lib.alloc_attention_workspace(q)
    ws.fill_(255)
    args = (q, *caches, i32(table), i32(seq), i32(np.concatenate([[0], np.cumsum(new)])))
    kw = dict(max_len=max(1, max(new)), window=window, scale=scale, want_lse=True)
    out, lse = lib.spec_verify_attention(*args, out=out, workspace=ws, dev_error=err, **kw)
    assert err.item() == 0
    again, lse2 = lib.spec_verify_attention(*args, **kw)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    o, x, qn = out.double().cpu().numpy(), lse.double().cpu().numpy(), q.double().cpu().numpy()
    sc = D ** -0.5 if scale is None else scale
    at = 0
    for r, (n, l) in enumerate(lens):
        want, wl, mag = S.attention_request(qn[at:at + l], *flat[r], sc, window)
        got, gl = o[at:at + l], x[at:at + l]
        tol = mag * (2.0 ** -12 if dtype == F32 else 2.0 ** -7) + 1e-30
        assert np.isfinite(got).all(), (r, n, l)
        assert (np.abs(got - want) <= tol).all(), (r, n, l, np.max(np.abs(got - want) / tol))
        fin = np.isfinite(wl)
        assert (np.isfinite(gl) == fin).all() and (gl[~fin] == -np.inf).all()
        assert (np.abs(gl[fin] - wl[fin]) <= 2.0 ** -12).all()
        at += l
    return out


LENS = [(1, 1), (5, 5), (16, 1), (17, 16), (127, 16), (128, 16), (129, 7), (200, 3), (255, 5),
        (257, 16), (300, 300), (1000, 16)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [8, 64, 72, 80, 128, 256])
@pytest.mark.parametrize("Hk,G", [(1, 1), (2, 4), (1, 16), (3, 5)])
def test_attention_shapes(cuda_lib, dtype, D, Hk, G):
    check_attention(cuda_lib, dtype, LENS, Hk, G, D, 16)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [1, 2, 5, 8, 16, 24, 32, 64, 128, 192, 256, 1000])
@pytest.mark.parametrize("layout", ["tokens", "heads"])
def test_attention_pages(cuda_lib, page, layout, D):
    for G, strided in ((2, False), (9, True)):
        check_attention(cuda_lib, BF, LENS, 2, G, D, page, layout=layout, strided=strided)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("window", [1, 2, 31, 128, 129, 500])
def test_attention_window(cuda_lib, dtype, window):
    for G in (1, 6):
        check_attention(cuda_lib, dtype, LENS, 2, G, 64, 16, window=window)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attention_rows_that_see_nothing(cuda_lib, dtype):
    """Requests without new tokens, without tokens, and with more rows than
    tokens: zeros and -inf."""
    lens = [(0, 0), (7, 0), (0, 3), (2, 9), (1, 1), (0, 1), (130, 140), (0, 0)]
    for G in (1, 8):
        check_attention(cuda_lib, dtype, lens, 2, G, 128, 16)


@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("l", [1, 2, 16, 33])
def test_attention_long(cuda_lib, G, l):
    check_attention(cuda_lib, BF, [(9001, l), (20000, l), (37, l), (4096, l)], 2, G, 128, 32, seed=l)


@pytest.mark.parametrize("D", [64, 96, 256])
@pytest.mark.parametrize("page", [1, 24, 64])
@pytest.mark.parametrize("layout", ["tokens", "heads"])
def test_attention_float_long(cuda_lib, D, page, layout):
    """fp32: requests cut into many parts, ragged pages, strided rows, both layouts."""
    lens = [(3001, 1), (37, 5), (5000, 16), (4096, 3)]
    check_attention(cuda_lib, F32, lens, 2, 3, D, page, layout=layout, strided=True, seed=page)
    check_attention(cuda_lib, F32, lens, 1, 2, D, page, layout=layout, window=300, seed=page)


def test_attention_many_requests(cuda_lib):
    rng = np.random.default_rng(9)
    lens = [(int(n), int(min(n, l))) for n, l in zip(rng.integers(1, 400, 700),
                                                     rng.integers(1, 17, 700))]
    check_attention(cuda_lib, BF, lens, 1, 4, 64, 16)
    check_attention(cuda_lib, BF, [(n, 1) for n, _ in lens], 2, 3, 128, 16)


@pytest.mark.parametrize("G", [1, 8])
def test_attention_chunks(cuda_lib, G):
    check_attention(cuda_lib, BF, [(1500, 1000), (700, 700), (2049, 129), (513, 257)], 1, G, 128, 64)
    check_attention(cuda_lib, BF, [(900, 640), (300, 300)], 2, G, 64, 16, window=200)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("G,l", [(1, 6), (4, 16), (2, 130)])
def test_attention_unseen_values_do_not_reach_a_row(cuda_lib, dtype, G, l):
    """NaN and infinities in the keys and values of later chunk positions, and of
    keys that left the window, leave the earlier rows as they were."""
    g = torch.Generator(device=DEV).manual_seed(4)
    n, D, Hk, page = 300, 64, 2, 16
    for window in (0, 200):
        kc, vc = (torch.randn(20, page, Hk, D, device=DEV, generator=g).to(dtype) for _ in range(2))
        q = torch.randn(l, Hk * G, D, device=DEV, generator=g).to(dtype)
        table = i32(np.arange(20)[None])
        args = (q, kc, vc, table, i32([n]), i32([0, l]))
        clean, _ = cuda_lib.spec_verify_attention(*args, max_len=l, window=window)
        bad = n - l + l // 2  # rows before this position do not see it
        for c, x in ((kc, float("nan")), (vc, float("nan")), (vc, float("inf"))):
            keep = c[bad // page, bad % page].clone()
            c[bad // page, bad % page] = x
            got, _ = cuda_lib.spec_verify_attention(*args, max_len=l, window=window)
            assert torch.equal(got[:l // 2], clean[:l // 2])
            assert not torch.isfinite(got[l // 2:]).any()
            c[bad // page, bad % page] = keep
        if window:
            old = n - l - window + 1 + l // 2  # rows from l // 2 + 1 on do not see it
            vc[old // page, old % page] = float("nan")
            got, _ = cuda_lib.spec_verify_attention(*args, max_len=l, window=window)
            assert torch.equal(got[l // 2 + 1:], clean[l // 2 + 1:])
            assert torch.isnan(got[:l // 2 + 1]).all()


def test_attention_infinite_scores_and_masks(cuda_lib):
    """Keys that drive scores to -inf drop out; scores far apart do not overflow."""
    kc = torch.zeros(2, 16, 1, 64, device=DEV, dtype=BF)
    vc = torch.randn(2, 16, 1, 64, device=DEV).to(BF)
    q = torch.zeros(1, 1, 64, device=DEV, dtype=BF)
    q[0, 0, 0] = 1.0
    kc[0, :, 0, 0] = -float("inf")
    kc[0, 3, 0, 0] = 0.0
    a = (i32([[0, 1]]), i32([16]), i32([0, 1]))
    out, lse = cuda_lib.spec_verify_attention(q, kc, vc, *a, max_len=1, scale=1.0, want_lse=True)
    assert torch.equal(out[0, 0], vc[0, 3, 0]) and lse.item() == 0.0
    kc[0, :, 0, 0] = torch.arange(16, device=DEV).to(BF) * 1e30
    out, lse = cuda_lib.spec_verify_attention(q, kc, vc, *a, max_len=1, scale=1.0, want_lse=True)
    assert torch.equal(out[0, 0], vc[0, 15, 0]) and np.isfinite(lse.item())


def test_attention_error_flags(cuda_lib):
    kc = torch.randn(4, 16, 1, 64, device=DEV).to(BF)
    q = torch.randn(6, 2, 64, device=DEV).to(BF)

    def call(table, seq, offs, max_len=3):
        err, out = dev_error(), torch.zeros_like(q)
        cuda_lib.spec_verify_attention(q, kc, kc.clone(), i32(table), i32(seq), i32(offs),
                                       max_len=max_len, out=out, dev_error=err)
        return err.item(), out
    good, ref = call([[0, 1], [2, 3]], [20, 30], [0, 3, 6])
    assert good == 0
    for table, seq, offs, max_len, flag in (
            ([[0, 1], [2, 9]], [20, 30], [0, 3, 6], 3, cuda_lib.SV_DEVERR_PAGE),
            ([[0, 1], [2, -1]], [20, 30], [0, 3, 6], 3, cuda_lib.SV_DEVERR_PAGE),
            ([[0, 1], [2, 3]], [20, 33], [0, 3, 6], 3, cuda_lib.SV_DEVERR_LEN),
            ([[0, 1], [2, 3]], [20, -1], [0, 3, 6], 3, cuda_lib.SV_DEVERR_LEN),
            ([[0, 1], [2, 3]], [20, 30], [0, 3, 7], 4, cuda_lib.SV_DEVERR_LEN),
            ([[0, 1], [2, 3]], [20, 30], [0, 3, 2], 3, cuda_lib.SV_DEVERR_LEN)):
        err, out = call(table, seq, offs, max_len)
        assert err == flag
        assert torch.equal(out[:3], ref[:3])  # the sound request keeps its answer
    assert call([[0, 1], [2, 3]], [20, 30], [0, 3, 6], 2)[0] == cuda_lib.SV_DEVERR_LEN


def test_attention_refusals(cuda_lib):
    kc = torch.zeros(2, 16, 2, 64, device=DEV, dtype=BF)
    base = dict(query=torch.zeros(4, 4, 64, device=DEV, dtype=BF), key_cache=kc,
                value_cache=kc.clone(), block_table=i32([[0, 1]]), seq_lens=i32([20]),
                row_offsets=i32([0, 4]))
    for bad in (dict(query=base["query"].float()), dict(seq_lens=i32([20, 1])),
                dict(row_offsets=i32([0])), dict(block_table=base["block_table"].long()),
                dict(value_cache=kc[:1]), dict(key_cache=kc[..., :32]),
                dict(query=base["query"].half()), dict(seq_lens=i32([20]).cpu())):
        with pytest.raises((TypeError, ValueError)):
            cuda_lib.spec_verify_attention(*{**base, **bad}.values(), max_len=4)
    for bad in (dict(max_len=0), dict(scale=float("nan")),
                dict(workspace=torch.empty(16, dtype=torch.uint8, device=DEV))):
        with pytest.raises(cuda_lib.SpecVerifyError):
            cuda_lib.spec_verify_attention(*base.values(), **{**dict(max_len=4), **bad})
    with pytest.raises(cuda_lib.SpecVerifyError):  # three heads over two
        cuda_lib.spec_verify_attention(base["query"][:, :3], *list(base.values())[1:], max_len=4)


# ---------------------------------------------------------------- streams and graphs

def test_a_step_on_its_own_stream_and_in_a_graph(cuda_lib):
    """Slots, append, attention and sampling enqueued on a side stream, and
    replayed from a graph after the inputs have changed, match eager calls."""
    g = torch.Generator(device=DEV).manual_seed(2)
    B, Hk, G, D, page, V = 4, 2, 4, 64, 16, 5003
    ctx, new = i32([30, 0, 77, 15]), i32([4, 9, 1, 2])
    table, held = torch.zeros(B, 8, dtype=torch.int32, device=DEV), i32([2, 0, 5, 1])
    table[0, :2], table[2, :5], table[3, :1] = i32([1, 2]), i32([3, 4, 5, 6, 7]), i32([8])
    free, count = i32(list(range(9, 30))), i32([21])
    kc, vc = (torch.randn(30, page, Hk, D, device=DEV, generator=g).to(BF) for _ in range(2))
    qkv = torch.randn(16, (G + 2) * Hk, D, device=DEV, generator=g).to(BF)
    logits, u = torch.randn(16, V, device=DEV, generator=g), torch.rand(16, device=DEV, generator=g)

    def step(stream=None):
        s = cuda_lib.spec_verify_slots(ctx, new, table, held, free, count, page_size=page,
                                       n_rows=16, stream=stream)
        cuda_lib.spec_verify_append(qkv[:, G * Hk:(G + 1) * Hk], qkv[:, (G + 1) * Hk:], s.slots,
                                    kc, vc, stream=stream)
        out = torch.zeros(16, G * Hk, D, device=DEV, dtype=BF)
        _, lse = cuda_lib.spec_verify_attention(qkv[:, :G * Hk], kc, vc, table, s.seq_lens,
                                                s.row_offsets, max_len=16, out=out, want_lse=True,
                                                stream=stream)
        tok, _ = cuda_lib.spec_verify_sample(logits, u, stream=stream)
        return s.slots, out, tok

    want = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    side.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held_tensors = step()
    ctx.copy_(i32([31, 3, 70, 16]))
    held.copy_(i32([3, 1, 5, 2]))
    qkv.normal_(generator=g)
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in held_tensors]
    for a, b in zip(step(), got):
        assert torch.equal(a, b)
