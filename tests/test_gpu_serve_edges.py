"""Edges of the paged serving operators on the GPU: tokens without weight,
requests that get no pages, calls without rows, scales and windows at the ends of
their ranges, many rows of a real vocabulary."""

import importlib.util
import os

import numpy as np
import pytest
import torch

from oracle import serve_oracle as S
from test_gpu_serve import BF, DEV, F32, check_attention, check_sample, dev_error, f32, i32

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- sampling

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [300, 512, 40000])
def test_tokens_without_weight_are_never_drawn(cuda_lib, dtype, V):
    """The largest random numbers leave the target at the rounding of the kept
    mass.  Kept by top-k are also tokens whose weight underflows (T = 0.05: ids more
    than 7 below the best have exp(-140), below every fp32 number) or is masked: they
    have no probability, so none may come out, whatever the sums' rounding."""
    rng = np.random.default_rng(V)
    N = 600
    x = np.full((N, V), -np.inf) if V <= 512 else rng.uniform(-40, -20, (N, V))
    for i in range(N):
        n = 3 + i % 7
        # among masked tokens top-k takes the lowest ids: the finite ones lie below them
        x[i, rng.choice(12 if V <= 512 else V, n, replace=False)] = rng.uniform(0, 0.2, n)
    xt = torch.tensor(x, dtype=dtype, device=DEV)
    u = np.where(np.arange(N) % 2 == 0, 1 - 2.0 ** -24, 1 - 2.0 ** -23)
    T = [0.05] * N
    for k in (20, 64):
        check_sample(cuda_lib, xt, u, T, [k] * N)
        tok, prob = cuda_lib.spec_verify_sample(xt, f32(u), temperature=f32(T), top_k=i32([k] * N),
                                                want_probs=True)
        assert (xt.gather(1, tok.long()[:, None]) >= 0).all()
        assert (prob > 0).all()


@pytest.mark.parametrize("tail", [2.0 ** -23 * 1.7, 2.0 ** -23 * 1.3, 0.7, 0.3])
def test_running_masses_do_not_drift(cuda_lib, tail):
    """511 equal weights below the best: added one by one to a sum of 1 or more, each
    rounds the same way, and the running mass at their end is off by 511 roundings
    (2^-25 each, 1.5e-5 in all).  The draw has to stay within 1e-6 of the mass."""
    V = 512
    rng = np.random.default_rng(7)
    x = np.full((40, V), np.log(tail))
    x[np.arange(40), rng.integers(0, V, 40)] = 0.0
    rest = 511 * tail / (1 + 511 * tail)
    u = 1 - min(rest, 0.999) * (np.arange(40) + 0.5) / 40
    check_sample(cuda_lib, torch.tensor(x, dtype=F32, device=DEV), u, k=[500] * 40)
    check_sample(cuda_lib, torch.tensor(x, dtype=F32, device=DEV), u, p=[0.9999999] * 40)


@pytest.mark.parametrize("dtype,V,N", [(BF, 32003, 200), (F32, 20011, 330), (BF, 151936, 160)])
def test_many_rows(cuda_lib, dtype, V, N):
    """More rows than SMs, where a row has one CTA: settings of every kind, masked
    rows among them."""
    rng = np.random.default_rng(N)
    x = rng.normal(0, 3, (N, V))
    x[::5, :] += 12 * (rng.random((len(x[::5]), V)) < 20 / V)
    x[3::20][rng.random((len(x[3::20]), V)) < 0.999] = -np.inf
    x[3::20, V // 3] = 1.0
    kind = np.arange(N) % 6
    T = np.where(kind == 5, 0.0, rng.choice([0.6, 1.0, 1.3], N))
    k = np.where((kind == 0) | (kind == 2), rng.choice([20, 1000, V], N), 0)
    p = np.where((kind == 1) | (kind == 2), rng.uniform(0.7, 0.97, N), 1.0)
    m = np.where(kind == 3, 0.05, 0.0)
    check_sample(cuda_lib, torch.tensor(x, dtype=dtype, device=DEV), rng.random(N), T, k, p, m)


# ---------------------------------------------------------------- shortage

@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_request_without_pages_reads_no_other_requests_cache(cuda_lib, dtype):
    """Three requests want pages, the second finds none.  Its table still holds ids
    of pages that others own; its rows come out as zeros, flagged, and the others'
    rows as they are without it."""
    lib = cuda_lib
    page, H, D = 16, 2, 64
    g = torch.Generator(device=DEV).manual_seed(0)
    kc, vc = (torch.randn(8, page, H, D, device=DEV, generator=g).to(dtype) for _ in range(2))
    q, k, v = (torch.randn(9, H, D, device=DEV, generator=g).to(dtype) for _ in range(3))
    # request 1 holds page 5; its row's next entries are pages that it gave back long ago
    table = i32([[1, 2, 0, 0], [5, 1, 2, 3], [3, 4, 0, 0]])
    err = dev_error()
    plan = lib.spec_verify_slots(i32([20, 15, 18]), i32([3, 40, 2]), table, i32([2, 1, 2]),
                                 i32([6, 0]), i32([1]), page_size=page, n_rows=48, dev_error=err)
    assert err.item() == lib.SV_DEVERR_BLOCKS
    assert plan.seq_lens.tolist() == [23, -1, 20]
    plan = lib.spec_verify_slots(i32([20, 15, 18]), i32([3, 4, 2]), table, i32([2, 1, 2]),
                                 i32([6, 0]), i32([0]), page_size=page, n_rows=9, dev_error=err)
    assert plan.seq_lens.tolist() == [23, -1, 20] and plan.held.tolist() == [2, 1, 2]
    err.zero_()
    lib.spec_verify_append(k, v, plan.slots, kc, vc, dev_error=err)
    out = torch.full((9, H, D), 7.0, device=DEV, dtype=dtype)
    lse = torch.full((9, H), 7.0, device=DEV)
    lib.spec_verify_attention(q, kc, vc, table, plan.seq_lens, plan.row_offsets, max_len=4, out=out,
                              lse=lse, dev_error=err)
    assert err.item() == lib.SV_DEVERR_LEN
    assert (out[3:7] == 0).all() and (lse[3:7] == -float("inf")).all()
    rest = torch.cat([q[:3], q[7:]])
    want, wl = lib.spec_verify_attention(rest, kc, vc, table[[0, 2]], i32([23, 20]), i32([0, 3, 5]),
                                         max_len=4, want_lse=True)
    assert torch.equal(torch.cat([out[:3], out[7:]]), want)
    assert torch.equal(torch.cat([lse[:3], lse[7:]]), wl)


def test_requests_out_of_range_get_no_length(cuda_lib):
    """A negative context, more pages than the table has columns, a count of pages
    outside it: the length that comes out is one that attention refuses."""
    lib, err = cuda_lib, dev_error()
    out = lib.spec_verify_slots(i32([-1, 5, 3, 2, 3]), i32([2, 20, 1, -4, 0]),
                                i32(np.arange(20).reshape(5, 4)), i32([1, 2, 1, 9, 1]),
                                i32([90, 91, 92]), i32([3]), page_size=4, n_rows=30, dev_error=err)
    assert err.item() == lib.SV_DEVERR_LEN
    assert out.seq_lens.tolist() == [-1, -1, 4, -1, 3]


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_of_a_request_that_is_left_out_are_zeros(cuda_lib, dtype):
    kc = torch.randn(4, 16, 1, 64, device=DEV).to(dtype)
    q = torch.randn(6, 2, 64, device=DEV).to(dtype)
    ok, okl = cuda_lib.spec_verify_attention(q, kc, kc.clone(), i32([[0, 1], [2, 3]]), i32([20, 30]),
                                             i32([0, 3, 6]), max_len=3, want_lse=True)
    for seq, offs, max_len in (([20, 33], [0, 3, 6], 3), ([20, -1], [0, 3, 6], 3),
                               ([20, 30], [0, 2, 6], 3)):
        err = dev_error()
        out, lse = torch.full_like(q, 9.0), torch.full((6, 2), 9.0, device=DEV)
        cuda_lib.spec_verify_attention(q, kc, kc.clone(), i32([[0, 1], [2, 3]]), i32(seq), i32(offs),
                                       max_len=max_len, out=out, lse=lse, dev_error=err)
        assert err.item() == cuda_lib.SV_DEVERR_LEN
        n = offs[1]
        assert (out[n:] == 0).all() and (lse[n:] == -float("inf")).all()
        if n == 3:
            assert torch.equal(out[:3], ok[:3]) and torch.equal(lse[:3], okl[:3])


# ---------------------------------------------------------------- attention

@pytest.mark.parametrize("dtype", [BF, F32])
def test_attention_without_rows(cuda_lib, dtype):
    """A step in which no request has new tokens."""
    kc = torch.randn(4, 16, 2, 64, device=DEV).to(dtype)
    q = torch.empty(0, 4, 64, dtype=dtype, device=DEV)
    out, lse = cuda_lib.spec_verify_attention(q, kc, kc.clone(), i32([[0, 1], [2, 3]]), i32([20, 30]),
                                              i32([0, 0, 0]), max_len=1, want_lse=True)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("scale", [0.0, -0.125])
def test_attention_signs_of_the_scale(cuda_lib, dtype, D, scale):
    """Requests cut into parts, tiles on the causal edge, chunks; the scores are no
    larger than at the default scale, so the same bounds hold."""
    check_attention(cuda_lib, dtype, [(9001, 16), (700, 5), (37, 1), (0, 2)], 2, 4, D, 16,
                    scale=scale * (64 / D) ** 0.5)
    check_attention(cuda_lib, dtype, [(700, 300), (257, 257)], 1, 2, D, 64, window=200,
                    scale=scale * (64 / D) ** 0.5)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("scale", [6.0, -6.0])
@pytest.mark.parametrize("lens,G", [([(9001, 16), (700, 5), (37, 1)], 4), ([(700, 300), (260, 9)], 2)])
def test_attention_of_large_scores(cuda_lib, dtype, scale, lens, G):
    """Scores of some hundreds, across rescalings and the join of parts.

    A score is a sum of D products in 32 bits, off by at most D 2^-24 sum |q k|
    |scale| =: e, and two roundings of its own size (scaling, and m c) add 2^-23 |score|
    <= 2^-23 sum |q k| |scale|, below e.  A weight exp(s - m) is then off by at
    most 4 e relatively (both scores, twice e each) and so is the sum of weights; over
    both the output by 8 e mag, beside its roundings as at any scale.  lse: 2 e."""
    D, Hk, page = 64, 2, 16
    g = torch.Generator(device=DEV).manual_seed(1)
    need = [-(-n // page) for n, _ in lens]
    ids = np.random.default_rng(1).permutation(sum(need))
    table, at = np.zeros((len(lens), max(need)), int), 0
    for r, n in enumerate(need):
        table[r, :n] = ids[at:at + n]
        at += n
    kc, vc = (torch.randn(sum(need), page, Hk, D, device=DEV, generator=g).to(dtype) for _ in range(2))
    N = sum(l for _, l in lens)
    q = (2 * torch.randn(N, Hk * G, D, device=DEV, generator=g)).to(dtype)
    offs = np.concatenate([[0], np.cumsum([l for _, l in lens])])
    err = dev_error()
    out, lse = cuda_lib.spec_verify_attention(
        q, kc, vc, i32(table), i32([n for n, _ in lens]), i32(offs), max_len=max(l for _, l in lens),
        scale=scale, want_lse=True, dev_error=err)
    assert err.item() == 0
    o, x, qn = out.double().cpu().numpy(), lse.double().cpu().numpy(), q.double().cpu().numpy()
    for r, (n, l) in enumerate(lens):
        k, v = (c[torch.tensor(table[r, :need[r]], device=DEV)].flatten(0, 1)[:n].double().cpu().numpy()
                for c in (kc, vc))
        rows = slice(offs[r], offs[r + 1])
        want, wl, mag = S.attention_request(qn[rows], k, v, scale)
        e = np.zeros((l, Hk * G))
        for h in range(Hk * G):
            e[:, h] = D * 2.0 ** -24 * abs(scale) * (np.abs(qn[rows][:, h]) @ np.abs(k[:, h // G]).T).max(1)
        assert e.max() < 0.01
        tol = mag * ((2.0 ** -12 if dtype == F32 else 2.0 ** -7) + 8 * e[:, :, None]) + 1e-30
        assert (np.abs(o[rows] - want) <= tol).all(), np.max(np.abs(o[rows] - want) / tol)
        assert (np.abs(x[rows] - wl) <= 2.0 ** -12 + 2 * e).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attention_at_the_ends_of_the_scales(cuda_lib, dtype):
    """Scale 0 weighs all keys alike however large the products; the largest finite
    scales pick the best key."""
    n, D = 300, 64
    g = torch.Generator(device=DEV).manual_seed(2)
    q = torch.zeros(2, 1, D, device=DEV, dtype=dtype)
    q[:, 0, 0] = 1e18
    kc = torch.zeros(20, 16, 1, D, device=DEV, dtype=dtype)
    kc[..., 0] = (torch.rand(20, 16, 1, device=DEV, generator=g) * 1e20).to(dtype)
    vc = torch.randn(20, 16, 1, D, device=DEV, generator=g).to(dtype)
    a = (i32(np.arange(20)[None]), i32([n]), i32([0, 2]))
    out, lse = cuda_lib.spec_verify_attention(q, kc, vc, *a, max_len=2, scale=0.0, want_lse=True)
    v = vc.flatten(0, 1)[:, 0].double()
    for j in range(2):
        want, mag = v[:n - 1 + j].mean(0), v[:n - 1 + j].abs().mean(0)
        assert ((out[j, 0].double() - want).abs() <= 2.0 ** (-12 if dtype == F32 else -7) * mag).all()
        assert abs(lse[j, 0].item() - np.log(n - 1 + j)) <= 2.0 ** -12
    # a scale times log2(e) that leaves fp32: products of 0 and of 1
    for scale in (3e38, -3e38):
        q[:, 0, 0] = 1.0 if scale > 0 else -1.0
        kc.zero_()
        kc[7, 5, 0, 0] = 1.0
        out, _ = cuda_lib.spec_verify_attention(q, kc, vc, *a, max_len=2, scale=scale)
        assert torch.equal(out[:, 0], vc[7, 5].repeat(2, 1))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 5, 2 ** 30, 10 ** 6])
def test_attention_windows_past_every_context(cuda_lib, dtype, window):
    """A window that holds every key is no window, for requests with more rows than
    tokens too."""
    lens = [(2, 9), (0, 3), (130, 140), (9001, 4), (17, 16)]
    for G in (1, 4):
        a = check_attention(cuda_lib, dtype, lens, 2, G, 64, 16, window=window)
        b = check_attention(cuda_lib, dtype, lens, 2, G, 64, 16)
        assert torch.equal(a, b)


# ---------------------------------------------------------------- example

def test_the_example_sees_the_flags_of_every_operator(cuda_lib, monkeypatch):
    """Lengths that attention refuses, slots that append refuses: decoding stops."""
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "speculative_decode.py")
    spec = importlib.util.spec_from_file_location("speculative_decode", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    model = example.Toy(1009, 4, 2, 32, 50, 16, F32, 3)
    plan = example.Server.plan
    for break_it in (lambda p: p.seq_lens.fill_(10 ** 6), lambda p: p.slots.fill_(1 << 40)):
        def broken(self, *a):
            p = plan(self, *a)
            break_it(p)
            return p
        monkeypatch.setattr(example.Server, "plan", broken)
        with pytest.raises(AssertionError, match="device error"):
            example.generate(model, model, [[5, 9], [7]], 4, 3, page=16, pages=50, width=8)
