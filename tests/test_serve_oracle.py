"""Hand-computed pins of the serving operators' oracle, and the C ABI's host
checks of those operators (no GPU)."""

import ctypes

import numpy as np
import pytest

from oracle import serve_oracle as S

LOG = np.log


def only(d):
    assert len(d) == 1, d
    (t, p), = d.items()
    return t, p[0]


def test_sample_row_by_hand():
    x = LOG(np.array([0.1, 0.4, 0.2, 0.3]))
    assert only(S.sample_row(x, u=0.05)) == (0, pytest.approx(0.1))
    assert only(S.sample_row(x, u=0.49)) == (1, pytest.approx(0.4))
    assert only(S.sample_row(x, u=0.51)) == (2, pytest.approx(0.2))
    assert only(S.sample_row(x, u=0.71)) == (3, pytest.approx(0.3))
    assert only(S.sample_row(x, T=0, u=0.99)) == (1, 1.0)
    # top-k 2 keeps ids 1 and 3
    assert only(S.sample_row(x, top_k=2, u=0.56)) == (1, pytest.approx(4 / 7))
    assert only(S.sample_row(x, top_k=2, u=0.58)) == (3, pytest.approx(3 / 7))
    # top-p 0.65: 0.4 + 0.3 reaches it; of the top-3's 0.9, 0.65 needs 0.585
    assert only(S.sample_row(x, top_p=0.65, u=0.58)) == (3, pytest.approx(3 / 7))
    assert only(S.sample_row(x, top_k=3, top_p=0.8, u=0.5)) == (2, pytest.approx(2 / 9))
    # min-p 0.6: 0.6 * 0.4 = 0.24 keeps 0.4 and 0.3
    assert only(S.sample_row(x, min_p=0.6, u=0.58)) == (3, pytest.approx(3 / 7))
    # T = 0.5 squares the weights: 0.16 / 0.30
    assert only(S.sample_row(x, T=0.5, u=0.1)) == (1, pytest.approx(0.16 / 0.30))


def test_sample_row_ties_and_masks():
    x = np.array([1.0, 3.0, 3.0, 3.0, -np.inf])
    assert only(S.sample_row(x, T=0)) == (1, 1.0)
    assert only(S.sample_row(x, top_k=2, u=0.6)) == (2, pytest.approx(0.5))
    assert only(S.sample_row(np.array([-0.0, 0.0]), top_k=1, u=0.9)) == (0, 1.0)
    both = S.sample_row(np.zeros(2), u=0.5)  # the draw lies on an edge
    assert set(both) == {0, 1}
    assert set(S.sample_row(LOG(np.array([0.5, 0.3, 0.2])), top_p=0.8, u=0.9)) >= {1, 2}


def test_slots_by_hand():
    # page 4; request 0: 3 + 2 tokens, holds 1, takes 1; request 1: 4 + 0, holds
    # 3, gives 2 back; request 2: 0 + 5, takes 2
    table = np.array([[7, 0, 0], [1, 2, 3], [0, 0, 0]])
    got = S.slots([3, 4, 0], [2, 0, 5], table, [1, 3, 0], np.array([9, 8, 0, 0, 0]), 2, 4, 9)
    assert got["stack"] == [9, 8, 2, 3]
    assert got["table"].tolist() == [[7, 3, 0], [1, 2, 3], [2, 8, 0]]
    assert got["count"] == 1 and got["held"] == [2, 1, 2]
    assert got["row_offsets"].tolist() == [0, 2, 2, 7]
    assert got["positions"].tolist() == [3, 4, 0, 1, 2, 3, 4, 0, 0]
    assert got["slots"].tolist() == [31, 12, 8, 9, 10, 11, 32, -1, -1]
    short = S.slots([0, 0], [5, 1], np.zeros((2, 2), int), [0, 0], np.array([4]), 1, 4, 6)
    assert short["errors"] == {"blocks"} and short["held"] == [0, 0] and short["count"] == 1
    assert short["slots"].tolist() == [-1] * 6


def test_attention_by_hand():
    q = np.ones((2, 1, 1))
    k = np.array([0.0, LOG(3.0), 0.0]).reshape(3, 1, 1)
    v = np.array([1.0, 2.0, 10.0]).reshape(3, 1, 1)
    out, lse, _ = S.attention_request(q, k, v, 1.0)
    assert out[:, 0, 0] == pytest.approx([7 / 4, 17 / 5]) and lse[:, 0] == pytest.approx(LOG([4, 5]))
    out, lse, _ = S.attention_request(q, k, v, 1.0, window=1)
    assert out[:, 0, 0] == pytest.approx([2, 10])
    out, lse, _ = S.attention_request(np.ones((2, 1, 1)), k[:1], v[:1], 1.0)  # l > n
    assert out[0, 0, 0] == 0 and lse[0, 0] == -np.inf and out[1, 0, 0] == 1


# ---------------------------------------------------------------- C ABI host checks

P = 1 << 20  # an aligned address that is never dereferenced
ERR_ARG, ERR_DTYPE, ERR_UNSUPPORTED, ERR_WORKSPACE = -1, -2, -4, -5


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_verification_16_gb300 import build
    build.build()
    from speculative_decoding_verification_16_gb300 import binding
    return binding._lib


SAMPLE = dict(logits=P, stride=1000, N=4, V=1000, dtype=0, T=P, k=P, p=P, m=P, u=P, tok=P, prob=P,
              err=P, stream=None)


@pytest.mark.parametrize("over,code", [
    (dict(dtype=3), ERR_DTYPE), (dict(N=-1), ERR_ARG), (dict(V=0), ERR_ARG),
    (dict(stride=999), ERR_ARG), (dict(logits=None), ERR_ARG), (dict(logits=P + 1), ERR_ARG),
    (dict(u=None), ERR_ARG), (dict(tok=None), ERR_ARG), (dict(tok=P + 2), ERR_ARG),
    (dict(k=P + 1), ERR_ARG), (dict(V=786433, stride=786433), ERR_UNSUPPORTED),
    (dict(V=393217, stride=393217, dtype=1), ERR_UNSUPPORTED),
    (dict(N=0), 0),
])
def test_sample_host_checks(lib, over, code):
    assert lib.spec_verify_sample(*{**SAMPLE, **over}.values()) == code


SLOTS = dict(ctx=P, new=P, B=4, page=16, table=P, stride=8, width=8, held=P, free=P, cap=64,
             count=P, rows=10, offs=P, seq=P, pos=P, slots=P, held_out=2 * P, count_out=2 * P,
             err=P, stream=None)


@pytest.mark.parametrize("over,code", [
    (dict(B=0), ERR_ARG), (dict(page=0), ERR_ARG), (dict(width=0), ERR_ARG),
    (dict(stride=7), ERR_ARG), (dict(ctx=None), ERR_ARG), (dict(free=None), ERR_ARG),
    (dict(slots=None), ERR_ARG), (dict(slots=P + 4), ERR_ARG), (dict(held_out=P), ERR_ARG),
    (dict(count_out=P), ERR_ARG), (dict(rows=-1), ERR_ARG), (dict(B=8193), ERR_UNSUPPORTED),
    (dict(width=1 << 30, stride=1 << 30), ERR_UNSUPPORTED),
])
def test_slots_host_checks(lib, over, code):
    assert lib.spec_verify_slots(*{**SLOTS, **over}.values()) == code


APPEND = dict(k=P, v=P, kr=1024, kh=128, vr=1024, vh=128, slots=P, rows=4, heads=8, dim=128, kc=P,
              vc=P, sb=16384, st=1024, sh=128, blocks=9, page=16, dtype=0, err=None, stream=None)


@pytest.mark.parametrize("over,code", [
    (dict(dtype=2), ERR_DTYPE), (dict(rows=-1), ERR_ARG), (dict(heads=0), ERR_ARG),
    (dict(page=0), ERR_ARG), (dict(blocks=0), ERR_ARG), (dict(k=None), ERR_ARG),
    (dict(vc=None), ERR_ARG), (dict(slots=P + 4), ERR_ARG), (dict(k=P + 1), ERR_ARG),
    (dict(st=-1), ERR_ARG), (dict(rows=0), 0),
])
def test_append_host_checks(lib, over, code):
    assert lib.spec_verify_append(*{**APPEND, **over}.values()) == code


ATTN = dict(q=P, qr=1024, qh=128, k=P, v=P, sb=16384, st=1024, sh=128, table=P, ts=8, width=8,
            seq=P, offs=P, B=4, rows=8, max_len=4, heads=8, kv=8, dim=128, blocks=9, page=16,
            dtype=0, scale=0.1, window=0, out=P, orow=1024, ohead=128, lse=P, err=P, ws=P,
            ws_bytes=1 << 40, stream=None)


@pytest.mark.parametrize("over,code", [
    (dict(dtype=5), ERR_DTYPE), (dict(B=0), ERR_ARG), (dict(max_len=0), ERR_ARG),
    (dict(heads=9), ERR_ARG), (dict(kv=0), ERR_ARG), (dict(dim=12), ERR_UNSUPPORTED),
    (dict(dim=264), ERR_UNSUPPORTED), (dict(q=None), ERR_ARG), (dict(q=P + 8), ERR_ARG),
    (dict(st=1020), ERR_ARG), (dict(qr=-1024), ERR_ARG), (dict(scale=float("nan")), ERR_ARG),
    (dict(scale=float("inf")), ERR_ARG), (dict(ts=7), ERR_ARG), (dict(seq=None), ERR_ARG),
    (dict(ws=None), ERR_WORKSPACE), (dict(ws=P + 128), ERR_WORKSPACE),
    (dict(ws_bytes=64), ERR_WORKSPACE), (dict(width=1 << 28, ts=1 << 28), ERR_UNSUPPORTED),
    (dict(rows=0), 0),
])
def test_attention_host_checks(lib, over, code):
    assert lib.spec_verify_attention(*[ctypes.c_float(v) if k == "scale" else v
                                       for k, v in {**ATTN, **over}.items()]) == code


def test_attention_workspace_is_aligned(lib):
    for dtype in (0, 1):
        n = lib.spec_verify_attention_workspace_size(512, 32, 128, dtype)
        assert n > 0 and n % 256 == 0
