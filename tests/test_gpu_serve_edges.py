"""Edges of the paged serving operators on the GPU: tokens without weight,
requests that get no pages, calls without rows, scales and windows at the ends of
their ranges, many rows of a real vocabulary."""

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
