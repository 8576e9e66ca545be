"""The AdamW step where second moments are below f32's normal range: with eps of 0 the update is still
l m / (1 - b1^t) / sqrt(v / (1 - b2^t)), not m over a root flushed to zero."""
import numpy as np
import pytest
import torch

from tests._util import dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("g", [1e-18, 2e-19, 1e-19, 7e-21, 3e-22])
def test_adamw_second_moments_below_the_normal_range(f8, g):
    import semi_structured_sparsity_amd as nm
    n, lr, b1, b2, step = 300, 0.1, 0.9, 0.95, 2
    dt = torch.float8_e4m3fn if f8 else torch.float32
    p, gr = torch.full((n,), 3.0, device=dev()), torch.full((n,), g, device=dev())
    m, v = (torch.zeros(n, device=dev()).to(dt) for _ in range(2))
    ms, vs = (torch.zeros(2, device=dev()) for _ in range(2))
    t = nm.AdamWTensors([p], [gr], [m], [v], [ms] if f8 else None, [vs] if f8 else None)
    nm.nm_adamw(t, lr=lr, step=step, beta1=b1, beta2=b2, eps=0.0)
    # the states in f32, one rounding per operation (v loses bits below 2^-126: it is an input of the rest)
    f = np.float32
    m1, v1 = f(f(1 - b1) * f(g)), f(f(f(1 - b2) * f(g)) * f(g))
    assert 0 < v1 < 2.0 ** -125 * 1e3
    want = 3.0 - lr / (1 - b1 ** step) * float(m1) / np.sqrt(float(v1) / (1 - b2 ** step))
    # a reciprocal (2^-22), and one rounding of each of four operations and of p
    upd = abs(3.0 - want)
    assert torch.isfinite(p).all() and (p.double() - want).abs().max().item() <= 2.0 ** -20 * upd + 2.0 ** -23 * 3.0
    if not f8:
        assert (m == float(m1)).all() and (v == float(v1)).all()
