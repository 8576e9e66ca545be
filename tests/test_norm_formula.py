"""The gradients the norms' tests hold the kernels to, against differences of the forward formula."""
import numpy as np
import pytest

from tests import _rounded as R


@pytest.mark.parametrize("post", [R.NONE, R.RMS, R.LAYER])
@pytest.mark.parametrize("pre", [R.NONE, R.RMS, R.LAYER])
@pytest.mark.parametrize("gated", [False, True])
def test_gradients_are_those_of_differences(post, pre, gated):
    g = np.random.default_rng(post * 6 + pre * 2 + gated)
    M, C, eps, res = 3, 7, 1e-3, 0.7
    p = {"x": g.standard_normal((M, C)), "y": g.standard_normal((M, C)) + 0.5}
    if gated:
        p["gate"] = g.standard_normal((1, C))
    for k, kind in (("p", post), ("n", pre)):
        if kind:
            p["w" + k], p["b" + k] = 1 + 0.3 * g.standard_normal(C), g.standard_normal(C)
    dz, dn = g.standard_normal((M, C)), g.standard_normal((M, C)) if pre else None

    def loss(q):
        z, n = R.forward(q["x"], q["y"], res, q.get("gate"), post, q.get("wp"), q.get("bp"), pre, q.get("wn"), q.get("bn"), eps)
        return (z.v * dz).sum() + (0 if n is None else (n.v * dn).sum())

    z, _ = R.forward(p["x"], p["y"], res, p.get("gate"), post, p.get("wp"), p.get("bp"), pre, p.get("wn"), p.get("bn"), eps)
    got = R.backward(z.v, dz, dn, p["y"], res, p.get("gate"), post, p.get("wp"), p.get("bp"), pre, p.get("wn"), eps)
    names = {"x": "dX", "y": "dY", "gate": "dgate", "wp": "dw_post", "bp": "db_post", "wn": "dw_pre", "bn": "db_pre"}
    for k, t in p.items():
        grad = got[names[k]].v
        if t.shape != grad.shape:
            grad = grad.sum(0).reshape(t.shape)
        for i in np.ndindex(t.shape):
            h = 1e-6
            up, down = ({**p, k: t + s * h * (np.indices(t.shape) == np.reshape(i, (-1,) + (1,) * t.ndim)).all(0)} for s in (1, -1))
            diff = (loss(up) - loss(down)) / (2 * h)
            assert abs(diff - grad[i]) <= 1e-6 * (1 + abs(diff)), (k, i)
