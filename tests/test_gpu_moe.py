"""A mixture of sparse blocks (nm_moe) against its formula in 64 bits."""
import numpy as np
import pytest
import torch

import oracle as O
from tests import _block as B
from tests import _layers as L
from tests._util import dev, np_bf16

pytestmark = pytest.mark.gpu
BF16 = 1


@pytest.fixture(scope="module")
def nm():
    import semi_structured_sparsity_amd as m
    return m


def _x(g, T, K, scale=1.0):
    X = O.f32_to_bf16((g.standard_normal((T, K)) * scale).astype(np.float32))
    return np_bf16(X).to(dev()), O.bf16_to_f32(X).astype(np.float64)


def _stack(nm, g, E, R, K, Ns, vdt, group, apart):
    """E experts' weights stacked, with gaps between experts and rows where apart: (dense [E, R, K], vals, idx, scales)."""
    dense, parts = [], []
    for _ in range(E):
        if vdt == BF16:
            W, v, i = B.weight(g, R, K, Ns, scale=1 / np.sqrt(K))
            s = None
        else:
            W, v, i, s = L.w4_weight(nm, g, R, K, Ns, vdt, group)
            s = s.as_strided((s.shape[0], -(-R // 4) * 4), (s.stride(0), 1))
        dense.append(W)
        parts.append((v, i, s))

    def stack(ts, unit):
        if ts[0] is None:
            return None
        r, c = ts[0].shape
        pr, pc = (r + 2, (c + 2 * unit - 1) // unit * unit) if apart else (r, (c + unit - 1) // unit * unit)
        out = torch.zeros((len(ts), pr, pc), dtype=ts[0].dtype, device=dev())
        if ts[0].dtype == torch.bfloat16:
            out.fill_(float("nan"))
        for k, t in enumerate(ts):
            out[k, :r, :c] = t
        return out[:, :r, :c]
    v = stack([p[0] for p in parts], 8 if vdt == BF16 else 16)
    i = stack([p[1] for p in parts], 1)
    s = stack([p[2] for p in parts], 4)
    return np.stack(dense), v, i, s


def _layer(nm, g, E, K, F, Ns, vdt, group, bias=False, apart=False, router=None):
    gd, gv, gi, gs = _stack(nm, g, E, F, K, Ns, vdt, group, apart)
    ud, uv, ui, us = _stack(nm, g, E, F, K, Ns, vdt, group, apart)
    dd, dv, di, ds = _stack(nm, g, E, K, F, Ns, vdt, group, apart)
    if router is None:
        router = _x(g, E, K, K ** -0.5)
    b = (0.2 * g.standard_normal(E)).astype(np.float32) if bias else None
    layer = nm.MoELayer(router[0], gv, gi, uv, ui, dv, di, F, vdt=vdt, group=group, Ns=Ns, gate_scales=gs, up_scales=us,
                        down_scales=ds, bias=None if b is None else torch.from_numpy(b).to(dev()))
    return layer, (router[1], gd, ud, dd, b)


def _check(nm, layer, dense, X, Xf, topk, a, route, renorm, scale, ydt, out=None):
    R, gd, ud, dd, b = dense
    T, K = Xf.shape
    E, F = gd.shape[:2]
    ws = B.nan_ws(nm.raw.nm_moe_workspace(T, K, F, E, topk))
    Y, sel, wts = nm.nm_moe(layer, X, topk, act=a, route=route, renorm=renorm, route_scale=scale, ydt=ydt, want_routing=True,
                            out=out, ws=ws)
    assert torch.equal(Y.view(torch.uint8) if Y.is_contiguous() else Y,
                       (lambda t: t.view(torch.uint8) if Y.is_contiguous() else t)(
                           nm.nm_moe(layer, X, topk, act=a, route=route, renorm=renorm, route_scale=scale, ydt=ydt)))
    sel, wts = sel.cpu().numpy(), wts.cpu().numpy().astype(np.float64)
    lg = Xf @ R.T
    eL = (K + 8) * 2.0 ** -24 * (np.abs(Xf) @ np.abs(R).T)
    if route == nm.NM_ROUTE_SIGMOID:
        p = B.sigmoid(lg)
    else:
        p = np.exp(lg - lg.max(1, keepdims=True))
        p = p / p.sum(1, keepdims=True)
    # a probability's error: its logit's (and the largest's) twice over, the f32 exponential and sum
    rel = 4 * eL.max(1, keepdims=True) + (E + 16 + 4 * np.abs(lg)) * 2.0 ** -23
    key = lg if b is None else p + b.astype(np.float64)
    eK = eL if b is None else 4 * eL.max(1, keepdims=True) * p + (E + 16) * 2.0 ** -23 * p + 2.0 ** -40
    y = np.zeros((T, K))
    err = np.zeros((T, K))
    for t in range(T):
        assert len(set(sel[t])) == topk and sel[t].min() >= 0 and sel[t].max() < E
        left = np.ones(E, bool)
        for j in range(topk):
            e = sel[t, j]
            assert key[t, e] + eK[t, e] >= (key[t] - eK[t])[left].max()      # the largest left, as far as f32 sums tell
            left[e] = False
        want = p[t, sel[t]]
        r = rel[t, sel[t]].copy()
        if renorm:
            r = r + r.max() + topk * 2.0 ** -24
            want = want / want.sum()
        want, r = scale * want, r + 2 * 2.0 ** -24
        assert (np.abs(wts[t] - want) <= r * np.abs(want) + 1e-37).all()
        for j in range(topk):
            e = sel[t, j]
            G, U = Xf[t:t + 1] @ gd[e].T, Xf[t:t + 1] @ ud[e].T
            eG, eU = L.product_bound(Xf[t:t + 1], gd[e], K), L.product_bound(Xf[t:t + 1], ud[e], K)
            f, d, ra = B.act(a, G)
            H = f * U
            eH = (np.abs(d) * eG + B.CURVE[a] * eG * eG) * (np.abs(U) + eU) + np.abs(f) * eU + ra * np.abs(H) + 2.0 ** -24 * np.abs(H)
            eH += 2.0 ** -8 * (np.abs(H) + eH)          # H's rounding
            D = (H @ dd[e].T)[0]
            eD = (eH @ np.abs(dd[e]).T + L.product_bound(np.abs(H) + eH, dd[e], F))[0]
            y[t] += want[j] * D
            err[t] += np.abs(want[j]) * (1 + r[j]) * eD + r[j] * np.abs(want[j] * D) + (topk + 8) * 2.0 ** -24 * np.abs(want[j] * D)
    got = Y.float().cpu().numpy().astype(np.float64)
    assert np.isfinite(got).all()
    tol = err + (2.0 ** -8 if ydt == nm.NM_BF16 else 2.0 ** -24) * (np.abs(y) + err) + 1e-37
    assert (np.abs(got - y) <= tol).all(), float((np.abs(got - y) / tol).max())
    return sel


@pytest.mark.parametrize("T,E,topk,K,F", [(1, 1, 1, 16, 16), (1, 8, 2, 256, 128), (1, 64, 8, 512, 144), (2, 70, 5, 272, 64),
                                          (5, 4, 4, 320, 80), (16, 16, 2, 512, 256), (17, 8, 1, 128, 272), (40, 3, 2, 1040, 528),
                                          (64, 130, 16, 64, 32), (64, 2, 1, 256, 48), (7, 300, 3, 48, 16), (3, 512, 16, 32, 16)])
@pytest.mark.parametrize("vdt", [BF16, L.I4, L.FP4])
def test_layer(nm, T, E, topk, K, F, vdt):
    g = np.random.default_rng(T + E + K + F + vdt)
    layer, dense = _layer(nm, g, E, K, F, 0, vdt, (64, 128, 256)[T % 3])
    X, Xf = _x(g, T, K)
    _check(nm, layer, dense, X, Xf, topk, B.SILU, nm.NM_ROUTE_SOFTMAX, True, 1.0, nm.NM_F32)
    _check(nm, layer, dense, X, Xf, topk, B.GELU, nm.NM_ROUTE_SIGMOID, False, 2.5, nm.NM_BF16)


@pytest.mark.parametrize("Ns,K,F", [(3, 96, 48), (4, 512, 288), (5, 160, 80), (6, 96, 192), (7, 112, 224), (8, 256, 128)])
@pytest.mark.parametrize("vdt", [BF16, L.I4, L.FP4])
def test_lifted_experts_apart(nm, Ns, K, F, vdt):
    """Windows of (2N-2):2N weights, experts and rows with gaps of NaN between them, strided tokens and outputs."""
    g = np.random.default_rng(K + F + vdt)
    layer, dense = _layer(nm, g, 6, K, F, Ns, vdt, 64, bias=True, apart=True)
    X, Xf = _x(g, 9, K)
    out = B.strided(torch.zeros((9, K), dtype=torch.float32, device=dev()), 5)
    _check(nm, layer, dense, B.strided(X, 8), Xf, 3, B.GELU_TANH, nm.NM_ROUTE_SIGMOID, True, 1.5, nm.NM_F32, out=out)
    assert torch.isnan(out.as_strided((8, 5), (K + 5, 1), K)).all()
    _check(nm, layer, dense, X, Xf, 6, B.RELU2, nm.NM_ROUTE_SOFTMAX, False, 1.0, nm.NM_BF16)


@pytest.mark.parametrize("vdt", [BF16, L.I4])
@pytest.mark.parametrize("T", [1, 9])
def test_experts_gigabytes_apart(nm, T, vdt):
    """Experts whose values, positions and scales start more than 2^32 bytes after the one before."""
    g = np.random.default_rng(T + vdt)
    K, F, E = 128, 64, 3
    weights, dense = [], []
    for rows, width in ((F, K), (F, K), (K, F)):
        d, v, i, s = _stack(nm, g, E, rows, width, 0, vdt, 64, False)
        dense.append(d)
        weights.append((v, i, s))

    def spread(t):
        _, r, c = t.shape
        rs, far = t.stride(1), ((1 << 32) + 256) // t.element_size()
        out = torch.empty((E - 1) * far + r * rs, dtype=t.dtype, device=dev()).as_strided((E, r, c), (far, rs, 1))
        out.copy_(t)
        return out
    far_w = [[None if t is None else spread(t) for t in w] for w in weights]
    router = _x(g, E, K, K ** -0.5)
    (gv, gi, gs), (uv, ui, us), (dv, di, ds) = far_w
    layer = nm.MoELayer(router[0], gv, gi, uv, ui, dv, di, F, vdt=vdt, group=64, gate_scales=gs, up_scales=us, down_scales=ds)
    X, Xf = _x(g, T, K)
    _check(nm, layer, (router[1], *dense, None), X, Xf, 3, B.SILU, nm.NM_ROUTE_SOFTMAX, True, 1.0, nm.NM_F32)


@pytest.mark.parametrize("E", [4, 65, 200])
def test_equal_scores_go_to_the_lower_index(nm, E):
    """Router rows of small integers: exact logits, most of them equal."""
    g = np.random.default_rng(E)
    r = O.f32_to_bf16(g.integers(-1, 2, (E, 16)).astype(np.float32))
    layer, _ = _layer(nm, g, E, 16, 16, 0, BF16, 64, router=(np_bf16(r).to(dev()), None))
    x = g.integers(-1, 2, (20, 16)).astype(np.float32)
    x[3] = 0
    X = np_bf16(O.f32_to_bf16(x)).to(dev())
    lg = x.astype(np.float64) @ O.bf16_to_f32(r).astype(np.float64).T
    want = np.argsort(-lg, axis=1, kind="stable")[:, :4]
    for route in (nm.NM_ROUTE_SOFTMAX, nm.NM_ROUTE_SIGMOID):
        sel = nm.nm_moe(layer, X, 4, route=route, want_routing=True)[1]
        assert np.array_equal(sel.cpu().numpy(), want)
    # a bias of zeros: the same order, by probability
    layer.bias = torch.zeros(E, device=dev())
    assert np.array_equal(nm.nm_moe(layer, X, 4, want_routing=True)[1].cpu().numpy(), want)


def test_a_token_of_nan_stays_alone(nm):
    """Its row is NaN, the others are as without it; its experts are valid ones."""
    g = np.random.default_rng(2)
    layer, _ = _layer(nm, g, 8, 64, 32, 0, L.FP4, 64)
    X, _ = _x(g, 6, 64)
    ref = nm.nm_moe(layer, X, 2)
    X[4] = float("nan")
    Y, sel, _ = nm.nm_moe(layer, X, 2, want_routing=True)
    assert torch.isnan(Y[4]).all() and sel.min() >= 0 and sel.max() < 8
    keep = [0, 1, 2, 3, 5]
    assert torch.equal(Y[keep], ref[keep])


def _routed(nm, E, T, logits, topk, route, renorm, bias):
    """(experts, weights) of tokens that all have the given logits, rounded to bf16: column 0 of the router times 1."""
    g = np.random.default_rng(E + T)
    r = torch.zeros((E, 16))
    r[:, 0] = torch.from_numpy(np.asarray(logits, np.float32))
    layer, _ = _layer(nm, g, E, 16, 16, 0, BF16, 64, bias=True, router=(r.bfloat16().to(dev()), None))
    layer.bias.copy_(torch.from_numpy(np.asarray(bias, np.float32)))
    X = torch.zeros((T, 16), dtype=torch.bfloat16, device=dev())
    X[:, 0] = 1
    _, sel, wts = nm.nm_moe(layer, X, topk, route=route, renorm=renorm, want_routing=True)
    return sel.cpu().numpy(), wts.cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("E", [8, 100, 500])
@pytest.mark.parametrize("T", [1, 6])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_infinite_logits_with_a_bias(nm, E, T, sigmoid):
    """A logit of -inf is a probability of 0 (and +inf a sigmoid of 1): its expert is placed by its bias."""
    lg = np.tile([-1.0, -np.inf, 0.5, -np.inf], E)[:E]
    if sigmoid:
        lg[4] = np.inf
    p = B.sigmoid(lg) if sigmoid else np.exp(lg - lg.max()) / np.exp(lg - lg.max()).sum()
    rising = np.linspace(0.0, 3.0, E)
    for bias in (rising, rising + 10.0 * np.isinf(lg)):
        want = np.argsort(-(p + bias.astype(np.float32)), kind="stable")[:5]
        sel, wts = _routed(nm, E, T, lg, 5, nm.NM_ROUTE_SIGMOID if sigmoid else nm.NM_ROUTE_SOFTMAX, False, bias)
        assert (sel == want).all()
        # a probability of f32: the exponential and the sum of E of them
        assert (np.abs(wts - p[want]) <= (E + 20) * 2.0 ** -23 * p[want]).all()


@pytest.mark.parametrize("E", [8, 100, 500])
@pytest.mark.parametrize("T", [1, 6])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_weights_of_probabilities_below_the_types_range(nm, E, T, sigmoid):
    """Divided by their sum they are ordinary numbers: all of the sigmoid's, and those behind a softmax's top."""
    lg = -100.0 - 0.5 * np.arange(E)
    lg[0] = -100.0 if sigmoid else 60.0
    lg = torch.from_numpy(lg).bfloat16().double().numpy()
    bias = np.zeros(E)
    bias[2:6] = [4, 3, 2.5, 2]        # experts 2 to 5, whatever their probabilities
    sel, wts = _routed(nm, E, T, lg, 4, nm.NM_ROUTE_SIGMOID if sigmoid else nm.NM_ROUTE_SOFTMAX, True, bias)
    assert (sel == [2, 3, 4, 5]).all()
    d = lg[2:6] - lg[2]
    want = np.exp(d) / np.exp(d).sum()          # a sigmoid this far below 0 is its exponential to 1e-43
    # an f32 exponential of d and (the sigmoid's) its reciprocal, twice for the sum, three more roundings
    tol = (2 * (2 * np.abs(d).max() + 4) + 7) * 2.0 ** -23
    assert (np.abs(wts - want) <= tol * want).all(), np.abs(wts / want - 1).max() / tol


def test_a_new_bias_is_checked(nm):
    g = np.random.default_rng(4)
    layer, _ = _layer(nm, g, 8, 64, 32, 0, BF16, 64)
    for bad in (torch.zeros(7, device=dev()), torch.zeros(8, dtype=torch.bfloat16, device=dev()), torch.zeros(16, device=dev())[::2],
                torch.zeros(8), torch.zeros((1, 8), device=dev())):
        with pytest.raises(ValueError):
            layer.bias = bad
    layer.bias = torch.zeros(8, device=dev())
    layer.bias = None


def test_every_token_on_one_expert(nm):
    """A bias sends all 64 tokens to one expert; the others' weights of NaN are not read."""
    g = np.random.default_rng(3)
    layer, dense = _layer(nm, g, 5, 128, 64, 0, BF16, 64, bias=True)
    layer.bias.copy_(torch.tensor([0, 0, 0, 9.0, 0]))
    dense[4][:] = [0, 0, 0, 9, 0]
    for k in (1, 4, 7):     # gate, up, down values
        for e in (0, 1, 2, 4):
            layer.keep[k][e] = float("nan")
    X, Xf = _x(g, 64, 128)
    sel = _check(nm, layer, dense, X, Xf, 1, B.SILU, nm.NM_ROUTE_SOFTMAX, False, 1.0, nm.NM_F32)
    assert (sel == 3).all()


def test_graph_and_stream(nm):
    """Captured once, replayed with other tokens between eager calls; on a stream of its own."""
    g = np.random.default_rng(9)
    layer, _ = _layer(nm, g, 16, 256, 128, 0, L.I4, 128)
    X, _ = _x(g, 3, 256)
    ws = torch.empty(nm.raw.nm_moe_workspace(3, 256, 128, 16, 4), dtype=torch.uint8, device=dev())
    eager = nm.nm_moe(layer, X, 4)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        side = nm.nm_moe(layer, X, 4)
    torch.cuda.synchronize()
    assert torch.equal(side, eager)
    out, graph = torch.empty_like(eager), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nm.nm_moe(layer, X, 4, out=out, ws=ws)
    for k in range(4):
        X.copy_(_x(np.random.default_rng(30 + k), 3, 256)[0])
        out.fill_(float("nan"))
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, nm.nm_moe(layer, X, 4))


def test_wrappers_refuse(nm):
    g = np.random.default_rng(1)
    layer, _ = _layer(nm, g, 4, 64, 32, 0, L.I4, 64)
    X, _ = _x(g, 2, 64)
    nm.nm_moe(layer, X, 2)
    assert nm.nm_moe(layer, X[:0], 2).shape == (0, 64)
    for bad in (dict(X=X.float()), dict(X=X[:, :48]), dict(X=X.cpu()), dict(topk=0), dict(topk=5), dict(act=9), dict(route=2),
                dict(out=torch.zeros((2, 32), device=dev())), dict(X=_x(g, 65, 64)[0])):
        with pytest.raises((ValueError, nm.NMError)):
            nm.nm_moe(layer, **{"X": X, "topk": 2, **bad})
    k = layer.keep
    ok = dict(router=k[0], gate=k[1], gate_idx=k[2], gate_scales=k[3], up=k[4], up_idx=k[5], up_scales=k[6], down=k[7], down_idx=k[8],
              down_scales=k[9], hidden=32, vdt=L.I4, group=64)
    nm.MoELayer(**ok)
    for bad in (dict(router=k[0].float()), dict(gate=k[1][:3]), dict(up_idx=k[5][:, :, :1]), dict(down_scales=None), dict(vdt=BF16), dict(vdt=4),
                dict(hidden=64), dict(Ns=2), dict(bias=torch.zeros(3, device=dev())), dict(gate_scales=k[3].cpu())):
        with pytest.raises(ValueError):
            nm.MoELayer(**{**ok, **bad})
