"""Gradients of the packed layer (nm_spmm_backward) and of the gated block
(nm_spmm_glu_backward) against their formulas in 64 bits and against differences of the
forward pass in 64 bits."""
import numpy as np
import pytest
import torch

import oracle as O
from tests import _block as B
from tests._util import dev, np_bf16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nm():
    import semi_structured_sparsity_amd as m
    return m


def _rand(g, shape, scale=1.0, integer=0):
    b = O.f32_to_bf16((g.integers(-integer, integer + 1, shape) if integer else g.standard_normal(shape) * scale)
                      .astype(np.float32))
    return np_bf16(b).to(dev()), O.bf16_to_f32(b).astype(np.float64)


def _np(t):
    return t.float().cpu().numpy().astype(np.float64)


# (the last five: weights large enough that dX's tiles decode them, ragged everywhere, and many tokens of
# small weights, which split dV's sum)
SIZES = [(1, 1, 16), (1, 64, 64), (3, 70, 48), (17, 33, 272), (64, 64, 64), (65, 130, 528), (129, 200, 1024),
         (200, 1000, 272), (300, 257, 512), (513, 520, 784),
         (130, 4100, 4112), (257, 8195, 2064), (600, 2111, 8208), (1400, 130, 272), (900, 301, 528)]


@pytest.mark.parametrize("Mt,R,K", SIZES)
@pytest.mark.parametrize("extra", [0, 8, 3])
def test_backward_integers_exact(nm, Mt, R, K, extra):
    """Small integers: every product and sum is exact in f32, so every value is."""
    g = np.random.default_rng(Mt + R + K + extra)
    dY, dYf = _rand(g, (Mt, R), integer=2)
    X, Xf = _rand(g, (Mt, K), integer=2)
    W, v, i = B.weight(g, R, K, integer=True)
    if extra:
        dY, X, v, i = B.strided(dY, extra), B.strided(X, 16), B.strided(v, 16), B.strided(i, extra)
    ws = B.nan_ws(nm.raw.nm_spmm_backward_workspace(Mt, K, R, 0))
    dX, dV = nm.nm_spmm_backward(dY, X, v, i, dxdt=nm.NM_F32, dvdt=nm.NM_F32, ws=ws)
    assert np.array_equal(_np(dX), dYf @ W)
    assert np.array_equal(_np(dV), B.take(dYf.T @ Xf, i.contiguous(), K))
    ws.fill_(0xFF)
    dX2, dV2 = nm.nm_spmm_backward(dY, X, v, i, ws=ws)
    assert torch.equal(dX2, dX.to(torch.bfloat16)) and torch.equal(dV2, dV.to(torch.bfloat16))


@pytest.mark.parametrize("Mt,R,K", [(1, 300, 512), (200, 130, 1040), (700, 1000, 512), (1500, 300, 2048), (64, 4096, 1024)])
def test_backward_random(nm, Mt, R, K):
    g = np.random.default_rng(Mt * 3 + R + K)
    dY, dYf = _rand(g, (Mt, R), 0.1)
    X, Xf = _rand(g, (Mt, K))
    W, v, i = B.weight(g, R, K)
    dX, dV = nm.nm_spmm_backward(dY, X, v, i, dxdt=nm.NM_F32, dvdt=nm.NM_F32)
    assert (np.abs(_np(dX) - dYf @ W) <= (R + 16) * 2.0 ** -24 * (np.abs(dYf) @ np.abs(W)) + 1e-37).all()
    tol = (Mt + 16) * 2.0 ** -24 * (np.abs(dYf).T @ np.abs(Xf)) + 1e-37
    assert (np.abs(_np(dV) - B.take(dYf.T @ Xf, i, K)) <= B.take(tol, i, K)).all()


@pytest.mark.parametrize("Mt,R,K", SIZES)
@pytest.mark.parametrize("extra", [0, 8, 3])
def test_glu_backward_integers_exact(nm, Mt, R, K, extra):
    """With max(g, 0)^2 and small integers dG and dU are exact in bf16 (below 2^8) and every sum
    is exact in f32."""
    g = np.random.default_rng(Mt + R + K + extra)
    dH, dHf = _rand(g, (Mt, R), integer=1)
    G, Gf = _rand(g, (Mt, R), integer=4)
    U, Uf = _rand(g, (Mt, R), integer=4)
    X, Xf = _rand(g, (Mt, K), integer=2)
    Wg, vg, ig = B.weight(g, R, K, integer=True)
    Wu, vu, iu = B.weight(g, R, K, integer=True)
    if extra:
        dH, G, U, X = B.strided(dH, extra), B.strided(G, extra), B.strided(U, extra), B.strided(X, 8)
        vg, vu, ig, iu = B.strided(vg, 8), B.strided(vu, 8), B.strided(ig, extra), B.strided(iu, extra)
    f, d, _ = B.act(B.RELU2, Gf)
    dG, dU = dHf * Uf * d, dHf * f
    ws = B.nan_ws(nm.raw.nm_spmm_glu_backward_workspace(Mt, K, R, 0))
    dX, dVg, dVu = nm.nm_spmm_glu_backward(dH, G, U, X, vg, ig, vu, iu, act=B.RELU2, dxdt=nm.NM_F32, dvdt=nm.NM_F32, ws=ws)
    assert np.array_equal(_np(dX), dG @ Wg + dU @ Wu)
    assert np.array_equal(_np(dVg), B.take(dG.T @ Xf, ig.contiguous(), K))
    assert np.array_equal(_np(dVu), B.take(dU.T @ Xf, iu.contiguous(), K))
    ws.fill_(0xFF)
    only, n1, n2 = nm.nm_spmm_glu_backward(dH, G, U, X, vg, ig, vu, iu, act=B.RELU2, want_dv=False, ws=ws)
    assert n1 is None and n2 is None and torch.equal(only, dX.to(torch.bfloat16))
    n1, a, b = nm.nm_spmm_glu_backward(dH, G, U, X, vg, ig, vu, iu, act=B.RELU2, want_dx=False, ws=ws)
    assert n1 is None and torch.equal(a, dVg.to(torch.bfloat16)) and torch.equal(b, dVu.to(torch.bfloat16))


# (2N-2):2N weights: every N, tokens on both sides of each kernel's range, the last two decoded by
# dX's tiles; row lengths that are no multiple of 8 among them (N = 3, 5, 7)
LIFTED = [(3, 1, 40, 12), (3, 140, 130, 540), (4, 17, 33, 224), (4, 300, 257, 512), (5, 64, 70, 170), (5, 520, 260, 1310),
          (6, 33, 100, 528), (6, 700, 200, 480), (7, 100, 130, 308), (7, 800, 120, 644), (8, 128, 65, 448), (8, 200, 90, 320),
          (4, 130, 6161, 2080), (7, 300, 4100, 2548), (4, 1100, 70, 160)]


@pytest.mark.parametrize("Ns,Mt,R,K", LIFTED)
@pytest.mark.parametrize("extra", [0, 8])
def test_lifted_backward_integers_exact(nm, Ns, Mt, R, K, extra):
    g = np.random.default_rng(Ns + Mt + R + K + extra)
    dY, dYf = _rand(g, (Mt, R), integer=2)
    X, Xf = _rand(g, (Mt, K), integer=2)
    W, v, i = B.weight(g, R, K, Ns=Ns, integer=True)
    X = B.strided(X, 8 - K % 8 if K % 8 else extra)      # rows of 16-byte alignment
    if extra:
        dY, v, i = B.strided(dY, extra), B.strided(v, 16), B.strided(i, extra)
    ws = B.nan_ws(nm.raw.nm_spmm_backward_workspace(Mt, K, R, Ns))
    dX, dV = nm.nm_spmm_backward(dY, X, v, i, Ns=Ns, dxdt=nm.NM_F32, dvdt=nm.NM_F32, ws=ws)
    assert np.array_equal(_np(dX), dYf @ W)
    assert np.array_equal(_np(dV), B.take(dYf.T @ Xf, i.contiguous(), K, Ns))
    ws.fill_(0xFF)
    dX2, dV2 = nm.nm_spmm_backward(dY, X, v, i, Ns=Ns, ws=ws)
    assert torch.equal(dX2, dX.to(torch.bfloat16)) and torch.equal(dV2, dV.to(torch.bfloat16))
    only, n1 = nm.nm_spmm_backward(dY, X, v, i, Ns=Ns, want_dv=False, ws=ws)
    assert n1 is None and torch.equal(only, dX2)


@pytest.mark.parametrize("Ns,Mt,R,K", LIFTED)
def test_lifted_glu_backward_integers_exact(nm, Ns, Mt, R, K):
    g = np.random.default_rng(Ns + Mt + R + K)
    dH, dHf = _rand(g, (Mt, R), integer=1)
    G, Gf = _rand(g, (Mt, R), integer=4)
    U, Uf = _rand(g, (Mt, R), integer=4)
    X, Xf = _rand(g, (Mt, K), integer=2)
    X = B.strided(X, -K % 8)
    Wg, vg, ig = B.weight(g, R, K, Ns=Ns, integer=True)
    Wu, vu, iu = B.weight(g, R, K, Ns=Ns, integer=True)
    f, d, _ = B.act(B.RELU2, Gf)
    dG, dU = dHf * Uf * d, dHf * f
    ws = B.nan_ws(nm.raw.nm_spmm_glu_backward_workspace(Mt, K, R, Ns))
    dX, dVg, dVu = nm.nm_spmm_glu_backward(dH, G, U, X, vg, ig, vu, iu, Ns=Ns, act=B.RELU2, dxdt=nm.NM_F32,
                                           dvdt=nm.NM_F32, ws=ws)
    assert np.array_equal(_np(dX), dG @ Wg + dU @ Wu)
    assert np.array_equal(_np(dVg), B.take(dG.T @ Xf, ig, K, Ns))
    assert np.array_equal(_np(dVu), B.take(dU.T @ Xf, iu, K, Ns))


def test_lifted_backward_adds_windows(nm):
    """Two slots may place a value at one column: dX sees their sum, and each slot has the
    column's derivative."""
    Ns, Mt, R, K = 4, 3, 8, 32
    g = np.random.default_rng(12)
    dY, dYf = _rand(g, (Mt, R), integer=2)
    X, Xf = _rand(g, (Mt, K), integer=2)
    v, vf = _rand(g, (R, O.lifted_width(K, Ns) // 2), integer=3)
    # pairs of ascending positions in every window
    pairs = np.array([(a, b) for a in range(4) for b in range(a + 1, 4)])[g.integers(0, 6, (R, 12))].reshape(R, 24)
    words = np.zeros((R, 2), np.uint32)
    for j in range(24):
        words[:, j // 16] |= (pairs[:, j].astype(np.uint32) << np.uint32(2 * (j % 16)))
    i = torch.from_numpy(words.view(np.int32)).to(dev())
    cols = B.columns(i, K, Ns)
    W = np.zeros((R, K))
    np.add.at(W, (np.arange(R)[:, None], cols), vf)
    assert any(len(set(c)) < len(c) for c in cols)
    dX, dV = nm.nm_spmm_backward(dY, X, v, i, Ns=Ns, dxdt=nm.NM_F32, dvdt=nm.NM_F32)
    assert np.array_equal(_np(dX), dYf @ W)
    assert np.array_equal(_np(dV), np.take_along_axis(dYf.T @ Xf, cols, axis=1))
    assert np.array_equal(_np(nm.nm_spmm(X, v, i, Ns=Ns, ydt=nm.NM_F32)), Xf @ W.T)


@pytest.mark.parametrize("Ns,Mt,R,K", [(4, 20, 300, 512), (5, 700, 200, 640)])
def test_lifted_backward_random(nm, Ns, Mt, R, K):
    g = np.random.default_rng(Mt)
    dY, dYf = _rand(g, (Mt, R), 0.1)
    X, Xf = _rand(g, (Mt, K))
    W, v, i = B.weight(g, R, K, Ns=Ns)
    dX, dV = nm.nm_spmm_backward(dY, X, v, i, Ns=Ns, dxdt=nm.NM_F32, dvdt=nm.NM_F32)
    # a column's two windows are one sum more
    assert (np.abs(_np(dX) - dYf @ W) <= (R + 17) * 2.0 ** -24 * (np.abs(dYf) @ np.abs(W)) + 1e-37).all()
    tol = (Mt + 16) * 2.0 ** -24 * (np.abs(dYf).T @ np.abs(Xf)) + 1e-37
    assert (np.abs(_np(dV) - B.take(dYf.T @ Xf, i, K, Ns)) <= B.take(tol, i, K, Ns)).all()


def _operands(a, dHf, Gf, Uf):
    """dG and dU in 64 bits, and the error of their evaluation in f32."""
    f, d, rel = B.act(a, Gf)
    dG, dU = dHf * Uf * d, dHf * f
    # act' is a sum of terms of at most |g| + 1 in size, each with the activation's error
    eG = 2.0 ** -22 * np.abs(dG) + np.abs(dHf * Uf) * rel * (1 + np.abs(Gf))
    eU = 2.0 ** -22 * np.abs(dU) + np.abs(dHf * f) * rel
    return dG, dU, eG, eU


def _rounded(x, e):
    """x as a bf16 operand, and how far an operand evaluated with the error e may be from it: the
    two agree unless that error moves x across a midpoint, then they are one unit apart."""
    r = B.bf16(x)
    return r, np.maximum(np.abs(B.bf16(x + 1.01 * e) - r), np.abs(B.bf16(x - 1.01 * e) - r))


@pytest.mark.parametrize("Mt,R,K", [(1, 100, 256), (130, 257, 528), (400, 600, 512)])
@pytest.mark.parametrize("a", B.ACTS)
def test_glu_backward_random(nm, Mt, R, K, a):
    g = np.random.default_rng(Mt + R + K + a)
    dH, dHf = _rand(g, (Mt, R), 0.1)
    G, Gf = _rand(g, (Mt, R), 2.0)
    U, Uf = _rand(g, (Mt, R))
    X, Xf = _rand(g, (Mt, K))
    Wg, vg, ig = B.weight(g, R, K)
    Wu, vu, iu = B.weight(g, R, K)
    dG, dU, eG, eU = _operands(a, dHf, Gf, Uf)
    dG, eG = _rounded(dG, eG)
    dU, eU = _rounded(dU, eU)
    dX, dVg, dVu = nm.nm_spmm_glu_backward(dH, G, U, X, vg, ig, vu, iu, act=a, dxdt=nm.NM_F32, dvdt=nm.NM_F32)
    n = (2 * R + 16) * 2.0 ** -24
    tol = eG @ np.abs(Wg) + eU @ np.abs(Wu) + n * 1.01 * (np.abs(dG) @ np.abs(Wg) + np.abs(dU) @ np.abs(Wu))
    assert (np.abs(_np(dX) - (dG @ Wg + dU @ Wu)) <= tol).all()
    for got, d, e, i in ((dVg, dG, eG, ig), (dVu, dU, eU, iu)):
        tol = e.T @ np.abs(Xf) + (Mt + 16) * 1.01 * 2.0 ** -24 * (np.abs(d).T @ np.abs(Xf))
        assert (np.abs(_np(got) - B.take(d.T @ Xf, i, K)) <= B.take(tol, i, K)).all()


@pytest.mark.parametrize("a", B.ACTS)
def test_glu_backward_against_differences(nm, a):
    """Differences of the 64-bit forward pass sum(C . H) along single values of X and of the
    weights.  The kernel differentiates at the rounded G and U, at most 2^-8 away from the
    exact ones, so each gradient may differ by that step times the second derivatives."""
    g = np.random.default_rng(40 + a)
    Mt, R, K = 6, 40, 64
    C, Cf = _rand(g, (Mt, R))
    X, Xf = _rand(g, (Mt, K))
    Wg, vg, ig = B.weight(g, R, K, scale=0.2)
    Wu, vu, iu = B.weight(g, R, K, scale=0.2)
    H, G, U = nm.nm_spmm_glu(X, vg, ig, vu, iu, act=a, save=True)
    dX, dVg, dVu = (_np(t) for t in nm.nm_spmm_glu_backward(C, G, U, X, vg, ig, vu, iu, act=a, dxdt=nm.NM_F32,
                                                           dvdt=nm.NM_F32))

    def loss(x, wg, wu):
        return (Cf * B.act(a, x @ wg.T)[0] * (x @ wu.T)).sum()

    Gx, Ux = Xf @ Wg.T, Xf @ Wu.T
    dG, dU, eG, eU = _operands(a, Cf, Gx, Ux)
    eG, eU = eG + 2.0 ** -8 * np.abs(dG), eU + 2.0 ** -8 * np.abs(dU)
    f, d, _ = B.act(a, Gx)
    sG, sU = 2.0 ** -8 * np.abs(Gx), 2.0 ** -8 * np.abs(Ux)
    eG = eG + np.abs(Cf) * (np.abs(d) * sU + B.CURVE[a] * sG * (np.abs(Ux) + sU))
    eU = eU + np.abs(Cf) * (np.abs(d) * sG + B.CURVE[a] * sG * sG)
    h, small = 1e-5, 1e-6
    tX = eG @ np.abs(Wg) + eU @ np.abs(Wu)
    for _ in range(12):
        m, k = g.integers(Mt), g.integers(K)
        e = np.zeros_like(Xf)
        e[m, k] = h
        diff = (loss(Xf + e, Wg, Wu) - loss(Xf - e, Wg, Wu)) / (2 * h)
        assert abs(dX[m, k] - diff) <= tX[m, k] * 1.01 + small
    for got, W, i, err, up in ((dVg, Wg, ig, eG, False), (dVu, Wu, iu, eU, True)):
        cols, t = B.columns(i, K), err.T @ np.abs(Xf)
        for _ in range(12):
            r, j = g.integers(R), g.integers(K // 2)
            e = np.zeros_like(W)
            e[r, cols[r, j]] = h
            diff = (loss(Xf, Wg, W + e) - loss(Xf, Wg, W - e) if up else loss(Xf, W + e, Wu) - loss(Xf, W - e, Wu)) / (2 * h)
            assert abs(got[r, j] - diff) <= t[r, cols[r, j]] * 1.01 + small


def test_backward_against_differences(nm):
    g = np.random.default_rng(77)
    Mt, R, K = 7, 24, 48
    C, Cf = _rand(g, (Mt, R))
    X, Xf = _rand(g, (Mt, K))
    W, v, i = B.weight(g, R, K, scale=0.3)
    dX, dV = (_np(t) for t in nm.nm_spmm_backward(C, X, v, i, dxdt=nm.NM_F32, dvdt=nm.NM_F32))
    cols = B.columns(i, K)
    for _ in range(20):   # the layer is linear: one-sided differences are exact up to rounding
        m, k, r, j = g.integers(Mt), g.integers(K), g.integers(R), g.integers(K // 2)
        e = np.zeros_like(Xf)
        e[m, k] = 1.0
        assert abs(dX[m, k] - (Cf * ((Xf + e) @ W.T - Xf @ W.T)).sum()) < 1e-5
        e = np.zeros_like(W)
        e[r, cols[r, j]] = 1.0
        assert abs(dV[r, j] - (Cf * (Xf @ (W + e).T - Xf @ W.T)).sum()) < 1e-5


@pytest.mark.parametrize("Mt", [5, 300])
def test_backward_values_stay_in_their_rows(nm, Mt):
    """A token row of NaN reaches its own dX row and the weight rows whose dY is involved, and
    nothing outside the outputs is written."""
    g = np.random.default_rng(Mt)
    R, K = 90, 144
    dY, _ = _rand(g, (Mt, R))
    X, _ = _rand(g, (Mt, K))
    _, v, i = B.weight(g, R, K)
    dX0, dV0 = nm.nm_spmm_backward(dY, X, v, i)
    dY[2] = float("nan")
    out_dx = B.strided(torch.zeros((Mt, K), dtype=torch.bfloat16, device=dev()), 5)
    out_dv = B.strided(torch.zeros((R, K // 2), dtype=torch.bfloat16, device=dev()), 8)
    dX, dV = nm.nm_spmm_backward(dY, X, v, i, out_dx=out_dx, out_dv=out_dv)
    keep = torch.arange(Mt, device=dev()) != 2
    assert torch.equal(dX[keep], dX0[keep]) and torch.isnan(dX[2]).all() and torch.isnan(dV).all()
    assert torch.isnan(out_dx.as_strided((Mt - 1, 5), (out_dx.stride(0), 1), K)).all()
    assert torch.isnan(out_dv.as_strided((R - 1, 8), (out_dv.stride(0), 1), K // 2)).all()


def test_backward_empty(nm):
    g = np.random.default_rng(0)
    _, v, i = B.weight(g, 8, 64)
    X = torch.empty((0, 64), dtype=torch.bfloat16, device=dev())
    dY = torch.empty((0, 8), dtype=torch.bfloat16, device=dev())
    out = torch.full((8, 32), float("nan"), device=dev())
    dX, dV = nm.nm_spmm_backward(dY, X, v, i, out_dv=out, dvdt=nm.NM_F32)
    assert dX.shape == (0, 64) and torch.equal(dV, torch.zeros_like(out))
    _, a, b = nm.nm_spmm_glu_backward(dY, dY, dY, X, v, i, v, i)
    assert not a.any() and not b.any()


def test_backward_runs_twice_alike_on_other_streams_and_in_a_graph(nm):
    g = np.random.default_rng(6)
    Mt, R, K = 300, 700, 512
    dY, _ = _rand(g, (Mt, R))
    G, _ = _rand(g, (Mt, R))
    X, _ = _rand(g, (Mt, K))
    _, v, i = B.weight(g, R, K)
    ref = nm.nm_spmm_glu_backward(dY, G, dY, X, v, i, v, i)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        again = nm.nm_spmm_glu_backward(dY, G, dY, X, v, i, v, i)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(ref, again))
    outs = [torch.empty_like(t) for t in ref]
    ws = B.nan_ws(nm.raw.nm_spmm_glu_backward_workspace(Mt, K, R, 0))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nm.nm_spmm_glu_backward(dY, G, dY, X, v, i, v, i, out_dx=outs[0], out_dv=(outs[1], outs[2]), ws=ws)
    for _ in range(3):
        for t in outs:
            t.fill_(float("nan"))
        graph.replay()
        now = nm.nm_spmm_glu_backward(dY, G, dY, X, v, i, v, i)
        assert all(torch.equal(x, y) for x, y in zip(outs, now))


def test_backward_binding_refuses(nm):
    g = np.random.default_rng(2)
    dY, _ = _rand(g, (4, 8))
    X, _ = _rand(g, (4, 64))
    _, v, i = B.weight(g, 8, 64)
    for bad in (lambda: nm.nm_spmm_backward(dY[:3], X, v, i), lambda: nm.nm_spmm_backward(dY, X.float(), v, i),
                lambda: nm.nm_spmm_backward(dY, X, v[:, :8], i), lambda: nm.nm_spmm_backward(dY.t(), X, v, i),
                lambda: nm.nm_spmm_backward(dY, X, v, i, out_dv=torch.empty((8, 31), dtype=torch.bfloat16, device=dev())),
                lambda: nm.nm_spmm_glu_backward(dY, dY, dY[:, :4], X, v, i, v, i),
                lambda: nm.nm_spmm_glu_backward(dY, dY, dY, X, v, i, v[:4], i[:4]),
                lambda: nm.nm_spmm_backward(dY, X, v, i, Ns=5), lambda: nm.nm_spmm_backward(dY, X, v.cpu(), i),
                lambda: nm.nm_spmm_backward(dY, X, v, i, ws=torch.empty(1 << 20, dtype=torch.uint8)),
                lambda: nm.nm_spmm_backward(dY, X, v, i, ws=torch.empty((1, 64), device=dev()).expand(4096, 64))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(nm.NMError):
        nm.nm_spmm_glu_backward(dY, dY, dY, X, v, i, v, i, act=7)
    with pytest.raises(nm.NMError):
        nm.nm_spmm_backward(dY, X, v, i, out_dx=X)
