"""The gated block's forward pass (nm_spmm_glu) against its formula in 64 bits."""
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


def _inputs(g, Mt, K, dtype, integer=False):
    """(X on the device, X in f64, x_scale or None)."""
    if dtype == "int8":
        X = g.integers(-127, 128, (Mt, K)).astype(np.int8)
        xs = (g.random(Mt) * 0.02 + 0.001).astype(np.float32)
        return torch.from_numpy(X).to(dev()), X.astype(np.float64), xs
    if dtype == "fp8":
        X = torch.from_numpy((g.integers(-8, 9, (Mt, K)) if integer else g.standard_normal((Mt, K))).astype(np.float32))
        X = X.to(torch.float8_e4m3fn)
        xs = (g.random(Mt) * 0.5 + 0.1).astype(np.float32)
        return X.to(dev()), X.float().numpy().astype(np.float64), xs
    X = O.f32_to_bf16(g.standard_normal((Mt, K)).astype(np.float32))
    return np_bf16(X).to(dev()), O.bf16_to_f32(X).astype(np.float64), None


def _check(nm, Mt, R, K, Ns, a, dtype, hdt, save, seed, extra=0, integer=False):
    g = np.random.default_rng(seed)
    X, Xf, xs = _inputs(g, Mt, K, dtype, integer)
    Wg, vg, ig = B.weight(g, R, K, Ns, dtype=dtype, integer=integer)
    Wu, vu, iu = B.weight(g, R, K, Ns, dtype=dtype, integer=integer)
    gs, us = (1.0, 1.0) if dtype == "bf16" else (0.031, 0.017)
    if extra:
        X = B.strided(X, 16 * extra)
        vg, vu = B.strided(vg, 16 * extra), B.strided(vu, 16 * extra)
        ig, iu = B.strided(ig, extra), B.strided(iu, extra)
    out = None
    if extra:
        out = B.strided(torch.zeros((Mt, R), dtype=torch.float32 if hdt == nm.NM_F32 else torch.bfloat16, device=dev()), 3)
    ws = B.nan_ws(nm.raw.nm_spmm_glu_workspace(Mt, K, R, Ns, nm.dtype_code(X)))
    got = nm.nm_spmm_glu(X, vg, ig, vu, iu, Ns=Ns, act=a, x_scale=None if xs is None else torch.from_numpy(xs).to(dev()),
                         g_scale=gs, u_scale=us, hdt=hdt, save=save, out=out, ws=ws)
    H = (got[0] if save else got).float().cpu().numpy().astype(np.float64)
    sx = np.ones((Mt, 1)) if xs is None else xs[:, None].astype(np.float64)
    sg, su = np.float64(np.float32(gs)) * sx, np.float64(np.float32(us)) * sx
    G, U = Xf @ Wg.T * sg, Xf @ Wu.T * su
    if dtype == "int8" or (dtype == "fp8" and integer):     # exact sums, the scale and the product rounded once each
        eG, eU = 4 * 2.0 ** -24 * np.abs(G), 4 * 2.0 ** -24 * np.abs(U)
    else:
        n = K * 2.0 ** -24 + 4 * 2.0 ** -24
        eG, eU = n * (np.abs(Xf) @ np.abs(Wg).T) * sg, n * (np.abs(Xf) @ np.abs(Wu).T) * su
    f, d, rel = B.act(a, G)
    ref = f * U
    tol = (np.abs(d) * eG + B.CURVE[a] * eG * eG) * (np.abs(U) + eU) + np.abs(f) * eU + rel * np.abs(ref)
    tol += (2.0 ** -8 if hdt == nm.NM_BF16 else 2.0 ** -23) * (np.abs(ref) + tol) + 1e-37
    assert np.isfinite(H).all()
    assert (np.abs(H - ref) <= tol).all(), float((np.abs(H - ref) / tol).max())
    if save:
        for t, r, e in ((got[1], G, eG), (got[2], U, eU)):
            t = t.float().cpu().numpy().astype(np.float64)
            assert (np.abs(t - r) <= e + 2.0 ** -8 * (np.abs(r) + e)).all()
    if extra:
        gap = out.as_strided((Mt, 3), (out.stride(0), 1), R) if Mt > 1 else torch.full((1,), float("nan"))
        assert torch.isnan(gap.float()).all()      # nothing written between the rows


# one token to several tiles, widths on and off the stage grid, rows that fill no tile
@pytest.mark.parametrize("Mt,R,K", [(1, 1, 16), (1, 96, 256), (2, 33, 272), (1, 700, 4096), (5, 130, 512), (16, 700, 1024),
                                    (31, 64, 128), (33, 200, 640), (64, 300, 1024), (65, 129, 512), (100, 520, 768),
                                    (129, 257, 1024), (200, 1000, 512), (256, 130, 256), (257, 300, 512), (520, 400, 768)])
@pytest.mark.parametrize("a", B.ACTS)
def test_glu_bf16(nm, Mt, R, K, a):
    _check(nm, Mt, R, K, 0, a, "bf16", nm.NM_F32, False, Mt + R + K + a)
    _check(nm, Mt, R, K, 0, a, "bf16", nm.NM_BF16, True, Mt + R + K + a + 1)


@pytest.mark.parametrize("dtype", ["bf16", "int8", "fp8"])
@pytest.mark.parametrize("Ns", [0, 3, 4, 5])
@pytest.mark.parametrize("Mt,R", [(1, 300), (3, 97), (40, 130), (70, 64), (130, 300), (300, 260)])
def test_glu_types_and_windows(nm, dtype, Ns, Mt, R):
    K = {0: 512, 3: 768, 4: 1024, 5: 640}[Ns]
    _check(nm, Mt, R, K, Ns, B.RELU2 if dtype == "int8" else B.SILU, dtype, nm.NM_F32, True, Mt * 7 + R + Ns)
    _check(nm, Mt, R, K, Ns, B.GELU_TANH, dtype, nm.NM_BF16, False, Mt * 7 + R + Ns + 1)


# widths that end inside a 256-byte stage, the first one or a later one, on every token range's kernel;
# FP8 on small integers, whose sums are
# exact: the matrix instruction adds products of unlike size with less than f32's precision, which
# few terms do not average out
@pytest.mark.parametrize("dtype,Ns,K", [("bf16", 0, 48), ("bf16", 0, 176), ("bf16", 0, 1104), ("bf16", 4, 64), ("bf16", 4, 896),
                                        ("int8", 0, 96), ("int8", 0, 544), ("int8", 4, 192), ("int8", 4, 1216),
                                        ("fp8", 0, 32), ("fp8", 0, 1184), ("fp8", 4, 320), ("fp8", 4, 960)])
@pytest.mark.parametrize("Mt,R", [(1, 130), (20, 70), (50, 200), (100, 65), (200, 300), (300, 129)])
def test_glu_widths_inside_a_stage(nm, dtype, Ns, K, Mt, R):
    fp8 = dtype == "fp8"
    _check(nm, Mt, R, K, Ns, B.SILU, dtype, nm.NM_F32, True, Mt + R + K + Ns, integer=fp8)
    _check(nm, Mt, R, K, Ns, B.GELU, dtype, nm.NM_BF16, False, Mt + R + K + Ns + 1, extra=1, integer=fp8)


@pytest.mark.parametrize("Mt", [1, 20, 50, 100, 200, 300])
@pytest.mark.parametrize("K,Ns", [(400, 0), (896, 4)])
def test_glu_widths_inside_a_stage_keep_rows_apart(nm, Mt, K, Ns):
    """A weight row or a token row of NaN stays in its own outputs, with rows that follow each other
    without a gap."""
    g = np.random.default_rng(Mt + K)
    R = 100
    X, _, _ = _inputs(g, Mt, K, "bf16")
    _, vg, ig = B.weight(g, R, K, Ns)
    _, vu, iu = B.weight(g, R, K, Ns)
    ref = nm.nm_spmm_glu(X, vg, ig, vu, iu, Ns=Ns, hdt=nm.NM_F32)
    vg[6], vu[51] = float("nan"), float("nan")
    X[Mt // 2] = float("nan")
    H = nm.nm_spmm_glu(X, vg, ig, vu, iu, Ns=Ns, hdt=nm.NM_F32)
    rows, cols = torch.arange(Mt, device=dev()) != Mt // 2, torch.ones(R, dtype=torch.bool, device=dev())
    cols[[6, 51]] = False
    assert torch.isnan(H[~rows]).all() and torch.isnan(H[:, ~cols]).all()
    assert torch.equal(H[rows][:, cols], ref[rows][:, cols])


@pytest.mark.parametrize("dtype,K,Ns", [("bf16", 400, 0), ("int8", 320, 4)])
def test_glu_rows_far_apart(nm, dtype, K, Ns):
    """Token rows whose offsets pass 32 bits: two products and a combination, the same answer."""
    g = np.random.default_rng(K)
    Mt, R, es = 9, 200, 2 if dtype == "bf16" else 1
    X, _, xs = _inputs(g, Mt, K, dtype)
    _, vg, ig = B.weight(g, R, K, Ns, dtype=dtype)
    _, vu, iu = B.weight(g, R, K, Ns, dtype=dtype)
    x_scale = None if xs is None else torch.from_numpy(xs).to(dev())
    far = torch.empty(((Mt - 1) * 2 ** 29 // es + K,), dtype=X.dtype, device=dev()).as_strided((Mt, K), (2 ** 29 // es, 1))
    far.copy_(X)
    near = nm.nm_spmm_glu(X, vg, ig, vu, iu, Ns=Ns, x_scale=x_scale, hdt=nm.NM_F32)
    H = nm.nm_spmm_glu(far, vg, ig, vu, iu, Ns=Ns, x_scale=x_scale, hdt=nm.NM_F32)
    # the sums' orders differ (int8: exact); |terms| of a sum is at most K times its largest
    assert torch.allclose(H, near, rtol=1e-4, atol=1e-4 * near.abs().max().item())


# many-token tiles in whole and ragged rounds, a split of few-token stages
@pytest.mark.parametrize("Mt,R,K,dtype,Ns", [(2048, 1500, 512, "bf16", 0), (1030, 4100, 256, "bf16", 0),
                                             (700, 2100, 1024, "int8", 0), (900, 1900, 512, "fp8", 4),
                                             (128, 4100, 2048, "bf16", 0), (17, 9000, 1024, "bf16", 0),
                                             (8, 6912, 2560, "int8", 4)])
def test_glu_larger(nm, Mt, R, K, dtype, Ns):
    _check(nm, Mt, R, K, Ns, B.SILU, dtype, nm.NM_BF16, True, Mt + R)
    _check(nm, Mt, R, K, Ns, B.GELU, dtype, nm.NM_F32, False, Mt + R + 1)


# rows further apart than their width, on every operand; index rows off 16-byte boundaries
@pytest.mark.parametrize("extra", [1, 4])
@pytest.mark.parametrize("Mt,R,K,dtype", [(1, 96, 512, "bf16"), (9, 130, 1024, "int8"), (70, 130, 512, "bf16"),
                                          (300, 300, 512, "bf16"), (300, 260, 1024, "fp8")])
def test_glu_strides(nm, Mt, R, K, dtype, extra):
    _check(nm, Mt, R, K, 0, B.SILU, dtype, nm.NM_F32, True, Mt + R, extra=extra)
    _check(nm, Mt, R, K, 0, B.SILU, dtype, nm.NM_BF16, False, Mt + R + 1, extra=extra)


@pytest.mark.parametrize("Mt", [1, 40, 130, 300])
def test_glu_large_and_nonfinite_gates(nm, Mt):
    """Gates of any size give the limits of the activation; a NaN or infinite activation row
    touches its own token only."""
    g = np.random.default_rng(Mt)
    R, K = 128, 256
    Wg, vg, ig = B.weight(g, R, K)
    _, vu, iu = B.weight(g, R, K)
    X = np.zeros((Mt, K), np.float32)
    X[:, :] = g.standard_normal((Mt, K)) * 2000
    bad = Mt - 1
    if Mt > 1:
        X[bad, 3] = np.nan
    Xt = torch.from_numpy(X).to(torch.bfloat16).to(dev())
    for a in B.ACTS:
        H = nm.nm_spmm_glu(Xt, vg, ig, vu, iu, act=a, hdt=nm.NM_F32)
        ok = torch.ones(Mt, dtype=torch.bool)
        if Mt > 1:
            ok[bad] = False
        assert torch.isfinite(H.cpu()[ok]).all()
        if Mt > 1:      # rows that keep column 3 see the NaN, in the gate or in the up product
            kept = torch.from_numpy((Wg[:, 3] != 0))
            assert torch.isnan(H.cpu()[bad][kept]).all()


def test_glu_runs_twice_alike_on_other_streams_and_in_a_graph(nm):
    g = np.random.default_rng(5)
    for Mt, R, K in [(1, 11008, 1024), (100, 1000, 1024), (300, 600, 512)]:
        X, _, _ = _inputs(g, Mt, K, "bf16")
        _, vg, ig = B.weight(g, R, K)
        _, vu, iu = B.weight(g, R, K)
        ref = nm.nm_spmm_glu(X, vg, ig, vu, iu)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            again = nm.nm_spmm_glu(X, vg, ig, vu, iu)
        torch.cuda.synchronize()
        assert torch.equal(ref, again)
        out = torch.empty_like(ref)
        ws = B.nan_ws(nm.raw.nm_spmm_glu_workspace(Mt, K, R, 0, nm.NM_BF16))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            nm.nm_spmm_glu(X, vg, ig, vu, iu, out=out, ws=ws)
        for _ in range(3):
            out.fill_(float("nan"))
            ws.fill_(0xFF)
            graph.replay()
            assert torch.equal(out, nm.nm_spmm_glu(X, vg, ig, vu, iu))


def test_glu_empty(nm):
    _, vg, ig = B.weight(np.random.default_rng(0), 8, 64)
    X = torch.empty((0, 64), dtype=torch.bfloat16, device=dev())
    assert nm.nm_spmm_glu(X, vg, ig, vg, ig).shape == (0, 8)


def test_glu_binding_refuses(nm):
    g = np.random.default_rng(1)
    X, _, _ = _inputs(g, 4, 64, "bf16")
    _, vg, ig = B.weight(g, 8, 64)
    with pytest.raises(ValueError):
        nm.nm_spmm_glu(X.t(), vg, ig, vg, ig)
    with pytest.raises(ValueError):
        nm.nm_spmm_glu(X, vg[:, :16], ig, vg, ig)
    with pytest.raises(ValueError):
        nm.nm_spmm_glu(X, vg, ig, vg[:4], ig[:4])
    with pytest.raises(ValueError):
        nm.nm_spmm_glu(X, vg, ig, vg, ig, out=torch.empty((4, 9), dtype=torch.bfloat16, device=dev()))
    with pytest.raises(ValueError):
        nm.nm_spmm_glu(X, vg, ig, vg, ig, x_scale=torch.ones(3, device=dev()))
    with pytest.raises(ValueError):
        nm.nm_spmm_glu(X, vg, ig, vg, ig, ws=torch.empty(1 << 20, dtype=torch.uint8))
    with pytest.raises(nm.NMError):
        nm.nm_spmm_glu(X, vg, ig, vg, ig, act=9)
    with pytest.raises(nm.NMError):
        nm.nm_spmm_glu(X, vg, ig, vg, ig, hdt=nm.NM_F32, out=X.view(torch.float32)[:, :8])


def test_glu_infinite_gates(nm):
    """An infinite pre-activation: max(g, 0)^2 has its limits, and the other activations' positive
    side is infinite."""
    K, R = 64, 8
    v = torch.ones((R, K // 2), dtype=torch.bfloat16, device=dev())
    i = torch.full((R, 2), 0x44444444, dtype=torch.int32, device=dev())      # columns 0 and 1 of every four
    X = torch.zeros((3, K), dtype=torch.bfloat16, device=dev())
    X[0, 0], X[1, 0], X[2, 0] = float("-inf"), float("inf"), 1.0
    up = torch.ones_like(v) * 0.5
    for a in B.ACTS:
        H = nm.nm_spmm_glu(X, v, i, up, i, act=a, hdt=nm.NM_F32).cpu()
        assert torch.isposinf(H[1]).all() and torch.isfinite(H[2]).all()
        if a == B.RELU2:
            assert torch.isnan(H[0]).all()      # 0 times an up product of -inf
    inf = torch.full((1, R), float("-inf"), dtype=torch.bfloat16, device=dev())
    one = torch.ones((1, R), dtype=torch.bfloat16, device=dev())
    X1 = torch.ones((1, K), dtype=torch.bfloat16, device=dev())
    dX, dvg, dvu = nm.nm_spmm_glu_backward(one, inf, one, X1, v, i, up, i, act=B.RELU2)
    assert not dX.any() and not dvg.any() and not dvu.any()
