"""4-bit packed weights: the quantiser bit for bit, the products against their formula in 64 bits."""
import numpy as np
import pytest
import torch

import oracle as O
from tests import _block as B
from tests import _layers as L
from tests._util import dev, np_bf16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nm():
    import semi_structured_sparsity_amd as m
    return m


# ------------------------------------------------------------------ quantiser
def _vals(g, R, slots):
    """Values of unlike size with zero groups, ties, a NaN, infinities and numbers below the normal range."""
    v = g.standard_normal((R, slots)) * np.exp(g.standard_normal((R, 1)))
    v[0, :] = 0
    if R > 3:
        v[1, :8] = [7, -3.5, 2.5, 0.5, -0.5, 1.5, -6.5, 4.5]      # halves of a scale of 1 (and e2m1's borders at 6)
        v[2, :8] = [6, 0.25, -0.75, 1.25, 1.75, -2.5, 3.5, 5]
        v[1, 8:] = v[2, 8:] = 0
        v[3] *= 1e-40
    if R > 6:
        v[4, 3], v[5, 5], v[6, 7] = np.nan, np.inf, -np.inf
    return v.astype(np.float32)


@pytest.mark.parametrize("qdt", [L.I4, L.FP4])
@pytest.mark.parametrize("group", [64, 128, 256])
@pytest.mark.parametrize("R,slots", [(1, 8), (7, 40), (16, 128), (33, 344), (200, 2048)])
@pytest.mark.parametrize("f32", [False, True])
def test_quantiser(nm, qdt, group, R, slots, f32):
    v = _vals(np.random.default_rng(R * slots + group), R, slots)
    t = torch.from_numpy(v) if f32 else np_bf16(O.f32_to_bf16(v))
    v = t.float().numpy()
    codes, scales, values = nm.nm_quant_w4(t.to(dev()), qdt=qdt, group=group, want_values=True)
    rc, rs, rv = L.quant(v, qdt, group)
    assert scales.shape == rs.shape and codes.shape == (R, -(-slots // 32) * 16)
    assert np.array_equal(scales.float().cpu().numpy(), rs, equal_nan=True)
    assert np.array_equal(L.unpack_codes(codes, slots), rc)
    assert not codes[:, slots // 2:].any()
    want = torch.from_numpy(rv).to(torch.float32).to(t.dtype)
    ok = torch.isfinite(want)
    assert torch.equal(values.cpu()[ok], want[ok]) and torch.isnan(values.cpu()[~ok]).all()
    again = nm.nm_quant_w4(t.to(dev()), qdt=qdt, group=group)
    assert len(again) == 2 and torch.equal(again[0], codes)


def test_quantiser_of_strided_rows(nm):
    g = np.random.default_rng(5)
    v = g.standard_normal((9, 72)).astype(np.float32)
    t = B.strided(torch.from_numpy(v).to(dev()), 4)
    codes, scales = nm.nm_quant_w4(t, qdt=nm.NM_FP4, group=64)
    rc, rs, _ = L.quant(v, L.FP4, 64)
    assert np.array_equal(L.unpack_codes(codes, 72), rc) and np.array_equal(scales.float().cpu().numpy(), rs)


# ------------------------------------------------------------------ products
def _x(g, T, K, integer=False):
    X = O.f32_to_bf16((g.integers(-8, 9, (T, K)) if integer else g.standard_normal((T, K))).astype(np.float32))
    return np_bf16(X).to(dev()), O.bf16_to_f32(X).astype(np.float64)


def _close(got, ref, err, bf16):
    got = got.float().cpu().numpy().astype(np.float64)
    tol = err + (2.0 ** -8 if bf16 else 2.0 ** -24) * (np.abs(ref) + err) + 1e-37
    assert np.isfinite(got).all()
    assert (np.abs(got - ref) <= tol).all(), float((np.abs(got - ref) / tol).max())


def _check(nm, T, R, K, Ns, qdt, group, seed, extra=0, integer=False):
    g = np.random.default_rng(seed)
    X, Xf = _x(g, T, K, integer)
    W, codes, idx, scales = L.w4_weight(nm, g, R, K, Ns, qdt, group, integer)
    if extra:
        X, codes, idx = B.strided(X, 8 * extra), B.strided(codes, 16 * extra), B.strided(idx, extra)
    ref, err = Xf @ W.T, L.product_bound(Xf, W, K)
    if integer:
        err = 0 * err
    for ydt in (nm.NM_F32, nm.NM_BF16):
        out = None
        if extra:
            out = B.strided(torch.zeros((T, R), dtype=nm._binding._TORCH[ydt], device=dev()), 3)
        Y = nm.nm_spmm_w4(X, codes, idx, scales, qdt=qdt, group=group, Ns=Ns, ydt=ydt, out=out)
        _close(Y, ref, err, ydt == nm.NM_BF16)
        if extra and T > 1:
            assert torch.isnan(out.as_strided((T - 1, 3), (out.stride(0), 1), R).float()).all()


@pytest.mark.parametrize("T,R,K", [(1, 1, 16), (1, 16, 256), (1, 33, 272), (1, 700, 4096), (3, 50, 48), (5, 130, 512),
                                   (16, 100, 1024), (17, 64, 1040), (31, 96, 768), (33, 200, 640), (64, 100, 1024),
                                   (65, 40, 512), (130, 70, 304)])
@pytest.mark.parametrize("qdt", [L.I4, L.FP4])
@pytest.mark.parametrize("group", [64, 128, 256])
def test_product(nm, T, R, K, qdt, group):
    _check(nm, T, R, K, 0, qdt, group, T + R + K + group)
    _check(nm, T, R, K, 0, qdt, group, T + R + K + group + 1, extra=1)
    _check(nm, T, R, K, 0, qdt, group, T + R + K + group + 2, integer=True)


@pytest.mark.parametrize("Ns,K", [(3, 48), (3, 768), (4, 32), (4, 1024), (4, 2528), (5, 640), (6, 480), (7, 336), (8, 1152)])
@pytest.mark.parametrize("T,R", [(1, 40), (7, 33), (40, 130)])
@pytest.mark.parametrize("qdt", [L.I4, L.FP4])
def test_product_of_lifted_weights(nm, Ns, K, T, R, qdt):
    _check(nm, T, R, K, Ns, qdt, 128, T + R + K + Ns)
    _check(nm, T, R, K, Ns, qdt, 64, T + R + K + Ns + 1, extra=1, integer=True)


@pytest.mark.parametrize("T,R,K,Ns", [(1, 1, 16, 0), (1, 300, 4096, 0), (4, 97, 336, 0), (20, 64, 512, 0), (50, 130, 1104, 0),
                                      (2, 70, 1024, 4), (35, 30, 480, 6)])
@pytest.mark.parametrize("a", B.ACTS)
@pytest.mark.parametrize("qdt", [L.I4, L.FP4])
def test_glu(nm, T, R, K, Ns, a, qdt):
    g = np.random.default_rng(T + R + K + a)
    X, Xf = _x(g, T, K)
    group = (64, 128, 256)[(T + a) % 3]
    Wg, cg, ig, sg = L.w4_weight(nm, g, R, K, Ns, qdt, group)
    Wu, cu, iu, su = L.w4_weight(nm, g, R, K, Ns, qdt, group)
    G, U, eG, eU = Xf @ Wg.T, Xf @ Wu.T, L.product_bound(Xf, Wg, K), L.product_bound(Xf, Wu, K)
    f, d, rel = B.act(a, G)
    ref = f * U
    err = (np.abs(d) * eG + B.CURVE[a] * eG * eG) * (np.abs(U) + eU) + np.abs(f) * eU + rel * np.abs(ref) + 2.0 ** -24 * np.abs(ref)
    for hdt in (nm.NM_F32, nm.NM_BF16):
        H = nm.nm_spmm_glu_w4(X, cg, ig, sg, cu, iu, su, qdt=qdt, group=group, Ns=Ns, act=a, hdt=hdt)
        _close(H, ref, err, hdt == nm.NM_BF16)


@pytest.mark.parametrize("T,R,K,Ns", [(17, 64, 4096, 0), (33, 40, 8192, 0), (48, 130, 4112, 0), (64, 33, 6144, 0), (90, 70, 4096, 0),
                                      (40, 70, 4096, 4), (20, 97, 5120, 5)])
@pytest.mark.parametrize("qdt", [L.I4, L.FP4])
def test_widths_split_over_blocks(nm, T, R, K, Ns, qdt):
    """Few rows of a wide weight: partial sums through the workspace (full of NaN before), plain and gated."""
    g = np.random.default_rng(T + R + K)
    X, Xf = _x(g, T, K)
    group = (64, 128, 256)[T % 3]
    assert nm.raw.nm_spmm_w4_workspace(T, K, R, Ns) > 0
    Wg, cg, ig, sg = L.w4_weight(nm, g, R, K, Ns, qdt, group)
    Wu, cu, iu, su = L.w4_weight(nm, g, R, K, Ns, qdt, group)
    G, U, eG, eU = Xf @ Wg.T, Xf @ Wu.T, L.product_bound(Xf, Wg, K), L.product_bound(Xf, Wu, K)
    for ydt in (nm.NM_F32, nm.NM_BF16):
        Y = nm.nm_spmm_w4(X, cg, ig, sg, qdt=qdt, group=group, Ns=Ns, ydt=ydt, ws=B.nan_ws(nm.raw.nm_spmm_w4_workspace(T, K, R, Ns)))
        _close(Y, G, eG, ydt == nm.NM_BF16)
        assert torch.equal(Y, nm.nm_spmm_w4(X, cg, ig, sg, qdt=qdt, group=group, Ns=Ns, ydt=ydt))
    f, d, rel = B.act(B.SILU, G)
    ref = f * U
    err = (np.abs(d) * eG + B.CURVE[B.SILU] * eG * eG) * (np.abs(U) + eU) + np.abs(f) * eU + rel * np.abs(ref) + 2.0 ** -24 * np.abs(ref)
    H = nm.nm_spmm_glu_w4(X, cg, ig, sg, cu, iu, su, qdt=qdt, group=group, Ns=Ns, hdt=nm.NM_F32,
                          ws=B.nan_ws(nm.raw.nm_spmm_glu_w4_workspace(T, K, R, Ns)))
    _close(H, ref, err, False)


def test_rows_stay_apart(nm):
    """A token of NaN and a weight row with a NaN scale stay in their own outputs."""
    g = np.random.default_rng(3)
    X, Xf = _x(g, 5, 320)
    W, codes, idx, scales = L.w4_weight(nm, g, 40, 320, 0, L.I4, 64)
    X[2] = float("nan")
    scales[1, 7] = float("nan")
    Y = nm.nm_spmm_w4(X, codes, idx, scales, group=64).float().cpu()
    assert torch.isnan(Y[2]).all() and torch.isnan(Y[:, 7]).all()
    Y[2], Y[:, 7] = 0, 0
    assert torch.isfinite(Y).all()


def test_an_infinite_activation(nm):
    """An infinite activation gives an infinity where the weight has a value, as in the plain product."""
    g = np.random.default_rng(4)
    X, _ = _x(g, 1, 64)
    _, codes, idx, scales = L.w4_weight(nm, g, 16, 64, 0, L.I4, 64, integer=True)
    X[0, 5] = float("inf")
    v = np.where(L.unpack_codes(codes, 32) >= 8, -1, 1) * (L.unpack_codes(codes, 32) & 7)
    cols = B.columns(idx, 64)
    Y = nm.nm_spmm_w4(X, codes, idx, scales, group=64, ydt=nm.NM_F32).cpu().numpy()[0]
    for r in range(16):
        c = v[r][cols[r] == 5]
        if len(c) == 0:
            assert np.isfinite(Y[r])
        elif (c != 0).all() and len(c) == 1:
            assert Y[r] == np.sign(c[0]) * np.inf
        else:
            assert not np.isfinite(Y[r])


def test_offsets_past_32_bits(nm):
    """Rows of codes, tokens and outputs that lie gigabytes apart."""
    g = np.random.default_rng(8)
    T, R, K = 3, 70, 256
    X, Xf = _x(g, T, K)
    W, codes, idx, scales = L.w4_weight(nm, g, R, K, 0, L.FP4, 128)
    far = torch.empty(((R - 1) * ((1 << 26) - 16) + 64,), dtype=torch.uint8, device=dev())
    c = far.as_strided((R, 64), ((1 << 26) - 16, 1))
    c.copy_(codes[:, :64])
    xs = torch.empty(((T - 1) * (1 << 31) + K,), dtype=torch.bfloat16, device=dev()).as_strided((T, K), (1 << 31, 1))
    xs.copy_(X)
    out = torch.empty(((T - 1) * (1 << 31) + R,), dtype=torch.bfloat16, device=dev()).as_strided((T, R), (1 << 31, 1))
    _close(nm.nm_spmm_w4(xs, c, idx, scales, qdt=nm.NM_FP4, out=out), Xf @ W.T, L.product_bound(Xf, W, K), True)


def test_graph_and_stream(nm):
    """Captured once and replayed with other inputs between eager work; on a stream of its own."""
    g = np.random.default_rng(9)
    X, Xf = _x(g, 4, 512)
    W, codes, idx, scales = L.w4_weight(nm, g, 120, 512, 0, L.I4, 128)
    call = lambda out=None: nm.nm_spmm_w4(X, codes, idx, scales, ydt=nm.NM_F32, out=out)  # noqa: E731
    eager = call()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        side = call()
    torch.cuda.synchronize()
    assert torch.equal(side, eager)
    out, graph = torch.empty_like(eager), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out)
    for k in range(3):
        X.copy_(_x(np.random.default_rng(20 + k), 4, 512)[0])
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, call())


def test_nothing_to_do(nm):
    g = np.random.default_rng(1)
    _, codes, idx, scales = L.w4_weight(nm, g, 8, 64, 0, L.I4, 64)
    X = torch.empty((0, 64), dtype=torch.bfloat16, device=dev())
    assert nm.nm_spmm_w4(X, codes, idx, scales, group=64).shape == (0, 8)
    assert nm.nm_quant_w4(torch.empty((0, 64), device=dev()))[0].shape[0] == 0


def test_wrappers_refuse(nm):
    g = np.random.default_rng(1)
    X, _ = _x(g, 2, 64)
    _, codes, idx, scales = L.w4_weight(nm, g, 8, 64, 0, L.I4, 64)
    ok = dict(X=X, codes=codes, idx=idx, scales=scales, group=64)
    nm.nm_spmm_w4(**ok)
    for k, v in (("X", X.float()), ("X", X[:, :48].t()), ("codes", codes.view(torch.int8)), ("idx", idx[:4]), ("scales", scales.float()),
                 ("scales", scales[:, :4]), ("codes", codes.cpu()), ("X", torch.zeros((2, 128), dtype=torch.bfloat16, device=dev())),
                 ("out", torch.zeros((2, 9), device=dev())), ("out", torch.zeros((2, 8), dtype=torch.int32, device=dev()))):
        with pytest.raises((ValueError, nm.NMError)):
            nm.nm_spmm_w4(**{**ok, k: v})
    with pytest.raises((ValueError, nm.NMError)):
        nm.nm_spmm_w4(**{**ok, "group": 32})
    with pytest.raises(ValueError):
        nm.nm_quant_w4(torch.zeros((4, 12), device=dev()))
    with pytest.raises(ValueError):
        nm.nm_spmm_w4(**{**ok, "X": X.cpu(), "codes": codes.cpu(), "idx": idx.cpu(), "scales": scales.cpu()})
