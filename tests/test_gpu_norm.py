"""The norms around a block (nm_block_norm) and their gradients against the formulas in 64 bits; the bound is an
error analysis of the same steps (tests/_rounded.py)."""
import numpy as np
import pytest
import torch

from tests import _block as B
from tests import _rounded as R
from tests._util import dev

pytestmark = pytest.mark.gpu
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def nm():
    import semi_structured_sparsity_amd as m
    return m


def _t(a, dtype):
    return torch.from_numpy(np.asarray(a, np.float32)).to(dtype).to(dev())


def _f(t):
    return None if t is None else t.float().cpu().numpy().astype(np.float64)


def _close(got, ref, name=""):
    """got within the bound of the f32 steps and one rounding to its type."""
    half = 2.0 ** -8 if got.dtype == torch.bfloat16 else 2.0 ** -24
    g = _f(got)
    tol = ref.e + half * (np.abs(ref.v) + ref.e) + 1e-37
    assert np.isfinite(g).all(), name
    assert (np.abs(g - ref.v) <= tol).all(), (name, float((np.abs(g - ref.v) / tol).max()))


def _case(g, M, C, xt, wt, post, pre, gates, block=True, bias=True):
    w = lambda: _t(1 + 0.2 * g.standard_normal(C), TYPES[wt])  # noqa: E731
    b = lambda: _t(0.3 * g.standard_normal(C), TYPES[wt]) if bias else None  # noqa: E731
    c = {"X": _t(g.standard_normal((M, C)) * np.exp(g.standard_normal(C)), TYPES[xt]),
         "Y": _t(g.standard_normal((M, C)) + 0.2, torch.bfloat16) if block else None,
         "post": post, "pre": pre, "w_post": w() if post else None, "b_post": b() if post else None,
         "w_pre": w() if pre else None, "b_pre": b() if pre else None, "gate": None, "gate_rows": 0}
    if gates:
        c["gate_rows"] = -(-M // gates) if gates > 1 else 0
        c["gate"] = _t(0.5 + g.standard_normal((-(-M // c["gate_rows"]) if c["gate_rows"] else 1, C)), TYPES[wt])
    return c


def _gate(c, M):
    if c["gate"] is None:
        return None
    rows = c["gate_rows"] or M
    return _f(c["gate"])[np.arange(M) // rows]


def _forward(c, res):
    M = c["X"].shape[0]
    return R.forward(_f(c["X"]), _f(c["Y"]), np.float64(np.float32(res)), _gate(c, M), c["post"], _f(c["w_post"]), _f(c["b_post"]),
                     c["pre"], _f(c["w_pre"]), _f(c["b_pre"]), np.float64(np.float32(EPS)))


# (tokens, columns): single values, ragged widths, rows in whole vectors and not, every width's kernel
SIZES = [(1, 1), (3, 8), (2, 100), (5, 1000), (129, 1025), (40, 2560), (33, 4096), (7, 4100), (3, 8200), (2, 12001), (2, 16392),
         (2, 32768), (1, 32767), (600, 264)]


@pytest.mark.parametrize("M,C", SIZES)
@pytest.mark.parametrize("post,pre", [(R.RMS, R.RMS), (R.LAYER, R.LAYER), (R.NONE, R.RMS), (R.RMS, R.NONE), (R.LAYER, R.RMS)])
@pytest.mark.parametrize("xt", ["bf16", "f32"])
def test_forward(nm, M, C, post, pre, xt):
    g = np.random.default_rng(M * 7 + C + post * 3 + pre)
    for wt, gates, res, ndt in (("bf16", 1, 1.0, nm.NM_BF16), ("f32", 3, 0.5, nm.NM_F32), ("bf16", 0, -2.0, nm.NM_BF16)):
        c = _case(g, M, C, xt, wt, post, pre, min(gates, M))
        z, n = _forward(c, res)
        Z, N, s = nm.nm_block_norm(**c, res_scale=res, eps=EPS, ndt=ndt)
        assert s is None and (N is None) == (pre == R.NONE)
        _close(Z, z, "Z")
        if pre:
            _close(N, n, "N")
            Z2, N2, _ = nm.nm_block_norm(**c, res_scale=res, eps=EPS, ndt=ndt, want_z=False)
            assert Z2 is None and torch.equal(N, N2)


@pytest.mark.parametrize("M,C", [(1, 16), (9, 257), (30, 2048), (2, 9000)])
@pytest.mark.parametrize("pre", [R.RMS, R.LAYER])
def test_norm_alone(nm, M, C, pre):
    """Without a block: N of X; weights and biases left out."""
    g = np.random.default_rng(M + C)
    c = _case(g, M, C, "f32", "f32", R.NONE, pre, 0, block=False, bias=False)
    for w in (c["w_pre"], None):
        c["w_pre"] = w
        z, n = _forward(c, 1.0)
        Z, N, _ = nm.nm_block_norm(**c, eps=EPS)
        assert torch.equal(Z, c["X"])
        _close(N, n)


@pytest.mark.parametrize("C", [64, 250, 4096])
def test_strides_in_place_and_gaps(nm, C):
    """Rows apart (nothing is written between them), Z written over X, odd strides."""
    g = np.random.default_rng(C)
    for extra in (8, 3):
        c = _case(g, 6, C, "f32", "bf16", R.RMS, R.LAYER, 2)
        ref = nm.nm_block_norm(**c, res_scale=0.5)
        c["X"], c["Y"], c["gate"] = B.strided(c["X"], extra), B.strided(c["Y"], extra), B.strided(c["gate"], extra)
        Z, N, _ = nm.nm_block_norm(**c, res_scale=0.5, out_z=c["X"])
        assert Z.data_ptr() == c["X"].data_ptr()
        assert torch.isnan(c["X"].as_strided((5, extra), (C + extra, 1), C)).all()
        if extra == 8:
            assert torch.equal(Z, ref[0]) and torch.equal(N, ref[1])
        else:      # another kernel's order of sums
            z, n = R.A(_f(ref[0])), R.A(_f(ref[1]))
            assert (np.abs(_f(Z) - z.v) <= 1e-4 * np.abs(z.v).max()).all() and (np.abs(_f(N) - n.v) <= 2e-2 * np.abs(n.v).max()).all()


# ------------------------------------------------------------------ codes
@pytest.mark.parametrize("M,C", [(1, 240), (5, 2560), (300, 480), (3, 13440)])
@pytest.mark.parametrize("code", ["int8", "fp8"])
@pytest.mark.parametrize("pre", [R.RMS, R.LAYER])
def test_codes(nm, M, C, code, pre):
    g = np.random.default_rng(M + C)
    c = _case(g, M, C, "bf16", "bf16", R.RMS, pre, 1)
    z, n = _forward(c, 0.5)
    ndt, top = (nm.NM_I8, 127.0) if code == "int8" else (nm.NM_FP8, 448.0)
    Z, N, s = nm.nm_block_norm(**c, res_scale=0.5, eps=EPS, ndt=ndt)
    _close(Z, z)
    big = np.abs(n.v).max(1)
    es = n.e.max(1) / top + 2 * R.U * big / top
    S = _f(s)
    assert (np.abs(S - big / top) <= es).all()
    q = n.v / S[:, None]
    slack = n.e / S[:, None] + 2 * R.U * np.abs(q)
    half = 0.5 if code == "int8" else np.maximum(2.0 ** -4 * np.abs(q), 2.0 ** -10)
    got = _f(N)
    assert (np.abs(got - q) <= half + slack * (1 + 2.0 ** -4)).all()
    for Ns in (3, 4, 5, 6, 7, 8):
        if C % (2 * Ns):
            continue
        _, NL, sl = nm.nm_block_norm(**c, res_scale=0.5, eps=EPS, ndt=ndt, Ns=Ns)
        j = np.arange(nm.lifted_width(C, Ns))
        w = j // 4
        cols = 2 * Ns * (w // (Ns - 1)) + 2 * (w % (Ns - 1)) + j % 4
        assert torch.equal(sl, s) and np.array_equal(_f(NL), got[:, cols])


def test_codes_of_a_zero_row(nm):
    X = torch.zeros((2, 64), dtype=torch.bfloat16, device=dev())
    X[1] = 1
    _, N, s = nm.nm_block_norm(X, ndt=nm.NM_FP8)
    assert s[0] == 0 and not N[0].float().any() and (N[1].float() == 448).all()


# ------------------------------------------------------------------ backward
def _check_backward(nm, c, M, C, res, dz, dn, ws=None):
    fwd = {k: v for k, v in c.items() if k != "X"}
    Z = nm.nm_block_norm(**c, res_scale=res, eps=EPS)[0]
    got = nm.nm_block_norm_backward(Z, dZ=dz, dN=dn, res_scale=res, eps=EPS, ws=ws, **fwd)
    gate = _gate(c, M)
    ref = R.backward(_f(Z), _f(dz), _f(dn), _f(c["Y"]), np.float64(np.float32(res)), gate, c["post"], _f(c["w_post"]),
                     _f(c["b_post"]), c["pre"], _f(c["w_pre"]), np.float64(np.float32(EPS)))
    _close(got.dX, ref["dX"], "dX")
    if c["Y"] is not None:
        _close(got.dY, ref["dY"], "dY")
    for k in ("dw_pre", "db_pre", "dw_post", "db_post"):
        if getattr(got, k) is not None:
            _close(getattr(got, k), ref[k].sum(0), k)
    assert (got.dw_pre is None) == (c["w_pre"] is None) and (got.dw_post is None) == (c["w_post"] is None)
    assert (got.dgate is None) == (c["gate"] is None)
    if got.dgate is not None:
        rows = c["gate_rows"] or M
        for k, a in enumerate(range(0, M, rows)):
            t = ref["dgate"]
            _close(got.dgate[k], R.A(t.v[a:a + rows], t.e[a:a + rows]).sum(0), "dgate")
    return got


@pytest.mark.parametrize("M,C", SIZES)
@pytest.mark.parametrize("post,pre", [(R.RMS, R.RMS), (R.LAYER, R.LAYER), (R.NONE, R.RMS), (R.LAYER, R.RMS)])
@pytest.mark.parametrize("xt", ["bf16", "f32"])
def test_backward(nm, M, C, post, pre, xt):
    g = np.random.default_rng(M * 5 + C + post * 3 + pre)
    for wt, gates, res in (("bf16", 1, 0.5), ("f32", 3, 1.0), ("f32", M, 1.0), ("bf16", 0, 2.0)):
        c = _case(g, M, C, xt, wt, post, pre, min(gates, M), bias=gates != 3)
        dz, dn = _t(g.standard_normal((M, C)), TYPES[xt]), _t(g.standard_normal((M, C)), TYPES["f32" if gates == 3 else "bf16"])
        ws = B.nan_ws(nm.raw.nm_block_norm_backward_workspace(M, C, c["gate_rows"]))
        _check_backward(nm, c, M, C, res, dz, dn, ws)


def test_backward_of_parts(nm):
    """Without dZ, without a block, without a norm, without parameter gradients; dX over dZ; twice the same bits."""
    g = np.random.default_rng(4)
    M, C = 70, 520
    c = _case(g, M, C, "bf16", "bf16", R.RMS, R.RMS, 2)
    dz, dn = (_t(g.standard_normal((M, C)), torch.bfloat16) for _ in range(2))
    _check_backward(nm, c, M, C, 0.5, None, dn)
    full = _check_backward(nm, c, M, C, 0.5, dz, dn)
    again = _check_backward(nm, c, M, C, 0.5, dz, dn)
    assert all(torch.equal(a, b) for a, b in zip(full, again) if a is not None)
    fwd = {k: v for k, v in c.items() if k != "X"}
    Z = nm.nm_block_norm(**c, res_scale=0.5, eps=EPS)[0]
    only = nm.nm_block_norm_backward(Z, dZ=dz, dN=dn, res_scale=0.5, eps=EPS, want_params=False, **fwd)
    assert torch.equal(only.dX, full.dX) and torch.equal(only.dY, full.dY) and not any(t is not None for t in only[2:])
    params = nm.nm_block_norm_backward(Z, dZ=dz, dN=dn, res_scale=0.5, eps=EPS, want_dx=False, want_dy=False, **fwd)
    assert params.dX is None and params.dY is None and all(torch.equal(a, b) for a, b in zip(params[2:], full[2:]) if a is not None)
    over = dz.clone()
    got = nm.nm_block_norm_backward(Z, dZ=over, dN=dn, res_scale=0.5, eps=EPS, out_dx=over, **fwd)
    assert got.dX.data_ptr() == over.data_ptr() and torch.equal(over, full.dX)
    _check_backward(nm, _case(g, M, C, "bf16", "bf16", R.NONE, R.LAYER, 0, block=False), M, C, 1.0, dz, dn)
    _check_backward(nm, _case(g, M, C, "f32", "f32", R.LAYER, R.NONE, 1), M, C, 1.0, dz.float(), None)


def test_no_tokens(nm):
    c = _case(np.random.default_rng(0), 1, 40, "bf16", "f32", R.LAYER, R.LAYER, 1)
    X, Y = c["X"][:0], c["Y"][:0]
    rest = {k: v for k, v in c.items() if k not in ("X", "Y")}
    Z, N, _ = nm.nm_block_norm(X, Y, **rest)
    assert Z.shape == N.shape == (0, 40)
    got = nm.nm_block_norm_backward(X, dZ=X, dN=X, Y=Y, **rest)
    assert got.dX.shape == (0, 40) and all(not t.any() for t in got[2:]) and got.dgate.shape == (1, 40)


def test_offsets_past_32_bits(nm):
    """Rows gigabytes apart."""
    g = np.random.default_rng(6)
    M, C, ld = 3, 512, 1 << 31
    c = _case(g, M, C, "bf16", "bf16", R.RMS, R.RMS, 1)
    ref = nm.nm_block_norm(**c)
    far = torch.empty((M - 1) * ld + C, dtype=torch.bfloat16, device=dev()).as_strided((M, C), (ld, 1))
    far.copy_(c["X"])
    Z, N, _ = nm.nm_block_norm(**{**c, "X": far}, out_z=far)
    assert torch.equal(Z, ref[0]) and torch.equal(N, ref[1])


def test_a_token_of_nan_stays_alone(nm):
    g = np.random.default_rng(7)
    c = _case(g, 5, 264, "bf16", "bf16", R.RMS, R.RMS, 0)
    ref = nm.nm_block_norm(**c)
    c["X"][2, 7] = float("nan")
    Z, N, _ = nm.nm_block_norm(**c)
    assert torch.isnan(N[2]).all() and torch.isnan(Z[2, 7]) and not torch.isnan(Z[2, 8])
    keep = [0, 1, 3, 4]
    assert torch.equal(N[keep], ref[1][keep])


def test_graph_and_stream(nm):
    """Both directions captured in one graph, replayed with other inputs between eager calls."""
    g = np.random.default_rng(11)
    M, C = 50, 640
    c = _case(g, M, C, "bf16", "bf16", R.RMS, R.RMS, 2)
    fwd = {k: v for k, v in c.items() if k != "X"}
    dz, dn = (_t(g.standard_normal((M, C)), torch.bfloat16) for _ in range(2))

    def step():
        Z, N, _ = nm.nm_block_norm(**c)
        return [Z, N, *[t for t in nm.nm_block_norm_backward(Z, dZ=dz, dN=dn, **fwd) if t is not None]]
    eager = step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        side = step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(eager, side))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(3):
        c["X"].copy_(_t(np.random.default_rng(k).standard_normal((M, C)), torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, step()))


def test_wrappers_refuse(nm):
    c = _case(np.random.default_rng(0), 4, 64, "bf16", "bf16", R.RMS, R.RMS, 2)
    nm.nm_block_norm(**c)
    for bad in (dict(X=c["X"].half()), dict(Y=c["Y"].float()), dict(Y=c["Y"][:3]), dict(gate=c["gate"][:1]), dict(w_post=c["w_post"][:60]),
                dict(w_post=c["w_post"].float()), dict(gate=c["gate"].cpu()), dict(pre=3), dict(post=R.NONE), dict(pre=R.NONE),
                dict(Ns=4), dict(ndt=nm.NM_I32), dict(Y=None), dict(eps=-1.0), dict(out_z=c["Y"][:, :32]), dict(out_z=c["Y"]),
                dict(ndt=nm.NM_FP8, Ns=5), dict(gate_rows=-1)):
        with pytest.raises((ValueError, nm.NMError)):
            nm.nm_block_norm(**{**c, **bad})
    fwd = {k: v for k, v in c.items() if k != "X"}
    ok = dict(Z=c["X"], dZ=c["X"].clone(), dN=c["X"].clone(), **fwd)
    nm.nm_block_norm_backward(**ok)
    for bad in (dict(dN=None), dict(dZ=ok["dZ"].float()), dict(dN=ok["dN"][:2]), dict(Y=None), dict(pre=R.NONE), dict(out_dx=c["Y"]),
                dict(Z=c["X"].cpu())):
        with pytest.raises((ValueError, nm.NMError)):
            nm.nm_block_norm_backward(**{**ok, **bad})
