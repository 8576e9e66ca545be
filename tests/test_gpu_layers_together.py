"""The operators of nmsparse_layers.h run together, as a served and as a trained layer uses them."""
import numpy as np
import pytest
import torch

from tests import _layers as L
from tests import _rounded as R
from tests._util import dev

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module")
def nm():
    import semi_structured_sparsity_amd as m
    return m


def _rand(g, *shape, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g) * scale).to(dtype).to(dev())


def _f(t):
    return t.float().cpu().numpy().astype(np.float64)


class Layer:
    """A decoder layer's feed-forward half, twice: a mixture of 4-bit experts, then a 4-bit gated block and its
    down projection, with norms before, between and after, and an FP8 6:8 block for the next layer."""

    def __init__(self, nm, K=256, F=128, E=8):
        self.nm, self.K, self.F = nm, K, F
        g = torch.Generator().manual_seed(5)
        prune = lambda rows, cols: nm.nm_prune_pack(_rand(g, rows, cols, scale=cols ** -0.5), None, 0.0, nm.NM_SCORE_MAGNITUDE, 2, 4)[:2]  # noqa: E731

        def four(rows, cols, count=None):
            """(codes, idx, scales) of a pruned weight, or of `count` stacked ones, and its dense values."""
            parts, dense = [], []
            for _ in range(count or 1):
                vals, idx = prune(rows, cols)
                codes, scales, values = nm.nm_quant_w4(vals, qdt=nm.NM_FP4, group=64, want_values=True)
                _, sc, _ = L.quant(vals.float().cpu().numpy(), L.FP4, 64)
                c = L.unpack_codes(codes, cols // 2)
                v = np.where(c >= 8, -1, 1) * L.E2M1[c & 7] * sc.astype(np.float64).repeat(32, 0)[:cols // 2].T
                assert np.array_equal(torch.from_numpy(v).float().bfloat16().float().numpy(), values.float().cpu().numpy())
                dense.append(L.scatter(v, idx, cols))
                parts.append((codes, idx, scales))
            stack = [torch.stack(t) if count else t[0] for t in zip(*parts)]
            return stack, np.stack(dense) if count else dense[0]

        (eg, self.eg), (eu, self.eu), (ed, self.ed) = four(F, K, E), four(F, K, E), four(K, F, E)
        self.router = _rand(g, E, K, scale=K ** -0.5)
        self.moe = nm.MoELayer(self.router, eg[0], eg[1], eu[0], eu[1], ed[0], ed[1], F, vdt=nm.NM_FP4, group=64, gate_scales=eg[2],
                               up_scales=eu[2], down_scales=ed[2])
        (self.g, self.dg), (self.u, self.du), (self.d, self.dd) = four(F, K), four(F, K), four(K, F)
        self.w = [_rand(g, K, scale=0.1) + 1 for _ in range(5)]
        self.gate = _rand(g, 1, K, scale=0.3)

    def __call__(self, x):
        nm = self.nm
        _, n0, _ = nm.nm_block_norm(x, w_pre=self.w[0], want_z=False)
        y0, sel, wts = nm.nm_moe(self.moe, n0, 2, renorm=True, want_routing=True)
        z1, n1, _ = nm.nm_block_norm(x, Y=y0, gate=self.gate, res_scale=0.5, post=nm.NM_NORM_RMS, w_post=self.w[1], w_pre=self.w[2])
        h = nm.nm_spmm_glu_w4(n1, *self.g, *self.u, qdt=nm.NM_FP4, group=64)
        y1 = nm.nm_spmm_w4(h, *self.d, qdt=nm.NM_FP4, group=64)
        z2, n2, s2 = nm.nm_block_norm(z1, Y=y1, post=nm.NM_NORM_RMS, w_post=self.w[3], w_pre=self.w[4], ndt=nm.NM_FP8, Ns=4)
        return n0, y0, sel, wts, z1, n1, h, y1, z2, n2, s2


@pytest.mark.parametrize("T", [1, 5, 33])
def test_a_served_layer(nm, T):
    """Every stage against its formula in 64 bits from the stage before's output, in one captured graph too."""
    layer = Layer(nm)
    x = _rand(torch.Generator().manual_seed(T), T, layer.K)
    n0, y0, sel, wts, z1, n1, h, y1, z2, n2, s2 = out = layer(x)
    silu = lambda v: v / (1 + np.exp(-v))  # noqa: E731
    half = 2.0 ** -8
    w = [_f(t) for t in layer.w]

    def near(got, ref, slack):
        got, ref = _f(got), np.asarray(ref)
        assert (np.abs(got - ref) <= half * np.abs(ref) + slack).all(), float(np.abs(got - ref).max())
    near(n0, R.norm(R.A(_f(x)), R.RMS, w[0], None, EPS).v, 1e-5)
    X, S, W = _f(n0), sel.cpu().numpy(), wts.cpu().numpy().astype(np.float64)
    ref, size = np.zeros((T, layer.K)), np.zeros((T, layer.K))
    for t in range(T):
        for j in range(2):
            e = S[t, j]
            H = silu(X[t] @ layer.eg[e].T) * (X[t] @ layer.eu[e].T)
            ref[t] += W[t, j] * (H @ layer.ed[e].T)
            size[t] += W[t, j] * (np.abs(H) @ np.abs(layer.ed[e]).T)
    near(y0, ref, half * size + 1e-5)              # H is rounded to bf16 between
    z, n = R.forward(_f(x), _f(y0), 0.5, _f(layer.gate), R.RMS, w[1], None, R.RMS, w[2], None, EPS)
    near(z1, z.v, z.e)
    near(n1, n.v, n.e)
    near(h, silu(_f(n1) @ layer.dg.T) * (_f(n1) @ layer.du.T), 1e-4)
    near(y1, _f(h) @ layer.dd.T, 1e-4)
    z, n = R.forward(_f(z1), _f(y1), 1.0, None, R.RMS, w[3], None, R.RMS, w[4], None, EPS)
    near(z2, z.v, z.e)
    # the codes feed the sliding-window block as nm_quant_lift's do
    code, scale = _f(n2), _f(s2)[:, None]
    j = np.arange(nm.lifted_width(layer.K, 4))
    cols = 8 * (j // 12) + 2 * (j % 12 // 4) + j % 4
    assert (np.abs(code * scale - n.v[:, cols]) <= 2.0 ** -4 * np.abs(n.v[:, cols]) + (2.0 ** -10 + 1e-4) * scale).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer(x)
    for k in range(3):
        x.copy_(_rand(torch.Generator().manual_seed(100 + k), T, layer.K))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a.view(torch.uint8) if a.dtype == torch.float8_e4m3fn else a,
                               b.view(torch.uint8) if b.dtype == torch.float8_e4m3fn else b) for a, b in zip(got, layer(x)))
    assert len(out) == len(got)


def test_two_streams_at_once(nm):
    """Two layers on two streams, each with its own workspaces, give what they give alone."""
    a, b = Layer(nm), Layer(nm, K=512, F=256, E=16)
    xa, xb = _rand(torch.Generator().manual_seed(1), 3, 256), _rand(torch.Generator().manual_seed(2), 9, 512)
    ra, rb = a(xa), b(xb)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(s):
            ga = a(xa)
        with torch.cuda.stream(t):
            gb = b(xb)
    torch.cuda.synchronize()
    for g, r in ((ga, ra), (gb, rb)):
        assert all(torch.equal(u.float(), v.float()) for u, v in zip(g, r))


def test_a_trained_block(nm):
    """norm -> gated block -> down projection -> norm, forward and backward, against automatic differentiation in
    64 bits.  Every gradient has passed at most ten roundings to bf16, of 2^-8 each: within 10 2^-8 of its size."""
    g = torch.Generator().manual_seed(3)
    M, K, F = 48, 128, 96
    x = _rand(g, M, K)
    vals, dense = {}, {}
    for k, (r, c) in {"g": (F, K), "u": (F, K), "d": (K, F)}.items():
        v, i, m = nm.nm_prune_pack(_rand(g, r, c, scale=c ** -0.5), None, 0.0, nm.NM_SCORE_MAGNITUDE, 2, 4)
        vals[k], dense[k] = (v, i), torch.from_numpy(L.scatter(_f(v), i, c)).requires_grad_()
    w = {k: _rand(g, K, scale=0.1) + 1 for k in ("n0", "post", "n1")}
    gate = _rand(g, 2, K, scale=0.3) + 1
    dz, dn = _rand(g, M, K, scale=0.1), _rand(g, M, K, scale=0.1)
    _, n0, _ = nm.nm_block_norm(x, w_pre=w["n0"], want_z=False)
    h, G, U = nm.nm_spmm_glu(n0, *vals["g"], *vals["u"], save=True)
    y = nm.nm_spmm(h, *vals["d"])
    around = dict(Y=y, gate=gate, gate_rows=24, res_scale=0.5, post=nm.NM_NORM_RMS, w_post=w["post"], w_pre=w["n1"])
    z, n, _ = nm.nm_block_norm(x, **around)
    b1 = nm.nm_block_norm_backward(z, dZ=dz, dN=dn, **around)
    dh, dvd = nm.nm_spmm_backward(b1.dY, h, *vals["d"])
    dn0, dvg, dvu = nm.nm_spmm_glu_backward(dh, G, U, n0, *vals["g"], *vals["u"])
    b0 = nm.nm_block_norm_backward(x, dZ=b1.dX, dN=dn0, w_pre=w["n0"])
    # the same in 64 bits
    leaf = lambda t: torch.from_numpy(_f(t)).requires_grad_()  # noqa: E731
    X, W, A = leaf(x), {k: leaf(t) for k, t in w.items()}, leaf(gate)
    rms = lambda v: v * (v.square().mean(1, keepdim=True) + EPS).rsqrt()  # noqa: E731
    N0 = rms(X) * W["n0"]
    Yd = (torch.nn.functional.silu(N0 @ dense["g"].t()) * (N0 @ dense["u"].t())) @ dense["d"].t()
    Z = 0.5 * X + A.repeat_interleave(24, 0) * (rms(Yd) * W["post"])
    N = rms(Z) * W["n1"]
    ((Z * torch.from_numpy(_f(dz))).sum() + (N * torch.from_numpy(_f(dn))).sum()).backward()
    take = lambda full, i, c: np.take_along_axis(full.numpy(), L.B.columns(i, c), 1)  # noqa: E731
    for name, got, ref in (("x", b0.dX, X.grad), ("w n0", b0.dw_pre, W["n0"].grad), ("w post", b1.dw_post, W["post"].grad),
                           ("w n1", b1.dw_pre, W["n1"].grad), ("gate", b1.dgate, A.grad),
                           ("down", dvd, take(dense["d"].grad, vals["d"][1], F)), ("gate proj", dvg, take(dense["g"].grad, vals["g"][1], K)),
                           ("up", dvu, take(dense["u"].grad, vals["u"][1], K))):
        ref = ref if isinstance(ref, np.ndarray) else ref.numpy()
        assert np.linalg.norm(_f(got) - ref) <= 10 * 2.0 ** -8 * np.linalg.norm(ref), name
    z64, n64 = Z.detach().numpy(), N.detach().numpy()
    assert np.linalg.norm(_f(z) - z64) <= 10 * 2.0 ** -8 * np.linalg.norm(z64) and np.linalg.norm(_f(n) - n64) <= 10 * 2.0 ** -8 * np.linalg.norm(n64)
