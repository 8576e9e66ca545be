"""The AdamW step (nm_adamw) against its formula in 64 bits.

f32 arithmetic of about ten roundings and the hardware's square root and reciprocal (2^-22 each):
states within 2^-21 of their terms' sizes; the parameter within 2^-23 of itself plus 2^-19 of
the update (and one rounding to its type)."""
import numpy as np
import pytest
import torch

from tests._util import dev

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def nm():
    import semi_structured_sparsity_amd as m
    return m


def _blocks(x, n):
    pad = (-n) % 256
    return np.pad(x, (0, pad)).reshape(-1, 256)


def encode64(x, least):
    """(values of the codes, scales) of 8-bit states in 64 bits."""
    n = x.size
    b = _blocks(x, n)
    fin = np.where(np.isfinite(b), np.abs(b), 0)
    top = fin.max(1)
    top = np.where(top < 2.0 ** -118, 0, top)
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.where(top[:, None] > 0, b / (top[:, None] / 448), 0)
    a = np.abs(q)
    e = np.maximum(np.floor(np.log2(np.maximum(a, 2.0 ** -60))), -6)
    u = 2.0 ** (e - 3)
    r = np.round(a / u) * u
    if least:
        r = np.where((a > 0) & (r == 0), 2.0 ** -9, r)
    return (np.where(np.isfinite(b), r * np.sign(q), np.nan)).reshape(-1)[:n], top / 448, q.reshape(-1)[:n]


def _state(g, n, mag):
    return (g.standard_normal(n) * 0.3 * mag), (g.standard_normal(n) * mag) ** 2


class Case:
    def __init__(self, g, sizes, pdt, gdt, f8, copy, offset=0):
        self.sizes, self.f8 = sizes, f8
        new = lambda n, dt: torch.zeros(n + offset, dtype=dt, device=dev())[offset:]  # noqa: E731
        self.p, self.g, self.m, self.v, self.ms, self.vs, self.c = ([] for _ in range(7))
        for k, n in enumerate(sizes):
            mag = 10.0 ** (-(k % 6))
            p, gr = new(n, pdt), new(n, gdt)
            p.copy_(torch.from_numpy(g.standard_normal(n)))
            gr.copy_(torch.from_numpy(g.standard_normal(n) * mag))
            m, v = _state(g, n, mag)
            if f8:
                mq, ms, _ = encode64(m, False)
                vq, vs, _ = encode64(np.sqrt(v), True)
                a, b = new(n, F8), new(n, F8)
                a.copy_(torch.from_numpy(mq).float().to(F8))
                b.copy_(torch.from_numpy(vq).float().to(F8))
                self.ms.append(torch.from_numpy(ms.astype(np.float32)).to(dev()))
                self.vs.append(torch.from_numpy(vs.astype(np.float32)).to(dev()))
            else:
                a, b = new(n, torch.float32), new(n, torch.float32)
                a.copy_(torch.from_numpy(m))
                b.copy_(torch.from_numpy(v))
            self.p.append(p), self.g.append(gr), self.m.append(a), self.v.append(b)
            if copy:
                self.c.append(new(n, torch.bfloat16))

    def tensors(self, nm, **kw):
        return nm.AdamWTensors(self.p, self.g, self.m, self.v, self.ms if self.f8 else None,
                               self.vs if self.f8 else None, self.c or None, **kw)

    def host(self, k):
        f = lambda t: t.float().cpu().numpy().astype(np.float64)  # noqa: E731
        n = self.sizes[k]
        m, v = f(self.m[k]), f(self.v[k])
        if self.f8:
            m = (_blocks(m, n) * f(self.ms[k])[:, None]).reshape(-1)[:n]
            v = (_blocks(v, n) * f(self.vs[k])[:, None]).reshape(-1)[:n] ** 2
        return f(self.p[k]), f(self.g[k]), m, v


def _step(nm, case, step, clip, decay, lr_scale, lr=1e-2, b1=0.9, b2=0.999, eps=1e-8):
    before = [case.host(k) for k in range(len(case.sizes))]
    scale = torch.tensor([clip], dtype=torch.float32, device=dev()) if clip is not None else None
    nm.nm_adamw(case.tensors(nm, lr_scale=lr_scale, weight_decay=decay), lr=lr, step=step, beta1=b1, beta2=b2, eps=eps,
                grad_scale=scale)
    for k, n in enumerate(case.sizes):
        p, g, m, v = before[k]
        g = g * (np.float64(np.float32(clip)) if clip is not None else 1.0)
        m1, v1 = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
        tm = 2.0 ** -21 * (np.abs(m) + np.abs(g)) + 1e-44
        tv = 2.0 ** -21 * (v + g * g) + 1e-44
        l = lr * lr_scale[k]
        den = np.sqrt(v1 / (1 - b2 ** step)) + eps
        upd = l / (1 - b1 ** step) * m1 / den
        p1 = p * (1 - l * decay[k]) - upd
        # the update's error: m's, v's (half of it through the root) and the arithmetic's
        tu = l / (1 - b1 ** step) * tm / den + np.abs(upd) * (2.0 ** -19 + tv / np.maximum(v1, 1e-60))
        tp = 2.0 ** -22 * np.abs(p) + tu
        got = case.p[k].float().cpu().numpy().astype(np.float64)
        bf = case.p[k].dtype == torch.bfloat16
        assert (np.abs(got - p1) <= tp + (2.0 ** -8 * np.abs(p1) if bf else 0)).all(), k
        if case.c:
            assert torch.equal(case.c[k], case.p[k].to(torch.bfloat16)), k
        if not case.f8:
            assert (np.abs(case.m[k].cpu().numpy() - m1) <= tm).all(), k
            assert (np.abs(case.v[k].cpu().numpy() - v1) <= tv).all(), k
            continue
        for codes, scales, x, t, least in ((case.m[k], case.ms[k], m1, tm, False),
                                           (case.v[k], case.vs[k], np.sqrt(v1), 2.0 ** -20 * np.sqrt(v + g * g) + 1e-30, True)):
            want, sc, q = encode64(x, least)
            s = scales.cpu().numpy().astype(np.float64)
            assert (np.abs(s - sc) <= 2.0 ** -20 * sc + _blocks(t, n).max(1) / 448 + 1e-45).all(), k
            c = codes.float().cpu().numpy().astype(np.float64)
            # the code nearest the quotient, or its neighbour where the quotient is within its
            # error of the midpoint: the value is half a unit plus that error away at most
            unit = 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(np.abs(q), 2.0 ** -60))), -6) - 3)
            slack = 2.0 ** -18 * np.abs(q) + np.repeat(1 / np.maximum(sc, 1e-60), 256)[:n] * t * 2
            half = 0.5 * unit * (1 + 2.0 ** -10)
            least_ok = (c == 2.0 ** -9) & (np.abs(q) <= 2.0 ** -9) & least
            assert ((np.abs(c - q) <= half + slack) | least_ok).all(), k
            if least:
                assert (c[x > 1e-30] > 0).all(), k


SIZES = [1, 255, 256, 257, 1000, 4096, 4097, 8191, 20000, 3]


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("pdt,gdt,copy", [(torch.float32, torch.bfloat16, True), (torch.float32, torch.float32, False),
                                          (torch.bfloat16, torch.bfloat16, False), (torch.bfloat16, torch.float32, False)])
@pytest.mark.parametrize("offset", [0, 1, 8])
def test_adamw_step(nm, f8, pdt, gdt, copy, offset):
    g = np.random.default_rng(11 + offset)
    case = Case(g, SIZES, pdt, gdt, f8, copy, offset)
    n = len(SIZES)
    _step(nm, case, 1, None, [0.0] * n, [1.0] * n)
    _step(nm, case, 2, 0.37, [0.1] * n, [1.0 + 0.1 * k for k in range(n)])
    _step(nm, case, 5000, 2.0, [0.01 * k for k in range(n)], [1.0] * n, b1=0.8, b2=0.95, eps=1e-6)


@pytest.mark.parametrize("f8", [False, True])
def test_adamw_more_tensors_than_one_launch_takes(nm, f8):
    g = np.random.default_rng(12)
    sizes = [int(x) for x in g.integers(0, 700, 131)]
    sizes[7] = 0
    case = Case(g, sizes, torch.float32, torch.bfloat16, f8, True)
    _step(nm, case, 3, None, [0.1] * len(sizes), [1.0] * len(sizes))


def test_adamw_from_zero_states(nm):
    """Zeroed states (codes and scales) are the state before the first step; zero gradients leave
    parameters at their decay."""
    for f8 in (False, True):
        n = 1000
        p = torch.randn(n, device=dev())
        gr = torch.randn(n, device=dev())
        gr[300:] = 0
        dt = F8 if f8 else torch.float32
        m, v = torch.zeros(n, device=dev()).to(dt), torch.zeros(n, device=dev()).to(dt)
        ms, vs = torch.zeros(4, device=dev()), torch.zeros(4, device=dev())
        t = nm.AdamWTensors([p], [gr], [m], [v], [ms] if f8 else None, [vs] if f8 else None, weight_decay=0.5)
        p0 = p.clone()
        nm.nm_adamw(t, lr=0.01, step=1)
        # the first step is lr * sign(g) where g is well above eps
        want = p0 * (1 - 0.01 * 0.5)
        want[:300] -= 0.01 * torch.sign(gr[:300])
        assert torch.allclose(p, want, rtol=0, atol=1e-5)
        assert not m.float()[300:].any() and not v.float()[300:].any()
        if f8:
            assert not ms[2:].any() and not vs[2:].any()


def test_adamw_nonfinite_gradients_stay_in_place(nm):
    """NaN and infinities reach their own element only; the others of their block keep their
    values."""
    for f8 in (False, True):
        out = []
        for bad in (False, True):
            g = np.random.default_rng(13)
            case = Case(g, [1024], torch.float32, torch.float32, f8, False)
            # a large element keeps the block's scale the same with and without the bad ones
            case.g[0][5] = 100.0
            if bad:
                case.g[0][7], case.g[0][300], case.g[0][301] = float("nan"), float("inf"), float("-inf")
            else:
                case.g[0][7], case.g[0][300], case.g[0][301] = 0, 0, 0
            nm.nm_adamw(case.tensors(nm), lr=0.01, step=4)
            out.append(case)
        a, b = out
        keep = torch.ones(1024, dtype=torch.bool, device=dev())
        keep[[7, 300, 301]] = False
        assert torch.equal(a.p[0][keep], b.p[0][keep])
        assert torch.isnan(b.p[0][7])
        ma, mb = a.m[0].float(), b.m[0].float()
        assert torch.isnan(mb[7]) and not torch.isfinite(mb[300]) and not torch.isfinite(mb[301])
        if f8:
            keep[256:512] = False      # without its largest elements a block may have another scale
            assert torch.isfinite(b.ms[0]).all() and torch.isfinite(b.vs[0]).all()
        assert torch.equal(ma[keep], mb[keep])


def test_adamw_all_codes_read_and_written(nm):
    """beta = 0 decay of nothing: with lr 0, b1 -> m' = b1 m exactly for powers of two, every code's
    value is read, and written back as the same code."""
    codes = torch.arange(256, dtype=torch.uint8).view(F8).float()
    codes = torch.where(torch.isnan(codes), torch.zeros_like(codes), codes)
    m = codes.to(F8).to(dev())
    r = codes.abs().to(F8).to(dev())
    ms, vs = torch.full((1,), 2.0 ** -5, device=dev()), torch.full((1,), 2.0 ** -7, device=dev())
    p, gr = torch.zeros(256, device=dev()), torch.zeros(256, device=dev())
    t = nm.AdamWTensors([p], [gr], [m], [r], [ms], [vs])
    m0, r0 = m.float().clone(), r.float().clone()
    nm.nm_adamw(t, lr=0.0, step=1, beta1=0.5, beta2=0.25)
    assert torch.equal(m.float(), m0) and torch.equal(r.float(), r0)
    assert abs(ms.item() - 2.0 ** -6) < 1e-8 and abs(vs.item() - 2.0 ** -8) < 1e-9


def test_adamw_long_tensor(nm):
    """More elements than 32 bits count."""
    n = 2 ** 32 + 4097
    p = torch.zeros(n, dtype=torch.bfloat16, device=dev())
    g = torch.ones(n, dtype=torch.bfloat16, device=dev())
    m, v = (torch.zeros(n, dtype=torch.uint8, device=dev()).view(F8) for _ in range(2))
    ms, vs = (torch.zeros((n + 255) // 256, device=dev()) for _ in range(2))
    nm.nm_adamw(nm.AdamWTensors([p], [g], [m], [v], [ms], [vs]), lr=0.5, step=1)
    for a in (0, 2 ** 31 - 64, 2 ** 32 - 64, n - 4097, n - 64):
        assert (p[a:a + 64] == -0.5).all() and (m[a:a + 64].float() == 448).all()
    assert (ms[-1] > 0) and (vs[-1] > 0)
    assert p.float().sum().item() < 0 and bool((p == -0.5).all())


def test_adamw_runs_twice_alike_on_a_stream_and_in_a_graph(nm):
    for f8 in (False, True):
        runs = []
        for how in range(3):
            g = np.random.default_rng(14)
            case = Case(g, [5000, 77], torch.float32, torch.bfloat16, f8, True)
            t = case.tensors(nm)
            torch.cuda.synchronize()
            if how == 0:
                for _ in range(3):
                    nm.nm_adamw(t, lr=1e-3, step=2)
            elif how == 1:
                s = torch.cuda.Stream()
                with torch.cuda.stream(s):
                    for _ in range(3):
                        nm.nm_adamw(t, lr=1e-3, step=2)
            else:
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    nm.nm_adamw(t, lr=1e-3, step=2)
                for _ in range(3):
                    graph.replay()
            torch.cuda.synchronize()
            runs.append(case)
        for c in runs[1:]:
            for a, b in ((runs[0].p, c.p), (runs[0].m, c.m), (runs[0].v, c.v), (runs[0].c, c.c)):
                assert all(torch.equal(x.float(), y.float()) for x, y in zip(a, b))


def test_adamw_binding_refuses(nm):
    x = torch.zeros(300, device=dev())
    y, z, w = x.clone(), x.clone(), x.clone()
    s = torch.zeros(2, device=dev())
    with pytest.raises(ValueError):
        nm.AdamWTensors([x], [y[:299]], [z], [w])
    with pytest.raises(ValueError):
        nm.AdamWTensors([x], [y], [z.to(F8)], [w])
    with pytest.raises(ValueError):
        nm.AdamWTensors([x], [y], [z.to(F8)], [w.to(F8)])
    with pytest.raises(ValueError):
        nm.AdamWTensors([x], [y], [z.to(F8)], [w.to(F8)], [s[:1]], [s])
    with pytest.raises(ValueError):
        nm.AdamWTensors([x], [y], [z], [w], copies=[x.clone()])
    with pytest.raises(ValueError):
        nm.AdamWTensors([torch.zeros((4, 8), device=dev()).t()], [y[:32]], [z[:32]], [w[:32]])
    t = nm.AdamWTensors([x], [y], [z], [w])
    for kw in (dict(lr=-1.0, step=1), dict(lr=1.0, step=0), dict(lr=1.0, step=1, beta1=1.0), dict(lr=1.0, step=1, eps=-1.0)):
        with pytest.raises(nm.NMError):
            nm.nm_adamw(t, **kw)
    with pytest.raises(ValueError):
        nm.AdamWTensors([x], [y], [x], [w])
    with pytest.raises(ValueError):
        nm.AdamWTensors([x, x], [y, y], [z, z.clone()], [w, w.clone()])
    with pytest.raises(ValueError):
        nm.AdamWTensors([x.half()], [y], [z], [w])
    with pytest.raises(nm.NMError):
        nm.nm_adamw(nm.AdamWTensors([x], [x], [z], [w]), lr=1.0, step=1)
    with pytest.raises(ValueError):
        nm.nm_adamw(t, lr=1.0, step=1, grad_scale=torch.ones(2, device=dev()))
    with pytest.raises(ValueError):
        nm.nm_adamw(t, lr=1.0, step=1, grad_scale=torch.ones(1))
