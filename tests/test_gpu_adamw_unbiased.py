"""The optimiser step with unbiased 8-bit states (nm_adamw_unbiased): every code, scale and parameter against
the header's definition bit for bit, and thousands of steps against f32 states."""
import warnings

import numpy as np
import pytest
import torch

from tests._util import dev

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn
U64 = np.uint64
f = np.float32


@pytest.fixture(scope="module")
def nm():
    import semi_structured_sparsity_amd as m
    return m


def splitmix(seed, i):
    """Output number i of SplitMix64 seeded with seed."""
    with np.errstate(over="ignore"):
        z = U64(seed) + (np.asarray(i, U64) + U64(1)) * U64(0x9E3779B97F4A7C15)
        z = (z ^ (z >> U64(30))) * U64(0xBF58476D1CE4E5B9)
        z = (z ^ (z >> U64(27))) * U64(0x94D049BB133111EB)
        return z ^ (z >> U64(31))


def draws(seed, step, tensor, n):
    e = np.arange(n, dtype=np.uint64)
    z = splitmix(splitmix(splitmix(seed, step), tensor), e >> U64(1))
    w = np.where(e & U64(1), z >> U64(32), z).astype(np.uint64).astype(np.uint32)
    return w & 0xFFFF, w >> 16


def encode(x, u, least):
    """(values of the codes, scales) of f32 x by the header's rule."""
    n = x.size
    fin = np.where(np.isfinite(x), np.abs(x), f(0))
    top = np.pad(fin, (0, -n % 256)).reshape(-1, 256).max(1)
    some = top >= f(2.0 ** -118)
    with np.errstate(divide="ignore", over="ignore", invalid="ignore"):
        inv = np.where(some, f(448) * (f(1) / top), f(0)).astype(f)
        a = np.minimum(np.abs(np.where(np.isfinite(x), x, f(0)) * np.repeat(inv, 256)[:n]), f(448)).astype(f)
    sub = a < f(2.0 ** -6)
    z = np.where(sub, a + f(2.0 ** -6), a).astype(f)
    r = ((z.view(np.uint32) + (u << 4) + 8) & np.uint32(0xFFF00000)).astype(np.uint32).view(f)
    r = np.minimum(np.where(sub, r - f(2.0 ** -6), r), f(448)).astype(f)
    if least:
        r = np.where((x > 0) & np.repeat(some, 256)[:n], np.maximum(r, f(2.0 ** -9)), r)
    r = np.where(np.isfinite(x), np.copysign(r, x), f("nan"))
    return r, np.where(some, top * f(1 / 448), f(0)).astype(f)


def _states(g, n, zero):
    """(m, r) in f32 and their (codes, scales) on the device."""
    out = []
    for k in range(2):
        x = np.zeros(n, f) if zero else (g.standard_normal(n) * np.exp(2 * g.standard_normal(n))).astype(f)
        x = np.abs(x) if k else x
        q, sc = encode(x, np.full(n, 32767, np.uint32), k == 1)
        out.append((torch.from_numpy(q).to(F8).to(dev()), torch.from_numpy(sc).to(dev()),
                    q.astype(f) * np.repeat(sc, 256)[:n]))
    return out


SIZES = [1, 255, 256, 257, 1000, 4096, 4097, 0, 8191, 20000, 3]


@pytest.mark.parametrize("offset", [0, 1, 8])
@pytest.mark.parametrize("step,zero", [(1, True), (3, False), (100000, False)])
def test_codes_scales_and_parameters(nm, step, zero, offset):
    g = np.random.default_rng(step + offset)
    b1, b2, seed = 0.9, 0.999, 0xFEDCBA9876543210 + step
    ps, gs, ms, vs, ss, rs, ref = [], [], [], [], [], [], []
    new = lambda n, dt: torch.zeros(n + offset, dtype=dt, device=dev())[offset:]  # noqa: E731
    for n in SIZES:
        gr = (g.standard_normal(n) * np.exp(3 * g.standard_normal(n))).astype(f)
        gr[: n // 8] = 0
        (mq, msc, m), (rq, rsc, r) = _states(g, n, zero)
        p = g.standard_normal(n).astype(f)
        ps.append(new(n, torch.float32)), gs.append(new(n, torch.float32)), ms.append(new(n, F8)), vs.append(new(n, F8))
        ps[-1].copy_(torch.from_numpy(p)), gs[-1].copy_(torch.from_numpy(gr)), ms[-1].copy_(mq), vs[-1].copy_(rq)
        ss.append(msc), rs.append(rsc)
        m1 = f(b1) * m + f(1 - b1) * gr
        v1 = f(b2) * (r * r) + (f(1 - b2) * gr) * gr
        ref.append((p, m1, np.sqrt(v1)))
    near = [[t.clone() for t in x] for x in (ps, ms, vs, ss, rs)]
    nm.nm_adamw_unbiased(nm.AdamWTensors(ps, gs, ms, vs, ss, rs), lr=0.01, step=step, seed=seed, beta1=b1, beta2=b2)
    with warnings.catch_warnings():
        warnings.simplefilter("ignore")
        nm.nm_adamw(nm.AdamWTensors(near[0], gs, *near[1:]), lr=0.01, step=step, beta1=b1, beta2=b2)
    for i, n in enumerate(SIZES):
        um, ur = draws(seed, step, i, n)
        for got, sc, near_sc, x, u, least in ((ms[i], ss[i], near[3][i], ref[i][1], um, False),
                                              (vs[i], rs[i], near[4][i], ref[i][2], ur, True)):
            q, scale = encode(x.astype(f), u, least)
            off = int((got.float().cpu().numpy() != q).sum())
            assert off == 0, (i, n, off)
            assert np.array_equal(sc.cpu().numpy(), scale) and torch.equal(sc, near_sc), (i, n)
        assert torch.equal(ps[i], near[0][i]), i       # updated before any rounding


def test_nonfinite_values_and_zeros(nm):
    n = 600
    gr = torch.randn(n, device=dev())
    gr[7], gr[300], gr[301], gr[400:420] = float("nan"), float("inf"), float("-inf"), 0
    p, m, v = torch.randn(n, device=dev()), *(torch.zeros(n, dtype=torch.uint8, device=dev()).view(F8) for _ in range(2))
    ms, vs = (torch.zeros(3, device=dev()) for _ in range(2))
    nm.nm_adamw_unbiased(nm.AdamWTensors([p], [gr], [m], [v], [ms], [vs]), lr=0.01, step=1, seed=3)
    bad = torch.zeros(n, dtype=torch.bool, device=dev())
    bad[[7, 300, 301]] = True
    assert torch.isnan(m.float()[bad]).all() and torch.isnan(v.float()[bad]).all()
    assert torch.isfinite(m.float()[~bad]).all() and torch.isfinite(v.float()[~bad]).all() and torch.isfinite(ms).all()
    assert not m.float()[400:420].any() and not v.float()[400:420].any()
    assert (v.float()[~bad & (gr != 0)] > 0).all()


def _gradients(kind, gr, g):
    if kind == "normal":
        gr.normal_(generator=g)
    elif kind == "uniform":
        gr.uniform_(-1, 1, generator=g)
    elif kind == "constant":      # signs
        gr.uniform_(-1, 1, generator=g).sign_()
    else:                         # a mean of its own for every element, with 10% noise
        gr.normal_(generator=g).mul_(0.1).add_(1.0).mul_(torch.linspace(0.2, 1.7, 256, device=gr.device).repeat(gr.numel() // 256))


def _train(nm, step_of, b2, f8, steps, fall_at, kind="normal", n=8192):
    """The second moments' roots after gradients whose second half of every block falls tenfold."""
    g = torch.Generator(device=dev())
    g.manual_seed(5)
    dt = F8 if f8 else torch.float32
    p, gr = torch.zeros(n, device=dev()), torch.zeros(n, device=dev())
    m, v = (torch.zeros(n, device=dev()).to(dt) for _ in range(2))
    ms, vs = (torch.zeros(n // 256, device=dev()) for _ in range(2))
    t = nm.AdamWTensors([p], [gr], [m], [v], [ms] if f8 else None, [vs] if f8 else None)
    small = (torch.arange(n, device=dev()) % 256) >= 128
    for s in range(1, steps + 1):
        _gradients(kind, gr, g)
        if s > fall_at:
            gr.mul_(torch.where(small, 0.1, 1.0))
        step_of(t, s, b2)
    r = v.float() * vs.repeat_interleave(256) if f8 else v.sqrt()
    return r, m.float() * ms.repeat_interleave(256) if f8 else m, small


@pytest.mark.parametrize("kind,b2", [("normal", 0.95), ("normal", 0.99), ("normal", 0.999), ("uniform", 0.95), ("uniform", 0.999),
                                     ("constant", 0.95), ("constant", 0.999), ("mean", 0.95), ("mean", 0.999)])
def test_thousands_of_steps_follow_f32_states(nm, kind, b2):
    """An unbiased code of r adds its variance to v: per step at most |change| unit, in the mean
    (1 - b2) / 2 E|g^2 / v - 1| r unit <= (1 - b2) r^2 / 16 (the mean is 0.97 for normal gradients, less for the
    others and at most 1 while r falls), so v settles at most 6.3% and r 3.1% above.  The stationary spread of r by that
    variance is at most 0.18 of it, more while r still falls (its units were larger); the mean over 4096
    elements then has a standard error of 0.4%, five of which are allowed.  m's rounding adds at most 1.4% of m^2 to its
    variance (u <= m / 8, 5.3 steps), 0.7% to its mean size."""
    steps, fall_at = 5000, 1000
    r32, m32, small = _train(nm, lambda t, s, b: nm.nm_adamw(t, lr=1e-4, step=s, beta2=b), b2, False, steps, fall_at, kind)
    r8, m8, _ = _train(nm, lambda t, s, b: nm.nm_adamw_unbiased(t, lr=1e-4, step=s, seed=11, beta2=b), b2, True, steps, fall_at, kind)
    for half in (small, ~small):
        ratio = (r8 / r32)[half]
        assert abs(ratio.mean().item() - 1) < 0.031 + 5 * 0.004, ratio.mean()
        assert ratio.std().item() < 0.6
        assert abs(m8[half].abs().mean().item() / m32[half].abs().mean().item() - 1) < 0.05


def test_nearest_codes_say_what_they_are_not_for(nm):
    """Once a list, with 8-bit states only; the unbiased step says nothing."""
    near = lambda t, s, b: nm.nm_adamw(t, lr=1e-4, step=s, beta2=b)  # noqa: E731
    for b2 in (0.9, 0.999):
        with pytest.warns(UserWarning, match="nm_adamw_unbiased") as said:
            _train(nm, near, b2, True, 3, 1)
        assert len(said) == 1 and said[0].filename == __file__
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        _train(nm, near, 0.999, False, 2, 1)
        _train(nm, lambda t, s, b: nm.nm_adamw_unbiased(t, lr=1e-4, step=s, beta2=b), 0.999, True, 2, 1)


def test_runs_twice_alike_on_a_stream_and_in_a_graph(nm):
    runs = []
    for how in range(3):
        g = torch.Generator(device=dev())
        g.manual_seed(9)
        p, gr = torch.randn(5000, generator=g, device=dev()), torch.randn(5000, generator=g, device=dev())
        m, v = (torch.zeros(5000, dtype=torch.uint8, device=dev()).view(F8) for _ in range(2))
        ms, vs = (torch.zeros(20, device=dev()) for _ in range(2))
        t = nm.AdamWTensors([p], [gr], [m], [v], [ms], [vs])
        step = lambda: nm.nm_adamw_unbiased(t, lr=1e-3, step=2, seed=1)  # noqa: E731
        torch.cuda.synchronize()
        if how == 0:
            for _ in range(3):
                step()
        elif how == 1:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(3):
                    step()
        else:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
            for _ in range(3):
                graph.replay()
        torch.cuda.synchronize()
        runs.append((p, m.view(torch.uint8), v.view(torch.uint8), ms, vs))
    for other in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(runs[0], other))


def test_seeds_steps_and_tensors_draw_their_own_bits(nm):
    def codes(seed, step):
        gr = torch.randn(4096, device=dev(), generator=torch.Generator(device=dev()).manual_seed(1))
        t = [[torch.zeros(4096, device=dev()) for _ in range(2)], [gr, gr.clone()]]
        t += [[torch.zeros(4096, dtype=torch.uint8, device=dev()).view(F8) for _ in range(2)] for _ in range(2)]
        t += [[torch.zeros(16, device=dev()) for _ in range(2)] for _ in range(2)]
        nm.nm_adamw_unbiased(nm.AdamWTensors(*t), lr=0.1, step=step, seed=seed)
        return [x.view(torch.uint8) for x in t[2] + t[3]]
    a, b, c, d = codes(1, 1), codes(1, 1), codes(2, 1), codes(1, 2)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    for other in (c, d):
        assert all((x != y).float().mean() > 0.2 for x, y in zip(a, other))
    assert (a[0] != a[1]).float().mean() > 0.2 and (a[2] != a[3]).float().mean() > 0.2


def test_binding_refuses(nm):
    x = [torch.zeros(300, device=dev()) for _ in range(4)]
    t = nm.AdamWTensors([x[0]], [x[1]], [x[2]], [x[3]])
    with pytest.raises(ValueError):
        nm.nm_adamw_unbiased(t, lr=0.1, step=1)
    s = [torch.zeros(2, device=dev()) for _ in range(2)]
    t = nm.AdamWTensors([x[0]], [x[1]], [x[2].to(F8)], [x[3].to(F8)], [s[0]], [s[1]])
    for kw in (dict(lr=-1.0, step=1), dict(lr=1.0, step=0), dict(lr=1.0, step=1, beta2=1.0)):
        with pytest.raises(nm.NMError):
            nm.nm_adamw_unbiased(t, **kw)
    with pytest.raises(ValueError):
        nm.nm_adamw_unbiased(t, lr=1.0, step=1, grad_scale=torch.ones(2, device=dev()))
