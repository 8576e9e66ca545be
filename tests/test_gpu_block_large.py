"""Outputs and operands whose offsets pass 32 bits: the gated block and its gradients on small
integers (every sum exact), compared on the first, the last and random rows."""
import numpy as np
import pytest
import torch

from tests import _block as B
from tests._util import dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nm():
    import semi_structured_sparsity_amd as m
    return m


def _ints(seed, shape, lim, dtype=torch.bfloat16):
    g = torch.Generator(device=dev())
    g.manual_seed(seed)
    return torch.randint(-lim, lim + 1, shape, generator=g, device=dev(), dtype=torch.int8).to(dtype)


def _rows(n, seed):
    g = np.random.default_rng(seed)
    return torch.from_numpy(np.unique(np.concatenate([[0, 1, n - 2, n - 1], g.integers(0, n, 60)]))).to(dev())


def test_glu_output_past_32_bits(nm):
    g = np.random.default_rng(1)
    Mt, R, K = 70001, 16400, 64           # H: 4.6 GB in f32
    Wg, vg, ig = B.weight(g, R, K, integer=True)
    Wu, vu, iu = B.weight(g, R, K, integer=True)
    X = _ints(2, (Mt, K), 2)
    H = nm.nm_spmm_glu(X, vg, ig, vu, iu, act=B.RELU2, hdt=nm.NM_F32)
    assert H.numel() * 4 > 2 ** 32
    r = _rows(Mt, 3)
    x = X[r].double()
    G, U = x @ torch.from_numpy(Wg).to(dev()).t(), x @ torch.from_numpy(Wu).to(dev()).t()
    ref = G.clamp(min=0).square() * U
    # |g| <= 64 * 4, g^2 u below 2^24: exact in f32
    assert ref.abs().max() < 2 ** 24 and torch.equal(H[r].double(), ref)


def test_glu_backward_operands_past_32_bits(nm):
    g = np.random.default_rng(4)
    Mt, R, K = 70001, 16400, 64           # dG | dU and their transpose: 4.6 GB each
    Wg, vg, ig = B.weight(g, R, K, integer=True)
    Wu, vu, iu = B.weight(g, R, K, integer=True)
    X, dH = _ints(5, (Mt, K), 2), _ints(6, (Mt, R), 1)
    G, U = _ints(7, (Mt, R), 1), _ints(8, (Mt, R), 1)
    dX, dVg, dVu = nm.nm_spmm_glu_backward(dH, G, U, X, vg, ig, vu, iu, act=B.RELU2, dxdt=nm.NM_F32, dvdt=nm.NM_F32)
    r = _rows(Mt, 9)
    h, p, u = dH[r].double(), G[r].double(), U[r].double()
    dG, dU = h * u * 2 * p.clamp(min=0), h * p.clamp(min=0).square()
    ref = dG @ torch.from_numpy(Wg).to(dev()) + dU @ torch.from_numpy(Wu).to(dev())
    assert torch.equal(dX[r].double(), ref)
    c = _rows(R, 10)
    h, p, u = dH[:, c].float(), G[:, c].float(), U[:, c].float()
    for got, d, i in ((dVg, h * u * 2 * p.clamp(min=0), ig), (dVu, h * p.clamp(min=0).square(), iu)):
        full = (d.double().t() @ X.double()).cpu().numpy()          # |sums| below 2^24: exact in f32
        assert np.abs(full).max() < 2 ** 24
        cols = B.columns(i[c], K)
        assert np.array_equal(got[c].double().cpu().numpy(), np.take_along_axis(full, cols, axis=1))
