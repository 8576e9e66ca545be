"""Training a weight whose mask keeps fewer weights than its groups have slots: the padding slots' gradients are
zeroed (kept_slots), and weights outside the mask stay zero, exactly."""
import numpy as np
import pytest
import torch

import oracle as O
from tests import _block as B
from tests._util import dev, np_bf16

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def nm():
    import semi_structured_sparsity_amd as m
    return m


def _sparse_mask(g, R, K, M, most):
    """bool [R, K]: 0 .. most kept of every M."""
    score, count = g.random((R, K // M, M)), g.integers(0, most + 1, (R, K // M, 1))
    return (score.argsort(-1).argsort(-1) < count).reshape(R, K)


def _packed(g, R, K, Ns):
    """(mask bool, mask bits, vals, idx, kept by the oracle)"""
    keep = _sparse_mask(g, R, K, 2 * Ns if Ns else 4, 2 * Ns - 2 if Ns else 2)
    bits = np.packbits(keep, axis=1, bitorder="little")
    W = O.f32_to_bf16(np.where(keep, g.standard_normal((R, K)) * 0.2 + np.sign(g.standard_normal((R, K))) * 0.1, 0).astype(np.float32))
    ones = np.ones((R, K), np.int8)
    if Ns:
        (vals, idx, bad), kept = O.slide_decompose(W, bits, Ns), O.slide_decompose(ones, bits, Ns)[0]
        assert bad == 0
    else:
        (vals, idx), kept = O.pack(W, bits, 2, 4), O.pack(ones, bits, 2, 4)[0]
    return keep, torch.from_numpy(bits).to(dev()), np_bf16(vals).to(dev()), \
        torch.from_numpy(np.ascontiguousarray(idx).view(np.int32)).to(dev()), kept.astype(bool)


def _dense(vals, idx, K, Ns):
    W = np.zeros((vals.shape[0], K))
    np.add.at(W, (np.arange(vals.shape[0])[:, None], B.columns(idx, K, Ns)), vals.float().cpu().numpy().astype(np.float64))
    return W


@pytest.mark.parametrize("Ns,R,K", [(0, 33, 64), (0, 130, 528), (3, 20, 48), (4, 70, 256), (5, 16, 160), (8, 9, 128)])
def test_kept_slots_are_the_packers(nm, Ns, R, K):
    g = np.random.default_rng(R + K + Ns)
    keep, mask, vals, idx, kept = _packed(g, R, K, Ns)
    got = nm.kept_slots(mask, K, Ns)
    assert got.dtype == torch.bool and got.shape == vals.shape and np.array_equal(got.cpu().numpy(), kept)
    assert int(got.sum()) == int(keep.sum()) and not vals.float()[~got].any() and (vals.float()[got] != 0).all()
    full = nm.nm_mask(torch.randn((R, K), device=dev()), 2, 4) if Ns == 0 else None
    if full is not None:
        assert nm.kept_slots(full, K).all()


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("Ns,R,K,Mt", [(0, 70, 256, 5), (0, 300, 512, 300), (4, 70, 256, 5), (4, 300, 512, 300), (5, 64, 320, 150)])
def test_pruned_weights_stay_zero(nm, Ns, R, K, Mt, f8):
    g = np.random.default_rng(R + K + Ns + f8)
    keep, mask, vals, idx, _ = _packed(g, R, K, Ns)
    before = _dense(vals, idx, K, Ns)
    pad = ~nm.kept_slots(mask, K, Ns)
    master, dV = vals.float(), torch.empty_like(vals)
    dt = F8 if f8 else torch.float32
    m, v = (torch.zeros(master.numel(), device=dev()).to(dt) for _ in range(2))
    ms, vs = (torch.zeros((master.numel() + 255) // 256, device=dev()) for _ in range(2))
    t = nm.AdamWTensors([master], [dV], [m], [v], [ms] if f8 else None, [vs] if f8 else None, copies=[vals], weight_decay=0.1)
    for step in range(1, 7):
        X = torch.from_numpy(g.standard_normal((Mt, K)).astype(np.float32)).to(torch.bfloat16).to(dev())
        dY = torch.from_numpy(g.standard_normal((Mt, R)).astype(np.float32)).to(torch.bfloat16).to(dev())
        nm.nm_spmm_backward(dY, X, vals, idx, Ns=Ns, want_dx=False, out_dv=dV)
        if step == 1:
            assert dV.float()[pad].abs().max() > 0        # what the step leaves out
        dV.masked_fill_(pad, 0)
        if f8:
            nm.nm_adamw_unbiased(t, lr=0.01, step=step, seed=4)
        else:
            nm.nm_adamw(t, lr=0.01, step=step)
        W = _dense(vals, idx, K, Ns)
        assert not W[~keep].any() and not master[pad].any() and not m.float()[pad.view(-1)].any()
    assert (W[keep] != before[keep]).mean() > 0.9
    # and the forward pass multiplies the masked weight
    Y = nm.nm_spmm(X, vals, idx, Ns=Ns, ydt=nm.NM_F32).double().cpu().numpy()
    x = X.float().cpu().numpy().astype(np.float64)
    assert (np.abs(Y - x @ W.T) <= (K + 4) * 2.0 ** -24 * (np.abs(x) @ np.abs(W).T) + 1e-30).all()
