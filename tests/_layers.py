"""Plain 64-bit forms of the operators of nmsparse_layers.h.  Bounds as in _block.py: sums of n terms
in f32 n 2^-24 sum |terms|, one rounding to bf16 2^-8 relative."""
import numpy as np
import torch

import oracle as O
from tests import _block as B
from tests._util import dev

I4, FP4 = 5, 6
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def bf16_round(a):
    """f32 array rounded to bf16 (nearest even), as f32."""
    return O.bf16_to_f32(O.f32_to_bf16(np.asarray(a, np.float32)))


def magnitudes(qdt):
    return np.arange(8.0) if qdt == I4 else E2M1


def quant(vals, qdt, group):
    """(codes [R, slots] of 0..15, scales [groups, R] f32, values [R, slots] f64) of f32 values."""
    vals = np.asarray(vals, np.float32)
    R, slots = vals.shape
    half, mags = group // 2, magnitudes(qdt)
    codes, scales = np.zeros((R, slots), np.uint8), []
    values = np.zeros((R, slots))
    for a in range(0, slots, half):
        b = vals[:, a:a + half]
        top = np.abs(b).max(1)
        bad = ~np.isfinite(top)
        with np.errstate(all="ignore"):
            s = bf16_round(top / np.float32(mags[-1]))
        s = np.where(bad, np.float32(np.nan), s).astype(np.float32)
        with np.errstate(all="ignore"):
            q = np.abs(b / s[:, None]).astype(np.float64)       # the f32 quotient
        q = np.where((s[:, None] > 0) & np.isfinite(q), q, 0.0)
        # nearest magnitude, of two equally near the one with the even code
        d = np.abs(np.minimum(q, mags[-1])[..., None] - mags)
        m = (d - 1e-9 * (np.arange(8) % 2 == 0)).argmin(-1)
        neg = (np.signbit(b)) & (m > 0)
        codes[:, a:a + half] = m + 8 * neg
        scales.append(s)
        values[:, a:a + half] = np.where(neg, -1.0, 1.0) * mags[m] * s[:, None].astype(np.float64)
    return codes, np.stack(scales), values


def unpack_codes(codes, slots):
    c = codes.cpu().numpy()
    return np.stack([c & 15, c >> 4], -1).reshape(c.shape[0], -1)[:, :slots]


def scatter(values, idx, K, Ns=0):
    """Dense f64 [R, K] of packed values (sums where windows overlap)."""
    full = np.zeros((values.shape[0], K))
    np.add.at(full, (np.arange(values.shape[0])[:, None], B.columns(idx, K, Ns)), values)
    return full


def w4_weight(nm, g, R, K, Ns, qdt, group, integer=False):
    """(dense f64 [R, K], codes, idx, scales) of a random pruned weight, codes by the library's quantiser's
    rule.  integer: scales are powers of two, so that sums of small integers are exact."""
    _, vals, idx = B.weight(g, R, K, Ns)
    slots = vals.shape[1]
    ngroups = -(-2 * slots // group)
    if integer:
        codes = g.integers(0, 16, (R, slots)).astype(np.uint8)
        scales = 2.0 ** g.integers(-2, 3, (ngroups, R))
        mags = magnitudes(qdt)
        values = np.where(codes >= 8, -1.0, 1.0) * mags[codes & 7] * scales.repeat(group // 2, 0)[:slots].T
    else:
        codes, scales, values = quant(vals.float().cpu().numpy(), qdt, group)
    ldc = -(-slots // 32) * 16
    packed = np.full((R, ldc), 0xFF, np.uint8)       # garbage past a row's codes
    even = np.zeros((R, slots + slots % 2), np.uint8)
    even[:, :slots] = codes
    packed[:, :slots // 2] = (even[:, 0::2] | even[:, 1::2] << 4)[:, :slots // 2]
    sc = torch.full((ngroups, -(-R // 4) * 4), float("nan"), dtype=torch.bfloat16)
    sc[:, :R] = torch.from_numpy(scales.astype(np.float32)).to(torch.bfloat16)
    return scatter(values, idx, K, Ns), torch.from_numpy(packed).to(dev()), idx, sc.to(dev())[:, :R]


def product_bound(Xf, W, K):
    """Error of an f32 evaluation of X W^T."""
    return (K + 8) * 2.0 ** -24 * (np.abs(Xf) @ np.abs(W).T)
