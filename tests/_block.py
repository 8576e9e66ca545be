"""Plain 64-bit forms of the gated block, its gradients and the AdamW step, and the bounds the
kernels are held to.  Every bound is a worst case of the arithmetic the header states:
  sums of n terms in f32            n 2^-24 sum |terms|
  an activation evaluated in f32    (8 + 4 a) 2^-23 relative, a the size of the exponent's
                                    argument (its rounding is what a large one magnifies)
  one rounding to bf16              2^-8 relative (8 significant bits: half a unit)
"""
import numpy as np
import torch
from scipy.special import erfc

import oracle as O
from tests._util import dev, np_bf16

SILU, GELU, GELU_TANH, RELU2 = range(4)
ACTS = [SILU, GELU, GELU_TANH, RELU2]
_C = np.sqrt(2 / np.pi)


def sigmoid(x):
    return 0.5 * (1 + np.tanh(0.5 * x))


def act(a, g):
    """(act(g), act'(g), relative error of an f32 evaluation)."""
    if a == SILU:
        s = sigmoid(g)
        return g * s, s * (1 + g * (1 - s)), (8 + 4 * np.abs(g)) * 2.0 ** -23
    if a == GELU:
        p = 0.5 * erfc(-g / np.sqrt(2))
        return g * p, p + g * np.exp(-g * g / 2) / np.sqrt(2 * np.pi), (8 + 4 * g * g) * 2.0 ** -23
    if a == GELU_TANH:
        t = _C * (g + 0.044715 * g ** 3)
        s = sigmoid(2 * t)
        return g * s, s + g * s * (1 - s) * 2 * _C * (1 + 3 * 0.044715 * g * g), (8 + 8 * np.abs(t)) * 2.0 ** -23
    r = np.maximum(g, 0)
    return r * r, 2 * r, 4 * 2.0 ** -23 * np.ones_like(g)


# largest |act''| of each activation
CURVE = {SILU: 0.5, GELU: 0.8, GELU_TANH: 0.9, RELU2: 2.0}


def bf16(a):
    """numpy array rounded to bf16, as float64."""
    return O.bf16_to_f32(O.f32_to_bf16(np.asarray(a, np.float32))).astype(np.float64)


def weight(g, R, K, Ns=0, scale=0.05, integer=False, dtype="bf16"):
    """A random weight pruned by magnitude: (dense masked f64 [R, K], vals, idx) on the device."""
    if dtype == "int8":
        Wb = g.integers(-1, 2, (R, K)).astype(np.int8)
        dense = Wb.astype(np.float64)
    elif dtype == "fp8":
        Wt = torch.from_numpy((g.integers(-8, 9, (R, K)) if integer else g.standard_normal((R, K))).astype(np.float32))
        Wt = Wt.to(torch.float8_e4m3fn)
        Wb, dense = Wt.view(torch.uint8).numpy(), Wt.float().numpy().astype(np.float64)
    else:
        Wb = O.f32_to_bf16((g.integers(-2, 3, (R, K)) if integer else g.standard_normal((R, K)) * scale).astype(np.float32))
        dense = O.bf16_to_f32(Wb).astype(np.float64)
    key = (np.abs(dense) + 1e-6 * g.random((R, K))).astype(np.float32)
    mask = O.topn_mask(key, 2 * Ns - 2, 2 * Ns) if Ns else O.topn_mask(key, 2, 4)
    if dtype == "fp8":
        Wb = Wb.view(np.int8)      # the packers move one-byte codes as they are
    if Ns:
        vals, idx, bad = O.slide_decompose(Wb, mask, Ns)
        assert bad == 0
    else:
        vals, idx = O.pack(Wb, mask, 2, 4)
    dense = np.where(O.mask_to_bool(mask, K), dense, 0.0)
    v = np_bf16(vals) if dtype == "bf16" else torch.from_numpy(np.ascontiguousarray(vals))
    if dtype == "fp8":
        v = v.view(torch.float8_e4m3fn)
    return dense, v.to(dev()), torch.from_numpy(np.ascontiguousarray(idx).view(np.int32)).to(dev())


def columns(idx, K, Ns=0):
    """Column of every packed value: [R, K/2], or [R, K'/2] of a lifted weight."""
    w = idx.cpu().numpy().view(np.uint32)
    j = np.arange((O.lifted_width(K, Ns) if Ns else K) // 2)
    win = j // 2
    start = 2 * Ns * (win // (Ns - 1)) + 2 * (win % (Ns - 1)) if Ns else 4 * win
    return start[None] + ((w[:, j // 16] >> (2 * (j % 16)).astype(np.uint32)[None]) & 3).astype(np.int64)


def take(full, idx, K, Ns=0):
    return np.take_along_axis(full, columns(idx, K, Ns), axis=1)


def strided(t, extra):
    """A copy of t [rows, cols] whose rows are extra elements further apart (the gap holds NaN
    where the type has one)."""
    if not extra:
        return t.contiguous()
    buf = torch.empty((t.shape[0], t.shape[1] + extra), dtype=t.dtype, device=t.device)
    if t.dtype in (torch.bfloat16, torch.float32):
        buf.fill_(float("nan"))
    buf[:, :t.shape[1]] = t
    return buf[:, :t.shape[1]]


def nan_ws(nbytes):
    """A workspace whose contents are NaN in every type."""
    return torch.full((max(int(nbytes), 16),), 0xFF, dtype=torch.uint8, device=dev())
