"""ctypes binding of include/nmsparse_layers.h, in the manner of _binding.py: ``raw.<name>`` is the C
function, ``<name>(...)`` the wrapper that takes tensors, allocates outputs and raises NMError.
These run in every layer of every token, so their checks are one expression each, and every wrapper makes
its tensors' device current for the call."""
from __future__ import annotations

import ctypes

import torch

from ._binding import (NM_ACT_SILU, NM_BF16, _DT, _F, _I, _I64, _P, _SZ, _TORCH, _check, _enter, _leave, _mat,
                       _need, _ptr, _refuse, dtype_code, lifted_width, raw)

NM_ROUTE_SOFTMAX, NM_ROUTE_SIGMOID = range(2)
NM_I4, NM_FP4 = 5, 6      # 4-bit codes of packed values: sign and 3-bit magnitude, or OCP e2m1

LAYER_SIGNATURES = {
    "nm_quant_w4": (_I, [_P, _I, _I64, _I64, _I64, _I, _I, _P, _I64, _P, _I64, _P, _I64, _P]),
    "nm_spmm_w4": (_I, [_P, _I64, _I64, _I64, _P, _I, _P, _P, _I64, _I64, _I64, _I64, _I, _I, _P, _I, _I64, _P]),
    "nm_spmm_glu_w4": (_I, [_P, _I64, _I64, _I64, _P, _P, _P, _P, _P, _P, _I, _I64, _I64, _I64, _I64, _I, _I, _I, _P, _I,
                            _I64, _P]),
    "nm_moe_workspace": (_SZ, [_I64, _I64, _I64, _I, _I]),
    "nm_moe": (_I, [_P, _I64, _I64, _I64, _P, _I64, _P, _I, _I, _I, _I, _F, _P, _P, _P, _I, _I, _I64, _I, _I, _P, _I, _I64, _P,
                    _P, _P, _SZ, _P]),
}
for _name, (_res, _args) in LAYER_SIGNATURES.items():
    _fn = getattr(raw, _name)
    _fn.restype = _res
    _fn.argtypes = _args


# ---------------------------------------------------------------- 4-bit packed weights
def nm_quant_w4(vals: torch.Tensor, qdt: int = NM_I4, group: int = 128, want_values: bool = False):
    """4-bit codes of packed values (bf16 or f32, as nm_pack and its kin write them): (codes [R, bytes] uint8, rows
    of whole 16 bytes; scales [groups, R] bf16), and with want_values the values they stand for, in vals' type.
    A scale serves group consecutive columns of the (lifted) width."""
    v = _mat(vals)
    if not v or vals.dtype not in (torch.bfloat16, torch.float32):
        _refuse("vals must be a row-major bf16 or f32 matrix", vals=vals)
    R, slots, ldv = v
    if group not in (64, 128, 256) or slots % 8:
        _refuse(f"group must be 64, 128 or 256 (got {group}) and a row a multiple of 8 values", vals=vals)
    ldc, lds = (slots // 2 + 15) // 16 * 16, (R + 3) // 4 * 4
    # the bytes past a row's codes are never read as codes; zeroed where there are any, so that no
    # stale memory travels with the weight
    codes = vals.new_empty((R, ldc), dtype=torch.uint8)
    if ldc > slots // 2:
        codes[:, slots // 2:].zero_()
    scales = vals.new_empty(((2 * slots + group - 1) // group, lds), dtype=torch.bfloat16)[:, :R]
    values = vals.new_empty((R, slots)) if want_values else None
    stream, back = _enter(vals)
    try:
        st = raw.nm_quant_w4(vals.data_ptr(), _DT[vals.dtype], R, slots, ldv, qdt, group, codes.data_ptr(), ldc,
                             scales.data_ptr(), lds, _ptr(values), slots, stream)
    finally:
        _leave(back)
    if st:
        _check(st)
    return (codes, scales, values) if want_values else (codes, scales)


def _w4(codes, idx, scales, Kl, group):
    """(rows, row strides of codes, idx and scales) of a 4-bit weight of Kl columns, or None."""
    c, i, s = _mat(codes), _mat(idx), _mat(scales)
    if not (c and i and s and codes.dtype == torch.uint8 and idx.dtype == torch.int32 and scales.dtype == torch.bfloat16):
        return None
    R = c[0]
    if i[0] != R or s[1] < R or c[1] < Kl // 4 or i[1] < (Kl + 31) // 32 or s[0] * group < Kl:
        return None
    # one group's scales may have any stride: their row is as long as it is
    return R, c[2], i[2], s[2] if s[0] > 1 else (s[1] + 3) // 4 * 4


def _out(t, dt, rows, cols, X):
    """(output, its row stride, its type)."""
    if t is None:
        return X.new_empty((rows, cols), dtype=_TORCH[dt]), cols, dt
    m = _mat(t)
    if not (m and m[:2] == (rows, cols) and t.dtype in (torch.bfloat16, torch.float32) and t.device == X.device):
        _refuse(f"out must be a row-major bf16 or f32 tensor of ({rows}, {cols})", out=t)
    return t, m[2], dtype_code(t)


def nm_spmm_w4(X: torch.Tensor, codes: torch.Tensor, idx: torch.Tensor, scales: torch.Tensor, qdt: int = NM_I4,
               group: int = 128, Ns: int = 0, ydt: int = NM_BF16, out: torch.Tensor | None = None) -> torch.Tensor:
    """Y = X W^T on a 4-bit packed weight (nm_quant_w4's codes and scales, the packers' idx), made for few tokens."""
    x = _mat(X)
    Kl = lifted_width(x[1], Ns) if x and Ns >= 2 else x[1] if x else 0
    w, dev = _w4(codes, idx, scales, Kl, group), X.device
    if not (x and w and X.dtype == torch.bfloat16 and dev == codes.device and dev == idx.device and dev == scales.device):
        _refuse(f"X must be row-major bf16 and the weight codes, idx and scales of {Kl} columns", X=X, codes=codes, idx=idx,
                scales=scales)
    (Mtok, K, ldx), (R, ldc, ldi, lds) = x, w
    Y, ldy, ydt = _out(out, ydt, Mtok, R, X)
    stream, back = _enter(X)
    try:
        st = raw.nm_spmm_w4(X.data_ptr(), Mtok, K, ldx, codes.data_ptr(), qdt, idx.data_ptr(), scales.data_ptr(), R, ldc, ldi,
                            lds, group, Ns, Y.data_ptr(), ydt, ldy, stream)
    finally:
        _leave(back)
    if st:
        _check(st)
    return Y


def nm_spmm_glu_w4(X: torch.Tensor, codes_g: torch.Tensor, idx_g: torch.Tensor, scales_g: torch.Tensor,
                   codes_u: torch.Tensor, idx_u: torch.Tensor, scales_u: torch.Tensor, qdt: int = NM_I4, group: int = 128,
                   Ns: int = 0, act: int = NM_ACT_SILU, hdt: int = NM_BF16, out: torch.Tensor | None = None) -> torch.Tensor:
    """H = act(X Wg^T) . (X Wu^T) on two 4-bit weights packed alike, in one pass."""
    x = _mat(X)
    Kl = lifted_width(x[1], Ns) if x and Ns >= 2 else x[1] if x else 0
    w, dev = _w4(codes_g, idx_g, scales_g, Kl, group), X.device
    if not (x and w and w == _w4(codes_u, idx_u, scales_u, Kl, group) and X.dtype == torch.bfloat16 and
            all(t.device == dev for t in (codes_g, idx_g, scales_g, codes_u, idx_u, scales_u))):
        _refuse(f"X must be row-major bf16 and the gate and up weights codes, idx and scales of {Kl} columns, packed alike",
                X=X, codes_g=codes_g, idx_g=idx_g, scales_g=scales_g, codes_u=codes_u, idx_u=idx_u, scales_u=scales_u)
    (Mtok, K, ldx), (R, ldc, ldi, lds) = x, w
    H, ldh, hdt = _out(out, hdt, Mtok, R, X)
    stream, back = _enter(X)
    try:
        st = raw.nm_spmm_glu_w4(X.data_ptr(), Mtok, K, ldx, codes_g.data_ptr(), idx_g.data_ptr(), scales_g.data_ptr(),
                                codes_u.data_ptr(), idx_u.data_ptr(), scales_u.data_ptr(), qdt, R, ldc, ldi, lds, group, Ns,
                                act, H.data_ptr(), hdt, ldh, stream)
    finally:
        _leave(back)
    if st:
        _check(st)
    return H


# ---------------------------------------------------------------- mixture of sparse blocks
class _Experts(ctypes.Structure):
    _fields_ = [("vals", _P), ("idx", _P), ("scales", _P), ("ld_vals", _I64), ("ld_idx", _I64), ("ld_scales", _I64),
                ("es_vals", _I64), ("es_idx", _I64), ("es_scales", _I64)]


class MoELayer:
    """The weights of a mixture-of-experts layer, as nm_moe takes them: router [E, K] bf16, the experts' gate and up
    [E, hidden, .] and down [E, K, .] weights stacked (the packers' vals or nm_quant_w4's codes, their idx, and scales
    [E, groups, rows] of 4-bit ones), an optional f32 selection bias [E].  Checked once and kept for as long as the
    object lives; build it once and use it every step."""

    def __init__(self, router, gate, gate_idx, up, up_idx, down, down_idx, hidden, vdt=NM_BF16, group=128, Ns=0,
                 gate_scales=None, up_scales=None, down_scales=None, bias=None):
        r = _mat(router)
        if not (r and router.dtype == torch.bfloat16 and router.device.type == "cuda"):
            _refuse("router must be a row-major bf16 matrix on a GPU", router=router)
        if vdt not in (NM_BF16, NM_I4, NM_FP4):
            raise ValueError("vdt is NM_BF16, NM_I4 or NM_FP4")
        if Ns and not 3 <= Ns <= 8:
            raise ValueError(f"Ns is 0 or 3 to 8, got {Ns}")
        self.experts, self.K, self.ldr = r
        self.hidden, self.vdt, self.group, self.Ns, self.device = int(hidden), vdt, group, Ns, router.device
        E, dev, four = self.experts, router.device, vdt != NM_BF16
        lift = lambda n: lifted_width(n, Ns) if Ns else n  # noqa: E731
        self.keep = [router, gate, gate_idx, gate_scales, up, up_idx, up_scales, down, down_idx, down_scales, bias]
        self.router, self.bias = router, bias
        if bias is not None and not (bias.dtype == torch.float32 and bias.shape == (E,) and bias.is_contiguous() and
                                     bias.device == dev):
            _refuse(f"bias must be {E} contiguous f32 values on {dev}", bias=bias)
        self.weights = []
        for name, rows, width, v, i, s in (("gate", self.hidden, lift(self.K), gate, gate_idx, gate_scales),
                                           ("up", self.hidden, lift(self.K), up, up_idx, up_scales),
                                           ("down", self.K, lift(self.hidden), down, down_idx, down_scales)):
            slots = width // 4 if four else width // 2
            ok = (v.dim() == 3 and i.dim() == 3 and v.dtype == (torch.uint8 if four else torch.bfloat16) and
                  i.dtype == torch.int32 and v.shape[:2] == (E, rows) == i.shape[:2] and v.shape[2] >= slots and
                  i.shape[2] >= (width + 31) // 32 and v.stride(2) == 1 == i.stride(2) and v.device == dev == i.device)
            if four and ok:
                ok = (s is not None and s.dim() == 3 and s.dtype == torch.bfloat16 and s.shape[0] == E and
                      s.shape[1] * group >= width and s.shape[2] >= rows and s.stride(2) == 1 and s.device == dev)
            if not ok:
                _refuse(f"{name}: {slots} values{' and scales' if four else ''} and {(width + 31) // 32} index words a row for "
                        f"{E} experts of {rows} rows", vals=v, idx=i, scales=s)
            lds = 0 if not four else s.stride(1) if s.shape[1] > 1 else (s.shape[2] + 3) // 4 * 4
            one = lambda t: t.stride(0) if E > 1 else 0  # noqa: E731
            self.weights.append(_Experts(v.data_ptr(), i.data_ptr(), s.data_ptr() if four else None, v.stride(1), i.stride(1), lds,
                                         one(v), one(i), one(s) if four else 0))
        self.address = [ctypes.addressof(w) for w in self.weights]

    def get_device(self) -> int:
        return self.router.get_device()


def nm_moe(layer: MoELayer, X: torch.Tensor, topk: int, act: int = NM_ACT_SILU, route: int = NM_ROUTE_SOFTMAX,
           renorm: bool = False, route_scale: float = 1.0, ydt: int = NM_BF16, want_routing: bool = False,
           out: torch.Tensor | None = None, ws: torch.Tensor | None = None):
    """Y = sum over a token's topk experts of weight * gated block, for up to 64 tokens: Y, or with want_routing
    (Y, experts [tokens, topk] int32, weights [tokens, topk] f32)."""
    x = _mat(X)
    if not (x and x[1] == layer.K and X.dtype == torch.bfloat16 and X.device == layer.device):
        _refuse(f"X must be row-major bf16 tokens of {layer.K} columns on {layer.device}", X=X)
    Mtok, K, ldx = x
    Y, ldy, ydt = _out(out, ydt, Mtok, K, X)
    sel = X.new_empty((Mtok, topk), dtype=torch.int32) if want_routing else None
    wts = X.new_empty((Mtok, topk), dtype=torch.float32) if want_routing else None
    ws = _need(raw.nm_moe_workspace(Mtok, K, layer.hidden, layer.experts, topk), ws, X)
    stream, back = _enter(X)
    try:
        st = raw.nm_moe(X.data_ptr(), Mtok, K, ldx, layer.router.data_ptr(), layer.ldr, _ptr(layer.bias), layer.experts, topk, route,
                        renorm, route_scale, *layer.address, layer.vdt, layer.group, layer.hidden, layer.Ns, act, Y.data_ptr(),
                        ydt, ldy, _ptr(sel), _ptr(wts), _ptr(ws), 0 if ws is None else ws.nbytes, stream)
    finally:
        _leave(back)
    if st:
        _check(st)
    return (Y, sel, wts) if want_routing else Y
