"""ctypes binding of libnmsparse (the C ABI in include/nmsparse.h).

Argument marshalling only: torch tensors supply device memory and the current
HIP stream; every step runs in the library's HIP kernels.  There is no CPU
fallback -- importing this module without the built library raises.

Each C entry point is exposed twice:
  * ``raw.<name>`` -- the ctypes function with the exact C signature;
  * ``<name>(...)``  -- a wrapper with the same name that takes tensors,
    allocates outputs with ``torch.empty`` on the input's device, passes
    pointers, and raises ``NMError`` with the library's message on failure.
"""
from __future__ import annotations

import bisect
import ctypes
import functools
import warnings
from pathlib import Path

import torch

_PKG = Path(__file__).resolve().parent
LIB_PATH = _PKG / "libnmsparse.so"

NM_OK, NM_ERR_NULL, NM_ERR_SHAPE, NM_ERR_PATTERN, NM_ERR_DTYPE, NM_ERR_ALIGN, NM_ERR_WORKSPACE, NM_ERR_DEVICE, NM_ERR_ALIAS = range(9)
STATUS_NAMES = ["NM_OK", "NM_ERR_NULL", "NM_ERR_SHAPE", "NM_ERR_PATTERN", "NM_ERR_DTYPE", "NM_ERR_ALIGN",
                "NM_ERR_WORKSPACE", "NM_ERR_DEVICE", "NM_ERR_ALIAS"]
NM_F32, NM_BF16, NM_I8, NM_I32, NM_FP8 = 0, 1, 2, 3, 4
NM_SCORE_HESSIAN, NM_SCORE_MAGNITUDE = 0, 1
NM_FLAG_VALIDATE = 1
NM_ACT_SILU, NM_ACT_GELU, NM_ACT_GELU_TANH, NM_ACT_RELU2 = range(4)

# NM_FP8 travels as torch.float8_e4m3fn (OCP e4m3 codes, one byte each)
_DT = {torch.float32: NM_F32, torch.bfloat16: NM_BF16, torch.int8: NM_I8, torch.int32: NM_I32,
       torch.float8_e4m3fn: NM_FP8}
_TORCH = {v: k for k, v in _DT.items()}


class NMError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS_NAMES[status] if 0 <= status < len(STATUS_NAMES) else status}: {msg}")
        self.status = status


if not LIB_PATH.exists():
    raise ImportError(f"{LIB_PATH} is not built; run `python -c 'import __graft_entry__ as g; g.build()'` "
                      "(or semi_structured_sparsity_amd/build.py) first")

raw = ctypes.CDLL(str(LIB_PATH))

_P, _I64, _I, _F, _U64, _SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_uint64, ctypes.c_size_t
_U = ctypes.c_uint
_D = ctypes.c_double

SIGNATURES = {
    "nm_abi_version": (_I, []),
    "nm_last_error": (ctypes.c_char_p, []),
    "nm_colsumsq_workspace": (_SZ, [_I64, _I64]),
    "nm_hdiag_colsumsq": (_I, [_P, _I, _I64, _I64, _I64, _P, _P, _SZ, _P]),
    "nm_hutchinson_workspace": (_SZ, [_I64, _I64, _I64, _I]),
    "nm_hdiag_hutchinson": (_I, [_P, _I64, _I64, _I64, _I64, _I, _U64, _P, _I64, _P, _SZ, _P]),
    "nm_hutchinson_score_workspace": (_SZ, [_I64, _I64, _I64, _I]),
    "nm_hutchinson_score": (_I, [_P, _I64, _I64, _I64, _I64, _I, _U64, _P, _I, _I64, _F, _P, _I64, _P, _P, _SZ, _P]),
    "nm_score": (_I, [_P, _I, _I64, _I64, _I64, _P, _I64, _F, _I, _P, _I64, _P]),
    "nm_stats_workspace": (_SZ, [_I64, _I64]),
    "nm_score_stats": (_I, [_P, _I64, _I64, _I64, _P, _P, _SZ, _P]),
    "nm_gate_workspace": (_SZ, [_I64, _I64, _I]),
    "nm_gate": (_I, [_P, _I64, _I64, _I64, _P, _I, _I, _F, _F, _I, _I, _P, _I64, _P, _I64, _P, _P, _SZ, _P]),
    "nm_gate_pack": (_I, [_P, _I64, _I64, _I64, _P, _I, _I, _F, _F, _I, _I, _P, _I64, _P, _I64, _P,
                          _P, _I, _I64, _I, _P, _I64, _P, _I64, _P, _SZ, _P]),
    "nm_mask": (_I, [_P, _I64, _I64, _I64, _I, _I, _P, _I64, _P]),
    "nm_pack": (_I, [_P, _I, _I64, _I64, _I64, _P, _I64, _I, _I, _I, _P, _I64, _P, _I64, _U, _P]),
    "nm_prune_pack": (_I, [_P, _I, _I64, _P, _I64, _F, _I, _P, _I, _I64, _I64, _I64, _I, _I, _P, _I64, _I, _P, _I64,
                           _P, _I64, _P]),
    "nm_slide_decompose": (_I, [_P, _I, _I64, _I64, _I64, _P, _I64, _I, _I, _P, _I64, _P, _I64, _U, _P]),
    "nm_prune_slide": (_I, [_P, _I, _I64, _P, _I64, _F, _I, _P, _I, _I64, _I64, _I64, _I, _P, _I64, _I, _P, _I64, _P,
                            _I64, _P]),
    "nm_absmean": (_I, [_P, _I, _I64, _I64, _I64, _P, _P, _SZ, _P]),
    "nm_quant_lift": (_I, [_P, _I, _I64, _I64, _I64, _I, _I, _P, _I64, _P, _P]),
    "nm_spmm_workspace": (_SZ, [_I64, _I64, _I64, _I, _I]),
    "nm_spmm": (_I, [_P, _I, _I64, _I64, _I64, _P, _I, _P, _I64, _I64, _I64, _I, _P, _F, _P, _I, _I64, _P, _SZ, _P]),
    "nm_spmm_noalloc": (_I, [_P, _I, _I64, _I64, _I64, _P, _I, _P, _I64, _I64, _I64, _I, _P, _F, _P, _I, _I64, _P]),
    "nm_spmm_lowrank_workspace": (_SZ, [_I64, _I64, _I64, _I, _I]),
    "nm_bitmap_encode": (_I, [_P, _I, _I64, _I64, _I64, _P, _I64, _P, _I64, _P, _I64, _P]),
    "nm_spmm_bitmap_workspace": (_SZ, [_I64, _I64, _I64]),
    "nm_spmm_bitmap": (_I, [_P, _I64, _I64, _I64, _P, _I64, _P, _I64, _P, _I64, _I64, _P, _I, _I64, _P, _SZ, _P]),
    "nm_spmm_lowrank": (_I, [_P, _I64, _I64, _I64, _P, _P, _I64, _I64, _I64, _I, _P, _I64, _P, _I64, _I, _P, _I, _I64,
                             _P, _SZ, _P]),
    "nm_spmm_glu_workspace": (_SZ, [_I64, _I64, _I64, _I, _I]),
    "nm_spmm_glu": (_I, [_P, _I, _I64, _I64, _I64, _P, _P, _P, _P, _I, _I64, _I64, _I64, _I, _P, _F, _F, _I, _P, _I,
                         _I64, _P, _P, _I64, _P, _SZ, _P]),
    "nm_spmm_backward_workspace": (_SZ, [_I64, _I64, _I64, _I]),
    "nm_spmm_backward": (_I, [_P, _I64, _P, _I64, _I64, _I64, _P, _P, _I64, _I64, _I64, _I, _P, _I, _I64, _P, _I, _I64,
                              _P, _SZ, _P]),
    "nm_spmm_glu_backward_workspace": (_SZ, [_I64, _I64, _I64, _I]),
    "nm_spmm_glu_backward": (_I, [_P, _I64, _P, _P, _I64, _I, _P, _I64, _I64, _I64, _P, _P, _P, _P, _I64, _I64, _I64, _I,
                                  _P, _I, _I64, _P, _P, _I, _I64, _P, _SZ, _P]),
    "nm_adamw": (_I, [_P, _I, _I, _D, _D, _D, _D, _I64, _P, _P]),
    "nm_adamw_unbiased": (_I, [_P, _I, _D, _D, _D, _D, _I64, _U64, _P, _P]),
}
for _name, (_res, _args) in SIGNATURES.items():
    _fn = getattr(raw, _name)
    _fn.restype = _res
    _fn.argtypes = _args


def last_error() -> str:
    m = raw.nm_last_error()
    return m.decode() if m else ""


def _check(st: int):
    if st != NM_OK:
        raise NMError(st, last_error())


def _ptr(t):
    return None if t is None else t.data_ptr()


def _ld(t: torch.Tensor) -> int:
    """Leading dimension (elements) of a 2-D row-major view."""
    if t.dim() == 1:
        return t.shape[0]
    assert t.stride(1) == 1, "tensors must be row-major (unit stride along the last dimension)"
    return t.stride(0)


def _stream(t: torch.Tensor | None = None):
    index = -1 if t is None else t.get_device()
    return torch.cuda.current_stream().cuda_stream if index < 0 else torch._C._cuda_getCurrentRawStream(index)


def _ws(nbytes: int, device) -> torch.Tensor | None:
    return torch.empty(max(int(nbytes), 1), dtype=torch.uint8, device=device) if nbytes else None


def dtype_code(t: torch.Tensor) -> int:
    return _DT[t.dtype]


def index_words(slots: int, M: int) -> int:
    b = (M - 1).bit_length()
    return (slots * b + 31) // 32


def lifted_width(K: int, Ns: int) -> int:
    return K // (2 * Ns) * 4 * (Ns - 1)


# ---------------------------------------------------------------- wrappers
def nm_abi_version() -> int:
    return raw.nm_abi_version()


def nm_hdiag_colsumsq(X: torch.Tensor) -> torch.Tensor:
    n, K = X.shape
    H = torch.empty(K, dtype=torch.float32, device=X.device)
    ws = _ws(raw.nm_colsumsq_workspace(n, K), X.device)
    _check(raw.nm_hdiag_colsumsq(_ptr(X), dtype_code(X), n, K, _ld(X), _ptr(H), _ptr(ws),
                                 0 if ws is None else ws.numel(), _stream(X)))
    return H


def nm_hdiag_hutchinson(X: torch.Tensor, R: int, probes: int, seed: int) -> torch.Tensor:
    n, K = X.shape
    D = torch.empty((R, K), dtype=torch.float32, device=X.device)
    ws = _ws(raw.nm_hutchinson_workspace(n, K, R, probes), X.device)
    _check(raw.nm_hdiag_hutchinson(_ptr(X), n, K, _ld(X), R, probes, seed, _ptr(D), K, _ptr(ws),
                                   0 if ws is None else ws.numel(), _stream(X)))
    return D


def nm_hutchinson_score(X: torch.Tensor, W: torch.Tensor, probes: int, seed: int, eps: float,
                        want_stats: bool = True):
    """S = (D + eps) W^2 with D the Hutchinson diagonal of ||X W^T||^2 (never stored), and
    the per-tensor (mean, std) of S: returns (S [R, K] f32, stats [2] f64 or None)."""
    n, K = X.shape
    R = W.shape[0]
    S = torch.empty((R, K), dtype=torch.float32, device=X.device)
    st = torch.empty(2, dtype=torch.float64, device=X.device) if want_stats else None
    ws = _ws(raw.nm_hutchinson_score_workspace(n, K, R, probes), X.device)
    _check(raw.nm_hutchinson_score(_ptr(X), n, K, _ld(X), R, probes, seed, _ptr(W), dtype_code(W), _ld(W), eps,
                                   _ptr(S), K, _ptr(st), _ptr(ws), 0 if ws is None else ws.numel(), _stream(X)))
    return S, st


def nm_score(W: torch.Tensor, H: torch.Tensor | None, eps: float, mode: int = NM_SCORE_HESSIAN) -> torch.Tensor:
    R, K = W.shape
    S = torch.empty((R, K), dtype=torch.float32, device=W.device)
    ldh = 0 if (H is None or H.dim() == 1) else _ld(H)
    _check(raw.nm_score(_ptr(W), dtype_code(W), R, K, _ld(W), _ptr(H), ldh, eps, mode, _ptr(S), K, _stream(W)))
    return S


def nm_score_stats(S: torch.Tensor) -> torch.Tensor:
    R, K = S.shape
    st = torch.empty(2, dtype=torch.float64, device=S.device)
    ws = _ws(raw.nm_stats_workspace(R, K), S.device)
    _check(raw.nm_score_stats(_ptr(S), R, K, _ld(S), _ptr(st), _ptr(ws), ws.numel(), _stream(S)))
    return st


def nm_gate(S: torch.Tensor, stats: torch.Tensor, N: int, M: int, T0: float, rho: float, steps: int,
            want_m: bool = True, m_step: int | None = None):
    """Returns (m_t [R, K] f32 of step m_step (default the last) or None, hard mask, lmid [steps])."""
    R, K = S.shape
    t = steps - 1 if m_step is None else m_step
    mf = torch.empty((R, K), dtype=torch.float32, device=S.device) if want_m else None
    hm = torch.empty((R, (K + 7) // 8), dtype=torch.uint8, device=S.device)
    lm = torch.empty(steps, dtype=torch.float64, device=S.device)
    ws = _ws(raw.nm_gate_workspace(R, K, steps), S.device)
    _check(raw.nm_gate(_ptr(S), R, K, _ld(S), _ptr(stats), N, M, T0, rho, steps, t, _ptr(mf), K, _ptr(hm),
                       hm.shape[1], _ptr(lm), _ptr(ws), ws.numel(), _stream(S)))
    return mf, hm, lm


def nm_gate_pack(S: torch.Tensor, stats: torch.Tensor, W: torch.Tensor, N: int, M: int, T0: float, rho: float,
                 steps: int, want_m: bool = True, m_step: int | None = None, vdt: int | None = None):
    """nm_gate and the pack of W under its hard mask in one call: returns (m_t or None,
    hard mask, lmid, vals, idx)."""
    R, K = S.shape
    t = steps - 1 if m_step is None else m_step
    vdt = dtype_code(W) if vdt is None else vdt
    mf = torch.empty((R, K), dtype=torch.float32, device=S.device) if want_m else None
    hm = torch.empty((R, (K + 7) // 8), dtype=torch.uint8, device=S.device)
    lm = torch.empty(steps, dtype=torch.float64, device=S.device)
    slots = K // M * N
    vals, idx = _pack_out(R, slots, index_words(slots, M), vdt, S.device)
    ws = _ws(raw.nm_gate_workspace(R, K, steps), S.device)
    _check(raw.nm_gate_pack(_ptr(S), R, K, _ld(S), _ptr(stats), N, M, T0, rho, steps, t, _ptr(mf), K, _ptr(hm),
                            hm.shape[1], _ptr(lm), _ptr(W), dtype_code(W), _ld(W), vdt, _ptr(vals), slots, _ptr(idx),
                            idx.shape[1], _ptr(ws), ws.numel(), _stream(S)))
    return mf, hm, lm, vals, idx


def nm_mask(S: torch.Tensor, N: int, M: int) -> torch.Tensor:
    R, K = S.shape
    mask = torch.empty((R, (K + 7) // 8), dtype=torch.uint8, device=S.device)
    _check(raw.nm_mask(_ptr(S), R, K, _ld(S), N, M, _ptr(mask), mask.shape[1], _stream(S)))
    return mask


def _pack_out(R, slots, words, vdt, device):
    vals = torch.empty((R, slots), dtype=_TORCH[vdt], device=device)
    idx = torch.empty((R, words), dtype=torch.int32, device=device)
    return vals, idx


def nm_pack(W: torch.Tensor, mask: torch.Tensor, N: int, M: int, vdt: int | None = None, flags: int = 0):
    R, K = W.shape
    vdt = dtype_code(W) if vdt is None else vdt
    slots = K // M * N
    vals, idx = _pack_out(R, slots, index_words(slots, M), vdt, W.device)
    _check(raw.nm_pack(_ptr(W), dtype_code(W), R, K, _ld(W), _ptr(mask), _ld(mask), N, M, vdt, _ptr(vals), slots,
                       _ptr(idx), idx.shape[1], flags, _stream(W)))
    return vals, idx


def nm_prune_pack(W: torch.Tensor, H: torch.Tensor | None, eps: float, mode: int, N: int, M: int,
                  Wv: torch.Tensor | None = None, vdt: int | None = None, want_mask: bool = True):
    """Fused score -> top-N -> pack.  Score from W, values from Wv (default W)."""
    R, K = W.shape
    Wv = W if Wv is None else Wv
    vdt = (NM_BF16 if Wv.dtype == torch.float32 else dtype_code(Wv)) if vdt is None else vdt
    slots = K // M * N
    vals, idx = _pack_out(R, slots, index_words(slots, M), vdt, W.device)
    mask = torch.empty((R, (K + 7) // 8), dtype=torch.uint8, device=W.device) if want_mask else None
    ldh = 0 if (H is None or H.dim() == 1) else _ld(H)
    _check(raw.nm_prune_pack(_ptr(W), dtype_code(W), _ld(W), _ptr(H), ldh, eps, mode, _ptr(Wv), dtype_code(Wv),
                             _ld(Wv), R, K, N, M, _ptr(mask), (K + 7) // 8, vdt, _ptr(vals), slots, _ptr(idx),
                             idx.shape[1], _stream(W)))
    return vals, idx, mask


def nm_slide_decompose(W: torch.Tensor, mask: torch.Tensor, Ns: int, vdt: int | None = None, flags: int = 0):
    R, K = W.shape
    vdt = dtype_code(W) if vdt is None else vdt
    Kl = lifted_width(K, Ns)
    vals, idx = _pack_out(R, Kl // 2, (Kl + 31) // 32, vdt, W.device)
    _check(raw.nm_slide_decompose(_ptr(W), dtype_code(W), R, K, _ld(W), _ptr(mask), _ld(mask), Ns, vdt, _ptr(vals),
                                  vals.shape[1], _ptr(idx), idx.shape[1], flags, _stream(W)))
    return vals, idx


def nm_prune_slide(W: torch.Tensor, H: torch.Tensor | None, eps: float, mode: int, Ns: int,
                   Wv: torch.Tensor | None = None, vdt: int | None = None, want_mask: bool = True):
    R, K = W.shape
    Wv = W if Wv is None else Wv
    vdt = dtype_code(Wv) if vdt is None else vdt
    Kl = lifted_width(K, Ns)
    vals, idx = _pack_out(R, Kl // 2, (Kl + 31) // 32, vdt, W.device)
    mask = torch.empty((R, (K + 7) // 8), dtype=torch.uint8, device=W.device) if want_mask else None
    ldh = 0 if (H is None or H.dim() == 1) else _ld(H)
    _check(raw.nm_prune_slide(_ptr(W), dtype_code(W), _ld(W), _ptr(H), ldh, eps, mode, _ptr(Wv), dtype_code(Wv),
                              _ld(Wv), R, K, Ns, _ptr(mask), (K + 7) // 8, vdt, _ptr(vals), vals.shape[1], _ptr(idx),
                              idx.shape[1], _stream(W)))
    return vals, idx, mask


def nm_absmean(W: torch.Tensor) -> torch.Tensor:
    R, K = W.shape
    a = torch.empty(1, dtype=torch.float32, device=W.device)
    ws = _ws(raw.nm_stats_workspace(R, K), W.device)
    _check(raw.nm_absmean(_ptr(W), dtype_code(W), R, K, _ld(W), _ptr(a), _ptr(ws), ws.numel(), _stream(W)))
    return a


def nm_quant_lift(X: torch.Tensor, Ns: int = 4, qdt: int = NM_I8) -> tuple[torch.Tensor, torch.Tensor]:
    """Per-token int8 or FP8 codes of bf16 X (lifted for Ns >= 3) and their scales."""
    Mtok, K = X.shape
    Kl = lifted_width(K, Ns) if Ns else K
    Xq = torch.empty((Mtok, Kl), dtype=_TORCH[qdt], device=X.device)
    sx = torch.empty(Mtok, dtype=torch.float32, device=X.device)
    _check(raw.nm_quant_lift(_ptr(X), dtype_code(X), Mtok, K, _ld(X), Ns, qdt, _ptr(Xq), Kl, _ptr(sx), _stream(X)))
    return Xq, sx


def nm_bitmap_encode(W: torch.Tensor, mask: torch.Tensor, ldv: int | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """Bitmap format of bf16 W under mask: (vals [R, ldv] bf16, offs [R, K/64 + 1] int32)."""
    R, K = W.shape
    ldv = K if ldv is None else ldv
    vals = torch.zeros((R, ldv), dtype=torch.bfloat16, device=W.device)
    offs = torch.empty((R, K // 64 + 1), dtype=torch.int32, device=W.device)
    _check(raw.nm_bitmap_encode(_ptr(W), dtype_code(W), R, K, _ld(W), _ptr(mask), _ld(mask), _ptr(vals), ldv,
                                _ptr(offs), _ld(offs), _stream(W)))
    return vals, offs


def nm_spmm_bitmap(X: torch.Tensor, vals: torch.Tensor, mask: torch.Tensor, offs: torch.Tensor, R: int | None = None,
                   ydt: int = NM_BF16, out: torch.Tensor | None = None, ws: torch.Tensor | None = None) -> torch.Tensor:
    """Y = X W_hat^T with W_hat in the bitmap format (decode into LDS, then dense MFMA)."""
    Mtok, K = X.shape
    R = vals.shape[0] if R is None else R
    Y = out if out is not None else torch.empty((Mtok, R), dtype=_TORCH[ydt], device=X.device)
    need = raw.nm_spmm_bitmap_workspace(Mtok, K, R)
    if need and (ws is None or ws.numel() < need):
        ws = _ws(need, X.device)
    _check(raw.nm_spmm_bitmap(_ptr(X), Mtok, K, _ld(X), _ptr(vals), _ld(vals), _ptr(mask), _ld(mask), _ptr(offs),
                              _ld(offs), R, _ptr(Y), ydt, _ld(Y), _ptr(ws), 0 if ws is None else ws.numel(),
                              _stream(X)))
    return Y


def nm_spmm_lowrank(X: torch.Tensor, vals: torch.Tensor, idx: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                    R: int | None = None, Ns: int = 0, ydt: int = NM_BF16, out: torch.Tensor | None = None,
                    ws: torch.Tensor | None = None) -> torch.Tensor:
    """Y = X W_hat^T + bf16(X A^T) B^T: sparse layer plus stacked low-rank adapters (bf16)."""
    Mtok, K = X.shape
    R = vals.shape[0] if R is None else R
    rank = A.shape[0]
    Y = out if out is not None else torch.empty((Mtok, R), dtype=_TORCH[ydt], device=X.device)
    need = raw.nm_spmm_lowrank_workspace(Mtok, K, R, Ns, rank)
    if need and (ws is None or ws.numel() < need):
        ws = _ws(need, X.device)
    _check(raw.nm_spmm_lowrank(_ptr(X), Mtok, K, _ld(X), _ptr(vals), _ptr(idx), R, _ld(vals), _ld(idx), Ns,
                               _ptr(A), _ld(A), _ptr(B), _ld(B), rank, _ptr(Y), ydt, _ld(Y), _ptr(ws),
                               0 if ws is None else ws.numel(), _stream(X)))
    return Y


def nm_spmm(X: torch.Tensor, vals: torch.Tensor, idx: torch.Tensor, R: int | None = None, Ns: int = 0,
            x_scale: torch.Tensor | None = None, w_scale: float = 1.0, ydt: int | None = None,
            out: torch.Tensor | None = None, ws: torch.Tensor | None = None) -> torch.Tensor:
    Mtok, K = X.shape
    R = vals.shape[0] if R is None else R
    xdt = dtype_code(X)
    if ydt is None:
        ydt = {NM_BF16: NM_BF16, NM_I8: NM_I32, NM_FP8: NM_F32}[xdt]
    Y = out if out is not None else torch.empty((Mtok, R), dtype=_TORCH[ydt], device=X.device)
    need = raw.nm_spmm_workspace(Mtok, K, R, Ns, xdt)
    if need and (ws is None or ws.numel() < need):
        ws = _ws(need, X.device)
    _check(raw.nm_spmm(_ptr(X), xdt, Mtok, K, _ld(X), _ptr(vals), dtype_code(vals), _ptr(idx), R, _ld(vals), _ld(idx),
                       Ns, _ptr(x_scale), w_scale, _ptr(Y), ydt, _ld(Y), _ptr(ws), 0 if ws is None else ws.numel(),
                       _stream(X)))
    return Y


NM_SPMM_SCRATCH_BYTES = 64 << 20


def nm_spmm_noalloc(X: torch.Tensor, vals: torch.Tensor, idx: torch.Tensor, R: int | None = None, Ns: int = 0,
                    x_scale: torch.Tensor | None = None, w_scale: float = 1.0, ydt: int | None = None,
                    out: torch.Tensor | None = None) -> torch.Tensor:
    """nm_spmm with the library's own per-device scratch buffer instead of a workspace (for
    callers that cannot allocate); give `out` to allocate nothing here either."""
    Mtok, K = X.shape
    R = vals.shape[0] if R is None else R
    xdt = dtype_code(X)
    if ydt is None:
        ydt = {NM_BF16: NM_BF16, NM_I8: NM_I32, NM_FP8: NM_F32}[xdt]
    Y = out if out is not None else torch.empty((Mtok, R), dtype=_TORCH[ydt], device=X.device)
    _check(raw.nm_spmm_noalloc(_ptr(X), xdt, Mtok, K, _ld(X), _ptr(vals), dtype_code(vals), _ptr(idx), R, _ld(vals),
                               _ld(idx), Ns, _ptr(x_scale), w_scale, _ptr(Y), ydt, _ld(Y), _stream(X)))
    return Y


# ---------------------------------------------------------------- gated feed-forward block, training
# These run every layer of every step, so their checks are one expression each; what it found is
# looked up only when it fails.
def _enter(t) -> tuple[int, int]:
    """t's device made current, for the call of the library (it launches there, and a default stream is the same
    0 on every device): (the current stream, the device to go back to or -1)."""
    index = t.get_device()
    if index < 0:
        raise ValueError(f"tensors must be on a GPU, got {t.device}")
    now = torch._C._cuda_getDevice()
    if now == index:
        return torch._C._cuda_getCurrentRawStream(index), -1
    torch._C._cuda_setDevice(index)
    return torch._C._cuda_getCurrentRawStream(index), now


def _leave(back: int):
    if back >= 0:
        torch._C._cuda_setDevice(back)


def _mat(t: torch.Tensor):
    """(rows, columns, leading dimension) of a row-major 2-D view (a one-row view's may be
    anything), or None.  Each property of a tensor costs about 0.1 us and these calls are short:
    they are read once."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 2 or (stride[1] != 1 and shape[1] > 1):
        return None
    r, c = shape
    return r, c, stride[0] if r > 1 else max(stride[0], c)


def _need(need: int, ws: torch.Tensor | None, like: torch.Tensor) -> torch.Tensor | None:
    """The caller's workspace where it has need bytes, else a new one."""
    if need and (ws is None or ws.nbytes < need):
        ws = like.new_empty(need, dtype=torch.uint8)
    elif ws is not None and not (ws.is_contiguous() and ws.device == like.device):
        _refuse(f"ws must be contiguous and on {like.device}", ws=ws)
    return ws


def _same(what: str, *pairs):
    for a, b in pairs:
        if a != b:
            raise ValueError(f"{what}: got {a}, expected {b}")


def _refuse(what: str, **tensors):
    got = ", ".join(f"{k} {tuple(t.shape)} strides {t.stride()} {t.dtype} {t.device}" for k, t in tensors.items()
                    if isinstance(t, torch.Tensor))
    raise ValueError(f"{what}; got {got}")


def nm_spmm_glu(X: torch.Tensor, vals_g: torch.Tensor, idx_g: torch.Tensor, vals_u: torch.Tensor, idx_u: torch.Tensor,
                Ns: int = 0, act: int = NM_ACT_SILU, x_scale: torch.Tensor | None = None, g_scale: float = 1.0,
                u_scale: float = 1.0, hdt: int | None = None, save: bool = False, out: torch.Tensor | None = None,
                ws: torch.Tensor | None = None):
    """H = act(G) . U with G = X Wg^T and U = X Wu^T on packed weights, in one pass: H, or with
    save (H, G, U), the bf16 pre-activations that nm_spmm_glu_backward takes."""
    x, v, i, dev = _mat(X), _mat(vals_g), _mat(idx_g), X.device
    if not (x and v and i and v == _mat(vals_u) and i == _mat(idx_u) and
            vals_g.dtype == X.dtype == vals_u.dtype and idx_g.dtype == torch.int32 == idx_u.dtype and X.dtype in _DT and
            dev == vals_g.device and dev == idx_g.device and dev == vals_u.device and dev == idx_u.device):
        _refuse("X must be row-major and the gate and up weights packed alike, in X's type", X=X, vals_g=vals_g,
                idx_g=idx_g, vals_u=vals_u, idx_u=idx_u)
    (Mtok, K, ldx), (R, slots, ldv), (irows, words, ldi) = x, v, i
    Kl = lifted_width(K, Ns) if Ns >= 2 else K
    if slots < Kl // 2 or irows != R or words < (Kl + 31) // 32:
        _refuse(f"{Kl // 2} values and {(Kl + 31) // 32} index words per row are needed", vals=vals_g, idx=idx_g)
    if x_scale is not None and not (x_scale.dtype == torch.float32 and x_scale.numel() == Mtok and x_scale.is_contiguous()
                                    and x_scale.device == dev):
        _refuse(f"x_scale must be {Mtok} contiguous f32 values", x_scale=x_scale)
    xdt = _DT[X.dtype]
    if out is None:
        hdt = NM_BF16 if hdt is None else hdt
        H, ldh = X.new_empty((Mtok, R), dtype=_TORCH[hdt]), R
    else:
        hdt = dtype_code(out) if hdt is None else hdt
        h = _mat(out)
        if not (h and h[:2] == (Mtok, R) and out.dtype == _TORCH[hdt] and out.device == dev):
            _refuse(f"out must be a row-major {_TORCH[hdt]} tensor of ({Mtok}, {R})", out=out)
        H, ldh = out, h[2]
    G = X.new_empty((Mtok, R), dtype=torch.bfloat16) if save else None
    U = X.new_empty((Mtok, R), dtype=torch.bfloat16) if save else None
    ws = _need(raw.nm_spmm_glu_workspace(Mtok, K, R, Ns, xdt), ws, X)
    stream, back = _enter(X)
    try:
        st = raw.nm_spmm_glu(X.data_ptr(), xdt, Mtok, K, ldx, vals_g.data_ptr(), idx_g.data_ptr(), vals_u.data_ptr(),
                             idx_u.data_ptr(), xdt, R, ldv, ldi, Ns, _ptr(x_scale), g_scale, u_scale, act, H.data_ptr(), hdt,
                             ldh, _ptr(G), _ptr(U), R, _ptr(ws), 0 if ws is None else ws.nbytes, stream)
    finally:
        _leave(back)
    if st:
        _check(st)
    return (H, G, U) if save else H


def _grad_out(t: torch.Tensor | None, want: bool, rows: int, cols: int, dt: int, X: torch.Tensor):
    """(output or None, its leading dimension)."""
    if not want:
        return None, cols
    dtype = _TORCH[dt]
    if t is None:
        return X.new_empty((rows, cols), dtype=dtype), cols
    m = _mat(t)
    if not (m and m[:2] == (rows, cols) and t.dtype == dtype and t.device == X.device):
        _refuse(f"an output must be a row-major {dtype} tensor of {(rows, cols)}", out=t)
    return t, m[2]


def _grad_inputs(X, dY, vals, idx, Ns):
    """(tokens, columns, rows, lifted columns) of a backward call and the leading dimensions of X,
    dY, vals and idx."""
    x, y, v, i, dev, bf16 = _mat(X), _mat(dY), _mat(vals), _mat(idx), X.device, torch.bfloat16
    if not (x and y and v and i and X.dtype == bf16 and dY.dtype == bf16 and vals.dtype == bf16 and
            idx.dtype == torch.int32 and dev == dY.device and dev == vals.device and dev == idx.device):
        _refuse("the backward pass takes row-major bf16 tensors and an int32 idx", X=X, dY=dY, vals=vals, idx=idx)
    (Mtok, K, ldx), (R, slots, ldv), (irows, words, ldi) = x, v, i
    Kl = lifted_width(K, Ns) if Ns >= 2 else K
    if not (y[0] == Mtok and y[1] == R and slots >= Kl // 2 and irows == R and words >= (Kl + 31) // 32):
        _refuse("the shapes do not belong to one sparse layer", X=X, dY=dY, vals=vals, idx=idx)
    return Mtok, K, R, Kl, ldx, y[2], ldv, ldi


def nm_spmm_backward(dY: torch.Tensor, X: torch.Tensor, vals: torch.Tensor, idx: torch.Tensor, Ns: int = 0,
                     want_dx: bool = True, want_dv: bool = True, dxdt: int = NM_BF16, dvdt: int = NM_BF16,
                     out_dx: torch.Tensor | None = None, out_dv: torch.Tensor | None = None, ws: torch.Tensor | None = None):
    """(dX, dvals) of Y = X W^T on a packed bf16 weight; what is not wanted is None."""
    Mtok, K, R, Kl, ldx, ldy, ldv, ldi = _grad_inputs(X, dY, vals, idx, Ns)
    dX, lddx = _grad_out(out_dx, want_dx, Mtok, K, dxdt, X)
    dV, lddv = _grad_out(out_dv, want_dv, R, Kl // 2, dvdt, X)
    ws = _need(raw.nm_spmm_backward_workspace(Mtok, K, R, Ns), ws, X)
    stream, back = _enter(X)
    try:
        st = raw.nm_spmm_backward(dY.data_ptr(), ldy, X.data_ptr(), ldx, Mtok, K, vals.data_ptr(), idx.data_ptr(), R, ldv,
                                  ldi, Ns, _ptr(dX), dxdt, lddx, _ptr(dV), dvdt, lddv, _ptr(ws),
                                  0 if ws is None else ws.nbytes, stream)
    finally:
        _leave(back)
    if st:
        _check(st)
    return dX, dV


def nm_spmm_glu_backward(dH: torch.Tensor, G: torch.Tensor, U: torch.Tensor, X: torch.Tensor, vals_g: torch.Tensor,
                         idx_g: torch.Tensor, vals_u: torch.Tensor, idx_u: torch.Tensor, Ns: int = 0,
                         act: int = NM_ACT_SILU, want_dx: bool = True, want_dv: bool = True, dxdt: int = NM_BF16,
                         dvdt: int = NM_BF16, out_dx: torch.Tensor | None = None,
                         out_dv: tuple[torch.Tensor, torch.Tensor] | None = None, ws: torch.Tensor | None = None):
    """(dX, dvals_g, dvals_u) of nm_spmm_glu from its saved pre-activations; what is not wanted
    is None."""
    Mtok, K, R, Kl, ldx, ldh, ldv, ldi = _grad_inputs(X, dH, vals_g, idx_g, Ns)
    v, i, dev, bf16 = _mat(vals_u), _mat(idx_u), X.device, torch.bfloat16
    if not (v and i and v == (R, vals_g.shape[1], ldv) and i == (R, idx_g.shape[1], ldi) and vals_u.dtype == bf16 and
            idx_u.dtype == torch.int32 and dev == vals_u.device and dev == idx_u.device):
        _refuse("the gate and up weights must be packed alike", vals_g=vals_g, idx_g=idx_g, vals_u=vals_u, idx_u=idx_u)
    m = _mat(G)
    if not (m and m == _mat(U) and m[0] == Mtok and m[1] == R and G.dtype == bf16 and U.dtype == bf16 and
            dev == G.device and dev == U.device):
        _refuse("G and U must be row-major bf16 tensors of dH's shape with the same row stride", dH=dH, G=G, U=U)
    dX, lddx = _grad_out(out_dx, want_dx, Mtok, K, dxdt, X)
    dVg, lddv = _grad_out(out_dv[0] if out_dv else None, want_dv, R, Kl // 2, dvdt, X)
    dVu, lddu = _grad_out(out_dv[1] if out_dv else None, want_dv, R, Kl // 2, dvdt, X)
    if lddu != lddv:
        _refuse("the two weight gradients must have the same row stride", dVg=dVg, dVu=dVu)
    ws = _need(raw.nm_spmm_glu_backward_workspace(Mtok, K, R, Ns), ws, X)
    stream, back = _enter(X)
    try:
        st = raw.nm_spmm_glu_backward(dH.data_ptr(), ldh, G.data_ptr(), U.data_ptr(), m[2], act, X.data_ptr(), ldx, Mtok, K,
                                      vals_g.data_ptr(), idx_g.data_ptr(), vals_u.data_ptr(), idx_u.data_ptr(), R, ldv,
                                      ldi, Ns, _ptr(dX), dxdt, lddx, _ptr(dVg), _ptr(dVu), dvdt, lddv, _ptr(ws),
                                      0 if ws is None else ws.nbytes, stream)
    finally:
        _leave(back)
    if st:
        _check(st)
    return dX, dVg, dVu


def kept_slots(mask: torch.Tensor, K: int, Ns: int = 0) -> torch.Tensor:
    """Which slots of a weight packed 2:4 (or decomposed, Ns >= 3) under mask hold kept weights: bool, the shape of
    vals.  The others are padding, of groups with fewer mask bits than slots, and their gradients are those of
    pruned weights: a training step zeroes them (dvals.masked_fill_(~kept, 0)), or the optimiser brings the weights
    back.  A mask of exactly N of M has none."""
    ones = torch.ones((mask.shape[0], K), dtype=torch.int8, device=mask.device)
    vals, _ = nm_slide_decompose(ones, mask, Ns) if Ns else nm_pack(ones, mask, 2, 4)
    return vals.view(torch.bool)


class _AdamWTensor(ctypes.Structure):
    _fields_ = [("p", _P), ("g", _P), ("m", _P), ("v", _P), ("m_scale", _P), ("v_scale", _P), ("copy", _P), ("n", _I64),
                ("pdt", _I), ("gdt", _I), ("lr_scale", _F), ("weight_decay", _F)]


class AdamWTensors:
    """The tensors of an optimiser, as nm_adamw takes them: lists of contiguous parameters,
    gradients and states (f32, or float8_e4m3fn codes with f32 scales per 256 elements), kept
    for as long as the object lives.  copies: bf16 copies of the parameters, or None; lr_scale
    and weight_decay: one number, or one per tensor.  Build it once and use it every step: it holds
    the tensors' addresses (about 4 us a tensor to build, a launch of many is 6), so gradients go into the same tensors
    every step (out_dv of the backward calls); tensors allocated anew need a new list."""

    def __init__(self, params, grads, m, v, m_scale=None, v_scale=None, copies=None, lr_scale=1.0, weight_decay=0.0):
        n = len(params)
        lists = {"grads": grads, "m": m, "v": v, "m_scale": m_scale, "v_scale": v_scale, "copies": copies}
        for name, t in lists.items():
            if t is not None and len(t) != n:
                raise ValueError(f"{name}: {len(t)} tensors for {n} parameters")
        per = lambda x: [float(x)] * n if isinstance(x, (int, float)) else [float(y) for y in x]  # noqa: E731
        lr_scale, weight_decay = per(lr_scale), per(weight_decay)
        _same("lr_scale and weight_decay", (len(lr_scale), n), (len(weight_decay), n))
        if any(t.device.type != "cuda" for t in params):
            raise ValueError("the tensors of an optimiser step are on a GPU")
        self.keep = [list(params)] + [None if t is None else list(t) for t in lists.values()]
        self.device = params[0].device if n else None
        kinds = {t.dtype for t in [*m, *v]}
        if kinds - {torch.float32} and kinds != {torch.float8_e4m3fn}:
            raise ValueError(f"states must all be float32 or all float8_e4m3fn, got {kinds}")
        self.sdt = NM_FP8 if kinds == {torch.float8_e4m3fn} else NM_F32
        if self.sdt == NM_FP8 and (m_scale is None or v_scale is None):
            raise ValueError("8-bit states need m_scale and v_scale")
        self.count, self.array, self.warned = n, (_AdamWTensor * max(n, 1))(), False
        self.address = ctypes.addressof(self.array)
        f8, spans, read = self.sdt == NM_FP8, [], []      # (first byte, past the last, tensor) of what a step writes, and of the gradients
        for i in range(n):
            p, k, dev = params[i], params[i].numel(), params[i].device
            for name, t in lists.items():
                scale = name.endswith("scale")
                if t is None or (scale and not f8):
                    continue
                want = (k + 255) // 256 if scale else k
                if t[i].numel() != want or not t[i].is_contiguous() or t[i].device != dev:
                    raise ValueError(f"{name}[{i}]: {want} contiguous elements on {dev} expected")
            if not p.is_contiguous() or dev != self.device:
                raise ValueError(f"params[{i}] must be contiguous and on {self.device}")
            if copies is not None and copies[i].dtype != torch.bfloat16:
                raise ValueError("copies are bf16")
            if f8 and (m_scale[i].dtype != torch.float32 or v_scale[i].dtype != torch.float32):
                raise ValueError("scales are float32")
            pdt, gdt = _DT.get(p.dtype), _DT.get(grads[i].dtype)
            if pdt not in (NM_F32, NM_BF16) or gdt not in (NM_F32, NM_BF16):
                raise ValueError(f"params[{i}] and its gradient must be float32 or bfloat16")
            at = (_ptr(p), _ptr(grads[i]), _ptr(m[i]), _ptr(v[i]), _ptr(m_scale[i]) if f8 else None,
                  _ptr(v_scale[i]) if f8 else None, None if copies is None else _ptr(copies[i]))
            self.array[i] = _AdamWTensor(*at, k, pdt, gdt, lr_scale[i], weight_decay[i])
            if k:
                es, ss, blocks = (4, 2)[pdt], 1 if f8 else 4, (k + 255) // 256
                read.append((at[1], at[1] + k * (4, 2)[gdt], i))
                spans += [(a, a + b, i) for a, b in ((at[0], k * es), (at[2], k * ss), (at[3], k * ss), (at[4], 4 * blocks),
                                                     (at[5], 4 * blocks), (at[6], 2 * k)) if a is not None]
        # what a step writes, by address: a tensor listed twice would be updated by two blocks at once, and a
        # gradient inside another tensor's would be read while it is written (inside its own: the call refuses)
        spans.sort()
        if any(a[1] > b[0] for a, b in zip(spans, spans[1:])):
            raise ValueError("the tensors of a step must not overlap")
        starts = [a for a, _, _ in spans]
        for a, b, i in read:
            for k in range(max(bisect.bisect_right(starts, a) - 1, 0), bisect.bisect_left(starts, b)):
                if spans[k][1] > a and spans[k][2] != i:
                    raise ValueError(f"grads[{i}] overlaps what the step writes of tensor {spans[k][2]}")

    def get_device(self) -> int:
        return -1 if self.device is None else self.device.index


def _adamw_ready(tensors: AdamWTensors, grad_scale: torch.Tensor | None) -> bool:
    if grad_scale is not None and (grad_scale.dtype != torch.float32 or grad_scale.numel() != 1):
        raise ValueError("grad_scale must be one f32 value on the device")
    if tensors.count == 0:
        return False
    if grad_scale is not None and grad_scale.device != tensors.device:
        raise ValueError(f"grad_scale must be on {tensors.device}, got {grad_scale.device}")
    return True


def nm_adamw(tensors: AdamWTensors, lr: float, step: int, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
             grad_scale: torch.Tensor | None = None) -> None:
    """One AdamW step over every tensor of the list, in place; step counts from 1.  8-bit states are held
    to the nearest codes, which do not follow gradients that fall (a warning, once a list): train with
    nm_adamw_unbiased."""
    if not _adamw_ready(tensors, grad_scale):
        return
    if tensors.sdt == NM_FP8 and not tensors.warned:
        tensors.warned = True
        warnings.warn("8-bit states held to the nearest codes do not follow gradients that fall: train with nm_adamw_unbiased",
                      stacklevel=3)
    stream, back = _enter(tensors)
    try:
        st = raw.nm_adamw(tensors.address, tensors.count, tensors.sdt, lr, beta1, beta2, eps, step, _ptr(grad_scale), stream)
    finally:
        _leave(back)
    if st:
        _check(st)


def nm_adamw_unbiased(tensors: AdamWTensors, lr: float, step: int, seed: int = 0, beta1: float = 0.9, beta2: float = 0.999,
                      eps: float = 1e-8, grad_scale: torch.Tensor | None = None) -> None:
    """nm_adamw on 8-bit states with unbiased codes, for any beta2.  The codes are a function of seed, step,
    tensor and element."""
    if tensors.sdt != NM_FP8 and tensors.count:
        raise ValueError("unbiased codes are of 8-bit states")
    if not _adamw_ready(tensors, grad_scale):
        return
    stream, back = _enter(tensors)
    try:
        st = raw.nm_adamw_unbiased(tensors.address, tensors.count, lr, beta1, beta2, eps, step, seed & (2 ** 64 - 1),
                                   _ptr(grad_scale), stream)
    finally:
        _leave(back)
    if st:
        _check(st)


# ---------------------------------------------------------------- the current device
def _on_device(fn):
    """fn with its tensors' device current, as _enter makes it (the wrappers that use that are not wrapped)."""
    @functools.wraps(fn)
    def call(*args, **kwargs):
        first = args[0] if args else next((x for x in kwargs.values() if isinstance(x, torch.Tensor)), None)
        try:
            index = first.get_device()
        except AttributeError:      # no tensor: fn says so
            index = -1
        if index < 0 or index == torch._C._cuda_getDevice():
            return fn(*args, **kwargs)
        with torch.cuda.device(index):
            return fn(*args, **kwargs)
    return call


_ENTER = ("nm_spmm_glu", "nm_spmm_backward", "nm_spmm_glu_backward", "nm_adamw", "nm_adamw_unbiased")
for _name in SIGNATURES:
    if not _name.endswith("_workspace") and _name not in ("nm_abi_version", "nm_last_error", *_ENTER):
        globals()[_name] = _on_device(globals()[_name])
