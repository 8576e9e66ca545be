"""Host-side checks of nmsparse_layers.h: the header's functions are exported and bound, bad arguments are
refused before anything reaches a GPU (the pointers below are never dereferenced), and every wrapper
makes its tensors' device current."""
import ctypes
import re
from pathlib import Path

import pytest
import torch

import semi_structured_sparsity_amd as nm

P = ctypes.c_void_p
X, C, I, S, C2, I2, S2, Y, V = (P((i + 1) << 32) for i in range(9))
HEADER = Path(__file__).resolve().parents[1] / "include" / "nmsparse_layers.h"


def _name(st):
    return nm.STATUS_NAMES[st]


def test_header_library_and_binding_agree():
    text = re.sub(r"/\*.*?\*/", "", HEADER.read_text(), flags=re.S)
    declared = set(re.findall(r"\b(nm_[a-z0-9_]+)\s*\(", text))
    assert declared == set(nm.LAYER_SIGNATURES)
    for s in declared:
        assert hasattr(nm.raw, s) and (s.endswith("_workspace") or callable(getattr(nm, s)))
    assert not declared & set(nm.SIGNATURES)


# ------------------------------------------------------------------ 4-bit weights
def _quant(**kw):
    a = dict(vals=X, vdt=1, R=8, slots=64, ldv=64, qdt=5, group=64, codes=C, ldc=32, scales=S, lds=8, values=V, ldo=64)
    a.update(kw)
    return _name(nm.raw.nm_quant_w4(*a.values(), None))


def test_quant_refuses():
    assert _quant(vdt=2) == "NM_ERR_DTYPE" and _quant(qdt=4) == "NM_ERR_DTYPE" and _quant(qdt=7) == "NM_ERR_DTYPE"
    for g in (0, 32, 96, 512, -64):
        assert _quant(group=g) == "NM_ERR_SHAPE"
    assert _quant(slots=60) == "NM_ERR_SHAPE" and _quant(R=-1) == "NM_ERR_SHAPE" and _quant(slots=-8) == "NM_ERR_SHAPE"
    assert _quant(R=1 << 25) == "NM_ERR_SHAPE" and _quant(slots=1 << 25) == "NM_ERR_SHAPE"
    for k, v in (("ldv", 56), ("ldc", 28), ("lds", 7), ("ldo", 56)):
        assert _quant(**{k: v}) == "NM_ERR_SHAPE", k
    for k in ("vals", "codes", "scales"):
        assert _quant(**{k: None}) == "NM_ERR_NULL", k
    for k, p, off in (("vals", X, 8), ("codes", C, 2), ("scales", S, 1), ("values", V, 8)):
        assert _quant(**{k: P(p.value + off)}) == "NM_ERR_ALIGN", k
    for k, v in (("ldv", 68), ("ldc", 34), ("ldo", 68)):
        assert _quant(**{k: v}) == "NM_ERR_ALIGN", k
    for k in ("codes", "scales", "values"):
        assert _quant(**{k: X}) == "NM_ERR_ALIAS", k
    assert _quant(codes=S) == "NM_ERR_ALIAS" and _quant(values=C) == "NM_ERR_ALIAS"
    assert _quant(R=0, vals=None) == "NM_OK" and _quant(slots=0, vals=None) == "NM_OK"


def _w4(two=False, **kw):
    a = dict(X=X, M=4, K=64, ldx=64, c=C)
    if two:
        a.update(i=I, s=S, c2=C2, i2=I2, s2=S2, qdt=5)
    else:
        a.update(qdt=5, i=I, s=S)
    a.update(R=8, ldc=16, ldi=2, lds=8, group=64, Ns=0)
    if two:
        a.update(act=0)
    a.update(Y=Y, ydt=1, ldy=8, ws=V, n=1 << 40)
    a.update(kw)
    return _name((nm.raw.nm_spmm_glu_w4 if two else nm.raw.nm_spmm_w4)(*a.values(), None))


@pytest.mark.parametrize("two", [False, True])
def test_products_refuse(two):
    f = lambda **kw: _w4(two, **kw)  # noqa: E731
    assert f(qdt=1) == "NM_ERR_DTYPE" and f(ydt=2) == "NM_ERR_DTYPE" and f(ydt=5) == "NM_ERR_DTYPE"
    assert f(group=32) == "NM_ERR_SHAPE" and f(group=0) == "NM_ERR_SHAPE"
    assert f(Ns=2) == "NM_ERR_PATTERN" and f(Ns=9) == "NM_ERR_PATTERN" and f(Ns=-1) == "NM_ERR_PATTERN"
    assert f(K=40) == "NM_ERR_SHAPE" and f(K=60, Ns=4) == "NM_ERR_SHAPE" and f(K=24, Ns=4) == "NM_ERR_SHAPE"
    assert f(M=-1) == "NM_ERR_SHAPE" and f(K=-16) == "NM_ERR_SHAPE" and f(R=-1) == "NM_ERR_SHAPE" and f(K=0) == "NM_ERR_SHAPE"
    assert f(M=(1 << 20) + 1) == "NM_ERR_SHAPE" and f(R=(1 << 24) + 1) == "NM_ERR_SHAPE"
    for k, v in (("ldx", 56), ("ldc", 0), ("ldi", 1), ("lds", 4), ("ldy", 7), ("ldc", 1 << 26), ("ldi", 1 << 24)):
        assert f(**{k: v}) == "NM_ERR_SHAPE", k
    for k, v in (("ldx", 68), ("ldc", 24), ("lds", 10)):
        assert f(**{k: v}) == "NM_ERR_ALIGN", k
    ptrs = [("X", X, 8), ("c", C, 8), ("i", I, 2), ("s", S, 4), ("Y", Y, 1)]
    if two:
        ptrs += [("c2", C2, 8), ("i2", I2, 2), ("s2", S2, 4)]
        assert f(act=4) == "NM_ERR_SHAPE" and f(act=-1) == "NM_ERR_SHAPE"
    for k, p, off in ptrs:
        assert f(**{k: None}) == "NM_ERR_NULL", k
        assert f(**{k: P(p.value + off)}) == "NM_ERR_ALIGN", k
        if k != "Y":
            assert f(Y=p) == "NM_ERR_ALIAS", k
    assert f(M=0, X=None, Y=None) == "NM_OK" and f(R=0, Y=None) == "NM_OK"


@pytest.mark.parametrize("two", [False, True])
def test_products_that_need_a_workspace(two):
    big = dict(M=33, K=8192, ldx=8192, R=64, ldc=2048, ldi=256, lds=64, ldy=64)
    f = lambda **kw: _w4(two, **{**big, **kw})  # noqa: E731
    query = nm.raw.nm_spmm_glu_w4_workspace if two else nm.raw.nm_spmm_w4_workspace
    need = query(33, 8192, 64, 0)
    assert need >= 2 * (1 + two) * 33 * 64 * 4
    assert f(ws=None) == "NM_ERR_WORKSPACE" and f(n=need - 1) == "NM_ERR_WORKSPACE" and f(ws=P(V.value + 8)) == "NM_ERR_ALIGN"
    for p in (X, C, I, S, Y) + ((C2, I2, S2) if two else ()):
        assert f(ws=p) == "NM_ERR_ALIAS"
    assert query(16, 8192, 64, 0) == 0 and query(33, 256, 64, 0) == 0
    for bad in ((0, 8192, 64, 0), (33, 8200, 64, 0), (33, 8192, 0, 0), (33, 8192, 64, 2), (33, 8192, 64, 9), (33, 8192, 64, 3), (33, 1 << 40, 64, 0),
                ((1 << 20) + 1, 8192, 64, 0), (33, 8192, -4, 0)):
        assert query(*bad) == 0, bad


# ------------------------------------------------------------------ mixture of sparse blocks
def _experts(base, rows, slots, words, groups, **kw):
    e = nm._layers._Experts(base, base + (1 << 20), base + (2 << 20), slots, words, rows, rows * slots, rows * words, rows * groups)
    for k, v in kw.items():
        setattr(e, k, v)
    return e


def _moe(w=None, **kw):
    """w: (which weight, field, value)"""
    es = [_experts((20 + i) << 32, 32 if i < 2 else 64, 16, 2, 1) for i in range(3)]
    if w:
        setattr(es[w[0]], w[1], w[2])
    a = dict(X=X, M=4, K=64, ldx=64, router=C, ldr=64, bias=None, E=4, topk=2, route=0, renorm=1, scale=1.0, gate=0, up=1, down=2,
             vdt=5, group=64, F=32, Ns=0, act=0, Y=Y, ydt=1, ldy=64, sel=I, wts=S, ws=V, n=1 << 40)
    a.update(kw)
    for k in ("gate", "up", "down"):
        a[k] = ctypes.byref(es[a[k]]) if a[k] is not None else None
    return _name(nm.raw.nm_moe(*a.values(), None))


def test_moe_refuses():
    assert _moe(M=65) == "NM_ERR_SHAPE" and _moe(M=-1) == "NM_ERR_SHAPE" and _moe(K=-16) == "NM_ERR_SHAPE"
    assert _moe(topk=0) == "NM_ERR_SHAPE" and _moe(topk=5) == "NM_ERR_SHAPE" and _moe(E=32, topk=17) == "NM_ERR_SHAPE"
    assert _moe(E=0) == "NM_ERR_SHAPE" and _moe(E=513) == "NM_ERR_SHAPE"
    assert _moe(route=2) == "NM_ERR_SHAPE" and _moe(act=4) == "NM_ERR_SHAPE" and _moe(group=96) == "NM_ERR_SHAPE"
    assert _moe(vdt=2) == "NM_ERR_DTYPE" and _moe(ydt=2) == "NM_ERR_DTYPE"
    assert _moe(Ns=2) == "NM_ERR_PATTERN" and _moe(Ns=9) == "NM_ERR_PATTERN"
    assert _moe(K=40) == "NM_ERR_SHAPE" and _moe(F=40) == "NM_ERR_SHAPE" and _moe(F=0) == "NM_ERR_SHAPE" and _moe(Ns=3) == "NM_ERR_SHAPE"
    assert _moe(K=0) == "NM_ERR_SHAPE" and _moe(M=0, K=0, X=None) == "NM_OK"      # no columns to pick experts by
    for k in ("ldx", "ldr", "ldy"):
        assert _moe(**{k: 56}) == "NM_ERR_SHAPE", k
    for k in ("X", "router", "gate", "up", "down", "Y"):
        assert _moe(**{k: None}) == "NM_ERR_NULL", k
    for k, p, off in (("X", X, 8), ("router", C, 8), ("Y", Y, 1), ("sel", I, 2), ("wts", S, 2), ("ws", V, 8), ("bias", C2, 2)):
        assert _moe(**{k: P(p.value + off)}) == "NM_ERR_ALIGN", k
    assert _moe(ldx=68) == "NM_ERR_ALIGN" and _moe(ldr=68) == "NM_ERR_ALIGN"
    assert _moe(ws=None) == "NM_ERR_WORKSPACE" and _moe(n=16) == "NM_ERR_WORKSPACE"
    for w in range(3):
        for f, v in (("vals", None), ("idx", None), ("scales", None)):
            assert _moe(w=(w, f, v)) == "NM_ERR_NULL", (w, f)
        for f, v in (("ld_vals", 0), ("ld_idx", 0), ("ld_scales", 28), ("es_vals", -16), ("es_idx", -1), ("es_scales", -4),
                     ("ld_vals", 1 << 26), ("ld_idx", 1 << 24)):
            assert _moe(w=(w, f, v)) == "NM_ERR_SHAPE", (w, f)
        for f, v in (("vals", (30 << 32) + 8), ("idx", (30 << 32) + 2), ("scales", (30 << 32) + 4), ("ld_vals", 24), ("es_vals", 8),
                     ("ld_scales", 66), ("es_scales", 66)):
            assert _moe(w=(w, f, v)) == "NM_ERR_ALIGN", (w, f)
        assert _moe(Y=P(((20 + w) << 32) + 3 * 16)) == "NM_ERR_ALIAS" and _moe(ws=P((20 + w) << 32)) == "NM_ERR_ALIAS"
    assert _moe(Y=X) == "NM_ERR_ALIAS" and _moe(sel=S) == "NM_ERR_ALIAS" and _moe(ws=C) == "NM_ERR_ALIAS" and _moe(wts=Y) == "NM_ERR_ALIAS"
    assert _moe(M=0, X=None, Y=None, gate=None) == "NM_OK"


def test_moe_workspace_of_refused_sizes():
    ws = nm.raw.nm_moe_workspace
    assert ws(4, 64, 32, 4, 2) > 0
    for bad in ((0, 64, 32, 4, 2), (65, 64, 32, 4, 2), (4, 0, 32, 4, 2), (4, 64, -1, 4, 2), (4, 64, 32, 0, 1), (4, 64, 32, 513, 2),
                (4, 64, 32, 4, 5), (4, 64, 32, 64, 17), (4, 64, 32, 4, 0), (4, 1 << 40, 32, 4, 2), (-3, 64, 32, 4, 2)):
        assert ws(*bad) == 0, bad


# ------------------------------------------------------------------ norms around a block
Q = [P((40 + i) << 32) for i in range(14)]


def _norm(**kw):
    a = dict(X=X, xdt=1, M=4, C=64, ldx=64, res=1.0, Y=Y, ldy=64, gate=Q[0], ldg=64, rows=2, post=1, wp=Q[1], bp=Q[2], pre=2, wn=Q[3],
             bn=Q[4], wdt=1, eps=1e-6, Z=Q[5], ldz=64, N=Q[6], ndt=1, Ns=0, ldn=96, s=Q[7])
    a.update(kw)
    return _name(nm.raw.nm_block_norm(*a.values(), None))


def test_norm_refuses():
    assert _norm(M=-1) == "NM_ERR_SHAPE" and _norm(C=-1) == "NM_ERR_SHAPE" and _norm(C=0) == "NM_ERR_SHAPE"
    assert _norm(C=32769, ldx=1 << 17) == "NM_ERR_SHAPE" and _norm(M=1 << 25) == "NM_ERR_SHAPE"
    assert _norm(xdt=2) == "NM_ERR_DTYPE" and _norm(wdt=3) == "NM_ERR_DTYPE" and _norm(ndt=3) == "NM_ERR_DTYPE" and _norm(ndt=5) == "NM_ERR_DTYPE"
    assert _norm(post=3) == "NM_ERR_SHAPE" and _norm(pre=-1) == "NM_ERR_SHAPE" and _norm(post=0) == "NM_ERR_SHAPE"
    assert _norm(post=0, wp=None) == "NM_ERR_SHAPE" and _norm(pre=0) == "NM_ERR_SHAPE"
    assert _norm(pre=0, wn=None, bn=None) == "NM_ERR_NULL" and _norm(N=None) == "NM_ERR_NULL"
    assert _norm(Y=None) == "NM_ERR_NULL" and _norm(X=None) == "NM_ERR_NULL" and _norm(ndt=2, s=None) == "NM_ERR_NULL"
    assert _norm(rows=-1) == "NM_ERR_SHAPE" and _norm(eps=-1.0) == "NM_ERR_SHAPE" and _norm(eps=float("nan")) == "NM_ERR_SHAPE"
    assert _norm(Ns=4) == "NM_ERR_PATTERN" and _norm(Ns=2, ndt=4) == "NM_ERR_PATTERN" and _norm(Ns=9, ndt=4) == "NM_ERR_PATTERN"
    assert _norm(Ns=3, ndt=4) == "NM_ERR_SHAPE" and _norm(C=60, ndt=2) == "NM_ERR_SHAPE"
    for k in ("ldx", "ldy", "ldg", "ldz", "ldn"):
        assert _norm(**{k: 63}) == "NM_ERR_SHAPE", k
    assert _norm(Ns=4, ndt=4, ldn=92) == "NM_ERR_SHAPE"
    for k, p in (("X", X), ("Y", Y), ("gate", Q[0]), ("wp", Q[1]), ("bp", Q[2]), ("wn", Q[3]), ("bn", Q[4]), ("Z", Q[5]), ("N", Q[6])):
        assert _norm(**{k: P(p.value + 1)}) == "NM_ERR_ALIGN", k
        if k != "N":
            assert _norm(ndt=4, **{k: P(p.value + 8)}) == "NM_ERR_ALIGN", k
    assert _norm(ndt=4, N=P(Q[6].value + 2)) == "NM_ERR_ALIGN" and _norm(ndt=4, ldn=98) == "NM_ERR_ALIGN" and _norm(ndt=4, ldx=68) == "NM_ERR_ALIGN"
    for k in ("Z", "N"):
        for p in (Y, *Q[:5]):
            assert _norm(**{k: p}) == "NM_ERR_ALIAS", k
    assert _norm(N=X) == "NM_ERR_ALIAS" and _norm(Z=Q[6]) == "NM_ERR_ALIAS" and _norm(Z=X, ldz=72) == "NM_ERR_ALIAS"
    assert _norm(Z=P(X.value + 128)) == "NM_ERR_ALIAS" and _norm(ndt=2, s=Q[6]) == "NM_ERR_ALIAS"
    assert _norm(M=0, X=None) == "NM_OK"


def _norm_bwd(**kw):
    a = dict(Z=X, xdt=1, M=4, C=64, ldz=64, dZ=C, lddz=64, dN=I, dndt=1, lddn=64, res=1.0, Y=Y, ldy=64, gate=Q[0], ldg=64, rows=2, post=1,
             wp=Q[1], bp=Q[2], pre=2, wn=Q[3], wdt=1, eps=1e-6, dX=Q[4], lddx=64, dY=Q[5], lddy=64, dwn=Q[6], dbn=Q[7], dwp=Q[8],
             dbp=Q[9], dgate=Q[10], ws=Q[11], n=1 << 31)
    a.update(kw)
    return _name(nm.raw.nm_block_norm_backward(*a.values(), None))


def test_norm_backward_refuses():
    f = _norm_bwd
    assert f(M=-1) == "NM_ERR_SHAPE" and f(C=0) == "NM_ERR_SHAPE" and f(C=32769) == "NM_ERR_SHAPE" and f(pre=4) == "NM_ERR_SHAPE"
    assert f(xdt=2) == "NM_ERR_DTYPE" and f(wdt=2) == "NM_ERR_DTYPE" and f(dndt=4) == "NM_ERR_DTYPE"
    assert f(pre=0, wn=None) == "NM_ERR_NULL" and f(dN=None) == "NM_ERR_NULL" and f(Z=None) == "NM_ERR_NULL"
    assert f(post=0, wp=None, bp=None) == "NM_ERR_NULL" and f(Y=None) == "NM_ERR_NULL" and f(gate=None) == "NM_ERR_NULL"
    assert f(Y=None, gate=None, post=0, wp=None, bp=None, dwp=None, dbp=None, dgate=None) == "NM_ERR_NULL"      # dY is left
    for k in ("ldz", "lddz", "lddn", "ldy", "ldg", "lddx", "lddy"):
        assert f(**{k: 63}) == "NM_ERR_SHAPE", k
    for k in ("Z", "dZ", "dN", "Y", "gate", "wp", "dX", "dY", "dwn", "dgate"):
        v = dict(Z=X, dZ=C, dN=I, Y=Y, gate=Q[0], wp=Q[1], dX=Q[4], dY=Q[5], dwn=Q[6], dgate=Q[10])[k]
        assert f(**{k: P(v.value + 1)}) == "NM_ERR_ALIGN", k
    assert f(ws=P(Q[11].value + 8)) == "NM_ERR_ALIGN" and f(ws=None) == "NM_ERR_WORKSPACE" and f(n=8) == "NM_ERR_WORKSPACE"
    for k in ("dX", "dY", "dwn", "dbn", "dwp", "dbp", "dgate", "ws"):
        for p in (X, I, Y, Q[0], Q[1], Q[3]):
            assert f(**{k: p}) == "NM_ERR_ALIAS", k
        if k != "dX":
            assert f(**{k: C}) == "NM_ERR_ALIAS" and f(**{k: Q[4]}) == "NM_ERR_ALIAS", k
    assert f(dX=C, lddx=72) == "NM_ERR_ALIAS"


def test_norm_workspace_of_refused_sizes():
    ws = nm.raw.nm_block_norm_backward_workspace
    assert ws(4, 64, 0) > 0 and ws(4096, 4096, 1) > 0
    assert all(ws(*a) == 0 for a in ((0, 64, 0), (-1, 64, 0), (4, 0, 0), (4, 32769, 0), (1 << 25, 64, 0), (4, 64, -1)))


# ------------------------------------------------------------------ the current device
@pytest.fixture
def seen(monkeypatch):
    """The current device, where the tensors are, and (device, stream) of the library's calls; devices are
    stood in for."""
    state = {"current": 0, "log": [], "status": 0}
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: state["current"], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_setDevice", lambda i: state.update(current=i), raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 100 + i, raising=False)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 1)
    for name in CALLS:
        def call(*args, n=len(nm.LAYER_SIGNATURES[name][1])):
            assert len(args) == n
            state["log"].append((state["current"], args[-1]))
            return state["status"]
        monkeypatch.setattr(nm.raw, name, call)
    return state


def _bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def _u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


def _layer():
    """A layer's handle, as one on a GPU is."""
    t = nm.MoELayer.__new__(nm.MoELayer)
    t.experts, t.K, t.ldr, t.hidden, t.vdt, t.group, t.Ns, t.device = 4, 64, 64, 32, 1, 64, 0, torch.device("cpu")
    t.router, t.bias, t.address = _bf16(4, 64), None, [0, 0, 0]
    return t


_CODES, _IDX, _SC = _u8(8, 16), torch.zeros((8, 2), dtype=torch.int32), _bf16(1, 8)
DO = {
    "nm_quant_w4": lambda: nm.nm_quant_w4(_bf16(8, 64)),
    "nm_spmm_w4": lambda: nm.nm_spmm_w4(_bf16(2, 64), _CODES, _IDX, _SC),
    "nm_spmm_glu_w4": lambda: nm.nm_spmm_glu_w4(_bf16(2, 64), _CODES, _IDX, _SC, _CODES, _IDX, _SC),
    "nm_moe": lambda: nm.nm_moe(_layer(), _bf16(2, 64), 2),
    "nm_block_norm": lambda: nm.nm_block_norm(_bf16(2, 64)),
    "nm_block_norm_backward": lambda: nm.nm_block_norm_backward(_bf16(2, 64), dN=_bf16(2, 64), w_pre=_bf16(64)),
}
CALLS = sorted(DO)


def test_every_call_is_tested():
    assert set(CALLS) == {n for n in nm.LAYER_SIGNATURES if not n.endswith("_workspace")}


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("current", [0, 1, 3])
def test_the_tensors_device_is_current_during_a_call(seen, name, current):
    seen["current"] = current
    DO[name]()
    assert seen["log"] == [(1, 101)] and seen["current"] == current


@pytest.mark.parametrize("name", CALLS)
def test_an_error_goes_back_too(seen, name):
    seen["status"] = nm.NM_ERR_SHAPE
    with pytest.raises(nm.NMError):
        DO[name]()
    assert seen["log"] == [(1, 101)] and seen["current"] == 0
