"""Host-side checks of the gated block, the gradients and the optimiser: bad arguments are
refused before anything reaches a GPU (the pointers below are never dereferenced)."""
import ctypes

import pytest

P = ctypes.c_void_p
X, VG, IG, VU, IU, H, G, U, WS, XS = (P((i + 1) << 32) for i in range(10))
BIG = 1 << 40


@pytest.fixture(scope="module")
def nm():
    import semi_structured_sparsity_amd as m
    return m


def _name(nm, st):
    return nm.STATUS_NAMES[st]


def _glu(nm, **kw):
    a = dict(X=X, xdt=1, M=4, K=64, ldx=64, vg=VG, ig=IG, vu=VU, iu=IU, vdt=1, R=8, ldv=32, ldi=4, Ns=0, xs=None, gs=1.0,
             us=1.0, act=0, H=H, hdt=1, ldh=8, G=None, U=None, ldg=8, ws=WS, n=BIG)
    a.update(kw)
    return _name(nm, nm.raw.nm_spmm_glu(*a.values(), None))


def test_glu_refuses(nm):
    assert _glu(nm, act=4) == "NM_ERR_SHAPE" and _glu(nm, act=-1) == "NM_ERR_SHAPE"
    assert _glu(nm, hdt=3) == "NM_ERR_DTYPE" and _glu(nm, xdt=2) == "NM_ERR_DTYPE" and _glu(nm, xdt=2, vdt=2, hdt=3) == "NM_ERR_DTYPE"
    assert _glu(nm, Ns=2) == "NM_ERR_PATTERN" and _glu(nm, Ns=9) == "NM_ERR_PATTERN"
    assert _glu(nm, K=40, ldx=40) == "NM_ERR_SHAPE"           # not a multiple of 16
    assert _glu(nm, M=-1) == "NM_ERR_SHAPE"
    for k in ("ldx", "ldv", "ldi", "ldh"):
        assert _glu(nm, **{k: 1}) == "NM_ERR_SHAPE", k
    for k in ("X", "vg", "ig", "vu", "iu", "H"):
        assert _glu(nm, **{k: None}) == "NM_ERR_NULL", k
    assert _glu(nm, G=G) == "NM_ERR_NULL" and _glu(nm, U=U) == "NM_ERR_NULL"
    assert _glu(nm, G=G, U=U, ldg=7) == "NM_ERR_SHAPE"
    for k, p in (("X", X), ("vg", VG), ("vu", VU)):
        assert _glu(nm, **{k: P(p.value + 8)}) == "NM_ERR_ALIGN", k
    for k, p in (("ig", IG), ("iu", IU)):
        assert _glu(nm, **{k: P(p.value + 2)}) == "NM_ERR_ALIGN", k
    assert _glu(nm, H=P(H.value + 1)) == "NM_ERR_ALIGN" and _glu(nm, G=P(G.value + 1), U=U) == "NM_ERR_ALIGN"
    assert _glu(nm, ws=P(WS.value + 8)) == "NM_ERR_ALIGN"
    assert _glu(nm, ws=None) == "NM_ERR_WORKSPACE" and _glu(nm, n=1) == "NM_ERR_WORKSPACE"
    assert _glu(nm, H=X) == "NM_ERR_ALIAS" and _glu(nm, H=VU) == "NM_ERR_ALIAS" and _glu(nm, G=H, U=U) == "NM_ERR_ALIAS"
    assert _glu(nm, G=G, U=G) == "NM_ERR_ALIAS" and _glu(nm, ws=X) == "NM_ERR_ALIAS" and _glu(nm, ws=H) == "NM_ERR_ALIAS"
    assert _glu(nm, xdt=2, vdt=2, xs=H) == "NM_ERR_ALIAS"
    # int8 sums must stay exact in int32
    assert _glu(nm, xdt=2, vdt=2, K=1 << 20, ldx=1 << 20, ldv=1 << 19, ldi=1 << 15) == "NM_ERR_SHAPE"


def test_glu_nothing_to_do(nm):
    assert _glu(nm, M=0, X=None, H=None) == "NM_OK" and _glu(nm, R=0, H=None) == "NM_OK"
    assert nm.raw.nm_spmm_glu_workspace(0, 64, 8, 0, 1) == 0


def test_glu_workspace_covers_the_plain_form(nm):
    """The query does not know the index pointers, which decide whether the fused kernels run: it
    covers the two products in f32 as well, in passes of bounded size."""
    ws = nm.raw.nm_spmm_glu_workspace
    assert ws(1, 4096, 11008, 0, nm.NM_BF16) >= 2 * 11008 * 4
    assert ws(16384, 4096, 11008, 0, nm.NM_BF16) < 1 << 30
    # the lifted activation, and K splits of a small weight
    assert ws(512, 4096, 14336, 4, nm.NM_FP8) >= 512 * 6144
    assert ws(1, 4096, 64, 0, nm.NM_BF16) >= 2 * 2 * 64 * 4


def _bwd(nm, two=False, **kw):
    a = dict(dY=H, lddy=8)
    if two:
        a.update(G=G, U=U, ldg=8, act=0)
    a.update(X=X, ldx=64, M=4, K=64, vg=VG, ig=IG)
    if two:
        a.update(vu=VU, iu=IU)
    a.update(R=8, ldv=32, ldi=2, Ns=0, dX=P(11 << 32), dxdt=1, lddx=64, dV=P(12 << 32))
    if two:
        a.update(dVu=P(13 << 32))
    a.update(dvdt=1, lddv=32, ws=WS, n=BIG)
    assert set(kw) <= set(a), set(kw) - set(a)
    a.update(kw)
    return _name(nm, (nm.raw.nm_spmm_glu_backward if two else nm.raw.nm_spmm_backward)(*a.values(), None))


@pytest.mark.parametrize("two", [False, True])
def test_backward_refuses(nm, two):
    b = lambda **kw: _bwd(nm, two, **kw)  # noqa: E731
    assert b(K=40) == "NM_ERR_SHAPE" and b(M=-1) == "NM_ERR_SHAPE" and b(M=(1 << 21) + 1) == "NM_ERR_SHAPE"
    assert b(Ns=2) == "NM_ERR_PATTERN" and b(Ns=9) == "NM_ERR_PATTERN" and b(Ns=-1) == "NM_ERR_PATTERN"
    assert b(Ns=5) == "NM_ERR_SHAPE" and b(Ns=4, K=80, ldx=80) == "NM_ERR_SHAPE"      # 64 % 10, 120 % 16
    assert b(Ns=4, ldv=47) in ("NM_ERR_SHAPE", "NM_ERR_ALIGN") and b(Ns=4, lddv=32, ldv=48, ldi=3) == "NM_ERR_ALIGN"
    assert b(dxdt=2) == "NM_ERR_DTYPE" and b(dvdt=4) == "NM_ERR_DTYPE"
    for k in ["dY", "X", "vg", "ig"] + (["G", "U", "vu", "iu"] if two else []):
        assert b(**{k: None}) == "NM_ERR_NULL", k
    for k in ["lddy", "ldx", "ldv", "ldi", "lddx"] + (["ldg"] if two else []):
        assert b(**{k: 1}) in ("NM_ERR_SHAPE", "NM_ERR_ALIGN"), k
    assert b(lddv=31) == "NM_ERR_ALIGN" and b(lddv=33) == "NM_ERR_ALIGN" and b(dV=P((12 << 32) + 8)) == "NM_ERR_ALIGN"
    assert b(X=P(X.value + 8)) == "NM_ERR_ALIGN" and b(ldx=68) == "NM_ERR_ALIGN" and b(vg=P(VG.value + 8)) == "NM_ERR_ALIGN"
    assert b(dY=P(H.value + 1)) == "NM_ERR_ALIGN" and b(ig=P(IG.value + 2)) == "NM_ERR_ALIGN"
    assert b(ws=None) == "NM_ERR_WORKSPACE" and b(n=16) == "NM_ERR_WORKSPACE" and b(ws=P(WS.value + 8)) == "NM_ERR_ALIGN"
    assert b(dX=X) == "NM_ERR_ALIAS" and b(dX=H) == "NM_ERR_ALIAS" and b(dV=VG) == "NM_ERR_ALIAS"
    assert b(dV=P(11 << 32)) == "NM_ERR_ALIAS" and b(ws=X) == "NM_ERR_ALIAS" and b(ws=P(11 << 32)) == "NM_ERR_ALIAS"
    if two:
        assert b(act=9) == "NM_ERR_SHAPE"
        assert b(dVu=None) == "NM_ERR_NULL" and b(dVu=P(12 << 32)) == "NM_ERR_ALIAS"


@pytest.mark.parametrize("two", [False, True])
def test_backward_nothing_to_do(nm, two):
    none = dict(dX=None, dV=None, **({"dVu": None} if two else {}))
    assert _bwd(nm, two, **none) == "NM_OK"
    assert _bwd(nm, two, K=0) == "NM_OK"


def test_backward_workspace(nm):
    one, two = nm.raw.nm_spmm_backward_workspace, nm.raw.nm_spmm_glu_backward_workspace
    assert one(0, 64, 8, 0) == 0 and two(4, 64, 0, 0) == 0
    # the transposed operands and the dense transposed weights of many tokens
    M, K, R = 2048, 4096, 11008
    assert two(M, K, R, 0) >= 2 * (2 * M * R * 2) + K * M * 2 + K * 2 * R * 2
    # a lifted dX is folded from f32
    assert two(M, K, R, 4) >= M * K * 3 // 2 * 4 and two(M, K, R, 2) == 0
    # few tokens stream the packed weight: no dense copy of it
    assert two(8, K, R, 0) < K * 2 * R * 2


def _adamw(nm, n=300, sdt=0, lr=1e-3, b1=0.9, b2=0.999, eps=1e-8, step=1, gs=None, count=1, **kw):
    from semi_structured_sparsity_amd._binding import _AdamWTensor
    t = _AdamWTensor(1 << 32, 2 << 32, 3 << 32, 4 << 32, 5 << 32, 6 << 32, 7 << 32, n, 0, 1, 1.0, 0.0)
    for k, v in kw.items():
        setattr(t, k, v)
    arr = (_AdamWTensor * 1)(t)
    return _name(nm, nm.raw.nm_adamw(ctypes.addressof(arr) if count else None, count, sdt, lr, b1, b2, eps, step, gs, None))


def test_adamw_refuses(nm):
    assert _adamw(nm, sdt=1) == "NM_ERR_DTYPE" and _adamw(nm, pdt=2) == "NM_ERR_DTYPE" and _adamw(nm, gdt=4) == "NM_ERR_DTYPE"
    assert _adamw(nm, step=0) == "NM_ERR_SHAPE" and _adamw(nm, b1=1.0) == "NM_ERR_SHAPE" and _adamw(nm, b2=-0.1) == "NM_ERR_SHAPE"
    assert _adamw(nm, eps=-1.0) == "NM_ERR_SHAPE" and _adamw(nm, lr=float("nan")) == "NM_ERR_SHAPE"
    assert _adamw(nm, n=-1) == "NM_ERR_SHAPE" and _adamw(nm, count=-1) == "NM_ERR_SHAPE"
    for k in ("p", "g", "m", "v"):
        assert _adamw(nm, **{k: None}) == "NM_ERR_NULL", k
    for k in ("m_scale", "v_scale"):
        assert _adamw(nm, sdt=4, **{k: None}) == "NM_ERR_NULL", k
    assert _adamw(nm, p=(1 << 32) + 2) == "NM_ERR_ALIGN" and _adamw(nm, m=(3 << 32) + 2) == "NM_ERR_ALIGN"
    assert _adamw(nm, copy=(7 << 32) + 1) == "NM_ERR_ALIGN" and _adamw(nm, sdt=4, v_scale=(6 << 32) + 2) == "NM_ERR_ALIGN"
    assert _adamw(nm, gs=P((9 << 32) + 2)) == "NM_ERR_ALIGN"
    assert _adamw(nm, g=1 << 32) == "NM_ERR_ALIAS" and _adamw(nm, v=(3 << 32) + 4 * 299) == "NM_ERR_ALIAS"
    assert _adamw(nm, copy=2 << 32) == "NM_ERR_ALIAS" and _adamw(nm, sdt=4, m_scale=6 << 32) == "NM_ERR_ALIAS"
    assert _adamw(nm, gs=P((1 << 32) + 8)) == "NM_ERR_ALIAS"


def test_adamw_nothing_to_do(nm):
    assert _adamw(nm, count=0) == "NM_OK" and _adamw(nm, n=0, p=None, g=None, m=None, v=None) == "NM_OK"


def test_descriptor_layout_matches_the_header(nm):
    """The struct of the header: seven pointers, a 64-bit count, two enums, two floats."""
    from semi_structured_sparsity_amd._binding import _AdamWTensor
    assert ctypes.sizeof(_AdamWTensor) == 7 * 8 + 8 + 2 * 4 + 2 * 4
    assert _AdamWTensor.n.offset == 56 and _AdamWTensor.pdt.offset == 64 and _AdamWTensor.weight_decay.offset == 76
