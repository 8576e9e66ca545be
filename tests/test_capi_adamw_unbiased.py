"""Host-side checks of the optimiser step with unbiased 8-bit states (the pointers are never dereferenced)."""
import ctypes
import warnings

import pytest

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def nm():
    import semi_structured_sparsity_amd as m
    return m


def _step(nm, n=300, lr=1e-3, b1=0.9, b2=0.999, eps=1e-8, step=1, seed=7, gs=None, count=1, **kw):
    from semi_structured_sparsity_amd._binding import _AdamWTensor
    t = _AdamWTensor(1 << 32, 2 << 32, 3 << 32, 4 << 32, 5 << 32, 6 << 32, 7 << 32, n, 0, 1, 1.0, 0.0)
    for k, v in kw.items():
        setattr(t, k, v)
    arr = (_AdamWTensor * 1)(t)
    st = nm.raw.nm_adamw_unbiased(ctypes.addressof(arr) if count else None, count, lr, b1, b2, eps, step, seed, gs, None)
    return nm.STATUS_NAMES[st]


def test_refuses(nm):
    assert _step(nm, pdt=2) == "NM_ERR_DTYPE" and _step(nm, gdt=4) == "NM_ERR_DTYPE"
    assert "nm_adamw_unbiased" in nm.last_error()
    assert _step(nm, step=0) == "NM_ERR_SHAPE" and _step(nm, b1=1.0) == "NM_ERR_SHAPE" and _step(nm, b2=-0.1) == "NM_ERR_SHAPE"
    assert _step(nm, eps=-1.0) == "NM_ERR_SHAPE" and _step(nm, lr=float("nan")) == "NM_ERR_SHAPE"
    assert _step(nm, n=-1) == "NM_ERR_SHAPE" and _step(nm, n=1 << 40) == "NM_ERR_SHAPE" and _step(nm, count=-1) == "NM_ERR_SHAPE"
    for k in ("p", "g", "m", "v", "m_scale", "v_scale"):
        assert _step(nm, **{k: None}) == "NM_ERR_NULL", k
    assert _step(nm, v_scale=(6 << 32) + 2) == "NM_ERR_ALIGN" and _step(nm, gs=P((9 << 32) + 2)) == "NM_ERR_ALIGN"
    assert _step(nm, g=1 << 32) == "NM_ERR_ALIAS" and _step(nm, v=(3 << 32) + 299) == "NM_ERR_ALIAS"
    assert _step(nm, gs=P((1 << 32) + 8)) == "NM_ERR_ALIAS"


def test_nothing_to_do(nm):
    assert _step(nm, count=0) == "NM_OK" and _step(nm, n=0, p=None, g=None, m=None, v=None) == "NM_OK"


def test_wrappers_without_tensors(nm):
    """Empty lists do nothing; nothing is said where nothing is held to 8 bits."""
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        none = nm.AdamWTensors([], [], [], [])
        nm.nm_adamw(none, lr=0.1, step=1)
        nm.nm_adamw_unbiased(none, lr=0.1, step=1)
