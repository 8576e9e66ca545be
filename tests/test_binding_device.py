"""Every wrapper makes its tensors' device current for its call: a default stream is 0 on every device, so with
another one current the launch would go there.  Host-only: devices, streams and the library's calls are
stood in for."""
import inspect

import pytest
import torch

import semi_structured_sparsity_amd as nm
from semi_structured_sparsity_amd import _binding as B

CALLS = sorted(n for n in nm.SIGNATURES if not n.endswith("_workspace") and n not in ("nm_last_error", "nm_abi_version"))


@pytest.fixture
def seen(monkeypatch):
    """The current device, where the tensors are, and (device, stream) of the library's calls."""
    state = {"current": 0, "at": 1, "log": []}

    class device:
        def __init__(self, i):
            self.i = i

        def __enter__(self):
            self.before, state["current"] = state["current"], self.i

        def __exit__(self, *a):
            state["current"] = self.before

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: state["current"], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_setDevice", lambda i: state.update(current=i), raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 100 + i, raising=False)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: state["at"])

    def library(name):
        real = getattr(nm.raw, name)

        def call(*args):
            assert len(args) == len(real.argtypes)
            state["log"].append((state["current"], args[-1]))
            return state.get("status", 0)
        return call

    for name in CALLS:
        monkeypatch.setattr(nm.raw, name, library(name))
    return state


def _bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def _list(f8):
    """An optimiser's list, as one on a GPU is."""
    t = nm.AdamWTensors([], [], [], [])
    t.count, t.device, t.sdt, t.warned = 1, torch.device("cuda:1"), nm.NM_FP8 if f8 else nm.NM_F32, True
    return t


X, V, I = _bf16(4, 64), _bf16(8, 32), torch.zeros((8, 4), dtype=torch.int32)
Y, F, M = _bf16(4, 8), torch.zeros((8, 64)), torch.zeros((8, 8), dtype=torch.uint8)
STATS = torch.zeros(2, dtype=torch.float64)
DO = {
    "nm_hdiag_colsumsq": lambda: nm.nm_hdiag_colsumsq(X),
    "nm_hdiag_hutchinson": lambda: nm.nm_hdiag_hutchinson(_bf16(64, 64), 8, 1, 0),
    "nm_hutchinson_score": lambda: nm.nm_hutchinson_score(_bf16(64, 64), _bf16(8, 64), 1, 0, 1e-6),
    "nm_score": lambda: nm.nm_score(W=F, H=None, eps=0.0, mode=nm.NM_SCORE_MAGNITUDE),
    "nm_score_stats": lambda: nm.nm_score_stats(F),
    "nm_gate": lambda: nm.nm_gate(F, STATS, 2, 4, 1.0, 0.5, 2),
    "nm_gate_pack": lambda: nm.nm_gate_pack(F, STATS, _bf16(8, 64), 2, 4, 1.0, 0.5, 2),
    "nm_mask": lambda: nm.nm_mask(F, 2, 4),
    "nm_pack": lambda: nm.nm_pack(F, M, 2, 4, vdt=nm.NM_BF16),
    "nm_prune_pack": lambda: nm.nm_prune_pack(F, None, 0.0, nm.NM_SCORE_MAGNITUDE, 2, 4),
    "nm_slide_decompose": lambda: nm.nm_slide_decompose(_bf16(8, 64), M, 4),
    "nm_prune_slide": lambda: nm.nm_prune_slide(_bf16(8, 64), None, 0.0, nm.NM_SCORE_MAGNITUDE, 4),
    "nm_absmean": lambda: nm.nm_absmean(F),
    "nm_quant_lift": lambda: nm.nm_quant_lift(X),
    "nm_bitmap_encode": lambda: nm.nm_bitmap_encode(_bf16(8, 64), M),
    "nm_spmm_bitmap": lambda: nm.nm_spmm_bitmap(X, _bf16(8, 64), M, torch.zeros((8, 2), dtype=torch.int32)),
    "nm_spmm_lowrank": lambda: nm.nm_spmm_lowrank(X, V, I, _bf16(8, 64), _bf16(8, 8)),
    "nm_spmm": lambda: nm.nm_spmm(X, V, I),
    "nm_spmm_noalloc": lambda: nm.nm_spmm_noalloc(X, vals=V, idx=I),
    "nm_spmm_glu": lambda: nm.nm_spmm_glu(X, V, I, V, I),
    "nm_spmm_backward": lambda: nm.nm_spmm_backward(Y, X=X, vals=V, idx=I),
    "nm_spmm_glu_backward": lambda: nm.nm_spmm_glu_backward(Y, Y, Y, X, V, I, V, I),
    "nm_adamw": lambda: nm.nm_adamw(_list(False), lr=0.1, step=1),
    "nm_adamw_unbiased": lambda: nm.nm_adamw_unbiased(_list(True), lr=0.1, step=1),
}


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("current", [0, 1, 3])
def test_the_tensors_device_is_current_during_a_call(seen, name, current):
    seen["current"] = current
    DO[name]()
    assert seen["log"] == [(1, 101)] and seen["current"] == current      # on their device and its stream, and back


@pytest.mark.parametrize("name", CALLS)
def test_an_error_goes_back_too(seen, name):
    seen["status"] = nm.NM_ERR_SHAPE
    with pytest.raises(nm.NMError):
        DO[name]()
    assert seen["log"] == [(1, 101)] and seen["current"] == 0


def test_a_device_is_not_needed(seen):
    """Lists of nothing do nothing; a call without tensors says what is missing."""
    none = nm.AdamWTensors([], [], [], [])
    assert none.device is None and none.get_device() == -1
    nm.nm_adamw(none, lr=0.1, step=1)
    nm.nm_adamw_unbiased(none, lr=0.1, step=1)
    with pytest.raises(TypeError):
        nm.nm_spmm()
    seen["at"] = -1
    with pytest.raises(ValueError, match="on a GPU"):
        nm.nm_spmm_glu(X, V, I, V, I)
    assert seen["log"] == []


def test_wrappers_keep_their_signatures():
    for name in CALLS:
        first = next(iter(inspect.signature(getattr(nm, name)).parameters.values()))
        assert getattr(nm, name).__name__ == name and first.annotation in ("torch.Tensor", "AdamWTensors")
