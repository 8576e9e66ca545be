"""Every wrapper makes its tensors' device current for its call: a default stream is 0 on every device, so with
another one current the launch would go there.  Host-only: devices are stood in for."""
import inspect

import pytest
import torch

import semi_structured_sparsity_amd as nm
from semi_structured_sparsity_amd import _binding as B

WRAPPERS = sorted(n for n in nm.SIGNATURES if not n.endswith("_workspace") and n not in ("nm_last_error", "nm_abi_version"))


class Tensor(nm.AdamWTensors):
    """What a wrapper's first argument has."""

    def __init__(self, device):
        self.device = torch.device(device)

    def get_device(self):
        return -1 if self.device.type == "cpu" else self.device.index


@pytest.fixture
def seen(monkeypatch):
    """[current device], and the devices made current meanwhile."""
    state = {"current": 0, "log": []}

    class device:
        def __init__(self, i):
            self.i = i

        def __enter__(self):
            self.before, state["current"] = state["current"], self.i

        def __exit__(self, *a):
            state["current"] = self.before

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: state["current"], raising=False)
    monkeypatch.setattr(torch.cuda, "device", device)
    return state


def test_the_tensors_device_is_current_during_a_call(seen):
    call = B._on_device(lambda x, y=1, fail=False: seen["log"].append((seen["current"], y)) or (1 / 0 if fail else y))
    assert call(Tensor("cuda:0"), y=2) == 2 and call(Tensor("cuda:1"), 3) == 3 and call(x=Tensor("cuda:3"), y=4) == 4
    assert call(Tensor("cpu")) == 1 and call(y=5, x=Tensor("cuda:2")) == 5 and call(None) == 1
    assert seen["log"] == [(0, 2), (1, 3), (3, 4), (0, 1), (2, 5), (0, 1)] and seen["current"] == 0
    with pytest.raises(ZeroDivisionError):
        call(Tensor("cuda:2"), fail=True)
    assert seen["log"][-1] == (2, 1) and seen["current"] == 0
    seen["current"] = 1
    call(Tensor("cuda:0"))
    assert seen["log"][-1][0] == 0 and seen["current"] == 1


def test_lists_without_a_device_pass(seen):
    none = nm.AdamWTensors([], [], [], [])
    assert none.device is None and none.get_device() == -1
    nm.nm_adamw(none, lr=0.1, step=1)


@pytest.mark.parametrize("name", WRAPPERS)
def test_every_wrapper_does(name):
    fn = getattr(nm, name)
    assert getattr(fn, "__wrapped__", None) is not None and fn is getattr(B, name) and fn.__name__ == name
    first = next(iter(inspect.signature(fn).parameters.values()))
    assert first.annotation in ("torch.Tensor", "AdamWTensors"), "the first argument says which device"
