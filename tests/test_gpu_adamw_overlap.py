"""A gradient that lies inside what the step writes of another tensor would be read while it is written: the list
of an optimiser's tensors refuses it, wherever it lies and whatever is overlapped (nothing is launched)."""
import pytest
import torch

from tests._util import dev

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


def _list(nm, f8, n=3, size=512, **put):
    z = lambda dt: [torch.zeros(size, device=dev()).to(dt) for _ in range(n)]  # noqa: E731
    sc = lambda: [torch.zeros(2, device=dev()) for _ in range(n)] if f8 else None  # noqa: E731
    t = dict(params=z(torch.float32), grads=z(torch.float32), m=z(F8 if f8 else torch.float32), v=z(F8 if f8 else torch.float32),
             m_scale=sc(), v_scale=sc(), copies=z(torch.bfloat16))
    for name, (i, x) in put.items():
        t[name][i] = x(t) if callable(x) else x
    return nm.AdamWTensors(**t)


@pytest.mark.parametrize("f8", [False, True])
def test_gradients_inside_another_tensors_arrays_are_refused(f8):
    import semi_structured_sparsity_amd as nm
    _list(nm, f8)
    for name in ("params", "m", "v", "copies"):
        for i, j in ((0, 2), (2, 0), (1, 2)):
            if f8 and name in ("m", "v"):
                continue        # states of codes are shorter than any gradient of their size: below
            with pytest.raises(ValueError, match="overlaps"):      # a bf16 gradient over the other tensor's first bytes
                _list(nm, f8, grads=(i, lambda t: t[name][j].view(torch.uint8)[:1024].view(torch.bfloat16)))
    # one buffer: the gradient of tensor 0 reaches one byte into what follows it
    flat = torch.zeros(4 * 512 * 4, dtype=torch.uint8, device=dev())
    g = flat[:2048].view(torch.float32)
    for dt, name in ((F8 if f8 else torch.float32, "m"), (F8 if f8 else torch.float32, "v"), (torch.bfloat16, "copies")):
        es = torch.empty(0, dtype=dt).element_size()
        touch = flat[2048 - es:2048 - es + 512 * es].view(dt)
        with pytest.raises(ValueError, match="overlaps"):
            _list(nm, f8, grads=(0, g), **{name: (1, touch)})
        _list(nm, f8, grads=(0, g), **{name: (1, flat[2048:2048 + 512 * es].view(dt))})
    # gradients may share memory with each other
    t = torch.zeros(512, device=dev())
    z = lambda: torch.zeros(512, device=dev())  # noqa: E731
    nm.nm_adamw(nm.AdamWTensors([z(), z()], [t, t], [z(), z()], [z(), z()]), lr=0.1, step=1)
    # over its own tensor the call refuses it
    p = z()
    with pytest.raises(nm.NMError):
        nm.nm_adamw(nm.AdamWTensors([p], [p], [z()], [z()]), lr=0.1, step=1)
    # empty tensors overlap nothing
    e = torch.zeros(0, device=dev())
    nm.AdamWTensors([e, z()], [e, z()], [e, z()], [e, z()])
