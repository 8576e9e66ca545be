"""The example that trains a pruned block: the forward pass, both backward passes and the
optimiser step together, against the same training of the masked dense block by automatic
differentiation in f32."""
import importlib.util
from pathlib import Path

import pytest
import torch

pytestmark = pytest.mark.gpu


def _reference(width, hidden, tokens, steps, lr, seed, Ns):
    """Masked dense weights, f32 throughout, on the example's random numbers."""
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g, device=dev)  # noqa: E731
    dense = {"g": rand(hidden, width) * width ** -0.5, "u": rand(hidden, width) * width ** -0.5,
             "d": rand(width, hidden) * hidden ** -0.5}
    mask, param = {}, {}
    for k, w in dense.items():
        a = w.view(w.shape[0], -1, 2 * Ns if Ns else 4).abs()
        mask[k] = torch.zeros_like(a).scatter_(-1, a.topk(2 * Ns - 2 if Ns else 2, -1).indices, 1.0).view_as(w)
        param[k] = (w * mask[k]).to(torch.bfloat16).float().requires_grad_()
    opt = torch.optim.AdamW(list(param.values()), lr=lr, betas=(0.9, 0.999), weight_decay=0.0)
    mix = rand(width // 8, width) * (width // 8) ** -0.5

    def block(x, w):
        return (torch.nn.functional.silu(x @ w["g"].t()) * (x @ w["u"].t())) @ w["d"].t()

    def batch():
        x = (rand(tokens, width // 8) @ mix).to(torch.bfloat16).float()
        return x, block(x, dense)

    def loss(x, want):
        return (block(x, {k: param[k] * mask[k] for k in param}) - want).square().mean()

    held = batch()
    before = loss(*held).item()
    for step in range(1, steps + 1):
        data = batch()
        opt.zero_grad()
        loss(*data).backward()
        for group in opt.param_groups:
            group["lr"] = lr * min(1.0, step / 10)
        opt.step()
    return before, loss(*held).item()


@pytest.mark.parametrize("Ns", [0, 4])
def test_training_follows_the_masked_dense_block(Ns):
    path = Path(__file__).resolve().parents[1] / "examples" / "train_pruned_block.py"
    spec = importlib.util.spec_from_file_location("train_pruned_block", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    size = dict(width=256, hidden=704, tokens=256, steps=40, lr=5e-4, seed=3, Ns=Ns)
    before, after, one, many = example.train(**size)
    ref_before, ref_after = _reference(**size)
    assert abs(before - ref_before) < 0.02 * ref_before
    assert after < 0.6 * before
    # bf16 activations and gradients and 8-bit states against f32 throughout
    assert abs(after - ref_after) < 0.1 * ref_after
    # the same token through the few-token and the many-token kernels: f32 sums in another order,
    # h and y rounded to bf16
    assert torch.allclose(one.float(), many[:1].float(), rtol=2.0 ** -6, atol=2.0 ** -6 * many.float().abs().max().item())
