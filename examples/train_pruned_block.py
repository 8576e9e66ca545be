"""Recover a pruned gated feed-forward block by training its kept values.

A dense block y = (silu(x Wg^T) . (x Wu^T)) Wd^T is pruned to 2:4 (or with
--slide N to (2N-2):2N) and packed; its mask stays fixed while AdamW moves the kept values (f32 masters, bf16 copies that the products read,
states in 8 bits) towards the dense block's outputs.  The trained block then answers a single
token, as it would in serving.

    python examples/train_pruned_block.py [--width 1024 --hidden 2816 --tokens 512 --steps 60 --slide 0]
"""
from __future__ import annotations

import argparse
import sys
from pathlib import Path

import torch

sys.path.insert(0, str(Path(__file__).resolve().parents[1]))
import semi_structured_sparsity_amd as nm  # noqa: E402


def train(width: int = 1024, hidden: int = 2816, tokens: int = 512, steps: int = 60, lr: float = 5e-4, seed: int = 0,
          Ns: int = 0):
    """(loss before, loss after, single-token output of the trained block, its batch output)."""
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g, device=dev)  # noqa: E731
    dense = {"g": rand(hidden, width) * width ** -0.5, "u": rand(hidden, width) * width ** -0.5,
             "d": rand(width, hidden) * hidden ** -0.5}

    # prune by magnitude, pack; the masters hold the kept values in f32
    vals, idx = {}, {}
    for k, w in dense.items():
        if Ns:
            vals[k], idx[k], _ = nm.nm_prune_slide(w, None, 0.0, nm.NM_SCORE_MAGNITUDE, Ns, vdt=nm.NM_BF16)
        else:
            vals[k], idx[k], _ = nm.nm_prune_pack(w, None, 0.0, nm.NM_SCORE_MAGNITUDE, 2, 4)
    master = {k: v.float() for k, v in vals.items()}
    grad = {k: torch.empty_like(v) for k, v in vals.items()}
    f8 = lambda t: torch.zeros(t.shape, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn)  # noqa: E731
    scales = lambda t: torch.zeros((t.numel() + 255) // 256, device=dev)  # noqa: E731
    names = list(vals)
    trained = nm.AdamWTensors(
        params=[master[k] for k in names], grads=[grad[k] for k in names], m=[f8(master[k]) for k in names],
        v=[f8(master[k]) for k in names], m_scale=[scales(master[k]) for k in names],
        v_scale=[scales(master[k]) for k in names], copies=[vals[k] for k in names])

    ws = torch.empty(max(nm.raw.nm_spmm_glu_workspace(tokens, width, hidden, Ns, nm.NM_BF16),
                         nm.raw.nm_spmm_glu_backward_workspace(tokens, width, hidden, Ns),
                         nm.raw.nm_spmm_backward_workspace(tokens, hidden, width, Ns),
                         nm.raw.nm_spmm_workspace(tokens, hidden, width, Ns, nm.NM_BF16), 1), dtype=torch.uint8, device=dev)

    def forward(x, save):
        out = nm.nm_spmm_glu(x, vals["g"], idx["g"], vals["u"], idx["u"], Ns=Ns, save=save, ws=ws)
        h, pre = (out[0], out[1:]) if save else (out, None)
        return nm.nm_spmm(h, vals["d"], idx["d"], Ns=Ns, ws=ws), h, pre

    # activations of a model lie near a subspace: an eighth of the width here
    mix = rand(width // 8, width) * (width // 8) ** -0.5

    def batch():
        x = (rand(tokens, width // 8) @ mix).to(torch.bfloat16)
        xf = x.float()
        return x, (torch.nn.functional.silu(xf @ dense["g"].t()) * (xf @ dense["u"].t())) @ dense["d"].t()

    def loss_of(x, want):
        return (forward(x, False)[0].float() - want).square().mean().item()

    held, held_want = batch()
    before = loss_of(held, held_want)
    for step in range(1, steps + 1):
        x, want = batch()
        y, h, (pre_g, pre_u) = forward(x, True)
        dy = ((y.float() - want) * (2.0 / y.numel())).to(torch.bfloat16)
        dh, _ = nm.nm_spmm_backward(dy, h, vals["d"], idx["d"], Ns=Ns, out_dv=grad["d"], ws=ws)
        nm.nm_spmm_glu_backward(dh, pre_g, pre_u, x, vals["g"], idx["g"], vals["u"], idx["u"], Ns=Ns,
                                want_dx=False, out_dv=(grad["g"], grad["u"]), ws=ws)
        nm.nm_adamw_unbiased(trained, lr=lr * min(1.0, step / 10), step=step, seed=seed)
    after = loss_of(held, held_want)
    return before, after, forward(held[:1], False)[0], forward(held, False)[0]


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("width", 1024), ("hidden", 2816), ("tokens", 512), ("steps", 60), ("slide", 0)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    before, after, one, many = train(a.width, a.hidden, a.tokens, a.steps, Ns=a.slide)
    print(f"mean squared error to the dense block: pruned {before:.5f}, after {a.steps} steps {after:.5f}")
    print(f"one token alone against the same token in the batch: max difference {(one - many[:1]).abs().max().item():.2e}")
