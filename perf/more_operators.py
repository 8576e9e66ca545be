"""Cases of the operators around a pruned feed-forward block: its packed weights in 4 bits, a
mixture of such blocks, and the norms before and after it.

  quant    4-bit codes of packed values, one bf16 scale per group, and the values they stand for
  w4       y = x W^T for a few tokens on a 2:4 (or 6:8 sliding-window) packed weight in 4 bits
  w4_glu   h = act(x Wg^T) * (x Wu^T) on such weights
  moe      a router and the gated blocks of the experts it picks, for a few tokens
  norm     z = a x + gate * norm(y), n = norm(z): bf16, or FP8 codes with a scale per token
  norm_bwd its gradients

`own` False computes the plain forms in elementary torch operations; `own` True calls the
library.  Weights are packed as the library's headers lay them out: two kept values per 4
consecutive columns, their 2-bit positions in an LSB-first bitstream; 4-bit codes two to a
byte, low half first; scales [groups, rows].
"""
import math

import torch

own = False

_F8 = torch.float8_e4m3fn
_T = {"bf16": torch.bfloat16, "f32": torch.float32}
_FP4 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)      # e2m1 magnitudes


# ------------------------------------------------------------------ cases
def listed():
    return [
        # an adapter-sized weight, and the gate projection of a layer, when a model is made ready to serve
        {"name": "quant_small", "op": "quant", "code": "i4", "group": 64, "rows": 1000, "cols": 1376, "from": "f32"},
        {"name": "quant_layer", "op": "quant", "code": "fp4", "group": 128, "rows": 11008, "cols": 4096, "from": "bf16"},
        # one token through an 11008-row projection (decoding)
        {"name": "w4_one_token", "op": "w4", "code": "i4", "group": 128, "ns": 0, "tokens": 1, "cols": 4096, "rows": 11008},
        # a batch of requests, one token each, through the down projection
        {"name": "w4_requests", "op": "w4", "code": "fp4", "group": 64, "ns": 0, "tokens": 33, "cols": 11008, "rows": 4096},
        # the gate and up projections for one token, and for a few on a 6:8 layer
        {"name": "w4_glu_one_token", "op": "w4_glu", "code": "i4", "group": 128, "ns": 0, "act": "silu", "tokens": 1,
         "cols": 4096, "rows": 11008},
        {"name": "w4_glu_68", "op": "w4_glu", "code": "fp4", "group": 128, "ns": 4, "act": "relu2", "tokens": 16,
         "cols": 2560, "rows": 6912},
        # one token through many small experts, in 4 bits
        {"name": "moe_one_token", "op": "moe", "code": "i4", "group": 128, "tokens": 1, "cols": 2048, "rows": 1024,
         "experts": 64, "topk": 8, "act": "silu", "route": "softmax", "renorm": True},
        # a batch of requests through a few large experts, in bf16
        {"name": "moe_requests", "op": "moe", "code": "bf16", "group": 128, "tokens": 40, "cols": 4096, "rows": 2816,
         "experts": 16, "topk": 2, "act": "silu", "route": "sigmoid", "renorm": False},
        # the norm ahead of an FP8 6:8 block, for a few requests
        {"name": "norm_requests", "op": "norm", "x": "bf16", "tokens": 5, "cols": 2560, "post": "none", "pre": "rms",
         "gates": 0, "scale": 1.0, "out": "fp8", "ns": 4, "weights": "bf16"},
        # both norms around a block, for a training step's tokens
        {"name": "norm_train", "op": "norm", "x": "bf16", "tokens": 4096, "cols": 4096, "post": "rms", "pre": "rms",
         "gates": 1, "scale": 0.5, "out": "bf16", "ns": 0, "weights": "bf16"},
        # the backward pass: a short ragged batch gated per sequence, and a training step's tokens
        {"name": "norm_bwd_small", "op": "norm_bwd", "x": "f32", "tokens": 129, "cols": 1025, "post": "layer", "pre": "layer",
         "gates": 3, "scale": 0.7, "weights": "f32"},
        {"name": "norm_bwd_train", "op": "norm_bwd", "x": "bf16", "tokens": 4096, "cols": 4096, "post": "rms", "pre": "rms",
         "gates": 1, "scale": 0.5, "weights": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quant", "w4", "w4", "w4_glu", "moe", "moe", "norm", "norm", "norm_bwd", "norm_bwd"])
    code, group = rng.choice(["i4", "fp4"]), rng.choice([64, 128, 256])
    act = rng.choice(["silu", "gelu", "gelu_tanh", "relu2"])
    if op == "quant":
        return {"op": op, "code": code, "group": group, "rows": _log_int(rng, 16, 11008),
                "cols": 16 * _log_int(rng, 4, 256), "from": rng.choice(["bf16", "f32"])}
    if op in ("w4", "w4_glu"):
        ns = rng.choice([0, 0, 4])
        unit = 32 if ns else 16
        case = {"op": op, "code": code, "group": group, "ns": ns, "tokens": _log_int(rng, 1, 64),
                "cols": unit * max(2, _log_int(rng, 64, 8192) // unit), "rows": _log_int(rng, 64, 11008)}
        if op == "w4_glu":
            case["act"] = act
        return case
    if op == "moe":
        experts = rng.choice([4, 8, 16, 60, 64, 128])
        tokens = _log_int(rng, 1, 40)
        cols = 16 * _log_int(rng, 16, 256)
        rows = 16 * _log_int(rng, 8, max(8, min(176, 11534336 // (experts * cols))))
        return {"op": op, "code": rng.choice(["bf16", "i4", "fp4"]), "group": group, "tokens": tokens, "cols": cols,
                "rows": rows, "experts": experts, "topk": rng.randint(1, min(8, experts)), "act": act,
                "route": rng.choice(["softmax", "sigmoid"]), "renorm": rng.random() < 0.5}
    kind = lambda *more: rng.choice(["rms", "layer", *more])  # noqa: E731
    case = {"op": op, "x": rng.choice(["bf16", "f32"]), "tokens": _log_int(rng, 1, 4096), "post": kind("none"), "pre": kind(),
            "gates": rng.choice([0, 1, 3]), "scale": rng.choice([1.0, 0.5]), "weights": rng.choice(["bf16", "f32"])}
    case["gates"] = min(case["gates"], case["tokens"])
    most = min(8192, 3600 * 4096 // case["tokens"])
    if op == "norm":
        case["out"] = rng.choice(["bf16", "bf16", "fp8"])
        case["ns"] = rng.choice([0, 4]) if case["out"] == "fp8" else 0
        case["cols"] = 8 * _log_int(rng, 16, most // 8) if case["out"] == "fp8" else _log_int(rng, 100, most)
    else:
        case["cols"] = _log_int(rng, 100, most)
    return case


# ------------------------------------------------------------------ inputs
def _lifted(cols, ns):
    return cols // (2 * ns) * 4 * (ns - 1) if ns else cols


def _pad(t, unit):
    return torch.nn.functional.pad(t, (0, (-t.shape[-1]) % unit))


def _positions(g, rows, lifted, dev):
    """The index words of two random positions in every window of four columns."""
    lo, hi = torch.tensor([0, 0, 0, 1, 1, 2], device=dev), torch.tensor([1, 2, 3, 2, 3, 3], device=dev)
    pair = torch.randint(0, 6, (rows, lifted // 4), generator=g, device=dev)
    pos = torch.stack([lo[pair], hi[pair]], -1).reshape(rows, -1)
    p = _pad(pos, 16).view(rows, -1, 16)
    words = _pad((p << (2 * torch.arange(16, device=dev))).sum(-1), 4)     # index rows of whole 16 bytes
    return (words - ((words >> 31) << 32)).to(torch.int32)


def _nearest4(q, code):
    """4-bit codes (sign, 3 bits of magnitude) nearest q, ties to even codes."""
    a = q.abs()
    if code == "i4":
        mag = a.round().clamp(max=7)
    else:
        edge = [a > 0.25, a >= 0.75, a > 1.25, a >= 1.75, a > 2.5, a >= 3.5, a > 5.0]
        mag = sum(e.to(torch.float32) for e in edge)
    return mag.to(torch.uint8) | ((q < 0) & (mag > 0)).to(torch.uint8) * 8


def _quantise(v, code, group):
    """(codes, bf16 scales [rows, groups]) of packed values, group / 2 values to a scale."""
    rows, slots = v.shape
    b = _pad(v.float(), group // 2).view(rows, -1, group // 2)
    scale = (b.abs().amax(-1) / (7.0 if code == "i4" else 6.0)).to(torch.bfloat16)
    s = scale.float()[:, :, None]
    q = torch.where(s > 0, b / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(b))
    return _nearest4(q, code).view(rows, -1)[:, :slots], scale


def _weight(g, rows, cols, ns, code, group, scale, dev):
    """A random packed weight: {"v", "i"} in bf16, or with scales "s" in 4 bits."""
    lifted = _lifted(cols, ns)
    w = {"i": _positions(g, rows, lifted, dev)}
    v = (torch.randn((rows, lifted // 2), generator=g, device=dev) * scale).to(torch.bfloat16)
    if code == "bf16":
        w["v"] = _pad(v, 8)
        return w
    codes, s = _quantise(v, code, group)
    codes = _pad(codes, 2)
    w["v"] = _pad(codes[:, 0::2] | (codes[:, 1::2] << 4), 16).contiguous()
    w["s"] = _pad(s.t(), 4).contiguous()
    return w


def _experts(g, count, rows, cols, code, group, scale, dev):
    """The same weight of every expert, stacked."""
    each = [_weight(g, rows, cols, 0, code, group, scale, dev) for _ in range(count)]
    return {k: torch.stack([w[k] for w in each]) for k in each[0]}


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(1000003 * int(seed) + 29)
    rand = lambda *shape: torch.randn(shape, generator=g, device=dev)  # noqa: E731
    s = {"case": dict(case)}
    op, cols = case["op"], case["cols"]
    if op == "quant":
        s["vals"] = (rand(case["rows"], cols // 2) * 0.02).to(_T[case["from"]])
        return s
    tokens = case["tokens"]
    if op in ("norm", "norm_bwd"):
        wt = _T[case["weights"]]
        # a residual stream: channels of unlike size, a few large ones
        size = torch.exp(0.5 * rand(cols)) * torch.where(torch.rand(cols, generator=g, device=dev) < 0.003, 20.0, 1.0)
        s["x"] = (rand(tokens, cols) * size).to(_T[case["x"]])
        block = case["post"] != "none" or op == "norm_bwd"
        s["y"] = (rand(tokens, cols) * 0.7 + 0.1).to(torch.bfloat16) if block else None
        s["gate"] = (0.3 + 0.2 * rand(case["gates"], cols)).to(wt) if block and case["gates"] else None
        s["gate_rows"] = -(-tokens // case["gates"]) if case["gates"] else 0
        if s["gate"] is not None:     # the last sequences may be empty where the tokens do not fill them
            s["gate"] = s["gate"][:-(-tokens // s["gate_rows"])].contiguous()
        for k in ("post", "pre"):
            some = case[k] != "none"
            s["w_" + k] = (1 + 0.1 * rand(cols)).to(wt) if some else None
            s["b_" + k] = (0.1 * rand(cols)).to(wt) if case[k] == "layer" else None
        if op == "norm_bwd":          # z as the forward pass kept it, gradients from above
            s["dz"] = (rand(tokens, cols) * 0.01).to(_T[case["x"]])
            s["dn"] = (rand(tokens, cols) * 0.01).to(torch.bfloat16)
        return s
    s["x"] = rand(tokens, cols).to(torch.bfloat16)
    args = (case["code"], case["group"])
    scale = 1.4 / math.sqrt(cols)
    if op == "moe":
        experts, rows = case["experts"], case["rows"]
        s["router"] = (rand(experts, cols) / math.sqrt(cols)).to(torch.bfloat16)
        s["bias"] = 0.1 * rand(experts) if case["route"] == "sigmoid" else None
        s["g"], s["u"] = (_experts(g, experts, rows, cols, *args, scale, dev) for _ in range(2))
        s["d"] = _experts(g, experts, cols, rows, *args, 1.4 / math.sqrt(rows), dev)
        return s
    for k in ("g", "u") if op == "w4_glu" else ("w",):
        s[k] = _weight(g, case["rows"], cols, case["ns"], *args, scale, dev)
    return s


# ------------------------------------------------------------------ plain forms
def _columns(idx, slots, ns):
    """Column of every packed value: [rows, slots]."""
    dev = idx.device
    pos = ((idx[:, :, None] >> (2 * torch.arange(16, device=dev, dtype=torch.int32))) & 3).reshape(idx.shape[0], -1)
    win = torch.arange(slots, device=dev) // 2
    base = 4 * win if ns == 0 else 2 * ns * (win // (ns - 1)) + 2 * (win % (ns - 1))
    return pos[:, :slots].long() + base


def _table(code, dev, dtype=torch.float32):
    mag = torch.arange(8, device=dev, dtype=dtype) if code == "i4" else torch.tensor(_FP4, device=dev, dtype=dtype)
    return torch.cat([mag, -mag])


def _values(w, slots, code, group):
    """The packed values a weight's bytes stand for, in 32 bits."""
    if code == "bf16":
        return w["v"][:, :slots].float()
    nib = torch.stack([w["v"] & 15, w["v"] >> 4], -1).reshape(w["v"].shape[0], -1)[:, :slots].long()
    s = w["s"].float().t()[:nib.shape[0]].repeat_interleave(group // 2, dim=1)[:, :slots]
    return _table(code, nib.device)[nib] * s


def _dense(w, cols, ns, code, group):
    slots = _lifted(cols, ns) // 2
    full = torch.zeros((w["v"].shape[0], cols), dtype=torch.float32, device=w["v"].device)
    return full.scatter_add_(1, _columns(w["i"], slots, ns), _values(w, slots, code, group))


def _act(g, kind):
    if kind == "silu":
        return g / (1 + torch.exp(-g))
    if kind == "relu2":
        return g.clamp(min=0).square()
    if kind == "gelu":
        return 0.5 * g * (1 + torch.erf(g * math.sqrt(0.5)))
    return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g)))


def _route(s):
    """(experts, weights) of every token: the largest scores, the lower index first where two
    are the same.  Logits in 64 bits, because two of them may be close."""
    case = s["case"]
    logits = s["x"].double() @ s["router"].double().t()
    if case["route"] == "sigmoid":
        p = 1 / (1 + torch.exp(-logits))
    else:
        p = torch.exp(logits - logits.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
    key = p if s["bias"] is None else p + s["bias"].double()
    sel = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :case["topk"]]
    wt = p.gather(1, sel)
    if case["renorm"]:
        wt = wt / wt.sum(1, keepdim=True)
    return sel, wt


def _pick(w, e):
    return {k: t.index_select(0, e)[0] for k, t in w.items()}


def _plain_moe(s):
    case = s["case"]
    cols, rows, args = case["cols"], case["rows"], (0, case["code"], case["group"])
    sel, wt = _route(s)
    x, w32 = s["x"].float(), wt.float()
    y = torch.zeros((case["tokens"], cols), dtype=torch.float32, device=x.device)

    def block(xs, e):
        wg, wu, wd = (_dense(_pick(s[k], e), *c, *args) for k, c in (("g", (cols,)), ("u", (cols,)), ("d", (rows,))))
        return (_act(xs @ wg.t(), case["act"]) * (xs @ wu.t())) @ wd.t()

    if case["tokens"] * case["topk"] <= case["experts"]:     # each token's experts, one after the other
        for t in range(case["tokens"]):
            for j in range(case["topk"]):
                y[t] += w32[t, j] * block(x[t:t + 1], sel[t, j:j + 1])[0]
    else:                                                    # every expert on all tokens, weighted by their shares
        for e in range(case["experts"]):
            share = torch.where(sel == e, w32, torch.zeros_like(w32)).sum(1, keepdim=True)
            y += share * block(x, torch.full((1,), e, device=x.device))
    return {"y": y.to(torch.bfloat16), "experts": sel.to(torch.int32), "weights": w32}


def _norm(v, kind, w, b, eps):
    if kind == "none":
        return v
    if kind == "layer":
        v = v - v.mean(1, keepdim=True)
    v = v / torch.sqrt(v.square().mean(1, keepdim=True) + eps)
    v = v * w if w is not None else v
    return v if b is None else v + b


def _gate_of(s, tokens):
    if s["gate"] is None:
        return None
    return s["gate"].float().repeat_interleave(s["gate_rows"], dim=0)[:tokens]


_EPS = 1e-6


def _float(t):
    return None if t is None else t.float()


def _lift(q, ns):
    if not ns:
        return q
    m, c = q.shape
    b = q.view(m, c // (2 * ns), 2 * ns)
    return torch.stack([b[:, :, 2 * w:2 * w + 4] for w in range(ns - 1)], 2).reshape(m, -1)


def _plain_norm(s):
    case = s["case"]
    z = case["scale"] * s["x"].float()
    if s["y"] is not None:
        u = _norm(s["y"].float(), case["post"], _float(s["w_post"]), _float(s["b_post"]), _EPS)
        gate = _gate_of(s, case["tokens"])
        z = z + (u if gate is None else gate * u)
    n = _norm(z, case["pre"], _float(s["w_pre"]), _float(s["b_pre"]), _EPS)
    out = {"z": z.to(s["x"].dtype)} if s["y"] is not None else {}
    if case["out"] == "bf16":
        out["n"] = n.to(torch.bfloat16)
        return out
    top = n.abs().amax(1)
    scale = top / 448
    q = torch.where(scale[:, None] > 0, n / scale[:, None], torch.zeros_like(n)).clamp(-448, 448)
    out["n"], out["n_scale"] = _lift(q, case["ns"]).to(_F8), scale
    return out


def _norm_grad(v, d, kind, w, eps):
    """(dv, sum d vhat, sum d) of norm(v) with gradient d."""
    if kind == "none":
        return d, None, None
    if kind == "layer":
        v = v - v.mean(1, keepdim=True)
    r = 1 / torch.sqrt(v.square().mean(1, keepdim=True) + eps)
    hat = v * r
    dh = d if w is None else d * w
    dv = dh - hat * (dh * hat).mean(1, keepdim=True)
    if kind == "layer":
        dv = dv - dh.mean(1, keepdim=True)
    return dv * r, (d * hat).sum(0), d.sum(0) if kind == "layer" else None


def _plain_norm_bwd(s):
    case, tokens = s["case"], s["case"]["tokens"]
    z = s["x"].float()
    d, dw, db = _norm_grad(z, s["dn"].float(), case["pre"], _float(s["w_pre"]), _EPS)
    d = d + s["dz"].float()
    out = {"dx": (case["scale"] * d).to(s["x"].dtype), "dw_pre": dw, "db_pre": db}
    gate = _gate_of(s, tokens)
    y = s["y"].float()
    if gate is not None:
        u = d * _norm(y, case["post"], _float(s["w_post"]), _float(s["b_post"]), _EPS)
        rows = s["gate_rows"]
        out["dgate"] = torch.stack([u[a:a + rows].sum(0) for a in range(0, tokens, rows)])
        d = d * gate
    dy, out["dw_post"], out["db_post"] = _norm_grad(y, d, case["post"], _float(s["w_post"]), _EPS)
    out["dy"] = dy.to(torch.bfloat16)
    return {k: v for k, v in out.items() if v is not None}


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "quant":
        codes, scale = _quantise(s["vals"], case["code"], case["group"])
        slots = codes.shape[1]
        v = _table(case["code"], codes.device)[codes.long()] * scale.float().repeat_interleave(case["group"] // 2, 1)[:, :slots]
        return {"values": v.to(s["vals"].dtype), "scales": scale.t().contiguous()}
    if op == "moe":
        return _plain_moe(s)
    if op == "norm":
        return _plain_norm(s)
    if op == "norm_bwd":
        return _plain_norm_bwd(s)
    x, args = s["x"].float(), (case["cols"], case["ns"], case["code"], case["group"])
    if op == "w4":
        return {"y": (x @ _dense(s["w"], *args).t()).to(torch.bfloat16)}
    g, u = (x @ _dense(s[k], *args).t() for k in "gu")
    return {"h": (_act(g, case["act"]) * u).to(torch.bfloat16)}


# ------------------------------------------------------------------ the library
def _own(s):
    import semi_structured_sparsity_amd as nm

    case = s["case"]
    op = case["op"]
    code = {"i4": "NM_I4", "fp4": "NM_FP4", "bf16": "NM_BF16"}.get(case.get("code"))
    if op == "quant":
        _, scales, values = nm.nm_quant_w4(s["vals"], qdt=getattr(nm, code), group=case["group"], want_values=True)
        return {"values": values, "scales": scales}
    if op in ("norm", "norm_bwd"):
        kinds = {"none": nm.NM_NORM_NONE, "rms": nm.NM_NORM_RMS, "layer": nm.NM_NORM_LAYER}
        args = dict(Y=s["y"], gate=s["gate"], gate_rows=s["gate_rows"], res_scale=case["scale"], post=kinds[case["post"]],
                    w_post=s["w_post"], b_post=s["b_post"], pre=kinds[case["pre"]], w_pre=s["w_pre"], eps=_EPS)
        if op == "norm_bwd":
            out = nm.nm_block_norm_backward(s["x"], dZ=s["dz"], dN=s["dn"], **args)._asdict()
            names = {"dX": "dx", "dY": "dy"}
            return {names.get(k, k): v for k, v in out.items() if v is not None}
        fp8 = case["out"] == "fp8"
        z, n, scale = nm.nm_block_norm(s["x"], b_pre=s["b_pre"], ndt=nm.NM_FP8 if fp8 else nm.NM_BF16, Ns=case["ns"],
                                       want_z=s["y"] is not None, **args)
        return {k: v for k, v in (("z", z), ("n", n), ("n_scale", scale)) if v is not None}
    if op == "w4":
        return {"y": nm.nm_spmm_w4(s["x"], s["w"]["v"], s["w"]["i"], s["w"]["s"], qdt=getattr(nm, code), group=case["group"],
                                   Ns=case["ns"])}
    act = {"silu": nm.NM_ACT_SILU, "gelu": nm.NM_ACT_GELU, "gelu_tanh": nm.NM_ACT_GELU_TANH,
           "relu2": nm.NM_ACT_RELU2}[case["act"]]
    if op == "w4_glu":
        g, u = s["g"], s["u"]
        return {"h": nm.nm_spmm_glu_w4(s["x"], g["v"], g["i"], g["s"], u["v"], u["i"], u["s"], qdt=getattr(nm, code),
                                       group=case["group"], Ns=case["ns"], act=act)}
    if "layer" not in s:      # the program's handle of its experts, made once
        s["layer"] = nm.MoELayer(s["router"], gate=s["g"]["v"], gate_idx=s["g"]["i"], gate_scales=s["g"].get("s"),
                                 up=s["u"]["v"], up_idx=s["u"]["i"], up_scales=s["u"].get("s"), down=s["d"]["v"],
                                 down_idx=s["d"]["i"], down_scales=s["d"].get("s"), vdt=getattr(nm, code),
                                 hidden=case["rows"], group=case["group"], bias=s["bias"])
    y, experts, weights = nm.nm_moe(s["layer"], s["x"], topk=case["topk"], act=act, renorm=case["renorm"],
                                    route=nm.NM_ROUTE_SIGMOID if case["route"] == "sigmoid" else nm.NM_ROUTE_SOFTMAX,
                                    want_routing=True)
    return {"y": y, "experts": experts, "weights": weights}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ work
def _weight_bytes(rows, cols, ns, code, group):
    lifted = _lifted(cols, ns)
    if code == "bf16":
        return rows * (lifted + lifted // 8)
    return rows * (lifted // 4 + lifted // 8 + 2 * -(-lifted // group))


def work(case):
    op, cols = case["op"], case["cols"]
    if op == "quant":
        n, es = case["rows"] * cols // 2, 2 if case["from"] == "bf16" else 4
        return {"bytes": n * (2 * es + 0.5) + 2 * case["rows"] * -(-cols // case["group"]), "flops": 4 * n}
    t = case["tokens"]
    if op in ("norm", "norm_bwd"):
        n, es, ws = t * cols, 2 if case["x"] == "bf16" else 4, 2 if case["weights"] == "bf16" else 4
        block = case["post"] != "none" or op == "norm_bwd"
        vecs = (case["post"] != "none") + 1 + (case["post"] == "layer") + (case["pre"] == "layer") + (case["gates"] if block else 0)
        if op == "norm_bwd":
            return {"bytes": n * (3 * es + 2 * 3) + vecs * cols * (ws + 4), "flops": 30 * n}
        out = n * 2 if case["out"] == "bf16" else t * (_lifted(cols, case["ns"]) + 4)
        return {"bytes": n * es * (2 if block else 1) + (2 * n if block else 0) + out + vecs * cols * ws, "flops": 12 * n}
    r, args = case["rows"], (case.get("ns", 0), case["code"], case["group"])
    if op == "moe":
        # an expert that nobody picked is not read: the expected number of picked ones
        e, pairs = case["experts"], t * case["topk"]
        picked = e * (1 - (1 - case["topk"] / e) ** t)
        one = 2 * _weight_bytes(r, cols, *args) + _weight_bytes(cols, r, *args)
        return {"bytes": picked * one + 2 * e * cols + 4 * t * cols, "flops": 2 * pairs * 3 * r * cols // 2 + 2 * t * e * cols}
    n = 2 if op == "w4_glu" else 1
    lifted = _lifted(cols, case["ns"])
    return {"bytes": n * _weight_bytes(r, cols, *args) + 2 * t * (cols + r), "flops": n * t * r * lifted}


# ------------------------------------------------------------------ 64 bits
def _dense64(w, cols, ns, code, group):
    """The dense weight in 64 bits, window by window and position by position."""
    lifted = _lifted(cols, ns)
    rows, slots = w["v"].shape[0], lifted // 2
    slot = torch.arange(slots, device=w["v"].device)
    if code == "bf16":
        v = w["v"][:, :slots].double()
    else:
        c = (w["v"].to(torch.int64)[:, slot // 2] >> (4 * (slot % 2))[None]) & 15
        m = (c & 7).double()
        if code == "fp4":     # e2m1: a subnormal half, then 1.f times powers of two
            m = torch.where((c & 7) < 2, m * 0.5, torch.exp2(((c >> 1) & 3).double() - 1) * (1 + 0.5 * (c & 1).double()))
        v = torch.where(c >= 8, -m, m) * w["s"].double()[slot // (group // 2)].t()[:rows]
    pos = ((w["i"].to(torch.int64) & 0xFFFFFFFF)[:, slot // 16] >> (2 * (slot % 16))[None]) & 3
    win = torch.zeros((rows, slots // 2, 4), dtype=torch.float64, device=v.device)
    for j in range(4):
        win[:, :, j] = torch.where(pos == j, v, torch.zeros_like(v)).view(rows, -1, 2).sum(-1)
    if ns == 0:
        return win.view(rows, cols)
    full = torch.zeros((rows, cols // (2 * ns), 2 * ns), dtype=torch.float64, device=v.device)
    win = win.view(rows, -1, ns - 1, 4)
    for k in range(ns - 1):
        full[:, :, 2 * k:2 * k + 4] += win[:, :, k]
    return full.reshape(rows, cols)


def _act64(g, kind):
    if kind == "silu":
        return g * torch.sigmoid(g)
    if kind == "relu2":
        return torch.where(g > 0, g * g, 0 * g)
    if kind == "gelu":
        return g * 0.5 * torch.erfc(-g / math.sqrt(2))
    return g * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3))


def _exact_moe(s):
    case = s["case"]
    x = s["x"].double()
    logits = torch.matmul(x, s["router"].double().t())
    p = torch.sigmoid(logits) if case["route"] == "sigmoid" else torch.softmax(logits, 1)
    key = p if s["bias"] is None else p + s["bias"].double()
    # an expert's place: how many are before it
    before = (key[:, None, :] > key[:, :, None]).sum(-1)
    lower = torch.ones(key.shape[1], key.shape[1], device=x.device).tril(-1).bool()
    before = before + ((key[:, None, :] == key[:, :, None]) & lower[None]).sum(-1)
    sel = torch.argsort(before, 1)[:, :case["topk"]]
    wt = p.gather(1, sel)
    wt = wt / wt.sum(1, keepdim=True) if case["renorm"] else wt
    y = torch.zeros((case["tokens"], case["cols"]), dtype=torch.float64, device=x.device)
    args = (0, case["code"], case["group"])
    for e in torch.unique(sel).tolist():
        t, j = torch.nonzero(sel == e, as_tuple=True)
        w = [{k: v[e] for k, v in s[n].items()} for n in "gud"]
        h = _act64(torch.matmul(x[t], _dense64(w[0], case["cols"], *args).t()), case["act"])
        h = h * torch.matmul(x[t], _dense64(w[1], case["cols"], *args).t())
        y.index_add_(0, t, wt[t, j][:, None] * torch.matmul(h, _dense64(w[2], case["rows"], *args).t()))
    return {"y": y, "experts": None, "weights": wt}


def _stats64(v, kind):
    mean = v.mean(1, keepdim=True) if kind == "layer" else 0.0
    return mean, ((v - mean) ** 2).mean(1, keepdim=True).add(_EPS).rsqrt()


def _double(t):
    return None if t is None else t.double()


def _affine64(v, kind, w, b):
    if kind == "none":
        return v
    mean, r = _stats64(v, kind)
    v = (v - mean) * r
    v = v if w is None else v * w.double()
    return v if b is None else v + b.double()


def _backward64(v, d, kind, w):
    """v's gradient: with hat = (v - mean) r, each value moves hat through itself, the spread
    and (layer) the mean."""
    if kind == "none":
        return d, None, None
    mean, r = _stats64(v, kind)
    hat, c = (v - mean) * r, v.shape[1]
    dh = d if w is None else d * w.double()
    dv = r * dh - r * hat * ((dh * hat).sum(1, keepdim=True) / c)
    if kind == "layer":
        dv = dv - r * (dh.sum(1, keepdim=True) / c)
    return dv, (d * hat).sum(0), d.sum(0) if kind == "layer" else None


def _exact_norm(s):
    case = s["case"]
    gate = None if s["gate"] is None else s["gate"].double()[torch.arange(case["tokens"], device=s["x"].device) // s["gate_rows"]]
    if case["op"] == "norm":
        z = s["x"].double() * case["scale"]
        if s["y"] is not None:
            u = _affine64(s["y"].double(), case["post"], s["w_post"], s["b_post"])
            z = z + (u if gate is None else gate * u)
        n = _affine64(z, case["pre"], s["w_pre"], s["b_pre"])
        out = {"z": z} if s["y"] is not None else {}
        if case["out"] == "bf16":
            out["n"] = n
            return out
        scale = n.abs().amax(1) / 448
        q = n / torch.where(scale > 0, scale, torch.ones_like(scale))[:, None]
        a = q.abs()
        unit = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -40))).clamp(min=-6) - 3)
        q = (torch.round(a / unit) * unit).clamp(max=448) * q.sign()
        if case["ns"]:
            j = torch.arange(_lifted(case["cols"], case["ns"]), device=q.device)
            w = j // 4
            q = q[:, 2 * case["ns"] * (w // (case["ns"] - 1)) + 2 * (w % (case["ns"] - 1)) + j % 4]
        out["n"], out["n_scale"] = q, scale
        return out
    d, dw, db = _backward64(s["x"].double(), s["dn"].double(), case["pre"], s["w_pre"])
    d = d + s["dz"].double()
    out = {"dx": case["scale"] * d, "dw_pre": dw, "db_pre": db}
    y = s["y"].double()
    if gate is not None:
        u = d * _affine64(y, case["post"], s["w_post"], s["b_post"])
        dg = torch.zeros_like(s["gate"], dtype=torch.float64)
        out["dgate"] = dg.index_add_(0, torch.arange(case["tokens"], device=y.device) // s["gate_rows"], u)
        d = d * gate
    out["dy"], out["dw_post"], out["db_post"] = _backward64(y, d, case["post"], s["w_post"])
    return {k: v for k, v in out.items() if v is not None}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quant":
        v, half = s["vals"].double(), case["group"] // 2
        rows, slots = v.shape
        out, scales = torch.zeros_like(v), []
        for a in range(0, slots, half):
            b = v[:, a:a + half]
            sc = (b.abs().amax(1) / (7 if case["code"] == "i4" else 6)).to(torch.float32).to(torch.bfloat16).double()
            q = b / torch.where(sc > 0, sc, torch.ones_like(sc))[:, None]
            if case["code"] == "i4":
                q = q.round().clamp(-7, 7)
            else:
                a4 = q.abs()
                unit = torch.exp2(torch.floor(torch.log2(a4.clamp(min=1.0))) - 1)
                q = (torch.round(a4 / unit) * unit).clamp(max=6) * q.sign()
            out[:, a:a + half] = q * sc[:, None]
            scales.append(sc)
        return {"values": out, "scales": torch.stack(scales)}
    if op == "moe":
        return _exact_moe(s)
    if op in ("norm", "norm_bwd"):
        return _exact_norm(s)
    x, args = s["x"].double(), (case["cols"], case["ns"], case["code"], case["group"])
    if op == "w4":
        return {"y": torch.matmul(x, _dense64(s["w"], *args).t())}
    g, u = (torch.matmul(x, _dense64(s[k], *args).t()) for k in "gu")
    return {"h": _act64(g, case["act"]) * u}
