"""Cases of the sparse feed-forward and optimiser operators: fine-tuning and serving a pruned
gated feed-forward block.

  glu      h = act(x Wg^T) * (x Wu^T) on 2:4 (or 6:8 sliding-window) packed weights
  glu_bwd  its gradients: dx and the gradients of the packed values of Wg and Wu
  spmm_bwd the gradients of the plain packed layer y = x W^T (the block's down projection)
  adamw    one AdamW step over many tensors, with states in 32 bits or in e4m3 codes

`own` False computes the plain forms in elementary torch operations in 32 bits; `own` True
calls the library.  Weights are packed as include/nmsparse.h lays them out: two kept values
per 4 consecutive columns, their 2-bit positions in an LSB-first bitstream.
"""
import math

import torch

own = False

_BLOCK = 256          # elements that share a scale of 8-bit states
_F8 = torch.float8_e4m3fn
_T = {"bf16": torch.bfloat16, "f32": torch.float32, "int8": torch.int8, "fp8": _F8}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one token through the gate and up projections of an 11008-row layer (decoding)
        {"name": "glu_one_token", "op": "glu", "dtype": "bf16", "ns": 0, "act": "silu", "tokens": 1, "cols": 4096,
         "rows": 11008, "save": False},
        # a few requests' tokens on a ternary 6:8 layer with int8 activations
        {"name": "glu_int8_68", "op": "glu", "dtype": "int8", "ns": 4, "act": "relu2", "tokens": 16, "cols": 2560,
         "rows": 6912, "save": False},
        # a prompt's tokens on a 6:8 layer in FP8
        {"name": "glu_fp8_68", "op": "glu", "dtype": "fp8", "ns": 4, "act": "gelu_tanh", "tokens": 512, "cols": 4096,
         "rows": 14336, "save": False},
        # the forward pass of a training step, with the pre-activations kept for the backward
        {"name": "glu_train", "op": "glu", "dtype": "bf16", "ns": 0, "act": "silu", "tokens": 2048, "cols": 4096,
         "rows": 11008, "save": True},
        # its backward pass: a short ragged batch on a small block, and a training step's
        {"name": "glu_bwd_small", "op": "glu_bwd", "act": "gelu", "tokens": 129, "cols": 1024, "rows": 2730},
        {"name": "glu_bwd_train", "op": "glu_bwd", "act": "silu", "tokens": 2048, "cols": 4096, "rows": 11008},
        # the down projection's backward pass, small and ragged, and a training step's
        {"name": "spmm_bwd_small", "op": "spmm_bwd", "tokens": 200, "cols": 2736, "rows": 1000},
        {"name": "spmm_bwd_train", "op": "spmm_bwd", "tokens": 2048, "cols": 11008, "rows": 4096},
        # a handful of adapter-sized tensors: launch latency
        {"name": "adamw_small", "op": "adamw", "state": "f32", "param": "f32", "copy": True, "tensors": 9, "numel": 8192},
        # the packed values of a layer's projections: f32 masters with bf16 copies
        {"name": "adamw_f32", "op": "adamw", "state": "f32", "param": "f32", "copy": True, "tensors": 12,
         "numel": 22544384},
        # the same with states in 8 bits
        {"name": "adamw_8bit", "op": "adamw", "state": "fp8", "param": "f32", "copy": True, "tensors": 12,
         "numel": 22544384},
        # bf16 parameters without masters, many tensors of mixed sizes
        {"name": "adamw_8bit_bf16", "op": "adamw", "state": "fp8", "param": "bf16", "copy": False, "tensors": 40,
         "numel": 1048576},
    ]


_MOST = 2048 * 4096 * 11008     # tokens * cols * rows of the largest listed case


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["glu", "glu", "glu_bwd", "spmm_bwd", "adamw", "adamw"])
    if op == "adamw":
        param = rng.choice(["f32", "bf16"])
        return {"op": "adamw", "state": rng.choice(["f32", "fp8"]), "param": param,
                "copy": param == "f32" and rng.random() < 0.75, "tensors": rng.randint(1, 48),
                "numel": _log_int(rng, 300, 4000000)}
    tokens = _log_int(rng, 1, 2048)
    if op == "glu":
        dtype = rng.choice(["bf16", "bf16", "int8", "fp8"])
        ns = rng.choice([0, 4])
        # whole 16-byte rows of the (lifted) width in every type
        unit = 64 if ns else 32
        cols = unit * max(2, _log_int(rng, 128, 4096) // unit)
        rows = min(_log_int(rng, 64, 14336), _MOST // (tokens * cols))
        return {"op": "glu", "dtype": dtype, "ns": ns, "act": rng.choice(["silu", "gelu", "gelu_tanh", "relu2"]),
                "tokens": tokens, "cols": cols, "rows": rows, "save": dtype == "bf16" and rng.random() < 0.5}
    cols = 16 * max(4, _log_int(rng, 64, 8192) // 16)
    rows = min(_log_int(rng, 64, 11008), _MOST // (tokens * cols))
    case = {"op": op, "tokens": tokens, "cols": cols, "rows": rows}
    if op == "glu_bwd":
        case["act"] = rng.choice(["silu", "gelu", "gelu_tanh", "relu2"])
    return case


# ------------------------------------------------------------------ inputs
def _lifted(cols, ns):
    return cols // (2 * ns) * 4 * (ns - 1) if ns else cols


def _packed(g, rows, cols, ns, dtype, scale, dev):
    """(vals, idx) of a random weight pruned by magnitude: 2 of 4, or 2*ns-2 of 2*ns spread
    over overlapping windows of 4 columns (each kept column in the first window with room)."""
    w = torch.randn((rows, cols), generator=g, device=dev)
    if ns == 0:
        x = w.view(rows, cols // 4, 4).abs()
        # the two largest of four, lower column first
        lo, hi = [0, 0, 0, 1, 1, 2], [1, 2, 3, 2, 3, 3]
        pair = torch.stack([x[..., a] + x[..., b] for a, b in zip(lo, hi)], dim=-1).argmax(-1)
        pos = torch.stack([torch.tensor(lo, device=dev)[pair], torch.tensor(hi, device=dev)[pair]], -1)
        col = pos + 4 * torch.arange(cols // 4, device=dev)[None, :, None]
    else:
        m = 2 * ns
        x = w.view(rows, cols // m, m)
        drop = x.abs().topk(2, dim=-1, largest=False).indices
        keep = torch.ones_like(x, dtype=torch.bool).scatter_(-1, drop, False)
        used = torch.zeros((rows, cols // m, ns - 1), dtype=torch.long, device=dev)
        pos = torch.zeros((rows, cols // m, ns - 1, 2), dtype=torch.long, device=dev)
        for k in range(m):
            left = keep[..., k].clone()
            for v in range(max(0, (k - 2) // 2), min(ns - 2, k // 2) + 1):
                if not 0 <= k - 2 * v <= 3:
                    continue
                take = left & (used[..., v] < 2)
                pos[..., v, 0] = torch.where(take & (used[..., v] == 0), k - 2 * v, pos[..., v, 0])
                pos[..., v, 1] = torch.where(take & (used[..., v] == 1), k - 2 * v, pos[..., v, 1])
                used[..., v] += take.long()
                left &= ~take
        col = pos + 2 * torch.arange(ns - 1, device=dev)[:, None]
        col = (col + m * torch.arange(cols // m, device=dev)[None, :, None, None])
    pos, col = pos.reshape(rows, -1), col.reshape(rows, -1)
    kept = w.gather(1, col)
    if dtype == "int8":
        vals = torch.where(kept.abs() <= 0.553, torch.zeros_like(kept), kept.sign()).to(torch.int8)
    elif dtype == "fp8":
        vals = kept.clamp(-448, 448).to(_F8)
    else:
        vals = (kept * scale).to(torch.bfloat16)
    slots = pos.shape[1]
    pad = (-slots) % 16
    p = torch.nn.functional.pad(pos, (0, pad)).view(rows, -1, 16)
    words = (p << (2 * torch.arange(16, device=dev))).sum(-1)
    # index rows of whole 16 bytes, as a program that packs once would lay them out
    words = torch.nn.functional.pad(words, (0, (-words.shape[1]) % 4))
    idx = (words - ((words >> 31) << 32)).to(torch.int32)
    return vals.contiguous(), idx.contiguous()


def _sizes(case):
    """Ragged sizes of the tensors of one optimiser step, and their places in the flat
    buffers (each starts on a block of its own)."""
    sizes = [max(1, (case["numel"] >> (i % 6)) - (i * 37) % 251) for i in range(case["tensors"])]
    starts, at = [], 0
    for n in sizes:
        starts.append(at)
        at += -(-n // _BLOCK) * _BLOCK
    return sizes, starts, at


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(1000003 * int(seed) + 17)
    s = {"case": dict(case)}
    if case["op"] == "adamw":
        sizes, starts, total = _sizes(case)
        param, f8 = _T[case["param"]], case["state"] == "fp8"
        real = torch.zeros(total, dtype=torch.bool, device=dev)
        for n, a in zip(sizes, starts):
            real[a:a + n] = True
        rand = lambda: torch.randn(total, generator=g, device=dev)  # noqa: E731
        # gradients of tensors differ in size by orders of magnitude, as a model's do
        mag = torch.exp(torch.randn(total // _BLOCK, generator=g, device=dev) * 1.5 - 7.0).repeat_interleave(_BLOCK)
        s["p"] = (rand() * 0.02 * real).to(param)
        s["g"] = (rand() * mag * real).to(torch.bfloat16)
        m, v = rand() * 0.3 * mag * real, (rand() * mag).square() * 0.5 * real
        if f8:
            s["m"], s["ms"] = _encode(m, False)
            s["v"], s["vs"] = _encode(v.sqrt(), True)
        else:
            s["m"], s["v"] = m, v
        s["c"] = s["p"].to(torch.bfloat16) if case["copy"] else None
        s["clip"] = torch.full((1,), 0.73, device=dev)
        # decay for the weights, none for the small tensors (norms, biases)
        s["decay"] = [0.1 if n >= 1024 else 0.0 for n in sizes]
        s["decay_of"] = torch.tensor(s["decay"], device=dev).repeat_interleave(
            torch.tensor([-(-n // _BLOCK) for n in sizes], device=dev))
        s["sizes"], s["starts"] = sizes, starts
        s["step"], s["lr"], s["betas"], s["eps"] = 100, 3e-4, (0.9, 0.95), 1e-8
        return s
    tokens, cols, rows = case["tokens"], case["cols"], case["rows"]
    ns, dtype = case.get("ns", 0), case.get("dtype", "bf16")
    x = torch.randn((tokens, cols), generator=g, device=dev)
    wscale = 1.4 / math.sqrt(cols)
    s["xs"], s["gs"], s["us"] = None, 1.0, 1.0
    if dtype == "bf16":
        s["x"] = x.to(torch.bfloat16)
    else:
        top = 127.0 if dtype == "int8" else 448.0
        s["xs"] = x.abs().amax(1) / top
        q = x / s["xs"][:, None]
        s["x"] = q.round().to(torch.int8) if dtype == "int8" else q.to(_F8)
        s["gs"], s["us"] = 1.2 * wscale, 0.9 * wscale
    for k in ("g", "u") if case["op"] != "spmm_bwd" else ("w",):
        s["v" + k], s["i" + k] = _packed(g, rows, cols, ns, dtype, wscale, dev)
    if case["op"] == "glu_bwd":
        s["gate"] = torch.randn((tokens, rows), generator=g, device=dev).to(torch.bfloat16)
        s["up"] = torch.randn((tokens, rows), generator=g, device=dev).to(torch.bfloat16)
    if case["op"] != "glu":
        s["dy"] = (torch.randn((tokens, rows), generator=g, device=dev) * 0.01).to(torch.bfloat16)
    return s


# ------------------------------------------------------------------ plain forms
def _columns(idx, slots, ns):
    """Column of every packed value: [rows, slots]."""
    dev = idx.device
    pos = ((idx[:, :, None] >> (2 * torch.arange(16, device=dev, dtype=torch.int32))) & 3).reshape(idx.shape[0], -1)
    win = torch.arange(slots, device=dev) // 2
    base = 4 * win if ns == 0 else 2 * ns * (win // (ns - 1)) + 2 * (win % (ns - 1))
    return pos[:, :slots].long() + base


def _dense(vals, idx, cols, ns):
    w = torch.zeros((vals.shape[0], cols), dtype=torch.float32, device=vals.device)
    return w.scatter_add_(1, _columns(idx, vals.shape[1], ns), vals.float())


def _act(g, kind):
    if kind == "silu":
        return g / (1 + torch.exp(-g))
    if kind == "relu2":
        return g.clamp(min=0).square()
    if kind == "gelu":
        return 0.5 * g * (1 + torch.erf(g * math.sqrt(0.5)))
    return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g)))


def _act_grad(g, kind):
    if kind == "silu":
        t = 1 / (1 + torch.exp(-g))
        return t * (1 + g * (1 - t))
    if kind == "relu2":
        return 2 * g.clamp(min=0)
    if kind == "gelu":
        return 0.5 * (1 + torch.erf(g * math.sqrt(0.5))) + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)


def _encode(x, nonzero):
    """e4m3 codes and f32 scales of blocks of 256: scale = max|x| / 448.  `nonzero`: a value
    above zero keeps at least the smallest code."""
    b = x.view(-1, _BLOCK)
    top = b.abs().amax(1)
    some = top >= 2.0 ** -118
    q = b * torch.where(some, 448.0 / top, torch.zeros_like(top))[:, None]
    if nonzero:
        q = torch.where((b > 0) & some[:, None], q.clamp(min=2.0 ** -9), q)
    return q.clamp(-448, 448).to(_F8).view(-1), torch.where(some, top * (1 / 448.0), torch.zeros_like(top))


def _decode(q, scale):
    return (q.view(-1, _BLOCK).float() * scale[:, None]).view(-1)


def _plain_adamw(s):
    b1, b2 = s["betas"]
    f8 = s["case"]["state"] == "fp8"
    p, g = s["p"].float(), s["g"].float() * s["clip"]
    m = _decode(s["m"], s["ms"]) if f8 else s["m"]
    v = _decode(s["v"], s["vs"]).square() if f8 else s["v"]
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    new = p.view(-1, _BLOCK) * (1 - s["lr"] * s["decay_of"])[:, None]
    denom = torch.sqrt(v * (1 / (1 - b2 ** s["step"]))) + s["eps"]
    new = new.view(-1) - (s["lr"] / (1 - b1 ** s["step"])) * m / denom
    s["p"].copy_(new)
    if s["c"] is not None:
        s["c"].copy_(new)
    if f8:
        q, scale = _encode(m, False)
        s["m"].copy_(q)
        s["ms"].copy_(scale)
        q, scale = _encode(v.sqrt(), True)
        s["v"].copy_(q)
        s["vs"].copy_(scale)
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)


def _adamw_out(s):
    return {k: s[k] for k in ("p", "c", "m", "v", "ms", "vs") if s.get(k) is not None}


def _plain(s):
    case = s["case"]
    if case["op"] == "adamw":
        _plain_adamw(s)
        return _adamw_out(s)
    x, cols, ns = s["x"].float(), case["cols"], case.get("ns", 0)
    if case["op"] == "glu":
        g = (x @ _dense(s["vg"], s["ig"], cols, ns).t()) * s["gs"]
        u = (x @ _dense(s["vu"], s["iu"], cols, ns).t()) * s["us"]
        if s["xs"] is not None:
            g, u = g * s["xs"][:, None], u * s["xs"][:, None]
        h = (_act(g, case["act"]) * u).to(torch.bfloat16)
        return {"h": h, "g": g.to(torch.bfloat16), "u": u.to(torch.bfloat16)} if case["save"] else {"h": h}
    dy = s["dy"].float()
    if case["op"] == "spmm_bwd":
        dx = dy @ _dense(s["vw"], s["iw"], cols, 0)
        dw = (dy.t() @ x).gather(1, _columns(s["iw"], cols // 2, 0))
        return {"dx": dx.to(torch.bfloat16), "dv": dw.to(torch.bfloat16)}
    g, u = s["gate"].float(), s["up"].float()
    dg, du = dy * u * _act_grad(g, case["act"]), dy * _act(g, case["act"])
    dx = dg @ _dense(s["vg"], s["ig"], cols, 0) + du @ _dense(s["vu"], s["iu"], cols, 0)
    dvg = (dg.t() @ x).gather(1, _columns(s["ig"], cols // 2, 0))
    dvu = (du.t() @ x).gather(1, _columns(s["iu"], cols // 2, 0))
    return {"dx": dx.to(torch.bfloat16), "dvg": dvg.to(torch.bfloat16), "dvu": dvu.to(torch.bfloat16)}


# ------------------------------------------------------------------ the library
def _own(s):
    import semi_structured_sparsity_amd as nm

    case = s["case"]
    if case["op"] == "adamw":
        if "list" not in s:      # the program's list of what it trains, made once
            views = lambda t: [t[a:a + n] for n, a in zip(s["sizes"], s["starts"])]  # noqa: E731
            scales = lambda t: [t[a // _BLOCK:a // _BLOCK + -(-n // _BLOCK)]  # noqa: E731
                                for n, a in zip(s["sizes"], s["starts"])]
            f8 = case["state"] == "fp8"
            s["list"] = nm.AdamWTensors(
                params=views(s["p"]), grads=views(s["g"]), m=views(s["m"]), v=views(s["v"]),
                m_scale=scales(s["ms"]) if f8 else None, v_scale=scales(s["vs"]) if f8 else None,
                copies=None if s["c"] is None else views(s["c"]), weight_decay=s["decay"])
        nm.nm_adamw(s["list"], lr=s["lr"], beta1=s["betas"][0], beta2=s["betas"][1], eps=s["eps"], step=s["step"],
                    grad_scale=s["clip"])
        return _adamw_out(s)
    if case["op"] == "spmm_bwd":
        dx, dv = nm.nm_spmm_backward(s["dy"], s["x"], s["vw"], s["iw"])
        return {"dx": dx, "dv": dv}
    act = {"silu": nm.NM_ACT_SILU, "gelu": nm.NM_ACT_GELU, "gelu_tanh": nm.NM_ACT_GELU_TANH,
           "relu2": nm.NM_ACT_RELU2}[case["act"]]
    if case["op"] == "glu":
        out = nm.nm_spmm_glu(s["x"], s["vg"], s["ig"], s["vu"], s["iu"], Ns=case["ns"], act=act, x_scale=s["xs"],
                             g_scale=s["gs"], u_scale=s["us"], hdt=nm.NM_BF16, save=case["save"])
        return {"h": out[0], "g": out[1], "u": out[2]} if case["save"] else {"h": out}
    dx, dvg, dvu = nm.nm_spmm_glu_backward(s["dy"], s["gate"], s["up"], s["x"], s["vg"], s["ig"], s["vu"], s["iu"],
                                           act=act)
    return {"dx": dx, "dvg": dvg, "dvu": dvu}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ work
def work(case):
    if case["op"] == "adamw":
        n = sum(_sizes(case)[0])
        p = 4 if case["param"] == "f32" else 2
        st = 4 if case["state"] == "f32" else 1 + 4 / _BLOCK
        return {"bytes": n * (2 * p + 2 + 4 * st + (2 if case["copy"] else 0)), "flops": 20 * n}
    t, k, r = case["tokens"], case["cols"], case["rows"]
    es = {"bf16": 2, "int8": 1, "fp8": 1}[case.get("dtype", "bf16")]
    kl = _lifted(k, case.get("ns", 0))
    packed = r * (kl // 2 * es + kl // 8)        # values and positions of one weight
    kept = 2 * t * r * (kl // 2)                 # multiply-adds of one product on kept weights
    if case["op"] == "glu":
        return {"bytes": 2 * packed + t * k * es + t * r * 2 * (3 if case["save"] else 1), "flops": 2 * kept}
    if case["op"] == "spmm_bwd":
        return {"bytes": packed + 2 * t * r + 2 * 2 * t * k + r * k, "flops": 2 * kept}
    return {"bytes": 2 * packed + 3 * 2 * t * r + 2 * 2 * t * k + 2 * r * k, "flops": 4 * kept}


# ------------------------------------------------------------------ 64 bits
def _weight64(vals, idx, cols, ns):
    """The dense weight in 64 bits, position by position of the windows of four columns."""
    rows, slots = vals.shape
    code = idx.to(torch.int64) & 0xFFFFFFFF
    slot = torch.arange(slots, device=vals.device)
    pos = (code[:, slot // 16] >> (2 * (slot % 16))[None]) & 3
    v = vals.to(torch.float32).double()
    win = torch.zeros((rows, slots // 2, 4), dtype=torch.float64, device=vals.device)
    for j in range(4):
        win[:, :, j] = torch.where(pos == j, v, torch.zeros_like(v)).view(rows, -1, 2).sum(-1)
    if ns == 0:
        return win.view(rows, cols)
    w = torch.zeros((rows, cols // (2 * ns), 2 * ns), dtype=torch.float64, device=vals.device)
    win = win.view(rows, -1, ns - 1, 4)
    for k in range(ns - 1):
        w[:, :, 2 * k:2 * k + 4] += win[:, :, k]
    return w.reshape(rows, cols)


def _take64(full, idx, slots):
    code = idx.to(torch.int64) & 0xFFFFFFFF
    slot = torch.arange(slots, device=full.device)
    pos = (code[:, slot // 16] >> (2 * (slot % 16))[None]) & 3
    four = full.view(full.shape[0], -1, 4).repeat_interleave(2, dim=1)
    return four.gather(2, pos[:, :, None])[:, :, 0]


def _e4m3_64(q, least):
    a = q.abs()
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** -40))).clamp(min=-6)
    unit = torch.exp2(e - 3)
    r = (torch.round(a / unit) * unit).clamp(max=448)
    if least:
        r = torch.where((a > 0) & (r == 0), torch.full_like(r, 2.0 ** -9), r)
    return r * q.sign()


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "adamw":
        b1, b2 = s["betas"]
        f8 = case["state"] == "fp8"
        g = s["g"].double() * s["clip"].double()
        block = lambda q, sc: (q.to(torch.float32).double().view(-1, _BLOCK) * sc.double()[:, None]).view(-1)  # noqa: E731
        m = block(s["m"], s["ms"]) if f8 else s["m"].double()
        v = block(s["v"], s["vs"]) ** 2 if f8 else s["v"].double()
        m = m + (1 - b1) * (g - m)
        v = v + (1 - b2) * (g * g - v)
        decay = s["decay_of"].double().repeat_interleave(_BLOCK)
        p = s["p"].double()
        p = p - s["lr"] * (decay * p + (m / (1 - b1 ** s["step"])) / ((v / (1 - b2 ** s["step"])).sqrt() + s["eps"]))
        out = {"p": p, "m": m, "v": v}
        if s["c"] is not None:
            out["c"] = p
        if f8:
            for k, t, least in (("m", m, False), ("v", v.sqrt(), True)):
                b = t.view(-1, _BLOCK)
                top = b.abs().amax(1)
                sc = top / 448
                out[k] = _e4m3_64(b / torch.where(sc > 0, sc, torch.ones_like(sc))[:, None], least).view(-1)
                out[k + "s"] = sc
        return out
    cols, ns = case["cols"], case.get("ns", 0)
    x = s["x"].to(torch.float32).double()
    act = case.get("act")
    if act == "silu":
        fn, d = lambda g: g * torch.sigmoid(g), lambda g: torch.sigmoid(g) + g * torch.sigmoid(g) * torch.sigmoid(-g)
    elif act == "relu2":
        fn, d = lambda g: torch.where(g > 0, g * g, 0 * g), lambda g: torch.where(g > 0, 2 * g, 0 * g)
    elif act == "gelu":
        fn = lambda g: g * 0.5 * torch.erfc(-g / math.sqrt(2))  # noqa: E731
        d = lambda g: 0.5 * torch.erfc(-g / math.sqrt(2)) + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)  # noqa: E731
    else:
        c = 2 * math.sqrt(2 / math.pi)
        fn = lambda g: g * torch.sigmoid(c * (g + 0.044715 * g ** 3))  # noqa: E731

        def d(g):
            t = torch.sigmoid(c * (g + 0.044715 * g ** 3))
            return t + g * t * (1 - t) * c * (1 + 0.134145 * g ** 2)
    if case["op"] == "glu":
        sx = 1.0 if s["xs"] is None else s["xs"].double()[:, None]
        g = torch.matmul(x, _weight64(s["vg"], s["ig"], cols, ns).t()) * (s["gs"] * sx)
        u = torch.matmul(x, _weight64(s["vu"], s["iu"], cols, ns).t()) * (s["us"] * sx)
        return {"h": fn(g) * u, "g": g, "u": u} if case["save"] else {"h": fn(g) * u}
    dy = s["dy"].double()
    if case["op"] == "spmm_bwd":
        return {"dx": torch.matmul(dy, _weight64(s["vw"], s["iw"], cols, 0)),
                "dv": _take64(torch.matmul(dy.t(), x), s["iw"], cols // 2)}
    g, u = s["gate"].double(), s["up"].double()
    dg, du = dy * u * d(g), dy * fn(g)
    return {"dx": torch.matmul(dg, _weight64(s["vg"], s["ig"], cols, 0)) +
            torch.matmul(du, _weight64(s["vu"], s["iu"], cols, 0)),
            "dvg": _take64(torch.matmul(dg.t(), x), s["ig"], cols // 2),
            "dvu": _take64(torch.matmul(du.t(), x), s["iu"], cols // 2)}
