"""The operators around the SSD core in a Mamba-2 decoder, as they are timed and checked.

Kinds of cases:

  norm        RMS norm with the residual's addition              ssd_rms_norm
  norm_mx     the same with an 8-bit output and block scales     ssd_rms_norm_mx
  norm_bwd    its gradients                                      ssd_rms_norm_bwd
  linear      act(x W^T + bias) + residual                       ssd_linear
  linear_bwd  its gradients                                      ssd_linear_bwd
  linear_mx   the same from 8-bit operands with block scales     ssd_mx_quantize, ssd_linear_mx
  select      beam search's choice of the next tokens            ssd_beam_select
  step        the decode step from the chosen beams' states      ssd_step_beam

Every kind has a plain form in elementary torch operations (run with own = False), the
framework's call (own = True), and a definition in 64 bits (exact).
"""
import math

import torch

own = False

EPS = 1e-5
LINEAR_FLOPS = 2.9e11   # the largest matrix work of a drawn case
NORM_VALUES = 1 << 26   # the largest row-times-column count of a drawn norm


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # one token of one sequence between two layers of the 1.3B shape: latency is all of it
        {"name": "norm_one_token", "kind": "norm", "rows": 1, "dim": 2048, "groups": 1, "dtype": "bf16",
         "residual": "bf16"},
        # a prompt batch (4 x 2048 tokens) of the 1.3B layer, an fp32 residual stream, 8 bits for the projection
        {"name": "norm_mx_prompt", "kind": "norm_mx", "rows": 8192, "dim": 2048, "groups": 1, "dtype": "bf16",
         "residual": "f32"},
        # training the 125M layer (8 x 2048 tokens): gradients of the norm before its output projection
        {"name": "norm_bwd_125m", "kind": "norm_bwd", "rows": 16384, "dim": 1536, "groups": 1, "dtype": "bf16",
         "residual": "bf16"},
        # decoding 8 sequences: the 1.3B layer's input projection (z, x, B, C, dt in one), bound by its weights
        {"name": "linear_decode", "kind": "linear", "rows": 8, "in": 2048, "out": 8512, "dtype": "bf16",
         "act": "none", "bias": False, "residual": False},
        # a prompt batch of the 1.3B layer's output projection, added to the residual stream
        {"name": "linear_prompt", "kind": "linear", "rows": 8192, "in": 4096, "out": 2048, "dtype": "bf16",
         "act": "none", "bias": False, "residual": True},
        # odd sizes in fp32, with every part of the epilogue
        {"name": "linear_odd_f32", "kind": "linear", "rows": 777, "in": 1003, "out": 515, "dtype": "f32",
         "act": "gelu", "bias": True, "residual": True},
        # training the 125M layer's input projection (8 x 2048 tokens), a SiLU behind it
        {"name": "linear_bwd_125m", "kind": "linear_bwd", "rows": 16384, "in": 768, "out": 3352, "dtype": "bf16",
         "act": "silu", "bias": True},
        # a prompt batch of the 1.3B layer's input projection in 8 bits
        {"name": "linear_mx_prompt", "kind": "linear_mx", "rows": 8192, "in": 2048, "out": 8512, "act": "none",
         "bias": False, "residual": False},
        # one sequence with four beams
        {"name": "select_one_sequence", "kind": "select", "batch": 1, "beams": 4, "vocab": 50257, "dtype": "bf16",
         "masked": False, "finished": False},
        # a serving batch: forbidden tokens and finished beams among it
        {"name": "select_batch", "kind": "select", "batch": 64, "beams": 8, "vocab": 65536, "dtype": "f32",
         "masked": True, "finished": True},
        # two sequences of four beams through the 125M layer's step, with its convolution and gate
        {"name": "step_small", "kind": "step", "batch": 2, "beams": 4, "heads": 24, "headdim": 64, "state": 128,
         "groups": 1, "dtype": "bf16", "fused": True},
        # the decode benchmark's 256 states of 64 heads, as 32 sequences of 8 beams
        {"name": "step_batch", "kind": "step", "batch": 32, "beams": 8, "heads": 64, "headdim": 64, "state": 128,
         "groups": 1, "dtype": "bf16", "fused": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["norm", "norm_mx", "norm_bwd", "linear", "linear", "linear_bwd", "linear_mx", "select", "step"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if kind.startswith("norm"):
        groups = rng.choice([1, 1, 2, 8])
        per = _log(rng, 48, 8192 // groups)
        if kind == "norm_mx":
            per = 32 * max(1, per // 32)
        elif rng.random() < 0.6:
            per = 8 * max(1, per // 8)
        dim = per * groups
        rows = min(_log(rng, 1, 32768), max(1, NORM_VALUES // dim))
        residual = "f32" if dtype == "f32" else rng.choice(["bf16", "f32"])
        return {"kind": kind, "rows": rows, "dim": dim, "groups": groups, "dtype": dtype, "residual": residual}
    if kind.startswith("linear"):
        rows = _log(rng, 1, 16384)
        k, n = _log(rng, 64, 8192), _log(rng, 64, 16384)
        if kind == "linear_mx":
            k = 32 * max(1, k // 32)
        elif rng.random() < 0.7:
            k, n = 8 * max(1, k // 8), 8 * max(1, n // 8)
        most = LINEAR_FLOPS / (8 if dtype == "f32" and kind != "linear_mx" else 1)
        most /= 3 if kind == "linear_bwd" else 1
        rows = max(1, min(rows, int(most / (2.0 * k * n))))
        case = {"kind": kind, "rows": rows, "in": k, "out": n, "act": rng.choice(["none", "silu", "gelu"]),
                "bias": rng.random() < 0.5}
        if kind != "linear_mx":
            case["dtype"] = dtype
        if kind != "linear_bwd":
            case["residual"] = rng.random() < 0.5
        return case
    if kind == "select":
        beams = rng.choice([1, 2, 3, 4, 5, 8, 12, 16])
        vocab = _log(rng, 1000, 131072)
        batch = min(_log(rng, 1, 256), max(1, (64 * 8 * 65536) // (beams * vocab)))
        return {"kind": kind, "batch": batch, "beams": beams, "vocab": vocab, "dtype": dtype,
                "masked": rng.random() < 0.5, "finished": rng.random() < 0.5}
    beams = rng.choice([1, 2, 3, 4, 5, 8])
    heads, headdim, state = rng.choice([8, 24, 32, 64]), rng.choice([16, 32, 50, 64, 128]), rng.choice([16, 32, 64, 128, 256])
    batch = min(_log(rng, 1, 64), max(1, (256 * 64 * 64 * 128) // (beams * heads * headdim * state)))
    return {"kind": kind, "batch": batch, "beams": beams, "heads": heads, "headdim": headdim, "state": state,
            "groups": rng.choice([1, 2, 8]), "dtype": dtype, "fused": rng.random() < 0.5}


# --------------------------------------------------------------------------- inputs
def _type(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _quantised(t):
    """8-bit weights as a user's program keeps them: (e4m3 values, e8m0 scales), 32 to a scale."""
    blocks = t.reshape(t.shape[0], -1, 32)
    p = _scale_exponent(blocks.abs().amax(-1))
    q = torch.ldexp(blocks, -p[..., None].to(blocks.dtype)).to(torch.float8_e4m3fn).reshape(t.shape)
    return q, (p + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _scale_exponent(largest):
    """The smallest whole p >= -127 with largest <= 448 * 2^p (448 = 0.875 * 2^9)."""
    m, e = torch.frexp(largest)
    p = torch.where(m > 0.875, e - 8, e - 9)
    return torch.where(largest > 0, p, torch.full_like(p, -127)).clamp(min=-127)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype=torch.float32, scale=1.0):
        return (torch.randn(*shape, device="cuda", generator=g) * scale).to(dtype)

    def uniform(*shape):
        return torch.rand(*shape, device="cuda", generator=g)

    s = dict(case)
    kind = case["kind"]
    if kind.startswith("norm"):
        rows, dim, dtype, rtype = case["rows"], case["dim"], _type(case["dtype"]), _type(case["residual"])
        s["weight"] = 1.0 + normal(dim, scale=0.1)
        if kind == "norm_bwd":
            s["h"] = normal(rows, dim, dtype=rtype, scale=2.0)
            s["dy"] = normal(rows, dim, dtype=dtype)
            s["dres"] = normal(rows, dim, dtype=rtype)
            grouped = s["h"].double().reshape(rows, case["groups"], -1)
            s["rstd"] = (grouped.square().mean(-1) + EPS).rsqrt().float()
        else:
            s["x"] = normal(rows, dim, dtype=dtype)
            s["residual_in"] = normal(rows, dim, dtype=rtype, scale=2.0)
    elif kind.startswith("linear"):
        rows, k, n = case["rows"], case["in"], case["out"]
        dtype = _type(case.get("dtype", "bf16"))
        s["x"] = normal(rows, k, dtype=dtype)
        w = normal(n, k, scale=k ** -0.5)
        if kind == "linear_mx":
            s["wq"], s["wscale"] = _quantised(w)
        else:
            s["w"] = w.to(dtype)
        s["b"] = normal(n, scale=0.5) if case["bias"] else None
        s["r"] = normal(rows, n, dtype=dtype) if case.get("residual") else None
        if kind == "linear_bwd":
            s["dy"] = normal(rows, n, dtype=dtype)
            s["pre"] = normal(rows, n, dtype=dtype) if case["act"] != "none" else None
    elif kind == "select":
        b, k, v = case["batch"], case["beams"], case["vocab"]
        s["logits"] = normal(b, k, v, dtype=_type(case["dtype"]), scale=3.0)
        if case["masked"]:  # forbidden tokens
            s["logits"].masked_fill_(uniform(b, k, v) < 0.3, -math.inf)
        s["scores"] = -20.0 * uniform(b, k)
        s["scores"][0, 1:] = -math.inf  # a sequence that has just begun: one beam so far
        s["done"] = (uniform(b, k) < 0.2) if case["finished"] else None
        s["eos"] = v // 3
    else:
        rows, h, p, n, grp = case["batch"] * case["beams"], case["heads"], case["headdim"], case["state"], case["groups"]
        dtype = _type(case["dtype"])
        s["state_in"] = normal(rows, h, p, n)
        s["state_out"] = torch.empty_like(s["state_in"])
        # the chosen parents: rows of the same sequence, some twice and some not at all
        base = torch.arange(case["batch"], device="cuda").repeat_interleave(case["beams"]) * case["beams"]
        s["parent"] = (base + (uniform(rows) * case["beams"]).long().clamp(max=case["beams"] - 1)).int()
        s["x"] = normal(rows, h, p, dtype=dtype)
        s["A"] = -torch.exp(uniform(h) * math.log(16.0))
        s["B"] = normal(rows, grp, n, dtype=dtype, scale=n ** -0.5)
        s["C"] = normal(rows, grp, n, dtype=dtype, scale=n ** -0.5)
        s["D"] = normal(h)
        if case["fused"]:
            s["dt"] = normal(rows, h, dtype=dtype)
            s["dt_bias"] = normal(h) - 4.0
            s["z"] = normal(rows, h, p, dtype=dtype)
            s["conv_in"] = normal(rows, h * p, 3, dtype=dtype)
            s["conv_out"] = torch.empty_like(s["conv_in"])
            s["conv_w"], s["conv_b"] = normal(h * p, 4, scale=0.5), normal(h * p, scale=0.5)
        else:
            s["dt"] = torch.nn.functional.softplus(normal(rows, h) - 4.0).to(dtype)
    return s


# --------------------------------------------------------------------------- one pass
def run(s):
    return (_framework if own else _plain)(s)


def _framework(s):
    import ssd_sequence_mixing_amd as ssd
    kind = s["kind"]
    if kind == "norm":
        y, h, _ = ssd.ssd_rms_norm(s["x"], s["weight"], EPS, residual=s["residual_in"], groups=s["groups"])
        return {"y": y, "h": h}
    if kind == "norm_mx":
        q, scale, h = ssd.ssd_rms_norm_mx(s["x"], s["weight"], EPS, residual=s["residual_in"], groups=s["groups"])
        return {"q": q, "scale": scale, "h": h}
    if kind == "norm_bwd":
        dx, dh, dw = ssd.ssd_rms_norm_bwd(s["dy"], s["h"], s["weight"], s["rstd"], d_residual_out=s["dres"],
                                          groups=s["groups"])
        return {"dx": dx, "dh": dh, "dw": dw}  # dh is None where dx serves for both
    if kind == "linear":
        y, _ = ssd.ssd_linear(s["x"], s["w"], bias=s["b"], act=s["act"], residual=s["r"])
        return {"y": y}
    if kind == "linear_bwd":
        dx, dw, db = ssd.ssd_linear_bwd(s["dy"], s["x"], s["w"], act=s["act"], preact=s["pre"],
                                        want_bias=s["bias"])
        return {"dx": dx, "dw": dw, "db": db}
    if kind == "linear_mx":
        xq, xscale = ssd.ssd_mx_quantize(s["x"])
        return {"y": ssd.ssd_linear_mx(xq, xscale, s["wq"], s["wscale"], bias=s["b"], act=s["act"], residual=s["r"])}
    if kind == "select":
        scores, parent, token, done = ssd.ssd_beam_select(s["logits"], s["scores"], finished=s["done"], eos=s["eos"])
        return {"scores": scores, "parent": parent, "token": token, "done": done}
    more = dict(dt_bias=s["dt_bias"], dt_softplus=1, z=s["z"], conv_in=s["conv_in"], conv_out=s["conv_out"],
                conv_w=s["conv_w"], conv_b=s["conv_b"]) if s["fused"] else {}
    y = ssd.ssd_step_beam(s["state_in"], s["state_out"], s["parent"], s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"],
                          **more)
    return {"y": y, "state": s["state_out"], "conv": s.get("conv_out")}


def _norm(s):
    h = s["x"].float() + s["residual_in"].float()
    grouped = h.reshape(h.shape[0], s["groups"], -1)
    y = (grouped * torch.rsqrt(grouped.square().mean(-1, keepdim=True) + EPS)).reshape(h.shape) * s["weight"]
    return y, h.to(s["residual_in"].dtype)


def _silu(v):
    return v / (1.0 + torch.exp(-v))


def _act(v, act):
    if act == "silu":
        return _silu(v)
    return 0.5 * v * (1.0 + torch.erf(v * math.sqrt(0.5))) if act == "gelu" else v


def _act_slope(v, act):
    if act == "silu":
        g = 1.0 / (1.0 + torch.exp(-v))
        return g * (1.0 + v * (1.0 - g))
    return 0.5 * (1.0 + torch.erf(v * math.sqrt(0.5))) + v * torch.exp(-0.5 * v * v) / math.sqrt(2.0 * math.pi)


def _values(q, scale):
    """What 8-bit codes with a scale for each 32 stand for."""
    return (q.float().reshape(*scale.shape, 32) * scale.float()[..., None]).reshape(q.shape)


def _plain(s):
    kind = s["kind"]
    if kind == "norm":
        y, h = _norm(s)
        return {"y": y.to(s["x"].dtype), "h": h}
    if kind == "norm_mx":
        y, h = _norm(s)
        q, scale = _quantised(y)
        return {"q": q, "scale": scale, "h": h}
    if kind == "norm_bwd":
        dy, h, inv = s["dy"].float(), s["h"].float(), s["rstd"][..., None]
        shape = (h.shape[0], s["groups"], -1)
        hh = h.reshape(shape) * inv
        gw = (dy * s["weight"]).reshape(shape)
        dh = (inv * (gw - hh * (gw * hh).mean(-1, keepdim=True))).reshape(h.shape) + s["dres"].float()
        dw = (dy * hh.reshape(h.shape)).sum(0)
        same = s["dy"].dtype == s["h"].dtype
        return {"dx": dh.to(s["dy"].dtype), "dh": None if same else dh.to(s["h"].dtype), "dw": dw}
    if kind in ("linear", "linear_mx"):
        if kind == "linear":
            x, w = s["x"].float(), s["w"].float()
        else:
            x, w = _values(*_quantised(s["x"].float())), _values(s["wq"], s["wscale"])
        y = x @ w.t()
        if s["b"] is not None:
            y = y + s["b"]
        y = _act(y, s["act"])
        if s["r"] is not None:
            y = y + s["r"].float()
        return {"y": y.to(s["x"].dtype)}
    if kind == "linear_bwd":
        dz, dtype = s["dy"].float(), s["x"].dtype
        if s["pre"] is not None:
            dz = dz * _act_slope(s["pre"].float(), s["act"])
        dx, dw = dz @ s["w"].float(), dz.t() @ s["x"].float()
        return {"dx": dx.to(dtype), "dw": dw.to(dtype), "db": dz.sum(0) if s["bias"] else None}
    if kind == "select":
        return _choose(s, torch.logsumexp)
    p = s["parent"].long()
    x, dt = s["x"].float(), s["dt"].float()
    conv = None
    if s["fused"]:
        dt = torch.log1p(torch.exp(dt + s["dt_bias"]))
        window = torch.cat([s["conv_in"][p], s["x"].reshape(len(p), -1, 1)], -1)
        conv = window[..., 1:].contiguous()
        x = _silu((window.float() * s["conv_w"]).sum(-1) + s["conv_b"]).to(s["x"].dtype).float().reshape(x.shape)
    per = s["heads"] // s["groups"]
    bm, cm = (s[k].float().repeat_interleave(per, 1)[:, :, None] for k in ("B", "C"))
    state = torch.exp(dt * s["A"])[..., None, None] * s["state_in"][p] + (dt[..., None] * x)[..., None] * bm
    y = (state * cm).sum(-1) + s["D"][:, None] * x
    if s["fused"]:
        y = y * _silu(s["z"].float())
    return {"y": y.to(s["x"].dtype), "state": state, "conv": conv}


def _choose(s, logsumexp):
    """In 64 bits: neighbouring candidates can be closer than 32 bits tell apart."""
    b, k, v = s["logits"].shape
    l = s["logits"].double()
    cand = s["scores"].double()[..., None] + l - logsumexp(l, -1, keepdim=True)
    if s["done"] is not None:
        cand = cand.masked_fill(s["done"][..., None], -math.inf)
        cand[:, :, s["eos"]] = torch.where(s["done"], s["scores"].double(), cand[:, :, s["eos"]])
    best, at = torch.sort(cand.reshape(b, k * v), dim=-1, descending=True, stable=True)
    best, at = best[:, :k], at[:, :k]
    beam, token = at // v, at % v
    parent = beam + torch.arange(b, device=at.device)[:, None] * k
    done = token == s["eos"]
    if s["done"] is not None:
        done = done | s["done"].gather(1, beam)
    return {"scores": best.float(), "parent": parent.int(), "token": token.int(), "done": done}


# --------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    kind = case["kind"]
    es = 2 if case.get("dtype", "bf16") == "bf16" else 4
    if kind.startswith("norm"):
        n, rs = case["rows"] * case["dim"], 2 if case["residual"] == "bf16" else 4
        if kind == "norm":
            return {"bytes": n * (2 * es + 2 * rs) + 4 * case["dim"], "flops": 5 * n}
        if kind == "norm_mx":
            return {"bytes": n * (es + 2 * rs + 1 + 1 / 32) + 4 * case["dim"], "flops": 7 * n}
        return {"bytes": n * (2 * es + 2 * rs + (rs if rs != es else 0)) + 8 * case["dim"], "flops": 12 * n}
    if kind.startswith("linear"):
        m, k, n = case["rows"], case["in"], case["out"]
        flops = 2.0 * m * k * n
        if kind == "linear":
            return {"bytes": es * (m * k + n * k + m * n * (2 if case["residual"] else 1)), "flops": flops}
        if kind == "linear_mx":
            return {"bytes": 2 * m * k + n * k * (1 + 1 / 32) + 2 * m * n * (2 if case["residual"] else 1), "flops": flops}
        return {"bytes": es * (2 * m * k + 2 * n * k + m * n * (1 if case["act"] == "none" else 2)), "flops": 2 * flops}
    if kind == "select":
        return {"bytes": case["batch"] * case["beams"] * (case["vocab"] * es + 17), "flops": 4 * case["batch"] * case["beams"] * case["vocab"]}
    rows = case["batch"] * case["beams"]
    n = rows * case["heads"] * case["headdim"]
    small = n * 2 * es + rows * case["groups"] * case["state"] * 2 * es + (n * 7 * es if case["fused"] else 0)
    return {"bytes": 8 * n * case["state"] + small, "flops": 5 * n * case["state"]}


# --------------------------------------------------------------------------- the definition in 64 bits
def _round_e4m3(u):
    """The nearest e4m3 value (3 bits of mantissa, exponents from -6, ties to even) to |u| <= 448."""
    step = torch.exp2(torch.floor(torch.log2(u.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(u / step) * step


def _to_blocks(t):
    """(values in 8 bits, their scales) of t in 64 bits, from the definition."""
    blocks = t.reshape(t.shape[0], -1, 32)
    top = blocks.abs().amax(-1, keepdim=True)
    scale = torch.exp2(torch.ceil(torch.log2(top / 448.0)).clamp(min=-127))
    scale = torch.where(top > 448.0 * scale, 2 * scale, torch.where((top <= 224.0 * scale) & (scale > 2.0 ** -127), scale / 2, scale))
    return _round_e4m3(blocks / scale).reshape(t.shape), scale[..., 0]


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    f = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() and "float8" not in str(v.dtype) else v
         for k, v in s.items() if k not in ("state_out", "conv_out")}
    if kind in ("norm", "norm_mx"):
        h = f["x"] + f["residual_in"]
        parts = h.unflatten(1, (case["groups"], -1))
        y = (parts / torch.sqrt((parts * parts).sum(-1, keepdim=True) / parts.shape[-1] + EPS)).flatten(1) * f["weight"]
        if kind == "norm":
            return {"y": y, "h": h}
        q, scale = _to_blocks(y)
        return {"q": q, "scale": scale, "h": h}
    if kind == "norm_bwd":
        parts, inv = f["h"].unflatten(1, (case["groups"], -1)), f["rstd"][..., None]
        up = (f["dy"] * f["weight"]).unflatten(1, (case["groups"], -1))
        along = (up * parts).sum(-1, keepdim=True) / parts.shape[-1]
        dh = (up * inv - parts * along * inv ** 3).flatten(1) + f["dres"]
        dw = (f["dy"] * (parts * inv).flatten(1)).sum(0)
        return {"dx": dh, "dh": None if s["dy"].dtype == s["h"].dtype else dh, "dw": dw}
    if kind.startswith("linear"):
        x = f["x"]
        if kind == "linear_mx":
            q, scale = _to_blocks(x)
            x = q * scale.repeat_interleave(32, 1)
            w = s["wq"].float().double() * s["wscale"].float().double().repeat_interleave(32, 1)
        else:
            w = f["w"]
        if kind == "linear_bwd":
            dz, v = f["dy"], f["pre"]
            if case["act"] == "silu":
                dz = dz * (torch.sigmoid(v) + v * torch.sigmoid(v) * torch.sigmoid(-v))
            elif case["act"] == "gelu":
                dz = dz * (0.5 * torch.erfc(-v / math.sqrt(2.0)) + v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi))
            return {"dx": torch.mm(dz, w), "dw": torch.mm(dz.t().contiguous(), x), "db": dz.sum(0) if case["bias"] else None}
        y = torch.mm(x, w.t().contiguous())
        if f["b"] is not None:
            y += f["b"]
        if case["act"] == "silu":
            y = y * torch.sigmoid(y)
        elif case["act"] == "gelu":
            y = y * 0.5 * torch.erfc(-y / math.sqrt(2.0))
        return {"y": y if f["r"] is None else y + f["r"]}
    if kind == "select":
        top = f["logits"].amax(-1, keepdim=True)
        top = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
        lse = top + torch.log(torch.exp(f["logits"] - top).sum(-1, keepdim=True))
        cand = f["scores"][..., None] + (f["logits"] - lse)
        if s["done"] is not None:
            only = torch.full_like(cand, -math.inf)
            only[..., s["eos"]] = f["scores"]
            cand = torch.where(s["done"][..., None], only, cand)
        return {"scores": torch.topk(cand.flatten(1), case["beams"]).values, "parent": None, "token": None, "done": None}
    rows = s["parent"].long()
    x, dt, conv = f["x"], f["dt"], None
    if case["fused"]:
        dt = torch.nn.functional.softplus(dt + f["dt_bias"])
        old, now = f["conv_in"][rows], f["x"].flatten(1)
        conv = torch.stack([old[..., 1], old[..., 2], now], -1)
        w = f["conv_w"]
        v = f["conv_b"] + w[:, 0] * old[..., 0] + w[:, 1] * old[..., 1] + w[:, 2] * old[..., 2] + w[:, 3] * now
        x = (v * torch.sigmoid(v)).to(s["x"].dtype).double().unflatten(1, x.shape[1:])
    group = torch.arange(case["heads"], device=x.device) * case["groups"] // case["heads"]
    bm, cm = f["B"][:, group], f["C"][:, group]
    state = torch.exp(dt * f["A"])[..., None, None] * f["state_in"][rows]
    state += (dt[..., None] * x)[..., None] * bm[:, :, None]
    y = (state @ cm[..., None])[..., 0] + f["D"][:, None] * x
    if case["fused"]:
        y = y * f["z"] * torch.sigmoid(f["z"])
    return {"y": y, "state": state, "conv": conv}
