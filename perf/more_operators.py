"""Operators of a decoder that mixes by a gated linear recurrence, from its tokens to its logits, as they are timed
and checked.

Kinds of cases:

  scan       h_t = a_t h_(t-1) + c_t sigmoid(i_t) x_t over sequences      ssd_gated_scan_fwd
  scan_bwd   its gradients                                                ssd_gated_scan_bwd
  step       one token of it, rows from their parents' states             ssd_gated_step
  embed      rows of a table, scaled                                      ssd_embedding
  embed_bwd  the table's gradient                                         ssd_embedding_bwd
  logits     penalties for repeated tokens, a bias, a grammar's mask      ssd_logits_process
  linear_int  act(x W^T + bias) + residual from 8-bit integers             ssd_int_quantize, ssd_linear_int

Every kind has a plain form in elementary torch operations (run with own = False), the framework's call
(own = True), and a definition in 64 bits (exact).
"""
import math

import torch

own = False

SCAN_VALUES = 48 << 20   # the largest batch x tokens x channels of a drawn scan
TABLE_VALUES = 1 << 27   # the largest vocabulary x channels of a drawn table
LOGITS = 1 << 25         # the largest rows x vocabulary of drawn logits
LINEAR_FLOPS = 1.37e11   # the largest matrix work of a drawn product
LINEAR_VALUES = 9 << 23  # the most values that it reads and writes by rows
CHUNK = 128              # tokens between the states that a scan keeps for its gradients


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # a prompt batch (4 x 2048 tokens) through a mixer as wide as the 1.3B layer's, learned rates, gated input
        {"name": "scan_prompt", "kind": "scan", "batch": 4, "seqlen": 2048, "dim": 4096, "dtype": "bf16",
         "decay": "rate", "in_gate": True, "resets": False, "initial": False},
        # the long-context shape (16384 tokens) of several documents laid end to end, continued from a state
        {"name": "scan_long", "kind": "scan", "batch": 1, "seqlen": 16384, "dim": 4096, "dtype": "bf16",
         "decay": "sigmoid", "in_gate": False, "resets": True, "initial": True},
        # training the 125M shape (8 x 2048 tokens, 24 heads of 64 channels)
        {"name": "scan_bwd_125m", "kind": "scan_bwd", "batch": 8, "seqlen": 2048, "dim": 1536, "dtype": "bf16",
         "decay": "rate", "in_gate": True, "resets": False, "initial": False},
        # odd sizes in fp32, given log-decays, documents laid end to end
        {"name": "scan_bwd_odd_f32", "kind": "scan_bwd", "batch": 3, "seqlen": 1000, "dim": 515, "dtype": "f32",
         "decay": "log", "in_gate": True, "resets": True, "initial": True},
        # decoding two sequences of four beams through the 125M shape: latency is all of it
        {"name": "step_small", "kind": "step", "rows": 8, "dim": 1536, "dtype": "bf16", "decay": "rate", "in_gate": True},
        # a prompt batch's tokens into an fp32 residual stream of the 1.3B shape
        {"name": "embed_prompt", "kind": "embed", "rows": 8192, "vocab": 50257, "dim": 2048, "dtype": "bf16", "out": "f32",
         "scaled": True, "padded": False},
        # training the 125M shape: the table's gradient, tokens as frequent as words are
        {"name": "embed_bwd_125m", "kind": "embed_bwd", "rows": 16384, "vocab": 50257, "dim": 768, "dtype": "bf16",
         "grad": "f32", "scaled": True, "padded": False},
        # a small vocabulary (bytes and marks), so that every row of the table sums many; padded sequences
        {"name": "embed_bwd_bytes", "kind": "embed_bwd", "rows": 16384, "vocab": 259, "dim": 1003, "dtype": "f32",
         "grad": "f32", "scaled": False, "padded": True},
        # one sequence of four beams: latency
        {"name": "logits_one_sequence", "kind": "logits", "rows": 4, "vocab": 50257, "history": 512, "dtype": "bf16",
         "bias": "none", "mask": "none"},
        # a serving batch of 64 sequences of 8 beams, a bias for all and a grammar for each
        {"name": "logits_batch", "kind": "logits", "rows": 512, "vocab": 65536, "history": 2048, "dtype": "f32",
         "bias": "one", "mask": "rows"},
        # decoding 8 sequences: the 1.3B layer's input projection, bound by its weights
        {"name": "linear_int_decode", "kind": "linear_int", "rows": 8, "in": 2048, "out": 8512, "dtype": "bf16", "act": "none",
         "bias": False, "residual": False},
        # a prompt batch of the 1.3B layer's output projection, added to the residual stream
        {"name": "linear_int_prompt", "kind": "linear_int", "rows": 8192, "in": 4096, "out": 2048, "dtype": "bf16",
         "act": "none", "bias": True, "residual": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _eights(rng, n, odd=0.4):
    return n if rng.random() < odd else 8 * max(1, n // 8)


def draw(rng):
    kind = rng.choice(["scan", "scan", "scan_bwd", "scan_bwd", "step", "embed", "embed_bwd", "embed_bwd", "logits", "logits",
                       "linear_int", "linear_int"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if kind in ("scan", "scan_bwd"):
        most = SCAN_VALUES // (2 if kind == "scan_bwd" else 1) // (2 if dtype == "f32" else 1)
        dim, seqlen = _eights(rng, _log(rng, 48, 4096)), _log(rng, 1, 16384)
        batch = max(1, min(_log(rng, 1, 16), most // (seqlen * dim)))
        seqlen = min(seqlen, most // (batch * dim))
        return {"kind": kind, "batch": batch, "seqlen": seqlen, "dim": dim, "dtype": dtype,
                "decay": rng.choice(["rate", "sigmoid", "log"]), "in_gate": rng.random() < 0.6,
                "resets": rng.random() < 0.4, "initial": rng.random() < 0.5}
    if kind == "step":
        return {"kind": kind, "rows": _log(rng, 1, 512), "dim": _eights(rng, _log(rng, 48, 8192)), "dtype": dtype,
                "decay": rng.choice(["rate", "sigmoid", "log"]), "in_gate": rng.random() < 0.6}
    if kind in ("embed", "embed_bwd"):
        vocab, dim = _log(rng, 200, 131072), _eights(rng, _log(rng, 48, 4096))
        vocab = min(vocab, TABLE_VALUES // dim // (2 if kind == "embed_bwd" else 1))
        rows = min(_log(rng, 1, 65536), (1 << 24) // dim)
        return {"kind": kind, "rows": rows, "vocab": vocab, "dim": dim, "dtype": dtype,
                "out" if kind == "embed" else "grad": rng.choice([dtype, "f32"]), "scaled": rng.random() < 0.5,
                "padded": rng.random() < 0.5}
    if kind == "logits":
        vocab = _log(rng, 1000, 131072)
        bias = rng.choice(["none", "one", "rows"])
        rows = min(_log(rng, 1, 512), LOGITS // vocab // (2 if bias == "rows" else 1))
        return {"kind": kind, "rows": rows, "vocab": vocab, "history": _log(rng, 1, 8192), "dtype": dtype, "bias": bias,
                "mask": rng.choice(["none", "one", "rows"])}
    k, n = 16 * _log(rng, 4, 512), _eights(rng, _log(rng, 64, 16384))
    rows = max(1, min(_log(rng, 1, 16384), int(LINEAR_FLOPS / (2.0 * k * n)), LINEAR_VALUES // (k + 2 * n)))
    return {"kind": kind, "rows": rows, "in": k, "out": n, "dtype": dtype, "act": rng.choice(["none", "silu", "gelu"]),
            "bias": rng.random() < 0.5, "residual": rng.random() < 0.5}


# --------------------------------------------------------------------------- inputs
def _type(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _codes(x):
    """8-bit integers with a scale for each row: the nearest to x / scale (in 64 bits: two codes' border is decided)."""
    scale = (x.float().abs().amax(-1) / 127.0)[:, None]
    q = torch.round(x.double() / scale.double())
    return torch.where(scale > 0, q, torch.zeros_like(q)).to(torch.int8), scale[:, 0]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype=torch.float32, scale=1.0):
        return (torch.randn(*shape, device="cuda", generator=g) * scale).to(dtype)

    def uniform(*shape):
        return torch.rand(*shape, device="cuda", generator=g)

    def words(*shape, vocab):  # as frequent as words are: the k-th about 1 / k
        return (torch.exp(uniform(*shape) * math.log(vocab + 1.0)) - 1.0).int().clamp(max=vocab - 1)

    s = dict(case)
    kind = case["kind"]
    dtype = _type(case["dtype"])
    if kind in ("scan", "scan_bwd", "step"):
        d = case["dim"]
        shape = (case["rows"], d) if kind == "step" else (case["batch"], case["seqlen"], d)
        s["x"] = normal(*shape, dtype=dtype)
        # the recurrence's memory: some 10 to 1000 tokens
        if case["decay"] == "log":
            s["f"] = (-0.1 * torch.exp(normal(*shape, scale=1.5))).to(dtype)
        else:
            s["f"] = normal(*shape, dtype=dtype) if case["decay"] == "rate" else (3.0 + normal(*shape)).to(dtype)
        s["rate"] = torch.log(0.9 + 0.099 * uniform(d)) if case["decay"] == "rate" else None
        s["i"] = normal(*shape, dtype=dtype) if case["in_gate"] else None
        if kind == "step":
            s["state_in"], s["state_out"] = normal(*shape), torch.empty(*shape, device="cuda")
            s["parent"] = (uniform(shape[0]) * shape[0]).int().clamp(max=shape[0] - 1)
            return s
        s["reset"] = (uniform(*shape[:2]) < 1 / 500) if case["resets"] else None
        s["h0"] = normal(shape[0], d) if case["initial"] else None
        if kind == "scan_bwd":
            s["dy"] = normal(*shape, dtype=dtype)
            s["dfinal"] = normal(shape[0], d) if case["initial"] else None
            # the states before each chunk's first token, as the forward pass leaves them
            h = _states64(s)
            first = s["h0"].double() if case["initial"] else torch.zeros_like(h[:, 0])
            s["states"] = torch.cat([first[:, None], h[:, CHUNK - 1:-1:CHUNK]], 1).float()
    elif kind in ("embed", "embed_bwd"):
        s["tokens"] = words(case["rows"], vocab=case["vocab"])
        if case["padded"]:  # a third of the places hold no token
            s["tokens"].masked_fill_(uniform(case["rows"]) < 1 / 3, -1)
        s["scale"] = math.sqrt(case["dim"]) if case["scaled"] else 1.0
        if kind == "embed":
            s["table"] = normal(case["vocab"], case["dim"], dtype=dtype, scale=case["dim"] ** -0.5)
        else:
            s["dy"] = normal(case["rows"], case["dim"], dtype=dtype)
    elif kind == "logits":
        rows, v, n = case["rows"], case["vocab"], case["history"]
        s["l"] = normal(rows, v, dtype=dtype, scale=3.0)
        s["tokens"] = words(rows, n, vocab=v)
        s["lengths"] = (uniform(rows) * (n + 1)).int().clamp(max=n)
        s["prompt"] = (uniform(rows) * 0.5 * n).int()
        s["repetition"], s["presence"], s["frequency"] = 1.0 + uniform(rows), uniform(rows), 0.5 * uniform(rows)
        many = {"none": 0, "one": 1, "rows": rows}
        s["b"] = normal(many[case["bias"]], v, scale=0.5) if case["bias"] != "none" else None
        s["m"] = None
        if case["mask"] != "none":  # 32 tokens to a word; grammars allow few or many
            m = torch.zeros(many[case["mask"]], -(-v // 32), dtype=torch.int64, device="cuda")
            allowed = uniform(m.shape[0], 1)
            for bit in range(32):
                m |= (uniform(*m.shape) < allowed).long() << bit
            s["m"] = torch.where(m >= 1 << 31, m - (1 << 32), m).int()
    else:
        rows, k, n = case["rows"], case["in"], case["out"]
        s["x"] = normal(rows, k, dtype=dtype)
        s["wq"], s["wscale"] = _codes(normal(n, k, scale=k ** -0.5))
        s["b"] = normal(n, scale=0.5) if case["bias"] else None
        s["r"] = normal(rows, n, dtype=dtype) if case["residual"] else None
    return s


# --------------------------------------------------------------------------- one pass
def run(s):
    return (_framework if own else _plain)(s)


def _framework(s):
    import ssd_sequence_mixing_amd as ssd
    kind = s["kind"]
    if kind == "scan":
        y, final, _ = ssd.ssd_gated_scan_fwd(s["x"], s["f"], decay=s["decay"], rate=s["rate"], in_gate=s["i"],
                                             reset=s["reset"], initial_state=s["h0"])
        return {"y": y, "final": final}
    if kind == "scan_bwd":
        dx, df, di, drate, dh0 = ssd.ssd_gated_scan_bwd(s["dy"], s["x"], s["f"], s["states"], decay=s["decay"],
                                                        rate=s["rate"], in_gate=s["i"], reset=s["reset"],
                                                        d_final_state=s["dfinal"])
        return {"dx": dx, "df": df, "di": di, "drate": drate, "dh0": dh0}
    if kind == "step":
        y = ssd.ssd_gated_step(s["state_in"], s["state_out"], s["x"], s["f"], decay=s["decay"], rate=s["rate"],
                               in_gate=s["i"], parent=s["parent"])
        return {"y": y, "state": s["state_out"]}
    if kind == "embed":
        return {"y": ssd.ssd_embedding(s["tokens"], s["table"], scale=s["scale"], dtype=_type(s["out"]))}
    if kind == "embed_bwd":
        return {"dtable": ssd.ssd_embedding_bwd(s["dy"], s["tokens"], s["vocab"], scale=s["scale"], dtype=_type(s["grad"]))}
    if kind == "logits":
        return {"y": ssd.ssd_logits_process(s["l"], tokens=s["tokens"], lengths=s["lengths"], prompt=s["prompt"],
                                            repetition=s["repetition"], presence=s["presence"], frequency=s["frequency"],
                                            bias=s["b"], mask=s["m"])}
    xq, xscale = ssd.ssd_int_quantize(s["x"])
    return {"y": ssd.ssd_linear_int(xq, xscale, s["wq"], s["wscale"], bias=s["b"], act=s["act"], residual=s["r"],
                                   dtype=s["x"].dtype)}


def _sigmoid(v):
    return 1.0 / (1.0 + torch.exp(-v))


def _coefficients(s):
    """(a, c, sigmoid(i) x) of a recurrence in fp32."""
    f, x = s["f"].float(), s["x"].float()
    if s["decay"] == "log":
        a, c = torch.exp(f), torch.ones_like(f)
    elif s["decay"] == "sigmoid":
        a, c = _sigmoid(f), _sigmoid(-f)
    else:
        la = s["rate"] * _sigmoid(f)
        a, c = torch.exp(la), torch.sqrt(-torch.expm1(2.0 * la))
    return a, c, x if s["i"] is None else _sigmoid(s["i"].float()) * x


def _doubling(a, u):
    """All h_t = a_t h_(t-1) + u_t along dimension 1, in steps of 1, 2, 4 ..."""
    step = 1
    while step < a.shape[1]:
        u = torch.cat([u[:, :step], u[:, step:] + a[:, step:] * u[:, :-step]], 1)
        if 2 * step < a.shape[1]:
            a = torch.cat([a[:, :step], a[:, step:] * a[:, :-step]], 1)
        step *= 2
    return u


def _act(v, act):
    if act == "silu":
        return v * _sigmoid(v)
    return 0.5 * v * (1.0 + torch.erf(v * math.sqrt(0.5))) if act == "gelu" else v


def _counts(s):
    """How often each row has each token: in all of its history, and behind the prompt."""
    at = torch.arange(s["tokens"].shape[1], device=s["tokens"].device)
    lived = (at < s["lengths"][:, None]).float()
    zero = torch.zeros(s["l"].shape, device=at.device)
    return (zero.scatter_add(1, s["tokens"].long(), lived),
            zero.scatter_add(1, s["tokens"].long(), lived * (at >= s["prompt"][:, None]).float()))


def _allowed(s):
    return ((s["m"][:, :, None] >> torch.arange(32, device=s["m"].device, dtype=torch.int32)) & 1).flatten(1)[:, :s["vocab"]] != 0


def _plain(s):
    kind = s["kind"]
    if kind in ("scan", "scan_bwd"):
        dtype = s["x"].dtype
        a, c, v = _coefficients(s)
        kept = a if s["reset"] is None else a.masked_fill(s["reset"][..., None], 0.0)
        u = c * v
        first = s["h0"] if kind == "scan" else s["states"][:, 0]
        if first is not None:
            u = torch.cat([u[:, :1] + kept[:, :1] * first[:, None], u[:, 1:]], 1)
        h = _doubling(kept, u)
        if kind == "scan":
            return {"y": h.to(dtype), "final": h[:, -1].clone()}
        before = torch.cat([s["states"][:, :1], h[:, :-1]], 1)
        dy = s["dy"].float()
        if s["dfinal"] is not None:
            dy = torch.cat([dy[:, :-1], dy[:, -1:] + s["dfinal"][:, None]], 1)
        # g_t = dy_t + a_(t+1) g_(t+1)
        later = torch.cat([kept[:, 1:], torch.zeros_like(kept[:, :1])], 1)
        g = _doubling(later.flip(1), dy.flip(1)).flip(1)
        out = {"dx": g * c, "di": None, "drate": None, "dh0": kept[:, 0] * g[:, 0]}
        if s["i"] is not None:
            gate = _sigmoid(s["i"].float())
            out["dx"] = out["dx"] * gate
            out["di"] = (g * c * v * (1.0 - gate)).to(dtype)
        out["dx"] = out["dx"].to(dtype)
        dla = g * kept * before
        if s["decay"] == "sigmoid":
            dla = (dla - g * a * v) * c   # c = 1 - a
        elif s["decay"] == "rate":
            dla = dla - g * v * a * a / c
            gate = _sigmoid(s["f"].float())
            out["drate"] = (dla * gate).sum((0, 1))
            dla = dla * s["rate"] * gate * _sigmoid(-s["f"].float())
        out["df"] = dla.to(dtype)
        return out
    if kind == "step":
        a, c, v = _coefficients(s)
        state = a * s["state_in"][s["parent"].long()] + c * v
        return {"y": state.to(s["x"].dtype), "state": state}
    if kind == "embed":
        t = s["tokens"].long()
        y = s["table"][t.clamp(min=0)].float() * s["scale"]
        return {"y": y.masked_fill((t < 0)[:, None], 0.0).to(_type(s["out"]))}
    if kind == "embed_bwd":
        t = s["tokens"].long()
        table = torch.zeros(s["vocab"] + 1, s["dim"], device=t.device)  # one row more for the places without a token
        table.index_add_(0, torch.where(t < 0, s["vocab"], t), s["dy"].float())
        return {"dtable": (table[:-1] * s["scale"]).to(_type(s["grad"]))}
    if kind == "logits":
        every, said = _counts(s)
        l = s["l"].float()
        rep = s["repetition"][:, None]
        l = torch.where(every > 0, torch.where(l > 0, l / rep, l * rep), l)
        l = l - s["frequency"][:, None] * said - s["presence"][:, None] * (said > 0).float()
        if s["b"] is not None:
            l = l + s["b"]
        if s["m"] is not None:
            l = l.masked_fill(~_allowed(s), -math.inf)
        return {"y": l.to(s["l"].dtype)}
    xq, xscale = _codes(s["x"])
    y = (xq.float() @ s["wq"].float().t()) * xscale[:, None] * s["wscale"]
    if s["b"] is not None:
        y = y + s["b"]
    y = _act(y, s["act"])
    if s["r"] is not None:
        y = y + s["r"].float()
    return {"y": y.to(s["x"].dtype)}


# --------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    kind = case["kind"]
    es = 2 if case["dtype"] == "bf16" else 4
    if kind in ("scan", "scan_bwd"):
        n = case["batch"] * case["seqlen"] * case["dim"]
        gates = 2 if case["in_gate"] else 1
        state = 4 * case["batch"] * case["dim"] * (2 if case["initial"] else 1)
        if kind == "scan":
            return {"bytes": n * es * (2 + gates) + state, "flops": 12 * n}
        kept = 4 * case["batch"] * -(-case["seqlen"] // CHUNK) * case["dim"]
        return {"bytes": n * es * (3 + 2 * gates) + state + kept, "flops": 30 * n}
    if kind == "step":
        n = case["rows"] * case["dim"]
        return {"bytes": n * (8 + es * (4 if case["in_gate"] else 3)), "flops": 12 * n}
    if kind == "embed":
        n, out = case["rows"] * case["dim"], 2 if case["out"] == "bf16" else 4
        return {"bytes": min(n, case["vocab"] * case["dim"]) * es + n * out + 4 * case["rows"], "flops": n}
    if kind == "embed_bwd":
        n, out = case["rows"] * case["dim"], 2 if case["grad"] == "bf16" else 4
        return {"bytes": n * es + case["vocab"] * case["dim"] * out + 4 * case["rows"], "flops": n}
    if kind == "logits":
        n, v = case["rows"] * case["vocab"], case["vocab"]
        many = {"none": 0, "one": 1, "rows": case["rows"]}
        extra = 4 * v * many[case["bias"]] + v / 8 * many[case["mask"]] + 4 * case["rows"] * case["history"]
        return {"bytes": 2 * n * es + extra, "flops": 4 * n}
    m, k, n = case["rows"], case["in"], case["out"]
    return {"bytes": es * m * k + n * k + es * m * n * (2 if case["residual"] else 1), "flops": 2.0 * m * k * n}


# --------------------------------------------------------------------------- the definition in 64 bits
def _gate64(v):
    return torch.sigmoid(v.double())


def _decay64(s):
    """(log a, c) in 64 bits."""
    f = s["f"].double()
    if s["decay"] == "log":
        return f, torch.ones_like(f)
    if s["decay"] == "sigmoid":
        return torch.nn.functional.logsigmoid(f), torch.sigmoid(-f)
    la = s["rate"].double() * torch.sigmoid(f)
    return la, (-torch.expm1(2 * la)).sqrt()


def _input64(s):
    return s["x"].double() * (1.0 if s["i"] is None else _gate64(s["i"]))


def _states64(s):
    """Every h_t, token by token."""
    la, c = _decay64(s)
    a, u = torch.exp(la), c * _input64(s)
    if s["reset"] is not None:
        a[s["reset"]] = 0
    h = torch.empty_like(u)
    last = s["h0"].double() if s["h0"] is not None else torch.zeros_like(u[:, 0])
    for t in range(u.shape[1]):
        last = torch.addcmul(u[:, t], a[:, t], last)
        h[:, t] = last
    return h


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "scan":
        h = _states64(s)
        return {"y": h, "final": h[:, -1].clone()}
    if kind == "scan_bwd":
        la, c = _decay64(s)
        a, x = torch.exp(la), s["x"].double()
        carried = a.clone()
        if s["reset"] is not None:
            carried[s["reset"]] = 0
        # what the call is given: the states before each chunk, which it goes on from
        h0, n = s["states"], case["seqlen"]
        prev, h = torch.empty_like(a), None
        u = c * _input64(s)
        for t in range(n):
            h = h0[:, t // CHUNK].double() if t % CHUNK == 0 else h
            prev[:, t] = h
            h = carried[:, t] * h + u[:, t]
        g = torch.empty_like(a)
        back = s["dfinal"].double() if s["dfinal"] is not None else torch.zeros_like(a[:, 0])
        for t in range(n - 1, -1, -1):
            g[:, t] = s["dy"][:, t].double() + back
            back = carried[:, t] * g[:, t]
        gate = 1.0 if s["i"] is None else _gate64(s["i"])
        out = {"dx": g * c * gate, "di": None, "drate": None, "dh0": back}
        if s["i"] is not None:
            out["di"] = g * c * x * gate * (1 - gate)
        slope = {"log": 0.0, "sigmoid": -a, "rate": -a * a / c}[s["decay"]]  # of c, for log a
        dla = g * (carried * prev + slope * gate * x)
        if s["decay"] == "log":
            out["df"] = dla
        elif s["decay"] == "sigmoid":
            out["df"] = dla * torch.sigmoid(-s["f"].double())
        else:
            p = _gate64(s["f"])
            out["drate"] = (dla * p).sum((0, 1))
            out["df"] = dla * s["rate"].double() * p * (1 - p)
        return out
    if kind == "step":
        la, c = _decay64(s)
        state = torch.exp(la) * s["state_in"].double()[s["parent"].long()] + c * _input64(s)
        return {"y": state, "state": state}
    if kind == "embed":
        rows = torch.zeros(case["rows"], case["dim"], dtype=torch.float64, device="cuda")
        there = s["tokens"] >= 0
        rows[there] = s["table"][s["tokens"][there].long()].double() * s["scale"]
        return {"y": rows}
    if kind == "embed_bwd":
        order = torch.argsort(s["tokens"], stable=True)
        sums = torch.cumsum(s["dy"].double()[order], 0)
        sums = torch.cat([torch.zeros_like(sums[:1]), sums])
        ends = torch.searchsorted(s["tokens"][order].contiguous(), torch.arange(-1, case["vocab"], device="cuda", dtype=torch.int32), right=True)
        return {"dtable": (sums[ends[1:]] - sums[ends[:-1]]) * s["scale"]}
    if kind == "logits":
        out = s["l"].double()
        tokens, lengths, prompt = s["tokens"].cpu(), s["lengths"].tolist(), s["prompt"].tolist()
        for r in range(case["rows"]):
            seen = tokens[r, :lengths[r]].unique().long().cuda()
            said = torch.bincount(tokens[r, prompt[r]:lengths[r]], minlength=case["vocab"]).cuda() if lengths[r] > prompt[r] else None
            rep = float(s["repetition"][r])
            v = out[r, seen]
            out[r, seen] = torch.where(v > 0, v / rep, v * rep)
            if said is not None:
                out[r] -= float(s["frequency"][r]) * said + float(s["presence"][r]) * (said > 0)
        if s["b"] is not None:
            out += s["b"].double()
        if s["m"] is not None:
            at = torch.arange(case["vocab"], device="cuda")
            bits = (s["m"].long()[:, at // 32] >> (at % 32)) & 1
            out[(bits == 0).expand_as(out)] = -math.inf
        return {"y": out}
    x = s["x"].double()
    scale = (x.abs().amax(1) / 127.0).float().double()
    q = torch.round(x / torch.where(scale > 0, scale, torch.ones_like(scale))[:, None])
    y = torch.mm(q, s["wq"].double().t().contiguous()) * scale[:, None] * s["wscale"].double()
    if s["b"] is not None:
        y = y + s["b"].double()
    if case["act"] == "silu":
        y = y * torch.sigmoid(y)
    elif case["act"] == "gelu":
        y = y * 0.5 * torch.special.erfc(-y / math.sqrt(2.0))
    return {"y": y if s["r"] is None else y + s["r"].double()}
