"""The operators around and beside the matrix-state cells, as cases that can be run and measured.

  scan      gated linear recurrence with a vector state, h_t = e^{g_t} h_{t-1} + m(g_t) x_t:
            forward, forward and backward together (a training step), one decoding step
  addnorm   residual sum and norm before a block: r = res + alpha rscale x, y = norm(r) w
  headnorm  norm and gate after a cell: y = norm(o) w act(z) per head, from the cell's
            [B,H,L,D] to the out-projection's [B,L,H,D]

`own` chooses between the plain form (elementary torch operations in fp32) and the calls that a
user makes of the framework.
"""
import math

import torch

own = False

DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


# ----------------------------------------------------------------------------------- cases

def listed():
    return [
        # a short prompt entering a small layer: latency counts, nothing is a round number
        _scan("scan_fwd_short", "fwd", 1, 4, 77, 64, "bf16", "complement", "slow"),
        # the batch of heads of the GLA forward workload (8 x 16 heads, 2048 tokens, 64 wide)
        _scan("scan_fwd_heads", "fwd", 8, 16, 2048, 64, "bf16", "complement", "slow"),
        # one long document, few heads: the long-context workload, continued from a state
        _scan("scan_fwd_long", "fwd", 1, 8, 65536, 128, "bf16", "plain", "slow", h0=True),
        # a training step at the size of the main GLA workload
        _scan("scan_train", "train", 4, 16, 4096, 256, "bf16", "norm", "slow"),
        # a training step on packed documents (a gate of minus infinity starts one), odd sizes
        _scan("scan_train_packed", "train", 3, 5, 1021, 100, "f32", "norm", "packed", h0=True),
        # one token for 64 sequences x 16 heads, as in the decoding workload
        _scan("scan_decode", "decode", 64, 16, 1, 256, "bf16", "complement", "forget", h0=True),
        # the same 64 tokens through the residual sum and norm of a 4096-wide model
        _addnorm("addnorm_fwd_decode", "fwd", 64, 4096, "bf16", "bf16", "rms"),
        # the training batch of the main workload (4 x 4096 tokens of 16 x 256), fp32 residual
        _addnorm("addnorm_fwd", "fwd", 16384, 4096, "bf16", "f32", "rms", rscale=True),
        # the backward at the width of the mLSTM workload (2 x 8192 tokens of 8 x 256)
        _addnorm("addnorm_bwd", "bwd", 16384, 2048, "bf16", "bf16", "layer", rscale=True),
        # the output of the main workload's cell, with the swish gate
        _headnorm("headnorm_fwd", "fwd", 4, 16, 4096, 256, "bf16", "rms", "silu"),
        # the mLSTM cell's output norm and output gate, weights per head, backward
        _headnorm("headnorm_bwd", "bwd", 2, 8, 8192, 256, "bf16", "layer", "sigmoid", per_head=True),
        # odd sizes in fp32
        _headnorm("headnorm_bwd_odd", "bwd", 3, 5, 1021, 100, "f32", "rms", "silu"),
    ]


def _scan(name, pass_, B, H, L, D, io, input, gates, h0=False):
    return {"name": name, "op": "scan", "pass": pass_, "B": B, "H": H, "L": L, "D": D, "io": io, "input": input,
            "gates": gates, "h0": h0}


def _addnorm(name, pass_, rows, D, io, res, kind, rscale=False):
    return {"name": name, "op": "addnorm", "pass": pass_, "rows": rows, "D": D, "io": io, "res": res, "kind": kind,
            "rscale": rscale}


def _headnorm(name, pass_, B, H, L, D, io, kind, act, per_head=False):
    return {"name": name, "op": "headnorm", "pass": pass_, "B": B, "H": H, "L": L, "D": D, "io": io, "kind": kind,
            "act": act, "per_head": per_head}


def draw(rng):
    def size(lo, hi):
        """Spread over the logarithm; multiples of a power of two as often as odd sizes."""
        n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        step = rng.choice([1, 1, 2, 8, 32, 64])
        return max(lo, min(hi, n // step * step if n >= step else n))

    op = rng.choice(["scan", "scan", "addnorm", "headnorm"])
    io = rng.choice(["bf16", "bf16", "f32"])
    if op == "scan":
        pass_ = rng.choice(["fwd", "train", "decode"])
        B, H, D = size(1, 64 if pass_ == "decode" else 8), size(1, 16), size(8, 2048)
        most = (1 << 26) // (2 if io == "f32" else 1) // (B * H * D)
        L = 1 if pass_ == "decode" else size(1, max(1, min(65536, most)))
        case = _scan("", pass_, B, H, L, D, io, rng.choice(["plain", "complement", "norm"]),
                     rng.choice(["slow", "forget", "packed"]), h0=pass_ == "decode" or rng.random() < 0.5)
    elif op == "addnorm":
        D = size(16, 8192)
        rows = size(1, min(65536, (1 << 25) // D))
        res = "f32" if io == "f32" else rng.choice(["bf16", "f32"])
        case = _addnorm("", rng.choice(["fwd", "bwd"]), rows, D, io, res, rng.choice(["rms", "layer"]),
                        rscale=rng.random() < 0.5)
    else:
        B, H, D = size(1, 8), size(1, 32), size(8, 1024)
        L = size(1, max(1, min(65536, (1 << 25) // (B * H * D))))
        case = _headnorm("", rng.choice(["fwd", "bwd"]), B, H, L, D, io, rng.choice(["rms", "layer"]),
                         rng.choice(["silu", "sigmoid"]), per_head=rng.random() < 0.5)
    del case["name"]
    return case


# ---------------------------------------------------------------------------------- inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    io = DTYPE[case["io"]]

    def normal(*shape, dtype=torch.float32, mul=1.0, add=0.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * mul + add).to(dtype)

    s = {"case": case}
    if case["op"] == "scan":
        B, H, L, D = case["B"], case["H"], case["L"], case["D"]
        s["x"] = normal(B, H, L, D, dtype=io)
        if case["gates"] == "slow":       # the gated linear attention workloads' gates
            s["g"] = torch.nn.functional.logsigmoid(normal(B, H, L, D)) / 16
        else:                             # the mLSTM workload's forget gates
            s["g"] = torch.nn.functional.logsigmoid(normal(B, H, L, D, add=3.0))
        if case["gates"] == "packed":     # some tokens start a document
            starts = torch.rand(B, 1, L, 1, generator=gen, device="cuda") < 1 / 256
            s["g"] = s["g"].masked_fill(starts, float("-inf"))
        s["h0"] = normal(B, H, D) if case["h0"] else None
        if case["pass"] == "train":
            s["dO"] = normal(B, H, L, D, dtype=io)
            s["dhT"] = normal(B, H, D) if case["h0"] else None
    elif case["op"] == "addnorm":
        N, D, res = case["rows"], case["D"], DTYPE[case["res"]]
        s["x"] = normal(N, D, dtype=io)
        s["res"] = normal(N, D, dtype=res, mul=3.0)   # the residual stream (the backward's r)
        s["w"] = normal(D, mul=0.2, add=1.0)
        s["rscale"] = normal(D, mul=0.1, add=0.5) if case["rscale"] else None
        if case["pass"] == "bwd":
            s["dy"] = normal(N, D, dtype=io)
            s["dr"] = normal(N, D, dtype=res)
    else:
        B, H, L, D = case["B"], case["H"], case["L"], case["D"]
        s["o"] = normal(B, H, L, D, dtype=io, mul=2.0)
        s["z"] = normal(B, L, H, D, dtype=io)
        s["w"] = normal(H, D, mul=0.2, add=1.0) if case["per_head"] else normal(D, mul=0.2, add=1.0)
        if case["pass"] == "bwd":
            s["dy"] = normal(B, L, H, D, dtype=io)
    return s


# ------------------------------------------------------------------------------------- run

def run(s):
    case = s["case"]
    if own:
        return _own(s, case)
    if case["op"] == "scan":
        return {"fwd": _scan_fwd, "train": _scan_train, "decode": _scan_decode}[case["pass"]](s, case)
    if case["op"] == "addnorm":
        return {"fwd": _addnorm_fwd, "bwd": _addnorm_bwd}[case["pass"]](s, case)
    return {"fwd": _headnorm_fwd, "bwd": _headnorm_bwd}[case["pass"]](s, case)


def _own(s, case):
    from linear_rnn_b200 import ops
    if case["op"] == "scan":
        if case["pass"] == "decode":
            o = ops.gla_scan_decode(s["x"], s["g"], s["h0"], input=case["input"])
            return {"o": o, "state": s["h0"]}
        if case["pass"] == "fwd":
            o, hT = ops.gla_scan_fwd(s["x"], s["g"], s["h0"], input=case["input"])
            return {"o": o, "hT": hT}
        prob = ops.make_scan_problem(s["x"])
        saved = torch.empty(ops.gla_scan_saved_bytes(prob), dtype=torch.uint8, device=s["x"].device)
        o, hT = ops.gla_scan_fwd(s["x"], s["g"], s["h0"], input=case["input"], saved_states=saved)
        grads = ops.gla_scan_bwd(s["x"], s["g"], s["h0"], s["dO"], s["dhT"], input=case["input"], saved_states=saved)
        return {"o": o, "hT": hT, **grads}
    if case["op"] == "addnorm":
        if case["pass"] == "fwd":
            r, y = ops.gla_addnorm_fwd(s["x"], s["res"], s["w"], rscale=s["rscale"], alpha=0.5, kind=case["kind"],
                                       eps=EPS)
            return {"r": r, "y": y}
        return ops.gla_addnorm_bwd(s["x"], s["res"], s["w"], s["dy"], s["dr"], rscale=s["rscale"], alpha=0.5,
                                   kind=case["kind"], eps=EPS)
    if case["pass"] == "fwd":
        return ops.gla_headnorm_fwd(s["o"], s["z"], s["w"], act=case["act"], kind=case["kind"], eps=EPS)
    return ops.gla_headnorm_bwd(s["o"], s["z"], s["w"], s["dy"], act=case["act"], kind=case["kind"], eps=EPS)


# ----------------------------------------------------------------------- plain form: scan

def _input_scale(g, kind):
    """m(g), the factor on the input, and its derivative dm/dg."""
    if kind == "plain":
        return torch.ones_like(g), torch.zeros_like(g)
    if kind == "complement":
        return -torch.expm1(g), -torch.exp(g)
    m = torch.sqrt(-torch.expm1(2 * g))
    return m, torch.where(m > 0, -torch.exp(2 * g) / m, 0)


def _linear_scan(a, b):
    """All h_t = a_t h_{t-1} + b_t (from zero) along dim 2, by doubling the reach of every element."""
    reach, L = 1, a.shape[2]
    while reach < L:
        b = torch.cat([b[:, :, :reach], b[:, :, reach:] + a[:, :, reach:] * b[:, :, :-reach]], 2)
        a = torch.cat([a[:, :, :reach], a[:, :, reach:] * a[:, :, :-reach]], 2)
        reach *= 2
    return b


def _states(s, case):
    """a, m, dm, and every state in fp32."""
    g = s["g"]
    a = torch.exp(g)
    m, dm = _input_scale(g, case["input"])
    b = m * s["x"].float()
    if s["h0"] is not None:
        b[:, :, 0] += a[:, :, 0] * s["h0"]
    return a, m, dm, _linear_scan(a, b)


def _scan_fwd(s, case):
    _, _, _, h = _states(s, case)
    return {"o": h.to(s["x"].dtype), "hT": h[:, :, -1].clone()}


def _scan_train(s, case):
    x, dO = s["x"], s["dO"]
    a, m, dm, h = _states(s, case)
    out = {"o": h.to(x.dtype), "hT": h[:, :, -1].clone()}
    first = torch.zeros_like(h[:, :, :1]) if s["h0"] is None else s["h0"].unsqueeze(2)
    prev = torch.cat([first, h[:, :, :-1]], 2)
    # the gradient of h_t is dO_t + a_{t+1} dh_{t+1}: the same recurrence from the other end
    up = dO.float()
    if s["dhT"] is not None:
        up = up.clone()       # an fp32 dO is the case's own
        up[:, :, -1] += s["dhT"]
    after = torch.cat([a[:, :, 1:], torch.zeros_like(a[:, :, :1])], 2)
    dh = _linear_scan(after.flip(2), up.flip(2)).flip(2)
    out["dx"] = (m * dh).to(x.dtype)
    out["dg"] = dh * (a * prev + dm * x.float())
    out["dh0"] = a[:, :, 0] * dh[:, :, 0]
    return out


def _scan_decode(s, case):
    a = torch.exp(s["g"][:, :, 0])
    m, _ = _input_scale(s["g"][:, :, 0], case["input"])
    h = a * s["h0"] + m * s["x"][:, :, 0].float()
    s["h0"].copy_(h)
    return {"o": h.unsqueeze(2).to(s["x"].dtype), "state": s["h0"]}


# -------------------------------------------------------------------- plain form: the norms

def _normalise(r, kind):
    """(normalised rows, 1 / their root mean square)"""
    if kind == "layer":
        r = r - r.mean(-1, keepdim=True)
    rstd = torch.rsqrt(r.square().mean(-1, keepdim=True) + EPS)
    return r * rstd, rstd


def _normalise_grad(d, n, rstd, kind):
    """The gradient of the rows from that of the normalised rows n."""
    d = d - n * (d * n).mean(-1, keepdim=True) - (d.mean(-1, keepdim=True) if kind == "layer" else 0)
    return d * rstd


def _addnorm_fwd(s, case):
    x = s["x"].float() * 0.5
    r = s["res"].float() + (x if s["rscale"] is None else x * s["rscale"])
    n, _ = _normalise(r, case["kind"])
    return {"r": r.to(s["res"].dtype), "y": (n * s["w"]).to(s["x"].dtype)}


def _addnorm_bwd(s, case):
    dy, x = s["dy"].float(), s["x"].float()
    n, rstd = _normalise(s["res"].float(), case["kind"])
    dres = s["dr"].float() + _normalise_grad(dy * s["w"], n, rstd, case["kind"])
    dx = dres * 0.5
    out = {"dres": dres.to(s["res"].dtype), "dw": (dy * n).sum(0)}
    if s["rscale"] is not None:
        out["drscale"] = (dx * x).sum(0)
        dx = dx * s["rscale"]
    out["dx"] = dx.to(s["x"].dtype)
    return out


def _gate(z, act):
    """act(z) and its derivative."""
    p = torch.sigmoid(z)
    if act == "sigmoid":
        return p, p * (1 - p)
    return z * p, p * (1 + z * (1 - p))


def _headnorm_fwd(s, case):
    n, _ = _normalise(s["o"].float(), case["kind"])
    return (n.transpose(1, 2) * s["w"] * _gate(s["z"].float(), case["act"])[0]).to(s["o"].dtype)


def _headnorm_bwd(s, case):
    n, rstd = _normalise(s["o"].float(), case["kind"])
    nt, dy = n.transpose(1, 2), s["dy"].float()
    gate, dgate = _gate(s["z"].float(), case["act"])
    dn = dy * gate
    dw = (dn * nt).sum((0, 1) if case["per_head"] else (0, 1, 2))
    do = _normalise_grad((dn * s["w"]).transpose(1, 2), n, rstd, case["kind"])
    return {"do": do.to(s["o"].dtype).contiguous(), "dz": (dy * nt * s["w"] * dgate).to(s["z"].dtype), "dw": dw}


# ------------------------------------------------------------------------------------ work

def work(case):
    e = 2 if case["io"] == "bf16" else 4
    if case["op"] == "scan":
        heads = case["B"] * case["H"] * case["D"]
        n = heads * case["L"]
        extra = 1 if case["input"] == "plain" else 4
        if case["pass"] == "decode":      # x, g and the state in, the state and o out
            return {"bytes": n * (2 * e + 12), "flops": n * (3 + extra)}
        ends = 4 * heads * (2 if case["h0"] else 1)
        if case["pass"] == "fwd":         # x, g in, o out
            return {"bytes": n * (2 * e + 4) + ends, "flops": n * (3 + extra)}
        return {"bytes": n * (4 * e + 8) + 2 * ends, "flops": n * (10 + 2 * extra)}   # + dO in, dx, dg out
    if case["op"] == "addnorm":
        n, r = case["rows"] * case["D"], 2 if case["res"] == "bf16" else 4
        vec = 4 * case["D"] * (1 + case["rscale"])
        if case["pass"] == "fwd":         # x, res in, r, y out
            return {"bytes": n * (2 * e + 2 * r) + vec, "flops": 7 * n}
        # r, dy, dr in, dres, dx out; x where its scale learns
        return {"bytes": n * (2 * e + 3 * r + (e if case["rscale"] else 0)) + 2 * vec, "flops": 15 * n}
    n = case["B"] * case["H"] * case["L"] * case["D"]
    vec = 4 * case["D"] * (case["H"] if case["per_head"] else 1)
    if case["pass"] == "fwd":             # o, z in, y out
        return {"bytes": n * 3 * e + vec, "flops": 12 * n}
    return {"bytes": n * 5 * e + 2 * vec, "flops": 25 * n}   # o, z, dy in, do, dz out


# ----------------------------------------------------------------------------------- exact

def exact(case, seed):
    """The definitions in 64 bits: the recurrence token by token, the norms' gradients by
    differentiating their forward formula."""
    s = prepare(case, seed)
    d = {k: v.double() if torch.is_tensor(v) else v for k, v in s.items()}
    if case["op"] == "scan":
        return _exact_scan(d, case)
    leaf = {k: v.requires_grad_() for k, v in d.items() if torch.is_tensor(v) and k not in ("dy", "dr")}
    if case["op"] == "addnorm":
        if case["pass"] == "fwd":
            with torch.no_grad():
                r = d["res"] + 0.5 * d["x"] * (1 if d["rscale"] is None else d["rscale"])
                return {"r": r, "y": _exact_norm(r, case["kind"]) * d["w"]}
        # the sum whose value is the given r, as a function of each of its terms
        term = 0.5 * d["x"] * (1 if d["rscale"] is None else d["rscale"])
        r = d["res"] + (term - term.detach())
        loss = (d["dy"] * _exact_norm(r, case["kind"]) * d["w"]).sum() + (d["dr"] * r).sum()
        names = {"res": "dres", "w": "dw", "x": "dx", "rscale": "drscale"}
    else:
        act = d["z"] / (1 + torch.exp(-d["z"])) if case["act"] == "silu" else 1 / (1 + torch.exp(-d["z"]))
        y = _exact_norm(d["o"], case["kind"]).permute(0, 2, 1, 3) * d["w"] * act
        if case["pass"] == "fwd":
            return y.detach()
        loss = (d["dy"] * y).sum()
        names = {"o": "do", "z": "dz", "w": "dw"}
    grads = torch.autograd.grad(loss, [leaf[k] for k in leaf])
    return {names[k]: v for k, v in zip(leaf, grads)}


def _exact_norm(r, kind):
    if kind == "layer":
        return (r - r.mean(-1, keepdim=True)) / torch.sqrt(r.var(-1, unbiased=False, keepdim=True) + EPS)
    return r / torch.sqrt(r.pow(2).mean(-1, keepdim=True) + EPS)


def _exact_scan(d, case):
    x, a = d["x"].movedim(2, 0).contiguous(), torch.exp(d["g"]).movedim(2, 0).contiguous()
    L = x.shape[0]
    one = torch.ones((), dtype=torch.float64, device=x.device)
    g = d["g"].movedim(2, 0)
    m = {"plain": lambda: one.expand_as(a), "complement": lambda: -torch.expm1(g),
         "norm": lambda: torch.sqrt(-torch.expm1(2 * g))}[case["input"]]()
    b = m * x
    h0 = torch.zeros_like(x[0]) if d["h0"] is None else d["h0"]
    h, last = torch.empty_like(x), h0
    for t in range(L):
        torch.addcmul(b[t], a[t], last, out=h[t])
        last = h[t]
    if case["pass"] == "decode":
        return {"o": h.movedim(0, 2), "state": last.clone()}
    out = {"o": h.movedim(0, 2), "hT": last.clone()}
    if case["pass"] == "fwd":
        return out
    del b
    dh = d["dO"].movedim(2, 0).contiguous()
    if d["dhT"] is not None:
        dh[-1] += d["dhT"]
    for t in range(L - 2, -1, -1):
        dh[t].addcmul_(a[t + 1], dh[t + 1])
    out["dx"] = (m * dh).movedim(0, 2).contiguous()
    out["dh0"] = a[0] * dh[0]
    dg = torch.cat([h0.unsqueeze(0), h[:-1]]).mul_(a).mul_(dh)
    if case["input"] == "complement":
        dg -= a * x * dh
    elif case["input"] == "norm":     # d sqrt(1 - a^2) / dg = -a^2 / sqrt(1 - a^2), and 0 at a = 1
        dg -= torch.where(a < 1, a * a / torch.where(a < 1, m, one), 0) * x * dh
    out["dg"] = dg.movedim(0, 2).contiguous()
    return out
