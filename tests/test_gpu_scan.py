"""GPU parity of the gated linear recurrence with a vector state (gla_scan_*) against its float64
oracle, with tolerances that follow the roundings.

One token's step rounds a (relative error da), m (dm), the product m x, and the sum, and a
tree of products instead of a token-by-token walk only regroups those roundings. So the error
of h_t is at most e_t = a_t e_{t-1} + (da + 2u) a_t H_{t-1} + (dm + 2u) |m_t x_t|, with H the same
recurrence over absolute values and u = 2^-24; another 40 u H_t covers the levels of the tree. The
gate: for -0.30 <= g <= 0.05 a = 1 - t with t within 2u of itself, elsewhere the hardware's 2^x (2^-22)
of a product that one rounding moves by |g| u: da = (2 + 1.2 |g|) 2^-23 covers both. 1 - a at
g < -0.30, where it is at least 0.259: a's error 0.741 * 2.15 * 2^-23 and the subtraction's 2^-26 over
that are 6.7 * 2^-23, and less for larger |g|; its root halves that and adds 2^-22: dm = 7 * 2^-23 for
both. The slope a^2 / m: 2 da + dm + 3u.
The backward's dh obeys the same recurrence in reverse. A stored value adds half a step of its
type: finfo(t).eps / 2.
"""
import ctypes

import numpy as np
import pytest
import torch

from oracle import scan

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
ULP = 2.0 ** -23
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
IO = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def f64(t):
    return None if t is None else t.detach().to("cpu", torch.float64).numpy()


def errors_of_recurrence(a, da, b, db, start):
    """H and e of the module's docstring over axis 2 for |b| with relative error db, from |start|."""
    H = np.empty_like(b)
    e = np.empty_like(b)
    h, err = start, np.zeros_like(start)
    for t in range(b.shape[2]):
        err = a[:, :, t] * err + (da[:, :, t] + 2 * U) * a[:, :, t] * h + (db + 2 * U) * b[:, :, t]
        h = a[:, :, t] * h + b[:, :, t]
        H[:, :, t], e[:, :, t] = h, err
    return H, e + 40 * U * H


def bounds(x, g, h0, dO, dhT, kind, io):
    """Largest allowed |difference| of every output, from the inputs in float64."""
    a = np.exp(g)
    m, dm = scan.input_factor(g, kind)
    da = (2 + 1.2 * np.where(np.isfinite(g), np.abs(g), 0)) * ULP
    rm = 0.0 if kind == "plain" else 7 * ULP
    zero = np.zeros(x.shape[:2] + x.shape[3:])
    o, _ = scan.scan_fwd(x, g, h0, kind)
    H, e = errors_of_recurrence(a, da, np.abs(m * x), rm, zero if h0 is None else np.abs(h0))
    out = {"o": HALF[io] * np.abs(o) + e, "hT": e[:, :, -1] if x.shape[2] else zero + 0.0}
    if dO is None:
        return out
    L = x.shape[2]
    after = np.concatenate([a[:, :, 1:], np.ones_like(a[:, :, :1])], 2)
    dafter = np.concatenate([da[:, :, 1:], np.zeros_like(a[:, :, :1])], 2)
    G, eg = errors_of_recurrence(after[:, :, ::-1], dafter[:, :, ::-1], np.abs(dO)[:, :, ::-1], 0.0,
                                 zero if dhT is None else np.abs(dhT))
    G, eg = G[:, :, ::-1], eg[:, :, ::-1]
    ref = scan.scan_bwd(x, g, h0, dO, dhT, kind)
    first = (zero if h0 is None else np.abs(h0))[:, :, None]
    Hp = np.concatenate([first, H[:, :, :-1]], 2)
    ep = np.concatenate([np.zeros_like(first), e[:, :, :-1]], 2)
    fac, slope = a * Hp + np.abs(dm * x), 2 * da + rm + 3 * U
    out["dx"] = HALF[io] * np.abs(ref["dx"]) + m * eg + (rm + 2 * U) * m * G
    out["dg"] = fac * eg + G * (a * ep + (slope + 3 * U) * fac) + 4 * U * G * fac
    out["dh0"] = a[:, :, 0] * eg[:, :, 0] + (da[:, :, 0] + 2 * U) * a[:, :, 0] * G[:, :, 0] if L else zero + 0.0
    return out


def inputs(B, H, L, D, io, gates, seed, h0=True):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)
    x, pre, dO = n(B, H, L, D).to(IO[io]), n(B, H, L, D), n(B, H, L, D).to(IO[io])
    if gates == "slow":
        g = torch.nn.functional.logsigmoid(pre) / 16
    elif gates == "strong":
        g = -6 * pre.abs()
    elif gates == "packed":
        g = torch.nn.functional.logsigmoid(pre + 3)
        g[torch.rand(B, 1, L, 1, generator=gen).expand(B, H, L, D) < 0.02] = float("-inf")
    else:                                    # every kind of gate, some channels without any memory
        g = -pre.abs()
        g[..., ::3] = torch.nn.functional.logsigmoid(pre[..., ::3]) / 256
        g[..., 1::3][torch.rand(B, H, L, len(range(1, D, 3)), generator=gen) < 0.3] = float("-inf")
        if D > 4:
            g[..., 4] = float("-inf")
    return x, g, (n(B, H, D) if h0 else None), dO, (n(B, H, D) if h0 else None)


def cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


def within(got, ref, tol, name):
    got = f64(got)
    assert got.shape == ref.shape, name
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (name, int(bad.sum()), np.argwhere(bad)[0], np.nanmax(np.abs(got - ref)), got[bad][0],
                           ref[bad][0], tol[bad][0])


def check(B, H, L, D, io, kind, gates, seed, h0=True, save=True):
    from linear_rnn_b200 import ops
    x, g, s0, dO, dhT = inputs(B, H, L, D, io, gates, seed, h0)
    xd, gd, sd, dOd, dhd = cuda(x, g, s0, dO, dhT)
    saved = None
    if save:
        saved = torch.empty(max(16, ops.gla_scan_saved_bytes(ops.make_scan_problem(xd))), dtype=torch.uint8,
                            device="cuda")
    o, hT = ops.gla_scan_fwd(xd, gd, sd, input=kind, saved_states=saved)
    grads = ops.gla_scan_bwd(xd, gd, sd, dOd, dhd, input=kind, saved_states=saved)
    ro, rT = scan.scan_fwd(f64(x), f64(g), f64(s0), kind)
    ref = {"o": ro, "hT": rT, **scan.scan_bwd(f64(x), f64(g), f64(s0), f64(dO), f64(dhT), kind)}
    tol = bounds(f64(x), f64(g), f64(s0), f64(dO), f64(dhT), kind, IO[io])
    for name, got in {"o": o, "hT": hT, **grads}.items():
        within(got, ref[name], tol[name], name)


SIZES = [(1, 1, 1, 1), (2, 3, 1, 64), (1, 1, 2, 8), (2, 3, 63, 5), (1, 2, 64, 64), (1, 2, 65, 100), (2, 1, 127, 36),
         (1, 1, 128, 33), (2, 2, 129, 40), (1, 1, 300, 130), (1, 3, 517, 72), (2, 2, 1021, 24), (1, 2, 2049, 64),
         (1, 1, 4500, 96), (1, 1, 333, 257), (5, 7, 200, 16), (1, 1, 700, 74), (2, 1, 900, 130), (3, 2, 8, 64), (3, 2, 8, 66),
         (3, 2, 7, 67), (2, 2, 9, 40), (20, 1, 24, 1280), (20, 1, 25, 1282), (20, 1, 23, 1281), (60, 1, 64, 516)]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_scan_matches_oracle(size, io):
    kind = ["plain", "complement", "norm"][sum(size) % 3]
    check(*size, io, kind, "mixed", 41, save=sum(size) % 2 == 0)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["plain", "complement", "norm"])
@pytest.mark.parametrize("gates", ["slow", "strong", "packed"])
def test_scan_gates_and_factors(io, kind, gates):
    check(2, 3, 700, 72, io, kind, gates, 42)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_scan_without_states(io):
    check(2, 2, 130, 64, io, "complement", "slow", 43, h0=False)


@pytest.mark.parametrize("size", [(8, 16, 600, 64), (4, 16, 300, 256), (1, 8, 20000, 64), (1, 1, 30000, 128),
                                  (2, 1, 5000, 1024)], ids=str)
def test_scan_many_heads_and_long(size):
    check(*size, "bf16", "norm", "slow", 44)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_scan_empty(io):
    from linear_rnn_b200 import ops
    x, g, h0, dO, dhT = cuda(*inputs(2, 3, 0, 8, io, "slow", 45))
    o, hT = ops.gla_scan_fwd(x, g, h0)
    assert o.shape == (2, 3, 0, 8) and torch.equal(hT, h0)
    assert torch.equal(ops.gla_scan_bwd(x, g, h0, dO, dhT)["dh0"], dhT)
    _, hT = ops.gla_scan_fwd(x, g, None)
    assert (hT == 0).all()
    assert (ops.gla_scan_bwd(x, g, None, dO, None)["dh0"] == 0).all()
    x, g, h0, dO, dhT = cuda(*inputs(0, 3, 4, 8, io, "slow", 45))
    o, hT = ops.gla_scan_fwd(x, g, h0)
    assert o.shape == (0, 3, 4, 8) and hT.shape == (0, 3, 8)
    assert ops.gla_scan_bwd(x, g, h0, dO, dhT)["dx"].shape == (0, 3, 4, 8)


def test_scan_gradients_are_differences():
    """(f(v + e d) - f(v - e d)) / 2e of the GPU forward along a random direction d equals the
    gradient's projection. f is fp32: its own error over 2e is allowed for, with e^2 f''' / 6 far below."""
    from linear_rnn_b200 import ops
    x, g, h0, dO, dhT = cuda(*inputs(1, 2, 150, 20, "f32", "slow", 46))
    g = g - 0.05
    gen = torch.Generator(device="cuda").manual_seed(1)
    for kind in ("plain", "complement", "norm"):
        grads = ops.gla_scan_bwd(x, g, h0, dO, dhT, input=kind)
        for name, at in (("dx", 0), ("dg", 1), ("dh0", 2)):
            args = [x, g, h0]
            d = torch.randn(args[at].shape, generator=gen, device="cuda")
            e = 2.0 ** -8 if name != "dg" else 2.0 ** -11

            def f(sign):
                moved = list(args)
                moved[at] = args[at] + sign * e * d
                o, hT = ops.gla_scan_fwd(*moved, input=kind)
                return (dO.double() * o.double()).sum().item() + (dhT.double() * hT.double()).sum().item()
            o, _ = ops.gla_scan_fwd(*args, input=kind)
            # every o_t is within 60 u of its exact value's scale; the moved input rounds once more
            noise = 60 * U * (dO.abs().sum() * o.abs().max()).item() / (2 * e) / np.sqrt(dO.numel()) * 8
            want = (grads[name].double() * d.double()).sum().item()
            scale = (grads[name].abs().double() * d.abs().double()).sum().item()
            assert abs((f(1) - f(-1)) / (2 * e) - want) <= noise + 1e-3 * scale, (kind, name)


@pytest.mark.parametrize("kind", ["plain", "complement", "norm"])
def test_gate_of_zero_and_above(kind):
    """g = 0: no decay; 1 - a and sqrt(1 - a^2) are 0 there, and the root's slope counts as 0."""
    from linear_rnn_b200 import ops
    x, g, h0, dO, dhT = inputs(1, 2, 90, 12, "f32", "slow", 47)
    g[:, :, ::4] = 0.0
    if kind != "norm":
        g[:, :, 1::8] = 0.02
    xd, gd, sd, dOd, dhd = cuda(x, g, h0, dO, dhT)
    o, hT = ops.gla_scan_fwd(xd, gd, sd, input=kind)
    grads = ops.gla_scan_bwd(xd, gd, sd, dOd, dhd, input=kind)
    ref = dict(zip(("o", "hT"), scan.scan_fwd(f64(x), f64(g), f64(h0), kind)))
    ref.update(scan.scan_bwd(f64(x), f64(g), f64(h0), f64(dO), f64(dhT), kind))
    tol = bounds(f64(x), f64(g), f64(h0), f64(dO), f64(dhT), kind, torch.float32)
    for name, got in {"o": o, "hT": hT, **grads}.items():
        # g > 0 grows: 1 - a is negative there, so its magnitude enters the bounds
        within(got, ref[name], np.abs(tol[name]) + 1e-30, name)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_state_handoff_and_decode(io):
    """fwd over L = fwd over L1, then L2 from its hT; and a prompt's end continued token by token."""
    from linear_rnn_b200 import ops
    x, g, h0, _, _ = inputs(2, 3, 210, 48, io, "packed", 48)
    xd, gd, sd = cuda(x, g, h0)
    ref, rT = scan.scan_fwd(f64(x), f64(g), f64(h0), "complement")
    tol = bounds(f64(x), f64(g), f64(h0), None, None, "complement", IO[io])
    o1, h1 = ops.gla_scan_fwd(xd[:, :, :140].contiguous(), gd[:, :, :140].contiguous(), sd, input="complement")
    state = h1.clone()
    o2, h2 = ops.gla_scan_fwd(xd[:, :, 140:].contiguous(), gd[:, :, 140:].contiguous(), h1, input="complement")
    within(torch.cat([o1, o2], 2), ref, tol["o"], "o")
    within(h2, rT, tol["hT"], "hT")
    toks = [ops.gla_scan_decode(xd[:, :, t:t + 1].contiguous(), gd[:, :, t:t + 1].contiguous(), state,
                                input="complement") for t in range(140, 210)]
    within(torch.cat(toks, 2), ref[:, :, 140:], tol["o"][:, :, 140:], "decode")
    within(state, rT, tol["hT"], "state")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("size", [(1, 1, 1), (3, 5, 7), (64, 16, 256), (2, 3, 65), (1, 40, 4100)], ids=str)
@pytest.mark.parametrize("kind", ["plain", "complement", "norm"])
def test_decode_matches_oracle(io, size, kind):
    from linear_rnn_b200 import ops
    B, H, D = size
    x, g, h0, _, _ = inputs(B, H, 1, D, io, "mixed", 49)
    state = h0.cuda()
    o = ops.gla_scan_decode(x.cuda(), g.cuda(), state, input=kind)
    ro, rT = scan.scan_fwd(f64(x), f64(g), f64(h0), kind)
    tol = bounds(f64(x), f64(g), f64(h0), None, None, kind, IO[io])
    within(o, ro, tol["o"], "o")
    within(state, rT, tol["hT"], "state")


@pytest.mark.parametrize("L", [1, 100, 3000])
def test_saved_and_recomputed_states_agree_and_repeat(L):
    """The training pair, the backward alone, and a second run give the same bits."""
    from linear_rnn_b200 import ops
    x, g, h0, dO, dhT = cuda(*inputs(2, 2, L, 72, "bf16", "slow", 50))
    saved = torch.empty(ops.gla_scan_saved_bytes(ops.make_scan_problem(x)), dtype=torch.uint8, device="cuda")
    runs = []
    for _ in range(2):
        saved.fill_(255)
        o, hT = ops.gla_scan_fwd(x, g, h0, input="norm", saved_states=saved)
        runs.append((o, hT, *ops.gla_scan_bwd(x, g, h0, dO, dhT, input="norm", saved_states=saved).values()))
    runs.append((*ops.gla_scan_fwd(x, g, h0, input="norm"), *ops.gla_scan_bwd(x, g, h0, dO, dhT, input="norm").values()))
    for other in runs[1:]:
        for a, b in zip(runs[0], other):
            assert torch.equal(a, b)


def _call(fn, p, mode, *tensors, ws=()):
    from linear_rnn_b200 import _lib
    ptr = lambda t: None if t is None else ctypes.c_void_p(t.data_ptr())
    st = fn(ctypes.byref(p), mode, *map(ptr, tensors), *ws, ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert st == _lib.GLA_OK, _lib.status_string(st)


@pytest.mark.parametrize("size", [(2, 3, 70, 24), (1, 2, 333, 100), (1, 1, 65, 7), (1, 1, 1, 64)], ids=str)
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_outputs_are_written_whole_and_nothing_else(size, io):
    """Buffers filled with NaN become finite, and the bytes behind every buffer stay."""
    from linear_rnn_b200 import _lib, ops
    B, H, L, D = size
    x, g, h0, dO, dhT = cuda(*inputs(B, H, L, D, io, "slow", 51))
    p = ops.make_scan_problem(x)
    pad = 512

    def buffer(shape, dtype):
        n = int(np.prod(shape))
        flat = torch.full((n + pad,), float("nan"), dtype=dtype, device="cuda")
        flat[n:] = 7
        return flat, flat[:n].view(shape)
    fo, o = buffer(x.shape, IO[io])
    fT, hT = buffer(h0.shape, torch.float32)
    fs, sv = buffer((ops.gla_scan_saved_bytes(p) // 4,), torch.float32)
    fx, dx = buffer(x.shape, IO[io])
    fg, dg = buffer(x.shape, torch.float32)
    f0, dh0 = buffer(h0.shape, torch.float32)
    nb = ops.gla_scan_bwd_workspace_bytes(p)
    ws = torch.full((nb + pad,), 9, dtype=torch.uint8, device="cuda")
    lib = _lib.lib
    _call(lib.gla_scan_fwd_save, p, 1, x, g, h0, o, hT, sv)
    _call(lib.gla_scan_bwd_saved, p, 1, x, g, h0, dO, dhT, sv, dx, dg, dh0, ws=(None, 0))   # needs no workspace
    for flat in (fo, fT, fs, fx, fg, f0):
        assert torch.isfinite(flat[:-pad]).all() and (flat[-pad:] == 7).all()
    fx.fill_(float("nan")), fg.fill_(float("nan"))
    _call(lib.gla_scan_bwd, p, 1, x, g, h0, dO, dhT, dx, dg, None, ws=(ctypes.c_void_p(ws.data_ptr()), nb))
    assert torch.isfinite(dx).all() and torch.isfinite(dg).all()
    assert (ws[nb:] == 9).all()


def test_non_finite_inputs_spread_as_the_formula_says():
    from linear_rnn_b200 import ops
    x, g, h0, _, _ = inputs(1, 2, 200, 16, "f32", "slow", 52)
    x[0, 0, 50, 3] = float("inf")
    x[0, 0, 70, 5] = float("nan")
    g[0, 1, 120, 7] = float("nan")
    o, hT = ops.gla_scan_fwd(*cuda(x, g, h0))
    with np.errstate(invalid="ignore"):
        ro, rT = scan.scan_fwd(f64(x), f64(g), f64(h0), "plain")
    assert np.array_equal(np.isnan(f64(o)), np.isnan(ro)) and np.array_equal(np.isinf(f64(o)), np.isinf(ro))
    assert np.array_equal(np.isfinite(f64(hT)), np.isfinite(rT))


def test_graph_replays_side_stream_and_host_tensors():
    from linear_rnn_b200 import ops
    x, g, h0, dO, dhT = inputs(2, 2, 400, 64, "bf16", "slow", 53)
    xd, gd, sd, dOd, dhd = cuda(x, g, h0, dO, dhT)
    want = (*ops.gla_scan_fwd(xd, gd, sd), *ops.gla_scan_bwd(xd, gd, sd, dOd, dhd).values())
    host = (*ops.gla_scan_fwd(x, g, h0), *ops.gla_scan_bwd(x, g, h0, dO, dhT).values())
    for a, b in zip(want, host):
        assert b.device.type == "cpu" and torch.equal(a.cpu(), b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = (*ops.gla_scan_fwd(xd, gd, sd), *ops.gla_scan_bwd(xd, gd, sd, dOd, dhd).values())
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    state = sd.clone()
    xt, gt = xd[:, :, :1].contiguous(), gd[:, :, :1].contiguous()
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs = (*ops.gla_scan_fwd(xd, gd, sd), *ops.gla_scan_bwd(xd, gd, sd, dOd, dhd).values())
            ops.gla_scan_decode(xt, gt, state)
        graphs.append((gr, outs))
    for gr, outs in graphs:
        for t in outs:
            t.fill_(float("nan"))
    state.copy_(sd)
    for gr, _ in graphs:
        gr.replay()
    torch.cuda.synchronize()
    for _, outs in graphs:
        for a, b in zip(want, outs):
            assert torch.equal(a, b)
    s1 = sd.clone()
    for _ in range(2):
        ops.gla_scan_decode(xt, gt, s1)
    assert torch.equal(s1, state)


def test_offsets_past_32_bits():
    """More than 2^31 elements: a start near the end makes the last tokens a recurrence of their own."""
    from linear_rnn_b200 import ops
    L, D, tail = (1 << 19) + 5, 4112, 70
    x = torch.empty(1, 1, L, D, dtype=torch.bfloat16, device="cuda")
    for t in range(0, L, 1 << 16):
        x[:, :, t:t + (1 << 16)].normal_()
    g = torch.full((1, 1, L, D), -0.05, device="cuda")
    g[:, :, -tail] = float("-inf")
    o, hT = ops.gla_scan_fwd(x, g)
    ref, rT = scan.scan_fwd(f64(x[:, :, -tail:]), f64(g[:, :, -tail:]), None, "plain")
    tol = bounds(f64(x[:, :, -tail:]), f64(g[:, :, -tail:]), None, None, None, "plain", torch.bfloat16)
    within(o[:, :, -tail:], ref, tol["o"], "o")
    within(hT, rT, tol["hT"], "hT")
    at = L // 2
    ref = scan.scan_fwd(f64(x[:, :, :40]), f64(g[:, :, :40]), None, "plain")[0]
    within(o[:, :, :40], ref, bounds(f64(x[:, :, :40]), f64(g[:, :, :40]), None, None, None, "plain",
                                     torch.bfloat16)["o"], "head")
    # far from any start: 800 tokens of decay e^-0.05 leave e^-40 of the past
    lo = at - 800
    seg = scan.scan_fwd(f64(x[:, :, lo:at, :64]), f64(g[:, :, lo:at, :64]), None, "plain")[0]
    tol = bounds(f64(x[:, :, lo:at, :64]), f64(g[:, :, lo:at, :64]), None, None, None, "plain", torch.bfloat16)["o"]
    within(o[:, :, at - 1:at, :64], seg[:, :, -1:], tol[:, :, -1:] + 1e-12, "middle")
    del o
    dO = x.flip(2)
    grads = ops.gla_scan_bwd(x, g, None, dO, output_dh0=False)
    ref = scan.scan_bwd(f64(x[:, :, -tail:]), f64(g[:, :, -tail:]), None, f64(dO[:, :, -tail:]), None, "plain")
    tol = bounds(f64(x[:, :, -tail:]), f64(g[:, :, -tail:]), None, f64(dO[:, :, -tail:]), None, "plain",
                 torch.bfloat16)
    for name in ("dx", "dg"):
        within(grads[name][:, :, -tail:], ref[name], tol[name], name)


def test_refusals():
    from linear_rnn_b200 import _lib, ops
    x, g, h0, dO, dhT = cuda(*inputs(1, 2, 70, 16, "bf16", "slow", 54))
    for bad in (lambda: ops.gla_scan_fwd(x.half(), g), lambda: ops.gla_scan_fwd(x, g.bfloat16()),
                lambda: ops.gla_scan_fwd(x, g[..., :8].contiguous()), lambda: ops.gla_scan_fwd(x, None),
                lambda: ops.gla_scan_fwd(x, g, h0[:, :1].contiguous()), lambda: ops.gla_scan_fwd(x, g, input="gru"),
                lambda: ops.gla_scan_fwd(x.transpose(1, 2).contiguous().transpose(1, 2), g),
                lambda: ops.gla_scan_bwd(x, g, h0, dO.float()), lambda: ops.gla_scan_bwd(x, g, h0, None),
                lambda: ops.gla_scan_decode(x, g, h0), lambda: ops.gla_scan_fwd(x[0], g[0]),
                lambda: ops.gla_scan_decode(x[:, :, :1].contiguous(), g[:, :, :1].contiguous(), h0[:, :1].contiguous()),
                lambda: ops.gla_scan_bwd(x, g, h0, dO, workspace=torch.empty(1 << 20, dtype=torch.uint8))):
        with pytest.raises((ValueError, TypeError)):
            bad()
    small = torch.empty(64, dtype=torch.uint8, device="cuda")
    for bad in (lambda: ops.gla_scan_bwd(x, g, h0, dO, saved_states=small), lambda: ops.gla_scan_fwd(x, g, saved_states=small),
                lambda: ops.gla_scan_bwd(x, g, h0, dO, workspace=small)):
        with pytest.raises(_lib.GlaError) as e:
            bad()
        assert e.value.status == _lib.GLA_ERR_WORKSPACE
    odd = torch.empty(x.numel() + 1, dtype=torch.bfloat16, device="cuda")[1:].view(x.shape)
    with pytest.raises(_lib.GlaError) as e:
        ops.gla_scan_fwd(odd, g)
    assert e.value.status == _lib.GLA_ERR_INVALID_ARG
