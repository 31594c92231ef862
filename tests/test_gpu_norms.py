"""GPU parity of the norms before and after a block (gla_addnorm_*, gla_headnorm_*) against their
float64 oracle, with tolerances that follow the roundings.

u = 2^-24. A row's sums run over at most 16 terms a thread and then a tree: relative error below
(16 + 10 + 6) u of the sum of absolute values, so mu is within 32 u max|r|, and 1/sqrt(mean + eps)
within (32 / 2 + 4) u of itself plus what mu's error does (second order). With N = max|r| rstd a
bound of the normalised row, n is within (32 + 20 + 2) u N. A gate's exponential is within 4u (and
|z| u with bf16 data, |z| < 16 here), its sum and reciprocal within 3u, the products 2u: below 26 u of it,
its slope by a factor 1 + |z|. So y is within (54 + 26 + 4) u N |w f| and half a step
of its type. Gradient of the row: rstd (d - n mean(d n) - mean(d)), each mean with the sums' error:
within 192 u rstd (|d| + 2 N mean|d n| + N mean|d| + mean|d|). Row sums dw: every term dy n f is within
84 u |dy f| N, and at most 40 additions follow one another in each block and 64 in the sum over
blocks: 200 u sum |dy f| N.
"""
import ctypes

import numpy as np
import pytest
import torch

from oracle import norms, scan

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
IO = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def f64(t):
    return None if t is None else t.detach().to("cpu", torch.float64).numpy()


def cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


def within(got, ref, tol, name):
    got = f64(got)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    tol = np.broadcast_to(tol, ref.shape)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (name, int(bad.sum()), np.argwhere(bad)[0], got[bad][0], ref[bad][0], tol[bad][0])


def row_bound(r, kind):
    """(N, rstd) per row"""
    u = r - r.mean(-1, keepdims=True) if kind == "layer" else r
    rstd = 1 / np.sqrt((u * u).mean(-1, keepdims=True) + EPS)
    return np.abs(r).max(-1, keepdims=True) * rstd, rstd


def grad_bound(r, d, kind):
    """of the row's gradient from d, the gradient of its normalised row"""
    N, rstd = row_bound(r, kind)
    n = norms.norm(r, kind, EPS)
    mean = lambda v: np.abs(v).mean(-1, keepdims=True)
    return 192 * U * rstd * (np.abs(d) + 2 * N * mean(d * n) + N * mean(d) + mean(d))


ROWS = [(1, 1), (3, 7), (5, 8), (1, 33), (64, 64), (70, 100), (9, 257), (33, 256), (17, 512), (700, 520), (2, 1000),
        (5, 2048), (300, 2052), (3, 4096), (4, 4104), (2, 8192), (3, 8200), (2, 9999), (2, 16384),
        (400, 66), (2000, 78), (900, 330), (700, 333), (5, 2050), (3, 4098), (3, 4100), (2, 2049), (900, 1185),
        (301, 17), (70, 101), (2000, 9), (3, 4097), (300, 3001), (5, 8191), (2, 8193),
        (400, 5120), (9, 6144), (300, 6148), (5, 5004), (40, 5002),
        (3, 8190), (9, 6662), (170, 3333), (40, 6655), (3, 6657), (200, 8192), (200, 2560)]


def addnorm_inputs(N, D, io, res, seed):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)
    x, r0 = n(N, D).to(IO[io]), (2 * n(N, D) + 1).to(IO[res])
    return x, r0, 1 + 0.3 * n(D), 0.5 + 0.3 * n(D), n(N, D).to(IO[io]), n(N, D).to(IO[res])


def check_addnorm(N, D, io, res, kind, rscale, w, resid, dr, seed):
    from linear_rnn_b200 import ops
    x, r0, wv, rs, dy, dr0 = addnorm_inputs(N, D, io, res, seed)
    wv, rs, r0, dr0 = wv if w else None, rs if rscale else None, r0 if resid else None, dr0 if dr else None
    xd, r0d, wd, rsd, dyd, drd = cuda(x, r0, wv, rs, dy, dr0)
    r, y = ops.gla_addnorm_fwd(xd, r0d, wd, rscale=rsd, alpha=0.7, kind=kind, eps=EPS, res_dtype=IO[res])
    assert r.dtype == IO[res] and y.dtype == IO[io]
    alpha = float(np.float32(0.7))
    rr, ry = norms.addnorm_fwd(f64(x), f64(r0), f64(rs), f64(wv), alpha, kind, EPS)
    term = np.abs(alpha * f64(x) * (1 if rs is None else f64(rs)))
    exact = 2 * U * (term + np.abs(rr))
    within(r, rr, HALF[IO[res]] * (np.abs(rr) + exact) + exact, "r")
    N_, rstd = row_bound(rr, kind)
    wabs = 1 if wv is None else np.abs(f64(wv))
    # the sum's own rounding moves n by exact * rstd, at most 4 u (term + |r|) rstd over the row
    moved = 4 * U * (term + np.abs(rr)).max(-1, keepdims=True) * rstd * (2 + N_ * N_)
    within(y, ry, HALF[IO[io]] * np.abs(ry) + (84 * U * N_ + moved) * wabs, "y")

    grads = ops.gla_addnorm_bwd(xd, r, wd, dyd, drd, rscale=rsd, alpha=0.7, kind=kind, eps=EPS)
    r64 = f64(r)
    ref = norms.addnorm_bwd(f64(x), r64, f64(rs), f64(wv), f64(dy), f64(dr0), alpha, kind, EPS)
    d = f64(dy) * (1 if wv is None else f64(wv))
    e = grad_bound(r64, d, kind) + 2 * U * np.abs(ref["dres"])
    within(grads["dres"], ref["dres"], HALF[IO[res]] * np.abs(ref["dres"]) + e, "dres")
    sc = np.abs(alpha * (1 if rs is None else f64(rs)))
    within(grads["dx"], ref["dx"], HALF[IO[io]] * np.abs(ref["dx"]) + sc * (e + 4 * U * np.abs(ref["dres"])), "dx")
    N_, _ = row_bound(r64, kind)
    if w:
        within(grads["dw"], ref["dw"], 200 * U * (np.abs(f64(dy)) * N_).sum(0), "dw")
    else:
        assert grads["dw"] is None
    if rscale:
        xa = np.abs(alpha * f64(x))
        within(grads["drscale"], ref["drscale"], (xa * (e + 110 * U * np.abs(ref["dres"]))).sum(0), "drscale")
    else:
        assert grads["drscale"] is None


@pytest.mark.parametrize("io,res", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("size", ROWS, ids=str)
def test_addnorm_matches_oracle(size, io, res, kind):
    if size[0] * size[1] * size[1] > 3e9:      # the oracle's Jacobians
        size = (2, size[1])
    odd = sum(size) % 2 == 1
    check_addnorm(*size, io, res, kind, rscale=odd, w=True, resid=True, dr=True, seed=61)


@pytest.mark.parametrize("rscale", [False, True])
@pytest.mark.parametrize("w", [False, True])
@pytest.mark.parametrize("resid", [False, True])
@pytest.mark.parametrize("dr", [False, True])
def test_addnorm_optional_arguments(rscale, w, resid, dr):
    check_addnorm(37, 136, "bf16", "bf16", "rms", rscale, w, resid, dr, 62)
    check_addnorm(6, 75, "f32", "f32", "layer", rscale, w, resid, dr, 63)


HEADS = [(1, 1, 1, 1), (2, 3, 5, 7), (1, 2, 3, 8), (2, 2, 33, 64), (3, 5, 21, 100), (1, 4, 130, 128), (2, 3, 40, 256),
         (1, 17, 9, 36), (64, 4, 1, 64), (1, 2, 300, 24), (1, 2, 4, 512), (2, 1, 3, 1028), (1, 2, 2, 4096), (1, 1, 2, 9001),
         (3, 5, 700, 50), (2, 3, 200, 258), (3, 2, 500, 75), (1, 1, 2, 4102), (3, 5, 301, 9), (2, 3, 71, 101),
         (2, 3, 17, 129), (1, 3, 41, 1001), (1, 2, 5, 4095), (1, 2, 3, 8191)]


def headnorm_inputs(B, H, L, D, io, per_head, seed):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)
    return ((2 * n(B, H, L, D) + 0.5).to(IO[io]), (2 * n(B, L, H, D)).to(IO[io]),
            1 + 0.3 * (n(H, D) if per_head else n(D)), n(B, L, H, D).to(IO[io]))


def check_headnorm(B, H, L, D, io, kind, act, per_head, gate, w, seed):
    from linear_rnn_b200 import ops
    o, z, wv, dy = headnorm_inputs(B, H, L, D, io, per_head, seed)
    z, wv = z if gate else None, wv if w else None
    od, zd, wd, dyd = cuda(o, z, wv, dy)
    y = ops.gla_headnorm_fwd(od, zd, wd, act=act, kind=kind, eps=EPS)
    grads = ops.gla_headnorm_bwd(od, zd, wd, dyd, act=act, kind=kind, eps=EPS)
    ry = norms.headnorm_fwd(f64(o), f64(z), f64(wv), act, kind, EPS)
    ref = norms.headnorm_bwd(f64(o), f64(z), f64(wv), f64(dy), act, kind, EPS)
    N_, _ = row_bound(f64(o), kind)
    Nt = N_.transpose(0, 2, 1, 3)
    wabs = 1 if wv is None else np.abs(f64(wv))
    f, df, zabs = (1.0, 0.0, 0.0) if z is None else (*norms.act(f64(z), act), np.abs(f64(z)))
    within(y, ry, HALF[IO[io]] * np.abs(ry) + 84 * U * Nt * wabs * np.abs(f), "y")
    if gate:
        e = np.abs(f64(dy)) * wabs * Nt * (84 * U * np.abs(df) + 12 * U * (1 + zabs))
        within(grads["dz"], ref["dz"], HALF[IO[io]] * np.abs(ref["dz"]) + e, "dz")
    else:
        assert grads["dz"] is None
    d = (np.abs(f64(dy) * f) * wabs).transpose(0, 2, 1, 3)
    within(grads["do"], ref["do"], HALF[IO[io]] * np.abs(ref["do"]) + grad_bound(f64(o), d, kind), "do")
    if w:
        term = np.abs(f64(dy) * f) * Nt
        within(grads["dw"], ref["dw"], 200 * U * term.sum((0, 1) if per_head else (0, 1, 2)), "dw")
    else:
        assert grads["dw"] is None


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("kind,act,per_head", [("rms", "silu", False), ("layer", "sigmoid", True),
                                               ("rms", "sigmoid", True), ("layer", "silu", False)])
@pytest.mark.parametrize("size", HEADS, ids=str)
def test_headnorm_matches_oracle(size, io, kind, act, per_head):
    check_headnorm(*size, io, kind, act, per_head, True, True, 64)


@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("w", [False, True])
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_headnorm_optional_arguments(gate, w, io):
    check_headnorm(2, 3, 20, 64, io, "rms", "silu", False, gate, w, 65)


def test_gate_extremes():
    """Gates far on both sides: no overflow, the sigmoid's limits."""
    from linear_rnn_b200 import ops
    z = torch.tensor([-1e30, -200.0, -90.0, -20.0, 0.0, 20.0, 200.0, 1e30], device="cuda").view(1, 1, 1, 8)
    o, dy = torch.randn(1, 1, 1, 8, device="cuda"), torch.randn(1, 1, 1, 8, device="cuda")
    for act in ("silu", "sigmoid"):
        y = ops.gla_headnorm_fwd(o, z, None, act=act, eps=EPS)
        g = ops.gla_headnorm_bwd(o, z, None, dy, act=act, eps=EPS)
        n, (f, df) = norms.norm(f64(o), "rms", EPS), norms.act(f64(z), act)
        lim = np.abs(f64(z)) * 2.0 ** -126 if act == "silu" else 2.0 ** -126
        within(y, n * f, 100 * U * np.abs(n * f) + 4 * lim, act)
        within(g["dz"], f64(dy) * n * df, 100 * U * np.abs(f64(dy) * n) * (np.abs(df) + U * 0) + 4 * lim
               + 12 * U * np.abs(f64(dy) * n) * (np.abs(f64(z)) < 100) * (1 + np.minimum(np.abs(f64(z)), 100)), act)
        assert all(torch.isfinite(v).all() for v in (y, g["do"], g["dz"]))


@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_rows_of_zeros_constant_rows_and_large_offsets(kind):
    """A row of zeros gives zeros and finite gradients; a constant row's layer norm is zero; a row far
    from zero keeps the digits that its variance has (the mean is taken off before squaring)."""
    from linear_rnn_b200 import ops
    D = 320
    gen = torch.Generator().manual_seed(5)
    r = torch.randn(4, D, generator=gen)
    r[0] = 0
    r[1] = 3.0
    r[2] += 1000.0
    x, dy = torch.zeros(4, D), torch.randn(4, D, generator=gen)
    xd, rd, dyd = cuda(x, r, dy)
    _, y = ops.gla_addnorm_fwd(xd, rd, None, kind=kind, eps=EPS)
    g = ops.gla_addnorm_bwd(None, rd, None, dyd, kind=kind, eps=EPS)
    N_, _ = row_bound(f64(r), kind)
    within(y, norms.norm(f64(r), kind, EPS), 84 * U * N_, "y")
    assert (y[0] == 0).all()
    ref = norms.norm_vjp(f64(r), f64(dy), kind, EPS)
    within(g["dres"], ref, grad_bound(f64(r), f64(dy), kind) * (1 + N_), "dres")


def test_non_finite_rows_stay_in_their_row():
    from linear_rnn_b200 import ops
    r = torch.randn(6, 200, device="cuda")
    r[2, 7], r[4, 9] = float("inf"), float("nan")
    _, y = ops.gla_addnorm_fwd(torch.zeros_like(r), r)
    ok = [0, 1, 3, 5]
    assert torch.isfinite(y[ok]).all() and torch.isnan(y[4]).all() and torch.isnan(y[2, 7])


@pytest.mark.parametrize("shape", [(0, 8), (3, 0, 16)])
def test_empty_rows(shape):
    from linear_rnn_b200 import ops
    x, w, s = torch.empty(*shape, device="cuda"), torch.ones(shape[-1], device="cuda"), torch.ones(shape[-1], device="cuda")
    r, y = ops.gla_addnorm_fwd(x, x, w, rscale=s)
    assert r.shape == y.shape == x.shape
    g = ops.gla_addnorm_bwd(x, x, w, x, rscale=s)
    assert (g["dw"] == 0).all() and (g["drscale"] == 0).all() and g["dx"].shape == x.shape
    for B, H, L in ((0, 2, 3), (2, 0, 3), (2, 3, 0)):
        o, z, w = (torch.empty(B, H, L, 8, device="cuda"), torch.empty(B, L, H, 8, device="cuda"),
                   torch.ones(8, device="cuda"))
        assert ops.gla_headnorm_fwd(o, z, w).shape == (B, L, H, 8)
        assert (ops.gla_headnorm_bwd(o, z, w, z)["dw"] == 0).all()


def test_leading_dimensions_host_tensors_and_in_place():
    from linear_rnn_b200 import _lib, ops
    x, r0, w, rs, dy, dr = addnorm_inputs(30, 96, "bf16", "f32", 66)
    flat = ops.gla_addnorm_fwd(*cuda(x, r0, w), rscale=rs.cuda())
    deep = ops.gla_addnorm_fwd(*cuda(x.view(2, 3, 5, 96), r0.view(2, 3, 5, 96), w), rscale=rs.cuda())
    host = ops.gla_addnorm_fwd(x, r0, w, rscale=rs)
    for a, b, c in zip(flat, deep, host):
        assert torch.equal(a, b.view(30, 96)) and c.device.type == "cpu" and torch.equal(a.cpu(), c)
    g = ops.gla_addnorm_bwd(*cuda(x), flat[0], *cuda(w, dy, dr), rscale=rs.cuda())
    gh = ops.gla_addnorm_bwd(x, flat[0].cpu(), w, dy, dr, rscale=rs)
    for n in g:
        assert torch.equal(g[n].cpu(), gh[n]), n
    # r may be res, dres may be dr
    p = _lib.GlaNormProblem(1, 1, 30, 96, 1, 0, 0, 0, 0, 1e-6, 1.0)
    ptr = lambda t: None if t is None else ctypes.c_void_p(t.data_ptr())
    xd, rd, wd, rsd, dyd, drd = cuda(x, r0, w, rs, dy, dr)
    y = torch.empty_like(xd)
    st = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert _lib.lib.gla_addnorm_fwd(ctypes.byref(p), ptr(xd), ptr(rd), ptr(rsd), ptr(wd), ptr(rd), ptr(y), st) == 0
    assert torch.equal(rd, flat[0]) and torch.equal(y, flat[1])
    nb = _lib.lib.gla_addnorm_workspace_bytes(ctypes.byref(p))
    ws = torch.full((nb + 256,), 9, dtype=torch.uint8, device="cuda")
    assert _lib.lib.gla_addnorm_bwd(ctypes.byref(p), ptr(xd), ptr(rd), ptr(rsd), ptr(wd), ptr(dyd), ptr(drd), ptr(drd),
                                    None, None, None, ptr(ws), nb, st) == 0
    assert torch.equal(drd, g["dres"])
    assert (ws[nb:] == 9).all()


@pytest.mark.parametrize("D", [24, 100, 256, 1030])
def test_nothing_outside_the_outputs_is_written(D):
    from linear_rnn_b200 import ops
    B, H, L = 3, 2, 37
    o, z, w, dy = cuda(*headnorm_inputs(B, H, L, D, "bf16", True, 67))
    p = ops._headnorm_problem(o, w, "silu", "rms", 1e-6)
    from linear_rnn_b200 import _lib
    nb = _lib.lib.gla_headnorm_workspace_bytes(ctypes.byref(p))
    n = o.numel()
    bufs = [torch.full((n + 64,), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    dw = torch.full((H * D + 64,), float("nan"), device="cuda")
    ws = torch.full((nb + 64,), 9, dtype=torch.uint8, device="cuda")
    ptr = lambda t: ctypes.c_void_p(t.data_ptr())
    st = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert _lib.lib.gla_headnorm_fwd(ctypes.byref(p), ptr(o), ptr(z), ptr(w), ptr(bufs[0]), st) == 0
    assert _lib.lib.gla_headnorm_bwd(ctypes.byref(p), ptr(o), ptr(z), ptr(w), ptr(dy), ptr(bufs[1]), ptr(bufs[2]),
                                     ptr(dw), ptr(ws), nb, st) == 0
    for t, m in [(b, n) for b in bufs] + [(dw, H * D)]:
        assert torch.isfinite(t[:m]).all() and torch.isnan(t[m:]).all()
    assert (ws[nb:] == 9).all()


def test_row_sums_repeat_bit_for_bit():
    from linear_rnn_b200 import ops
    x, r0, w, rs, dy, dr = cuda(*addnorm_inputs(5000, 264, "bf16", "bf16", 68))
    a, b = (ops.gla_addnorm_bwd(x, r0, w, dy, dr, rscale=rs) for _ in range(2))
    o, z, hw, hdy = cuda(*headnorm_inputs(2, 4, 900, 64, "bf16", False, 69))
    c, d = (ops.gla_headnorm_bwd(o, z, hw, hdy) for _ in range(2))
    for p, q in ((a, b), (c, d)):
        for n in p:
            assert torch.equal(p[n], q[n]), n


def test_few_rows_need_no_workspace():
    """One block's column sums are the result: no workspace, nothing else launched."""
    from linear_rnn_b200 import _lib, ops
    x, r0, w, rs, dy, dr = cuda(*addnorm_inputs(3, 64, "bf16", "bf16", 76))
    n0 = _lib.launch_count()
    g = ops.gla_addnorm_bwd(x, r0, w, dy, dr, rscale=rs, eps=EPS)
    assert _lib.launch_count() == n0 + 1
    ref = norms.addnorm_bwd(f64(x), f64(r0), f64(rs), f64(w), f64(dy), f64(dr), 1.0, "rms", EPS)
    for n in ("dw", "drscale"):
        within(g[n], ref[n], 1e-5 * np.abs(ref[n]).max(), n)
    check_headnorm(1, 6, 2, 64, "f32", "layer", "silu", True, True, True, 77)    # one block per head, its own weights
    check_headnorm(1, 1, 2, 64, "f32", "layer", "silu", False, True, True, 78)
    check_headnorm(1, 6, 2, 64, "f32", "layer", "silu", False, True, True, 79)   # heads share them: summed


def test_many_rows():
    """More rows than any grid: every block walks several, and the sums over rows are long (their tolerance
    counts the additions that follow one another: rows over blocks and groups, here below 200 in all)."""
    check_headnorm(2, 2, 4000, 16, "f32", "layer", "silu", True, True, True, 70)
    check_addnorm(9000, 24, "bf16", "bf16", "rms", True, True, True, True, 71)


def test_graphs_and_streams():
    from linear_rnn_b200 import ops
    x, r0, w, rs, dy, dr = cuda(*addnorm_inputs(200, 512, "bf16", "bf16", 72))
    o, z, hw, hdy = cuda(*headnorm_inputs(2, 4, 60, 64, "bf16", False, 73))

    def run():
        r, y = ops.gla_addnorm_fwd(x, r0, w, rscale=rs)
        return (r, y, *ops.gla_addnorm_bwd(x, r, w, dy, dr, rscale=rs).values(), ops.gla_headnorm_fwd(o, z, hw),
                *ops.gla_headnorm_bwd(o, z, hw, hdy).values())
    want = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs = run()
        graphs.append((gr, outs))
    for _, outs in graphs:
        for t in outs:
            t.fill_(float("nan"))
    for gr, _ in graphs:
        gr.replay()
    torch.cuda.synchronize()
    for outs in (got, graphs[0][1], graphs[1][1]):
        for a, b in zip(want, outs):
            assert torch.equal(a, b)


def test_refusals():
    from linear_rnn_b200 import _lib, ops
    x, r0, w, rs, dy, dr = cuda(*addnorm_inputs(4, 32, "bf16", "bf16", 74))
    o, z, hw, hdy = cuda(*headnorm_inputs(2, 3, 4, 32, "bf16", True, 75))
    for bad in (lambda: ops.gla_addnorm_fwd(x.half(), r0, w), lambda: ops.gla_addnorm_fwd(x, r0, w.bfloat16()),
                lambda: ops.gla_addnorm_fwd(x, r0[:2].contiguous(), w), lambda: ops.gla_addnorm_fwd(x, r0, w, kind="batch"),
                lambda: ops.gla_addnorm_fwd(x, r0, w[:16].contiguous()), lambda: ops.gla_addnorm_fwd(x.t(), r0.t(), None),
                lambda: ops.gla_addnorm_fwd(x, r0, w, res_dtype=torch.float32),
                lambda: ops.gla_addnorm_bwd(None, r0, w, dy, rscale=rs), lambda: ops.gla_addnorm_bwd(x, r0, w, dy, dr.float()),
                lambda: ops.gla_headnorm_fwd(o, z.transpose(1, 2).contiguous(), hw), lambda: ops.gla_headnorm_fwd(o, z, hw.t()),
                lambda: ops.gla_headnorm_fwd(o, z.float(), hw), lambda: ops.gla_headnorm_fwd(o, z, hw, act="relu"),
                lambda: ops.gla_headnorm_bwd(o, z, hw, None), lambda: ops.gla_headnorm_fwd(o.transpose(1, 2), z, hw)):
        with pytest.raises((ValueError, TypeError)):
            bad()
    for bad, status in ((lambda: ops.gla_addnorm_fwd(x, r0, w, eps=0.0), _lib.GLA_ERR_INVALID_ARG),
                        (lambda: ops.gla_addnorm_fwd(x.float(), r0, w), _lib.GLA_ERR_UNSUPPORTED),
                        (lambda: ops.gla_addnorm_bwd(x, r0, w, dy, workspace=torch.empty(64, dtype=torch.uint8, device="cuda")),
                         _lib.GLA_ERR_WORKSPACE),
                        (lambda: ops.gla_addnorm_fwd(torch.zeros(1, 16385, device="cuda")), _lib.GLA_ERR_UNSUPPORTED)):
        with pytest.raises(_lib.GlaError) as e:
            bad()
        assert e.value.status == status


def layer_inputs(seed, B, H, L, D, io):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)
    M = H * D
    return {"x": n(B, L, M).to(IO[io]), "res": n(B, L, M).to(IO[io]), "w1": 1 + 0.2 * n(M), "rs": 0.5 + 0.2 * n(M),
            "g": torch.nn.functional.logsigmoid(n(B, H, L, D) + 2), "z": n(B, L, H, D).to(IO[io]),
            "w2": 1 + 0.2 * n(D), "h0": n(B, H, D), "dy": n(B, L, M).to(IO[io]), "dr": n(B, L, M).to(IO[io])}


@pytest.mark.parametrize("L", [1, 150])
def test_one_layer_forward_and_backward(L):
    """addnorm -> scan -> headnorm -> addnorm and back, in fp32, against the float64 oracles in a chain.
    Tolerance: each of the four stages is within 1e-5 of its output's largest value on these inputs
    (their own bounds above), and passes its input's error on with a gain below 8 here."""
    from linear_rnn_b200 import ops
    B, H, D = 2, 3, 40
    M = H * D
    t = layer_inputs(80, B, H, L, D, "f32")
    c = {k: v.cuda() for k, v in t.items()}
    f = {k: f64(v) for k, v in t.items()}
    split = lambda v: v.view(B, L, H, D).transpose(1, 2).contiguous()
    join = lambda v: v.transpose(1, 2).reshape(B, L, M).contiguous()
    r1, y1 = ops.gla_addnorm_fwd(c["x"], c["res"], c["w1"], rscale=c["rs"], eps=EPS)
    o, hT = ops.gla_scan_fwd(split(y1), c["g"], c["h0"], input="complement")
    u = ops.gla_headnorm_fwd(o, c["z"], c["w2"], eps=EPS)
    r2, y2 = ops.gla_addnorm_fwd(u.view(B, L, M), r1, c["w1"], rscale=c["rs"], kind="layer", eps=EPS)
    g4 = ops.gla_addnorm_bwd(u.view(B, L, M), r2, c["w1"], c["dy"], c["dr"], rscale=c["rs"], kind="layer", eps=EPS)
    g3 = ops.gla_headnorm_bwd(o, c["z"], c["w2"], g4["dx"].view(B, L, H, D), eps=EPS)
    g2 = ops.gla_scan_bwd(split(y1), c["g"], c["h0"], g3["do"], input="complement")
    g1 = ops.gla_addnorm_bwd(c["x"], r1, c["w1"], join(g2["dx"]), g4["dres"], rscale=c["rs"], eps=EPS)

    nsplit = lambda v: v.reshape(B, L, H, D).transpose(0, 2, 1, 3)
    njoin = lambda v: v.transpose(0, 2, 1, 3).reshape(B, L, M)
    flat = lambda v: v.reshape(B * L, M)
    R1, Y1 = norms.addnorm_fwd(f["x"], f["res"], f["rs"], f["w1"], 1.0, "rms", EPS)
    O, HT = scan.scan_fwd(nsplit(Y1), f["g"], f["h0"], "complement")
    Uu = norms.headnorm_fwd(O, f["z"], f["w2"], "silu", "rms", EPS)
    R2, Y2 = norms.addnorm_fwd(Uu.reshape(B, L, M), R1, f["rs"], f["w1"], 1.0, "layer", EPS)
    G4 = norms.addnorm_bwd(flat(Uu), flat(R2), f["rs"], f["w1"], flat(f["dy"]), flat(f["dr"]), 1.0, "layer", EPS)
    G3 = norms.headnorm_bwd(O, f["z"], f["w2"], G4["dx"].reshape(B, L, H, D), "silu", "rms", EPS)
    G2 = scan.scan_bwd(nsplit(Y1), f["g"], f["h0"], G3["do"], None, "complement")
    G1 = norms.addnorm_bwd(flat(f["x"]), flat(R1), f["rs"], f["w1"], flat(njoin(G2["dx"])), G4["dres"], 1.0, "rms", EPS)
    pairs = {"y2": (y2, Y2), "hT": (hT, HT), "dz": (g3["dz"], G3["dz"]), "dw2": (g3["dw"], G3["dw"]),
             "dg": (g2["dg"], G2["dg"]), "dh0": (g2["dh0"], G2["dh0"]), "dx": (g1["dx"].view(B * L, M), G1["dx"]),
             "dres": (g1["dres"].view(B * L, M), G1["dres"]), "drs": (g1["drscale"], G1["drscale"]),
             "dw1": (g1["dw"], G1["dw"])}
    for name, (a, b) in pairs.items():
        within(a, b, 4 * 8 * 1e-5 * np.abs(b).max(), name)


def test_layer_around_the_matrix_state_cell():
    """headnorm takes the gated linear attention forward's output as it is, and its gradient feeds that
    cell's backward: the chain equals the two float64 oracles joined (bf16 cell: its own 1e-2)."""
    import oracle
    from linear_rnn_b200 import inputs as I, ops
    w = I.WORKLOADS["c3"].replace(B=2, H=3, L=130, Dk=64, Dv=128)
    x = I.make_inputs(w, seed=81)
    xd = {k: (None if v is None else v.cuda()) for k, v in x.items()}
    _, z, hw, dy = headnorm_inputs(2, 3, 130, 128, "bf16", True, 82)
    o, _ = ops.gla_fwd(xd["q"], xd["k"], xd["v"], xd["g"], scale=w.scale)
    y = ops.gla_headnorm_fwd(o, z.cuda(), hw.cuda(), kind="layer", act="sigmoid", eps=EPS)
    gn = ops.gla_headnorm_bwd(o, z.cuda(), hw.cuda(), dy.cuda(), kind="layer", act="sigmoid", eps=EPS)
    # given the cell's own o, the norm adds only its own error
    ry = norms.headnorm_fwd(f64(o), f64(z), f64(hw), "sigmoid", "layer", EPS)
    rn = norms.headnorm_bwd(f64(o), f64(z), f64(hw), f64(dy), "sigmoid", "layer", EPS)
    within(y, ry, 2.0 ** -8 * np.abs(ry) + 1e-5 * np.abs(ry).max(), "y")
    within(gn["do"], rn["do"], 2.0 ** -8 * np.abs(rn["do"]) + 1e-5 * np.abs(rn["do"]).max(), "do")
    gb = ops.gla_bwd(xd["q"], xd["k"], xd["v"], xd["g"], None, None, gn["do"], scale=w.scale)
    rb = oracle.gla_bwd(x["q"], x["k"], x["v"], x["g"], None, None, gn["do"].cpu(), None, w.scale)
    for n in ("dq", "dk", "dv", "dg"):
        a = f64(gb[n])
        assert np.abs(a - rb[n]).max() <= 1e-2 * np.abs(rb[n]).max(), n


def test_offsets_past_32_bits():
    """More than 2^31 elements: the last rows against the oracle, in both operators and directions."""
    from linear_rnn_b200 import ops
    D, rows = 8208, (1 << 18) + 5
    x = torch.empty(rows, D, dtype=torch.bfloat16, device="cuda")
    for t in range(0, rows, 1 << 16):
        x[t:t + (1 << 16)].normal_()
    r, y = ops.gla_addnorm_fwd(x, x, None, eps=EPS)
    tail = f64(x[-3:])
    rr, ry = norms.addnorm_fwd(tail, tail, None, None, 1.0, "rms", EPS)
    within(r[-3:], rr, 2.0 ** -8 * np.abs(rr) + 1e-6, "r")
    within(y[-3:], ry, 2.0 ** -8 * np.abs(ry) + 1e-5, "y")
    del y
    g = ops.gla_addnorm_bwd(None, r, None, x, x, eps=EPS)
    rb = norms.addnorm_bwd(tail, f64(r[-3:]), None, None, tail, tail, 1.0, "rms", EPS)
    within(g["dres"][-3:], rb["dres"], 2.0 ** -8 * np.abs(rb["dres"]) + 1e-5, "dres")
    within(g["dx"][-3:], rb["dx"], 2.0 ** -8 * np.abs(rb["dx"]) + 1e-5, "dx")
    del g, r
    H, Dh = 19, 432                      # the same memory as heads of one sequence
    o, z = x.view(1, H, rows, Dh), x.view(1, rows, H, Dh)
    y = ops.gla_headnorm_fwd(o, z, None, eps=EPS)
    o2, z2 = f64(o[:, :, -2:]), f64(z[:, -2:])
    ry = norms.headnorm_fwd(o2, z2, None, "silu", "rms", EPS)
    within(y[:, -2:], ry, 2.0 ** -8 * np.abs(ry) + 1e-5, "head y")
    del y
    g = ops.gla_headnorm_bwd(o, z, None, z, eps=EPS)
    rb = norms.headnorm_bwd(o2, z2, None, z2, "silu", "rms", EPS)
    within(g["do"][:, :, -2:], rb["do"], 2.0 ** -8 * np.abs(rb["do"]) + 1e-5, "do")
    within(g["dz"][:, -2:], rb["dz"], 2.0 ** -8 * np.abs(rb["dz"]) + 3e-5, "dz")


FIRST_CALL_IN_CAPTURE = """
import torch
from linear_rnn_b200 import ops
n = lambda *s: torch.randn(*s, device="cuda")
x, g, dO = n(2, 3, 200, 64), -n(2, 3, 200, 64).abs(), n(2, 3, 200, 64)
a, w = n(600, 1000).bfloat16(), n(1000)
o, z, v = n(2, 3, 300, 96), n(2, 300, 3, 96), n(96)
torch.cuda.synchronize()
def run():
    r, y = ops.gla_addnorm_fwd(a, a, w, rscale=w, kind="layer")
    out = [*ops.gla_scan_fwd(x, g), *ops.gla_scan_bwd(x, g, None, dO).values(), r, y]
    out += list(ops.gla_addnorm_bwd(a, r, w, a, rscale=w, kind="layer").values())
    return out + [ops.gla_headnorm_fwd(o, z, v), *ops.gla_headnorm_bwd(o, z, v, z).values()]
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = run()
graph.replay()
want = run()
torch.cuda.synchronize()
assert all(torch.equal(p, q) for p, q in zip(got, want))
print("same")
"""


def test_first_call_of_a_process_may_be_captured():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL_IN_CAPTURE], cwd=root, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


def test_host_threads_with_their_own_streams():
    """Calls at once from several host threads, each on its own stream, give the single call's bits."""
    import threading
    from linear_rnn_b200 import ops
    x, r0, w, rs, dy, dr = cuda(*addnorm_inputs(900, 1024, "bf16", "bf16", 90))
    o, z, hw, hdy = cuda(*headnorm_inputs(2, 4, 300, 64, "bf16", False, 91))
    xs, g = torch.randn(2, 4, 700, 64, device="cuda"), -torch.rand(2, 4, 700, 64, device="cuda")

    def run():
        r, y = ops.gla_addnorm_fwd(x, r0, w, rscale=rs)
        return [y, *ops.gla_addnorm_bwd(x, r, w, dy, dr, rscale=rs).values(), ops.gla_headnorm_fwd(o, z, hw),
                *ops.gla_headnorm_bwd(o, z, hw, hdy).values(), *ops.gla_scan_fwd(xs, g),
                *ops.gla_scan_bwd(xs, g, None, xs).values()]
    want = run()
    torch.cuda.synchronize()
    bad = []

    def work():
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                got = run()
            torch.cuda.current_stream().synchronize()
            if not all(torch.equal(a, b) for a, b in zip(want, got)):
                bad.append(1)
    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_a_changed_scalar_is_seen():
    """alpha and eps given as tensors are read at each call."""
    from linear_rnn_b200 import ops
    x, r0 = torch.randn(5, 64).cuda(), torch.randn(5, 64).cuda()
    alpha, eps = torch.tensor(2.0), torch.tensor(1e-6)
    ops.gla_addnorm_fwd(x, r0, alpha=alpha, eps=eps)
    ops.gla_headnorm_fwd(x.view(1, 1, 5, 64), eps=eps)
    alpha.fill_(3.0)
    eps.fill_(0.5)
    r, y = ops.gla_addnorm_fwd(x, r0, alpha=alpha, eps=eps)
    want_r, want_y = ops.gla_addnorm_fwd(x, r0, alpha=3.0, eps=0.5)
    assert torch.equal(r, want_r) and torch.equal(y, want_y)
    got = ops.gla_addnorm_bwd(None, r, None, x, alpha=alpha, eps=eps)
    want = ops.gla_addnorm_bwd(None, r, None, x, alpha=3.0, eps=0.5)
    assert torch.equal(got["dres"], want["dres"]) and torch.equal(got["dx"], want["dx"])
    o = x.view(1, 1, 5, 64)
    assert torch.equal(ops.gla_headnorm_fwd(o, eps=eps), ops.gla_headnorm_fwd(o, eps=0.5))


def test_buffers_on_the_host_are_refused():
    """A host buffer next to host tensors would be written on the device only."""
    from linear_rnn_b200 import ops
    x, g = torch.randn(1, 1, 100, 8), -torch.rand(1, 1, 100, 8)
    buf = torch.zeros(1 << 16, dtype=torch.uint8)
    with pytest.raises(ValueError):
        ops.gla_scan_fwd(x, g, saved_states=buf)
    with pytest.raises(ValueError):
        ops.gla_scan_bwd(x, g, None, x, saved_states=buf)
    with pytest.raises(ValueError):
        ops.gla_scan_bwd(x, g, None, x, workspace=buf)
    with pytest.raises(ValueError):
        ops.gla_addnorm_bwd(None, x, None, x, workspace=buf)
    with pytest.raises(ValueError):
        ops.gla_headnorm_bwd(x, None, None, x.view(1, 100, 1, 8), workspace=buf)
    o, hT = ops.gla_scan_fwd(x, g, saved_states=buf.cuda())
    want_o, want_hT = ops.gla_scan_fwd(x, g)
    assert torch.equal(o, want_o) and torch.equal(hT, want_hT)
