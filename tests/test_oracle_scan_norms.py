"""Pins of the float64 oracles of the vector-state recurrence and of the norms: closed forms,
invariants and central differences; none re-types the oracle's formula."""
import numpy as np
import pytest

import oracle
from oracle import norms, scan

rng = np.random.default_rng


def close(a, b, tol=1e-9):
    a, b = np.asarray(a), np.asarray(b)
    assert a.shape == b.shape
    assert np.abs(a - b).max(initial=0.0) <= tol * (1 + np.abs(b).max(initial=0.0))


def differences(f, v, eps=1e-6):
    """Central differences of the scalar f with respect to every element of v (changed in place)."""
    out = np.empty_like(v)
    for i in np.ndindex(v.shape):
        keep = v[i]
        v[i] = keep + eps
        up = f()
        v[i] = keep - eps
        down = f()
        v[i] = keep
        out[i] = (up - down) / (2 * eps)
    return out


@pytest.mark.parametrize("kind", ["plain", "complement", "norm"])
def test_scan_is_the_sum_over_explicit_products_of_decays(kind):
    r = rng(1)
    x, g, h0 = r.normal(size=(2, 1, 9, 3)), -np.abs(r.normal(size=(2, 1, 9, 3))), r.normal(size=(2, 1, 3))
    a = np.exp(g)
    m = {"plain": 1.0 + 0 * a, "complement": 1 - a, "norm": np.sqrt(1 - a * a)}[kind]
    o, hT = scan.scan_fwd(x, g, h0, kind)
    for t in range(9):
        want = h0 * a[:, :, :t + 1].prod(2)
        for s in range(t + 1):
            want = want + a[:, :, s + 1:t + 1].prod(2) * m[:, :, s] * x[:, :, s]
        close(o[:, :, t], want)
    close(hT, o[:, :, -1])


def test_scan_is_the_diagonal_of_the_matrix_recurrence():
    """One key of ones and values x: every row of the matrix state with the same gate is h."""
    r = rng(2)
    L, D = 11, 4
    x, g = r.normal(size=(1, 1, L, D)), -np.abs(r.normal(size=(1, 1, L, D)))
    o, _ = scan.scan_fwd(x, g)
    for d in range(D):   # Dk = 1 is not a library size but the oracle takes any
        ro, _ = oracle.gla_fwd(np.ones((1, 1, L, 1)), np.ones((1, 1, L, 1)), x[..., d:d + 1], g[..., d:d + 1], None,
                               None, 1.0)
        close(np.asarray(ro)[..., 0], o[..., d], 1e-6)


def test_scan_special_gates_and_handoff():
    r = rng(3)
    x, h0 = r.normal(size=(2, 3, 10, 5)), r.normal(size=(2, 3, 5))
    close(scan.scan_fwd(x, np.zeros_like(x))[0], np.cumsum(x, 2))                     # no decay
    g = np.full_like(x, -np.inf)
    close(scan.scan_fwd(x, g, h0)[0], x)                                             # every token starts anew
    close(scan.scan_fwd(x, g, h0, "norm")[0], x)
    close(scan.scan_fwd(np.ones_like(x), np.full_like(x, -0.3), np.ones_like(h0), "complement")[0], np.ones_like(x))
    g = -np.abs(r.normal(size=x.shape))
    g[:, :, 6] = -np.inf
    o, hT = scan.scan_fwd(x, g, h0)
    close(o[:, :, 6:], scan.scan_fwd(x[:, :, 6:], g[:, :, 6:])[0])                    # a start cuts the past off
    o1, h1 = scan.scan_fwd(x[:, :, :4], g[:, :, :4], h0)
    o2, h2 = scan.scan_fwd(x[:, :, 4:], g[:, :, 4:], h1)
    close(np.concatenate([o1, o2], 2), o)
    close(h2, hT)
    o, hT = scan.scan_fwd(x[:, :, :0], g[:, :, :0], h0)
    assert o.shape == (2, 3, 0, 5)
    close(hT, h0)


@pytest.mark.parametrize("kind", ["plain", "complement", "norm"])
def test_scan_gradients_are_differences(kind):
    r = rng(4)
    x, g, h0 = r.normal(size=(1, 2, 6, 3)), -0.05 - np.abs(r.normal(size=(1, 2, 6, 3))), r.normal(size=(1, 2, 3))
    dO, dhT = r.normal(size=x.shape), r.normal(size=h0.shape)

    def loss():
        o, hT = scan.scan_fwd(x, g, h0, kind)
        return (dO * o).sum() + (dhT * hT).sum()
    got = scan.scan_bwd(x, g, h0, dO, dhT, kind)
    for name, v in (("dx", x), ("dg", g), ("dh0", h0)):
        close(got[name], differences(loss, v), 1e-6)


@pytest.mark.parametrize("kind", ["plain", "norm"])
def test_scan_gradient_stops_at_a_start(kind):
    r = rng(5)
    x, g, dO = r.normal(size=(1, 1, 8, 2)), -np.abs(r.normal(size=(1, 1, 8, 2))), r.normal(size=(1, 1, 8, 2))
    h0 = r.normal(size=(1, 1, 2))
    g[:, :, 5] = -np.inf
    got = scan.scan_bwd(x, g, h0, dO, None, kind)
    assert (got["dg"][:, :, 5] == 0).all()
    close(got["dx"][:, :, :5], scan.scan_bwd(x[:, :, :5], g[:, :, :5], h0, dO[:, :, :5], None, kind)["dx"])


@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_norm_statistics(kind):
    r = rng(6).normal(size=(7, 33)) * 3 + 2
    n = norms.norm(r, kind, 1e-12)
    close((n * n).mean(-1), np.ones(7), 1e-6)
    if kind == "layer":
        close(n.mean(-1), np.zeros(7), 1e-12)
        close(norms.norm(r + 5.0, kind, 1e-12), n)
    close(norms.norm(4.0 * r, kind, 1e-14), norms.norm(r, kind, 1e-14), 1e-9)
    close(norms.norm(np.zeros((2, 8)), kind, 1e-6), np.zeros((2, 8)))


@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_addnorm_gradients_are_differences(kind):
    r = rng(7)
    x, res, rs, w = r.normal(size=(3, 5)), r.normal(size=(3, 5)), r.normal(size=5), r.normal(size=5)
    dy, dr = r.normal(size=(3, 5)), r.normal(size=(3, 5))

    def loss():
        rr, y = norms.addnorm_fwd(x, res, rs, w, 0.7, kind, 1e-3)
        return (dy * y).sum() + (dr * rr).sum()
    rr, _ = norms.addnorm_fwd(x, res, rs, w, 0.7, kind, 1e-3)
    got = norms.addnorm_bwd(x, rr, rs, w, dy, dr, 0.7, kind, 1e-3)
    for name, v in (("dres", res), ("dx", x), ("dw", w), ("drscale", rs)):
        close(got[name], differences(loss, v), 1e-6)


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("act", ["silu", "sigmoid"])
@pytest.mark.parametrize("per_head", [False, True])
def test_headnorm_gradients_are_differences(kind, act, per_head):
    r = rng(8)
    o, z, dy = r.normal(size=(2, 3, 2, 4)), r.normal(size=(2, 2, 3, 4)), r.normal(size=(2, 2, 3, 4))
    w = r.normal(size=(3, 4) if per_head else 4)

    def loss():
        return (dy * norms.headnorm_fwd(o, z, w, act, kind, 1e-3)).sum()
    got = norms.headnorm_bwd(o, z, w, dy, act, kind, 1e-3)
    for name, v in (("do", o), ("dz", z), ("dw", w)):
        close(got[name], differences(loss, v), 1e-6)


def test_activations_closed_forms():
    z = np.array([-700.0, -3.0, 0.0, 2.0, 50.0])
    with np.errstate(over="ignore"):
        s = 1 / (1 + np.exp(-z))
    close(norms.act(z, "sigmoid")[0], s)
    close(norms.act(z, "silu")[0], z * s)
