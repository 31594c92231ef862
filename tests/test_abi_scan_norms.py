"""Host-only checks of gla_scan_*, gla_addnorm_* and gla_headnorm_*: sizes and refusals, before any
CUDA call (every call here fails validation, or asks for a size)."""
import ctypes

import pytest

from linear_rnn_b200 import _lib
from linear_rnn_b200._lib import GlaNormProblem, GlaProblem

lib = _lib.lib
vp = lambda x: None if x is None else ctypes.c_void_p(x)
INVALID, UNSUPPORTED, WORKSPACE = _lib.GLA_ERR_INVALID_ARG, _lib.GLA_ERR_UNSUPPORTED, _lib.GLA_ERR_WORKSPACE


def prob(**kw):
    d = dict(B=2, H=3, L=300, Dk=72, Dv=72, chunk=0, scale=0.0, io=_lib.GLA_BF16, gate=_lib.GLA_GATE_PER_KEY, plan=-3)
    d.update(kw)
    if "D" in kw:
        d["Dk"] = d["Dv"] = d.pop("D")
    return GlaProblem(*[d[f] for f, _ in GlaProblem._fields_])


BAD_SCAN = [(dict(B=-1), INVALID), (dict(L=-1), INVALID), (dict(D=0), INVALID), (dict(Dk=64), INVALID),
            (dict(io=2), INVALID), (dict(gate=_lib.GLA_GATE_NONE), INVALID), (dict(gate=_lib.GLA_GATE_PER_HEAD), INVALID),
            (dict(D=65537), UNSUPPORTED), (dict(B=1 << 20, H=1 << 20), UNSUPPORTED),
            (dict(B=(1 << 31) - 1, H=(1 << 31) - 1, D=65536), UNSUPPORTED)]


def scan_fwd(p, input=0, **kw):
    a = dict(x=16, g=16, h0=None, o=16, hT=None, saved=None)
    a.update(kw)
    return lib.gla_scan_fwd_save(ctypes.byref(p), input, *(vp(a[n]) for n in ("x", "g", "h0", "o", "hT", "saved")),
                                 None)


def scan_bwd(p, input=0, **kw):
    a = dict(x=16, g=16, h0=None, dO=16, dhT=None, saved=None, dx=16, dg=16, dh0=None, ws=16, nbytes=1 << 40)
    a.update(kw)
    names = ("x", "g", "h0", "dO", "dhT", "saved", "dx", "dg", "dh0", "ws")
    return lib.gla_scan_bwd_saved(ctypes.byref(p), input, *(vp(a[n]) for n in names), a["nbytes"], None)


def scan_decode(p, input=0, **kw):
    a = dict(x=16, g=16, state=16, o=16)
    a.update(kw)
    return lib.gla_scan_decode(ctypes.byref(p), input, *(vp(a[n]) for n in ("x", "g", "state", "o")), None)


def test_scan_sizes():
    p = prob()
    assert lib.gla_scan_saved_bytes(ctypes.byref(p)) == 4 * 6 * 5 * 72           # a state every 64 tokens
    assert lib.gla_scan_bwd_workspace_bytes(ctypes.byref(p)) >= 4 * 6 * 5 * 72   # those states
    empty = prob(L=0)
    assert lib.gla_scan_saved_bytes(ctypes.byref(empty)) == 0
    assert lib.gla_scan_bwd_workspace_bytes(ctypes.byref(empty)) > 0
    for kw, _ in BAD_SCAN:
        q = prob(**kw)
        assert lib.gla_scan_saved_bytes(ctypes.byref(q)) == 0
        assert lib.gla_scan_bwd_workspace_bytes(ctypes.byref(q)) == 0
    big = prob(B=8, H=16, L=1 << 20, D=4096)                                     # past 32 bits
    assert lib.gla_scan_saved_bytes(ctypes.byref(big)) == 4 * 128 * (1 << 14) * 4096


@pytest.mark.parametrize("kw,want", BAD_SCAN, ids=str)
def test_scan_refuses_problems(kw, want):
    p = prob(**kw)
    assert scan_fwd(p) == scan_bwd(p) == want
    if "L" not in kw:
        assert scan_decode(prob(**{**kw, "L": 1})) == want


def test_scan_refuses_arguments():
    p = prob()
    for call, names in ((scan_fwd, ("x", "g", "o")), (scan_bwd, ("x", "g", "dO", "dx", "dg", "ws"))):
        for n in names:
            assert call(p, **{n: None}) == INVALID, n
        for n in names + (("h0", "hT", "saved") if call is scan_fwd else ("h0", "dhT", "saved", "dh0")):
            assert call(p, **{n: 24}) == INVALID, n
        for mode in (-1, 3):
            assert call(p, input=mode) == INVALID
    assert scan_bwd(p, nbytes=16) == WORKSPACE
    one = prob(L=1)
    assert scan_decode(p) == INVALID                      # one token per (b, h)
    for n in ("x", "g", "state", "o"):
        assert scan_decode(one, **{n: None}) == INVALID
        assert scan_decode(one, **{n: 8}) == INVALID
    assert scan_decode(one, input=7) == INVALID
    assert lib.gla_scan_decode(None, 0, None, None, None, None, None) == INVALID
    assert lib.gla_scan_fwd(None, 0, None, None, None, None, None, None) == INVALID
    assert lib.gla_scan_bwd(None, 0, None, None, None, None, None, None, None, None, None, 0, None) == INVALID
    assert scan_decode(prob(B=0, L=1), x=None, g=None, state=None, o=None) == _lib.GLA_OK
    assert scan_fwd(prob(H=0), x=None, g=None, o=None) == _lib.GLA_OK


def nprob(**kw):
    d = dict(B=2, H=1, L=300, D=72, io=_lib.GLA_BF16, res=_lib.GLA_BF16, kind=0, act=0, w_per_head=0, eps=1e-6, alpha=1.0)
    d.update(kw)
    return GlaNormProblem(*[d[f] for f, _ in GlaNormProblem._fields_])


BAD_NORM = [(dict(B=-1), INVALID), (dict(L=-2), INVALID), (dict(D=0), INVALID), (dict(io=2), INVALID),
            (dict(kind=2), INVALID), (dict(kind=-1), INVALID), (dict(eps=0.0), INVALID), (dict(eps=float("nan")), INVALID),
            (dict(eps=float("inf")), INVALID), (dict(D=16385), UNSUPPORTED), (dict(B=1 << 20, L=1 << 20), UNSUPPORTED)]
BAD_ADD = BAD_NORM + [(dict(H=2), INVALID), (dict(res=5), INVALID), (dict(io=_lib.GLA_F32), UNSUPPORTED)]
BAD_HEAD = BAD_NORM + [(dict(H=-1), INVALID), (dict(act=2), INVALID), (dict(w_per_head=2), INVALID),
                       (dict(H=65536), UNSUPPORTED)]


def addnorm(p, **kw):
    a = dict(x=16, res=None, rscale=None, w=None, r=None, y=16)
    a.update(kw)
    return lib.gla_addnorm_fwd(ctypes.byref(p), *(vp(a[n]) for n in ("x", "res", "rscale", "w", "r", "y")), None)


def addnorm_bwd(p, **kw):
    a = dict(x=None, r=16, rscale=None, w=None, dy=16, dr=None, dres=None, dx=None, dw=None, drscale=None, ws=16,
             nbytes=1 << 40)
    a.update(kw)
    names = ("x", "r", "rscale", "w", "dy", "dr", "dres", "dx", "dw", "drscale", "ws")
    return lib.gla_addnorm_bwd(ctypes.byref(p), *(vp(a[n]) for n in names), a["nbytes"], None)


def headnorm(p, **kw):
    a = dict(o=16, z=None, w=None, y=16)
    a.update(kw)
    return lib.gla_headnorm_fwd(ctypes.byref(p), *(vp(a[n]) for n in ("o", "z", "w", "y")), None)


def headnorm_bwd(p, **kw):
    a = dict(o=16, z=16, w=None, dy=16, d_o=16, dz=16, dw=None, ws=16, nbytes=1 << 40)
    a.update(kw)
    return lib.gla_headnorm_bwd(ctypes.byref(p), *(vp(a[n]) for n in ("o", "z", "w", "dy", "d_o", "dz", "dw", "ws")),
                                a["nbytes"], None)


@pytest.mark.parametrize("kw,want", BAD_ADD, ids=str)
def test_addnorm_refuses_problems(kw, want):
    p = nprob(**kw)
    assert addnorm(p) == addnorm_bwd(p) == want
    assert lib.gla_addnorm_workspace_bytes(ctypes.byref(p)) == 0


@pytest.mark.parametrize("kw,want", BAD_HEAD, ids=str)
def test_headnorm_refuses_problems(kw, want):
    p = nprob(**kw)
    assert headnorm(p) == headnorm_bwd(p) == want
    assert lib.gla_headnorm_workspace_bytes(ctypes.byref(p)) == 0


def test_norms_refuse_arguments():
    p = nprob()
    assert addnorm(p, x=None) == addnorm(p, y=None) == INVALID
    for n in ("x", "res", "rscale", "w", "r", "y"):
        assert addnorm(p, **{n: 8}) == INVALID, n
    assert addnorm_bwd(p, r=None) == addnorm_bwd(p, dy=None) == addnorm_bwd(p, ws=None) == INVALID
    assert addnorm_bwd(p, drscale=16, x=16) == INVALID          # a gradient of a scale that is not there
    assert addnorm_bwd(p, drscale=16, rscale=16) == INVALID     # needs x
    for n in ("x", "r", "rscale", "w", "dy", "dr", "dres", "dx", "dw", "drscale", "ws"):
        assert addnorm_bwd(p, **{n: 8}) == INVALID, n
    assert addnorm_bwd(p, nbytes=64) == WORKSPACE
    assert headnorm(p, o=None) == headnorm(p, y=None) == INVALID
    for n in ("o", "z", "w", "y"):
        assert headnorm(p, **{n: 24}) == INVALID, n
    assert headnorm_bwd(p, z=None) == INVALID                   # dz without a gate
    for n in ("o", "dy", "d_o", "ws"):
        assert headnorm_bwd(p, **{n: None}) == INVALID, n
    for n in ("o", "z", "w", "dy", "d_o", "dz", "dw", "ws"):
        assert headnorm_bwd(p, **{n: 24}) == INVALID, n
    assert headnorm_bwd(p, nbytes=64) == WORKSPACE
    for f, n in ((lib.gla_addnorm_fwd, 7), (lib.gla_headnorm_fwd, 5)):
        assert f(*[None] * (n + 1)) == INVALID
    assert lib.gla_addnorm_bwd(*[None] * 12, 0, None) == INVALID
    assert lib.gla_headnorm_bwd(*[None] * 9, 0, None) == INVALID
    assert addnorm(nprob(L=0), x=None, y=None) == _lib.GLA_OK
    assert headnorm(nprob(B=0), o=None, y=None) == headnorm(nprob(H=0), o=None, y=None) == _lib.GLA_OK


def test_norm_workspace_holds_a_partial_row_per_block():
    """Never more partial rows than rows, and at least two each for dw and drscale where several blocks run; a
    single block writes the sums itself and needs none."""
    for D in (1, 72, 100, 4096, 16384):
        one = lib.gla_addnorm_workspace_bytes(ctypes.byref(nprob(B=1, L=1, D=D)))
        many = lib.gla_addnorm_workspace_bytes(ctypes.byref(nprob(B=8, L=8192, D=D)))
        assert one == 256 and 256 + 16 * D <= many < 1 << 28
        head = lib.gla_headnorm_workspace_bytes(ctypes.byref(nprob(B=8, L=8192, D=D, H=16)))
        assert 4 * D * 16 <= head < 1 << 28
        assert lib.gla_headnorm_workspace_bytes(ctypes.byref(nprob(B=1, L=1, D=D, H=16, w_per_head=1))) == 256
        assert lib.gla_headnorm_workspace_bytes(ctypes.byref(nprob(B=1, L=1, D=D, H=16))) >= 256 + 4 * 16 * D
