"""Refusals of the log-probability and distillation operators, and the plan of their rows: no GPU needed."""
import ctypes

import pytest
import torch

import vocabulary_cross_entropy_pass_gb300 as pkg
from vocabulary_cross_entropy_pass_gb300 import _lib

VP = ctypes.c_void_p
A = _lib.i64_array
ST = (3 * 4096, 4096, 1)


@pytest.fixture(scope="module")
def lib():
    from vocabulary_cross_entropy_pass_gb300 import build
    build.build()
    return _lib.load()


def rows(a):
    return [VP(a["x"]), a["dt"], a["d0"], a["d1"], a["V"], A(a["st"]) if a["st"] else None]


BASE = dict(x=0x1000, dt=1, d0=2, d1=3, V=4096, st=ST)


def logprobs(lib, **kw):
    a = dict(BASE, t=0x2000, ts=(6, 2, 1), n=2, ig=-100, lp=0x3000, ent=0x4000, k=5, top=0x5000, tlp=0x6000,
             stats=0x7000, ws=0x8000, wsb=1 << 30)
    a.update(kw)
    return lib.ce_logprobs_fwd(*rows(a), VP(a["t"]), A(a["ts"]) if a["ts"] else None, a["n"], a["ig"], VP(a["lp"]),
                               VP(a["ent"]), a["k"], VP(a["top"]), VP(a["tlp"]), VP(a["stats"]), VP(a["ws"]), a["wsb"],
                               None)


def row_refusals(call):
    assert call(dt=3) == 2
    assert call(x=0) == 1
    assert call(x=0x1001) == 1
    assert call(V=0) == 1
    assert call(V=1 << 31) == 1
    assert call(d0=-1) == 1
    assert call(d0=1 << 16, d1=1 << 16) == 1
    assert call(st=None) == 1
    assert call(st=(3 * 4096, 4096, 2)) == 3
    assert call(st=(3 * 4096, -1, 1)) == 3


def test_logprobs_refusals(lib):
    row_refusals(lambda **kw: logprobs(lib, **kw))
    assert logprobs(lib, t=0) == 1
    assert logprobs(lib, t=0x2004) == 1
    assert logprobs(lib, ts=None) == 1
    assert logprobs(lib, ts=(6, -2, 1)) == 3
    assert logprobs(lib, n=-1) == 1
    assert logprobs(lib, n=1025) == 1
    assert logprobs(lib, lp=0) == 1
    assert logprobs(lib, k=-1) == 1
    assert logprobs(lib, k=257) == 1
    assert logprobs(lib, k=5, V=4, st=(12, 4, 1)) == 1
    for p in ("top", "tlp", "ws"):
        assert logprobs(lib, **{p: 0}) == 1
    for p in ("lp", "ent", "top", "tlp", "stats", "ws"):
        assert logprobs(lib, **{p: 0x9002}) == 1
    assert logprobs(lib, n=0, k=0, ent=0, stats=0) == 1          # nothing asked for
    need = lib.ce_logprobs_workspace_bytes(6, 4096, 1, 5)
    assert need >= 256
    assert logprobs(lib, wsb=need - 1) == 4
    assert logprobs(lib, d1=0, x=0, t=0, lp=0, ws=0) == 0        # nothing to do
    assert lib.ce_logprobs_workspace_bytes(-1, 4096, 1, 5) == 0
    assert lib.ce_logprobs_workspace_bytes(6, 0, 1, 5) == 0
    assert lib.ce_logprobs_workspace_bytes(6, 4096, 5, 5) == 0
    assert lib.ce_logprobs_workspace_bytes(6, 4096, 1, 257) == 0


def logprobs_bwd(lib, **kw):
    a = dict(BASE, t=0x2000, ts=(6, 2, 1), n=2, ig=-100, stats=0x3000, gl=0x4000, ge=0x5000, g=0x9000, gst=ST)
    a.update(kw)
    return lib.ce_logprobs_bwd(*rows(a), VP(a["t"]), A(a["ts"]), a["n"], a["ig"], VP(a["stats"]), VP(a["gl"]),
                               VP(a["ge"]), VP(a["g"]), A(a["gst"]) if a["gst"] else None, None)


def grad_refusals(call):
    assert call(g=0) == 1
    assert call(g=0x9001) == 1
    assert call(gst=None) == 1
    assert call(gst=(3 * 4096, 4096, 2)) == 3
    assert call(gst=(3 * 4096, 4095, 1)) == 3                    # gradient rows that share memory
    assert call(gst=(0, 4096, 1)) == 3
    assert call(g=0x1000, gst=(3 * 4104, 4104, 1)) == 3          # in place means the same strides


def test_logprobs_bwd_refusals(lib):
    row_refusals(lambda **kw: logprobs_bwd(lib, **kw))
    grad_refusals(lambda **kw: logprobs_bwd(lib, **kw))
    assert logprobs_bwd(lib, stats=0) == 1
    assert logprobs_bwd(lib, stats=0x3008) == 1
    assert logprobs_bwd(lib, gl=0x4002) == 1
    assert logprobs_bwd(lib, ge=0x4002) == 1
    assert logprobs_bwd(lib, n=0) == 1                           # their gradients without tokens
    assert logprobs_bwd(lib, d0=0, x=0, g=0, t=0, stats=0) == 0


def distill(lib, step="fwd_bwd", **kw):
    a = dict(BASE, t=0x2000, ts=(60, 20, 1), z=0x3000, zdt=0, zs=(60, 20, 1), K=20, tau=2.0, norm=1, ig=-100, red=1,
             dl=0x4000, loss=0x5000, g=0x9000, gst=ST, n=0x6000, stats=0x7000, ws=0x8000, wsb=1 << 30)
    a.update(kw)
    first = rows(a) + [VP(a["t"]), A(a["ts"]) if a["ts"] else None, VP(a["z"]), a["zdt"], A(a["zs"]) if a["zs"] else None,
                       a["K"], a["tau"], a["norm"], a["ig"], a["red"]]
    gst = A(a["gst"]) if a["gst"] else None
    if step == "fwd_bwd":
        return lib.ce_distill_fwd_bwd(*first, VP(a["dl"]), VP(a["loss"]), VP(a["g"]), gst, VP(a["n"]), VP(a["ws"]),
                                      a["wsb"], None)
    if step == "fwd":
        return lib.ce_distill_fwd(*first, VP(a["loss"]), VP(a["stats"]), VP(a["n"]), VP(a["ws"]), a["wsb"], None)
    return lib.ce_distill_bwd(*first, VP(a["stats"]), VP(a["dl"]), VP(a["n"]), VP(a["g"]), gst, None)


@pytest.mark.parametrize("step", ["fwd_bwd", "fwd", "bwd"])
def test_distill_refusals(lib, step):
    def call(**kw):
        return distill(lib, step, **kw)

    row_refusals(call)
    assert call(t=0) == 1
    assert call(t=0x2004) == 1
    assert call(ts=None) == 1
    assert call(ts=(-60, 20, 1)) == 3
    assert call(z=0) == 1
    assert call(z=0x3002) == 1
    assert call(zdt=1, z=0x3001) == 1
    assert call(zdt=3) == 2
    assert call(zs=None) == 1
    assert call(zs=(60, 20, -1)) == 3
    assert call(K=0) == 1
    assert call(K=1025) == 1
    for tau in (0.0, -1.0, float("nan"), float("inf"), 1e-5, 1e5):
        assert call(tau=tau) == 1
    assert call(n=0x6004) == 1
    if step != "fwd":
        grad_refusals(call)
        assert call(dl=0x4002) == 1
    if step != "bwd":
        assert call(loss=0) == 1
        assert call(loss=0x5002) == 1
        assert call(ws=0) == 1
        assert call(ws=0x8008) == 1
        assert call(wsb=lib.ce_distill_workspace_bytes(6, 4096, 1) - 1) == 4
    if step != "fwd_bwd":
        assert call(stats=0x7008) == 1
    if step == "bwd":
        assert call(stats=0) == 1
        assert call(n=0) == 1                                     # the mean's gradient needs its count
        assert call(d0=0, x=0, g=0, t=0, z=0, stats=0) == 0


def test_distill_workspace_refusals(lib):
    assert lib.ce_distill_workspace_bytes(6, 4096, 1) > 256
    assert lib.ce_distill_workspace_bytes(-1, 4096, 1) == 0
    assert lib.ce_distill_workspace_bytes(6, 0, 1) == 0
    assert lib.ce_distill_workspace_bytes(6, 4096, 7) == 0


def test_python_refusals(lib):
    x = torch.zeros(4, 64)
    t = torch.zeros(4, dtype=torch.int64)
    z = torch.zeros(4, 3)
    with pytest.raises(ValueError):
        pkg.ce_logprobs_fwd(x, t)
    with pytest.raises(ValueError):
        pkg.ce_logprobs_bwd(x, torch.zeros(4, 4), t)
    for call in (pkg.ce_distill_fwd, pkg.ce_distill_fwd_bwd):
        with pytest.raises(ValueError):
            call(x, t[:, None].expand(4, 3), z)
    with pytest.raises(ValueError):
        pkg.ce_distill_bwd(x, t[:, None].expand(4, 3), z, torch.zeros(4, 4))
    with pytest.raises(TypeError):
        pkg.ce_logprobs_fwd("logits", t)
    with pytest.raises(TypeError):
        pkg.ce_distill_fwd_bwd(x, t, z, grad=False)
