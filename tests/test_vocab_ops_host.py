"""Refusals of the embedding, norm and logits operators: every call below is
rejected on the host, before any CUDA call (no GPU needed)."""
import ctypes

import pytest
import torch

import vocabulary_cross_entropy_pass_gb300 as pkg
from vocabulary_cross_entropy_pass_gb300 import _lib

VP = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    from vocabulary_cross_entropy_pass_gb300 import build
    build.build()
    return _lib.load()


def embed_fwd(lib, **kw):
    a = dict(tok=0x1000, d0=2, d1=3, ts=(3, 1), w=0x2000, dtype=1, V=100, H=64, ws=64, scale=1.0, ignore=-100,
             out=0x9000, os=64, wk=None, wkb=0)
    a.update(kw)
    return lib.ce_embed_fwd(VP(a["tok"]), a["d0"], a["d1"], _lib.i64_array(a["ts"]) if a["ts"] else None, VP(a["w"]),
                            a["dtype"], a["V"], a["H"], a["ws"], a["scale"], a["ignore"], VP(a["out"]), a["os"],
                            VP(a["wk"]), a["wkb"], None)


def test_embed_fwd_refusals(lib):
    assert embed_fwd(lib, dtype=3) == 2
    assert embed_fwd(lib, tok=0) == 1
    assert embed_fwd(lib, w=0) == 1
    assert embed_fwd(lib, out=0) == 1
    assert embed_fwd(lib, ts=None) == 1
    assert embed_fwd(lib, V=0) == 1
    assert embed_fwd(lib, H=0) == 1
    assert embed_fwd(lib, H=(1 << 20) + 1) == 1
    assert embed_fwd(lib, d0=-1) == 1
    assert embed_fwd(lib, d0=1 << 20, d1=1 << 20) == 1
    assert embed_fwd(lib, w=0x2001) == 1
    assert embed_fwd(lib, out=0x9001) == 1
    assert embed_fwd(lib, tok=0x1004) == 1
    assert embed_fwd(lib, ts=(-3, 1)) == 3
    assert embed_fwd(lib, ws=63) == 3
    assert embed_fwd(lib, os=63) == 3
    assert embed_fwd(lib, wk=0x4008, wkb=256) == 1
    assert embed_fwd(lib, wk=0x4000, wkb=255) == 4
    assert embed_fwd(lib, d1=0, tok=0, out=0) == 0     # nothing to do


def embed_bwd(lib, **kw):
    a = dict(g=0x1000, dtype=1, gs=64, tok=0x2000, d0=2, d1=3, ts=(3, 1), V=100, H=64, scale=1.0, ignore=-100,
             dw=0x9000, wdt=0, dws=64, acc=0, wk=0x4000, wkb=1 << 30)
    a.update(kw)
    return lib.ce_embed_bwd(VP(a["g"]), a["dtype"], a["gs"], VP(a["tok"]), a["d0"], a["d1"], _lib.i64_array(a["ts"]),
                            a["V"], a["H"], a["scale"], a["ignore"], VP(a["dw"]), a["wdt"], a["dws"], a["acc"],
                            VP(a["wk"]), a["wkb"], None)


def test_embed_bwd_refusals(lib):
    assert embed_bwd(lib, dtype=-1) == 2
    assert embed_bwd(lib, wdt=2) == 2                  # neither float32 nor grad_out's type
    assert embed_bwd(lib, wdt=1, acc=1) == 2           # adding needs float32
    assert embed_bwd(lib, g=0) == 1
    assert embed_bwd(lib, tok=0) == 1
    assert embed_bwd(lib, dw=0) == 1
    assert embed_bwd(lib, wk=0) == 1
    assert embed_bwd(lib, wk=0x4004) == 1
    assert embed_bwd(lib, g=0x1001) == 1
    assert embed_bwd(lib, dw=0x9002) == 1
    assert embed_bwd(lib, V=0) == 1
    assert embed_bwd(lib, H=0) == 1
    assert embed_bwd(lib, gs=-1) == 3
    assert embed_bwd(lib, dws=10) == 3
    assert embed_bwd(lib, ts=(3, -1)) == 3
    need = lib.ce_embed_bwd_workspace_bytes(6, 64, 100)
    assert need > 0
    assert embed_bwd(lib, wkb=need - 1) == 4
    assert lib.ce_embed_bwd_workspace_bytes(-1, 64, 100) == 0
    assert lib.ce_embed_bwd_workspace_bytes(1, 0, 100) == 0
    assert lib.ce_embed_bwd_workspace_bytes(1, 64, 1 << 31) == 0


def norm_fwd(lib, **kw):
    a = dict(x=0x1000, r=0x2000, w=0x3000, dt=1, wdt=1, N=4, H=64, xs=64, rs=64, eps=1e-6, y=0x5000, ys=64, q=0,
             group=0, sc=None, h=0x7000, hs=64)
    a.update(kw)
    return lib.ce_rmsnorm_fwd(VP(a["x"]), VP(a["r"]), VP(a["w"]), a["dt"], a["wdt"], a["N"], a["H"], a["xs"], a["rs"],
                              a["eps"], VP(a["y"]), a["ys"], a["q"], a["group"], VP(a["sc"]), VP(a["h"]), a["hs"],
                              None)


def test_rmsnorm_fwd_refusals(lib):
    assert norm_fwd(lib, dt=4) == 2
    assert norm_fwd(lib, wdt=2) == 2                   # bf16 rows take a bf16 or a float32 weight
    assert norm_fwd(lib, dt=0, wdt=1) == 2
    assert norm_fwd(lib, q=3) == 2
    for p in ("x", "w", "y", "h"):
        assert norm_fwd(lib, **{p: 0}) == 1            # a residual needs its sum's place
        assert norm_fwd(lib, **{p: 0x1001}) == 1
    assert norm_fwd(lib, N=-1) == 1
    assert norm_fwd(lib, H=0) == 1
    assert norm_fwd(lib, H=(1 << 20) + 1) == 1
    assert norm_fwd(lib, eps=-1.0) == 1
    assert norm_fwd(lib, eps=float("nan")) == 1
    assert norm_fwd(lib, y=0x7000) == 1                # y over h
    assert norm_fwd(lib, group=32) == 1                # groups without 8 bits
    assert norm_fwd(lib, q=1) == 1                     # 8 bits without scales
    assert norm_fwd(lib, q=1, sc=0x8000, group=48) == 1
    assert norm_fwd(lib, q=1, sc=0x8002) == 1
    assert norm_fwd(lib, q=1, sc=0x8000, y=0x1000) == 1  # 8 bits over the input
    assert norm_fwd(lib, xs=-64) == 3
    assert norm_fwd(lib, rs=-1) == 3
    assert norm_fwd(lib, ys=63) == 3
    assert norm_fwd(lib, hs=0) == 3
    assert norm_fwd(lib, y=0x1000, xs=80) == 3         # in place means the same strides
    assert norm_fwd(lib, h=0x2000, rs=0) == 3
    assert norm_fwd(lib, N=0, x=0, y=0) == 0


def norm_bwd(lib, **kw):
    a = dict(g=0x1000, h=0x2000, w=0x3000, dh=0x4000, dt=1, wdt=1, N=4, H=64, gs=64, hs=64, dhs=64, eps=1e-6,
             dx=0x5000, xs=64, dw=0x6000, wk=0x8000, wkb=1 << 20)
    a.update(kw)
    return lib.ce_rmsnorm_bwd(VP(a["g"]), VP(a["h"]), VP(a["w"]), VP(a["dh"]), a["dt"], a["wdt"], a["N"], a["H"],
                              a["gs"], a["hs"], a["dhs"], a["eps"], VP(a["dx"]), a["xs"], VP(a["dw"]), VP(a["wk"]),
                              a["wkb"], None)


def test_rmsnorm_bwd_refusals(lib):
    assert norm_bwd(lib, dt=4) == 2
    assert norm_bwd(lib, wdt=2) == 2
    for p in ("g", "h", "w", "dx"):
        assert norm_bwd(lib, **{p: 0}) == 1
        assert norm_bwd(lib, **{p: 0x1001}) == 1
    assert norm_bwd(lib, dh=0x4001) == 1
    assert norm_bwd(lib, dw=0x6002) == 1
    assert norm_bwd(lib, wk=0) == 1
    assert norm_bwd(lib, wk=0x8008) == 1
    assert norm_bwd(lib, eps=float("inf")) == 1
    assert norm_bwd(lib, gs=-1) == 3
    assert norm_bwd(lib, xs=32) == 3
    assert norm_bwd(lib, dx=0x2000, hs=80) == 3
    assert norm_bwd(lib, dx=0x1000, gs=0) == 3
    assert norm_bwd(lib, wkb=lib.ce_rmsnorm_bwd_workspace_bytes(4, 64) - 1) == 4
    assert lib.ce_rmsnorm_bwd_workspace_bytes(-1, 64) == 0
    assert lib.ce_rmsnorm_bwd_workspace_bytes(4, 0) == 0


def logits(lib, params=None, bwd=False, **kw):
    a = dict(x=0x1000, g=0x2000, dt=1, d0=2, d1=3, V=4096, st=(3 * 4096, 4096, 1), gst=(3 * 4096, 4096, 1),
             out=0x9000, ost=(3 * 4096, 4096, 1), wk=None, wkb=0)
    a.update(kw)
    p = _lib.ce_logits_params()
    for k, v in (params or {}).items():
        setattr(p, k, v)
    if bwd:
        return lib.ce_logits_process_bwd(VP(a["g"]), _lib.i64_array(a["gst"]), VP(a["x"]), a["dt"], a["d0"], a["d1"],
                                         a["V"], _lib.i64_array(a["st"]), ctypes.byref(p), VP(a["out"]),
                                         _lib.i64_array(a["ost"]), VP(a["wk"]), a["wkb"], None)
    return lib.ce_logits_process(VP(a["x"]), a["dt"], a["d0"], a["d1"], a["V"], _lib.i64_array(a["st"]),
                                 ctypes.byref(p), VP(a["out"]), _lib.i64_array(a["ost"]), VP(a["wk"]), a["wkb"],
                                 None)


@pytest.mark.parametrize("bwd", [False, True])
def test_logits_refusals(lib, bwd):
    assert logits(lib, bwd=bwd, dt=7) == 2
    assert logits(lib, bwd=bwd, x=0) == 1
    assert logits(lib, bwd=bwd, out=0) == 1
    assert logits(lib, bwd=bwd, x=0x1001) == 1
    assert logits(lib, bwd=bwd, out=0x9001) == 1
    assert logits(lib, bwd=bwd, V=0) == 1
    assert logits(lib, bwd=bwd, d0=-2) == 1
    assert logits(lib, bwd=bwd, st=(3 * 4096, 4096, 2)) == 3
    assert logits(lib, bwd=bwd, st=(-1, 4096, 1)) == 3
    assert logits(lib, bwd=bwd, ost=(3 * 4096, 4000, 1)) == 3   # output rows that share memory
    assert logits(lib, bwd=bwd, ost=(0, 4096, 1)) == 3
    assert logits(lib, dict(history_max=4), bwd=bwd) == 1
    assert logits(lib, dict(history_max=-1), bwd=bwd) == 1
    assert logits(lib, dict(history=0x100, history_max=4, history_stride=-4), bwd=bwd) == 3
    assert logits(lib, dict(bias_max=4, bias_tokens=0x100), bwd=bwd) == 1
    assert logits(lib, dict(mask=0x100, mask_stride=127), bwd=bwd) == 3  # 4096 tokens are 128 words
    p = _lib.ce_logits_params()
    p.reserved[0] = 1
    assert lib.ce_logits_process(VP(0x1000), 1, 2, 3, 4096, _lib.i64_array((3 * 4096, 4096, 1)), ctypes.byref(p),
                                 VP(0x9000), _lib.i64_array((3 * 4096, 4096, 1)), None, 0, None) == 1
    assert logits(lib, bwd=bwd, d1=0, x=0, out=0, g=0) == 0


def test_logits_workspace_refusals(lib):
    # few columns in all and no lists need none; else a table of touched columns a row
    assert lib.ce_logits_workspace_bytes(6, 4096, 1, 5000, 0) == 0
    assert lib.ce_logits_workspace_bytes(4096, 4096, 1, 0, 0) == 0
    assert lib.ce_logits_workspace_bytes(4096, 0, 1, 900, 0) == 0
    need = lib.ce_logits_workspace_bytes(4096, 4096, 1, 900, 0)
    assert need >= 4096 * 900 * 8
    one = (4096 * 4096, 4096, 1)
    for bwd in (False, True):
        p = dict(history=0x100, history_max=900, history_stride=900, repetition_penalty=0x200)
        kw = dict(bwd=bwd, d0=1, d1=4096, st=one, gst=one, ost=one)
        assert logits(lib, p, **kw) == 1
        assert logits(lib, p, wk=0x4008, wkb=need, **kw) == 1
        assert logits(lib, p, wk=0x4000, wkb=need - 1, **kw) == 4


def test_logits_in_place_refusals(lib):
    assert logits(lib, out=0x1000, ost=(3 * 4104, 4104, 1)) == 3
    assert logits(lib, bwd=True, out=0x2000, ost=(3 * 4104, 4104, 1)) == 3
    assert logits(lib, bwd=True, out=0x1000) == 1      # the gradient over the logits it still reads
    assert logits(lib, bwd=True, g=0) == 1


def test_python_refuses_cpu_tensors_and_types(lib):
    x = torch.zeros(4, 64)
    t = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError):
        pkg.ce_embed_fwd(t, x)
    with pytest.raises(ValueError):
        pkg.ce_embed_bwd(x, t, 10)
    with pytest.raises(ValueError):
        pkg.ce_rmsnorm_fwd(x, torch.zeros(64))
    with pytest.raises(ValueError):
        pkg.ce_rmsnorm_bwd(x, x, torch.zeros(64))
    with pytest.raises(ValueError):
        pkg.ce_logits_process(x)
    with pytest.raises(ValueError):
        pkg.ce_logits_process_bwd(x, x)


def test_row_strides_of_views(lib):
    from vocabulary_cross_entropy_pass_gb300.vocab_ops import _load
    stride = _load().row_stride
    x = torch.zeros(6, 5, 16)
    assert stride(x) == 16
    assert stride(x[:, :, :8]) == 16
    assert stride(x[:, 2]) == 80
    assert stride(x[:, :1]) == 80
    assert stride(x[0, 0]) == 16
    assert stride(x[:0]) == 16
    assert stride(torch.zeros(16).expand(3, 2, 16)) == 0
    for bad in (x[:, :4], x.transpose(0, 1), x[:, :, ::2]):
        with pytest.raises(ValueError):
            stride(bad)


def test_python_refuses_what_is_no_tensor(lib):
    x = torch.zeros(4, 64)
    with pytest.raises(TypeError):
        pkg.ce_embed_fwd([1, 2], x)
    with pytest.raises(TypeError):
        pkg.ce_rmsnorm_fwd(x, None)
    with pytest.raises(TypeError):
        pkg.ce_rmsnorm_fwd(x, x[0], quant=torch.int8)
    with pytest.raises(TypeError):
        pkg.ce_logits_process("logits")


@pytest.mark.parametrize("name", ["out", "workspace", "stream"])
def test_process_logits_takes_no_buffers(lib, name):
    # under autograd the logits are kept for the backward pass: an output over them would change its signs unseen
    x = torch.zeros(4, 64, requires_grad=True)
    for value in (x.detach(), None):
        with pytest.raises(TypeError, match=name):
            pkg.process_logits(x, **{name: value})


def test_logits_history_fits_its_count(lib):
    # a column's count has 30 bits beside its two flags
    p = dict(history=0x100, history_max=1 << 30, history_stride=1 << 30, frequency_penalty=0x200)
    for bwd in (False, True):
        assert logits(lib, p, bwd=bwd) == 1
        assert logits(lib, dict(p, history_max=(1 << 30) + 1), bwd=bwd) == 1
