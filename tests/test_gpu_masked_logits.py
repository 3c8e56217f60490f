"""The loss of logits masked by finite values of any size: a mask is what a row's maximum makes of it, nothing.

Bound: masked logits add nothing, so the loss is that of the row without them: |lse| and |x_y| rounded (a step
of 2^-23 each), log d off by 2^-24 * 128 (70 additions, an exponential of 2^-22, a base-2 product of |y| <= 40 rounded
to 2^-24 of itself); the gradient as p, 2^-24 (200 + 2 |lse|) relative, rounded to the type.
"""
import pytest
import torch

import vocabulary_cross_entropy_pass_gb300 as pkg

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
E = 2.0 ** -24
TINY = {torch.float32: 2.0 ** -125, torch.bfloat16: 2.0 ** -125, torch.float16: 2.0 ** -25}
VALUES = [-1e4, -1e9, -2e9, -4e9, -1e10, -1e15, -1e20, -1e30, -1e33]
PATHS = [("auto", pkg.CE_PATH_AUTO), ("row", pkg.CE_PATH_ROW), ("cluster", pkg.CE_PATH_CLUSTER),
         ("two_stage", pkg.CE_PATH_TWO_STAGE), ("stream", pkg.CE_PATH_STREAM), ("vecrow", pkg.CE_PATH_VECROW),
         ("warp", pkg.CE_PATH_WARP)]


def make(N, V, dtype, value, kind, seed=1):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = (torch.randn(N, V, generator=g, device=DEV) * 3).to(dtype)
    t = torch.randint(V // 2, V, (N,), generator=g, device=DEV)
    blocked = torch.zeros(N, V, dtype=torch.bool, device=DEV)
    if kind == "front":
        blocked[:, :V // 2] = True
    elif kind == "behind":
        blocked[:, -V // 3:] = True
        t = t % (V - V // 3 - 1)
    else:  # one token of 256 allowed
        blocked = torch.rand(N, V, generator=g, device=DEV) > 1 / 256
        blocked.scatter_(1, t[:, None], False)
    return x.masked_fill(blocked, value).unsqueeze(0), t.unsqueeze(0)


def check(x, t, loss, grad=None):
    y, i = x[0].double(), t[0]
    lse = torch.logsumexp(y, 1)
    xy = y.gather(1, i[:, None])[:, 0]
    bound = E * (128 + 4 * lse.abs() + 4 * xy.abs())
    assert bool(((loss.double().reshape(-1) - (lse - xy)).abs() <= bound).all())
    if grad is None:
        return
    p = torch.exp(y - lse[:, None])
    want = p.clone().scatter_add_(1, i[:, None], torch.full_like(xy, -1.0)[:, None])
    half = torch.finfo(x.dtype).eps / 2
    off = (grad[0].double() - want).abs() - half * want.abs() * (1 + half) - E * (200 + 2 * lse.abs())[:, None] * p - TINY[x.dtype]
    off.scatter_(1, i[:, None], off.gather(1, i[:, None]) - 2 * E)  # the target's own difference
    assert float(off.max()) <= 0, float(off.max())


@pytest.mark.parametrize("kind", ["front", "behind", "most"])
@pytest.mark.parametrize("name,path", PATHS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [4096, 12000, 32000, 50257])
def test_paths(V, dtype, name, path, kind):
    for value in VALUES:
        x, t = make(40, V, dtype, value, kind)
        try:
            loss = pkg.ce_fwd_only(x, t, label_smoothing=0.0, reduce_loss=False, force_path=path)
        except pkg.CEError as e:
            assert e.status == 8  # the path cannot run this shape
            return
        check(x, t, loss)
        g = x.clone()
        loss = pkg.ce_fwd_bwd(g, t, label_smoothing=0.0, reduce_loss=False, force_path=path)
        check(x, t, loss, g)


@pytest.mark.parametrize("kind", ["front", "most"])
def test_wide_and_many(kind):
    for N, V, dtype in ((1024, 32000, torch.bfloat16), (64, 128000, torch.bfloat16), (64, 256000, torch.float32)):
        for value in (-1e10, -1e30):
            x, t = make(N, V, dtype, value, kind)
            g = x.clone()
            check(x, t, pkg.ce_fwd_bwd(g, t, label_smoothing=0.0, reduce_loss=False), g)


def test_class_weights_chunks_and_backward():
    x, t = make(40, 32000, torch.bfloat16, -1e30, "front")
    ones = torch.ones(32000, device=DEV)
    check(x, t, pkg.ce_fwd_only(x, t, label_smoothing=0.0, reduce_loss=False, class_weights=ones))
    for chunks in (2, 8):
        g = x.clone()
        loss = pkg.ce_fwd_bwd(g, t, label_smoothing=0.0, reduce_loss=False, num_vocab_chunks=chunks)
        check(x, t, loss, g)
    # a shard of the vocabulary with no token allowed, and one with half
    y, off = x[:, :, :24000], [0, 12000, 24000]
    parts = torch.stack([pkg.ce_vp_partials(y[:, :, a:b].contiguous(), t.clamp(max=23999), a) for a, b in zip(off, off[1:])])
    t = t.clamp(max=23999)
    loss, lse = pkg.ce_vp_combine(parts, off, t)
    check(y, t, loss)


@pytest.mark.parametrize("name,path", PATHS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("V", [4096, 12000, 50257])
def test_masks_whose_sum_is_infinite(V, dtype, name, path):
    """Without smoothing the sum of the logits is not part of the loss, so -inf and the lowest values are masks too."""
    for value in (float(torch.finfo(dtype).min), -float("inf")):
        for kind in ("front", "most"):
            x, t = make(40, V, dtype, value, kind)
            g = x.clone()
            try:
                loss = pkg.ce_fwd_bwd(g, t, label_smoothing=0.0, reduce_loss=False, force_path=path)
            except pkg.CEError as e:
                assert e.status == 8
                return
            check(x, t, loss, g)
            check(x, t, pkg.ce_fwd_only(x, t, label_smoothing=0.0, reduce_loss=False, force_path=path))
            loss = pkg.ce_fwd_bwd(x.clone(), t, label_smoothing=0.0, reduce_loss=True, force_path=path)
            assert bool(torch.isfinite(loss).all())


def test_processed_logits_into_the_loss():
    """A mask of the default value, as process_logits leaves it, then the loss and its gradient."""
    g = torch.Generator(device=DEV).manual_seed(3)
    N, V = 24, 32000
    x = (torch.randn(N, V, generator=g, device=DEV) * 3).to(torch.bfloat16)
    bits = torch.randint(-2 ** 31, 2 ** 31, (N, (V + 31) // 32), generator=g, device=DEV).to(torch.int32)
    y = pkg.ce_logits_process(x, mask=bits)
    t = torch.argmax(y, 1)
    z = y.unsqueeze(0)
    grad = z.clone()
    check(z, t.unsqueeze(0), pkg.ce_fwd_bwd(grad, t.unsqueeze(0), label_smoothing=0.0, reduce_loss=False), grad)
    w = x.clone().requires_grad_()
    loss = pkg.parallel_cross_entropy(pkg.process_logits(w, mask=bits).unsqueeze(0), t.unsqueeze(0), 0.0, True)
    loss.backward()
    assert bool(torch.isfinite(w.grad).all()) and bool(torch.isfinite(loss).all())


@pytest.mark.parametrize("name,path", PATHS)
@pytest.mark.parametrize("smoothing", [0.0, 0.1])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_no_number_anywhere_in_the_row(name, path, smoothing, value):
    """A NaN or +inf makes its row's loss NaN wherever it lies, among the elements around the aligned body as well."""
    for V in (4099, 12000, 50257):
        for dtype in (torch.float32, torch.bfloat16):
            x = (torch.randn(1, 24, V, generator=torch.Generator(device=DEV).manual_seed(2), device=DEV) * 3).to(dtype)
            t = torch.full((1, 24), 9, dtype=torch.int64, device=DEV)
            for r, c in enumerate([0, 1, 2, 3, 4, 5, 6, 7, 8, V - 8, V - 7, V - 6, V - 5, V - 4, V - 3, V - 2, V - 1, V // 2]):
                x[0, r, c] = value
            try:
                loss = pkg.ce_fwd_only(x, t, label_smoothing=smoothing, reduce_loss=False, force_path=path)
            except pkg.CEError as e:
                assert e.status == 8
                continue
            assert bool(loss[:18].isnan().all()) and bool(torch.isfinite(loss[18:]).all())
            loss = pkg.ce_fwd_bwd(x.clone(), t, label_smoothing=smoothing, reduce_loss=False, force_path=path)
            assert bool(loss[:18].isnan().all()) and bool(torch.isfinite(loss[18:]).all())


@pytest.mark.parametrize("value", [-1e30, -float("inf")])
def test_shards_chunks_and_weights(value):
    V = 30011
    x, t = make(40, V, torch.bfloat16, value, "front")
    weights = torch.ones(V, device=DEV)
    for smooth_free in (None, weights):
        g = x.clone()
        loss = pkg.ce_fwd_bwd(g, t, label_smoothing=0.0, reduce_loss=False, class_weights=smooth_free)
        check(x, t, loss, g)
    for chunks in (3, 8):
        g = x.clone()
        loss = pkg.ce_fwd_bwd(g, t, label_smoothing=0.0, reduce_loss=False, num_vocab_chunks=chunks)
        check(x, t, loss, g)
    off = [0, 5003, 15001, 20003, V]
    parts = torch.stack([pkg.ce_vp_partials(x[:, :, a:b], t, a) for a, b in zip(off, off[1:])])
    loss, lse = pkg.ce_vp_combine(parts, off, t)
    check(x, t, loss)
    grads = [pkg.ce_vp_bwd(x[:, :, a:b], t, a, V, lse) for a, b in zip(off, off[1:])]
    check(x, t, loss, torch.cat(grads, 2))
    x[0, 3, [0, 5002, 5003, V - 1]] = float("nan")
    parts = torch.stack([pkg.ce_vp_partials(x[:, :, a:b], t, a) for a, b in zip(off, off[1:])])
    loss, lse = pkg.ce_vp_combine(parts, off, t)
    assert bool(loss.view(-1)[3].isnan()) and int(loss.isnan().sum()) == 1
