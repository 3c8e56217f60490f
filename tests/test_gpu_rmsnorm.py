"""The residual addition + root-mean-square norm and its gradients against plain float64.

Bounds.  h = x + r is one float32 addition (2^-24 relative to h) rounded to
the storage type.  The float32 sum of squares has at most 128 additions in a
row per thread and ten levels of a tree, all terms positive: 2^-17 relative
bounds it, half of that in rstd, and the roots and products add less than
2^-21: y is within 2^-17 |y| plus its one rounding.  The same 2^-17 bounds
each float32 term of the gradients; the mean of g w n is off by at most 2^-17
of the mean of its terms' magnitudes, and a column's sum over N rows by
(N + 64) 2^-24 of theirs.  8 bits: half a step of the value (2^-4 for e4m3,
2^-3 for e5m2) or of the smallest subnormal (2^-10, 2^-17 scales).
"""
import pytest
import torch

import vocabulary_cross_entropy_pass_gb300 as pkg

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
TYPES = [torch.float32, torch.bfloat16, torch.float16]
TINY = {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}
F = 2.0 ** -17
FP8 = {torch.float8_e4m3fn: (448.0, 2.0 ** -4, 2.0 ** -10), torch.float8_e5m2: (57344.0, 2.0 ** -3, 2.0 ** -17)}
WIDTHS = [1, 2, 7, 8, 31, 32, 100, 128, 130, 264, 1000, 1001, 2050, 4096, 5120, 8200, 9001, 16392]


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def rng(seed):
    return torch.Generator().manual_seed(seed)


def make(N, H, dtype, seed, residual=True, weight32=False):
    g = rng(seed)
    x = torch.randn(N, H, generator=g).to(dtype)
    r = (torch.randn(N, H, generator=g) * 3).to(dtype) if residual else None
    w = (1 + 0.2 * torch.randn(H, generator=g)).to(torch.float32 if weight32 else dtype)
    return x, r, w


def ref_fwd(x, r, w, eps):
    h = x.double().cpu() + (0 if r is None else r.double().cpu())
    return h, h / torch.sqrt((h * h).mean(-1, keepdim=True) + eps) * w.double().cpu()


def close(got, ref, rel, tiny=0.0):
    got = got.double().cpu()
    assert torch.equal(torch.isfinite(got), torch.isfinite(ref))
    worst = ((got - ref).abs() - rel * ref.abs() - tiny).max()
    assert float(worst) <= 0, float(worst)


def check_fwd(y, h, x, r, w, eps=1e-6):
    hr, yr = ref_fwd(x, r, w, eps)
    close(y, yr, half_step(y.dtype) + F, TINY[y.dtype])
    if r is not None:
        close(h, hr, half_step(h.dtype) + 2.0 ** -24, TINY[h.dtype])


def d(t):
    return None if t is None else t.to(DEV)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("H", WIDTHS)
def test_forward(H, dtype):
    for N, residual, w32 in ((1, True, False), (3, False, False), (5, True, True)):
        x, r, w = make(N, H, dtype, H + N, residual, w32)
        y, h, s = pkg.ce_rmsnorm_fwd(d(x), d(w), residual=d(r))
        assert s is None
        check_fwd(y, h, x, r, w)


@pytest.mark.parametrize("N", [1, 303, 305, 700])
def test_forward_many_rows(N):
    x, r, w = make(N, 4096, torch.bfloat16, N)
    y, h, _ = pkg.ce_rmsnorm_fwd(d(x), d(w), residual=d(r))
    check_fwd(y, h, x, r, w)


def check_q8(y, scales, x, r, w, quant, group, eps=1e-6):
    top, rel, sub = FP8[quant]
    _, yr = ref_fwd(x, r, w, eps)
    H = yr.shape[-1]
    group = group or H
    cols = torch.arange(H) // group
    G = int(cols[-1]) + 1
    m = torch.stack([yr[:, cols == k].abs().amax(1) for k in range(G)], 1)
    s = (m / top).clamp(min=2.0 ** -126)
    assert scales.shape == (yr.shape[0], G)
    assert bool(((scales.double().cpu() - s).abs() <= s * (F + 2.0 ** -23)).all())
    full = scales.double().cpu()[:, cols]
    got = y.float().double().cpu() * full
    # a value that saturates is the group's largest, off by the scale's own error
    bound = yr.abs() * (rel + 2 * F) + full * sub * (1 + F)
    assert bool(((got - yr).abs() <= bound).all())


@pytest.mark.parametrize("quant", [torch.float8_e4m3fn, torch.float8_e5m2])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("H", [1, 31, 32, 100, 130, 264, 1001, 2050, 4096, 8200, 9001, 16392])
def test_forward_8_bits(H, dtype, quant):
    for N, group in ((1, 0), (3, 128), (2, 32), (4, 64)):
        x, r, w = make(N, H, dtype, H + group, group != 64)
        x[0] *= 1e-3
        y, h, s = pkg.ce_rmsnorm_fwd(d(x), d(w), residual=d(r), quant=quant, group_size=group)
        assert y.dtype == quant
        check_q8(y, s, x, r, w, quant, group)
        if r is not None:
            close(h, ref_fwd(x, r, w, 1e-6)[0], half_step(dtype) + 2.0 ** -24, TINY[dtype])


@pytest.mark.parametrize("dtype", TYPES)
def test_rows_of_zeros(dtype):
    z = torch.zeros(3, 256, dtype=dtype, device=DEV)
    w = torch.ones(256, dtype=dtype, device=DEV)
    assert bool((pkg.ce_rmsnorm_fwd(z, w)[0] == 0).all())
    y, _, s = pkg.ce_rmsnorm_fwd(z, w, quant=torch.float8_e4m3fn, group_size=128)
    assert bool((y.float() == 0).all()) and bool((s == 2.0 ** -126).all())
    gx, gw = pkg.ce_rmsnorm_bwd(torch.ones_like(z), z, w)
    close(gx, torch.full((3, 256), 1e3, dtype=torch.float64), half_step(dtype) + F)
    assert bool((gw == 0).all())


@pytest.mark.parametrize("quant", [torch.float8_e4m3fn, torch.float8_e5m2])
@pytest.mark.parametrize("H", [256, 259])
def test_8_bits_of_the_smallest_values(H, quant):
    # scales at and just above their least value: y of about 2^-126 times 448 and below
    x, _, w = make(4, H, torch.float32, 9, residual=False)
    x = (x.double() * torch.tensor([2.0 ** -118, 2.0 ** -124, 2.0 ** -128, 2.0 ** -112])[:, None]).float()
    for group in (0, 32, 128):
        y, _, s = pkg.ce_rmsnorm_fwd(d(x), d(w), eps=1.0, quant=quant, group_size=group)
        top, rel, sub = FP8[quant]
        _, yr = ref_fwd(x, None, w, 1.0)
        full = s.double().cpu()[:, torch.arange(H) // (group or H)]
        assert bool((s >= 2.0 ** -126).all())
        # products below 2^-126 may be flushed or rounded by half the smallest float
        bound = yr.abs() * (rel + 2 * F) + full * sub * (1 + F) + 2.0 ** -126 * 2.0 ** -20
        assert bool(((y.float().double().cpu() * full - yr).abs() <= bound).all())


def test_infinities_stay_in_their_row():
    x, r, w = make(4, 512, torch.float32, 3)
    x[1, 7] = float("inf")
    x[2, 9] = float("nan")
    y, h, _ = pkg.ce_rmsnorm_fwd(d(x), d(w), residual=d(r))
    for k in (0, 3):
        check_fwd(y[k:k + 1], h[k:k + 1], x[k:k + 1], r[k:k + 1], w)
    assert bool(torch.isnan(y[2]).all()) and bool(torch.isnan(y[1, 7])) and bool(torch.isnan(h[2, 9]))


@pytest.mark.parametrize("dtype", TYPES)
def test_large_and_small_values(dtype):
    big = 1e15 if dtype != torch.float16 else 1e4
    for scale, eps in ((big, 1e-6), (1e-3, 1e-12), (1.0, 0.0)):
        x, _, w = make(3, 1024, dtype, 4, residual=False)
        x = (x.double() * scale).to(dtype)
        y, _, _ = pkg.ce_rmsnorm_fwd(d(x), d(w), eps=eps)
        hr, yr = ref_fwd(x, None, w, float(torch.tensor(eps)))
        close(y, yr, half_step(dtype) + F, TINY[dtype])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("H", [64, 65, 66, 2048, 9001])
def test_strides_and_in_place(H, dtype):
    g = rng(H)
    wide = torch.randn(2, 6, 2 * H + 8, generator=g).to(dtype).to(DEV)
    rbig = torch.randn(6, H + 3, generator=g).to(dtype).to(DEV)
    w = (1 + 0.1 * torch.randn(H, generator=g)).to(dtype).to(DEV)
    x, r = wide[0, :, 1:1 + H], rbig[:, 3:]
    for quant in (None, torch.float8_e4m3fn):
        y, h, s = pkg.ce_rmsnorm_fwd(x, w, residual=r, quant=quant)
        (check_fwd(y, h, x, r, w) if quant is None else check_q8(y, s, x.cpu(), r.cpu(), w.cpu(), quant, 0))
    y0, h0, _ = pkg.ce_rmsnorm_fwd(x, w, residual=r)
    # h over the residual, y over x; then h over x
    x1, r1 = wide.clone()[0, :, 1:1 + H], rbig.clone()[:, 3:]
    y, h, _ = pkg.ce_rmsnorm_fwd(x1, w, residual=r1, residual_out=r1, out=x1)
    assert torch.equal(y, y0) and torch.equal(h, h0) and torch.equal(r1, h0) and torch.equal(x1, y0)
    x2 = wide.clone()[0, :, 1:1 + H]
    y, h, _ = pkg.ce_rmsnorm_fwd(x2, w, residual=r, residual_out=x2)
    assert torch.equal(y, y0) and torch.equal(x2, h0)
    # one residual row for all
    one = r[:1].expand(6, H)
    y, h, _ = pkg.ce_rmsnorm_fwd(x, w, residual=one)
    check_fwd(y, h, x, one, w)
    y3, h3, _ = pkg.ce_rmsnorm_fwd(x.unflatten(0, (2, 3)), w, residual=r.unflatten(0, (2, 3)))
    assert torch.equal(y3.flatten(0, 1), y0) and torch.equal(h3.flatten(0, 1), h0)


def ref_bwd(go, h, w, dh, eps):
    go, h, w = (t.double().cpu() for t in (go, h, w))
    N, H = h.shape
    rstd = 1 / torch.sqrt((h * h).mean(-1, keepdim=True) + eps)
    n = h * rstd
    gw = go * w
    dx = rstd * (gw - n * (gw * n).mean(-1, keepdim=True))
    size = rstd * (gw.abs() + n.abs() * (gw * n).abs().mean(-1, keepdim=True))
    if dh is not None:
        dx = dx + dh.double().cpu()
        size = size + dh.double().cpu().abs()
    return dx, size, (go * n).sum(0), (go * n).abs().sum(0)


def check_bwd(gx, gw, go, h, w, dh, eps=1e-6):
    dx, size, dw, mag = ref_bwd(go, h, w, dh, eps)
    bound = half_step(gx.dtype) * dx.abs() + F * size + TINY[gx.dtype]
    assert bool(((gx.double().cpu() - dx).abs() <= bound).all())
    if gw is not None:
        assert gw.dtype == torch.float32
        assert bool(((gw.double().cpu() - dw).abs() <= ((h.shape[0] + 64) * 2.0 ** -24 + F) * mag).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("H", WIDTHS + [20000])
def test_backward(H, dtype):
    for N, residual, w32 in ((1, True, False), (3, False, True), (5, True, False)):
        h, dh, w = make(N, H, dtype, H + N, residual, w32)
        go = torch.randn(N, H, generator=rng(H + 77)).to(dtype)
        gx, gw = pkg.ce_rmsnorm_bwd(d(go), d(h), d(w), grad_h=d(dh))
        check_bwd(gx, gw, go, h, w, dh)
        only, none = pkg.ce_rmsnorm_bwd(d(go), d(h), d(w), grad_h=d(dh), grad_weight=None)
        assert none is None and torch.equal(only, gx)


@pytest.mark.parametrize("H", [72, 520, 1001, 1024, 2048, 4096, 9001])
@pytest.mark.parametrize("N", [455, 457, 1500])
def test_backward_many_rows(N, H):
    h, dh, w = make(N, H, torch.bfloat16, N)
    go = torch.randn(N, H, generator=rng(N)).to(torch.bfloat16)
    gx, gw = pkg.ce_rmsnorm_bwd(d(go), d(h), d(w), grad_h=d(dh))
    check_bwd(gx, gw, go, h, w, dh)
    ws = torch.full((pkg.ce_rmsnorm_bwd_workspace_bytes(N, H),), 171, dtype=torch.uint8, device=DEV)
    gx2, gw2 = pkg.ce_rmsnorm_bwd(d(go), d(h), d(w), grad_h=d(dh), workspace=ws)
    assert torch.equal(gx, gx2) and torch.equal(gw, gw2)
    assert pkg.ce_get_error(ws) == (0, 0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("H", [1, 40, 63, 128, 129, 130, 256, 257, 258, 396, 512, 513])
@pytest.mark.parametrize("N", [1, 9, 10007])
def test_backward_short_rows(N, H, dtype):
    h, dh, w = make(N, H, dtype, H + N)
    go = torch.randn(N, H, generator=rng(N + 5)).to(dtype)
    gx, gw = pkg.ce_rmsnorm_bwd(d(go), d(h), d(w), grad_h=d(dh))
    check_bwd(gx, gw, go, h, w, dh)
    gx2, gw2 = pkg.ce_rmsnorm_bwd(d(go), d(h), d(w))
    check_bwd(gx2, gw2, go, h, w, None)
    assert torch.equal(gw, gw2)
    # rows of a wider matrix, a row's end followed by numbers that must not count
    wide = torch.full((3, N, H + 3), float("nan"), dtype=dtype, device=DEV)
    for k, t in enumerate((go, h, dh)):
        wide[k, :, :H] = d(t)
    x3, w3 = pkg.ce_rmsnorm_bwd(wide[0, :, :H], wide[1, :, :H], d(w), grad_h=wide[2, :, :H])
    check_bwd(x3, w3, go, h, w, dh)
    # in place, and into a tensor of its own with the same strides (another stride may add in another order)
    apart = torch.full_like(wide[0], float("nan"))[:, :H]
    x4, w4 = pkg.ce_rmsnorm_bwd(wide[0, :, :H], wide[1, :, :H], d(w), grad_h=wide[2, :, :H], grad_x=apart)
    x5, w5 = pkg.ce_rmsnorm_bwd(wide[0, :, :H], wide[1, :, :H], d(w), grad_h=wide[2, :, :H], grad_x=wide[0, :, :H])
    check_bwd(x5, w5, go, h, w, dh)
    assert torch.equal(x4, x5) and torch.equal(w4, w5) and bool(wide[0, :, H:].isnan().all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("H", [64, 65, 66, 9001])
def test_backward_strides_and_in_place(H, dtype):
    g = rng(H)
    big = torch.randn(3, 7, H + 5, generator=g).to(dtype).to(DEV)
    w = torch.randn(H, generator=g).to(dtype).to(DEV)
    go, h, dh = big[0, :, :H], big[1, :, 3:3 + H], big[2, :, 5:]
    gx, gw = pkg.ce_rmsnorm_bwd(go, h, w, grad_h=dh)
    check_bwd(gx, gw, go, h, w, dh)
    for k in range(3):
        c = big.clone()
        views = (c[0, :, :H], c[1, :, 3:3 + H], c[2, :, 5:])
        x2, w2 = pkg.ce_rmsnorm_bwd(views[0], views[1], w, grad_h=views[2], grad_x=views[k])
        assert torch.equal(x2, gx) and torch.equal(w2, gw)
    one = go[:1].expand(7, H)  # one gradient row for all
    gx, gw = pkg.ce_rmsnorm_bwd(one, h, w)
    check_bwd(gx, gw, one, h, w, None)


@pytest.mark.parametrize("H", [1, 5, 1024, 4097, 8190])
@pytest.mark.parametrize("N", [1, 2, 300, 1300])
def test_backward_rows_off_the_grid(H, N):
    # each tensor at its own offset from 16 bytes, the first and last rows at the storage's ends
    g = rng(H + N)
    flat = [torch.randn(N * H + 8, generator=g).to(torch.float16).to(DEV) for _ in range(3)]
    go, h, dh = (f[k:k + N * H].view(N, H) for f, k in zip(flat, (1, 3, 6)))
    w = torch.randn(H, generator=g).to(torch.float16).to(DEV)
    gx, gw = pkg.ce_rmsnorm_bwd(go, h, w, grad_h=dh)
    check_bwd(gx, gw, go, h, w, dh)
    gx, gw = pkg.ce_rmsnorm_bwd(go, h, w)
    check_bwd(gx, gw, go, h, w, None)


def test_no_rows():
    w = torch.ones(40, device=DEV)
    e = torch.empty(0, 40, device=DEV)
    y, h, _ = pkg.ce_rmsnorm_fwd(e, w, residual=e)
    assert y.shape == h.shape == (0, 40)
    gx, gw = pkg.ce_rmsnorm_bwd(e, e, w)
    assert gx.shape == (0, 40) and bool((gw == 0).all())


def test_autograd_and_differences():
    g = rng(21)
    x = torch.randn(3, 4, 200, generator=g).to(DEV).requires_grad_()
    r = torch.randn(3, 4, 200, generator=g).to(DEV).requires_grad_()
    w = (1 + 0.1 * torch.randn(200, generator=g)).to(DEV).requires_grad_()
    cy, ch = (torch.randn(3, 4, 200, generator=g).to(DEV) for _ in range(2))

    def loss(x, r, w):
        y, h = pkg.rms_norm(x, w, residual=r)
        return (y.double() * cy.double()).sum() + (h.double() * ch.double()).sum()

    loss(x, r, w).backward()
    hr = (x + r).detach().flatten(0, 1)
    check_bwd(x.grad.flatten(0, 1), w.grad, cy.flatten(0, 1), hr, w.detach(), ch.flatten(0, 1))
    assert torch.equal(x.grad, r.grad)
    e = 2.0 ** -6
    for k, t in enumerate((x, r, w)):
        v = torch.randn(t.shape, generator=g).to(DEV)
        args = [a.detach() for a in (x, r, w)]
        up, dn = list(args), list(args)
        up[k], dn[k] = args[k] + e * v, args[k] - e * v
        diff = float(loss(*up) - loss(*dn)) / (2 * e)
        slope = float((t.grad.double() * v.double()).sum())
        # third derivatives of size about one over 2400 values, and their float32 rounding over 2e
        assert abs(diff - slope) <= 2400 * (e * e + 2.0 ** -22 / e), (k, diff, slope)
    # without a residual, and gradients that reach only one of the outputs
    x.grad = None
    pkg.rms_norm(x, w).backward(cy)
    check_bwd(x.grad.flatten(0, 1), None, cy.flatten(0, 1), x.detach().flatten(0, 1), w.detach(), None)
    x.grad = None
    pkg.rms_norm(x, w, residual=r)[1].backward(ch)
    assert torch.equal(x.grad, ch)
    x.grad = None
    pkg.rms_norm(x, w).sum().backward()  # a gradient expanded from one value
    check_bwd(x.grad.flatten(0, 1), None, torch.ones(12, 200), x.detach().flatten(0, 1), w.detach(), None)


def test_other_stream_and_graph():
    x, r, w = (t.to(DEV) for t in make(64, 1024, torch.bfloat16, 31))
    want = pkg.ce_rmsnorm_fwd(x, w, residual=r)
    wantb = pkg.ce_rmsnorm_bwd(x, want[1], w, grad_h=r)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, h = torch.empty_like(x), torch.empty_like(x)
    pkg.ce_rmsnorm_fwd(x, w, residual=r, out=out, residual_out=h, stream=side)
    side.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(h, want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, h, _ = pkg.ce_rmsnorm_fwd(x, w, residual=r)
        gx, gw = pkg.ce_rmsnorm_bwd(x, h, w, grad_h=r)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want[0]) and torch.equal(gx, wantb[0]) and torch.equal(gw, wantb[1])
    x.mul_(2)
    want = pkg.ce_rmsnorm_fwd(x, w, residual=r)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want[0])


def test_rows_past_32_bits():
    N, H = 600000, 4096  # 2.5e9 elements, 4.9 GB
    x = torch.empty(N, H, dtype=torch.bfloat16, device=DEV).fill_(1.0)
    g = torch.Generator(device=DEV).manual_seed(3)
    at = torch.tensor([0, 300000, 524287, 524288, 599999], device=DEV)
    x[at] = torch.randn(5, H, generator=g, device=DEV).to(torch.bfloat16)
    w = torch.ones(H, dtype=torch.bfloat16, device=DEV)
    y, _, _ = pkg.ce_rmsnorm_fwd(x, w, out=x[:0].new_empty(N, H))
    check_fwd(y[at], None, x[at], None, w)
    go = y[at]
    gx, _ = pkg.ce_rmsnorm_bwd(y, x, w, grad_x=y)
    check_bwd(gx[at], None, go, x[at], w, None)


@pytest.mark.parametrize("quant,least,bits", [(torch.float8_e4m3fn, -6, 3), (torch.float8_e5m2, -14, 2)])
@pytest.mark.parametrize("N,H,group", [(1000, 1024, 128), (200, 8192, 0), (1000, 1003, 64), (100, 20480, 32)])
def test_8_bits_on_rounding_borders(N, H, group, quant, least, bits):
    """q_j is t_j top / max|t| (t = h w in float32) with one rounding of 2^-24 before
    that to 8 bits: within half a step and 2^-23 of it, and half-way values, which
    a float holds, go to the even neighbour."""
    top = FP8[quant][0]
    x, r, w = make(N, H, torch.bfloat16, N + H)
    y, _, _ = pkg.ce_rmsnorm_fwd(d(x), d(w), residual=d(r), quant=quant, group_size=group)
    t = (x.float() + r.float()) * w.float()
    cols = torch.arange(H) // (group or H)
    m = torch.zeros(N, int(cols[-1]) + 1).scatter_reduce_(1, cols[None].expand(N, -1), t.abs(), "amax")
    v = t.double() * top / m.double()[:, cols]
    powers = 2.0 ** torch.arange(-40, 40, dtype=torch.float64)
    step = powers[(torch.frexp(v.abs())[1] - 1).clamp(min=least) - bits + 40]
    even = torch.round(v / step) * step
    half = (v / step).abs() % 1 == 0.5
    got = y.float().double().cpu()
    assert int(half.sum()) > 10
    assert torch.equal(got[half], even[half])
    assert bool(((got - v).abs() <= step / 2 + v.abs() * 2.0 ** -23).all())
