"""Log-probabilities, entropies, likeliest tokens and their gradient against float64.

Bounds.  A row's statistics are sums of positive float32 terms: each term is off by 2^-22 (the
exponential) and by 2^-23 of its exponent |y| (a difference and a product, each rounded; weighted
by the terms themselves that is at most log V <= 13), each of the at most 70 additions on a term's
way by 2^-24: log d is off by less than 128 * 2^-24, and by 2^-24 of itself.  A log-probability adds
two rounded differences: 2^-24 (128 + 2 |lp| + 2 log V).  The entropy's second sum has terms e y with the
same relative errors: 2^-24 * 160 (1 + log V).  A gradient is a sum of terms t with the relative error of
p, 2^-24 (160 + 2 |lp|), then one rounding to the storage type (half a step, or half the least subnormal).
"""
import math

import pytest
import torch

import vocabulary_cross_entropy_pass_gb300 as pkg

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
TYPES = [torch.float32, torch.bfloat16, torch.float16]
TINY = {torch.float32: 2.0 ** -125, torch.bfloat16: 2.0 ** -125, torch.float16: 2.0 ** -25}
E = 2.0 ** -24
NEG = -math.inf
LOWEST = {t: torch.finfo(t).min for t in TYPES}


def rng(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def reference(x, tokens, ignore=-100):
    """(lp (N, V), entropy, skipped) in float64; an all -inf row has lp = -inf and entropy 0."""
    x = x.reshape(-1, x.shape[-1]).double()
    m = x.amax(1, keepdim=True)
    none = (m == NEG)[:, 0] & ~x.isnan().any(1)
    y = x - m.masked_fill(none[:, None], 0.0)
    lp = y - torch.log(torch.exp(y).sum(1, keepdim=True))
    lp[none] = NEG
    p = torch.exp(lp)
    ent = -(p * torch.where(p > 0, lp, 0.0)).sum(1)
    ent[x.isnan().any(1) | (x == math.inf).any(1)] = math.nan
    skipped = torch.zeros(x.shape[0], dtype=torch.bool, device=DEV)
    if tokens is not None:
        skipped = (tokens.reshape(x.shape[0], -1) == ignore).all(1)
    return lp, ent, skipped


def order(x):
    """Columns by falling value, equal ones by rising column, NaN left out at the end."""
    v = x.reshape(-1, x.shape[-1]).double() + 0.0
    v = torch.where(v.isnan(), -math.inf, v)  # (after every -inf: those tests look at counts)
    return torch.sort(v, dim=1, descending=True, stable=True).indices


def check_forward(x, tokens=None, top_k=0, entropy=True, ignore=-100, **kw):
    V = x.shape[-1]
    lp, ent, top, top_lp, stats = pkg.ce_logprobs_fwd(x, tokens, top_k=top_k, entropy=entropy, stats=True,
                                                      ignore_idx=ignore, **kw)
    ref, ref_ent, skipped = reference(x, tokens, ignore)
    N = ref.shape[0]
    rows = torch.arange(N, device=DEV)[:, None]

    def near(got, want):
        assert got.dtype == torch.float32
        got, want = got.double(), want
        fine = torch.isfinite(want)
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(got[~fine].nan_to_num(7.0), want[~fine].nan_to_num(7.0))
        off = ((got - want).abs() - E * (128 + 2 * want.abs() + 2 * math.log(V)))[fine]
        assert off.numel() == 0 or float(off.max()) <= 0, float(off.max())

    if tokens is not None:
        assert lp.shape == tokens.shape
        t = tokens.reshape(N, -1)
        inside = (t >= 0) & (t < V)
        want = torch.where(inside, ref[rows, t.clamp(0, V - 1)], torch.where(t == ignore, 0.0, math.nan))
        near(lp.reshape(N, -1), want)
    if entropy:
        assert ent.shape == x.shape[:-1]
        want = torch.where(skipped, 0.0, ref_ent)
        got = ent.reshape(-1).double()
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        off = ((got - want).abs() - E * 160 * (1 + math.log(V))).nan_to_num(-1.0)
        assert float(off.max()) <= 0
    else:
        assert ent is None
    if top_k:
        assert top.shape == x.shape[:-1] + (top_k,) and top_lp.shape == top.shape
        want = order(x)[:, :top_k]
        got = top.reshape(N, -1)
        assert torch.equal(got, torch.where(skipped[:, None], ignore, want))
        near(top_lp.reshape(N, -1), torch.where(skipped[:, None], 0.0, ref[rows, want]))
    else:
        assert top is None and top_lp is None
    return lp, ent, top, top_lp, stats


def logits(N, V, dtype, seed, sigma=3.0):
    return (torch.randn(N, V, generator=rng(seed), device=DEV) * sigma).to(dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [1, 2, 7, 33, 300, 1001, 4095, 4096, 8193, 32000, 50257])
def test_rows(V, dtype):
    for k, (N, G, top) in enumerate([(1, 1, 1), (3, 5, 20), (2, 0, 21), (5, 1, 22), (4, 2, 64), (2, 1, 256)]):
        x = logits(N, V, dtype, V + k)
        t = torch.randint(0, V, (N, G), generator=rng(k), device=DEV) if G else None
        check_forward(x, t[:, 0].contiguous() if G == 1 else t, top_k=min(top, V), entropy=k % 2 == 0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N,V", [(1300, 8192), (1217, 4097), (2500, 1000), (1220, 20011)])
def test_rows_in_one_piece(N, V, dtype):
    x = logits(N, V, dtype, 7)
    t = torch.randint(0, V, (N,), generator=rng(1), device=DEV)
    t[::9] = -100
    check_forward(x, t, top_k=20)
    check_forward(x, None, top_k=130, entropy=False)


@pytest.mark.parametrize("dtype", TYPES)
def test_wide_rows(dtype):
    x = logits(2, 300001, dtype, 3)
    check_forward(x, torch.tensor([3, 300000], device=DEV), top_k=100)


# Rows on which a threshold is least use: equal logits, rising, falling, few distinct, a large one at each end, the
# likeliest all in one place.
def hard_rows(V, dtype):
    i = torch.arange(V, device=DEV, dtype=torch.float32)
    few = torch.randint(0, 3, (V,), generator=rng(5), device=DEV).float()
    ends = torch.zeros(V, device=DEV)
    ends[0] = ends[-1] = 2.0
    block = torch.randn(V, generator=rng(6), device=DEV)
    block[V // 2:V // 2 + 600] += 50.0
    low = torch.full((V,), LOWEST[dtype], device=DEV)
    few_left = low.clone()
    few_left[::max(1, V // 5)] = 1.0
    signs = torch.zeros(V, device=DEV)
    signs[::2] = -0.0
    return torch.stack([torch.full((V,), 1.5, device=DEV), i / 64, -i / 64, few, ends, block, low, few_left, signs,
                        torch.cat([torch.zeros(V // 2, device=DEV), i[V // 2:] / 8])]).to(dtype)


@pytest.mark.parametrize("copies", [1, 130])  # few rows: in segments; many: in one piece
@pytest.mark.parametrize("top", [1, 20, 64, 256])
@pytest.mark.parametrize("dtype", TYPES)
def test_ties_and_orders(dtype, top, copies):
    for V in (600, 9001, 40000):
        x = hard_rows(V, dtype).repeat(copies, 1)
        check_forward(x, None, top_k=top, entropy=top == 20)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N", [4, 1300])
def test_masks(dtype, N):
    V = 9000
    x = logits(N, V, dtype, 11)
    keep = torch.rand(N, V, generator=rng(3), device=DEV) < 1 / 64
    keep[1::4] = False            # nothing
    keep[2::4] = False
    keep[2::4, 17] = True         # one token
    keep[3::4] = False
    keep[3::4, 7000:8990] = True  # a range
    for blocked in (NEG, -3e4):
        y = x.masked_fill(~keep, blocked)
        t = torch.randint(0, V, (N,), generator=rng(4), device=DEV)
        t[2::4] = 17
        check_forward(y, t, top_k=20)
        check_forward(y, t, top_k=200)


@pytest.mark.parametrize("N", [3, 1300])
def test_no_numbers(N):
    V = 5000
    x = logits(N, V, torch.float32, 1)
    x[0, 4999] = math.nan
    x[1, 17] = math.inf
    x[2, :] = math.nan
    x[2, 40] = 3.0
    t = torch.full((N,), 5, device=DEV)
    lp, ent, top, top_lp, stats = pkg.ce_logprobs_fwd(x, t, top_k=4, entropy=True, stats=True)
    assert bool(lp[:3].isnan().all()) and bool(ent[:3].isnan().all()) and bool(top_lp[:3].isnan().all())
    assert torch.equal(top[0], torch.sort(x[0].nan_to_num(-99.0), descending=True, stable=True).indices[:4])
    assert int(top[1, 0]) == 17
    assert top[2].tolist() == [40, -1, -1, -1]
    g = pkg.ce_logprobs_bwd(x, stats, t, grad_logprobs=torch.ones(N, device=DEV))
    assert bool(g[0].isnan().all()) and bool(g[1].isnan().all()) and bool(g[2].isnan().all())
    if N > 3:
        assert bool(torch.isfinite(g[3:]).all())


def test_layouts():
    # (dim0, dim1, V) views of padded, transposed and shifted buffers, tokens with strides of their own
    base = logits(6 * 5, 3011, torch.bfloat16, 2).view(6, 5, 3011)
    for x in (base, base.transpose(0, 1), base[:, :, 3:], base[::2, 1:, 1:2900], base[:, :1], base[:1]):
        d0, d1, V = x.shape
        t = torch.randint(0, V, (d1, d0, 6), generator=rng(9), device=DEV).transpose(0, 1)
        check_forward(x, t[:, :, ::2], top_k=5)
        check_forward(x, t[:, :, 0], top_k=0)
    flat = logits(40, 3011, torch.float16, 3)[::2, 5:]
    check_forward(flat, torch.arange(40, device=DEV)[::2], top_k=3)
    row = logits(1, 3011, torch.float16, 3)
    check_forward(row.expand(4, 3011), None, top_k=3)  # rows may share memory when they are only read


def test_range_and_ignored():
    x = logits(4, 1000, torch.float32, 5)
    ws = torch.empty(pkg.ce_logprobs_workspace_bytes(4, 1000, torch.float32, 3), dtype=torch.uint8, device=DEV)
    t = torch.tensor([[1, 2], [-100, 999], [-100, -100], [1000, -1]], device=DEV)
    check_forward(x, t, top_k=3, workspace=ws)
    assert pkg.ce_get_error(ws) == (6, 1)
    check_forward(x[:3], t[:3], top_k=3, workspace=ws)
    assert pkg.ce_get_error(ws) == (0, 0)
    check_forward(x, t[:, 0].contiguous().clamp(0), top_k=3, workspace=ws, ignore=2)
    assert pkg.ce_get_error(ws) == (6, 1)
    big = logits(1300, 64, torch.float32, 5)
    tb = torch.zeros(1300, dtype=torch.int64, device=DEV)
    check_forward(big, tb, workspace=ws)
    assert pkg.ce_get_error(ws) == (0, 0)
    tb[1299] = 64
    check_forward(big, tb, workspace=ws)
    assert pkg.ce_get_error(ws) == (6, 1)


def test_no_rows():
    x = torch.empty(0, 100, device=DEV)
    lp, ent, top, top_lp, stats = pkg.ce_logprobs_fwd(x, torch.empty(0, dtype=torch.int64, device=DEV), top_k=3,
                                                      entropy=True, stats=True)
    assert lp.shape == (0,) and ent.shape == (0,) and top.shape == (0, 3) and stats.shape == (0, 4)
    assert pkg.ce_logprobs_bwd(x, stats).shape == (0, 100)


# ------------------------------------------------------------------------------------- gradient
def check_backward(x, tokens, gl, ge, out=None, ignore=-100):
    V = x.shape[-1]
    given = x.clone() if out is x else x
    stats = pkg.ce_logprobs_fwd(x, tokens, stats=True, ignore_idx=ignore)[4]
    got = pkg.ce_logprobs_bwd(x, stats, tokens, grad_logprobs=gl, grad_entropy=ge, ignore_idx=ignore, grad=out)
    assert got.dtype == x.dtype and got.shape == x.shape
    lp, ent, skipped = reference(given, tokens, ignore)
    N = lp.shape[0]
    nothing = skipped | (given.reshape(N, V).double().amax(1) == NEG)
    p = torch.exp(lp)
    safe = torch.where(p > 0, lp, 0.0)
    want, mag = torch.zeros_like(p), torch.zeros_like(p)
    if gl is not None:
        t, c = tokens.reshape(N, -1), gl.reshape(N, -1).double()
        ok = (t >= 0) & (t < V) & (t != ignore)
        c = torch.where(ok, c, 0.0)
        hit = torch.zeros_like(p).scatter_add_(1, t.clamp(0, V - 1), c)
        habs = torch.zeros_like(p).scatter_add_(1, t.clamp(0, V - 1), c.abs())
        want += hit - p * c.sum(1, keepdim=True)
        mag += habs + p * c.abs().sum(1, keepdim=True)
    if ge is not None:
        h = ge.reshape(N, 1).double()
        want -= h * p * (safe + ent[:, None])
        mag += h.abs() * p * (safe.abs() + ent[:, None] + 1)
    want[nothing] = 0.0
    mag[nothing] = 0.0
    got64 = got.reshape(N, V).double()
    assert bool((got64[nothing] == 0).all())
    half = torch.finfo(x.dtype).eps / 2
    off = (got64 - want).abs() - half * want.abs() - E * (160 + 2 * safe.abs()) * mag * (1 + half) - TINY[x.dtype] * (
        1 + mag)
    assert float(off.max()) <= 0, float(off.max())
    return got


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [1, 7, 33, 1001, 4096, 8193, 50257])
def test_gradient(V, dtype):
    for k, (N, G, ent) in enumerate([(1, 1, False), (3, 5, True), (700, 1, True), (4, 0, True), (2, 300, False)]):
        if V > 20000 and N > 100:
            N = 40
        x = logits(N, V, dtype, V + k)
        t = torch.randint(0, V, (N, G), generator=rng(k), device=DEV) if G else None
        gl = torch.randn(N, G, generator=rng(k), device=DEV) if G else None
        if G == 1:
            t, gl = t[:, 0].contiguous(), gl[:, 0].contiguous()
        ge = torch.randn(N, generator=rng(k + 1), device=DEV) if ent else None
        check_backward(x, t, gl, ge)
        check_backward(x, t, gl, ge, out=x)


@pytest.mark.parametrize("dtype", TYPES)
def test_gradient_masks_and_ignored(dtype):
    N, V = 8, 9001
    x = logits(N, V, dtype, 21)
    x[0, ::2] = NEG
    x[1] = NEG
    x[2] = NEG
    x[2, 100] = 1.0
    x[3] = LOWEST[dtype]
    t = torch.randint(0, V, (N, 3), generator=rng(1), device=DEV)
    t[2] = 100
    t[4] = -100
    t[5, 0] = -100
    t[6, 1] = V
    t[7] = 8
    gl = torch.randn(N, 3, generator=rng(2), device=DEV)
    ge = torch.randn(N, generator=rng(3), device=DEV)
    check_backward(x, t, gl, ge)
    check_backward(x, t, gl, None)
    check_backward(x, t, None, ge)


@pytest.mark.parametrize("shift", [0, 1, 3, 8])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gradient_layouts(dtype, shift):
    N, V = 6, 5003
    buf = logits(N, V + 16, dtype, 4)
    x = buf[:, shift:shift + V]
    t = torch.randint(0, V, (N,), generator=rng(5), device=DEV)
    gl = torch.randn(N, generator=rng(6), device=DEV)
    for to in (0, 2, 5):
        room = torch.full((N, V + 16), 7.0, dtype=dtype, device=DEV)
        check_backward(x, t, gl, gl, out=room[:, to:to + V])
        assert bool((room[:, :to] == 7).all()) and bool((room[:, to + V:] == 7).all())
    x3 = x.reshape(3, 2, V)
    check_backward(x3.transpose(0, 1), t.view(3, 2).t(), gl.view(2, 3), None)


def test_autograd_and_differences():
    x = logits(5, 41, torch.float32, 8, sigma=1.5).requires_grad_()
    t = torch.tensor([[1, 1], [4, 40], [-100, 7], [-100, -100], [0, 3]], device=DEV)
    w = torch.randn(5, 2, generator=rng(1), device=DEV)
    h = torch.randn(5, generator=rng(2), device=DEV)
    lp, ent, top, top_lp = pkg.token_logprobs(x, t, top_k=3, entropy=True)
    assert not top.requires_grad and not top_lp.requires_grad
    ((lp * w).sum() + (ent * h).sum()).backward()

    def f(z):
        ref, e, skipped = reference(z, t)
        got = torch.where(t == -100, 0.0, ref[torch.arange(5, device=DEV)[:, None], t.clamp(min=0)])
        return (got * w).sum() + (torch.where(skipped, 0.0, e) * h).sum()

    z = x.detach().double()
    for r in range(5):
        for j in range(0, 41, 5):
            d = torch.zeros_like(z)
            d[r, j] = 1e-5
            diff = float((f(z + d) - f(z - d)) / 2e-5)
            # the central difference's own error: 1e-10 / 6 of a third derivative of order one, and 1e-11 of rounding
            assert abs(float(x.grad[r, j]) - diff) <= 1e-6 + 1e-6 * abs(diff)
    x.grad = None
    pkg.token_logprobs(x, t, entropy=True)[1].sum().backward()
    assert bool(torch.isfinite(x.grad).all())
    assert pkg.token_logprobs(x, None, top_k=2)[0] is None


def test_autograd_of_lists_without_tokens():
    x = logits(3, 40, torch.float32, 9).requires_grad_()
    lp, ent, *_ = pkg.token_logprobs(x, torch.empty(3, 0, dtype=torch.int64, device=DEV), entropy=True)
    assert lp.shape == (3, 0)
    got, = torch.autograd.grad(lp.sum() + ent.sum(), x)
    want, = torch.autograd.grad(pkg.token_logprobs(x, entropy=True)[1].sum(), x)
    assert torch.equal(got, want)
    assert bool((want != 0).any())


def test_graph_and_streams():
    x = logits(6, 9000, torch.bfloat16, 1)
    t = torch.randint(0, 9000, (6,), generator=rng(1), device=DEV)
    gl = torch.ones(6, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        pkg.ce_logprobs_fwd(x, t, top_k=8, entropy=True, stats=True)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = pkg.ce_logprobs_fwd(x, t, top_k=8, entropy=True, stats=True)
        g = pkg.ce_logprobs_bwd(x, out[4], t, grad_logprobs=gl)
    for seed in (2, 3):
        x.copy_(logits(6, 9000, torch.bfloat16, seed))
        graph.replay()
        want = pkg.ce_logprobs_fwd(x, t, top_k=8, entropy=True, stats=True)
        for a, b in zip(out, want):
            assert torch.equal(a, b)
        assert torch.equal(g, pkg.ce_logprobs_bwd(x, want[4], t, grad_logprobs=gl))
    # a stream handed in: behind what it holds
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        y = x * 2
    got = pkg.ce_logprobs_fwd(y, t, top_k=8, stream=side)
    side.synchronize()
    want = pkg.ce_logprobs_fwd(y, t, top_k=8)
    assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])


def test_same_on_every_run():
    x = logits(300, 20011, torch.bfloat16, 1)
    t = torch.randint(0, 20011, (300, 4), generator=rng(1), device=DEV)
    a = pkg.ce_logprobs_fwd(x, t, top_k=50, entropy=True, stats=True)
    for _ in range(5):
        for u, v in zip(a, pkg.ce_logprobs_fwd(x, t, top_k=50, entropy=True, stats=True)):
            assert torch.equal(u, v)
