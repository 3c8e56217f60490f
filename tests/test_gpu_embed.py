"""The embedding rows and their gradient against plain float64.

Forward: float32(scale) * W is one float32 product (half a step, 2^-24
relative) rounded once more to the storage type (eps/2): the bound is
(eps/2 + 2^-23) |ref| plus half the type's smallest subnormal.

Gradient: the float32 sum of n rows is off by at most (n + 1) 2^-24 of the
sum of their magnitudes, times the scale (one product more), then rounded once
to the gradient's type; adding to what is there rounds once more.
"""
import pytest
import torch

import vocabulary_cross_entropy_pass_gb300 as pkg

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
TYPES = [torch.float32, torch.bfloat16, torch.float16]
TINY = {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def rng(seed):
    return torch.Generator().manual_seed(seed)


def fwd_ref(tokens, weight, scale, ignore):
    V, H = weight.shape
    flat = tokens.reshape(-1)
    out = torch.full((flat.numel(), H), float("nan"), dtype=torch.float64)
    ok = (flat >= 0) & (flat < V)
    out[ok] = weight.double()[flat[ok]] * scale
    out[flat == ignore] = 0.0
    return out.view(*tokens.shape, H)


def check_fwd(got, tokens, weight, scale, ignore=-100):
    ref = fwd_ref(tokens, weight, scale, ignore)
    got = got.double().cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(ref))
    ref, got = ref.nan_to_num(), got.nan_to_num()
    bound = (half_step(weight.dtype) + 2.0 ** -23) * ref.abs() + TINY[weight.dtype]
    assert bool(((got - ref).abs() <= bound).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N,V,H", [(1, 1, 1), (1, 7, 5), (3, 100, 8), (33, 257, 65), (16, 500, 4096), (1000, 50, 130),
                                   (257, 1000, 1001), (2000, 300, 2056)])
def test_forward(N, V, H, dtype):
    g = rng(N * 7 + H)
    w = torch.randn(V, H, generator=g).to(dtype)
    t = torch.randint(0, V, (N,), generator=g)
    for scale in (1.0, 0.125, 1.7):
        scale = float(torch.tensor(scale))
        check_fwd(pkg.ce_embed_fwd(t.to(DEV), w.to(DEV), scale=scale), t, w, scale)


def test_forward_no_rows():
    w = torch.zeros(5, 8, device=DEV)
    assert pkg.ce_embed_fwd(torch.zeros(0, dtype=torch.int64, device=DEV), w).shape == (0, 8)
    assert pkg.ce_embed_fwd(torch.zeros(2, 0, dtype=torch.int64, device=DEV), w).shape == (2, 0, 8)


def test_forward_ignored_and_out_of_range():
    g = rng(5)
    w = torch.randn(50, 72, generator=g).to(torch.bfloat16)
    t = torch.randint(0, 50, (4, 9), generator=g)
    t[0, 0], t[1, 2], t[3, 8] = -100, -1, 50
    ws = torch.full((256,), 255, dtype=torch.uint8, device=DEV)
    check_fwd(pkg.ce_embed_fwd(t.to(DEV), w.to(DEV), workspace=ws), t, w, 1.0)
    assert pkg.ce_get_error(ws) == (6, 1)
    t[1, 2] = t[3, 8] = -100
    check_fwd(pkg.ce_embed_fwd(t.to(DEV), w.to(DEV), workspace=ws), t, w, 1.0)
    assert pkg.ce_get_error(ws) == (0, 0)
    # the ignored value comes first, also inside the vocabulary
    got = pkg.ce_embed_fwd(t.clamp(min=0).to(DEV), w.to(DEV), ignore_idx=7)
    check_fwd(got, t.clamp(min=0), w, 1.0, ignore=7)


@pytest.mark.parametrize("dtype", TYPES)
def test_forward_strides(dtype):
    g = rng(6)
    wide = torch.randn(40, 201, generator=g).to(dtype).to(DEV)
    t = torch.randint(0, 40, (7, 5), generator=g).to(DEV)
    for w in (wide[:, 1:130], wide[:, :128], wide[::2, 3:3 + 64]):
        tt = t % w.shape[0]
        for tok in (tt, tt.t(), tt[:, ::2], tt[1:, 1:]):
            check_fwd(pkg.ce_embed_fwd(tok, w), tok.cpu(), w.cpu(), 1.0)
        big = torch.full((7, 5, 200), 9.0, dtype=dtype, device=DEV)
        pkg.ce_embed_fwd(tt, w, out=big[:, :, 1:1 + w.shape[1]])
        check_fwd(big[:, :, 1:1 + w.shape[1]], tt.cpu(), w.cpu(), 1.0)
        assert bool((big[:, :, 0] == 9).all()) and bool((big[:, :, 1 + w.shape[1]:] == 9).all())


def bwd_ref(grad_out, tokens, V, scale, ignore, base):
    """(gradient, sum of magnitudes, tokens per row) in float64."""
    H = grad_out.shape[-1]
    flat = tokens.reshape(-1)
    rows = grad_out.reshape(-1, H).double()
    keep = (flat >= 0) & (flat < V) & (flat != ignore)
    ref = torch.zeros(V, H, dtype=torch.float64).index_add_(0, flat[keep], rows[keep]) * scale
    mag = torch.zeros(V, H, dtype=torch.float64).index_add_(0, flat[keep], rows[keep].abs()) * abs(scale)
    n = torch.zeros(V, dtype=torch.float64).index_add_(0, flat[keep], torch.ones(int(keep.sum()), dtype=torch.float64))
    if base is not None:
        ref = ref + base.double()
        mag = mag + base.double().abs()
    return ref, mag, n


def check_bwd(got, grad_out, tokens, V, scale, ignore=-100, base=None):
    ref, mag, n = bwd_ref(grad_out, tokens, V, scale, ignore, base)
    bound = (n[:, None] + 3) * 2.0 ** -24 * mag + half_step(got.dtype) * ref.abs() + TINY[got.dtype]
    assert bool(((got.double().cpu() - ref).abs() <= bound).all())
    absent = n == 0
    if base is None:
        assert bool((got.cpu()[absent] == 0).all())
    else:
        assert torch.equal(got.cpu()[absent], base.cpu()[absent])


def run_bwd(N, V, H, dtype, tokens, scale=1.0, seed=0, twice=True):
    g = rng(seed + N)
    go = torch.randn(N, H, generator=g).to(dtype)
    god, td = go.to(DEV), tokens.to(DEV)
    got = pkg.ce_embed_bwd(god, td, V, scale=scale)
    check_bwd(got, go, tokens, V, scale)
    if twice:  # the same bits on every run, also from a dirty workspace and output
        ws = torch.full((pkg.ce_embed_bwd_workspace_bytes(N, H, V),), 171, dtype=torch.uint8, device=DEV)
        out = torch.full_like(got, float("nan"))
        assert torch.equal(pkg.ce_embed_bwd(god, td, V, scale=scale, grad_weight=out, workspace=ws), got)
    if dtype != torch.float32:
        low = pkg.ce_embed_bwd(god, td, V, scale=scale, grad_dtype=dtype)
        assert low.dtype == dtype
        check_bwd(low, go, tokens, V, scale)
    base = torch.randn(V, H, generator=g)
    acc = base.to(DEV)
    pkg.ce_embed_bwd(god, td, V, scale=scale, grad_weight=acc, accumulate=True)
    check_bwd(acc, go, tokens, V, scale, base=base)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N,V,H", [(1, 1, 1), (1, 5, 3), (7, 100, 8), (8, 3, 17), (9, 3, 16), (31, 1000, 40),
                                   (33, 40, 130), (1000, 50, 24), (1023, 8192, 33), (1025, 2000, 64), (2049, 5000, 8)])
def test_backward(N, V, H, dtype):
    t = torch.randint(0, V, (N,), generator=rng(N + H))
    run_bwd(N, V, H, dtype, t, scale=float(torch.tensor(1.3)))


@pytest.mark.parametrize("N", [15, 16, 17, 255, 1024, 1025, 5000, 9000])
def test_backward_one_token_takes_all(N):
    run_bwd(N, 77, 40, torch.bfloat16, torch.full((N,), 76))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N,H", [(2, 256), (9, 257), (128, 4096), (129, 4096), (1000, 300), (1024, 512), (1023, 513)])
def test_backward_on_both_sides_of_few_tokens(N, H, dtype):
    # a kernel of its own below, the sort above; values seen once, often, and never
    V = 3 * N + 5
    g = rng(N + H)
    t = torch.randint(0, V, (N,), generator=g)
    t[torch.rand(N, generator=g) < 0.3] = V - 1
    run_bwd(N, V, H, dtype, t, scale=2.0)


def test_backward_few_tokens_strides_and_strangers():
    g = rng(17)
    go = torch.randn(6, 10, 40, generator=g).to(torch.bfloat16)
    t = torch.randint(0, 9000, (6, 10), generator=g)
    t[1, 1], t[2, 3], t[5, 9] = -100, 9000, -7
    ws = torch.empty(pkg.ce_embed_bwd_workspace_bytes(60, 33, 9000), dtype=torch.uint8, device=DEV)
    wide, td = go.to(DEV), t.t().contiguous().to(DEV).t()
    got = pkg.ce_embed_bwd(wide[:, :, 2:35], td, 9000, workspace=ws)
    check_bwd(got, go[:, :, 2:35], t, 9000, 1.0)
    assert pkg.ce_get_error(ws) == (6, 1)


@pytest.mark.parametrize("N,V", [(3000, 3000), (9000, 9001)])
def test_backward_all_different(N, V):
    run_bwd(N, V, 16, torch.float32, torch.randperm(V, generator=rng(3))[:N])


def test_backward_long_and_skewed():
    # several CTAs sort; runs of every length cross the chunks
    g = rng(9)
    N, V = 40001, 50257
    t = (torch.exp(torch.rand(N, generator=g, dtype=torch.float64) * 10.8).long() * 7919) % V
    run_bwd(N, V, 72, torch.bfloat16, t, scale=8.0)


def test_backward_more_than_fits_on_chip():
    N, V = 70001, 3001
    run_bwd(N, V, 8, torch.float32, torch.randint(0, V, (N,), generator=rng(10)))


@pytest.mark.parametrize("V,H", [(1, 3), (7, 1001), (4096, 8), (513, 16), (100, 33)])
def test_backward_zeros_what_is_absent(V, H):
    # contiguous, padded and odd rows, from a dirty buffer
    g = rng(V)
    t = torch.randint(0, V, (3,), generator=g)
    for dtype in (torch.float32, torch.bfloat16):
        go = torch.randn(3, H, generator=g).to(dtype)
        for pad in (0, 1, 5):
            big = torch.full((V, H + pad), 7.0, dtype=dtype, device=DEV)
            pkg.ce_embed_bwd(go.to(DEV), t.to(DEV), V, grad_weight=big[:, :H])
            check_bwd(big[:, :H], go, t, V, 1.0)
            assert bool((big[:, H:] == 7).all())


@pytest.mark.parametrize("V", [1023, 1024, 1025, (1 << 20) - 1, (1 << 20) + 3])
def test_backward_digit_counts(V):
    # one, two and three digits of up to ten bits; the highest token
    t = torch.randint(0, V, (700,), generator=rng(11))
    t[5] = V - 1
    run_bwd(700, V, 2, torch.float32, t)


def test_backward_ignored_and_out_of_range():
    g = rng(12)
    go = torch.randn(600, 24, generator=g)
    t = torch.randint(0, 30, (600,), generator=g)
    t[::7] = -100
    t[3], t[10], t[599] = 30, -1, 1 << 40
    ws = torch.empty(pkg.ce_embed_bwd_workspace_bytes(600, 24, 30), dtype=torch.uint8, device=DEV)
    got = pkg.ce_embed_bwd(go.to(DEV), t.to(DEV), 30, workspace=ws)
    check_bwd(got, go, t, 30, 1.0)
    assert pkg.ce_get_error(ws) == (6, 1)
    t[3] = t[10] = t[599] = -100
    check_bwd(pkg.ce_embed_bwd(go.to(DEV), t.to(DEV), 30, workspace=ws), go, t, 30, 1.0)
    assert pkg.ce_get_error(ws) == (0, 0)
    t[:] = -100
    assert bool((pkg.ce_embed_bwd(go.to(DEV), t.to(DEV), 30) == 0).all())
    t[:] = 4
    check_bwd(pkg.ce_embed_bwd(go.to(DEV), t.to(DEV), 30, ignore_idx=4), go, t, 30, 1.0, ignore=4)


def test_backward_no_rows():
    go = torch.zeros(0, 24, device=DEV)
    t = torch.zeros(0, dtype=torch.int64, device=DEV)
    out = torch.full((9, 24), 3.0, device=DEV)
    pkg.ce_embed_bwd(go, t, 9, grad_weight=out, accumulate=True)
    assert bool((out == 3).all())
    pkg.ce_embed_bwd(go, t, 9, grad_weight=out)
    assert bool((out == 0).all())


@pytest.mark.parametrize("dtype", TYPES)
def test_backward_strides(dtype):
    g = rng(13)
    wide = torch.randn(6, 11, 90, generator=g).to(dtype).to(DEV)
    t = torch.randint(0, 20, (11, 6), generator=g).to(DEV).t()
    for go in (wide[:, :, :64], wide[:, :, 1:66], wide[:, :, 2:90]):
        H = go.shape[-1]
        check_bwd(pkg.ce_embed_bwd(go, t, 20), go.cpu(), t.cpu(), 20, 1.0)
        big = torch.full((20, 100), 5.0, device=DEV)
        pkg.ce_embed_bwd(go, t, 20, grad_weight=big[:, 3:3 + H])
        check_bwd(big[:, 3:3 + H], go.cpu(), t.cpu(), 20, 1.0)
        assert bool((big[:, :3] == 5).all()) and bool((big[:, 3 + H:] == 5).all())
    one = torch.randn(1, 64, generator=g).to(dtype).to(DEV).expand(66, 64)  # one row for all tokens
    flat = t.reshape(-1)
    check_bwd(pkg.ce_embed_bwd(one, flat, 20), one.cpu(), flat.cpu(), 20, 1.0)


def test_tables_past_32_bits():
    # 2.5e9 elements: offsets in bytes and in elements pass 32 bits
    V, H = 305000, 8192
    w = torch.empty(V, H, dtype=torch.bfloat16, device=DEV)
    t = torch.tensor([0, V - 1, V - 2, 262144, 300001, V - 1], device=DEV)
    for k, r in enumerate(t.tolist()):
        w[r] = 0.5 + k
    got = pkg.ce_embed_fwd(t, w, scale=2.0)
    assert torch.equal(got, w[t] * 2)
    go = torch.randn(6, H, device=DEV).to(torch.bfloat16)
    dw = pkg.ce_embed_bwd(go, t, V, grad_weight=w, grad_dtype=torch.bfloat16)
    check_bwd(dw[t.unique()], go.cpu(), torch.searchsorted(t.unique(), t).cpu(), 5, 1.0)
    assert int((dw[::997] != 0).any(1).sum()) == int((t.unique() % 997 == 0).sum())


def test_autograd_and_differences():
    g = rng(14)
    w = (torch.randn(30, 20, generator=g)).to(DEV).requires_grad_()
    t = torch.randint(0, 30, (4, 9), generator=g).to(DEV)
    c = torch.randn(4, 9, 20, generator=g).to(DEV)
    (pkg.embedding(t, w, scale=3.0) * c).sum().backward()
    check_bwd(w.grad, c.cpu(), t.cpu(), 30, 3.0)
    d = torch.randn(30, 20, generator=g).to(DEV)
    e = 2.0 ** -5
    up = (pkg.ce_embed_fwd(t, (w + e * d).detach(), scale=3.0).double() * c.double()).sum()
    dn = (pkg.ce_embed_fwd(t, (w - e * d).detach(), scale=3.0).double() * c.double()).sum()
    slope = float((w.grad.double() * d.double()).sum())
    # linear in w: the difference is off by the rounding of 720 values of about 5 over 2e alone
    assert abs(float(up - dn) / (2 * e) - slope) <= 720 * 20 * 2.0 ** -23 / (2 * e)


def test_tied_with_linear_cross_entropy():
    # the lm_head's gradient and the embedding's meet in one float32 buffer
    g = rng(15)
    V, H, N = 500, 64, 96
    w = (torch.randn(V, H, generator=g) * 0.1).to(torch.bfloat16)
    t = torch.randint(0, V, (N,), generator=g)
    go = torch.randn(N, H, generator=g).to(torch.bfloat16)
    h = torch.randn(N, H, generator=g).to(torch.bfloat16)
    _, _, gw = pkg.ce_linear_fwd_bwd(h.to(DEV), w.to(DEV), t.to(DEV), reduce_loss=True)
    base = gw.cpu()
    pkg.ce_embed_bwd(go.to(DEV), t.to(DEV), V, scale=8.0, grad_weight=gw, accumulate=True)
    check_bwd(gw, go, t, V, 8.0, base=base)


def test_other_stream_and_graph():
    g = rng(16)
    go = torch.randn(3000, 64, generator=g).to(DEV)
    t = torch.randint(0, 700, (3000,), generator=g).to(DEV)
    want = pkg.ce_embed_bwd(go, t, 700)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ws = torch.empty(pkg.ce_embed_bwd_workspace_bytes(3000, 64, 700), dtype=torch.uint8, device=DEV)
    out = torch.empty(700, 64, device=DEV)
    pkg.ce_embed_bwd(go, t, 700, grad_weight=out, workspace=ws, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkg.ce_embed_bwd(go, t, 700, grad_weight=out, workspace=ws)
        rows = pkg.ce_embed_fwd(t, out)
    t.copy_(torch.randint(0, 700, (3000,), generator=g).to(DEV))
    want = pkg.ce_embed_bwd(go, t, 700)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(rows, want[t])
