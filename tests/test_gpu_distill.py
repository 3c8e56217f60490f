"""Distillation from a teacher's top logits against float64.

Bounds.  log p and log q are off by 2^-24 (128 + 2 |lp| + 2 log V) as in the log-probabilities' tests (with
the temperature's reciprocal and its products 2^-23 of |x - m| / temperature more), q by that relative to
itself; a loss sums K such terms in float32: temperature^2 2^-24 sum q (300 + 4 |lq| + 4 |lp| + K/8)
(1 + |lq - lp|).  A gradient is (Q p - q) times two factors: relative errors of its terms as of p and q, four
rounded products, then one rounding to the storage type.
"""
import math
import os
import subprocess
import sys

import pytest
import torch

import vocabulary_cross_entropy_pass_gb300 as pkg

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
TYPES = [torch.float32, torch.bfloat16, torch.float16]
TINY = {torch.float32: 2.0 ** -125, torch.bfloat16: 2.0 ** -125, torch.float16: 2.0 ** -25}
E = 2.0 ** -24
NEG = -math.inf


def rng(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def make(N, V, K, dtype, seed, teacher_dtype=torch.float32, ignored=0.2):
    g = rng(seed)
    x = (torch.randn(N, V, generator=g, device=DEV) * 3).to(dtype)
    t = torch.stack([torch.randperm(V, generator=g, device=DEV)[:K] for _ in range(N)]) if N <= 64 else torch.randint(
        0, V, (N, K), generator=g, device=DEV)
    z = (torch.randn(N, K, generator=g, device=DEV) * 4).to(teacher_dtype)
    drop = torch.rand(N, generator=g, device=DEV) < ignored
    t[drop] = -100
    if K > 2:
        t[1::3, K // 2:] = -100
    return x, t, z


def reference(x, t, z, tau, normalize, ignore=-100):
    """(loss, gradient before its factors, magnitude of its terms, loss bound, rows that count) in float64."""
    V = x.shape[-1]
    x = x.reshape(-1, V).double()
    N = x.shape[0]
    t, z = t.reshape(N, -1), z.reshape(N, -1).double()
    K = t.shape[1]
    row = t[:, 0] != ignore
    keep = (t != ignore) & row[:, None]
    bad = (keep & ((t < 0) | (t >= V))).any(1)
    zz = torch.where(keep, z / tau, NEG)
    if normalize:
        top = zz.amax(1, keepdim=True).clamp(min=-1e300)
        total = torch.exp(zz - top).sum(1, keepdim=True)
        lq = zz - top - torch.log(total)
    else:
        lq = zz
    q = torch.where(zz == NEG, 0.0, torch.exp(lq))
    m = x.amax(1, keepdim=True)
    none = (m == NEG)[:, 0]
    y = (x - m.masked_fill(none[:, None], 0.0)) / tau
    lp = y - torch.log(torch.exp(y).sum(1, keepdim=True))
    lp[none] = NEG
    lpt = lp[torch.arange(N, device=DEV)[:, None], t.clamp(0, V - 1)]
    term = torch.where(q > 0, q * (lq - lpt), 0.0)
    loss = tau * tau * term.sum(1)
    bound = tau * tau * E * torch.where(q > 0, q * (300 + 4 * lq.abs() + 4 * lpt.abs() + K / 8) * (1 + (lq - lpt).abs()),
                                        0.0).sum(1)
    p = torch.exp(lp)
    Q = q.sum(1, keepdim=True)
    hit = torch.zeros_like(p).scatter_add_(1, t.clamp(0, V - 1), q)
    grad = Q * p - hit
    mag = (Q * p + hit) * (200 + 2 * torch.where(p > 0, lp.abs(), 0.0) + 4 * hit.clamp(min=1e-300).log().abs().clamp(max=40))
    dead = ~row | bad | none
    grad[dead] = 0.0
    mag[dead] = 0.0
    loss[~row] = 0.0
    loss[bad] = math.nan
    return loss, grad, mag, bound, row


def check(x, t, z, tau=1.0, normalize=True, reduce=False, dloss=None, in_place=False, **kw):
    shape = x.shape
    V = shape[-1]
    loss, grad, mag, bound, row = reference(x, t, z, tau, normalize)
    N = loss.shape[0]
    n = int(row.sum())
    count = torch.full((1,), -7, dtype=torch.int64, device=DEV)
    g = torch.ones(N, dtype=torch.float64, device=DEV) if dloss is None else dloss.double().reshape(-1).expand(N)
    if reduce:
        g = g / n if n else torch.zeros_like(g)
    args = dict(temperature=tau, normalize=normalize, reduce_loss=reduce)
    fl, stats = pkg.ce_distill_fwd(x, t, z, stats=True, n_non_ignore_out=count, **args)
    assert int(count) == n
    got_b = pkg.ce_distill_bwd(x, t, z, stats, dloss=dloss, n_non_ignore=count if reduce else None, **args)
    own = x.clone() if in_place else x
    count.fill_(-7)
    got_l, got_g = pkg.ce_distill_fwd_bwd(own, t, z, dloss=dloss, grad=own if in_place else None,
                                          n_non_ignore_out=count, **args, **kw)
    assert int(count) == n
    if in_place:
        assert got_g.data_ptr() == own.data_ptr()
    want = loss
    if reduce:
        want = (loss.sum() / n).reshape(1) if n else torch.full((1,), math.nan, dtype=torch.float64, device=DEV)
        bound = (bound.sum() / max(n, 1)).reshape(1) + E * want.abs()
    for got in (fl, got_l):
        assert got.dtype == torch.float32 and got.shape == want.shape
        got = got.double()
        fine = torch.isfinite(want)
        assert torch.equal(got[~fine].nan_to_num(5.0), want[~fine].nan_to_num(5.0))
        assert bool(((got - want).abs() <= bound + 2.0 ** -140)[fine].all())
    scale = (g * tau)[:, None]
    half = torch.finfo(x.dtype).eps / 2
    for got in (got_b, got_g):
        assert got.dtype == x.dtype and got.shape == shape
        got = got.reshape(N, V).double()
        w = grad * scale
        off = (got - w).abs() - half * w.abs() - E * mag * scale.abs() * (1 + half) - TINY[x.dtype] * (1 + scale.abs())
        assert float(off.max()) <= 0, float(off.max())
        assert bool((got[mag.amax(1) == 0] == 0).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [1, 2, 9, 33, 1001, 4096, 8193, 50257])
def test_rows(V, dtype):
    for k, (N, K, tau, norm, reduce) in enumerate([(1, 1, 1.0, True, False), (5, 20, 2.0, True, True),
                                                   (3, 100, 0.5, True, False), (7, 300, 1.0, False, True),
                                                   (2, 1024, 4.0, True, False)]):
        K = min(K, V)
        x, t, z = make(N, V, K, dtype, V + k)
        if not norm:
            z = torch.log_softmax(z, 1) - 0.2
        dl = torch.rand(1 if reduce else N, generator=rng(k), device=DEV) + 0.3 if k % 2 else None
        check(x, t, z, tau, norm, reduce, dl, in_place=k % 2 == 1)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N,V,K", [(1300, 4096, 64), (1219, 20011, 7), (700, 33000, 256), (400, 70001, 32)])
def test_many_rows(N, V, K, dtype):
    x, t, z = make(N, V, K, dtype, 3)
    check(x, t, z, 2.0, True, True)
    check(x, t, z, 1.0, True, False, torch.rand(N, generator=rng(1), device=DEV), in_place=True)


def test_wide_rows():
    for dtype in (torch.float32, torch.bfloat16):
        x, t, z = make(3, 300001, 64, dtype, 4, ignored=0.0)
        check(x, t, z, 1.5, True, True)


@pytest.mark.parametrize("teacher", TYPES)
def test_teacher_types_and_strides(teacher):
    x, t, z = make(12, 3001, 40, torch.bfloat16, 6, teacher_dtype=teacher)
    check(x, t, z)
    check(x, t.t().contiguous().t(), z.t().contiguous().t())
    check(x, t[:, ::2], z[:, 1::2], 2.0)
    check(x, t, z[:1].expand(12, 40), 2.0)
    x3, t3, z3 = x.view(3, 4, 3001), t.view(3, 4, 40), z.view(3, 4, 40)
    check(x3, t3, z3)
    check(x3.transpose(0, 1), t3.transpose(0, 1), z3.transpose(0, 1), 1.0, True, True)
    check(x[:, 5:], t.clamp(max=2995), z)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("copies", [1, 200])
def test_edges_of_rows(dtype, copies):
    V, K = 2001, 8
    x, t, z = make(8, V, K, dtype, 9, ignored=0.0)
    t = torch.randint(0, V, (8, K), generator=rng(2), device=DEV)
    x[0] = NEG                      # the student allows nothing
    x[1, ::2] = NEG
    t[1] = torch.arange(K, device=DEV) * 2 + 1
    z[2] = NEG                      # the teacher gives nothing any probability
    t[3] = 5                        # one token eight times
    t[4, 3] = V                     # out of range
    t[5, 0] = -100                  # ignored, whatever follows
    z[6, 1:] = NEG
    x[7] = torch.finfo(dtype).min   # equal, as low as the type goes
    x, t, z = x.repeat(copies, 1), t.repeat(copies, 1), z.repeat(copies, 1)
    check(x, t, z, 1.0)
    check(x, t, z, 2.0, in_place=True)
    x[1, 1] = NEG                   # a token of the teacher's that the student forbids
    loss, _ = pkg.ce_distill_fwd(x, t, z)
    assert float(loss[1]) == math.inf and float(loss[0]) == math.inf and float(loss[2]) == 0.0
    ws = torch.empty(pkg.ce_distill_workspace_bytes(8 * copies, V, dtype), dtype=torch.uint8, device=DEV)
    pkg.ce_distill_fwd_bwd(x, t, z, workspace=ws)
    assert pkg.ce_get_error(ws) == (6, 1)
    pkg.ce_distill_fwd_bwd(x[:4], t[:4], z[:4], workspace=ws)
    assert pkg.ce_get_error(ws) == (0, 0)


def test_no_numbers():
    x, t, z = make(4, 500, 5, torch.float32, 1, ignored=0.0)
    t = torch.randint(0, 500, (4, 5), generator=rng(2), device=DEV)
    x[0, 300] = math.nan
    z[1, 2] = math.nan
    z[2, 2] = math.inf
    loss, g = pkg.ce_distill_fwd_bwd(x, t, z)
    assert bool(loss[:3].isnan().all()) and bool(torch.isfinite(loss[3]))
    assert bool(g[:3].isnan().all()) and bool(torch.isfinite(g[3]).all())


def test_all_ignored_and_no_rows():
    x, t, z = make(5, 700, 4, torch.bfloat16, 1)
    t[:] = -100
    check(x, t, z, 1.0, True, True)
    check(x, t, z, 1.0, True, False)
    x, t, z = x[:0], t[:0], z[:0]
    loss, g = pkg.ce_distill_fwd_bwd(x, t, z)
    assert loss.shape == (0,) and g.shape == (0, 700)
    loss, g = pkg.ce_distill_fwd_bwd(x, t, z, reduce_loss=True)
    assert bool(loss.isnan().all())


@pytest.mark.parametrize("shift", [0, 1, 8])
def test_gradient_elsewhere(shift):
    N, V = 20, 40003
    buf = torch.randn(N, V + 16, generator=rng(1), device=DEV).to(torch.bfloat16)
    x = buf[:, shift:shift + V]
    _, t, z = make(N, V, 16, torch.bfloat16, 3)
    want = pkg.ce_distill_fwd_bwd(x.contiguous(), t, z)
    for to in (0, 1, 6):
        room = torch.full((N, V + 16), 7.0, dtype=torch.bfloat16, device=DEV)
        loss, g = pkg.ce_distill_fwd_bwd(x, t, z, grad=room[:, to:to + V])
        # the sums' grouping goes with the rows' offset from 16 bytes: a bf16 step at most
        assert bool(((g.float() - want[1].float()).abs() <= 2.0 ** -7 * want[1].float().abs() + 2.0 ** -120).all())
        assert bool((room[:, :to] == 7).all()) and bool((room[:, to + V:] == 7).all())


def test_autograd_and_differences():
    x, t, z = make(5, 31, 6, torch.float32, 4, ignored=0.0)
    t[3] = -100
    w = torch.rand(5, generator=rng(1), device=DEV) + 0.5
    for reduce in (False, True):
        y = x.clone().requires_grad_()
        loss = pkg.distillation_loss(y, t, z, temperature=2.0, reduce_loss=reduce)
        assert loss.shape == (() if reduce else (5,))
        (loss if reduce else (loss * w).sum()).backward()

        def f(v):
            ref, _, _, _, row = reference(v, t, z, 2.0, True)
            return ref.sum() / row.sum() if reduce else (ref * w).sum()

        v = x.double()
        for r in range(5):
            for j in range(0, 31, 4):
                d = torch.zeros_like(v)
                d[r, j] = 1e-5
                diff = float((f(v + d) - f(v - d)) / 2e-5)
                # as for the log-probabilities: 1e-10 / 6 of a third derivative, 1e-11 / 2e-5 of rounding
                assert abs(float(y.grad[r, j]) - diff) <= 3e-6 + 1e-6 * abs(diff)
    y = x.clone().requires_grad_()
    h = y * 1.0
    pkg.distillation_loss(h, t, z, reduce_loss=True, inplace_grad=True).backward()
    assert bool(torch.isfinite(y.grad).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V,N", [(61, 20), (4096, 700), (70001, 400)])
def test_tokens_listed_often(V, N, dtype):
    # long lists of tokens drawn with replacement: of 61 columns each about 17 times, of others some
    # twice.  A column's entries are summed: at most 48 roundings, of the 200 that the bound allows.
    g = rng(V)
    x = (torch.randn(N, V, generator=g, device=DEV) * 3).to(dtype)
    t = torch.randint(0, V, (N, 1024), generator=g, device=DEV)
    t[::4, 1:] = t[::4, :1].clone()  # one token throughout ...
    t[::4, 40:] = -100               # ... of 40 entries
    z = torch.randn(N, 1024, generator=g, device=DEV) * 4
    check(x, t, z, 2.0, True, True)
    check(x, t[:, :300], z[:, :300], 1.0, True, False, in_place=True)


def test_second_backward_of_logits_given_up():
    """The first backward pass has replaced the logits: a second one is refused, not wrong."""
    x, t, z = make(5, 100, 6, torch.float32, 4, ignored=0.0)
    y = x.clone().requires_grad_()
    h = y * 1.0
    loss = pkg.distillation_loss(h, t, z, reduce_loss=True, inplace_grad=True)
    loss.backward(retain_graph=True)
    once = y.grad.clone()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    assert torch.equal(y.grad, once)
    y = x.clone().requires_grad_()
    loss = pkg.distillation_loss(y * 1.0, t, z, reduce_loss=True)
    loss.backward(retain_graph=True)
    assert torch.equal(y.grad, once)
    loss.backward()
    assert torch.equal(y.grad, 2 * once)


PROGRAM = """
import torch
import vocabulary_cross_entropy_pass_gb300 as pkg
x = torch.randn(20, 640, device="cuda")
t = torch.randint(0, 640, (20, 4), device="cuda")
z = torch.randn(20, 4, device="cuda")
ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
s = pkg.ce_logprobs_fwd(x, t, stats=True)[4]
d = pkg.ce_distill_fwd(x, t, z, stats=True)[1]
g = torch.ones(20, 4, device="cuda")
torch.cuda.synchronize()
calls = [lambda: pkg.ce_logprobs_fwd(x, t, top_k=3), lambda: pkg.ce_logprobs_bwd(x, s, t, grad_logprobs=g),
         lambda: pkg.ce_distill_fwd_bwd(x, t, z), lambda: pkg.ce_distill_bwd(x, t, z, d)]
for call in calls:
    call()
torch.cuda.synchronize()
for call in calls:
    with torch.cuda.stream(torch.cuda.Stream()):
        graph = torch.cuda.CUDAGraph()
        graph.capture_begin()
        status, _ = pkg.ce_get_error(ws)  # waits, which a capture does not allow
        try:
            graph.capture_end()
            print("captured")
        except RuntimeError:
            pass
    assert status == pkg.CEError(5).status == 5, status
    call()
torch.cuda.synchronize()
print("done")
"""


def test_a_refused_wait_is_not_the_next_launch_s_failure():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("done"), r.stdout + r.stderr[-2000:]


@pytest.mark.parametrize("N", [6, 1300])
def test_graph_and_streams(N):
    V = 9000
    x, t, z = make(N, V, 16, torch.bfloat16, 1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        pkg.ce_distill_fwd_bwd(x, t, z, reduce_loss=True)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = pkg.ce_distill_fwd_bwd(x, t, z, reduce_loss=True)
    for seed in (2, 3):
        x.copy_(make(N, V, 16, torch.bfloat16, seed)[0])
        graph.replay()
        graph.replay()
        want = pkg.ce_distill_fwd_bwd(x, t, z, reduce_loss=True)
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        y = x * 2
    got = pkg.ce_distill_fwd_bwd(y, t, z, stream=side)
    side.synchronize()
    want = pkg.ce_distill_fwd_bwd(y, t, z)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_teacher_to_student():
    """The operators as they are used together: the teacher's processed logits give the stored log-probabilities, the
    student is trained on them, in place, and its own log-probabilities of the teacher's first tokens rise."""
    N, V, K = 40, 6007, 32
    g = rng(3)
    teacher = (torch.randn(N, V, generator=g, device=DEV) * 3).to(torch.bfloat16)
    allowed = torch.randint(-2 ** 31, 2 ** 31, (N, (V + 31) // 32), generator=g, device=DEV).to(torch.int32)
    teacher = pkg.ce_logits_process(teacher, mask=allowed, temperature=torch.full((N,), 0.8, device=DEV))
    given = torch.randint(0, V, (N,), generator=g, device=DEV)
    given[::5] = -100
    _, _, top, top_lp, _ = pkg.ce_logprobs_fwd(teacher, given, top_k=K)
    student = torch.randn(N, V, generator=g, device=DEV).to(torch.bfloat16)
    check(student, top, top_lp, 1.0, False, True)
    check(student, top, top_lp, 2.0, True, True, in_place=True)
    first = top[:, 0].contiguous()
    before = pkg.ce_logprobs_fwd(student, first)[0]
    loss, grad = pkg.ce_distill_fwd_bwd(student, top, top_lp, normalize=False)
    after = pkg.ce_logprobs_fwd((student.float() - grad.float()), first)[0]
    kept = first != -100
    assert bool((after > before)[kept].all()) and bool((grad[~kept] == 0).all())
