"""Penalties, biases, masks and the temperature on logits, and the gradient
through them, against plain float64 loops.

Bounds: each of the at most eight float32 operations of an output rounds by
2^-24 of a value no larger than the sum of the magnitudes of its terms,
(|z| + freq count + pres + sum |bias|) / temp; a sum of K biases adds K 2^-24 of
theirs.  2^-20 plus K 2^-24 of that sum, and one rounding to the storage type.
"""
import math

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


def pack_mask(allowed):
    """(N, V) booleans as int32 words."""
    N, V = allowed.shape
    W = (V + 31) // 32
    bits = torch.zeros(N, W * 32, dtype=torch.int64)
    bits[:, :V] = allowed
    words = (bits.view(N, W, 32) << torch.arange(32)).sum(-1)
    return torch.where(words >= 2 ** 31, words - 2 ** 32, words).to(torch.int32)


def make(N, V, dtype, seed, L=0, K=0, mask=None, temp=True):
    g = rng(seed)
    x = (torch.randn(N, V, generator=g) * 3).to(dtype)
    p = {}
    if L:
        p["history"] = torch.randint(0, max(1, V // 2), (N, L), generator=g) * 2 % V
        p["history_lengths"] = torch.randint(0, L + 1, (N,), generator=g)
        p["prompt_lengths"] = torch.randint(0, L // 2 + 1, (N,), generator=g)
        p["repetition_penalty"] = 1 + torch.rand(N, generator=g)
        p["frequency_penalty"] = torch.rand(N, generator=g) - 0.3
        p["presence_penalty"] = torch.rand(N, generator=g)
    if K:
        p["bias_tokens"] = torch.randint(0, V, (N, K), generator=g)
        p["bias_values"] = torch.randn(N, K, generator=g) * 4
    if mask is not None:
        p["mask"] = pack_mask(torch.rand(N, V, generator=g) < mask)
    if temp:
        p["temperature"] = 0.5 + torch.rand(N, generator=g)
    return x, p


def reference(x, p, go=None):
    """(outputs or gradients, magnitude of their terms, allowed) in float64; rows flattened."""
    V = x.shape[-1]
    x = x.reshape(-1, V).double()
    N = x.shape[0]
    out, mag = torch.empty(N, V, dtype=torch.float64), torch.empty(N, V, dtype=torch.float64)
    allowed = torch.ones(N, V, dtype=torch.bool)
    for r in range(N):
        seen = torch.zeros(V, dtype=torch.bool)
        count = torch.zeros(V, dtype=torch.float64)
        if p.get("history") is not None:
            L = p["history"].shape[1]
            n = L if p.get("history_lengths") is None else min(max(int(p["history_lengths"][r]), 0), L)
            start = 0 if p.get("prompt_lengths") is None else int(p["prompt_lengths"][r])
            t = p["history"][r, :n]
            ok = (t >= 0) & (t < V)
            seen[t[ok]] = True
            new = ok & (torch.arange(n) >= start)
            count += torch.bincount(t[new], minlength=V)
        rep = 1.0 if p.get("repetition_penalty") is None else float(p["repetition_penalty"][r])
        freq = 0.0 if p.get("frequency_penalty") is None else float(p["frequency_penalty"][r])
        pres = 0.0 if p.get("presence_penalty") is None else float(p["presence_penalty"][r])
        temp = 1.0 if p.get("temperature") is None else float(p["temperature"][r])
        factor = torch.where(seen, torch.where(x[r] > 0, 1 / rep, rep), 1.0)
        if go is None:
            z = torch.where(seen, x[r] * factor, x[r])
            m = z.abs() + abs(freq) * count + abs(pres) * (count > 0)
            z = z - freq * count - pres * (count > 0)
            if p.get("bias_tokens") is not None:
                K = p["bias_tokens"].shape[1]
                for k in range(K):
                    t = int(p["bias_tokens"][r, k])
                    if 0 <= t < V:
                        z[t] += float(p["bias_values"][r, k])
                        m[t] += abs(float(p["bias_values"][r, k])) * (1 + K / 16)
            out[r], mag[r] = z / temp, m / temp
        else:
            out[r] = go.reshape(-1, V)[r].double() * factor / temp
            mag[r] = out[r].abs()
        if p.get("mask") is not None:
            words = p["mask"].reshape(-1, p["mask"].shape[-1])
            w = words[r if words.shape[0] > 1 else 0].long()
            v = torch.arange(V)
            allowed[r] = ((w[v // 32] >> (v % 32)) & 1) != 0
    return out, mag, allowed


def check(got, x, p, go=None, mask_value=-math.inf):
    ref, mag, allowed = reference(x.cpu(), p, go if go is None else go.cpu())
    blocked = 0.0 if go is not None else float(torch.tensor(mask_value, dtype=got.dtype))
    dtype, got = got.dtype, got.reshape(ref.shape).double().cpu()
    assert bool((got[~allowed] == blocked).all())
    a, b, m = got[allowed], ref[allowed], mag[allowed]
    same = torch.isfinite(b)
    assert torch.equal(a[~same].nan_to_num(7e300), b[~same].nan_to_num(7e300))
    worst = ((a - b).abs() - 2.0 ** -20 * m - half_step(dtype) * b.abs() - TINY[dtype])[same]
    assert worst.numel() == 0 or float(worst.max()) <= 0, float(worst.max())


def dev(p):
    return {k: v.to(DEV) if isinstance(v, torch.Tensor) else v for k, v in p.items()}


def bwd_params(p):
    return {k: v for k, v in p.items() if k in ("history", "history_lengths", "repetition_penalty", "mask",
                                                "temperature")}


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [1, 7, 31, 32, 33, 100, 4095, 4096, 4097, 8200, 10001])
def test_every_step(V, dtype):
    for k, (N, L, K, mask, temp) in enumerate([(1, 9, 5, 0.5, True), (3, 0, 0, 0.1, True), (2, 40, 0, None, False),
                                               (2, 0, 70, None, True), (4, 300, 3, 0.9, True), (1, 0, 0, None, False)]):
        x, p = make(N, V, dtype, V + k, L, K, mask, temp)
        check(pkg.ce_logits_process(x.to(DEV), **dev(p)), x, p)
        go = torch.randn(N, V, generator=rng(V)).to(dtype)
        check(pkg.ce_logits_process_bwd(go.to(DEV), x.to(DEV), **dev(bwd_params(p))), x, p, go=go)


@pytest.mark.parametrize("N,V,L", [(1, 32000, 2000), (42, 50257, 64), (3, 128000, 700)])
def test_wide_rows(N, V, L):
    x, p = make(N, V, torch.bfloat16, N, L, 20, 0.05)
    xd, pd = x.to(DEV), dev(p)
    got = pkg.ce_logits_process(xd, **pd)
    check(got, x, p)
    assert torch.equal(pkg.ce_logits_process(xd, **pd), got)
    go = torch.randn(N, V, generator=rng(V)).to(torch.bfloat16)
    check(pkg.ce_logits_process_bwd(go.to(DEV), xd, **dev(bwd_params(p))), x, p, go=go)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("L,K", [(1, 0), (0, 1), (63, 0), (61, 20), (127, 2), (513, 0), (600, 301)])
def test_tables_of_odd_sizes(L, K, dtype):
    # many columns in all: a kernel of its own finds the touched ones
    x, p = make(42, 50257, dtype, L + K, L, K, 0.3)
    xd = x.to(DEV)
    check(pkg.ce_logits_process(xd, **dev(p)), x, p)
    if L:
        go = torch.randn(42, 50257, generator=rng(L)).to(dtype)
        check(pkg.ce_logits_process_bwd(go.to(DEV), xd, **dev(bwd_params(p))), x, p, go=go)
    want = pkg.ce_logits_process(xd, **dev(p))
    assert torch.equal(pkg.ce_logits_process(xd, out=xd, **dev(p)), want)


@pytest.mark.parametrize("N,V,L,K", [(6, 400000, 9000, 3), (17, 128000, 70000, 0), (17, 128000, 1000, 3000),
                                     (520, 4096, 5000, 0), (3, 1 << 20, 300, 40), (2, 128000, 70000, 9),
                                     (3, 5000, 100000, 0)])
def test_long_lists(N, V, L, K):
    x, p = make(N, V, torch.bfloat16, L, L, K, 0.5)
    p["history_lengths"][0] = L
    xd, pd = x.to(DEV), dev(p)
    got = pkg.ce_logits_process(xd, **pd)
    check(got, x, p)
    assert torch.equal(pkg.ce_logits_process(xd, **pd), got)
    go = torch.randn(N, V, generator=rng(V)).to(torch.bfloat16)
    check(pkg.ce_logits_process_bwd(go.to(DEV), xd, **dev(bwd_params(p))), x, p, go=go)


def test_more_rows_than_a_grid_dimension():
    N, V = 70001, 64
    g = rng(20)
    x = torch.randn(N, V, generator=g).to(DEV)
    p = dict(history=torch.randint(0, V, (N, 3), generator=g).to(DEV), frequency_penalty=torch.rand(N, generator=g).to(DEV),
             mask=torch.randint(-2 ** 31, 2 ** 31, (N, 2), generator=g).to(torch.int32).to(DEV))
    got = pkg.ce_logits_process(x, **p)
    for rows in (slice(0, 40000), slice(40000, N)):
        assert torch.equal(got[rows], pkg.ce_logits_process(x[rows], **{k: v[rows] for k, v in p.items()}))
    some = torch.randint(0, N, (40,), generator=g)
    check(got[some.to(DEV)], x[some.to(DEV)], {k: v.cpu()[some] for k, v in p.items()})


def test_penalties_alone_and_signs():
    V = 64
    x = torch.linspace(-4, 4, V).repeat(2, 1)
    x[0, 5], x[0, 6], x[0, 7] = 0.0, float("inf"), -float("inf")
    hist = torch.tensor([[3, 5, 6, 7, 60, 60, 60, 3], [1, 1, 1, 1, 1, 1, 1, 1]])
    for name in ("repetition_penalty", "frequency_penalty", "presence_penalty"):
        p = {"history": hist, name: torch.tensor([1.5, 0.75])}
        check(pkg.ce_logits_process(x.to(DEV), **dev(p)), x, p)
        p["prompt_lengths"] = torch.tensor([5, 100])  # a prompt longer than the history counts nowhere
        check(pkg.ce_logits_process(x.to(DEV), **dev(p)), x, p)
    p = {"history": hist, "repetition_penalty": torch.tensor([1.5, 0.75])}
    go = torch.ones(2, V)
    check(pkg.ce_logits_process_bwd(go.to(DEV), x.to(DEV), **dev(p)), x, p, go=go)


def test_histories_of_no_length_and_of_strangers():
    V = 500
    x, p = make(4, V, torch.float32, 3, L=20)
    p["history_lengths"] = torch.tensor([0, -5, 1000, 20])  # clamped to what there is
    p["history"][2, ::2] = -100
    p["history"][3, 1], p["history"][3, 2] = V, 1 << 40
    check(pkg.ce_logits_process(x.to(DEV), **dev(p)), x, p)
    empty = {"history": torch.zeros(4, 0, dtype=torch.int64), "repetition_penalty": torch.full((4,), 2.0)}
    assert torch.equal(pkg.ce_logits_process(x.to(DEV), **dev(empty)), x.to(DEV))


def test_biases_repeat_and_ban():
    V = 300
    x, p = make(3, V, torch.float32, 4, K=100)
    p["bias_tokens"][0] = 17                    # all on one token
    p["bias_tokens"][1, ::3] = -1
    p["bias_tokens"][2, 5], p["bias_values"][2, 5] = 299, -float("inf")
    got = pkg.ce_logits_process(x.to(DEV), **dev(p))
    check(got, x, p)
    assert float(got[2, 299]) == -float("inf")
    # in list order: the same bits as a float32 loop
    p = {"bias_tokens": p["bias_tokens"][:1], "bias_values": p["bias_values"][:1]}
    s = torch.zeros(())
    for b in p["bias_values"][0]:
        s = s + b
    assert float(pkg.ce_logits_process(x[:1].to(DEV), **dev(p))[0, 17]) == float(x[0, 17] + s)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [70, 4096, 4133])
def test_masks(V, dtype):
    x, p = make(4, V, dtype, V, L=30, K=4)
    allowed = torch.rand(4, V, generator=rng(8)) < 0.5
    allowed[1] = False                          # nothing is left
    allowed[2] = True
    allowed[3] = False
    allowed[3, V - 1] = True
    x[0][~allowed[0]] = float("nan")            # what is masked plays no part
    x[1, ::2], x[1, 1::2] = float("inf"), float("nan")
    p["mask"] = pack_mask(allowed)
    for value in (-math.inf, -3e4, float(torch.finfo(dtype).min), 0.0):
        check(pkg.ce_logits_process(x.to(DEV), mask_value=value, **dev(p)), x, p, mask_value=value)
    go = torch.randn(4, V, generator=rng(9)).to(dtype)
    go[0][~allowed[0]] = float("nan")
    check(pkg.ce_logits_process_bwd(go.to(DEV), x.to(DEV), **dev(bwd_params(p))), x, p, go=go)
    p["mask"] = p["mask"][2:3]                  # one mask for all rows
    got = pkg.ce_logits_process(torch.zeros_like(x).to(DEV), **dev(p))
    check(got, torch.zeros_like(x), p)
    p["mask"] = p["mask"][0]
    assert torch.equal(pkg.ce_logits_process(torch.zeros_like(x).to(DEV), **dev(p)), got)


@pytest.mark.parametrize("dtype", TYPES)
def test_strides_layouts_and_in_place(dtype):
    g = rng(10)
    V = 777
    wide = torch.randn(3, 4, V + 23, generator=g).to(dtype).to(DEV)
    _, p = make(12, V, dtype, 10, L=25, K=6, mask=0.4)
    pd = dev(p)
    for x in (wide[:, :, :V], wide[:, :, 3:3 + V], wide.transpose(0, 1)[:, :, 1:1 + V]):
        got = pkg.ce_logits_process(x, **pd)
        assert got.shape == x.shape
        check(got, x.reshape(12, V), p)
        # into a place with another offset from 16 bytes, and into its own
        other = torch.full((*x.shape[:2], V + 9), 5.0, dtype=dtype, device=DEV)
        pkg.ce_logits_process(x, out=other[:, :, 2:2 + V], **pd)
        assert torch.equal(other[:, :, 2:2 + V], got)
        assert bool((other[:, :, :2] == 5).all()) and bool((other[:, :, 2 + V:] == 5).all())
        go = torch.randn(x.shape, generator=g).to(dtype).to(DEV)
        gx = pkg.ce_logits_process_bwd(go, x, **dev(bwd_params(p)))
        check(gx, x.reshape(12, V), p, go=go)
        pkg.ce_logits_process_bwd(go, x, grad=other[:, :, 2:2 + V], **dev(bwd_params(p)))
        assert torch.equal(other[:, :, 2:2 + V], gx)
        assert torch.equal(pkg.ce_logits_process_bwd(go, x, grad=go, **dev(bwd_params(p))), gx)
        pkg.ce_logits_process(x, out=x, **pd)
        assert torch.equal(x, got)
        wide.copy_(torch.randn(3, 4, V + 23, generator=g).to(dtype))
    # strided lists
    h = torch.randint(0, V, (12, 60), generator=g).to(DEV)
    q = dict(history=h[:, 7:40], frequency_penalty=pd["frequency_penalty"], bias_tokens=h[:, 40:50],
             bias_values=torch.randn(12, 30, generator=g).to(DEV)[:, 3:13])
    x = wide[:, :, :V]
    check(pkg.ce_logits_process(x, **q), x.reshape(12, V), {k: v.cpu() for k, v in q.items()})


def test_refusals():
    x = torch.zeros(4, 100, device=DEV)
    hist = torch.zeros(4, 9, dtype=torch.int64, device=DEV)
    one = torch.ones(4, device=DEV)
    bad = [dict(repetition_penalty=one), dict(history=hist.int()), dict(history=hist[:3]),
           dict(history=hist, repetition_penalty=one[:3]), dict(history=hist, repetition_penalty=one.double()),
           dict(history=hist, history_lengths=one), dict(history=hist.cpu()), dict(bias_tokens=hist),
           dict(bias_tokens=hist, bias_values=torch.zeros(4, 8, device=DEV)),
           dict(mask=torch.zeros(4, 3, dtype=torch.int32, device=DEV)),
           dict(mask=torch.zeros(3, 4, dtype=torch.int32, device=DEV)),
           dict(mask=torch.zeros(4, 4, dtype=torch.int64, device=DEV)), dict(temperature=one.half()),
           dict(history=torch.zeros(4, 18, dtype=torch.int64, device=DEV)[:, ::2])]
    for kw in bad:
        with pytest.raises((TypeError, ValueError)):
            pkg.ce_logits_process(x, **kw)
        with pytest.raises((TypeError, ValueError)):
            pkg.ce_logits_process_bwd(x, x, **kw)
    with pytest.raises(ValueError):
        pkg.ce_logits_process(x.t())
    with pytest.raises(ValueError):
        pkg.ce_logits_process(x, out=x[:, :50])
    with pytest.raises(pkg.CEError):
        pkg.ce_logits_process_bwd(torch.zeros_like(x), x, grad=x)
    with pytest.raises(TypeError):
        pkg.ce_logits_process(x.double())
    assert pkg.ce_logits_process(x[:0]).shape == (0, 100)


def test_autograd_and_differences():
    N, V = 5, 333
    x, p = make(N, V, torch.float32, 12, L=50, K=5, mask=0.6)
    x = torch.where(x.abs() < 0.2, 0.5 + x, x)  # away from the kink of the repetition penalty
    pd = dev(p)
    c = torch.randn(N, V, generator=rng(2)).to(DEV)
    xd = x.to(DEV).requires_grad_()

    def loss(t):
        out = pkg.ce_logits_process(t, mask_value=0.0, **pd)
        return float((out.double() * c.double()).sum())

    (pkg.process_logits(xd, mask_value=0.0, **pd) * c).sum().backward()
    check(xd.grad, x, p, go=c)
    v = torch.randn(N, V, generator=rng(3)).to(DEV)
    v = v.clamp(-2, 2)
    e = 2.0 ** -5
    diff = (loss(xd.detach() + e * v) - loss(xd.detach() - e * v)) / (2 * e)
    # piecewise linear: off by the rounding of 1665 values of about 16 over 2e
    assert abs(diff - float((xd.grad.double() * v.double()).sum())) <= 1665 * 16 * 2.0 ** -22 / (2 * e)


def test_policy_log_probabilities():
    """Cross-entropy on the processed logits: log-probabilities under the
    distribution the tokens were drawn from, and their gradient."""
    N, V = 24, 1000
    x, p = make(N, V, torch.float32, 13, L=30, K=3)
    allowed = torch.rand(N, V, generator=rng(4)) < 0.3
    t = torch.randint(0, V, (N,), generator=rng(5))
    allowed[torch.arange(N), t] = True
    p["mask"] = pack_mask(allowed)
    xd = x.to(DEV).requires_grad_()
    out = pkg.process_logits(xd, mask_value=-3e4, **dev(p))
    loss = pkg.parallel_cross_entropy(out.unsqueeze(0), t.to(DEV).unsqueeze(0))
    loss.sum().backward()
    ref, _, _ = reference(x, p)
    ref = torch.where(allowed, ref, -3e4).requires_grad_()
    want = torch.nn.functional.cross_entropy(ref, t, reduction="none")
    assert float((loss[0].detach().double().cpu() - want.detach()).abs().max()) <= 1e-4
    want.sum().backward()
    gref, _, _ = reference(x, p, go=ref.grad)
    gref = torch.where(allowed, gref, 0.0)
    assert float((xd.grad.double().cpu() - gref).abs().max()) <= 2e-5
    assert bool((xd.grad.cpu()[~allowed] == 0).all())


def test_other_stream_and_graph():
    x, p = make(8, 5000, torch.bfloat16, 14, L=100, K=10, mask=0.3)
    xd, pd = x.to(DEV), dev(p)
    want = pkg.ce_logits_process(xd, **pd)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(xd)
    pkg.ce_logits_process(xd, out=out, stream=side, **pd)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = pkg.ce_logits_process(xd, **pd)
        g = pkg.ce_logits_process_bwd(y, xd, grad=out, **bwd_params(pd))
    pd["history"].copy_(torch.randint(0, 5000, (8, 100), generator=rng(6)))
    want = pkg.ce_logits_process(xd, **pd)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want) and g.data_ptr() == out.data_ptr()


def test_offsets_past_32_bits():
    N, V = 20000, 128000  # 2.56e9 logits, 5 GB
    x = torch.zeros(N, V, dtype=torch.bfloat16, device=DEV)
    at = torch.tensor([0, 16776, 16777, 19999])
    g = rng(15)
    rows = (torch.randn(4, V, generator=g) * 3).to(torch.bfloat16)
    x[at.to(DEV)] = rows.to(DEV)
    hist = torch.randint(0, V, (4, 50), generator=g)
    full = torch.full((N, 50), -1, dtype=torch.int64)
    full[at] = hist
    rep = torch.full((N,), 1.5)
    got = pkg.ce_logits_process(x, out=x, history=full.to(DEV), repetition_penalty=rep.to(DEV))
    check(got[at.to(DEV)], rows, {"history": hist, "repetition_penalty": rep[:4]})
    assert bool((got[10000:10010] == 0).all())
