"""Logits under long lists of biases and histories, of every form of the list
kernel, against float64 on the GPU.

Bounds: a column's n biases, added one after another in float32, are off by at most
n 2^-24 of the sum of their magnitudes; the other at most eight operations by
2^-24 each of no more than the sum of the terms' magnitudes: 2^-20 + n 2^-24 of
that sum, over the temperature, and one rounding to the storage type.
"""
import pytest
import torch

import vocabulary_cross_entropy_pass_gb300 as pkg

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
TINY = {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}


def make(N, V, L, K, dtype, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def rand(*shape):
        return torch.rand(*shape, generator=g, device=DEV)

    x = (torch.randn(N, V, generator=g, device=DEV) * 3).to(dtype)
    p = {"temperature": 0.5 + rand(N)}
    if L:
        p["history"] = torch.randint(-2, V + 2, (N, L), generator=g, device=DEV)
        p["history_lengths"] = torch.randint(L // 2, L + 1, (N,), generator=g, device=DEV)
        p["prompt_lengths"] = torch.randint(0, L // 2 + 1, (N,), generator=g, device=DEV)
        p["repetition_penalty"] = 1 + rand(N)
        p["frequency_penalty"] = rand(N) - 0.3
        p["presence_penalty"] = rand(N)
    if K:
        p["bias_tokens"] = torch.randint(-2, V + 2, (N, K), generator=g, device=DEV)
        p["bias_values"] = torch.randn(N, K, generator=g, device=DEV) * 4
    return x, p


def spread(tokens, values, V):
    """Sum of the values at their tokens, per row; tokens outside [0, V) nowhere."""
    ok = (tokens >= 0) & (tokens < V)
    out = torch.zeros(tokens.shape[0], V, dtype=torch.float64, device=DEV)
    return out.scatter_add_(1, tokens.clamp(0, V - 1), torch.where(ok, values, 0.0).double())


def check(got, x, p, go=None):
    V = x.shape[1]
    for r in range(0, x.shape[0], 256):  # a few rows at a time
        s = slice(r, r + 256)
        q = {k: v[s] for k, v in p.items()}
        z = x[s].double()
        temp = q["temperature"].double()[:, None]
        add, n = torch.zeros_like(z), torch.zeros_like(z)
        size = z.abs()
        if "history" in q:
            at = torch.arange(q["history"].shape[1], device=DEV)[None]
            inside = at < q["history_lengths"][:, None]
            seen = spread(q["history"], inside.float(), V) > 0
            rep = q["repetition_penalty"].double()[:, None]
            factor = torch.where(seen, torch.where(z > 0, 1 / rep, rep), 1.0)
            count = spread(q["history"], (inside & (at >= q["prompt_lengths"][:, None])).float(), V)
            freq, pres = (q[k].double()[:, None] for k in ("frequency_penalty", "presence_penalty"))
            add = -freq * count - pres * (count > 0)
            size = size * factor + freq.abs() * count + pres * (count > 0)
        else:
            factor = torch.ones_like(z)
        if go is not None:
            ref = go[s].double() * factor / temp
            bound = 2.0 ** -20 * ref.abs()
        else:
            if "bias_tokens" in q:
                add = add + spread(q["bias_tokens"], q["bias_values"], V)
                n = spread(q["bias_tokens"], torch.ones_like(q["bias_values"]), V)
                size = size + spread(q["bias_tokens"], q["bias_values"].abs(), V)
            ref = (z * factor + add) / temp
            bound = (2.0 ** -20 + n * 2.0 ** -24) * size / temp
        bound = bound + torch.finfo(x.dtype).eps / 2 * ref.abs() + TINY[x.dtype]
        assert bool(((got[s].double() - ref).abs() <= bound).all())


# biases: by a key beside many entries; a sum to each entry; one run to a part; runs made shorter
@pytest.mark.parametrize("N,V,L,K,dtype", [
    (17, 128000, 6000, 40, torch.bfloat16), (17, 128000, 0, 4095, torch.bfloat16),
    (512, 128000, 0, 8193, torch.bfloat16), (100, 128000, 0, 9000, torch.float16), (70, 32000, 0, 32000, torch.float32),
    (17, 128000, 8192, 8192, torch.bfloat16), (17, 128000, 0, 20000, torch.float32),
    (17, 128000, 0, 128000, torch.bfloat16), (1400, 128000, 32768, 1025, torch.bfloat16),
    (700, 128000, 0, 9000, torch.float32), (17, 128001, 40000, 40000, torch.float16)])
def test_long_lists_of_biases(N, V, L, K, dtype):
    x, p = make(N, V, L, K, dtype, N + L + K)
    got = pkg.ce_logits_process(x, **p)
    check(got, x, p)
    ws = torch.full((pkg.ce_logits_workspace_bytes(N, V, dtype, L, K),), 171, dtype=torch.uint8, device=DEV)
    assert torch.equal(pkg.ce_logits_process(x, workspace=ws, **p), got)
    if L:
        q = {k: p[k] for k in ("history", "history_lengths", "repetition_penalty", "temperature")}
        go = torch.randn_like(x)
        check(pkg.ce_logits_process_bwd(go, x, **q), x, p, go=go)
    # in place, the same bits
    y = x.clone()
    assert torch.equal(pkg.ce_logits_process(y, out=y, **p), got)


def test_many_biases_of_one_token():
    x, p = make(40, 128000, 0, 9001, torch.float32, 5)
    p["bias_tokens"][0] = 77
    p["bias_tokens"][1, 1::2] = 127999
    got = pkg.ce_logits_process(x, **p)
    check(got, x, p)
    # in list order: the same bits as a float32 loop
    s = torch.zeros(())
    for b in p["bias_values"][0].cpu():
        s = s + b
    one = {"bias_tokens": p["bias_tokens"], "bias_values": p["bias_values"]}
    assert float(pkg.ce_logits_process(x, **one)[0, 77]) == float(x[0, 77].cpu() + s)


@pytest.mark.parametrize("N,V", [(3, 5000), (40, 70001)])
def test_float32_quotients_are_rounded_once(N, V):
    # the repetition penalty's and the temperature's division, bit for bit
    x, p = make(N, V, 300, 0, torch.float32, N)
    rep, temp = p["repetition_penalty"][:, None], p["temperature"][:, None]
    inside = torch.arange(300, device=DEV)[None] < p["history_lengths"][:, None]
    seen = spread(p["history"], inside.float(), V) > 0
    q = {k: p[k] for k in ("history", "history_lengths", "repetition_penalty")}
    z = torch.where(seen, torch.where(x > 0, x / rep, x * rep), x)
    assert torch.equal(pkg.ce_logits_process(x, temperature=p["temperature"]), x / temp)
    assert torch.equal(pkg.ce_logits_process(x, **q), z)
    assert torch.equal(pkg.ce_logits_process(x, temperature=p["temperature"], **q), z / temp)
    go = torch.randn_like(x)
    g = torch.where(seen, torch.where(x > 0, go / rep, go * rep), go)
    assert torch.equal(pkg.ce_logits_process_bwd(go, x, temperature=p["temperature"], **q), g / temp)
    # values that a quotient takes out of the ordinary range, and an odd offset
    x[0, :6] = torch.tensor([float("inf"), -float("inf"), 0.0, -0.0, 1e-40, 3e38])
    assert torch.equal(pkg.ce_logits_process(x[:, 1:], temperature=p["temperature"]), x[:, 1:] / temp)
    assert torch.equal(pkg.ce_logits_process(x, temperature=p["temperature"]), x / temp)
