"""The operators around the pass on a stream handed in: what a call allocates
itself belongs to that stream, so nothing that the caller's own stream allocates
meanwhile can meet it, and the same bits come out as on the caller's stream."""
import pytest
import torch

import vocabulary_cross_entropy_pass_gb300 as pkg

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
WAIT = 20_000_000  # cycles: about ten milliseconds


def rng(seed):
    return torch.Generator().manual_seed(seed)


def embed_calls(N, tokens_of=lambda t: t):
    g = rng(N)
    go = torch.randn(N, 64, generator=g).to(DEV)
    t = torch.randint(0, 700, (N,), generator=g).to(DEV)
    v = tokens_of(t)
    size = pkg.ce_embed_bwd_workspace_bytes(N, 64, 700)
    rows = go.view(*v.shape, 64)
    return lambda **kw: pkg.ce_embed_bwd(rows, v, 700, **kw), [size, N * 8]


def norm_call():
    g = rng(1)
    go, h = (torch.randn(3000, 1024, generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))
    w = torch.randn(1024, generator=g).to(torch.bfloat16).to(DEV)
    return lambda **kw: pkg.ce_rmsnorm_bwd(go, h, w, **kw), [pkg.ce_rmsnorm_bwd_workspace_bytes(3000, 1024)]


def logits_inputs():
    g = rng(2)
    x = torch.randn(64, 50257, generator=g).to(torch.bfloat16).to(DEV)
    p = dict(history=torch.randint(0, 50257, (64, 900), generator=g).to(DEV),
             repetition_penalty=(1 + torch.rand(64, generator=g)).to(DEV))
    size = pkg.ce_logits_workspace_bytes(64, 50257, torch.bfloat16, 900, 0)
    assert size > 0
    return x, p, size


def logits_call():
    x, p, size = logits_inputs()
    return lambda **kw: pkg.ce_logits_process(x, **p, **kw), [size]


def logits_bwd_call():
    x, p, size = logits_inputs()
    go = torch.randn(64, 50257, generator=rng(3)).to(torch.bfloat16).to(DEV)
    return lambda **kw: pkg.ce_logits_process_bwd(go, x, **p, **kw), [size]


CALLS = {
    "embedding gradient, few tokens": lambda: embed_calls(60),
    "embedding gradient, sorted": lambda: embed_calls(3000),
    "embedding gradient, tokens to be copied": lambda: embed_calls(
        3000, lambda t: t.view(10, 20, 15).transpose(0, 2).contiguous().transpose(0, 2)),
    "norm gradients": norm_call,
    "logits": logits_call,
    "logits gradient": logits_bwd_call,
}


def same(a, b):
    a, b = ([x] if isinstance(x, torch.Tensor) else list(x) for x in (a, b))
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("name", list(CALLS))
def test_memory_belongs_to_the_stream_handed_in(name):
    call, sizes = CALLS[name]()
    want = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(WAIT)
    got = call(stream=side)
    # the caller's stream takes blocks of the same sizes at once and writes them
    junk = [torch.full((n,), 171, dtype=torch.uint8, device=DEV) for n in sizes for _ in range(4)]
    side.synchronize()
    assert same(got, want)
    del junk


def test_output_lasts_as_long_as_its_reader():
    call, _ = CALLS["embedding gradient, sorted"]()
    want = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(WAIT)
    copy = got.clone()
    del got  # the other stream may not have its memory before the copy is made
    with torch.cuda.stream(side):
        junk = [torch.full_like(want, 7.0) for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(copy, want) and len(junk) == 4


def test_the_current_stream_handed_in_by_any_name():
    call, _ = CALLS["embedding gradient, sorted"]()
    want = call()
    assert same(call(stream=torch.cuda.current_stream()), want)
    assert same(call(stream=torch.cuda.default_stream()), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(stream=torch.cuda.ExternalStream(side.cuda_stream))
    side.synchronize()
    assert same(got, want)
    with torch.cuda.stream(side):
        got = call(stream=side)
    side.synchronize()
    assert same(got, want)
    assert torch.cuda.current_stream() == torch.cuda.default_stream()


def test_a_workspace_is_one_run_of_memory():
    # a view's elements say more than its memory holds
    one = torch.zeros(1, dtype=torch.uint8, device=DEV)
    spaced = torch.zeros(1 << 21, dtype=torch.uint8, device=DEV)
    x, p, size = logits_inputs()
    go, w = torch.zeros(60, 64, device=DEV), torch.ones(64, device=DEV)
    t = torch.zeros(60, dtype=torch.int64, device=DEV)
    many = 1 << 27
    assert size < many
    for ws in (one.expand(many), spaced[::2]):
        for call in (lambda: pkg.ce_embed_fwd(t, go, workspace=ws), lambda: pkg.ce_embed_bwd(go, t, 60, workspace=ws),
                     lambda: pkg.ce_rmsnorm_bwd(go, go, w, workspace=ws),
                     lambda: pkg.ce_logits_process(x, workspace=ws, **p),
                     lambda: pkg.ce_logits_process_bwd(x, x, workspace=ws, **p)):
            with pytest.raises(ValueError, match="contiguous"):
                call()


def pass_calls():
    """The cross-entropy passes, each with its inputs twice (one overwrites them)."""
    g = rng(7)
    N, V, H = 64, 50257, 72
    x = torch.randn(1, N, V, generator=g).to(torch.bfloat16).to(DEV)
    t = torch.randint(0, V, (1, N), generator=g).to(DEV)
    lse = torch.empty(N, device=DEV)
    n = torch.empty(1, dtype=torch.int64, device=DEV)
    pkg.ce_fwd_only(x, t, reduce_loss=True, lse_out=lse, n_non_ignore_out=n)
    part = pkg.ce_vp_partials(x, t, 0).unsqueeze(0).repeat(1, 1, 2)[:, :, :4]  # not contiguous
    hidden = torch.randn(N, 2 * H, generator=g).to(torch.bfloat16).to(DEV)[:, ::2]
    weight = torch.randn(900, H, generator=g).to(torch.bfloat16).to(DEV)
    few = t[0] % 900
    twice = [x.clone(), x.clone()]

    def in_place(**kw):
        y = twice.pop()
        return pkg.ce_fwd_bwd(y, t, reduce_loss=True, **kw), y

    size = pkg.ce_workspace_bytes(1, N, V, torch.bfloat16)
    return {
        "loss": (lambda **kw: pkg.ce_fwd_only(x, t, reduce_loss=True, **kw), [size]),
        "loss and gradient": (in_place, [size]),
        "gradient": (lambda **kw: pkg.ce_bwd(x, t, lse, reduce_loss=True, n_non_ignore=n, **kw), []),
        "partials": (lambda **kw: pkg.ce_vp_partials(x, t, 0, **kw), []),
        "combined": (lambda **kw: pkg.ce_vp_combine(part, [0, V], t, reduce_loss=True, **kw), [size, N * 16]),
        "shard's gradient": (lambda **kw: pkg.ce_vp_bwd(x, t, 0, V, lse, **kw), []),
        "lm_head": (lambda **kw: pkg.ce_linear_fwd_bwd(hidden, weight, few, reduce_loss=True, **kw),
                    [N * H * 2, 900 * H * 4]),
    }


@pytest.mark.parametrize("name", ["loss", "loss and gradient", "gradient", "partials", "combined", "shard's gradient",
                                  "lm_head"])
def test_the_passes_memory_belongs_to_the_stream_handed_in(name):
    call, sizes = pass_calls()[name]
    want = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(WAIT)
    got = call(stream=side)
    junk = [torch.full((n,), 171, dtype=torch.uint8, device=DEV) for n in sizes for _ in range(4)]
    side.synchronize()
    assert same(got, want)
    assert torch.cuda.current_stream() == torch.cuda.default_stream()
    del junk
