"""Logits and masks far from zero: finite mask values of any size, rows of nothing else, rows that are far from zero
throughout.

Bounds: those of the log-probabilities' and the distillation's tests, which hold at any size of the logits, since
log-probabilities are of differences from the row's maximum.  The exponents' reference is the maximum's product
with log2(e), rounded: off by `short`, 64 at most, and no product from 2^31 on.  Exponents of up to 64 are then
rounded by 2^-18, and so is the binary logarithm of their sum, which is below 64 + 17: together ln 2 (2^-18 + 2^-18) =
89 * 2^-24 of the 128 * 2^-24 that the bounds allow, whose other terms come to less than 2 log V at the sizes used
here.  The entropy is the difference of that logarithm and of a mean of the exponents, each of whose terms has 70
additions and two products behind it in the sum and 70 in the divisor: 2^-24 * 144 short more.
"""
import math

import pytest
import torch

import vocabulary_cross_entropy_pass_gb300 as pkg

from . import test_gpu_distill as distill
from . import test_gpu_logprobs as logprobs

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
WIDE = [torch.float32, torch.bfloat16]  # float16 has no such values
FAR = [-1e6, -3e7, -1e9, -4e9, -1e10, -1e12, -1e15, -1e20, -1e30, -1e35, -1e37, -2.2e38]


LOG2E = 1.4426950408889634


def rng(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def masked(N, V, dtype, value, seed):
    """A few tokens allowed, one, none, all but a range; the rest at `value`."""
    x = torch.randn(N, V, generator=rng(seed), device=DEV) * 3
    keep = torch.rand(N, V, generator=rng(seed + 1), device=DEV) < 1 / 256
    keep[1::4] = False
    keep[1::4, 17] = True
    keep[2::4] = False
    keep[3::4] = True
    keep[3::4, V // 3:V // 2] = False
    return x.to(dtype).masked_fill(~keep, value)


def distinct(N, V, K, seed):
    return (torch.randint(0, V, (N, 1), generator=rng(seed), device=DEV) + torch.arange(K, device=DEV) * (V // K)) % V


def short(x):
    m = x.amax(1).float()
    product = m * torch.tensor(LOG2E, device=DEV)  # rounded to float32
    off = (m.double() * float(torch.tensor(LOG2E)) - product.double()).abs()
    return torch.where(product.abs() < 2.0 ** 31, off, 0.0)


def check_forward(x, t, **kw):
    logprobs.check_forward(x, t, entropy=False, **kw)
    _, got, *_ = pkg.ce_logprobs_fwd(x, t, entropy=True, **kw)
    want = logprobs.reference(x, t)[1]
    bound = logprobs.E * (160 * (1 + math.log(x.shape[1])) + 144 * short(x))
    assert bool(((got.double() - want).abs() <= bound).all())


@pytest.mark.parametrize("value", FAR)
@pytest.mark.parametrize("dtype", WIDE)
@pytest.mark.parametrize("N,V", [(4, 9000), (1300, 9000), (5, 40008)])
def test_masked_log_probabilities(N, V, dtype, value):
    x = masked(N, V, dtype, value, 11)
    t = distinct(N, V, 3, 5)
    check_forward(x, t, top_k=20)
    check_forward(x, t)
    gl = torch.randn(N, 3, generator=rng(2), device=DEV)
    # (through the entropy where its bound is the other tests')
    logprobs.check_backward(x, t, gl, gl[:, 0].contiguous() if float(short(x).max()) <= 1 else None)


@pytest.mark.parametrize("value", FAR)
@pytest.mark.parametrize("dtype", WIDE)
@pytest.mark.parametrize("N", [4, 1300])
def test_masked_students(N, dtype, value):
    V, K = 9000, 16
    x = masked(N, V, dtype, value, 3)
    x[2::4] = value  # (log-probabilities of listed tokens that are masked are far below any bound elsewhere)
    t = distinct(N, V, K, 4)
    t[1::4] = distinct(N, V, K, 5)[1::4]
    x[0::4] = x[0::4].scatter(1, t[0::4], 1.0)
    x[1::4] = x[1::4].scatter(1, t[1::4], -2.0)
    x[3::4] = x[3::4].scatter(1, t[3::4], 0.5)
    z = torch.randn(N, K, generator=rng(6), device=DEV) * 4
    for tau in (0.5, 1.0, 4.0):
        distill.check(x, t, z, tau, reduce=tau == 1.0)
    distill.check(x, t, z, 2.0, in_place=True)


@pytest.mark.parametrize("scale", [1e7, 1e10, 1e25, 1e37])
@pytest.mark.parametrize("dtype", WIDE)
def test_rows_far_from_zero(dtype, scale):
    """Rows of one large value, or of large values next to each other: neighbours in the type."""
    V = 4104
    i = torch.arange(V, device=DEV, dtype=torch.float64)
    step = float(torch.finfo(dtype).eps)
    x = torch.stack([torch.full((V,), scale, device=DEV, dtype=torch.float64),
                     torch.full((V,), -scale, device=DEV, dtype=torch.float64),
                     scale * (1 + step * (i % 3)),
                     -scale * (1 + step * (i % 2)),
                     torch.where(i < 2000, scale, -scale),
                     torch.where(i % 8 == 3, 5.0, -scale)]).to(dtype)
    t = distinct(6, V, 4, 1)
    check_forward(x, t, top_k=8)
    check_forward(x.repeat(220, 1), t.repeat(220, 1), top_k=8)
    logprobs.check_backward(x, t, torch.ones(6, 4, device=DEV), torch.ones(6, device=DEV))


@pytest.mark.parametrize("dtype", WIDE)
def test_neighbours_at_the_reference(dtype):
    """Maxima on both sides of the size from which differences are taken: the warps of a row, its segments and the
    elements around its body meet with references of both kinds."""
    for top in (2.0 ** 29, 2.0 ** 31 / 1.4426950408889634, 2.0 ** 31, 2.0 ** 32):
        V = 40003
        i = torch.arange(V, device=DEV, dtype=torch.float64)
        eps = float(torch.finfo(dtype).eps)
        for sign in (1.0, -1.0):
            base = sign * top * (1 + eps * ((i // 977) % 3 - 1))
            x = torch.stack([base, base.flip(0), torch.full_like(i, sign * top)]).to(dtype)
            t = distinct(3, V, 4, 1)
            check_forward(x, t, top_k=8)
            check_forward(x.repeat(440, 1), t.repeat(440, 1))
