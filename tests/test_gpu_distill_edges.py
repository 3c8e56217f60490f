"""Listed tokens among the elements around a row's 16-byte vectors: each such column is stored by one lane as an element
of the row and again, with the teacher's part, by the lane that has its entry; the second has to be the one that stays."""
import pytest
import torch

import vocabulary_cross_entropy_pass_gb300 as pkg

from .test_gpu_distill import DEV, TYPES, check, rng

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N,V", [(9, 31), (40, 4099), (2500, 1003), (400, 70005)])
def test_tokens_around_the_body(N, V, dtype):
    g = rng(V)
    x = torch.randn(N, V + 9, generator=g, device=DEV).to(dtype)
    # the first and last seven columns and two inside, in an order of each row's own
    edges = torch.cat([torch.arange(7), torch.arange(V - 7, V), torch.tensor([V // 2, V // 3])]).to(DEV)
    t = edges[torch.rand(N, 16, generator=g, device=DEV).argsort(1)]
    z = torch.randn(N, 16, generator=g, device=DEV) * 2
    for shift in (0, 1, 5):
        rows = x[:, shift:shift + V]
        check(rows, t, z, 1.0)
        check(rows, t, z, 2.0, in_place=True)
    # in place in a padded buffer, which keeps what is around the rows
    own = x.clone()
    loss, grad = pkg.ce_distill_fwd_bwd(own[:, 3:3 + V], t, z, grad=own[:, 3:3 + V])
    other = pkg.ce_distill_fwd_bwd(x[:, 3:3 + V], t, z)[1]
    # both within (200 + 2 |lp| + 160) 2^-24 of terms of 2 in all, |lp| below 20, and a rounding to the type
    assert bool(((grad.double() - other.double()).abs() <= torch.finfo(dtype).eps * other.double().abs() + 1600 * 2.0 ** -24)
                .all())
    assert torch.equal(own[:, :3], x[:, :3]) and torch.equal(own[:, 3 + V:], x[:, 3 + V:])
