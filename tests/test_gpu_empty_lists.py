"""Lists without tokens, with and without rows, forward and backward."""
import pytest
import torch

import vocabulary_cross_entropy_pass_gb300 as pkg

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


@pytest.mark.parametrize("shape", [(0, 40), (3, 40), (0, 2, 40), (2, 0, 40), (2, 3, 40)])
@pytest.mark.parametrize("entropy", [True, False])
def test_autograd(shape, entropy):
    x = torch.randn(shape, device=DEV, requires_grad=True)
    t = torch.empty(*shape[:-1], 0, dtype=torch.int64, device=DEV)
    lp, ent, *_ = pkg.token_logprobs(x, t, entropy=entropy)
    assert lp.shape == t.shape
    total = lp.sum() + (ent.sum() if entropy else 0.0)
    got, = torch.autograd.grad(total, x, allow_unused=True)
    if not entropy:  # nothing reaches the logits
        assert got is None or bool((got == 0).all())
        return
    want, = torch.autograd.grad(pkg.token_logprobs(x, entropy=True)[1].sum(), x)
    assert got.shape == x.shape and torch.equal(got, want)


def test_rows_without_lists_and_lists_without_rows():
    for shape in ((0, 40), (0, 3, 40)):
        x = torch.randn(shape, device=DEV, requires_grad=True)
        for t in (torch.empty(shape[:-1], dtype=torch.int64, device=DEV),
                  torch.empty(*shape[:-1], 4, dtype=torch.int64, device=DEV)):
            lp, ent, top, top_lp = pkg.token_logprobs(x, t, top_k=2, entropy=True)
            assert lp.shape == t.shape and top.shape == (*shape[:-1], 2)
            got, = torch.autograd.grad(lp.sum() + ent.sum(), x)
            assert got.shape == x.shape
