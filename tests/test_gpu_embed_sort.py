"""The embedding gradient by sorted tokens (more than 1024 of them, or few but
wide): its digits, its vector widths, and what the few-token kernel otherwise
takes at small sizes.  Bounds as in test_gpu_embed.py."""
import pytest
import torch

import vocabulary_cross_entropy_pass_gb300 as pkg

from .test_gpu_embed import DEV, TYPES, check_bwd, rng, run_bwd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N", [1500, 9000])  # one CTA's run of tokens, several CTAs
@pytest.mark.parametrize("V", [1, 2, 511, 512, (1 << 18) - 1, 1 << 18, (1 << 20) + 3])
def test_digits(V, N):
    # keys 0 to V: one digit of up to nine bits, two, three
    t = torch.randint(0, V, (N,), generator=rng(V + N))
    t[5], t[N - 1] = V - 1, 0
    run_bwd(N, V, 2, torch.float32, t)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("H", [1, 2, 66, 129, 256, 1030])
def test_vector_widths(H, dtype):
    # 16 bytes, 4 bytes (even widths off the grid in 16 bits), one element
    V = 333
    t = torch.randint(0, V, (2000,), generator=rng(H))
    t[torch.rand(2000, generator=rng(H + 1)) < 0.2] = 17
    run_bwd(2000, V, H, dtype, t, scale=2.0)


@pytest.mark.parametrize("N", [1500, 9000, 70001])
def test_ignored_and_out_of_range(N):
    g = rng(N)
    V, H = 300, 24
    go = torch.randn(N, H, generator=g)
    t = torch.randint(0, V, (N,), generator=g)
    t[::7] = -100
    t[3], t[N // 2], t[N - 1] = V, -1, 1 << 40
    ws = torch.full((pkg.ce_embed_bwd_workspace_bytes(N, H, V),), 255, dtype=torch.uint8, device=DEV)
    got = pkg.ce_embed_bwd(go.to(DEV), t.to(DEV), V, workspace=ws)
    check_bwd(got, go, t, V, 1.0)
    assert pkg.ce_get_error(ws) == (6, 1)
    base = torch.randn(V, H, generator=g)
    acc = base.to(DEV)
    pkg.ce_embed_bwd(go.to(DEV), t.to(DEV), V, workspace=ws, grad_weight=acc, accumulate=True)
    check_bwd(acc, go, t, V, 1.0, base=base)
    assert pkg.ce_get_error(ws) == (6, 1)
    t[3] = t[N // 2] = t[N - 1] = -100
    check_bwd(pkg.ce_embed_bwd(go.to(DEV), t.to(DEV), V, workspace=ws), go, t, V, 1.0)
    assert pkg.ce_get_error(ws) == (0, 0)
    t[:] = -100
    assert bool((pkg.ce_embed_bwd(go.to(DEV), t.to(DEV), V) == 0).all())
    t[:] = 4  # the ignored value comes first, also inside the vocabulary
    t[1::2] = 5
    check_bwd(pkg.ce_embed_bwd(go.to(DEV), t.to(DEV), V, ignore_idx=4), go, t, V, 1.0, ignore=4)


@pytest.mark.parametrize("dtype", TYPES)
def test_strides(dtype):
    g = rng(23)
    V, A, B = 700, 50, 61
    wide = torch.randn(A, B, 90, generator=g).to(dtype).to(DEV)
    t = torch.randint(0, V, (B, A), generator=g).to(DEV).t()  # does not lie flat
    for go in (wide[:, :, :64], wide[:, :, 1:66], wide[:, :, 2:88]):
        H = go.shape[-1]
        check_bwd(pkg.ce_embed_bwd(go, t, V), go.cpu(), t.cpu(), V, 1.0)
        for at, width in ((0, H), (0, H + 2), (3, H + 7), (4, H + 8)):
            # written whole between columns that are not its own, then added to
            big = torch.full((V, width), 5.0, device=DEV)
            own = torch.zeros(width, dtype=torch.bool)
            own[at:at + H] = True
            part = big[:, at:at + H] if at + H <= width else None
            if part is None:
                continue
            pkg.ce_embed_bwd(go, t, V, grad_weight=part)
            check_bwd(part, go.cpu(), t.cpu(), V, 1.0)
            assert bool((big[:, (~own).to(DEV)] == 5).all())
            base = part.cpu().clone()
            pkg.ce_embed_bwd(go, t, V, scale=0.5, grad_weight=part, accumulate=True)
            check_bwd(part, go.cpu(), t.cpu(), V, 0.5, base=base)
            assert bool((big[:, (~own).to(DEV)] == 5).all())
            if dtype != torch.float32:
                low = torch.full((V, width), 5.0, dtype=dtype, device=DEV)
                pkg.ce_embed_bwd(go, t, V, grad_weight=low[:, at:at + H])
                check_bwd(low[:, at:at + H], go.cpu(), t.cpu(), V, 1.0)
                assert bool((low[:, (~own).to(DEV)] == 5).all())
    # tokens with a stride of their own, and one gradient row for all of them
    spaced = torch.randint(0, V, (3 * A * B,), generator=g).to(DEV)[::3]
    rows = wide.view(A * B, 90)[:, :64]
    check_bwd(pkg.ce_embed_bwd(rows, spaced, V), rows.cpu(), spaced.cpu(), V, 1.0)
    one = rows[:1].expand(A * B, 64)
    check_bwd(pkg.ce_embed_bwd(one, spaced, V), one.cpu(), spaced.cpu(), V, 1.0)
    assert bool((pkg.ce_embed_bwd(rows, spaced[:1].expand(A * B), V).count_nonzero(dim=1) > 0).sum() == 1)


def test_gradient_past_32_bits():
    # a gradient of 2.5e9 elements, written whole and added to
    V, H, N = 305000, 8192, 1100
    t = torch.randint(0, V, (N,), generator=rng(24))
    t[:6] = torch.tensor([0, V - 1, V - 2, 262144, 300001, V - 1])
    td = t.to(DEV)
    go = torch.randn(N, H, generator=rng(25)).to(torch.bfloat16)
    dw = torch.empty(V, H, dtype=torch.float32, device=DEV).fill_(3.0)
    pkg.ce_embed_bwd(go.to(DEV), td, V, grad_weight=dw)
    ids = t.unique()
    check_bwd(dw[ids.to(DEV)], go, torch.searchsorted(ids, t), len(ids), 1.0)
    assert int((dw[::997] != 0).any(1).sum()) == int((ids % 997 == 0).sum())
    base = dw[ids.to(DEV)].cpu()
    pkg.ce_embed_bwd(go.to(DEV), td, V, scale=2.0, grad_weight=dw, accumulate=True)
    check_bwd(dw[ids.to(DEV)], go, torch.searchsorted(ids, t), len(ids), 2.0, base=base)


def test_rows_past_32_bits():
    # 300000 gradient rows of 8192: offsets of the rows that are summed pass 32 bits
    V, H, N = 5000, 8192, 300000
    t = torch.randint(0, V, (N,), generator=rng(26))
    go = torch.empty(N, H, dtype=torch.bfloat16, device=DEV)
    go.copy_(((torch.arange(N, device=DEV) % 61 - 30).to(torch.bfloat16))[:, None])
    dw = pkg.ce_embed_bwd(go, t.to(DEV), V)
    want = torch.zeros(V, dtype=torch.float64).index_add_(0, t, (torch.arange(N) % 61 - 30).double())
    assert torch.equal(dw[:, 0].double().cpu(), want)  # whole numbers: float32 sums are exact
    assert bool((dw == dw[:, :1]).all())
