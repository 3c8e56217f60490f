"""Many rows that are cut for their width: over 16384 vectors a row's groups' maxima have no room in one piece
(float32 beyond 65536 columns, 16 bits beyond 131072), so every row is put together from segments however many
there are."""
import pytest
import torch

import vocabulary_cross_entropy_pass_gb300 as pkg

from .test_gpu_logprobs import DEV, LOWEST, NEG, check_forward, rng

pytestmark = pytest.mark.gpu


def rows(N, V, dtype):
    """Random rows; among them equal logits across the borders of the segments, and masks."""
    g = rng(V)
    x = torch.randn(N, V, generator=g, device=DEV) * 3
    half = V // 2
    x[0] = 1.5                                    # all equal
    x[1, half - 300:half + 300] = 40.0            # the likeliest on both sides of a border, equal
    x[2] = torch.arange(V, device=DEV) / 4096.0   # rising: all in the last segment
    x[3] = -x[2]
    x[4] = NEG                                    # nothing
    x[5] = NEG
    x[5, V - 1] = 0.0                             # one token, the last
    x[6, :half + 1000] = NEG                      # a segment without any
    x[7] = float(LOWEST[dtype])
    x[7, ::V // 7] = 2.0
    x[8] = torch.randint(0, 3, (V,), generator=g, device=DEV).float()
    x[9, half:] = 30.0                            # many equal ones behind a border
    return x.to(dtype)


@pytest.mark.parametrize("top", [20, 64, 200])
@pytest.mark.parametrize("dtype,N,V", [(torch.float32, 400, 70001), (torch.float32, 700, 65544),
                                       (torch.bfloat16, 400, 140001), (torch.float16, 330, 131080)])
def test_many_rows_in_segments(dtype, N, V, top):
    x = rows(N, V, dtype)
    t = torch.randint(0, V, (N, 3), generator=rng(1), device=DEV)
    t[::11] = -100
    t[5::11, 0] = -100
    check_forward(x, t, top_k=top)
    check_forward(x, t[:, 1].contiguous(), top_k=top, entropy=False)
    check_forward(x, None, top_k=top, entropy=False)


def test_long_lists_of_given_tokens():
    N, V = 330, 65600
    x = rows(N, V, torch.float32)
    t = torch.randint(0, V, (N, 1024), generator=rng(2), device=DEV)
    t[:, 5::9] = -100
    t[17] = -100
    t[18, 1000] = V
    t[19, 31:33] = -1
    for top in (0, 20):
        ws = torch.empty(pkg.ce_logprobs_workspace_bytes(N, V, x.dtype, top), dtype=torch.uint8, device=DEV)
        check_forward(x, t, top_k=top, workspace=ws)
        assert pkg.ce_get_error(ws) == (6, 1)
