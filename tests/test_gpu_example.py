"""The example model: its operators together, in training and in answering."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))


def test_gradients_of_one_step_against_float64():
    import tied_language_model as ex
    V, H, N = 96, 64, 40
    m = ex.TiedModel(V, H, "cuda", dtype=torch.float32, seed=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    tokens = torch.randint(0, V, (2, N // 2), generator=g, device="cuda")
    targets = (3 * tokens + 1) % V
    w, a, n = (p.double().requires_grad_() for p in (m.matrix, m.mix, m.norm))
    loss = m.step(tokens, targets, lr=0.0)
    x = w[tokens] * m.scale
    h = torch.nn.functional.silu(x) @ a + x
    y = h / torch.sqrt((h * h).mean(-1, keepdim=True) + 1e-6) * n
    want = torch.nn.functional.cross_entropy((y @ w.t()).flatten(0, 1), targets.flatten())
    want.backward()
    assert abs(float(loss) - float(want.detach())) <= 2e-3
    # the float32 products of the lm_head and of the mixing layer may run in
    # tensor-float32 (a step of 2^-11 each, several in a row)
    off = (m.grad_matrix.double() - w.grad).norm() / w.grad.norm()
    assert float(off) <= 2.0 ** -7


def test_learns_and_answers_under_a_mask():
    import tied_language_model as ex
    model, losses = ex.train(steps=120)
    assert float(losses[-10:].mean()) < 0.2 * float(losses[0])
    prompt = torch.tensor([[5], [77], [200]], device="cuda")
    plain = model.answer(prompt, 6)
    right = [plain[:, k + 1] == (3 * plain[:, k] + 1) % model.V for k in range(6)]
    assert float(torch.stack(right).float().mean()) > 0.9
    even = torch.full(((model.V + 31) // 32,), 0x55555555, dtype=torch.int32, device="cuda")
    got = model.answer(prompt, 12, mask=even, presence=1e4)[:, 1:]
    assert bool((got % 2 == 0).all())
    assert all(len(set(row)) == 12 for row in got.tolist())  # none twice
