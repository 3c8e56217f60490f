"""A small language model whose embedding and lm_head are one matrix, trained and
then asked, on the operators around the cross-entropy pass.

    python examples/tied_language_model.py [--steps 120]

Training: rows of the matrix by token (ce_embed_fwd), one mixing layer in
torch, residual + norm (rms_norm), lm_head + loss without the full logits
(ce_linear_fwd_bwd).  The matrix's gradient is one float32 buffer: the lm_head
step adds to it, then the embedding's gradient does (ce_embed_bwd with
accumulate).  Answering: the same steps for the last token, then the logits'
penalties and a grammar mask (ce_logits_process) before the largest is taken.

The task is synthetic: the next token is (3 t + 1) mod V.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import vocabulary_cross_entropy_pass_gb300 as ce  # noqa: E402


class TiedModel:
    def __init__(self, V: int, H: int, device, dtype=torch.bfloat16, seed: int = 0):
        g = torch.Generator(device=device).manual_seed(seed)
        self.V, self.H, self.dtype, self.scale = V, H, dtype, float(H) ** 0.5
        # float32 masters; the operators take copies of the storage type
        self.matrix = torch.randn(V, H, generator=g, device=device) * (0.5 / H ** 0.5)
        self.mix = torch.randn(H, H, generator=g, device=device) * (0.5 / H ** 0.5)
        self.norm = torch.ones(H, device=device)
        self.grad_matrix = torch.zeros(V, H, device=device)
        self.moments = [[torch.zeros_like(p), torch.zeros_like(p)] for p in (self.matrix, self.mix, self.norm)]
        self.t = 0

    def hidden(self, tokens, table, mix, norm):
        """(input rows, normed rows) of a batch of tokens."""
        x = ce.ce_embed_fwd(tokens, table, scale=self.scale).requires_grad_()
        y, _ = ce.rms_norm(torch.nn.functional.silu(x) @ mix, norm, residual=x)
        return x, y

    def step(self, tokens, targets, lr: float) -> torch.Tensor:
        """One training step; returns the mean loss (on the GPU)."""
        table = self.matrix.to(self.dtype)
        mix = self.mix.to(self.dtype, copy=True).requires_grad_()
        norm = self.norm.clone().requires_grad_()
        x, y = self.hidden(tokens, table, mix, norm)
        self.grad_matrix.zero_()
        loss, grad_y, _ = ce.ce_linear_fwd_bwd(y.detach().flatten(0, 1), table, targets.flatten(), reduce_loss=True,
                                               grad_weight=self.grad_matrix)
        y.backward(grad_y.view_as(y))
        ce.ce_embed_bwd(x.grad, tokens, self.V, scale=self.scale, grad_weight=self.grad_matrix, accumulate=True)
        self.t += 1
        for p, g, (m, v) in zip((self.matrix, self.mix, self.norm), (self.grad_matrix, mix.grad.float(), norm.grad),
                                self.moments):
            m.lerp_(g, 0.1)
            v.lerp_(g * g, 0.01)
            p -= lr * (m / (1 - 0.9 ** self.t)) / ((v / (1 - 0.99 ** self.t)).sqrt() + 1e-8)
        return loss

    @torch.no_grad()
    def answer(self, prompt: torch.Tensor, count: int, mask=None, repetition: float = 1.0, presence: float = 0.0):
        """``count`` more tokens after each row of ``prompt`` (N, L), the most likely
        one each time, under the penalties and the mask of allowed tokens."""
        N, L = prompt.shape
        dev = prompt.device
        table, mix = self.matrix.to(self.dtype), self.mix.to(self.dtype)
        history = torch.zeros(N, L + count, dtype=torch.int64, device=dev)
        history[:, :L] = prompt
        lengths = torch.full((N,), L, dtype=torch.int64, device=dev)
        params = dict(history=history, prompt_lengths=lengths.clone(), mask=mask,
                      repetition_penalty=torch.full((N,), repetition, device=dev),
                      presence_penalty=torch.full((N,), presence, device=dev),
                      temperature=torch.ones(N, device=dev))
        for k in range(L, L + count):
            x = ce.ce_embed_fwd(history[:, k - 1], table, scale=self.scale)
            y, _, _ = ce.ce_rmsnorm_fwd(torch.nn.functional.silu(x) @ mix, self.norm, residual=x)
            logits = y @ table.t()
            ce.ce_logits_process(logits, out=logits, history_lengths=lengths, **params)
            history[:, k] = logits.argmax(-1)
            lengths += 1
        return history


def train(steps: int = 120, V: int = 256, H: int = 128, batch: int = 8, length: int = 64, device="cuda", seed: int = 0):
    """(model, losses) after ``steps`` on random batches."""
    g = torch.Generator(device=device).manual_seed(seed + 1)
    model = TiedModel(V, H, device, seed=seed)
    losses = []
    for _ in range(steps):
        tokens = torch.randint(0, V, (batch, length), generator=g, device=device)
        losses.append(model.step(tokens, (3 * tokens + 1) % V, lr=2e-2))
    return model, torch.cat(losses)


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=120)
    args = ap.parse_args()
    model, losses = train(args.steps)
    print(f"loss {float(losses[0]):.3f} -> {float(losses[-1]):.3f} after {len(losses)} steps")
    prompt = torch.tensor([[5], [77]], device="cuda")
    print("answer:", model.answer(prompt, 8).tolist())
    words = (model.V + 31) // 32
    even = torch.full((words,), 0x55555555, dtype=torch.int32, device="cuda")
    print("even tokens only, none twice:", model.answer(prompt, 8, mask=even, presence=1e4).tolist())


if __name__ == "__main__":
    main()
