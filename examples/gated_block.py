"""A gated feed-forward block trained and then served with 4-bit weights.

    python examples/gated_block.py

Y = (SiLU(X Wg) * (X Wu)) Wd with BF16 weights learns a fixed random block: the
forward pass keeps G and U, the backward pass gives dX and the weights'
gradients, accumulated over two micro-batches (beta = 1).  The trained gate and
up weights are then quantised to MX4 once and a batch of tokens goes through
the 4-bit gated pair.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dense_gemm_mgemm_amd as mg  # noqa: E402

TOKENS, WIDTH, HIDDEN = 256, 256, 512


def weights(gen):
    shapes = ((WIDTH, HIDDEN), (WIDTH, HIDDEN), (HIDDEN, WIDTH))
    return [torch.randn(*s, generator=gen, device="cuda") / s[0] ** 0.5 for s in shapes]


class Block:
    def __init__(self, h, masters):
        self.h = h
        self.master = masters                                   # FP32, what the optimiser steps
        self.wg, self.wu, self.wd = (w.bfloat16() for w in masters)
        self.grads = [torch.zeros_like(w) for w in (self.wg, self.wu, self.wd)]
        new = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        self.z, self.g, self.u, self.dz = (new(TOKENS, HIDDEN) for _ in range(4))
        self.y, self.dx = new(TOKENS, WIDTH), new(TOKENS, WIDTH)
        x = self.dx
        sizes = [mg.mgemm_gated_workspace("row", TOKENS, HIDDEN, WIDTH, x, WIDTH, self.wg, self.wu, HIDDEN, "bf16", b,
                                          True) for b in (False, True)]
        self.work = torch.empty(max(sizes), dtype=torch.uint8, device="cuda")

    def forward(self, x):
        mg.mgemm_gated_forward(self.h, "row", TOKENS, HIDDEN, WIDTH, x, WIDTH, self.wg, self.wu, HIDDEN, self.z, HIDDEN,
                               self.g, self.u, HIDDEN, "bf16", self.work, self.work.numel())
        mg.mgemm_run(self.h, "row", "row", TOKENS, WIDTH, HIDDEN, 1.0, self.z, HIDDEN, self.wd, WIDTH, 0.0, self.y,
                     WIDTH, "bf16")
        return self.y

    def backward(self, x, dy, first):
        """Gradients of one micro-batch, added to those of the batch's earlier ones."""
        beta = 0.0 if first else 1.0
        dwg, dwu, dwd = self.grads
        # dWd = Z^T dY as the column-major product of Z stored M x N, and dZ = dY Wd^T.
        mg.mgemm_run(self.h, "col", "row", HIDDEN, WIDTH, TOKENS, 1.0, self.z, HIDDEN, dy, WIDTH, 0.0,
                     self._dwd_t(), HIDDEN, "bf16")
        dwd.mul_(beta).add_(self._dwd_t().t())
        mg.mgemm_run(self.h, "row", "col", TOKENS, HIDDEN, WIDTH, 1.0, dy, WIDTH, self.wd, WIDTH, 0.0, self.dz, HIDDEN,
                     "bf16")
        mg.mgemm_gated_backward(self.h, "row", TOKENS, HIDDEN, WIDTH, x, WIDTH, self.wg, self.wu, HIDDEN, self.g,
                                self.u, HIDDEN, self.dz, HIDDEN, self.dx, WIDTH, dwg, dwu, HIDDEN, beta, "bf16",
                                self.work, self.work.numel())

    def _dwd_t(self):
        if not hasattr(self, "_t"):
            self._t = torch.empty(WIDTH, HIDDEN, dtype=torch.bfloat16, device="cuda")
        return self._t

    def step(self, lr):
        for m, w, d in zip(self.master, (self.wg, self.wu, self.wd), self.grads):
            m.sub_(d.float(), alpha=lr)
            w.copy_(m)


def mx4(h, w):
    """Codes and scales of w^T (out x in)."""
    out = w.t().contiguous()
    rows, k = out.shape
    codes = torch.empty(rows, k // 2, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(rows, (k // 32 + 15) // 16 * 16, dtype=torch.uint8, device="cuda")
    mg.mgemm_quantize_mx4(h, rows, k, out, k, "bf16", codes, k // 2, scales, scales.stride(0))
    return codes, scales


def main(steps=40):
    gen = torch.Generator(device="cuda").manual_seed(1)
    h = mg.mgemm_create()
    try:
        target, block = Block(h, weights(gen)), Block(h, weights(gen))
        losses = []
        for _ in range(steps):
            loss = 0.0
            for micro in range(2):
                x = torch.randn(TOKENS, WIDTH, generator=gen, device="cuda").bfloat16()
                want = target.forward(x).clone()
                diff = block.forward(x).float() - want.float()
                loss += diff.square().mean() / 2
                block.backward(x, (diff / TOKENS).bfloat16(), micro == 0)
            block.step(0.5)
            losses.append(loss.item())
        # Served: eight tokens through the 4-bit gated pair.
        x = torch.randn(8, WIDTH, generator=gen, device="cuda").bfloat16()
        z4, z = (torch.empty(8, HIDDEN, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        (qg, sg), (qu, su) = mx4(h, block.wg), mx4(h, block.wu)
        mg.mgemm_gated_mx4(h, 8, HIDDEN, WIDTH, x, WIDTH, "bf16", qg, sg, qu, su, qg.stride(0), sg.stride(0), z4, HIDDEN,
                           "bf16")
        mg.mgemm_run_gated(h, 8, HIDDEN, WIDTH, x, WIDTH, block.wg, block.wu, HIDDEN, z, HIDDEN, "bf16")
        off = ((z4.float() - z.float()).norm() / z.float().norm()).item()
        torch.cuda.synchronize()
        print("loss %.4f -> %.4f; 4-bit gated pair off by %.1f%% of the BF16 one's norm" %
              (losses[0], losses[-1], 100 * off), flush=True)
        return losses, off
    finally:
        mg.mgemm_destroy(h)


if __name__ == "__main__":
    main()
