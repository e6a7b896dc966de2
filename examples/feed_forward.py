"""A gated feed-forward block, trained in bf16 and served from 8-bit integers.

    y = (silu(x Wg^T) * (x Wu^T)) Wd^T

Training runs gemm_glu (which keeps the two pre-activations) and
gemm_glu_bwd; the down projection and its gradient go through grouped_gemm
with one group.  Serving quantises the trained weights once, a row at a time,
and then runs quant_i8 -> gemm_glu_i8 -> quant_i8 -> gemm_i8 for any number of
tokens.

    python examples/feed_forward.py [--tokens 512] [--model 1024] [--hidden 2816] [--steps 20]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_gemm_02_amd as bsg  # noqa: E402

DEV, BF = "cuda", torch.bfloat16


class GatedFeedForward:
    """The block's bf16 weights, its gradients and the scratch it keeps."""

    def __init__(self, d_model, d_hidden, act="silu", seed=0):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.d, self.n, self.act = d_model, d_hidden, act

        def init(rows, cols):
            return (torch.randn(rows, cols, generator=g, device=DEV) * cols ** -0.5).to(BF)

        self.w_gate, self.w_up, self.w_down = init(d_hidden, d_model), init(d_hidden, d_model), init(d_model, d_hidden)
        self.scratch = {}

    def _workspace(self, op, m, n, k):
        need = bsg.workspace_bytes(op, m, n, k)
        if self.scratch.get(op) is None or self.scratch[op].numel() < need:
            self.scratch[op] = torch.empty(need, dtype=torch.uint8, device=DEV)
        return self.scratch[op]

    def _product(self, a, b, m, n, k):
        """a (m, k) b (n, k)^T through the grouped product with one group (m % 256 == 0)."""
        out = torch.empty(m, n, dtype=BF, device=DEV)
        ends = torch.tensor([m], dtype=torch.int32, device=DEV)
        bsg.grouped_gemm(a, b, ends, torch.ones(1, device=DEV), torch.ones(m, device=DEV), None, None, out, m, n, k, 1)
        return out

    def forward(self, x):
        """y and what the backward pass needs."""
        m = x.shape[0]
        h, g, u = (torch.empty(m, self.n, dtype=BF, device=DEV) for _ in range(3))
        bsg.gemm_glu(x, self.w_gate, self.w_up, h, g, u, m, self.n, self.d, act=self.act,
                     workspace=self._workspace("gemm_glu", m, self.n, self.d))
        return self._product(h, self.w_down, m, self.d, self.n), (x, h, g, u)

    def backward(self, dy, saved):
        """Gradients of x, w_gate, w_up and w_down."""
        x, h, g, u = saved
        m = x.shape[0]
        dh = self._product(dy, self.w_down.t().contiguous(), m, self.n, self.d)
        dx, dwg, dwu = torch.empty_like(x), torch.empty_like(self.w_gate), torch.empty_like(self.w_up)
        bsg.gemm_glu_bwd(dh, x, self.w_gate, self.w_up, g, u, dx, dwg, dwu, m, self.n, self.d, act=self.act,
                         workspace=self._workspace("gemm_glu_bwd", m, self.n, self.d))
        return dx, dwg, dwu, (dy.float().t() @ h.float()).to(BF)


class Int8FeedForward:
    """The same block from 8-bit weights: one scale a channel, and a token's
    scale found as it comes."""

    def __init__(self, block: GatedFeedForward):
        self.d, self.n, self.act = block.d, block.n, block.act
        self.gate, self.up, self.down = (self._quantise(w) for w in (block.w_gate, block.w_up, block.w_down))
        self.scratch = {}

    @staticmethod
    def _quantise(w):
        m, k = w.shape
        q, s = torch.empty(m, k, dtype=torch.int8, device=DEV), torch.empty(m, device=DEV)
        bsg.quant_i8(w, q, s, m, k)
        return q, s

    _workspace = GatedFeedForward._workspace

    def __call__(self, x):
        m = x.shape[0]
        h, y = torch.empty(m, self.n, dtype=BF, device=DEV), torch.empty(m, self.d, dtype=BF, device=DEV)
        a, sa = self._quantise(x)
        bsg.gemm_glu_i8(a, self.gate[0], self.up[0], sa, self.gate[1], self.up[1], h, m, self.n, self.d, act=self.act,
                        workspace=self._workspace("gemm_glu_i8", m, self.n, self.d))
        a, sa = self._quantise(h)
        bsg.gemm_i8(a, self.down[0], sa, self.down[1], None, y, m, self.d, self.n,
                    workspace=self._workspace("gemm_i8", m, self.d, self.n))
        return y


def train(block, tokens, steps, lr=0.03, seed=1):
    """Fits the block to another one of its kind by plain gradient descent;
    returns the mean squared error of every step."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    teacher = GatedFeedForward(block.d, block.n, block.act, seed=seed + 100)
    x = torch.randn(tokens, block.d, generator=g, device=DEV).to(BF)
    target = teacher.forward(x)[0].float()
    losses = []
    for _ in range(steps):
        y, saved = block.forward(x)
        diff = y.float() - target
        losses.append(float(diff.square().mean()))
        _, dwg, dwu, dwd = block.backward((diff * (2.0 / tokens)).to(BF), saved)
        for w, dw in ((block.w_gate, dwg), (block.w_up, dwu), (block.w_down, dwd)):
            w.sub_((lr * dw.float()).to(BF))
    return losses


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--tokens", type=int, default=512, help="tokens of the training batch (a multiple of 256)")
    p.add_argument("--model", type=int, default=1024)
    p.add_argument("--hidden", type=int, default=2816)
    p.add_argument("--steps", type=int, default=20)
    a = p.parse_args(argv)
    block = GatedFeedForward(a.model, a.hidden)
    losses = train(block, a.tokens, a.steps)
    print(f"training: mean squared error {losses[0]:.4f} -> {losses[-1]:.4f} in {a.steps} steps", flush=True)
    served = Int8FeedForward(block)
    errors = {}
    for m in (1, 7, 64, a.tokens):
        x = torch.randn(m, a.model, generator=torch.Generator(device=DEV).manual_seed(m), device=DEV).to(BF)
        pad = torch.zeros(-(-m // 256) * 256, a.model, dtype=BF, device=DEV)
        pad[:m] = x
        want = block.forward(pad)[0][:m].float()
        got = served(x).float()
        errors[m] = float((got - want).norm() / want.norm())
        print(f"serving {m:4d} tokens from 8-bit integers: {100 * errors[m]:.2f}% from the bf16 block", flush=True)
    return losses, errors


if __name__ == "__main__":
    main()
