"""The 4-bit operators as a training step and a decoding loop use them.

train   a linear layer learns a random teacher's outputs: forward, input
        gradient and weight gradient are 4-bit products, activations and
        weights rounded to nearest, output gradients stochastically.
serve   a mixture of experts with 4-bit weights takes one token at a time,
        its call captured once into a HIP graph.

Run on an MI355X: python examples/mx4_train_and_serve.py
"""
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_scaled_matmul_amd as fm      # noqa: E402


class Linear4(torch.autograd.Function):
    """y = x w^T of 4-bit operands.  Each tensor is read once for both of the
    copies that the three products need."""

    @staticmethod
    def forward(ctx, x, w, seed):
        xq, xqt = fm.mx4_quantize(x, want_t=True)
        wq, wqt = fm.mx4_quantize(w, want_t=True)
        ctx.held, ctx.seed = (xqt, wqt), seed
        return fm.mx4_mm(xq, wq)

    @staticmethod
    def backward(ctx, dy):
        xqt, wqt = ctx.held
        dq, dqt = fm.mx4_quantize(dy.contiguous(), want_t=True, seed=ctx.seed)
        return fm.mx4_mm(dq, wqt), fm.mx4_mm(dqt, xqt), None


def train(tokens=4096, hidden=1024, out=2048, steps=40, lr=0.5):
    """Losses, first to last."""
    torch.manual_seed(0)
    teacher = torch.randn(out, hidden, device="cuda") * hidden ** -0.5
    master = torch.zeros(out, hidden, device="cuda", requires_grad=True)
    seed = torch.zeros(1, dtype=torch.int64, device="cuda")
    losses = []
    for step in range(steps):
        x = torch.randn(tokens, hidden, device="cuda").bfloat16()
        seed.fill_(step)        # new bits for every step's gradients
        y = Linear4.apply(x, master, seed)
        loss = (y.float() - x.float() @ teacher.t()).square().mean()
        loss.backward()
        with torch.no_grad():
            master -= lr * 0.5 * out * master.grad.float()      # the loss is a mean over tokens and outputs
            master.grad = None
        losses.append(loss.item())
    return losses


def _experts(count, rows, cols):
    # one call for all of them, and views of what it gives
    held, _ = fm.mx4_quantize(torch.randn(count * rows, cols, device="cuda") * cols ** -0.5)
    return fm.Mx4(held.q.view(count, rows, -1), held.s.view(-1, count, rows, 16).transpose(0, 1), cols)


def serve(experts=16, top_k=2, hidden=1024, inner=704, tokens=200):
    """Microseconds a token, and the last token's output."""
    torch.manual_seed(1)
    router = (torch.randn(experts, hidden, device="cuda") * hidden ** -0.5).bfloat16()
    layer = fm.MoeMx4(router, _experts(experts, 2 * inner, hidden), _experts(experts, hidden, inner), top_k, max_tokens=1)
    x = torch.randn(1, hidden, device="cuda").bfloat16()
    layer(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, ids, weights = layer(x)
    graph.replay()          # capturing ran nothing: y is there from now on
    torch.cuda.synchronize()
    start = time.perf_counter()
    for _ in range(tokens):
        x.copy_(torch.nn.functional.rms_norm(x + y, (hidden,)))     # the next layer's input
        graph.replay()
    torch.cuda.synchronize()
    return (time.perf_counter() - start) / tokens * 1e6, y


if __name__ == "__main__":
    losses = train()
    print(f"train: loss {losses[0]:.4f} -> {losses[-1]:.4f} in {len(losses)} steps")
    us, y = serve()
    print(f"serve: {us:.1f} us a token, |y| {y.float().norm().item():.3f}")
