"""A small network trained and served on one GPU with the matrix operators together.

Training, per step: each of N simulated data-parallel ranks runs forward and
backward on its own batch with mx4_linear (all products on MXFP4 operands) and
leaves its bf16 gradient as one contribution row; MuonShardStep sums the rows,
decides on clipping and overflow, moves the weight matrices by their
orthogonalised momentum and the biases by AdamW, and writes the new bf16
parameters that the next forward reads.  Serving: the weights are quantised
once and single rows go through mx4_matmul.

    python examples/muon_mx4.py [--steps 60] [--ranks 4] [--width 256]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import zero_partitioned_mixed_amd as Z  # noqa: E402


def train(steps=60, ranks=4, width=256, batch=128, seed=0, lr=0.01):
    """Returns (losses, the parameters' views, the control block's last record)."""
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    depth = 2  # hidden layers: a stack of equal matrices
    inputs, outputs = 64, 16
    # flat parameter buffer: first matrix, hidden stack, last matrix, then the biases
    shapes = [(1, width, inputs), (depth, width, width), (1, outputs, width)]
    matrices, at = [], 0
    for count, rows, cols in shapes:
        matrices.append((at, count, rows, cols))
        at += count * rows * cols
    biases = at
    psi = at + (depth + 1) * width + outputs
    stride = -(-psi // 64) * 64

    master = torch.zeros(psi, device=dev)
    for start, count, rows, cols in matrices:
        end = start + count * rows * cols
        master[start:end] = torch.randn(end - start, device=dev, generator=gen) * cols ** -0.5
    state = (master, torch.zeros_like(master), torch.zeros_like(master))
    g = torch.empty(psi, device=dev)
    gather = master.to(torch.bfloat16)
    contrib = torch.zeros(ranks, stride, dtype=torch.bfloat16, device=dev)
    step = Z.MuonShardStep(ranks, stride, psi, 0, Z.BF16, Z.BF16, Z.hparams(lr=lr, max_grad_norm=1.0),
                           Z.muon_hparams(lr=lr), matrices, state, g)

    def views(flat):
        w = [flat[s:s + c * r * k].view(c, r, k) for s, c, r, k in matrices]
        b = flat[biases:psi]
        layers = [w[0][0], *w[1], w[2][0]]
        cuts = [width] * (depth + 1) + [outputs]
        return layers, list(b[:sum(cuts)].split(cuts))

    def forward(x, weights, bias):
        for i, (w, b) in enumerate(zip(weights, bias)):
            x = Z.mx4_linear(x, w) + b
            if i < len(weights) - 1:
                x = torch.nn.functional.gelu(x)
        return x

    teacher = torch.randn(inputs, outputs, device=dev, generator=gen) * inputs ** -0.5
    losses = []
    for _ in range(steps):
        total = 0.0
        for rank in range(ranks):
            x = torch.randn(batch, inputs, device=dev, generator=gen)
            y = torch.tanh(x @ teacher)
            leaf = gather.detach().clone().requires_grad_()
            loss = (forward(x.bfloat16(), *views(leaf)).float() - y).square().mean()
            contrib[rank, :psi] = torch.autograd.grad(loss, leaf)[0]
            total += loss.detach()
        losses.append(total / ranks)
        step.step(contrib, gather)
    return [float(v) for v in losses], views(gather), step.ctrl_dict()


def serve(weights, bias, rows):
    """Rows through the network with its weights quantised once."""
    packed = [Z.mx4_quantize(w) for w in weights]
    out = []
    for x in rows:
        x = x[None].bfloat16()
        for i, (w, b) in enumerate(zip(packed, bias)):
            x = Z.mx4_matmul(x, w) + b
            if i < len(packed) - 1:
                x = torch.nn.functional.gelu(x)
        out.append(x)
    return torch.cat(out)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--ranks", type=int, default=4)
    ap.add_argument("--width", type=int, default=256)
    a = ap.parse_args()
    losses, (weights, bias), ctrl = train(a.steps, a.ranks, a.width)
    for i in range(0, a.steps, max(1, a.steps // 10)):
        print(f"step {i:4d}  loss {losses[i]:.5f}")
    print(f"step {a.steps - 1:4d}  loss {losses[-1]:.5f}  ({ctrl['t']} steps applied, last norm {ctrl['norm']:.4f})")
    out = serve(weights, bias, torch.randn(3, 64, device="cuda"))
    print("three rows served:", [round(float(v), 3) for v in out[:, 0]])


if __name__ == "__main__":
    main()
