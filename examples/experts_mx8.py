"""A small next-token model trained and served on one GPU with the operators on rows of tokens.

The model: an embedding lookup, layers of (norm with the residual's addition, a router's two of
several experts for each token, dropout), a last norm and a projection.  Training, per step:
each of N simulated data-parallel ranks runs forward and backward on its own batch and leaves its
bf16 gradient as one contribution row; MuonShardStep sums the rows, decides on clipping and
overflow, moves the experts' matrices by their orthogonalised momentum and everything else by
AdamW, and writes the new bf16 parameters that the next forward reads.  Serving: the
weights are quantised to MXFP4 once; the norms leave MXFP8 rows for their products.

    python examples/experts_mx8.py [--steps 60] [--ranks 2] [--width 128]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import zero_partitioned_mixed_amd as Z  # noqa: E402

VOCAB, EXPERTS, CHOICES, LAYERS = 96, 4, 2, 2


def layout(width):
    """{name: (first element, shape)} of the flat parameter buffer, and its length."""
    parts = [("experts in", (LAYERS * EXPERTS, 2 * width, width)), ("experts out", (LAYERS * EXPERTS, width, 2 * width)),
             ("table", (VOCAB, width)), ("project", (VOCAB, width)), ("routers", (LAYERS, EXPERTS, width)), ("norms", (LAYERS + 1, width))]
    at, places = 0, {}
    for name, shape in parts:
        places[name] = (at, shape)
        at += torch.Size(shape).numel()
    return places, at


def views(flat, places):
    return {name: flat[at:at + torch.Size(shape).numel()].view(shape) for name, (at, shape) in places.items()}


def experts(y, p, layer):
    """The layer of experts on rows y: each token's two, weighted."""
    weights, chosen = torch.softmax(y.float() @ p["routers"][layer].float().t(), 1).topk(CHOICES, 1)
    plan = Z.expert_sort(chosen, EXPERTS)
    rows, out = Z.expert_rows(y, plan), []
    ends = plan.offsets.tolist()  # the products' sizes
    for e, (a, b) in enumerate(zip(ends, ends[1:])):
        if b > a:
            i = layer * EXPERTS + e
            out.append(Z.mx4_linear(torch.nn.functional.gelu(Z.mx4_linear(rows[a:b], p["experts in"][i])), p["experts out"][i]))
    return Z.expert_combine(torch.cat(out), weights, plan)


def forward(ids, p, drop=0.0, seed=0, offset=0):
    """The logits of every token in ids [tokens]."""
    h = Z.embedding(ids, p["table"])
    y = Z.rms_norm(h, p["norms"][0])
    for layer in range(LAYERS):
        # the layer's result, some of it dropped, goes into the stream with the next norm
        x = Z.dropout(experts(y, p, layer), drop, seed, offset * LAYERS + layer)
        y, h = Z.rms_norm(x, p["norms"][layer + 1], h)
    return Z.mx4_linear(y, p["project"])


def batch(gen, tokens):
    """Tokens of a sequence whose next one is mostly a fixed function of the last."""
    ids = torch.empty(tokens + 1, dtype=torch.int64)
    ids[0] = torch.randint(0, VOCAB, (1,), generator=gen)
    noise = torch.randint(0, VOCAB, (tokens + 1,), generator=gen)
    fresh = torch.rand(tokens + 1, generator=gen) < 0.1
    for i in range(1, tokens + 1):
        ids[i] = noise[i] if fresh[i] else (3 * ids[i - 1] + 1) % VOCAB
    ids = ids.cuda()
    return ids[:-1], ids[1:]


def train(steps=60, ranks=2, width=128, tokens=256, seed=0, lr=0.01):
    """Returns (losses, the parameters' views, the control block's last record)."""
    dev = torch.device("cuda")
    gen, host = torch.Generator(device=dev).manual_seed(seed), torch.Generator().manual_seed(seed)
    places, psi = layout(width)
    stride = -(-psi // 64) * 64
    master = torch.randn(psi, device=dev, generator=gen) * width ** -0.5
    views(master, places)["norms"].fill_(1.0)
    state = (master, torch.zeros_like(master), torch.zeros_like(master))
    matrices = [(at, *shape) for name, (at, shape) in places.items() if name.startswith("experts")]
    gather = master.to(torch.bfloat16)
    contrib = torch.zeros(ranks, stride, dtype=torch.bfloat16, device=dev)
    step = Z.MuonShardStep(ranks, stride, psi, 0, Z.BF16, Z.BF16, Z.hparams(lr=lr, max_grad_norm=1.0), Z.muon_hparams(lr=lr),
                           matrices, state, torch.empty(psi, device=dev))
    losses = []
    for i in range(steps):
        total = 0.0
        for rank in range(ranks):
            ids, following = batch(host, tokens)
            leaf = gather.detach().clone().requires_grad_()
            logits = forward(ids, views(leaf, places), drop=0.05, seed=seed, offset=i * ranks + rank)
            loss = torch.nn.functional.cross_entropy(logits.float(), following)
            contrib[rank, :psi] = torch.autograd.grad(loss, leaf)[0]
            total += loss.detach()
        losses.append(total / ranks)
        step.step(contrib, gather)
    return [float(v) for v in losses], views(gather, places), step.ctrl_dict()


@torch.no_grad()
def serve(p, ids):
    """The logits of ids with 4-bit weights and 8-bit rows into the last projection and the experts."""
    packed = {name: [Z.mx4_quantize(w) for w in p[name]] for name in ("experts in", "experts out")}
    project = Z.mx4_quantize(p["project"])
    h = Z.embedding(ids, p["table"])
    y = Z.rms_norm(h, p["norms"][0])
    for layer in range(LAYERS):
        weights, chosen = torch.softmax(y.float() @ p["routers"][layer].float().t(), 1).topk(CHOICES, 1)
        plan = Z.expert_sort(chosen, EXPERTS)
        rows, out = Z.expert_rows(y, plan), []
        ends = plan.offsets.tolist()
        for e, (a, b) in enumerate(zip(ends, ends[1:])):
            if b > a:
                i = layer * EXPERTS + e
                hidden = torch.nn.functional.gelu(Z.mx8_matmul(rows[a:b], packed["experts in"][i]))
                out.append(Z.mx8_matmul(hidden, packed["experts out"][i]))
        x = Z.expert_combine(torch.cat(out), weights, plan)
        if layer < LAYERS - 1:
            y, h = Z.rms_norm(x, p["norms"][layer + 1], h)
    rows8, _ = Z.rms_norm_mx8(x, p["norms"][LAYERS], h)
    return Z.mx8_matmul(rows8, project, torch.float32)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--ranks", type=int, default=2)
    ap.add_argument("--width", type=int, default=128)
    a = ap.parse_args()
    losses, p, ctrl = train(a.steps, a.ranks, a.width)
    for i in range(0, a.steps, max(1, a.steps // 10)):
        print(f"step {i:4d}  loss {losses[i]:.4f}")
    print(f"step {a.steps - 1:4d}  loss {losses[-1]:.4f}  ({ctrl['t']} steps applied, last norm {ctrl['norm']:.4f})")
    ids, following = batch(torch.Generator().manual_seed(1), 200)
    right = (serve(p, ids).argmax(1) == following).float().mean()
    print(f"next tokens found by the served model: {float(right):.2f}")


if __name__ == "__main__":
    main()
