"""Adapters of several tenants on a frozen layer in four bits: trained together with
dropout, their gradients clipped, then served.

The base layer is quantised once (0.53 bytes a weight) and stays as it is; each tenant
has a low-rank adapter on top.  A prompt may run with its activations in four bits too.

    python examples/four_bit_finetune.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import unstructured_sparse_linear_amd as S  # noqa: E402


def finetune(steps=30, tenants=3, features=512, rank=8, tokens=257, dropout=0.05, seed=0):
    """Losses of the steps, the base layer and the trained adapters."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    base = S.Mx4Linear(normal(features, features) * features ** -0.5)
    # packed sequences of unequal lengths, one tenant each
    cuts = [0] + [tokens * (i + 1) // (tenants + 1) + i for i in range(tenants - 1)] + [tokens]
    requests = torch.tensor(cuts, dtype=torch.int32, device="cuda")
    adapter = torch.arange(tenants, dtype=torch.int32, device="cuda")
    xt = normal(features, tokens)
    # what each tenant wants: its own low-rank change of the layer
    target = base(xt)
    for i in range(tenants):
        t = slice(cuts[i], cuts[i + 1])
        change = normal(features, rank) @ normal(rank, features) / (rank * features) ** 0.5
        target[:, t] += change @ xt[:, t]
    layer = S.LowRankAdapters(tenants, rank, features, features, dropout=dropout, seed=seed)
    opt = torch.optim.Adam(layer.parameters(), lr=0.02)
    losses = []
    for _ in range(steps):
        opt.zero_grad()
        y = layer(base(xt), xt, requests, adapter)
        loss = (y - target).square().mean()
        loss.backward()
        S.clip_grad_norm([p.grad for p in layer.parameters()], 0.05)
        opt.step()
        losses.append(loss.detach())
    return [float(v) for v in losses], base, layer


@torch.no_grad()
def serve(base, layer, requests=5, prompt=40, seed=1):
    """A decode step of some requests, and a prompt with its activations in 16 and in 4
    bits."""
    layer.eval()
    g = torch.Generator(device="cuda").manual_seed(seed)
    features, tenants = layer.A.shape[2], layer.A.shape[0]
    xt = torch.randn(features, requests, generator=g, device="cuda")
    offsets = torch.arange(requests + 1, dtype=torch.int32, device="cuda")
    adapter = torch.tensor([i % tenants for i in range(requests)], dtype=torch.int32,
                           device="cuda")
    step = layer.project(base.weight, xt, offsets, adapter)
    long = torch.randn(features, prompt, generator=g, device="cuda").bfloat16()
    whole = base(long)
    four = S.mx4_matmul(base.weight, S.mx4_quantize(long.t()), out_dtype=long.dtype)
    return step, whole, four


if __name__ == "__main__":
    losses, base, layer = finetune()
    step, whole, four = serve(base, layer)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f}")
    apart = (whole.float() - four.float()).square().mean() / whole.float().square().mean()
    print(f"a prompt in four bits is {float(apart) ** 0.5:.3f} of its size away")
