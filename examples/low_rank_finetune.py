"""Low-rank adapters of several tenants on one sparse layer: trained together,
with their gradients clipped, then served.

A frozen sparse layer S (features x features) makes the base output; each tenant
has an adapter of its own on top.  Training packs the tenants' sequences into one
batch; serving makes one token per request beside a dense projection.

    python examples/low_rank_finetune.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import unstructured_sparse_linear_amd as S  # noqa: E402


def finetune(steps=30, tenants=3, features=512, rank=8, tokens=257, seed=0):
    """Losses of the steps, the norms before clipping, and the trained adapters."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    # a sparse base layer, 5% full
    mask = torch.rand(features, features, generator=g, device="cuda") < 0.05
    dense = normal(features, features) * mask * (20.0 / features) ** 0.5
    csr = dense.to_sparse_csr()
    offsets = csr.crow_indices().to(torch.int32)
    columns = csr.col_indices().to(torch.int32)
    order = S.sort_rows_by_nnz(offsets, features)
    # packed sequences of unequal lengths, one tenant each
    cuts = [0] + [tokens * (i + 1) // (tenants + 1) + i for i in range(tenants - 1)] + [tokens]
    requests = torch.tensor(cuts, dtype=torch.int32, device="cuda")
    adapter = torch.arange(tenants, dtype=torch.int32, device="cuda")
    xt = normal(features, tokens)
    base = S.spmm(csr.values(), offsets, order, columns, xt, features)
    # what each tenant wants: its own low-rank change of the layer
    target = base.clone()
    for i in range(tenants):
        t = slice(cuts[i], cuts[i + 1])
        change = normal(features, rank) @ normal(rank, features) / (rank * features) ** 0.5
        target[:, t] += change @ xt[:, t]
    layer = S.LowRankAdapters(tenants, rank, features, features)
    opt = torch.optim.Adam(layer.parameters(), lr=0.02)
    losses, norms = [], []
    for _ in range(steps):
        opt.zero_grad()
        y = layer(base, xt, requests, adapter)
        loss = (y - target).square().mean()
        loss.backward()
        norms.append(S.clip_grad_norm([p.grad for p in layer.parameters()], 0.05))
        opt.step()
        losses.append(loss.detach())
    return [float(v) for v in losses], [float(v) for v in norms], layer, dense


def serve(layer, dense, requests=5, seed=1):
    """One token for each of some requests: the projection and the adapters in one
    pass, and the two apart."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    features, tenants = dense.shape[1], layer.A.shape[0]
    xt = torch.randn(features, requests, generator=g, device="cuda")
    offsets = torch.arange(requests + 1, dtype=torch.int32, device="cuda")
    # every last request of a round of tenants runs on the base layer alone
    adapter = torch.tensor([i % (tenants + 1) if i % (tenants + 1) < tenants else -1
                            for i in range(requests)], dtype=torch.int32, device="cuda")
    together = layer.project(dense, xt, offsets, adapter)
    with torch.no_grad():
        apart = layer(dense @ xt, xt, offsets, adapter)
    return together, apart


if __name__ == "__main__":
    losses, norms, layer, dense = finetune()
    together, apart = serve(layer, dense)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f}, gradient norm {norms[0]:.3f} -> {norms[-1]:.3f}")
    print(f"serving, together against apart: {float((together - apart).abs().max()):.2e}")
