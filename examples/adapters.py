"""Fine-tuning and serving low-rank adapters beside a frozen sparse projection.

``finetune`` trains several adapters at once, one per task: every batch mixes
the tasks' rows, the shared sparse layer gives the base, the gradients of all
adapters are clipped by their global norm.  ``serve`` answers single rows of
many requests, each with its own adapter, and checks them against the same
products computed one by one.

    python examples/adapters.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import unstructured_sparse_nn_amd as snk  # noqa: E402


def sparse_layer(K, M, density, max_batch, dtype=torch.float32, seed=0):
    """A SparseLinear with random connections, its values frozen."""
    g = torch.Generator().manual_seed(seed)
    flat = torch.randperm(K * M, generator=g)[:int(K * M * density)].sort().values
    row, col = (flat // K).int(), (flat % K).int()
    vals = torch.randn(flat.numel(), generator=g) * (density * K) ** -0.5
    layer = snk.SparseLinear(K, M, row.cuda(), col.cuda(), vals.to(dtype).cuda(), max_batch)
    layer.vals.requires_grad_(False)
    return layer


def finetune(tasks=4, K=256, M=192, rank=8, rows=256, steps=60, lr=0.02, max_norm=1.0):
    """The loss of the first and of the last step."""
    torch.manual_seed(0)
    layer = sparse_layer(K, M, 0.1, rows)
    adapters = snk.LoraAdapters(K, M, tasks, rank, alpha=rank)
    opt = torch.optim.Adam(adapters.parameters(), lr=lr)
    shift = torch.randn(tasks, M, 4, device="cuda") @ torch.randn(4, K, device="cuda") / K
    losses = []
    for _ in range(steps):
        x = torch.randn(rows, K, device="cuda")
        ids = torch.randint(0, tasks, (rows,), device="cuda").int()
        with torch.no_grad():
            base = layer(x)
            want = base + (shift[ids.long()] @ x[:, :, None])[:, :, 0]
        loss = (adapters(x, ids, base) - want).square().mean()
        opt.zero_grad(set_to_none=True)
        loss.backward()
        snk.clip_grad_norm_(adapters.parameters(), max_norm)
        opt.step()
        losses.append(loss.detach())
    return float(losses[0]), float(losses[-1])


@torch.no_grad()
def serve(requests=13, K=512, M=384, tasks=6, dtype=torch.bfloat16):
    """One row of each request through the sparse layer and its adapter."""
    torch.manual_seed(1)
    layer = sparse_layer(K, M, 0.05, 32, dtype)
    adapters = snk.LoraAdapters(K, M, tasks, 16, ranks=[16, 8, 4, 16, 8, 4], dtype=dtype)
    adapters.B.normal_(std=0.1)
    x = torch.randn(requests, K, device="cuda").to(dtype)
    ids = torch.randint(-1, tasks, (requests,), device="cuda").int()
    base = layer(x)
    y = adapters(x, ids, base)
    for i, a in enumerate(ids.tolist()):
        want = base[i].double()
        if a >= 0:
            r = int(adapters.ranks[a])
            t = adapters.A[a, :r].double() @ x[i].double()
            want = want + float(adapters.scale[a]) * (t @ adapters.B[a, :r].double())
        # the output's rounding, half a step of bf16
        assert ((y[i].double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-3).all(), i
    return y


if __name__ == "__main__":
    first, last = finetune()
    print(f"mean squared error of 4 tasks: {first:.5f} at the first step, {last:.5f} at the last")
    y = serve()
    print(f"served {y.shape[0]} requests, {y.shape[1]} features each")
