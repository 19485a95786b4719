"""Adapters on frozen 4-bit projections: trained, then served to mixed requests.

Two W4A16 projections with a ReLU between them stay as they are; every task has
its own low-rank adapter on both.  A step takes tokens of all tasks at once:
forward (keeping u), loss, backward (dx through the packed weights, the
adapters' gradients), one AdamW launch over all adapters with 8-bit moments that
also writes the bf16 copies the next forward reads.  Afterwards single tokens of
different tasks are decoded in one call.

    python examples/adapters.py
"""
import os
import sys

import numpy as np

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

GROUP = 128


class Projection:
    """A frozen 4-bit weight [N, K] with a stack of adapters of rank R beside it."""

    def __init__(self, N, K, tasks, R, rng, dtype):
        import torch
        import int4_weight_only_linear_amd as L
        self.codes = rng.integers(0, 16, (N, K), dtype=np.uint8)
        self.wq = torch.from_numpy(L.w4a16_pack_weights(self.codes)).cuda()
        # codes - 8 have a root mean square of 4.6: outputs about as large as inputs
        self.scales = torch.full((N, K // GROUP), 1 / (4.6 * K**0.5), dtype=dtype, device="cuda")
        a = rng.standard_normal((tasks, R, K)).astype(np.float32) / K**0.5
        self.masters = [torch.from_numpy(a).cuda(), torch.zeros((tasks, N, R), device="cuda")]
        self.factors = [m.to(dtype) for m in self.masters]  # what the kernels read
        self.grads = [torch.zeros_like(f) for f in self.factors]

    def forward(self, x, ids, save_u=False):
        import int4_weight_only_linear_amd as L
        return L.w4a16_lora_linear(x, self.wq, self.scales, *self.factors, ids, group_size=GROUP, save_u=save_u)

    def backward(self, dy, x, u, ids, need_dx=True):
        """The adapters' gradients into self.grads; returns dx."""
        import torch
        import int4_weight_only_linear_amd as L
        dx = torch.empty_like(x) if need_dx else None
        L.w4a16_lora_backward(dy, x, u, self.wq, self.scales, *self.factors, ids, group_size=GROUP,
                              out=(dx, *self.grads))
        return dx


def train(tasks=3, K=512, H=768, N=256, R=16, tokens=384, steps=150, lr=4e-3, seed=0):
    """Teaches each task's adapters a target of its own; returns (losses, up, down, targets)."""
    import torch
    import int4_weight_only_linear_amd as L
    dtype, rng = torch.bfloat16, np.random.default_rng(seed)
    up, down = Projection(H, K, tasks, R, rng, dtype), Projection(N, H, tasks, R, rng, dtype)
    # the targets: the frozen projections' output through a rotation of each task's own
    turn = torch.from_numpy(np.stack([np.linalg.qr(rng.standard_normal((N, 4)))[0] for _ in range(tasks)])).to("cuda", torch.float32)
    masters, copies, grads = up.masters + down.masters, up.factors + down.factors, up.grads + down.grads
    moments = [(torch.zeros(m.numel(), dtype=torch.int8, device="cuda"), torch.zeros(m.numel(), dtype=torch.uint8, device="cuda"),
                torch.zeros((m.numel() + 255) // 256, device="cuda"), torch.zeros((m.numel() + 255) // 256, device="cuda"))
               for m in masters]
    m, v, ms, vs = map(list, zip(*moments))
    plan = L.w4a16_adamw_plan(masters, grads, m, v, m_scales=ms, v_scales=vs, copies=copies)
    none = torch.full((tokens,), -1, dtype=torch.int32, device="cuda")

    def target(x, ids):
        y = down.forward(torch.relu(up.forward(x, none)), none).float()
        q = turn[ids.long()]  # [tokens, N, 4]: the output without its part in a subspace
        return y - 2 * (q @ (q.transpose(1, 2) @ y[:, :, None]))[:, :, 0]

    losses = []
    for step in range(1, steps + 1):
        x = torch.from_numpy(rng.standard_normal((tokens, K)).astype(np.float32)).to("cuda", dtype)
        ids = torch.from_numpy(rng.integers(0, tasks, tokens).astype(np.int32)).cuda()
        want = target(x, ids)
        h, u1 = up.forward(x, ids, save_u=True)
        a = torch.relu(h)
        y, u2 = down.forward(a, ids, save_u=True)
        diff = y.float() - want
        losses.append(float((diff * diff).mean() / (want * want).mean()))
        dy = (diff * (2 / diff.numel())).to(dtype)
        da = down.backward(dy, a, u2, ids)
        up.backward(da * (h > 0), x, u1, ids, need_dx=False)
        L.w4a16_adamw_step(plan, lr=lr, weight_decay=0.0, step=step, seed=step)
    return losses, up, down, target


def serve(up, down, x, ids):
    """Single tokens of several requests, each through its own adapters."""
    import torch
    return down.forward(torch.relu(up.forward(x, ids)), ids)


def main():
    import torch
    losses, up, down, target = train()
    for step in (0, len(losses) // 4, len(losses) // 2, len(losses) - 1):
        print(f"step {step + 1:4d}  relative squared error {losses[step]:.4f}")
    x = torch.randn(4, 512, device="cuda").to(torch.bfloat16)
    ids = torch.tensor([2, 0, -1, 1], dtype=torch.int32, device="cuda")
    y = serve(up, down, x, ids)
    print("served", tuple(y.shape), "tokens of tasks", ids.tolist())


if __name__ == "__main__":
    main()
