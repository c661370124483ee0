"""A training step of one MoE layer with gated experts, from token ids to the updated weights.

    python examples/train_moe_experts.py --steps 40

The task is that of train_moe_tokens.py: given a token id, name the id that
follows it in a fixed random cycle.  The model: an embedding, a linear router
with sigmoid scores, groups of experts and a bias that balances them, E gated
experts (silu(x G) * (x U), then a second product) and a linear head.  Weights
are BF16 with FP32 master copies; AdamW keeps its moments in 8 bits.

    forward    embed -> router product -> route_scored -> dispatch + stash push
               -> expert_linear (gated) -> expert_linear -> combine -> head
    backward   head -> combine_backward -> expert_linear_dw, expert_linear_dx
               (through the second product and the gate) -> stash pop ->
               expert_linear_dw, expert_linear_dx -> dispatch_backward ;
               dw -> route_scored_backward -> router product -> embed_backward
    update     grad_norm, AdamW step (skipped when the pool overflowed),
               route_bias_step

Everything runs on the pool's paging stream; live counts never leave the GPU.
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import activation_paging_gb300 as ap  # noqa: E402

PAD = 0


class Layer:
    def __init__(self, V=257, H=64, F=96, E=16, k=4, groups=4, top_groups=2, max_tokens=1024, lr=2e-2, seed=0, device="cuda"):
        self.V, self.H, self.F, self.E, self.k, self.groups, self.top_groups = V, H, F, E, k, groups, top_groups
        g = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape, scale):
            return (torch.randn(*shape, generator=g, device=device) * scale).bfloat16()
        self.scale = math.sqrt(H)
        self.params = {"table": normal(V, H, scale=1 / math.sqrt(H)), "router": normal(E, H, scale=0.1),
                       "gate_up": normal(E, 2 * F, H, scale=1 / math.sqrt(H)), "down": normal(E, H, F, scale=1 / math.sqrt(F)),
                       "down_bias": normal(E, H, scale=0.1), "head": normal(H, V, scale=1 / math.sqrt(H))}
        self.grads = {n: torch.zeros(p.shape, device=device) for n, p in self.params.items()}
        self.bias = torch.zeros(E, device=device)  # balances the experts; has no gradient
        self.counts = torch.zeros(E, dtype=torch.int32, device=device)
        self.opt = ap.AdamW(list(self.params.values()), list(self.grads.values()), lr=lr, betas=(0.9, 0.95), weight_decay=0.01,
                            master=True, state_bits=8, seed=seed)
        P = 16
        self.pool = ap.Pool(P, ap.page_bytes_for(P, (2 * H,)), max_tokens * k // P + E, 1, 2, E)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)

    def step(self, ids: torch.Tensor, target: torch.Tensor, mask: torch.Tensor) -> torch.Tensor:
        """Forward and backward of one batch (ids, target [T], mask [T] bool: positions that are not padding); adds to the
        gradients and counts.  Call it on the pool's stream."""
        s, p, q = self.pool.stream, self.params, self.grads
        H, E, k, st = self.H, self.E, self.k, self.status
        # forward
        x = ap.embed(p["table"], ids, scale=self.scale, status=st, stream=s)
        logits = x.float() @ p["router"].float().t()
        idx, w = ap.route_scored(logits, k, bias=self.bias, groups=self.groups, top_groups=self.top_groups, scale=2.0, mask=mask,
                                 counts=self.counts, stream=s)
        d = self.pool.dispatch_stash(0, x, idx, E, status=st)
        rows = d["xd"].shape[0]
        seg, live = d["seg_off"], d["live"]
        z = torch.empty(rows, 2 * self.F, dtype=torch.bfloat16, device=ids.device)
        h = ap.expert_linear(d["xd"], p["gate_up"], seg, live, act="swiglu", pre=z, status=st, stream=s)
        y = ap.expert_linear(h, p["down"], seg, live, bias=p["down_bias"].float(), status=st, stream=s)
        del d["xd"]  # the rows wait in the stash
        out = ap.combine_unpermute(y, d["dest"], w, status=st, stream=s)
        lz = out.float() @ p["head"].float()
        lse = torch.logsumexp(lz, 1)
        n = mask.sum().clamp(min=1)
        loss = ((lse - lz.gather(1, target[:, None])[:, 0]) * mask).sum() / n
        # backward
        dz = torch.softmax(lz, 1)
        dz.scatter_add_(1, target[:, None], torch.full((ids.shape[0], 1), -1.0, device=ids.device))
        dz *= (mask / n)[:, None]
        q["head"] += out.float().t() @ dz
        dout = (dz @ p["head"].float().t()).bfloat16()
        dy = torch.empty_like(y)
        _, dw = ap.combine_backward(dout, y, d["dest"], w, dy=dy, status=st, stream=s)
        ap.expert_linear_dw(dy, h, seg, live, dW=q["down"], dbias=q["down_bias"], accumulate=True, status=st, stream=s)
        dzz = ap.expert_linear_dx(dy, p["down"], seg, live, act="swiglu", pre=z, status=st, stream=s)
        back = torch.empty(rows, H, dtype=torch.bfloat16, device=ids.device)
        self.pool.pop(0, [back])
        ap.expert_linear_dw(dzz, back, seg, live, dW=q["gate_up"], accumulate=True, status=st, stream=s)
        dxd = ap.expert_linear_dx(dzz, p["gate_up"], seg, live, status=st, stream=s)
        dx = ap.dispatch_backward(dxd, d["dest"], status=st, stream=s).float()
        dlogits = ap.route_scored_backward(logits, idx, dw, scale=2.0, status=st, stream=s, w=w)
        q["router"] += dlogits.t() @ x.float()
        dx += dlogits @ p["router"].float()
        ap.embed_backward(dx, ids, self.V, scale=self.scale, padding_idx=PAD, dtable=q["table"], accumulate=True, status=st, stream=s)
        return loss

    def update(self, max_norm: float = 1.0):
        s = self.pool.stream
        norm = self.opt.grad_norm(max_norm, stream=s)
        self.opt.step(scale=norm[1:], skip=self.pool, stream=s)
        ap.route_bias_step(self.bias, self.counts, 1e-3, reset=True, stream=s)
        for g in self.grads.values():
            g.zero_()


def batch(follow: torch.Tensor, sequences: int, length: int, g: torch.Generator):
    """ids of `sequences` sequences of `length` positions with padded ends, their followers, and the mask."""
    V = follow.shape[0]
    ids = torch.randint(1, V, (sequences, length), generator=g, device=follow.device)
    used = torch.randint(length // 2, length + 1, (sequences, 1), generator=g, device=follow.device)
    mask = torch.arange(length, device=follow.device)[None, :] < used
    ids = torch.where(mask, ids, PAD).view(-1)
    return ids, follow[ids], mask.view(-1)


def train(steps: int = 40, sequences: int = 8, length: int = 64, report=None) -> list:
    layer = Layer(max_tokens=sequences * length)
    g = torch.Generator(device="cuda").manual_seed(1)
    order = torch.randperm(layer.V - 1, generator=g, device="cuda") + 1
    follow = torch.zeros(layer.V, dtype=torch.int64, device="cuda")
    follow[order] = order.roll(-1)
    s = layer.pool.stream
    s.wait_stream(torch.cuda.current_stream())
    history = []
    with torch.cuda.stream(s):
        for step in range(steps):
            loss = layer.step(*batch(follow, sequences, length, g))
            history.append((loss, layer.counts.clone()))
            layer.update()
            if report and (step % 10 == 0 or step + 1 == steps):
                report(step, float(loss), history[-1][1].tolist())
    torch.cuda.synchronize()
    assert int(layer.status) == 0 and layer.pool.overflow() == 0
    assert int(layer.opt.state["step"][0]) == steps
    return [(float(a), c.tolist()) for a, c in history]


def main():
    a = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    a.add_argument("--steps", type=int, default=40)
    a = a.parse_args()
    train(a.steps, report=lambda step, loss, counts: print(f"step {step:4d}  loss {loss:.4f}  pairs per expert {counts}"))


if __name__ == "__main__":
    main()
