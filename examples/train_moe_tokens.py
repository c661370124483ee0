"""A training step of one MoE layer from token ids to the embedding's gradient.

    python examples/train_moe_tokens.py --steps 60

The task: given a token id, name the id that follows it in a fixed random
cycle.  The model: an embedding (FP32, scaled by sqrt(H)), a linear router
with its balance loss, E linear experts, and a linear head.  The token
movement of both passes runs on the package; the matrix products are torch's.

    forward    embed -> router product -> route_balance -> dispatch + stash push
               -> experts -> combine -> head
    backward   head -> combine_backward (dy, dw) -> stash pop -> expert products
               -> dispatch_backward (dx) ; dw, slope -> route_backward (dlogits)
               -> router product -> embed_backward (added over micro-batches)

Everything runs on the pool's paging stream.  Ids outside the first `length`
positions of a sequence are padding: they count neither for the balance loss
nor for the embedding's gradient.
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
    def __init__(self, V=257, H=64, E=8, k=2, max_tokens=1024, coef=0.02, seed=0, device="cuda"):
        self.V, self.H, self.E, self.k, self.coef = V, H, E, k, coef
        g = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape, scale):
            return torch.randn(*shape, generator=g, device=device) * scale
        self.scale = math.sqrt(H)
        self.params = {"table": normal(V, H, scale=1 / math.sqrt(H)), "router": normal(H, E, scale=0.1),
                       "experts": normal(E, H, H, scale=1 / math.sqrt(H)), "head": normal(H, V, scale=1 / math.sqrt(H))}
        self.grads = {n: torch.zeros_like(p) for n, p in self.params.items()}
        P = 16
        # room for one record of all pairs, every expert's last page partly filled
        self.pool = ap.Pool(P, ap.page_bytes_for(P, (2 * H,)), max_tokens * k // P + E, 1, 2, E)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)

    def step(self, ids: torch.Tensor, target: torch.Tensor, mask: torch.Tensor, group_tokens: int, weight: float) -> dict:
        """Forward and backward of one micro-batch: ids, target [T], mask [T] bool (positions that are not padding);
        adds ``weight`` x the gradients.  Call it on the pool's stream."""
        s, p, q = self.pool.stream, self.params, self.grads
        T, H, E = ids.shape[0], self.H, self.E
        # forward
        x = ap.embed(p["table"], ids, scale=self.scale, dtype=torch.bfloat16, status=self.status, stream=s)
        logits = x.float() @ p["router"]
        r = ap.route_balance(logits, self.k, coef=self.coef, group_tokens=group_tokens, mask=mask, stream=s)
        d = self.pool.dispatch_stash(0, x, r["idx"], E, capacity=T, padded=True, status=self.status)
        W = p["experts"].bfloat16()
        live = (torch.arange(T, device=ids.device)[None, :] < d["live"][:, None])[..., None]
        xd = torch.where(live, d["xd"].view(E, T, H), 0)
        y = torch.bmm(xd, W).view(E * T, H)
        del xd, d["xd"]  # the rows wait in the stash
        out = ap.combine_unpermute(y, d["dest"], r["w"], status=self.status, stream=s)
        z = out.float() @ p["head"]
        lse = torch.logsumexp(z, 1)
        n = mask.sum().clamp(min=1)
        loss = ((lse - z.gather(1, target[:, None])[:, 0]) * mask).sum() / n
        # backward
        dz = torch.softmax(z, 1)
        dz.scatter_add_(1, target[:, None], torch.full((T, 1), -1.0, device=ids.device))
        dz *= (mask * (weight / n))[:, None]
        q["head"] += out.float().t() @ dz
        dout = (dz @ p["head"].t()).bfloat16()
        dy, dw = ap.combine_backward(dout, y, d["dest"], r["w"], status=self.status, stream=s)
        back = torch.zeros(E * T, H, dtype=torch.bfloat16, device=ids.device)
        self.pool.pop(0, [back])
        q["experts"] += torch.bmm(back.view(E, T, H).transpose(1, 2), dy.view(E, T, H)).float()
        dxd = torch.bmm(dy.view(E, T, H), W.transpose(1, 2)).view(E * T, H)
        dx = ap.dispatch_backward(dxd, d["dest"], status=self.status, stream=s).float()
        dlogits = ap.route_backward(logits, r["idx"], r["w"], dw=dw, slope=r["slope"],
                                    dloss=torch.full((1,), weight, device=ids.device), group_tokens=group_tokens,
                                    mask=mask, status=self.status, stream=s)
        q["router"] += x.float().t() @ dlogits
        dx += dlogits @ p["router"].t()
        ap.embed_backward(dx, ids, self.V, scale=self.scale, padding_idx=PAD, dtable=q["table"], accumulate=True,
                          status=self.status, stream=s)
        return {"loss": loss, "balance": r["loss"], "counts": r["counts"]}

    def update(self, lr: float):
        for n, p in self.params.items():
            p -= lr * self.grads[n]
            self.grads[n].zero_()


def batch(follow: torch.Tensor, sequences: int, length: int, g: torch.Generator):
    """ids of `sequences` sequences of `length` positions with padded ends, their followers, and the mask."""
    V = follow.shape[0]
    ids = torch.randint(1, V, (sequences, length), generator=g, device=follow.device)
    used = torch.randint(length // 2, length + 1, (sequences, 1), generator=g, device=follow.device)
    mask = torch.arange(length, device=follow.device)[None, :] < used
    ids = torch.where(mask, ids, PAD).view(-1)
    return ids, follow[ids], mask.view(-1)


def train(steps: int = 60, sequences: int = 8, length: int = 64, micro: int = 2, lr: float = 2.0, report=None) -> list:
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
            parts = [layer.step(*batch(follow, sequences, length, g), length, 1.0 / micro) for _ in range(micro)]
            layer.update(lr)
            history.append([torch.stack([p[n] for p in parts]).mean() for n in ("loss", "balance")] +
                           [sum(p["counts"].sum(0) for p in parts)])
            if report and (step % 10 == 0 or step + 1 == steps):
                loss, balance, counts = history[-1]
                report(step, float(loss), float(balance), counts.tolist())
    torch.cuda.synchronize()
    assert int(layer.status) == 0 and layer.pool.overflow() == 0
    return [(float(a), float(b), c.tolist()) for a, b, c in history]


def main():
    a = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    a.add_argument("--steps", type=int, default=60)
    a.add_argument("--lr", type=float, default=2.0)
    a = a.parse_args()
    train(a.steps, lr=a.lr, report=lambda step, loss, balance, counts: print(
        f"step {step:4d}  loss {loss:.4f}  balance loss {balance:.5f}  pairs per expert {counts}"))


if __name__ == "__main__":
    main()
