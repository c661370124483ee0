"""Cases that measure the training operators at the two ends of the MoE token path.

Four operators, each in a plain form of elementary torch operations (``own`` false) and as a user calls it (``own`` true):

    balance     routing with its balance loss: expert ids and weights, per-expert counts, mean probabilities, the loss and
                its slope, over groups of tokens and a mask of padding tokens
    router_grad gradient of the router's logits from the gradient of the routing weights and from the balance loss
    embed       rows of an embedding table for token ids, scaled
    embed_grad  gradient of the table: the rows of each id added up, written whole or added to a kept gradient

Sizes come from the workloads of ``activation_paging_gb300/inputs.py`` (256 tokens over 8 experts, top 2; 8192 tokens over
128 experts, top 8, H = 2048; 32768 tokens over 256 experts, top 8, H = 7168); the vocabularies (32003, 131072 and 151936
rows) are generic.  Token ids follow a Zipf law over the vocabulary (a few ids take a large share, most occur once), as
text does.
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}


def _balance(name, T, E, k, group=0, pad=False, zipf=0.0, op="balance"):
    return {"name": name, "op": op, "T": T, "E": E, "k": k, "group": group, "pad": pad, "zipf": zipf}


def _embed(name, T, H, V, table="bf16", out="bf16", wide=False):
    return {"name": name, "op": "embed", "T": T, "H": H, "V": V, "table": table, "out": out, "wide": wide}


def _embed_grad(name, T, H, V, dout="bf16", grad="f32", accumulate=True, pad=0.0, wide=False):
    return {"name": name, "op": "embed_grad", "T": T, "H": H, "V": V, "dout": dout, "grad": grad,
            "accumulate": accumulate, "pad": pad, "wide": wide}


def listed():
    return [
        # one small batch through a small router: latency counts
        _balance("balance 256x8", 256, 8, 2),
        # one chunk of a training step's layer
        _balance("balance 8192x128", 8192, 128, 8),
        # a skewed router with a loss for each sequence of 4096 positions, padded at the ends, one sequence all padding
        _balance("balance 32768x256 seqs", 32768, 256, 8, 4096, True, 1.0),
        # an odd batch of three padded sequences over an odd number of experts
        _balance("router grad 999x60 seqs", 999, 60, 6, 333, True, op="router_grad"),
        # one chunk of a training step's layer
        _balance("router grad 8192x128", 8192, 128, 8, op="router_grad"),
        # the skewed, padded sequences of the third case, backwards
        _balance("router grad 32768x256 seqs", 32768, 256, 8, 4096, True, 1.0, op="router_grad"),
        # one decoding step of four sequences
        _embed("embed 4 tokens", 4, 2048, 151936),
        # the tokens of one training step
        _embed("embed 16384 tokens", 16384, 2048, 151936),
        # a small batch with rows of odd length, everything in single precision
        _embed_grad("embed grad 777 odd", 777, 1001, 32003, "f32", "f32", True, 0.1),
        # one chunk, added to the gradient kept over a step's chunks
        _embed_grad("embed grad 8192 add", 8192, 2048, 151936),
        # the tokens of one step, the gradient written whole in the parameters' type
        _embed_grad("embed grad 16384 whole", 16384, 2048, 151936, "bf16", "bf16", False),
        # the largest rows and batch, 30% of the positions padding
        _embed_grad("embed grad 32768 padded", 32768, 7168, 131072, "bf16", "f32", True, 0.3),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["balance", "router_grad", "embed", "embed_grad"])
    if op in ("balance", "router_grad"):
        E = _log(rng, 4, 1024)
        T = _log(rng, 1, min(32768, 32768 * 256 // E))
        k = rng.randint(1, min(E, 12))
        group = rng.choice([0, 0, max(1, -(-T // rng.randint(2, 9)))])
        case = _balance("", T, E, k, group, rng.random() < 0.5, rng.choice([0.0, 0.5, 1.0]), op)
    elif op == "embed":
        H = _log(rng, 64, 7168)
        V = _log(rng, 1000, 262144)
        case = _embed("", _log(rng, 1, 32768), H, V, rng.choice(["bf16", "f32"]), rng.choice(["bf16", "bf16", "f32"]),
                      rng.random() < 0.25)
        while case["V"] * case["H"] * BYTES[case["table"]] > 3 << 30:
            case["V"] //= 2
        while case["T"] * case["H"] * BYTES[case["out"]] > 480 << 20:
            case["T"] //= 2
    else:
        H = _log(rng, 64, 7168)
        V = _log(rng, 1000, 262144)
        case = _embed_grad("", _log(rng, 1, 32768), H, V, rng.choice(["bf16", "bf16", "f32"]),
                           rng.choice(["f32", "f32", "bf16"]), rng.random() < 0.6, rng.choice([0.0, 0.0, 0.3]),
                           rng.random() < 0.25)
        most = (3 << 30) if case["accumulate"] else (600 << 20)
        while case["V"] * case["H"] * BYTES[case["grad"]] > most:
            case["V"] //= 2
        while case["T"] * case["H"] * BYTES[case["dout"]] > 240 << 20:
            case["T"] //= 2
    del case["name"]
    return case


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 2654435761 % (1 << 62))


def _ids(g, T, V):
    """T ids of a Zipf law (s = 1) over V, the frequent ones low, as byte-pair vocabularies have them."""
    cdf = torch.cumsum(1.0 / torch.arange(1, V + 1, device="cuda", dtype=torch.float64), 0)
    u = torch.rand(T, generator=g, device="cuda", dtype=torch.float64) * cdf[-1]
    return torch.searchsorted(cdf, u).clamp_(max=V - 1)


def _rows(g, n, H, dtype, wide, scale=1.0):
    """n rows of H values; wide: the first H columns of wider rows, as a slice of a joint buffer has them."""
    pitch = H + 64 if wide else H
    a = torch.empty(n, pitch, device="cuda", dtype=DT[dtype])
    a.normal_(0.0, scale, generator=g)
    return a[:, :H]


def _groups(case):
    S = case["group"] or case["T"]
    return S, -(-case["T"] // S)


def prepare(case, seed):
    g = _gen(seed)
    T = case["T"]
    if case["op"] in ("balance", "router_grad"):
        E, k = case["E"], case["k"]
        S, G = _groups(case)
        logits = torch.randn(T, E, generator=g, device="cuda")
        if case["zipf"]:
            rank = torch.randperm(E, generator=g, device="cuda").float() + 1
            logits -= 0.375 * case["zipf"] * torch.log(rank)
        mask = None
        if case["pad"]:  # each sequence ends in padding; the last of several is all padding
            length = (torch.rand(G, generator=g, device="cuda") * 0.5 + 0.5).mul_(S).ceil_()
            if G > 2:
                length[-1] = 0
            t = torch.arange(T, device="cuda")
            mask = (t % S) < length[t // S]
        s = {"case": dict(case), "logits": logits, "mask": mask, "coef": 0.01}
        if case["op"] == "router_grad":  # what the forward pass left, and the gradient of the routing weights
            idx, w, _ = _choose(logits, k)
            s |= {"idx": idx, "w": w, "dw": torch.randn(T, k, generator=g, device="cuda") * (0.1 / T),
                  "slope": _slope(idx, mask, S, G, E, 0.01)[1], "dloss": torch.full((1,), 1.0, device="cuda")}
        return s
    H, V = case["H"], case["V"]
    ids = _ids(g, T, V)
    if T % 2:
        ids = ids.int()
    if case["op"] == "embed":
        return {"case": dict(case), "ids": ids, "table": _rows(g, V, H, case["table"], case["wide"], 0.02),
                "scale": math.sqrt(H)}
    pad = V - 1
    if case["pad"]:
        n = int(T * case["pad"])
        ids[T - n:] = pad
    dtable = torch.zeros(V, H, device="cuda", dtype=DT[case["grad"]])
    if case["accumulate"]:
        dtable.normal_(0.0, 1e-3, generator=g)
    return {"case": dict(case), "ids": ids, "dout": _rows(g, T, H, case["dout"], case["wide"], 1e-3), "dtable": dtable,
            "scale": math.sqrt(H), "pad": pad}


def _choose(logits, k):
    """(idx, w, p): the k largest logits of each row (ties to the lowest id), their renormalised weights, the softmax."""
    idx = torch.sort(logits, dim=1, descending=True, stable=True)[1][:, :k]
    z = torch.exp(logits - logits.amax(1, keepdim=True))
    zs = torch.gather(z, 1, idx)
    return idx.int(), zs / zs.sum(1, keepdim=True), z / z.sum(1, keepdim=True)


def _slope(idx, mask, S, G, E, coef):
    """(counts, slope): pairs of each group and expert, and d loss / d p of a group's tokens."""
    T, k = idx.shape
    group = torch.arange(T, device=idx.device) // S
    valid = torch.ones(T, dtype=torch.int32, device=idx.device) if mask is None else mask.int()
    counts = torch.zeros(G * E, dtype=torch.int32, device=idx.device)
    counts.scatter_add_(0, (group[:, None] * E + idx).reshape(-1), valid[:, None].expand(T, k).reshape(-1))
    counts = counts.view(G, E)
    n = torch.zeros(G, dtype=torch.int32, device=idx.device).scatter_add_(0, group, valid).clamp_(min=1).float()
    return counts, coef * E / (G * k) * counts / (n * n)[:, None]


def _run_balance(s):
    c, logits, mask = s["case"], s["logits"], s["mask"]
    T, E, k = c["T"], c["E"], c["k"]
    S, G = _groups(c)
    idx, w, p = _choose(logits, k)
    counts, slope = _slope(idx, mask, S, G, E, s["coef"])
    if mask is not None:
        p = torch.where(mask[:, None], p, torch.zeros_like(p))
    if T < G * S:
        p = torch.cat([p, torch.zeros(G * S - T, E, device=p.device)])
    total = p.view(G, S, E).sum(1)
    n = counts.sum(1, keepdim=True).clamp(min=1) / k
    prob = total / n
    loss = (slope * total).sum()
    return {"idx": idx, "w": w, "counts": counts, "prob": prob, "slope": slope, "loss": loss}


def _run_router_grad(s):
    c, logits, mask, idx, w, dw = s["case"], s["logits"], s["mask"], s["idx"], s["w"], s["dw"]
    S, G = _groups(c)
    z = torch.exp(logits - logits.amax(1, keepdim=True))
    p = z / z.sum(1, keepdim=True)
    slope = s["slope"].repeat_interleave(S, 0)[: c["T"]]
    d = p * (slope - (p * slope).sum(1, keepdim=True)) * s["dloss"]
    if mask is not None:
        d = torch.where(mask[:, None], d, torch.zeros_like(d))
    d.scatter_add_(1, idx.long(), w * (dw - (w * dw).sum(1, keepdim=True)))
    return d


def run(state):
    c = state["case"]
    if own:
        return _run_own(state)
    if c["op"] == "balance":
        return _run_balance(state)
    if c["op"] == "router_grad":
        return _run_router_grad(state)
    ids = state["ids"].long()
    if c["op"] == "embed":
        return (state["table"][ids].float() * state["scale"]).to(DT[c["out"]])
    dtable = state["dtable"]
    rows = state["dout"].float() * state["scale"]
    rows = torch.where((ids != state["pad"])[:, None], rows, torch.zeros_like(rows))
    if c["grad"] == "f32":
        if not c["accumulate"]:
            dtable.zero_()
        return dtable.index_add_(0, ids, rows)
    total = dtable.float() if c["accumulate"] else torch.zeros_like(dtable, dtype=torch.float32)
    return dtable.copy_(total.index_add_(0, ids, rows))


def _run_own(state):
    import activation_paging_gb300 as ap

    c = state["case"]
    if c["op"] == "balance":
        r = ap.route_balance(state["logits"], c["k"], coef=state["coef"], group_tokens=c["group"], mask=state["mask"])
        return {n: r[n] for n in ("idx", "w", "counts", "prob", "slope", "loss")}
    if c["op"] == "router_grad":
        return ap.route_backward(state["logits"], state["idx"], state["w"], dw=state["dw"], slope=state["slope"],
                                 dloss=state["dloss"], group_tokens=c["group"], mask=state["mask"])
    if c["op"] == "embed":
        return ap.embed(state["table"], state["ids"], scale=state["scale"], dtype=DT[c["out"]])
    return ap.embed_backward(state["dout"], state["ids"], c["V"], scale=state["scale"], padding_idx=state["pad"],
                             dtable=state["dtable"], accumulate=c["accumulate"])


def _distinct(T, V):
    """Expected number of different ids among T draws of the Zipf law over V."""
    p = 1.0 / np.arange(1, V + 1)
    p /= p.sum()
    return float(-np.expm1(T * np.log1p(-p)).sum()) if V > 1 else 1.0


def work(case):
    T = case["T"]
    if case["op"] in ("balance", "router_grad"):
        E, k = case["E"], case["k"]
        G = _groups(case)[1]
        mask = T if case["pad"] else 0
        if case["op"] == "balance":  # logits in; ids, weights, counts, means and slopes out
            return {"bytes": 4 * T * E + 8 * T * k + 12 * G * E + 4 + mask, "flops": 5 * T * E + 4 * T * k}
        # logits, ids, weights, their gradient and slopes in; the logits' gradient out
        return {"bytes": 8 * T * E + 12 * T * k + 4 * G * E + 4 + mask, "flops": 8 * T * E + 4 * T * k}
    H, V = case["H"], case["V"]
    idb = 4 if T % 2 else 8
    if case["op"] == "embed":  # each different row in once, each output row out once
        return {"bytes": idb * T + _distinct(T, V) * H * BYTES[case["table"]] + T * H * BYTES[case["out"]],
                "flops": T * H}
    n = T - int(T * case["pad"])  # rows that count; each different row of the gradient read and written, or all written
    rows = 2 * _distinct(n, V) if case["accumulate"] else V
    return {"bytes": idb * T + n * H * BYTES[case["dout"]] + rows * H * BYTES[case["grad"]], "flops": n * H}


def exact(case, seed):
    s = prepare(case, seed)
    T = case["T"]
    if case["op"] in ("balance", "router_grad"):
        E, k = case["E"], case["k"]
        S, G = _groups(case)
        x = s["logits"].cpu().numpy().astype(np.float64)
        valid = np.ones(T, bool) if s["mask"] is None else s["mask"].cpu().numpy()
        lse = np.log(np.exp(x - x.max(1, keepdims=True)).sum(1, keepdims=True)) + x.max(1, keepdims=True)
        p = np.exp(x - lse)
        if case["op"] == "balance":
            order = np.argsort(-x, axis=1, kind="stable")[:, :k]
            sel = np.take_along_axis(p, order, 1)
            w = sel / sel.sum(1, keepdims=True)
            counts = np.zeros((G, E), np.int64)
            prob, slope, loss = np.zeros((G, E)), np.zeros((G, E)), 0.0
            for q in range(G):
                m = np.flatnonzero(valid[q * S:(q + 1) * S]) + q * S
                if m.size:
                    counts[q] = np.bincount(order[m].ravel(), minlength=E)
                    prob[q] = p[m].mean(0)
                    share = counts[q] / (m.size * k)
                    slope[q] = s["coef"] * E * share / (G * m.size)
                    loss += s["coef"] * E * float(share @ prob[q]) / G
            return {"idx": None, "w": w, "counts": None, "prob": prob, "slope": slope, "loss": np.float64(loss)}
        slope = s["slope"].cpu().numpy().astype(np.float64)[np.arange(T) // S]
        # w and idx are inputs: the derivative of the selected softmax at them
        w, dw, idx = (s[n].cpu().numpy().astype(np.float64) for n in ("w", "dw", "idx"))
        mean = np.einsum("te,te->t", p, slope)
        d = np.where(valid[:, None], p * (slope - mean[:, None]), 0.0)
        dz = w * (dw - np.einsum("tk,tk->t", w, dw)[:, None])
        np.add.at(d, (np.arange(T)[:, None], idx.astype(np.int64)), dz)
        return d
    ids = s["ids"].long()
    if case["op"] == "embed":
        return torch.index_select(s["table"].double(), 0, ids) * s["scale"]
    keep = torch.nonzero(ids != s["pad"]).flatten()
    ids = ids[keep]
    total = s["dtable"].double()
    if not case["accumulate"]:
        total.zero_()
    order = torch.argsort(ids, stable=True)
    names, length = torch.unique_consecutive(ids[order], return_counts=True)
    rows = s["dout"][keep[order]].double()
    if names.numel():
        total[names] += torch.segment_reduce(rows, "sum", lengths=length, axis=0) * s["scale"]
    return total
