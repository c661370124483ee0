"""Cases that measure what a MoE layer's training and serving step does between and after the token movement.

Three families, each in a plain form of elementary torch operations (``own`` false) and as a user calls it (``own`` true):

    scored       routing by softmax or sigmoid scores with a balancing bias, groups of experts, top k and renormalised weights;
                 in training it adds up the pairs of each expert and moves the bias by them
    scored_grad  gradient of the router's logits from the gradient of the routing weights
    linear       the experts' products on expert-major rows, with bias, activation and residual in the epilogue
    linear_dx    their gradient towards the rows, times the derivative of the activation before it
    linear_dw    their gradient towards weights and bias
    update       norm of all gradients, clipping and an AdamW step over many tensors, moments in 32 or in 8 bits

Sizes come from the workloads of ``activation_paging_gb300/inputs.py`` (256 tokens over 8 experts, top 2; 8192 tokens over
128 experts, top 8, H = 2048; 32768 tokens over 256 experts, top 8); inner widths and tensor sizes are generic.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}
BLOCK = 256  # elements that share a scale of 8-bit moments; the parts of flat buffers begin at multiples of it


def _scored(name, T, E, k, score="sigmoid", bias=True, groups=1, top_groups=1, best=2, renorm=True, scale=1.0, pad=False,
            train=False, op="scored"):
    return {"name": name, "op": op, "T": T, "E": E, "k": k, "score": score, "bias": bias, "groups": groups,
            "top_groups": top_groups, "best": best, "renorm": renorm, "scale": scale, "pad": pad, "train": train}


def _linear(name, T, E, k, K, N, act="none", bias=False, residual=False, pre=False, padded=False, op="linear", out="bf16"):
    return {"name": name, "op": op, "T": T, "E": E, "k": k, "K": K, "N": N, "act": act, "bias": bias, "residual": residual,
            "pre": pre, "padded": padded, "out": out}


def _update(name, tensors, total, param="f32", grad="f32", master=False, bits=32, clip=True):
    return {"name": name, "op": "update", "tensors": tensors, "total": total, "param": param, "grad": grad,
            "master": master, "bits": bits, "clip": clip}


def listed():
    return [
        # one decoding step of 16 sequences: latency counts
        _scored("scored 16x256", 16, 256, 8, groups=8, top_groups=4, scale=2.5),
        # a training step's tokens, padded at the ends, with the counts and the bias moved by them
        _scored("scored 32768x256 train", 32768, 256, 8, groups=8, top_groups=4, scale=2.5, pad=True, train=True),
        # one chunk of a training step backwards, weights that are the chosen probabilities themselves
        _scored("scored grad 8192x128", 8192, 128, 8, "softmax", renorm=False, op="scored_grad"),
        # one decoding step of 4 sequences, gated experts
        _linear("experts 4 tokens", 4, 128, 8, 2048, 1024, "swiglu"),
        # one chunk of a training step: gate and up products, pre-activations kept for the way back
        _linear("experts 8192 swiglu", 8192, 128, 8, 2048, 1024, "swiglu", pre=True),
        # a small odd layer with everything in its epilogue, capacity-shaped rows
        _linear("experts 999 odd", 999, 60, 6, 1003, 517, "gelu", bias=True, residual=True, pre=True, padded=True),
        # the chunk backwards through the second product and the gate
        _linear("experts dx 8192", 8192, 128, 8, 1024, 2048, "swiglu", op="linear_dx"),
        # the chunk's gradient of the second product's weights, added to the kept gradient
        _linear("experts dw 8192", 8192, 128, 8, 1024, 2048, op="linear_dw", out="f32"),
        # a small batch over few experts, weights and bias
        _linear("experts dw 256", 256, 8, 2, 512, 512, bias=True, op="linear_dw", out="f32"),
        # the small tensors of a model (scales, biases, a router) alone: latency counts
        _update("update 48 small", 48, 400000),
        # a layer's weights in single precision with moments to match
        _update("update layer", 12, 67000000),
        # BF16 weights with a master copy, BF16 gradients and moments in 8 bits
        _update("update layer 8 bits", 12, 134000000, "bf16", "bf16", True, 8),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["scored", "scored", "scored_grad", "linear", "linear", "linear_dx", "linear_dw", "update", "update"])
    if op in ("scored", "scored_grad"):
        E = _log(rng, 4, 1024)
        T = _log(rng, 1, min(32768, 32768 * 256 // E))
        groups = rng.choice([1] + [g for g in range(2, 33) if E % g == 0 and E // g >= 2])
        k = rng.randint(1, min(E, 12))
        least = -(-k // (E // groups))
        top_groups = rng.randint(least, groups) if groups > 1 else 1
        case = _scored("", T, E, k, rng.choice(["sigmoid", "softmax"]), rng.random() < 0.7, groups, top_groups,
                       rng.choice([1, 2]), rng.random() < 0.7, rng.choice([1.0, 2.5]), rng.random() < 0.5,
                       rng.random() < 0.4, op)
    elif op == "update":
        param = rng.choice(["f32", "bf16"])
        case = _update("", _log(rng, 1, 200), _log(rng, 2000, 100000000), param, rng.choice(["f32", "bf16"]),
                       param == "bf16" and rng.random() < 0.7, rng.choice([8, 32]), rng.random() < 0.7)
    else:
        E = _log(rng, 1, 256)
        k = rng.randint(1, min(E, 8))
        odd = rng.random() < 0.3
        step = 1 if odd else 8
        K, N = (max(step, _log(rng, 32, 4096) // step * step) for _ in range(2))
        T = _log(rng, 1, 8192)
        act = rng.choice(["none", "silu", "gelu", "swiglu"]) if op != "linear_dw" else "none"
        while E * K * N * (2 if act == "swiglu" else 1) > 1 << 28:
            E = max(1, E // 2)
            k = min(k, E)
        most = 8.0e10 if odd else 5.0e11
        while 2.0 * T * k * K * N * (2 if act == "swiglu" else 1) > most:
            T //= 2
        case = _linear("", T, E, k, K, N, act, rng.random() < 0.5 and op != "linear_dx",
                       rng.random() < 0.4 and op != "linear_dw", rng.random() < 0.5 and op == "linear", rng.random() < 0.4, op,
                       rng.choice(["bf16", "bf16", "f32"]) if op != "linear_dw" else rng.choice(["bf16", "f32", "f32"]))
    del case["name"]
    return case


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 2654435761 % (1 << 62))


def _normal(g, *shape, scale=1.0, dtype=torch.float32):
    return torch.empty(*shape, device="cuda", dtype=dtype).normal_(0.0, scale, generator=g)


# ---- routing ------------------------------------------------------------------------------------------------------------

def _prepare_scored(case, g):
    T, E, k = case["T"], case["E"], case["k"]
    logits = _normal(g, T, E)
    rank = torch.randperm(E, generator=g, device="cuda").float() + 1
    logits -= 0.25 * torch.log(rank)  # some experts are preferred
    bias = _normal(g, E, scale=0.05 if case["score"] == "sigmoid" else 0.2 / E) if case["bias"] or case["train"] else None
    mask = None
    if case["pad"]:  # the last quarter or so is padding
        mask = torch.arange(T, device="cuda") < torch.rand((), generator=g, device="cuda") * 0.3 * T + 0.7 * T
    s = {"case": dict(case), "logits": logits, "bias": bias, "mask": mask}
    if case["train"]:
        s["counts"] = torch.zeros(E, dtype=torch.int32, device="cuda")
    if case["op"] == "scored_grad":
        s["idx"] = _choose(case, logits, bias)[0].int()
        s["dw"] = _normal(g, T, k, scale=0.1 / T)
    return s


def _scores(case, logits):
    """Scores in 64 bits: choices between near values need them."""
    x = logits.double()
    if case["score"] == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-x))
    z = torch.exp(x - x.amax(1, keepdim=True))
    return z / z.sum(1, keepdim=True)


def _choose(case, logits, bias):
    """(idx, scores): top k of score + bias in the best groups; ties go to the lowest index."""
    T, E, k, G = case["T"], case["E"], case["k"], case["groups"]
    s = _scores(case, logits)
    c = s + bias.double() if bias is not None else s
    if G > 1:
        by = torch.sort(c.view(T, G, E // G), dim=2, descending=True)[0][:, :, : case["best"]].sum(2)
        order = torch.sort(by, dim=1, descending=True, stable=True)[1][:, : case["top_groups"]]
        keep = torch.zeros(T, G, dtype=torch.bool, device=c.device).scatter_(1, order, True)
        c = torch.where(keep.repeat_interleave(E // G, 1), c, torch.full_like(c, -math.inf))
    return torch.sort(c, dim=1, descending=True, stable=True)[1][:, :k], s


def _run_scored(s):
    c = s["case"]
    idx, score = _choose(c, s["logits"], s["bias"])
    w = torch.gather(score, 1, idx)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    out = {"idx": idx.int(), "w": (w * c["scale"]).float()}
    if c["train"]:
        one = torch.ones(c["T"], dtype=torch.int32, device=idx.device) if s["mask"] is None else s["mask"].int()
        n = torch.zeros_like(s["counts"]).scatter_add_(0, idx.reshape(-1), one[:, None].expand(c["T"], c["k"]).reshape(-1))
        s["bias"] += 1e-3 * torch.sign(n.sum() - c["E"] * n).float()
        out |= {"counts": n, "bias": s["bias"]}
    return out


def _run_scored_grad(s):
    c, idx, dw = s["case"], s["idx"].long(), s["dw"]
    x = s["logits"]
    if c["score"] == "softmax" and not c["renorm"]:
        z = torch.exp(x - x.amax(1, keepdim=True))
        p = z / z.sum(1, keepdim=True)
        g = torch.zeros_like(x).scatter_add_(1, idx, dw * c["scale"])
        return p * (g - (p * g).sum(1, keepdim=True))
    l = torch.gather(x, 1, idx)
    if c["score"] == "softmax":
        z = torch.exp(l - l.amax(1, keepdim=True))
        w = z / z.sum(1, keepdim=True)
        d = c["scale"] * w * (dw - (w * dw).sum(1, keepdim=True))
    else:
        q = 1.0 / (1.0 + torch.exp(-l))
        one_less = 1.0 / (1.0 + torch.exp(l))
        if c["renorm"]:
            w = q / q.sum(1, keepdim=True)
            d = c["scale"] * w * one_less * (dw - (w * dw).sum(1, keepdim=True))
        else:
            d = c["scale"] * q * one_less * dw
    return torch.zeros_like(x).scatter_add_(1, idx, d)


# ---- the experts' products ----------------------------------------------------------------------------------------------

def _prepare_linear(case, g):
    T, E, k, K, N, op, act = (case[n] for n in ("T", "E", "k", "K", "N", "op", "act"))
    gates = _normal(g, T, E) - 0.25 * torch.log(torch.arange(1, E + 1, device="cuda").float())
    counts = torch.bincount(torch.sort(gates, dim=1, descending=True)[1][:, :k].reshape(-1), minlength=E)
    if case["padded"]:
        C = -(-5 * T * k // (4 * E))
        live, seg, rows = counts.clamp(max=C), torch.arange(E, device="cuda") * C, E * C
    else:
        live, seg, rows = counts, torch.cumsum(counts, 0) - counts, T * k
    s = {"case": dict(case), "seg": seg.int(), "live": live.int(), "most": int(live.max())}
    both = 2 if act == "swiglu" else 1
    if op == "linear":  # [rows, K] -> [rows, N]
        s["x"] = _normal(g, rows, K, dtype=torch.bfloat16)
        s["W"] = _normal(g, E, both * N, K, scale=K ** -0.5, dtype=torch.bfloat16)
        s["bias"] = _normal(g, E, both * N, scale=0.1) if case["bias"] else None
        wide, z = N, both * N
    elif op == "linear_dx":  # [rows, N] -> [rows, K], then through the activation that made those K
        s["x"] = _normal(g, rows, N, scale=1e-2, dtype=torch.bfloat16)
        s["W"] = _normal(g, E, N, K, scale=K ** -0.5, dtype=torch.bfloat16)
        wide, z = K, both * K
    else:
        s["x"] = _normal(g, rows, K, dtype=torch.bfloat16)
        s["dy"] = _normal(g, rows, N, scale=1e-2, dtype=torch.bfloat16)
        s["dW"] = _normal(g, E, N, K, scale=1e-2, dtype=DT[case["out"]])
        s["db"] = _normal(g, E, N, scale=1e-2) if case["bias"] else None
        return s
    s["residual"] = _normal(g, rows, wide, scale=1e-2 if op == "linear_dx" else 1.0, dtype=torch.bfloat16) if case["residual"] else None
    s["out"] = torch.zeros(rows, wide if op == "linear" else z, dtype=DT[case["out"]], device="cuda")
    if op == "linear":
        s["pre"] = torch.zeros(rows, z, dtype=torch.bfloat16, device="cuda") if case["pre"] else None
    else:
        s["pre"] = _normal(g, rows, z, dtype=torch.bfloat16) if act != "none" else None
    return s


def _at(s, rows):
    """(row [E, most] of each expert's place, whether it is live; for each row its place among those, and whether it is live)"""
    seg, live, most = s["seg"].long(), s["live"].long(), s["most"]
    at = torch.arange(most, device=seg.device)
    there = at[None, :] < live[:, None]
    row = (seg[:, None] + at[None, :]).clamp(max=rows - 1)
    place = torch.zeros(rows + 1, dtype=torch.int64, device=seg.device)
    place.scatter_(0, torch.where(there, row, rows).reshape(-1), torch.arange(1, there.numel() + 1, device=seg.device))
    place = place[:rows]
    return row, there, (place - 1).clamp(min=0), place > 0


def _gather(t, row, there):
    return torch.where(there[:, :, None], t[row].float(), torch.zeros((), device=t.device))


def _erf_cdf(x):
    return 0.5 * (1.0 + torch.erf(x * math.sqrt(0.5)))


def _run_linear(s):
    c, x = s["case"], s["x"]
    row, there, place, on = _at(s, x.shape[0])
    z = torch.matmul(_gather(x, row, there), s["W"].float().transpose(1, 2))
    if s["bias"] is not None:
        z = z + s["bias"][:, None, :]
    z = z.view(-1, z.shape[2])[place]
    if c["act"] == "swiglu":
        a, b = z[:, : c["N"]], z[:, c["N"]:]
        h = a / (1.0 + torch.exp(-a)) * b
    elif c["act"] == "silu":
        h = z / (1.0 + torch.exp(-z))
    elif c["act"] == "gelu":
        h = z * _erf_cdf(z)
    else:
        h = z
    if s["residual"] is not None:
        h = h + s["residual"].float()
    s["out"].copy_(torch.where(on[:, None], h.to(s["out"].dtype), s["out"]))
    if s["pre"] is not None:
        s["pre"].copy_(torch.where(on[:, None], z.to(torch.bfloat16), s["pre"]))
    return {"out": s["out"], "pre": s["pre"]}


def _run_linear_dx(s):
    c, dy = s["case"], s["x"]
    row, there, place, on = _at(s, dy.shape[0])
    d = torch.matmul(_gather(dy, row, there), s["W"].float())
    d = d.view(-1, d.shape[2])[place]
    if s["residual"] is not None:
        d = d + s["residual"].float()
    if c["act"] != "none":
        z = s["pre"].float()
        if c["act"] == "gelu":
            d = d * (_erf_cdf(z) + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi)))
        else:
            a = z[:, : c["K"]]
            q = 1.0 / (1.0 + torch.exp(-a))
            da = q * (1.0 + a * (1.0 - q))
            d = d * da if c["act"] == "silu" else torch.cat([d * z[:, c["K"]:] * da, d * a * q], 1)
    s["out"].copy_(torch.where(on[:, None], d.to(s["out"].dtype), s["out"]))
    return s["out"]


def _run_linear_dw(s):
    row, there, _, _ = _at(s, s["x"].shape[0])
    dy = _gather(s["dy"], row, there)
    s["dW"].copy_(s["dW"].float() + torch.matmul(dy.transpose(1, 2), _gather(s["x"], row, there)))
    if s["db"] is not None:
        s["db"] += dy.sum(1)
    return {"dW": s["dW"], "db": s["db"]}


# ---- the weights' update ------------------------------------------------------------------------------------------------

HYPER = {"lr": 1e-4, "betas": (0.9, 0.95), "eps": 1e-8, "weight_decay": 0.1}
MAX_NORM, SEED = 1.0, 11


def _sizes(case):
    """Elements of each tensor: a few large ones and many small, odd ones among them, about the total."""
    n, total = case["tensors"], case["total"]
    share = [(i % 7 + 1) ** 3 for i in range(n)]
    return [max(1, total * a // sum(share) + (3 if i % 5 == 2 else 0)) for i, a in enumerate(share)]


def _offsets(case):
    at, got = 0, []
    for n in _sizes(case):
        got.append((at, n))
        at += -(-n // BLOCK) * BLOCK
    return got, at


def _prepare_update(case, g):
    parts, flat = _offsets(case)
    used = torch.zeros(flat, dtype=torch.bool, device="cuda")
    for at, n in parts:
        used[at: at + n] = True

    def make(scale, dtype=torch.float32, positive=False):
        t = torch.empty(flat, device="cuda").normal_(0.0, 1.0, generator=g)
        t = t.square_().mul_(scale * scale).add_(0.1 * scale * scale) if positive else t.mul_(scale)
        return t.masked_fill_(~used, 0.0).to(dtype)
    spread = 1.0 / math.sqrt(case["total"])  # the gradients' norm is about 2: clipped
    p = make(0.02)
    s = {"case": dict(case), "parts": parts, "grad": make(2 * spread, DT[case["grad"]]), "step": 1000}
    s["master"] = p if case["master"] else None
    s["param"] = p.to(DT[case["param"]]) if case["master"] or case["param"] != "f32" else p
    m, v = make(0.5 * spread), make(spread, positive=True)
    if case["bits"] == 8:
        mb, rb = m.view(-1, BLOCK), v.sqrt_().view(-1, BLOCK)
        s["m_scale"], s["v_scale"] = mb.abs().amax(1) / 127 ** 2, rb.amax(1) / 255 ** 2
        s["m"] = (torch.sign(mb) * torch.sqrt(mb.abs() / s["m_scale"].clamp(min=1e-30)[:, None]).round_().clamp_(max=127)).to(torch.int8).view(-1)
        s["v"] = torch.sqrt(rb / s["v_scale"].clamp(min=1e-30)[:, None]).round_().clamp_(max=255).to(torch.uint8).view(-1)
    else:
        s["m"], s["v"], s["m_scale"], s["v_scale"] = m, v, None, None
    return s


def _views(flat, parts):
    return [flat[at: at + n] for at, n in parts]


def _mix(x):
    """A 32-bit mixing of integers (the finalizer of MurmurHash3), in 64-bit arithmetic."""
    x = (x ^ (x >> 16)) * 0x85EBCA6B & 0xFFFFFFFF
    x = (x ^ (x >> 13)) * 0xC2B2AE35 & 0xFFFFFFFF
    return x ^ (x >> 16)


def _noise(case, t, dev):
    """The 32 random bits of each element at step t: by the seed, the step, the tensor's number and the element's."""
    parts, flat = _offsets(case)
    start = torch.tensor([at for at, _ in parts], device=dev)
    which = torch.searchsorted(start, torch.arange(0, flat, BLOCK, device=dev), right=True) - 1
    key = _mix(which + _mix(torch.full_like(which, (SEED + 0x9E3779B9 * t) & 0xFFFFFFFF)) & 0xFFFFFFFF)
    at = torch.arange(flat, device=dev).view(-1, BLOCK) - start[which][:, None]
    return _mix((at * 0x9E3779B9 + key[:, None]) & 0xFFFFFFFF)


def _run_update(s):
    c = s["case"]
    g = s["grad"].float()
    scale = torch.ones((), device=g.device)
    norm = torch.sqrt((g.double() * g.double()).sum()).float()
    if c["clip"]:
        scale = torch.where(norm > MAX_NORM, MAX_NORM / norm, scale)
    s["step"] += 1
    t, (b1, b2) = s["step"], HYPER["betas"]
    g = g * scale
    eight = c["bits"] == 8
    if eight:
        cm, cv = s["m"].float().view(-1, BLOCK), s["v"].float().view(-1, BLOCK)
        m = (cm * cm.abs() * s["m_scale"][:, None]).view(-1)
        r = (cv * cv * s["v_scale"][:, None]).view(-1)
        v = r * r
    else:
        m, v = s["m"], s["v"]
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    p = (s["master"] if s["master"] is not None else s["param"]).float()
    step = HYPER["lr"] / (1 - b1 ** t)
    p = p * (1 - HYPER["lr"] * HYPER["weight_decay"]) - step * m / (torch.sqrt(v) * (1.0 / math.sqrt(1 - b2 ** t)) + HYPER["eps"])
    if s["master"] is not None:
        s["master"].copy_(p)
    s["param"].copy_(p)
    if not eight:
        s["m"].copy_(m)
        s["v"].copy_(v)
        return {"param": s["param"], "master": s["master"], "m": s["m"], "v": s["v"], "norm": norm}
    u = _noise(c, t, g.device)
    mb, rb = m.view(-1, BLOCK), torch.sqrt(v).view(-1, BLOCK)
    s["m_scale"].copy_(mb.abs().amax(1) * (1.0 / 127 ** 2))
    s["v_scale"].copy_(rb.amax(1) * (1.0 / 255 ** 2))
    zero = torch.zeros((), device=g.device)
    cm = torch.where(s["m_scale"][:, None] > 0, torch.sqrt(mb.abs() / s["m_scale"][:, None]), zero)
    cv = torch.where(s["v_scale"][:, None] > 0, torch.sqrt(rb / s["v_scale"][:, None]), zero)
    cm = torch.floor(cm + (u & 0xFFFF).float() * (1.0 / 65536)).clamp_(max=127) * torch.sign(mb)
    cv = torch.where(rb > 0, torch.floor(cv + (u >> 16).float() * (1.0 / 65536)).clamp_(min=1, max=255), zero)
    s["m"].copy_(cm.view(-1))
    s["v"].copy_(cv.view(-1))
    r = cv * cv * s["v_scale"][:, None]
    return {"param": s["param"], "master": s["master"], "m": (cm * cm.abs() * s["m_scale"][:, None]).to(torch.bfloat16).view(-1),
            "v": (r * r).to(torch.bfloat16).view(-1), "norm": norm}


# ---- the cases' functions -----------------------------------------------------------------------------------------------

def prepare(case, seed):
    g = _gen(seed)
    if case["op"].startswith("scored"):
        return _prepare_scored(case, g)
    return _prepare_update(case, g) if case["op"] == "update" else _prepare_linear(case, g)


def run(state):
    if own:
        return _run_own(state)
    return {"scored": _run_scored, "scored_grad": _run_scored_grad, "linear": _run_linear, "linear_dx": _run_linear_dx,
            "linear_dw": _run_linear_dw, "update": _run_update}[state["case"]["op"]](state)


def _run_own(s):
    import activation_paging_gb300 as ap

    c = s["case"]
    if c["op"] == "scored":
        if not c["train"]:
            idx, w = ap.route_scored(s["logits"], c["k"], score=c["score"], bias=s["bias"], groups=c["groups"],
                                     top_groups=c["top_groups"], group_best=c["best"], renorm=c["renorm"], scale=c["scale"])
            return {"idx": idx, "w": w}
        counts = torch.zeros_like(s["counts"])
        idx, w = ap.route_scored(s["logits"], c["k"], score=c["score"], bias=s["bias"], groups=c["groups"],
                                 top_groups=c["top_groups"], group_best=c["best"], renorm=c["renorm"], scale=c["scale"],
                                 mask=s["mask"], counts=counts)
        ap.route_bias_step(s["bias"], counts, 1e-3)
        return {"idx": idx, "w": w, "counts": counts, "bias": s["bias"]}
    if c["op"] == "scored_grad":
        return ap.route_scored_backward(s["logits"], s["idx"], s["dw"], score=c["score"], renorm=c["renorm"], scale=c["scale"])
    act = None if c.get("act") == "none" else c.get("act")
    if c["op"] == "linear":
        ap.expert_linear(s["x"], s["W"], s["seg"], s["live"], bias=s["bias"], act=act, residual=s["residual"], out=s["out"],
                         pre=s["pre"])
        return {"out": s["out"], "pre": s["pre"]}
    if c["op"] == "linear_dx":
        return ap.expert_linear_dx(s["x"], s["W"], s["seg"], s["live"], act=act, pre=s["pre"], residual=s["residual"],
                                   out=s["out"])
    if c["op"] == "linear_dw":
        ap.expert_linear_dw(s["dy"], s["x"], s["seg"], s["live"], dW=s["dW"], dbias=s["db"], accumulate=True)
        return {"dW": s["dW"], "db": s["db"]}
    opt = s.get("opt")
    if opt is None:  # the optimizer that a program keeps, over its parameters, gradients and moments
        state = {"m": s["m"], "v": s["v"], "step": torch.tensor([s["step"], 0], dtype=torch.int32, device="cuda")}
        if c["bits"] == 8:
            state |= {"m_scale": s["m_scale"], "v_scale": s["v_scale"]}
        opt = s["opt"] = ap.AdamW(_views(s["param"], s["parts"]), _views(s["grad"], s["parts"]),
                                  master=_views(s["master"], s["parts"]) if s["master"] is not None else None,
                                  state_bits=c["bits"], state=state, seed=SEED, **HYPER)
    norm = opt.grad_norm(MAX_NORM if c["clip"] else None)
    opt.step(scale=norm[1:])
    m, v = opt.moments(torch.bfloat16) if c["bits"] == 8 else (opt.state["m"], opt.state["v"])
    return {"param": s["param"], "master": s["master"], "m": m, "v": v, "norm": norm[0]}


def work(case):
    op = case["op"]
    if op.startswith("scored"):
        T, E, k = case["T"], case["E"], case["k"]
        if op == "scored":  # logits in; ids and weights out
            more = (4 * E * 3 if case["train"] else 4 * E if case["bias"] else 0) + (T if case["pad"] and case["train"] else 0)
            return {"bytes": 4 * T * E + 8 * T * k + more, "flops": 6 * T * E + 4 * T * k}
        dense = case["score"] == "softmax" and not case["renorm"]
        return {"bytes": 4 * T * E + 4 * T * (E if dense else k) + 8 * T * k, "flops": (8 * T * E if dense else 0) + 8 * T * k}
    if op == "update":
        n = sum(_sizes(case))
        each = BYTES[case["grad"]] + (16 if case["bits"] == 32 else 4 + 16 / BLOCK + 4)  # 8 bits: the moments' values too
        each += 8 + BYTES[case["param"]] if case["master"] else 2 * BYTES[case["param"]]
        return {"bytes": each * n, "flops": 20 * n}
    T, E, k, K, N = (case[n] for n in ("T", "E", "k", "K", "N"))
    rows = T * k  # at most: capacity-shaped rows may drop a few
    named = E * (1 - (1 - k / E) ** T)  # experts with rows, were they chosen evenly
    both = 2 if case["act"] == "swiglu" else 1
    if op == "linear":
        b = rows * (2 * K + BYTES[case["out"]] * N + (2 * both * N if case["pre"] else 0) + (2 * N if case["residual"] else 0))
        return {"bytes": b + 2 * named * both * N * K + (4 * E * both * N if case["bias"] else 0), "flops": 2 * rows * both * N * K}
    if op == "linear_dx":
        b = rows * (2 * N + BYTES[case["out"]] * both * K + (2 * both * K if case["act"] != "none" else 0) + (2 * K if case["residual"] else 0))
        return {"bytes": b + 2 * named * N * K, "flops": 2 * rows * N * K}
    return {"bytes": 2 * rows * (K + N) + 2 * named * N * K * BYTES[case["out"]], "flops": 2 * rows * N * K}


# ---- 64 bits ------------------------------------------------------------------------------------------------------------

def _exact_scored(case, s):
    x = s["logits"].double()
    q = torch.sigmoid(x) if case["score"] == "sigmoid" else torch.softmax(x, 1)
    if case["op"] == "scored":
        T, E, G = case["T"], case["E"], case["groups"]
        c = q if s["bias"] is None else q + s["bias"].double()
        best = torch.topk(c.view(T, G, E // G), case["best"], dim=2)[0].sum(2)
        least = torch.topk(best, case["top_groups"], dim=1)[0][:, -1:]
        c = c.view(T, G, E // G).masked_fill((best < least)[:, :, None], -math.inf).view(T, E)
        w = torch.gather(q, 1, torch.topk(c, case["k"], dim=1)[1])
        if case["renorm"]:
            w = w / w.sum(1, keepdim=True)
        got = {"idx": None, "w": w * case["scale"]}
        return got | {"counts": None, "bias": None} if case["train"] else got
    leaf = x.clone().requires_grad_()
    q = torch.sigmoid(leaf) if case["score"] == "sigmoid" else torch.softmax(leaf, 1)
    w = torch.gather(q, 1, s["idx"].long())
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True)
    (case["scale"] * w * s["dw"].double()).sum().backward()
    return leaf.grad


def _exact_linear(case, s):
    act, both, seg, live = case["act"], 2 if case["act"] == "swiglu" else 1, s["seg"].tolist(), s["live"].tolist()
    fn = {"none": lambda z: z, "silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu,
          "swiglu": lambda z: torch.nn.functional.silu(z[:, : z.shape[1] // 2]) * z[:, z.shape[1] // 2:]}[act]
    if case["op"] == "linear_dw":
        dW, db = s["dW"].double(), None if s["db"] is None else s["db"].double()
        for e, (a, n) in enumerate(zip(seg, live)):
            dy = s["dy"][a: a + n].double()
            dW[e] += dy.t() @ s["x"][a: a + n].double()
            if db is not None:
                db[e] += dy.sum(0)
        return {"dW": dW, "db": db}
    out = s["out"].double()
    pre = s["pre"].double() if s["pre"] is not None else None
    for e, (a, n) in enumerate(zip(seg, live)):
        at = slice(a, a + n)
        x, W = s["x"][at].double(), s["W"][e].double()
        add = 0.0 if s["residual"] is None else s["residual"][at].double()
        if case["op"] == "linear":
            z = x @ W.t() + (0.0 if s["bias"] is None else s["bias"][e].double())
            out[at] = fn(z) + add
            if pre is not None:
                pre[at] = z
        elif act == "none":
            out[at] = x @ W + add
        elif n:
            z = pre[at].clone().requires_grad_()
            (fn(z) * (x @ W + add)).sum().backward()
            out[at] = z.grad
    return {"out": out, "pre": pre} if case["op"] == "linear" else out


def _exact_update(case, s):
    g = s["grad"].double()
    norm = g.norm()
    if case["clip"] and float(norm) > MAX_NORM:
        g = g * (MAX_NORM / norm)
    (b1, b2), t, lr = HYPER["betas"], s["step"] + 1, HYPER["lr"]
    eight = case["bits"] == 8
    if eight:
        each = lambda scale: scale.double().repeat_interleave(BLOCK)  # noqa: E731
        m = s["m"].double() * s["m"].double().abs() * each(s["m_scale"])
        v = (s["v"].double().square() * each(s["v_scale"])).square()
    else:
        m, v = s["m"].double(), s["v"].double()
    m = torch.lerp(g, m, b1)
    v = torch.lerp(g * g, v, b2)
    p = (s["param"] if s["master"] is None else s["master"]).double()
    p = p - lr * (HYPER["weight_decay"] * p + m / (1 - b1 ** t) / ((v / (1 - b2 ** t)).sqrt() + HYPER["eps"]))
    got = {"param": p, "master": None if s["master"] is None else p, "m": m, "v": v, "norm": norm}
    if eight:
        u = _noise(case, t, g.device).view(-1)
        sm, sv = (x.view(-1, BLOCK).amax(1).repeat_interleave(BLOCK).clamp(min=1e-300) for x in (m.abs(), v.sqrt()))
        cm = ((m.abs() / sm).sqrt() * 127 + (u & 0xFFFF) / 65536.0).floor().clamp(max=127) / 127
        cv = ((v.sqrt() / sv).sqrt() * 255 + (u >> 16) / 65536.0).floor().clamp(1, 255) / 255
        got |= {"m": cm * cm * sm * m.sign(), "v": torch.where(v > 0, cv ** 4 * sv * sv, v)}
    return got


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("scored"):
        return _exact_scored(case, s)
    return _exact_update(case, s) if case["op"] == "update" else _exact_linear(case, s)
