"""GB300 token movement for a top-k MoE layer with a paged activation stash.

Thin Python binding of ``libap.so`` (C ABI in ``include/ap.h``).  Every step
runs in the library's CUDA kernels; this module only allocates tensors with
PyTorch (device memory, pinned host memory, streams) and passes their
addresses.  There is no CPU fallback: without the built library every call
raises.

    embed             rows of an embedding table, scaled (and embed_backward)
    route_topk        softmax -> top-k -> renormalised weights
    route_scored      top k by softmax or sigmoid scores, a balancing bias and groups
                      (and route_scored_backward, route_bias_step)
    route_balance     route_topk with a balance loss and per-expert counts
                      (and route_backward, the logits' gradient)
    expert_linear     the experts' products on dispatched rows, with bias,
                      activation and residual (and expert_linear_dx, _dw)
    dispatch_permute  expert-major, capacity-bounded permutation (BF16 / E4M3)
    Pool              paged stash: push / pop / reset / overflow read-out,
                      calibration and lazy growth (over an Arena)
    Arena             device memory that grows in place
    AdamW             the weights' update: gradient norm and clipping, a step over
                      many tensors, moments in 32 or 8 bits
    combine_unpermute top-k weighted un-permute to dense BF16 [T, H]
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import _lib
from ._lib import APError, PoolConfig, PoolState, RecordInfo, check

FLAG_POOL_OVERFLOW = 0x1
FLAG_SPILL_OVERFLOW = 0x2
FLAG_RECORD_OVERFLOW = 0x4
FLAG_BAD_COUNT = 0x8
FLAG_BAD_INDEX = 0x10
FLAG_CORRUPT = 0x20
DTYPE_BF16, DTYPE_E4M3, DTYPE_F32 = 0, 1, 2

__all__ = ["embed", "embed_backward", "embed_scratch_bytes", "route_balance", "route_balance_scratch_bytes",
           "route_backward", "route_scored", "route_scored_backward", "route_bias_step", "route_topk", "dispatch_permute",
           "dispatch_scratch_bytes", "combine_unpermute", "combine_backward", "dispatch_backward", "cast_e4m3", "expert_linear",
           "expert_linear_dx", "expert_linear_dw", "AdamW", "Pool", "Arena", "APError", "lib", "launch_count"]


def lib():
    return _lib.load()


def _stream(stream) -> int:
    if stream is not None:
        return stream.cuda_stream
    # the current stream's handle without a Stream object (a third of a call's host time)
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _p(t):
    return None if t is None else t.data_ptr()


def _need(t: torch.Tensor, dtype, name: str):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def route_topk(logits: torch.Tensor, k: int, idx: torch.Tensor | None = None, w: torch.Tensor | None = None,
               stream=None):
    """idx [T, k] int32 and w [T, k] float32 for float32 logits [T, E]."""
    _need(logits, torch.float32, "logits")
    T, E = logits.shape
    if idx is None:
        idx = torch.empty((T, k), dtype=torch.int32, device=logits.device)
    if w is None:
        w = torch.empty((T, k), dtype=torch.float32, device=logits.device)
    check(lib().ap_route_topk(_p(logits), T, E, k, _p(idx), _p(w), _stream(stream)), "route_topk")
    return idx, w


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    """A new tensor that belongs to the stream the call runs on, so that its memory is not handed
    out again before that stream is done with it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _groups(T: int, group_tokens: int) -> int:
    return -(-T // (group_tokens or T)) if T else 0


def _need_shape(t: torch.Tensor, dtype, shape: tuple, name: str) -> int:
    """_need, the shape too; returns the address."""
    if t.shape != shape or t.dtype != dtype or not t.is_cuda or not t.is_contiguous():
        _need(t, dtype, name)
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    return t.data_ptr()


def _mask(mask: torch.Tensor | None, T: int):
    if mask is None:
        return None
    if mask.dtype not in (torch.bool, torch.uint8):
        raise ValueError(f"mask must be bool or uint8, got {mask.dtype}")
    return _need_shape(mask, mask.dtype, (T,), "mask")


def _status(status: torch.Tensor | None):
    """Address of a status word: 32 bits on the GPU, of whatever type."""
    if status is None:
        return None
    if not status.is_cuda:
        raise ValueError("status must be a CUDA tensor")
    p = status.data_ptr()
    if status.numel() * status.element_size() < 4 or p & 3:
        raise ValueError("status must hold an aligned 32-bit word")
    return p


@functools.lru_cache(maxsize=1024)
def route_balance_scratch_bytes(T: int, E: int, group_tokens: int = 0) -> int:
    n = ctypes.c_int64(0)
    check(lib().ap_route_balance_scratch_bytes(T, E, group_tokens, ctypes.byref(n)), "route_balance_scratch_bytes")
    return n.value


def route_balance(logits: torch.Tensor, k: int, coef: float = 1.0, group_tokens: int = 0,
                  mask: torch.Tensor | None = None, out: dict | None = None, stream=None) -> dict:
    """``route_topk`` with the balance loss of each group of ``group_tokens``
    tokens (0: all tokens are one group): a dict of ``idx`` ([T, k] int32) and
    ``w`` ([T, k] float32) as route_topk's, ``counts`` ([G, E] int32, pairs per
    expert), ``prob`` ([G, E] float32, mean softmax probability), ``slope``
    ([G, E] float32, d loss / d p, for ``route_backward``), ``loss`` (float32
    scalar tensor, ``coef`` x the mean over groups of E sum_e share_e prob_e)
    and, for many tokens, ``scratch``.  ``mask`` ([T] bool or uint8): tokens that count.  Pass
    ``out`` (such a dict, whole or in part) to reuse buffers."""
    _need(logits, torch.float32, "logits")
    T, E = logits.shape
    m = _mask(mask, T)
    G = _groups(T, group_tokens)
    sb = route_balance_scratch_bytes(T, E, group_tokens)
    pairs, sums, dev = (T, k), (G, E), logits.device
    if out is None and stream is None:
        o = {"idx": torch.empty(pairs, dtype=torch.int32, device=dev),
             "w": torch.empty(pairs, dtype=torch.float32, device=dev),
             "counts": torch.empty(sums, dtype=torch.int32, device=dev),
             "prob": torch.empty(sums, dtype=torch.float32, device=dev),
             "slope": torch.empty(sums, dtype=torch.float32, device=dev),
             "loss": torch.empty((), dtype=torch.float32, device=dev)}
    else:
        o = dict(out) if out is not None else {}
        for name, shape, dtype in (("idx", pairs, torch.int32), ("w", pairs, torch.float32),
                                   ("counts", sums, torch.int32), ("prob", sums, torch.float32),
                                   ("slope", sums, torch.float32), ("loss", (), torch.float32)):
            if name in o:
                _need_shape(o[name], dtype, shape, name)
            else:
                o[name] = _empty(shape, dtype, dev, stream)
    scratch = o.get("scratch")
    if scratch is not None:
        _need(scratch, scratch.dtype, "scratch")
    if sb and (scratch is None or scratch.numel() < sb):
        scratch = o["scratch"] = _empty(sb, torch.uint8, dev, stream)
    check(lib().ap_route_balance(logits.data_ptr(), T, E, k, group_tokens, m, coef, o["idx"].data_ptr(),
                                 o["w"].data_ptr(), o["counts"].data_ptr(), o["prob"].data_ptr(),
                                 o["slope"].data_ptr(), o["loss"].data_ptr(), _p(scratch),
                                 scratch.numel() if scratch is not None else 0, _stream(stream)), "route_balance")
    return o


def route_backward(logits: torch.Tensor, idx: torch.Tensor | None = None, w: torch.Tensor | None = None,
                   dw: torch.Tensor | None = None, slope: torch.Tensor | None = None,
                   dloss: torch.Tensor | None = None, group_tokens: int = 0, mask: torch.Tensor | None = None,
                   dlogits: torch.Tensor | None = None, status: torch.Tensor | None = None, stream=None):
    """dlogits [T, E] float32 from the gradient ``dw`` of the routing weights
    (with the forward pass's ``idx`` and ``w``) and from the balance loss (with
    its ``slope`` and, if not 1, ``dloss``); either may be left out."""
    _need(logits, torch.float32, "logits")
    T, E = logits.shape
    m = _mask(mask, T)
    k, pi, pw, pdw, ps, pl = 1, None, None, None, None, None
    if dw is not None:
        if idx is None or w is None:
            raise ValueError("dw needs idx and w")
        if dw.dim() != 2:
            raise ValueError(f"dw must be [T, k], got {list(dw.shape)}")
        k = dw.shape[1]
        pdw = _need_shape(dw, torch.float32, (T, k), "dw")
        pi = _need_shape(idx, torch.int32, (T, k), "idx")
        pw = _need_shape(w, torch.float32, (T, k), "w")
    if slope is not None:
        ps = _need_shape(slope, torch.float32, (_groups(T, group_tokens), E), "slope")
    if dloss is not None:
        _need(dloss, torch.float32, "dloss")
        if dloss.numel() != 1:
            raise ValueError("dloss must hold one value")
        pl = dloss.data_ptr()
    if dlogits is None:
        dlogits = _empty((T, E), torch.float32, logits.device, stream)
    else:
        _need_shape(dlogits, torch.float32, (T, E), "dlogits")
    check(lib().ap_route_backward(_p(logits), T, E, k, pi, pw, pdw, ps, pl, group_tokens, m, _p(dlogits), _status(status),
                                  _stream(stream)), "route_backward")
    return dlogits


_SCORES = {"softmax": 0, "sigmoid": 1}


def _score(score: str) -> int:
    kind = _SCORES.get(score)
    if kind is None:
        raise ValueError(f"score must be 'softmax' or 'sigmoid', got {score!r}")
    return kind


def route_scored(logits: torch.Tensor, k: int, score: str = "sigmoid", bias: torch.Tensor | None = None, groups: int = 1,
                 top_groups: int = 1, group_best: int = 2, renorm: bool = True, scale: float = 1.0,
                 mask: torch.Tensor | None = None, counts: torch.Tensor | None = None, idx: torch.Tensor | None = None,
                 w: torch.Tensor | None = None, stream=None):
    """``idx`` [T, k] int32 and ``w`` [T, k] float32 for float32 logits [T, E]:
    the k largest of score + ``bias`` ([E] float32) in the ``top_groups`` of
    ``groups`` groups of experts whose ``group_best`` (1 or 2) largest have the
    largest sum.  The weights are the chosen scores themselves (``softmax`` or
    ``sigmoid`` of the logits), with ``renorm`` divided by their sum, times
    ``scale``.  ``counts`` ([E] int32): the pairs of each expert are added to
    it, of tokens that ``mask`` ([T] bool or uint8) lets count; see
    ``route_bias_step``."""
    kind = _score(score)
    _need(logits, torch.float32, "logits")
    T, E = logits.shape
    m = _mask(mask, T)
    if groups == 1:
        group_best = 1
    pb = None if bias is None else _need_shape(bias, torch.float32, (E,), "bias")
    pc = None if counts is None else _need_shape(counts, torch.int32, (E,), "counts")
    pairs = (T, k)
    if idx is None:
        idx = _empty(pairs, torch.int32, logits.device, stream)
    else:
        _need_shape(idx, torch.int32, pairs, "idx")
    if w is None:
        w = _empty(pairs, torch.float32, logits.device, stream)
    else:
        _need_shape(w, torch.float32, pairs, "w")
    check(lib().ap_route_scored(logits.data_ptr(), T, E, k, kind, pb, groups, top_groups, group_best, 1 if renorm else 0, scale,
                                m, idx.data_ptr(), w.data_ptr(), pc, _stream(stream)), "route_scored")
    return idx, w


def route_scored_backward(logits: torch.Tensor, idx: torch.Tensor, dw: torch.Tensor, score: str = "sigmoid",
                          renorm: bool = True, scale: float = 1.0, dlogits: torch.Tensor | None = None,
                          status: torch.Tensor | None = None, stream=None, w: torch.Tensor | None = None) -> torch.Tensor:
    """dlogits [T, E] float32 of ``route_scored`` from the gradient ``dw``
    [T, k] of its weights.  ``w``: the weights themselves, needed where rows may
    have fewer than k experts to choose from (logits or biases of -infinity):
    those chosen for want of others have weight 0, and no gradient."""
    kind = _score(score)
    _need(logits, torch.float32, "logits")
    T, E = logits.shape
    if dw.dim() != 2:
        raise ValueError(f"dw must be [T, k], got {list(dw.shape)}")
    k = dw.shape[1]
    pw = _need_shape(dw, torch.float32, (T, k), "dw")
    pi = _need_shape(idx, torch.int32, (T, k), "idx")
    p = None if w is None else _need_shape(w, torch.float32, (T, k), "w")
    if dlogits is None:
        dlogits = _empty((T, E), torch.float32, logits.device, stream)
    else:
        _need_shape(dlogits, torch.float32, (T, E), "dlogits")
    check(lib().ap_route_scored_backward_weighted(logits.data_ptr(), T, E, k, pi, pw, p, kind, 1 if renorm else 0, scale,
                                                  dlogits.data_ptr(), _status(status), _stream(stream)), "route_scored_backward")
    return dlogits


def route_bias_step(bias: torch.Tensor, counts: torch.Tensor, rate: float, reset: bool = False, stream=None) -> torch.Tensor:
    """Moves ``bias`` ([E] float32) by ``rate`` up where an expert has fewer
    than its share of ``counts`` ([E] int32), down where more; ``reset`` zeroes
    the counts."""
    _need(bias, torch.float32, "bias")
    if bias.dim() != 1:
        raise ValueError("bias must be [E]")
    E = bias.shape[0]
    check(lib().ap_route_bias_step(bias.data_ptr(), _need_shape(counts, torch.int32, (E,), "counts"), E, rate,
                                   1 if reset else 0, _stream(stream)), "route_bias_step")
    return bias


_ROW_TYPES = {torch.bfloat16: DTYPE_BF16, torch.float32: DTYPE_F32}


def _rows(t: torch.Tensor, name: str):
    """(n, H, distance of rows, type) of BF16 or FP32 rows [n, H], each contiguous; they may lie apart."""
    kind = _ROW_TYPES.get(t.dtype)
    if kind is None:
        raise ValueError(f"{name} must be bfloat16 or float32, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != 2:
        raise ValueError(f"{name} must be [rows, H]")
    (n, H), (pitch, step) = t.shape, t.stride()
    if pitch < H:
        if n > 1:
            raise ValueError(f"{name} must have rows that do not overlap")
        pitch = H
    if step != 1 and H > 1:
        raise ValueError(f"{name} must have contiguous rows")
    return n, H, pitch, kind


def _ids(ids: torch.Tensor):
    """(T, bytes of an id)"""
    size = 8 if ids.dtype == torch.int64 else 4 if ids.dtype == torch.int32 else 0
    if not size:
        raise ValueError(f"ids must be int32 or int64, got {ids.dtype}")
    _need(ids, ids.dtype, "ids")
    if ids.dim() != 1:
        raise ValueError("ids must be [T]")
    return ids.shape[0], size


def embed(table: torch.Tensor, ids: torch.Tensor, scale: float = 1.0, dtype: torch.dtype | None = None,
          out: torch.Tensor | None = None, status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """out[t] = scale * table[ids[t]]: [T, H] of ``dtype`` (default: the
    table's) for a BF16 or FP32 table [V, H] and int32 or int64 ids [T].  Rows
    of table and out may lie apart.  An id outside [0, V) gives zeros and sets
    FLAG_BAD_INDEX in ``status``."""
    V, H, ld, kind = _rows(table, "table")
    T, size = _ids(ids)
    if out is None:
        out_ld, out_kind = H, kind if dtype is None else _ROW_TYPES.get(dtype)
        if out_kind is None:
            raise ValueError(f"dtype must be bfloat16 or float32, got {dtype}")
        out = _empty((T, H), table.dtype if dtype is None else dtype, table.device, stream)
    else:
        n, h, out_ld, out_kind = _rows(out, "out")
        if n != T or h != H:
            raise ValueError(f"out must be {[T, H]}, got {[n, h]}")
    check(lib().ap_embed(_p(table), V, ld, kind, _p(ids), size, T, H, scale, _p(out), out_ld, out_kind, _status(status),
                         _stream(stream)), "embed")
    return out


@functools.lru_cache(maxsize=1024)
def embed_scratch_bytes(T: int, V: int, H: int) -> int:
    n = ctypes.c_int64(0)
    check(lib().ap_embed_scratch_bytes(T, V, H, ctypes.byref(n)), "embed_scratch_bytes")
    return n.value


def embed_backward(dout: torch.Tensor, ids: torch.Tensor, V: int, scale: float = 1.0, padding_idx: int | None = None,
                   dtable: torch.Tensor | None = None, accumulate: bool = False, dtype: torch.dtype = torch.float32,
                   scratch: torch.Tensor | None = None, status: torch.Tensor | None = None,
                   stream=None) -> torch.Tensor:
    """Gradient of ``embed``'s table: dtable [V, H], for every id the sum of its
    tokens' rows of dout [T, H] times ``scale`` (FP32 sums), written whole or,
    with ``accumulate``, added to ``dtable``.  Tokens whose id is
    ``padding_idx`` add nothing.  ``scratch``: a uint8 tensor of
    ``embed_scratch_bytes(T, V, H)`` bytes to reuse.  An id outside [0, V) adds
    nothing and sets FLAG_BAD_INDEX in ``status``.  FLAG_CORRUPT there says that
    rows did not arrive in the kernel; the ids that lack them hold NaN then,
    with ``status`` or without."""
    n, H, ld, kind = _rows(dout, "dout")
    T, size = _ids(ids)
    if n != T:
        raise ValueError(f"dout has {n} rows for {T} ids")
    if dtable is None:
        if accumulate:
            raise ValueError("accumulate needs dtable")
        dtable = _empty((V, H), dtype, dout.device, stream)
    v, h, g_ld, g_kind = _rows(dtable, "dtable")
    if v != V or h != H:
        raise ValueError(f"dtable must be {[V, H]}, got {[v, h]}")
    if scratch is not None:
        _need(scratch, torch.uint8, "scratch")
    else:
        sb = embed_scratch_bytes(T, V, H)
        if sb:
            scratch = _empty(sb, torch.uint8, dout.device, stream)
    check(lib().ap_embed_backward(_p(dout), ld, kind, _p(ids), size, T, H, V,
                                  -1 if padding_idx is None else padding_idx, scale, 1 if accumulate else 0, _p(dtable),
                                  g_ld, g_kind, _p(scratch), scratch.numel() if scratch is not None else 0,
                                  _status(status), _stream(stream)), "embed_backward")
    return dtable


_ROUNDINGS = {"codes": 0, "values": 1}


class AdamW:
    """AdamW over many tensors at once: one launch for the step, whatever their
    number (up to 440), with the step's number, the clipping factor and what
    skips the step on the GPU, so that steps are captured and replayed.

    ``params`` (BF16 or FP32, one type) and ``grads`` (BF16 or FP32, one type):
    lists of contiguous CUDA tensors; the optimizer keeps them, reads the
    gradients and writes the parameters at each step (``bind`` changes the
    gradients).  ``master``: FP32 copies of BF16 parameters, as a list or True
    (made here).  ``state_bits`` 32 or 8 (see ``ap_adamw_step``).  ``rounding`` of
    8-bit moments, at random: 'codes', fair between codes, which keeps moments
    far below their block's largest too large (of 1e-4 of it by a fifth), or
    'values', whose expectations are the moments.  Moments are
    flat buffers in which tensor i begins at element ``parts[i][0]``, a multiple
    of 256; ``state`` gives them with the step words (a checkpoint, or buffers
    to use): ``m``, ``v`` (float32, or int8 and uint8 with float32 ``m_scale``
    and ``v_scale``, one for each 256 elements) and ``step`` (int32 [2]: steps
    taken, 0).  All of them are used where they were when the optimizer was made
    (gradients: when they were bound): a call refuses tensors that have moved
    since (``p.data = ...``, another tensor in ``state``), so copy into them, or
    make a new optimizer with ``state``.  A captured graph does not look again.
    The calls of one optimizer are to follow one another (one stream, or events
    between)."""

    BLOCK = 256

    def __init__(self, params, grads, lr: float = 1e-3, betas=(0.9, 0.999), eps: float = 1e-8, weight_decay: float = 0.01,
                 master=None, state_bits: int = 32, state: dict | None = None, seed: int = 0, rounding: str = "codes"):
        self.params, self.lr = list(params), lr
        if not self.params:
            raise ValueError("params is empty")
        if state_bits not in (8, 32):
            raise ValueError(f"state_bits must be 8 or 32, got {state_bits}")
        if rounding not in _ROUNDINGS:
            raise ValueError(f"rounding must be 'codes' or 'values', got {rounding!r}")
        kind, dev = self.params[0].dtype, self.params[0].device
        if kind not in _ROW_TYPES:
            raise ValueError(f"params must be bfloat16 or float32, got {kind}")
        for i, p in enumerate(self.params):
            if p.dtype != kind or not p.is_cuda or not p.is_contiguous():
                _need(p, kind, f"params[{i}]")
        if master is True:
            master = [p.float() for p in self.params]
        self.master = None if master is None or master is False else list(master)
        if self.master is not None:
            if kind != torch.bfloat16:
                raise ValueError("master copies are of bfloat16 params")
            if len(self.master) != len(self.params):
                raise ValueError(f"{len(self.master)} master copies for {len(self.params)} params")
            for i, (p, q) in enumerate(zip(self.params, self.master)):
                _need_shape(q, torch.float32, p.shape, f"master[{i}]")
        self._apart(self.params + (self.master or []))
        self.parts, at = [], 0
        for p in self.params:
            self.parts.append((at, p.numel()))
            at += -(-p.numel() // self.BLOCK) * self.BLOCK
        self.state, self.state_bits, eight = dict(state or {}), state_bits, state_bits == 8
        need = {"m": (torch.int8 if eight else torch.float32, (at,)), "v": (torch.uint8 if eight else torch.float32, (at,)),
                "step": (torch.int32, (2,))}
        if eight:
            need |= {n: (torch.float32, (at // self.BLOCK,)) for n in ("m_scale", "v_scale")}
        for name, (dtype, shape) in need.items():
            if name in self.state:
                _need_shape(self.state[name], dtype, shape, "state " + name)
            else:
                self.state[name] = torch.zeros(shape, dtype=dtype, device=dev)
        self._apart([self.state[n] for n in need])
        self._names = list(need)
        self._held = self._hold(self._written())
        self._table = (_lib.AdamWTensor * len(self.params))()
        size = self.state["m"].element_size()
        at = {n: self.state[n].data_ptr() for n in need}
        for i, (p, (off, n)) in enumerate(zip(self.params, self.parts)):
            e = self._table[i]
            e.param, e.n, e.m, e.v = self._held[0][i], n, at["m"] + off * size, at["v"] + off * size
            if eight:
                e.m_scale, e.v_scale = at["m_scale"] + off // self.BLOCK * 4, at["v_scale"] + off // self.BLOCK * 4
            if self.master is not None:
                e.master = self.master[i].data_ptr()
        self._cfg = _lib.AdamWConfig(lr=lr, beta1=betas[0], beta2=betas[1], eps=eps, weight_decay=weight_decay,
                                     param_dtype=_ROW_TYPES[kind], master=1 if self.master is not None else 0,
                                     state_bits=state_bits, seed=seed & 0xFFFFFFFF, rounding=_ROUNDINGS[rounding], d_step=at["step"])
        self._cfg_ref = ctypes.byref(self._cfg)
        self.bind(grads)
        n = ctypes.c_int64(0)
        check(lib().ap_grad_norm_scratch_bytes(self._table, len(self._table), ctypes.byref(n)), "grad_norm_scratch_bytes")
        self._scratch_bytes = n.value
        self._scratch = torch.empty(n.value, dtype=torch.uint8, device=dev)
        self._norm = torch.empty(2, dtype=torch.float32, device=dev)

    def _written(self):
        """What a step writes."""
        return [*self.params, *(self.master or ()), *map(self.state.__getitem__, self._names)]

    @staticmethod
    def _hold(tensors):
        """(addresses, their indices, storages): as long as these are held, an address stays that of the same memory."""
        return list(map(torch.Tensor.data_ptr, tensors)), list(range(len(tensors))), [t.untyped_storage() for t in tensors]

    @staticmethod
    def _stay(tensors, held) -> bool:
        """Whether tensors are where the table has them (one call compares all: 32 ns each, 61 by data_ptr())."""
        at, all_of, _ = held
        return len(tensors) == len(at) and torch._C._tensors_data_ptrs_at_indices_equal(tensors, at, all_of)

    def _stay_written(self):
        if not self._stay(self._written(), self._held):
            raise ValueError("params, master copies or state have moved since the optimizer was made: copy into them, or make "
                             "a new optimizer")

    def _stay_grads(self):
        if not self._stay(self.grads, self._grads_held):
            raise ValueError("grads have moved since they were bound: bind them again")

    @staticmethod
    def _apart(tensors):
        """Refuses tensors that share memory: each is written by threads of its own."""
        spans = sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in tensors if t.numel())
        for (_, end), (start, _) in zip(spans, spans[1:]):
            if start < end:
                raise ValueError("params, master copies and moments must not share memory")

    def bind(self, grads):
        """The gradients of later steps: contiguous tensors of the parameters' shapes."""
        grads = list(grads)
        if len(grads) != len(self.params):
            raise ValueError(f"{len(grads)} grads for {len(self.params)} params")
        kind = grads[0].dtype
        if kind not in _ROW_TYPES:
            raise ValueError(f"grads must be bfloat16 or float32, got {kind}")
        for i, (p, g) in enumerate(zip(self.params, grads)):
            if g.shape != p.shape or g.dtype != kind or not g.is_cuda or not g.is_contiguous():
                _need_shape(g, kind, p.shape, f"grads[{i}]")
        held = self._hold(grads)
        for e, p in zip(self._table, held[0]):
            e.grad = p
        self.grads, self._cfg.grad_dtype = grads, _ROW_TYPES[kind]
        self._grads_held = held

    @staticmethod
    def _word(t, name: str):
        """Address of one float32 on the GPU."""
        if t is None:
            return None
        if t.dtype != torch.float32 or not t.is_cuda or t.numel() != 1:
            raise ValueError(f"{name} must be one float32 on the GPU")
        return t.data_ptr()

    def grad_norm(self, max_norm: float | None = None, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """[norm of all gradients, factor that clips it to ``max_norm``] (float32 [2]; the factor is 1 without clipping,
        NaN where the norm is not finite): pass ``out[1:]`` as ``scale`` to ``step``.  Without ``out`` the tensor is the
        optimizer's own, which the next call writes again."""
        self._stay_grads()
        if max_norm is not None and not max_norm > 0:
            raise ValueError(f"max_norm must be positive, got {max_norm}")
        if out is None:
            out = self._norm
        else:
            _need_shape(out, torch.float32, (2,), "out")
        check(lib().ap_grad_norm(self._table, len(self._table), self._cfg.grad_dtype, max_norm or 0.0, out.data_ptr(),
                                 self._scratch.data_ptr(), self._scratch_bytes, _stream(stream)), "grad_norm")
        return out

    def step(self, lr=None, scale: torch.Tensor | None = None, skip=None, stream=None):
        """One step.  ``lr``: a number or one float32 on the GPU (default: the optimizer's); ``scale``: one float32 on
        the GPU that multiplies the gradients, and skips the step where it is not finite; ``skip``: a 32-bit word on the
        GPU, or a ``Pool`` (its sticky flags): not 0 skips the step.  A skipped step changes nothing.  The word is read
        once for the whole step; to see the overflow of a pool's pushes, come after them (``stream=pool.stream``, or an
        event)."""
        self._stay_grads()
        self._stay_written()
        c = self._cfg
        if isinstance(lr, torch.Tensor):
            c.d_lr = self._word(lr, "lr")
        else:
            c.d_lr, c.lr = None, self.lr if lr is None else lr
        c.d_scale = self._word(scale, "scale")
        c.d_skip = skip.flags_device_ptr() if isinstance(skip, Pool) else _status(skip)
        check(lib().ap_adamw_step(self._table, len(self._table), self._cfg_ref, _stream(stream)), "adamw_step")

    def moments(self, dtype: torch.dtype = torch.float32, out=None, stream=None):
        """(m, v): the moments' values as flat float32 (or bfloat16) tensors; ``state``'s own where they are that already."""
        self._stay_written()
        s, n = self.state, self.state["m"].numel()
        if self.state_bits == 32:
            if dtype != torch.float32 or out is not None:
                raise ValueError("moments of 32 bits are state['m'] and state['v']")
            return s["m"], s["v"]
        if dtype not in _ROW_TYPES:
            raise ValueError(f"dtype must be bfloat16 or float32, got {dtype}")
        m, v = out if out is not None else (_empty((n,), dtype, s["m"].device, stream) for _ in range(2))
        check(lib().ap_adamw_moments(s["m"].data_ptr(), s["v"].data_ptr(), s["m_scale"].data_ptr(), s["v_scale"].data_ptr(), n,
                                     _ROW_TYPES[dtype], _need_shape(m, dtype, (n,), "m"), _need_shape(v, dtype, (n,), "v"),
                                     _stream(stream)), "adamw_moments")
        return m, v


_ACTS = {None: 0, "silu": 1, "gelu": 2, "swiglu": 3}


def _act(act) -> int:
    kind = _ACTS.get(act)
    if kind is None:
        raise ValueError(f"act must be None, 'silu', 'gelu' or 'swiglu', got {act!r}")
    return kind


def _rows16(t: torch.Tensor, name: str, shape: tuple | None = None):
    """(address, distance of rows) of BF16 rows that may lie apart."""
    n, H, pitch, kind = _rows(t, name)
    if kind != DTYPE_BF16:
        raise ValueError(f"{name} must be bfloat16, got {t.dtype}")
    if shape is not None and (n, H) != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {[n, H]}")
    return t.data_ptr(), pitch


def _segments(seg_off: torch.Tensor, live: torch.Tensor):
    _need(seg_off, torch.int32, "seg_off")
    if seg_off.dim() != 1:
        raise ValueError("seg_off must be [E]")
    E = seg_off.shape[0]
    return E, seg_off.data_ptr(), _need_shape(live, torch.int32, (E,), "live")


def _weights(W: torch.Tensor, E: int):
    """(N, K, distance of rows, distance of experts) of BF16 weights [E, N, K]."""
    if W.dtype != torch.bfloat16 or not W.is_cuda:
        raise ValueError(f"W must be a bfloat16 CUDA tensor, got {W.dtype}")
    if W.dim() != 3 or W.shape[0] != E:
        raise ValueError(f"W must be [{E}, N, K], got {list(W.shape)}")
    (_, N, K), (apart, pitch, step) = W.shape, W.stride()
    if step != 1 and K > 1:
        raise ValueError("W must have contiguous rows")
    return N, K, max(pitch, K) if N == 1 else pitch, apart


def _out_rows(out, rows: int, cols: int, dtype, device, stream, name: str):
    """(tensor, distance of rows, type) of BF16 or FP32 result rows, made here if not given."""
    if out is None:
        kind = DTYPE_BF16 if dtype is None else _ROW_TYPES.get(dtype)
        if kind is None:
            raise ValueError(f"dtype must be bfloat16 or float32, got {dtype}")
        return _empty((rows, cols), torch.bfloat16 if dtype is None else dtype, device, stream), cols, kind
    n, H, pitch, kind = _rows(out, name)
    if (n, H) != (rows, cols):
        raise ValueError(f"{name} must be {[rows, cols]}, got {[n, H]}")
    return out, pitch, kind


def _expert_scratch(scratch, a, lda, rows_a, cols_a, b, ldb, lde, rows_b, cols_b, device, stream):
    """(tensor, bytes) of the work space for operands that do not lie on 16-byte boundaries: none, as a rule."""
    if scratch is not None:
        _need(scratch, torch.uint8, "scratch")
        return scratch, scratch.numel()
    if not ((a | b) & 15 or (lda | ldb | lde) & 7):
        return None, 0
    n = ctypes.c_int64(0)
    check(lib().ap_expert_linear_scratch_bytes(a, lda, rows_a, cols_a, b, ldb, lde, rows_b, cols_b, ctypes.byref(n)),
          "expert_linear_scratch_bytes")
    return (_empty((n.value,), torch.uint8, device, stream), n.value) if n.value else (None, 0)


def expert_linear(x: torch.Tensor, W: torch.Tensor, seg_off: torch.Tensor, live: torch.Tensor,
                  bias: torch.Tensor | None = None, act: str | None = None, residual: torch.Tensor | None = None,
                  out: torch.Tensor | None = None, pre: torch.Tensor | None = None, dtype: torch.dtype | None = None,
                  scratch: torch.Tensor | None = None, status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """out[r] = act(x[r] W[e]^T + bias[e]) + residual[r] for the rows r of each
    expert e: ``live[e]`` rows from ``seg_off[e]`` ([E] int32 on the GPU, as the
    dispatch leaves them; the counts are read there).  x [rows, K] BF16, W [E, N, K]
    BF16, bias [E, N] float32, residual [rows, N] BF16, out [rows, N] BF16 (or
    float32: ``dtype``).  ``act``: None, 'silu', 'gelu', or 'swiglu' with W
    [E, 2 N, K], silu of the first N columns times the others.  ``pre``: a BF16
    tensor that receives the values before the activation, for
    ``expert_linear_dx``.  Rows may lie apart; rows of no expert are not written.
    ``scratch``: a uint8 tensor to reuse where rows do not lie on 16-byte
    boundaries (they are copied to such)."""
    E, ps, pl = _segments(seg_off, live)
    wide, K, ldw, lde = _weights(W, E)
    kind = _act(act)
    rows = x.shape[0]
    px, ldx = _rows16(x, "x", (rows, K))
    if kind == 3 and wide % 2:
        raise ValueError(f"W must have an even number of rows for swiglu, got {wide}")
    N = wide // 2 if kind == 3 else wide
    pb = None if bias is None else _need_shape(bias, torch.float32, (E, wide), "bias")
    pr, ldr = (None, 0) if residual is None else _rows16(residual, "residual", (rows, N))
    pp, ldp = (None, 0) if pre is None else _rows16(pre, "pre", (rows, wide))
    out, ldo, okind = _out_rows(out, rows, N, dtype, x.device, stream, "out")
    pw = W.data_ptr()
    scratch, sb = _expert_scratch(scratch, px, ldx, rows, K, pw, ldw, lde, E * wide, K, x.device, stream)
    check(lib().ap_expert_linear(px, ldx, rows, E, N, K, ps, pl, pw, ldw, lde, pb, kind, pr, ldr, pp, ldp, out.data_ptr(), ldo,
                                 okind, _p(scratch), sb, _status(status), _stream(stream)), "expert_linear")
    return out


def expert_linear_dx(dy: torch.Tensor, W: torch.Tensor, seg_off: torch.Tensor, live: torch.Tensor, act: str | None = None,
                     pre: torch.Tensor | None = None, residual: torch.Tensor | None = None, out: torch.Tensor | None = None,
                     dtype: torch.dtype | None = None, scratch: torch.Tensor | None = None,
                     status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Gradient of ``expert_linear``'s rows: (dy[r] W[e] + residual[r]) times the
    derivative of the activation ``act`` that made them, at ``pre``, from which
    they were made ([rows, K] BF16; 'swiglu': [rows, 2 K], as the result then)."""
    E, ps, pl = _segments(seg_off, live)
    N, K, ldw, lde = _weights(W, E)
    kind = _act(act)
    rows = dy.shape[0]
    py, ldy = _rows16(dy, "dy", (rows, N))
    wide = 2 * K if kind == 3 else K
    if kind and pre is None:
        raise ValueError("act needs pre")
    pp, ldp = _rows16(pre, "pre", (rows, wide)) if kind else (None, 0)
    pr, ldr = (None, 0) if residual is None else _rows16(residual, "residual", (rows, K))
    out, ldo, okind = _out_rows(out, rows, wide, dtype, dy.device, stream, "out")
    pw = W.data_ptr()
    scratch, sb = _expert_scratch(scratch, py, ldy, rows, N, pw, ldw, lde, E * N, K, dy.device, stream)
    check(lib().ap_expert_linear_dx(py, ldy, rows, E, N, K, ps, pl, pw, ldw, lde, kind, pp, ldp, pr, ldr, out.data_ptr(), ldo,
                                    okind, _p(scratch), sb, _status(status), _stream(stream)), "expert_linear_dx")
    return out


def expert_linear_dw(dy: torch.Tensor, x: torch.Tensor | None, seg_off: torch.Tensor, live: torch.Tensor,
                     dW: torch.Tensor | bool | None = None, dbias: torch.Tensor | None = None, accumulate: bool = False,
                     dtype: torch.dtype = torch.float32, scratch: torch.Tensor | None = None,
                     status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Gradient of ``expert_linear``'s weights: dW[e] = the sum of dy[r]^T x[r]
    over the expert's rows ([E, N, K] float32 or BF16), written whole or, with
    ``accumulate``, added to ``dW``; likewise ``dbias`` ([E, N] float32) where
    given.  ``dW=False``: the gradient of the bias alone, which is returned then
    (``x`` is of no account)."""
    E, ps, pl = _segments(seg_off, live)
    rows, N, ldy, kind = _rows(dy, "dy")
    py, ldy = _rows16(dy, "dy")
    if dW is False:
        if dbias is None:
            raise ValueError("dW=False needs dbias")
        check(lib().ap_expert_linear_dw(py, ldy, None, 1, rows, E, N, 1, ps, pl, 1 if accumulate else 0, None, DTYPE_F32,
                                        _need_shape(dbias, torch.float32, (E, N), "dbias"), None, 0, _status(status),
                                        _stream(stream)), "expert_linear_dw")
        return dbias
    K = x.shape[1] if x.dim() == 2 else -1
    px, ldx = _rows16(x, "x", (rows, K))
    if dW is None:
        if accumulate:
            raise ValueError("accumulate needs dW")
        dW = _empty((E, N, K), dtype, dy.device, stream)
    wkind = _ROW_TYPES.get(dW.dtype)
    if wkind is None:
        raise ValueError(f"dW must be bfloat16 or float32, got {dW.dtype}")
    pw = _need_shape(dW, dW.dtype, (E, N, K), "dW")
    pb = None if dbias is None else _need_shape(dbias, torch.float32, (E, N), "dbias")
    scratch, sb = _expert_scratch(scratch, py, ldy, rows, N, px, ldx, 0, rows, K, dy.device, stream)
    check(lib().ap_expert_linear_dw(py, ldy, px, ldx, rows, E, N, K, ps, pl, 1 if accumulate else 0, pw, wkind, pb, _p(scratch), sb,
                                    _status(status), _stream(stream)), "expert_linear_dw")
    return dW


def launch_count() -> int:
    """Kernels the library has enqueued in this process (a graph replay adds none)."""
    return int(lib().ap_launch_count())


def dispatch_scratch_bytes(T: int, k: int, E: int) -> int:
    n = ctypes.c_int64(0)
    check(lib().ap_dispatch_scratch_bytes(T, k, E, ctypes.byref(n)), "dispatch_scratch_bytes")
    return n.value


def count_rank(E: int, idx: torch.Tensor | None = None, logits: torch.Tensor | None = None, k: int | None = None,
               x: torch.Tensor | None = None, out: dict | None = None, status: torch.Tensor | None = None,
               stream=None, scan: bool = False, capacity: int = 0, padded: bool = False) -> dict:
    """Count/rank alone (``ap_count_rank``) on ``stream`` (default: the
    current stream): ``dest`` ([T, k] int32 ranks inside blocks of 64 tokens)
    and ``scratch`` (the blocks' expert histograms), for a later
    ``Pool.dispatch_stash(..., ranked=True, out=...)`` ordered after it.  With
    ``logits`` ([T, E] float32) it routes first and adds ``idx`` and ``w``;
    else ``idx`` is read.  ``x``: the rows the copy will read (an L2
    prefetch hint).  ``scan``: also the dispatch's expert scan for
    ``capacity`` / ``padded`` (adds ``counts``, ``live``, ``seg_off``; the
    scratch then holds block bases, and the dict is marked ``scanned``)."""
    o = dict(out) if out is not None else {}
    if logits is not None:
        _need(logits, torch.float32, "logits")
        T = logits.shape[0]
        dev = logits.device
        if "idx" not in o:
            o["idx"] = torch.empty((T, k), dtype=torch.int32, device=dev)
        if "w" not in o:
            o["w"] = torch.empty((T, k), dtype=torch.float32, device=dev)
        idx = o["idx"]
    else:
        _need(idx, torch.int32, "idx")
        T, k = idx.shape
        dev = idx.device
        o["idx"] = idx
    if "dest" not in o:
        o["dest"] = torch.empty((T, k), dtype=torch.int32, device=dev)
    sb = dispatch_scratch_bytes(T, k, E)
    if "scratch" not in o or o["scratch"].numel() < sb:
        o["scratch"] = torch.empty(sb, dtype=torch.uint8, device=dev)
    if scan:
        for name in ("counts", "live", "seg_off"):
            if name not in o:
                o[name] = torch.empty(E, dtype=torch.int32, device=dev)
    rb = x.shape[1] * x.element_size() if x is not None else 0
    check(lib().ap_count_rank(_p(logits), _p(o.get("w") if logits is not None else None), _p(idx), T, k, E, _p(x), rb,
                              _p(o["dest"]), _p(o["scratch"]), o["scratch"].numel(), capacity, int(padded),
                              _p(o["counts"] if scan else None), _p(o["live"] if scan else None),
                              _p(o["seg_off"] if scan else None), _p(status), _stream(stream)), "count_rank")
    o["scanned"] = scan
    return o


def dispatch_permute(x: torch.Tensor, idx: torch.Tensor, E: int, capacity: int = 0, padded: bool = False,
                     fp8: bool = False, out: dict | None = None, status: torch.Tensor | None = None, stream=None):
    """Permute BF16 rows x [T, H] into expert-major rows.

    Returns a dict with xd ([rows, H] bf16, or uint8 codes), xd_scale (E4M3
    only), counts, live, seg_off ([E] int32), dest ([T, k] int32), src_tok
    ([rows] int32, -1 where never written) and scratch.  Pass ``out`` (such a
    dict) to reuse buffers."""
    _need(x, torch.bfloat16, "x")
    _need(idx, torch.int32, "idx")
    T, H = x.shape
    k = idx.shape[1]
    dev = x.device
    rows = E * capacity if padded else T * k
    o = dict(out) if out is not None else {}
    if "xd" not in o:
        o["xd"] = torch.empty((rows, H), dtype=torch.uint8 if fp8 else torch.bfloat16, device=dev)
    if fp8 and "xd_scale" not in o:
        o["xd_scale"] = torch.empty(rows, dtype=torch.float32, device=dev)
    for name, shape in (("counts", (E,)), ("live", (E,)), ("seg_off", (E,)), ("dest", (T, k))):
        if name not in o:
            o[name] = torch.empty(shape, dtype=torch.int32, device=dev)
    if "src_tok" not in o:
        o["src_tok"] = torch.full((rows,), -1, dtype=torch.int32, device=dev)
    sb = dispatch_scratch_bytes(T, k, E)
    if "scratch" not in o or o["scratch"].numel() < sb:
        o["scratch"] = torch.empty(sb, dtype=torch.uint8, device=dev)
    xd = o["xd"]
    check(lib().ap_dispatch_permute(_p(x), T, H, _p(idx), k, E, capacity, int(padded),
                                    DTYPE_E4M3 if fp8 else DTYPE_BF16, _p(xd), _p(o.get("xd_scale")), xd.shape[0],
                                    _p(o["counts"]), _p(o["live"]), _p(o["seg_off"]), _p(o["dest"]),
                                    _p(o["src_tok"]), _p(o["scratch"]), o["scratch"].numel(), _p(status),
                                    _stream(stream)), "dispatch_permute")
    return o


def combine_unpermute(y: torch.Tensor, dest: torch.Tensor, w: torch.Tensor, out: torch.Tensor | None = None,
                      status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """out [T, H] bf16 = sum_j w[t, j] * y[dest[t, j]] (FP32 accumulation)."""
    _need(y, torch.bfloat16, "y")
    _need(dest, torch.int32, "dest")
    _need(w, torch.float32, "w")
    T, k = dest.shape
    H = y.shape[1]
    if out is None:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=y.device)
    check(lib().ap_combine_unpermute(_p(y), y.shape[0], H, _p(dest), _p(w), T, k, _p(out), _p(status),
                                     _stream(stream)), "combine_unpermute")
    return out


def combine_backward(dout: torch.Tensor, y: torch.Tensor, dest: torch.Tensor, w: torch.Tensor,
                     dy: torch.Tensor | None = None, dw: torch.Tensor | None = None,
                     status: torch.Tensor | None = None, stream=None):
    """dy [rows, H] bf16 (rows no pair maps to are left as given) and dw [T, k] f32."""
    _need(dout, torch.bfloat16, "dout")
    _need(y, torch.bfloat16, "y")
    _need(dest, torch.int32, "dest")
    _need(w, torch.float32, "w")
    T, k = dest.shape
    H = y.shape[1]
    if dy is None:
        dy = torch.zeros_like(y)
    if dw is None:
        dw = torch.empty((T, k), dtype=torch.float32, device=y.device)
    check(lib().ap_combine_backward(_p(dout), _p(y), y.shape[0], H, _p(dest), _p(w), T, k, _p(dy), _p(dw),
                                    _p(status), _stream(stream)), "combine_backward")
    return dy, dw


def dispatch_backward(dxd: torch.Tensor, dest: torch.Tensor, dx: torch.Tensor | None = None,
                      status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """dx [T, H] bf16 = sum_j dxd[dest[t, j]] (FP32 accumulation)."""
    _need(dxd, torch.bfloat16, "dxd")
    _need(dest, torch.int32, "dest")
    T, k = dest.shape
    H = dxd.shape[1]
    if dx is None:
        dx = torch.empty((T, H), dtype=torch.bfloat16, device=dxd.device)
    check(lib().ap_dispatch_backward(_p(dxd), dxd.shape[0], H, _p(dest), T, k, _p(dx), _p(status),
                                     _stream(stream)), "dispatch_backward")
    return dx


def cast_e4m3(x: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    _need(x, torch.float32, "x")
    if out is None:
        out = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    check(lib().ap_cast_e4m3(_p(x), _p(out), x.numel(), _stream(stream)), "cast_e4m3")
    return out


def page_bytes_for(page_tokens: int, row_bytes) -> int:
    """Smallest page (multiple of 256 bytes) holding page_tokens rows of each plane."""
    need = page_tokens * row_bytes[0]
    if len(row_bytes) == 2:
        need = (need + 15) // 16 * 16 + page_tokens * row_bytes[1]
    return (need + 255) // 256 * 256


class Arena:
    """Device memory whose size grows in place (``ap_arena_*``: reserved
    addresses, physical memory mapped on demand).  ``view(n)`` is a uint8
    tensor over the first n bytes; views stay valid while the arena lives."""

    def __init__(self, max_bytes: int, device="cuda"):
        self.lib = lib()
        self.device = torch.device(device)
        self.handle = ctypes.c_void_p()
        check(self.lib.ap_arena_create(ctypes.byref(self.handle), int(max_bytes), self.device.index or 0),
              "arena_create")

    def grow(self, nbytes: int):
        check(self.lib.ap_arena_grow(self.handle, int(nbytes)), "arena_grow")

    def info(self):
        base, mapped, reserved = ctypes.c_void_p(), ctypes.c_int64(), ctypes.c_int64()
        check(self.lib.ap_arena_info(self.handle, ctypes.byref(base), ctypes.byref(mapped), ctypes.byref(reserved)),
              "arena_info")
        return base.value or 0, mapped.value, reserved.value

    def view(self, nbytes: int) -> torch.Tensor:
        base, mapped, _ = self.info()
        if nbytes > mapped:
            raise ValueError(f"{nbytes} bytes requested, {mapped} mapped")
        if nbytes == 0:  # nothing mapped yet: no address to view
            return torch.empty(0, dtype=torch.uint8, device=self.device)
        return torch.as_tensor(_DeviceSpan(base, nbytes, self), device=self.device)

    def close(self):
        if getattr(self, "handle", None) and self.handle.value:
            check(self.lib.ap_arena_destroy(self.handle), "arena_destroy")
            self.handle = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class _DeviceSpan:
    """A device byte range in the CUDA array interface (keeps its owner alive)."""

    def __init__(self, ptr: int, nbytes: int, owner):
        self.owner = owner
        self.__cuda_array_interface__ = {"shape": (nbytes,), "typestr": "|u1", "data": (ptr, False),
                                         "version": 3, "strides": None}


class Pool:
    """Paged activation stash over PyTorch-owned memory.

    The device pool, its metadata and the pinned host spill are torch tensors
    held by this object; the library keeps only their addresses.  Every push,
    pop and reset runs on ``self.stream`` (a high-priority stream by
    default).  Order work on other streams with ``stream.wait_stream`` /
    ``self.stream.wait_stream``.

    ``max_num_pages > num_pages`` makes a growable pool: its pages live in an
    :class:`Arena` reserved for ``max_num_pages`` pages and mapped as the pool
    grows (``grow``); ``num_pages`` may then be 0, a calibration pool whose
    pushes park their live prefixes in the spill pages (or lose them) while
    ``state()["held_high_water"]`` measures the device pages the schedule
    needs (``calibrated_pages``)."""

    def __init__(self, page_tokens: int, page_bytes: int, num_pages: int, num_slots: int = 1,
                 max_records_per_slot: int = 8, max_segments: int = 1024, max_pages_per_record: int | None = None,
                 spill_pages: int = 0, max_ctas: int = 0, device="cuda", stream: torch.cuda.Stream | None = None,
                 fill: int | None = None, max_num_pages: int = 0):
        self.lib = lib()
        nmax = max(max_num_pages, num_pages)
        if max_pages_per_record is None:
            max_pages_per_record = nmax + spill_pages
        self.cfg = PoolConfig(page_tokens, num_slots, page_bytes, num_pages, spill_pages, max_records_per_slot,
                              max_segments, max_pages_per_record, max_ctas, 0, max_num_pages)
        a, b, c = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
        check(self.lib.ap_pool_required_bytes(ctypes.byref(self.cfg), ctypes.byref(a), ctypes.byref(b),
                                              ctypes.byref(c)), "pool_required_bytes")
        self.device = torch.device(device)
        self.fill = fill
        self.arena = None
        if nmax > num_pages:
            self.arena = Arena(nmax * page_bytes, self.device)
            self.arena.grow(a.value)
            self.pool = self.arena.view(a.value)
        else:
            self.pool = torch.empty(a.value, dtype=torch.uint8, device=self.device)
        self.meta = torch.empty(b.value, dtype=torch.uint8, device=self.device)
        self.spill = torch.empty(c.value, dtype=torch.uint8, pin_memory=True) if c.value else None
        if fill is not None:
            self.pool.fill_(fill)
            if self.spill is not None:
                self.spill.fill_(fill)
            torch.cuda.synchronize(self.device)
        self.stream = stream if stream is not None else torch.cuda.Stream(device=self.device, priority=-1)
        self.handle = ctypes.c_void_p()
        check(self.lib.ap_pool_init(ctypes.byref(self.handle), ctypes.byref(self.cfg),
                                    _p(self.pool) if num_pages else None, _p(self.meta), _p(self.spill),
                                    self.stream.cuda_stream), "pool_init")
        self.N, self.SP, self.P, self.NMAX = num_pages, spill_pages, page_tokens, nmax
        self.page_bytes = page_bytes
        self.max_pages = max_pages_per_record

    def grow(self, num_pages: int):
        """Grow the device pool to ``num_pages`` in place, with records still
        queued (``ap_pool_grow``).  New pages are filled with ``fill`` when the
        pool was created with one.  Graphs captured before must be captured
        again (they hold the old page count)."""
        if num_pages == self.N:
            return
        if self.arena is None:
            raise ValueError("this pool was created without room to grow (max_num_pages)")
        nbytes = num_pages * self.page_bytes
        self.arena.grow(nbytes)
        pool = self.arena.view(nbytes)
        if self.fill is not None:
            with torch.cuda.stream(self.stream):
                pool[self.N * self.page_bytes:].fill_(self.fill)
        check(self.lib.ap_pool_grow(self.handle, num_pages, self.arena.info()[0], self.stream.cuda_stream),
              "pool_grow")
        self.pool, self.N = pool, num_pages

    def calibrated_pages(self, margin: float = 1.0) -> int:
        """Device pages for the schedule run so far: the most pages its queued
        records ever held, times ``margin`` (synchronises the paging stream)."""
        import math
        return int(math.ceil(self.state()["held_high_water"] * margin))

    # -- lifecycle --------------------------------------------------------
    def close(self):
        if getattr(self, "handle", None) and self.handle.value:
            self.lib.ap_pool_destroy(self.handle)
            self.handle = ctypes.c_void_p()
        if getattr(self, "arena", None) is not None:
            # the paging stream's work on the pages ends before the mapping can
            # go; the arena itself is released with its last tensor view
            self.stream.synchronize()
            self.arena = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def reset(self):
        check(self.lib.ap_pool_reset(self.handle, self.stream.cuda_stream), "pool_reset")

    @property
    def max_ctas(self) -> int:
        v = ctypes.c_int32()
        check(self.lib.ap_pool_max_ctas(self.handle, ctypes.byref(v)), "pool_max_ctas")
        return v.value

    @max_ctas.setter
    def max_ctas(self, value: int):
        check(self.lib.ap_pool_set_max_ctas(self.handle, int(value)), "pool_set_max_ctas")

    # -- data path ----------------------------------------------------------
    @staticmethod
    def _planes(planes):
        rows = planes[0].shape[0]
        ptrs = (ctypes.c_void_p * 2)()
        rb = (ctypes.c_int64 * 2)()
        for i, t in enumerate(planes):
            if not t.is_contiguous() or t.shape[0] != rows:
                raise ValueError("planes must be contiguous with the same number of rows")
            ptrs[i] = t.data_ptr()
            rb[i] = (t.numel() // rows) * t.element_size() if rows else t[0:0].element_size()
        return ptrs, rb, rows

    def _order_after_caller(self, tensors):
        """Make the paging stream wait for the caller's current stream, and tell
        the caching allocator that the tensors are used on the paging stream."""
        cur = torch.cuda.current_stream(self.device)
        if cur != self.stream:
            self.stream.wait_stream(cur)
            for t in tensors:
                if t is not None and t.is_cuda:
                    t.record_stream(self.stream)

    def push(self, slot: int, planes, seg_off: torch.Tensor, live: torch.Tensor) -> int:
        """Stash the live prefixes of every segment of ``planes`` (list of 1-2 tensors).

        The paging stream first waits for the caller's current stream."""
        self._order_after_caller(list(planes) + [seg_off, live])
        ptrs, rb, rows = self._planes(planes)
        rid = ctypes.c_uint64()
        nseg = seg_off.numel()
        check(self.lib.ap_stash_push(self.handle, slot, len(planes), ptrs, rb, rows, nseg, _p(seg_off), _p(live),
                                     ctypes.byref(rid), self.stream.cuda_stream), "stash_push")
        return rid.value

    def dispatch_stash(self, slot: int, x: torch.Tensor, idx: torch.Tensor, E: int, capacity: int = 0,
                       padded: bool = False, fp8: bool = False, out: dict | None = None,
                       status: torch.Tensor | None = None, ranked: bool = False):
        """Fused dispatch + push into ``slot`` (BF16 rows, or E4M3 codes and
        row scales as two planes): returns the dispatch dict (as
        ``dispatch_permute``) with the record id under ``record_id``.
        ``ranked``: ``out`` holds ``count_rank``'s ``dest`` and ``scratch``
        for this idx (``ap_dispatch_stash_ranked``: no count/rank launch), and
        its ``counts``, ``live`` and ``seg_off`` when it ran the scan
        (``out["scanned"]``, for the same capacity and padded); the paging
        stream must already be ordered after the stream that ran it (this
        call orders it after the caller's current stream)."""
        _need(idx, torch.int32, "idx")
        if ranked and (out is None or "dest" not in out or "scratch" not in out):
            raise ValueError("ranked dispatch_stash needs out['dest'] and out['scratch'] from count_rank")
        if ranked and out.get("scanned") and any(n not in out for n in ("counts", "live", "seg_off")):
            raise ValueError("a scanned count_rank's counts, live and seg_off belong in out")
        return self._dispatch_stash(slot, x, idx, idx.shape[1], E, capacity, padded, fp8, out, status, ranked=ranked)

    def route_dispatch_stash(self, slot: int, logits: torch.Tensor, x: torch.Tensor, k: int, E: int | None = None,
                             capacity: int = 0, padded: bool = False, fp8: bool = False, out: dict | None = None,
                             status: torch.Tensor | None = None):
        """Route (as ``route_topk``) and fused dispatch + push in one call:
        the routing runs inside the count/rank launch.  Returns the dispatch
        dict with ``idx``, ``w`` and ``record_id`` added (``out`` may supply
        ``idx`` and ``w`` too)."""
        _need(logits, torch.float32, "logits")
        T, E_l = logits.shape
        E = E_l if E is None else E
        o = dict(out) if out is not None else {}
        if "idx" not in o:
            o["idx"] = torch.empty((T, k), dtype=torch.int32, device=logits.device)
        if "w" not in o:
            o["w"] = torch.empty((T, k), dtype=torch.float32, device=logits.device)
        return self._dispatch_stash(slot, x, o["idx"], k, E, capacity, padded, fp8, o, status, logits=logits,
                                    w=o["w"])

    def _dispatch_stash(self, slot, x, idx, k, E, capacity, padded, fp8, out, status, logits=None, w=None,
                        ranked=False):
        _need(x, torch.bfloat16, "x")
        T, H = x.shape
        dev = x.device
        rows = E * capacity if padded else T * k
        o = dict(out) if out is not None else {}
        if "xd" not in o:
            o["xd"] = torch.empty((rows, H), dtype=torch.uint8 if fp8 else torch.bfloat16, device=dev)
        if fp8 and "xd_scale" not in o:
            o["xd_scale"] = torch.empty(rows, dtype=torch.float32, device=dev)
        for name, shape in (("counts", (E,)), ("live", (E,)), ("seg_off", (E,)), ("dest", (T, k))):
            if name not in o:
                o[name] = torch.empty(shape, dtype=torch.int32, device=dev)
        if "src_tok" not in o:
            o["src_tok"] = torch.full((rows,), -1, dtype=torch.int32, device=dev)
        sb = dispatch_scratch_bytes(T, k, E)
        if "scratch" not in o or o["scratch"].numel() < sb:
            o["scratch"] = torch.empty(sb, dtype=torch.uint8, device=dev)
        self._order_after_caller([x, idx, status, logits] + [v for v in o.values() if isinstance(v, torch.Tensor)])
        rid = ctypes.c_uint64()
        xd = o["xd"]
        tail = (DTYPE_E4M3 if fp8 else DTYPE_BF16, _p(xd), _p(o.get("xd_scale") if fp8 else None), xd.shape[0],
                _p(o["counts"]), _p(o["live"]), _p(o["seg_off"]), _p(o["dest"]), _p(o["src_tok"]), _p(o["scratch"]),
                o["scratch"].numel(), _p(status), ctypes.byref(rid), self.stream.cuda_stream)
        if ranked:
            scanned = int(bool(o.get("scanned", False)))
            check(self.lib.ap_dispatch_stash_ranked(self.handle, slot, _p(x), T, H, _p(idx), k, E, capacity,
                                                    int(padded), *tail[:-1], scanned, tail[-1]),
                  "dispatch_stash_ranked")
        elif logits is None:
            check(self.lib.ap_dispatch_stash(self.handle, slot, _p(x), T, H, _p(idx), k, E, capacity, int(padded),
                                             *tail), "dispatch_stash")
        else:
            check(self.lib.ap_route_dispatch_stash(self.handle, slot, _p(logits), _p(w), _p(x), T, H, _p(idx), k, E,
                                                   capacity, int(padded), *tail), "route_dispatch_stash")
        o["record_id"] = rid.value
        return o

    def pop(self, slot: int, planes) -> int:
        """Reload the slot's oldest record into ``planes`` (same rows as pushed).

        The paging stream first waits for the caller's current stream; the
        caller orders later reads after ``self.stream``."""
        self._order_after_caller(list(planes))
        ptrs, _, rows = self._planes(planes)
        rid = ctypes.c_uint64()
        check(self.lib.ap_stash_pop(self.handle, slot, len(planes), ptrs, rows, ctypes.byref(rid),
                                    self.stream.cuda_stream), "stash_pop")
        return rid.value

    def time_copies(self, before: torch.cuda.Event | None, after: torch.cuda.Event | None):
        """Record ``before`` / ``after`` (timing events) around the copy kernel
        of every following push, fused dispatch + push and pop; None, None
        stops it.  The events must stay alive while set."""
        for e in (before, after):
            if e is not None and e.cuda_event == 0:
                e.record(self.stream)  # torch creates the event on its first record
        self._timing = (before, after)  # keep them alive while the library holds them
        check(self.lib.ap_pool_time_copies(self.handle, before.cuda_event if before is not None else None,
                                           after.cuda_event if after is not None else None), "pool_time_copies")

    def queue_len(self, slot: int) -> int:
        v = ctypes.c_int32()
        check(self.lib.ap_pool_queue_len(self.handle, slot, ctypes.byref(v)), "pool_queue_len")
        return v.value

    # -- read-outs (synchronise the paging stream) -------------------------------
    def overflow(self, wait: bool = True) -> int:
        f = ctypes.c_uint32()
        check(self.lib.ap_overflow_query(self.handle, ctypes.byref(f), int(wait)), "overflow_query")
        return f.value

    def flags_device_ptr(self) -> int:
        p = ctypes.c_void_p()
        check(self.lib.ap_pool_flags_device_ptr(self.handle, ctypes.byref(p)), "pool_flags_device_ptr")
        return p.value

    def state(self) -> dict:
        s = PoolState()
        check(self.lib.ap_pool_read_state(self.handle, ctypes.byref(s)), "pool_read_state")
        return dict(head=s.head, tail=s.tail, spill_head=s.spill_head, spill_tail=s.spill_tail, flags=s.flags,
                    high_water=s.high_water, spill_high_water=s.spill_high_water, held=s.held,
                    held_high_water=s.held_high_water, num_pages=s.num_pages)

    def stats(self, wait: bool = True) -> dict:
        """Device pages in use, their high-water mark and spill pages in use
        (``ap_pool_stats``).  ``wait=False`` touches no GPU and returns the
        figures of the last synchronising read-out."""
        a, b, c = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
        check(self.lib.ap_pool_stats(self.handle, ctypes.byref(a), ctypes.byref(b), ctypes.byref(c), int(wait)),
              "pool_stats")
        return dict(pages_in_use=a.value, high_water=b.value, spill_in_use=c.value)

    def rings(self):
        import numpy as np
        ring = np.empty(self.N, np.int32)
        sring = np.empty(max(self.SP, 1), np.int32)
        check(self.lib.ap_pool_read_rings(self.handle, ring.ctypes.data, sring.ctypes.data if self.SP else None),
              "pool_read_rings")
        return ring, sring[: self.SP]

    def record(self, slot: int, qpos: int = 0) -> dict:
        import numpy as np
        info = RecordInfo()
        check(self.lib.ap_pool_read_record(self.handle, slot, qpos, ctypes.byref(info), None, None, None, 0),
              "pool_read_record")
        n = info.npages
        pt = np.empty(max(n, 1), np.int32)
        r0 = np.empty(max(n, 1), np.int64)
        nr = np.empty(max(n, 1), np.int32)
        check(self.lib.ap_pool_read_record(self.handle, slot, qpos, ctypes.byref(info), pt.ctypes.data,
                                           r0.ctypes.data, nr.ctypes.data, n), "pool_read_record")
        return dict(id=info.record_id, npages=n, ndev=info.ndev, nspill=info.nspill, nlost=info.nlost,
                    nseg=info.nseg, page_table=pt[:n], row0=r0[:n], nrows=nr[:n])
