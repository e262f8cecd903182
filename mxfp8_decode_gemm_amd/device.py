"""Device-memory plumbing around the C ABI (torch allocates, the library computes).

``Mailbox`` owns the slot and state buffers of one mailbox; ``Workspace`` owns
a split-K workspace; ``upload`` places MXFP8 operands in HBM; ``route``,
``Experts`` and ``AdaptedLinear`` are the operators whose weights are chosen
per row, on torch tensors. Nothing here computes any part of an operator or of
the mailbox protocol: every call goes through ``binding``.
"""

from __future__ import annotations

import numpy as np
import torch

from . import binding as mx


def _dev(device) -> torch.device:
    d = torch.device(device if device is not None else "cuda")
    if d.type != "cuda":
        raise ValueError("the MXFP8 publishing GEMM runs on a HIP device")
    return d


def upload(a: np.ndarray, device=None) -> torch.Tensor:
    """A contiguous device copy of a numpy array (uint8/uint16/...)."""
    t = torch.from_numpy(np.ascontiguousarray(a))
    return t.to(_dev(device))


class Mailbox:
    """A three-generation mailbox of ``ranks`` slots of ``capacity_bytes``."""

    def __init__(self, ranks: int, capacity_bytes: int, rank: int = 0, device=None,
                 stream=None) -> None:
        dev = _dev(device)
        nbytes = mx.mxg_mailbox_slots_bytes(ranks, capacity_bytes)
        if nbytes == 0:
            raise ValueError("invalid mailbox geometry")
        self.slots = torch.empty(nbytes // 4, dtype=torch.int32, device=dev)
        self.state = torch.empty(mx.STATE_WORDS, dtype=torch.int32, device=dev)
        self.ranks, self.rank, self.capacity_bytes = ranks, rank, capacity_bytes
        self.mb = mx.mailbox_init(self.slots, self.state, ranks, rank, capacity_bytes, stream)

    def reinit(self, stream=None) -> None:
        self.mb = mx.mailbox_init(self.slots, self.state, self.ranks, self.rank,
                                  self.capacity_bytes, stream)

    @property
    def spin_limit(self) -> int:
        """Polls before a device wait of a call on this mailbox gives up (0:
        the library's default); carried in the descriptor, read at launch."""
        return int(self.mb.spin_limit)

    @spin_limit.setter
    def spin_limit(self, polls: int) -> None:
        self.mb.spin_limit = polls

    def state_words(self) -> np.ndarray:
        return self.state.cpu().numpy().view(np.uint32).copy()

    def slot_words(self) -> np.ndarray:
        """uint32 [3, ranks, capacity/4] copy of the whole mailbox."""
        w = self.slots.cpu().numpy().view(np.uint32)
        return w.reshape(mx.GENERATIONS, self.ranks, self.capacity_bytes // 4).copy()


class Workspace:
    """A split-K workspace large enough for ``n`` output columns at ``split_k``."""

    def __init__(self, n: int, split_k: int, device=None, stream=None) -> None:
        self.nbytes = max(mx.mxgemm_workspace_bytes(8, n, 128 * split_k, split_k),
                          mx.WS_HEADER_BYTES + mx.WS_FLAG_BYTES)
        self.buf = torch.empty(self.nbytes // 4, dtype=torch.int32, device=_dev(device))
        mx.mxgemm_workspace_init(self.buf, self.nbytes, stream)

    def header(self) -> np.ndarray:
        return self.buf[: mx.WS_HEADER_BYTES // 4].cpu().numpy().view(np.uint32).copy()


def pack_weight(w: torch.Tensor, ws: torch.Tensor, n: int, k: int, stream=None):
    """Device copies of W and its scales in the GEMM's packed tile layout."""
    wp = torch.empty(mx.mxgemm_packed_weight_bytes(n, k), dtype=torch.uint8, device=w.device)
    wsp = torch.empty(mx.mxgemm_packed_scale_bytes(n, k), dtype=torch.uint8, device=w.device)
    mx.mxgemm_pack_weight(w, ws, n, k, wp, wsp, stream)
    return wp, wsp


class Operands:
    """A problem's MXFP8 operands in HBM; W and its scales packed once."""

    def __init__(self, problem, device=None) -> None:
        self.m, self.n, self.k = problem.m, problem.n, problem.k
        w = upload(problem.w, device)
        ws = upload(problem.ws, device)
        self.w, self.ws = pack_weight(w, ws, self.n, self.k)
        self.x = upload(problem.x, device)
        self.xs = upload(problem.xs, device)


def publish(mailbox: Mailbox, ops: Operands, split_k: int = 1, workspace: Workspace = None,
            c_out: torch.Tensor = None, stream=None) -> None:
    """One mxgemm_publish call on device operands."""
    mx.mxgemm_publish(mailbox.mb, ops.w, ops.ws, ops.x, ops.xs, ops.m, ops.n, ops.k, split_k,
                      workspace.buf if workspace is not None else None,
                      workspace.nbytes if workspace is not None else 0, c_out, stream)


def collect(mailbox: Mailbox, nbytes: int, out: torch.Tensor = None, stream=None) -> torch.Tensor:
    """One mailbox_collect; returns the [ranks * nbytes] byte output as uint16."""
    if out is None:
        out = torch.empty(mailbox.ranks * nbytes // 2, dtype=torch.int16,
                          device=mailbox.slots.device)
    mx.mailbox_collect(mailbox.mb, out, nbytes, stream)
    return out


def collect_sum(mailbox: Mailbox, nbytes: int, out: torch.Tensor = None,
                stream=None) -> torch.Tensor:
    """One mailbox_collect_sum; returns the [nbytes] byte all-reduce as uint16."""
    if out is None:
        out = torch.empty(nbytes // 2, dtype=torch.int16, device=mailbox.slots.device)
    mx.mailbox_collect_sum(mailbox.mb, out, nbytes, stream)
    return out


def all_gather(mailbox: Mailbox, src: torch.Tensor, nbytes: int, out: torch.Tensor = None,
               stream=None) -> torch.Tensor:
    """One mailbox_all_gather of slot mailbox.rank; returns the [ranks * nbytes]
    byte output as int32 words."""
    if out is None:
        out = torch.empty(mailbox.ranks * nbytes // 4, dtype=torch.int32,
                          device=mailbox.slots.device)
    mx.mailbox_all_gather(mailbox.mb, src, out, nbytes, stream)
    return out


def as_u16(t: torch.Tensor) -> np.ndarray:
    """uint16 host copy of a 16-bit device tensor."""
    return t.cpu().numpy().view(np.uint16).copy()


# ---------------------------------------------------------------------------
# operators whose weights are chosen per row (include/mxdecode.h)
# ---------------------------------------------------------------------------


def _tensor(t, name: str, dtype, shape, device=None, contiguous: bool = True) -> torch.Tensor:
    """``t`` itself when it is a device tensor of this type and shape (None in
    ``shape``: any size)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name}: a device tensor is needed")
    if t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise ValueError(f"{name}: {t.dtype} instead of {dtype}")
    if t.dim() != len(shape) or any(w is not None and w != g for g, w in zip(t.shape, shape)):
        raise ValueError(f"{name}: shape {tuple(t.shape)} instead of {tuple(shape)}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name}: not contiguous")
    if device is not None and t.device != device:
        raise ValueError(f"{name}: on {t.device}, not on {device}")
    return t


def _current(device: torch.device) -> None:
    """A call runs on the current device: its tensors have to be there."""
    if device.index != torch.cuda.current_device():
        raise ValueError(f"tensors on {device}, but the current device is "
                         f"cuda:{torch.cuda.current_device()}")


_SCORES = {"softmax": mx.ROUTE_SOFTMAX, "sigmoid": mx.ROUTE_SIGMOID}


def route(logits: torch.Tensor, top_k: int, score: str = "softmax", bias: torch.Tensor = None,
          groups: int = 1, top_groups: int = 1, group_best: int = 1, renormalize: bool = False,
          scale: float = 1.0, ids: torch.Tensor = None, weights: torch.Tensor = None,
          stream=None):
    """One mxmoe_route call on [tokens, experts] logits (float32 or bfloat16,
    rows of any stride): (ids int32, weights float32), each [tokens, top_k]."""
    _tensor(logits, "logits", (torch.float32, torch.bfloat16), (None, None), contiguous=False)
    tokens, experts = logits.shape
    dev = logits.device
    _current(dev)
    row_stride, step = logits.stride()
    if step != 1 and experts > 1:
        raise ValueError("logits: a row's values have to be contiguous")
    if tokens == 1:
        row_stride = experts
    if score not in _SCORES:
        raise ValueError(f"score: {score!r} instead of one of {sorted(_SCORES)}")
    if bias is not None:
        _tensor(bias, "bias", torch.float32, (experts,), dev)
    if ids is None:
        ids = torch.empty(tokens, max(top_k, 0), dtype=torch.int32, device=dev)
    else:
        _tensor(ids, "ids", torch.int32, (tokens, top_k), dev)
    if weights is None:
        weights = torch.empty(tokens, max(top_k, 0), dtype=torch.float32, device=dev)
    else:
        _tensor(weights, "weights", torch.float32, (tokens, top_k), dev)
    router = mx.mxmoe_router(experts, top_k, _SCORES[score], groups, top_groups, group_best,
                             int(renormalize), scale)
    mx.mxmoe_route(router, logits, mx.F32 if logits.dtype == torch.float32 else mx.BF16,
                   row_stride, bias, tokens, ids, weights, stream)
    return ids, weights


def pack_experts(w: torch.Tensor, ws: torch.Tensor, stream=None):
    """Packed copies of [experts, n, k] codes and their scales."""
    _tensor(w, "w", torch.uint8, (None, None, None))
    e, n, k = w.shape
    _tensor(ws, "w_scale", torch.uint8, (e, n, k // 32), w.device)
    _current(w.device)
    wp = torch.empty(mx.mxmoe_packed_weight_bytes(e, n, k), dtype=torch.uint8, device=w.device)
    wsp = torch.empty(mx.mxmoe_packed_scale_bytes(e, n, k), dtype=torch.uint8, device=w.device)
    mx.mxmoe_pack_weight(w, ws, e, n, k, wp, wsp, stream)
    return wp, wsp


class Experts:
    """The experts of one layer: MXFP8 weights packed once (w13 [experts,
    2 inter, hidden]: gate rows, then up rows; w2 [experts, hidden, inter];
    uint8 codes and scale bytes) and a workspace for ``max_pairs`` (token,
    choice) pairs. Calls go one at a time, in order, on one stream."""

    def __init__(self, w13: torch.Tensor, w13_scale: torch.Tensor, w2: torch.Tensor,
                 w2_scale: torch.Tensor, max_pairs: int = mx.MOE_MAX_PAIRS, stream=None) -> None:
        _tensor(w13, "w13", torch.uint8, (None, None, None))
        self.experts, two, self.hidden = w13.shape
        self.inter = two // 2
        _tensor(w2, "w2", torch.uint8, (self.experts, self.hidden, self.inter), w13.device)
        self.nbytes = mx.mxmoe_workspace_bytes(max_pairs, 1, self.hidden, self.inter)
        if two % 2 or self.nbytes == 0:
            raise ValueError("w13, w2 or max_pairs: sizes that mxmoe_experts does not take")
        self.max_pairs, self.device = max_pairs, w13.device
        self.w13, self.w13_scale = pack_experts(w13, w13_scale, stream)
        self.w2, self.w2_scale = pack_experts(w2, w2_scale, stream)
        self.workspace = torch.empty(self.nbytes, dtype=torch.uint8, device=w13.device)

    def __call__(self, x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor,
                 out: torch.Tensor = None, stream=None) -> torch.Tensor:
        """One mxmoe_experts call: BF16 x [tokens, hidden], ids and weights as
        ``route`` returns them; BF16 [tokens, hidden]."""
        dev = self.device
        _current(dev)
        _tensor(ids, "ids", torch.int32, (None, None), dev)
        tokens, top_k = ids.shape
        _tensor(x, "x", torch.bfloat16, (tokens, self.hidden), dev)
        _tensor(weights, "weights", torch.float32, (tokens, top_k), dev)
        if out is None:
            out = torch.empty_like(x)
        else:
            _tensor(out, "out", torch.bfloat16, (tokens, self.hidden), dev)
        mx.mxmoe_experts(x, ids, weights, self.w13, self.w13_scale, self.w2, self.w2_scale,
                         tokens, top_k, self.experts, self.hidden, self.inter, self.workspace,
                         self.nbytes, out, stream)
        return out


class AdaptedLinear:
    """An MXFP8 projection [n, k] (uint8 codes and scale bytes, packed once)
    with a stack of low-rank adapters: a [adapters, rank, k] and b [adapters,
    n, rank] in BF16, scale [adapters] in FP32. Owns the split-K workspace and
    the scratch; calls go one at a time, in order, on one stream."""

    def __init__(self, w: torch.Tensor, w_scale: torch.Tensor, a: torch.Tensor, b: torch.Tensor,
                 scale: torch.Tensor, split_k: int = 1, stream=None) -> None:
        _tensor(w, "w", torch.uint8, (None, None))
        self.n, self.k = w.shape
        dev = self.device = w.device
        _current(dev)
        _tensor(w_scale, "w_scale", torch.uint8, (self.n, self.k // 32), dev)
        _tensor(a, "a", torch.bfloat16, (None, None, self.k), dev)
        adapters, rank = a.shape[:2]
        _tensor(b, "b", torch.bfloat16, (adapters, self.n, rank), dev)
        _tensor(scale, "scale", torch.float32, (adapters,), dev)
        self.scratch_bytes = mx.mxgemm_lora_scratch_bytes(self.n)
        if self.scratch_bytes == 0 or adapters < 1 or rank % 8 or not 8 <= rank <= mx.LORA_MAX_RANK:
            raise ValueError("w or a: sizes that mxgemm_lora does not take")
        self.split_k = split_k
        self.w, self.w_scale = pack_weight(w, w_scale, self.n, self.k, stream)
        self.a, self.b, self.scale = a, b, scale
        self.workspace = Workspace(self.n, split_k, dev, stream) if split_k > 1 else None
        self.scratch = torch.empty(self.scratch_bytes // 4, dtype=torch.int32, device=dev)
        mx.mxgemm_lora_scratch_init(self.scratch, self.scratch_bytes, stream)
        self.lora = mx.mxg_lora(a.data_ptr(), b.data_ptr(), scale.data_ptr(), None, adapters, rank)

    def _call(self, mb, x, ids, x_scale, c_out, stream):
        dev = self.device
        _current(dev)
        m = x.shape[0]
        if x_scale is None:
            _tensor(x, "x", torch.bfloat16, (None, self.k), dev)
            form = (None, None, x)
        else:
            _tensor(x, "x", torch.uint8, (None, self.k), dev)
            _tensor(x_scale, "x_scale", torch.uint8, (m, self.k // 32), dev)
            form = (x, x_scale, None)
        _tensor(ids, "ids", torch.int32, (m,), dev)
        if c_out is not None:
            _tensor(c_out, "c_out", torch.bfloat16, (m, self.n), dev)
        self.lora.ids = ids.data_ptr()
        ws = self.workspace
        mx.mxgemm_lora(mb, self.w, self.w_scale, *form, m, self.n, self.k, self.split_k,
                       ws.buf if ws else None, ws.nbytes if ws else 0, self.lora, self.scratch,
                       self.scratch_bytes, c_out, stream)

    def __call__(self, x: torch.Tensor, ids: torch.Tensor, x_scale: torch.Tensor = None,
                 c_out: torch.Tensor = None, stream=None) -> torch.Tensor:
        """One mxgemm_lora call without a mailbox: BF16 x [m, k], or uint8 codes
        with x_scale [m, k/32]; ids int32 [m] (outside 0..adapters-1: none).
        BF16 [m, n]."""
        if c_out is None:
            c_out = torch.empty(x.shape[0], self.n, dtype=torch.bfloat16, device=x.device)
        self._call(None, x, ids, x_scale, c_out, stream)
        return c_out

    def publish(self, mailbox: Mailbox, x: torch.Tensor, ids: torch.Tensor,
                x_scale: torch.Tensor = None, c_out: torch.Tensor = None, stream=None) -> None:
        """The same into the mailbox (then collect it)."""
        self._call(mailbox.mb, x, ids, x_scale, c_out, stream)
