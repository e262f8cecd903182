"""Device-memory plumbing around the C ABI (torch allocates, the library computes).

``Mailbox`` owns the slot and state buffers of one mailbox; ``Workspace`` owns
a split-K workspace; ``upload`` places MXFP8 operands in HBM; ``route``,
``Experts`` and ``AdaptedLinear`` are the operators whose weights are chosen
per row, on torch tensors (without a backward pass: tensors that require a
gradient are taken under ``torch.no_grad`` only). Nothing here computes any part
of an operator or of the mailbox protocol: every call goes through ``binding``.
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


# A decode step's calls take a few microseconds on the GPU, so the checks below
# are written to cost less than that on the host.
_raw_stream = torch._C._cuda_getCurrentRawStream
_device = torch._C._cuda_getDevice


def _refuse(t, name: str, dtype, shape, device) -> None:
    """The reason why ``t`` is not a contiguous tensor of this type, shape (None:
    any size) and device."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name}: a device tensor is needed")
    if t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise ValueError(f"{name}: {t.dtype} instead of {dtype}")
    if t.dim() != len(shape) or any(w is not None and w != g for g, w in zip(t.shape, shape)):
        raise ValueError(f"{name}: shape {tuple(t.shape)} instead of {tuple(shape)}")
    if device is not None and t.device != device:
        raise ValueError(f"{name}: on {t.device}, not on {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: not contiguous")
    _refuse_gradient(t, name)


def _refuse_gradient(t: torch.Tensor, name: str) -> None:
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{name}: requires a gradient, and the decode operators have none "
                         "(call them under torch.no_grad)")


def _address(t, name: str, dtype, shape: tuple, device) -> int:
    """The address of a contiguous device tensor of this type and shape."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape
            and t.device == device and t.is_contiguous() and not t.requires_grad):
        return t.data_ptr()
    _refuse(t, name, dtype, shape, device)
    return t.data_ptr()


def _on(device: torch.device, stream):
    """The stream handle of a call whose tensors are on ``device``, which has to
    be the current one."""
    if device.index != _device():
        raise ValueError(f"tensors on {device}, but the current device is cuda:{_device()}")
    if stream is None:
        return _raw_stream(device.index)
    if isinstance(stream, int):
        return stream
    if stream.device != device:
        raise ValueError(f"a stream of {stream.device} for tensors on {device}")
    return stream.cuda_stream


# Memory and streams. A fresh tensor of a call on a given stream is allocated on that
# stream: on the current one it could be memory that work queued there still uses.
# The current stream, where the caller goes on, is noted for it. Tensors that a call
# on a given stream is handed are noted as used there, so that memory the caller
# drops is not given out while the call runs. A handle (an int) names a stream whose
# end this module cannot see: nothing is noted for it, and what such a call uses has to
# live until it has ended.


def _stream(stream, device: torch.device):
    """The given stream as torch's (None for the current one)."""
    return torch.cuda.ExternalStream(stream, device) if isinstance(stream, int) else stream


def _fresh(like: torch.Tensor, shape: tuple, dtype, stream) -> torch.Tensor:
    """An output's memory, for a call on the given stream."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(_stream(stream, like.device)):
        t = like.new_empty(shape, dtype=dtype)
    t.record_stream(torch.cuda.current_stream(like.device))
    return t


def _lend(stream, *tensors) -> None:
    """Notes the tensors as used on the given stream."""
    if stream is not None and not isinstance(stream, int):
        for t in tensors:
            if t is not None:
                t.record_stream(stream)


class _Home:
    """The tensors an object owns, made on one stream: other streams it is used on are
    noted for them."""

    def __init__(self, handle: int, tensors: tuple) -> None:
        self._seen, self._tensors = {handle}, tensors

    def used(self, handle: int, stream) -> None:
        if handle not in self._seen and not isinstance(stream, int):
            self._seen.add(handle)
            _lend(stream or torch.cuda.current_stream(self._tensors[0].device), *self._tensors)


_SCORES = {"softmax": mx.ROUTE_SOFTMAX, "sigmoid": mx.ROUTE_SIGMOID}
_LOGITS = {torch.float32: mx.F32, torch.bfloat16: mx.BF16}
_lib = mx.library()


def route(logits: torch.Tensor, top_k: int, score: str = "softmax", bias: torch.Tensor = None,
          groups: int = 1, top_groups: int = 1, group_best: int = 1, renormalize: bool = False,
          scale: float = 1.0, ids: torch.Tensor = None, weights: torch.Tensor = None,
          stream=None):
    """One mxmoe_route call on [tokens, experts] logits (float32 or bfloat16,
    rows of any stride): (ids int32, weights float32), each [tokens, top_k]."""
    kind = _LOGITS.get(logits.dtype) if isinstance(logits, torch.Tensor) else None
    if kind is None or logits.dim() != 2 or not logits.is_cuda:
        raise ValueError("logits: a float32 or bfloat16 device tensor [tokens, experts] is needed")
    if logits.requires_grad:
        _refuse_gradient(logits, "logits")
    tokens, experts = logits.shape
    row_stride, step = logits.stride()
    if step != 1 and experts > 1:
        raise ValueError("logits: a row's values have to be contiguous")
    if tokens == 1:
        row_stride = experts
    if score not in _SCORES:
        raise ValueError(f"score: {score!r} instead of one of {sorted(_SCORES)}")
    dev = logits.device
    handle = _on(dev, stream)
    out = (tokens, top_k if top_k > 0 else 0)
    if ids is None:
        ids = _fresh(logits, out, torch.int32, stream)
    else:
        _address(ids, "ids", torch.int32, out, dev)
    if weights is None:
        weights = _fresh(logits, out, torch.float32, stream)
    else:
        _address(weights, "weights", torch.float32, out, dev)
    router = mx.mxmoe_router(experts, top_k, _SCORES[score], groups, top_groups, group_best,
                             int(renormalize), scale)
    code = _lib.mxmoe_route(
        router, logits.data_ptr(), kind, row_stride,
        None if bias is None else _address(bias, "bias", torch.float32, (experts,), dev), tokens,
        ids.data_ptr(), weights.data_ptr(), handle)
    if code:
        mx._check(code, "mxmoe_route")
    if stream is not None:
        _lend(stream, logits, bias, ids, weights)
    return ids, weights


def pack_experts(w: torch.Tensor, ws: torch.Tensor, stream=None):
    """Packed copies of [experts, n, k] codes and their scales."""
    _refuse(w, "w", torch.uint8, (None, None, None), None)
    e, n, k = w.shape
    _refuse(ws, "w_scale", torch.uint8, (e, n, k // 32), w.device)
    handle = _on(w.device, stream)
    wp = _fresh(w, (mx.mxmoe_packed_weight_bytes(e, n, k),), torch.uint8, stream)
    wsp = _fresh(w, (mx.mxmoe_packed_scale_bytes(e, n, k),), torch.uint8, stream)
    mx.mxmoe_pack_weight(w, ws, e, n, k, wp, wsp, handle)
    _lend(stream, w, ws)
    return wp, wsp


class Experts:
    """The experts of one layer: MXFP8 weights packed once (w13 [experts,
    2 inter, hidden]: gate rows, then up rows; w2 [experts, hidden, inter];
    uint8 codes and scale bytes) and a workspace for ``max_pairs`` (token,
    choice) pairs. Calls go one at a time, in order, on one stream. Its tensors
    may be written, not replaced."""

    w13 = property(lambda self: self._packed[0])
    w13_scale = property(lambda self: self._packed[1])
    w2 = property(lambda self: self._packed[2])
    w2_scale = property(lambda self: self._packed[3])
    workspace = property(lambda self: self._workspace)

    def __init__(self, w13: torch.Tensor, w13_scale: torch.Tensor, w2: torch.Tensor,
                 w2_scale: torch.Tensor, max_pairs: int = mx.MOE_MAX_PAIRS, stream=None) -> None:
        _refuse(w13, "w13", torch.uint8, (None, None, None), None)
        self.experts, two, self.hidden = w13.shape
        self.inter = two // 2
        dev = self.device = w13.device
        _refuse(w2, "w2", torch.uint8, (self.experts, self.hidden, self.inter), dev)
        self.nbytes = mx.mxmoe_workspace_bytes(max_pairs, 1, self.experts, self.hidden, self.inter)
        if two % 2 or self.nbytes == 0:
            raise ValueError("w13, w2 or max_pairs: sizes that mxmoe_experts does not take")
        self._packed = (*pack_experts(w13, w13_scale, stream), *pack_experts(w2, w2_scale, stream))
        self._workspace = _fresh(w13, (self.nbytes,), torch.uint8, stream)
        self._weights = tuple(t.data_ptr() for t in self._packed)
        self._home = _Home(_on(dev, stream), (*self._packed, self._workspace))

    def __call__(self, x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor,
                 out: torch.Tensor = None, stream=None) -> torch.Tensor:
        """One mxmoe_experts call: BF16 x [tokens, hidden], ids and weights as
        ``route`` returns them; BF16 [tokens, hidden]."""
        dev = self.device
        handle = _on(dev, stream)
        if not isinstance(ids, torch.Tensor) or ids.dim() != 2:
            raise ValueError("ids: a device tensor [tokens, top_k] is needed")
        chosen = ids.shape
        rows = (chosen[0], self.hidden)
        px = _address(x, "x", torch.bfloat16, rows, dev)
        if out is None:
            out = _fresh(x, rows, torch.bfloat16, stream)
        else:
            _address(out, "out", torch.bfloat16, rows, dev)
        self._home.used(handle, stream)
        code = _lib.mxmoe_experts(
            px, _address(ids, "ids", torch.int32, chosen, dev),
            _address(weights, "weights", torch.float32, chosen, dev), *self._weights, chosen[0],
            chosen[1], self.experts, self.hidden, self.inter, self._workspace.data_ptr(),
            self.nbytes, out.data_ptr(), handle)
        if code:
            mx._check(code, "mxmoe_experts")
        if stream is not None:
            _lend(stream, x, ids, weights, out)
        return out


class AdaptedLinear:
    """An MXFP8 projection [n, k] (uint8 codes and scale bytes, packed once)
    with a stack of low-rank adapters: a [adapters, rank, k] and b [adapters,
    n, rank] in BF16, scale [adapters] in FP32. Owns the split-K workspace and
    the scratch; calls go one at a time, in order, on one stream. A result whose
    split-K exchange failed is NaN (or not published); ``errors`` names it, and
    ``rearm`` makes the object good again.

    ``a``, ``b`` and ``scale`` are the caller's tensors, read by every call as they
    are then: they may be written, or replaced (a call after that looks at the new
    ones; a captured graph keeps those it was captured with, which have to
    live). ``scratch`` may be another armed one, as for projections that share
    it. The packed weight and the workspace may be written, not replaced."""

    w = property(lambda self: self._packed[0])
    w_scale = property(lambda self: self._packed[1])
    workspace = property(lambda self: self._workspace)
    scratch = property(lambda self: self._scratch)
    scratch_bytes = property(lambda self: self._scratch_bytes)

    @scratch.setter
    def scratch(self, t: torch.Tensor) -> None:
        _refuse(t, "scratch", torch.int32, (None,), self.device)
        if 4 * t.numel() < mx.mxgemm_lora_scratch_bytes(self.n):
            raise ValueError(f"scratch: {4 * t.numel()} bytes are too few for n = {self.n}")
        self._scratch, self._scratch_bytes = t, 4 * t.numel()

    @scratch_bytes.setter
    def scratch_bytes(self, nbytes: int) -> None:
        if nbytes > 4 * self._scratch.numel():
            raise ValueError(f"scratch_bytes: {nbytes} are more than the scratch has")
        self._scratch_bytes = nbytes

    def __init__(self, w: torch.Tensor, w_scale: torch.Tensor, a: torch.Tensor, b: torch.Tensor,
                 scale: torch.Tensor, split_k: int = 1, stream=None) -> None:
        _refuse(w, "w", torch.uint8, (None, None), None)
        self.n, self.k = w.shape
        dev = self.device = w.device
        handle = _on(dev, stream)
        _refuse(w_scale, "w_scale", torch.uint8, (self.n, self.k // 32), dev)
        self.a, self.b, self.scale = a, b, scale
        self._take_adapters()
        nbytes = mx.mxgemm_lora_scratch_bytes(self.n)
        if nbytes == 0:
            raise ValueError("w: sizes that mxgemm_lora does not take")
        self.split_k = split_k
        with torch.cuda.stream(_stream(stream, dev)):  # its memory is that stream's
            self._packed = pack_weight(w, w_scale, self.n, self.k, handle)
            self._workspace = Workspace(self.n, split_k, dev, handle) if split_k > 1 else None
            self.scratch = torch.empty(nbytes // 4, dtype=torch.int32, device=dev)
        mx.mxgemm_lora_scratch_init(self.scratch, nbytes, handle)
        _lend(stream, w, w_scale)
        self._weights = tuple(t.data_ptr() for t in self._packed)
        ws = self._workspace
        self._home = _Home(handle, (*self._packed, self.scratch) + ((ws.buf,) if ws else ()))
        self._memory = (ws.buf.data_ptr(), ws.nbytes) if ws else (None, 0)

    def _take_adapters(self) -> None:
        """Looks at a, b and scale, and keeps them and their addresses."""
        a, b, scale = self.a, self.b, self.scale
        _refuse(a, "a", torch.bfloat16, (None, None, self.k), self.device)
        adapters, rank = a.shape[:2]
        _refuse(b, "b", torch.bfloat16, (adapters, self.n, rank), self.device)
        _refuse(scale, "scale", torch.float32, (adapters,), self.device)
        if adapters < 1 or rank % 8 or not 8 <= rank <= mx.LORA_MAX_RANK:
            raise ValueError("a: sizes that mxgemm_lora does not take")
        self._adapters = a, b, scale
        self._places = a.data_ptr(), b.data_ptr(), scale.data_ptr()
        self.lora = mx.mxg_lora(*self._places, None, adapters, rank)

    def errors(self) -> int:
        """MXG_ERR_* bits of the calls since the last arming, the scratch's and
        the workspace's (waits for the device)."""
        bits = int(self.scratch[mx.WS_ERROR])
        return bits | int(self.workspace.header()[mx.WS_ERROR]) if self.workspace else bits

    def rearm(self, stream=None) -> None:
        """Arms the scratch and the workspace again; no call may be in flight."""
        handle = _on(self.device, stream)
        mx.mxgemm_lora_scratch_init(self.scratch, self.scratch_bytes, handle)
        if self.workspace:
            mx.mxgemm_workspace_init(self.workspace.buf, self.workspace.nbytes, handle)

    def _call(self, mb, x, ids, x_scale, c_out, stream):
        dev = self.device
        handle = _on(dev, stream)
        if not isinstance(x, torch.Tensor) or x.dim() != 2:
            raise ValueError("x: a device tensor [m, k] is needed")
        m = x.shape[0]
        if x_scale is None:
            form = None, None, _address(x, "x", torch.bfloat16, (m, self.k), dev)
        else:
            form = (_address(x, "x", torch.uint8, (m, self.k), dev),
                    _address(x_scale, "x_scale", torch.uint8, (m, self.k // 32), dev), None)
        a, b, scale = self.a, self.b, self.scale
        was = self._adapters
        if (a is not was[0] or b is not was[1] or scale is not was[2]
                or (a.data_ptr(), b.data_ptr(), scale.data_ptr()) != self._places
                or a.requires_grad or b.requires_grad or scale.requires_grad):
            self._take_adapters()
        # (Read by the library within the call.)
        self.lora.ids = _address(ids, "ids", torch.int32, (m,), dev)
        pc = None
        if c_out is not None:
            pc = _address(c_out, "c_out", torch.bfloat16, (m, self.n), dev)
        elif mb is None:
            c_out = _fresh(x, (m, self.n), torch.bfloat16, stream)
            pc = c_out.data_ptr()
        self._home.used(handle, stream)
        code = _lib.mxgemm_lora(mb, *self._weights, *form, m, self.n, self.k, self.split_k,
                                *self._memory, self.lora, self._scratch.data_ptr(),
                                self._scratch_bytes, pc, handle)
        if code:
            mx._check(code, "mxgemm_lora")
        if stream is not None:
            _lend(stream, x, ids, x_scale, c_out, a, b, scale, self._scratch)
        return c_out

    def __call__(self, x: torch.Tensor, ids: torch.Tensor, x_scale: torch.Tensor = None,
                 c_out: torch.Tensor = None, stream=None) -> torch.Tensor:
        """One mxgemm_lora call without a mailbox: BF16 x [m, k], or uint8 codes
        with x_scale [m, k/32]; ids int32 [m] (outside 0..adapters-1: none).
        BF16 [m, n]."""
        return self._call(None, x, ids, x_scale, c_out, stream)

    def publish(self, mailbox: Mailbox, x: torch.Tensor, ids: torch.Tensor,
                x_scale: torch.Tensor = None, c_out: torch.Tensor = None, stream=None) -> None:
        """The same into the mailbox (then collect it)."""
        self._call(mailbox.mb, x, ids, x_scale, c_out, stream)
