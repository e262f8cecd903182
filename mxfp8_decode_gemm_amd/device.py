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


# ---------------------------------------------------------------------------
# products of any number of rows (include/mxrows.h)
# ---------------------------------------------------------------------------

_TYPES = {torch.float32: mx.F32, torch.bfloat16: mx.BF16, torch.float16: mx.F16}
_FORMATS = {"mxfp4": mx.MXFP4, "mxfp8": mx.MXFP8}
_MOST = (1 << 31) - 1


def _matrix(t, name: str) -> torch.Tensor:
    """A device tensor of two dimensions, each in the 32 bits that the library takes sizes in
    (ctypes cuts a longer number without a word)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dim() != 2:
        raise ValueError(f"{name}: a device tensor of two dimensions is needed")
    rows, width = t.shape
    if rows > _MOST or width > _MOST:
        raise ValueError(f"{name}: shape {tuple(t.shape)} is beyond 32 bits")
    return t


def _count(value, name: str, most: int) -> None:
    if not 0 <= value <= most:
        raise ValueError(f"{name}: {value} is not within 0..{most}")


def quantize4(x: torch.Tensor, codes: torch.Tensor = None, scales: torch.Tensor = None,
              stream=None):
    """One mxfp4_quantize call on [rows, k] float32, bfloat16 or float16 values (rows of
    any stride that is a multiple of 16 bytes): (codes uint8 [rows, k/2], scales uint8
    [rows, k/32])."""
    kind = _TYPES.get(_matrix(x, "x").dtype)
    if kind is None:
        raise ValueError(f"x: {x.dtype} instead of one of {sorted(map(str, _TYPES))}")
    if x.requires_grad:
        _refuse_gradient(x, "x")
    rows, k = x.shape
    row_stride, step = x.stride()
    if step != 1:
        raise ValueError("x: a row's values have to be contiguous")
    if rows == 1:
        row_stride = k
    dev = x.device
    handle = _on(dev, stream)
    if codes is None:
        codes = _fresh(x, (rows, k // 2), torch.uint8, stream)
    else:
        _address(codes, "codes", torch.uint8, (rows, k // 2), dev)
    if scales is None:
        scales = _fresh(x, (rows, k // 32), torch.uint8, stream)
    else:
        _address(scales, "scales", torch.uint8, (rows, k // 32), dev)
    code = _lib.mxfp4_quantize(x.data_ptr(), kind, row_stride, rows, k, codes.data_ptr(),
                               scales.data_ptr(), handle)
    if code:
        mx._check(code, "mxfp4_quantize")
    if stream is not None:
        _lend(stream, x, codes, scales)
    return codes, scales


def dequantize4(codes: torch.Tensor, scales: torch.Tensor, dtype=torch.bfloat16,
                out: torch.Tensor = None, stream=None) -> torch.Tensor:
    """One mxfp4_dequantize call: the values of codes [rows, k/2] and scales [rows, k/32]
    as float32, bfloat16 or float16 [rows, k]."""
    rows, half = _matrix(codes, "codes").shape
    _count(half, "half a row", _MOST // 2)
    dev = codes.device
    handle = _on(dev, stream)
    pc = _address(codes, "codes", torch.uint8, (rows, half), dev)
    ps = _address(scales, "scales", torch.uint8, (rows, half // 16), dev)
    if dtype not in _TYPES:
        raise ValueError(f"dtype: {dtype} instead of one of {sorted(map(str, _TYPES))}")
    if out is None:
        out = _fresh(codes, (rows, 2 * half), dtype, stream)
    else:
        _address(out, "out", dtype, (rows, 2 * half), dev)
    code = _lib.mxfp4_dequantize(pc, ps, rows, 2 * half, _TYPES[dtype], out.data_ptr(), handle)
    if code:
        mx._check(code, "mxfp4_dequantize")
    if stream is not None:
        _lend(stream, codes, scales, out)
    return out


def quantize8(x: torch.Tensor, stream=None):
    """One mxfp8_quantize call on contiguous [rows, k] bfloat16 values: (codes uint8 [rows,
    k], scales uint8 [rows, k/32])."""
    rows, k = _matrix(x, "x").shape
    handle = _on(x.device, stream)
    px = _address(x, "x", torch.bfloat16, (rows, k), x.device)
    codes = _fresh(x, (rows, k), torch.uint8, stream)
    scales = _fresh(x, (rows, k // 32), torch.uint8, stream)
    code = _lib.mxfp8_quantize(px, rows, k, codes.data_ptr(), scales.data_ptr(), handle)
    if code:
        mx._check(code, "mxfp8_quantize")
    if stream is not None:
        _lend(stream, x, codes, scales)
    return codes, scales


_QUANTIZE = {mx.MXFP4: quantize4, mx.MXFP8: quantize8}


class _RowsWeight:
    """A stack of weights packed once for the products of any number of rows:
    uint8 codes [experts, n, k/2] (MXFP4) or [experts, n, k] (MXFP8) and scale bytes
    [experts, n, k/32], which say the format. Its tensors may be written, not
    replaced; calls keep nothing in it, so they may run at once."""

    w = property(lambda self: self._packed[0])
    w_scale = property(lambda self: self._packed[1])

    def _pack(self, w, w_scale, gated, activation, fast, stream) -> None:
        _refuse(w, "w", torch.uint8, (None, None, None), None)
        e, n, width = w.shape
        dev = self.device = w.device
        blocks = w_scale.shape[-1] if isinstance(w_scale, torch.Tensor) and w_scale.dim() else 0
        self.format = mx.MXFP4 if width == 16 * blocks else mx.MXFP8
        self.experts, self.n, self.k = e, n, 32 * blocks
        _count(max(e, n, self.k), "w's sizes", _MOST)
        if width not in (16 * blocks, 32 * blocks):
            raise ValueError("w: 16 (MXFP4) or 32 (MXFP8) bytes for each scale byte are needed")
        _refuse(w_scale, "w_scale", torch.uint8, (e, n, blocks), dev)
        nbytes = mx.mxrows_packed_weight_bytes(self.format, e, n, self.k)
        if nbytes == 0 or (gated and n % 64):
            raise ValueError("w: sizes that the products of any number of rows do not take")
        if activation is not None and activation not in _FORMATS:
            raise ValueError(f"activation: {activation!r} instead of one of {sorted(_FORMATS)}")
        self.activation = _FORMATS[activation] if activation else self.format
        if (self.format, self.activation) == (mx.MXFP8, mx.MXFP4):
            raise ValueError("activation: an MXFP8 weight takes MXFP8 activations")
        self.gated, self.out_n = bool(gated), n // 2 if gated else n
        self._mxfp8 = mx.MXFP8_FAST if fast else mx.MXFP8  # MXFP8 rows, to the library
        handle = _on(dev, stream)
        wp = _fresh(w, (nbytes,), torch.uint8, stream)
        wsp = _fresh(w, (mx.mxrows_packed_scale_bytes(self.format, e, n, self.k),), torch.uint8,
                     stream)
        mx.mxrows_pack_weight(self.format, w, w_scale, e, n, self.k, wp, wsp, handle)
        _lend(stream, w, w_scale)
        self._packed = wp, wsp
        self._weight = mx.mxrows_weight(wp.data_ptr(), wsp.data_ptr(), self.format, e, n, self.k,
                                        int(self.gated))
        self._home = _Home(handle, self._packed)

    def _codes(self, x, x_scale, rows, stream):
        """x as codes: (format, codes, scales, their addresses); BF16 x is quantized."""
        dev, k = self.device, self.k
        if x_scale is None:
            _address(x, "x", torch.bfloat16, (rows, k), dev)
            x, x_scale = _QUANTIZE[self.activation](x, stream=stream)
            kind = mx.MXFP4 if self.activation == mx.MXFP4 else self._mxfp8
            return kind, x, x_scale, x.data_ptr(), x_scale.data_ptr()
        kind = mx.MXFP4 if 2 * x.shape[1] == k else self._mxfp8
        px = _address(x, "x", torch.uint8, (rows, k // 2 if kind == mx.MXFP4 else k), dev)
        return kind, x, x_scale, px, _address(x_scale, "x_scale", torch.uint8, (rows, k // 32), dev)


class Linear(_RowsWeight):
    """A projection [n, k] in MXFP4 or MXFP8, packed once, for any number of rows
    (``Operands`` and ``publish`` are the projection of at most 8). gated: the rows are
    [gate; up], and a result is silu(gate) * up of them. activation ("mxfp4" or "mxfp8",
    by default the weight's format): what BF16 rows are quantized to. fast: products of MXFP8
    rows may lose what lies 2^-13 below the largest of eight (mxrows.h says when that
    matters); many rows then take about half the time."""

    def __init__(self, w: torch.Tensor, w_scale: torch.Tensor, gated: bool = False,
                 activation: str = None, stream=None, fast: bool = False) -> None:
        _refuse(w, "w", torch.uint8, (None, None), None)
        if not isinstance(w_scale, torch.Tensor) or w_scale.dim() != 2:
            raise ValueError("w_scale: a device tensor [n, k/32] is needed")
        self._pack(w.unsqueeze(0), w_scale.unsqueeze(0), gated, activation, fast, stream)

    def __call__(self, x: torch.Tensor, x_scale: torch.Tensor = None, out: torch.Tensor = None,
                 stream=None) -> torch.Tensor:
        """One mxrows_product call: uint8 codes [rows, k/2] or [rows, k] with x_scale
        [rows, k/32], or BF16 [rows, k], quantized first; BF16 [rows, n] (gated: n/2)."""
        dev = self.device
        handle = _on(dev, stream)
        rows = _matrix(x, "x").shape[0]
        kind, x, x_scale, px, ps = self._codes(x, x_scale, rows, stream)
        if out is None:
            out = _fresh(x, (rows, self.out_n), torch.bfloat16, stream)
        else:
            _address(out, "out", torch.bfloat16, (rows, self.out_n), dev)
        self._home.used(handle, stream)
        nbytes = _lib.mxrows_workspace_bytes(self._weight, kind, rows)
        workspace = _fresh(x, (nbytes,), torch.uint8, stream) if nbytes else None
        code = _lib.mxrows_product(self._weight, kind, px, ps, rows,
                                   workspace.data_ptr() if nbytes else None, nbytes,
                                   out.data_ptr(), handle)
        if code:
            mx._check(code, "mxrows_product")
        if stream is not None:
            _lend(stream, x, x_scale, out, workspace)
        return out


def sort_pairs(ids: torch.Tensor, experts: int, order: torch.Tensor = None,
               offsets: torch.Tensor = None, stream=None):
    """One mxmoe_sort call on a router's ids [tokens, top_k]: (order int32 [tokens *
    top_k], offsets int32 [experts + 1])."""
    tokens, top_k = _matrix(ids, "ids").shape
    _count(experts, "experts", mx.MOE_MAX_EXPERTS)
    dev = ids.device
    handle = _on(dev, stream)
    pi = _address(ids, "ids", torch.int32, (tokens, top_k), dev)
    if order is None:
        order = _fresh(ids, (tokens * top_k,), torch.int32, stream)
    else:
        _address(order, "order", torch.int32, (tokens * top_k,), dev)
    if offsets is None:
        offsets = _fresh(ids, (experts + 1,), torch.int32, stream)
    else:
        _address(offsets, "offsets", torch.int32, (experts + 1,), dev)
    nbytes = _lib.mxmoe_sort_workspace_bytes(tokens, top_k, experts)
    workspace = _fresh(ids, (nbytes,), torch.uint8, stream) if nbytes else None
    code = _lib.mxmoe_sort(pi, tokens, top_k, experts, workspace.data_ptr() if nbytes else None,
                           nbytes, order.data_ptr(), offsets.data_ptr(), handle)
    if code:
        mx._check(code, "mxmoe_sort")
    if stream is not None:
        _lend(stream, ids, order, offsets, workspace)
    return order, offsets


class GroupedLinear(_RowsWeight):
    """Every expert's projection in MXFP4 or MXFP8 (uint8 codes [experts, n, k/2] or
    [experts, n, k], scale bytes [experts, n, k/32]), packed once, on the rows of its
    pairs. gated, activation and fast: as ``Linear``."""

    def __init__(self, w: torch.Tensor, w_scale: torch.Tensor, gated: bool = False,
                 activation: str = None, stream=None, fast: bool = False) -> None:
        self._pack(w, w_scale, gated, activation, fast, stream)

    def __call__(self, x: torch.Tensor, x_scale, offsets: torch.Tensor,
                 order: torch.Tensor = None, gather: int = 0, scatter: bool = False,
                 out: torch.Tensor = None, stream=None) -> torch.Tensor:
        """One mxmoe_grouped call. x, x_scale: codes, or BF16 rows and None; offsets and
        order: of ``sort_pairs``. gather (a router's top_k): sorted row i is x[order[i] //
        gather], else x[i]; scatter: its result is row order[i], else row i. BF16 [rows, n]
        (gated: n/2), a row for each of order's, or of x without one; rows without an
        expert are left as they were."""
        dev = self.device
        handle = _on(dev, stream)
        x_rows = _matrix(x, "x").shape[0]
        _count(gather, "gather", mx.ROUTE_MAX_TOP_K)
        rows = x_rows
        po = None
        if order is not None:
            rows = order.numel() if isinstance(order, torch.Tensor) else None
            po = _address(order, "order", torch.int32, (rows,), dev)
            _count(rows, "order's length", mx.ROWS_MAX)
        poff = _address(offsets, "offsets", torch.int32, (self.experts + 1,), dev)
        kind, x, x_scale, px, ps = self._codes(x, x_scale, x_rows, stream)
        if out is None:
            out = _fresh(x, (rows, self.out_n), torch.bfloat16, stream)
        else:
            _address(out, "out", torch.bfloat16, (rows, self.out_n), dev)
        self._home.used(handle, stream)
        code = _lib.mxmoe_grouped(self._weight, kind, px, ps, x_rows, po, gather, int(scatter),
                                  poff, rows, out.data_ptr(), handle)
        if code:
            mx._check(code, "mxmoe_grouped")
        if stream is not None:
            _lend(stream, x, x_scale, offsets, order, out)
        return out


def combine(y: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, experts: int,
            out: torch.Tensor = None, stream=None) -> torch.Tensor:
    """One mxmoe_combine call: BF16 y [tokens * top_k, hidden] (a row for each pair), ids
    and weights as ``route`` returns them; BF16 [tokens, hidden]."""
    tokens, top_k = _matrix(ids, "ids").shape
    hidden = _matrix(y, "y").shape[1]
    _count(experts, "experts", mx.MOE_MAX_EXPERTS)
    dev = y.device
    handle = _on(dev, stream)
    py = _address(y, "y", torch.bfloat16, (tokens * top_k, hidden), dev)
    pi = _address(ids, "ids", torch.int32, (tokens, top_k), dev)
    pw = _address(weights, "weights", torch.float32, (tokens, top_k), dev)
    if out is None:
        out = _fresh(y, (tokens, hidden), torch.bfloat16, stream)
    else:
        _address(out, "out", torch.bfloat16, (tokens, hidden), dev)
    code = _lib.mxmoe_combine(py, pi, pw, tokens, top_k, experts, hidden, out.data_ptr(), handle)
    if code:
        mx._check(code, "mxmoe_combine")
    if stream is not None:
        _lend(stream, y, ids, weights, out)
    return out


class PromptExperts:
    """The experts of one layer on a prompt's rows, where ``Experts`` takes a decode step's
    (at most 1024 pairs): w13 [experts, 2 inter, hidden] (gate rows, then up rows) and w2
    [experts, hidden, inter] in MXFP4 or MXFP8, packed once. activation ("mxfp4" or "mxfp8",
    by default each weight's format): what the rows of both products are quantized to. fast:
    as ``Linear``."""

    def __init__(self, w13: torch.Tensor, w13_scale: torch.Tensor, w2: torch.Tensor,
                 w2_scale: torch.Tensor, activation: str = None, stream=None,
                 fast: bool = False) -> None:
        self.up = GroupedLinear(w13, w13_scale, gated=True, activation=activation, stream=stream,
                                fast=fast)
        self.down = GroupedLinear(w2, w2_scale, activation=activation, stream=stream, fast=fast)
        self.experts, self.hidden, self.inter = self.up.experts, self.up.k, self.up.out_n
        if (self.down.experts, self.down.n, self.down.k) != (self.experts, self.hidden, self.inter):
            raise ValueError("w2: [experts, hidden, inter] of w13 is needed")

    def __call__(self, x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor,
                 out: torch.Tensor = None, stream=None) -> torch.Tensor:
        """BF16 x [tokens, hidden], ids and weights as ``route`` returns them; BF16 [tokens,
        hidden]: sort_pairs, both products with the rows quantized before each, combine."""
        tokens, top_k = _matrix(ids, "ids").shape
        if _matrix(x, "x").shape[0] != tokens:
            raise ValueError(f"x: {x.shape[0]} rows for the choices of {tokens} tokens")
        order, offsets = sort_pairs(ids, self.experts, stream=stream)
        h = self.up(x, None, offsets, order, gather=top_k, stream=stream)
        y = self.down(h, None, offsets, order, scatter=True, stream=stream)
        return combine(y, ids, weights, self.experts, out, stream)
