"""Thin Python binding of libsb (include/sb.h): argument marshalling only.

Every step of the head runs in libsb's HIP kernels.  PyTorch provides device
memory and the stream; this module builds the C descriptor from tensors,
allocates the workspace through torch when none is given, and raises
``SbError`` on a non-zero status.  A workspace allocated here is allocated on
the call's stream and recorded as used by it.  There is no fallback: if libsb.so is
missing, loading fails with an error.
"""
import contextlib
import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsb.so")

SB_OK = 0
SB_ERR_NULL = -1
SB_ERR_SHAPE = -2
SB_ERR_LANES = -3
SB_ERR_ALIGN = -4
SB_ERR_WORKSPACE = -5
SB_ERR_UNSUPPORTED = -6
SB_ERR_HIP = -7

SB_SURF_TOKENS = 0
SB_SURF_LOGPROBS = 1
SB_SURF_LOGPROBS_FULL = 2
SB_SURF_FULL_LOGITS = 3

SB_MAX_LANES = 64

SB_FP32 = 0
SB_BF16 = 1

SB_RED_SUM = 0
SB_RED_PROD = 1
SB_RED_MIN = 2
SB_RED_MAX = 3
REDUCE_OPS = {"sum": SB_RED_SUM, "prod": SB_RED_PROD, "min": SB_RED_MIN, "max": SB_RED_MAX}

EXPORTS = ("sb_workspace_bytes", "sb_project_tokens", "sb_project_tokens_static",
           "sb_project_lane_results",
           "sb_project_logprobs", "sb_full_logits", "sb_partial_workspace_bytes",
           "sb_partial_complete", "sb_cross_entropy_workspace_bytes", "sb_cross_entropy",
           "sb_cross_entropy_grad", "sb_int8_quantize_rows", "sb_int8_quantize_head",
           "sb_int8_workspace_bytes", "sb_int8_project_tokens", "sb_int8_logits",
           "sb_layer_norm", "sb_layer_norm_grad_workspace_bytes", "sb_layer_norm_grad",
           "sb_embed", "sb_embed_grad_workspace_bytes", "sb_embed_grad",
           "sb_verify_workspace_bytes", "sb_verify_drafts", "sb_status_string")


class SbError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


class sb_head_desc(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int32), ("H", ctypes.c_int32),
        ("V", ctypes.c_int32), ("k", ctypes.c_int32),
        ("lane_off", ctypes.POINTER(ctypes.c_int32)),
        ("x", ctypes.c_void_p), ("ldx", ctypes.c_int64),
        ("w", ctypes.POINTER(ctypes.c_void_p)), ("ldw", ctypes.c_int64),
    ]


class sb_partial_desc(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int32), ("N", ctypes.c_int32), ("k", ctypes.c_int32),
        ("lane_k", ctypes.POINTER(ctypes.c_int32)),
        ("x", ctypes.POINTER(ctypes.c_void_p)), ("ldx", ctypes.c_int64),
        ("w", ctypes.POINTER(ctypes.c_void_p)), ("ldw", ctypes.c_int64),
    ]


class sb_int8_desc(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int32), ("H", ctypes.c_int32),
        ("V", ctypes.c_int32), ("k", ctypes.c_int32),
        ("lane_off", ctypes.POINTER(ctypes.c_int32)),
        ("x", ctypes.c_void_p), ("ldx", ctypes.c_int64), ("x_scale", ctypes.c_void_p),
        ("w", ctypes.POINTER(ctypes.c_void_p)), ("ldw", ctypes.c_int64),
        ("w_scale", ctypes.POINTER(ctypes.c_void_p)),
    ]


class sb_norm_desc(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int32), ("H", ctypes.c_int32),
        ("x", ctypes.c_void_p), ("x_type", ctypes.c_int), ("ldx", ctypes.c_int64),
        ("weight", ctypes.c_void_p), ("bias", ctypes.c_void_p), ("param_type", ctypes.c_int),
        ("eps", ctypes.c_float),
    ]


class sb_table_desc(ctypes.Structure):
    _fields_ = [
        ("V", ctypes.c_int32), ("H", ctypes.c_int32), ("k", ctypes.c_int32),
        ("lane_off", ctypes.POINTER(ctypes.c_int32)),
        ("w", ctypes.POINTER(ctypes.c_void_p)), ("ldw", ctypes.c_int64), ("type", ctypes.c_int),
    ]


class sb_drafts_desc(ctypes.Structure):
    _fields_ = [
        ("N", ctypes.c_int32), ("K", ctypes.c_int32), ("V", ctypes.c_int32), ("drafts", ctypes.c_int32),
        ("offsets", ctypes.c_void_p), ("tokens", ctypes.c_void_p),
        ("target", ctypes.c_void_p), ("ldt", ctypes.c_int64),
        ("draft", ctypes.c_void_p), ("ldd", ctypes.c_int64), ("type", ctypes.c_int),
        ("temperature", ctypes.c_void_p),
    ]


_lib = None


def lib():
    """The loaded libsb.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            f"libsb.so not found at {LIB_PATH}; build it first "
            "(python -c 'import __graft_entry__ as g; g.build()')")
    L = ctypes.CDLL(LIB_PATH)
    P = ctypes.POINTER(sb_head_desc)
    vp, i64, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t
    L.sb_workspace_bytes.restype = sz
    L.sb_workspace_bytes.argtypes = [P, ctypes.c_int, ctypes.POINTER(ctypes.c_int)]
    L.sb_project_tokens.restype = ctypes.c_int
    L.sb_project_tokens.argtypes = [P, vp, vp, sz, vp]
    L.sb_project_tokens_static.restype = ctypes.c_int
    L.sb_project_tokens_static.argtypes = [P, vp, vp]
    L.sb_project_lane_results.restype = ctypes.c_int
    L.sb_project_lane_results.argtypes = [P, vp, vp, vp, vp, sz, vp]
    L.sb_project_logprobs.restype = ctypes.c_int
    L.sb_project_logprobs.argtypes = [P, vp, vp, vp, vp, i64, vp, sz, vp]
    L.sb_full_logits.restype = ctypes.c_int
    L.sb_full_logits.argtypes = [P, vp, i64, vp, vp, sz, vp]
    PP = ctypes.POINTER(sb_partial_desc)
    L.sb_partial_workspace_bytes.restype = sz
    L.sb_partial_workspace_bytes.argtypes = [PP, ctypes.POINTER(ctypes.c_int)]
    L.sb_partial_complete.restype = ctypes.c_int
    L.sb_partial_complete.argtypes = [PP, ctypes.c_int, vp, i64, vp, sz, vp]
    L.sb_cross_entropy_workspace_bytes.restype = sz
    L.sb_cross_entropy_workspace_bytes.argtypes = [P, ctypes.c_int, ctypes.POINTER(ctypes.c_int)]
    L.sb_cross_entropy.restype = ctypes.c_int
    L.sb_cross_entropy.argtypes = [P, vp, vp, vp, vp, sz, vp]
    L.sb_cross_entropy_grad.restype = ctypes.c_int
    L.sb_cross_entropy_grad.argtypes = [P, vp, vp, vp, vp, i64, ctypes.POINTER(vp), i64, vp, sz,
                                        vp]
    PI, pvp, i32 = ctypes.POINTER(sb_int8_desc), ctypes.POINTER(vp), ctypes.c_int32
    L.sb_int8_quantize_rows.restype = ctypes.c_int
    L.sb_int8_quantize_rows.argtypes = [vp, i64, i32, i32, vp, i64, vp, vp]
    L.sb_int8_quantize_head.restype = ctypes.c_int
    L.sb_int8_quantize_head.argtypes = [P, pvp, i64, pvp, vp]
    L.sb_int8_workspace_bytes.restype = sz
    L.sb_int8_workspace_bytes.argtypes = [PI, ctypes.c_int, ctypes.POINTER(ctypes.c_int)]
    L.sb_int8_project_tokens.restype = ctypes.c_int
    L.sb_int8_project_tokens.argtypes = [PI, vp, vp, sz, vp]
    L.sb_int8_logits.restype = ctypes.c_int
    L.sb_int8_logits.argtypes = [PI, vp, ctypes.c_int, i64, vp, sz, vp]
    PN = ctypes.POINTER(sb_norm_desc)
    L.sb_layer_norm.restype = ctypes.c_int
    L.sb_layer_norm.argtypes = [PN, vp, ctypes.c_int, i64, vp, vp, vp]
    L.sb_layer_norm_grad_workspace_bytes.restype = sz
    L.sb_layer_norm_grad_workspace_bytes.argtypes = [PN, ctypes.POINTER(ctypes.c_int)]
    L.sb_layer_norm_grad.restype = ctypes.c_int
    L.sb_layer_norm_grad.argtypes = [PN, vp, ctypes.c_int, i64, vp, vp, vp, i64, vp, vp, vp, sz, vp]
    PT, f32, cint = ctypes.POINTER(sb_table_desc), ctypes.c_float, ctypes.c_int
    L.sb_embed.restype = cint
    L.sb_embed.argtypes = [PT, vp, i32, f32, vp, cint, i64, vp]
    L.sb_embed_grad_workspace_bytes.restype = sz
    L.sb_embed_grad_workspace_bytes.argtypes = [PT, i32, cint, ctypes.POINTER(cint)]
    L.sb_embed_grad.restype = cint
    L.sb_embed_grad.argtypes = [PT, vp, i32, f32, vp, cint, i64, cint, vp, sz, vp]
    PD = ctypes.POINTER(sb_drafts_desc)
    L.sb_verify_workspace_bytes.restype = sz
    L.sb_verify_workspace_bytes.argtypes = [PD, ctypes.POINTER(cint)]
    L.sb_verify_drafts.restype = cint
    L.sb_verify_drafts.argtypes = [PD, vp, vp, vp, i64, vp, vp, sz, vp]
    L.sb_status_string.restype = ctypes.c_char_p
    L.sb_status_string.argtypes = [ctypes.c_int]
    _lib = L
    return L


def status_string(status):
    return lib().sb_status_string(int(status)).decode()


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


# Argument checks of the binding: a host tensor, a wrong dtype or a strided
# layout the C ABI cannot express would otherwise reach a kernel as a raw
# pointer.  They raise before anything is enqueued.
def _device(t, name, dtype):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")


def _vector(t, name, dtype, n):
    """A contiguous device buffer of at least n elements (None allowed)."""
    if t is None:
        return
    _device(t, name, dtype)
    if not t.is_contiguous() or t.numel() < n:
        raise ValueError(f"{name} must be contiguous with at least {n} elements")


def _matrix(t, name, dtype, rows, cols):
    """A [>= rows, >= cols] device matrix with unit column stride (None allowed)."""
    if t is None:
        return
    _device(t, name, dtype)
    if t.dim() != 2 or t.shape[0] < rows or t.shape[1] < cols or (
            t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be a [>= {rows}, >= {cols}] matrix with unit column stride")


def _holds(t, name, rows, cols):
    if t.dim() != 2 or t.shape[0] < rows or t.shape[1] < cols:
        raise ValueError(f"{name} must be a [>= {rows}, >= {cols}] matrix, not {list(t.shape)}")


def _operands(tensors, name):
    """The bf16 operands a descriptor was built from: on the device, rows
    with unit column stride."""
    for t in tensors:
        _device(t, name, torch.bfloat16)
        if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
            raise ValueError(f"{name} must be 2-D with unit column stride")


def _stream(stream):
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


class Head:
    """Descriptor of a head: hidden rows x [B, H] (bf16) and the lane shards.

    ``w`` is either one [H, V] bf16 tensor (lanes are column ranges of it;
    every lane offset must then be a multiple of 8) or a list of k tensors,
    lane i of shape [H, V_i] with one common row stride.  ``lane_off`` holds
    the k+1 vocab offsets.  Raw values (pointers, strides) can be overridden
    to exercise the ABI's validation.
    """

    def __init__(self, x, w, lane_off, *, B=None, H=None, V=None, ldx=None,
                 ldw=None, x_ptr=None, w_ptrs=None):
        self.x = x
        self.w = w
        # built from tensors (checked on every call) or from raw pointers
        self.from_tensors = x_ptr is None and w_ptrs is None
        self._device = None
        off = [int(o) for o in lane_off]
        self.lane_off = off
        k = len(off) - 1
        self._off = (ctypes.c_int32 * max(1, k + 1))(*off)
        if isinstance(w, (list, tuple)):
            ptrs = [t.data_ptr() for t in w]
            stride = w[0].stride(0) if len(w) else 0
        else:
            base = w.data_ptr()
            ptrs = [base + 2 * off[i] for i in range(k)]
            stride = w.stride(0)
        if w_ptrs is not None:
            ptrs = list(w_ptrs)
        self._w = (ctypes.c_void_p * max(1, len(ptrs)))(*ptrs)
        self.desc = sb_head_desc(
            B=x.shape[0] if B is None else B,
            H=x.shape[1] if H is None else H,
            V=off[-1] if V is None else V,
            k=k,
            lane_off=self._off,
            x=x.data_ptr() if x_ptr is None else x_ptr,
            ldx=x.stride(0) if ldx is None else ldx,
            w=self._w,
            ldw=stride if ldw is None else ldw)

    @property
    def B(self):
        return self.desc.B

    @property
    def V(self):
        return self.desc.V

    def ref(self):
        return ctypes.byref(self.desc)

    def check(self):
        if self.from_tensors:
            _operands([self.x], "x")
            _operands(self.w if isinstance(self.w, (list, tuple)) else [self.w], "w")

    def check_shapes(self):
        """The operands hold what the descriptor says."""
        d, off = self.desc, self.lane_off
        _holds(self.x, "x", d.B, d.H)
        if isinstance(self.w, (list, tuple)):
            if len(self.w) != len(off) - 1:
                raise ValueError(f"w must hold one tensor per lane, {len(off) - 1}")
            for i, t in enumerate(self.w):
                _holds(t, f"w[{i}]", d.H, off[i + 1] - off[i])
            if d.H > 1 and len({t.stride(0) for t in self.w}) > 1:
                raise ValueError("the tensors of w must have one row stride")
        else:
            _holds(self.w, "w", d.H, off[-1])

    def device(self):
        """The one device of the operands (None for raw pointers).  The
        descriptor holds their addresses, so their shapes are checked once."""
        if self._device is None and self.from_tensors:
            self.check_shapes()
            self._device = _one_device([self.x] + _as_list(self.w))
        return self._device


def sb_workspace_bytes(head, surface):
    st = ctypes.c_int(0)
    n = lib().sb_workspace_bytes(head.ref(), int(surface), ctypes.byref(st))
    if st.value != SB_OK:
        raise SbError(st.value, "sb_workspace_bytes")
    return int(n)


def workspace(head, surface, device="cuda"):
    """A workspace for `surface` (its contents on entry do not matter: every
    call clears what it relies on)."""
    n = sb_workspace_bytes(head, surface)
    return torch.empty(max(n, 16), dtype=torch.uint8, device=device)


def _workspace(nbytes_fn, ws, device, stream):
    """The caller's workspace, or a temporary one allocated on the call's
    stream and marked as used by it, so that the caching allocator does not
    hand its memory to other work before the call's kernels are done."""
    if ws is not None:
        return ws
    s = _torch_stream(stream, device)
    with torch.cuda.stream(s):
        t = torch.empty(max(nbytes_fn(), 16), dtype=torch.uint8, device=device)
    t.record_stream(s)
    return t


def _torch_stream(stream, device):
    if stream is None:
        return torch.cuda.current_stream(device)
    if isinstance(stream, torch.cuda.Stream):
        return stream
    return torch.cuda.ExternalStream(int(stream), device=device)


def _check(status, where):
    if status != SB_OK:
        raise SbError(status, where)


def sb_project_tokens(head, ids, ws=None, stream=None):
    """Token-only surface: ids (int32 [B], device) <- argmax token IDs."""
    head.check()
    _vector(ids, "ids", torch.int32, head.B)
    _vector(ws, "ws", torch.uint8, 0)
    ws = _workspace(lambda: sb_workspace_bytes(head, SB_SURF_TOKENS), ws, ids.device, stream)
    _check(lib().sb_project_tokens(head.ref(), _ptr(ids), _ptr(ws), ws.numel(),
                                   _stream(stream)), "sb_project_tokens")
    return ids


def sb_project_tokens_static(head, ids, stream=None):
    """Token-only surface with the library's static device scratch as the
    workspace (no allocation; SB_STATIC_SCRATCH_BYTES at most)."""
    head.check()
    _vector(ids, "ids", torch.int32, head.B)
    _check(lib().sb_project_tokens_static(head.ref(), _ptr(ids), _stream(stream)),
           "sb_project_tokens_static")
    return ids


SB_STATIC_SCRATCH_BYTES = 32 << 20


def sb_project_lane_results(head, ids, lane_ids=None, lane_max=None, ws=None, stream=None):
    """Token surface plus each lane's own result: lane_ids (int32 [B, k]) and
    lane_max (fp32 [B, k]) of every row, either optional."""
    head.check()
    k = head.desc.k
    _vector(ids, "ids", torch.int32, head.B)
    _vector(lane_ids, "lane_ids", torch.int32, head.B * k)
    _vector(lane_max, "lane_max", torch.float32, head.B * k)
    _vector(ws, "ws", torch.uint8, 0)
    ws = _workspace(lambda: sb_workspace_bytes(head, SB_SURF_TOKENS), ws, ids.device, stream)
    _check(lib().sb_project_lane_results(head.ref(), _ptr(ids), _ptr(lane_ids), _ptr(lane_max),
                                         _ptr(ws), ws.numel(), _stream(stream)),
           "sb_project_lane_results")
    return ids


def sb_project_logprobs(head, ids, lse, sel_lp=None, logprobs=None, ws=None,
                        stream=None):
    """Log-probability surface: ids, lse, optional sel_lp and complete
    fp32 log-probs [B, V] (row stride logprobs.stride(0))."""
    head.check()
    _vector(ids, "ids", torch.int32, head.B)
    _vector(lse, "lse", torch.float32, head.B)
    _vector(sel_lp, "sel_lp", torch.float32, head.B)
    _matrix(logprobs, "logprobs", torch.float32, head.B, head.V)
    _vector(ws, "ws", torch.uint8, 0)
    surf = SB_SURF_LOGPROBS_FULL if logprobs is not None else SB_SURF_LOGPROBS
    ws = _workspace(lambda: sb_workspace_bytes(head, surf), ws, ids.device, stream)
    ld = logprobs.stride(0) if logprobs is not None else 0
    _check(lib().sb_project_logprobs(head.ref(), _ptr(ids), _ptr(lse), _ptr(sel_lp),
                                     _ptr(logprobs), ld, _ptr(ws), ws.numel(),
                                     _stream(stream)), "sb_project_logprobs")
    return ids


def sb_full_logits(head, logits, ids=None, ws=None, stream=None):
    """Full-logit plan: logits fp32 [B, V] (row stride logits.stride(0)),
    optional ids."""
    head.check()
    _matrix(logits, "logits", torch.float32, head.B, head.V)
    _vector(ids, "ids", torch.int32, head.B)
    _vector(ws, "ws", torch.uint8, 0)
    ws = _workspace(lambda: sb_workspace_bytes(head, SB_SURF_FULL_LOGITS), ws, logits.device,
                    stream)
    _check(lib().sb_full_logits(head.ref(), _ptr(logits), logits.stride(0), _ptr(ids),
                                _ptr(ws), ws.numel(), _stream(stream)), "sb_full_logits")
    return logits


class Partial:
    """Descriptor of a row-parallel partial-completion boundary: k activation
    shards x[i] [B, K_i] (bf16, one common row stride) and weight blocks
    w[i] [K_i, N] (bf16, one common row stride).  Raw values can be
    overridden to exercise the ABI's validation."""

    def __init__(self, x, w, *, B=None, N=None, lane_k=None, ldx=None, ldw=None,
                 x_ptrs=None, w_ptrs=None):
        self.x, self.w = list(x), list(w)
        # built from tensors (checked on every call) or from raw pointers
        self.from_tensors = x_ptrs is None and w_ptrs is None
        Ks = [t.shape[1] for t in self.x]
        off = [0]
        for kk in Ks:
            off.append(off[-1] + kk)
        if lane_k is not None:
            off = [int(o) for o in lane_k]
        k = len(off) - 1
        self._off = (ctypes.c_int32 * max(1, k + 1))(*off)
        xp = [t.data_ptr() for t in self.x] if x_ptrs is None else list(x_ptrs)
        wp = [t.data_ptr() for t in self.w] if w_ptrs is None else list(w_ptrs)
        self._x = (ctypes.c_void_p * max(1, len(xp)))(*xp)
        self._w = (ctypes.c_void_p * max(1, len(wp)))(*wp)
        self.desc = sb_partial_desc(
            B=self.x[0].shape[0] if B is None else B,
            N=self.w[0].shape[1] if N is None else N,
            k=k, lane_k=self._off, x=self._x,
            ldx=self.x[0].stride(0) if ldx is None else ldx,
            w=self._w,
            ldw=self.w[0].stride(0) if ldw is None else ldw)

    @property
    def B(self):
        return self.desc.B

    @property
    def N(self):
        return self.desc.N

    def ref(self):
        return ctypes.byref(self.desc)

    def check(self):
        if self.from_tensors:
            _operands(self.x, "x")
            _operands(self.w, "w")


def sb_partial_workspace_bytes(part):
    st = ctypes.c_int(0)
    n = lib().sb_partial_workspace_bytes(part.ref(), ctypes.byref(st))
    if st.value != SB_OK:
        raise SbError(st.value, "sb_partial_workspace_bytes")
    return int(n)


def sb_partial_complete(part, op, out, ws=None, stream=None):
    """out (fp32 [B, N], row stride out.stride(0)) <- the registered
    reduction `op` ("sum", "prod", "min", "max" or an SB_RED_* code) of the
    lane partials."""
    code = REDUCE_OPS[op] if isinstance(op, str) else int(op)
    part.check()
    _matrix(out, "out", torch.float32, part.B, part.N)
    _vector(ws, "ws", torch.uint8, 0)
    ws = _workspace(lambda: sb_partial_workspace_bytes(part), ws, out.device, stream)
    _check(lib().sb_partial_complete(part.ref(), code, _ptr(out), out.stride(0), _ptr(ws),
                                     ws.numel(), _stream(stream)), "sb_partial_complete")
    return out


# ---------------------------------------------------------------------------
# Training surface.  These calls run on the device of their tensors, whatever
# the current one is; a stream that is not given is that device's current one, and a
# given one has to be that device's.
# ---------------------------------------------------------------------------
def _one_device(tensors, device=None):
    """The device that holds every tensor of a call (and the operands of its
    descriptor, `device`)."""
    for t in tensors:
        if t is None:
            continue
        if device is None:
            device = t.device
        elif t.device != device:
            raise ValueError(f"tensors on different devices: {device} and {t.device}")
    return device


def _as_list(w):
    return list(w) if isinstance(w, (list, tuple)) else [w]


def _on(device):
    """`device` made current for the block (no-op where it already is)."""
    if device.index == torch.cuda.current_device():
        return contextlib.nullcontext()
    return torch.cuda.device(device)


def _stream_on(stream, device):
    """The stream's handle: the given one's, or the device's current one's
    (taken as a number: a torch.cuda.Stream object costs 3 us a call)."""
    if stream is None:
        return ctypes.c_void_p(torch._C._cuda_getCurrentRawStream(device.index))
    if getattr(stream, "device", device) != device:
        raise ValueError(f"a stream of {stream.device} for tensors on {device}")
    return _stream(stream)


def _run(name, device, stream, nbytes_fn, ws, call):
    """call(workspace pointer, its size, stream) on `device`."""
    with _on(device):
        s = _stream_on(stream, device)
        if ws is None:
            ws = _workspace(nbytes_fn, ws, device, stream)
        _check(call(ws.data_ptr(), ws.numel(), s), name)


def sb_cross_entropy_workspace_bytes(head, grad):
    st = ctypes.c_int(0)
    n = lib().sb_cross_entropy_workspace_bytes(head.ref(), int(bool(grad)), ctypes.byref(st))
    if st.value != SB_OK:
        raise SbError(st.value, "sb_cross_entropy_workspace_bytes")
    return int(n)


def cross_entropy_workspace(head, grad=False, device=None):
    """A workspace for sb_cross_entropy, or with grad for sb_cross_entropy_grad
    (its contents on entry do not matter)."""
    return torch.empty(max(sb_cross_entropy_workspace_bytes(head, grad), 16), dtype=torch.uint8,
                       device=head.x.device if device is None else device)


def sb_cross_entropy(head, targets, loss, lse, ws=None, stream=None):
    """loss and lse (fp32 [B]) <- softmax cross entropy of every row with its
    target (int32 [B]; negative = ignored, loss 0).  Returns loss."""
    head.check()
    B = head.B
    _vector(targets, "targets", torch.int32, B)
    _vector(loss, "loss", torch.float32, B)
    _vector(lse, "lse", torch.float32, B)
    _vector(ws, "ws", torch.uint8, 0)
    dev = _one_device([targets, loss, lse, ws], head.device())
    _run("sb_cross_entropy", dev, stream, lambda: sb_cross_entropy_workspace_bytes(head, False), ws,
         lambda p, n, s: lib().sb_cross_entropy(head.ref(), _ptr(targets), _ptr(loss), _ptr(lse), p,
                                                n, s))
    return loss


def sb_cross_entropy_grad(head, targets, lse, dloss, dx=None, dw=None, ws=None, stream=None):
    """dx (bf16 [B, H]) and / or dw <- the gradient of sum(dloss * loss).  dw
    has the head weight's form: one bf16 [H, V] tensor, or a list of one
    [H, V_i] tensor per lane with a common row stride.  lse is what
    sb_cross_entropy returned; dloss (fp32 [B]) the gradient of each row's
    loss.  Returns (dx, dw)."""
    head.check()
    B, H, V, off = head.B, head.desc.H, head.V, head.lane_off
    _vector(targets, "targets", torch.int32, B)
    _vector(lse, "lse", torch.float32, B)
    _vector(dloss, "dloss", torch.float32, B)
    _matrix(dx, "dx", torch.bfloat16, B, H)
    _vector(ws, "ws", torch.uint8, 0)
    dws, ptrs, lddw = [], None, 0
    if isinstance(dw, (list, tuple)):
        dws = list(dw)
        if len(dws) != len(off) - 1:
            raise ValueError(f"dw must hold one tensor per lane, {len(off) - 1}")
        for i, t in enumerate(dws):
            _matrix(t, f"dw[{i}]", torch.bfloat16, H, off[i + 1] - off[i])
        if len({t.stride(0) for t in dws}) > 1:
            raise ValueError("the tensors of dw must have one row stride")
        ptrs, lddw = [t.data_ptr() for t in dws], dws[0].stride(0)
    elif dw is not None:
        _matrix(dw, "dw", torch.bfloat16, H, V)
        dws = [dw]
        ptrs, lddw = [dw.data_ptr() + 2 * o for o in off[:-1]], dw.stride(0)
    arr = None if ptrs is None else (ctypes.c_void_p * len(ptrs))(*ptrs)
    dev = _one_device([targets, lse, dloss, dx, ws] + dws, head.device())
    _run("sb_cross_entropy_grad", dev, stream,
         lambda: sb_cross_entropy_workspace_bytes(head, True), ws,
         lambda p, n, s: lib().sb_cross_entropy_grad(
             head.ref(), _ptr(targets), _ptr(lse), _ptr(dloss), _ptr(dx),
             0 if dx is None else dx.stride(0), arr, lddw, p, n, s))
    return dx, dw


# ---------------------------------------------------------------------------
# The head in 8-bit integers.
# ---------------------------------------------------------------------------
class Int8Head:
    """Descriptor of an 8-bit head: row codes x [B, H] (int8) with scales
    x_scale [B], and the channels of every lane with their scales.

    ``w`` is either one [V, H] int8 tensor with w_scale [V], or lists of k
    tensors, lane i of shape [V_i, H] (one common row stride) and [V_i].
    ``lane_off`` holds the k+1 vocab offsets.  Row strides are multiples of
    16.  Raw values can be overridden to exercise the ABI's validation."""

    def __init__(self, x, x_scale, w, w_scale, lane_off, *, B=None, H=None, V=None, ldx=None,
                 ldw=None, x_ptr=None, x_scale_ptr=None, w_ptrs=None, w_scale_ptrs=None):
        self.x, self.x_scale, self.w, self.w_scale = x, x_scale, w, w_scale
        self.from_tensors = x_ptr is None and w_ptrs is None
        self._device = None
        off = [int(o) for o in lane_off]
        self.lane_off = off
        k = len(off) - 1
        self._off = (ctypes.c_int32 * max(1, k + 1))(*off)
        if w_ptrs is not None:
            wp, sp, stride = list(w_ptrs), list(w_scale_ptrs), 0
        elif isinstance(w, (list, tuple)):
            if len(w) != k or len(w_scale) != k:
                raise ValueError(f"w and w_scale must hold one tensor per lane, {k}")
            wp, sp = [t.data_ptr() for t in w], [t.data_ptr() for t in w_scale]
            stride = w[0].stride(0)
        else:
            stride = w.stride(0)
            wp = [w.data_ptr() + stride * o for o in off[:-1]]
            sp = [w_scale.data_ptr() + 4 * o for o in off[:-1]]
        self._w = (ctypes.c_void_p * max(1, len(wp)))(*wp)
        self._ws = (ctypes.c_void_p * max(1, len(sp)))(*sp)
        self.desc = sb_int8_desc(
            B=x.shape[0] if B is None else B,
            H=x.shape[1] if H is None else H,
            V=off[-1] if V is None else V,
            k=k, lane_off=self._off,
            x=x.data_ptr() if x_ptr is None else x_ptr,
            ldx=x.stride(0) if ldx is None else ldx,
            x_scale=x_scale.data_ptr() if x_scale_ptr is None else x_scale_ptr,
            w=self._w, ldw=stride if ldw is None else ldw, w_scale=self._ws)

    @property
    def B(self):
        return self.desc.B

    @property
    def V(self):
        return self.desc.V

    def ref(self):
        return ctypes.byref(self.desc)

    def check(self):
        if not self.from_tensors or self._device is not None:
            return
        d, off = self.desc, self.lane_off
        _matrix(self.x, "x", torch.int8, d.B, d.H)
        _vector(self.x_scale, "x_scale", torch.float32, d.B)
        if isinstance(self.w, (list, tuple)):
            for i, (t, s) in enumerate(zip(self.w, self.w_scale)):
                n = off[i + 1] - off[i]
                _matrix(t, f"w[{i}]", torch.int8, n, d.H)
                _vector(s, f"w_scale[{i}]", torch.float32, n)
            if len({t.stride(0) for t in self.w}) > 1:
                raise ValueError("the tensors of w must have one row stride")
        else:
            _matrix(self.w, "w", torch.int8, d.V, d.H)
            _vector(self.w_scale, "w_scale", torch.float32, d.V)

    def device(self):
        """The one device of the operands (None for raw pointers).  The
        descriptor holds their addresses, so they are checked once."""
        self.check()
        if self._device is None and self.from_tensors:
            self._device = _one_device([self.x, self.x_scale] + _as_list(self.w) +
                                       _as_list(self.w_scale))
        return self._device


def sb_int8_quantize_rows(x, q, scale, stream=None):
    """q (int8 [B, H]) and scale (fp32 [B]) <- the codes of the rows of x
    (bf16 [B, H]).  Returns (q, scale)."""
    _operands([x], "x")
    B, H = x.shape
    _matrix(q, "q", torch.int8, B, H)
    _vector(scale, "scale", torch.float32, B)
    device = _one_device([x, q, scale])
    with _on(device):
        _check(lib().sb_int8_quantize_rows(x.data_ptr(), x.stride(0), B, H, q.data_ptr(), q.stride(0),
                                           scale.data_ptr(), _stream_on(stream, device)),
               "sb_int8_quantize_rows")
    return q, scale


def sb_int8_quantize_head(head, q, scale, stream=None):
    """q and scale <- the codes of a bf16 head's weight, one channel per vocab
    column: int8 [V, H] and fp32 [V], or lists of one [V_i, H] and one [V_i]
    tensor per lane (one common row stride).  Returns (q, scale)."""
    head.check()
    off, H = head.lane_off, head.desc.H
    k = len(off) - 1
    if isinstance(q, (list, tuple)):
        if len(q) != k or len(scale) != k:
            raise ValueError(f"q and scale must hold one tensor per lane, {k}")
        for i, (t, s) in enumerate(zip(q, scale)):
            _matrix(t, f"q[{i}]", torch.int8, off[i + 1] - off[i], H)
            _vector(s, f"scale[{i}]", torch.float32, off[i + 1] - off[i])
        if len({t.stride(0) for t in q}) > 1:
            raise ValueError("the tensors of q must have one row stride")
        qp, sp, ldq = [t.data_ptr() for t in q], [t.data_ptr() for t in scale], q[0].stride(0)
    else:
        _matrix(q, "q", torch.int8, head.V, H)
        _vector(scale, "scale", torch.float32, head.V)
        ldq = q.stride(0)
        qp = [q.data_ptr() + ldq * o for o in off[:-1]]
        sp = [scale.data_ptr() + 4 * o for o in off[:-1]]
    device = _one_device(_as_list(q) + _as_list(scale), head.device())
    with _on(device):
        _check(lib().sb_int8_quantize_head(head.ref(), (ctypes.c_void_p * k)(*qp), ldq,
                                           (ctypes.c_void_p * k)(*sp), _stream_on(stream, device)),
               "sb_int8_quantize_head")
    return q, scale


def sb_int8_workspace_bytes(head, surface):
    st = ctypes.c_int(0)
    n = lib().sb_int8_workspace_bytes(head.ref(), int(surface), ctypes.byref(st))
    if st.value != SB_OK:
        raise SbError(st.value, "sb_int8_workspace_bytes")
    return int(n)


def int8_workspace(head, surface, device=None):
    """A workspace for `surface` (its contents on entry do not matter)."""
    return torch.empty(max(sb_int8_workspace_bytes(head, surface), 16), dtype=torch.uint8,
                       device=head.x.device if device is None else device)


def sb_int8_project_tokens(head, ids, ws=None, stream=None):
    """Greedy token IDs (int32 [B]) of the 8-bit head.  Returns ids."""
    device = head.device()
    _vector(ids, "ids", torch.int32, head.B)
    _vector(ws, "ws", torch.uint8, 0)
    dev = _one_device([ids, ws], device)
    _run("sb_int8_project_tokens", dev, stream,
         lambda: sb_int8_workspace_bytes(head, SB_SURF_TOKENS), ws,
         lambda p, n, s: lib().sb_int8_project_tokens(head.ref(), _ptr(ids), p, n, s))
    return ids


def sb_int8_logits(head, out, ws=None, stream=None):
    """out (fp32 or bf16 [B, V], row stride out.stride(0)) <- the scaled
    product.  Returns out."""
    device = head.device()
    if isinstance(out, torch.Tensor) and out.dtype == torch.bfloat16:
        _matrix(out, "out", torch.bfloat16, head.B, head.V)
    else:
        _matrix(out, "out", torch.float32, head.B, head.V)
    _vector(ws, "ws", torch.uint8, 0)
    dev = _one_device([out, ws], device)
    dtype = SB_BF16 if out.dtype == torch.bfloat16 else SB_FP32
    _run("sb_int8_logits", dev, stream,
         lambda: sb_int8_workspace_bytes(head, SB_SURF_FULL_LOGITS), ws,
         lambda p, n, s: lib().sb_int8_logits(head.ref(), _ptr(out), dtype, out.stride(0), p, n, s))
    return out


# ---------------------------------------------------------------------------
# Layer norm.  Like the training surface, these calls run on the device of their
# tensors; fp32 and bf16 tensors are taken as they are.
# ---------------------------------------------------------------------------
_TYPES = {torch.float32: SB_FP32, torch.bfloat16: SB_BF16}


def _on_device(t, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")


def _padded(n, size):
    """n columns rounded up to whole 16-byte units."""
    return -(-n * size // 16) * 16 // size


def _row_stride(t):
    """The stride between rows (a single row has none of its own: torch gives any)."""
    return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), _padded(t.shape[1], t.element_size()))


# The checks below also give what the C ABI takes; `index` is the number of the device that
# the call's other tensors are on, or None.  They are written out: at a few microseconds
# a call, those of several tensors are what a small call waits for.
def _rows(t, name, rows, cols, index=None, dtype=None):
    """(type code, address, row stride) of a [>= rows, >= cols] matrix with unit column
    stride, fp32 or bf16 or of the given type."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    code = _TYPES.get(t.dtype)
    if code is None and dtype is None:
        raise TypeError(f"{name} must be torch.float32 or torch.bfloat16, not {t.dtype}")
    if t.dim() != 2:
        raise ValueError(f"{name} must be a [>= {rows}, >= {cols}] matrix with unit column stride")
    (n, m), (s0, s1) = t.size(), t.stride()
    if n < rows or m < cols or (m > 1 and s1 != 1):
        raise ValueError(f"{name} must be a [>= {rows}, >= {cols}] matrix with unit column stride")
    if index is not None and t.get_device() != index:
        raise ValueError(f"tensors on different devices: cuda:{index} and {t.device}")
    return code, t.data_ptr(), s0 if n > 1 else max(s0, _padded(m, t.element_size()))


def _buffer(t, name, dtype, n, index=None):
    """The address of a contiguous buffer of at least n elements (None of None)."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if not t.is_contiguous() or t.numel() < n:
        raise ValueError(f"{name} must be contiguous with at least {n} elements")
    if index is not None and t.get_device() != index:
        raise ValueError(f"tensors on different devices: cuda:{index} and {t.device}")
    return t.data_ptr()


def _call(name, index, stream, fn, *args):
    """fn(*args, stream) on device `index`, which is made current for it where it is not."""
    if torch._C._cuda_getDevice() != index:
        with torch.cuda.device(index):
            return _call(name, index, stream, fn, *args)
    if stream is None:
        s = torch._C._cuda_getCurrentRawStream(index)
    else:
        s = _stream_on(stream, torch.device("cuda", index))
    _check(fn(*args, s), name)


def _space(ws, nbytes_fn, index, stream):
    """(address, bytes) of the caller's workspace or of one for this call, and the tensor
    that holds it."""
    if ws is None:
        device = torch.device("cuda", index)
        if stream is not None:
            _stream_on(stream, device)  # (one of another device is refused here already)
        with _on(device):
            ws = _workspace(nbytes_fn, None, device, stream)
    return _buffer(ws, "ws", torch.uint8, 0, index), ws.numel(), ws


class Norm:
    """Descriptor of a layer norm: rows x [B, H] (fp32 or bf16), and weight and
    bias [H] of one type (fp32 or bf16; None for 1 and 0).  Raw values can be
    overridden to exercise the ABI's validation."""

    def __init__(self, x, weight=None, bias=None, eps=1e-5, *, B=None, H=None, x_type=None, ldx=None,
                 x_ptr=None, weight_ptr=None, bias_ptr=None, param_type=None):
        self.x, self.weight, self.bias = x, weight, bias
        self.from_tensors = x_ptr is None
        self._index = None
        one = weight if weight is not None else bias
        self.param_dtype = torch.float32 if one is None else one.dtype
        self.desc = sb_norm_desc(
            B=x.shape[0] if B is None else B, H=x.shape[1] if H is None else H,
            x=x.data_ptr() if x_ptr is None else x_ptr,
            x_type=_TYPES.get(x.dtype, -1) if x_type is None else x_type,
            ldx=_row_stride(x) if ldx is None else ldx,
            weight=weight_ptr if weight is None else weight.data_ptr(),
            bias=bias_ptr if bias is None else bias.data_ptr(),
            param_type=_TYPES.get(self.param_dtype, -1) if param_type is None else param_type, eps=eps)

    @property
    def B(self):
        return self.desc.B

    @property
    def H(self):
        return self.desc.H

    def ref(self):
        return ctypes.byref(self.desc)

    def index(self):
        """The number of the operands' one device (None for raw pointers).  The
        descriptor holds their addresses, so they are checked once."""
        if self._index is None and self.from_tensors:
            d = self.desc
            _rows(self.x, "x", d.B, d.H)
            index = self.x.get_device()
            for t, name in ((self.weight, "weight"), (self.bias, "bias")):
                if t is not None:
                    _on_device(t, name)
                    if t.dtype not in _TYPES:
                        raise TypeError(f"{name} must be torch.float32 or torch.bfloat16, not {t.dtype}")
                    _buffer(t, name, self.param_dtype, d.H, index)
            self._index = index
        return self._index


def sb_layer_norm(norm, y, mean=None, rstd=None, stream=None):
    """y (fp32 or bf16 [B, H]) <- layer norm of the rows; mean and rstd (fp32
    [B], either optional) are what sb_layer_norm_grad takes.  Returns y."""
    index = norm.index()
    d = norm.desc
    B = d.B
    code, p, ld = _rows(y, "y", B, d.H, index)
    mean = _buffer(mean, "mean", torch.float32, B, index)
    rstd = _buffer(rstd, "rstd", torch.float32, B, index)
    _call("sb_layer_norm", y.get_device(), stream, lib().sb_layer_norm, norm.ref(), p, code, ld, mean, rstd)
    return y


def sb_layer_norm_grad_workspace_bytes(norm):
    st = ctypes.c_int(0)
    n = lib().sb_layer_norm_grad_workspace_bytes(norm.ref(), ctypes.byref(st))
    if st.value != SB_OK:
        raise SbError(st.value, "sb_layer_norm_grad_workspace_bytes")
    return int(n)


def layer_norm_grad_workspace(norm, device=None):
    """A workspace for sb_layer_norm_grad (its contents on entry do not matter)."""
    return torch.empty(max(sb_layer_norm_grad_workspace_bytes(norm), 16), dtype=torch.uint8,
                       device=norm.x.device if device is None else device)


def sb_layer_norm_grad(norm, dy, mean, rstd, dx=None, dweight=None, dbias=None, ws=None, stream=None):
    """dx ([B, H] of x's type), dweight and dbias ([H] of the parameters' type; fp32
    where there are none) <- the gradient of sum(dy * y), any of them optional.
    dy (fp32 or bf16 [B, H]) is of any type; mean and rstd are what
    sb_layer_norm returned.  Returns (dx, dweight, dbias)."""
    index = norm.index()
    d = norm.desc
    B, H = d.B, d.H
    code, pdy, lddy = _rows(dy, "dy", B, H, index)
    index = dy.get_device()
    mean = _buffer(mean, "mean", torch.float32, B, index)
    rstd = _buffer(rstd, "rstd", torch.float32, B, index)
    _, pdx, lddx = (None, None, 0) if dx is None else _rows(dx, "dx", B, H, index, norm.x.dtype)
    pw = _buffer(dweight, "dweight", norm.param_dtype, H, index)
    pb = _buffer(dbias, "dbias", norm.param_dtype, H, index)
    pws, n, ws = _space(ws, lambda: sb_layer_norm_grad_workspace_bytes(norm), index, stream)
    _call("sb_layer_norm_grad", index, stream, lib().sb_layer_norm_grad, norm.ref(), pdy, code, lddy, mean, rstd,
          pdx, lddx, pw, pb, pws, n)
    return dx, dweight, dbias


# ---------------------------------------------------------------------------
# Embedding.
# ---------------------------------------------------------------------------
def _counted(t, name, dtype, index=None):
    """(elements, address) of a contiguous buffer, as the C ABI counts them."""
    p = _buffer(t, name, dtype, 0, index)
    if t is None or t.numel() >= 1 << 31:
        raise ValueError(f"{name} must be a tensor of fewer than 2^31 elements")
    return t.numel(), p


class Table:
    """Descriptor of an embedding table, or of its gradient: one [V, H] tensor
    (fp32 or bf16), or a list of k tensors, lane i of shape [V_i, H] (one type
    and row stride).  ``lane_off`` holds the k+1 vocab offsets; one lane
    where it is not given.  Raw values can be overridden to exercise the ABI's
    validation."""

    def __init__(self, w, lane_off=None, *, V=None, H=None, ldw=None, type=None, w_ptrs=None):
        self.w = w
        self.from_tensors = w_ptrs is None
        self._index = None
        one = _as_list(w)[0]
        if lane_off is None:
            lane_off = [0]
            for t in _as_list(w):
                lane_off.append(lane_off[-1] + t.shape[0])
        off = [int(o) for o in lane_off]
        self.lane_off = off
        k = len(off) - 1
        self._off = (ctypes.c_int32 * max(1, k + 1))(*off)
        stride = _row_stride(one)
        if w_ptrs is not None:
            ptrs = list(w_ptrs)
        elif isinstance(w, (list, tuple)):
            if len(w) != k:
                raise ValueError(f"w must hold one tensor per lane, {k}")
            ptrs = [t.data_ptr() for t in w]
            stride = max([t.stride(0) for t in w if t.shape[0] > 1] or [stride])
        else:
            ptrs = [w.data_ptr() + w.element_size() * stride * o for o in off[:-1]]
        self._w = (ctypes.c_void_p * max(1, len(ptrs)))(*ptrs)
        self.desc = sb_table_desc(
            V=off[-1] if V is None else V, H=one.shape[1] if H is None else H, k=k, lane_off=self._off,
            w=self._w, ldw=stride if ldw is None else ldw,
            type=_TYPES.get(one.dtype, -1) if type is None else type)

    @property
    def V(self):
        return self.desc.V

    @property
    def H(self):
        return self.desc.H

    def ref(self):
        return ctypes.byref(self.desc)

    def index(self):
        """The number of the table's one device (None for raw pointers).  The
        descriptor holds its addresses, so it is checked once."""
        if self._index is None and self.from_tensors:
            d, off, w = self.desc, self.lane_off, _as_list(self.w)
            if isinstance(self.w, (list, tuple)):
                for i, t in enumerate(w):
                    if i == 0:
                        _rows(t, "w[0]", off[1] - off[0], d.H)
                    else:
                        _rows(t, f"w[{i}]", off[i + 1] - off[i], d.H, w[0].get_device(), w[0].dtype)
                if len({t.stride(0) for t in w if t.shape[0] > 1}) > 1:
                    raise ValueError("the tensors of w must have one row stride")
            else:
                _rows(self.w, "w", d.V, d.H)
            self._index = w[0].get_device()
        return self._index


def sb_embed(table, ids, out, scale=1.0, stream=None):
    """out (fp32 or bf16 [B, H]) <- scale times the table's rows that ids (int32
    [B]) name; zeros for a negative ID, NaN for one past the table.  Returns out."""
    index = table.index()
    B, pids = _counted(ids, "ids", torch.int32, index)
    code, p, ld = _rows(out, "out", B, table.desc.H, index)
    _call("sb_embed", out.get_device(), stream, lib().sb_embed, table.ref(), pids, B, scale, p, code, ld)
    return out


def sb_embed_grad_workspace_bytes(table, B, accumulate=False):
    st = ctypes.c_int(0)
    n = lib().sb_embed_grad_workspace_bytes(table.ref(), B, int(bool(accumulate)), ctypes.byref(st))
    if st.value != SB_OK:
        raise SbError(st.value, "sb_embed_grad_workspace_bytes")
    return int(n)


def embed_grad_workspace(table, B, accumulate=False, device=None):
    """A workspace for sb_embed_grad on B rows (its contents on entry do not matter)."""
    return torch.empty(max(sb_embed_grad_workspace_bytes(table, B, accumulate), 16), dtype=torch.uint8,
                       device=_as_list(table.w)[0].device if device is None else device)


def sb_embed_grad(table, ids, dout, scale=1.0, accumulate=False, ws=None, stream=None):
    """The gradient of sum(dout * sb_embed(...)): written to the tensors of `table`
    (a Table of the gradient), all of whose rows are overwritten; with
    accumulate it is added to the rows that ids name.  dout (fp32 or bf16 [B, H])
    is of any type.  Returns the table's tensor or tensors."""
    index = table.index()
    B, pids = _counted(ids, "ids", torch.int32, index)
    code, p, ld = _rows(dout, "dout", B, table.desc.H, index)
    index = dout.get_device()
    add = int(bool(accumulate))
    pws, n, ws = _space(ws, lambda: sb_embed_grad_workspace_bytes(table, B, accumulate), index, stream)
    _call("sb_embed_grad", index, stream, lib().sb_embed_grad, table.ref(), pids, B, scale, p, code, ld, add, pws, n)
    return table.w


# ---------------------------------------------------------------------------
# Verification of drafted tokens.
# ---------------------------------------------------------------------------
class Drafts:
    """Descriptor of N sequences' drafted tokens: tokens (int32, all sequences'
    one after another), offsets (int32 [N + 1], on the device: sequence i has
    tokens[offsets[i]:offsets[i + 1]], at most max_drafts of them), the target's
    logits [len(tokens) + N, V] (fp32 or bf16; a sequence's rows are those of its
    drafts and one behind the last), and optionally the draft model's logits
    [len(tokens), V] of the same type and temperatures (fp32 [N]; 1 where there
    are none)."""

    def __init__(self, target, tokens, offsets, max_drafts, draft=None, temperature=None):
        self.target, self.tokens, self.offsets = target, tokens, offsets
        self.draft, self.temperature = draft, temperature
        self._index = None
        self.desc = sb_drafts_desc(
            N=max(0, offsets.numel() - 1), K=int(max_drafts), V=target.shape[1], drafts=tokens.numel(),
            offsets=offsets.data_ptr(), tokens=tokens.data_ptr(), target=target.data_ptr(),
            ldt=_row_stride(target), draft=None if draft is None else draft.data_ptr(),
            ldd=0 if draft is None else _row_stride(draft), type=_TYPES.get(target.dtype, -1),
            temperature=None if temperature is None else temperature.data_ptr())

    @property
    def N(self):
        return self.desc.N

    @property
    def K(self):
        return self.desc.K

    def ref(self):
        return ctypes.byref(self.desc)

    def index(self):
        """The number of the operands' one device.  The descriptor holds their
        addresses, so they are checked once."""
        if self._index is None:
            d, t = self.desc, self.target
            _rows(t, "target", 0, d.V)
            index = t.get_device()
            drafts, _ = _counted(self.tokens, "tokens", torch.int32, index)
            if _counted(self.offsets, "offsets", torch.int32, index)[0] < 1:
                raise ValueError("offsets must hold one number more than there are sequences")
            _rows(t, "target", drafts + d.N, d.V)
            if self.draft is not None:
                _rows(self.draft, "draft", drafts, d.V, index, t.dtype)
            _buffer(self.temperature, "temperature", torch.float32, d.N, index)
            self._index = index
        return self._index


def sb_verify_workspace_bytes(drafts):
    st = ctypes.c_int(0)
    n = lib().sb_verify_workspace_bytes(drafts.ref(), ctypes.byref(st))
    if st.value != SB_OK:
        raise SbError(st.value, "sb_verify_workspace_bytes")
    return int(n)


def verify_workspace(drafts, device=None):
    """A workspace for sb_verify_drafts (its contents on entry do not matter)."""
    return torch.empty(max(sb_verify_workspace_bytes(drafts), 16), dtype=torch.uint8,
                       device=drafts.target.device if device is None else device)


def sb_verify_drafts(drafts, u, u_next, out, accepted, ws=None, stream=None):
    """out (int32 [N, max_drafts + 1]) <- every sequence's accepted drafts, the
    token behind them, and -1 up to the end; accepted (int32 [N]) <- how many
    are accepted.  u (fp32, one per drafted token) and u_next (fp32 [N]) are
    random numbers from [0, 1).  Returns (out, accepted)."""
    index = drafts.index()
    d = drafts.desc
    N, K = d.N, d.K
    u = _buffer(u, "u", torch.float32, d.drafts, index)
    u_next = _buffer(u_next, "u_next", torch.float32, N, index)
    _, p, ldo = _rows(out, "out", N, K + 1, index, torch.int32)
    acc = _buffer(accepted, "accepted", torch.int32, N, index)
    pws, n, ws = _space(ws, lambda: sb_verify_workspace_bytes(drafts), index, stream)
    _call("sb_verify_drafts", index, stream, lib().sb_verify_drafts, drafts.ref(), u, u_next, p, ldo, acc, pws, n)
    return out, accepted


def to_device_bf16(bits, device="cuda"):
    """uint16 numpy bf16 bit patterns -> torch.bfloat16 tensor on device."""
    import numpy as np
    t = torch.from_numpy(np.ascontiguousarray(bits).view(np.int16))
    return t.to(device).view(torch.bfloat16)
