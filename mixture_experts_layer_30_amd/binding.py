"""ctypes binding of libmoe_layer.so: one Python function per C entry point,
same names, argument marshalling only (device pointers from torch tensors,
the current HIP stream).  Every step of the layer runs in the library's HIP
kernels; if the library is missing this module raises instead of computing
anything another way.
"""
import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_layer.so")

MOE_OK, MOE_EINVAL, MOE_EUNSUPPORTED, MOE_ECAPACITY, MOE_EHIP = range(5)
MOE_F32, MOE_BF16 = 0, 1
SCHED_AUTO, SCHED_STREAM, SCHED_TILE, SCHED_RING, SCHED_SPAN = 0, 1, 2, 3, 4
PAD_BLOCK, PAD_MAX = 0, 1
NORM_NONE, NORM_RMS, NORM_LAYER = 0, 1, 2

# every function the C header declares
EXPORTS = ["moe_last_error", "moe_status_string", "moe_align_capacity", "moe_align_capacity_ex",
           "moe_ffn_workspace_bytes", "moe_ffn_workspace_bytes_ex", "dense_ffn_workspace_bytes",
           "moe_route", "moe_route_var", "moe_align", "moe_align_ex", "moe_route_align", "moe_grouped_ffn", "moe_grouped_gate_up", "moe_grouped_down",
           "moe_combine", "dense_ffn_fa", "moe_grouped_gate_up_fp8", "moe_grouped_down_fp8",
           "dense_ffn_fp8", "moe_grouped_ffn_noalloc", "moe_permute", "moe_permute_backward",
           "moe_unpermute", "moe_unpermute_backward", "moe_route_backward",
           "moe_norm_workspace_bytes", "moe_norm", "moe_norm_backward", "moe_norm_residual",
           "moe_norm_residual_backward", "moe_combine_norm_residual"]

# workspace bytes held per GPU by moe_grouped_ffn_noalloc (MOE_NOALLOC_SCRATCH_BYTES)
NOALLOC_SCRATCH_BYTES = 128 << 20


class MoEError(RuntimeError):
    def __init__(self, status, msg):
        super().__init__(f"{msg} (status {status})")
        self.status = status


class moe_plan(ctypes.Structure):
    _fields_ = [("expert_counts", ctypes.c_void_p), ("expert_offsets", ctypes.c_void_p),
                ("sorted_ids", ctypes.c_void_p), ("block_expert", ctypes.c_void_p),
                ("inv_pos", ctypes.c_void_p), ("block_m", ctypes.c_int32), ("cap", ctypes.c_int64)]


class moe_norm_params(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("eps", ctypes.c_float), ("weight", ctypes.c_void_p),
                ("bias", ctypes.c_void_p)]


class moe_gate_params(ctypes.Structure):
    _fields_ = [("alpha", ctypes.c_float), ("channel", ctypes.c_void_p), ("token", ctypes.c_void_p)]


_lib = None


def lib():
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is not built; run `python -m mixture_experts_layer_30_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
        P = ctypes.POINTER(moe_plan)
        L.moe_last_error.restype = ctypes.c_char_p
        L.moe_last_error.argtypes = []
        L.moe_status_string.restype = ctypes.c_char_p
        L.moe_status_string.argtypes = [i32]
        L.moe_align_capacity.restype = i64
        L.moe_align_capacity.argtypes = [i64, i32, i32, i32]
        L.moe_align_capacity_ex.restype = i64
        L.moe_align_capacity_ex.argtypes = [i64, i32, i32, i32, i32]
        L.moe_ffn_workspace_bytes.restype = i64
        L.moe_ffn_workspace_bytes.argtypes = [i64, i32]
        L.moe_ffn_workspace_bytes_ex.restype = i64
        L.moe_ffn_workspace_bytes_ex.argtypes = [i64, i64, i32, i32, i32, i32]
        L.dense_ffn_workspace_bytes.restype = i64
        L.dense_ffn_workspace_bytes.argtypes = [i64, i32, i32]
        L.moe_route.restype = i32
        L.moe_route.argtypes = [vp, i64, i32, i32, vp, vp, vp]
        L.moe_route_var.restype = i32
        L.moe_route_var.argtypes = [vp, i64, i32, i32, vp, vp, vp, vp]
        L.moe_align.restype = i32
        L.moe_align.argtypes = [vp, i64, i32, i32, P, vp]
        L.moe_align_ex.restype = i32
        L.moe_align_ex.argtypes = [vp, i64, i32, i32, P, i32, vp]
        L.moe_route_align.restype = i32
        L.moe_route_align.argtypes = [vp, i64, i32, i32, vp, vp, vp, P, i32, vp]
        L.moe_grouped_ffn.restype = i32
        L.moe_grouped_ffn.argtypes = [vp, i32, i64, i32, i32, i32, i32, vp, vp, P, vp, i64, vp, vp]
        L.moe_grouped_ffn_noalloc.restype = i32
        L.moe_grouped_ffn_noalloc.argtypes = [vp, i32, i64, i32, i32, i32, i32, vp, vp, P, vp, vp]
        L.moe_grouped_gate_up.restype = i32
        L.moe_grouped_gate_up.argtypes = [vp, i32, i64, i32, i32, i32, i32, vp, P, vp, i64, i32, vp]
        L.moe_grouped_down.restype = i32
        L.moe_grouped_down.argtypes = [vp, i32, i64, i32, i32, i32, i32, P, vp, i64, vp, i32, vp]
        L.moe_combine.restype = i32
        L.moe_combine.argtypes = [vp, i32, vp, vp, i32, i64, i32, i32, vp, i32, vp]
        L.dense_ffn_fa.restype = i32
        L.dense_ffn_fa.argtypes = [vp, i32, i64, i32, i32, vp, vp, vp, i64, vp, i32, i32, vp]
        L.moe_grouped_gate_up_fp8.restype = i32
        L.moe_grouped_gate_up_fp8.argtypes = [vp, i64, i32, i32, i32, i32, vp, vp, P, vp, i64, vp]
        L.moe_grouped_down_fp8.restype = i32
        L.moe_grouped_down_fp8.argtypes = [vp, vp, i64, i32, i32, i32, i32, P, vp, i64, vp, vp]
        L.dense_ffn_fp8.restype = i32
        L.dense_ffn_fp8.argtypes = [vp, i64, i32, i32, vp, vp, vp, vp, vp, i64, vp, i32, vp]
        N, G = ctypes.POINTER(moe_norm_params), ctypes.POINTER(moe_gate_params)
        for name, args in (
                ("moe_permute", [vp, i32, i64, i32, i32, i32, P, vp, vp]),
                ("moe_permute_backward", [vp, i32, i64, i32, i32, i32, P, vp, vp]),
                ("moe_unpermute", [vp, i32, vp, vp, i32, i64, i32, i32, i32, P, vp, i32, vp]),
                ("moe_unpermute_backward", [vp, vp, i32, vp, i64, i32, i32, i32, P, vp, vp, vp]),
                ("moe_route_backward", [vp, vp, vp, i64, i32, i32, vp, vp]),
                ("moe_norm", [vp, i32, i64, i32, N, i32, vp, i32, vp]),
                ("moe_norm_backward", [vp, i32, vp, i32, vp, i64, i32, N, i32, vp, vp, vp, vp, i64,
                                       vp]),
                ("moe_norm_residual", [vp, i32, vp, i32, i64, i32, N, G, i32, vp, N, vp, vp]),
                ("moe_combine_norm_residual", [vp, i32, vp, vp, i32, vp, i32, i64, i32, i32, N, G,
                                               i32, vp, N, vp, vp]),
                ("moe_norm_residual_backward", [vp, i32, vp, i32, i64, i32, N, G, i32, vp, vp, vp,
                                                vp, vp, vp, i64, vp])):
            getattr(L, name).restype = i32
            getattr(L, name).argtypes = args
        L.moe_norm_workspace_bytes.restype = i64
        L.moe_norm_workspace_bytes.argtypes = [i64, i32]
        _lib = L
    return _lib


def _check(status):
    if status != MOE_OK:
        raise MoEError(status, lib().moe_last_error().decode())


def _dt(t):
    if t.dtype is torch.bfloat16:
        return MOE_BF16
    if t.dtype is torch.float32:
        return MOE_F32
    raise MoEError(MOE_EUNSUPPORTED, f"dtype {t.dtype}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        # the current stream's handle alone: building torch's Stream object around it
        # takes 2.5 us (measured on MI355X: one token's norm 9.2 -> 7.2 us a call)
        return ctypes.c_void_p(torch._C._cuda_getCurrentRawStream(torch.cuda.current_device()))
    return ctypes.c_void_p(stream.cuda_stream)


def moe_align_capacity(T, K, E, block_m):
    return lib().moe_align_capacity(T, K, E, block_m)


def moe_align_capacity_ex(T, K, E, block_m, pad):
    return lib().moe_align_capacity_ex(T, K, E, block_m, pad)


def moe_ffn_workspace_bytes(cap, I):
    return lib().moe_ffn_workspace_bytes(cap, I)


def moe_ffn_workspace_bytes_ex(cap, T, K, E, H, I):
    return lib().moe_ffn_workspace_bytes_ex(cap, T, K, E, H, I)


def dense_ffn_workspace_bytes(T, H, I):
    return lib().dense_ffn_workspace_bytes(T, H, I)


class Plan:
    """Device arrays of one alignment (see moe_plan in include/moe_layer.h)."""

    def __init__(self, T, K, E, block_m, device, cap=None, pad=PAD_BLOCK):
        self.T, self.K, self.E, self.block_m, self.pad = T, K, E, block_m, pad
        self.cap = moe_align_capacity_ex(T, K, E, block_m, pad) if cap is None else cap
        i32 = torch.int32
        self.expert_counts = torch.empty(E, dtype=i32, device=device)
        self.expert_offsets = torch.empty(E + 1, dtype=i32, device=device)
        self.sorted_ids = torch.empty(max(self.cap, 1), dtype=i32, device=device)
        self.block_expert = torch.empty(max(self.cap // block_m, 1), dtype=i32, device=device)
        self.inv_pos = torch.empty(max(T * K, 1), dtype=i32, device=device)
        self.c = moe_plan(self.expert_counts.data_ptr(), self.expert_offsets.data_ptr(),
                          self.sorted_ids.data_ptr(), self.block_expert.data_ptr(),
                          self.inv_pos.data_ptr(), block_m, self.cap)

    def arrays(self):
        return dict(expert_counts=self.expert_counts, expert_offsets=self.expert_offsets,
                    sorted_ids=self.sorted_ids[:self.cap], block_expert=self.block_expert[:self.cap // self.block_m],
                    inv_pos=self.inv_pos[:self.T * self.K])


def moe_route(logits, K, topk_ids, topk_w, stream=None):
    T, E = logits.shape
    _check(lib().moe_route(_ptr(logits), T, E, K, _ptr(topk_ids), _ptr(topk_w), _stream(stream)))


def moe_route_var(logits, Kmax, k_tok, topk_ids, topk_w, stream=None):
    """Routing with a per-token budget k_tok [T] int32 (device)."""
    T, E = logits.shape
    _check(lib().moe_route_var(_ptr(logits), T, E, Kmax, _ptr(k_tok), _ptr(topk_ids), _ptr(topk_w),
                               _stream(stream)))


def moe_align(topk_ids, E, plan, stream=None):
    T, K = topk_ids.shape
    _check(lib().moe_align(_ptr(topk_ids), T, K, E, ctypes.byref(plan.c), _stream(stream)))


def moe_align_ex(topk_ids, E, plan, pad, stream=None):
    T, K = topk_ids.shape
    _check(lib().moe_align_ex(_ptr(topk_ids), T, K, E, ctypes.byref(plan.c), pad, _stream(stream)))


def moe_route_align(logits, K, topk_ids, topk_w, plan, pad=None, k_tok=None, stream=None):
    """moe_route (or moe_route_var with budgets k_tok) then moe_align_ex, in one
    launch for small batches."""
    T, E = logits.shape
    _check(lib().moe_route_align(_ptr(logits), T, E, K, _ptr(k_tok) if k_tok is not None else None,
                                 _ptr(topk_ids), _ptr(topk_w), ctypes.byref(plan.c),
                                 PAD_BLOCK if pad is None else pad, _stream(stream)))


def moe_grouped_ffn(x, w13, w2, K, plan, workspace, y_pairs, stream=None):
    T, H = x.shape
    E, I2, _ = w13.shape
    _check(lib().moe_grouped_ffn(_ptr(x), _dt(x), T, H, I2 // 2, E, K, _ptr(w13), _ptr(w2),
                                 ctypes.byref(plan.c), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                 _ptr(y_pairs), _stream(stream)))


def moe_grouped_ffn_noalloc(x, w13, w2, K, plan, y_pairs, stream=None):
    """moe_grouped_ffn with the library's own per-GPU workspace (no workspace argument)."""
    T, H = x.shape
    E, I2, _ = w13.shape
    _check(lib().moe_grouped_ffn_noalloc(_ptr(x), _dt(x), T, H, I2 // 2, E, K, _ptr(w13), _ptr(w2),
                                         ctypes.byref(plan.c), _ptr(y_pairs), _stream(stream)))


def moe_grouped_gate_up(x, w13, K, plan, workspace, sched=SCHED_AUTO, stream=None):
    T, H = x.shape
    E, I2, _ = w13.shape
    _check(lib().moe_grouped_gate_up(_ptr(x), _dt(x), T, H, I2 // 2, E, K, _ptr(w13),
                                     ctypes.byref(plan.c), _ptr(workspace),
                                     workspace.numel() * workspace.element_size(), sched, _stream(stream)))


def moe_grouped_down(w2, T, K, plan, workspace, y_pairs, sched=SCHED_AUTO, stream=None):
    E, H, I = w2.shape
    _check(lib().moe_grouped_down(_ptr(w2), _dt(w2), T, H, I, E, K, ctypes.byref(plan.c),
                                  _ptr(workspace), workspace.numel() * workspace.element_size(),
                                  _ptr(y_pairs), sched, _stream(stream)))


def moe_combine(y_pairs, topk_w, out, shared=None, stream=None):
    T, K = topk_w.shape
    H = out.shape[1]
    sdt = _dt(shared) if shared is not None else MOE_F32
    _check(lib().moe_combine(_ptr(y_pairs), _dt(y_pairs), _ptr(topk_w), _ptr(shared), sdt, T, K, H,
                             _ptr(out), _dt(out), _stream(stream)))


def dense_ffn_fa(x, w13, w2, workspace, out, sched=SCHED_AUTO, stream=None):
    T, H = x.shape
    I = w2.shape[1]
    _check(lib().dense_ffn_fa(_ptr(x), _dt(x), T, H, I, _ptr(w13), _ptr(w2), _ptr(workspace),
                              workspace.numel() * workspace.element_size(), _ptr(out), _dt(out),
                              sched, _stream(stream)))


def _need(t, dtype, what):
    """The FP8 entry points take no dtype argument for these tensors: check here."""
    if t.dtype != dtype:
        raise MoEError(MOE_EUNSUPPORTED, f"{what} must be {dtype}, got {t.dtype}")


def _fp8_weights(q, s, what):
    _need(q, torch.uint8, what + " codes")
    _need(s, torch.float32, what + " row scales")


def moe_grouped_gate_up_fp8(x, q13, s13, K, plan, workspace, stream=None):
    """FP8 E4M3 expert weights: q13 uint8 [E,2I,H] codes, s13 fp32 [E,2I] row scales; x bf16."""
    _need(x, torch.bfloat16, "x")
    _fp8_weights(q13, s13, "w13")
    T, H = x.shape
    E, I2, _ = q13.shape
    _check(lib().moe_grouped_gate_up_fp8(_ptr(x), T, H, I2 // 2, E, K, _ptr(q13), _ptr(s13),
                                         ctypes.byref(plan.c), _ptr(workspace),
                                         workspace.numel() * workspace.element_size(), _stream(stream)))


def moe_grouped_down_fp8(q2, s2, T, K, plan, workspace, y_pairs, stream=None):
    """q2 uint8 [E,H,I] codes, s2 fp32 [E,H] row scales; y_pairs bf16."""
    _need(y_pairs, torch.bfloat16, "y_pairs")
    _fp8_weights(q2, s2, "w2")
    E, H, I = q2.shape
    _check(lib().moe_grouped_down_fp8(_ptr(q2), _ptr(s2), T, H, I, E, K, ctypes.byref(plan.c),
                                      _ptr(workspace), workspace.numel() * workspace.element_size(),
                                      _ptr(y_pairs), _stream(stream)))


def dense_ffn_fp8(x, q13, s13, q2, s2, workspace, out, stream=None):
    """x bf16 [T,H]; q13/s13, q2/s2 FP8 codes and row scales; out bf16 or fp32."""
    _need(x, torch.bfloat16, "x")
    _fp8_weights(q13, s13, "w13")
    _fp8_weights(q2, s2, "w2")
    T, H = x.shape
    I = q2.shape[1]
    _check(lib().dense_ffn_fp8(_ptr(x), T, H, I, _ptr(q13), _ptr(s13), _ptr(q2), _ptr(s2),
                               _ptr(workspace), workspace.numel() * workspace.element_size(),
                               _ptr(out), _dt(out), _stream(stream)))



# ---------------------------------------------- around the experts: rows, norms, gates
#
# These calls are outside torch's autograd: a tensor that requires grad gets none from
# them, and buffers are written without autograd's knowledge.  The gradients are the
# *_backward calls, in the caller's order; the grouped FFN has none.


def _refuse(what):
    raise MoEError(MOE_EINVAL, what)


def _shaped(t, shape, what, dtype=None):
    """t is a tensor of this shape (and type), its elements in row-major order."""
    if t.shape == shape and (dtype is None or t.dtype is dtype) and t.is_contiguous():
        return
    if t.shape != shape:
        _refuse(f"{what} must have shape {list(shape)}, got {list(t.shape)}")
    if dtype is not None and t.dtype is not dtype:
        raise MoEError(MOE_EUNSUPPORTED, f"{what} must be {dtype}, got {t.dtype}")
    _refuse(f"{what} must be contiguous")


def _addr(t):
    return None if t is None else t.data_ptr()


def _call(fn, device, stream, *args):
    """fn(*args, stream) with GPU `device` (an index) current: on `stream`, or that GPU's
    current one."""
    if device < 0:
        _refuse("tensors must be on a GPU")
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(device)   # (see _stream)
    elif stream.device.index != device:
        _refuse(f"a stream of {stream.device} for tensors on GPU {device}")
    else:
        stream = stream.cuda_stream
    if device == torch.cuda.current_device():
        status = fn(*args, stream)
    else:
        with torch.cuda.device(device):
            status = fn(*args, stream)
    if status != MOE_OK:
        _check(status)


def _one_device(first, *rest):
    """The index of the GPU that holds every tensor given; -1: none does."""
    dev = first.get_device()
    for t in rest:
        if t is not None and t.get_device() != dev:
            _refuse(f"tensors on {first.device} and {t.device}")
    return dev


def _ref(o):
    """The C struct of a Norm or Gate by reference, as the object is now; None: NULL."""
    return None if o is None else o.ref()


class _Params:
    """Holds the C struct that a call reads; a copy has one of its own."""
    _type = None

    def __init__(self):
        self._c = self._type()
        self._ref = ctypes.byref(self._c)

    def __getstate__(self):
        return {k: v for k, v in self.__dict__.items() if k not in ("_c", "_ref")}

    def __setstate__(self, state):
        self.__dict__.update(state)
        _Params.__init__(self)


class Norm(_Params):
    """A norm's kind, eps and parameters (see moe_norm_params in include/moe_layer.h).
    weight, bias [H] fp32 or bf16, or None: ones, zeros.  Holds the tensors it points to."""
    _type = moe_norm_params

    def __init__(self, kind=NORM_RMS, eps=1e-6, weight=None, bias=None):
        self.kind, self.eps, self.weight, self.bias = kind, eps, weight, bias
        super().__init__()

    def ref(self):
        c, w, b = self._c, self.weight, self.bias
        c.kind = self.kind
        c.eps = self.eps
        c.weight = None if w is None else w.data_ptr()
        c.bias = None if b is None else b.data_ptr()
        return self._ref


class Gate(_Params):
    """alpha * channel[h] * token[t] (see moe_gate_params): channel [H] of the parameters'
    type, token [T] fp32, either None.  Holds the tensors it points to."""
    _type = moe_gate_params

    def __init__(self, alpha=1.0, channel=None, token=None):
        self.alpha, self.channel, self.token = alpha, channel, token
        super().__init__()

    def ref(self):
        c, ch, tok = self._c, self.channel, self.token
        c.alpha = self.alpha
        c.channel = None if ch is None else ch.data_ptr()
        c.token = None if tok is None else tok.data_ptr()
        return self._ref


def _param(t, shape, dt, device, what):
    """Checks a parameter against those before it, of type dt (None: any); returns its type."""
    dtype = t.dtype
    if t.shape != shape or not t.is_contiguous():
        _shaped(t, shape, what)
    if dt is not None and dtype is not dt:
        raise MoEError(MOE_EUNSUPPORTED, f"parameters of {dt} and {dtype} in one call")
    if t.get_device() != device:
        _refuse(f"{what} on {t.device}, the tokens on another")
    return dtype


def _params(T, H, device, norm, gate=None, next_norm=None):
    """Checks the parameters of a call; returns their type."""
    dt, shape = None, (H,)
    for n in (norm, next_norm):
        if n is not None:
            if n.weight is not None:
                dt = _param(n.weight, shape, dt, device, "weight")
            if n.bias is not None:
                dt = _param(n.bias, shape, dt, device, "bias")
    if gate is not None:
        if gate.channel is not None:
            dt = _param(gate.channel, shape, dt, device, "channel")
        if gate.token is not None:
            _shaped(gate.token, (T,), "token", torch.float32)
            if gate.token.get_device() != device:
                _refuse(f"token on {gate.token.device}, the tokens on another")
    if dt is None or dt is torch.float32:
        return MOE_F32
    if dt is torch.bfloat16:
        return MOE_BF16
    raise MoEError(MOE_EUNSUPPORTED, f"parameter dtype {dt}")


def _rows(t, plan, H, what, dtype=None):
    """t holds the plan's rows: [cap][H] or more."""
    if t.dim() != 2 or t.shape[0] < plan.cap or t.shape[1] != H:
        _refuse(f"{what} must have shape [{plan.cap}, {H}] or more rows, got {list(t.shape)}")
    if dtype is not None and t.dtype != dtype:
        raise MoEError(MOE_EUNSUPPORTED, f"{what} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        _refuse(f"{what} must be contiguous")


def _tokens(t, what):
    if t.dim() != 2 or not t.is_contiguous():
        _refuse(f"{what} must be a contiguous [T, H] tensor, got {list(t.shape)}")
    return t.shape


def _planned(t, plan, what):
    """(T, H) of the tokens t, as many as the plan's"""
    T, H = _tokens(t, what)
    if T != plan.T:
        _refuse(f"{what} has {T} tokens, the plan {plan.T}")
    return T, H


def moe_permute(x, plan, rows, stream=None):
    """rows[r] = the token of alignment row r; zeros in padding rows; rows past the
    padded total are left as they were.  x [T,H], rows [plan.cap,H] of x's type."""
    T, H = _planned(x, plan, "x")
    _rows(rows, plan, H, "rows", x.dtype)
    dev = _one_device(x, rows, plan.inv_pos)
    _call(lib().moe_permute, dev, stream, _addr(x), _dt(x), T, H, plan.E, plan.K,
          ctypes.byref(plan.c), _addr(rows))


def moe_permute_backward(drows, plan, dx, stream=None):
    """dx[t] = the sum of the rows of token t, in slot order."""
    T, H = _planned(dx, plan, "dx")
    _rows(drows, plan, H, "drows", dx.dtype)
    dev = _one_device(dx, drows, plan.inv_pos)
    _call(lib().moe_permute_backward, dev, stream, _addr(drows), _dt(dx), T, H, plan.E, plan.K,
          ctypes.byref(plan.c), _addr(dx))


def moe_unpermute(rows, topk_w, plan, out, shared=None, stream=None):
    """out[t] = sum_k topk_w[t,k] * (row of pair t,k) (+ shared[t]); topk_w None: weights 1."""
    T, H = _planned(out, plan, "out")
    _rows(rows, plan, H, "rows")
    if topk_w is not None:
        _shaped(topk_w, (T, plan.K), "topk_w", torch.float32)
    if shared is not None:
        _shaped(shared, (T, H), "shared")
    dev = _one_device(out, rows, topk_w, shared, plan.inv_pos)
    _call(lib().moe_unpermute, dev, stream, _addr(rows), _dt(rows), _addr(topk_w), _addr(shared),
          _dt(shared) if shared is not None else MOE_F32, T, H, plan.E, plan.K,
          ctypes.byref(plan.c), _addr(out), _dt(out))


def moe_unpermute_backward(dout, rows, topk_w, plan, drows=None, dw=None, stream=None):
    """Gradients of moe_unpermute: drows (padding rows as by moe_permute; may be rows) and
    dw [T,K] fp32, either None.  rows may be None where dw is."""
    T, H = _planned(dout, plan, "dout")
    for t, what in ((rows, "rows"), (drows, "drows")):
        if t is not None:
            _rows(t, plan, H, what, dout.dtype)
    for t, what in ((topk_w, "topk_w"), (dw, "dw")):
        if t is not None:
            _shaped(t, (T, plan.K), what, torch.float32)
    dev = _one_device(dout, rows, topk_w, drows, dw, plan.inv_pos)
    _call(lib().moe_unpermute_backward, dev, stream, _addr(dout), _addr(rows), _dt(dout),
          _addr(topk_w), T, H, plan.E, plan.K, ctypes.byref(plan.c), _addr(drows), _addr(dw))


def moe_route_backward(topk_ids, topk_w, dw, dlogits, stream=None):
    """dlogits [T,E] fp32 from the gradient dw [T,K] of the routing weights."""
    if topk_ids.dim() != 2 or dlogits.dim() != 2:
        _refuse("topk_ids must be [T, K] and dlogits [T, E]")
    T, K = topk_ids.shape
    E = dlogits.shape[1]
    _shaped(topk_ids, (T, K), "topk_ids", torch.int32)
    _shaped(topk_w, (T, K), "topk_w", torch.float32)
    _shaped(dw, (T, K), "dw", torch.float32)
    _shaped(dlogits, (T, E), "dlogits", torch.float32)
    dev = _one_device(topk_ids, topk_w, dw, dlogits)
    _call(lib().moe_route_backward, dev, stream, _addr(topk_ids), _addr(topk_w), _addr(dw), T, E, K,
          _addr(dlogits))


def moe_norm_workspace_bytes(T, H):
    return lib().moe_norm_workspace_bytes(T, H)


def _workspace(t):
    if t is None:
        return None, 0
    if not t.is_contiguous():
        _refuse("workspace must be contiguous")
    return _addr(t), t.numel() * t.element_size()


def _optional(H, **named):
    for what, t in named.items():
        if t is not None:
            _shaped(t, (H,), what, torch.float32)


def moe_norm(x, norm, out, stream=None):
    """out = norm(x): x, out [T,H], each fp32 or bf16."""
    T, H = _tokens(x, "x")
    _shaped(out, (T, H), "out")
    dev = _one_device(x, out)
    pdt = _params(T, H, dev, norm)
    _call(lib().moe_norm, dev, stream, _addr(x), _dt(x), T, H, _ref(norm), pdt, _addr(out),
          _dt(out))


def moe_norm_backward(dout, x, norm, dx, workspace=None, dres=None, dweight=None, dbias=None,
                      stream=None):
    """Gradients of moe_norm: dx (+ dres, both of x's type), dweight and dbias [H] fp32, where
    given (they need a workspace of moe_norm_workspace_bytes(T, H))."""
    T, H = _tokens(x, "x")
    _shaped(dout, (T, H), "dout")
    _shaped(dx, (T, H), "dx", x.dtype)
    if dres is not None:
        _shaped(dres, (T, H), "dres", x.dtype)
    _optional(H, dweight=dweight, dbias=dbias)
    dev = _one_device(x, dout, dx, dres, dweight, dbias, workspace)
    pdt = _params(T, H, dev, norm)
    ws, n = _workspace(workspace)
    _call(lib().moe_norm_backward, dev, stream, _addr(dout), _dt(dout), _addr(x), _dt(x), _addr(dres),
          T, H, _ref(norm), pdt, _addr(dx), _addr(dweight), _addr(dbias), ws, n)


def _next_norm(pre, n, T, H, dtype):
    if n is not None:
        _shaped(n, (T, H), "n", dtype)
    return _ref(pre)


def moe_norm_residual(y, x, post, gate, r, pre=None, n=None, stream=None):
    """r = x + gate * post(y) and, with pre, n = pre(r): x, r of one type, y, n of one type."""
    T, H = _tokens(x, "x")
    _shaped(y, (T, H), "y")
    _shaped(r, (T, H), "r", x.dtype)
    nx = _next_norm(pre, n, T, H, y.dtype)
    dev = _one_device(x, y, r, n)
    pdt = _params(T, H, dev, post, gate, pre)
    _call(lib().moe_norm_residual, dev, stream, _addr(y), _dt(y), _addr(x), _dt(x), T, H,
          _ref(post), _ref(gate), pdt, _addr(r), nx, _addr(n))


def moe_combine_norm_residual(y_pairs, topk_w, x, post, gate, r, pre=None, n=None, shared=None,
                              stream=None):
    """moe_norm_residual of y[t] = sum_k topk_w[t,k] y_pairs[t*K + k] (+ shared[t])."""
    T, H = _tokens(x, "x")
    if topk_w.dim() != 2:
        _refuse("topk_w must be [T, K]")
    K = topk_w.shape[1]
    _shaped(topk_w, (T, K), "topk_w", torch.float32)
    if y_pairs.dim() != 2 or y_pairs.shape[0] < T * K or y_pairs.shape[1] != H or \
            not y_pairs.is_contiguous():
        _refuse(f"y_pairs must be a contiguous [{T * K}, {H}] tensor, got {list(y_pairs.shape)}")
    _shaped(r, (T, H), "r", x.dtype)
    if shared is not None:
        _shaped(shared, (T, H), "shared")
    nx = _next_norm(pre, n, T, H, y_pairs.dtype)
    dev = _one_device(x, y_pairs, topk_w, shared, r, n)
    pdt = _params(T, H, dev, post, gate, pre)
    _call(lib().moe_combine_norm_residual, dev, stream, _addr(y_pairs), _dt(y_pairs), _addr(topk_w),
          _addr(shared), _dt(shared) if shared is not None else MOE_F32, _addr(x), _dt(x), T, K, H,
          _ref(post), _ref(gate), pdt, _addr(r), nx, _addr(n))


def moe_norm_residual_backward(dr, y, post, gate, dy, workspace=None, dweight=None, dbias=None,
                               dchannel=None, dtoken=None, stream=None):
    """Gradients of moe_norm_residual's y, of post's parameters and of the gates, where given;
    that of x is dr itself."""
    T, H = _tokens(y, "y")
    _shaped(dr, (T, H), "dr")
    _shaped(dy, (T, H), "dy", y.dtype)
    _optional(H, dweight=dweight, dbias=dbias, dchannel=dchannel)
    if dtoken is not None:
        _shaped(dtoken, (T,), "dtoken", torch.float32)
    dev = _one_device(y, dr, dy, dweight, dbias, dchannel, dtoken, workspace)
    pdt = _params(T, H, dev, post, gate)
    ws, n = _workspace(workspace)
    _call(lib().moe_norm_residual_backward, dev, stream, _addr(dr), _dt(dr), _addr(y), _dt(y), T, H,
          _ref(post), _ref(gate), pdt, _addr(dy), _addr(dweight), _addr(dbias),
          _addr(dchannel), _addr(dtoken), ws, n)
