"""MoE token dispatch / combine on MI355X: thin Python binding over libmoe_ep.so.

Every step of the path runs in the HIP kernels of ``csrc/``; this
module only allocates outputs with torch (device memory + the current stream)
and marshals pointers to the C ABI of ``include/moe_ep.h``. There is no CPU
fallback: importing works without the library, but any call raises when
``libmoe_ep.so`` has not been built (``python -m combine_ep_recv_amd._build``
or ``__graft_entry__.build()``).

    expand_x, dynamic_scales, assist_info, ep_recv_count = dispatch(
        x, expert_ids, ep_world, experts_per_rank, quant_mode=0)
    x_out = combine(expand_x, assist_info, ep_recv_count, expert_ids,
                    expert_scales, ep_world, experts_per_rank)

Around them: ``gate`` makes expert_ids and expert_scales from a router's logits
(``gate_backward`` its gradient), and ``quantize_mx`` / ``expert_product`` run
the experts on microscaled rows and 4-bit weights, ``quantize_int8`` /
``expert_product`` on int8 rows and weights:

    expert_ids, expert_scales = gate(logits, topk)
    rows, row_scales, assist_info, ep_recv_count = dispatch(..., quant_mode=MOE_QUANT_MX)
    y = expert_product(rows, row_scales, weights, weight_scales, ep_recv_count)

``combine_backward`` and ``dispatch_backward`` are the gradients of the two calls:

    grad_rows, grad_scales = combine_backward(grad_out, expand_x, ...)
    grad_x = dispatch_backward(grad_expand_x, ...)
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmoe_ep.so")

MOE_OK = 0
(MOE_ERR_NULLPTR, MOE_ERR_SHAPE, MOE_ERR_DTYPE, MOE_ERR_QUANT, MOE_ERR_WORKSPACE, MOE_ERR_LAUNCH, MOE_ERR_SCHEDULE,
 MOE_ERR_ALIGN, MOE_ERR_MASK) = range(1, 10)
MOE_INT32, MOE_FP16, MOE_BF16, MOE_FP32 = 0, 1, 2, 3
MOE_QUANT_NONE, MOE_QUANT_STATIC, MOE_QUANT_DYN_TOKEN, MOE_QUANT_DYN_GROUP, MOE_QUANT_MX = 0, 1, 2, 3, 4
MOE_SCHED_TOKEN, MOE_SCHED_SEGMENT, MOE_SCHED_ADAPTIVE = 0, 1, 2
MOE_MASK_NONE, MOE_MASK_TOKEN, MOE_MASK_PAIR = 0, 1, 2
MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID = 0, 1
MOE_GROUP_MAX, MOE_GROUP_TOP2 = 0, 1
MOE_MX_E2M1, MOE_MX_E4M3 = 0, 1
MOE_ACT_NONE, MOE_ACT_SWIGLU = 0, 1

EXPORTS = ("moe_dispatch_workspace_size", "moe_dispatch", "moe_dispatch_noalloc", "moe_combine_workspace_size",
           "moe_combine", "moe_combine_backward_workspace_size", "moe_combine_backward", "moe_dispatch_backward",
           "moe_gate", "moe_gate_backward", "moe_mx_quantize", "moe_mx_dequantize",
           "moe_expert_product", "moe_int8_quantize", "moe_int8_dequantize", "moe_expert_product_int8", "moe_status_str")
NOALLOC_SCRATCH_BYTES = 32 << 20      # MOE_NOALLOC_SCRATCH_BYTES


class MoeError(RuntimeError):
    def __init__(self, fn, status, msg):
        super().__init__("%s failed: status %d (%s)" % (fn, status, msg))
        self.status = status


class MoeSpecialExperts(ctypes.Structure):
    _fields_ = [("zero_expert_num", ctypes.c_int32), ("copy_expert_num", ctypes.c_int32),
                ("const_expert_num", ctypes.c_int32), ("reserved", ctypes.c_int32), ("ori_x", ctypes.c_void_p),
                ("const_x", ctypes.c_void_p)]


def _special(zero_experts: int, copy_experts: int, ori_x: Optional[torch.Tensor] = None, const_experts: int = 0,
             const_x: Optional[torch.Tensor] = None):
    """byref(moe_special_experts) or None when there are no special experts."""
    if not zero_experts and not copy_experts and not const_experts:
        return None
    sp = MoeSpecialExperts(zero_expert_num=int(zero_experts), copy_expert_num=int(copy_experts),
                           const_expert_num=int(const_experts),
                           ori_x=None if ori_x is None else ori_x.data_ptr(),
                           const_x=None if const_x is None else const_x.data_ptr())
    return ctypes.byref(sp)


class MoeSchedule(ctypes.Structure):
    """moe_schedule; by default the adaptive mode with the README's 2 MiB threshold (what a NULL schedule
    selects)."""
    _fields_ = [("mode", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("large_segment_bytes", ctypes.c_int64), ("segment_is_large", ctypes.c_void_p)]

    def __init__(self, mode=MOE_SCHED_ADAPTIVE, large_segment_bytes=-1, segment_is_large=None, reserved=0):
        super().__init__(mode, reserved, large_segment_bytes, segment_is_large)


_lib = None


def library() -> ctypes.CDLL:
    """Load libmoe_ep.so (raises if it was not built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError("libmoe_ep.so is not built (%s); build it with __graft_entry__.build()" % LIB_PATH)
    lib = ctypes.CDLL(LIB_PATH)
    P, I, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    lib.moe_dispatch_workspace_size.argtypes = [I, I, I, I, I, I, I, ctypes.POINTER(SZ)]
    lib.moe_dispatch_workspace_size.restype = I
    lib.moe_dispatch.argtypes = [P, P, P, P, I, ctypes.POINTER(MoeSpecialExperts), I, I, I, I, I, I, I, P,
                                 ctypes.c_int64, P, P, P, P, P, ctypes.POINTER(MoeSchedule), P, SZ, P]
    lib.moe_dispatch.restype = I
    lib.moe_dispatch_noalloc.argtypes = [P, P, P, P, I, ctypes.POINTER(MoeSpecialExperts), I, I, I, I, I, I, I, P,
                                         ctypes.c_int64, P, P, P, P, P, ctypes.POINTER(MoeSchedule), P]
    lib.moe_dispatch_noalloc.restype = I
    lib.moe_combine_workspace_size.argtypes = [I, I, I, I, I, I, ctypes.POINTER(SZ)]
    lib.moe_combine_workspace_size.restype = I
    lib.moe_combine.argtypes = [P, P, P, P, P, P, I, ctypes.POINTER(MoeSpecialExperts), I, I, I, I, I, I, P, P,
                                SZ, P]
    lib.moe_combine.restype = I
    lib.moe_combine_backward_workspace_size.argtypes = [I, I, I, I, I, I, I, ctypes.POINTER(SZ)]
    lib.moe_combine_backward_workspace_size.restype = I
    lib.moe_combine_backward.argtypes = [P, P, P, P, P, P, P, I, ctypes.POINTER(MoeSpecialExperts), I, I, I, I, I, I,
                                         P, P, P, P, P, SZ, P]
    lib.moe_combine_backward.restype = I
    lib.moe_dispatch_backward.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, I, P, P, P]
    lib.moe_dispatch_backward.restype = I
    F, L = ctypes.c_float, ctypes.c_int64
    lib.moe_gate.argtypes = [P, P, P, I, I, I, I, I, I, I, I, I, F, P, P, P, P]
    lib.moe_gate.restype = I
    lib.moe_gate_backward.argtypes = [P, P, P, P, I, I, I, I, I, I, F, P, P]
    lib.moe_gate_backward.restype = I
    lib.moe_mx_quantize.argtypes = [P, L, I, I, I, P, P, P]
    lib.moe_mx_quantize.restype = I
    lib.moe_mx_dequantize.argtypes = [P, P, L, I, I, I, P, P]
    lib.moe_mx_dequantize.restype = I
    lib.moe_expert_product.argtypes = [P, P, I, P, P, P, I, I, I, I, I, I, I, P, P]
    lib.moe_expert_product.restype = I
    lib.moe_int8_quantize.argtypes = [P, L, I, I, P, P, P]
    lib.moe_int8_quantize.restype = I
    lib.moe_int8_dequantize.argtypes = [P, P, L, I, I, P, P]
    lib.moe_int8_dequantize.restype = I
    lib.moe_expert_product_int8.argtypes = [P, P, P, P, P, I, I, I, I, I, I, I, P, P]
    lib.moe_expert_product_int8.restype = I
    lib.moe_status_str.argtypes = [I]
    lib.moe_status_str.restype = ctypes.c_char_p
    _lib = lib
    return lib


def status_str(status: int) -> str:
    return library().moe_status_str(int(status)).decode()


def _check(fn, status):
    if status != MOE_OK:
        raise MoeError(fn, status, status_str(status))


def dtype_code(dt: torch.dtype) -> int:
    if dt == torch.int32:
        return MOE_INT32
    if dt == torch.float16:
        return MOE_FP16
    if dt == torch.bfloat16:
        return MOE_BF16
    raise MoeError("dtype", MOE_ERR_DTYPE, "unsupported token dtype %s" % dt)


def _check_tensor(name, t, dtype, shape, device):
    """A contiguous tensor of this dtype and shape (a tuple) on this device, else MoeError before
    any launch. Callers first make sure that the device is a GPU. About 0.3 us per tensor."""
    try:
        ok = t.dtype == dtype and t.shape == shape and t.device == device and t.is_contiguous()
    except AttributeError:
        ok = False
    if not ok:
        raise MoeError(name, MOE_ERR_SHAPE, "%s must be a contiguous %s tensor of shape %s on %s; got %r"
                       % (name, dtype, tuple(shape), device, t if not isinstance(t, torch.Tensor)
                          else "%s %s on %s" % (t.dtype, tuple(t.shape), t.device)))


def _gpu_device(name, t):
    """The device of t, which must be a GPU tensor."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise MoeError(name, MOE_ERR_SHAPE, "%s must be a tensor on a GPU" % name)
    return t.device


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_ptr(device) -> int:
    """torch's current HIP stream on this GPU, as the raw handle: torch's own accessor when this build
    has it (0.07 us per call), else the public one (1.8 us)."""
    if _raw_stream is not None:
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def _mask_args(mask: Optional[torch.Tensor], N: int, K: int, device):
    """(pointer, kind) for a token mask: None, bool/uint8 [N] (per token) or [N, K] (per pair)."""
    if mask is None:
        return None, MOE_MASK_NONE
    if mask.dtype not in (torch.bool, torch.uint8) or not mask.is_contiguous() or mask.device != device:
        raise MoeError("x_active_mask", MOE_ERR_MASK, "mask must be a contiguous bool or uint8 tensor on %s" % device)
    if tuple(mask.shape) == (N,):
        return _ptr(mask), MOE_MASK_TOKEN
    if tuple(mask.shape) == (N, K):
        return _ptr(mask), MOE_MASK_PAIR
    raise MoeError("x_active_mask", MOE_ERR_MASK,
                   "mask shape %s is neither (%d,) nor (%d, %d)" % (tuple(mask.shape), N, N, K))


def dispatch_workspace_size(ep_world, bs, experts_per_rank, h, topk, dtype, quant_mode=0) -> int:
    n = ctypes.c_size_t(0)
    _check("moe_dispatch_workspace_size",
           library().moe_dispatch_workspace_size(ep_world, bs, experts_per_rank, h, topk, dtype, quant_mode,
                                                 ctypes.byref(n)))
    return n.value


def combine_workspace_size(ep_world, bs, experts_per_rank, h, topk, dtype) -> int:
    n = ctypes.c_size_t(0)
    _check("moe_combine_workspace_size",
           library().moe_combine_workspace_size(ep_world, bs, experts_per_rank, h, topk, dtype, ctypes.byref(n)))
    return n.value


def _out_dtype(quant_mode, dtype):
    """expand_x's element type: int8 codes (quantMode 1, 2), E4M3 codes (3, 4), else the token dtype."""
    return {MOE_QUANT_STATIC: torch.int8, MOE_QUANT_DYN_TOKEN: torch.int8, MOE_QUANT_DYN_GROUP: torch.float8_e4m3fn,
            MOE_QUANT_MX: torch.float8_e4m3fn}.get(quant_mode, dtype)


class DispatchBuffers:
    """Preallocated outputs + workspace for repeated dispatch calls of one shape."""

    def __init__(self, ep_world, bs, experts_per_rank, h, topk, dtype: torch.dtype, quant_mode=0,
                 device="cuda", with_expand_scales=False):
        rows = ep_world * bs * topk
        self.shape = (ep_world, bs, experts_per_rank, h, topk)
        self.dtype, self.quant_mode = dtype, quant_mode
        self.expand_x = torch.empty((rows, h), dtype=_out_dtype(quant_mode, dtype), device=device)
        if quant_mode == MOE_QUANT_DYN_TOKEN:
            self.dynamic_scales = torch.empty((rows,), dtype=torch.float32, device=device)
        elif quant_mode == MOE_QUANT_DYN_GROUP:          # one scale per 128-element group
            self.dynamic_scales = torch.empty((rows, (h + 127) // 128), dtype=torch.float32, device=device)
        elif quant_mode == MOE_QUANT_MX:                 # one E8M0 byte per 32-element block
            self.dynamic_scales = torch.empty((rows, (h + 31) // 32), dtype=torch.uint8, device=device)
        else:
            self.dynamic_scales = None
        self.assist_info = torch.empty((rows, 3), dtype=torch.int32, device=device)
        self.ep_recv_count = torch.empty((ep_world, experts_per_rank * ep_world), dtype=torch.int32,
                                         device=device)
        self.expand_scales = (torch.empty((rows,), dtype=torch.float32 if dtype != torch.int32 else torch.int32,
                                          device=device) if with_expand_scales else None)
        ws = dispatch_workspace_size(ep_world, bs, experts_per_rank, h, topk, dtype_code(dtype), quant_mode)
        self.workspace = torch.empty((max(ws, 16),), dtype=torch.uint8, device=device)
        self._checked = None

    def check(self):
        """Check the buffers against the shape (once per set of tensor objects: the attributes are
        public, and a replaced tensor must fit before a kernel writes it). Returns the device."""
        now = (self.expand_x, self.dynamic_scales, self.assist_info, self.ep_recv_count, self.expand_scales,
               self.workspace)
        if self._checked is not None and all(a is b for a, b in zip(now, self._checked)):
            return self.expand_x.device
        W, bs, epr, h, K = self.shape
        rows = W * bs * K
        dev = _gpu_device("expand_x", self.expand_x)
        _check_tensor("expand_x", self.expand_x, _out_dtype(self.quant_mode, self.dtype), (rows, h), dev)
        if self.quant_mode == MOE_QUANT_DYN_TOKEN:
            _check_tensor("dynamic_scales", self.dynamic_scales, torch.float32, (rows,), dev)
        elif self.quant_mode == MOE_QUANT_DYN_GROUP:
            _check_tensor("dynamic_scales", self.dynamic_scales, torch.float32, (rows, (h + 127) // 128), dev)
        elif self.quant_mode == MOE_QUANT_MX:
            _check_tensor("dynamic_scales", self.dynamic_scales, torch.uint8, (rows, (h + 31) // 32), dev)
        _check_tensor("assist_info", self.assist_info, torch.int32, (rows, 3), dev)
        _check_tensor("ep_recv_count", self.ep_recv_count, torch.int32, (W, epr * W), dev)
        if self.expand_scales is not None:
            _check_tensor("expand_scales", self.expand_scales,
                          torch.int32 if self.expand_scales.dtype == torch.int32 else torch.float32, (rows,), dev)
        _check_tensor("workspace", self.workspace, torch.uint8, (self.workspace.numel(),), dev)
        self._checked = now          # held, so the objects compared by identity stay these ones
        return dev


def _quant_scales_args(qs: Optional[torch.Tensor], device):
    """(pointer, count) for quantMode 1's fp32 coefficients: 1, h or E*h values."""
    if qs is None:
        return None, 0
    if qs.dtype != torch.float32 or not qs.is_contiguous() or qs.device != device:
        raise MoeError("quant_scales", MOE_ERR_QUANT,
                       "quant_scales must be a contiguous float32 tensor on %s" % device)
    return _ptr(qs), qs.numel()


def dispatch_into(buf: DispatchBuffers, x: torch.Tensor, expert_ids: torch.Tensor,
                  expert_scales: Optional[torch.Tensor] = None, schedule: Optional[MoeSchedule] = None,
                  x_active_mask: Optional[torch.Tensor] = None, zero_experts: int = 0, copy_experts: int = 0,
                  quant_scales: Optional[torch.Tensor] = None, const_experts: int = 0):
    """moe_dispatch into preallocated buffers on the current stream. quant_scales: the static
    quantiser's coefficients (quantMode 1 only): 1, h or E*h fp32 values. The C ABI sees only
    pointers, so the tensors' shapes, dtypes and device are checked here against buf."""
    W, bs, epr, h, K = buf.shape
    dev = buf.check()
    _check_tensor("x", x, buf.dtype, (W * bs, h), dev)
    _check_tensor("expert_ids", expert_ids, torch.int32, (W * bs, K), dev)
    if expert_scales is not None:
        _check_tensor("expert_scales", expert_scales,
                      torch.int32 if getattr(expert_scales, "dtype", None) == torch.int32 else torch.float32,
                      (W * bs, K), dev)
    mp, mk = _mask_args(x_active_mask, W * bs, K, dev)
    qp, qn = _quant_scales_args(quant_scales, dev)
    rc = library().moe_dispatch(
        _ptr(x), _ptr(expert_ids), _ptr(expert_scales), mp, mk, _special(zero_experts, copy_experts, None,
                                                                         const_experts), W, bs, epr,
        h, K, dtype_code(buf.dtype),
        buf.quant_mode, qp, ctypes.c_int64(qn),
        _ptr(buf.expand_x), _ptr(buf.dynamic_scales), _ptr(buf.assist_info), _ptr(buf.ep_recv_count),
        _ptr(buf.expand_scales), ctypes.byref(schedule) if schedule is not None else None,
        _ptr(buf.workspace), buf.workspace.numel(), _stream_ptr(dev))
    _check("moe_dispatch", rc)
    return buf


def dispatch_noalloc_into(buf: DispatchBuffers, x: torch.Tensor, expert_ids: torch.Tensor,
                          expert_scales: Optional[torch.Tensor] = None, schedule: Optional[MoeSchedule] = None,
                          x_active_mask: Optional[torch.Tensor] = None, zero_experts: int = 0,
                          copy_experts: int = 0, quant_scales: Optional[torch.Tensor] = None,
                          const_experts: int = 0):
    """moe_dispatch_noalloc into preallocated buffers on the current stream: the same outputs as
    dispatch_into, with the library's own per-GPU scratch in place of buf.workspace (which is not
    used). The same checks run first."""
    W, bs, epr, h, K = buf.shape
    dev = buf.check()
    _check_tensor("x", x, buf.dtype, (W * bs, h), dev)
    _check_tensor("expert_ids", expert_ids, torch.int32, (W * bs, K), dev)
    if expert_scales is not None:
        _check_tensor("expert_scales", expert_scales,
                      torch.int32 if getattr(expert_scales, "dtype", None) == torch.int32 else torch.float32,
                      (W * bs, K), dev)
    mp, mk = _mask_args(x_active_mask, W * bs, K, dev)
    qp, qn = _quant_scales_args(quant_scales, dev)
    rc = library().moe_dispatch_noalloc(
        _ptr(x), _ptr(expert_ids), _ptr(expert_scales), mp, mk, _special(zero_experts, copy_experts, None,
                                                                         const_experts), W, bs, epr,
        h, K, dtype_code(buf.dtype), buf.quant_mode, qp, ctypes.c_int64(qn),
        _ptr(buf.expand_x), _ptr(buf.dynamic_scales), _ptr(buf.assist_info), _ptr(buf.ep_recv_count),
        _ptr(buf.expand_scales), ctypes.byref(schedule) if schedule is not None else None, _stream_ptr(dev))
    _check("moe_dispatch_noalloc", rc)
    return buf


def dispatch(x: torch.Tensor, expert_ids: torch.Tensor, ep_world: int, experts_per_rank: int,
             quant_mode: int = MOE_QUANT_NONE, expert_scales: Optional[torch.Tensor] = None,
             schedule: Optional[MoeSchedule] = None, x_active_mask: Optional[torch.Tensor] = None,
             zero_experts: int = 0, copy_experts: int = 0, quant_scales: Optional[torch.Tensor] = None,
             const_experts: int = 0):
    """Dispatch tokens into expert-grouped rows.

    x: [ep_world*bs, h] int32/fp16/bf16 on a GPU; expert_ids: [ep_world*bs, topk]
    int32. Returns (expand_x, dynamic_scales or None, assist_info, ep_recv_count)
    and, when expert_scales is given, a fifth item expand_scales. With a token
    mask (bool/uint8 [N] or [N, topk]) only the first ep_recv_count[:, -1].sum()
    rows of the row-indexed outputs are written; the same holds with special
    experts (ids E.. for zero_experts, then copy_experts, then const_experts), whose
    pairs get no row.
    quant_mode 1 (static int8) takes its coefficients in quant_scales (fp32, 1, h or
    E*h values) and returns no dynamic scales. quant_mode 3 returns float8_e4m3fn
    codes and fp32 scales per 128-element group; quant_mode 4 (MXFP8) returns
    float8_e4m3fn codes and uint8 E8M0 bytes per 32-element block (the scale
    2^(byte - 127)).
    """
    dev = _gpu_device("x", x)
    _gpu_device("expert_ids", expert_ids)
    if x.dim() != 2 or expert_ids.dim() != 2:
        raise MoeError("moe_dispatch", MOE_ERR_SHAPE, "x and expert_ids must be 2-D")
    N, h = x.shape
    K = expert_ids.shape[1]
    if N % ep_world:
        raise MoeError("moe_dispatch", MOE_ERR_SHAPE,
                       "token count %d is not a multiple of ep_world %d" % (N, ep_world))
    _check_tensor("expert_ids", expert_ids, torch.int32, (N, K), dev)
    buf = DispatchBuffers(ep_world, N // ep_world, experts_per_rank, h, K, x.dtype, quant_mode, dev,
                          with_expand_scales=expert_scales is not None)
    if expert_scales is not None:            # expand_scales takes the dtype of the scales given
        buf.expand_scales = torch.empty((N * K,), dtype=getattr(expert_scales, "dtype", torch.float32),
                                        device=dev)
    dispatch_into(buf, x, expert_ids, expert_scales, schedule, x_active_mask, zero_experts, copy_experts,
                  quant_scales, const_experts)
    out = (buf.expand_x, buf.dynamic_scales, buf.assist_info, buf.ep_recv_count)
    return out + (buf.expand_scales,) if expert_scales is not None else out


def combine_into(x_out: torch.Tensor, expand_x: torch.Tensor, assist_info: torch.Tensor,
                 ep_recv_count: torch.Tensor, expert_ids: torch.Tensor, expert_scales: torch.Tensor,
                 ep_world: int, experts_per_rank: int, workspace: Optional[torch.Tensor] = None,
                 x_active_mask: Optional[torch.Tensor] = None, zero_experts: int = 0, copy_experts: int = 0,
                 ori_x: Optional[torch.Tensor] = None, const_experts: int = 0,
                 const_x: Optional[torch.Tensor] = None):
    """moe_combine into a preallocated x_out on the current stream. Copy experts need ori_x,
    the tokens given to dispatch, and const experts const_x [const_experts, h], their fixed
    outputs, both in expand_x's dtype. The C ABI sees only pointers, so the tensors' shapes,
    dtypes and device are checked here."""
    dev = _gpu_device("expand_x", expand_x)
    _gpu_device("expert_ids", expert_ids)
    if expand_x.dim() != 2 or expert_ids.dim() != 2:
        raise MoeError("moe_combine", MOE_ERR_SHAPE, "expand_x and expert_ids must be 2-D")
    N, K = expert_ids.shape
    rows, h = expand_x.shape
    if N % ep_world or rows != N * K:
        raise MoeError("moe_combine", MOE_ERR_SHAPE, "expand_x must have ep_world*bs*topk rows")
    _check_tensor("expand_x", expand_x, expand_x.dtype, (rows, h), dev)
    _check_tensor("x_out", x_out, expand_x.dtype, (N, h), dev)
    _check_tensor("assist_info", assist_info, torch.int32, (rows, 3), dev)
    _check_tensor("ep_recv_count", ep_recv_count, torch.int32, (ep_world, experts_per_rank * ep_world), dev)
    _check_tensor("expert_ids", expert_ids, torch.int32, (N, K), dev)
    sdt = torch.int32 if expand_x.dtype == torch.int32 else torch.float32
    _check_tensor("expert_scales", expert_scales, sdt, (N, K), dev)
    mp, mk = _mask_args(x_active_mask, N, K, dev)
    if copy_experts:
        if ori_x is None:
            raise MoeError("moe_combine", MOE_ERR_NULLPTR, "copy experts need ori_x, the tokens given to dispatch")
        _check_tensor("ori_x", ori_x, expand_x.dtype, (N, h), dev)
    if const_experts:
        if const_x is None:
            raise MoeError("moe_combine", MOE_ERR_NULLPTR, "const experts need const_x, their outputs")
        _check_tensor("const_x", const_x, expand_x.dtype, (int(const_experts), h), dev)
    dt = dtype_code(expand_x.dtype)
    if workspace is None:
        workspace = combine_workspace(ep_world, N // ep_world, experts_per_rank, h, K, expand_x.dtype, dev)
    else:
        _check_tensor("workspace", workspace, torch.uint8, (workspace.numel(),), dev)
    rc = library().moe_combine(
        _ptr(expand_x), _ptr(assist_info), _ptr(ep_recv_count), _ptr(expert_ids), _ptr(expert_scales), mp, mk,
        _special(zero_experts, copy_experts, ori_x, const_experts, const_x), ep_world, N // ep_world,
        experts_per_rank, h, K, dt,
        _ptr(x_out), _ptr(workspace), workspace.numel(), _stream_ptr(dev))
    _check("moe_combine", rc)
    return x_out


def combine_workspace(ep_world, bs, experts_per_rank, h, topk, dtype: torch.dtype, device="cuda"):
    """Workspace tensor for moe_combine of this shape."""
    n = combine_workspace_size(ep_world, bs, experts_per_rank, h, topk, dtype_code(dtype))
    return torch.empty((max(n, 16),), dtype=torch.uint8, device=device)


def combine(expand_x: torch.Tensor, assist_info: torch.Tensor, ep_recv_count: torch.Tensor,
            expert_ids: torch.Tensor, expert_scales: torch.Tensor, ep_world: int, experts_per_rank: int,
            x_active_mask: Optional[torch.Tensor] = None, zero_experts: int = 0, copy_experts: int = 0,
            ori_x: Optional[torch.Tensor] = None, const_experts: int = 0, const_x: Optional[torch.Tensor] = None):
    """x_out[t] = sum over active k of expand_x[row(t,k)] * expert_scales[t,k] (fp32 accumulation);
    x_active_mask: the dispatch's."""
    dev = _gpu_device("expand_x", expand_x)
    _gpu_device("expert_ids", expert_ids)
    if expand_x.dim() != 2 or expert_ids.dim() != 2:
        raise MoeError("moe_combine", MOE_ERR_SHAPE, "expand_x and expert_ids must be 2-D")
    x_out = torch.empty((expert_ids.shape[0], expand_x.shape[1]), dtype=expand_x.dtype, device=dev)
    return combine_into(x_out, expand_x, assist_info, ep_recv_count, expert_ids, expert_scales, ep_world,
                        experts_per_rank, x_active_mask=x_active_mask, zero_experts=zero_experts,
                        copy_experts=copy_experts, ori_x=ori_x, const_experts=const_experts, const_x=const_x)


# ---- launches of what stands around dispatch and combine ----

_raw_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _launch(name: str, device, *args):
    """Call the library with `device` current (a launch on a device's default stream goes to the current
    device) and raise on an error status."""
    f = getattr(library(), name)
    if device.index is None or device.index == _raw_device():
        rc = f(*args)
    else:
        with torch.cuda.device(device):
            rc = f(*args)
    if rc != MOE_OK:
        _check(name, rc)


_FLOAT_CODES = {torch.float32: MOE_FP32, torch.bfloat16: MOE_BF16, torch.float16: MOE_FP16}
_HALF_CODES = {torch.bfloat16: MOE_BF16, torch.float16: MOE_FP16}


def _float_code(name, dt: torch.dtype) -> int:
    """moe_dtype of a floating tensor."""
    code = _FLOAT_CODES.get(dt)
    if code is None:
        raise MoeError(name, MOE_ERR_DTYPE, "unsupported dtype %s" % dt)
    return code


def _address(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _new(shape, dtype, device):
    """torch.empty, at three quarters of its cost for one or two dimensions."""
    if len(shape) > 2:
        return torch.empty(shape, dtype=dtype, device=device)
    return torch.empty_strided(shape, shape[1:] + (1,), dtype=dtype, device=device)


def _check_int(fn, bits):
    """Refuse sizes that a C int does not hold, which ctypes would cut off without a word; bits: all of them, or-ed."""
    if bits >> 31:
        raise MoeError(fn, MOE_ERR_SHAPE, "a size or option is negative or above 2^31 - 1")


# ---- the gradients of combine and dispatch ----

def combine_backward_workspace_size(ep_world, bs, experts_per_rank, h, topk, dtype, const_experts=0) -> int:
    _check_int("moe_combine_backward", ep_world | bs | experts_per_rank | h | topk | const_experts)
    n = ctypes.c_size_t(0)
    _check("moe_combine_backward_workspace_size",
           library().moe_combine_backward_workspace_size(ep_world, bs, experts_per_rank, h, topk, dtype, const_experts,
                                                         ctypes.byref(n)))
    return n.value


def combine_backward_workspace(ep_world, bs, experts_per_rank, h, topk, dtype: torch.dtype, const_experts=0,
                               device="cuda"):
    """Workspace tensor for moe_combine_backward of this shape, or None where it needs none."""
    n = combine_backward_workspace_size(ep_world, bs, experts_per_rank, h, topk, dtype_code(dtype), const_experts)
    return torch.empty((n,), dtype=torch.uint8, device=device) if n else None


def _row_call(fn, rows, expert_ids, ep_world, experts_per_rank):
    """(device, tokens, topk, h, dtype code) of a gradient call on dispatch's rows, its sizes checked."""
    dev = _gpu_device("the rows", rows)
    try:
        (R, h), (N, K) = rows.shape, expert_ids.shape
    except (AttributeError, ValueError):
        raise MoeError(fn, MOE_ERR_SHAPE, "the rows and expert_ids must be 2-D tensors") from None
    dt = _HALF_CODES.get(rows.dtype)
    if dt is None:
        raise MoeError(fn, MOE_ERR_DTYPE, "gradients are fp16 or bf16, got %s" % rows.dtype)
    _check_int(fn, N | K | h | ep_world | experts_per_rank)
    if ep_world < 1 or N % ep_world or R != N * K:
        raise MoeError(fn, MOE_ERR_SHAPE, "there must be ep_world*bs*topk rows")
    return dev, N, K, h, dt


def _check_routing(assist_info, ep_recv_count, expert_ids, N, K, ep_world, experts_per_rank, device):
    _check_tensor("assist_info", assist_info, torch.int32, (N * K, 3), device)
    _check_tensor("ep_recv_count", ep_recv_count, torch.int32, (ep_world, experts_per_rank * ep_world), device)
    _check_tensor("expert_ids", expert_ids, torch.int32, (N, K), device)


def _combine_backward(head, grad_expand_x, grad_scales, grad_out, expand_x, assist_info, ep_recv_count, expert_ids,
                      expert_scales, ep_world, experts_per_rank, workspace, x_active_mask, zero_experts, copy_experts,
                      ori_x, grad_ori_x, const_experts, const_x, grad_const_x):
    """moe_combine_backward on outputs that have been checked (or made); head: _row_call's result."""
    fn = "moe_combine_backward"
    dev, N, K, h, dt = head
    dtype = expand_x.dtype
    _check_routing(assist_info, ep_recv_count, expert_ids, N, K, ep_world, experts_per_rank, dev)
    _check_tensor("expand_x", expand_x, dtype, (N * K, h), dev)
    _check_tensor("grad_out", grad_out, dtype, (N, h), dev)
    _check_tensor("expert_scales", expert_scales, torch.float32, (N, K), dev)
    mp, mk = (None, MOE_MASK_NONE) if x_active_mask is None else _mask_args(x_active_mask, N, K, dev)
    special = None
    if zero_experts or copy_experts or const_experts:
        _check_int(fn, zero_experts | copy_experts | const_experts)
        for name, count, t, shape in (("ori_x", copy_experts, ori_x, (N, h)),
                                      ("const_x", const_experts, const_x, (const_experts, h))):
            if count and t is None:
                raise MoeError(fn, MOE_ERR_NULLPTR, "%s is needed: it was combine's" % name)
            if count:
                _check_tensor(name, t, dtype, shape, dev)
        special = _special(zero_experts, copy_experts, ori_x, const_experts, const_x)
    if workspace is not None:
        _check_tensor("workspace", workspace, torch.uint8, (workspace.numel(),), dev)
    elif grad_const_x is not None:
        workspace = combine_backward_workspace(ep_world, N // ep_world, experts_per_rank, h, K, dtype, const_experts, dev)
    _launch(fn, dev, grad_out.data_ptr(), expand_x.data_ptr(), assist_info.data_ptr(), ep_recv_count.data_ptr(),
            expert_ids.data_ptr(), expert_scales.data_ptr(), mp, mk, special, ep_world, N // ep_world, experts_per_rank, h,
            K, dt, grad_expand_x.data_ptr(), grad_scales.data_ptr(), _address(grad_ori_x), _address(grad_const_x),
            _address(workspace), 0 if workspace is None else workspace.numel(), _stream_ptr(dev))


def combine_backward_into(grad_expand_x: torch.Tensor, grad_scales: torch.Tensor, grad_out: torch.Tensor,
                          expand_x: torch.Tensor, assist_info: torch.Tensor, ep_recv_count: torch.Tensor,
                          expert_ids: torch.Tensor, expert_scales: torch.Tensor, ep_world: int, experts_per_rank: int,
                          workspace: Optional[torch.Tensor] = None, x_active_mask: Optional[torch.Tensor] = None,
                          zero_experts: int = 0, copy_experts: int = 0, ori_x: Optional[torch.Tensor] = None,
                          grad_ori_x: Optional[torch.Tensor] = None, const_experts: int = 0,
                          const_x: Optional[torch.Tensor] = None, grad_const_x: Optional[torch.Tensor] = None):
    """moe_combine_backward into preallocated grad_expand_x [rows, h] (rows behind the last counted one are left as
    they were), grad_scales fp32 [N, topk] and, when given, grad_ori_x [N, h] and grad_const_x [const_experts, h], on
    the current stream. workspace: combine_backward_workspace's, needed (and otherwise made) for grad_const_x. See
    combine_backward for the rest."""
    fn = "moe_combine_backward"
    head = _row_call(fn, expand_x, expert_ids, ep_world, experts_per_rank)
    dev, N, K, h, _ = head
    _check_tensor("grad_expand_x", grad_expand_x, expand_x.dtype, (N * K, h), dev)
    _check_tensor("grad_scales", grad_scales, torch.float32, (N, K), dev)
    for name, count, t, shape in (("grad_ori_x", copy_experts, grad_ori_x, (N, h)),
                                  ("grad_const_x", const_experts, grad_const_x, (const_experts, h))):
        if t is None:
            continue
        if not count:
            raise MoeError(fn, MOE_ERR_NULLPTR, "%s without such experts" % name)
        _check_tensor(name, t, expand_x.dtype, shape, dev)
    _combine_backward(head, grad_expand_x, grad_scales, grad_out, expand_x, assist_info, ep_recv_count, expert_ids,
                      expert_scales, ep_world, experts_per_rank, workspace, x_active_mask, int(zero_experts),
                      int(copy_experts), ori_x, grad_ori_x, int(const_experts), const_x, grad_const_x)
    return grad_expand_x, grad_scales


def combine_backward(grad_out: torch.Tensor, expand_x: torch.Tensor, assist_info: torch.Tensor,
                     ep_recv_count: torch.Tensor, expert_ids: torch.Tensor, expert_scales: torch.Tensor, ep_world: int,
                     experts_per_rank: int, x_active_mask: Optional[torch.Tensor] = None, zero_experts: int = 0,
                     copy_experts: int = 0, ori_x: Optional[torch.Tensor] = None, const_experts: int = 0,
                     const_x: Optional[torch.Tensor] = None):
    """Gradients of combine's inputs from grad_out [N, h], the gradient of its x_out; the other arguments are the
    combine's (fp16 or bf16 rows).

    Returns (grad_expand_x [rows, h], grad_scales fp32 [N, topk]), then grad_ori_x [N, h] with copy experts and
    grad_const_x [const_experts, h] with const experts. grad_expand_x[row(t, k)] = expert_scales[t, k] * grad_out[t], rows
    behind the last counted one uninitialised; grad_scales[t, k] is the product of the pair's row (ori_x[t], const_x[j])
    with grad_out[t], and 0 for a zero expert's or an inactive pair: gate_backward takes it.
    """
    head = _row_call("moe_combine_backward", expand_x, expert_ids, ep_world, experts_per_rank)
    dev, N, K, h, _ = head
    made = (_new((N * K, h), expand_x.dtype, dev), _new((N, K), torch.float32, dev))
    zero_experts, copy_experts, const_experts = int(zero_experts), int(copy_experts), int(const_experts)
    ori = _new((N, h), expand_x.dtype, dev) if copy_experts > 0 and ori_x is not None else None
    const = torch.empty_like(const_x) if const_experts > 0 and isinstance(const_x, torch.Tensor) else None
    _combine_backward(head, *made, grad_out, expand_x, assist_info, ep_recv_count, expert_ids, expert_scales, ep_world,
                      experts_per_rank, None, x_active_mask, zero_experts, copy_experts, ori_x, ori, const_experts, const_x,
                      const)
    return made + tuple(t for t in (ori, const) if t is not None)


def _dispatch_backward(head, grad_x, grad_expand_x, assist_info, ep_recv_count, expert_ids, ep_world, experts_per_rank,
                       x_active_mask, add, grad_expand_scales, grad_scales):
    """moe_dispatch_backward on outputs that have been checked (or made); head: _row_call's result."""
    fn = "moe_dispatch_backward"
    dev, N, K, h, dt = head
    _check_routing(assist_info, ep_recv_count, expert_ids, N, K, ep_world, experts_per_rank, dev)
    _check_tensor("grad_expand_x", grad_expand_x, grad_expand_x.dtype, (N * K, h), dev)
    if add is not None:
        _check_tensor("add", add, grad_expand_x.dtype, (N, h), dev)
    if grad_expand_scales is not None:
        _check_tensor("grad_expand_scales", grad_expand_scales, torch.float32, (N * K,), dev)
    mp, mk = (None, MOE_MASK_NONE) if x_active_mask is None else _mask_args(x_active_mask, N, K, dev)
    _launch(fn, dev, grad_expand_x.data_ptr(), assist_info.data_ptr(), ep_recv_count.data_ptr(), expert_ids.data_ptr(),
            _address(grad_expand_scales), _address(add), mp, mk, ep_world, N // ep_world, experts_per_rank, h, K, dt,
            grad_x.data_ptr(), _address(grad_scales), _stream_ptr(dev))


def dispatch_backward_into(grad_x: torch.Tensor, grad_expand_x: torch.Tensor, assist_info: torch.Tensor,
                           ep_recv_count: torch.Tensor, expert_ids: torch.Tensor, ep_world: int, experts_per_rank: int,
                           x_active_mask: Optional[torch.Tensor] = None, add: Optional[torch.Tensor] = None,
                           grad_expand_scales: Optional[torch.Tensor] = None,
                           grad_scales: Optional[torch.Tensor] = None):
    """moe_dispatch_backward into a preallocated grad_x [N, h] (which may be add itself) and, with grad_expand_scales,
    grad_scales fp32 [N, topk], on the current stream. See dispatch_backward for the rest."""
    fn = "moe_dispatch_backward"
    head = _row_call(fn, grad_expand_x, expert_ids, ep_world, experts_per_rank)
    dev, N, K, h, _ = head
    _check_tensor("grad_x", grad_x, grad_expand_x.dtype, (N, h), dev)
    if (grad_expand_scales is None) != (grad_scales is None):
        raise MoeError(fn, MOE_ERR_NULLPTR, "grad_expand_scales and grad_scales go together")
    if grad_scales is not None:
        _check_tensor("grad_scales", grad_scales, torch.float32, (N, K), dev)
    _dispatch_backward(head, grad_x, grad_expand_x, assist_info, ep_recv_count, expert_ids, ep_world, experts_per_rank,
                       x_active_mask, add, grad_expand_scales, grad_scales)
    return grad_x


def dispatch_backward(grad_expand_x: torch.Tensor, assist_info: torch.Tensor, ep_recv_count: torch.Tensor,
                      expert_ids: torch.Tensor, ep_world: int, experts_per_rank: int,
                      x_active_mask: Optional[torch.Tensor] = None, add: Optional[torch.Tensor] = None,
                      grad_expand_scales: Optional[torch.Tensor] = None):
    """Gradient of dispatch's tokens from grad_expand_x [rows, h] (fp16 or bf16), the gradient of its expand_x (or of
    what its codes stand for): grad_x[t] is the sum of the rows of t's pairs, plus add[t], in fp32, rounded once. add
    [N, h] is what else flows back to the tokens, combine_backward's grad_ori_x among it. With grad_expand_scales
    fp32 [rows], the gradient of dispatch's expand_scales, returns (grad_x, grad_scales fp32 [N, topk]), else
    grad_x [N, h]. Pairs of special experts and inactive ones have no row and get 0."""
    head = _row_call("moe_dispatch_backward", grad_expand_x, expert_ids, ep_world, experts_per_rank)
    dev, N, K, h, _ = head
    out = _new((N, h), grad_expand_x.dtype, dev)
    scales = _new((N, K), torch.float32, dev) if grad_expand_scales is not None else None
    _dispatch_backward(head, out, grad_expand_x, assist_info, ep_recv_count, expert_ids, ep_world, experts_per_rank,
                       x_active_mask, add, grad_expand_scales, scales)
    return out if scales is None else (out, scales)


# ---- the gate ----

def _logits(fn, logits):
    """(device, tokens, experts, dtype code) of a gate's logits, checked."""
    dev = _gpu_device("logits", logits)
    if logits.dim() != 2:
        raise MoeError(fn, MOE_ERR_SHAPE, "logits must be 2-D")
    dt = _float_code(fn, logits.dtype)
    _check_tensor("logits", logits, logits.dtype, logits.shape, dev)
    return (dev, *logits.shape, dt)


def _byte_mask(name, mask, shape, device):
    if (not isinstance(mask, torch.Tensor) or mask.dtype not in (torch.bool, torch.uint8) or mask.shape != shape
            or mask.device != device or not mask.is_contiguous()):
        raise MoeError(name, MOE_ERR_MASK, "%s must be a contiguous bool or uint8 tensor of shape %s on %s"
                       % (name, tuple(shape), device))


def _gate(head, ids, w, logits, topk, score, bias, groups, topk_groups, group_score, renormalize, scale, token_mask,
          pair_mask):
    """moe_gate on outputs that have been checked (or made); head: _logits' result."""
    dev, N, E, dt = head
    if bias is not None:
        _check_tensor("bias", bias, torch.float32, (E,), dev)
    if token_mask is not None:
        _byte_mask("token_mask", token_mask, (N,), dev)
    score, groups, topk_groups, group_score = int(score), int(groups), int(topk_groups), int(group_score)
    _check_int("moe_gate", N | E | topk | score | groups | topk_groups | group_score)
    _launch("moe_gate", dev, logits.data_ptr(), _address(bias), _address(token_mask), N, E, topk, dt, score,
            groups, topk_groups, group_score, 1 if renormalize else 0, float(scale), ids.data_ptr(),
            w.data_ptr(), _address(pair_mask), _stream_ptr(dev))


def gate_into(expert_ids: torch.Tensor, expert_scales: torch.Tensor, logits: torch.Tensor,
              score: int = MOE_SCORE_SOFTMAX, bias: Optional[torch.Tensor] = None, groups: int = 1,
              topk_groups: int = 1, group_score: int = MOE_GROUP_MAX, renormalize: bool = True, scale: float = 1.0,
              token_mask: Optional[torch.Tensor] = None, pair_mask: Optional[torch.Tensor] = None):
    """moe_gate into preallocated expert_ids [N, topk] int32, expert_scales [N, topk] fp32 and, when given,
    pair_mask [N, topk] bool or uint8, on the current stream. See gate for the rest."""
    head = _logits("moe_gate", logits)
    if not isinstance(expert_ids, torch.Tensor) or expert_ids.dim() != 2:
        raise MoeError("moe_gate", MOE_ERR_SHAPE, "expert_ids must be 2-D")
    dev, N, K = head[0], head[1], expert_ids.shape[1]
    _check_tensor("expert_ids", expert_ids, torch.int32, (N, K), dev)
    _check_tensor("expert_scales", expert_scales, torch.float32, (N, K), dev)
    if pair_mask is not None:
        _byte_mask("pair_mask", pair_mask, (N, K), dev)
    _gate(head, expert_ids, expert_scales, logits, K, score, bias, groups, topk_groups, group_score, renormalize,
          scale, token_mask, pair_mask)
    return expert_ids, expert_scales


def gate(logits: torch.Tensor, topk: int, score: int = MOE_SCORE_SOFTMAX, bias: Optional[torch.Tensor] = None,
         groups: int = 1, topk_groups: int = 1, group_score: int = MOE_GROUP_MAX, renormalize: bool = True,
         scale: float = 1.0, token_mask: Optional[torch.Tensor] = None, with_pair_mask: bool = False):
    """Choose each token's experts and weights from a router's logits [N, E] (fp16, bf16 or fp32).

    score: MOE_SCORE_SOFTMAX or MOE_SCORE_SIGMOID. bias: fp32 [E], added to the scores for the choice
    alone. groups > 1: only the experts of the topk_groups best groups can be chosen, a group being
    worth its best expert (MOE_GROUP_MAX) or the sum of its two best (MOE_GROUP_TOP2). The weights are
    the chosen scores, divided by their sum if renormalize, times scale.
    Returns (expert_ids int32 [N, topk], expert_scales fp32 [N, topk]) and, with_pair_mask, a bool
    [N, topk] that is False where there was no expert to choose (logits of -inf or NaN) or the token is
    not in token_mask (bool or uint8 [N]); such pairs have id -1 and weight 0, and dispatch and combine
    take the mask as x_active_mask. The outputs carry no autograd graph: gate_backward gives the
    gradient of the logits.
    """
    head = _logits("moe_gate", logits)
    topk = int(topk)
    if not 1 <= topk <= head[2]:
        raise MoeError("moe_gate", MOE_ERR_SHAPE, "topk must be between 1 and the number of experts")
    dev, shape = head[0], (head[1], topk)
    ids, w = _new(shape, torch.int32, dev), _new(shape, torch.float32, dev)
    on = _new(shape, torch.bool, dev) if with_pair_mask else None
    _gate(head, ids, w, logits, topk, score, bias, groups, topk_groups, group_score, renormalize, scale, token_mask,
          on)
    return (ids, w, on) if with_pair_mask else (ids, w)


def _gate_backward(head, out, logits, ids, w, grad, score, renormalize, scale):
    dev, N, E, dt = head
    if not isinstance(ids, torch.Tensor) or ids.dim() != 2:
        raise MoeError("moe_gate_backward", MOE_ERR_SHAPE, "expert_ids must be 2-D")
    K = ids.shape[1]
    _check_tensor("expert_ids", ids, torch.int32, (N, K), dev)
    _check_tensor("expert_scales", w, torch.float32, (N, K), dev)
    _check_tensor("grad_scales", grad, torch.float32, (N, K), dev)
    _check_int("moe_gate_backward", N | E | K | int(score))
    _launch("moe_gate_backward", dev, logits.data_ptr(), ids.data_ptr(), w.data_ptr(), grad.data_ptr(), N, E, K, dt,
            int(score), 1 if renormalize else 0, float(scale), out.data_ptr(), _stream_ptr(dev))
    return out


def gate_backward_into(grad_logits: torch.Tensor, logits: torch.Tensor, expert_ids: torch.Tensor,
                       expert_scales: torch.Tensor, grad_scales: torch.Tensor, score: int = MOE_SCORE_SOFTMAX,
                       renormalize: bool = True, scale: float = 1.0):
    """moe_gate_backward into a preallocated grad_logits (logits' shape and dtype; every element is
    written) on the current stream."""
    head = _logits("moe_gate_backward", logits)
    _check_tensor("grad_logits", grad_logits, logits.dtype, logits.shape, head[0])
    return _gate_backward(head, grad_logits, logits, expert_ids, expert_scales, grad_scales, score, renormalize, scale)


def gate_backward(logits: torch.Tensor, expert_ids: torch.Tensor, expert_scales: torch.Tensor,
                  grad_scales: torch.Tensor, score: int = MOE_SCORE_SOFTMAX, renormalize: bool = True,
                  scale: float = 1.0) -> torch.Tensor:
    """Gradient of gate's logits from grad_scales, the gradient of its expert_scales: [N, E] in the
    logits' dtype. expert_ids and expert_scales are gate's outputs for the same score, renormalize and
    scale; pairs with id -1 give and get nothing."""
    head = _logits("moe_gate_backward", logits)
    return _gate_backward(head, _new((head[1], head[2]), logits.dtype, head[0]), logits, expert_ids, expert_scales,
                          grad_scales, score, renormalize, scale)


# ---- microscaled rows and the experts' product ----

MX_BLOCK = 32                # elements that share a scale byte


def _mx_codes(element):
    """(torch dtype of the codes, codes a byte): E2M1 is packed two a byte in uint8."""
    if element == MOE_MX_E2M1:
        return torch.uint8, 2
    if element == MOE_MX_E4M3:
        return torch.float8_e4m3fn, 1
    raise MoeError("element", MOE_ERR_QUANT, "unknown microscaled element type %r" % (element,))


def _mx_rows(name, codes):
    """(element, rows shape) of microscaled codes: float8_e4m3fn [..., cols] or packed uint8 [..., cols / 2]."""
    if codes.dtype == torch.float8_e4m3fn:
        return MOE_MX_E4M3, tuple(codes.shape)
    if codes.dtype == torch.uint8:
        return MOE_MX_E2M1, tuple(codes.shape[:-1]) + (2 * codes.shape[-1],)
    raise MoeError(name, MOE_ERR_DTYPE, "microscaled codes are float8_e4m3fn or packed uint8, got %s" % codes.dtype)


def _quantize(codes, scales, x, cols, element):
    """moe_mx_quantize of checked tensors; cols is not 0."""
    dev = x.device
    _launch("moe_mx_quantize", dev, x.data_ptr(), x.numel() // cols, cols, _float_code("moe_mx_quantize", x.dtype),
            element, codes.data_ptr(), scales.data_ptr(), _stream_ptr(dev))
    return codes, scales


def _columns(fn, cols):
    if cols < 1 or cols % 16:
        raise MoeError(fn, MOE_ERR_SHAPE, "the last dimension must be a multiple of 16")
    _check_int(fn, cols)


def quantize_mx_into(codes: torch.Tensor, scales: torch.Tensor, x: torch.Tensor):
    """moe_mx_quantize of x [..., cols] into preallocated codes (float8_e4m3fn [..., cols], or uint8
    [..., cols / 2] for packed E2M1) and scales (uint8 [..., ceil(cols / 32)]), on the current stream."""
    dev = _gpu_device("x", x)
    _gpu_device("codes", codes)
    if x.dim() < 1 or codes.dim() < 1:
        raise MoeError("moe_mx_quantize", MOE_ERR_SHAPE, "x must have at least one dimension")
    element, shape = _mx_rows("codes", codes)
    _columns("moe_mx_quantize", shape[-1])
    _check_tensor("x", x, x.dtype, shape, dev)
    _check_tensor("codes", codes, codes.dtype, codes.shape, dev)
    _check_tensor("scales", scales, torch.uint8, shape[:-1] + (-(-shape[-1] // MX_BLOCK),), dev)
    return _quantize(codes, scales, x, shape[-1], element)


def quantize_mx(x: torch.Tensor, element: int = MOE_MX_E2M1):
    """Microscaled rows of x [..., cols] (fp16, bf16 or fp32; cols a multiple of 16): (codes, scales).
    E2M1 codes are packed two a byte (uint8 [..., cols / 2], the even element in the low nibble), E4M3
    ones are float8_e4m3fn [..., cols]; scales are E8M0 bytes, uint8 [..., ceil(cols / 32)], each the
    power 2^(byte - 127) of a block of 32 elements. A block with an infinity or NaN gets byte 255 (NaN)."""
    dev = _gpu_device("x", x)
    dt, per = _mx_codes(element)
    shape = tuple(x.shape)
    cols = shape[-1] if shape else 0
    _columns("moe_mx_quantize", cols)
    if x.dtype not in _FLOAT_CODES or not x.is_contiguous():
        raise MoeError("moe_mx_quantize", MOE_ERR_DTYPE if x.dtype not in _FLOAT_CODES else MOE_ERR_SHAPE,
                       "x must be a contiguous fp16, bf16 or fp32 tensor, got %s" % x.dtype)
    lead = shape[:-1]
    return _quantize(_new(lead + (cols // per,), dt, dev), _new(lead + (-(-cols // MX_BLOCK),), torch.uint8, dev), x,
                     cols, element)


def _dequantize(out, codes, scales, shape, element):
    """moe_mx_dequantize of a checked out."""
    dev, cols = out.device, shape[-1]
    _columns("moe_mx_dequantize", cols)
    _check_tensor("codes", codes, codes.dtype, codes.shape, dev)
    _check_tensor("scales", scales, torch.uint8, shape[:-1] + (-(-cols // MX_BLOCK),), dev)
    _launch("moe_mx_dequantize", dev, codes.data_ptr(), scales.data_ptr(), out.numel() // cols, cols,
            _float_code("moe_mx_dequantize", out.dtype), element, out.data_ptr(), _stream_ptr(dev))
    return out


def dequantize_mx_into(out: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor):
    """moe_mx_dequantize into a preallocated out [..., cols] (fp16, bf16 or fp32) on the current stream."""
    _gpu_device("codes", codes)
    dev = _gpu_device("out", out)
    if codes.dim() < 1:
        raise MoeError("moe_mx_dequantize", MOE_ERR_SHAPE, "codes must have at least one dimension")
    element, shape = _mx_rows("codes", codes)
    _check_tensor("out", out, out.dtype, shape, dev)
    return _dequantize(out, codes, scales, shape, element)


def dequantize_mx(codes: torch.Tensor, scales: torch.Tensor, dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """What microscaled codes and scales stand for, code * 2^(byte - 127), in dtype."""
    dev = _gpu_device("codes", codes)
    if codes.dim() < 1:
        raise MoeError("moe_mx_dequantize", MOE_ERR_SHAPE, "codes must have at least one dimension")
    _float_code("moe_mx_dequantize", dtype)
    element, shape = _mx_rows("codes", codes)
    return _dequantize(_new(shape, dtype, dev), codes, scales, shape, element)


# ---- rows of 8-bit integers ----

def _int8_rows(fn, x):
    """(device, shape, dtype code) of rows to quantise, checked."""
    dev = _gpu_device("x", x)
    shape = tuple(x.shape)
    if not shape or not 0 < shape[-1] < 1 << 31 or not x.is_contiguous():
        raise MoeError(fn, MOE_ERR_SHAPE, "x must be contiguous, with 1 to 2^31 - 1 columns; got %s" % (shape,))
    return dev, shape, _float_code(fn, x.dtype)


def _quantize_int8(codes, scales, x, head):
    """moe_int8_quantize into checked (or new) outputs; head: _int8_rows' result."""
    dev, shape, dt = head
    _launch("moe_int8_quantize", dev, x.data_ptr(), x.numel() // shape[-1], shape[-1], dt, codes.data_ptr(),
            scales.data_ptr(), _stream_ptr(dev))
    return codes, scales


def quantize_int8_into(codes: torch.Tensor, scales: torch.Tensor, x: torch.Tensor):
    """moe_int8_quantize of x [..., cols] into preallocated codes (int8 [..., cols]) and scales (fp32 [...]), on the
    current stream."""
    head = _int8_rows("moe_int8_quantize", x)
    _check_tensor("codes", codes, torch.int8, head[1], head[0])
    _check_tensor("scales", scales, torch.float32, head[1][:-1], head[0])
    return _quantize_int8(codes, scales, x, head)


def quantize_int8(x: torch.Tensor):
    """Rows of x [..., cols] (fp16, bf16 or fp32) as int8 codes with one scale each: (codes int8 [..., cols], scales
    fp32 [...]), scale = max|x| / 127 and code = x / scale rounded to the nearest, ties to even: what dispatch writes
    under MOE_QUANT_DYN_TOKEN. A row of zeros has scale 0; one with an infinity or NaN has scale NaN and codes 0."""
    head = _int8_rows("moe_int8_quantize", x)
    dev, shape, _ = head
    scales = _new(shape[:-1], torch.float32, dev) if len(shape) > 1 else torch.empty((), dtype=torch.float32, device=dev)
    return _quantize_int8(_new(shape, torch.int8, dev), scales, x, head)


def _dequantize_int8(out, codes, scales, dt):
    """moe_int8_dequantize into a checked (or new) out."""
    fn, dev, shape = "moe_int8_dequantize", out.device, tuple(codes.shape)
    if not shape or not 0 < shape[-1] < 1 << 31:
        raise MoeError(fn, MOE_ERR_SHAPE, "codes must have 1 to 2^31 - 1 columns")
    _check_tensor("codes", codes, torch.int8, shape, dev)
    _check_tensor("scales", scales, torch.float32, shape[:-1], dev)
    _launch(fn, dev, codes.data_ptr(), scales.data_ptr(), codes.numel() // shape[-1], shape[-1], dt, out.data_ptr(),
            _stream_ptr(dev))
    return out


def dequantize_int8_into(out: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor):
    """moe_int8_dequantize into a preallocated out [..., cols] (fp16, bf16 or fp32) on the current stream."""
    dev = _gpu_device("codes", codes)
    _gpu_device("out", out)
    dt = _float_code("moe_int8_dequantize", out.dtype)
    _check_tensor("out", out, out.dtype, codes.shape, dev)
    return _dequantize_int8(out, codes, scales, dt)


def dequantize_int8(codes: torch.Tensor, scales: torch.Tensor, dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """What int8 codes [..., cols] and scales fp32 [...] stand for, code * scale, in dtype: quantize_int8's rows, or
    dispatch's under MOE_QUANT_DYN_TOKEN."""
    dev = _gpu_device("codes", codes)
    dt = _float_code("moe_int8_dequantize", dtype)
    if codes.dim() < 1:
        raise MoeError("moe_int8_dequantize", MOE_ERR_SHAPE, "codes must have columns")
    return _dequantize_int8(_new(tuple(codes.shape), dtype, dev), codes, scales, dt)


# ---- the experts' product ----

def _product_int8(out, x, x_scales, weights, weight_scales, ep_recv_count, activation):
    """moe_expert_product_int8 of rows x on a GPU."""
    fn, dev = "moe_expert_product_int8", x.device
    try:
        (rows, k), (E, n, _), (W, _), dt = x.shape, weights.shape, ep_recv_count.shape, _HALF_CODES.get(out.dtype)
    except (AttributeError, ValueError):
        raise MoeError(fn, MOE_ERR_SHAPE, "x, weights and ep_recv_count must have 2, 3 and 2 dimensions") from None
    if W < 1 or E % W:
        raise MoeError(fn, MOE_ERR_SHAPE, "%d experts are not a multiple of %d ranks" % (E, W))
    if dt is None:
        raise MoeError(fn, MOE_ERR_DTYPE, "out must be fp16 or bf16, got %s" % out.dtype)
    _check_tensor("x", x, torch.int8, (rows, k), dev)
    if x_scales is not None:
        _check_tensor("x_scales", x_scales, torch.float32, (rows,), dev)
    _check_tensor("weights", weights, torch.int8, (E, n, k), dev)
    _check_tensor("weight_scales", weight_scales, torch.float32, (E, n), dev)
    _check_tensor("ep_recv_count", ep_recv_count, torch.int32, (W, E), dev)
    _check_tensor("out", out, out.dtype, (rows, n // 2 if activation == MOE_ACT_SWIGLU else n), dev)
    _check_int(fn, W | E | rows | k | n | int(activation))
    _launch(fn, dev, x.data_ptr(), _address(x_scales), weights.data_ptr(), weight_scales.data_ptr(),
            ep_recv_count.data_ptr(), W, E // W, rows, k, n, int(activation), dt, out.data_ptr(), _stream_ptr(dev))
    return out


def expert_product_into(out: torch.Tensor, x: torch.Tensor, x_scales: Optional[torch.Tensor], weights: torch.Tensor,
                        weight_scales: torch.Tensor, ep_recv_count: torch.Tensor, activation: int = MOE_ACT_NONE):
    """moe_expert_product (or, with int8 rows, moe_expert_product_int8) into a preallocated out [rows, n] ([rows, n / 2]
    with MOE_ACT_SWIGLU) in fp16 or bf16, on the current stream. Rows behind the last that ep_recv_count counts are left as
    they were."""
    dev = _gpu_device("x", x)
    if x.dtype == torch.int8:
        return _product_int8(out, x, x_scales, weights, weight_scales, ep_recv_count, activation)
    _gpu_device("weights", weights)
    _gpu_device("ep_recv_count", ep_recv_count)
    _gpu_device("out", out)
    if x.dim() != 2 or weights.dim() != 3 or ep_recv_count.dim() != 2 or out.dim() != 2:
        raise MoeError("moe_expert_product", MOE_ERR_SHAPE,
                       "x, weights, ep_recv_count and out must have 2, 3, 2 and 2 dimensions")
    element, (rows, k) = _mx_rows("x", x)
    E, n = weights.shape[:2]
    W, nb = ep_recv_count.shape[0], -(-k // MX_BLOCK)
    if W < 1 or E % W:
        raise MoeError("moe_expert_product", MOE_ERR_SHAPE, "%d experts are not a multiple of %d ranks" % (E, W))
    if out.dtype not in (torch.float16, torch.bfloat16):
        raise MoeError("moe_expert_product", MOE_ERR_DTYPE, "out must be fp16 or bf16, got %s" % out.dtype)
    _check_tensor("x", x, x.dtype, x.shape, dev)
    _check_tensor("x_scales", x_scales, torch.uint8, (rows, nb), dev)
    _check_tensor("weights", weights, torch.uint8, (E, n, k // 2), dev)
    _check_tensor("weight_scales", weight_scales, torch.uint8, (E, n, nb), dev)
    _check_tensor("ep_recv_count", ep_recv_count, torch.int32, (W, E), dev)
    _check_tensor("out", out, out.dtype, (rows, n // 2 if activation == MOE_ACT_SWIGLU else n), dev)
    _check_int("moe_expert_product", W | E | rows | k | n | int(activation))
    _launch("moe_expert_product", dev, x.data_ptr(), x_scales.data_ptr(), element, weights.data_ptr(),
            weight_scales.data_ptr(), ep_recv_count.data_ptr(), W, E // W, rows, k, n, int(activation),
            dtype_code(out.dtype), out.data_ptr(), _stream_ptr(dev))
    return out


def expert_product(x: torch.Tensor, x_scales: Optional[torch.Tensor], weights: torch.Tensor, weight_scales: torch.Tensor,
                   ep_recv_count: torch.Tensor, activation: int = MOE_ACT_NONE,
                   dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """Each row of dispatch's order times its expert's weights.

    Either x, x_scales: microscaled rows [rows, k], from dispatch under MOE_QUANT_MX or from quantize_mx;
    weights, weight_scales: quantize_mx of [E, n, k] in E2M1. Or x int8 [rows, k] and x_scales fp32 [rows],
    from dispatch under MOE_QUANT_DYN_TOKEN or from quantize_int8 (x_scales None: 1, for dispatch's rows under
    MOE_QUANT_STATIC); weights, weight_scales: quantize_int8 of [E, n, k], int8 and fp32 [E, n]. Static rows stand
    for code / coefficient: one coefficient divides weight_scales; those of the columns, quant_scales [k] or [E, k],
    divide the weights before these are quantised, quantize_int8(w / c[..., None, :]).
    ep_recv_count: dispatch's. Returns [rows, n], or with MOE_ACT_SWIGLU [rows, n / 2]: silu(first n / 2
    weight rows) * the others. Rows behind the last counted one are uninitialised.
    """
    dev = _gpu_device("x", x)
    if x.dim() != 2 or not isinstance(weights, torch.Tensor) or weights.dim() != 3:
        raise MoeError("moe_expert_product", MOE_ERR_SHAPE, "x must be 2-D and weights 3-D")
    n = weights.shape[1]
    out = _new((x.shape[0], n // 2 if activation == MOE_ACT_SWIGLU else n), dtype, dev)
    return expert_product_into(out, x, x_scales, weights, weight_scales, ep_recv_count, activation)
