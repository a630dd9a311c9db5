"""ctypes binding of libbf16_linear.so — argument marshalling only.

Every step of the computation runs in the library's CUDA kernels; this module
(and csrc/torch_calls.cpp for the calls that a decode step makes most) turns torch tensors into (pointer, size, stream) arguments, checks dtype /
contiguity / device on the Python side (the dtype guards the vLLM PR #42562
review asked for: both x and W must be bfloat16), and raises on a nonzero
status.  There is no fallback: if the library is missing the import-time
loader raises.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import NamedTuple

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libbf16_linear.so")

OK, EINVAL, EALIGN, EARCH, ELAUNCH, ETIMEOUT, EUNSUPPORTED, ENOSCRATCH = 0, -1, -2, -3, -4, -5, -6, -7
FLAG_PDL = 1      # weights read before the grid-dependency wait
FLAG_SERIAL = 2   # no programmatic dependent launch
(KERNEL_DOTPROD, KERNEL_SPLITK, KERNEL_TILE, KERNEL_SPLITK_WS, KERNEL_STREAM, KERNEL_TILE2, KERNEL_WARPROW,
 KERNEL_WARPMMA, KERNEL_DOTMMA, KERNEL_DOTMMA_WS, KERNEL_TILE_T) = range(11)
KERNEL_NAMES = {KERNEL_DOTPROD: "dotprod", KERNEL_SPLITK: "splitk", KERNEL_TILE: "tile",
                KERNEL_SPLITK_WS: "splitk_ws", KERNEL_STREAM: "stream", KERNEL_TILE2: "tile2",
                KERNEL_WARPROW: "warprow", KERNEL_WARPMMA: "warpmma", KERNEL_DOTMMA: "dotmma",
                KERNEL_DOTMMA_WS: "dotmma_ws", KERNEL_TILE_T: "tile_t"}


class Plan(ctypes.Structure):
    """Mirror of bf16l_plan in include/bf16_linear.h."""
    _fields_ = [("kernel", ctypes.c_int32), ("threads", ctypes.c_int32),
                ("rows_per_cta", ctypes.c_int32), ("tokens_per_cta", ctypes.c_int32),
                ("split_k", ctypes.c_int32), ("stages", ctypes.c_int32),
                ("grid", ctypes.c_int32), ("flags", ctypes.c_int32), ("chunks_per_stage", ctypes.c_int32)]

    def as_dict(self) -> dict:
        d = {f[0]: int(getattr(self, f[0])) for f in self._fields_}
        d["kernel_name"] = KERNEL_NAMES.get(d["kernel"], "?")
        return d

    def __repr__(self):
        return f"Plan({self.as_dict()})"


class Device(ctypes.Structure):
    """Mirror of bf16l_device."""
    _fields_ = [("cc_major", ctypes.c_int32), ("cc_minor", ctypes.c_int32), ("num_sms", ctypes.c_int32)]


class Call(ctypes.Structure):
    """Mirror of bf16l_call (the argument block of bf16_linear_run)."""
    _fields_ = [("x", ctypes.c_void_p), ("W", ctypes.c_void_p), ("bias", ctypes.c_void_p), ("out", ctypes.c_void_p),
                ("M", ctypes.c_int32), ("N", ctypes.c_int32), ("K", ctypes.c_int32), ("out_f32", ctypes.c_int32),
                ("flags", ctypes.c_uint32), ("plan", ctypes.POINTER(Plan)), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_size_t), ("stream", ctypes.c_void_p)]


class BF16LinearError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(msg)
        self.status = status


_lib = None
_calls = None  # csrc/torch_calls.cpp, where it was built for this PyTorch: the usual calls without Python's share
_lock = threading.Lock()


def _load_calls(lib):
    """The compiled marshalling module, bound to this library's entry points; None without one."""
    import importlib.util

    from . import build as _build
    try:
        path = _build.calls_path()
        if not os.path.exists(path):
            return None
        spec = importlib.util.spec_from_file_location("_torch_calls", path)
        mod = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(mod)
    except (ImportError, OSError):
        return None
    mod.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
        lib.bf16_rmsnorm, lib.bf16_route, lib.bf16_quant_mxfp4, lib.bf16_dequant_mxfp4, lib.bf16_linear_mxfp4,
        lib.bf16_linear_mxfp4_dynamic, lib.bf16_linear_mxfp4_dynamic_workspace, lib.bf16_group_rows,
        lib.bf16_linear_grouped, lib.bf16_combine_rows, lib.bf16_linear_lora, lib.bf16_linear_lora_workspace,
        lib.bf16_linear_grouped_workspace)))
    return mod


def load(path: str | None = None) -> ctypes.CDLL:
    """Load the built library (raises if it has not been built)."""
    global _lib, _calls
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise ImportError(f"{p} is missing: build it with `python -m moe_router_gemm_gb300.build` "
                              "(there is no CPU fallback)")
        lib = ctypes.CDLL(p)
        vp, i32 = ctypes.c_void_p, ctypes.c_int
        lib.bf16_linear.argtypes = [vp, vp, vp, vp, i32, i32, i32, vp]
        lib.bf16_linear.restype = i32
        lib.bf16_linear_ex.argtypes = [vp, vp, vp, vp, i32, i32, i32, ctypes.c_uint32, vp]
        lib.bf16_linear_ex.restype = i32
        lib.bf16_linear_host.argtypes = [vp, vp, vp, vp, i32, i32, i32, vp, ctypes.c_size_t, ctypes.c_uint32, vp]
        lib.bf16_linear_host.restype = i32
        lib.bf16_linear_host_staging_bytes.argtypes = [i32, i32, i32, i32]
        lib.bf16_linear_host_staging_bytes.restype = ctypes.c_size_t
        lib.bf16_linear_f32out.argtypes = [vp, vp, vp, vp, i32, i32, i32, ctypes.c_uint32, vp]
        lib.bf16_linear_f32out.restype = i32
        lib.bf16_linear_f32out_with_plan.argtypes = [vp, vp, vp, vp, i32, i32, i32, ctypes.POINTER(Plan), vp]
        lib.bf16_linear_f32out_with_plan.restype = i32
        lib.bf16_linear_with_plan.argtypes = [vp, vp, vp, vp, i32, i32, i32, ctypes.POINTER(Plan), vp]
        lib.bf16_linear_with_plan.restype = i32
        lib.bf16_linear_plan.argtypes = [i32, i32, i32, ctypes.POINTER(Plan)]
        lib.bf16_linear_plan.restype = i32
        lib.bf16_linear_plan_for_device.argtypes = [i32, i32, i32, ctypes.POINTER(Device), ctypes.POINTER(Plan)]
        lib.bf16_linear_plan_for_device.restype = i32
        lib.bf16_linear_plan_check.argtypes = [i32, i32, i32, ctypes.POINTER(Device), ctypes.POINTER(Plan)]
        lib.bf16_linear_plan_check.restype = i32
        lib.bf16_linear_run.argtypes = [ctypes.POINTER(Call)]
        lib.bf16_linear_run.restype = i32
        lib.bf16_linear_workspace_size.argtypes = [i32, i32, i32, ctypes.POINTER(Plan)]
        lib.bf16_linear_workspace_size.restype = ctypes.c_size_t
        lib.bf16_linear_plan_ws.argtypes = [i32, i32, i32, ctypes.POINTER(Device), ctypes.c_size_t,
                                            ctypes.POINTER(Plan)]
        lib.bf16_linear_plan_ws.restype = i32
        lib.bf16_linear_noalloc.argtypes = [vp, vp, vp, vp, i32, i32, i32, vp]
        lib.bf16_linear_noalloc.restype = i32
        lib.bf16_quant_fp8.argtypes = [vp, vp, vp, ctypes.c_int64, ctypes.c_uint32, vp]
        lib.bf16_quant_fp8.restype = i32
        lib.bf16_linear_fp8.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, i32, ctypes.c_uint32, vp]
        lib.bf16_linear_fp8.restype = i32
        lib.bf16_linear_fp8_with_plan.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, i32, ctypes.POINTER(Plan), vp]
        lib.bf16_linear_fp8_with_plan.restype = i32
        lib.bf16_linear_fp8_split.argtypes = [i32, i32, i32, i32]
        lib.bf16_linear_fp8_split.restype = i32
        lib.bf16_quant_mxfp8.argtypes = [vp, ctypes.c_int64, i32, vp, vp, ctypes.c_uint32, vp]
        lib.bf16_quant_mxfp8.restype = i32
        lib.bf16_linear_mxfp8.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, i32, ctypes.c_uint32, vp]
        lib.bf16_linear_mxfp8.restype = i32
        lib.bf16_linear_mxfp8_with_plan.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, i32, ctypes.POINTER(Plan), vp]
        lib.bf16_linear_mxfp8_with_plan.restype = i32
        lib.bf16_linear_mxfp8_split.argtypes = [i32, i32, i32, i32, i32]
        lib.bf16_linear_mxfp8_split.restype = i32
        i64, u32, f32 = ctypes.c_int64, ctypes.c_uint32, ctypes.c_float
        lib.bf16_rmsnorm.argtypes = [vp, i64, vp, vp, vp, vp, vp, vp, vp, i64, i32, f32, i32, u32, vp]
        lib.bf16_rmsnorm.restype = i32
        lib.bf16_route.argtypes = [vp, i64, vp, vp, vp, i64, i32, i32, i32, i32, i32, i32, i32, f32, i32, u32, vp]
        lib.bf16_route.restype = i32
        lib.bf16_quant_mxfp4.argtypes = [vp, i64, i32, vp, vp, u32, vp]
        lib.bf16_quant_mxfp4.restype = i32
        lib.bf16_dequant_mxfp4.argtypes = [vp, vp, i64, i32, vp, u32, vp]
        lib.bf16_dequant_mxfp4.restype = i32
        lib.bf16_linear_mxfp4.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, i32, u32, vp]
        lib.bf16_linear_mxfp4.restype = i32
        lib.bf16_linear_mxfp4_dynamic.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, vp, ctypes.c_size_t, u32, vp]
        lib.bf16_linear_mxfp4_dynamic.restype = i32
        lib.bf16_linear_mxfp4_dynamic_workspace.argtypes = [i32, i32, i32]
        lib.bf16_linear_mxfp4_dynamic_workspace.restype = ctypes.c_size_t
        lib.bf16_group_rows.argtypes = [vp, i64, i32, i32, vp, vp, vp, u32, vp]
        lib.bf16_group_rows.restype = i32
        lib.bf16_linear_grouped.argtypes = [vp, i64, vp, vp, vp, vp, vp, i64, i32, i32, i32, i32, vp, ctypes.c_size_t, u32, vp]
        lib.bf16_linear_grouped.restype = i32
        lib.bf16_linear_grouped_workspace.argtypes = [i64, i32, i32, i32, i32]
        lib.bf16_linear_grouped_workspace.restype = ctypes.c_size_t
        lib.bf16_combine_rows.argtypes = [vp, i64, vp, vp, vp, vp, i64, i32, i32, u32, vp]
        lib.bf16_combine_rows.restype = i32
        lib.bf16_linear_lora.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, vp, ctypes.c_size_t, u32, vp]
        lib.bf16_linear_lora.restype = i32
        lib.bf16_linear_lora_workspace.argtypes = [i32, i32, i32, i32, i32]
        lib.bf16_linear_lora_workspace.restype = ctypes.c_size_t
        lib.bf16_linear_probe_read.argtypes = [vp, ctypes.c_size_t, i32, i32, vp, ctypes.c_uint32, vp]
        lib.bf16_linear_probe_read.restype = i32
        lib.bf16_linear_noalloc_scratch_bytes.argtypes = []
        lib.bf16_linear_noalloc_scratch_bytes.restype = ctypes.c_size_t
        lib.bf16_linear_device_status.argtypes = [ctypes.POINTER(ctypes.c_int32), i32]
        lib.bf16_linear_device_status.restype = i32
        lib.bf16_linear_selftest_wait.argtypes = [ctypes.c_uint32, vp]
        lib.bf16_linear_selftest_wait.restype = i32
        lib.bf16_linear_strerror.argtypes = [i32]
        lib.bf16_linear_strerror.restype = ctypes.c_char_p
        lib.bf16_linear_cuda_error.argtypes = []
        lib.bf16_linear_cuda_error.restype = i32
        lib.bf16_linear_version.argtypes = []
        lib.bf16_linear_version.restype = i32
        _calls = _load_calls(lib)
        _lib = lib
        return lib


def strerror(status: int) -> str:
    return load().bf16_linear_strerror(int(status)).decode()


def _raise(status: int, what: str):
    lib = load()
    extra = ""
    if status == ELAUNCH:
        extra = f" (cuda error {lib.bf16_linear_cuda_error()})"
    raise BF16LinearError(status, f"{what}: {strerror(status)}{extra}")


def plan(M: int, N: int, K: int, device: tuple[int, int, int] | None = None) -> Plan:
    """The kernel and parameters chosen for (M, N, K); device = (cc_major, cc_minor, num_sms)."""
    p = Plan()
    if device is None:
        st = load().bf16_linear_plan(int(M), int(N), int(K), ctypes.byref(p))
    else:
        st = load().bf16_linear_plan_for_device(int(M), int(N), int(K), ctypes.byref(Device(*device)),
                                                ctypes.byref(p))
    if st != OK:
        _raise(st, f"bf16_linear_plan({M},{N},{K})")
    return p


def plan_check(M: int, N: int, K: int, p: Plan, device: tuple[int, int, int] | None = None) -> Plan:
    """Validate an explicit plan for (M, N, K); fills p.grid, raises BF16LinearError if unusable."""
    dev = Device(*device) if device is not None else None
    st = load().bf16_linear_plan_check(int(M), int(N), int(K), ctypes.byref(dev) if dev is not None else None,
                                       ctypes.byref(p))
    if st != OK:
        _raise(st, f"bf16_linear_plan_check({M},{N},{K}, {p})")
    return p


def plan_ws(M: int, N: int, K: int, workspace_bytes: int, device: tuple[int, int, int] | None = None) -> Plan:
    """The dispatcher's choice when `workspace_bytes` of workspace are available."""
    p = Plan()
    dev = Device(*device) if device is not None else None
    st = load().bf16_linear_plan_ws(int(M), int(N), int(K), ctypes.byref(dev) if dev is not None else None,
                                    int(workspace_bytes), ctypes.byref(p))
    if st != OK:
        _raise(st, f"bf16_linear_plan_ws({M},{N},{K})")
    return p


def workspace_size(M: int, N: int, K: int, p: Plan | None = None) -> int:
    """Workspace bytes a call needs (for plan p, else for the dispatcher's choice with workspace allowed)."""
    return int(load().bf16_linear_workspace_size(int(M), int(N), int(K), ctypes.byref(p) if p is not None else None))


def make_plan(kernel: int | str, **fields) -> Plan:
    """Build an explicit plan (for with_plan); unspecified fields are 0."""
    if isinstance(kernel, str):
        kernel = {v: k for k, v in KERNEL_NAMES.items()}[kernel]
    p = Plan()
    p.kernel = int(kernel)
    for k, v in fields.items():
        setattr(p, k, int(v))
    return p


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _check(x, W, bias, out, out_dtype=None):
    import torch
    if x.dtype != torch.bfloat16 or W.dtype != torch.bfloat16:
        raise TypeError(f"x and W must be torch.bfloat16 (got {x.dtype}, {W.dtype})")
    if bias is not None and bias.dtype != torch.bfloat16:
        raise TypeError(f"bias must be torch.bfloat16 (got {bias.dtype})")
    if x.dim() != 2 or W.dim() != 2 or x.shape[1] != W.shape[1]:
        raise ValueError(f"need x[M,K] and W[N,K], got {tuple(x.shape)} and {tuple(W.shape)}")
    M, K = x.shape
    N = W.shape[0]
    if bias is not None and tuple(bias.shape) != (N,):
        raise ValueError(f"bias must be [{N}], got {tuple(bias.shape)}")
    for name, t in (("x", x), ("W", W), ("bias", bias)):
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    odt = out_dtype or torch.bfloat16
    if out is None:
        out = torch.empty((M, N), dtype=odt, device=x.device)
    elif out.dtype != odt or tuple(out.shape) != (M, N) or not out.is_contiguous() or not out.is_cuda:
        raise ValueError(f"out must be a contiguous CUDA {odt} tensor of shape [M, N]")
    devs = {t.device for t in (x, W, bias, out) if t is not None}
    if len(devs) != 1:
        raise ValueError(f"all tensors must be on one device, got {devs}")
    return M, N, K, out


def _stream_handle(stream, device):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream)


def host_staging_bytes(M: int, N: int, K: int, with_bias: bool) -> int:
    """Device staging bytes bf16_linear_host needs (bf16_linear_host_staging_bytes)."""
    return int(load().bf16_linear_host_staging_bytes(int(M), int(N), int(K), 1 if with_bias else 0))


def new_host_staging(M: int, N: int, K: int, with_bias: bool, device=None):
    """A device staging tensor for bf16_linear_host (the caching allocator aligns blocks to 512 bytes)."""
    import torch
    return torch.empty(max(256, host_staging_bytes(M, N, K, with_bias)), dtype=torch.uint8,
                       device=device or "cuda")


def bf16_linear_host(x, W, bias=None, out=None, *, staging, flags: int = 0, stream=None):
    """bf16_linear_host: x[M,K], W[N,K], bias[N] and out[M,N] are CPU bf16 tensors (page-locked for
    asynchronous copies; out is allocated page-locked when None); the library copies them through the
    CUDA tensor `staging`, runs the planned kernel and copies out back, all on the given (or current)
    stream.  Returns out, complete once the stream has reached the final copy."""
    import torch
    for name, t in (("x", x), ("W", W), ("bias", bias)):
        if t is not None and (t.dtype != torch.bfloat16 or t.is_cuda or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous CPU bf16 tensor")
    if x.dim() != 2 or W.dim() != 2 or x.shape[1] != W.shape[1]:
        raise ValueError(f"need x[M,K] and W[N,K], got {tuple(x.shape)} and {tuple(W.shape)}")
    M, K = x.shape
    N = W.shape[0]
    if bias is not None and tuple(bias.shape) != (N,):
        raise ValueError(f"bias must be [{N}], got {tuple(bias.shape)}")
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16).pin_memory()
    elif out.dtype != torch.bfloat16 or out.is_cuda or tuple(out.shape) != (M, N) or not out.is_contiguous():
        raise ValueError("out must be a contiguous CPU bf16 tensor of shape [M, N]")
    if not staging.is_cuda or not staging.is_contiguous():
        raise ValueError("staging must be a contiguous CUDA tensor")
    dev = staging.device
    if torch.cuda.current_device() == dev.index:  # (entering a device context costs more than the call)
        h = _stream_handle(stream, dev)
        st = load().bf16_linear_host(_ptr(x), _ptr(W), _ptr(bias), _ptr(out), M, N, K, _ptr(staging),
                                     staging.numel() * staging.element_size(), int(flags), h)
    else:
        with torch.cuda.device(dev):
            st = load().bf16_linear_host(_ptr(x), _ptr(W), _ptr(bias), _ptr(out), M, N, K, _ptr(staging),
                                         staging.numel() * staging.element_size(), int(flags),
                                         _stream_handle(stream, dev))
    if st != OK:
        _raise(st, f"bf16_linear_host(M={M}, N={N}, K={K})")
    return out


def bf16_linear(x, W, bias=None, out=None, stream=None):
    """out[M,N] = x[M,K] @ W[N,K]^T (+ bias[N]) in bf16, on the given (or current) stream."""
    import torch
    M, N, K, out = _check(x, W, bias, out)
    with torch.cuda.device(x.device):
        st = load().bf16_linear(_ptr(x), _ptr(W), _ptr(bias), _ptr(out), M, N, K,
                                _stream_handle(stream, x.device))
    if st != OK:
        _raise(st, f"bf16_linear(M={M}, N={N}, K={K})")
    return out


def run(x, W, bias=None, out=None, *, out_f32=False, flags=0, plan_: Plan | None = None, workspace=None,
        stream=None):
    """The general entry point (bf16_linear_run): optional explicit plan and workspace tensor."""
    import torch
    M, N, K, out = _check(x, W, bias, out, out_dtype=torch.float32 if out_f32 else torch.bfloat16)
    c = Call()
    c.x, c.W, c.bias, c.out = x.data_ptr(), W.data_ptr(), (bias.data_ptr() if bias is not None else None), \
        out.data_ptr()
    c.M, c.N, c.K = M, N, K
    c.out_f32 = 1 if out_f32 else 0
    c.flags = int(flags)
    c.plan = ctypes.pointer(plan_) if plan_ is not None else None
    if workspace is not None:
        if not workspace.is_cuda or workspace.device != x.device or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous CUDA tensor on the inputs' device")
        c.workspace = workspace.data_ptr()
        c.workspace_bytes = workspace.numel() * workspace.element_size()
    with torch.cuda.device(x.device):
        c.stream = _stream_handle(stream, x.device).value
        st = load().bf16_linear_run(ctypes.byref(c))
    if st != OK:
        _raise(st, f"bf16_linear_run(M={M}, N={N}, K={K}, plan={plan_})")
    return out


def bf16_linear_with_plan(x, W, bias=None, out=None, plan_: Plan | None = None, stream=None, workspace=None):
    """Run exactly `plan_` (no fallback: an unusable plan raises)."""
    if plan_ is None:
        raise ValueError("plan_ is required")
    return run(x, W, bias, out, plan_=plan_, workspace=workspace, stream=stream)


def new_workspace(nbytes: int, device=None):
    """A zero-filled workspace tensor of at least nbytes (256-byte aligned by the caching allocator)."""
    import torch
    return torch.zeros(max(256, int(nbytes)), dtype=torch.uint8, device=device or "cuda")


def bf16_linear_f32out(x, W, bias=None, out=None, stream=None, flags: int = 0, plan_: Plan | None = None):
    """fp32 out[M,N] = x @ W^T (+ bias): the router-logits variant (no rounding to bf16)."""
    import torch
    M, N, K, out = _check(x, W, bias, out, out_dtype=torch.float32)
    with torch.cuda.device(x.device):
        if plan_ is None:
            st = load().bf16_linear_f32out(_ptr(x), _ptr(W), _ptr(bias), _ptr(out), M, N, K, int(flags),
                                           _stream_handle(stream, x.device))
        else:
            st = load().bf16_linear_f32out_with_plan(_ptr(x), _ptr(W), _ptr(bias), _ptr(out), M, N, K,
                                                     ctypes.byref(plan_), _stream_handle(stream, x.device))
    if st != OK:
        _raise(st, f"bf16_linear_f32out(M={M}, N={N}, K={K})")
    return out


def bf16_linear_ex(x, W, bias=None, out=None, flags: int = 0, stream=None):
    """bf16_linear with BF16L_FLAG_* launch flags (1 = programmatic dependent launch)."""
    import torch
    M, N, K, out = _check(x, W, bias, out)
    with torch.cuda.device(x.device):
        st = load().bf16_linear_ex(_ptr(x), _ptr(W), _ptr(bias), _ptr(out), M, N, K, int(flags),
                                   _stream_handle(stream, x.device))
    if st != OK:
        _raise(st, f"bf16_linear_ex(M={M}, N={N}, K={K})")
    return out


def bf16_linear_noalloc(x, W, bias=None, out=None, stream=None):
    """bf16 out = x @ W^T (+ bias) for callers that cannot allocate device memory.

    Runs the workspace split-K kernel with its scratch in the library's fixed
    device array (see bf16_linear.h); the library allocates nothing.  Pass
    `out` to avoid the allocation this wrapper would otherwise make for it.
    Calls share the array: keep them on one stream.
    """
    import torch
    M, N, K, out = _check(x, W, bias, out)
    with torch.cuda.device(x.device):
        st = load().bf16_linear_noalloc(_ptr(x), _ptr(W), _ptr(bias), _ptr(out), M, N, K,
                                        _stream_handle(stream, x.device))
    if st != OK:
        _raise(st, f"bf16_linear_noalloc(M={M}, N={N}, K={K})")
    return out


def quant_fp8(x, scale, out=None, flags: int = 0, stream=None):
    """Static per-tensor quantisation (bf16_quant_fp8): bf16 x -> e4m3 codes (torch.uint8, same shape).

    `scale` is a one-element fp32 CUDA tensor (read on the device)."""
    import torch
    if x.dtype != torch.bfloat16:
        raise TypeError(f"x must be torch.bfloat16 (got {x.dtype})")
    if scale.dtype != torch.float32 or scale.numel() != 1 or not scale.is_cuda:
        raise ValueError("scale must be a one-element float32 CUDA tensor")
    if not x.is_cuda or not x.is_contiguous():
        raise ValueError("x must be a contiguous CUDA tensor")
    if out is None:
        out = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    elif out.dtype != torch.uint8 or out.shape != x.shape or not out.is_contiguous():
        raise ValueError("out must be a contiguous uint8 tensor shaped like x")
    with torch.cuda.device(x.device):
        st = load().bf16_quant_fp8(_ptr(x), _ptr(scale), _ptr(out), x.numel(), int(flags),
                                   _stream_handle(stream, x.device))
    if st != OK:
        _raise(st, f"bf16_quant_fp8(n={x.numel()})")
    return out


def bf16_linear_fp8(xq, wq, scale_x, scale_w, bias=None, out=None, flags: int = 0, stream=None,
                    plan_: Plan | None = None):
    """Per-tensor FP8 linear (bf16_linear_fp8): e4m3 codes xq[M,K], wq[N,K] (torch.uint8),
    one-element fp32 CUDA scale tensors, optional bf16 bias[N]; bf16 out[M,N]."""
    import torch
    for name, t in (("xq", xq), ("wq", wq)):
        if t.dtype != torch.uint8 or t.dim() != 2 or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous 2-D uint8 (e4m3 code) CUDA tensor")
    for name, t in (("scale_x", scale_x), ("scale_w", scale_w)):
        if t.dtype != torch.float32 or t.numel() != 1 or not t.is_cuda:
            raise ValueError(f"{name} must be a one-element float32 CUDA tensor")
    M, K = xq.shape
    N = wq.shape[0]
    if wq.shape[1] != K:
        raise ValueError(f"need xq[M,K] and wq[N,K], got {tuple(xq.shape)} and {tuple(wq.shape)}")
    if bias is not None and (bias.dtype != torch.bfloat16 or tuple(bias.shape) != (N,) or not bias.is_cuda):
        raise ValueError(f"bias must be a bf16 CUDA tensor of shape ({N},)")
    if out is None:
        out = torch.empty(M, N, dtype=torch.bfloat16, device=xq.device)
    with torch.cuda.device(xq.device):
        if plan_ is None:
            st = load().bf16_linear_fp8(_ptr(xq), _ptr(wq), _ptr(scale_x), _ptr(scale_w), _ptr(bias), _ptr(out),
                                        M, N, K, int(flags), _stream_handle(stream, xq.device))
        else:
            st = load().bf16_linear_fp8_with_plan(_ptr(xq), _ptr(wq), _ptr(scale_x), _ptr(scale_w), _ptr(bias),
                                                  _ptr(out), M, N, K, ctypes.byref(plan_),
                                                  _stream_handle(stream, xq.device))
    if st != OK:
        _raise(st, f"bf16_linear_fp8(M={M}, N={N}, K={K})")
    return out


def quant_mxfp8(x, out=None, scales=None, flags: int = 0, stream=None):
    """MXFP8 quantisation (bf16_quant_mxfp8) of a contiguous bf16 CUDA tensor x[rows, K], K % 32 == 0:
    returns (codes uint8 [rows, K], scales uint8 [rows, K / 32])."""
    import torch
    if x.dtype != torch.bfloat16 or x.dim() != 2 or not x.is_cuda or not x.is_contiguous():
        raise ValueError("x must be a contiguous 2-D bf16 CUDA tensor")
    rows, K = x.shape
    if out is None:
        out = torch.empty((rows, K), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty((rows, max(1, K // 32)), dtype=torch.uint8, device=x.device)
    with torch.cuda.device(x.device):
        st = load().bf16_quant_mxfp8(_ptr(x), rows, K, _ptr(out), _ptr(scales), int(flags),
                                     _stream_handle(stream, x.device))
    if st != OK:
        _raise(st, f"bf16_quant_mxfp8(rows={rows}, K={K})")
    return out, scales


def bf16_linear_mxfp8(xq, xs, wq, ws, bias=None, out=None, flags: int = 0, stream=None, plan_: Plan | None = None):
    """MXFP8 linear (bf16_linear_mxfp8): e4m3 codes xq[M,K], wq[N,K] (uint8) with E8M0 block scales
    xs[M,K/32], ws[N,K/32] (uint8), optional bf16 bias[N]; bf16 out[M,N]."""
    import torch
    for name, t in (("xq", xq), ("wq", wq), ("xs", xs), ("ws", ws)):
        if t.dtype != torch.uint8 or t.dim() != 2 or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous 2-D uint8 CUDA tensor")
    M, K = xq.shape
    N = wq.shape[0]
    if wq.shape[1] != K or tuple(xs.shape) != (M, K // 32) or tuple(ws.shape) != (N, K // 32):
        raise ValueError(f"shapes xq{tuple(xq.shape)} xs{tuple(xs.shape)} wq{tuple(wq.shape)} ws{tuple(ws.shape)}")
    if bias is not None and (bias.dtype != torch.bfloat16 or tuple(bias.shape) != (N,) or not bias.is_cuda):
        raise ValueError(f"bias must be a bf16 CUDA tensor of shape ({N},)")
    if out is None:
        out = torch.empty(M, N, dtype=torch.bfloat16, device=xq.device)
    with torch.cuda.device(xq.device):
        h = _stream_handle(stream, xq.device)
        if plan_ is None:
            st = load().bf16_linear_mxfp8(_ptr(xq), _ptr(xs), _ptr(wq), _ptr(ws), _ptr(bias), _ptr(out), M, N, K,
                                          int(flags), h)
        else:
            st = load().bf16_linear_mxfp8_with_plan(_ptr(xq), _ptr(xs), _ptr(wq), _ptr(ws), _ptr(bias), _ptr(out),
                                                    M, N, K, ctypes.byref(plan_), h)
    if st != OK:
        _raise(st, f"bf16_linear_mxfp8(M={M}, N={N}, K={K})")
    return out


def mxfp8_split(M: int, N: int, K: int, threads: int = 128, num_sms: int = 152) -> int:
    """The K split bf16_linear_mxfp8 uses (host logic, no GPU)."""
    return int(load().bf16_linear_mxfp8_split(M, N, K, threads, num_sms))


def fp8_split(M: int, N: int, K: int, num_sms: int = 152) -> int:
    """The K split bf16_linear_fp8 uses for a shape (host logic, no GPU)."""
    return int(load().bf16_linear_fp8_split(M, N, K, num_sms))


def _call(fn, device, stream, *args) -> int:
    """fn(*args, stream) with `device` current (entering a device context costs more than the call)."""
    import torch
    i = device.index
    if torch._C._cuda_getDevice() == i:
        # the raw handle: building a torch.cuda.Stream for it takes as long as the launch
        return fn(*args, torch._C._cuda_getCurrentRawStream(i) if stream is None else stream.cuda_stream)
    with torch.cuda.device(device):
        return fn(*args, torch._C._cuda_getCurrentRawStream(i) if stream is None else stream.cuda_stream)


def _empty(shape, dtype, device, stream):
    """A tensor that work on `stream` (None: the current one) may write at once: it comes from that stream's own memory,
    so nothing that the current stream still has to read or write can share it."""
    import torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _need(t, name, dtype, shape, device):
    """The address of t, a contiguous CUDA tensor of this dtype and shape on `device`."""
    if t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
        return t.data_ptr()
    raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}, got {t.dtype} "
                     f"{tuple(t.shape)} on {t.device}, strides {t.stride()}")


def _cuda(t, name):
    """t's device, a CUDA one."""
    if not t.is_cuda or t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D CUDA tensor, got {tuple(t.shape)} on {t.device}")
    return t.device


def _pitch(t, name):
    """Elements between the rows of a 2-D tensor whose rows are contiguous."""
    rows, cols = t.shape
    ld, step = t.stride()
    if (step != 1 and cols > 1) or (ld < cols and rows > 1):
        raise ValueError(f"{name}'s rows must be contiguous and apart, got strides {t.stride()}")
    return ld if ld > cols else cols


def _ints(*sizes) -> bool:
    """Whether the C ABI's ints hold these sizes (ctypes would pass their low 32 bits)."""
    return all(-(1 << 31) <= v < 1 << 31 for v in sizes)


def _fits(what, flags, *sizes):
    """Refuse what the C ABI's 32 bits do not hold (ctypes would pass the low ones)."""
    if not 0 <= flags < 1 << 32 or not _ints(*sizes):
        _raise(EINVAL, f"{what}: sizes {sizes}, flags {flags}")


QUANT_FORMATS = {None: 0, "fp8": 1, "mxfp8": 2, "mxfp4": 3}


class Norm(NamedTuple):
    """What rmsnorm gives: the norm in bf16, x + residual, and the codes and scales of the asked format (or None)."""
    out: object
    residual: object
    codes: object
    scales: object


def rmsnorm(x, weight, residual=None, eps: float = 1e-6, *, quant: str | None = None, scale=None, bf16_out: bool = True,
            out=None, residual_out=None, codes=None, scales=None, flags: int = 0, stream=None) -> Norm:
    """Root-mean-square norm of the rows of x[rows, H] (bf16_rmsnorm): h = x, or the bf16 sum x + residual[rows, H];
    y = h / sqrt(mean(h^2) + eps) * weight[H] in fp32.  Gives y in bf16 (left out with bf16_out=False), h where there is a
    residual, and y's codes in `quant`: "fp8" (e4m3 with the one-element fp32 CUDA tensor `scale`), "mxfp8" or "mxfp4"
    (uint8 codes [rows, H] or [rows, H / 2], uint8 E8M0 scales [rows, H / 32]).  All bf16; x may be a column range of a
    wider matrix.  residual_out may be residual itself (in place)."""
    if out is residual_out is codes is scales is stream is None and _calls is not None and quant in QUANT_FORMATS:
        r = _calls.rmsnorm(x, weight, residual, eps, QUANT_FORMATS[quant], scale, bf16_out, flags)
        if type(r) is tuple:
            return tuple.__new__(Norm, r)
        if r is not None:
            _raise(r, f"bf16_rmsnorm(x{tuple(x.shape)}, quant={quant})")
    import torch
    bf16, u8 = torch.bfloat16, torch.uint8
    if x.dtype is not bf16:
        raise TypeError(f"x must be torch.bfloat16 (got {x.dtype})")
    if quant not in QUANT_FORMATS:
        raise ValueError(f"quant must be one of {list(QUANT_FORMATS)}, got {quant!r}")
    dev, shape, ld = _cuda(x, "x"), x.shape, _pitch(x, "x")
    rows, H = shape
    _fits("bf16_rmsnorm", flags, H)
    w = _need(weight, "weight", bf16, (H,), dev)
    r = ro = o = c = sc = s1 = None
    if residual is not None:
        r = _need(residual, "residual", bf16, shape, dev)
        if residual_out is None:
            residual_out = _empty(shape, bf16, dev, stream)
            ro = residual_out.data_ptr()
        else:
            ro = _need(residual_out, "residual_out", bf16, shape, dev)
    elif residual_out is not None:
        raise ValueError("residual_out without a residual")
    if not bf16_out:
        if out is not None or quant is None:
            raise ValueError("bf16_out=False needs a quant format and no out")
    elif out is None:
        out = _empty(shape, bf16, dev, stream)
        o = out.data_ptr()
    else:
        o = _need(out, "out", bf16, shape, dev)
    if quant is None:
        if codes is not None or scales is not None or scale is not None:
            raise ValueError("codes, scales and scale need a quant format")
    else:
        packed = (rows, H // 2 if quant == "mxfp4" else H)
        if codes is None:
            codes = _empty(packed, u8, dev, stream)
        c = _need(codes, "codes", u8, packed, dev)
        if quant == "fp8":
            if scale is None or scales is not None:
                raise ValueError("quant='fp8' takes the one-element `scale` and no `scales`")
            s1 = _need(scale.reshape(-1), "scale", torch.float32, (1,), dev)
        else:
            if scale is not None:
                raise ValueError("scale is for quant='fp8'")
            if scales is None:
                scales = _empty((rows, H // 32), u8, dev, stream)
            sc = _need(scales, "scales", u8, (rows, H // 32), dev)
    st = _call(load().bf16_rmsnorm, dev, stream, x.data_ptr(), ld, r, w, o, ro, c, sc, s1, rows, H, eps,
               QUANT_FORMATS[quant], flags)
    if st != OK:
        _raise(st, f"bf16_rmsnorm(rows={rows}, H={H}, quant={quant})")
    return Norm(out, residual_out, codes, scales)


SCORES = {"softmax": 0, "sigmoid": 1}


def route(logits, k: int, *, scoring: str = "softmax", bias=None, groups: int = 1, top_groups: int = 1,
          group_best: int = 1, renormalize: bool = True, scale: float = 1.0, weights=None, ids=None, flags: int = 0,
          stream=None):
    """The k experts of each token from the router's logits[tokens, experts], fp32 or bf16 (bf16_route): (weights fp32
    [tokens, k], ids int32 [tokens, k]), the best first.  scoring "softmax" or "sigmoid"; bias[experts] (fp32) is added to
    the scores for the choice alone; with groups > 1 only the experts of the top_groups best of `groups` equal runs of
    experts stay, a group ranked by the sum of its group_best largest.  renormalize divides the weights by their sum; scale
    multiplies them.  Experts with a logit of -inf are out."""
    if weights is ids is stream is None and _calls is not None and scoring in SCORES:
        r = _calls.route(logits, k, SCORES[scoring], bias, groups, top_groups, group_best, renormalize, scale, flags)
        if type(r) is tuple:
            return r
        if r is not None:
            _raise(r, f"bf16_route(logits{tuple(logits.shape)}, k={k}, groups={groups}, top_groups={top_groups})")
    import torch
    f32, dt = torch.float32, logits.dtype
    if dt is not f32 and dt is not torch.bfloat16:
        raise TypeError(f"logits must be float32 or bfloat16 (got {dt})")
    if scoring not in SCORES:
        raise ValueError(f"scoring must be one of {list(SCORES)}, got {scoring!r}")
    dev, (T, E), ld = _cuda(logits, "logits"), logits.shape, _pitch(logits, "logits")
    _fits("bf16_route", flags, E, k, groups, top_groups, group_best)
    b = None if bias is None else _need(bias, "bias", f32, (E,), dev)
    if weights is None:
        weights = _empty((T, k if k > 0 else 0), f32, dev, stream)
    if ids is None:
        ids = _empty((T, k if k > 0 else 0), torch.int32, dev, stream)
    st = _call(load().bf16_route, dev, stream, logits.data_ptr(), ld, b, _need(weights, "weights", f32, (T, k), dev),
               _need(ids, "ids", torch.int32, (T, k), dev), T, E, k, SCORES[scoring], groups, top_groups, group_best,
               renormalize, scale, dt is not f32, flags) if k > 0 else EINVAL
    if st != OK:
        _raise(st, f"bf16_route(tokens={T}, experts={E}, k={k}, groups={groups}, top_groups={top_groups})")
    return weights, ids


def quant_mxfp4(x, out=None, scales=None, flags: int = 0, stream=None):
    """MXFP4 quantisation (bf16_quant_mxfp4) of a contiguous bf16 CUDA tensor x[rows, K], K % 32 == 0: returns (codes uint8
    [rows, K / 2], two to a byte, scales uint8 [rows, K / 32])."""
    if out is scales is stream is None and _calls is not None:
        r = _calls.quant_mxfp4(x, flags)
        if type(r) is tuple:
            return r
        if r is not None:
            _raise(r, f"bf16_quant_mxfp4(x{tuple(x.shape)})")
    import torch
    dev, u8 = _cuda(x, "x"), torch.uint8
    rows, K = x.shape
    p = _need(x, "x", torch.bfloat16, (rows, K), dev)
    _fits("bf16_quant_mxfp4", flags, K)
    if out is None:
        out = _empty((rows, K // 2), u8, dev, stream)
    if scales is None:
        scales = _empty((rows, K // 32), u8, dev, stream)
    st = _call(load().bf16_quant_mxfp4, dev, stream, p, rows, K, _need(out, "out", u8, (rows, K // 2), dev),
               _need(scales, "scales", u8, (rows, K // 32), dev), flags)
    if st != OK:
        _raise(st, f"bf16_quant_mxfp4(rows={rows}, K={K})")
    return out, scales


def dequant_mxfp4(codes, scales, out=None, flags: int = 0, stream=None):
    """The bf16 values [rows, K] that MXFP4 codes [rows, K / 2] and scales [rows, K / 32] stand for (bf16_dequant_mxfp4)."""
    if out is stream is None and _calls is not None:
        r = _calls.dequant_mxfp4(codes, scales, flags)
        if type(r) is int:
            _raise(r, f"bf16_dequant_mxfp4(codes{tuple(codes.shape)})")
        if r is not None:
            return r
    import torch
    dev, u8 = _cuda(codes, "codes"), torch.uint8
    rows, h = codes.shape
    q, s = _need(codes, "codes", u8, (rows, h), dev), _need(scales, "scales", u8, (rows, h // 16), dev)
    _fits("bf16_dequant_mxfp4", flags, 2 * h)
    if out is None:
        out = _empty((rows, 2 * h), torch.bfloat16, dev, stream)
    st = _call(load().bf16_dequant_mxfp4, dev, stream, q, s, rows, 2 * h,
               _need(out, "out", torch.bfloat16, (rows, 2 * h), dev), flags)
    if st != OK:
        _raise(st, f"bf16_dequant_mxfp4(rows={rows}, K={2 * h})")
    return out


def bf16_linear_mxfp4(xq, xs, wq, ws, bias=None, out=None, flags: int = 0, stream=None):
    """MXFP4 linear (bf16_linear_mxfp4): packed e2m1 codes xq[M, K / 2], wq[N, K / 2] with E8M0 block scales xs[M, K / 32],
    ws[N, K / 32] (all uint8), optional bf16 bias[N]; bf16 out[M, N]."""
    if out is stream is None and _calls is not None and xs is not None:
        r = _calls.linear_mxfp4(xq, xs, wq, ws, bias, flags)
        if type(r) is int:
            _raise(r, f"bf16_linear_mxfp4(xq{tuple(xq.shape)}, wq{tuple(wq.shape)})")
        if r is not None:
            return r
    import torch
    dev, u8, bf16 = _cuda(xq, "xq"), torch.uint8, torch.bfloat16
    (M, h), N = xq.shape, wq.shape[0]
    a, b = _need(xq, "xq", u8, (M, h), dev), _need(xs, "xs", u8, (M, h // 16), dev)
    c, d = _need(wq, "wq", u8, (N, h), dev), _need(ws, "ws", u8, (N, h // 16), dev)
    _fits("bf16_linear_mxfp4", flags, M, N, 2 * h)
    e = None if bias is None else _need(bias, "bias", bf16, (N,), dev)
    if out is None:
        out = _empty((M, N), bf16, dev, stream)
    st = _call(load().bf16_linear_mxfp4, dev, stream, a, b, c, d, e, _need(out, "out", bf16, (M, N), dev), M, N, 2 * h, flags)
    if st != OK:
        _raise(st, f"bf16_linear_mxfp4(M={M}, N={N}, K={2 * h})")
    return out


def mxfp4_dynamic_workspace(M: int, N: int, K: int) -> int:
    """Workspace bytes of bf16_linear_mxfp4_dynamic (0 where the product quantises x itself, and for sizes that it refuses)."""
    return int(load().bf16_linear_mxfp4_dynamic_workspace(M, N, K)) if _ints(M, N, K) else 0


def bf16_linear_mxfp4_dynamic(x, wq, ws, bias=None, out=None, workspace=None, flags: int = 0, stream=None):
    """MXFP4 linear with x[M, K] in bf16, quantised by the call (bf16_linear_mxfp4_dynamic): bit for bit quant_mxfp4 and
    then bf16_linear_mxfp4.  `workspace`: a contiguous CUDA tensor of at least mxfp4_dynamic_workspace(M, N, K) bytes to
    reuse from call to call on one stream; allocated for the call when None."""
    if out is workspace is stream is None and _calls is not None:
        r = _calls.linear_mxfp4(x, None, wq, ws, bias, flags)
        if type(r) is int:
            _raise(r, f"bf16_linear_mxfp4_dynamic(x{tuple(x.shape)}, wq{tuple(wq.shape)})")
        if r is not None:
            return r
    import torch
    dev, u8, bf16 = _cuda(x, "x"), torch.uint8, torch.bfloat16
    (M, K), N = x.shape, wq.shape[0]
    a = _need(x, "x", bf16, (M, K), dev)
    c, d = _need(wq, "wq", u8, (N, K // 2), dev), _need(ws, "ws", u8, (N, K // 32), dev)
    _fits("bf16_linear_mxfp4_dynamic", flags, M, N, K)
    e = None if bias is None else _need(bias, "bias", bf16, (N,), dev)
    if out is None:
        out = _empty((M, N), bf16, dev, stream)
    lib = load()
    wp, wn = None, 0
    if workspace is None:
        wn = lib.bf16_linear_mxfp4_dynamic_workspace(M, N, K)
        if wn:
            workspace = _empty((wn,), u8, dev, stream)
            wp = workspace.data_ptr()
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor on x's device")
    else:
        wp, wn = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    st = _call(lib.bf16_linear_mxfp4_dynamic, dev, stream, a, c, d, e, _need(out, "out", bf16, (M, N), dev), M, N, K, wp, wn,
               flags)
    if st != OK:
        _raise(st, f"bf16_linear_mxfp4_dynamic(M={M}, N={N}, K={K})")
    return out


class Groups(NamedTuple):
    """What group_rows gives: the groups' first positions, the token of each position, and each pair's position."""
    offsets: object
    rows: object
    place: object


def group_rows(ids, groups: int, *, offsets=None, rows=None, place=None, flags: int = 0, stream=None) -> Groups:
    """The pairs of ids[tokens, k] or ids[tokens] (int32) ordered by id, equal ids in their own order (bf16_group_rows):
    offsets int32 [groups + 1], where each group's positions start; rows int32 [tokens * k], the token of each position, -1
    past offsets[groups]; place int32 like ids, each pair's position, -1 for an id outside 0 .. groups - 1, which is left
    out.  Outputs that the call makes may lie in one allocation."""
    if offsets is rows is place is stream is None and _calls is not None:
        r = _calls.group_rows(ids, groups, flags)
        if type(r) is tuple:
            return tuple.__new__(Groups, r)
        if r is not None:
            _raise(r, f"bf16_group_rows(ids{tuple(ids.shape)}, groups={groups})")
    import torch
    i32 = torch.int32
    if ids.dtype is not i32:
        raise TypeError(f"ids must be torch.int32 (got {ids.dtype})")
    if not ids.is_cuda or ids.dim() not in (1, 2):
        raise ValueError(f"ids must be a 1-D or 2-D CUDA tensor, got {tuple(ids.shape)} on {ids.device}")
    dev, shape = ids.device, ids.shape
    T, k = shape[0], shape[1] if len(shape) == 2 else 1
    p = _need(ids, "ids", i32, shape, dev)
    _fits("bf16_group_rows", flags, k, groups)
    if groups < 1:
        _raise(EINVAL, f"bf16_group_rows(ids{tuple(shape)}, groups={groups})")
    if offsets is None:
        offsets = _empty((groups + 1,), i32, dev, stream)
    if rows is None:
        rows = _empty((T * k,), i32, dev, stream)
    if place is None:
        place = _empty(shape, i32, dev, stream)
    st = _call(load().bf16_group_rows, dev, stream, p, T, k, groups, _need(offsets, "offsets", i32, (groups + 1,), dev),
               _need(rows, "rows", i32, (T * k,), dev), _need(place, "place", i32, shape, dev), flags)
    if st != OK:
        _raise(st, f"bf16_group_rows(ids{tuple(shape)}, groups={groups})")
    return Groups(offsets, rows, place)


def grouped_workspace(P: int, groups: int, N: int, K: int, swiglu: bool = False) -> int:
    """Workspace bytes of bf16_linear_grouped for P rows of out (0 where it needs none, and for sizes that it refuses)."""
    return int(load().bf16_linear_grouped_workspace(P, groups, N, K, bool(swiglu))) if _ints(P, groups, N, K) else 0


def bf16_linear_grouped(x, w, offsets, bias=None, *, rows=None, swiglu: bool = False, out=None, workspace=None, flags: int = 0,
                        stream=None):
    """A linear for each group's rows (bf16_linear_grouped): out[p] = x[p] @ w[e]^T (+ bias[e]) for the positions p from
    offsets[e] to offsets[e + 1], x[rows[p]] where rows (int32) is given.  x[x_rows, K], w[groups, N, K], bias[groups, N] bf16,
    offsets int32 [groups + 1]; out bf16 [len(rows) or x_rows, N], in which rows of no group are not written.  swiglu: w and
    bias hold N gate rows and N up rows a group, out = silu(gate) * up.  `workspace`: a contiguous CUDA tensor of at least
    grouped_workspace(rows of out, groups, N, K, swiglu) bytes to reuse from call to call on one stream; allocated for the
    call when None."""
    if out is workspace is stream is None and _calls is not None:
        r = _calls.linear_grouped(x, w, offsets, bias, rows, swiglu, flags)
        if type(r) is int:
            _raise(r, f"bf16_linear_grouped(x{tuple(x.shape)}, w{tuple(w.shape)}, swiglu={bool(swiglu)})")
        if r is not None:
            return r
    import torch
    bf16, i32 = torch.bfloat16, torch.int32
    if x.dtype is not bf16 or w.dtype is not bf16:
        raise TypeError(f"x and w must be torch.bfloat16 (got {x.dtype}, {w.dtype})")
    dev, (xr, K) = _cuda(x, "x"), x.shape
    if w.dim() != 3 or (swiglu and w.shape[1] % 2):
        raise ValueError(f"w must be [groups, N, K], with swiglu [groups, 2 N, K], got {tuple(w.shape)}")
    G, W = w.shape[:2]
    P, N = xr if rows is None else rows.numel(), W // 2 if swiglu else W
    a, b = _need(x, "x", bf16, (xr, K), dev), _need(w, "w", bf16, (G, W, K), dev)
    c = _need(offsets, "offsets", i32, (G + 1,), dev)
    d = None if rows is None else _need(rows, "rows", i32, (P,), dev)
    e = None if bias is None else _need(bias, "bias", bf16, (G, W), dev)
    _fits("bf16_linear_grouped", flags, G, W, K)
    if out is None:
        out = _empty((P, N), bf16, dev, stream)
    lib = load()
    wp, wn = None, 0
    if workspace is None:
        wn = lib.bf16_linear_grouped_workspace(P, G, N, K, bool(swiglu))
        if wn:
            workspace = _empty((wn,), torch.uint8, dev, stream)
            wp = workspace.data_ptr()
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor on x's device")
    else:
        wp, wn = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    st = _call(lib.bf16_linear_grouped, dev, stream, a, xr, b, e, c, d, _need(out, "out", bf16, (P, N), dev), P, G, N, K,
               bool(swiglu), wp, wn, flags)
    if st != OK:
        _raise(st, f"bf16_linear_grouped(x{tuple(x.shape)}, w{tuple(w.shape)}, swiglu={bool(swiglu)})")
    return out


def combine_rows(y, place, weights=None, addend=None, *, out=None, flags: int = 0, stream=None):
    """out[t] = sum over j of weights[t, j] * y[place[t, j]] (+ addend[t]) in bf16, summed in fp32 (bf16_combine_rows).
    y[y_rows, H] and addend[tokens, H] bf16, place[tokens, k] int32, weights[tokens, k] fp32 (None: all 1).  A place outside y
    adds nothing.  out may be addend itself (in place)."""
    if out is stream is None and _calls is not None:
        r = _calls.combine_rows(y, place, weights, addend, flags)
        if type(r) is int:
            _raise(r, f"bf16_combine_rows(y{tuple(y.shape)}, place{tuple(place.shape)})")
        if r is not None:
            return r
    import torch
    bf16 = torch.bfloat16
    dev, (yr, H) = _cuda(y, "y"), y.shape
    if place.dim() != 2:
        raise ValueError(f"place must be [tokens, k], got {tuple(place.shape)}")
    T, k = place.shape
    a, b = _need(y, "y", bf16, (yr, H), dev), _need(place, "place", torch.int32, (T, k), dev)
    c = None if weights is None else _need(weights, "weights", torch.float32, (T, k), dev)
    d = None if addend is None else _need(addend, "addend", bf16, (T, H), dev)
    _fits("bf16_combine_rows", flags, k, H)
    if out is None:
        out = _empty((T, H), bf16, dev, stream)
    st = _call(load().bf16_combine_rows, dev, stream, a, yr, b, c, d, _need(out, "out", bf16, (T, H), dev), T, k, H, flags)
    if st != OK:
        _raise(st, f"bf16_combine_rows(y{tuple(y.shape)}, place{tuple(place.shape)})")
    return out


def lora_workspace(M: int, N: int, K: int, R: int, L: int) -> int:
    """Workspace bytes of bf16_linear_lora (0 for sizes that it refuses)."""
    return int(load().bf16_linear_lora_workspace(M, N, K, R, L)) if _ints(M, N, K, R, L) else 0


def bf16_linear_lora(x, w, a, b, ids, bias=None, *, scale=None, out=None, workspace=None, flags: int = 0, stream=None):
    """A linear with a low-rank adapter for each row (bf16_linear_lora): out[t] = x[t] @ w^T (+ bias) +
    scale[id] * (x[t] @ a[id]^T) @ b[id]^T, id = ids[t]; rows whose id lies outside 0 .. L - 1 have none.  x[M, K], w[N, K],
    a[L, R, K], b[L, N, R], bias[N] bf16, ids[M] int32, scale[L] fp32 (None: 1).  `workspace`: a contiguous CUDA tensor of at
    least lora_workspace(M, N, K, R, L) bytes to reuse from call to call on one stream; allocated for the call when None."""
    if out is workspace is stream is None and _calls is not None:
        r = _calls.linear_lora(x, w, a, b, ids, bias, scale, flags)
        if type(r) is int:
            _raise(r, f"bf16_linear_lora(x{tuple(x.shape)}, w{tuple(w.shape)}, a{tuple(a.shape)})")
        if r is not None:
            return r
    import torch
    bf16 = torch.bfloat16
    if x.dtype is not bf16 or w.dtype is not bf16:
        raise TypeError(f"x and w must be torch.bfloat16 (got {x.dtype}, {w.dtype})")
    dev, (M, K) = _cuda(x, "x"), x.shape
    if w.dim() != 2 or a.dim() != 3:
        raise ValueError(f"need w[N, K] and a[L, R, K], got {tuple(w.shape)} and {tuple(a.shape)}")
    N, (L, R) = w.shape[0], a.shape[:2]
    args = [_need(x, "x", bf16, (M, K), dev), _need(w, "w", bf16, (N, K), dev),
            None if bias is None else _need(bias, "bias", bf16, (N,), dev), _need(a, "a", bf16, (L, R, K), dev),
            _need(b, "b", bf16, (L, N, R), dev), None if scale is None else _need(scale, "scale", torch.float32, (L,), dev),
            _need(ids, "ids", torch.int32, (M,), dev)]
    _fits("bf16_linear_lora", flags, M, N, K, R, L)
    if out is None:
        out = _empty((M, N), bf16, dev, stream)
    lib = load()
    wp, wn = None, 0
    if workspace is None:
        wn = lib.bf16_linear_lora_workspace(M, N, K, R, L)
        if wn:
            workspace = _empty((wn,), torch.uint8, dev, stream)
            wp = workspace.data_ptr()
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor on x's device")
    else:
        wp, wn = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    st = _call(lib.bf16_linear_lora, dev, stream, *args, _need(out, "out", bf16, (M, N), dev), M, N, K, R, L, wp, wn, flags)
    if st != OK:
        _raise(st, f"bf16_linear_lora(M={M}, N={N}, K={K}, R={R}, L={L})")
    return out


def probe_read(src, grid: int, threads: int, sink, nbytes: int | None = None, stream=None, flags: int = 0):
    """Launch the read-floor probe (bf16_linear_probe_read) over the bytes of the CUDA tensor `src`
    (the first nbytes of them, or none when src is None); CTA b XORs its checksum into sink[b] of the
    int32 CUDA tensor `sink` (at least `grid` elements).  flags: 0 (the library's launch mode) or
    FLAG_SERIAL."""
    import torch
    if sink is not None and sink.numel() < grid:
        raise ValueError(f"sink needs {grid} elements, has {sink.numel()}")
    nb = 0 if src is None else (src.numel() * src.element_size() if nbytes is None else int(nbytes))
    dev = sink.device if sink is not None else torch.device("cuda", torch.cuda.current_device())
    st = load().bf16_linear_probe_read(_ptr(src), nb, int(grid), int(threads), _ptr(sink), int(flags),
                                       _stream_handle(stream, dev))
    if st != OK:
        _raise(st, f"bf16_linear_probe_read(bytes={nb}, grid={grid}, threads={threads})")


def device_status(clear: bool = False) -> int:
    """The device's kernel status word (0 = no kernel wait gave up).  Synchronises."""
    v = ctypes.c_int32(0)
    st = load().bf16_linear_device_status(ctypes.byref(v), int(bool(clear)))
    if st != OK:
        _raise(st, "bf16_linear_device_status")
    return int(v.value)


def selftest_wait(limit_us: int, stream=None):
    """Launch the bounded-wait diagnostic (see bf16_linear.h)."""
    import torch
    st = load().bf16_linear_selftest_wait(int(limit_us), _stream_handle(stream, torch.cuda.current_device()))
    if st != OK:
        _raise(st, "bf16_linear_selftest_wait")


def version() -> int:
    return int(load().bf16_linear_version())
