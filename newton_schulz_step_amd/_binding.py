"""ctypes binding of libmuonstep (argument marshalling only).

Every step of the Muon step runs in the library's HIP kernels; this module only
turns torch tensors into device pointers and the current HIP stream, and turns
status codes into MuonError. It never computes a result itself, and it raises
if the library is missing.
"""
from __future__ import annotations

import ctypes
import functools
import operator
import os
import threading
from typing import Dict, Iterable, List, Optional, Sequence, Tuple

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmuonstep.so")

# status codes (include/muon_step.h)
OK, ERR_NULL, ERR_BAD_METHOD, ERR_BAD_SHAPE, ERR_RANGE, ERR_OVERLAP, ERR_ALIGN, \
    ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_HIP, ERR_BAD_HYPER = range(11)
STATUS_NAMES = {
    0: "MUON_OK", 1: "MUON_ERR_NULL", 2: "MUON_ERR_BAD_METHOD", 3: "MUON_ERR_BAD_SHAPE",
    4: "MUON_ERR_RANGE", 5: "MUON_ERR_OVERLAP", 6: "MUON_ERR_ALIGN", 7: "MUON_ERR_UNSUPPORTED",
    8: "MUON_ERR_WORKSPACE", 9: "MUON_ERR_HIP", 10: "MUON_ERR_BAD_HYPER",
}
DTYPES = {"f32": 0, "bf16": 1, "f16": 2}
NS_METHODS = {"standard": 0, "gram": 1}
FP8_FORMATS = {"e4m3": 0, "e5m2": 1}
FP8_BLOCK = 128                        # MUON_FP8_BLOCK
ROUTE_SCORES = {"softmax": 0, "sigmoid": 1}

EXPORTED = (
    "muon_default_hyper", "muon_default_adamw_hyper", "muon_workspace_size", "muon_step",
    "muon_step_window", "adamw_step", "muon_pack", "muon_unpack", "muon_last_error", "muon_release_plans",
    "muon_profile_begin", "muon_profile_end", "muon_version", "muon_ns_flops",
    "muon_plan_owners", "muon_comm_elements", "muon_step_noalloc",
    "muon_fp8_quantize", "muon_fp8_matmul", "muon_fp8_matmul_grouped_k",
    "muon_default_route_hyper", "muon_route", "muon_route_backward", "muon_expert_order",
    "muon_expert_order_workspace_size", "muon_combine", "muon_combine_backward",
)
NOALLOC_WORKSPACE_BYTES = 64 << 20     # MUON_NOALLOC_WORKSPACE_BYTES


class MuonError(RuntimeError):
    """A non-zero status from libmuonstep."""

    def __init__(self, status: int, message: str):
        self.status = status
        self.message = message
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")


class MuonMatrix(ctypes.Structure):
    _fields_ = [("offset", ctypes.c_int64), ("rows", ctypes.c_int64),
                ("cols", ctypes.c_int64), ("split_rows", ctypes.c_int64),
                ("split_cols", ctypes.c_int64)]


class MuonHyper(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("momentum", ctypes.c_float),
                ("weight_decay", ctypes.c_float), ("ns_a", ctypes.c_float),
                ("ns_b", ctypes.c_float), ("ns_c", ctypes.c_float),
                ("ns_steps", ctypes.c_int32), ("ns_eps", ctypes.c_float),
                ("ns_method", ctypes.c_int32), ("param_dtype", ctypes.c_int32),
                ("grad_dtype", ctypes.c_int32), ("ns_dtype", ctypes.c_int32)]


class MuonWindow(ctypes.Structure):
    _fields_ = [("lo", ctypes.c_int64), ("hi", ctypes.c_int64), ("param_offset", ctypes.c_int64)]


class MuonParam(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("split_rows", ctypes.c_int64),
                ("layer", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("split_cols", ctypes.c_int64)]


class MuonAssign(ctypes.Structure):
    _fields_ = [("owner", ctypes.c_int32), ("reserved", ctypes.c_int32), ("offset", ctypes.c_int64)]


class MuonOwner(ctypes.Structure):
    _fields_ = [("numel", ctypes.c_int64), ("max_layer_numel", ctypes.c_int64),
                ("ns_flops", ctypes.c_int64), ("n_matrices", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class AdamWHyper(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("beta1", ctypes.c_float), ("beta2", ctypes.c_float),
                ("eps", ctypes.c_float), ("weight_decay", ctypes.c_float),
                ("step", ctypes.c_int32), ("grad_dtype", ctypes.c_int32)]


class KernelStat(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 48), ("launches", ctypes.c_int32),
                ("total_ms", ctypes.c_double)]


class Fp8Operand(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("batch", ctypes.c_int64),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("format", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class Fp8Source(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("batch_stride", ctypes.c_int64), ("ld", ctypes.c_int64),
                ("batch", ctypes.c_int64), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("row_div", ctypes.c_int32), ("row_index", ctypes.c_void_p),
                ("out_rows", ctypes.c_int64), ("row_weight", ctypes.c_void_p), ("n_weights", ctypes.c_int64)]


class Fp8Result(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("batch_stride", ctypes.c_int64), ("ld", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("accumulate", ctypes.c_int32)]


class RouteHyper(ctypes.Structure):
    _fields_ = [("score", ctypes.c_int32), ("top_k", ctypes.c_int32), ("n_groups", ctypes.c_int32),
                ("top_groups", ctypes.c_int32), ("group_top", ctypes.c_int32),
                ("renormalize", ctypes.c_int32), ("scale", ctypes.c_float), ("reserved", ctypes.c_int32)]


_lib = None
_lock = threading.Lock()


def load() -> ctypes.CDLL:
    """Load the built library (raises if it has not been built).

    torch is imported first: torch ships its own HIP runtime under the same
    soname (libamdhip64.so.7) as the system one the library links against, and
    the first one loaded serves the whole process. Loaded in this order the
    library shares torch's runtime (and torch's tensors and streams); loaded
    the other way round, torch ran on the system runtime and the library's
    first HIP call failed."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing; build it with "
                              "`python -m newton_schulz_step_amd.build`")
        import torch  # noqa: F401  (see above)
        lib = ctypes.CDLL(LIB_PATH)
        vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        pm = ctypes.POINTER(MuonMatrix)
        lib.muon_default_hyper.argtypes = [ctypes.POINTER(MuonHyper)]
        lib.muon_default_hyper.restype = None
        lib.muon_default_adamw_hyper.argtypes = [ctypes.POINTER(AdamWHyper)]
        lib.muon_default_adamw_hyper.restype = None
        lib.muon_workspace_size.argtypes = [pm, i32, ctypes.POINTER(MuonHyper), ctypes.POINTER(sz)]
        lib.muon_step.argtypes = [vp, vp, vp, i64, pm, i32, ctypes.POINTER(MuonHyper), vp, sz,
                                  vp, vp, vp]
        lib.muon_step_noalloc.argtypes = [vp, vp, vp, i64, pm, i32, ctypes.POINTER(MuonHyper), vp, vp, vp]
        lib.muon_step_window.argtypes = [vp, i64, vp, vp, i64, pm, ctypes.POINTER(MuonWindow), i32,
                                         ctypes.POINTER(MuonHyper), vp, sz, vp, vp, vp]
        lib.adamw_step.argtypes = [vp, vp, vp, vp, i64, ctypes.POINTER(AdamWHyper), vp]
        lib.muon_pack.argtypes = [vp, i64, ctypes.POINTER(vp), pm, i32, i32, vp]
        lib.muon_unpack.argtypes = [ctypes.POINTER(vp), vp, i64, pm, i32, i32, vp]
        lib.muon_ns_flops.argtypes = [i64, i64, i32, i32]
        lib.muon_ns_flops.restype = i64
        lib.muon_plan_owners.argtypes = [ctypes.POINTER(MuonParam), i32, i32, i32, i32, i64,
                                         ctypes.POINTER(MuonAssign), ctypes.POINTER(MuonOwner)]
        lib.muon_comm_elements.argtypes = [i64, i32, i32, i32]
        lib.muon_comm_elements.restype = ctypes.c_double
        lib.muon_last_error.restype = ctypes.c_char_p
        lib.muon_version.restype = ctypes.c_char_p
        lib.muon_profile_end.argtypes = [ctypes.POINTER(KernelStat), i32, ctypes.POINTER(i32)]
        po, ps, pr = ctypes.POINTER(Fp8Operand), ctypes.POINTER(Fp8Source), ctypes.POINTER(Fp8Result)
        ph = ctypes.POINTER(RouteHyper)
        lib.muon_fp8_quantize.argtypes = [ps, i32, po, po, vp]
        lib.muon_fp8_matmul.argtypes = [po, po, vp, pr, vp]
        lib.muon_fp8_matmul_grouped_k.argtypes = [po, po, vp, i32, pr, vp]
        lib.muon_default_route_hyper.argtypes = [ph]
        lib.muon_default_route_hyper.restype = None
        lib.muon_route.argtypes = [vp, i32, i64, i32, i64, vp, ph, vp, vp, vp]
        lib.muon_route_backward.argtypes = [vp, vp, i32, i64, i32, i64, vp, ph, vp, i64, vp]
        lib.muon_expert_order.argtypes = [vp, i64, i32, i32, vp, vp, vp, i64, vp, vp, sz, vp]
        lib.muon_expert_order_workspace_size.argtypes = [i64, i32, ctypes.POINTER(sz)]
        lib.muon_combine.argtypes = [vp, i32, i64, i64, i64, vp, vp, i64, i32, vp, i64, vp]
        lib.muon_combine_backward.argtypes = [vp, i32, i64, i64, i64, vp, i64, i64, vp, vp, i32, vp, vp, i64, vp]
        for name in ("muon_fp8_quantize", "muon_fp8_matmul", "muon_fp8_matmul_grouped_k",
                     "muon_route", "muon_route_backward", "muon_expert_order",
                     "muon_expert_order_workspace_size", "muon_combine", "muon_combine_backward"):
            getattr(lib, name).restype = ctypes.c_int
        for name in ("muon_workspace_size", "muon_step", "muon_step_noalloc", "muon_step_window", "muon_plan_owners",
                     "adamw_step", "muon_pack", "muon_unpack",
                     "muon_release_plans", "muon_profile_begin", "muon_profile_end"):
            getattr(lib, name).restype = ctypes.c_int
        _lib = lib
        return lib


def _check(status: int) -> None:
    if status != OK:
        raise MuonError(status, load().muon_last_error().decode(errors="replace"))


def version() -> str:
    return load().muon_version().decode()


# ----------------------------------------------------------------------------- hyperparameters

def hyper(**kw) -> MuonHyper:
    """Muon-group hyperparameters: the library defaults, then keyword overrides.

    Accepts lr / muon_lr (muon_lr wins, as in the DeepSpeed config), momentum,
    weight_decay, ns_method ("standard" | "gram"), ns_steps, ns_eps, ns_a/b/c,
    grad_dtype and ns_dtype ("f32" | "bf16" | "f16"), param_dtype ("f32" | "bf16")."""
    h = MuonHyper()
    load().muon_default_hyper(ctypes.byref(h))
    kw = dict(kw)
    if "muon_lr" in kw:
        kw["lr"] = kw.pop("muon_lr")
    for k, v in kw.items():
        if k == "ns_method":
            v = NS_METHODS.get(v, v) if isinstance(v, str) else v
            if isinstance(v, str):
                v = -1
        elif k in ("grad_dtype", "ns_dtype", "param_dtype") and isinstance(v, str):
            v = DTYPES[v]
        if not hasattr(h, k):
            raise TypeError(f"unknown Muon hyperparameter {k!r}")
        setattr(h, k, v)
    return h


def table(entries: Iterable[Sequence[int]]):
    """ctypes array of muon_matrix_t from (offset, rows, cols[, split_rows[,
    split_cols]]) tuples."""
    rows = [tuple(e) + (0,) * (5 - len(e)) for e in entries]
    arr = (MuonMatrix * max(len(rows), 1))()
    for i, (o, r, c, s, sc) in enumerate(rows):
        arr[i] = MuonMatrix(o, r, c, s, sc)
    return arr, len(rows)


def workspace_size(entries, h: MuonHyper) -> int:
    arr, n = table(entries)
    out = ctypes.c_size_t(0)
    _check(load().muon_workspace_size(arr, n, ctypes.byref(h), ctypes.byref(out)))
    return out.value


# ----------------------------------------------------------------------------- torch plumbing

_TORCH_DT = None


def _torch():
    import torch
    return torch


def _dtype_code(t) -> int:
    torch = _torch()
    m = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
    if t.dtype not in m:
        raise TypeError(f"unsupported tensor dtype {t.dtype}")
    return m[t.dtype]


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors passed to libmuonstep must be on a GPU")
    if not t.is_contiguous():
        raise ValueError("tensors passed to libmuonstep must be contiguous")
    return t.data_ptr()


def _stream(t, stream) -> Optional[int]:
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream(t.device)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _device(*tensors):
    """The one GPU all given tensors (None skipped) live on; every call runs with
    it as the current device."""
    devs = {t.device for t in tensors if t is not None}
    if len(devs) != 1:
        raise ValueError(f"tensors passed to libmuonstep must share one GPU, got {sorted(map(str, devs))}")
    dev = devs.pop()
    if dev.type != "cuda":
        raise ValueError("tensors passed to libmuonstep must be on a GPU")
    return dev


_ws_cache: Dict[Tuple[int, int], object] = {}
_ws_lock = threading.Lock()
_WS_CACHE_MAX = 16      # (device, stream) pairs kept; the oldest is dropped first


def workspace(nbytes: int, device, stream=None) -> "torch.Tensor":
    """A device workspace of at least `nbytes` bytes, cached per (device, stream).

    Steps enqueued on one stream reuse it in stream order; steps on different
    streams get different buffers, so they may run concurrently. A torch stream's
    buffer is allocated on that stream, so when a larger one replaces it the old
    memory is recycled in that stream's order. With a raw stream handle the
    caller orders the stream against torch's current stream. At most
    _WS_CACHE_MAX buffers are kept (a dropped one was allocated on its own
    stream, so torch reuses its memory in that stream's order)."""
    torch = _torch()
    dev = torch.device(device)
    idx = dev.index if dev.index is not None else torch.cuda.current_device()
    s = stream if stream is not None else torch.cuda.current_stream(idx)
    key = (idx, s.cuda_stream if hasattr(s, "cuda_stream") else int(s))
    with _ws_lock:
        buf = _ws_cache.get(key)
        if buf is None or buf.numel() < nbytes:
            _ws_cache.pop(key, None)
            size = max(nbytes, 256)
            if isinstance(s, torch.cuda.Stream):
                with torch.cuda.stream(s):
                    buf = torch.empty(size, dtype=torch.uint8, device=torch.device("cuda", idx))
            else:
                buf = torch.empty(size, dtype=torch.uint8, device=torch.device("cuda", idx))
            _ws_cache[key] = buf
            while len(_ws_cache) > _WS_CACHE_MAX:
                _ws_cache.pop(next(iter(_ws_cache)))
    return buf


def step(params, grads, momentum, entries, h: MuonHyper, ws=None, update_out=None,
         bf16_shadow=None, stream=None) -> None:
    """One Muon step (muon_step) on packed torch tensors; updates params and momentum."""
    torch = _torch()
    if momentum.dtype != torch.float32:
        raise TypeError("momentum must be float32")
    if params.dtype not in (torch.float32, torch.bfloat16) or _dtype_code(params) != h.param_dtype:
        raise TypeError("params must be float32 or bfloat16, matching hyper.param_dtype")
    if _dtype_code(grads) != h.grad_dtype:
        raise TypeError("grads dtype does not match hyper.grad_dtype")
    numel = params.numel()
    if grads.numel() != numel or momentum.numel() != numel:
        raise ValueError("params, grads and momentum must have the same numel")
    dev = _device(params, grads, momentum, ws, update_out, bf16_shadow)
    arr, n = table(entries)
    need = ctypes.c_size_t(0)
    _check(load().muon_workspace_size(arr, n, ctypes.byref(h), ctypes.byref(need)))
    if ws is None:
        ws = workspace(need.value, dev, stream)
    if update_out is not None and (update_out.dtype != torch.float32 or update_out.numel() != numel):
        raise ValueError("update_out must be float32 with params' numel")
    if bf16_shadow is not None and (bf16_shadow.element_size() != 2 or bf16_shadow.numel() != numel):
        raise ValueError("bf16_shadow must be a 16-bit tensor with params' numel")
    with torch.cuda.device(dev):
        _check(load().muon_step(_ptr(params), _ptr(grads), _ptr(momentum), numel, arr, n,
                                ctypes.byref(h), _ptr(ws), ws.numel() * ws.element_size(),
                                _ptr(update_out), _ptr(bf16_shadow), _stream(params, stream)))


def step_noalloc(params, grads, momentum, entries, h: MuonHyper, update_out=None,
                 bf16_shadow=None, stream=None) -> None:
    """One Muon step through muon_step_noalloc: no workspace argument, nothing
    allocated (the library's per-GPU device array serves as the workspace)."""
    torch = _torch()
    if momentum.dtype != torch.float32:
        raise TypeError("momentum must be float32")
    if params.dtype not in (torch.float32, torch.bfloat16) or _dtype_code(params) != h.param_dtype:
        raise TypeError("params must be float32 or bfloat16, matching hyper.param_dtype")
    if _dtype_code(grads) != h.grad_dtype:
        raise TypeError("grads dtype does not match hyper.grad_dtype")
    numel = params.numel()
    if grads.numel() != numel or momentum.numel() != numel:
        raise ValueError("params, grads and momentum must have the same numel")
    if update_out is not None and (update_out.dtype != torch.float32 or update_out.numel() != numel):
        raise ValueError("update_out must be float32 with params' numel")
    if bf16_shadow is not None and (bf16_shadow.element_size() != 2 or bf16_shadow.numel() != numel):
        raise ValueError("bf16_shadow must be a 16-bit tensor with params' numel")
    dev = _device(params, grads, momentum, update_out, bf16_shadow)
    arr, n = table(entries)
    with torch.cuda.device(dev):
        _check(load().muon_step_noalloc(_ptr(params), _ptr(grads), _ptr(momentum), numel, arr, n,
                                        ctypes.byref(h), _ptr(update_out), _ptr(bf16_shadow),
                                        _stream(params, stream)))


def windows(ws: Iterable[Sequence[int]], n: int):
    """ctypes array of muon_window_t from (lo, hi, param_offset) tuples, one per entry."""
    rows = [tuple(w) for w in ws]
    if len(rows) != n:
        raise ValueError("one window per table entry")
    arr = (MuonWindow * max(n, 1))()
    for i, (lo, hi, po) in enumerate(rows):
        arr[i] = MuonWindow(lo, hi, po)
    return arr


def step_window(partition, grads, momentum, entries, wins, h: MuonHyper, ws=None,
                update_out=None, bf16_shadow=None, stream=None) -> None:
    """One Muon step for the holder of a parameter partition (muon_step_window):
    momentum and Newton-Schulz on every listed matrix in full, the update
    applied to the window (lo, hi, param_offset) of each entry in `partition`."""
    torch = _torch()
    if partition.dtype != torch.float32 or momentum.dtype != torch.float32:
        raise TypeError("partition and momentum must be float32")
    if _dtype_code(grads) != h.grad_dtype:
        raise TypeError("grads dtype does not match hyper.grad_dtype")
    numel = momentum.numel()
    if grads.numel() != numel:
        raise ValueError("grads and momentum must have the same numel")
    dev = _device(partition, grads, momentum, ws, update_out, bf16_shadow)
    arr, n = table(entries)
    warr = windows(wins, n)
    need = ctypes.c_size_t(0)
    _check(load().muon_workspace_size(arr, n, ctypes.byref(h), ctypes.byref(need)))
    if ws is None:
        ws = workspace(need.value, dev, stream)
    if update_out is not None and (update_out.dtype != torch.float32 or update_out.numel() != numel):
        raise ValueError("update_out must be float32 with momentum's numel")
    if bf16_shadow is not None and (bf16_shadow.element_size() != 2 or
                                    bf16_shadow.numel() != partition.numel()):
        raise ValueError("bf16_shadow must be a 16-bit tensor with the partition's numel")
    with torch.cuda.device(dev):
        _check(load().muon_step_window(_ptr(partition), partition.numel(), _ptr(grads), _ptr(momentum),
                                       numel, arr, warr, n, ctypes.byref(h), _ptr(ws),
                                       ws.numel() * ws.element_size(), _ptr(update_out),
                                       _ptr(bf16_shadow), _stream(momentum, stream)))


def _method_code(method) -> int:
    return NS_METHODS[method] if isinstance(method, str) else int(method)


def ns_flops(m: int, n: int, method="standard", steps: int = 5) -> int:
    """Nominal Newton-Schulz FLOPs of one problem with short side m, long side n."""
    f = load().muon_ns_flops(m, n, _method_code(method), steps)
    if f < 0:
        raise ValueError("invalid problem for the FLOP model")
    return int(f)


def plan_owners(params: Sequence[Sequence[int]], n_owners: int, method="standard",
                steps: int = 5, align: int = 64):
    """Owner plan (muon_plan_owners) for matrices given as (rows, cols, split_rows,
    layer[, split_cols]). Returns (assign, owners): assign[i] = (owner, offset);
    owners[o] = dict(numel, max_layer_numel, ns_flops, n_matrices, table), where
    `table` is the owner's muon_step table [(offset, rows, cols, split_rows,
    split_cols), ...] in packed order, and `index` the matching input indices."""
    rows = [tuple(p) + (0,) * (5 - len(p)) for p in params]
    n = len(rows)
    arr = (MuonParam * max(n, 1))()
    for i, (r, c, s, layer, sc) in enumerate(rows):
        arr[i] = MuonParam(r, c, s, layer, 0, sc)
    out_a = (MuonAssign * max(n, 1))()
    out_o = (MuonOwner * max(n_owners, 1))()
    _check(load().muon_plan_owners(arr, n, n_owners, _method_code(method), steps, align, out_a,
                                   out_o))
    assign = [(out_a[i].owner, out_a[i].offset) for i in range(n)]
    owners = []
    for o in range(n_owners):
        idx = sorted((i for i in range(n) if assign[i][0] == o), key=lambda i: assign[i][1])
        owners.append({"numel": out_o[o].numel, "max_layer_numel": out_o[o].max_layer_numel,
                       "ns_flops": out_o[o].ns_flops, "n_matrices": out_o[o].n_matrices,
                       "index": idx,
                       "table": [(assign[i][1], rows[i][0], rows[i][1], rows[i][2], rows[i][4])
                                 for i in idx]})
    return assign, owners


def comm_elements(p_m: int, n_ranks: int, zero_stage: int = 2, dedicated: bool = True) -> float:
    """Elements sent per step on the shard group (muon_comm_elements)."""
    v = load().muon_comm_elements(p_m, n_ranks, zero_stage, int(bool(dedicated)))
    if v < 0:
        raise ValueError("invalid arguments for the communication model")
    return v


def adamw(params, grads, m, v, lr=3e-4, beta1=0.9, beta2=0.95, eps=1e-10, weight_decay=0.0,
          step: int = 1, stream=None) -> None:
    """AdamW step (adamw_step) on flat torch tensors; updates params, m and v."""
    torch = _torch()
    for t in (params, m, v):
        if t.dtype != torch.float32:
            raise TypeError("params, m and v must be float32")
    numel = params.numel()
    if any(t.numel() != numel for t in (grads, m, v)):
        raise ValueError("params, grads, m and v must have the same numel")
    h = AdamWHyper()
    load().muon_default_adamw_hyper(ctypes.byref(h))
    h.lr, h.beta1, h.beta2, h.eps, h.weight_decay = lr, beta1, beta2, eps, weight_decay
    h.step = step
    h.grad_dtype = _dtype_code(grads)
    dev = _device(params, grads, m, v)
    with torch.cuda.device(dev):
        _check(load().adamw_step(_ptr(params), _ptr(grads), _ptr(m), _ptr(v), numel, ctypes.byref(h),
                                 _stream(params, stream)))


def _copy_args(packed, tensors: Sequence, entries):
    """Table and pointer array for pack / unpack; each tensor must hold exactly its
    entry's rows * cols elements of the packed buffer's dtype (the copy is sized
    from the table and that dtype)."""
    tensors = list(tensors)
    arr, n = table(entries)
    if len(tensors) != n:
        raise ValueError(f"{len(tensors)} tensors for {n} table entries")
    for i, t in enumerate(tensors):
        if t.dtype != packed.dtype or t.numel() != arr[i].rows * arr[i].cols:
            raise ValueError(f"tensor {i} must be {packed.dtype} with {arr[i].rows * arr[i].cols} elements, "
                             f"got {t.dtype} with {t.numel()}")
    ptrs = (ctypes.c_void_p * max(n, 1))(*[_ptr(t) for t in tensors])
    return arr, n, ptrs, _device(packed, *tensors)


def pack(packed, tensors: Sequence, entries, stream=None) -> None:
    """Copy each tensor bit for bit into `packed` at its table offset."""
    torch = _torch()
    arr, n, ptrs, dev = _copy_args(packed, tensors, entries)
    with torch.cuda.device(dev):
        _check(load().muon_pack(_ptr(packed), packed.numel(), ptrs, arr, n, _dtype_code(packed),
                                _stream(packed, stream)))


def unpack(tensors: Sequence, packed, entries, stream=None) -> None:
    """Copy each table entry of `packed` bit for bit into its tensor."""
    torch = _torch()
    arr, n, ptrs, dev = _copy_args(packed, tensors, entries)
    with torch.cuda.device(dev):
        _check(load().muon_unpack(ptrs, _ptr(packed), packed.numel(), arr, n, _dtype_code(packed),
                                  _stream(packed, stream)))


def release_plans() -> None:
    _check(load().muon_release_plans())


def profile_begin() -> None:
    _check(load().muon_profile_begin())


def profile_end() -> Dict[str, Tuple[int, float]]:
    """{kernel kind: (launches, summed milliseconds)} since profile_begin()."""
    out = (KernelStat * 64)()
    n = ctypes.c_int32(0)
    _check(load().muon_profile_end(out, 64, ctypes.byref(n)))
    return {out[i].name.decode(): (out[i].launches, out[i].total_ms) for i in range(min(n.value, 64))}


# ----------------------------------------------------------------------------- 8-bit operands and experts

_FP8_TYPES = None


def _fp8_types():
    global _FP8_TYPES
    if _FP8_TYPES is None:
        torch = _torch()
        _FP8_TYPES = {torch.float8_e4m3fn: 0, torch.float8_e5m2: 1}
    return _FP8_TYPES


def _i32(v, name) -> int:
    """v as the C ABI's 32-bit integer; ctypes alone would drop the upper bits."""
    v = operator.index(v)
    if not -(1 << 31) <= v < 1 << 31:
        raise ValueError(f"{name} must be a 32-bit integer, got {v}")
    return v


def _same_device(first, *others):
    """The GPU that `first` and the others (None skipped) live on."""
    dev = first.device
    if dev.type != "cuda":
        raise ValueError("tensors passed to libmuonstep must be on a GPU")
    for t in others:
        if t is not None and t.device != dev:
            raise ValueError(f"tensors passed to libmuonstep must share one GPU, got {dev} and {t.device}")
    return dev


def _flat(t) -> Optional[int]:
    """Pointer of a contiguous tensor whose device is checked elsewhere (None stays None)."""
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to libmuonstep must be contiguous")
    return t.data_ptr()


def _last_dense(t, name):
    """(pointer, row pitch, batch stride) of a 2-D or 3-D tensor whose rows are contiguous."""
    shape, stride = t.shape, t.stride()
    n = len(shape)
    if n != 2 and n != 3:
        raise ValueError(f"{name} must be a matrix or a batch of matrices")
    if shape[-1] > 1 and stride[-1] != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    ld = stride[-2] if shape[-2] > 1 else shape[-1]
    bs = stride[0] if n == 3 and shape[0] > 1 else 0
    return t.data_ptr(), ld, bs


class _on:
    """Runs a call on `dev` and `stream`: outputs and workspaces that the binding
    allocates belong to that stream. A raw stream handle has no torch allocator,
    so it takes calls whose outputs are given (`fresh` then refuses)."""

    __slots__ = ("dev", "raw", "handle", "_ctx", "_stream")

    def __init__(self, dev, stream):
        torch = _torch()
        self.dev, self.raw, self._ctx, self._stream = dev, False, None, stream
        if stream is None:
            if torch.cuda.current_device() != dev.index:
                self._ctx = torch.cuda.device(dev)
        elif isinstance(stream, torch.cuda.Stream):
            if stream.device != dev:
                raise ValueError(f"the stream is on {stream.device}, the tensors on {dev}")
            self._ctx = torch.cuda.stream(stream)
        else:
            self.raw, self._ctx = True, torch.cuda.device(dev)

    def __enter__(self):
        if self._ctx is not None:
            self._ctx.__enter__()
        self.handle = int(self._stream) if self.raw else _torch()._C._cuda_getCurrentRawStream(self.dev.index)
        return self

    def __exit__(self, *exc):
        if self._ctx is not None:
            self._ctx.__exit__(*exc)

    def fresh(self, shape, dtype):
        if self.raw:
            raise ValueError("with a raw stream handle the outputs must be given")
        return _torch().empty(shape, dtype=dtype, device=self.dev)

    def scratch(self, nbytes, ws=None):
        """Workspace of a call: the caller's, or one of its own. Calls of two launches pass
        data through it, and other threads' calls may come between them on the same stream;
        under graph capture it is from the graph's memory, so that no two graphs share it."""
        if ws is not None or nbytes == 0:
            return ws
        if self.raw:
            raise ValueError("with a raw stream handle the workspace must be given")
        torch = _torch()
        return torch.empty(nbytes, dtype=torch.uint8, device=self.dev)


class Fp8:
    """A quantised operand (muon_fp8_t): float8 `data` [..., rows, cols padded to 128],
    float8_e8m0fnu `scale` [..., rows, blocks of 128 padded to 4], and its number of
    columns. One matrix, or a batch of them in the first dimension."""

    __slots__ = ("data", "scale", "cols")

    def __init__(self, data, scale, cols: int):
        torch = _torch()
        if data.dtype not in _fp8_types() or scale.dtype != torch.float8_e8m0fnu:
            raise TypeError("data must be float8_e4m3fn or float8_e5m2, scale float8_e8m0fnu")
        pitch = -(-cols // FP8_BLOCK) * FP8_BLOCK
        want = tuple(data.shape[:-1]) + (-(-(pitch // FP8_BLOCK) // 4) * 4,)
        if data.dim() not in (2, 3) or data.shape[-1] != pitch or tuple(scale.shape) != want:
            raise ValueError(f"{cols} columns take data of {pitch} columns and scale of shape {want}, "
                             f"got {tuple(data.shape)} and {tuple(scale.shape)}")
        self.data, self.scale, self.cols = data, scale, cols

    @property
    def rows(self) -> int:
        return self.data.shape[-2]

    @property
    def format(self) -> str:
        return "e4m3" if _fp8_types()[self.data.dtype] == 0 else "e5m2"

    def _c(self) -> Fp8Operand:
        d = self.data
        shape = d.shape
        return Fp8Operand(_flat(d), _flat(self.scale), shape[0] if len(shape) == 3 else 1, shape[-2], self.cols,
                          _fp8_types()[d.dtype], 0)

    @classmethod
    def _of(cls, data, scale, cols):
        """Parts that are known to fit."""
        self = cls.__new__(cls)
        self.data, self.scale, self.cols = data, scale, cols
        return self


def fp8_empty(rows: int, cols: int, fmt: str = "e4m3", device="cuda", batch: Optional[int] = None) -> Fp8:
    """An uninitialised operand of rows x cols (a batch of them with `batch`)."""
    torch = _torch()
    if fmt not in FP8_FORMATS:
        raise ValueError(f"format must be one of {sorted(FP8_FORMATS)}, got {fmt!r}")
    lead = () if batch is None else (batch,)
    pitch = -(-cols // FP8_BLOCK) * FP8_BLOCK
    dt = torch.float8_e4m3fn if fmt == "e4m3" else torch.float8_e5m2
    data = torch.empty(lead + (rows, pitch), dtype=dt, device=device)
    scale = torch.empty(lead + (rows, -(-(pitch // FP8_BLOCK) // 4) * 4), dtype=torch.float8_e8m0fnu, device=device)
    return Fp8._of(data, scale, cols)


def fp8_quantize(x, fmt: str = "e4m3", blocks: bool = False, transposed="no", row_index=None, row_div: int = 1,
                 row_weight=None, out: Optional[Fp8] = None, out_t: Optional[Fp8] = None, stream=None):
    """Quantise x (muon_fp8_quantize): [rows, cols] or a batch of them, float32,
    bfloat16 or float16, rows contiguous (any row pitch: a view into a packed
    buffer will do). transposed: "no" returns the operand, "only" the transposed
    one, "both" the pair. row_index (int32): row r of the result is x's row
    row_index[r] // row_div, zeros for a negative one, times
    row_weight[row_index[r]] where that is given. out / out_t: results of an
    earlier call to write into."""
    torch = _torch()
    if transposed not in ("no", "only", "both"):
        raise ValueError('transposed must be "no", "only" or "both"')
    if fmt not in FP8_FORMATS:
        raise ValueError(f"format must be one of {sorted(FP8_FORMATS)}, got {fmt!r}")
    if (out is not None and transposed == "only") or (out_t is not None and transposed == "no"):
        raise ValueError("an output was given that `transposed` does not ask for")
    row_div = _i32(row_div, "row_div")
    for t, dt, name in ((row_index, torch.int32, "row_index"), (row_weight, torch.float32, "row_weight")):
        if t is not None and t.dtype != dt:
            raise TypeError(f"{name} must be {dt}")
    ptr, ld, bs = _last_dense(x, "x")
    batch = x.shape[0] if x.dim() == 3 else None
    cols = x.shape[-1]
    rows = x.shape[-2] if row_index is None else row_index.numel()
    dev = _same_device(x, row_index, row_weight, *(t for o in (out, out_t) if o is not None for t in (o.data, o.scale)))
    with _on(dev, stream) as on:
        def make(r, c):
            if on.raw:
                raise ValueError("with a raw stream handle the outputs must be given")
            return fp8_empty(r, c, fmt, dev, batch)
        q = None if transposed == "only" else out if out is not None else make(rows, cols)
        qt = None if transposed == "no" else out_t if out_t is not None else make(cols, rows)
        for o in (q, qt):
            if o is not None and o.format != fmt:
                raise ValueError(f"outputs are {o.format}, the call asks for {fmt}")
        src = Fp8Source(ptr, bs, ld, 1 if batch is None else batch, x.shape[-2], cols, _dtype_code(x), row_div,
                        _flat(row_index), rows, _flat(row_weight), 0 if row_weight is None else row_weight.numel())
        _check(load().muon_fp8_quantize(ctypes.byref(src), int(bool(blocks)),
                                        None if q is None else ctypes.byref(q._c()),
                                        None if qt is None else ctypes.byref(qt._c()), on.handle))
    return (q, qt) if transposed == "both" else qt if transposed == "only" else q


def _result(out, shape, on, out_dtype, accumulate):
    """(tensor, muon_fp8_result_t) of a product's result."""
    torch = _torch()
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        out = on.fresh(shape, torch.bfloat16 if out_dtype is None else out_dtype)
    elif tuple(out.shape) != tuple(shape):
        raise ValueError(f"out must have shape {tuple(shape)}, got {tuple(out.shape)}")
    elif out_dtype is not None and out.dtype != out_dtype:
        raise TypeError(f"out is {out.dtype}, the call asks for {out_dtype}")
    ptr, ld, bs = _last_dense(out, "out")
    return out, Fp8Result(ptr, bs, ld, _dtype_code(out), int(bool(accumulate)))


def _int32(t, n, name):
    torch = _torch()
    if t.dtype != torch.int32 or (n is not None and t.numel() != n):
        raise ValueError(f"{name} must be int32" + ("" if n is None else f" with {n} elements"))


def fp8_matmul(a: Fp8, b: Fp8, out=None, out_dtype=None, accumulate: bool = False, offsets=None, stream=None):
    """a b^T (muon_fp8_matmul): [M, N] of a [M, K] and b [N, K], or batches of them.
    With `offsets` (int32, groups + 1) rows offsets[g] .. offsets[g + 1] of a meet
    matrix g of b [groups, N, K]; rows outside every group are not written.
    out: a tensor or view to write into (e.g. a matrix of the packed gradients),
    else a new one of out_dtype (bfloat16). accumulate adds to out."""
    if offsets is not None:
        if b.data.dim() != 3 or a.data.dim() != 2:
            raise ValueError("a grouped product takes one matrix a and a batch b")
        _int32(offsets, b.data.shape[0] + 1, "offsets")
        shape = (a.rows, b.rows)
    else:
        if a.data.dim() != b.data.dim():
            raise ValueError("a and b must both be single matrices or both be batches")
        shape = tuple(a.data.shape[:-1]) + (b.rows,)
    dev = _same_device(a.data, a.scale, b.data, b.scale, out, offsets)
    with _on(dev, stream) as on:
        out, c = _result(out, shape, on, out_dtype, accumulate)
        _check(load().muon_fp8_matmul(ctypes.byref(a._c()), ctypes.byref(b._c()), _flat(offsets), ctypes.byref(c),
                                      on.handle))
    return out


def fp8_matmul_grouped_k(a: Fp8, b: Fp8, offsets, out=None, out_dtype=None, accumulate: bool = False, stream=None):
    """Grouped contractions (muon_fp8_matmul_grouped_k): out[g] = the product of
    columns offsets[g] .. offsets[g + 1] of a [M, K] and b [N, K], each offset a
    multiple of 128: [groups, M, N]."""
    _int32(offsets, None, "offsets")
    groups = offsets.numel() - 1
    if groups < 0 or a.data.dim() != 2 or b.data.dim() != 2:
        raise ValueError("a grouped contraction takes single matrices and groups + 1 offsets")
    dev = _same_device(a.data, a.scale, b.data, b.scale, out, offsets)
    with _on(dev, stream) as on:
        out, c = _result(out, (groups, a.rows, b.rows), on, out_dtype, accumulate)
        _check(load().muon_fp8_matmul_grouped_k(ctypes.byref(a._c()), ctypes.byref(b._c()), _flat(offsets), groups,
                                                ctypes.byref(c), on.handle))
    return out


def route_hyper(**kw) -> RouteHyper:
    """Router hyperparameters: the library defaults, then keyword overrides (score:
    "softmax" | "sigmoid", top_k, n_groups, top_groups, group_top, renormalize, scale)."""
    h = RouteHyper()
    load().muon_default_route_hyper(ctypes.byref(h))
    for k, v in kw.items():
        if k == "score" and isinstance(v, str):
            v = ROUTE_SCORES.get(v, -1)
        if not hasattr(h, k) or k == "reserved":
            raise TypeError(f"unknown router hyperparameter {k!r}")
        setattr(h, k, v if k == "scale" else _i32(v, k))
    return h


def _logits(t):
    if t.dim() != 2:
        raise ValueError("logits must be [tokens, experts]")
    return _last_dense(t, "logits")


def _given(t, shape, dtype, on, name):
    if t is None:
        return on.fresh(shape, dtype)
    if t.dtype != dtype or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {dtype} of shape {tuple(shape)}, got {t.dtype} of {tuple(t.shape)}")
    return t


def route(logits, h: RouteHyper, bias=None, ids=None, weights=None, stream=None):
    """Route rows to experts (muon_route): (ids int32, weights float32), both [tokens, top_k]."""
    torch = _torch()
    ptr, ld, _ = _logits(logits)
    tokens, experts = logits.shape
    if bias is not None and (bias.dtype != torch.float32 or bias.numel() != experts):
        raise ValueError("bias must be float32 with one element per expert")
    dev = _same_device(logits, bias, ids, weights)
    with _on(dev, stream) as on:
        k = max(h.top_k, 0)
        ids = _given(ids, (tokens, k), torch.int32, on, "ids")
        weights = _given(weights, (tokens, k), torch.float32, on, "weights")
        _check(load().muon_route(ptr, _dtype_code(logits), tokens, experts, ld, _flat(bias), ctypes.byref(h), _flat(ids),
                                 _flat(weights), on.handle))
    return ids, weights


def route_backward(dweights, logits, ids, h: RouteHyper, dlogits=None, stream=None):
    """Gradient of route's weights with respect to the logits (muon_route_backward)."""
    torch = _torch()
    ptr, ld, _ = _logits(logits)
    tokens, experts = logits.shape
    if dweights.dtype != torch.float32 or tuple(dweights.shape) != (tokens, h.top_k):
        raise ValueError(f"dweights must be float32 of shape {(tokens, h.top_k)}")
    if ids.dtype != torch.int32 or tuple(ids.shape) != (tokens, h.top_k):
        raise ValueError(f"ids must be int32 of shape {(tokens, h.top_k)}")
    dev = _same_device(dweights, logits, ids, dlogits)
    with _on(dev, stream) as on:
        dlogits = _given(dlogits, (tokens, experts), logits.dtype, on, "dlogits")
        dptr, ldd, _ = _last_dense(dlogits, "dlogits")
        _check(load().muon_route_backward(_flat(dweights), ptr, _dtype_code(logits), tokens, experts, ld, _flat(ids),
                                          ctypes.byref(h), dptr, ldd, on.handle))
    return dlogits


@functools.lru_cache(maxsize=256)
def expert_order_workspace_size(n: int, n_experts: int) -> int:
    """Bytes of workspace that ordering n slots takes (muon_expert_order_workspace_size);
    0 for few slots."""
    need = ctypes.c_size_t(0)
    _check(load().muon_expert_order_workspace_size(n, _i32(n_experts, "n_experts"), ctypes.byref(need)))
    return need.value


def expert_order(ids, n_experts: int, align: int = 128, offsets=None, counts=None, rows=None, pos=None, stream=None,
                 ws=None):
    """Order of routed slots by expert (muon_expert_order): (offsets [experts + 1],
    counts [experts], rows [capacity], pos like ids), all int32. The capacity
    that any routing fits is ids.numel() + n_experts * (align - 1). Where none of
    offsets, counts and rows is given they are views of one new tensor. ws: a
    workspace of expert_order_workspace_size bytes that no other call uses until this
    one is done; without it the call allocates its own on its stream (with a raw
    stream handle it has to be given where the size is not 0)."""
    torch = _torch()
    _int32(ids, None, "ids")
    n, n_experts, align = ids.numel(), _i32(n_experts, "n_experts"), _i32(align, "align")
    dev = _same_device(ids, offsets, counts, rows, pos, ws)
    with _on(dev, stream) as on:
        need = expert_order_workspace_size(n, n_experts)
        capacity = max(n + n_experts * (align - 1), 0)
        if offsets is None and counts is None and rows is None:
            # one allocation: three cost as much time as the launch
            parts = (n_experts + 1, n_experts, capacity)
            offsets, counts, rows = on.fresh((sum(parts),), torch.int32).split_with_sizes(parts)
        else:
            offsets = _given(offsets, (n_experts + 1,), torch.int32, on, "offsets")
            counts = _given(counts, (n_experts,), torch.int32, on, "counts")
            if rows is None:
                rows = on.fresh((capacity,), torch.int32)
            else:
                _int32(rows, None, "rows")
        pos = _given(pos, ids.shape, torch.int32, on, "pos")
        ws = on.scratch(need, ws)
        _check(load().muon_expert_order(_flat(ids), n, n_experts, align, _flat(offsets), _flat(counts), _flat(rows),
                                        rows.numel(), _flat(pos), _flat(ws),
                                        0 if ws is None else ws.numel() * ws.element_size(), on.handle))
    return offsets, counts, rows, pos


def _slots(o_or_dy, pos, weights):
    torch = _torch()
    if pos.dim() != 2 or pos.dtype != torch.int32:
        raise ValueError("pos must be int32 [tokens, top_k]")
    if weights.dtype != torch.float32 or weights.shape != pos.shape:
        raise ValueError("weights must be float32 with pos's shape")
    if o_or_dy.dim() != 2:
        raise ValueError("expected a matrix of rows")


def combine(o, pos, weights, out=None, stream=None):
    """Weighted sum of each token's expert rows (muon_combine): [tokens, cols] of
    o [rows, cols], pos and weights [tokens, top_k]."""
    _slots(o, pos, weights)
    optr, ldo, _ = _last_dense(o, "o")
    tokens, k = pos.shape
    dev = _same_device(o, pos, weights, out)
    with _on(dev, stream) as on:
        out = _given(out, (tokens, o.shape[1]), o.dtype, on, "out")
        yptr, ldy, _ = _last_dense(out, "out")
        _check(load().muon_combine(optr, _dtype_code(o), o.shape[0], o.shape[1], ldo, _flat(pos), _flat(weights), tokens,
                                   k, yptr, ldy, on.handle))
    return out


def combine_backward(dy, o, pos, weights, dweights=None, do=None, stream=None):
    """Gradients of combine (muon_combine_backward): (dweights, do). Rows of `do` that
    no slot points at are not written (zeros in a new one)."""
    torch = _torch()
    _slots(dy, pos, weights)
    if o.dim() != 2 or dy.dtype != o.dtype or tuple(dy.shape) != (pos.shape[0], o.shape[1]):
        raise ValueError("dy must be [tokens, cols] with o's dtype")
    tokens, k = pos.shape
    dyptr, lddy, _ = _last_dense(dy, "dy")
    optr, ldo, _ = _last_dense(o, "o")
    dev = _same_device(dy, o, pos, weights, dweights, do)
    with _on(dev, stream) as on:
        dweights = _given(dweights, (tokens, k), torch.float32, on, "dweights")
        do = on.fresh(o.shape, o.dtype).zero_() if do is None else _given(do, o.shape, o.dtype, on, "do")
        doptr, lddo, _ = _last_dense(do, "do")
        _check(load().muon_combine_backward(dyptr, _dtype_code(dy), tokens, o.shape[1], lddy, optr, o.shape[0], ldo,
                                            _flat(pos), _flat(weights), k, _flat(dweights), doptr, lddo, on.handle))
    return dweights, do
