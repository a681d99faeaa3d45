"""Thin ctypes binding of libmuon (include/muon.h): argument marshalling only.

Every step of the Muon path runs in the library's CUDA kernels; this module
only turns tensors into pointers, shapes and a stream handle.  Loading fails
loudly when the library has not been built (there is no fallback path).
"""
from __future__ import annotations

import ctypes
import os
from typing import Iterable, NamedTuple, Optional, Sequence

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmuon.so")

MUON_OK = 0
STATUS_NAMES = {
    0: "MUON_OK", 1: "MUON_ERR_INVALID_ARGUMENT", 2: "MUON_ERR_UNSUPPORTED",
    3: "MUON_ERR_ALIAS", 4: "MUON_ERR_OUT_OF_MEMORY", 5: "MUON_ERR_CUDA",
    6: "MUON_ERR_TIMEOUT", 7: "MUON_ERR_NONFINITE", 8: "MUON_ERR_BOUNDS",
}
MUON_F32, MUON_BF16, MUON_E4M3 = 0, 1, 2
ROUTE_SOFTMAX, ROUTE_SIGMOID = 0, 1
GROUP_MAX, GROUP_SUM2 = 0, 1
SCALE_SQRT_MAX1_R_OVER_C, SCALE_RMS_0P2_SQRT_MAXDIM, SCALE_ONE = 0, 1, 2
NS_BF16, NS_TF32 = 0, 1
PROFILE_KINDS = ("prep", "gram", "poly", "apply", "update", "fused_small", "adamw")

EXPORTED = (
    "muon_ns_default_config", "muon_ns_batched", "muon_ns_batched_ex", "muon_step_grouped",
    "muon_step_grouped_ex", "muon_step_grouped_host", "muon_query_status", "muon_status_string",
    "muon_release_workspace", "muon_last_launch_count", "muon_profile_enable",
    "muon_profile_read", "muon_adamw_grouped", "muon_ns_cost_table", "muon_assign_owners",
    "muon_ns_batched_noalloc", "muon_debug_inject_stall", "muon_debug_guard_check",
    "muon_ns_path",
    "muon_ns_gram_restart",
    "muon_debug_build",
    "muon_rmsnorm_forward", "muon_rmsnorm_backward",
    "muon_route_forward", "muon_route_plan", "muon_route_backward",
    "muon_experts_forward", "muon_experts_backward",
)
PATH_SMALL, PATH_XSPACE, PATH_GRAM_SPACE = 0, 1, 2
INJECT_NONE, INJECT_GEMM, INJECT_SMALL = 0, 1, 2


class MuonError(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__(f"{where}: {STATUS_NAMES.get(code, code)}")
        self.code = code


class NsConfig(ctypes.Structure):
    _fields_ = [("steps", ctypes.c_int32), ("coeffs", ctypes.POINTER(ctypes.c_float)),
                ("a", ctypes.c_float), ("b", ctypes.c_float), ("c", ctypes.c_float),
                ("eps", ctypes.c_float), ("precision", ctypes.c_int32)]


class Group(ctypes.Structure):
    _fields_ = [("W", ctypes.c_void_p), ("w_dtype", ctypes.c_int32),
                ("G", ctypes.c_void_p), ("g_dtype", ctypes.c_int32),
                ("Mom", ctypes.c_void_p),
                ("B", ctypes.c_int64), ("M", ctypes.c_int64), ("N", ctypes.c_int64)]


class AdamwGroup(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("p_dtype", ctypes.c_int32),
                ("grad", ctypes.c_void_p), ("g_dtype", ctypes.c_int32),
                ("exp_avg", ctypes.c_void_p), ("exp_avg_sq", ctypes.c_void_p),
                ("numel", ctypes.c_int64)]


class AdamwConfig(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("beta1", ctypes.c_float), ("beta2", ctypes.c_float),
                ("eps", ctypes.c_float), ("weight_decay", ctypes.c_float),
                ("step", ctypes.c_int64)]


class Unit(ctypes.Structure):
    _fields_ = [("cost", ctypes.c_double), ("bytes", ctypes.c_int64), ("elems", ctypes.c_int64),
                ("layer", ctypes.c_int32)]


class RmsNorm(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("x", ctypes.c_void_p), ("x_stride", ctypes.c_int64),
                ("residual", ctypes.c_void_p), ("residual_stride", ctypes.c_int64),
                ("gain", ctypes.c_void_p),
                ("h", ctypes.c_void_p), ("h_stride", ctypes.c_int64),
                ("y", ctypes.c_void_p), ("y_stride", ctypes.c_int64),
                ("scales", ctypes.c_void_p),
                ("x_dtype", ctypes.c_int32), ("residual_dtype", ctypes.c_int32),
                ("gain_dtype", ctypes.c_int32), ("h_dtype", ctypes.c_int32),
                ("y_dtype", ctypes.c_int32), ("group", ctypes.c_int32), ("eps", ctypes.c_float)]


class RmsNormGrad(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("dy", ctypes.c_void_p), ("dy_stride", ctypes.c_int64),
                ("h", ctypes.c_void_p), ("h_stride", ctypes.c_int64),
                ("gain", ctypes.c_void_p),
                ("dres", ctypes.c_void_p), ("dres_stride", ctypes.c_int64),
                ("dh", ctypes.c_void_p), ("dh_stride", ctypes.c_int64),
                ("dgain", ctypes.c_void_p),
                ("dy_dtype", ctypes.c_int32), ("h_dtype", ctypes.c_int32),
                ("gain_dtype", ctypes.c_int32), ("dres_dtype", ctypes.c_int32),
                ("dh_dtype", ctypes.c_int32), ("eps", ctypes.c_float)]


class RouteConfig(ctypes.Structure):
    _fields_ = [("experts", ctypes.c_int32), ("top_k", ctypes.c_int32), ("score", ctypes.c_int32),
                ("groups", ctypes.c_int32), ("top_groups", ctypes.c_int32),
                ("group_score", ctypes.c_int32), ("renormalize", ctypes.c_int32),
                ("scale", ctypes.c_float)]


class Experts(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("hidden", ctypes.c_int64), ("inner", ctypes.c_int64),
                ("experts", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("x", ctypes.c_void_p), ("x_stride", ctypes.c_int64),
                ("w_in", ctypes.c_void_p), ("w_out", ctypes.c_void_p),
                ("weights", ctypes.c_void_p), ("offsets", ctypes.c_void_p),
                ("src", ctypes.c_void_p), ("pos", ctypes.c_void_p)]


class Route(NamedTuple):
    """A routing as muon_route_forward returns it (int32, f32, int32 ...)."""
    idx: object       # [tokens, top_k] expert of each slot, -1: none
    weights: object   # [tokens, top_k]
    offsets: object   # [experts + 1] rows of each expert; None without a plan
    src: object       # [tokens * top_k] token * top_k + slot of each row, -1 past the last
    pos: object       # [tokens, top_k] row of each slot, -1: none


_lib = None


def load(path: str = None) -> ctypes.CDLL:
    """Load libmuon.so, or the library MUON_LIB_PATH names (the -DMUON_DEBUG
    build, libmuon_debug.so); raises OSError when it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or os.environ.get("MUON_LIB_PATH") or LIB_PATH
    if not os.path.exists(path):
        raise OSError(f"{path} not found: build it with `python -m newton_schulz_gb300.build`")
    lib = ctypes.CDLL(path)
    i32, i64, vp, f32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_float
    lib.muon_ns_default_config.argtypes = [ctypes.POINTER(NsConfig)]
    lib.muon_ns_default_config.restype = i32
    lib.muon_ns_batched.argtypes = [vp, i64, i64, i64, ctypes.c_int, f32, f32, f32, vp]
    lib.muon_ns_batched.restype = i32
    lib.muon_ns_batched_ex.argtypes = [vp, i32, i64, i64, i64, ctypes.POINTER(NsConfig), vp, vp]
    lib.muon_ns_batched_ex.restype = i32
    lib.muon_step_grouped.argtypes = [ctypes.POINTER(Group), ctypes.c_int, f32, ctypes.c_int,
                                      f32, f32, ctypes.c_int, vp]
    lib.muon_step_grouped.restype = i32
    lib.muon_step_grouped_ex.argtypes = [ctypes.POINTER(Group), ctypes.c_int, f32, ctypes.c_int,
                                         f32, f32, ctypes.c_int, ctypes.POINTER(NsConfig), vp]
    lib.muon_step_grouped_ex.restype = i32
    lib.muon_adamw_grouped.argtypes = [ctypes.POINTER(AdamwGroup), ctypes.c_int,
                                       ctypes.POINTER(AdamwConfig), vp]
    lib.muon_adamw_grouped.restype = i32
    lib.muon_ns_cost_table.argtypes = [ctypes.POINTER(ctypes.c_int64), ctypes.c_int,
                                       ctypes.POINTER(NsConfig), ctypes.c_int,
                                       ctypes.POINTER(ctypes.c_double), vp]
    lib.muon_ns_cost_table.restype = i32
    lib.muon_assign_owners.argtypes = [ctypes.POINTER(Unit), ctypes.c_int, ctypes.c_int,
                                       ctypes.c_double, ctypes.POINTER(ctypes.c_int32)]
    lib.muon_assign_owners.restype = i32
    lib.muon_step_grouped_host.argtypes = lib.muon_step_grouped_ex.argtypes
    lib.muon_step_grouped_host.restype = i32
    lib.muon_ns_batched_noalloc.argtypes = [vp, i64, i64, i64, ctypes.c_int, f32, f32, f32, vp]
    lib.muon_ns_batched_noalloc.restype = i32
    lib.muon_debug_inject_stall.argtypes = [ctypes.c_int]
    lib.muon_debug_inject_stall.restype = i32
    lib.muon_ns_path.argtypes = [i64, i64, ctypes.POINTER(NsConfig)]
    lib.muon_ns_path.restype = ctypes.c_int
    lib.muon_ns_gram_restart.argtypes = [i64]
    lib.muon_ns_gram_restart.restype = ctypes.c_int
    lib.muon_debug_build.argtypes = []
    lib.muon_debug_build.restype = ctypes.c_int
    lib.muon_debug_guard_check.argtypes = [vp, ctypes.POINTER(ctypes.c_int64)]
    lib.muon_debug_guard_check.restype = i32
    for name, args in (
            ("muon_rmsnorm_forward", [ctypes.POINTER(RmsNorm), vp]),
            ("muon_rmsnorm_backward", [ctypes.POINTER(RmsNormGrad), vp]),
            ("muon_route_forward", [ctypes.POINTER(RouteConfig), vp, i32, i64, i64, vp, vp, vp, vp,
                                    vp, vp, vp, vp]),
            ("muon_route_plan", [vp, i64, i32, i32, vp, vp, vp, vp]),
            ("muon_route_backward", [ctypes.POINTER(RouteConfig), vp, i32, i64, i64, vp, vp, vp,
                                     i64, vp]),
            ("muon_experts_forward", [ctypes.POINTER(Experts), vp, i64, vp, vp]),
            ("muon_experts_backward", [ctypes.POINTER(Experts), vp, i64, vp, vp, i64, vp, vp, i32,
                                       vp, vp])):
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = args, i32
    lib.muon_query_status.argtypes = [vp]
    lib.muon_query_status.restype = i32
    lib.muon_status_string.argtypes = [i32]
    lib.muon_status_string.restype = ctypes.c_char_p
    lib.muon_release_workspace.argtypes = []
    lib.muon_release_workspace.restype = None
    lib.muon_last_launch_count.argtypes = []
    lib.muon_last_launch_count.restype = ctypes.c_int
    lib.muon_profile_enable.argtypes = [ctypes.c_int]
    lib.muon_profile_enable.restype = ctypes.c_int
    lib.muon_profile_read.argtypes = [ctypes.POINTER(ctypes.c_double),
                                      ctypes.POINTER(ctypes.c_int64), ctypes.c_int]
    lib.muon_profile_read.restype = ctypes.c_int
    _lib = lib
    return lib


# ---- marshalling helpers ----------------------------------------------------------
def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.float32:
        return MUON_F32
    if t.dtype == torch.bfloat16:
        return MUON_BF16
    raise TypeError(f"unsupported dtype {t.dtype}")


def _stream_ptr(stream) -> Optional[int]:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _shape3(t):
    if t.dim() == 2:
        return 1, t.shape[0], t.shape[1]
    if t.dim() == 3:
        return t.shape[0], t.shape[1], t.shape[2]
    raise ValueError("tensors must be [M,N] or [B,M,N]")


def _check_contig(*ts):
    for t in ts:
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous row-major")


def check(code: int, where: str) -> None:
    if code != MUON_OK:
        raise MuonError(code, where)


def make_config(steps: int = 5, coeffs: Optional[Sequence[Sequence[float]]] = None,
                a: float = 3.4445, b: float = -4.7750, c: float = 2.0315,
                eps: float = 1e-7, precision: int = NS_BF16):
    """Build an NsConfig; keeps the coefficient array alive on the object."""
    cfg = NsConfig()
    cfg.steps, cfg.a, cfg.b, cfg.c, cfg.eps, cfg.precision = steps, a, b, c, eps, precision
    if coeffs is not None:
        flat = [float(v) for row in coeffs for v in row]
        arr = (ctypes.c_float * max(1, len(flat)))(*flat)
        cfg.coeffs = ctypes.cast(arr, ctypes.POINTER(ctypes.c_float))
        cfg._keep = arr
    return cfg


# ---- entry points (same names as the C ABI) -------------------------------------------
def muon_ns_batched(X, steps: int = 5, a: float = 3.4445, b: float = -4.7750,
                    c: float = 2.0315, stream=None) -> None:
    """In-place NS of every [M,N] slice of a contiguous bf16 CUDA tensor."""
    _check_contig(X)
    B, M, N = _shape3(X)
    check(load().muon_ns_batched(X.data_ptr(), B, M, N, steps, a, b, c, _stream_ptr(stream)),
          "muon_ns_batched")


def muon_ns_batched_noalloc(X, steps: int = 5, a: float = 3.4445, b: float = -4.7750,
                            c: float = 2.0315, stream=None) -> None:
    """As muon_ns_batched, with the library's fixed workspace array (the call
    allocates no device memory)."""
    _check_contig(X)
    B, M, N = _shape3(X)
    check(load().muon_ns_batched_noalloc(X.data_ptr(), B, M, N, steps, a, b, c,
                                         _stream_ptr(stream)), "muon_ns_batched_noalloc")


def muon_ns_batched_ex(X, cfg=None, out=None, stream=None) -> None:
    """NS of every [M,N] slice of X (f32 or bf16) into X, or into `out`,
    which the library writes in X's dtype and shape (checked here: the C
    entry point sees only a pointer)."""
    _check_contig(X)
    B, M, N = _shape3(X)
    if out is not None:
        _check_contig(out)
        if out.dtype != X.dtype or tuple(out.shape) != tuple(X.shape):
            raise ValueError(f"out must match X: {out.dtype} {tuple(out.shape)} against "
                             f"{X.dtype} {tuple(X.shape)}")
    check(load().muon_ns_batched_ex(X.data_ptr(), _dtype_code(X), B, M, N,
                                    ctypes.byref(cfg) if cfg is not None else None,
                                    out.data_ptr() if out is not None else None,
                                    _stream_ptr(stream)), "muon_ns_batched_ex")


def make_groups(groups: Iterable[dict]):
    """[{"W","G","Mom"}] of contiguous CUDA tensors -> ctypes array."""
    groups = list(groups)
    arr = (Group * max(1, len(groups)))()
    for i, g in enumerate(groups):
        W, G, Mom = g["W"], g["G"], g["Mom"]
        _check_contig(W, G, Mom)
        B, M, N = _shape3(W)
        arr[i] = Group(W.data_ptr(), _dtype_code(W), G.data_ptr(), _dtype_code(G),
                       Mom.data_ptr(), B, M, N)
    return arr, len(groups)


def muon_step_grouped(groups, mu: float = 0.95, nesterov: bool = True, lr: float = 0.02,
                      wd: float = 0.01, scale_rule: int = SCALE_SQRT_MAX1_R_OVER_C,
                      ns_cfg=None, stream=None) -> None:
    """One fused Muon step over groups of [B,M,N] tensors (W, G, Mom)."""
    arr, n = groups if isinstance(groups, tuple) else make_groups(groups)
    lib = load()
    if ns_cfg is None:
        code = lib.muon_step_grouped(arr, n, mu, int(nesterov), lr, wd, scale_rule,
                                     _stream_ptr(stream))
    else:
        code = lib.muon_step_grouped_ex(arr, n, mu, int(nesterov), lr, wd, scale_rule,
                                        ctypes.byref(ns_cfg), _stream_ptr(stream))
    check(code, "muon_step_grouped")


muon_step_grouped_ex = muon_step_grouped


def muon_step_grouped_host(groups, mu: float = 0.95, nesterov: bool = True, lr: float = 0.02,
                           wd: float = 0.01, scale_rule: int = SCALE_SQRT_MAX1_R_OVER_C,
                           ns_cfg=None, stream=None) -> None:
    """One Muon step over groups of HOST (ideally pinned) [B,M,N] tensors; the
    library stages them through device memory.  Synchronise `stream` before
    reading the results."""
    arr, n = groups if isinstance(groups, tuple) else make_groups(groups)
    code = load().muon_step_grouped_host(arr, n, mu, int(nesterov), lr, wd, scale_rule,
                                         ctypes.byref(ns_cfg) if ns_cfg is not None else None,
                                         _stream_ptr(stream))
    check(code, "muon_step_grouped_host")


def muon_query_status(stream=None) -> int:
    return load().muon_query_status(_stream_ptr(stream))


def muon_debug_inject_stall(what: int) -> None:
    """Testing hook: the next launch of kind `what` (INJECT_GEMM or
    INJECT_SMALL) stalls on a wait nothing satisfies until its bound runs out."""
    check(load().muon_debug_inject_stall(int(what)), "muon_debug_inject_stall")


def muon_ns_path(rows: int, cols: int, cfg=None) -> int:
    """0 small-m kernel, 1 grouped GEMMs in X space, 2 grouped GEMMs in Gram
    space, for a stored [rows, cols] matrix (host-side decision)."""
    return load().muon_ns_path(rows, cols, ctypes.byref(cfg) if cfg is not None else None)


def muon_ns_gram_restart(m: int) -> int:
    """Restart period (NS steps) of the Gram-space path for small side m;
    0 = no restart."""
    return load().muon_ns_gram_restart(m)


def muon_debug_build() -> bool:
    """True for the -DMUON_DEBUG build (libmuon_debug.so)."""
    return bool(load().muon_debug_build())


def muon_debug_guard_check(stream=None) -> int:
    """Bytes found changed in the workspace guard bands since the last read
    (calls made with MUON_WS_GUARD=1); synchronises the stream."""
    bad = ctypes.c_int64(0)
    check(load().muon_debug_guard_check(_stream_ptr(stream), ctypes.byref(bad)),
          "muon_debug_guard_check")
    return bad.value


def muon_status_string(code: int) -> str:
    return load().muon_status_string(code).decode()


def muon_release_workspace() -> None:
    load().muon_release_workspace()


def muon_last_launch_count() -> int:
    return load().muon_last_launch_count()


def muon_profile_enable(enable: bool = True) -> int:
    return load().muon_profile_enable(int(enable))


def muon_profile_read():
    """{kind: (ms_total, launches)} since the last read (stream synchronised first)."""
    n = len(PROFILE_KINDS)
    ms = (ctypes.c_double * n)()
    cnt = (ctypes.c_int64 * n)()
    load().muon_profile_read(ms, cnt, n)
    return {k: (ms[i], cnt[i]) for i, k in enumerate(PROFILE_KINDS)}


def muon_adamw_grouped(groups, step: int, lr: float = 1e-3, betas=(0.9, 0.999),
                       eps: float = 1e-8, weight_decay: float = 0.01, stream=None) -> None:
    """One AdamW step over [{"param", "grad", "exp_avg", "exp_avg_sq"}] of
    contiguous CUDA tensors (any shape; fp32 state)."""
    groups = list(groups)
    arr = (AdamwGroup * max(1, len(groups)))()
    for i, g in enumerate(groups):
        p, gr, m, v = g["param"], g["grad"], g["exp_avg"], g["exp_avg_sq"]
        _check_contig(p, gr, m, v)
        arr[i] = AdamwGroup(p.data_ptr(), _dtype_code(p), gr.data_ptr(), _dtype_code(gr),
                            m.data_ptr(), v.data_ptr(), p.numel())
    cfg = AdamwConfig(lr, betas[0], betas[1], eps, weight_decay, step)
    check(load().muon_adamw_grouped(arr, len(groups), ctypes.byref(cfg), _stream_ptr(stream)),
          "muon_adamw_grouped")


def muon_ns_cost_table(shapes, cfg=None, reps: int = 5, stream=None):
    """Measured NS milliseconds per matrix for each (rows, cols) in `shapes`."""
    shapes = [(int(r), int(c)) for r, c in shapes]
    n = len(shapes)
    flat = (ctypes.c_int64 * max(1, 2 * n))(*[v for rc in shapes for v in rc])
    out = (ctypes.c_double * max(1, n))()
    check(load().muon_ns_cost_table(flat, n, ctypes.byref(cfg) if cfg is not None else None,
                                    reps, out, _stream_ptr(stream)), "muon_ns_cost_table")
    return [out[i] for i in range(n)]


def muon_assign_owners(costs, n_ranks: int, nbytes=None, elems=None, layers=None,
                       eps: float = 0.1):
    """Owner rank of each assignment unit (greedy LPT with a byte cap and
    layer spreading); host only."""
    n = len(costs)
    nbytes = nbytes if nbytes is not None else [0] * n
    elems = elems if elems is not None else [0] * n
    layers = layers if layers is not None else [-1] * n
    arr = (Unit * max(1, n))(*[Unit(float(costs[i]), int(nbytes[i]), int(elems[i]), int(layers[i]))
                               for i in range(n)])
    out = (ctypes.c_int32 * max(1, n))()
    check(load().muon_assign_owners(arr, n, n_ranks, eps, out), "muon_assign_owners")
    return [out[i] for i in range(n)]


# ---- the mixture-of-experts block ------------------------------------------------------
_DTYPE_CODES = {}


def _code(dtype) -> int:
    code = _DTYPE_CODES.get(dtype)
    if code is None:
        import torch
        _DTYPE_CODES.update({torch.float32: MUON_F32, torch.bfloat16: MUON_BF16,
                             torch.float8_e4m3fn: MUON_E4M3})
        code = _DTYPE_CODES.get(dtype)
        if code is None:
            raise TypeError(f"unsupported dtype {dtype}")
    return code


def _rows(t, name: str, cols: Optional[int] = None, rows: Optional[int] = None):
    """(pointer, row stride, dtype code) of a CUDA tensor [rows, cols] whose
    columns are adjacent in memory."""
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must be [rows, cols]")
    r, c = shape
    if (cols is not None and c != cols) or (rows is not None and r != rows):
        raise ValueError(f"{name} is {tuple(shape)}, expected {(rows, cols)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.is_contiguous():
        return t.data_ptr(), c, _code(t.dtype)
    if c > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: neighbouring columns must be adjacent in memory")
    stride = t.stride(0) if r > 1 else c
    if r > 1 and stride < c:
        raise ValueError(f"{name}: rows overlap")
    return t.data_ptr(), stride, _code(t.dtype)


def _current_handle() -> int:
    """The current stream's handle.  torch.cuda.current_stream() builds a Stream
    object, several microseconds of a small call; where torch has no cheaper
    way to the handle, it is taken from there."""
    import torch
    try:
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    except AttributeError:
        return torch.cuda.current_stream().cuda_stream


def _as_current(stream):
    """Context in which `stream` (a torch stream or a raw handle) is the current
    one.  The block's calls allocate their outputs in it: memory of another
    stream may still be written by work that was enqueued there before the call."""
    import torch
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


def _like(t, dtype=None):
    """An uninitialised contiguous tensor of t's shape (torch.empty_like is the
    cheapest allocation from Python; it would keep a view's strides)."""
    import torch
    if t.is_contiguous():
        return torch.empty_like(t) if dtype is None else torch.empty_like(t, dtype=dtype)
    return torch.empty(t.shape, dtype=dtype or t.dtype, device=t.device)


def _dense(t, name: str, shape, dtype) -> int:
    """Pointer of a contiguous CUDA tensor of exactly this shape and dtype."""
    if t.shape != shape or t.dtype != dtype or not t.is_contiguous() or not t.is_cuda:
        raise ValueError(f"{name} must be a contiguous CUDA {dtype} tensor {tuple(shape)}, got "
                         f"{t.dtype} {tuple(t.shape)}")
    return t.data_ptr()


def muon_rmsnorm_forward(x, gain=None, residual=None, eps: float = 1e-6, y_dtype=None, group: int = 0,
                         h=None, y=None, scales=None, stream=None):
    """(y, h, scales) of h = x + residual, y = gain h / sqrt(mean(h^2) + eps)
    for CUDA tensors [rows, cols]; see include/muon.h.

    y has dtype `y_dtype` (x's by default; float8_e4m3fn adds `scales`, one per
    row or, with group = 128, per 128 columns).  h has the residual's dtype; it
    is None without a residual unless given.  Outputs that are not given are
    allocated; h may be `residual` itself."""
    import torch
    if stream is not None:
        with _as_current(stream):
            return muon_rmsnorm_forward(x, gain, residual, eps, y_dtype, group, h, y, scales)
    xp, xs, xc = _rows(x, "x")
    rows, cols = x.shape
    rp, rs, rc, gp, gc, hp, hs, hc, sp = None, 0, 0, None, 0, None, 0, 0, None
    if residual is not None:
        rp, rs, rc = _rows(residual, "residual", cols, rows)
        if h is None:
            h = _like(residual)
    if gain is not None:
        gp, gc = _dense(gain, "gain", (cols,), gain.dtype), _code(gain.dtype)
    if h is not None:
        hp, hs, hc = _rows(h, "h", cols, rows)
    if y is None:
        y = _like(x, y_dtype)
    elif y_dtype is not None and y.dtype != y_dtype:
        raise ValueError(f"y is {y.dtype}, expected {y_dtype}")
    yp, ys, yc = _rows(y, "y", cols, rows)
    if yc == MUON_E4M3:
        n = -(-cols // group) if group > 0 else 1
        if scales is None:
            scales = torch.empty((rows, n), dtype=torch.float32, device=x.device)
        sp = _dense(scales, "scales", (rows, n), torch.float32)
    else:
        scales = None
    a = RmsNorm(rows, cols, xp, xs, rp, rs, gp, hp, hs, yp, ys, sp, xc, rc, gc, hc, yc, group, eps)
    check(load().muon_rmsnorm_forward(a, _current_handle()), "muon_rmsnorm_forward")
    return y, h, scales


def muon_rmsnorm_backward(dy, h, gain=None, dres=None, eps: float = 1e-6, dh=None, dgain=None,
                          want_dgain: bool = True, stream=None):
    """(dh, dgain) of muon_rmsnorm_forward: dh (h's dtype unless given) is the
    gradient of x and of the residual, with `dres`, the gradient that reaches
    h along the residual stream, added; dgain is f32 [cols] (None when not
    wanted)."""
    import torch
    if stream is not None:
        with _as_current(stream):
            return muon_rmsnorm_backward(dy, h, gain, dres, eps, dh, dgain, want_dgain)
    dp, ds, dc = _rows(dy, "dy")
    rows, cols = dy.shape
    hp, hs, hc = _rows(h, "h", cols, rows)
    gp, gc, rp, rs, rc, wp = None, 0, None, 0, 0, None
    if gain is not None:
        gp, gc = _dense(gain, "gain", (cols,), gain.dtype), _code(gain.dtype)
    if dres is not None:
        rp, rs, rc = _rows(dres, "dres", cols, rows)
    if dh is None:
        dh = _like(h)
    op, os_, oc = _rows(dh, "dh", cols, rows)
    if dgain is None and want_dgain:
        dgain = torch.empty(cols, dtype=torch.float32, device=dy.device)
    if dgain is not None:
        wp = _dense(dgain, "dgain", (cols,), torch.float32)
    a = RmsNormGrad(rows, cols, dp, ds, hp, hs, gp, rp, rs, op, os_, wp, dc, hc, gc, rc, oc, eps)
    check(load().muon_rmsnorm_backward(a, _current_handle()), "muon_rmsnorm_backward")
    return dh, dgain


def make_route_config(experts: int, top_k: int, score: int = ROUTE_SOFTMAX, groups: int = 1,
                      top_groups: Optional[int] = None, group_score: int = GROUP_MAX,
                      renormalize: bool = False, scale: float = 1.0) -> RouteConfig:
    """Build a RouteConfig (include/muon.h); top_groups defaults to every group."""
    return RouteConfig(experts, top_k, score, groups, groups if top_groups is None else top_groups,
                       group_score, int(renormalize), scale)


def _plan_tensors(dev, tokens: int, top_k: int, experts: int):
    import torch
    return (torch.empty(experts + 1, dtype=torch.int32, device=dev),
            torch.empty(tokens * top_k, dtype=torch.int32, device=dev),
            torch.empty((tokens, top_k), dtype=torch.int32, device=dev))


def muon_route_forward(logits, cfg: RouteConfig, bias=None, mask=None, plan: bool = True,
                       stream=None) -> Route:
    """Experts and weights of every token from CUDA logits [tokens, experts]
    (f32 or bf16), and their rows in expert order unless `plan` is false.
    bias: f32 [experts], seen by the choice only.  mask: bool or uint8
    [tokens], tokens to leave out are false."""
    import torch
    if stream is not None:
        with _as_current(stream):
            return muon_route_forward(logits, cfg, bias, mask, plan)
    ptr, stride, code = _rows(logits, "logits", cfg.experts)
    tokens, k, dev = logits.shape[0], cfg.top_k, logits.device
    idx = torch.empty((tokens, k), dtype=torch.int32, device=dev)
    weights = torch.empty((tokens, k), dtype=torch.float32, device=dev)
    off = src = pos = op = sp = pp = None
    if plan:
        off, src, pos = _plan_tensors(dev, tokens, k, cfg.experts)
        op, sp, pp = off.data_ptr(), src.data_ptr(), pos.data_ptr()
    b = _dense(bias, "bias", (cfg.experts,), torch.float32) if bias is not None else None
    m = None
    if mask is not None:
        m = _dense(mask, "mask", (tokens,), torch.bool if mask.dtype == torch.bool else torch.uint8)
    check(load().muon_route_forward(cfg, ptr, code, stride, tokens, b, m, idx.data_ptr(),
                                    weights.data_ptr(), op, sp, pp, _current_handle()),
          "muon_route_forward")
    return Route(idx, weights, off, src, pos)


def muon_route_plan(idx, experts: int, stream=None):
    """(offsets, src, pos) of int32 CUDA idx [tokens, top_k]: the pairs' rows in expert order."""
    import torch
    if stream is not None:
        with _as_current(stream):
            return muon_route_plan(idx, experts)
    tokens, top_k = idx.shape
    p = _dense(idx, "idx", (tokens, top_k), torch.int32)
    off, src, pos = _plan_tensors(idx.device, tokens, top_k, experts)
    check(load().muon_route_plan(p, tokens, top_k, experts, off.data_ptr(), src.data_ptr(),
                                 pos.data_ptr(), _current_handle()), "muon_route_plan")
    return off, src, pos


def muon_route_backward(logits, cfg: RouteConfig, idx, dweights, dlogits=None, stream=None):
    """Gradient of the routing weights with respect to the logits (their dtype)."""
    import torch
    if stream is not None:
        with _as_current(stream):
            return muon_route_backward(logits, cfg, idx, dweights, dlogits)
    ptr, stride, code = _rows(logits, "logits", cfg.experts)
    tokens = logits.shape[0]
    if dlogits is None:
        dlogits = _like(logits)
    dptr, dstride, dcode = _rows(dlogits, "dlogits", cfg.experts, tokens)
    if dcode != code:
        raise ValueError("dlogits must have the logits' dtype")
    i = _dense(idx, "idx", (tokens, cfg.top_k), torch.int32)
    w = _dense(dweights, "dweights", (tokens, cfg.top_k), torch.float32)
    check(load().muon_route_backward(cfg, ptr, code, stride, tokens, i, w, dptr, dstride,
                                     _current_handle()), "muon_route_backward")
    return dlogits


def _experts_args(x, w_in, w_out, route: Route):
    import torch
    if w_out.dim() != 3:
        raise ValueError("w_out must be [experts, hidden, inner]")
    experts, hidden, inner = w_out.shape
    bf16, i32 = torch.bfloat16, torch.int32
    if x.dtype != bf16:
        raise TypeError(f"x must be bfloat16, got {x.dtype}")
    ptr, stride, _ = _rows(x, "x", hidden)
    tokens, top_k = x.shape[0], route.weights.shape[1]
    if route.offsets is None:
        raise ValueError("the routing has no plan")
    return Experts(
        tokens, hidden, inner, experts, top_k, ptr, stride,
        _dense(w_in, "w_in", (experts, 2 * inner, hidden), bf16),
        _dense(w_out, "w_out", (experts, hidden, inner), bf16),
        _dense(route.weights, "weights", (tokens, top_k), torch.float32),
        _dense(route.offsets, "offsets", (experts + 1,), i32),
        _dense(route.src, "src", (tokens * top_k,), i32),
        _dense(route.pos, "pos", (tokens, top_k), i32))


def muon_experts_forward(x, w_in, w_out, route: Route, save: bool = False, out=None, stream=None):
    """(out, gu): out[t] = sum over slots of weight * W_out silu(W_gate x) (W_up x)
    for bf16 CUDA x [tokens, hidden], w_in [experts, 2 * inner, hidden] (gate
    rows, then up rows), w_out [experts, hidden, inner].  gu, what
    muon_experts_backward needs, is None unless `save`."""
    import torch
    if stream is not None:
        with _as_current(stream):
            return muon_experts_forward(x, w_in, w_out, route, save, out)
    a = _experts_args(x, w_in, w_out, route)
    if out is None:
        out = _like(x)
    elif out.dtype != torch.bfloat16:
        raise TypeError(f"out must be bfloat16, got {out.dtype}")
    optr, ostride, _ = _rows(out, "out", a.hidden, a.tokens)
    gu = None
    if save:
        gu = torch.empty((a.tokens * a.top_k, 2 * a.inner), dtype=torch.bfloat16, device=x.device)
    check(load().muon_experts_forward(a, optr, ostride,
                                      gu.data_ptr() if save else None, _current_handle()),
          "muon_experts_forward")
    return out, gu


def muon_experts_backward(dout, x, w_in, w_out, route: Route, gu, dw_dtype=None, dx=None, dw_in=None,
                          dw_out=None, want_dx: bool = True, want_dw: bool = True, stream=None):
    """(dx, dw_in, dw_out, dweights) of muon_experts_forward.  The weights'
    gradients have dtype `dw_dtype` (f32 by default, or bf16) and the weights'
    shapes, as muon_step_grouped takes them; dweights is f32 [tokens, top_k]
    for muon_route_backward."""
    import torch
    if stream is not None:
        with _as_current(stream):
            return muon_experts_backward(dout, x, w_in, w_out, route, gu, dw_dtype, dx, dw_in, dw_out, want_dx,
                                         want_dw)
    a = _experts_args(x, w_in, w_out, route)
    bf16 = torch.bfloat16
    if dout.dtype != bf16 or (dx is not None and dx.dtype != bf16):
        raise TypeError("dout and dx must be bfloat16")
    dptr, dstride, _ = _rows(dout, "dout", a.hidden, a.tokens)
    g = _dense(gu, "gu", (a.tokens * a.top_k, 2 * a.inner), bf16)
    xptr, xstride = None, a.hidden
    if dx is None and want_dx:
        dx = _like(x)
    if dx is not None:
        xptr, xstride, _ = _rows(dx, "dx", a.hidden, a.tokens)
    if want_dw:
        dw_dtype = dw_dtype or (dw_in.dtype if dw_in is not None else torch.float32)
        if dw_in is None:
            dw_in = torch.empty_like(w_in, dtype=dw_dtype)
        if dw_out is None:
            dw_out = torch.empty_like(w_out, dtype=dw_dtype)
    code = _code(dw_dtype) if dw_dtype is not None else MUON_F32
    dweights = torch.empty((a.tokens, a.top_k), dtype=torch.float32, device=x.device)
    check(load().muon_experts_backward(
        a, dptr, dstride, g, xptr, xstride,
        _dense(dw_in, "dw_in", w_in.shape, dw_dtype) if want_dw else None,
        _dense(dw_out, "dw_out", w_out.shape, dw_dtype) if want_dw else None,
        code, dweights.data_ptr(), _current_handle()), "muon_experts_backward")
    return dx, dw_in, dw_out, dweights
