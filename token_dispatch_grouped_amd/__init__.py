"""MI355X (gfx950) MoE expert layer on one rank's share: Python binding.

Thin ctypes marshalling over libmoe.so (include/moe.h). Every step of the path
runs in the library's HIP kernels; PyTorch only provides device memory and the
current stream. With its `stream` argument, a call runs on that stream and what
it allocates (results, workspaces) belongs to it. There is no fallback: if the
library is missing, importing the binding works only for introspection
(`lib_path`, `declared_symbols`) and every compute call raises.

Every wrapper checks the dtype and shape of each tensor it is given (inputs and
caller-provided outputs alike) against the sizes of the call before anything
reaches the library: a wrong dtype raises TypeError, a wrong shape ValueError.

Debug mode (`set_debug(True)`, or MOE_DEBUG=1 in the environment at import)
loads libmoe_debug.so instead, whose dispatch also counts the expert ids outside
[0, E) on the device; `dispatch` then waits for its stream and raises ValueError
when there are any. That wait makes the dispatch synchronous, so debug mode is
for finding bad input, not for graph capture or timing.
"""
from __future__ import annotations

import array
import ctypes
import os
import re
from dataclasses import dataclass

_PKG = os.path.dirname(os.path.abspath(__file__))
_ROOT = os.path.dirname(_PKG)
lib_path = os.path.join(_PKG, "libmoe.so")
debug_lib_path = os.path.join(_PKG, "libmoe_debug.so")
header_path = os.path.join(_ROOT, "include", "moe.h")
_SIZE_MAX = ctypes.c_size_t(-1).value

MOE_OK, MOE_EINVAL, MOE_EUNSUPPORTED, MOE_EHIP = 0, 1, 2, 3
MOE_F32, MOE_BF16 = 0, 1


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


class moe_shape(ctypes.Structure):
    _fields_ = [
        ("T", ctypes.c_int64),
        ("d", ctypes.c_int32),
        ("d_ff", ctypes.c_int32),
        ("E", ctypes.c_int32),
        ("k", ctypes.c_int32),
        ("e_begin", ctypes.c_int32),
        ("e_end", ctypes.c_int32),
    ]


class moe_tensor(ctypes.Structure):
    _fields_ = [
        ("data", ctypes.c_void_p),
        ("numel", ctypes.c_int64),
        ("dt", ctypes.c_int),
    ]


_libs: dict = {}
_debug = os.environ.get("MOE_DEBUG", "") not in ("", "0")


def set_debug(enabled: bool) -> None:
    """Use libmoe_debug.so (True) or libmoe.so (False) for the calls that follow."""
    global _debug
    _debug = bool(enabled)


def debug_enabled() -> bool:
    return _debug


def _load():
    path = debug_lib_path if _debug else lib_path
    if path not in _libs:
        if not os.path.exists(path):
            raise ImportError(
                f"{path} is missing: build it with token_dispatch_grouped_amd.build.build() "
                "(there is no fallback path)")
        lib = ctypes.CDLL(path)
        P, S, I32, I64, SZ = ctypes.c_void_p, ctypes.POINTER(moe_shape), ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        sigs = {
            "moe_status_string": (ctypes.c_char_p, [ctypes.c_int]),
            "moe_expert_range": (ctypes.c_int, [I32, I32, I32, ctypes.POINTER(I32), ctypes.POINTER(I32)]),
            "moe_route_topk": (ctypes.c_int, [S, P, P, P, P]),
            "moe_dispatch_workspace_bytes": (SZ, [S]),
            "moe_dispatch_debug_word_offset": (SZ, []),
            "moe_dispatch": (ctypes.c_int, [S, ctypes.c_int, P, P, P, P, P, P, P, P, P]),
            "moe_dispatch_indices": (ctypes.c_int, [S, P, P, P, P, P, P, P]),
            "moe_dispatch_indices_noalloc": (ctypes.c_int, [S, P, P, P, P, P, P]),
            "moe_grouped_gemm_gather": (ctypes.c_int, [S, ctypes.c_int, P, P, P, P, P, P, P, P, P]),
            "moe_grouped_gemm_workspace_bytes": (SZ, [S, ctypes.c_int]),
            "moe_grouped_gemm": (ctypes.c_int, [S, ctypes.c_int, P, P, P, P, P, P, P, P]),
            "moe_combine": (ctypes.c_int, [S, ctypes.c_int, P, P, P, P, P]),
            "moe_combine_backward": (ctypes.c_int, [S, ctypes.c_int, P, P, P, P, P, P, P]),
            "moe_grouped_gemm_backward_workspace_bytes": (SZ, [S, ctypes.c_int]),
            "moe_grouped_gemm_backward": (ctypes.c_int, [S, ctypes.c_int, P, P, P, P, P, P, P, P, P, P, P, P]),
            "moe_dispatch_backward": (ctypes.c_int, [S, ctypes.c_int, P, P, P, P]),
            "moe_route_topk_backward": (ctypes.c_int, [S, P, P, P, P, P]),
            "moe_grouped_gemm_gather_save": (ctypes.c_int, [S, ctypes.c_int, P, P, P, P, P, P, P, P, P, P]),
            "moe_grouped_gemm_backward_saved": (ctypes.c_int,
                                                [S, ctypes.c_int, P, P, P, P, P, P, P, P, P, P, P, P, P]),
            "moe_layer_norm": (ctypes.c_int, [S, ctypes.c_int, P, P, ctypes.c_int, P, P, ctypes.c_float, P, P, P, P, P]),
            "moe_layer_norm_backward_workspace_bytes": (SZ, [S]),
            "moe_layer_norm_backward": (ctypes.c_int,
                                        [S, ctypes.c_int, P, P, ctypes.c_int, P, P, P, P, P, P, P, P, P]),
            "moe_quantize_experts": (ctypes.c_int, [S, ctypes.c_int, P, P, P, P, P, P, P]),
            "moe_grouped_gemm_int8_workspace_bytes": (SZ, [S]),
            "moe_grouped_gemm_int8": (ctypes.c_int, [S, ctypes.c_int, P, P, P, P, P, P, P, P, P, P]),
            "moe_grad_norm_workspace_bytes": (SZ, [I32]),
            "moe_grad_norm": (ctypes.c_int, [P, I32, P, P, P]),
            "moe_clip_grads": (ctypes.c_int, [P, P, I32, P, ctypes.c_float, P]),
            "moe_clip_grad_norm": (ctypes.c_int, [P, P, I32, ctypes.c_float, P, P, P]),
        }
        for name, (res, args) in sigs.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _libs[path] = lib
    return _libs[path]


def lib():
    """The loaded ctypes library (raises ImportError when it is not built)."""
    return _load()


def declared_symbols() -> list[str]:
    """Function names declared in include/moe.h."""
    with open(header_path) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(moe_[a-z_0-9]+)\s*\(", text)))


def status_string(status: int) -> str:
    try:
        return _load().moe_status_string(int(status)).decode()
    except ImportError:
        return f"status {status}"


def _check(status: int, where: str) -> None:
    if status != MOE_OK:
        raise MoeError(status, where)


# ----------------------------------------------------------------------------- torch helpers

_TORCH = None
_CODES: dict = {}  # torch dtype -> moe_dtype


def _torch():
    """torch, imported by the first call that needs it."""
    global _TORCH
    if _TORCH is None:
        import torch
        _CODES.update({torch.float32: MOE_F32, torch.bfloat16: MOE_BF16})
        _TORCH = torch  # last: another thread's call that finds it finds the table filled
    return _TORCH


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _dtype_code(t) -> int:
    torch = _torch()
    if t.dtype == torch.bfloat16:
        return MOE_BF16
    if t.dtype == torch.float32:
        return MOE_F32
    raise TypeError(f"unsupported dtype {t.dtype}; expected bfloat16 or float32")


def _dev(*ts):
    for t in ts:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("every tensor must be on the GPU")
        if not t.is_contiguous():
            raise ValueError("every tensor must be contiguous (row-major)")


def _want(t, name: str, dtype=None, shape=None, min_rows=None):
    """Check one tensor argument: its dtype (TypeError) and its shape (ValueError).
    `shape` is the exact shape; with `min_rows`, shape[0] may be any count of at
    least min_rows (a buffer sized for more rows than this call's N_max)."""
    if t is None:
        raise ValueError(f"{name} is required")
    if dtype is not None:
        allowed = dtype if isinstance(dtype, tuple) else (dtype,)
        if t.dtype not in allowed:
            want = " or ".join(str(a) for a in allowed)
            raise TypeError(f"{name} must be {want}, got {t.dtype}")
    if shape is not None:
        got = tuple(t.shape)
        if min_rows is not None:
            ok = len(got) == len(shape) and got[1:] == tuple(shape[1:]) and got[0] >= min_rows
            if not ok:
                raise ValueError(f"{name} must have shape [>= {min_rows}, {', '.join(map(str, shape[1:]))}], "
                                 f"got {list(got)}")
        elif got != tuple(shape):
            raise ValueError(f"{name} must have shape {list(shape)}, got {list(got)}")


class _SameStream:
    """The caller's own stream."""

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        return False

    def give(self, *ts):
        pass


class _OnStream:
    """Another stream made current: what is allocated inside belongs to it."""

    def __init__(self, stream, caller):
        self._ctx, self._caller = _torch().cuda.stream(stream), caller

    def __enter__(self):
        self._ctx.__enter__()
        return self

    def __exit__(self, *exc):
        return self._ctx.__exit__(*exc)

    def give(self, *ts):
        """What the call returns: once the caller's stream has waited, it may use these
        and free them, before the uses have run."""
        for t in ts:
            if t is not None and self._caller is not None:
                t.record_stream(self._caller)


_SAME = _SameStream()


def _place(stream, ts):
    """Where a call on the GPU tensors `ts` runs: (stream handle, context), on
    `stream` or their GPU's current stream. The context makes both the GPU and the
    stream current, so that memory allocated inside belongs to that stream. The
    tensors that the call is given are recorded on a stream other than the current
    one, so that freeing them early does not hand their memory out while it runs."""
    torch = _torch()
    devices = set(map(torch.Tensor.get_device, ts))
    index = devices.pop()
    if devices or index < 0:
        _dev(*ts)
        raise ValueError(f"every tensor must be on one GPU, got GPUs {sorted({index, *devices})}")
    if index == torch.cuda.current_device():
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # without building a Stream object
        here = raw(index) if raw else torch.cuda.current_stream(index).cuda_stream
        if stream is None or (stream.cuda_stream == here and stream.device_index == index):
            return here, _SAME
    dev = ts[0].device
    current = torch.cuda.current_stream(dev)
    if stream is None or stream == current:
        return current.cuda_stream, _OnStream(current, None)
    if stream.device != dev:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {dev}")
    for t in ts:
        t.record_stream(stream)
    return stream.cuda_stream, _OnStream(stream, current)


def _dense(stream, ts):
    """_place after checking that every tensor (None: not given) is dense and on the GPU."""
    ts = [t for t in ts if t is not None]
    if not all(map(_torch().Tensor.is_contiguous, ts)):
        _dev(*ts)
    return _place(stream, ts)


def _ready(stream, vectors, others=()):
    """_dense after checking that `vectors`, which move in 16-byte pieces, start at such
    a boundary."""
    ts = [t for t in vectors if t is not None]
    low = 0
    for t in ts:
        low |= t.data_ptr()
    placed = _dense(stream, [*ts, *others])
    if low & 15:
        bad = next(t for t in ts if t.data_ptr() & 15)
        raise ValueError(f"a tensor of shape {list(bad.shape)} does not start at a 16-byte boundary")
    return placed


def _addr(t):
    return None if t is None else t.data_ptr()


def _act_dtypes():
    torch = _torch()
    return (torch.bfloat16, torch.float32)


def _n_max(T: int, k: int, e_begin: int, e_end: int) -> int:
    return T * min(k, e_end - e_begin)


def _expert_weights(w_gate_up, w_down, dtype, d: int, e_begin: int, e_end: int) -> int:
    """Checks the local experts' weights against the activations; returns d_ff."""
    _want(w_down, "w_down", dtype)
    if w_down.dim() != 3:
        raise ValueError(f"w_down must be [E_loc, d_ff, d], got {list(w_down.shape)}")
    e_loc, d_ff = int(w_down.shape[0]), int(w_down.shape[1])
    if e_loc != e_end - e_begin:
        raise ValueError(f"expert weights must hold exactly the {e_end - e_begin} local experts, got {e_loc}")
    _want(w_down, "w_down", dtype, (e_loc, d_ff, d))
    _want(w_gate_up, "w_gate_up", dtype, (e_loc, d, 2 * d_ff))
    return d_ff


def _range(E: int, k: int, e_begin: int, e_end: int) -> None:
    if not 1 <= k <= E:
        raise ValueError(f"need 1 <= k <= E, got k={k}, E={E}")
    if not 0 <= e_begin < e_end <= E:
        raise ValueError(f"local experts [{e_begin}, {e_end}) must be a non-empty range inside [0, {E})")


def shape(T, d, d_ff, E, k, e_begin, e_end) -> moe_shape:
    """The sizes as the library takes them: T in 64 bits, the others in 32 (ctypes by
    itself would take a size modulo 2^32)."""
    if max(d, d_ff, E, k, e_begin, e_end) > 0x7FFFFFFF or min(d, d_ff, E, k, e_begin, e_end) < -0x80000000:
        raise ValueError(f"sizes must fit 32 bits, got {dict(d=d, d_ff=d_ff, E=E, k=k, e_begin=e_begin, e_end=e_end)}")
    if not -(1 << 63) <= T < 1 << 63:
        raise ValueError(f"T must fit 64 bits, got {T}")
    return moe_shape(int(T), int(d), int(d_ff), int(E), int(k), int(e_begin), int(e_end))


def expert_range(E: int, ep: int, rank: int) -> tuple[int, int]:
    lo, hi = ctypes.c_int32(), ctypes.c_int32()
    _check(_load().moe_expert_range(E, ep, rank, ctypes.byref(lo), ctypes.byref(hi)), "moe_expert_range")
    return lo.value, hi.value


# ----------------------------------------------------------------------------- the four steps

def route_topk(logits, k: int, topk_idx=None, topk_w=None, stream=None):
    """logits [T, E] fp32 -> (topk_idx [T, k] int32, topk_w [T, k] fp32)."""
    torch = _torch()
    _want(logits, "logits", torch.float32)
    if logits.dim() != 2:
        raise ValueError(f"logits must be [T, E], got {list(logits.shape)}")
    T, E = (int(v) for v in logits.shape)
    if not 1 <= k <= E:
        raise ValueError(f"need 1 <= k <= E, got k={k}, E={E}")
    if topk_idx is not None:
        _want(topk_idx, "topk_idx", torch.int32, (T, k))
    if topk_w is not None:
        _want(topk_w, "topk_w", torch.float32, (T, k))
    st, ctx = _dense(stream, (logits, topk_idx, topk_w))
    s = shape(T, 8, 8, E, k, 0, E)
    with ctx:
        if topk_idx is None:
            topk_idx = torch.empty((T, k), dtype=torch.int32, device=logits.device)
        if topk_w is None:
            topk_w = torch.empty((T, k), dtype=torch.float32, device=logits.device)
        ctx.give(topk_idx, topk_w)
        _check(_load().moe_route_topk(ctypes.byref(s), _ptr(logits), _ptr(topk_idx), _ptr(topk_w), st),
               "moe_route_topk")
    return topk_idx, topk_w


@dataclass
class Dispatch:
    counts: object
    offsets: object
    perm: object
    pair_pos: object
    x_perm: object
    workspace: object


def dispatch_workspace_bytes(T: int, k: int, E: int) -> int:
    s = shape(T, 8, 8, E, k, 0, E)
    return int(_load().moe_dispatch_workspace_bytes(ctypes.byref(s)))


def dispatch_alloc(x, k: int, E: int, e_begin: int, e_end: int, gather: bool = True) -> Dispatch:
    """Allocate every dispatch output (sized on the host, no device read); without
    `gather` there is no x_perm (the fused path reads rows straight from x)."""
    torch = _torch()
    T, d = x.shape
    n_max = _n_max(T, k, e_begin, e_end)
    ws_bytes = dispatch_workspace_bytes(T, k, E)
    dev = x.device
    return Dispatch(
        counts=torch.empty(E, dtype=torch.int32, device=dev),
        offsets=torch.empty(E + 1, dtype=torch.int32, device=dev),
        perm=torch.empty(T * k, dtype=torch.int32, device=dev),
        pair_pos=torch.empty(T * k, dtype=torch.int32, device=dev),
        x_perm=torch.empty((n_max, d), dtype=x.dtype, device=dev) if gather else None,
        workspace=torch.empty(max(1, ws_bytes), dtype=torch.uint8, device=dev),
    )


def _check_dispatch(out: Dispatch, x, T: int, k: int, E: int, n_max: int, gather: bool) -> None:
    torch = _torch()
    _want(out.counts, "counts", torch.int32, (E,))
    _want(out.offsets, "offsets", torch.int32, (E + 1,))
    _want(out.perm, "perm", torch.int32, (T * k,))
    _want(out.pair_pos, "pair_pos", torch.int32, (T * k,))
    if gather:
        if out.x_perm is None:
            raise ValueError("this Dispatch has no x_perm; allocate it with gather=True")
        _want(out.x_perm, "x_perm", x.dtype, (n_max, x.shape[1]), min_rows=n_max)
    _want(out.workspace, "workspace", torch.uint8)
    need = dispatch_workspace_bytes(T, k, E)
    if out.workspace.numel() < need:
        raise ValueError(f"workspace must hold at least {need} bytes, got {out.workspace.numel()}")


def _debug_word(out: Dispatch, E: int) -> None:
    """Debug mode: wait for the dispatch on the current stream, then refuse ids outside [0, E)."""
    torch = _torch()
    off = int(_load().moe_dispatch_debug_word_offset())
    if off == _SIZE_MAX:
        return
    torch.cuda.current_stream().synchronize()
    bad = int(out.workspace[off:off + 4].view(torch.int32).item())
    if bad:
        raise ValueError(f"moe_dispatch: topk_idx holds {bad} expert id(s) outside [0, {E})")


def dispatch(x, topk_idx, E: int, e_begin: int, e_end: int, out: Dispatch | None = None, stream=None,
             gather: bool = True) -> Dispatch:
    """Histogram, offsets, stable permutation and (with `gather`) the local-row
    gather into x_perm; without it, moe_dispatch_indices (no x_perm)."""
    torch = _torch()
    _want(x, "x", _act_dtypes())
    if x.dim() != 2:
        raise ValueError(f"x must be [T, d], got {list(x.shape)}")
    T, d = (int(v) for v in x.shape)
    _want(topk_idx, "topk_idx", torch.int32)
    if topk_idx.dim() != 2 or topk_idx.shape[0] != T:
        raise ValueError(f"topk_idx must be [T={T}, k], got {list(topk_idx.shape)}")
    k = int(topk_idx.shape[1])
    _range(E, k, e_begin, e_end)
    n_max = _n_max(T, k, e_begin, e_end)
    if out is not None:
        _check_dispatch(out, x, T, k, E, n_max, gather)
    st, ctx = _dense(stream, (x, topk_idx) if out is None else
                     (x, topk_idx, out.counts, out.offsets, out.perm, out.pair_pos, out.x_perm if gather else None,
                      out.workspace))
    s = shape(T, d, 8, E, k, e_begin, e_end)
    with ctx:
        if out is None:
            out = dispatch_alloc(x, k, E, e_begin, e_end, gather=gather)
        ctx.give(out.counts, out.offsets, out.perm, out.pair_pos, out.x_perm, out.workspace)
        if gather:
            _check(_load().moe_dispatch(ctypes.byref(s), _dtype_code(x), _ptr(x), _ptr(topk_idx), _ptr(out.counts),
                                        _ptr(out.offsets), _ptr(out.perm), _ptr(out.pair_pos), _ptr(out.x_perm),
                                        _ptr(out.workspace), st), "moe_dispatch")
        else:
            _check(_load().moe_dispatch_indices(ctypes.byref(s), _ptr(topk_idx), _ptr(out.counts), _ptr(out.offsets),
                                                _ptr(out.perm), _ptr(out.pair_pos), _ptr(out.workspace), st),
                   "moe_dispatch_indices")
        if _debug:
            _debug_word(out, E)
    return out


def dispatch_indices_noalloc(topk_idx, E: int, e_begin: int, e_end: int, counts, offsets, perm, pair_pos,
                             stream=None) -> None:
    """moe_dispatch_indices_noalloc: the dispatch's indices into caller-provided
    buffers, with the library's per-GPU array as workspace (nothing allocated;
    calls that overlap on one GPU race)."""
    torch = _torch()
    _want(topk_idx, "topk_idx", torch.int32)
    if topk_idx.dim() != 2:
        raise ValueError(f"topk_idx must be [T, k], got {list(topk_idx.shape)}")
    T, k = (int(v) for v in topk_idx.shape)
    _range(E, k, e_begin, e_end)
    _want(counts, "counts", torch.int32, (E,))
    _want(offsets, "offsets", torch.int32, (E + 1,))
    _want(perm, "perm", torch.int32, (T * k,))
    _want(pair_pos, "pair_pos", torch.int32, (T * k,))
    st, ctx = _dense(stream, (topk_idx, counts, offsets, perm, pair_pos))
    s = shape(T, 8, 8, E, k, e_begin, e_end)
    with ctx:
        _check(_load().moe_dispatch_indices_noalloc(ctypes.byref(s), _ptr(topk_idx), _ptr(counts), _ptr(offsets),
                                                    _ptr(perm), _ptr(pair_pos), st), "moe_dispatch_indices_noalloc")


def _check_gemm_outputs(h, y, n_max: int, d: int, d_ff: int, dtype) -> None:
    if h is not None:
        _want(h, "h", dtype, (n_max, d_ff), min_rows=n_max)
    if y is not None:
        _want(y, "y", dtype, (n_max, d), min_rows=n_max)


def _gemm_outputs(h, y, n_max: int, d: int, d_ff: int, dtype, device):
    torch = _torch()
    if h is None:
        h = torch.empty((n_max, d_ff), dtype=dtype, device=device)
    if y is None:
        y = torch.empty((n_max, d), dtype=dtype, device=device)
    return h, y


def grouped_gemm(x_perm, offsets, w_gate_up, w_down, T: int, k: int, E: int, e_begin: int, e_end: int,
                 h=None, y=None, stream=None):
    """Local experts' SwiGLU FFN: returns (h [N_max, d_ff], y [N_max, d])."""
    torch = _torch()
    _range(E, k, e_begin, e_end)
    n_max = _n_max(T, k, e_begin, e_end)
    _want(x_perm, "x_perm", _act_dtypes())
    if x_perm.dim() != 2:
        raise ValueError(f"x_perm must be [N_max, d], got {list(x_perm.shape)}")
    d = int(x_perm.shape[1])
    _want(x_perm, "x_perm", x_perm.dtype, (n_max, d), min_rows=n_max)
    _want(offsets, "offsets", torch.int32, (E + 1,))
    d_ff = _expert_weights(w_gate_up, w_down, x_perm.dtype, d, e_begin, e_end)
    _check_gemm_outputs(h, y, n_max, d, d_ff, x_perm.dtype)
    st, ctx = _dense(stream, (x_perm, offsets, w_gate_up, w_down, h, y))
    s = shape(T, d, d_ff, E, k, e_begin, e_end)
    dt = _dtype_code(x_perm)
    ws_bytes = _load().moe_grouped_gemm_workspace_bytes(ctypes.byref(s), dt)
    with ctx:
        h, y = _gemm_outputs(h, y, n_max, d, d_ff, x_perm.dtype, x_perm.device)
        ctx.give(h, y)
        ws = torch.empty(ws_bytes, dtype=torch.uint8, device=x_perm.device) if ws_bytes else None
        _check(_load().moe_grouped_gemm(ctypes.byref(s), dt, _ptr(x_perm), _ptr(offsets), _ptr(w_gate_up),
                                        _ptr(w_down), _ptr(h), _ptr(y), _ptr(ws), st), "moe_grouped_gemm")
    return h, y


def grouped_gemm_gather(x, perm, offsets, w_gate_up, w_down, k: int, E: int, e_begin: int, e_end: int,
                        h=None, y=None, stream=None, gu=None):
    """grouped_gemm reading each local row straight from x through perm (no
    x_perm): returns (h [N_max, d_ff], y [N_max, d]), bit-identical to
    dispatch + grouped_gemm. With gu (a [N_max, 2*d_ff] tensor) the gate/up
    pre-activations are kept there as well (moe_grouped_gemm_gather_save)."""
    torch = _torch()
    _range(E, k, e_begin, e_end)
    _want(x, "x", _act_dtypes())
    if x.dim() != 2:
        raise ValueError(f"x must be [T, d], got {list(x.shape)}")
    T, d = (int(v) for v in x.shape)
    n_max = _n_max(T, k, e_begin, e_end)
    _want(perm, "perm", torch.int32, (T * k,))
    _want(offsets, "offsets", torch.int32, (E + 1,))
    d_ff = _expert_weights(w_gate_up, w_down, x.dtype, d, e_begin, e_end)
    _check_gemm_outputs(h, y, n_max, d, d_ff, x.dtype)
    if gu is not None:
        _want(gu, "gu", x.dtype, (n_max, 2 * d_ff), min_rows=n_max)
    st, ctx = _dense(stream, (x, perm, offsets, w_gate_up, w_down, h, y, gu))
    s = shape(T, d, d_ff, E, k, e_begin, e_end)
    dt = _dtype_code(x)
    ws_bytes = _load().moe_grouped_gemm_workspace_bytes(ctypes.byref(s), dt)
    with ctx:
        h, y = _gemm_outputs(h, y, n_max, d, d_ff, x.dtype, x.device)
        ctx.give(h, y)
        ws = torch.empty(ws_bytes, dtype=torch.uint8, device=x.device) if ws_bytes else None
        if gu is None:
            _check(_load().moe_grouped_gemm_gather(ctypes.byref(s), dt, _ptr(x), _ptr(perm), _ptr(offsets),
                                                   _ptr(w_gate_up), _ptr(w_down), _ptr(h), _ptr(y), _ptr(ws), st),
                   "moe_grouped_gemm_gather")
        else:
            _check(_load().moe_grouped_gemm_gather_save(ctypes.byref(s), dt, _ptr(x), _ptr(perm), _ptr(offsets),
                                                        _ptr(w_gate_up), _ptr(w_down), _ptr(h), _ptr(y), _ptr(gu),
                                                        _ptr(ws), st), "moe_grouped_gemm_gather_save")
    return h, y


def combine(y, pair_pos, topk_w, T: int, k: int, E: int, e_begin: int, e_end: int, out=None, stream=None):
    """out[t] = sum_j topk_w[t, j] * y[pair_pos[t*k + j]] over local pairs; [T, d]."""
    torch = _torch()
    _range(E, k, e_begin, e_end)
    n_max = _n_max(T, k, e_begin, e_end)
    _want(y, "y", _act_dtypes())
    if y.dim() != 2:
        raise ValueError(f"y must be [N_max, d], got {list(y.shape)}")
    d = int(y.shape[1])
    _want(y, "y", y.dtype, (n_max, d), min_rows=n_max)
    _want(pair_pos, "pair_pos", torch.int32, (T * k,))
    _want(topk_w, "topk_w", torch.float32, (T, k))
    if out is not None:
        _want(out, "out", y.dtype, (T, d))
    st, ctx = _dense(stream, (y, pair_pos, topk_w, out))
    s = shape(T, d, 8, E, k, e_begin, e_end)
    with ctx:
        if out is None:
            out = torch.empty((T, d), dtype=y.dtype, device=y.device)
        ctx.give(out)
        _check(_load().moe_combine(ctypes.byref(s), _dtype_code(y), _ptr(y), _ptr(pair_pos), _ptr(topk_w),
                                   _ptr(out), st), "moe_combine")
    return out


def layer(x, logits, w_gate_up, w_down, k: int, e_begin: int, e_end: int, stream=None, fused: bool = False,
          save: bool = False, norm=None) -> dict:
    """The whole forward of one rank: route -> dispatch -> grouped GEMM -> combine.
    With `fused`, the dispatch writes indices only and the GEMM gathers the rows.
    With `save` (fused path), the gate/up pre-activations are kept in the result
    as "gu", for layer_backward to use instead of recomputing them.
    With `norm` = (weight, bias or None, eps), out is added to the residual x and
    normalised (layer_norm): the result has "sum" = x + out, "normed", "mean" and
    "rstd" as well. On a rank that holds a share of the experts, out is a partial
    sum over ranks: join the ranks' first and call layer_norm then."""
    torch = _torch()
    T = x.shape[0]
    if logits.dim() != 2 or logits.shape[0] != T:
        raise ValueError(f"logits must be [T={T}, E], got {list(logits.shape)}")
    E = logits.shape[1]
    if save and not fused:
        raise ValueError("save needs the fused path")
    _check_layer_norm_arg(norm, E, e_begin, e_end)
    idx, w = route_topk(logits, k, stream=stream)
    disp = dispatch(x, idx, E, e_begin, e_end, stream=stream, gather=not fused)
    gu = None
    if fused:
        if save:
            e_loc, d_ff = w_down.shape[0], w_down.shape[1]
            _, ctx = _dense(stream, (x,))
            with ctx:
                gu = torch.empty((T * min(k, e_loc), 2 * d_ff), dtype=x.dtype, device=x.device)
                ctx.give(gu)
        h, y = grouped_gemm_gather(x, disp.perm, disp.offsets, w_gate_up, w_down, k, E, e_begin, e_end,
                                   stream=stream, gu=gu)
    else:
        h, y = grouped_gemm(disp.x_perm, disp.offsets, w_gate_up, w_down, T, k, E, e_begin, e_end, stream=stream)
    out = combine(y, disp.pair_pos, w, T, k, E, e_begin, e_end, stream=stream)
    res = dict(idx=idx, w=w, counts=disp.counts, offsets=disp.offsets, perm=disp.perm,
               pair_pos=disp.pair_pos, x_perm=disp.x_perm, h=h, y=y, out=out, gu=gu)
    return _with_norm(res, x, E, e_begin, e_end, norm, stream)


def _check_layer_norm_arg(norm, E: int, e_begin: int, e_end: int):
    if norm is None:
        return
    if len(norm) != 3:
        raise ValueError("norm must be (weight, bias or None, eps)")
    if (e_begin, e_end) != (0, E):
        raise ValueError(f"norm needs the whole layer output; experts [{e_begin}, {e_end}) of {E} give a partial sum")


def _with_norm(res: dict, x, E: int, e_begin: int, e_end: int, norm, stream) -> dict:
    if norm is not None:
        weight, bias, eps = norm
        res["normed"], res["sum"], res["mean"], res["rstd"] = layer_norm(res["out"], weight, bias, eps, residual=x,
                                                                         stream=stream)
    return res


# ----------------------------------------------------------------------------- backward

def combine_backward(d_out, y, pair_pos, topk_w, T: int, k: int, E: int, e_begin: int, e_end: int,
                     d_y=None, d_topk_w=None, stream=None):
    """(d_y [N_max, d], d_topk_w [T, k] fp32): the gradient of combine."""
    torch = _torch()
    _range(E, k, e_begin, e_end)
    n_max = _n_max(T, k, e_begin, e_end)
    _want(d_out, "d_out", _act_dtypes())
    if d_out.dim() != 2:
        raise ValueError(f"d_out must be [T, d], got {list(d_out.shape)}")
    d = int(d_out.shape[1])
    _want(d_out, "d_out", d_out.dtype, (T, d))
    _want(y, "y", d_out.dtype, (n_max, d), min_rows=n_max)
    _want(pair_pos, "pair_pos", torch.int32, (T * k,))
    _want(topk_w, "topk_w", torch.float32, (T, k))
    if d_y is not None:
        _want(d_y, "d_y", d_out.dtype, (n_max, d), min_rows=n_max)
    if d_topk_w is not None:
        _want(d_topk_w, "d_topk_w", torch.float32, (T, k))
    st, ctx = _dense(stream, (d_out, y, pair_pos, topk_w, d_y, d_topk_w))
    s = shape(T, d, 8, E, k, e_begin, e_end)
    with ctx:
        if d_y is None:
            d_y = torch.empty_like(y)
        if d_topk_w is None:
            d_topk_w = torch.empty((T, k), dtype=torch.float32, device=d_out.device)
        ctx.give(d_y, d_topk_w)
        _check(_load().moe_combine_backward(ctypes.byref(s), _dtype_code(d_out), _ptr(d_out), _ptr(y), _ptr(pair_pos),
                                            _ptr(topk_w), _ptr(d_y), _ptr(d_topk_w), st), "moe_combine_backward")
    return d_y, d_topk_w


def grouped_gemm_backward_workspace_bytes(T: int, d: int, d_ff: int, E: int, k: int, e_begin: int, e_end: int) -> int:
    s = shape(T, d, d_ff, E, k, e_begin, e_end)
    return int(_load().moe_grouped_gemm_backward_workspace_bytes(ctypes.byref(s), MOE_BF16))


def grouped_gemm_backward(x, perm, offsets, w_gate_up, w_down, h, d_y, k: int, E: int, e_begin: int, e_end: int,
                          d_x_perm=None, d_w_gate_up=None, d_w_down=None, workspace=None, stream=None, gu=None):
    """(d_x_perm, d_w_gate_up, d_w_down): the gradient of the grouped expert FFN.
    With gu (the pre-activations the saving forward kept) they are not
    recomputed (moe_grouped_gemm_backward_saved)."""
    torch = _torch()
    _range(E, k, e_begin, e_end)
    _want(x, "x", _act_dtypes())
    if x.dim() != 2:
        raise ValueError(f"x must be [T, d], got {list(x.shape)}")
    T, d = (int(v) for v in x.shape)
    n_max = _n_max(T, k, e_begin, e_end)
    dt_ = x.dtype
    _want(perm, "perm", torch.int32, (T * k,))
    _want(offsets, "offsets", torch.int32, (E + 1,))
    d_ff = _expert_weights(w_gate_up, w_down, dt_, d, e_begin, e_end)
    _want(h, "h", dt_, (n_max, d_ff), min_rows=n_max)
    _want(d_y, "d_y", dt_, (n_max, d), min_rows=n_max)
    if d_x_perm is not None:
        _want(d_x_perm, "d_x_perm", dt_, (n_max, d), min_rows=n_max)
    if d_w_gate_up is not None:
        _want(d_w_gate_up, "d_w_gate_up", dt_, tuple(w_gate_up.shape))
    if d_w_down is not None:
        _want(d_w_down, "d_w_down", dt_, tuple(w_down.shape))
    if gu is not None:
        _want(gu, "gu", dt_, (n_max, 2 * d_ff), min_rows=n_max)
    s = shape(T, d, d_ff, E, k, e_begin, e_end)
    dt = _dtype_code(x)
    ws_bytes = int(_load().moe_grouped_gemm_backward_workspace_bytes(ctypes.byref(s), dt))
    if workspace is not None:
        _want(workspace, "workspace", torch.uint8)
        if workspace.numel() < ws_bytes:
            raise ValueError(f"workspace must hold at least {ws_bytes} bytes, got {workspace.numel()}")
    st, ctx = _dense(stream, (x, perm, offsets, w_gate_up, w_down, h, d_y, d_x_perm, d_w_gate_up, d_w_down, gu,
                              workspace))
    with ctx:
        if d_x_perm is None:
            d_x_perm = torch.empty((n_max, d), dtype=dt_, device=x.device)
        if d_w_gate_up is None:
            d_w_gate_up = torch.empty_like(w_gate_up)
        if d_w_down is None:
            d_w_down = torch.empty_like(w_down)
        ctx.give(d_x_perm, d_w_gate_up, d_w_down)
        ws = workspace
        if ws is None:
            ws = torch.empty(ws_bytes, dtype=torch.uint8, device=x.device) if ws_bytes else None
        if gu is None:
            _check(_load().moe_grouped_gemm_backward(ctypes.byref(s), dt, _ptr(x), _ptr(perm), _ptr(offsets),
                                                     _ptr(w_gate_up), _ptr(w_down), _ptr(h), _ptr(d_y),
                                                     _ptr(d_x_perm), _ptr(d_w_gate_up), _ptr(d_w_down), _ptr(ws), st),
                   "moe_grouped_gemm_backward")
        else:
            _check(_load().moe_grouped_gemm_backward_saved(ctypes.byref(s), dt, _ptr(x), _ptr(perm), _ptr(offsets),
                                                           _ptr(w_gate_up), _ptr(w_down), _ptr(h), _ptr(gu),
                                                           _ptr(d_y), _ptr(d_x_perm), _ptr(d_w_gate_up),
                                                           _ptr(d_w_down), _ptr(ws), st),
                   "moe_grouped_gemm_backward_saved")
    return d_x_perm, d_w_gate_up, d_w_down


def dispatch_backward(d_x_perm, pair_pos, T: int, k: int, E: int, e_begin: int, e_end: int, d_x=None, stream=None):
    """d_x [T, d]: the gradient of the row gather."""
    torch = _torch()
    _range(E, k, e_begin, e_end)
    n_max = _n_max(T, k, e_begin, e_end)
    _want(d_x_perm, "d_x_perm", _act_dtypes())
    if d_x_perm.dim() != 2:
        raise ValueError(f"d_x_perm must be [N_max, d], got {list(d_x_perm.shape)}")
    d = int(d_x_perm.shape[1])
    _want(d_x_perm, "d_x_perm", d_x_perm.dtype, (n_max, d), min_rows=n_max)
    _want(pair_pos, "pair_pos", torch.int32, (T * k,))
    if d_x is not None:
        _want(d_x, "d_x", d_x_perm.dtype, (T, d))
    st, ctx = _dense(stream, (d_x_perm, pair_pos, d_x))
    s = shape(T, d, 8, E, k, e_begin, e_end)
    with ctx:
        if d_x is None:
            d_x = torch.empty((T, d), dtype=d_x_perm.dtype, device=d_x_perm.device)
        ctx.give(d_x)
        _check(_load().moe_dispatch_backward(ctypes.byref(s), _dtype_code(d_x_perm), _ptr(d_x_perm), _ptr(pair_pos),
                                             _ptr(d_x), st), "moe_dispatch_backward")
    return d_x


def route_topk_backward(topk_idx, topk_w, d_topk_w, E: int, d_logits=None, stream=None):
    """d_logits [T, E] fp32: the gradient of route_topk's weights w.r.t. the logits."""
    torch = _torch()
    _want(topk_idx, "topk_idx", torch.int32)
    if topk_idx.dim() != 2:
        raise ValueError(f"topk_idx must be [T, k], got {list(topk_idx.shape)}")
    T, k = (int(v) for v in topk_idx.shape)
    if not 1 <= k <= E:
        raise ValueError(f"need 1 <= k <= E, got k={k}, E={E}")
    _want(topk_w, "topk_w", torch.float32, (T, k))
    _want(d_topk_w, "d_topk_w", torch.float32, (T, k))
    if d_logits is not None:
        _want(d_logits, "d_logits", torch.float32, (T, E))
    st, ctx = _dense(stream, (topk_idx, topk_w, d_topk_w, d_logits))
    s = shape(T, 8, 8, E, k, 0, E)
    with ctx:
        if d_logits is None:
            d_logits = torch.empty((T, E), dtype=torch.float32, device=topk_idx.device)
        ctx.give(d_logits)
        _check(_load().moe_route_topk_backward(ctypes.byref(s), _ptr(topk_idx), _ptr(topk_w), _ptr(d_topk_w),
                                               _ptr(d_logits), st), "moe_route_topk_backward")
    return d_logits


def layer_backward(x, w_gate_up, w_down, fwd: dict, d_out, k: int, e_begin: int, e_end: int, stream=None,
                   norm=None, d_sum=None) -> dict:
    """The whole backward of one rank, given the forward's dict (from layer()):
    combine -> experts -> row gather -> router softmax. The gate/up
    pre-activations come from the forward's "gu" when it kept them.
    With the forward's `norm`, d_out is the gradient of "normed" (and d_sum, if
    given, that of "sum"): the result has "d_norm_weight", "d_norm_bias" (None
    without a bias) and "d_sum", the gradient of x + out. d_x is then still the
    gradient through the experts alone; x's whole gradient adds d_sum (the
    residual) and what comes through the logits."""
    T = x.shape[0]
    E = fwd["counts"].shape[0]
    extra = {}
    if norm is not None:
        if "sum" not in fwd:
            raise ValueError("the forward was run without norm")
        weight, bias, _ = norm
        d_out, d_nw, d_nb = layer_norm_backward(d_out, fwd["sum"], weight, fwd["mean"], fwd["rstd"], d_s=d_sum,
                                                bias=bias is not None, stream=stream)
        extra = dict(d_sum=d_out, d_norm_weight=d_nw, d_norm_bias=d_nb)
    elif d_sum is not None:
        raise ValueError("d_sum needs norm")
    d_y, d_w = combine_backward(d_out, fwd["y"], fwd["pair_pos"], fwd["w"], T, k, E, e_begin, e_end, stream=stream)
    d_x_perm, d_wgu, d_wdn = grouped_gemm_backward(x, fwd["perm"], fwd["offsets"], w_gate_up, w_down, fwd["h"], d_y,
                                                   k, E, e_begin, e_end, stream=stream, gu=fwd.get("gu"))
    d_x = dispatch_backward(d_x_perm, fwd["pair_pos"], T, k, E, e_begin, e_end, stream=stream)
    d_logits = route_topk_backward(fwd["idx"], fwd["w"], d_w, E, stream=stream)
    return dict(d_y=d_y, d_w=d_w, d_x_perm=d_x_perm, d_w_gate_up=d_wgu, d_w_down=d_wdn, d_x=d_x, d_logits=d_logits,
                **extra)


# ----------------------------------------------------------------------------- residual add and layer norm

def _rows(x, name: str):
    if x.dtype not in _CODES:
        _want(x, name, _act_dtypes())
    size = x.shape
    if len(size) != 2:
        raise ValueError(f"{name} must be [T, d], got {list(size)}")
    return size


def _like(t, name: str, dtype, size):
    """_want of a tensor that may be left out (None)."""
    if t is not None and (t.dtype is not dtype or t.shape != size):
        _want(t, name, dtype, tuple(size))


def _norm_params(x, weight, bias, d: int):
    if weight.dtype is not x.dtype or weight.shape != (d,):
        _want(weight, "weight", (x.dtype, _torch().float32), (d,))
    _like(bias, "bias", weight.dtype, (d,))


def layer_norm(x, weight, bias=None, eps: float = 1e-5, residual=None, y=None, s=None, mean=None, rstd=None,
               stream=None):
    """(y, s, mean, rstd): s = x + residual (x itself without one), normalised to
    y = (s - mean) * rstd * weight + bias, with fp32 statistics [T]. weight and
    bias [d] are of x's dtype or fp32. y may be x or residual, and so may s. With
    y = x and no residual, the rows that were normalised are overwritten: s is
    None, and there is nothing for layer_norm_backward to start from."""
    torch = _torch()
    T, d = size = _rows(x, "x")
    _norm_params(x, weight, bias, d)
    if residual is None and s is not None:
        raise ValueError("s is written only with a residual")
    _like(residual, "residual", x.dtype, size)
    _like(y, "y", x.dtype, size)
    _like(s, "s", x.dtype, size)
    _like(mean, "mean", torch.float32, (T,))
    _like(rstd, "rstd", torch.float32, (T,))
    sh = shape(T, d, 8, 1, 1, 0, 1)
    h, ctx = _ready(stream, (x, weight, bias, residual, y, s), (mean, rstd))
    if residual is None and not (y is not None and T > 0 and y.data_ptr() == x.data_ptr()):
        s = x
    with ctx:
        if y is None:
            y = torch.empty_like(x)
        if residual is not None and s is None:
            s = torch.empty_like(x)
        if mean is None:
            mean = torch.empty(T, dtype=torch.float32, device=x.device)
        if rstd is None:
            rstd = torch.empty(T, dtype=torch.float32, device=x.device)
        ctx.give(y, s, mean, rstd)
        _check(_load().moe_layer_norm(ctypes.byref(sh), _CODES[x.dtype], x.data_ptr(), _addr(residual),
                                      _CODES[weight.dtype], weight.data_ptr(), _addr(bias), eps, y.data_ptr(),
                                      None if residual is None else s.data_ptr(), mean.data_ptr(), rstd.data_ptr(), h),
               "moe_layer_norm")
    return y, s, mean, rstd


def layer_norm_backward_workspace_bytes(T: int, d: int) -> int:
    sh = shape(T, d, 8, 1, 1, 0, 1)
    return int(_load().moe_layer_norm_backward_workspace_bytes(ctypes.byref(sh)))


def layer_norm_backward(d_y, s, weight, mean, rstd, d_s=None, bias: bool = True, d_x=None, d_weight=None, d_bias=None,
                        workspace=None, stream=None):
    """(d_x, d_weight, d_bias): the gradient of layer_norm, given the forward's s,
    mean and rstd. d_s, the gradient that reaches s on other ways, is added to
    d_x. Without `bias`, d_bias is None. d_x may be d_y or d_s."""
    torch = _torch()
    T, d = size = _rows(d_y, "d_y")
    if s is None or mean is None or rstd is None:
        raise ValueError("s, mean and rstd of the forward are required")
    _like(s, "s", d_y.dtype, size)
    _norm_params(d_y, weight, None, d)
    _like(mean, "mean", torch.float32, (T,))
    _like(rstd, "rstd", torch.float32, (T,))
    _like(d_s, "d_s", d_y.dtype, size)
    _like(d_x, "d_x", d_y.dtype, size)
    _like(d_weight, "d_weight", weight.dtype, (d,))
    _like(d_bias, "d_bias", weight.dtype, (d,))
    if d_bias is not None and not bias:
        raise ValueError("d_bias is written only with bias")
    sh = shape(T, d, 8, 1, 1, 0, 1)
    ws_bytes = _load().moe_layer_norm_backward_workspace_bytes(ctypes.byref(sh))
    if workspace is not None:
        _want(workspace, "workspace", torch.uint8)
        if workspace.numel() < ws_bytes:
            raise ValueError(f"workspace must hold at least {ws_bytes} bytes, got {workspace.numel()}")
    h, ctx = _ready(stream, (d_y, s, weight, d_s, d_x, d_weight, d_bias, workspace), (mean, rstd))
    with ctx:
        if d_x is None:
            d_x = torch.empty_like(d_y)
        if d_weight is None:
            d_weight = torch.empty_like(weight)
        if d_bias is None and bias:
            d_bias = torch.empty_like(weight)
        ctx.give(d_x, d_weight, d_bias)
        if workspace is None and ws_bytes:
            workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=d_y.device)
        _check(_load().moe_layer_norm_backward(ctypes.byref(sh), _CODES[d_y.dtype], d_y.data_ptr(), s.data_ptr(),
                                               _CODES[weight.dtype], weight.data_ptr(), mean.data_ptr(),
                                               rstd.data_ptr(), _addr(d_s), d_x.data_ptr(), d_weight.data_ptr(),
                                               _addr(d_bias), _addr(workspace), h), "moe_layer_norm_backward")
    return d_x, d_weight, d_bias


# ----------------------------------------------------------------------------- experts in 8-bit integers

@dataclass
class Int8Experts:
    """The local experts' weights as 8-bit codes in K-blocks of 64 with one fp32
    scale per output channel: w_gate_up int8 [E_loc, ceil(d / 64), 2 * d_ff, 64],
    gate_up_scale [E_loc, 2 * d_ff], w_down int8 [E_loc, ceil(d_ff / 64), d, 64],
    down_scale [E_loc, d]. Weight [e, k, n] is w[e, k // 64, n, k % 64] * scale[e, n]."""
    w_gate_up: object
    gate_up_scale: object
    w_down: object
    down_scale: object


def _kblocks(k: int) -> int:
    return (k + 63) // 64


def _want_int8_experts(experts: Int8Experts, d: int, e_loc: int) -> int:
    """Checks the quantised experts against the activations; returns d_ff."""
    torch = _torch()
    sc = experts.gate_up_scale
    _want(sc, "gate_up_scale", torch.float32)
    if sc.dim() != 2 or sc.shape[0] != e_loc or sc.shape[1] % 2:
        raise ValueError(f"gate_up_scale must be [{e_loc}, 2 * d_ff], got {list(sc.shape)}")
    d_ff = sc.shape[1] // 2
    for t, name, dtype, size in ((experts.w_gate_up, "w_gate_up", torch.int8, (e_loc, _kblocks(d), 2 * d_ff, 64)),
                                 (experts.w_down, "w_down", torch.int8, (e_loc, _kblocks(d_ff), d, 64)),
                                 (experts.down_scale, "down_scale", torch.float32, (e_loc, d))):
        if t is None or t.dtype is not dtype or t.shape != size:
            _want(t, name, dtype, size)
    return d_ff


def quantize_experts(w_gate_up, w_down, out: Int8Experts | None = None, stream=None) -> Int8Experts:
    """The experts' weights (w_gate_up [E_loc, d, 2 * d_ff], w_down [E_loc, d_ff, d])
    as 8-bit codes, one scale per output channel: once, before serving."""
    torch = _torch()
    _want(w_down, "w_down", _act_dtypes())
    if w_down.dim() != 3:
        raise ValueError(f"w_down must be [E_loc, d_ff, d], got {list(w_down.shape)}")
    e_loc, d_ff, d = (int(v) for v in w_down.shape)
    _want(w_gate_up, "w_gate_up", w_down.dtype, (e_loc, d, 2 * d_ff))
    if out is not None:
        _want_int8_experts(out, d, e_loc)
    mine = () if out is None else (out.w_gate_up, out.gate_up_scale, out.w_down, out.down_scale)
    s = shape(0, d, d_ff, max(e_loc, 1), 1, 0, e_loc)
    h, ctx = _ready(stream, (w_gate_up, w_down, *mine[::2]), mine[1::2])
    dev = w_down.device
    with ctx:
        if out is None:
            out = Int8Experts(torch.empty((e_loc, _kblocks(d), 2 * d_ff, 64), dtype=torch.int8, device=dev),
                              torch.empty((e_loc, 2 * d_ff), dtype=torch.float32, device=dev),
                              torch.empty((e_loc, _kblocks(d_ff), d, 64), dtype=torch.int8, device=dev),
                              torch.empty((e_loc, d), dtype=torch.float32, device=dev))
        ctx.give(out.w_gate_up, out.gate_up_scale, out.w_down, out.down_scale)
        _check(_load().moe_quantize_experts(ctypes.byref(s), _dtype_code(w_down), _ptr(w_gate_up), _ptr(w_down),
                                            _ptr(out.w_gate_up), _ptr(out.gate_up_scale), _ptr(out.w_down),
                                            _ptr(out.down_scale), h), "moe_quantize_experts")
    return out


def grouped_gemm_int8_workspace_bytes(T: int, d: int, d_ff: int, E: int, k: int, e_begin: int, e_end: int) -> int:
    s = shape(T, d, d_ff, E, k, e_begin, e_end)
    return int(_load().moe_grouped_gemm_int8_workspace_bytes(ctypes.byref(s)))


def grouped_gemm_int8(x, perm, offsets, experts: Int8Experts, k: int, E: int, e_begin: int, e_end: int, y=None,
                      workspace=None, stream=None):
    """y [N_max, d]: the local experts' SwiGLU FFN in 8-bit integers, on rows of x
    (bf16) quantised as they are gathered through perm."""
    torch = _torch()
    _range(E, k, e_begin, e_end)
    _want(x, "x", torch.bfloat16)
    T, d = _rows(x, "x")
    n_max = _n_max(T, k, e_begin, e_end)
    _want(perm, "perm", torch.int32, (T * k,))
    _want(offsets, "offsets", torch.int32, (E + 1,))
    d_ff = _want_int8_experts(experts, d, e_end - e_begin)
    if y is not None:
        _want(y, "y", x.dtype, (n_max, d), min_rows=n_max)
    s = shape(T, d, d_ff, E, k, e_begin, e_end)
    ws_bytes = _load().moe_grouped_gemm_int8_workspace_bytes(ctypes.byref(s))
    if workspace is not None:
        _want(workspace, "workspace", torch.uint8)
        if workspace.numel() < ws_bytes:
            raise ValueError(f"workspace must hold at least {ws_bytes} bytes, got {workspace.numel()}")
    wgu, sgu, wdn, sdn = experts.w_gate_up, experts.gate_up_scale, experts.w_down, experts.down_scale
    h, ctx = _ready(stream, (x, wgu, wdn, y, workspace), (perm, offsets, sgu, sdn))
    with ctx:
        if y is None:
            y = torch.empty((n_max, d), dtype=x.dtype, device=x.device)
        ctx.give(y)
        if workspace is None and ws_bytes:
            workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=x.device)
        _check(_load().moe_grouped_gemm_int8(ctypes.byref(s), MOE_BF16, x.data_ptr(), perm.data_ptr(),
                                             offsets.data_ptr(), wgu.data_ptr(), sgu.data_ptr(), wdn.data_ptr(),
                                             sdn.data_ptr(), y.data_ptr(), _addr(workspace), h),
               "moe_grouped_gemm_int8")
    return y


def layer_int8(x, logits, experts: Int8Experts, k: int, e_begin: int, e_end: int, stream=None, norm=None) -> dict:
    """layer() for serving, with the experts in 8-bit integers: route -> dispatch
    (indices) -> grouped_gemm_int8 -> combine, and with `norm` the residual add
    and layer norm."""
    T = x.shape[0]
    if logits.dim() != 2 or logits.shape[0] != T:
        raise ValueError(f"logits must be [T={T}, E], got {list(logits.shape)}")
    E = logits.shape[1]
    _check_layer_norm_arg(norm, E, e_begin, e_end)
    idx, w = route_topk(logits, k, stream=stream)
    disp = dispatch(x, idx, E, e_begin, e_end, stream=stream, gather=False)
    y = grouped_gemm_int8(x, disp.perm, disp.offsets, experts, k, E, e_begin, e_end, stream=stream)
    out = combine(y, disp.pair_pos, w, T, k, E, e_begin, e_end, stream=stream)
    res = dict(idx=idx, w=w, counts=disp.counts, offsets=disp.offsets, perm=disp.perm, pair_pos=disp.pair_pos, y=y,
               out=out)
    return _with_norm(res, x, E, e_begin, e_end, norm, stream)


# ----------------------------------------------------------------------------- gradient norm and clipping

def _tensor_list(ts, name: str):
    """A list of gradients after checking its types, and their lengths and dtype codes."""
    torch = _torch()
    if torch.is_tensor(ts):
        raise TypeError(f"{name} must be a list of tensors")
    ts = list(ts)
    if not ts:
        raise ValueError(f"{name} is empty")
    try:
        kinds = [_CODES[t.dtype] for t in ts]
    except KeyError:
        for i, t in enumerate(ts):
            _want(t, f"{name}[{i}]", _act_dtypes())
        raise
    return ts, list(map(torch.Tensor.numel, ts)), kinds


def _host_list(ts, numels, kinds):
    """The host array of moe_tensor (address, length and dtype code, eight bytes each) as a C pointer."""
    flat = [0] * (3 * len(ts))
    flat[::3] = map(_torch().Tensor.data_ptr, ts)
    flat[1::3] = numels
    flat[2::3] = kinds
    return array.array("q", flat)


def grad_norm_workspace_bytes(n: int) -> int:
    return int(_load().moe_grad_norm_workspace_bytes(n))


def _norm_buffers(n: int, norm, workspace) -> int:
    torch = _torch()
    if norm is not None:
        _want(norm, "norm", torch.float32, (1,))
    need = grad_norm_workspace_bytes(n)
    if workspace is not None:
        _want(workspace, "workspace", torch.uint8)
        if workspace.numel() < need or workspace.data_ptr() % 8:
            raise ValueError(f"workspace must hold at least {need} bytes at an 8-byte boundary")
    return need


def _clip_out(ts, out):
    if out is None:
        return []
    out = list(out)
    if len(out) != len(ts):
        raise ValueError(f"out must hold {len(ts)} tensors, got {len(out)}")
    for i, (o, t) in enumerate(zip(out, ts)):
        if o.dtype is not t.dtype or o.shape != t.shape:
            _want(o, f"out[{i}]", t.dtype, tuple(t.shape))
    return out


def grad_norm(grads, norm=None, workspace=None, stream=None):
    """norm [1] fp32: the 2-norm over a list of gradients (bf16 or fp32, dense, any
    length and alignment), summed in fp64."""
    torch = _torch()
    ts, numels, kinds = _tensor_list(grads, "grads")
    need = _norm_buffers(len(ts), norm, workspace)
    h, ctx = _dense(stream, [*ts, norm, workspace])
    src = _host_list(ts, numels, kinds)
    with ctx:
        if norm is None:
            norm = torch.empty(1, dtype=torch.float32, device=ts[0].device)
        ctx.give(norm)
        if workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=ts[0].device)
        _check(_load().moe_grad_norm(src.buffer_info()[0], len(ts), norm.data_ptr(), workspace.data_ptr(), h),
               "moe_grad_norm")
    return norm


def clip_grads(grads, norm, max_norm: float, out=None, stream=None) -> None:
    """Scales the gradients by min(1, max_norm / (norm + 1e-6)) for a norm [1] fp32
    in device memory, in place or into the tensors of `out`."""
    torch = _torch()
    ts, numels, kinds = _tensor_list(grads, "grads")
    outs = _clip_out(ts, out)
    _want(norm, "norm", torch.float32, (1,))
    h, ctx = _dense(stream, [*ts, *outs, norm])
    src = _host_list(ts, numels, kinds)
    dst = _host_list(outs, numels, kinds) if outs else None
    with ctx:
        _check(_load().moe_clip_grads(src.buffer_info()[0], dst.buffer_info()[0] if outs else None, len(ts),
                                      norm.data_ptr(), max_norm, h), "moe_clip_grads")


def clip_grad_norm(grads, max_norm: float, out=None, norm=None, workspace=None, stream=None):
    """grad_norm, then clip_grads with it; returns the norm [1] before clipping."""
    torch = _torch()
    ts, numels, kinds = _tensor_list(grads, "grads")
    outs = _clip_out(ts, out)
    need = _norm_buffers(len(ts), norm, workspace)
    h, ctx = _dense(stream, [*ts, *outs, norm, workspace])
    src = _host_list(ts, numels, kinds)
    dst = _host_list(outs, numels, kinds) if outs else None
    with ctx:
        if norm is None:
            norm = torch.empty(1, dtype=torch.float32, device=ts[0].device)
        ctx.give(norm)
        if workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=ts[0].device)
        _check(_load().moe_clip_grad_norm(src.buffer_info()[0], dst.buffer_info()[0] if outs else None, len(ts),
                                          max_norm, norm.data_ptr(), workspace.data_ptr(), h), "moe_clip_grad_norm")
    return norm
