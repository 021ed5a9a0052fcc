"""Python binding of libpgemm (persistent-tile-scheduled GEMM for MI355X).

Argument marshalling only: every step of the GEMM runs in the HIP kernels
behind the C ABI declared in include/pgemm.h, and the functions here carry
the same names as its entry points. torch is used only to hand over device
memory (``tensor.data_ptr()``) and streams. There is no fallback: if the
HIP library has not been built, importing this package raises.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpgemm.so")

PGEMM_OK = 0
PGEMM_ERR_INVALID_ARG = 1
PGEMM_ERR_UNSUPPORTED = 2
PGEMM_ERR_HIP = 3
PGEMM_ERR_OOM = 4
PGEMM_ERR_TIMEOUT = 5

PGEMM_F16 = 0
PGEMM_BF16 = 1
PGEMM_F8E4M3_BF16 = 2

PGEMM_SCHED_NONPERSISTENT = 0
PGEMM_SCHED_STATIC = 1
PGEMM_SCHED_DYNAMIC = 2
PGEMM_SCHED_CANCEL = 3
PGEMM_SCHED_STREAMK = 4

PGEMM_TILE_AUTO = 0
PGEMM_TILE_256 = 1
PGEMM_TILE_128 = 2

PGEMM_B_KN = 0
PGEMM_B_NK = 1

PGEMM_IDS_I32 = 0
PGEMM_IDS_I64 = 1

PGEMM_GROUPED_ANY = 0
PGEMM_GROUPED_PINGPONG = 1
PGEMM_GROUPED_FEW16 = 2
PGEMM_GROUPED_FEW16_WIDE = 3
PGEMM_GROUPED_FEW32_WIDE = 4
PGEMM_GROUPED_FEW_GRAD = 5

PGEMM_W4_INT4 = 0
PGEMM_W4_E2M1 = 1

PGEMM_LOGITS_F16 = 0
PGEMM_LOGITS_BF16 = 1
PGEMM_LOGITS_F32 = 3

PGEMM_SCORE_SOFTMAX = 0
PGEMM_SCORE_SIGMOID = 1

PGEMM_ACT_NONE = 0
PGEMM_ACT_RELU = 1
PGEMM_ACT_GELU = 2
PGEMM_ACT_GELU_TANH = 3
PGEMM_ACT_SILU = 4

PGEMM_DENSE_DX = 1
PGEMM_DENSE_DW = 2
PGEMM_DENSE_DB = 4

PGEMM_DENSE_FEW8 = 0
PGEMM_DENSE_FEW16 = 1
PGEMM_DENSE_FEW32 = 2
PGEMM_DENSE_TILE64 = 3
PGEMM_DENSE_TILE128 = 4
PGEMM_DENSE_TILE128_PAIR = 5
PGEMM_DENSE_PINGPONG = 6

PGEMM_MAINLOOP_AUTO = 0
PGEMM_MAINLOOP_LOCKSTEP = 1
PGEMM_MAINLOOP_PINGPONG = 2
PGEMM_MAINLOOP_PRODUCER = 3

DTYPE_NAMES = {"f16": PGEMM_F16, "bf16": PGEMM_BF16, "e4m3fn": PGEMM_F8E4M3_BF16}
SCHED_NAMES = {"nonpersistent": PGEMM_SCHED_NONPERSISTENT, "static": PGEMM_SCHED_STATIC,
               "dynamic": PGEMM_SCHED_DYNAMIC, "cancel": PGEMM_SCHED_CANCEL, "streamk": PGEMM_SCHED_STREAMK}

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with "
                      "`python -m persistent_tile_scheduling_macro_amd.build` (hipcc, gfx950)")


def _load_hip_runtime() -> None:
    """Load torch's own HIP runtime before the library asks for one, whichever of the two is imported first: a process
    that holds both it and the system's passes streams of one to the other. Without a torch that has one, the system's."""
    try:
        torch = importlib.util.find_spec("torch")
        if torch is not None and torch.origin:
            path = os.path.join(os.path.dirname(torch.origin), "lib", "libamdhip64.so")
            if os.path.exists(path):
                ctypes.CDLL(path)
    except (ValueError, OSError):  # a module without a spec in torch's place, a runtime that does not load
        pass


_load_hip_runtime()
_lib = ctypes.CDLL(LIB_PATH)
_vp, _i64, _i32, _int = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_int
_ip = ctypes.POINTER(ctypes.c_int)


def _sig(name, restype, *argtypes):
    f = getattr(_lib, name)
    f.restype = restype
    f.argtypes = list(argtypes)
    return f


_create = _sig("pgemm_create", _int, ctypes.POINTER(_vp), _int)
_set_stream = _sig("pgemm_set_stream", _int, _vp, _vp)
_run = _sig("pgemm_run", _int, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _int, _int, _int)
_run_noalloc = _sig("pgemm_run_noalloc", _int, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _int, _int, _int)
_run_ld = _sig("pgemm_run_ld", _int, _vp, _vp, _i64, _vp, _i64, _vp, _i64, _i64, _i64, _i64, _int, _int, _int)
_destroy = _sig("pgemm_destroy", _int, _vp)
_status_string = _sig("pgemm_status_string", ctypes.c_char_p, _int)
_last_error = _sig("pgemm_last_error", ctypes.c_char_p, _vp)
_set_tile_counter = _sig("pgemm_set_tile_counter", _int, _vp, _vp, _i64)
_set_owner_log = _sig("pgemm_set_owner_log", _int, _vp, _vp, _i64)
_set_tile_trace = _sig("pgemm_set_tile_trace", _int, _vp, _vp, _i64)
_clock_khz = _sig("pgemm_clock_khz", _int, _int, _ip)
_wait = _sig("pgemm_wait", _int, _vp, _int)
_query_launch = _sig("pgemm_query_launch", _int, _vp, _i64, _i64, _i64, _int, _int, _int,
                     _ip, _ip, _ip, _ip, _ip, _ip, _ip)
_query_streamk = _sig("pgemm_query_streamk", _int, _vp, _i64, _i64, _i64, _int, _int, _ip, _ip, _ip, _ip,
                      ctypes.POINTER(_i64))
_set_tile_order = _sig("pgemm_set_tile_order", _int, _vp, _int, _int)
_set_tile_config = _sig("pgemm_set_tile_config", _int, _vp, _int)
_set_b_layout = _sig("pgemm_set_b_layout", _int, _vp, _int)
_set_mainloop = _sig("pgemm_set_mainloop", _int, _vp, _int)
_set_fp8_scales = _sig("pgemm_set_fp8_scales", _int, _vp, ctypes.c_float, ctypes.c_float)
_tile_coords = _sig("pgemm_tile_coords", _int, _i64, _i64, _i64, _int, _int, _ip, _ip)
_read_work_counter = _sig("pgemm_read_work_counter", _int, _vp, ctypes.POINTER(_i32))
_moe_dispatch_workspace = _sig("pgemm_moe_dispatch_workspace", _int, _i64, _i64, _i64, ctypes.POINTER(_i64))
_moe_dispatch = _sig("pgemm_moe_dispatch", _int, _vp, _vp, _i64, _vp, _int, _i64, _i64, _i64, _i64, _int, _vp, _vp, _vp,
                     _vp, _vp, _i64)
_moe_dispatch_backward = _sig("pgemm_moe_dispatch_backward", _int, _vp, _vp, _i64, _vp, _i64, _i64, _i64, _int, _vp)
_moe_combine = _sig("pgemm_moe_combine", _int, _vp, _vp, _i64, _vp, _vp, _i64, _i64, _i64, _int, _vp)
_moe_combine_backward = _sig("pgemm_moe_combine_backward", _int, _vp, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _i64, _i64,
                             _i64, _i64, _int, _vp, _vp)
_moe_combine_backward_plan = _sig("pgemm_moe_combine_backward_plan", _int, _vp, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _i64,
                                  _i64, _i64, _i64, _int, _vp, _vp)
_grouped_run = _sig("pgemm_grouped_run", _int, _vp, _vp, _i64, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _int, _int)
_grouped_weight_grad = _sig("pgemm_grouped_weight_grad", _int, _vp, _vp, _i64, _vp, _i64, _vp, _vp, _i64, _i64, _i64,
                            _i64, _int, _vp, _i64)
_grouped_weight_grad_workspace = _sig("pgemm_grouped_weight_grad_workspace", _int, _i64, _i64, _i64, _i64,
                                      ctypes.POINTER(_i64))
_w4_run = _sig("pgemm_w4_run", _int, _vp, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _int, _int, _int)
_grouped_query = _sig("pgemm_grouped_query", _int, _i64, _i64, _i64, _i64, _int, _int, _ip)
_grouped_weight_grad_query = _sig("pgemm_grouped_weight_grad_query", _int, _i64, _i64, _i64, _i64, _int, _ip, _ip)
_w4_query = _sig("pgemm_w4_query", _int, _i64, _i64, _i64, _int, _int, _ip, _ip)
_dense_run = _sig("pgemm_dense_run", _int, _vp, _vp, _i64, _vp, _i64, _vp, _vp, _i64, _vp, _vp, _i64, _i64, _i64, _int, _int,
                  _int, _int, _vp, _i64)
_dense_workspace = _sig("pgemm_dense_workspace", _int, _i64, _i64, _i64, _int, _int, _int, ctypes.POINTER(_i64))
_dense_backward = _sig("pgemm_dense_backward", _int, _vp, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _i64, _i64, _i64,
                       _int, _int, _int, _int, _vp, _i64)
_dense_backward_workspace = _sig("pgemm_dense_backward_workspace", _int, _i64, _i64, _i64, _int, _int, _int, _int, _int,
                                 ctypes.POINTER(_i64))
_dense_query = _sig("pgemm_dense_query", _int, _i64, _i64, _i64, _int, _int, _ip, _ip)
_dense_weight_grad_query = _sig("pgemm_dense_weight_grad_query", _int, _i64, _i64, _i64, _ip, _ip)
_dense_gradients_query = _sig("pgemm_dense_gradients_query", _int, _i64, _i64, _i64, _int, _ip, _ip, _ip)
_moe_route = _sig("pgemm_moe_route", _int, _vp, _vp, _i64, _int, _i64, _i64, _i64, _int, _int, _vp, _vp)
_moe_route_backward = _sig("pgemm_moe_route_backward", _int, _vp, _vp, _vp, _i64, _int, _vp, _vp, _i64, _i64, _i64, _int, _int, _vp)
_moe_layer = _sig("pgemm_moe_layer", _int, _vp, _vp, _i64, _vp, _int, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _i64, _int, _int,
                  _int, _vp, _i64)
_moe_layer_workspace = _sig("pgemm_moe_layer_workspace", _int, _i64, _i64, _i64, _i64, _i64, ctypes.POINTER(_i64))
_hold_cus = _sig("pgemm_hold_cus", _int, _vp, _int, _int, _int)


class PgemmError(RuntimeError):
    def __init__(self, status: int, detail: str = ""):
        self.status = status
        msg = pgemm_status_string(status)
        super().__init__(f"{msg}: {detail}" if detail else msg)


def _check(status: int, h=None) -> None:
    if status != PGEMM_OK:
        raise PgemmError(status, pgemm_last_error(h) if h else "")


def _ptr(x) -> int:
    """Device address of a torch tensor (or an int address / None)."""
    if x is None:
        return 0
    if isinstance(x, int):
        return x
    return int(x.data_ptr())


def pgemm_status_string(status: int) -> str:
    return _status_string(int(status)).decode()


def pgemm_last_error(h) -> str:
    return _last_error(h).decode()


def pgemm_create(device: int = 0):
    """Create a handle on `device`; returns an opaque handle (ctypes c_void_p)."""
    h = _vp()
    _check(_create(ctypes.byref(h), int(device)))
    return h


def _stream_ptr(stream):
    """hipStream_t of a torch.cuda.Stream, a raw int handle, or None (null stream)."""
    if stream is not None and not isinstance(stream, int):
        stream = int(stream.cuda_stream)
    return stream or None


def pgemm_set_stream(h, stream) -> None:
    """Bind a stream: a torch.cuda.Stream, a raw hipStream_t int, or None (null stream)."""
    _check(_set_stream(h, _stream_ptr(stream)), h)


def pgemm_run(h, A, B, C, M: int, N: int, K: int, dtype: int, sched_mode: int, grid_multiple: int = 0) -> None:
    """Enqueue C = A @ B (device pointers or tensors) on the handle's stream."""
    _check(_run(h, _ptr(A), _ptr(B), _ptr(C), int(M), int(N), int(K), int(dtype), int(sched_mode),
                int(grid_multiple)), h)


def pgemm_run_noalloc(h, A, B, C, M: int, N: int, K: int, dtype: int, sched_mode: int,
                      grid_multiple: int = 0) -> None:
    """pgemm_run that allocates nothing (stream-K partial tiles in the device's fixed scratch)."""
    _check(_run_noalloc(h, _ptr(A), _ptr(B), _ptr(C), int(M), int(N), int(K), int(dtype), int(sched_mode),
                        int(grid_multiple)), h)


PGEMM_NOALLOC_SCRATCH_BYTES = 96 << 20


def pgemm_run_ld(h, A, lda: int, B, ldb: int, C, ldc: int, M: int, N: int, K: int, dtype: int,
                 sched_mode: int, grid_multiple: int = 0) -> None:
    """pgemm_run with leading dimensions (in elements) for row-major views; pointers or tensors
    (a tensor's data_ptr() is the view's first element)."""
    _check(_run_ld(h, _ptr(A), int(lda), _ptr(B), int(ldb), _ptr(C), int(ldc), int(M), int(N), int(K),
                   int(dtype), int(sched_mode), int(grid_multiple)), h)


def pgemm_destroy(h) -> None:
    _check(_destroy(h))


def pgemm_set_tile_counter(h, visits, n_tiles: int = 0) -> None:
    """Attach an int32 device buffer of n_tiles visit counters (tensor or pointer); None detaches."""
    if visits is not None and not isinstance(visits, int) and not n_tiles:
        n_tiles = visits.numel()
    _check(_set_tile_counter(h, _ptr(visits) or None, int(n_tiles)), h)


def pgemm_set_owner_log(h, owner, n_tiles: int = 0) -> None:
    if owner is not None and not isinstance(owner, int) and not n_tiles:
        n_tiles = owner.numel()
    _check(_set_owner_log(h, _ptr(owner) or None, int(n_tiles)), h)


def pgemm_set_tile_trace(h, trace, n_tiles: int = 0) -> None:
    """trace: int64 device tensor of 4 * n_tiles entries ({wg, xcd, start, end} per tile), or None."""
    if trace is not None and not isinstance(trace, int) and not n_tiles:
        n_tiles = trace.numel() // 4
    _check(_set_tile_trace(h, _ptr(trace) or None, int(n_tiles)), h)


def pgemm_wait(h, timeout_ms: int) -> None:
    """Watchdog wait on the handle's stream; raises PgemmError(PGEMM_ERR_TIMEOUT) past the deadline."""
    _check(_wait(h, int(timeout_ms)), h)


def pgemm_clock_khz(device: int = 0) -> int:
    v = ctypes.c_int()
    _check(_clock_khz(int(device), ctypes.byref(v)))
    return v.value


def pgemm_query_launch(h, M: int, N: int, K: int, dtype: int, sched_mode: int, grid_multiple: int = 0) -> dict:
    out = [ctypes.c_int() for _ in range(7)]
    _check(_query_launch(h, int(M), int(N), int(K), int(dtype), int(sched_mode), int(grid_multiple),
                         *[ctypes.byref(o) for o in out]), h)
    keys = ["tiles", "grid", "occupancy", "bm", "bn", "bk", "body"]
    d = {k: o.value for k, o in zip(keys, out)}
    d["fast_path"] = int(d["body"] != 0)  # 0: generic kernel; body 1 lockstep, 2 ping-pong, 3 producer waves
    return d


def pgemm_query_streamk(h, M: int, N: int, K: int, dtype: int, grid_multiple: int = 0) -> dict:
    out = [ctypes.c_int() for _ in range(4)]
    ws = _i64()
    _check(_query_streamk(h, int(M), int(N), int(K), int(dtype), int(grid_multiple),
                          *[ctypes.byref(o) for o in out], ctypes.byref(ws)), h)
    keys = ["whole_tiles", "split_tiles", "split_groups", "pieces_split"]
    d = {k: o.value for k, o in zip(keys, out)}
    d["workspace_bytes"] = ws.value
    return d


def pgemm_set_tile_order(h, group_m: int = 8, xcd_remap=True) -> None:
    """xcd_remap: True/1 on, False/0 off, None/-1 automatic (on when a launch has more tiles than CUs)."""
    if xcd_remap is None or (not isinstance(xcd_remap, bool) and int(xcd_remap) < 0):
        v = -1
    else:
        v = int(bool(xcd_remap))
    _check(_set_tile_order(h, int(group_m), v), h)


def pgemm_set_tile_config(h, tile: int) -> None:
    _check(_set_tile_config(h, int(tile)), h)


def pgemm_set_mainloop(h, mainloop: int) -> None:
    """Wave schedule of the 256-row tile: PGEMM_MAINLOOP_AUTO, _LOCKSTEP, _PINGPONG or _PRODUCER."""
    _check(_set_mainloop(h, int(mainloop)), h)


def pgemm_set_fp8_scales(h, scale_a: float, scale_b: float) -> None:
    """Per-tensor scales of e4m3 A and B (C = scale_a * scale_b * sum of decoded products)."""
    _check(_set_fp8_scales(h, float(scale_a), float(scale_b)), h)


def pgemm_set_b_layout(h, layout: int) -> None:
    """PGEMM_B_KN: B is K x N row-major (default); PGEMM_B_NK: B is N x K row-major."""
    _check(_set_b_layout(h, int(layout)), h)


def pgemm_tile_coords(t: int, n_m: int, n_n: int, group_m: int = 8, cu_chunk: int = 0):
    pm, pn = ctypes.c_int(), ctypes.c_int()
    _check(_tile_coords(int(t), int(n_m), int(n_n), int(group_m), int(cu_chunk), ctypes.byref(pm),
                        ctypes.byref(pn)))
    return pm.value, pn.value


def pgemm_read_work_counter(h) -> int:
    v = ctypes.c_int32()
    _check(_read_work_counter(h, ctypes.byref(v)), h)
    return v.value


def pgemm_dense_run(h, x, ldx: int, w, ldw: int, bias, residual, ldr: int, y, z, M: int, N: int, K: int, layout: int, act: int,
                    gated: int, dtype: int, work=None, work_bytes: int = 0) -> None:
    """Enqueue y = act(x W + bias) + residual, and z, its pre-activations, unless None."""
    _check(_dense_run(h, _ptr(x), ldx, _ptr(w), ldw, _ptr(bias) or None, _ptr(residual) or None, ldr, _ptr(y), _ptr(z) or None,
                      M, N, K, layout, act, gated, dtype, _ptr(work) or None, work_bytes), h)


def pgemm_dense_workspace(M: int, N: int, K: int, layout: int, gated: int = 0, wide: bool = True) -> int:
    """Bytes of device scratch that pgemm_dense_run needs."""
    v = _i64()
    _check(_dense_workspace(M, N, K, layout, gated, int(wide), ctypes.byref(v)))
    return v.value


def pgemm_dense_backward(h, dy, lddy: int, x, ldx: int, w, ldw: int, z, dx, dw, db, M: int, N: int, K: int, layout: int, act: int,
                         gated: int, dtype: int, work=None, work_bytes: int = 0) -> None:
    """Enqueue the gradients dx, dw and db, each unless None."""
    _check(_dense_backward(h, _ptr(dy), lddy, _ptr(x), ldx, _ptr(w), ldw, _ptr(z) or None, _ptr(dx) or None, _ptr(dw) or None,
                           _ptr(db) or None, M, N, K, layout, act, gated, dtype, _ptr(work) or None, work_bytes), h)


def pgemm_dense_backward_workspace(M: int, N: int, K: int, layout: int, act: int, gated: int = 0, needs: int = 7,
                                   wide: bool = True) -> int:
    """Bytes of device scratch that pgemm_dense_backward needs for the gradients in `needs` (PGEMM_DENSE_D*, added up)."""
    v = _i64()
    _check(_dense_backward_workspace(M, N, K, layout, act, gated, needs, int(wide), ctypes.byref(v)))
    return v.value


def pgemm_dense_query(M: int, N: int, K: int, layout: int, gated: int = 0) -> tuple:
    """(PGEMM_DENSE_* body, pieces of the sum) of pgemm_dense_run."""
    body, pieces = ctypes.c_int(), ctypes.c_int()
    _check(_dense_query(M, N, K, layout, gated, ctypes.byref(body), ctypes.byref(pieces)))
    return body.value, pieces.value


def pgemm_dense_weight_grad_query(R: int, I: int, J: int) -> tuple:
    """(PGEMM_DENSE_* body, pieces of the sum) of the linear layer's weight gradient, [I, J] over R rows."""
    body, pieces = ctypes.c_int(), ctypes.c_int()
    _check(_dense_weight_grad_query(R, I, J, ctypes.byref(body), ctypes.byref(pieces)))
    return body.value, pieces.value


def pgemm_dense_gradients_query(M: int, C: int, K: int, layout: int) -> tuple:
    """(PGEMM_DENSE_* body, pieces of dx, pieces of dw) of the launch that computes both gradients, -1 for two launches."""
    body, px, pw = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
    _check(_dense_gradients_query(M, C, K, layout, ctypes.byref(body), ctypes.byref(px), ctypes.byref(pw)))
    return body.value, px.value, pw.value


def pgemm_moe_route(h, logits, ld: int, type: int, T: int, E: int, k: int, score: int, normalize: int, ids, weights) -> None:
    """Enqueue the choice of each token's k experts and their weights."""
    _check(_moe_route(h, _ptr(logits), ld, type, T, E, k, score, normalize, _ptr(ids), _ptr(weights)), h)


def pgemm_moe_route_backward(h, dweights, logits, ld: int, type: int, ids, weights, T: int, E: int, k: int, score: int,
                             normalize: int, dlogits) -> None:
    """Enqueue the gradient of the logits."""
    _check(_moe_route_backward(h, _ptr(dweights), _ptr(logits), ld, type, _ptr(ids), _ptr(weights), T, E, k, score, normalize,
                               _ptr(dlogits)), h)


def pgemm_moe_layer(h, x, ldx: int, ids, ids_type: int, weights, w_in, w_out, out, T: int, k: int, E: int, H: int, I: int, act: int,
                    gated: int, dtype: int, work=None, work_bytes: int = 0) -> None:
    """Enqueue a whole routed layer of few tokens."""
    _check(_moe_layer(h, _ptr(x), ldx, _ptr(ids), ids_type, _ptr(weights), _ptr(w_in), _ptr(w_out), _ptr(out), T, k, E, H, I, act,
                      gated, dtype, _ptr(work) or None, work_bytes), h)


def pgemm_moe_layer_workspace(T: int, k: int, E: int, H: int, I: int) -> int:
    """Bytes of device scratch that pgemm_moe_layer needs."""
    v = _i64()
    _check(_moe_layer_workspace(T, k, E, H, I, ctypes.byref(v)))
    return v.value


def pgemm_hold_cus(stream, device: int, n_cus: int, microseconds: int) -> None:
    """Benchmark aid: hold about n_cus CUs for about `microseconds` on `stream`."""
    _check(_hold_cus(_stream_ptr(stream), int(device), int(n_cus), int(microseconds)))


def pgemm_moe_dispatch_workspace(T: int, k: int, E: int) -> int:
    """Bytes of device scratch that pgemm_moe_dispatch needs."""
    v = _i64()
    _check(_moe_dispatch_workspace(int(T), int(k), int(E), ctypes.byref(v)))
    return v.value


def pgemm_moe_dispatch(h, x, ldx: int, ids, ids_type: int, T: int, k: int, E: int, H: int, dtype: int, offsets, order,
                       pos, xs, work=None, work_bytes: int = 0) -> None:
    """Sort T*k slots by expert and move the token rows (pointers or tensors)."""
    _check(_moe_dispatch(h, _ptr(x), ldx, _ptr(ids), ids_type, T, k, E, H, dtype, _ptr(offsets), _ptr(order), _ptr(pos),
                         _ptr(xs), _ptr(work), work_bytes), h)


def pgemm_moe_dispatch_backward(h, dxs, lddxs: int, pos, T: int, k: int, H: int, dtype: int, dx) -> None:
    _check(_moe_dispatch_backward(h, _ptr(dxs), lddxs, _ptr(pos), T, k, H, dtype, _ptr(dx)), h)


def pgemm_moe_combine(h, ys, ldys: int, w, pos, T: int, k: int, H: int, dtype: int, out) -> None:
    _check(_moe_combine(h, _ptr(ys), ldys, _ptr(w), _ptr(pos), T, k, H, dtype, _ptr(out)), h)


def pgemm_moe_combine_backward(h, dout, lddout: int, ys, ldys: int, w, offsets, pos, T: int, k: int, E: int, H: int,
                               dtype: int, dys, dw) -> None:
    _check(_moe_combine_backward(h, _ptr(dout), lddout, _ptr(ys), ldys, _ptr(w), _ptr(offsets), _ptr(pos), T, k, E, H,
                                 dtype, _ptr(dys), _ptr(dw)), h)


def pgemm_moe_combine_backward_plan(h, dout, lddout: int, ys, ldys: int, w, offsets, order, pos, T: int, k: int, E: int,
                                    H: int, dtype: int, dys, dw) -> None:
    """The same where slots were taken out of the plan after the sort."""
    _check(_moe_combine_backward_plan(h, _ptr(dout), lddout, _ptr(ys), ldys, _ptr(w), _ptr(offsets), _ptr(order), _ptr(pos),
                                      T, k, E, H, dtype, _ptr(dys), _ptr(dw)), h)


def pgemm_grouped_run(h, x, ldx: int, w, offsets, y, R: int, E: int, K: int, N: int, layout: int, dtype: int) -> None:
    """Enqueue y[r] = x[r] @ w[expert of r] for rows sorted by expert (pointers or tensors)."""
    _check(_grouped_run(h, _ptr(x), ldx, _ptr(w), _ptr(offsets), _ptr(y), R, E, K, N, layout, dtype), h)


def pgemm_grouped_weight_grad(h, a, lda: int, b, ldb: int, offsets, c, R: int, E: int, I: int, J: int, dtype: int,
                              work=None, work_bytes: int = 0) -> None:
    """Enqueue c[e] = a_e^T @ b_e over the rows of each expert."""
    _check(_grouped_weight_grad(h, _ptr(a), lda, _ptr(b), ldb, _ptr(offsets), _ptr(c), R, E, I, J, dtype, _ptr(work),
                                work_bytes), h)


def pgemm_grouped_weight_grad_workspace(R: int, E: int, I: int, J: int) -> int:
    """Bytes of device scratch that pgemm_grouped_weight_grad needs."""
    v = _i64()
    _check(_grouped_weight_grad_workspace(int(R), int(E), int(I), int(J), ctypes.byref(v)))
    return v.value


def pgemm_w4_run(h, x, ldx: int, q, scales, zeros, offsets, y, M: int, N: int, K: int, E: int, group: int, fmt: int,
                 dtype: int) -> None:
    """Enqueue y = x times 4-bit weights with group scales (pointers or tensors; zeros and offsets may be None)."""
    _check(_w4_run(h, _ptr(x), ldx, _ptr(q), _ptr(scales), _ptr(zeros) or None, _ptr(offsets) or None, _ptr(y), M, N, K,
                   E, group, fmt, dtype), h)


def pgemm_grouped_query(R: int, E: int, K: int, N: int, layout: int, wide: bool = True) -> int:
    """The PGEMM_GROUPED_* body that pgemm_grouped_run would launch."""
    body = _int()
    _check(_grouped_query(R, E, K, N, layout, int(wide), ctypes.byref(body)))
    return body.value


def pgemm_grouped_weight_grad_query(R: int, E: int, I: int, J: int, wide: bool = True) -> tuple:
    """(PGEMM_GROUPED_* body, pieces an expert's rows are cut into) of pgemm_grouped_weight_grad."""
    body, pieces = _int(), _int()
    _check(_grouped_weight_grad_query(R, E, I, J, int(wide), ctypes.byref(body), ctypes.byref(pieces)))
    return body.value, pieces.value


def pgemm_w4_query(M: int, N: int, E: int = 1, experts: bool = False, cus: int = 256) -> tuple:
    """(rows at once, blocks of 16 columns a wave takes) of pgemm_w4_run."""
    rows, blocks = _int(), _int()
    _check(_w4_query(M, N, E, int(experts), cus, ctypes.byref(rows), ctypes.byref(blocks)))
    return rows.value, blocks.value


def matmul(A, B, C=None, *, sched: str | int = "static", grid_multiple: int = 0, handle=None):
    """C = A @ B for 2-D CUDA tensors (fp16, bf16, or float8_e4m3fn with a bf16 C).

    Marshals shapes and pointers into pgemm_run; no arithmetic happens here.
    """
    import torch  # the binding itself does not need torch; this helper does

    dtypes = {torch.float16: PGEMM_F16, torch.bfloat16: PGEMM_BF16, torch.float8_e4m3fn: PGEMM_F8E4M3_BF16}
    if A.dtype != B.dtype or A.dtype not in dtypes:
        raise TypeError(f"unsupported dtypes {A.dtype}, {B.dtype}")
    if A.dim() != 2 or B.dim() != 2 or A.shape[1] != B.shape[0]:
        raise ValueError(f"shape mismatch {tuple(A.shape)} @ {tuple(B.shape)}")
    if not (A.is_cuda and B.is_cuda and A.is_contiguous() and B.is_contiguous()):
        raise ValueError("A and B must be contiguous device tensors")
    M, K = A.shape
    N = B.shape[1]
    out_dtype = torch.bfloat16 if A.dtype == torch.float8_e4m3fn else A.dtype
    if C is None:
        C = torch.empty((M, N), dtype=out_dtype, device=A.device)
    elif C.shape != (M, N) or C.dtype != out_dtype or not C.is_contiguous():
        raise ValueError("C has the wrong shape, dtype or layout")
    own = handle is None
    h = pgemm_create(A.device.index or 0) if own else handle
    try:
        if own:
            pgemm_set_stream(h, torch.cuda.current_stream(A.device))
        s = SCHED_NAMES[sched] if isinstance(sched, str) else int(sched)
        pgemm_run(h, A, B, C, M, N, K, dtypes[A.dtype], s, grid_multiple)
    finally:
        if own:
            pgemm_destroy(h)
    return C
