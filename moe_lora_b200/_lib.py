"""ctypes binding to libmoe_lora.so (argument marshalling only).

Every function here checks tensor placement and dtype, allocates the outputs and the
workspace with torch when the caller does not pass them, and calls the C ABI on the
current torch CUDA stream.  All arithmetic happens in the CUDA kernels of the library;
there is no fallback: a missing library or a non-OK status raises.
"""
from __future__ import annotations

import ctypes
import functools
import operator
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe_lora.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_CUDA, ERR_DEVICE_CHECK, ERR_TIMEOUT = range(6)
ML_F32, ML_BF16, ML_E4M3 = 0, 1, 2
OP_ROUTE, OP_FORWARD, OP_SGMV_SHRINK, OP_SGMV_EXPAND, OP_DENSE, OP_FORWARD_BF16, OP_FORWARD_E4M3 = range(7)
OP_ROUTE_SCORED, OP_DENSE_FUSED = 7, 8
SCORES = {"softmax": 0, "sigmoid": 1}
GROUP_RULES = {"max": 0, "top2": 1}
ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4, "silu_and_mul": 5}

EXPORTS = ("moe_lora_route", "moe_lora_forward", "sgmv_shrink", "sgmv_expand", "dense_lora_forward",
           "moe_lora_workspace_size", "moe_lora_check_status", "moe_lora_last_error", "moe_lora_version",
           "moe_lora_profile_enable", "moe_lora_profile_read", "moe_lora_launch_count",
           "moe_lora_route_noalloc", "moe_lora_route_scored", "dense_lora_fused")
KERNEL_IDS = {"router_logits": 0, "topk": 1, "sort": 2, "shrink": 3, "gemm_gateup": 4, "gemm_down": 5,
              "combine": 6, "expand": 7, "dense_f32": 8, "gemm_dense": 9, "quant": 10,
              "lora": 11, "route": 12, "lora_down": 13,
              "gather": 14, "dense_fused": 15, "fused_shrink": 16, "route_scored": 17}


class AdapterFormat(ctypes.Structure):
    """moe_lora_adapter_format: gate_up adapter layout (0 fused, 1 separate gate and up
    adapters) and the per-projection scales of the LoRA deltas."""
    _fields_ = [("gate_up_split", ctypes.c_int), ("scale_gu", ctypes.c_float), ("scale_d", ctypes.c_float)]


class RouteFormat(ctypes.Structure):
    """moe_lora_route_format: scores, expert groups, renormalisation and scale of the weights."""
    _fields_ = [("score", ctypes.c_int), ("n_group", ctypes.c_int), ("topk_group", ctypes.c_int),
                ("group_rule", ctypes.c_int), ("renormalize", ctypes.c_int), ("scale", ctypes.c_float)]


class MoELoRAError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"moe_lora status {status}: {msg}")
        self.status = status


_lib = None
_P = ctypes.c_void_p
_I = ctypes.c_int
_SZ = ctypes.c_size_t


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m moe_lora_b200.build` "
                               "(there is no CPU fallback)")
        L = ctypes.CDLL(LIB_PATH)
        L.moe_lora_route.argtypes = [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _SZ, _P]
        L.moe_lora_forward.argtypes = [_P, _I, _I, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _I, _P,
                                       _P, _P, _P, _P, ctypes.POINTER(AdapterFormat), _P, _P, _SZ, _P]
        L.sgmv_shrink.argtypes = [_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _SZ, _P]
        L.sgmv_expand.argtypes = [_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _SZ, _P]
        L.dense_lora_forward.argtypes = [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _P, _P, _SZ, _P]
        L.moe_lora_route_scored.argtypes = [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, ctypes.POINTER(RouteFormat),
                                            _P, _P, _P, _P, _P, _P, _SZ, _P]
        L.dense_lora_fused.argtypes = [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, ctypes.c_float, _P,
                                       _I, _P, _P, _SZ, _P]
        L.moe_lora_workspace_size.argtypes = [_I] * 8
        L.moe_lora_workspace_size.restype = _SZ
        L.moe_lora_check_status.argtypes = [_P, _P]
        L.moe_lora_last_error.restype = ctypes.c_char_p
        L.moe_lora_version.restype = ctypes.c_char_p
        L.moe_lora_profile_enable.argtypes = [_I]
        L.moe_lora_profile_enable.restype = _I
        L.moe_lora_profile_read.argtypes = [_I, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(_I)]
        L.moe_lora_profile_read.restype = _I
        L.moe_lora_launch_count.restype = ctypes.c_longlong
        for name in ("moe_lora_route", "moe_lora_forward", "sgmv_shrink", "sgmv_expand",
                     "dense_lora_forward", "moe_lora_route_scored", "dense_lora_fused", "moe_lora_check_status"):
            getattr(L, name).restype = _I
        _lib = L
    return _lib


def _check(status: int):
    if status != OK:
        raise MoELoRAError(status, lib().moe_lora_last_error().decode())


def _ptr(t: torch.Tensor | None):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors passed to the library must be CUDA tensors")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # no stream object is made


def _stream(stream=None, device=None):
    if stream is None and _current_raw_stream is not None:
        return _current_raw_stream(torch.cuda.current_device() if device is None else device)
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _dt(t: torch.Tensor) -> int:
    return {torch.float32: ML_F32, torch.bfloat16: ML_BF16, torch.float8_e4m3fn: ML_E4M3}[t.dtype]


def workspace_size(op: int, M=0, H=0, I=0, E=0, k=0, L=0, r=0) -> int:
    return int(lib().moe_lora_workspace_size(op, M, H, I, E, k, L, r))


def new_workspace(nbytes: int, device) -> torch.Tensor:
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


def check_status(workspace: torch.Tensor, stream=None) -> None:
    _check(lib().moe_lora_check_status(_ptr(workspace), _stream(stream)))


def version() -> str:
    return lib().moe_lora_version().decode()


def profile_enable(max_launches: int) -> None:
    _check(lib().moe_lora_profile_enable(int(max_launches)))


def profile_read(kernel: str) -> tuple[float, int]:
    ms, n = ctypes.c_double(0.0), _I(0)
    _check(lib().moe_lora_profile_read(KERNEL_IDS[kernel], ctypes.byref(ms), ctypes.byref(n)))
    return ms.value, n.value


def launch_count() -> int:
    return int(lib().moe_lora_launch_count())


# ------------------------------------------------------------------------------ MoE layer

def route(adapter_ids: torch.Tensor, k: int, L: int, *, x=None, w_router=None, bias=None,
          logits_in=None, want_logits=False, out=None, workspace=None, stream=None) -> dict:
    """moe_lora_route.  Returns topk_ids [M,k], topk_w [M,k], sorted_pairs [M*k],
    seg_offsets [E*(L+1)+1] (and logits [M,E] when asked)."""
    dev = adapter_ids.device
    M = adapter_ids.shape[0]
    if logits_in is not None:
        E = logits_in.shape[1]
        H = 0
    else:
        E, H = w_router.shape
    o = out if out is not None else {}

    def buf(name, shape, dtype):
        t = o.get(name)
        return t if t is not None else torch.empty(shape, dtype=dtype, device=dev)

    ids = buf("topk_ids", (M, k), torch.int32)
    w = buf("topk_w", (M, k), torch.float32)
    sp = buf("sorted_pairs", (max(M * k, 1),), torch.int32)
    so = buf("seg_offsets", (E * (L + 1) + 1,), torch.int32)
    lg = buf("logits", (M, E), torch.float32) if want_logits else None
    if workspace is None:
        workspace = new_workspace(workspace_size(OP_ROUTE, M, H, 0, E, k, L, 0), dev)
    _check(lib().moe_lora_route(_ptr(x), _ptr(w_router), _ptr(bias), _ptr(logits_in), _ptr(adapter_ids),
                                M, H, E, k, L, _ptr(lg), _ptr(ids), _ptr(w), _ptr(sp), _ptr(so),
                                _ptr(workspace), workspace.numel(), _stream(stream)))
    res = {"topk_ids": ids, "topk_w": w, "sorted_pairs": sp[: M * k], "seg_offsets": so,
           "workspace": workspace}
    if want_logits:
        res["logits"] = lg
    return res


def _expect(name: str, t: torch.Tensor | None, shape: tuple, dtype: torch.dtype) -> None:
    if t is not None and (t.dtype != dtype or t.shape != shape):
        raise ValueError(f"{name} must be {dtype} of shape {shape}, got {t.dtype} of shape {tuple(t.shape)}")


def _addresses(*tensors) -> tuple[int, list]:
    """The current device's index and the tensors' addresses (None stays None): they have to be
    contiguous and on that device, since the library launches on the current one."""
    dev, at = -2, []
    for t in tensors:
        if t is None:
            at.append(None)
            continue
        if t.get_device() != dev:
            if dev != -2:
                raise ValueError(f"tensors on several devices, cuda:{dev} and {t.device} among them")
            dev = t.get_device()
            if dev < 0:
                raise ValueError("tensors passed to the library must be CUDA tensors")
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")
        at.append(t.data_ptr())
    if dev != torch.cuda.current_device():
        raise ValueError(f"the tensors are on cuda:{dev}, the current device is cuda:{torch.cuda.current_device()}")
    return dev, at


@functools.lru_cache(maxsize=4096)
def _sized(op: int, M: int, H: int, I: int, E: int, k: int, L: int, r: int) -> int:
    return workspace_size(op, M, H, I, E, k, L, r)


def _made(stream, n, dtype: torch.dtype, device: torch.device) -> torch.Tensor:
    """A buffer for a call on `stream` (None: the current one).  It comes from that stream's memory,
    since a block of the current one's may still wait for work queued there; and as the caller goes
    on on the current stream, it is not reused before that one is done with it either."""
    if stream is None:
        return torch.empty(n, dtype=dtype, device=device)
    if stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
    with torch.cuda.stream(stream):
        t = torch.empty(n, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(device))
    return t


def _choice(name: str, value: str, of: dict) -> int:
    if value not in of:
        raise ValueError(f"{name} must be one of {', '.join(of)}, got {value!r}")
    return of[value]


@functools.lru_cache(maxsize=256)
def _kept_format(score, n_group, topk_group, group_rule, renormalize, scale) -> RouteFormat:
    return RouteFormat(_choice("score", score, SCORES), n_group, topk_group,
                       _choice("group_rule", group_rule, GROUP_RULES), renormalize, scale)


def _route_format(score, n_group, topk_group, group_rule, renormalize, scale) -> RouteFormat:
    # plain numbers only are kept: a tensor would be by its identity, with the value of its first call
    if type(scale) is not float:
        scale = float(scale)
    if not type(n_group) is type(topk_group) is int:
        n_group, topk_group = int(n_group), int(topk_group)
    return _kept_format(score, n_group, topk_group, group_rule, 1 if renormalize else 0, scale)


def route_scored(adapter_ids: torch.Tensor, k: int, L: int, *, x=None, w_router=None, bias=None, logits_in=None,
                 score: str = "softmax", score_bias=None, n_group: int = 1, topk_group: int = 1,
                 group_rule: str = "max", renormalize: bool = True, scale: float = 1.0, want_logits=False,
                 out=None, workspace=None, stream=None) -> dict:
    """moe_lora_route_scored: routing by "softmax" or "sigmoid" scores.  score_bias (fp32 [E])
    moves the choice of experts, not their weights; topk_group of n_group groups of experts
    are kept by group_rule ("max", or "top2": the sum of the two largest); the weights are
    divided by their sum if renormalize, then multiplied by scale.  Returns what route() does."""
    if logits_in is None and (x is None or w_router is None):
        raise ValueError("route_scored needs x and w_router, or logits_in")
    M, k, L = adapter_ids.shape[0], operator.index(k), operator.index(L)
    E, H = (logits_in.shape[1], 0) if logits_in is not None else w_router.shape
    _expect("adapter_ids", adapter_ids, (M,), torch.int32)
    if logits_in is not None:
        _expect("logits_in", logits_in, (M, E), torch.float32)
    else:
        _expect("x", x, (M, H), torch.bfloat16)
        _expect("w_router", w_router, (E, H), torch.bfloat16)
        _expect("bias", bias, (E,), torch.float32)
    _expect("score_bias", score_bias, (E,), torch.float32)
    fmt = _route_format(score, n_group, topk_group, group_rule, renormalize, scale)
    mk, ns = M * k, E * (L + 1) + 1
    ids = w = sp = so = lg = None
    if out:
        ids, w, sp, so = out.get("topk_ids"), out.get("topk_w"), out.get("sorted_pairs"), out.get("seg_offsets")
        lg = out.get("logits") if want_logits else None
        for name, t, n, dtype in (("topk_ids", ids, mk, torch.int32), ("topk_w", w, mk, torch.float32),
                                  ("sorted_pairs", sp, mk, torch.int32), ("seg_offsets", so, ns, torch.int32),
                                  ("logits", lg, M * E, torch.float32)):
            if t is not None and (t.dtype != dtype or t.numel() < n):
                raise ValueError(f"out[{name!r}] must be {dtype} with at least {n} elements")
    dev, at = _addresses(adapter_ids, x, w_router, bias, logits_in, score_bias, workspace, ids, w, sp, so, lg)
    # what the caller did not pass is cut from one buffer, in pieces of whole 256 bytes (64 words)
    wsn = 0 if workspace is not None else (_sized(OP_ROUTE_SCORED, M, H, 0, E, k, L, 0) + 255) // 256 * 64
    pmk, pns = (mk + 63) // 64 * 64, (ns + 63) // 64 * 64
    total = wsn
    if not out:
        total += 3 * pmk + pns
    else:
        total += pmk * ((ids is None) + (w is None) + (sp is None)) + pns * (so is None)
    if want_logits and lg is None:
        total += M * E
    buf, o = None, wsn
    if total:
        buf = _made(stream, total, torch.int32, adapter_ids.device)
        base = buf.data_ptr()
    if workspace is None:
        workspace, at[6], wsb = buf.as_strided((wsn,), (1,), 0).view(torch.uint8), base, 4 * wsn
    else:
        wsb = workspace.numel()
    if ids is None:
        ids, at[7] = buf.as_strided((M, k), (k, 1), o), base + 4 * o
        o += pmk
    if w is None:
        w, at[8] = buf.as_strided((M, k), (k, 1), o).view(torch.float32), base + 4 * o
        o += pmk
    if sp is None:
        sp, at[9] = buf.as_strided((mk,), (1,), o), base + 4 * o
        o += pmk
    if so is None:
        so, at[10] = buf.as_strided((ns,), (1,), o), base + 4 * o
        o += pns
    if want_logits and lg is None:
        lg, at[11] = buf.as_strided((M, E), (E, 1), o).view(torch.float32), base + 4 * o
    st = lib().moe_lora_route_scored(at[1], at[2], at[3], at[4], at[5], at[0], M, H, E, k, L, ctypes.byref(fmt), at[11],
                                     at[7], at[8], at[9], at[10], at[6], wsb, _stream(stream, dev))
    if st != OK:
        _check(st)
    res = {"topk_ids": ids, "topk_w": w, "sorted_pairs": sp if sp.shape[0] == mk else sp[:mk], "seg_offsets": so,
           "workspace": workspace}
    if want_logits:
        res["logits"] = lg
    return res


def forward(x: torch.Tensor, routing: dict, weights: dict, *, k: int, L: int, y=None, workspace=None,
            stream=None, scale_gu: float = 1.0, scale_d: float = 1.0) -> torch.Tensor:
    """moe_lora_forward.  weights: w_gu [E,2I,H], w_d [E,H,I] (bf16 or e4m3), scales [E,2]
    (e4m3 only), a_gu [L,E,r,H], b_gu [L,E,r,2I] -- or separate gate and up adapters
    a_gu [L,E,2,r,H], b_gu [L,E,2,r,I] -- a_d [L,E,r,I], b_d [L,E,r,H] (bf16).
    scale_gu / scale_d multiply each projection's delta."""
    M, H = x.shape
    E, twoI, _ = weights["w_gu"].shape
    I = twoI // 2
    split = L > 0 and weights["a_gu"].dim() == 5
    r = weights["a_gu"].shape[-2] if L > 0 else 0
    fmt = AdapterFormat(1 if split else 0, float(scale_gu), float(scale_d))
    wdt = _dt(weights["w_gu"])
    if y is None:
        y = torch.empty((M, H), dtype=torch.bfloat16, device=x.device)
    if workspace is None:
        op = OP_FORWARD_E4M3 if wdt == ML_E4M3 else OP_FORWARD_BF16
        workspace = new_workspace(workspace_size(op, M, H, I, E, k, L, r), x.device)
    scales = weights.get("scales") if wdt == ML_E4M3 else None
    _check(lib().moe_lora_forward(
        _ptr(x), M, H, I, E, k, L, r, _ptr(routing["topk_w"]), _ptr(routing["sorted_pairs"]),
        _ptr(routing["seg_offsets"]), _ptr(weights["w_gu"]), _ptr(weights["w_d"]), wdt, _ptr(scales),
        _ptr(weights["a_gu"]) if L else None, _ptr(weights["b_gu"]) if L else None,
        _ptr(weights["a_d"]) if L else None, _ptr(weights["b_d"]) if L else None, ctypes.byref(fmt),
        _ptr(y), _ptr(workspace), workspace.numel(), _stream(stream)))
    return y


# ------------------------------------------------------------------------------ SGMV / dense

def sgmv_shrink(x, lora_a, seg_offsets, seg_adapter, *, z=None, workspace=None, stream=None):
    T, h_in = x.shape
    L, r, _ = lora_a.shape
    if z is None:
        z = torch.empty((T, r), dtype=torch.float32, device=x.device)
    if workspace is None:
        workspace = new_workspace(workspace_size(OP_SGMV_SHRINK), x.device)
    S = seg_adapter.shape[0]
    _check(lib().sgmv_shrink(_ptr(x), _ptr(lora_a) if L else None, _ptr(seg_offsets), _ptr(seg_adapter),
                             S, T, h_in, r, L, _dt(x), _ptr(z), _ptr(workspace), workspace.numel(),
                             _stream(stream)))
    return z


def sgmv_expand(z, lora_b, seg_offsets, seg_adapter, y, *, workspace=None, stream=None):
    T, r = z.shape
    L, _, h_out = lora_b.shape
    if workspace is None:
        workspace = new_workspace(workspace_size(OP_SGMV_EXPAND), z.device)
    S = seg_adapter.shape[0]
    _check(lib().sgmv_expand(_ptr(z), _ptr(lora_b) if L else None, _ptr(seg_offsets), _ptr(seg_adapter),
                             S, T, h_out, r, L, _dt(y), _ptr(y), _ptr(workspace), workspace.numel(),
                             _stream(stream)))
    return y


def dense_lora_forward(x, w, lora_a, lora_b, seg_offsets, seg_adapter, *, y=None, workspace=None,
                       stream=None):
    T, h_in = x.shape
    h_out = w.shape[0]
    L, r, _ = lora_a.shape
    if y is None:
        y = torch.empty((T, h_out), dtype=x.dtype, device=x.device)
    if workspace is None:
        workspace = new_workspace(workspace_size(OP_DENSE, T, h_in, h_out, 1, 1, L, r), x.device)
    S = seg_adapter.shape[0]
    _check(lib().dense_lora_forward(_ptr(x), _ptr(w), _ptr(lora_a) if L else None,
                                    _ptr(lora_b) if L else None, _ptr(seg_offsets), _ptr(seg_adapter),
                                    S, T, h_in, h_out, r, L, _dt(x), _ptr(y), _ptr(workspace),
                                    workspace.numel(), _stream(stream)))
    return y


def dense_lora_fused(x, w, lora_a=None, lora_b=None, seg_offsets=None, seg_adapter=None, *, bias=None,
                     activation: str = "none", residual=None, lora_scale: float = 1.0, y=None, workspace=None,
                     stream=None):
    """dense_lora_fused: y = act(x w^T + bias + lora_scale (x A) B) + residual, bf16 or fp32.
    activation: "none", "relu", "gelu", "gelu_tanh", "silu", or "silu_and_mul", where w (and
    bias and lora_b) hold 2 h_out features, the gate first.  Without lora_a and lora_b no
    segments are needed, and given ones are not looked at; y may be the residual (an update in
    place).  What the kernels find wrong (segments out of order, an adapter id out of range, a wait
    that ran out) is recorded in the workspace alone: pass one and give it to check_status()."""
    act = _choice("activation", activation, ACTIVATIONS)
    if x.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"x must be torch.bfloat16 or torch.float32, got {x.dtype}")
    T, h_in = x.shape
    n = w.shape[0]
    if act == 5 and n % 2:
        raise ValueError("silu_and_mul needs an even number of weight rows (gate, then up)")
    h_out = n // 2 if act == 5 else n
    if (lora_a is None) != (lora_b is None):
        raise ValueError("lora_a and lora_b go together")
    L, r = (lora_a.shape[0], lora_a.shape[1]) if lora_a is not None else (0, 0)
    if L > 0 and (seg_offsets is None or seg_adapter is None):
        raise ValueError("adapters need seg_offsets and seg_adapter")
    S = seg_adapter.shape[0] if seg_adapter is not None else 0
    dt = x.dtype
    for name, t, shape in (("w", w, (n, h_in)), ("bias", bias, (n,)), ("residual", residual, (T, h_out)),
                           ("lora_a", lora_a, (L, r, h_in)), ("lora_b", lora_b, (L, r, n)), ("y", y, (T, h_out))):
        if t is not None and (t.dtype is not dt or t.shape != shape):
            _expect(name, t, shape, dt)
    if seg_adapter is not None:
        _expect("seg_adapter", seg_adapter, (S,), torch.int32)
        _expect("seg_offsets", seg_offsets, (S + 1,), torch.int32)
    dev, at = _addresses(x, w, bias, lora_a, lora_b, seg_offsets, seg_adapter, residual, y, workspace)
    if L == 0:
        at[3] = at[4] = None
    if y is None:
        y = _made(stream, (T, h_out), dt, x.device)
        at[8] = y.data_ptr()
    wsb = workspace.numel() if workspace is not None else max(_sized(OP_DENSE_FUSED, T, h_in, h_out, 1, 1, L, r), 256)
    if workspace is None:
        workspace = _made(stream, wsb, torch.uint8, x.device)
        at[9] = workspace.data_ptr()
    st = lib().dense_lora_fused(at[0], at[1], at[2], at[3], at[4], at[5], at[6], S, T, h_in, h_out, r, L, act,
                                float(lora_scale), at[7], ML_BF16 if dt is torch.bfloat16 else ML_F32, at[8], at[9], wsb,
                                _stream(stream, dev))
    if st != OK:
        _check(st)
    return y
