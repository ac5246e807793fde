"""Thin Python binding of libmoe.so (include/moe.h): argument marshalling only.

Every step of the layer runs in the library's HIP kernels; torch supplies device memory and the current
stream.  Importing works without a GPU; calling a function without the built library raises.
"""
import contextlib
import ctypes
import os

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmoe.so")

MOE_F32, MOE_BF16, MOE_FP8_E4M3, MOE_MXFP4, MOE_MXFP8 = 0, 1, 2, 3, 4
STATUS = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED", 3: "MOE_ERR_WORKSPACE", 4: "MOE_ERR_HIP",
          5: "MOE_ERR_SCRATCH"}
EXPORTS = ("moe_workspace_size", "moe_route", "moe_forward", "moe_forward_staged", "moe_route_limited",
           "moe_route_grouped", "moe_forward_shard", "moe_expert_utilization", "moe_forward_noalloc",
           "moe_quantize_e4m3", "moe_quantize_mx", "moe_dequantize_mx", "moe_forward_routed", "moe_few_workspace_size", "moe_forward_few",
           "moe_status_string")
NOALLOC_SCRATCH_BYTES = 64 << 20
FEW_MAX_T = 16
NUM_STAGES = 7
STAGE_NAMES = ("router_logits", "topk_softmax", "permute", "x_quant", "up_gemm", "down_gemm", "combine")


class MoeError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {STATUS.get(status, status)} ({moe_status_string(status)})")
        self.status = status


class moe_shape_t(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("d", ctypes.c_int64), ("E", ctypes.c_int64), ("k", ctypes.c_int64),
                ("inter", ctypes.c_int64), ("inter_shared", ctypes.c_int64),
                ("act_dtype", ctypes.c_int32), ("w_dtype", ctypes.c_int32)]


_LIB = None


def lib() -> ctypes.CDLL:
    """The loaded library; raises if it has not been built (no fallback path exists)."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m sparse_mixture_experts_08_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, sp = ctypes.c_void_p, ctypes.POINTER(moe_shape_t)
        L.moe_workspace_size.restype = ctypes.c_size_t
        L.moe_workspace_size.argtypes = [sp]
        L.moe_route.restype = ctypes.c_int
        L.moe_route.argtypes = [sp] + [vp] * 10 + [ctypes.c_size_t, vp]
        L.moe_forward.restype = ctypes.c_int
        L.moe_forward.argtypes = [sp] + [vp] * 20 + [ctypes.c_size_t, vp]
        L.moe_forward_staged.restype = ctypes.c_int
        L.moe_forward_staged.argtypes = [sp] + [vp] * 20 + [ctypes.c_size_t, vp, vp]
        L.moe_route_limited.restype = ctypes.c_int
        L.moe_route_limited.argtypes = [sp] + [vp] * 11 + [ctypes.c_size_t, vp]
        i64 = ctypes.c_int64
        L.moe_route_grouped.restype = ctypes.c_int
        L.moe_route_grouped.argtypes = [sp, i64] + [vp] * 10 + [ctypes.c_size_t, vp]
        L.moe_quantize_e4m3.restype = ctypes.c_int
        L.moe_quantize_e4m3.argtypes = [i64, i64, vp, vp, vp, vp]
        i32 = ctypes.c_int32
        L.moe_quantize_mx.restype = ctypes.c_int
        L.moe_quantize_mx.argtypes = [i64, i64, vp, i32, i32, vp, vp, vp]
        L.moe_dequantize_mx.restype = ctypes.c_int
        L.moe_dequantize_mx.argtypes = [i64, i64, vp, vp, i32, i32, vp, vp]
        L.moe_forward_shard.restype = ctypes.c_int
        L.moe_forward_shard.argtypes = [sp] + [vp] * 4 + [i64] * 3 + [vp] * 17 + [ctypes.c_size_t, vp, vp]
        L.moe_few_workspace_size.restype = ctypes.c_size_t
        L.moe_few_workspace_size.argtypes = [sp]
        L.moe_forward_few.restype = ctypes.c_int
        L.moe_forward_few.argtypes = [sp] + [vp] * 20 + [ctypes.c_size_t, vp]
        L.moe_forward_routed.restype = ctypes.c_int
        L.moe_forward_routed.argtypes = [sp] + [vp] * 18 + [ctypes.c_size_t, vp]
        L.moe_expert_utilization.restype = ctypes.c_int
        L.moe_expert_utilization.argtypes = [i64] + [vp] * 5
        L.moe_forward_noalloc.restype = ctypes.c_int
        L.moe_forward_noalloc.argtypes = [sp] + [vp] * 19 + [vp]
        L.moe_status_string.restype = ctypes.c_char_p
        L.moe_status_string.argtypes = [ctypes.c_int]
        _LIB = L
    return _LIB


def moe_status_string(status: int) -> str:
    return lib().moe_status_string(status).decode()


def _act_code(t: torch.Tensor) -> int:
    return {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16}.get(t.dtype, -1)


def _w_code(t: torch.Tensor, cols=None) -> int:
    """Weight type of a stored matrix [.., out, in]; byte tensors of half the `cols` input features hold MXFP4."""
    if cols is not None and t.element_size() == 1 and t.shape[-1] * 2 == cols:
        return MOE_MXFP4
    return {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16, torch.uint8: MOE_FP8_E4M3,
            torch.float8_e4m3fn: MOE_FP8_E4M3}.get(t.dtype, -1)


def make_shape(T, d, E, k, inter, inter_shared, act_dtype, w_dtype) -> moe_shape_t:
    return moe_shape_t(T, d, E, k, inter, inter_shared, act_dtype, w_dtype)


def moe_workspace_size(shape: moe_shape_t) -> int:
    return int(lib().moe_workspace_size(ctypes.byref(shape)))


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(dev):
    if dev.type != "cuda":
        raise ValueError(f"Expected a cuda device, but got: {dev}")
    # the handle alone: a torch.cuda.Stream object costs 2 us, a sixth of a small call
    return ctypes.c_void_p(torch._C._cuda_getCurrentRawStream(dev.index))


def _on(dev):
    """A context in which `dev` is the current device (kernels are launched there)."""
    here = dev.type == "cuda" and dev.index == torch.cuda.current_device()
    return contextlib.nullcontext() if here else torch.cuda.device(dev)


def _workspace(shape, dev, workspace):
    need = moe_workspace_size(shape)
    if need == 0:
        raise MoeError(2, "moe_workspace_size")
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    return workspace, need


def moe_route(x, Wg, bias, k, workspace=None, allowed=None, n_group=None):
    """Routing of x [T, d]: returns dict(idx, w, counts, offsets, sorted_slots, pos) as device tensors.

    With `allowed` (uint8 [E] device tensor) calls moe_route_limited (device-limited routing); with
    `n_group` moe_route_grouped (group-limited routing)."""
    T, d = x.shape
    E = Wg.shape[0]
    shape = make_shape(T, d, E, k, 128, 128, _act_code(x), _act_code(x))
    dev = x.device
    workspace, need = _workspace(shape, dev, workspace)
    i32 = dict(dtype=torch.int32, device=dev)
    out = dict(idx=torch.empty((T, k), **i32), w=torch.empty((T, k), dtype=torch.float32, device=dev),
               counts=torch.empty(E, **i32), offsets=torch.empty(E + 1, **i32),
               sorted_slots=torch.empty(T * k, **i32), pos=torch.empty(T * k, **i32))
    tail = [_ptr(out["idx"]), _ptr(out["w"]), _ptr(out["counts"]), _ptr(out["offsets"]),
            _ptr(out["sorted_slots"]), _ptr(out["pos"]), _ptr(workspace), workspace.numel(), _stream(dev)]
    if allowed is not None and n_group is not None:
        raise ValueError("a routing mask and group-limited routing do not combine")
    if allowed is not None:
        _check_allowed(allowed, E)
        st, name = lib().moe_route_limited(ctypes.byref(shape), _ptr(x), _ptr(Wg), _ptr(bias), _ptr(allowed),
                                           *tail), "moe_route_limited"
    elif n_group is not None:
        st, name = lib().moe_route_grouped(ctypes.byref(shape), int(n_group), _ptr(x), _ptr(Wg), _ptr(bias),
                                           *tail), "moe_route_grouped"
    else:
        st, name = lib().moe_route(ctypes.byref(shape), _ptr(x), _ptr(Wg), _ptr(bias), *tail), "moe_route"
    if st:
        raise MoeError(st, name)
    return out


def moe_route_limited(x, Wg, bias, allowed, k, workspace=None):
    """Device-limited routing: moe_route with the per-expert mask `allowed` (uint8 [E] device tensor)."""
    return moe_route(x, Wg, bias, k, workspace=workspace, allowed=allowed)


def moe_quantize_e4m3(x):
    """fp8 activation quantisation of a bf16 [rows, cols] device tensor: (E4M3 codes uint8 [rows, cols],
    fp32 scales [rows, cols / 128])."""
    if x.dtype != torch.bfloat16 or x.dim() != 2 or not x.is_contiguous():
        raise ValueError("x must be a contiguous 2-D bf16 tensor")
    rows, cols = x.shape
    q = torch.empty((rows, cols), dtype=torch.uint8, device=x.device)
    s = torch.empty((rows, max(cols // 128, 0)), dtype=torch.float32, device=x.device)
    st = lib().moe_quantize_e4m3(rows, cols, _ptr(x), _ptr(q), _ptr(s), _stream(x.device))
    if st:
        raise MoeError(st, "moe_quantize_e4m3")
    return q, s


def moe_quantize_mx(x, fmt):
    """Quantise a bf16 or fp32 [rows, cols] device tensor to MOE_MXFP4 or MOE_MXFP8: (codes, scales), uint8.

    Codes [rows, cols / 2] (MXFP4, two to a byte, the lower column in the low half) or [rows, cols] (MXFP8:
    E4M3); scales [rows, cols / 32], E8M0 bytes."""
    if x.dtype not in (torch.bfloat16, torch.float32) or x.dim() != 2 or not x.is_contiguous():
        raise ValueError("x must be a contiguous 2-D bf16 or fp32 tensor")
    rows, cols = x.shape
    q = torch.empty((rows, cols // 2 if fmt == MOE_MXFP4 else cols), dtype=torch.uint8, device=x.device)
    s = torch.empty((rows, cols // 32), dtype=torch.uint8, device=x.device)
    with _on(x.device):
        st = lib().moe_quantize_mx(rows, cols, _ptr(x), _act_code(x), fmt, _ptr(q), _ptr(s), _stream(x.device))
    if st:
        raise MoeError(st, "moe_quantize_mx")
    return q, s


def moe_dequantize_mx(q, scales, fmt, dtype=torch.bfloat16):
    """The values [rows, cols] (bf16 or fp32) of what moe_quantize_mx returned for format `fmt`."""
    rows, cols = scales.shape[0], scales.shape[-1] * 32
    if q.shape != (rows, cols // 2 if fmt == MOE_MXFP4 else cols) or scales.dim() != 2:
        raise ValueError("codes and scales do not have the shapes of one matrix")
    if q.element_size() != 1 or scales.element_size() != 1 or not q.is_contiguous() or not scales.is_contiguous():
        raise ValueError("codes and scales must be contiguous byte tensors")
    if q.device != scales.device:
        raise ValueError("codes and scales must be on one device")
    if dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("dtype must be bf16 or fp32")
    out = torch.empty((rows, cols), dtype=dtype, device=q.device)
    with _on(q.device):
        st = lib().moe_dequantize_mx(rows, cols, _ptr(q), _ptr(scales), fmt, _act_code(out), _ptr(out), _stream(q.device))
    if st:
        raise MoeError(st, "moe_dequantize_mx")
    return out


def moe_route_grouped(x, Wg, bias, k, n_group, workspace=None):
    """Group-limited routing: two experts from each of the k / 2 best of n_group expert groups."""
    return moe_route(x, Wg, bias, k, workspace=workspace, n_group=n_group)


def _check_allowed(allowed, E):
    if allowed.dtype != torch.uint8 or allowed.numel() != E or not allowed.is_contiguous():
        raise ValueError("allowed must be a contiguous uint8 tensor of E entries")


def moe_forward(x, Wg, bias, W1, W3, W2, S1, S3, S2, k, scales=None, y=None, workspace=None, routing=False,
                events=None):
    """Layer output y [T, d] (x's dtype).  `scales`: dict of W1s, W3s, W2s, S1s, S3s, S2s for fp8
    (fp32 block scales) and MXFP4 weights (E8M0 bytes; the weights [.., out, in / 2] bytes).

    With routing=True returns (y, dict(idx, w, counts)).  With `events` (a ctypes array of
    NUM_STAGES + 1 hipEvent_t handles) calls moe_forward_staged, which records them between stages.
    """
    T, d = x.shape
    E, inter = W1.shape[0], W1.shape[1]
    inter_s = S1.shape[0]
    shape = make_shape(T, d, E, k, inter, inter_s, _act_code(x), _w_code(W1, d))
    dev = x.device
    workspace, need = _workspace(shape, dev, workspace)
    if y is None:
        y = torch.empty_like(x)
    sc = scales or {}
    r = None
    if routing:
        r = dict(idx=torch.empty((T, k), dtype=torch.int32, device=dev),
                 w=torch.empty((T, k), dtype=torch.float32, device=dev),
                 counts=torch.empty(E, dtype=torch.int32, device=dev))
    args = [ctypes.byref(shape), _ptr(x), _ptr(Wg), _ptr(bias), _ptr(W1), _ptr(W3), _ptr(W2),
            _ptr(sc.get("W1s")), _ptr(sc.get("W3s")), _ptr(sc.get("W2s")), _ptr(S1), _ptr(S3), _ptr(S2),
            _ptr(sc.get("S1s")), _ptr(sc.get("S3s")), _ptr(sc.get("S2s")), _ptr(y),
            _ptr(r and r["idx"]), _ptr(r and r["w"]), _ptr(r and r["counts"]),
            _ptr(workspace), workspace.numel(), _stream(dev)]
    if events is not None:
        st = lib().moe_forward_staged(*args, ctypes.cast(events, ctypes.c_void_p))
    else:
        st = lib().moe_forward(*args)
    if st:
        raise MoeError(st, "moe_forward")
    return (y, r) if routing else y


_SCALES = ("W1s", "W3s", "W2s", "S1s", "S3s", "S2s")


def _layer(x, k, E, W1, W3, W2, S1, S3, S2, scales, y, vectors):
    """Checks one layer call's tensors; returns (shape, scales, y).  `vectors`: (name, tensor or None, dtype, shape)
    of the call's other inputs."""
    if x.dim() != 2 or x.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("x must be a 2-D bf16 or fp32 tensor")
    T, d = x.shape
    if W1.dim() != 3 or S1.dim() != 2:
        raise ValueError("W1 must be [E, inter, d], S1 [inter_shared, d]")
    inter, inter_s = W1.shape[1], S1.shape[0]
    w = _w_code(W1, d)
    half = 2 if w == MOE_MXFP4 else 1
    sc = dict(scales or {})
    want = [("W1", W1, (E, inter, d // half)), ("W3", W3, (E, inter, d // half)), ("W2", W2, (E, d, inter // half)),
            ("S1", S1, (inter_s, d // half)), ("S3", S3, (inter_s, d // half)), ("S2", S2, (d, inter_s // half))]
    tensors = [("x", x, None)]
    for name, t, size in want:
        if t.shape != size or _w_code(t, size[-1] * half) != w:
            raise ValueError(f"{name} must be {list(size)} with W1's type")
        tensors.append((name, t, None))
        if w in (MOE_FP8_E4M3, MOE_MXFP4):
            s = sc.get(name + "s")
            ssize = size[:-2] + ((size[-2], size[-1] * half // 32) if half == 2 else (size[-2] // 128, size[-1] // 128))
            if s is None or s.shape != ssize or s.element_size() != (1 if half == 2 else 4):
                raise ValueError(f"scales[{name}s] must be {list(ssize)} {'E8M0 bytes' if half == 2 else 'fp32'}")
            tensors.append((name + "s", s, None))
    for name, t, dtype, size in vectors:
        if t is not None and (t.dtype != dtype or t.shape != size):
            raise ValueError(f"{name} must be {list(size)} {dtype}")
        tensors.append((name, t, None))
    if y is None:
        y = torch.empty_like(x, memory_format=torch.contiguous_format)
    elif y.shape != x.shape or y.dtype != x.dtype:
        raise ValueError("y must have x's shape and type")
    for name, t, _ in tensors + [("y", y, None)]:
        if t is not None and (not t.is_contiguous() or t.device != x.device):
            raise ValueError(f"{name} must be contiguous and on x's device")
    return make_shape(T, d, E, k, inter, inter_s, _act_code(x), w), sc, y


def moe_forward_routed(x, idx, w, W1, W3, W2, S1, S3, S2, scales=None, y=None, workspace=None, counts=False):
    """The layer for a given routing: idx int32 [T, k] (an entry outside [0, E) is a slot without an expert), w fp32
    [T, k].  Weights and `scales` as moe_forward.  With counts=True returns (y, counts int32 [E])."""
    if idx.dim() != 2:
        raise ValueError("idx must be [T, k]")
    k, E = idx.shape[1], W1.shape[0]
    shape, sc, y = _layer(x, k, E, W1, W3, W2, S1, S3, S2, scales, y,
                          [("idx", idx, torch.int32, (x.shape[0], k)), ("w", w, torch.float32, (x.shape[0], k))])
    dev = x.device
    with _on(dev):
        workspace, need = _workspace(shape, dev, workspace)
        c = torch.empty(E, dtype=torch.int32, device=dev) if counts else None
        if counts and x.shape[0] == 0:
            c.zero_()                                  # no tokens: the library writes nothing
        st = lib().moe_forward_routed(ctypes.byref(shape), _ptr(x), _ptr(idx), _ptr(w), _ptr(W1), _ptr(W3), _ptr(W2),
                                      *[_ptr(sc.get(n)) for n in _SCALES[:3]], _ptr(S1), _ptr(S3), _ptr(S2),
                                      *[_ptr(sc.get(n)) for n in _SCALES[3:]], _ptr(y), _ptr(c), _ptr(workspace),
                                      workspace.numel(), _stream(dev))
    if st:
        raise MoeError(st, "moe_forward_routed")
    return (y, c) if counts else y


def moe_few_workspace_size(shape: moe_shape_t) -> int:
    return int(lib().moe_few_workspace_size(ctypes.byref(shape)))


def moe_forward_few(x, Wg, bias, W1, W3, W2, S1, S3, S2, k, scales=None, y=None, workspace=None, routing=False):
    """moe_forward for at most FEW_MAX_T tokens, in two launches made for latency.  Arguments and results as
    moe_forward; the workspace holds moe_few_workspace_size bytes."""
    T, d = x.shape
    E = W1.shape[0]
    shape, sc, y = _layer(x, k, E, W1, W3, W2, S1, S3, S2, scales, y,
                          [("Wg", Wg, torch.float32, (E, d)), ("bias", bias, torch.float32, (E,))])
    dev = x.device
    with _on(dev):
        if workspace is None:
            need = moe_few_workspace_size(shape)
            if need == 0:
                raise MoeError(2, "moe_few_workspace_size")
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        r = None
        if routing:
            r = dict(idx=torch.empty((T, k), dtype=torch.int32, device=dev),
                     w=torch.empty((T, k), dtype=torch.float32, device=dev),
                     counts=torch.empty(E, dtype=torch.int32, device=dev))
            if T == 0:
                r["counts"].zero_()                    # no tokens: the library writes nothing
        st = lib().moe_forward_few(ctypes.byref(shape), _ptr(x), _ptr(Wg), _ptr(bias), _ptr(W1), _ptr(W3), _ptr(W2),
                                   *[_ptr(sc.get(n)) for n in _SCALES[:3]], _ptr(S1), _ptr(S3), _ptr(S2),
                                   *[_ptr(sc.get(n)) for n in _SCALES[3:]], _ptr(y), _ptr(r and r["idx"]),
                                   _ptr(r and r["w"]), _ptr(r and r["counts"]), _ptr(workspace), workspace.numel(),
                                   _stream(dev))
    if st:
        raise MoeError(st, "moe_forward_few")
    return (y, r) if routing else y


def moe_forward_noalloc(x, Wg, bias, W1, W3, W2, S1, S3, S2, k, scales=None, y=None, routing=False):
    """moe_forward_noalloc: moe_forward with the library's static device scratch as its workspace (nothing is
    allocated by the call itself; y and the routing copies are allocated here unless given)."""
    T, d = x.shape
    E, inter = W1.shape[0], W1.shape[1]
    shape = make_shape(T, d, E, k, inter, S1.shape[0], _act_code(x), _w_code(W1, d))
    dev = x.device
    if y is None:
        y = torch.empty_like(x)
    sc = scales or {}
    r = None
    if routing:
        r = dict(idx=torch.empty((T, k), dtype=torch.int32, device=dev),
                 w=torch.empty((T, k), dtype=torch.float32, device=dev),
                 counts=torch.empty(E, dtype=torch.int32, device=dev))
    with _on(dev):      # the library uses the current device's scratch array
        st = lib().moe_forward_noalloc(ctypes.byref(shape), _ptr(x), _ptr(Wg), _ptr(bias), _ptr(W1), _ptr(W3),
                                       _ptr(W2), _ptr(sc.get("W1s")), _ptr(sc.get("W3s")), _ptr(sc.get("W2s")),
                                       _ptr(S1), _ptr(S3), _ptr(S2), _ptr(sc.get("S1s")), _ptr(sc.get("S3s")),
                                       _ptr(sc.get("S2s")), _ptr(y), _ptr(r and r["idx"]), _ptr(r and r["w"]),
                                       _ptr(r and r["counts"]), _stream(dev))
    if st:
        raise MoeError(st, "moe_forward_noalloc")
    return (y, r) if routing else y


def forward_inputs_noalloc(inp: dict, k: int, **kw):
    """moe_forward_noalloc over a dict produced by workloads.generate (device tensors)."""
    scales = {n: inp[n] for n in ("W1s", "W3s", "W2s", "S1s", "S3s", "S2s") if inp.get(n) is not None}
    return moe_forward_noalloc(inp["x"], inp["Wg"], inp.get("bias"), inp["W1"], inp["W3"], inp["W2"], inp["S1"],
                               inp["S3"], inp["S2"], k, scales=scales or None, **kw)


def forward_inputs(inp: dict, k: int, **kw):
    """moe_forward over a dict produced by workloads.generate (device tensors)."""
    scales = {n: inp[n] for n in ("W1s", "W3s", "W2s", "S1s", "S3s", "S2s") if inp.get(n) is not None}
    return moe_forward(inp["x"], inp["Wg"], inp.get("bias"), inp["W1"], inp["W3"], inp["W2"], inp["S1"], inp["S3"],
                       inp["S2"], k, scales=scales or None, **kw)


def moe_forward_shard(x, Wg, bias, k, e0, e1, W1, W3, W2, S1, S3, S2, inter, inter_shared, allowed=None,
                      scales=None, y_partial=None, workspace=None, routing=False, events=None):
    """One expert-parallel rank's fp32 partial output [T, d] (moe_forward_shard).

    W1, W3 [e1-e0, inter, d], W2 [e1-e0, d, inter]: the rank's experts (None when e0 == e1);
    S1, S3 [n_shared, d], S2 [d, n_shared]: its shared slice (None for none); `inter`, `inter_shared`:
    the layer's full widths.  With routing=True returns (y_partial, dict(idx, w, counts)).  `events`: as in
    moe_forward (NUM_STAGES + 1 hipEvent_t handles recorded between stages).
    """
    T, d = x.shape
    E = Wg.shape[0]
    n_shared = 0 if S1 is None else S1.shape[0]
    wt = W1 if W1 is not None else S1
    shape = make_shape(T, d, E, k, inter, inter_shared, _act_code(x), _w_code(wt, d) if wt is not None else _act_code(x))
    dev = x.device
    workspace, need = _workspace(shape, dev, workspace)
    if y_partial is None:
        y_partial = torch.empty((T, d), dtype=torch.float32, device=dev)
    if allowed is not None:
        _check_allowed(allowed, E)
    sc = scales or {}
    r = None
    if routing:
        r = dict(idx=torch.empty((T, k), dtype=torch.int32, device=dev),
                 w=torch.empty((T, k), dtype=torch.float32, device=dev),
                 counts=torch.empty(E, dtype=torch.int32, device=dev))
    st = lib().moe_forward_shard(ctypes.byref(shape), _ptr(x), _ptr(Wg), _ptr(bias), _ptr(allowed), e0, e1, n_shared,
                                 _ptr(W1), _ptr(W3), _ptr(W2), _ptr(sc.get("W1s")), _ptr(sc.get("W3s")),
                                 _ptr(sc.get("W2s")), _ptr(S1), _ptr(S3), _ptr(S2), _ptr(sc.get("S1s")),
                                 _ptr(sc.get("S3s")), _ptr(sc.get("S2s")), _ptr(y_partial),
                                 _ptr(r and r["idx"]), _ptr(r and r["w"]), _ptr(r and r["counts"]),
                                 _ptr(workspace), workspace.numel(), _stream(dev),
                                 None if events is None else ctypes.cast(events, ctypes.c_void_p))
    if st:
        raise MoeError(st, "moe_forward_shard")
    return (y_partial, r) if routing else y_partial


def shard_weights(inp: dict, e0: int, e1: int, s0: int, s1: int) -> dict:
    """The rank-local weight arrays of experts [e0, e1) and shared features [s0, s1) of a full-layer dict
    (as workloads.generate makes), stored densely as moe_forward_shard expects."""
    scaled = inp.get("W1s") is not None
    half = 2 if inp["S2"].shape[1] * 2 == inp["S1"].shape[0] else 1          # MXFP4: two codes to a byte
    out = {}
    if e1 > e0:
        for n in ("W1", "W3", "W2") + (("W1s", "W3s", "W2s") if scaled else ()):
            out[n] = inp[n][e0:e1].contiguous()
    if s1 > s0:
        out["S1"] = inp["S1"][s0:s1].contiguous()
        out["S3"] = inp["S3"][s0:s1].contiguous()
        out["S2"] = inp["S2"][:, s0 // half:s1 // half].contiguous()
        if half == 2:
            out["S1s"] = inp["S1s"][s0:s1].contiguous()
            out["S3s"] = inp["S3s"][s0:s1].contiguous()
            out["S2s"] = inp["S2s"][:, s0 // 32:s1 // 32].contiguous()
        elif scaled:
            out["S1s"] = inp["S1s"][s0 // 128:s1 // 128].contiguous()
            out["S3s"] = inp["S3s"][s0 // 128:s1 // 128].contiguous()
            out["S2s"] = inp["S2s"][:, s0 // 128:s1 // 128].contiguous()
    return out


def shard_inputs(inp: dict, k: int, e0: int, e1: int, s0: int, s1: int, **kw):
    """moe_forward_shard over a workloads.generate dict: slices the rank's weights, then calls it."""
    lw = shard_weights(inp, e0, e1, s0, s1)
    scales = {n: lw[n] for n in ("W1s", "W3s", "W2s", "S1s", "S3s", "S2s") if n in lw}
    return moe_forward_shard(inp["x"], inp["Wg"], inp.get("bias"), k, e0, e1, lw.get("W1"), lw.get("W3"),
                             lw.get("W2"), lw.get("S1"), lw.get("S3"), lw.get("S2"), inp["W1"].shape[1],
                             inp["S1"].shape[0], scales=scales or None, **kw)


def moe_expert_utilization(counts):
    """(util fp32 [E], flags int32 [E], summary int32 [2]) of an int32 [E] device tensor of counts."""
    E = counts.numel()
    dev = counts.device
    util = torch.empty(E, dtype=torch.float32, device=dev)
    flags = torch.empty(E, dtype=torch.int32, device=dev)
    summary = torch.empty(2, dtype=torch.int32, device=dev)
    st = lib().moe_expert_utilization(E, _ptr(counts), _ptr(util), _ptr(flags), _ptr(summary), _stream(dev))
    if st:
        raise MoeError(st, "moe_expert_utilization")
    return util, flags, summary
