"""Thin Python binding of libkmoe.so (include/kmoe.h).

Argument marshalling only: every step of the layer runs in the CUDA library.
PyTorch supplies device memory and the current stream. There is no CPU
fallback: if the library is missing or a call fails, an exception is raised.
"""
from __future__ import annotations

import ctypes
import os

import torch

from ._build import LIB

KMOE_OK, KMOE_ERR_INVALID_ARG, KMOE_ERR_UNSUPPORTED, KMOE_ERR_CUDA, KMOE_ERR_WORKSPACE, KMOE_ERR_DEVICE = range(6)
KMOE_F32, KMOE_BF16, KMOE_E4M3_B128, KMOE_E4M3_B128_A8, KMOE_W4 = range(5)
SCORES = {"sigmoid": 0, "softmax": 1}     # kmoe_score, kmoe_route_score
GROUP_SCORES = {"max": 0, "top2": 1}      # kmoe_group_score

# Bytes at the head of a moe_grouped_ffn workspace: the status word, tickets
# and the grouped FFN's unit counters (include/kmoe.h).
FFN_STATUS_BYTES = (64 + 1088) * 4

EXPORTS = ["moe_workspace_size", "moe_router_topk", "moe_permute", "moe_permute_noalloc", "moe_grouped_ffn",
           "moe_combine", "moe_forward", "moe_block_workspace_size", "moe_block_forward", "moe_quant_1x128",
           "moe_route", "moe_linear_w4", "moe_linear_w4_workspace_size", "moe_forward_routed", "moe_block_forward_routed", "moe_quant_w4",
           "moe_dequant_w4",
           "moe_device_status", "moe_set_wait_limit", "moe_last_error", "moe_abi_version"]


class KmoeError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"kmoe status {status}: {msg}")
        self.status = status


class _W4Struct(ctypes.Structure):
    """kmoe_w4: matrices held in 4 bits with group scales."""
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("zeros", ctypes.c_void_p),
                ("group", ctypes.c_int)]


class Experts(ctypes.Structure):
    """kmoe_experts: one stack of SwiGLU experts."""
    _fields_ = [("w_gate", ctypes.c_void_p), ("w_up", ctypes.c_void_p), ("w_down", ctypes.c_void_p),
                ("s_gate", ctypes.c_void_p), ("s_up", ctypes.c_void_p), ("s_down", ctypes.c_void_p),
                ("dtype", ctypes.c_int), ("w4", ctypes.POINTER(_W4Struct))]


class _RoutingStruct(ctypes.Structure):
    """kmoe_routing."""
    _fields_ = [("score", ctypes.c_int), ("n_groups", ctypes.c_int), ("topk_groups", ctypes.c_int),
                ("group_score", ctypes.c_int), ("renormalise", ctypes.c_int), ("scale", ctypes.c_float)]


class _Fixed:
    """An object whose C struct is made once: setting an attribute afterwards would not reach it."""
    _ref = None

    def __setattr__(self, name, value):
        if self._ref is not None:
            raise AttributeError(f"{type(self).__name__} is fixed: make another for a different {name}")
        object.__setattr__(self, name, value)


class Routing(_Fixed):
    """How experts are chosen and weighted (kmoe_routing in include/kmoe.h): scores from a sigmoid or
    a softmax over all experts, the correction bias added to the score, selection limited to the best
    groups of experts, weights optionally renormalised and scaled."""

    def __init__(self, score: str = "sigmoid", n_groups: int = 1, topk_groups: int | None = None,
                 group_score: str = "top2", renormalise: bool = True, scale: float = 1.0):
        if score not in SCORES:
            raise ValueError(f"score {score!r}: one of {sorted(SCORES)}")
        if group_score not in GROUP_SCORES:
            raise ValueError(f"group_score {group_score!r}: one of {sorted(GROUP_SCORES)}")
        self.score, self.n_groups, self.group_score = score, n_groups, group_score
        self.topk_groups = n_groups if topk_groups is None else topk_groups
        self.renormalise, self.scale = renormalise, scale
        self._struct = _RoutingStruct(SCORES[score], self.n_groups, self.topk_groups, GROUP_SCORES[group_score],
                                      int(bool(renormalise)), float(scale))
        self._ref = ctypes.byref(self._struct)


class W4(_Fixed):
    """Weights in the 4-bit format of kmoe_w4: codes uint8 [..., rows, cols / 2], scales BF16
    [..., rows, cols / group], zeros uint8 of the scales' shape or None (8 everywhere). One leading
    dimension stacks the matrices of several experts."""

    def __init__(self, codes, scales, zeros=None):
        if codes.dim() not in (2, 3) or codes.dtype != torch.uint8 or not codes.is_contiguous():
            raise ValueError("codes: a dense uint8 tensor [rows, cols / 2] or [E, rows, cols / 2]")
        self.rows, self.cols = codes.shape[-2], codes.shape[-1] * 2
        self.E = codes.shape[0] if codes.dim() == 3 else 1
        groups = scales.shape[-1] if scales.dim() else 0
        if groups < 1 or self.cols % groups:
            raise ValueError("scales: [..., rows, cols / group]")
        self.group = self.cols // groups
        shape = tuple(codes.shape[:-1]) + (groups,)
        _dense(scales, "scales", torch.bfloat16, shape, codes.device)
        if zeros is not None:
            _dense(zeros, "zeros", torch.uint8, shape, codes.device)
        self.codes, self.scales, self.zeros = codes, scales, zeros
        self._struct = _W4Struct(codes.data_ptr(), scales.data_ptr(), None if zeros is None else zeros.data_ptr(),
                                 self.group)
        self._ref = ctypes.byref(self._struct)


def _dense(t, name, dtype, shape, device):
    """Refuses a tensor that the library would read wrongly."""
    if t.dtype is not dtype and (dtype is not _ACT_DTYPES or t.dtype not in _ACT_DTYPES):
        raise ValueError(f"{name}: dtype {t.dtype} is not {dtype}")
    if t.shape != shape:                          # a tuple
        raise ValueError(f"{name}: shape {tuple(t.shape)} is not {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, not on {device}")


_lib = None


def load(path: str | None = None):
    """Load libkmoe.so (or the library named by KMOE_LIBRARY, e.g. the KMOE_DEBUG build);
    raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or os.environ.get("KMOE_LIBRARY") or LIB
    if not os.path.exists(path):
        raise RuntimeError(f"CUDA library {path} is missing: build it with __graft_entry__.build()")
    lib = ctypes.CDLL(path)
    vp, i, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    lib.moe_workspace_size.restype = sz
    lib.moe_workspace_size.argtypes = [i, i, i, i, i, i, i]
    lib.moe_last_error.restype = ctypes.c_char_p
    lib.moe_abi_version.restype = i
    lib.moe_router_topk.argtypes = [vp, i, vp, vp, i, i, i, i, i, vp, vp, vp, vp, sz, vp]
    lib.moe_permute.argtypes = [vp, i, i, i, vp, vp, vp, vp, vp, sz, vp]
    lib.moe_permute_noalloc.argtypes = [vp, i, i, i, vp, vp, vp, vp, vp]
    lib.moe_grouped_ffn.argtypes = [vp, i, i, i, i, i, i, vp, vp, ctypes.POINTER(Experts),
                                    ctypes.POINTER(Experts), vp, vp, vp, sz, vp]
    lib.moe_combine.argtypes = [vp, vp, i, vp, vp, i, i, i, vp, i, vp]
    lib.moe_forward.argtypes = [vp, i, i, i, i, i, i, i, vp, vp, ctypes.POINTER(Experts),
                                ctypes.POINTER(Experts), vp, i, vp, vp, vp, vp, sz, vp]
    lib.moe_block_workspace_size.restype = sz
    lib.moe_block_workspace_size.argtypes = [i, i, i, i, i, i]
    lib.moe_block_forward.argtypes = [vp, i, i, i, i, i, i, vp, vp, ctypes.c_float, vp, vp,
                                      ctypes.POINTER(Experts), ctypes.POINTER(Experts), vp, vp, vp, vp, vp, vp, sz, vp]
    lib.moe_quant_1x128.argtypes = [vp, i, i, vp, vp, vp]
    lib.moe_route.argtypes = [vp, i, vp, i, i, i, vp, vp, vp, vp]
    lib.moe_linear_w4.argtypes = [vp, i, i, i, i, i, i, vp, vp, vp, vp, i, vp, sz, vp]
    lib.moe_linear_w4_workspace_size.restype = sz
    lib.moe_linear_w4_workspace_size.argtypes = [i, i, i, i, i, i, i]
    lib.moe_forward_routed.argtypes = [vp, i, i, i, i, i, i, vp, vp, vp, ctypes.POINTER(Experts),
                                       ctypes.POINTER(Experts), vp, i, vp, vp, vp, vp, sz, vp]
    lib.moe_block_forward_routed.argtypes = [vp, i, i, i, i, i, vp, vp, vp, ctypes.c_float, vp, vp,
                                             ctypes.POINTER(Experts), ctypes.POINTER(Experts), vp, vp, vp, vp, vp,
                                             vp, sz, vp]
    lib.moe_quant_w4.argtypes = [vp, i, i, i, i, vp, vp, vp, vp]
    lib.moe_dequant_w4.argtypes = [vp, i, i, vp, i, vp]
    lib.moe_device_status.argtypes = [vp, ctypes.POINTER(ctypes.c_int), vp]
    lib.moe_set_wait_limit.argtypes = [ctypes.c_longlong]
    for f in ("moe_router_topk", "moe_permute", "moe_permute_noalloc", "moe_grouped_ffn", "moe_combine",
              "moe_forward", "moe_block_forward", "moe_quant_1x128", "moe_device_status", "moe_set_wait_limit",
              "moe_route", "moe_linear_w4", "moe_forward_routed", "moe_block_forward_routed", "moe_quant_w4",
              "moe_dequant_w4"):
        getattr(lib, f).restype = i
    if lib.moe_abi_version() != 3:
        raise RuntimeError("libkmoe ABI version mismatch")
    _lib = lib
    return lib


def _check(status: int):
    if status != KMOE_OK:
        raise KmoeError(status, load().moe_last_error().decode())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _call(name, t, stream, *args):
    """Calls entry point `name` for tensors on t's device: on `stream`, or on that device's current
    stream, with that device current."""
    dev = t.device.index
    if stream is None:
        s = torch._C._cuda_getCurrentRawStream(dev)
    elif stream.device != t.device:
        raise ValueError(f"stream of {stream.device} for tensors on {t.device}")
    else:
        s = stream.cuda_stream
    fn = getattr(_lib or load(), name)
    if torch._C._cuda_getDevice() == dev:
        status = fn(*args, s)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, s)
    if status:
        _check(status)


def _empty(shape, dtype, device, stream):
    """New memory of the stream that writes it: what it held before was used on that stream alone."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _on_gpu(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name}: must be on a CUDA device")


_DTYPE_CODES = {torch.float32: KMOE_F32, torch.bfloat16: KMOE_BF16}
_ACT_DTYPES = tuple(_DTYPE_CODES)


def dtype_code(t: torch.dtype) -> int:
    return _DTYPE_CODES[t]


def _act_code(t, name):
    if t not in _DTYPE_CODES:
        raise ValueError(f"{name}: dtype {t}, must be torch.float32 or torch.bfloat16")
    return _DTYPE_CODES[t]


def w_dtype_code(name: str) -> int:
    return {"f32": KMOE_F32, "bf16": KMOE_BF16, "e4m3": KMOE_E4M3_B128, "e4m3_a8": KMOE_E4M3_B128_A8,
            "w4": KMOE_W4}[name]


def act_dtype_for(w_dtype: str) -> torch.dtype:
    """dtype of the grouped FFN outputs for a weight dtype (FP32 weights -> FP32)."""
    return torch.float32 if w_dtype == "f32" else torch.bfloat16


def experts_of(layer: dict, which: str = "routed") -> Experts:
    """kmoe_experts for a generator-layout layer: routed = experts 0..E-1, shared = index E."""
    cfg = layer["cfg"]
    e = cfg.E if which == "shared" else 0
    if cfg.w_dtype == "w4":
        shapes = {"gate": (cfg.I, cfg.d), "up": (cfg.I, cfg.d), "down": (cfg.d, cfg.I)}
        w4 = []
        for m, (rows, cols) in shapes.items():
            w = W4(layer["w_" + m], layer["s_" + m], layer.get("z_" + m))
            if w.codes.dim() != 3 or (w.E <= e or w.E < cfg.E or (w.rows, w.cols) != (rows, cols)):
                raise ValueError(f"w_{m}: shape {tuple(w.codes.shape)} is not [{cfg.E} + 1, {rows}, {cols // 2}]")
            w4.append(_W4Struct(*(None if t is None else t[e].data_ptr() for t in (w.codes, w.scales, w.zeros)),
                                w.group))
        return Experts(dtype=KMOE_W4, w4=(_W4Struct * 3)(*w4))

    def at(name):
        t = layer.get(name)
        return None if t is None else ctypes.c_void_p(t[e].data_ptr() if which == "shared" else t.data_ptr())

    return Experts(at("w_gate"), at("w_up"), at("w_down"), at("s_gate"), at("s_up"), at("s_down"),
                   w_dtype_code(cfg.w_dtype))


def moe_workspace_size(N, d, E, K, I, x_dtype: int, w_dtype: int) -> int:
    return int(load().moe_workspace_size(N, d, E, K, I, x_dtype, w_dtype))


def workspace(N, d, E, K, I, x_dtype: int, w_dtype: int, device="cuda") -> torch.Tensor:
    n = moe_workspace_size(N, d, E, K, I, x_dtype, w_dtype)
    if n == 0:
        _check(KMOE_ERR_UNSUPPORTED)
    return torch.empty(n, dtype=torch.uint8, device=device)


def moe_router_topk(x, w_router, bias, K, logits=None, topk_idx=None, topk_w=None, ws=None, stream=None,
                    score="sigmoid"):
    N, d = x.shape
    E = w_router.shape[0]
    if topk_idx is None:
        topk_idx = torch.empty((N, K), dtype=torch.int32, device=x.device)
    if topk_w is None:
        topk_w = torch.empty((N, K), dtype=torch.float32, device=x.device)
    if ws is None:   # logits (if not supplied) + status + the three BF16 router terms
        ws = torch.empty(((N * E * 4 + 255) // 256) * 256 + 256 + 3 * E * d * 2, dtype=torch.uint8,
                         device=x.device)
    _check(load().moe_router_topk(_ptr(x), dtype_code(x.dtype), _ptr(w_router), _ptr(bias), N, d, E, K,
                                  SCORES[score], _ptr(logits), _ptr(topk_idx), _ptr(topk_w), _ptr(ws),
                                  0 if ws is None else ws.numel(), _stream(stream)))
    return topk_idx, topk_w


def moe_permute(topk_idx, E, ws=None, stream=None):
    N, K = topk_idx.shape
    dev = topk_idx.device
    counts = torch.empty(E, dtype=torch.int32, device=dev)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    perm = torch.empty(max(N * K, 1), dtype=torch.int32, device=dev)
    inv = torch.empty((N, K), dtype=torch.int32, device=dev)
    if ws is None:
        ws = torch.empty(max(((N + 255) // 256) * E * 4, 16), dtype=torch.uint8, device=dev)
    _check(load().moe_permute(_ptr(topk_idx), N, K, E, _ptr(counts), _ptr(offsets), _ptr(perm), _ptr(inv),
                              _ptr(ws), ws.numel(), _stream(stream)))
    return counts, offsets, perm[: N * K], inv


def moe_permute_noalloc(topk_idx, E, counts=None, offsets=None, perm=None, inv=None, stream=None):
    """moe_permute for callers that cannot hand the library a workspace.

    The library keeps the scratch in its own fixed 1 MiB device array, so the
    C call allocates nothing; the caller passes every output buffer (any left
    as None is allocated here by torch, for convenience in tests)."""
    N, K = topk_idx.shape
    dev = topk_idx.device
    counts = torch.empty(E, dtype=torch.int32, device=dev) if counts is None else counts
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev) if offsets is None else offsets
    perm = torch.empty(max(N * K, 1), dtype=torch.int32, device=dev) if perm is None else perm
    inv = torch.empty((N, K), dtype=torch.int32, device=dev) if inv is None else inv
    _check(load().moe_permute_noalloc(_ptr(topk_idx), N, K, E, _ptr(counts), _ptr(offsets), _ptr(perm), _ptr(inv),
                                      _stream(stream)))
    return counts, offsets, perm[: N * K], inv


def moe_grouped_ffn(x, layer, perm_token, offsets, with_shared=True, ws=None, stream=None, out=None):
    cfg = layer["cfg"]
    N, d = x.shape
    I, E, K = cfg.I, cfg.E, cfg.K
    adt = act_dtype_for(cfg.w_dtype)
    if out is not None:
        y_perm, y_shared = out
    else:
        y_perm = torch.empty((N * K, d), dtype=adt, device=x.device)
        y_shared = torch.empty((N, d), dtype=adt, device=x.device) if with_shared else None
    if ws is None:
        ws = workspace(N, d, E, K, I, dtype_code(x.dtype), w_dtype_code(cfg.w_dtype), x.device)
    routed = experts_of(layer, "routed")
    shared = experts_of(layer, "shared") if with_shared else None
    _check(load().moe_grouped_ffn(_ptr(x), dtype_code(x.dtype), N, d, I, E, K, _ptr(perm_token), _ptr(offsets),
                                  ctypes.byref(routed), ctypes.byref(shared) if shared is not None else None,
                                  _ptr(y_perm), _ptr(y_shared), _ptr(ws), ws.numel(), _stream(stream)))
    return y_perm, y_shared


def moe_device_status(ws, stream=None) -> int:
    """Synchronises `stream` and returns the device status word of workspace `ws` (0 = ok)."""
    st = ctypes.c_int(-1)
    rc = load().moe_device_status(_ptr(ws), ctypes.byref(st), _stream(stream))
    if rc not in (KMOE_OK, KMOE_ERR_DEVICE):
        _check(rc)
    return st.value


def moe_set_wait_limit(cycles: int):
    """Give-up limit (SM cycles) of the FFN kernels' pipeline waits for this host thread; 0 = default."""
    _check(load().moe_set_wait_limit(int(cycles)))


def moe_combine(y_perm, y_shared, topk_w, inv_pos, y_dtype=torch.bfloat16, out=None, stream=None):
    N, K = topk_w.shape
    d = y_perm.shape[1]
    y = out if out is not None else torch.empty((N, d), dtype=y_dtype, device=y_perm.device)
    _check(load().moe_combine(_ptr(y_perm), _ptr(y_shared), dtype_code(y_perm.dtype), _ptr(topk_w), _ptr(inv_pos),
                              N, K, d, _ptr(y), dtype_code(y.dtype), _stream(stream)))
    return y


def moe_block_workspace_size(N, d, E, K, I, w_dtype: int) -> int:
    return int(load().moe_block_workspace_size(N, d, E, K, I, w_dtype))


class Layer:
    """Device-resident weights of one layer plus a reusable workspace.

    `forward(x)` is one moe_forward call and `block_forward(h, ...)` one
    moe_block_forward call (workspace sized for it when `block` is set);
    outputs are written into tensors owned here (or passed in). With `routing`
    (a Routing) both choose and weigh the experts by it (moe_forward_routed,
    moe_block_forward_routed), `score` is not used and the layer's bias may be
    None. `grouped_ffn` is one moe_grouped_ffn call on the same workspace. A
    workspace serves one call at a time: calls on several streams, and graphs
    that may run at the same time, need a Layer each."""

    def __init__(self, layer: dict, max_tokens: int, y_dtype=torch.bfloat16, score: str = "sigmoid",
                 block: bool = False, routing: Routing | None = None):
        self.layer = layer
        self.routing = routing
        cfg = self.cfg = layer["cfg"]
        self.routed = experts_of(layer, "routed")
        self.shared = experts_of(layer, "shared")
        self._routed_ref, self._shared_ref = ctypes.byref(self.routed), ctypes.byref(self.shared)
        dev = layer["w_gate"].device
        self.x_code = w_dtype_code(cfg.x_dtype)
        if block:
            n = moe_block_workspace_size(max_tokens, cfg.d, cfg.E, cfg.K, cfg.I, w_dtype_code(cfg.w_dtype))
            if n == 0:
                _check(KMOE_ERR_UNSUPPORTED)
            self.ws = torch.empty(n, dtype=torch.uint8, device=dev)
        else:
            self.ws = workspace(max_tokens, cfg.d, cfg.E, cfg.K, cfg.I, self.x_code, w_dtype_code(cfg.w_dtype), dev)
        self.y_dtype = y_dtype
        self.max_tokens = max_tokens
        self.score = SCORES[score]

    def _check_routed(self, x, topk_idx, topk_w, counts):
        """Refuses what a call with `routing` on x [N, d] would misread."""
        cfg, L, dev = self.cfg, self.layer, x.device
        _on_gpu(x, "x")
        _dense(L["w_router"], "w_router", torch.float32, (cfg.E, cfg.d), dev)
        for t, name, dtype, shape in ((L["bias"], "bias", torch.float32, (cfg.E,)),
                                      (topk_idx, "topk_idx", torch.int32, (x.shape[0], cfg.K)),
                                      (topk_w, "topk_w", torch.float32, (x.shape[0], cfg.K)),
                                      (counts, "counts", torch.int32, (cfg.E,))):
            if t is not None:
                _dense(t, name, dtype, shape, dev)

    def forward(self, x, y=None, topk_idx=None, topk_w=None, counts=None, stream=None):
        cfg = self.cfg
        N = x.shape[0]
        if N > self.max_tokens:
            raise ValueError("more tokens than the workspace was sized for")
        if y is None:
            y = _empty((N, cfg.d), self.y_dtype, x.device, stream)
        L = self.layer
        if self.routing is not None:
            _dense(x, "x", _ACT_DTYPES, (N, cfg.d), self.ws.device)
            _dense(y, "y", _ACT_DTYPES, (N, cfg.d), x.device)
            self._check_routed(x, topk_idx, topk_w, counts)
            _call("moe_forward_routed", x, stream, _ptr(x), dtype_code(x.dtype), N, cfg.d, cfg.E, cfg.K, cfg.I,
                  self.routing._ref, _ptr(L["w_router"]), _ptr(L["bias"]), ctypes.byref(self.routed),
                  ctypes.byref(self.shared), _ptr(y), dtype_code(y.dtype), _ptr(topk_idx), _ptr(topk_w), _ptr(counts),
                  _ptr(self.ws), self.ws.numel())
            return y
        _check(load().moe_forward(_ptr(x), dtype_code(x.dtype), N, cfg.d, cfg.E, cfg.K, cfg.I, self.score,
                                  _ptr(L["w_router"]), _ptr(L["bias"]), ctypes.byref(self.routed),
                                  ctypes.byref(self.shared), _ptr(y), dtype_code(y.dtype), _ptr(topk_idx),
                                  _ptr(topk_w), _ptr(counts), _ptr(self.ws), self.ws.numel(), _stream(stream)))
        return y

    def block_forward(self, h, gamma_pre, gamma_post, eps: float, h_out=None, topk_idx=None, topk_w=None,
                      counts=None, x_out=None, stream=None):
        """h_out = h + RMSNorm(layer(x)) * gamma_post with x = bf16(RMSNorm(h) * gamma_pre); h_out may
        be h; x_out (optional) receives x."""
        cfg = self.cfg
        N = h.shape[0]
        if N > self.max_tokens:
            raise ValueError("more tokens than the workspace was sized for")
        if h_out is None:
            h_out = _empty(h.shape, h.dtype, h.device, stream)
        L = self.layer
        if self.routing is not None:
            for t, name in ((h, "h"), (h_out, "h_out"), (x_out, "x_out")):
                if t is not None:
                    _dense(t, name, torch.bfloat16, (N, cfg.d), self.ws.device)
            for t, name in ((gamma_pre, "gamma_pre"), (gamma_post, "gamma_post")):
                _dense(t, name, torch.bfloat16, (cfg.d,), h.device)
            self._check_routed(h, topk_idx, topk_w, counts)
            _call("moe_block_forward_routed", h, stream, _ptr(h), N, cfg.d, cfg.E, cfg.K, cfg.I, self.routing._ref,
                  _ptr(gamma_pre), _ptr(gamma_post), float(eps), _ptr(L["w_router"]), _ptr(L["bias"]),
                  ctypes.byref(self.routed), ctypes.byref(self.shared), _ptr(h_out), _ptr(x_out), _ptr(topk_idx),
                  _ptr(topk_w), _ptr(counts), _ptr(self.ws), self.ws.numel())
            return h_out
        _check(load().moe_block_forward(_ptr(h), N, cfg.d, cfg.E, cfg.K, cfg.I, self.score, _ptr(gamma_pre),
                                        _ptr(gamma_post), float(eps), _ptr(L["w_router"]), _ptr(L["bias"]),
                                        ctypes.byref(self.routed), ctypes.byref(self.shared), _ptr(h_out),
                                        _ptr(x_out), _ptr(topk_idx), _ptr(topk_w), _ptr(counts), _ptr(self.ws),
                                        self.ws.numel(), _stream(stream)))
        return h_out


    def grouped_ffn(self, x, perm_token, offsets, with_shared=True, out=None, stream=None):
        """moe_grouped_ffn: y_perm [N*K, d] and y_shared [N, d] (None without the shared expert) of x
        dispatched by perm_token and offsets (moe_permute)."""
        cfg = self.cfg
        N = x.shape[0]
        if N > self.max_tokens:
            raise ValueError("more tokens than the workspace was sized for")
        _dense(x, "x", _ACT_DTYPES, (N, cfg.d), self.ws.device)
        _dense(perm_token, "perm_token", torch.int32, (N * cfg.K,), x.device)
        _dense(offsets, "offsets", torch.int32, (cfg.E + 1,), x.device)
        adt = act_dtype_for(cfg.w_dtype)
        if out is None:
            y_perm = _empty((N * cfg.K, cfg.d), adt, x.device, stream)
            y_shared = _empty((N, cfg.d), adt, x.device, stream) if with_shared else None
        else:
            y_perm, y_shared = out
            _dense(y_perm, "y_perm", adt, (N * cfg.K, cfg.d), x.device)
            if with_shared:
                _dense(y_shared, "y_shared", adt, (N, cfg.d), x.device)
        _call("moe_grouped_ffn", x, stream, x.data_ptr(), _DTYPE_CODES[x.dtype], N, cfg.d, cfg.I, cfg.E, cfg.K,
              perm_token.data_ptr(), offsets.data_ptr(), self._routed_ref, self._shared_ref if with_shared else None,
              y_perm.data_ptr(), y_shared.data_ptr() if with_shared else None, self.ws.data_ptr(), self.ws.numel())
        return y_perm, y_shared


def moe_forward(x, layer, y_dtype=torch.bfloat16, with_outputs=False, stream=None, score="sigmoid", routing=None):
    """One whole-layer call; with_outputs also returns (topk_idx, topk_w, counts)."""
    cfg = layer["cfg"]
    N = x.shape[0]
    with torch.cuda.stream(stream):      # the workspace, given back on return, is that stream's, too
        lay = Layer(layer, N, y_dtype, score, routing=routing)
        if not with_outputs:
            return lay.forward(x, stream=stream)
        idx = torch.empty((N, cfg.K), dtype=torch.int32, device=x.device)
        w = torch.empty((N, cfg.K), dtype=torch.float32, device=x.device)
        counts = torch.empty(cfg.E, dtype=torch.int32, device=x.device)
        y = lay.forward(x, topk_idx=idx, topk_w=w, counts=counts, stream=stream)
        return y, idx, w, counts


def moe_block_forward(h, layer, gamma_pre, gamma_post, eps: float, with_outputs=False, stream=None,
                      score="sigmoid", h_out=None, routing=None):
    """One sandwich-block call; with_outputs also returns (x, topk_idx, topk_w, counts)."""
    cfg = layer["cfg"]
    N = h.shape[0]
    with torch.cuda.stream(stream):      # as in moe_forward
        lay = Layer(layer, N, torch.bfloat16, score, block=True, routing=routing)
        if not with_outputs:
            return lay.block_forward(h, gamma_pre, gamma_post, eps, h_out=h_out, stream=stream)
        idx = torch.empty((N, cfg.K), dtype=torch.int32, device=h.device)
        w = torch.empty((N, cfg.K), dtype=torch.float32, device=h.device)
        counts = torch.empty(cfg.E, dtype=torch.int32, device=h.device)
        x = torch.empty_like(h)
        out = lay.block_forward(h, gamma_pre, gamma_post, eps, h_out=h_out, topk_idx=idx, topk_w=w, counts=counts,
                                x_out=x, stream=stream)
        return out, x, idx, w, counts


def moe_quant_1x128(x, codes=None, scales=None, stream=None):
    """E4M3 codes (uint8 [rows, cols]) and FP32 scales ([rows, cols / 128]) of BF16 x."""
    rows, cols = x.shape
    if codes is None:
        codes = torch.empty((rows, cols), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty((rows, cols // 128), dtype=torch.float32, device=x.device)
    _check(load().moe_quant_1x128(_ptr(x), rows, cols, _ptr(codes), _ptr(scales), _stream(stream)))
    return codes, scales


def moe_route(logits, K, bias=None, routing=None, topk_idx=None, topk_w=None, stream=None):
    """Experts and weights of logits [N, E] (FP32 or BF16) by `routing` (a Routing; the default is a
    renormalised sigmoid): topk_idx [N, K] int32, topk_w [N, K] FP32."""
    if logits.dim() != 2:
        raise ValueError("logits: [N, E]")
    N, E = logits.shape
    dev = logits.device
    _on_gpu(logits, "logits")
    _dense(logits, "logits", _ACT_DTYPES, (N, E), dev)
    if bias is not None:
        _dense(bias, "bias", torch.float32, (E,), dev)
    if topk_idx is None:
        topk_idx = _empty((N, K), torch.int32, dev, stream)
    else:
        _dense(topk_idx, "topk_idx", torch.int32, (N, K), dev)
    if topk_w is None:
        topk_w = _empty((N, K), torch.float32, dev, stream)
    else:
        _dense(topk_w, "topk_w", torch.float32, (N, K), dev)
    _call("moe_route", logits, stream, logits.data_ptr(), _DTYPE_CODES[logits.dtype],
          None if bias is None else bias.data_ptr(), N, E, K, (routing or _DEFAULT_ROUTING)._ref, topk_idx.data_ptr(),
          topk_w.data_ptr())
    return topk_idx, topk_w


_DEFAULT_ROUTING = Routing()


def moe_quant_w4(w, group=128, zeros=False, out=None, stream=None) -> W4:
    """w [..., rows, cols] (FP32 or BF16) in the 4-bit format, with zero points if `zeros`. `out`: a W4 of
    the same shape, group and zero points, which is overwritten."""
    if w.dim() not in (2, 3):
        raise ValueError("w: [rows, cols] or [E, rows, cols]")
    _on_gpu(w, "w")
    _dense(w, "w", _ACT_DTYPES, w.shape, w.device)
    lead, cols = tuple(w.shape[:-1]), w.shape[-1]
    if group not in (32, 64, 128) or cols % 128 or cols < 128:
        raise ValueError(f"group {group} (32, 64 or 128) of cols {cols} (a multiple of 128)")
    if out is None:
        shape = lead + (cols // group,)
        out = W4(_empty(lead + (cols // 2,), torch.uint8, w.device, stream),
                 _empty(shape, torch.bfloat16, w.device, stream),
                 _empty(shape, torch.uint8, w.device, stream) if zeros else None)
    elif tuple(out.codes.shape) != lead + (cols // 2,) or out.group != group or (out.zeros is None) == bool(zeros) \
            or out.codes.device != w.device:
        raise ValueError("out: another shape, group, device or zero points")
    _call("moe_quant_w4", w, stream, w.data_ptr(), _DTYPE_CODES[w.dtype], w.numel() // cols, cols, group,
          out.codes.data_ptr(), out.scales.data_ptr(), None if out.zeros is None else out.zeros.data_ptr())
    return out


def moe_dequant_w4(w4: W4, dtype=torch.bfloat16, out=None, stream=None):
    """The values of 4-bit weights, [..., rows, cols] in FP32 (exact) or BF16 (rounded)."""
    shape = tuple(w4.codes.shape[:-1]) + (w4.cols,)
    _on_gpu(w4.codes, "codes")
    if out is None:
        _act_code(dtype, "out")
        out = _empty(shape, dtype, w4.codes.device, stream)
    else:
        _dense(out, "out", _ACT_DTYPES, shape, w4.codes.device)
    _call("moe_dequant_w4", w4.codes, stream, w4._ref, out.numel() // w4.cols, w4.cols, out.data_ptr(),
          _DTYPE_CODES[out.dtype])
    return out


def moe_linear_w4_workspace_size(N, P, rows, cols, E=1, group=128, y_dtype=torch.bfloat16) -> int:
    return int(load().moe_linear_w4_workspace_size(N, P, rows, cols, E, group, _act_code(y_dtype, "y")))


def moe_linear_w4(x, w4: W4, perm_token=None, offsets=None, y_dtype=torch.bfloat16, out=None, ws=None, stream=None):
    """y[p] = W_e x[perm_token[p]] with 4-bit weights: one matrix for all rows, or (offsets [E + 1], from
    moe_permute) the matrix of the expert whose range holds p. x [N, cols] BF16; y [P, rows]."""
    if x.dim() != 2:
        raise ValueError("x: [N, cols]")
    _on_gpu(x, "x")
    dev = x.device
    N = x.shape[0]
    _dense(x, "x", torch.bfloat16, (N, w4.cols), dev)
    if w4.codes.device != dev:
        raise ValueError(f"w4: on {w4.codes.device}, not on {dev}")
    P = N
    if perm_token is not None:
        P = perm_token.numel()
        _dense(perm_token, "perm_token", torch.int32, (P,), dev)
    if offsets is not None:
        _dense(offsets, "offsets", torch.int32, (w4.E + 1,), dev)
    if out is None:
        _act_code(y_dtype, "y")
        out = _empty((P, w4.rows), y_dtype, dev, stream)
    else:
        _dense(out, "out", _ACT_DTYPES, (P, w4.rows), dev)
    code = _DTYPE_CODES[out.dtype]
    if ws is None and code == KMOE_BF16:
        need = (_lib or load()).moe_linear_w4_workspace_size(N, P, w4.rows, w4.cols, w4.E, w4.group, code)
        if need:
            ws = _empty(need, torch.uint8, dev, stream)
    elif ws is not None:
        _dense(ws, "ws", torch.uint8, (ws.numel(),), dev)
    _call("moe_linear_w4", x, stream, x.data_ptr(), KMOE_BF16, N, P, w4.rows, w4.cols, w4.E,
          None if perm_token is None else perm_token.data_ptr(), None if offsets is None else offsets.data_ptr(),
          w4._ref, out.data_ptr(), code, None if ws is None else ws.data_ptr(), 0 if ws is None else ws.numel())
    return out
