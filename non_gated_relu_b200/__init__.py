"""Python binding of libnhmoe, the B200 (sm_100a) Nemotron-H non-gated MoE block.

Argument marshalling only: every step of the block runs in the CUDA kernels
behind the C ABI declared in ``include/nh_moe.h``.  PyTorch supplies device
memory and streams.  There is no CPU fallback: when the library cannot be
built or loaded, or no sm_100 device is present, the calls raise.

Low level (same names as the C ABI, minus the ``nh_moe_`` prefix):
``route``, ``permute``, ``forward``, ``shared``, ``zero_acc``, ``finalize``,
``check_device``, ``workspace_size``, ``workspace_layout``,
``shared_workspace_size``, ``validate``, ``selftest_timeout``.

From router logits: ``gate`` (sigmoid or softmax scores, bias, groups, top-k) and
its gradient ``gate_backward``; ``route_scored`` runs the router and the gate.

FP8 (E4M3 with a scale per block of 128): ``fp8_quantize`` (rows),
``fp8_quantize_weight``, ``fp8_weight``, ``fp8_linear``, and ``forward_fp8``,
``experts_up_fp8`` / ``experts_down_fp8``, ``shared_fp8`` / ``shared_store_fp8``
for a config with ``weight_format`` "fp8".

Block level: :class:`NemotronHMoE` (``block.py``) holds the weights and
buffers and runs one block call on two streams (optionally as a CUDA graph).
"""
from __future__ import annotations

import ctypes
import os
import threading

from . import build as _build

__all__ = ["NHMoEError", "Config", "Layout", "config_from", "load", "validate", "workspace_size",
           "workspace_layout", "shared_workspace_size", "route", "route_noalloc", "route_permute", "permute", "forward", "experts_up", "experts_down", "shared", "forward_nvfp4", "shared_nvfp4", "nvfp4_weight",
           "zero_acc", "finalize", "latent_config", "latent_workspace_size",
           "latent_in", "latent_out", "GateConfig", "Fp8Weight", "gate_config", "gate",
           "gate_backward", "route_scored", "fp8_weight", "fp8_quantize", "fp8_quantize_weight",
           "fp8_linear", "fp8_linear_workspace_size", "forward_fp8", "experts_up_fp8",
           "experts_down_fp8", "shared_fp8", "shared_store_fp8", "reset_status", "check_device", "selftest_timeout", "library_path", "NemotronHMoE"]

NH_OK, NH_ERR_INVALID_ARG, NH_ERR_UNSUPPORTED, NH_ERR_CUDA, NH_ERR_TIMEOUT, NH_ERR_DEVICE_CHECK = range(6)
STATUS_NAMES = {0: "NH_OK", 1: "NH_ERR_INVALID_ARG", 2: "NH_ERR_UNSUPPORTED", 3: "NH_ERR_CUDA",
                4: "NH_ERR_TIMEOUT", 5: "NH_ERR_DEVICE_CHECK"}
NH_F32, NH_BF16 = 0, 1


class NHMoEError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


class Config(ctypes.Structure):
    """nh_moe_config (field names of the model's config.json)."""
    _fields_ = [("hidden_size", ctypes.c_int32), ("n_routed_experts", ctypes.c_int32),
                ("n_group", ctypes.c_int32), ("topk_group", ctypes.c_int32),
                ("num_experts_per_tok", ctypes.c_int32), ("moe_intermediate_size", ctypes.c_int32),
                ("moe_shared_expert_intermediate_size", ctypes.c_int32),
                ("n_shared_experts", ctypes.c_int32), ("norm_topk_prob", ctypes.c_int32),
                ("routed_scaling_factor", ctypes.c_float), ("dtype", ctypes.c_int32),
                ("group_score", ctypes.c_int32), ("weight_format", ctypes.c_int32),
                ("latent_size", ctypes.c_int32)]


class NvFp4Weight(ctypes.Structure):
    """nh_nvfp4_weight: device pointers of one stacked NVFP4 tensor."""
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("global_scale", ctypes.c_void_p)]


class Fp8Weight(ctypes.Structure):
    """nh_fp8_weight: device pointers of one stacked FP8 tensor (and, on the Python
    side, its shape, device and the tensors themselves)."""
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


class GateConfig(ctypes.Structure):
    """nh_moe_gate_config."""
    _fields_ = [("n_routed_experts", ctypes.c_int32), ("n_group", ctypes.c_int32),
                ("topk_group", ctypes.c_int32), ("num_experts_per_tok", ctypes.c_int32),
                ("norm_topk_prob", ctypes.c_int32), ("routed_scaling_factor", ctypes.c_float),
                ("score_func", ctypes.c_int32), ("group_score", ctypes.c_int32),
                ("dtype", ctypes.c_int32)]


NH_WEIGHTS_NATIVE, NH_WEIGHTS_NVFP4, NH_WEIGHTS_FP8 = 0, 1, 2
NH_SCORE_SIGMOID, NH_SCORE_SOFTMAX = 0, 1
_WEIGHT_FORMATS = {"native": 0, "nvfp4": 1, "fp8": 2, 0: 0, 1: 1, 2: 2}
_SCORE_FUNCS = {"sigmoid": 0, "softmax": 1, 0: 0, 1: 1}


class Layout(ctypes.Structure):
    """nh_moe_ws_layout: byte offsets of the routed-path workspace regions."""
    _fields_ = [(n, ctypes.c_size_t) for n in (
        "total_bytes", "status", "logits", "router_w", "counts", "offsets", "chunk_counts", "perm_token",
        "perm_w", "inv_row", "tiles", "num_tiles", "x_perm", "h", "ready")] + [
        ("rows_alloc", ctypes.c_int64), ("tile_rows", ctypes.c_int32),
        ("max_tiles", ctypes.c_int32), ("n_chunks", ctypes.c_int32), ("swap_ab", ctypes.c_int32),
        ("x_direct", ctypes.c_int32)]


def config_from(c, group_score: int = 0) -> Config:
    """Build the C struct from any object with the config.json attribute names
    (and ``dtype`` in {"bf16", "f32"}; ``weight_format`` "native" (also None or without the
    field), "nvfp4" or "fp8")."""
    if isinstance(c, Config):
        return c
    dt = getattr(c, "dtype", "bf16")
    fmt = getattr(c, "weight_format", None)
    if fmt is not None and fmt not in _WEIGHT_FORMATS:
        raise ValueError(f"unknown weight_format {fmt!r}")
    return Config(int(c.hidden_size), int(c.n_routed_experts), int(c.n_group), int(c.topk_group),
                  int(c.num_experts_per_tok), int(c.moe_intermediate_size),
                  int(c.moe_shared_expert_intermediate_size), int(c.n_shared_experts),
                  int(bool(c.norm_topk_prob)), float(c.routed_scaling_factor),
                  NH_BF16 if dt in ("bf16", NH_BF16) else NH_F32,
                  int(getattr(c, "group_score", group_score)),
                  NH_WEIGHTS_NATIVE if fmt is None else _WEIGHT_FORMATS[fmt],
                  int(getattr(c, "latent_size", 0) or 0))


_lock = threading.Lock()
_lib = None

_EXPORTS = ["nh_moe_validate", "nh_moe_workspace_size", "nh_moe_workspace_layout",
            "nh_moe_shared_workspace_size", "nh_moe_route", "nh_moe_route_noalloc", "nh_moe_route_permute",
            "nh_moe_permute", "nh_moe_forward", "nh_moe_experts_up", "nh_moe_experts_down",
            "nh_moe_forward_nvfp4", "nh_moe_shared", "nh_moe_shared_store", "nh_moe_shared_nvfp4",
            "nh_moe_zero_acc",
            "nh_moe_finalize",
            "nh_moe_latent_config", "nh_moe_latent_workspace_size", "nh_moe_latent_in",
            "nh_moe_latent_out", "nh_moe_route_scored", "nh_moe_gate", "nh_moe_gate_backward",
            "nh_fp8_quantize", "nh_fp8_quantize_weight", "nh_fp8_linear_workspace_size",
            "nh_fp8_linear", "nh_moe_forward_fp8", "nh_moe_experts_up_fp8",
            "nh_moe_experts_down_fp8", "nh_moe_shared_fp8", "nh_moe_shared_store_fp8",
            "nh_moe_reset_status", "nh_moe_check_device",
            "nh_moe_selftest_timeout",
            "nh_last_error", "nh_version"]


def library_path() -> str:
    return _build.LIB


def load():
    """Build (if sources changed) and load libnhmoe.so; raise if impossible."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = _build.build()
        lib = ctypes.CDLL(path)
        P, S, I64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int64
        C = ctypes.POINTER(Config)
        G, W8, I32 = ctypes.POINTER(GateConfig), ctypes.POINTER(Fp8Weight), ctypes.c_int32
        sig = {
            "nh_moe_validate": [C],
            "nh_moe_workspace_size": [C, I64, ctypes.POINTER(S)],
            "nh_moe_workspace_layout": [C, I64, ctypes.POINTER(Layout)],
            "nh_moe_shared_workspace_size": [C, I64, ctypes.POINTER(S)],
            "nh_moe_route": [C, I64, P, P, P, P, P, P, S, P],
            "nh_moe_route_noalloc": [C, I64, P, P, P, P, P, P],
            "nh_moe_route_permute": [C, I64, P, P, P, P, P, P, S, P],
            "nh_moe_permute": [C, I64, P, P, P, P, S, P],
            "nh_moe_forward": [C, I64, P, P, P, P, S, P, P],
            "nh_moe_experts_up": [C, I64, P, P, P, S, P],
            "nh_moe_experts_down": [C, I64, P, P, S, P, P],
            "nh_moe_shared": [C, I64, P, P, P, P, P, S, P],
            "nh_moe_forward_nvfp4": [C, I64, P, ctypes.POINTER(NvFp4Weight),
                                     ctypes.POINTER(NvFp4Weight), P, S, P, P],
            "nh_moe_shared_nvfp4": [C, I64, P, ctypes.POINTER(NvFp4Weight),
                                    ctypes.POINTER(NvFp4Weight), P, P, S, P],
            "nh_moe_zero_acc": [C, I64, P, P],
            "nh_moe_finalize": [C, I64, P, P, P],
            "nh_moe_latent_config": [C, C],
            "nh_moe_latent_workspace_size": [C, I64, ctypes.POINTER(S)],
            "nh_moe_latent_in": [C, I64, P, P, P, P, S, P],
            "nh_moe_latent_out": [C, I64, P, P, P, P, S, P],
            "nh_moe_route_scored": [C, I32, I64, P, P, P, P, P, P, S, P],
            "nh_moe_gate": [G, I64, P, P, P, P, P],
            "nh_moe_gate_backward": [G, I64, P, P, P, P, P],
            "nh_fp8_quantize": [I64, I64, P, I32, P, P, P],
            "nh_fp8_quantize_weight": [I64, I64, I64, P, I32, P, P, P],
            "nh_fp8_linear_workspace_size": [I64, I64, I64, ctypes.POINTER(S)],
            "nh_fp8_linear": [I64, I64, I64, P, I32, W8, P, I32, P, S, P],
            "nh_moe_forward_fp8": [C, I64, P, W8, W8, P, S, P, P],
            "nh_moe_experts_up_fp8": [C, I64, P, W8, P, S, P],
            "nh_moe_experts_down_fp8": [C, I64, W8, P, S, P, P],
            "nh_moe_shared_fp8": [C, I64, P, W8, W8, P, P, S, P],
            "nh_moe_shared_store_fp8": [C, I64, P, W8, W8, P, P, S, P],
            "nh_moe_check_device": [P, P],
            "nh_moe_reset_status": [P, P],
            "nh_moe_selftest_timeout": [P, ctypes.c_uint64, P],
        }
        for name, args in sig.items():
            f = getattr(lib, name)
            f.argtypes = args
            f.restype = ctypes.c_int
        lib.nh_last_error.restype = ctypes.c_char_p
        lib.nh_version.restype = ctypes.c_char_p
        _lib = lib
        return lib


def _check(rc: int):
    if rc != NH_OK:
        raise NHMoEError(rc, load().nh_last_error().decode())


def _p(t):
    """Device pointer of a tensor (or None)."""
    if t is None:
        return None
    if hasattr(t, "data_ptr"):
        if not t.is_contiguous():
            raise ValueError("tensors passed to libnhmoe must be contiguous")
        return ctypes.c_void_p(t.data_ptr())
    return ctypes.c_void_p(int(t))


def _stream(stream):
    if stream is None:
        t = _types()
        if t.raw_stream is not None:     # 0.3 us; a Stream object takes 3.5
            return t.raw_stream(t.current_device())
        return ctypes.c_void_p(t.torch.cuda.current_stream().cuda_stream)
    if hasattr(stream, "cuda_stream"):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _nbytes(t):
    return t.numel() * t.element_size()


def validate(cfg):
    _check(load().nh_moe_validate(ctypes.byref(config_from(cfg))))


def workspace_size(cfg, T: int) -> int:
    n = ctypes.c_size_t()
    _check(load().nh_moe_workspace_size(ctypes.byref(config_from(cfg)), T, ctypes.byref(n)))
    return n.value


def workspace_layout(cfg, T: int) -> Layout:
    lay = Layout()
    _check(load().nh_moe_workspace_layout(ctypes.byref(config_from(cfg)), T, ctypes.byref(lay)))
    return lay


def shared_workspace_size(cfg, T: int) -> int:
    n = ctypes.c_size_t()
    _check(load().nh_moe_shared_workspace_size(ctypes.byref(config_from(cfg)), T,
                                               ctypes.byref(n)))
    return n.value


def _sigmoid_config(cfg) -> Config:
    """config_from for the routers whose scores are sigmoids: another ``scoring_func`` in
    the config is refused."""
    score = getattr(cfg, "scoring_func", None)
    if score is not None and _SCORE_FUNCS.get(score) != NH_SCORE_SIGMOID:
        raise ValueError(f"scoring_func {score!r}: this router's scores are sigmoids, "
                         "use route_scored")
    return config_from(cfg)


def route(cfg, x, w_router, bias, topk_idx, topk_w, ws, stream=None):
    c = _sigmoid_config(cfg)
    _check(load().nh_moe_route(ctypes.byref(c), x.shape[0], _p(x), _p(w_router), _p(bias),
                               _p(topk_idx), _p(topk_w), _p(ws), _nbytes(ws), _stream(stream)))


def route_noalloc(cfg, x, w_router, bias, topk_idx, topk_w, stream=None):
    """Router of decode-sized batches (T <= 32) without a workspace argument: its
    scratch is a fixed array inside the library (see nh_moe_route_noalloc)."""
    c = _sigmoid_config(cfg)
    _check(load().nh_moe_route_noalloc(ctypes.byref(c), x.shape[0], _p(x), _p(w_router),
                                       _p(bias), _p(topk_idx), _p(topk_w), _stream(stream)))


def route_permute(cfg, x, w_router, bias, topk_idx, topk_w, ws, stream=None):
    """route + permute in one call (one kernel for T <= 32)."""
    c = _sigmoid_config(cfg)
    _check(load().nh_moe_route_permute(ctypes.byref(c), x.shape[0], _p(x), _p(w_router), _p(bias),
                                       _p(topk_idx), _p(topk_w), _p(ws), _nbytes(ws),
                                       _stream(stream)))


def permute(cfg, x, topk_idx, topk_w, ws, stream=None):
    c = config_from(cfg)
    _check(load().nh_moe_permute(ctypes.byref(c), x.shape[0], _p(x), _p(topk_idx), _p(topk_w),
                                 _p(ws), _nbytes(ws), _stream(stream)))


def forward(cfg, x, w_up, w_down, ws, y_acc, stream=None):
    """Routed experts: y_acc[token] += the token's weighted expert outputs (float32)."""
    c = config_from(cfg)
    _check(load().nh_moe_forward(ctypes.byref(c), x.shape[0], _p(x), _p(w_up), _p(w_down), _p(ws),
                                 _nbytes(ws), _p(y_acc), _stream(stream)))


def experts_up(cfg, x, w_up, ws, stream=None):
    c = config_from(cfg)
    _check(load().nh_moe_experts_up(ctypes.byref(c), x.shape[0], _p(x), _p(w_up), _p(ws),
                                    _nbytes(ws), _stream(stream)))


def experts_down(cfg, T: int, w_down, ws, y_acc, stream=None):
    c = config_from(cfg)
    _check(load().nh_moe_experts_down(ctypes.byref(c), T, _p(w_down), _p(ws), _nbytes(ws),
                                      _p(y_acc), _stream(stream)))


def shared(cfg, x, w_shared_up, w_shared_down, y_acc, ws_shared, stream=None):
    """Shared expert: y_acc += relu(x W_su^T)^2 W_sd^T (float32)."""
    c = config_from(cfg)
    _check(load().nh_moe_shared(ctypes.byref(c), x.shape[0], _p(x), _p(w_shared_up),
                                _p(w_shared_down), _p(y_acc), _p(ws_shared),
                                _nbytes(ws_shared), _stream(stream)))


def shared_store(cfg, x, w_shared_up, w_shared_down, y_acc, ws_shared, stream=None):
    """Shared expert as y_acc's starting value: y_acc = relu(x W_su^T)^2 W_sd^T."""
    c = config_from(cfg)
    _check(load().nh_moe_shared_store(ctypes.byref(c), x.shape[0], _p(x), _p(w_shared_up),
                                      _p(w_shared_down), _p(y_acc), _p(ws_shared),
                                      _nbytes(ws_shared), _stream(stream)))


def nvfp4_weight(codes, scales, global_scale) -> NvFp4Weight:
    """Struct of device pointers for one stacked NVFP4 tensor (tensors stay owned by the caller)."""
    return NvFp4Weight(codes.data_ptr(), scales.data_ptr(), global_scale.data_ptr())


def forward_nvfp4(cfg, x, w_up, w_down, ws, y_acc, stream=None):
    """nh_moe_forward with NVFP4 weights; w_up / w_down are NvFp4Weight structs."""
    c = config_from(cfg)
    _check(load().nh_moe_forward_nvfp4(ctypes.byref(c), x.shape[0], _p(x), ctypes.byref(w_up),
                                       ctypes.byref(w_down), _p(ws), _nbytes(ws), _p(y_acc),
                                       _stream(stream)))


def shared_nvfp4(cfg, x, w_shared_up, w_shared_down, y_acc, ws_shared, stream=None):
    c = config_from(cfg)
    _check(load().nh_moe_shared_nvfp4(ctypes.byref(c), x.shape[0], _p(x), ctypes.byref(w_shared_up),
                                      ctypes.byref(w_shared_down), _p(y_acc), _p(ws_shared),
                                      _nbytes(ws_shared), _stream(stream)))


def zero_acc(cfg, T: int, y_acc, stream=None):
    """y_acc = 0 ([T, hidden_size] float32), asynchronously on `stream`."""
    c = config_from(cfg)
    _check(load().nh_moe_zero_acc(ctypes.byref(c), T, _p(y_acc), _stream(stream)))


def finalize(cfg, T: int, y_acc, y, stream=None):
    """y = dtype(y_acc): the one rounding of the block output."""
    c = config_from(cfg)
    _check(load().nh_moe_finalize(ctypes.byref(c), T, _p(y_acc), _p(y), _stream(stream)))


def latent_config(cfg) -> Config:
    """The expert-width config the routed-expert calls of a latent block take
    (hidden_size = latent_size, no latent projections, no shared expert)."""
    c = config_from(cfg)
    out = Config()
    _check(load().nh_moe_latent_config(ctypes.byref(c), ctypes.byref(out)))
    return out


def latent_workspace_size(cfg, T: int) -> int:
    c = config_from(cfg)
    n = ctypes.c_size_t()
    _check(load().nh_moe_latent_workspace_size(ctypes.byref(c), T, ctypes.byref(n)))
    return n.value


def latent_in(cfg, x, w_latent_fc1, x_lat, ws_latent, stream=None):
    """x_lat = dtype(x W_fc1^T)."""
    c = config_from(cfg)
    _check(load().nh_moe_latent_in(ctypes.byref(c), x.shape[0], _p(x), _p(w_latent_fc1),
                                   _p(x_lat), _p(ws_latent), _nbytes(ws_latent), _stream(stream)))


def latent_out(cfg, T: int, y_lat, w_latent_fc2, y_acc, ws_latent, stream=None):
    """y_acc += y_lat W_fc2^T (y_acc = ... without a shared expert), float32."""
    c = config_from(cfg)
    _check(load().nh_moe_latent_out(ctypes.byref(c), T, _p(y_lat), _p(w_latent_fc2), _p(y_acc),
                                    _p(ws_latent), _nbytes(ws_latent), _stream(stream)))


# ---------------------------------------------------------------------------
# The router's choice from logits, and FP8 (E4M3, a scale per block of 128).
# These calls check what they are given: types, shapes, contiguity and device.
# ---------------------------------------------------------------------------
def _dt(t) -> int:
    ty = _types()
    if t.dtype in ty.bf16:
        return NH_BF16
    if t.dtype in ty.f32:
        return NH_F32
    raise TypeError(f"expected bfloat16 or float32, got {t.dtype}")


class _Types:
    """torch and its types by what they hold (torch is imported with the first call)"""
    torch = act = f32 = bf16 = i32 = f8 = raw_stream = current_device = Tensor = None


def _types():
    if _Types.torch is None:
        import torch
        _Types.f32, _Types.bf16 = (torch.float32,), (torch.bfloat16,)
        _Types.i32, _Types.f8 = (torch.int32,), (torch.float8_e4m3fn, torch.uint8)
        _Types.act = _Types.bf16 + _Types.f32
        _Types.current_device, _Types.Tensor = torch.cuda.current_device, torch.Tensor
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        _Types.raw_stream = staticmethod(raw) if raw is not None else None
        _Types.torch = torch
    return _Types


def _args(*specs):
    """Check device tensors, each (name, tensor, types, shape); returns their pointers.
    Types, shapes and layout of all come before the device of any."""
    ty = _types()
    Tensor, dev, off, out = ty.Tensor, None, None, []
    for spec in specs:
        name, t, dtypes, shape = spec
        if not isinstance(t, Tensor):
            raise TypeError(f"{name}: expected a tensor, got {type(t).__name__}")
        if t.dtype not in dtypes:
            raise TypeError(f"{name}: expected {' or '.join(map(str, dtypes))}, got {t.dtype}")
        if t.shape != shape:
            raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
        if not t.is_contiguous():
            raise ValueError(f"{name}: tensors passed to libnhmoe must be contiguous")
        ptr = t.data_ptr()
        out.append(ptr or None)
        if ptr and off is None:
            if dev is None:
                dev = t.get_device()
                if dev < 0 or dev != ty.current_device():
                    off = spec
            elif t.get_device() != dev:
                off = spec
    if off is not None:
        raise ValueError(f"{off[0]}: on {off[1].device}, not on the current CUDA device")
    return out


def _ws_arg(name, ws):
    """(pointer, bytes) of a workspace tensor on the current device"""
    ty = _types()
    if not isinstance(ws, ty.Tensor):
        raise TypeError(f"{name}: expected a tensor, got {type(ws).__name__}")
    if not ws.is_contiguous():
        raise ValueError(f"{name}: tensors passed to libnhmoe must be contiguous")
    if ws.get_device() != ty.current_device():
        raise ValueError(f"{name}: on {ws.device}, not on the current CUDA device")
    return ws.data_ptr() or None, ws.numel() * ws.element_size()


def gate_config(n_routed_experts, num_experts_per_tok, n_group=1, topk_group=1,
                norm_topk_prob=True, routed_scaling_factor=1.0, scoring_func="sigmoid",
                group_score="max", dtype="f32") -> GateConfig:
    """Config of ``gate`` / ``gate_backward``: scoring_func "sigmoid" or "softmax",
    group_score "max" or "top2", dtype ("f32" or "bf16") of the logits."""
    try:
        score, group = _SCORE_FUNCS[scoring_func], {"max": 0, "top2": 1, 0: 0, 1: 1}[group_score]
        dt = {"f32": NH_F32, "bf16": NH_BF16, NH_F32: NH_F32, NH_BF16: NH_BF16}[dtype]
    except KeyError as e:
        raise ValueError(f"unknown scoring_func, group_score or dtype {e}") from None
    return GateConfig(int(n_routed_experts), int(n_group), int(topk_group),
                      int(num_experts_per_tok), int(bool(norm_topk_prob)),
                      float(routed_scaling_factor), score, group, dt)


def gate(cfg: GateConfig, logits, bias, topk_idx, topk_w, stream=None):
    """Choice and weights of every token from its router logits [T, E] (nh_moe_gate):
    writes topk_idx [T, k] int32 and topk_w [T, k] float32."""
    ty = _types()
    T, E, k = logits.shape[0], cfg.n_routed_experts, cfg.num_experts_per_tok
    specs = [("logits", logits, ty.bf16 if cfg.dtype == NH_BF16 else ty.f32, (T, E)),
             ("topk_idx", topk_idx, ty.i32, (T, k)), ("topk_w", topk_w, ty.f32, (T, k))]
    if bias is not None:
        specs.append(("bias", bias, ty.f32, (E,)))
    ptrs = _args(*specs)
    _check((_lib or load()).nh_moe_gate(ctypes.byref(cfg), T, ptrs[0], ptrs[3] if bias is not None else None,
                              ptrs[1], ptrs[2], _stream(stream)))


def gate_backward(cfg: GateConfig, logits, topk_idx, d_topk_w, d_logits, stream=None):
    """Gradient of the logits from that of topk_w (nh_moe_gate_backward): writes
    d_logits [T, E], in the logits' type."""
    ty = _types()
    T, E, k = logits.shape[0], cfg.n_routed_experts, cfg.num_experts_per_tok
    lt = ty.bf16 if cfg.dtype == NH_BF16 else ty.f32
    ptrs = _args(("logits", logits, lt, (T, E)), ("topk_idx", topk_idx, ty.i32, (T, k)),
                 ("d_topk_w", d_topk_w, ty.f32, (T, k)), ("d_logits", d_logits, lt, (T, E)))
    _check((_lib or load()).nh_moe_gate_backward(ctypes.byref(cfg), T, *ptrs, _stream(stream)))


def route_scored(cfg, scoring_func, x, w_router, bias, topk_idx, topk_w, ws, stream=None):
    """route with the scores of scoring_func ("sigmoid" or "softmax")."""
    c, ty = config_from(cfg), _types()
    if scoring_func not in _SCORE_FUNCS:
        raise ValueError(f"unknown scoring_func {scoring_func!r}")
    T, E, k = x.shape[0], c.n_routed_experts, c.num_experts_per_tok
    specs = [("x", x, ty.bf16 if c.dtype == NH_BF16 else ty.f32, (T, c.hidden_size)),
             ("w_router", w_router, ty.f32, (E, c.hidden_size)),
             ("topk_idx", topk_idx, ty.i32, (T, k)), ("topk_w", topk_w, ty.f32, (T, k))]
    if bias is not None:
        specs.append(("bias", bias, ty.f32, (E,)))
    ptrs = _args(*specs)
    _check(load().nh_moe_route_scored(ctypes.byref(c), _SCORE_FUNCS[scoring_func], T, ptrs[0],
                                      ptrs[1], ptrs[4] if bias is not None else None, ptrs[2],
                                      ptrs[3], *_ws_arg("ws", ws), _stream(stream)))


def fp8_weight(codes, scales) -> Fp8Weight:
    """Struct of one FP8 tensor: codes [n, rows, cols] (float8_e4m3fn or uint8) and
    scales [n, ceil(rows / 128), ceil(cols / 128)] float32.  It keeps the tensors alive."""
    ty = _types()
    if codes.dim() != 3:
        raise ValueError(f"codes: expected [n, rows, cols], got {tuple(codes.shape)}")
    n, rows, cols = codes.shape
    w = Fp8Weight(*_args(("codes", codes, ty.f8, (n, rows, cols)),
                         ("scales", scales, ty.f32, (n, -(-rows // 128), -(-cols // 128)))))
    w.shape, w.device, w.tensors = (n, rows, cols), codes.get_device(), (codes, scales)
    return w


def _fp8(name, w, shape):
    if not isinstance(w, Fp8Weight):
        raise TypeError(f"{name}: expected fp8_weight(codes, scales), got {type(w).__name__}")
    got = getattr(w, "shape", None)
    if got is not None and got != tuple(shape):
        raise ValueError(f"{name}: expected codes of shape {tuple(shape)}, got {got}")
    if got is not None and w.device != _types().current_device():
        raise ValueError(f"{name}: on cuda:{w.device}, not on the current CUDA device")
    return ctypes.byref(w)


def fp8_quantize(x, codes, scales, stream=None):
    """Rows x [T, K] (bfloat16 or float32) to E4M3 codes [T, K] and power-of-two scales
    [T, ceil(K / 128)] (nh_fp8_quantize)."""
    ty = _types()
    T, K = x.shape
    px, pc, ps = _args(("x", x, ty.act, (T, K)), ("codes", codes, ty.f8, (T, K)),
                       ("scales", scales, ty.f32, (T, -(-K // 128))))
    _check((_lib or load()).nh_fp8_quantize(T, K, px, _dt(x), pc, ps, _stream(stream)))


def _empty(shape, dtype, device, stream):
    """A tensor that a launch on `stream` writes.  torch hands memory out in the order of
    one stream's work: what the current stream still does to its last owner is not done
    when another stream's kernel starts."""
    torch = _types().torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(getattr(stream, "cuda_stream", stream)), device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(device))
    return t


def fp8_quantize_weight(w, codes=None, scales=None, stream=None):
    """w [n, rows, cols] (bfloat16 or float32) as FP8: returns (codes, scales), which
    are allocated where they are not given (on `stream`, for use on the current one, too)."""
    ty = _types()
    if w.dim() != 3:
        raise ValueError(f"w: expected [n, rows, cols], got {tuple(w.shape)}")
    n, rows, cols = w.shape
    blocks = (n, -(-rows // 128), -(-cols // 128))
    wspec = ("w", w, ty.act, (n, rows, cols))
    _args(wspec)
    if codes is None:
        codes = _empty((n, rows, cols), ty.torch.float8_e4m3fn, w.device, stream)
    if scales is None:
        scales = _empty(blocks, ty.torch.float32, w.device, stream)
    pw, pc, ps = _args(wspec, ("codes", codes, ty.f8, (n, rows, cols)), ("scales", scales, ty.f32, blocks))
    _check((_lib or load()).nh_fp8_quantize_weight(n, rows, cols, pw, _dt(w), pc, ps, _stream(stream)))
    return codes, scales


def fp8_linear_workspace_size(T: int, N: int, K: int) -> int:
    n = ctypes.c_size_t()
    _check((_lib or load()).nh_fp8_linear_workspace_size(T, N, K, ctypes.byref(n)))
    return n.value


def fp8_linear(x, w: Fp8Weight, y, ws, stream=None):
    """y [T, N] = x [T, K] W^T with E4M3 operands (nh_fp8_linear); w holds one [N, K]
    matrix, ws fp8_linear_workspace_size bytes (its status word cleared once by the
    caller: torch.zeros or reset_status)."""
    ty = _types()
    T, K = x.shape
    N = y.shape[1]
    ref = _fp8("w", w, (1, N, K))
    px, py = _args(("x", x, ty.act, (T, K)), ("y", y, ty.act, (T, N)))
    _check((_lib or load()).nh_fp8_linear(T, N, K, px, _dt(x), ref, py, _dt(y), *_ws_arg("ws", ws),
                                _stream(stream)))


def _f8_args(c, x, y_acc):
    """(T, pointer of x or None, pointer of y_acc or None)"""
    ty = _types()
    T = (x if x is not None else y_acc).shape[0]
    specs = [] if x is None else [("x", x, ty.bf16, (T, c.hidden_size))]
    if y_acc is not None:
        specs.append(("y_acc", y_acc, ty.f32, (T, c.hidden_size)))
    ptrs = _args(*specs)
    return T, None if x is None else ptrs[0], None if y_acc is None else ptrs[-1]


def forward_fp8(cfg, x, w_up: Fp8Weight, w_down: Fp8Weight, ws, y_acc, stream=None):
    """forward with FP8 weights (fp8_weight structs): y_acc += routed experts of x."""
    c = config_from(cfg)
    T, px, py = _f8_args(c, x, y_acc)
    E, H, I = c.n_routed_experts, c.hidden_size, c.moe_intermediate_size
    _check((_lib or load()).nh_moe_forward_fp8(ctypes.byref(c), T, px, _fp8("w_up", w_up, (E, I, H)),
                                     _fp8("w_down", w_down, (E, H, I)), *_ws_arg("ws", ws), py,
                                     _stream(stream)))


def experts_up_fp8(cfg, x, w_up: Fp8Weight, ws, stream=None):
    c = config_from(cfg)
    T, px, _ = _f8_args(c, x, None)
    shape = (c.n_routed_experts, c.moe_intermediate_size, c.hidden_size)
    _check(load().nh_moe_experts_up_fp8(ctypes.byref(c), T, px, _fp8("w_up", w_up, shape),
                                        *_ws_arg("ws", ws), _stream(stream)))


def experts_down_fp8(cfg, T: int, w_down: Fp8Weight, ws, y_acc, stream=None):
    c = config_from(cfg)
    _, _, py = _f8_args(c, None, y_acc)
    if y_acc.shape[0] != T:
        raise ValueError(f"y_acc: expected {T} rows, got {y_acc.shape[0]}")
    shape = (c.n_routed_experts, c.hidden_size, c.moe_intermediate_size)
    _check(load().nh_moe_experts_down_fp8(ctypes.byref(c), T, _fp8("w_down", w_down, shape),
                                          *_ws_arg("ws", ws), py, _stream(stream)))


def _shared_fp8(fn, cfg, x, w_su, w_sd, y_acc, ws_shared, stream):
    c = config_from(cfg)
    T, px, py = _f8_args(c, x, y_acc)
    H, S = c.hidden_size, c.moe_shared_expert_intermediate_size
    _check(fn(ctypes.byref(c), T, px, _fp8("w_shared_up", w_su, (1, S, H)),
              _fp8("w_shared_down", w_sd, (1, H, S)), py, *_ws_arg("ws_shared", ws_shared),
              _stream(stream)))


def shared_fp8(cfg, x, w_shared_up, w_shared_down, y_acc, ws_shared, stream=None):
    """Shared expert with FP8 weights: y_acc += relu(x W_su^T)^2 W_sd^T."""
    _shared_fp8(load().nh_moe_shared_fp8, cfg, x, w_shared_up, w_shared_down, y_acc, ws_shared,
                stream)


def shared_store_fp8(cfg, x, w_shared_up, w_shared_down, y_acc, ws_shared, stream=None):
    """shared_fp8 as y_acc's starting value."""
    _shared_fp8(load().nh_moe_shared_store_fp8, cfg, x, w_shared_up, w_shared_down, y_acc,
                ws_shared, stream)


def reset_status(ws, stream=None):
    """Clear a workspace's status word (asynchronously, on `stream`)."""
    _check(load().nh_moe_reset_status(_p(ws), _stream(stream)))


def check_device(ws, stream=None) -> int:
    """Synchronise the stream and return the workspace status word (raises on CUDA errors)."""
    rc = load().nh_moe_check_device(_p(ws), _stream(stream))
    if rc == NH_ERR_CUDA:
        _check(rc)
    return rc


def selftest_timeout(ws, timeout_ns: int, stream=None):
    _check(load().nh_moe_selftest_timeout(_p(ws), int(timeout_ns), _stream(stream)))


def last_error() -> str:
    return load().nh_last_error().decode()


from .block import NemotronHMoE  # noqa: E402
