"""ctypes binding of libparo (include/paro.h).

Argument marshalling only: every step of the rotated W4A16 linear runs in the
HIP kernels of libparo.so.  PyTorch provides device memory and streams.  The
library must have been built (rotation_int4_weight_amd.build); there is no
fallback of any kind: a missing library or a failing call raises.
"""
from __future__ import annotations

import ctypes
import os

PKG = os.path.dirname(os.path.abspath(__file__))
# PARO_LIB names another build of the same library (e.g. one with host-side
# sanitizers); by default the in-tree libparo.so is loaded.
LIB_PATH = os.environ.get("PARO_LIB") or os.path.join(PKG, "libparo.so")

F16, BF16, F32 = 0, 1, 2
KV4_F16, KV4_BF16 = 16, 17  # caches in four bits, for rows in fp16 or bf16
PATH_AUTO, PATH_DECODE_FUSED, PATH_DECODE_SPLIT, PATH_PREFILL = 0, 1, 2, 3
STATUS = {0: "PARO_OK", 1: "PARO_ERR_NULL", 2: "PARO_ERR_SHAPE", 3: "PARO_ERR_DTYPE",
          4: "PARO_ERR_ALIGN", 5: "PARO_ERR_UNSUPPORTED", 6: "PARO_ERR_PAIRS",
          7: "PARO_ERR_WORKSPACE", 8: "PARO_ERR_HIP"}
EXPORTS = ("paro_scale_rotate", "paro_w4_unpack_dequant", "paro_w4a16_linear",
           "paro_w4a16_linear_path", "paro_w4a16_linear_prerotated",
           "paro_w4a16_linear_prepared", "paro_w4a16_linear_prepared_workspace_bytes",
           "paro_w4a16_linear_prepared_multi", "paro_w4a16_linear_prepared_multi_workspace_bytes",
           "paro_w4a16_linear_tiled_multi",
           "paro_w4a16_linear_noalloc",
           "paro_w4_quantize_pack", "paro_scale_rotate_backward", "paro_w4a16_moe_linear",
           "paro_w4a16_moe_linear_workspace_bytes", "paro_mxfp4_quantize_weight",
           "paro_mxfp4_quantize_activations", "paro_mxfp4_gemm", "paro_mxfp4_linear",
           "paro_mxfp4_linear_workspace_bytes", "paro_mxfp4_activation_workspace_bytes",
           "paro_mxfp4_linear_prepared", "paro_mxfp4_linear_prepared_workspace_bytes",
           "paro_scale_rotate_backward_workspace_bytes",
           "paro_tiled_bytes", "paro_rotation_matrix_bytes", "paro_rotation_matrix",
           "paro_scale_rotate_tiled", "paro_w4a16_linear_tiled",
           "paro_w4a16_linear_workspace_bytes",
           "paro_w4a16_linear_choose_path", "paro_validate_layer", "paro_last_error",
           "paro_abi_version", "paro_attention_prompt", "paro_attention_prompt_cached",
           "paro_attention_prompt_cached_workspace_bytes", "paro_attention_decode", "paro_attention_decode_workspace_bytes", "paro_kv_append",
           "paro_kv_read", "paro_kv_reserve", "paro_kv_fork", "paro_kv_free", "paro_kv_compact",
           "paro_kv_workspace_bytes", "paro_rotary", "paro_rotary_frequencies")


class ParoError(RuntimeError):
    def __init__(self, status: int, what: str, msg: str):
        super().__init__(f"{what}: {STATUS.get(status, status)}: {msg}")
        self.status = status


class ParoLayerC(ctypes.Structure):
    _fields_ = [("in_features", ctypes.c_int64), ("out_features", ctypes.c_int64),
                ("group_size", ctypes.c_int32), ("krot", ctypes.c_int32),
                ("pairs", ctypes.c_void_p), ("theta", ctypes.c_void_p),
                ("channel_scales", ctypes.c_void_p), ("qweight", ctypes.c_void_p),
                ("qzeros", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("bias", ctypes.c_void_p)]


class ParoAttentionShapeC(ctypes.Structure):
    _fields_ = [("q_heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("causal", ctypes.c_int32), ("scale", ctypes.c_float),
                ("q_token", ctypes.c_int64), ("q_head", ctypes.c_int64),
                ("k_token", ctypes.c_int64), ("k_head", ctypes.c_int64),
                ("v_token", ctypes.c_int64), ("v_head", ctypes.c_int64),
                ("y_token", ctypes.c_int64), ("y_head", ctypes.c_int64)]


class ParoKvCacheC(ctypes.Structure):
    _fields_ = [("layers", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("num_pages", ctypes.c_int64), ("slots", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("dt", ctypes.c_int), ("k", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("refs", ctypes.c_void_p), ("table", ctypes.c_void_p),
                ("lengths", ctypes.c_void_p)]


class ParoRotaryShapeC(ctypes.Structure):
    _fields_ = [("heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("rot_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("inverse", ctypes.c_int32), ("magnitude", ctypes.c_float),
                ("x_token", ctypes.c_int64), ("x_head", ctypes.c_int64),
                ("y_token", ctypes.c_int64), ("y_head", ctypes.c_int64)]


class ParoRotaryScalingC(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("base", ctypes.c_double), ("factor", ctypes.c_double),
                ("context", ctypes.c_double), ("low", ctypes.c_double), ("high", ctypes.c_double)]


_lib = None


def load(path: str | None = None):
    """Load libparo.so; raises if it has not been built."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    path = path or LIB_PATH
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with `python -m rotation_int4_weight_amd.build`")
    lib = ctypes.CDLL(path)
    P, I64, I32, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    lib.paro_scale_rotate.argtypes = [P, P, I32, I64, P, I32, P]
    lib.paro_w4_unpack_dequant.argtypes = [P, P, P, P, I32, P]
    lib.paro_w4a16_linear.argtypes = [P, P, I32, I64, P, I32, P, SZ, P]
    lib.paro_w4a16_linear_path.argtypes = [P, P, I32, I64, P, I32, P, SZ, P, I32]
    lib.paro_w4a16_linear_prerotated.argtypes = [P, P, I32, I64, P, I32, P, SZ, P, I32]
    lib.paro_w4a16_linear_prepared.argtypes = [P, P, P, I32, I64, P, I32, P, SZ, P]
    lib.paro_w4a16_linear_prepared_workspace_bytes.argtypes = [P, I64]
    lib.paro_w4a16_linear_prepared_workspace_bytes.restype = SZ
    lib.paro_w4a16_linear_prepared_multi.argtypes = [P, ctypes.c_int, P, P, I32, I64, P, I32, P, SZ, P]
    lib.paro_w4a16_linear_prepared_multi_workspace_bytes.argtypes = [P, ctypes.c_int, I64]
    lib.paro_w4a16_linear_prepared_multi_workspace_bytes.restype = SZ
    lib.paro_w4a16_linear_tiled_multi.argtypes = [P, ctypes.c_int, P, I32, I64, P, I32, P]
    lib.paro_w4a16_linear_noalloc.argtypes = [P, P, I32, I64, P, I32, P]
    lib.paro_tiled_bytes.argtypes = [P, I64]
    lib.paro_tiled_bytes.restype = SZ
    lib.paro_w4_quantize_pack.argtypes = [P, P, I32, I32, P, P, P, P]
    lib.paro_w4a16_moe_linear.argtypes = [P, I32, P, P, I32, I64, P, I32, P, SZ, P]
    lib.paro_w4a16_moe_linear_workspace_bytes.argtypes = [P, I64, I32]
    lib.paro_w4a16_moe_linear_workspace_bytes.restype = SZ
    lib.paro_mxfp4_quantize_weight.argtypes = [P, P, I32, P, P, P]
    lib.paro_mxfp4_quantize_activations.argtypes = [P, P, I32, I64, P, P, P, SZ, P]
    lib.paro_mxfp4_activation_workspace_bytes.argtypes = [P]
    lib.paro_mxfp4_activation_workspace_bytes.restype = SZ
    lib.paro_mxfp4_gemm.argtypes = [P, P, I64, P, P, I64, I64, P, P, I32, P]
    lib.paro_mxfp4_linear.argtypes = [P, P, P, P, I32, I64, P, I32, P, SZ, P]
    lib.paro_mxfp4_linear_workspace_bytes.argtypes = [P, I64]
    lib.paro_mxfp4_linear_workspace_bytes.restype = SZ
    lib.paro_mxfp4_linear_prepared.argtypes = [P, P, P, P, P, I32, I64, P, I32, P, SZ, P]
    lib.paro_mxfp4_linear_prepared_workspace_bytes.argtypes = [P, I64]
    lib.paro_mxfp4_linear_prepared_workspace_bytes.restype = SZ
    lib.paro_scale_rotate_backward.argtypes = [P, P, I32, P, I32, I64, P, I32, P, P, P, SZ, P]
    lib.paro_scale_rotate_backward_workspace_bytes.argtypes = [P, I64]
    lib.paro_scale_rotate_backward_workspace_bytes.restype = SZ
    lib.paro_rotation_matrix_bytes.argtypes = [P]
    lib.paro_rotation_matrix_bytes.restype = SZ
    lib.paro_rotation_matrix.argtypes = [P, I32, P, P]
    lib.paro_scale_rotate_tiled.argtypes = [P, P, P, I32, I64, P, P]
    lib.paro_w4a16_linear_tiled.argtypes = [P, P, I32, I64, P, I32, P]
    lib.paro_w4a16_linear_workspace_bytes.argtypes = [P, I64, I32, I32]
    lib.paro_w4a16_linear_workspace_bytes.restype = SZ
    lib.paro_w4a16_linear_choose_path.argtypes = [P, I64]
    lib.paro_validate_layer.argtypes = [P]
    lib.paro_attention_prompt.argtypes = [P, P, P, P, I32, P, P, I64, I64, I64, P, P]
    lib.paro_attention_prompt_cached.argtypes = [P, I32, P, P, P, P, I64, I64, P, P, SZ, P]
    lib.paro_attention_prompt_cached_workspace_bytes.argtypes = [P, I64, I64, I32]
    lib.paro_attention_prompt_cached_workspace_bytes.restype = SZ
    lib.paro_attention_decode.argtypes = [P, I32, P, P, P, I64, P, P, SZ, P]
    lib.paro_attention_decode_workspace_bytes.argtypes = [P, I64, I32]
    lib.paro_attention_decode_workspace_bytes.restype = SZ
    lib.paro_kv_append.argtypes = [P, I32, P, I64, I64, P, I64, I64, P, P, P, I64, I64, P]
    lib.paro_kv_read.argtypes = [P, I32, P, I64, I64, P, I64, I64, I32, P, P, P, I64, I64, P]
    lib.paro_rotary.argtypes = [ctypes.POINTER(ParoRotaryShapeC), P, I32, P, P, I64, P, P]
    lib.paro_rotary_frequencies.argtypes = [P, I32, P, P]
    lib.paro_kv_reserve.argtypes = [P, P, P, I64, P, P, SZ, P]
    lib.paro_kv_fork.argtypes = [P, P, P, I64, P, P, SZ, P]
    lib.paro_kv_free.argtypes = [P, P, I64, P]
    lib.paro_kv_compact.argtypes = [P, P, P, SZ, P]
    lib.paro_kv_workspace_bytes.argtypes = [P]
    lib.paro_kv_workspace_bytes.restype = SZ
    lib.paro_last_error.argtypes = []
    lib.paro_last_error.restype = ctypes.c_char_p
    lib.paro_abi_version.argtypes = []
    for name in ("paro_scale_rotate", "paro_w4_unpack_dequant", "paro_w4a16_linear",
                 "paro_w4a16_linear_path", "paro_w4a16_linear_prerotated", "paro_w4a16_linear_prepared",
                 "paro_w4a16_linear_prepared_multi", "paro_w4a16_linear_tiled_multi", "paro_w4a16_linear_noalloc",
                 "paro_w4_quantize_pack", "paro_scale_rotate_backward", "paro_w4a16_moe_linear",
                 "paro_mxfp4_quantize_weight", "paro_mxfp4_quantize_activations", "paro_mxfp4_gemm",
                 "paro_mxfp4_linear",
                 "paro_rotation_matrix", "paro_scale_rotate_tiled", "paro_w4a16_linear_tiled",
                 "paro_w4a16_linear_choose_path",
                 "paro_validate_layer", "paro_abi_version", "paro_attention_prompt",
                 "paro_attention_prompt_cached", "paro_attention_decode", "paro_kv_append", "paro_kv_reserve",
                 "paro_kv_fork", "paro_kv_free", "paro_kv_compact", "paro_kv_read", "paro_rotary",
                 "paro_rotary_frequencies"):
        getattr(lib, name).restype = I32
    if path == LIB_PATH:
        _lib = lib
    return lib


def _check(rc: int, what: str):
    if rc != 0:
        raise ParoError(rc, what, load().paro_last_error().decode())


def paro_abi_version() -> int:
    return load().paro_abi_version()


def paro_last_error() -> str:
    return load().paro_last_error().decode()


def _stream_handle(stream):
    if stream is None:
        import torch
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return ctypes.c_void_p(stream)
    return ctypes.c_void_p(stream.cuda_stream)


def _ptr(t):
    return None if t is None else t.data_ptr()


_torch_module = _dtypes = None


def _torch():
    """The torch module (an import statement takes longer than a small call's other checks)."""
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _dt(t) -> int:
    global _dtypes
    if _dtypes is None:
        torch = _torch()
        _dtypes = {torch.float16: F16, torch.bfloat16: BF16, torch.float32: F32}
    return _dtypes[t.dtype]


class DeviceLayer:
    """A layer's stored tensors in device memory plus its C descriptor.

    Built from any object with the synth.Layer fields (numpy host arrays);
    torch allocates and owns the device copies.
    """

    def __init__(self, host, device="cuda"):
        import torch
        self.in_features = int(host.in_features)
        self.out_features = int(host.out_features)
        self.group_size = int(host.group_size)
        self.krot = int(host.krot)

        def up(a, dtype):
            return None if a is None else torch.from_numpy(a).to(device=device).view(dtype).contiguous()

        self.pairs = up(host.pairs, torch.int16)
        self.theta = up(host.theta, torch.float32)
        self.channel_scales = up(host.channel_scales, torch.float32)
        self.qweight = up(host.qweight, torch.int32)
        self.qzeros = up(host.qzeros, torch.int32)
        self.scales = up(host.scales.view("int16"), torch.float16)
        self.bias = None if host.bias is None else up(host.bias.view("int16"), torch.float16)
        self.c = ParoLayerC(self.in_features, self.out_features, self.group_size, self.krot,
                            self.pairs.data_ptr(), self.theta.data_ptr(),
                            self.channel_scales.data_ptr(), self.qweight.data_ptr(),
                            self.qzeros.data_ptr(), self.scales.data_ptr(),
                            None if self.bias is None else self.bias.data_ptr())

    @property
    def ref(self):
        return ctypes.byref(self.c)


def paro_validate_layer(host) -> None:
    """Host-side check of a layer's pair schedule and shape rules (numpy arrays)."""
    import numpy as np
    pairs = np.ascontiguousarray(host.pairs, dtype=np.int16)
    c = ParoLayerC(int(host.in_features), int(host.out_features), int(host.group_size),
                   int(host.krot), pairs.ctypes.data, None, None, None, None, None, None)
    _check(load().paro_validate_layer(ctypes.byref(c)), "paro_validate_layer")


def paro_scale_rotate(layer: DeviceLayer, x, x_r, stream=None) -> None:
    """x: (tokens, I) fp16/bf16 cuda tensor; x_r: (tokens, I) fp16/bf16/fp32 output."""
    _check(load().paro_scale_rotate(layer.ref, _ptr(x), _dt(x), x.shape[0], _ptr(x_r), _dt(x_r),
                                    _stream_handle(stream)), "paro_scale_rotate")


def paro_w4_unpack_dequant(layer: DeviceLayer, q_out=None, z_out=None, w_out=None, stream=None) -> None:
    w_dt = _dt(w_out) if w_out is not None else F32
    _check(load().paro_w4_unpack_dequant(layer.ref, _ptr(q_out), _ptr(z_out), _ptr(w_out), w_dt,
                                         _stream_handle(stream)), "paro_w4_unpack_dequant")


def paro_w4a16_linear_workspace_bytes(layer: DeviceLayer, tokens: int, x_dt: int = F16,
                                      path: int = PATH_AUTO) -> int:
    return int(load().paro_w4a16_linear_workspace_bytes(layer.ref, tokens, x_dt, path))


def paro_w4a16_linear_choose_path(layer: DeviceLayer, tokens: int) -> int:
    return int(load().paro_w4a16_linear_choose_path(layer.ref, tokens))


def make_workspace(nbytes: int, device="cuda"):
    """A zero-filled workspace (the contract requires zeros before first use)."""
    import torch
    return torch.zeros(max(int(nbytes), 16), dtype=torch.uint8, device=device)


def paro_w4a16_linear(layer: DeviceLayer, x, y, workspace=None, stream=None, path: int = PATH_AUTO) -> None:
    """y = rotated W4A16 linear of x.  x: (tokens, I) fp16/bf16; y: (tokens, O) x dtype or fp32."""
    ws_ptr = _ptr(workspace)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    lib = load()
    if path == PATH_AUTO:
        rc = lib.paro_w4a16_linear(layer.ref, _ptr(x), _dt(x), x.shape[0], _ptr(y), _dt(y), ws_ptr,
                                   ws_bytes, _stream_handle(stream))
    else:
        rc = lib.paro_w4a16_linear_path(layer.ref, _ptr(x), _dt(x), x.shape[0], _ptr(y), _dt(y), ws_ptr,
                                        ws_bytes, _stream_handle(stream), path)
    _check(rc, "paro_w4a16_linear")


def paro_w4a16_linear_prepared_workspace_bytes(layer: DeviceLayer, tokens: int) -> int:
    return int(load().paro_w4a16_linear_prepared_workspace_bytes(layer.ref, tokens))


def paro_w4a16_linear_prepared(layer: DeviceLayer, hl, x, y, workspace=None, stream=None) -> None:
    """The linear with the layer's dense rotation hl prebuilt by paro_rotation_matrix (for x's dtype)."""
    ws_ptr = _ptr(workspace)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().paro_w4a16_linear_prepared(layer.ref, _ptr(hl), _ptr(x), _dt(x), x.shape[0], _ptr(y), _dt(y),
                                             ws_ptr, ws_bytes, _stream_handle(stream)), "paro_w4a16_linear_prepared")


def _layer_array(layers):
    """A contiguous C array of the layers' descriptors (copies of their structs)."""
    arr = (ParoLayerC * len(layers))()
    for i, L in enumerate(layers):
        arr[i] = L.c
    return arr


def _ptr_array(ts):
    return (ctypes.c_void_p * len(ts))(*[t.data_ptr() for t in ts])


def paro_w4a16_linear_prepared_multi_workspace_bytes(layers, tokens: int) -> int:
    return int(load().paro_w4a16_linear_prepared_multi_workspace_bytes(_layer_array(layers), len(layers), tokens))


def paro_w4a16_linear_prepared_multi(layers, hls, x, ys, workspace=None, stream=None) -> None:
    """Layers of one shape over the same input x, each with its rotation matrix hls[i] and output ys[i]."""
    ws_ptr = _ptr(workspace)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().paro_w4a16_linear_prepared_multi(_layer_array(layers), len(layers), _ptr_array(hls), _ptr(x),
                                                   _dt(x), x.shape[0], _ptr_array(ys), _dt(ys[0]), ws_ptr,
                                                   ws_bytes, _stream_handle(stream)),
           "paro_w4a16_linear_prepared_multi")


def paro_w4a16_linear_tiled_multi(layers, x_ts, x_dt: int, tokens: int, ys, stream=None) -> None:
    """The prefill GEMM alone for layers of one shape, each over its tiled X_r, in one launch."""
    _check(load().paro_w4a16_linear_tiled_multi(_layer_array(layers), len(layers), _ptr_array(x_ts), x_dt, tokens,
                                                _ptr_array(ys), _dt(ys[0]), _stream_handle(stream)),
           "paro_w4a16_linear_tiled_multi")


def paro_w4a16_linear_noalloc(layer: DeviceLayer, x, y, stream=None) -> None:
    """The linear with the library-held workspace (no allocation in the call)."""
    _check(load().paro_w4a16_linear_noalloc(layer.ref, _ptr(x), _dt(x), x.shape[0], _ptr(y), _dt(y),
                                            _stream_handle(stream)), "paro_w4a16_linear_noalloc")


def paro_w4a16_linear_prerotated(layer: DeviceLayer, x_r, y, workspace=None, stream=None,
                                 path: int = PATH_AUTO) -> None:
    """The quantized projection alone over already rotated activations x_r."""
    ws_ptr = _ptr(workspace)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().paro_w4a16_linear_prerotated(layer.ref, _ptr(x_r), _dt(x_r), x_r.shape[0], _ptr(y), _dt(y),
                                               ws_ptr, ws_bytes, _stream_handle(stream), path),
           "paro_w4a16_linear_prerotated")


def paro_tiled_bytes(layer: DeviceLayer, tokens: int) -> int:
    """Bytes of an X_r buffer in the prefill GEMM's tiled layout."""
    return int(load().paro_tiled_bytes(layer.ref, tokens))


def paro_w4_quantize_pack(layer: DeviceLayer, w, symmetric: bool, qweight, qzeros, scales, stream=None) -> None:
    """w: (O, I) fp16/bf16/fp32 device tensor; qweight int32 (I, O/8), qzeros int32 (I/128, O/8),
    scales fp16/int16 view (I/128, O)."""
    _check(load().paro_w4_quantize_pack(layer.ref, _ptr(w), _dt(w), int(bool(symmetric)), _ptr(qweight),
                                        _ptr(qzeros), _ptr(scales), _stream_handle(stream)), "paro_w4_quantize_pack")


def paro_mxfp4_quantize_weight(layer: DeviceLayer, w, codes, scales, stream=None) -> None:
    """w: (O, I) fp16/bf16/fp32; codes uint8 (O, I/2); scales uint8 (O, I/32)."""
    _check(load().paro_mxfp4_quantize_weight(layer.ref, _ptr(w), _dt(w), _ptr(codes), _ptr(scales),
                                             _stream_handle(stream)), "paro_mxfp4_quantize_weight")


def paro_mxfp4_activation_workspace_bytes(layer: DeviceLayer) -> int:
    return int(load().paro_mxfp4_activation_workspace_bytes(layer.ref))


def paro_mxfp4_quantize_activations(layer: DeviceLayer, x, codes, scales, workspace, stream=None) -> None:
    """x: (tokens, I) fp16/bf16; codes uint8 (tokens, I/2); scales uint8 (tokens, I/32); workspace: device
    buffer of paro_mxfp4_activation_workspace_bytes() bytes."""
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().paro_mxfp4_quantize_activations(layer.ref, _ptr(x), _dt(x), x.shape[0], _ptr(codes),
                                                  _ptr(scales), _ptr(workspace), ws_bytes, _stream_handle(stream)),
           "paro_mxfp4_quantize_activations")


def paro_mxfp4_gemm(a_codes, a_scales, w_codes, w_scales, y, bias=None, stream=None) -> None:
    """y (tokens, O) = A . W^T (+ bias) from MXFP4 codes/scales (uint8 device tensors)."""
    tokens, O, I = a_codes.shape[0], w_codes.shape[0], w_codes.shape[1] * 2
    _check(load().paro_mxfp4_gemm(_ptr(a_codes), _ptr(a_scales), tokens, _ptr(w_codes), _ptr(w_scales), O, I,
                                  _ptr(bias), _ptr(y), _dt(y), _stream_handle(stream)), "paro_mxfp4_gemm")


def paro_mxfp4_linear_workspace_bytes(layer: DeviceLayer, tokens: int) -> int:
    return int(load().paro_mxfp4_linear_workspace_bytes(layer.ref, tokens))


def paro_mxfp4_linear(layer: DeviceLayer, w_codes, w_scales, x, y, workspace, stream=None) -> None:
    """The W4A4 MXFP4 linear (rotation, activation quantization, FP4 GEMM, layer bias)."""
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().paro_mxfp4_linear(layer.ref, _ptr(w_codes), _ptr(w_scales), _ptr(x), _dt(x), x.shape[0], _ptr(y),
                                    _dt(y), _ptr(workspace), ws_bytes, _stream_handle(stream)), "paro_mxfp4_linear")


def paro_mxfp4_linear_prepared_workspace_bytes(layer: DeviceLayer, tokens: int) -> int:
    return int(load().paro_mxfp4_linear_prepared_workspace_bytes(layer.ref, tokens))


def paro_mxfp4_linear_prepared(layer: DeviceLayer, hl, w_codes, w_scales, x, y, workspace, stream=None) -> None:
    """The W4A4 MXFP4 linear with the layer's dense rotation hl prebuilt by paro_rotation_matrix."""
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().paro_mxfp4_linear_prepared(layer.ref, _ptr(hl), _ptr(w_codes), _ptr(w_scales), _ptr(x), _dt(x),
                                             x.shape[0], _ptr(y), _dt(y), _ptr(workspace), ws_bytes,
                                             _stream_handle(stream)), "paro_mxfp4_linear_prepared")


def paro_w4a16_moe_linear_workspace_bytes(layer: DeviceLayer, tokens: int, x_dt: int = F16) -> int:
    """Workspace bytes of paro_w4a16_moe_linear for this many routed rows."""
    return int(load().paro_w4a16_moe_linear_workspace_bytes(layer.ref, tokens, x_dt))


def paro_w4a16_moe_linear(layer: DeviceLayer, num_experts: int, expert_offsets, x, y, workspace=None,
                          stream=None) -> None:
    """Experts stacked in `layer`'s weight tensors share its rotation.  expert_offsets: int64 device
    tensor (E+1,); x: (rows, I) fp16/bf16 grouped by expert; y: (rows, O) x dtype or fp32."""
    ws_ptr = _ptr(workspace)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().paro_w4a16_moe_linear(layer.ref, int(num_experts), _ptr(expert_offsets), _ptr(x), _dt(x),
                                        x.shape[0], _ptr(y), _dt(y), ws_ptr, ws_bytes, _stream_handle(stream)),
           "paro_w4a16_moe_linear")


def paro_scale_rotate_backward_workspace_bytes(layer: DeviceLayer, tokens: int) -> int:
    """Workspace bytes of paro_scale_rotate_backward for this many tokens."""
    return int(load().paro_scale_rotate_backward_workspace_bytes(layer.ref, tokens))


def paro_scale_rotate_backward(layer: DeviceLayer, x, g, gx, gtheta, gcs, workspace, stream=None) -> None:
    """x: (tokens, I) fp16/bf16; g = dL/dx_r: (tokens, I) fp32 or x's dtype; gx: (tokens, I) fp32 or x's
    dtype; gtheta: fp32 (krot, I/2); gcs: fp32 (I,); workspace: device buffer of
    paro_scale_rotate_backward_workspace_bytes() bytes."""
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().paro_scale_rotate_backward(layer.ref, _ptr(x), _dt(x), _ptr(g), _dt(g), x.shape[0], _ptr(gx),
                                             _dt(gx), _ptr(gtheta), _ptr(gcs), _ptr(workspace), ws_bytes,
                                             _stream_handle(stream)), "paro_scale_rotate_backward")


def paro_rotation_matrix_bytes(layer: DeviceLayer) -> int:
    """Bytes of the dense rotation (H and L) that paro_rotation_matrix writes."""
    return int(load().paro_rotation_matrix_bytes(layer.ref))


def paro_rotation_matrix(layer: DeviceLayer, x_dt: int, hl, stream=None) -> None:
    """Build H + L = diag(cs) . R per group into hl (device buffer of paro_rotation_matrix_bytes())."""
    _check(load().paro_rotation_matrix(layer.ref, x_dt, _ptr(hl), _stream_handle(stream)),
           "paro_rotation_matrix")


def paro_scale_rotate_tiled(layer: DeviceLayer, hl, x, x_t, stream=None) -> None:
    """x: (tokens, I) fp16/bf16; hl: from paro_rotation_matrix for x's dtype;
    x_t: device buffer of paro_tiled_bytes() bytes (any dtype view)."""
    _check(load().paro_scale_rotate_tiled(layer.ref, _ptr(hl), _ptr(x), _dt(x), x.shape[0], _ptr(x_t),
                                          _stream_handle(stream)), "paro_scale_rotate_tiled")


def paro_w4a16_linear_tiled(layer: DeviceLayer, x_t, x_dt: int, tokens: int, y, stream=None) -> None:
    """The prefill contraction over X_r in the tiled layout; y: (tokens, O) x dtype or fp32."""
    _check(load().paro_w4a16_linear_tiled(layer.ref, _ptr(x_t), x_dt, tokens, _ptr(y), _dt(y),
                                          _stream_handle(stream)), "paro_w4a16_linear_tiled")


# ---- attention and the key-value cache ----

class KVCache:
    """A paged key-value cache: its tensors and the C descriptor (paro_kv_cache).

    k, v: (layers, pages, kv_heads, page_size, head_dim) fp16/bf16; refs: (pages,), table: (slots, max_pages),
    lengths: (slots,), int32; contiguous, on one device.  KVCache.empty() makes them.
    In four bits k and v are uint8 of (layers, pages, kv_heads, page_size, 9 * head_dim // 16), the bytes of each
    head's page (include/paro.h gives their order), and dtype, fp16 or bf16, is that of the rows, queries and outputs.
    """

    def __init__(self, k, v, refs, table, lengths, dtype=None):
        torch = _torch()
        what = "KVCache"
        _need(k.dim() == 5 and v.shape == k.shape, 2, what, "k and v: (layers, pages, kv_heads, page_size, head_dim)")
        four = k.dtype == torch.uint8
        dtype = k.dtype if dtype is None else dtype
        _need(dtype in (torch.float16, torch.bfloat16) and v.dtype == k.dtype and (four or k.dtype == dtype), 3, what,
              "k and v: fp16 or bf16, or uint8 with dtype fp16 or bf16")
        _need(refs.shape == (k.shape[1],) and table.dim() == 2 and lengths.shape == (table.shape[0],), 2, what,
              "refs (pages,), table (slots, max_pages), lengths (slots,)")
        _need(all(t.dtype == torch.int32 for t in (refs, table, lengths)), 3, what, "refs, table and lengths: int32")
        _need(all(t.is_contiguous() and t.device == k.device for t in (k, v, refs, table, lengths)), 2, what,
              "contiguous tensors on one device")
        self.k, self.v, self.refs, self.table, self.lengths = k, v, refs, table, lengths
        layers, pages, kv_heads, page_size, head_dim = k.shape
        if four:
            _need(head_dim in (36, 72), 2, what, "four bits: 36 bytes for 64 channels or 72 for 128")
            head_dim = head_dim * 16 // 9
        self.dtype, self.device, self.bits = dtype, k.device, 4 if four else 16
        self.row_shape = kv_heads, head_dim  # of K and V rows
        dt = F16 if dtype == torch.float16 else BF16
        self.c = ParoKvCacheC(layers, kv_heads, head_dim, page_size, pages, table.shape[0], table.shape[1],
                              KV4_F16 + dt if four else dt, k.data_ptr(), v.data_ptr(), refs.data_ptr(),
                              table.data_ptr(), lengths.data_ptr())
        self.ref = ctypes.byref(self.c)

    @classmethod
    def empty(cls, layers, pages, kv_heads, page_size, head_dim, slots, max_pages, dtype, device="cuda", bits=16):
        """A cache with all slots empty and all pages free; bits: 16, or 4 for rows of dtype held in four bits."""
        torch = _torch()
        _need(bits in (4, 16), 5, "KVCache.empty", "bits: 4 or 16")
        _need(bits == 16 or head_dim in (64, 128), 5, "KVCache.empty", "four bits: heads of 64 or 128 channels")
        shape = (layers, pages, kv_heads, page_size, head_dim if bits == 16 else head_dim * 9 // 16)
        held = dtype if bits == 16 else torch.uint8
        return cls(torch.zeros(shape, dtype=held, device=device), torch.zeros(shape, dtype=held, device=device),
                   torch.zeros(pages, dtype=torch.int32, device=device),
                   torch.full((slots, max_pages), -1, dtype=torch.int32, device=device),
                   torch.zeros(slots, dtype=torch.int32, device=device), dtype=dtype)


def _need(good, status: int, what: str, msg: str):
    if not good:
        raise ParoError(status, what, msg)


def _scratch(workspace, device, what):
    """Bytes of a workspace tensor (0 for None, which the library refuses)."""
    if workspace is None:
        return 0
    _need(workspace.is_contiguous() and workspace.device == device, 7, what, "workspace: a contiguous tensor on q's device")
    return workspace.nbytes


def _index(t, dtype, n, device, what, name):
    """t: a contiguous 1-d tensor of n entries (None: any)."""
    shape = t.shape
    if t.dtype != dtype or len(shape) != 1 or not t.is_contiguous() or t.device != device:
        raise ParoError(3, what, f"{name}: a contiguous 1-d {dtype} tensor on {device}")
    if n is not None and shape[0] != n:
        raise ParoError(2, what, f"{name} has {shape[0]} entries, {n} expected")


def _rows(t, dtype, device, what, name):
    """t: a (tokens, heads, head_dim) view with channels together; returns its token and head strides."""
    stride = t.stride()
    if len(stride) != 3 or (stride[2] != 1 and t.numel()):
        raise ParoError(2, what, f"{name}: (tokens, heads, head_dim) with contiguous channels")
    if t.dtype != dtype or t.device != device:
        raise ParoError(3, what, f"{name}: {dtype} on {device}")
    return stride


def _launch(fn, device, stream, *args):
    """Calls fn(*args, stream) with `device` current; the stream defaults to that device's current one."""
    torch = _torch()
    if device.type != "cuda":
        raise ParoError(1, fn.__name__, f"tensors in device memory are required, not on {device}")
    # the raw handle: looking up a Stream object takes longer than the rest of a call's checks
    handle = torch._C._cuda_getCurrentRawStream(device.index) if stream is None else _stream_handle(stream)
    if device.index == torch._C._cuda_getDevice():
        return fn(*args, handle)
    with torch.cuda.device(device):
        return fn(*args, handle)


def _shape_of(q, kv_heads, scale, causal, qs, ys, ks=(0, 0), vs=(0, 0)):
    _, heads, d = q.shape
    return ParoAttentionShapeC(heads, kv_heads, d, bool(causal), d ** -0.5 if scale is None else scale, qs[0], qs[1],
                               ks[0], ks[1], vs[0], vs[1], ys[0], ys[1])


def paro_attention_prompt(q, k, v, cu_q, cu_k, y, scale=None, causal=True, stream=None) -> None:
    """q, y: (tokens, q_heads, head_dim); k, v: (keys, kv_heads, head_dim), fp16/bf16 views; cu_q, cu_k: int64
    (sequences + 1,) device tensors; scale: 1 / sqrt(head_dim) if None."""
    torch = _torch()
    what, dt, dev = "paro_attention_prompt", q.dtype, q.device
    qs, ks, vs, ys = (_rows(t, dt, dev, what, name) for t, name in ((q, "q"), (k, "k"), (v, "v"), (y, "y")))
    _need(dt in (torch.float16, torch.bfloat16), 3, what, "fp16 or bf16")
    _need(y.shape == q.shape and k.shape == v.shape and k.shape[2] == q.shape[2], 2, what,
          "y like q, v like k, one head_dim")
    n = cu_q.shape[0] if cu_q.dim() else 0
    _need(n > 0, 2, what, "cu_q has sequences + 1 entries")
    _index(cu_q, torch.int64, None, dev, what, "cu_q")
    _index(cu_k, torch.int64, n, dev, what, "cu_k")
    s = _shape_of(q, k.shape[1], scale, causal, qs, ys, ks, vs)
    _check(_launch(load().paro_attention_prompt, dev, stream, ctypes.byref(s), q.data_ptr(), k.data_ptr(),
                   v.data_ptr(), _dt(q), cu_q.data_ptr(), cu_k.data_ptr(), n - 1, q.shape[0], k.shape[0],
                   y.data_ptr()), what)


def paro_attention_prompt_cached_workspace_bytes(cache: KVCache, sequences: int, tokens: int, q_heads: int) -> int:
    return int(load().paro_attention_prompt_cached_workspace_bytes(cache.ref, sequences, tokens, q_heads))


def paro_attention_prompt_cached(cache: KVCache, layer: int, q, slots, cu_q, y, scale=None, causal=True,
                                 stream=None, workspace=None) -> None:
    """q, y: (tokens, q_heads, head_dim) of the cache's dtype: the newest rows of the slots; slots: int32
    (sequences,); cu_q: int64 (sequences + 1,); workspace: zero-filled before its first use, of
    paro_attention_prompt_cached_workspace_bytes() bytes: splits the keys of few rows over workgroups."""
    torch = _torch()
    what, dt, dev = "paro_attention_prompt_cached", cache.dtype, cache.device
    qs, ys = _rows(q, dt, dev, what, "q"), _rows(y, dt, dev, what, "y")
    _need(y.shape == q.shape, 2, what, "y like q")
    _index(slots, torch.int32, None, dev, what, "slots")
    n = slots.shape[0]
    _index(cu_q, torch.int64, n + 1, dev, what, "cu_q")
    s = _shape_of(q, cache.c.kv_heads, scale, causal, qs, ys)
    _check(_launch(load().paro_attention_prompt_cached, dev, stream, cache.ref, layer, ctypes.byref(s), q.data_ptr(),
                   slots.data_ptr(), cu_q.data_ptr(), n, q.shape[0], y.data_ptr(), _ptr(workspace),
                   _scratch(workspace, dev, what)), what)


def paro_attention_decode_workspace_bytes(cache: KVCache, rows: int, q_heads: int) -> int:
    return int(load().paro_attention_decode_workspace_bytes(cache.ref, rows, q_heads))


def paro_attention_decode(cache: KVCache, layer: int, q, slots, y, workspace, scale=None, stream=None) -> None:
    """q, y: (rows, q_heads, head_dim), one new token per row; slots: int32 (rows,); workspace: zero-filled before
    its first use, of paro_attention_decode_workspace_bytes() bytes."""
    torch = _torch()
    what, dt, dev = "paro_attention_decode", cache.dtype, cache.device
    qs, ys = _rows(q, dt, dev, what, "q"), _rows(y, dt, dev, what, "y")
    _need(y.shape == q.shape, 2, what, "y like q")
    n = q.shape[0]
    _index(slots, torch.int32, n, dev, what, "slots")
    ws_bytes = _scratch(workspace, dev, what)
    s = _shape_of(q, cache.c.kv_heads, scale, True, qs, ys)
    _check(_launch(load().paro_attention_decode, dev, stream, cache.ref, layer, ctypes.byref(s), q.data_ptr(),
                   slots.data_ptr(), n, y.data_ptr(), _ptr(workspace), ws_bytes), what)


def paro_kv_append(cache: KVCache, layer: int, k, v, slots, cu=None, stream=None, granted=None) -> None:
    """k, v: (tokens, kv_heads, head_dim) of the cache's dtype become the newest positions of the slots: rows
    cu[i]..cu[i + 1] of slot slots[i] (int32), one row per slot if cu (int64) is None; granted: paro_kv_reserve's,
    whose refused entries are then skipped."""
    torch = _torch()
    what, dt, dev = "paro_kv_append", cache.dtype, cache.device
    ks, vs = _rows(k, dt, dev, what, "k"), _rows(v, dt, dev, what, "v")
    shape = k.shape
    if v.shape != shape or tuple(shape[1:]) != cache.row_shape:
        raise ParoError(2, what, "k and v: (tokens, %d, %d)" % cache.row_shape)
    n = _entries(torch, dev, what, slots, cu, "granted", granted)
    rc = _launch(load().paro_kv_append, dev, stream, cache.ref, layer, k.data_ptr(), ks[0], ks[1], v.data_ptr(), vs[0],
                 vs[1], slots.data_ptr(), _ptr(cu), _ptr(granted), n, shape[0])
    if rc:
        _check(rc, what)


def _entries(torch, device, what, slots, cu, name, more):
    """The entries of a call on packed rows: int32 slots, int64 offsets or None, another int32 list or None."""
    _index(slots, torch.int32, None, device, what, "slots")
    n = slots.shape[0]
    if cu is not None:
        _index(cu, torch.int64, n + 1, device, what, "cu")
    if more is not None:
        _index(more, torch.int32, n, device, what, name)
    return n


def paro_kv_read(cache: KVCache, layer: int, k, v, slots, cu=None, first=None, stream=None) -> None:
    """k, v: (tokens, kv_heads, head_dim) of the cache's dtype or fp32 (either may be None) are set to what the slots
    hold: rows cu[i]..cu[i + 1] (one row per slot if cu is None) to positions first[i] and up (int32 (n,)), or to the
    newest ones if first is None; rows beyond what a slot holds are zero."""
    torch = _torch()
    what, dev = "paro_kv_read", cache.device
    one = v if k is None else k
    if one is None:
        raise ParoError(1, what, "k or v is required")
    out, shape = one.dtype, one.shape
    if out != cache.dtype and out != torch.float32:
        raise ParoError(3, what, f"k and v: {cache.dtype} or fp32")
    if tuple(shape[1:]) != cache.row_shape or (v is not None and v.shape != shape):
        raise ParoError(2, what, "k and v: (tokens, %d, %d)" % cache.row_shape)
    ks = (0, 0) if k is None else _rows(k, out, dev, what, "k")
    vs = (0, 0) if v is None else _rows(v, out, dev, what, "v")
    n = _entries(torch, dev, what, slots, cu, "first", first)
    rc = _launch(load().paro_kv_read, dev, stream, cache.ref, layer, _ptr(k), ks[0], ks[1], _ptr(v), vs[0], vs[1],
                 _dt(one), slots.data_ptr(), _ptr(cu), _ptr(first), n, shape[0])
    if rc:
        _check(rc, what)


def paro_kv_workspace_bytes(cache: KVCache) -> int:
    """Workspace bytes of paro_kv_reserve, paro_kv_fork and paro_kv_compact."""
    return int(load().paro_kv_workspace_bytes(cache.ref))


def _plan_call(fn, what, cache, names, a, b, out, workspace, stream):
    torch = _torch()
    dev = cache.device
    n = a.shape[0] if a.dim() else 0
    for t, name in zip((a, b, out), names):
        _index(t, torch.int32, n, dev, what, name)
    _check(_launch(fn, dev, stream, cache.ref, a.data_ptr(), b.data_ptr(), n, out.data_ptr(), _ptr(workspace),
                   _scratch(workspace, dev, what)), what)


def paro_kv_reserve(cache: KVCache, slots, grow, granted, workspace, stream=None) -> None:
    """Room for grow[i] new positions in slot slots[i]; granted[i] is set to 1 or 0 (int32 tensors)."""
    _plan_call(load().paro_kv_reserve, "paro_kv_reserve", cache, ("slots", "grow", "granted"), slots, grow, granted,
               workspace, stream)


def paro_kv_fork(cache: KVCache, parents, children, granted, workspace, stream=None) -> None:
    """The empty slot children[i] shares the pages of slot parents[i]; granted[i] is set to 1 or 0."""
    _plan_call(load().paro_kv_fork, "paro_kv_fork", cache, ("parents", "children", "granted"), parents, children,
               granted, workspace, stream)


def paro_kv_free(cache: KVCache, slots, stream=None) -> None:
    """Empties the slots (int32 tensor) and gives up their pages."""
    torch = _torch()
    _index(slots, torch.int32, None, cache.device, "paro_kv_free", "slots")
    _check(_launch(load().paro_kv_free, cache.device, stream, cache.ref, slots.data_ptr(), slots.shape[0]),
           "paro_kv_free")


def paro_kv_compact(cache: KVCache, used, workspace, stream=None) -> None:
    """Moves the pages in use to the lowest indices; used: int32 (1,), set to their number."""
    torch = _torch()
    what, dev = "paro_kv_compact", cache.device
    _index(used, torch.int32, 1, dev, what, "used")
    _check(_launch(load().paro_kv_compact, dev, stream, cache.ref, used.data_ptr(), _ptr(workspace),
                   _scratch(workspace, dev, what)), what)


# ---- rotary positions ----

ROTARY = {"none": 0, "linear": 1, "base": 2, "bands": 3, "ramp": 4}


def paro_rotary_frequencies(rot_dim: int, base: float = 10000.0, kind: str = "none", factor: float = 1.0,
                            context: float = 0.0, low: float | None = None, high: float | None = None, device="cuda"):
    """(freqs, magnitude): the angle per position of each pair of channels, float64 (rot_dim // 2,) on `device`, and
    what multiplies cosine and sine.  kind: "none", "linear", "base", "bands" or "ramp" (include/paro.h gives their
    formulas), stretching a trained `context` by `factor`; low, high: 1 and 4 ("bands") or 1 and 32 ("ramp") if None."""
    torch = _torch()
    what = "paro_rotary_frequencies"
    _need(kind in ROTARY, 5, what, f"kind: one of {', '.join(ROTARY)}")
    s = ParoRotaryScalingC(ROTARY[kind], base, factor, context, 1.0 if low is None else low,
                           (32.0 if kind == "ramp" else 4.0) if high is None else high)
    out, magnitude = (ctypes.c_double * max(1, rot_dim // 2))(), ctypes.c_float()
    _check(load().paro_rotary_frequencies(ctypes.byref(s), rot_dim, out, ctypes.byref(magnitude)), what)
    return torch.tensor(list(out), dtype=torch.float64, device=device), magnitude.value


def paro_rotary(x, positions, freqs, y, interleaved: bool = False, inverse: bool = False, magnitude: float = 1.0,
                stream=None) -> None:
    """x, y: (tokens, heads, head_dim) fp16/bf16/fp32 views, y may be x; positions: int32 (tokens,); freqs: float64
    (rot_dim // 2,), radians per position: channel pairs (i, i + rot_dim / 2), or (2i, 2i + 1) if interleaved, turn by
    positions * freqs (inverse: back, which is the gradient), the channels from rot_dim on are copied."""
    torch = _torch()
    what, dt, dev, shape = "paro_rotary", x.dtype, x.device, x.shape
    xs, ys = _rows(x, dt, dev, what, "x"), _rows(y, dt, dev, what, "y")
    if dt not in (torch.float16, torch.bfloat16, torch.float32):
        raise ParoError(3, what, "fp16, bf16 or fp32")
    if y.shape != shape:
        raise ParoError(2, what, "y like x")
    tokens, heads, d = shape
    _index(positions, torch.int32, tokens, dev, what, "positions")
    _index(freqs, torch.float64, None, dev, what, "freqs")
    s = ParoRotaryShapeC(heads, d, 2 * freqs.shape[0], bool(interleaved), bool(inverse), magnitude, xs[0], xs[1], ys[0], ys[1])
    rc = _launch(load().paro_rotary, dev, stream, s, x.data_ptr(), _dt(x), positions.data_ptr(), freqs.data_ptr(),
                 tokens, y.data_ptr())
    if rc:
        _check(rc, what)
