"""GB300 (sm_103a) routed-expert MoE layer of the qwen3_5_moe family.

This package is a thin Python binding of ``libmoe.so`` (the C ABI declared in
``include/moe.h``).  Every function named ``moe_*`` here marshals torch tensors
(device memory and streams only) into the C call of the same name; all of the
layer's arithmetic runs in the library's CUDA kernels.  There is no CPU
fallback: without the built library or a CUDA device the calls raise.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional

import numpy as np
import torch

from . import _build

MOE_OK = 0
MOE_ERR_INVALID_ARG = 1
MOE_ERR_UNSUPPORTED = 2
MOE_ERR_WORKSPACE = 3
MOE_ERR_CUDA = 4
MOE_ERR_TIMEOUT = 5
MOE_ERR_DEVICE = 6

MOE_PATH_AUTO = 0
MOE_PATH_DECODE = 1
MOE_PATH_PREFILL = 2

MOE_FORMAT_AFFINE = 0
MOE_FORMAT_NVFP4 = 1

MOE_SCALED_NVFP4 = 1
MOE_SCALED_MXFP8 = 2
MOE_SCALED_MXFP4 = 3
MOE_SCALED_WS_BYTES = 512

EXPORTED = ("moe_status_string", "moe_check_config", "moe_workspace_size", "moe_route", "moe_permute",
            "moe_expert_ffn", "moe_combine", "moe_forward", "moe_get_device_status", "moe_pack_down",
            "moe_expert_stages",
            "moe_decode_timeline", "moe_forward_decode_static",
            "moe_add_rmsnorm", "moe_quantize", "moe_quantize_routed", "moe_tile_scales", "moe_scaled_gemm",
            "moe_scaled_swiglu", "moe_scaled_workspace_size", "moe_scaled_forward")


class MoeError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn}: {status_string(status)} (status {status})")
        self.status = status


class moe_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in
                ("hidden", "inter", "n_experts", "top_k", "group", "bits", "router_bits", "has_shared",
                 "wait_polls", "format")]


class moe_qmat(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("biases", ctypes.c_void_p),
                ("gscale", ctypes.c_void_p)]


class moe_weights(ctypes.Structure):
    _fields_ = [(n, moe_qmat) for n in ("router", "gate", "up", "down", "s_gate", "s_up", "s_down")] + \
               [("shared_gate_vec", ctypes.c_void_p), ("down_packed", ctypes.c_void_p),
                ("s_down_packed", ctypes.c_void_p)]


class moe_scaled_rows(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("codes", "scales", "row_scale")]


class moe_scaled_mat(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("codes", "scales", "alpha")]


class moe_scaled_weights(ctypes.Structure):
    _fields_ = [("format", ctypes.c_int), ("router", moe_qmat), ("shared_gate_vec", ctypes.c_void_p),
                ("gate", moe_scaled_mat), ("up", moe_scaled_mat), ("down", moe_scaled_mat), ("h_scale", ctypes.c_void_p)]


_lock = threading.Lock()
_lib = None

_VP = ctypes.c_void_p
_I = ctypes.c_int
_SZ = ctypes.c_size_t


def library_path() -> str:
    return _build.LIB


def load(build: bool = True):
    """Load libmoe.so (building it with nvcc first if it is missing or stale)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if build:
            _build.build()
        if not os.path.exists(_build.LIB):
            raise RuntimeError(f"libmoe.so not built ({_build.LIB}); run quantised_moe_expert_gb300._build")
        lib = ctypes.CDLL(_build.LIB)
        P = ctypes.POINTER
        lib.moe_status_string.restype = ctypes.c_char_p
        lib.moe_status_string.argtypes = [_I]
        lib.moe_check_config.argtypes = [P(moe_config)]
        lib.moe_workspace_size.argtypes = [P(moe_config), _I, P(ctypes.c_size_t)]
        lib.moe_route.argtypes = [P(moe_config), P(moe_weights), _VP, _I, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _SZ, _VP]
        lib.moe_permute.argtypes = [P(moe_config), _VP, _I, _VP, _VP, _VP, _VP, _VP, _SZ, _VP]
        lib.moe_expert_ffn.argtypes = [P(moe_config), P(moe_weights), _VP, _I, _VP, _VP, _VP, _VP, _VP, _VP, _VP,
                                       _I, _VP, _SZ, _VP]
        lib.moe_combine.argtypes = [P(moe_config), _I, _VP, _VP, _VP]
        lib.moe_forward.argtypes = [P(moe_config), P(moe_weights), _VP, _I, _VP, _VP, _VP, _VP, _VP, _VP, _I, _VP,
                                    _SZ, _VP]
        lib.moe_get_device_status.argtypes = [_VP, _SZ, _VP, P(ctypes.c_int)]
        lib.moe_pack_down.argtypes = [P(moe_config), P(moe_weights), _VP, _VP, _VP]
        lib.moe_expert_stages.argtypes = [P(moe_config), P(moe_weights), _VP, _I, _VP, _VP, _VP, _VP, _VP, _VP, _I,
                                          _VP, _SZ, _VP]
        lib.moe_decode_timeline.argtypes = [P(moe_config), _I, _VP, _SZ, _VP, _VP, _I, P(ctypes.c_int)]
        lib.moe_forward_decode_static.argtypes = [P(moe_config), P(moe_weights), _VP, _I, _VP, _VP, _VP, _VP, _VP,
                                                  _VP, _VP]
        R, M, F = P(moe_scaled_rows), P(moe_scaled_mat), ctypes.c_float
        lib.moe_add_rmsnorm.argtypes = [_VP, _VP, _VP, F, F, _I, _I, _VP, _VP, _I, R, _VP]
        lib.moe_quantize.argtypes = [_I, _VP, _I, _I, _I, _I, _VP, R, _VP]
        lib.moe_quantize_routed.argtypes = [_I, _VP, _I, _I, _I, _I, _I, _VP, _VP, _VP, R, _VP, _SZ, _VP]
        lib.moe_tile_scales.argtypes = [_I, _VP, _I, _I, _I, _VP, _VP]
        lib.moe_scaled_gemm.argtypes = [_I, R, M, _I, _I, _I, _I, _VP, _VP, _I, _VP, _SZ, _VP]
        lib.moe_scaled_swiglu.argtypes = [_I, R, M, M, _I, _I, _I, _I, _VP, _VP, R, _VP, _SZ, _VP]
        lib.moe_scaled_workspace_size.argtypes = [P(moe_config), _I, _I, P(ctypes.c_size_t)]
        lib.moe_scaled_forward.argtypes = [P(moe_config), P(moe_scaled_weights), _VP, _I, _VP, _VP, _VP, _VP, _VP, _VP, _VP,
                                           _SZ, _VP]
        for name in EXPORTED:
            if name != "moe_status_string":
                getattr(lib, name).restype = ctypes.c_int
        _lib = lib
        return lib


def status_string(status: int) -> str:
    return load(build=False).moe_status_string(status).decode() if _lib is not None else f"status {status}"


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        # the current stream's handle, without the stream object that torch.cuda.current_stream() makes
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _check(fn: str, rc: int):
    if rc != MOE_OK:
        raise MoeError(fn, rc)


def config_of(shape, wait_polls: int = 0) -> moe_config:
    """moe_config from any object with the layer-shape attributes (e.g. synth.LayerShape)."""
    fmt = MOE_FORMAT_NVFP4 if getattr(shape, "fmt", "affine") == "nvfp4" else MOE_FORMAT_AFFINE
    return moe_config(shape.hidden, shape.inter, shape.n_experts, shape.top_k, shape.group, shape.bits,
                      shape.router_bits, shape.has_shared, wait_polls, fmt)


def _ptr(t):
    return None if t is None or t.numel() == 0 else t.data_ptr()


class DeviceLayer:
    """One layer's weights resident on a CUDA device, plus the C weight struct.

    pack=True also makes the decode layout of the down codes (moe_pack_down) and hands it to the
    library in moe_weights.down_packed / s_down_packed (4-bit experts only: the layout and the fused
    decode kernel that reads it are for 4-bit codes)."""

    def __init__(self, host, device="cuda", pack: bool = True):
        self.shape = host.shape
        self.cfg = config_of(host.shape)
        self.tensors = {}

        def up(name, arr):
            arr = np.ascontiguousarray(arr)
            if arr.dtype == np.uint16:
                arr = arr.view(np.int16)
            t = torch.from_numpy(arr).to(device)
            self.tensors[name] = t
            return t

        def q(name, m):
            c = up(name + ".codes", m.codes)
            s = up(name + ".scales", m.scales)
            b = up(name + ".biases", m.biases)
            g = None if m.gscale is None else up(name + ".gscale", m.gscale)
            return moe_qmat(c.data_ptr(), s.data_ptr(), _ptr(b), _ptr(g))

        self.w = moe_weights(q("router", host.router), q("gate", host.gate), q("up", host.up),
                             q("down", host.down), q("s_gate", host.s_gate), q("s_up", host.s_up),
                             q("s_down", host.s_down), up("v", host.shared_gate_vec).data_ptr(), None, None)
        if pack and host.shape.bits == 4 and getattr(host.shape, "fmt", "affine") == "affine":
            self.pack()

    def pack(self):
        """The decode layout of the down codes, made on the device by moe_pack_down."""
        d, sd = self.tensors["down.codes"], self.tensors["s_down.codes"]
        dp = torch.empty_like(d)
        sdp = torch.empty_like(sd) if self.shape.has_shared else None
        moe_pack_down(self.cfg, self.w, dp, sdp)
        self.tensors["down.packed"] = dp
        self.w.down_packed = dp.data_ptr()
        if sdp is not None:
            self.tensors["s_down.packed"] = sdp
            self.w.s_down_packed = sdp.data_ptr()

    def unpacked(self) -> "DeviceLayer":
        """The same layer without the packed down codes (the decode kernel gathers from the MLX layout)."""
        t = {k: v for k, v in self.tensors.items() if not k.endswith(".packed")}
        return DeviceLayer.from_tensors(self.shape, t)

    @staticmethod
    def from_tensors(shape, tensors):
        """Wrap device tensors already laid out as the C ABI expects (same keys as ``tensors``)."""
        obj = DeviceLayer.__new__(DeviceLayer)
        obj.shape = shape
        obj.cfg = config_of(shape)
        obj.tensors = tensors

        def q(name):
            return moe_qmat(tensors[name + ".codes"].data_ptr(), tensors[name + ".scales"].data_ptr(),
                            _ptr(tensors[name + ".biases"]), _ptr(tensors.get(name + ".gscale")))
        opt = lambda name: tensors[name].data_ptr() if name in tensors else None
        obj.w = moe_weights(q("router"), q("gate"), q("up"), q("down"), q("s_gate"), q("s_up"), q("s_down"),
                            tensors["v"].data_ptr(), opt("down.packed"), opt("s_down.packed"))
        return obj


# ---------------------------------------------------------------- C ABI, same names

def moe_check_config(cfg: moe_config) -> int:
    return load().moe_check_config(ctypes.byref(cfg))


def moe_workspace_size(cfg: moe_config, T: int) -> int:
    n = ctypes.c_size_t(0)
    _check("moe_workspace_size", load().moe_workspace_size(ctypes.byref(cfg), T, ctypes.byref(n)))
    return n.value


def moe_route(cfg, w, x, T, router_bias, logits_in, logits_out, ids, p, w_shared, ws, stream=None):
    rc = load().moe_route(ctypes.byref(cfg), ctypes.byref(w), _ptr(x), T, _ptr(router_bias), _ptr(logits_in),
                          _ptr(logits_out), _ptr(ids), _ptr(p), _ptr(w_shared), _ptr(ws),
                          ws.numel() * ws.element_size(), _stream(stream))
    _check("moe_route", rc)


def moe_permute(cfg, ids, T, counts, offsets, perm, inv_perm, ws, stream=None):
    rc = load().moe_permute(ctypes.byref(cfg), _ptr(ids), T, _ptr(counts), _ptr(offsets), _ptr(perm),
                            _ptr(inv_perm), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream))
    _check("moe_permute", rc)


def moe_expert_ffn(cfg, w, x, T, ids, p, w_shared, counts, offsets, perm, acc, path, ws, stream=None):
    rc = load().moe_expert_ffn(ctypes.byref(cfg), ctypes.byref(w), _ptr(x), T, _ptr(ids), _ptr(p), _ptr(w_shared),
                               _ptr(counts), _ptr(offsets), _ptr(perm), _ptr(acc), path, _ptr(ws),
                               ws.numel() * ws.element_size(), _stream(stream))
    _check("moe_expert_ffn", rc)


def moe_combine(cfg, T, acc, y, stream=None):
    _check("moe_combine", load().moe_combine(ctypes.byref(cfg), T, _ptr(acc), _ptr(y), _stream(stream)))


def moe_forward(cfg, w, x, T, router_bias, logits_in, y, ids_out, p_out, w_shared_out, path, ws, stream=None):
    rc = load().moe_forward(ctypes.byref(cfg), ctypes.byref(w), _ptr(x), T, _ptr(router_bias), _ptr(logits_in),
                            _ptr(y), _ptr(ids_out), _ptr(p_out), _ptr(w_shared_out), path, _ptr(ws),
                            ws.numel() * ws.element_size(), _stream(stream))
    _check("moe_forward", rc)


def moe_forward_decode_static(cfg, w, x, T, router_bias, logits_in, y, ids_out, p_out, w_shared_out, stream=None):
    """Decode layer (T <= 16) without a workspace, for callers that cannot allocate device memory.

    The scratch is a fixed array inside libmoe.so's device memory, shared by
    every call: keep calls ordered on the GPU (overlapping calls race).  The
    first call on a device must come before any stream capture.
    """
    rc = load().moe_forward_decode_static(ctypes.byref(cfg), ctypes.byref(w), _ptr(x), T, _ptr(router_bias),
                                          _ptr(logits_in), _ptr(y), _ptr(ids_out), _ptr(p_out), _ptr(w_shared_out),
                                          _stream(stream))
    _check("moe_forward_decode_static", rc)


def moe_get_device_status(ws, stream=None) -> int:
    st = ctypes.c_int(0)
    _check("moe_get_device_status", load().moe_get_device_status(_ptr(ws), ws.numel() * ws.element_size(),
                                                                 _stream(stream), ctypes.byref(st)))
    return st.value


def moe_pack_down(cfg, w, down_packed, s_down_packed=None, stream=None):
    rc = load().moe_pack_down(ctypes.byref(cfg), ctypes.byref(w), _ptr(down_packed), _ptr(s_down_packed),
                              _stream(stream))
    _check("moe_pack_down", rc)


def moe_expert_stages(cfg, w, x, T, ids, counts, offsets, perm, h_out, yslot_out, path, ws, stream=None):
    rc = load().moe_expert_stages(ctypes.byref(cfg), ctypes.byref(w), _ptr(x), T, _ptr(ids), _ptr(counts),
                                  _ptr(offsets), _ptr(perm), _ptr(h_out), _ptr(yslot_out), path, _ptr(ws),
                                  ws.numel() * ws.element_size(), _stream(stream))
    _check("moe_expert_stages", rc)


def moe_decode_timeline(cfg, T, ws, stream=None, max_ctas: int = 256) -> np.ndarray:
    """Per-CTA %globaltimer stamps (ns) of the last fused decode launch on ws: [n_ctas, 14] uint64."""
    buf = np.zeros((max_ctas, 14), dtype=np.uint64)
    n = ctypes.c_int(0)
    rc = load().moe_decode_timeline(ctypes.byref(cfg), T, _ptr(ws), ws.numel() * ws.element_size(),
                                    _stream(stream), ctypes.c_void_p(buf.ctypes.data), max_ctas, ctypes.byref(n))
    _check("moe_decode_timeline", rc)
    return buf[:min(n.value, max_ctas)]


# The block-scaled operators are microseconds on the device at small sizes, so their bindings do no more than
# they have to: no ctypes objects for pointers, the stream's handle and not its object.  The library sees addresses
# alone, so what a tensor holds is checked here.

_BITS16 = frozenset((torch.bfloat16, torch.int16, torch.uint16))   # bf16 values, or their bits
_BITS16_F32 = _BITS16 | {torch.float32}
_F32, _I32 = frozenset((torch.float32,)), frozenset((torch.int32,))


def _dense(fn, t, types):
    """Address of a dense tensor of one of these types."""
    if t.dtype not in types or not t.is_contiguous():
        raise MoeError(fn, MOE_ERR_INVALID_ARG)
    return t.data_ptr()


def _dense_or_none(fn, t, types):
    if t is None:
        return None
    if t.dtype not in types or not t.is_contiguous():
        raise MoeError(fn, MOE_ERR_INVALID_ARG)
    return t.data_ptr()


def _handle(stream):
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def moe_add_rmsnorm(x, residual, weight, weight_offset, eps, T, n, sum_out, y_out, fmt, q, stream=None):
    fn = "moe_add_rmsnorm"
    rc = (_lib or load()).moe_add_rmsnorm(_dense(fn, x, _BITS16), _dense_or_none(fn, residual, _BITS16),
                                          _dense_or_none(fn, weight, _BITS16), weight_offset, eps, T, n,
                                          _dense_or_none(fn, sum_out, _BITS16), _dense_or_none(fn, y_out, _BITS16), fmt, q,
                                          _handle(stream))
    if rc:
        raise MoeError(fn, rc)


def moe_quantize(fmt, x, T, n, groups, gscale, q, stream=None):
    """x: a bf16 (or its bits, as a 16-bit integer) or float32 tensor."""
    fn = "moe_quantize"
    rc = (_lib or load()).moe_quantize(fmt, _dense(fn, x, _BITS16_F32), x.dtype == torch.float32, T, n, groups,
                                       _dense_or_none(fn, gscale, _F32), q, _handle(stream))
    if rc:
        raise MoeError(fn, rc)


def moe_quantize_routed(fmt, x, T, n, k, E, has_shared, ids, inv_perm, offsets, q, ws, stream=None):
    fn = "moe_quantize_routed"
    rc = (_lib or load()).moe_quantize_routed(fmt, _dense(fn, x, _BITS16), T, n, k, E, has_shared, _dense(fn, ids, _I32),
                                              _dense(fn, inv_perm, _I32), _dense(fn, offsets, _I32), q, ws.data_ptr(), ws.nbytes,
                                              _handle(stream))
    if rc:
        raise MoeError(fn, rc)


def moe_tile_scales(fmt, src, G, N, n, dst, stream=None):
    """src, dst: tensors of one byte an element."""
    fn = "moe_tile_scales"
    if src.itemsize != 1 or dst.itemsize != 1 or not src.is_contiguous() or not dst.is_contiguous():
        raise MoeError(fn, MOE_ERR_INVALID_ARG)
    rc = (_lib or load()).moe_tile_scales(fmt, src.data_ptr(), G, N, n, dst.data_ptr(), _handle(stream))
    if rc:
        raise MoeError(fn, rc)


def moe_scaled_gemm(fmt, a, w, R, N, K, G, offsets, y, ws, stream=None):
    """y: a bf16 (or its bits, as a 16-bit integer) or float32 tensor [R, N]."""
    fn = "moe_scaled_gemm"
    rc = (_lib or load()).moe_scaled_gemm(fmt, a, w, R, N, K, G, _dense_or_none(fn, offsets, _I32), _dense(fn, y, _BITS16_F32),
                                          y.dtype == torch.float32, ws.data_ptr(), ws.nbytes, _handle(stream))
    if rc:
        raise MoeError(fn, rc)


def moe_scaled_swiglu(fmt, a, gate, up, R, inter, K, G, offsets, h_scale, h, ws, stream=None):
    fn = "moe_scaled_swiglu"
    rc = (_lib or load()).moe_scaled_swiglu(fmt, a, gate, up, R, inter, K, G, _dense_or_none(fn, offsets, _I32),
                                            _dense_or_none(fn, h_scale, _F32), h, ws.data_ptr(), ws.nbytes, _handle(stream))
    if rc:
        raise MoeError(fn, rc)


def moe_scaled_workspace_size(cfg: moe_config, fmt: int, T: int) -> int:
    n = ctypes.c_size_t(0)
    _check("moe_scaled_workspace_size", load().moe_scaled_workspace_size(ctypes.byref(cfg), fmt, T, ctypes.byref(n)))
    return n.value


def moe_scaled_forward(cfg, w, x, T, router_bias, logits_in, y, ids_out, p_out, w_shared_out, ws, stream=None):
    fn = "moe_scaled_forward"
    for t, types in ((x, _BITS16), (y, _BITS16), (router_bias, _F32), (logits_in, _F32), (ids_out, _I32), (p_out, _BITS16),
                     (w_shared_out, _BITS16)):
        _dense_or_none(fn, t, types)
    rc = load().moe_scaled_forward(ctypes.byref(cfg), ctypes.byref(w), _ptr(x), T, _ptr(router_bias), _ptr(logits_in), _ptr(y),
                                   _ptr(ids_out), _ptr(p_out), _ptr(w_shared_out), _ptr(ws), ws.numel() * ws.element_size(),
                                   _stream(stream))
    _check(fn, rc)


# ---------------------------------------------------------------- conveniences

def _dense_bytes(fn, codes, scales, factors):
    if not codes.is_contiguous() or not scales.is_contiguous():
        raise MoeError(fn, MOE_ERR_INVALID_ARG)
    _dense_or_none(fn, factors, _F32)


def scaled_rows(codes, scales, row_scale=None) -> moe_scaled_rows:
    """The C description of block-scaled rows held in these tensors (which it keeps alive)."""
    _dense_bytes("scaled_rows", codes, scales, row_scale)
    r = moe_scaled_rows(_ptr(codes), _ptr(scales), _ptr(row_scale))
    r.tensors = (codes, scales, row_scale)
    return r


def scaled_mat(codes, scales, alpha=None) -> moe_scaled_mat:
    """The C description of a stack of block-scaled matrices held in these tensors (which it keeps alive)."""
    _dense_bytes("scaled_mat", codes, scales, alpha)
    m = moe_scaled_mat(_ptr(codes), _ptr(scales), _ptr(alpha))
    m.tensors = (codes, scales, alpha)
    return m


def scaled_col_tiles(fmt: int, n: int) -> int:
    """Scale tiles across a row of n elements."""
    return -(-(n // (16 if fmt == MOE_SCALED_NVFP4 else 32)) // 4)


def scaled_rows_empty(fmt: int, R: int, n: int, groups: int = 1, row_scale: bool = True, device="cuda") -> moe_scaled_rows:
    """Room for R block-scaled rows of n elements in `groups` groups (row_scale: NVFP4 rows with their own factors)."""
    codes = torch.empty((R, n if fmt == MOE_SCALED_MXFP8 else n // 2), dtype=torch.uint8, device=device)
    scales = torch.zeros(((R // 128 + groups) * scaled_col_tiles(fmt, n) * 512,), dtype=torch.uint8, device=device)
    rs = torch.empty((R,), device=device) if row_scale and fmt == MOE_SCALED_NVFP4 else None
    return scaled_rows(codes, scales, rs)



class ScaledLayer:
    """One layer's weights for moe_scaled_forward: stacks of the routed experts' matrices and, last, the shared expert's.

    From an NVFP4 layer on the host (from_nvfp4, the layer DeviceLayer takes) or from matrices in floating
    point (quantized, either format)."""

    def __init__(self, shape, fmt, router, v, gate, up, down, h_scale=None):
        """router: DeviceLayer-style tensors (codes, scales, biases); v: bf16 bits [hidden] or None; gate, up, down:
        moe_scaled_mat; h_scale: float32 [G] (NVFP4)."""
        _dense_or_none("ScaledLayer", v, _BITS16)
        _dense_or_none("ScaledLayer", h_scale, _F32)
        if h_scale is not None and h_scale.numel() != shape.n_experts + shape.has_shared:
            raise MoeError("ScaledLayer", MOE_ERR_INVALID_ARG)
        self.shape, self.fmt, self.cfg = shape, fmt, config_of(shape)
        self.tensors = (router, v, gate, up, down, h_scale)
        self.w = moe_scaled_weights(fmt, moe_qmat(*[_ptr(t) for t in router], None), _ptr(v), gate, up, down, _ptr(h_scale))

    @staticmethod
    def _router(host, device):
        up = lambda a: torch.from_numpy(np.ascontiguousarray(a).view(np.int16 if a.dtype == np.uint16 else a.dtype)).to(device)
        return [up(host.router.codes), up(host.router.scales), up(host.router.biases)], up(host.shared_gate_vec)

    @classmethod
    def from_nvfp4(cls, host, h_scale, device="cuda"):
        """host: a synth.LayerWeights with NVFP4 experts; h_scale: the calibrated factor of h, a float32 tensor of one value
        per expert, shared expert last (see calibrate_h_scale)."""
        shape = host.shape

        def stack(m, s, N, n, factor):
            parts = [m, s] if shape.has_shared else [m]
            up = lambda name: torch.from_numpy(np.ascontiguousarray(np.concatenate([getattr(q, name) for q in parts]))).to(device)
            scales, codes, alpha = up("scales"), up("codes"), up("gscale")
            G = codes.shape[0]
            tiles = torch.empty(G * -(-N // 128) * scaled_col_tiles(MOE_SCALED_NVFP4, n) * 512, dtype=torch.uint8, device=device)
            moe_tile_scales(MOE_SCALED_NVFP4, scales, G, N, n, tiles)
            return scaled_mat(codes, tiles, alpha if factor is None else alpha * factor)

        H, I = shape.hidden, shape.inter
        h_scale = h_scale.to(device=device, dtype=torch.float32).contiguous()
        router, v = cls._router(host, device)
        return cls(shape, MOE_SCALED_NVFP4, router, v, stack(host.gate, host.s_gate, I, H, None),
                   stack(host.up, host.s_up, I, H, None), stack(host.down, host.s_down, H, I, h_scale), h_scale)

    @classmethod
    def quantized(cls, host, fmt, gate, up, down, h_scale=None, device="cuda"):
        """host: the layer's shape, router and gate vector; gate, up [G, inter, hidden], down [G, hidden, inter]: float32
        device tensors, quantised here to NVFP4 (fmt MOE_SCALED_NVFP4) or MXFP4 (MOE_SCALED_MXFP8).  h_scale (NVFP4): as in
        from_nvfp4."""
        nv = fmt == MOE_SCALED_NVFP4
        if h_scale is not None:
            h_scale = h_scale.to(device=device, dtype=torch.float32).contiguous()

        def mat(m, factor):
            G, N, n = m.shape
            g = (m.abs().amax((1, 2)) / 2688).clamp_min(2.0 ** -110) if nv else None
            codes = torch.empty((G, N, n // 2), dtype=torch.uint8, device=device)
            tiles = torch.zeros(G * -(-N // 128) * scaled_col_tiles(fmt, n) * 512, dtype=torch.uint8, device=device)
            moe_quantize(fmt if nv else MOE_SCALED_MXFP4, m.contiguous(), G * N, n, G, g, scaled_rows(codes, tiles))
            return scaled_mat(codes, tiles, g if factor is None else g * factor)

        router, v = cls._router(host, device)
        return cls(host.shape, fmt, router, v, mat(gate, None), mat(up, None), mat(down, h_scale), h_scale)


def calibrate_h_scale(layer: DeviceLayer, x: torch.Tensor, margin: float = 1.0) -> torch.Tensor:
    """The NVFP4 factor of h, the same for every expert (shared expert last), from a batch of tokens: the largest |h| the
    layer computes on x, over all experts, times margin, over 2688."""
    T, s = x.shape[0], layer.shape
    ws = workspace(layer.cfg, T, x.device)
    i32 = lambda *n: torch.empty(n, dtype=torch.int32, device=x.device)
    ids, p, w_s = i32(T, s.top_k), torch.empty((T, s.top_k), dtype=torch.int16, device=x.device), \
        torch.empty((T,), dtype=torch.int16, device=x.device)
    counts, offsets, perm, inv = i32(s.n_experts), i32(s.n_experts + 1), i32(T * s.top_k), i32(T * s.top_k)
    moe_route(layer.cfg, layer.w, x, T, None, None, None, ids, p, w_s, ws)
    moe_permute(layer.cfg, ids, T, counts, offsets, perm, inv, ws)
    h = torch.zeros((T * (s.top_k + 1), s.inter), device=x.device)
    moe_expert_stages(layer.cfg, layer.w, x, T, ids, counts, offsets, perm, h, None, MOE_PATH_AUTO, ws)
    return (h.abs().amax() * (margin / 2688)).clamp_min(2.0 ** -110).repeat(s.n_experts + s.has_shared)


def scaled_workspace(cfg: moe_config, fmt: int, T: int, device="cuda") -> torch.Tensor:
    """A zero-filled device workspace of moe_scaled_workspace_size bytes."""
    return torch.zeros(moe_scaled_workspace_size(cfg, fmt, T), dtype=torch.uint8, device=device)


def workspace(cfg: moe_config, T: int, device="cuda") -> torch.Tensor:
    """A zero-filled device workspace of moe_workspace_size bytes (uint8, 256-byte aligned by the allocator)."""
    return torch.zeros(moe_workspace_size(cfg, T), dtype=torch.uint8, device=device)


def forward(layer: DeviceLayer, x: torch.Tensor, ws: torch.Tensor, router_bias=None, logits_in=None,
            path: int = MOE_PATH_AUTO, stream=None, with_routing: bool = False, cfg: Optional[moe_config] = None):
    """y (int16 view of bf16 bits) = layer(x); optionally also (ids, p, w_s).  cfg overrides layer.cfg
    (e.g. to set wait_polls for one call)."""
    T = x.shape[0]
    dev = x.device
    y = torch.empty((T, layer.shape.hidden), dtype=torch.int16, device=dev)
    ids = p = w_s = None
    if with_routing:
        ids = torch.empty((T, layer.shape.top_k), dtype=torch.int32, device=dev)
        p = torch.empty((T, layer.shape.top_k), dtype=torch.int16, device=dev)
        w_s = torch.empty((max(T, 1),), dtype=torch.int16, device=dev)
    moe_forward(cfg if cfg is not None else layer.cfg, layer.w, x, T, router_bias, logits_in, y, ids, p, w_s, path,
                ws, stream)
    return (y, ids, p, w_s) if with_routing else y
