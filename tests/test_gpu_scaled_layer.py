"""The whole layer with block-scaled expert products: the composition of its operators, its routing that of
moe_forward, its refusals, and the example that chains norms and layers.

Each operator is checked against 64 bits on its own (test_gpu_scaled.py); here the layer must be exactly their
composition up to the weighted sum, which is taken in fp64 with the tolerance of an fp32 sum of k + 1 products
rounded to bf16.  Against the layer with 16-bit activations only the size of the difference is bounded: an
E2M1 code is within 1/4 of its value, an E4M3 one within 1/16, errors of many elements average out, so two
quantised stages stay below 0.3 (NVFP4) and 0.3 (MXFP8 activations against the same MXFP4 weights: 0.1).
"""
import ctypes
import dataclasses
import os
import sys

import numpy as np
import pytest
import torch

import quantised_moe_expert_gb300 as qm
from quantised_moe_expert_gb300 import synth

from . import scaled_ref as S

pytestmark = pytest.mark.gpu

NV, M8 = S.NV, S.M8
SMALL = synth.LayerShape(hidden=256, inter=128, n_experts=16, top_k=2, fmt="nvfp4")
ODD = synth.LayerShape(hidden=448, inter=192, n_experts=10, top_k=3, fmt="nvfp4")
QWEN = synth.QWEN_SHAPE_NVFP4


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    qm.load()


def tensor_x(shape, T, seed):
    return torch.from_numpy(synth.make_x(shape, T, seed).view(np.int16)).cuda()


def nvfp4_values(m):
    """fp32 device tensor of an NVFP4 host matrix stack."""
    v = S.dequantise(NV, S.unpack(NV, m.codes), m.scales) * m.gscale.astype(np.float64)[:, None, None]
    return torch.from_numpy(v.astype(np.float32)).cuda()


def make(shape, fmt, seed=3, x=None):
    host = synth.make_weights(shape, seed)
    if fmt == NV:
        plain = qm.DeviceLayer(host)
        x = tensor_x(shape, 64, 99) if x is None else x
        return host, qm.ScaledLayer.from_nvfp4(host, qm.calibrate_h_scale(plain, x, margin=1.5))
    cat = lambda a, b: torch.cat([nvfp4_values(a), nvfp4_values(b)]) if shape.has_shared else nvfp4_values(a)   # noqa: E731
    return host, qm.ScaledLayer.quantized(host, M8, cat(host.gate, host.s_gate), cat(host.up, host.s_up), cat(host.down, host.s_down))


def forward(layer, x, T, **kw):
    s = layer.shape
    y = torch.empty((T, s.hidden), dtype=torch.int16, device="cuda")
    ids = torch.empty((T, s.top_k), dtype=torch.int32, device="cuda")
    p = torch.empty((T, s.top_k), dtype=torch.int16, device="cuda")
    w_s = torch.empty((T,), dtype=torch.int16, device="cuda")
    ws = qm.scaled_workspace(layer.cfg, layer.fmt, T)
    qm.moe_scaled_forward(layer.cfg, layer.w, x, T, None, None, y, ids, p, w_s, ws, **kw)
    assert qm.moe_get_device_status(ws) == 0
    return y, ids, p, w_s


def f64(t):
    return t.view(torch.bfloat16).double().cpu().numpy()


@pytest.mark.parametrize("fmt", [NV, M8])
@pytest.mark.parametrize("shape,T", [(SMALL, 1), (SMALL, 5), (SMALL, 130), (QWEN, 1), (QWEN, 16), (QWEN, 200),
                                     (dataclasses.replace(SMALL, has_shared=0), 33), (ODD, 7)])
def test_layer_is_the_composition_of_its_operators(fmt, shape, T):
    if fmt == M8 and shape is ODD:
        pytest.skip("MXFP8 rows are multiples of 128")
    if fmt == M8 and shape.n_experts == 256:
        shape = dataclasses.replace(shape, n_experts=24)           # quantising 257 experts on the host takes long
    host, layer = make(shape, fmt)
    s, k, sh, E = shape, shape.top_k, shape.has_shared, shape.n_experts
    x = tensor_x(s, T, 7)
    y, ids, p, w_s = forward(layer, x, T)
    # routing: that of moe_route on the same x
    ws = qm.workspace(layer.cfg, T)
    i32 = lambda *n: torch.empty(n, dtype=torch.int32, device="cuda")              # noqa: E731
    ids2, p2, w2 = i32(T, k), torch.empty_like(p), torch.empty_like(w_s)
    mw = qm.moe_weights()
    mw.router, mw.shared_gate_vec = layer.w.router, layer.w.shared_gate_vec
    qm.moe_route(layer.cfg, mw, x, T, None, None, None, ids2, p2, w2, ws)
    assert torch.equal(ids, ids2) and torch.equal(p, p2) and (not sh or torch.equal(w_s, w2))
    # operators
    counts, offsets, perm, inv = i32(E), i32(E + 1), i32(T * k), i32(T * k)
    qm.moe_permute(layer.cfg, ids, T, counts, offsets, perm, inv, ws)
    R, G = T * (k + sh), E + sh
    xq, h = qm.scaled_rows_empty(fmt, R, s.hidden, G), qm.scaled_rows_empty(fmt, R, s.inter, G, row_scale=False)
    qm.moe_quantize_routed(fmt, x, T, s.hidden, k, E, sh, ids, inv, offsets, xq, ws)
    qm.moe_scaled_swiglu(fmt, xq, layer.w.gate, layer.w.up, R, s.inter, s.hidden, G, offsets, layer.tensors[5], h, ws)
    slots = torch.empty((R, s.hidden), device="cuda")
    qm.moe_scaled_gemm(fmt, h, layer.w.down, R, s.hidden, s.inter, G, offsets, slots, ws)
    assert qm.moe_get_device_status(ws) == 0
    v = slots.double().cpu().numpy()
    pos, pw = inv.cpu().numpy().reshape(T, k), f64(p)
    terms = v[pos] * pw[:, :, None]
    if sh:
        terms = np.concatenate([terms, (v[T * k:] * f64(w_s)[:, None])[:, None]], 1)
    want = terms.sum(1)
    tol = (k + 2) * 2.0 ** -24 * np.abs(terms).sum(1) + 2.0 ** -8 * np.abs(want)
    assert (np.abs(f64(y) - want) <= tol).all()
    # the expert-sorted rows' values against 64 bits, through the whole pair of products
    token = perm.cpu().numpy() // k
    assert np.isfinite(v).all() and len(token) == T * k


@pytest.mark.parametrize("shape,T", [(SMALL, 40), (QWEN, 16)])
def test_layer_against_16_bit_activations(shape, T):
    x = tensor_x(shape, T, 11)
    host, layer = make(shape, NV, x=x)
    plain = qm.DeviceLayer(host)
    ref = f64(qm.forward(plain, x, qm.workspace(plain.cfg, T)))
    got = f64(forward(layer, x, T)[0])
    assert np.linalg.norm(got - ref) <= 0.3 * np.linalg.norm(ref)


def test_mxfp8_layer_against_its_weights():
    """MXFP8 activations against fp64 products of the same MXFP4 weights."""
    T, s = 24, SMALL
    host, layer = make(s, M8)
    x = tensor_x(s, T, 5)
    y, ids, p, w_s = forward(layer, x, T)
    G, N, n = s.n_experts + 1, s.inter, s.hidden

    def values(m, N, n):
        codes, tiles = m.tensors[0].cpu().numpy(), m.tensors[1].cpu().numpy()
        rows = (np.arange(G)[:, None] * -(-N // 128) * 128 + np.arange(N)[None]).reshape(-1)
        return S.dequantise(S.M4, S.unpack(S.M4, codes), tiles[S.scale_index(S.M4, n, rows)].reshape(G, N, -1))

    gate, up, down = (values(m, *d) for m, d in zip(layer.tensors[2:5], ((s.inter, s.hidden),) * 2 + ((s.hidden, s.inter),)))
    xv = f64(x)
    h = S.silu(np.einsum("th,gih->tgi", xv, gate)) * np.einsum("th,gih->tgi", xv, up)
    out = np.einsum("tgi,ghi->tgh", h, down)
    pick, pw = ids.cpu().numpy(), f64(p)
    ref = (np.take_along_axis(out, pick[:, :, None], 1) * pw[:, :, None]).sum(1) + out[:, -1] * f64(w_s)[:, None]
    assert np.linalg.norm(f64(y) - ref) <= 0.1 * np.linalg.norm(ref)


def test_layer_reruns_and_streams_agree():
    T = 50
    host, layer = make(SMALL, NV)
    x = tensor_x(SMALL, T, 4)
    first = forward(layer, x, T)[0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert torch.equal(first, forward(layer, x, T)[0])
    y, ws = torch.empty_like(first), qm.scaled_workspace(layer.cfg, NV, T)
    torch.cuda.synchronize()
    qm.moe_scaled_forward(layer.cfg, layer.w, x, T, None, None, y, None, None, None, ws, stream=side)
    side.synchronize()
    assert torch.equal(first, y)


def test_layer_with_given_logits_and_bias():
    T = 20
    host, layer = make(SMALL, NV)
    x = tensor_x(SMALL, T, 8)
    logits = torch.randn(T, SMALL.n_experts, device="cuda")
    ws = qm.scaled_workspace(layer.cfg, NV, T)
    y, ids = torch.empty((T, SMALL.hidden), dtype=torch.int16, device="cuda"), torch.empty((T, 2), dtype=torch.int32, device="cuda")
    qm.moe_scaled_forward(layer.cfg, layer.w, x, T, None, logits, y, ids, None, None, ws)
    assert torch.equal(ids.long(), logits.topk(2, dim=1).indices)
    bias = torch.zeros(SMALL.n_experts, device="cuda")
    bias[5] = 100.0
    qm.moe_scaled_forward(layer.cfg, layer.w, x, T, bias, None, y, ids, None, None, ws)
    assert (ids[:, 0] == 5).all() and qm.moe_get_device_status(ws) == 0


def test_layer_refusals():
    host, layer = make(SMALL, NV)
    lib, T = qm.load(), 4
    x = tensor_x(SMALL, T, 1)
    y = torch.empty((T, SMALL.hidden), dtype=torch.int16, device="cuda")
    ws = qm.scaled_workspace(layer.cfg, NV, T)

    def call(cfg=layer.cfg, w=layer.w, x=x.data_ptr(), T=T, y=y.data_ptr(), ws_p=ws.data_ptr(), n=ws.numel()):
        return lib.moe_scaled_forward(ctypes.byref(cfg), ctypes.byref(w) if w is not None else None, x, T, None, None, y, None, None,
                                      None, ws_p, n, None)

    def change(**kw):
        w = qm.moe_scaled_weights.from_buffer_copy(layer.w)
        for k, v in kw.items():
            setattr(w, k, v)
        return w

    assert call() == qm.MOE_OK and call(T=0) == qm.MOE_OK
    assert call(w=None) == qm.MOE_ERR_INVALID_ARG and call(x=None) == qm.MOE_ERR_INVALID_ARG
    assert call(y=y.data_ptr() + 2) == qm.MOE_ERR_INVALID_ARG and call(T=-1) == qm.MOE_ERR_INVALID_ARG
    assert call(n=ws.numel() - 1) == qm.MOE_ERR_WORKSPACE
    assert call(w=change(h_scale=None)) == qm.MOE_ERR_INVALID_ARG
    assert call(w=change(format=3)) == qm.MOE_ERR_UNSUPPORTED
    assert call(w=change(format=M8)) == qm.MOE_ERR_INVALID_ARG                    # MXFP8 takes no h_scale
    assert call(w=change(gate=qm.moe_scaled_mat(None, None, None))) == qm.MOE_ERR_INVALID_ARG
    odd = qm.config_of(dataclasses.replace(SMALL, hidden=320))
    assert call(cfg=odd, w=change(format=M8, h_scale=None)) == qm.MOE_ERR_UNSUPPORTED
    torch.cuda.synchronize()


def test_example_runs():
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import scaled_layers
    d = scaled_layers.run(dataclasses.replace(SMALL, hidden=512), tokens=48, layers=3)
    assert len(d) == 3 and all(0 < v < 0.5 for v in d)


@pytest.mark.parametrize("T", [1, 40])
def test_waits_that_run_out_are_reported(T):
    """A limit of one poll on the in-kernel waits: MOE_ERR_TIMEOUT in the status word, the kernels return, and the same
    workspace serves the next call."""
    host, layer = make(SMALL, NV)
    x = tensor_x(SMALL, T, 2)
    want = forward(layer, x, T)[0]
    y, ws = torch.empty_like(want), qm.scaled_workspace(layer.cfg, NV, T)
    short = qm.config_of(SMALL, wait_polls=1)
    qm.moe_scaled_forward(short, layer.w, x, T, None, None, y, None, None, None, ws)
    assert qm.moe_get_device_status(ws) == qm.MOE_ERR_TIMEOUT
    qm.moe_scaled_forward(layer.cfg, layer.w, x, T, None, None, y, None, None, None, ws)
    assert qm.moe_get_device_status(ws) == 0 and torch.equal(y, want)
