"""The Python bindings of the block-scaled operators refuse tensors whose addresses the library would misread: another
element type, or elements that are not dense.  No call here has rows, and none reaches a GPU."""
import pytest
import torch

import quantised_moe_expert_gb300 as qm
from quantised_moe_expert_gb300 import synth

NV, M8 = qm.MOE_SCALED_NVFP4, qm.MOE_SCALED_MXFP8
STREAM = 0


def dense(n, dtype):
    """n elements at a 64-byte boundary."""
    raw = torch.zeros(n * torch.empty(0, dtype=dtype).element_size() + 64, dtype=torch.uint8)
    lo = -raw.data_ptr() % 64
    return raw[lo:lo + raw.numel() - 64].view(dtype)


def strided(n, dtype):
    return dense(2 * n, dtype)[::2]


X, Y = dense(256, torch.bfloat16), dense(256, torch.int16)
F, I, U = dense(64, torch.float32), dense(64, torch.int32), dense(4096, torch.uint8)
ROWS, FACTORS, MAT = qm.scaled_rows(U, U), qm.scaled_rows(U, U, F), qm.scaled_mat(U, U, F)
CFG = qm.config_of(synth.LayerShape(hidden=256, inter=128, n_experts=8, top_k=2))
W = qm.moe_scaled_weights(M8, qm.moe_qmat(*[U.data_ptr()] * 3, None), Y.data_ptr(), MAT, MAT, MAT, None)


def norm(x=X, residual=X, weight=X, sum_out=Y, y_out=X):
    qm.moe_add_rmsnorm(x, residual, weight, 0.0, 1e-6, 0, 256, sum_out, y_out, M8, ROWS, STREAM)


def quantize(x=X, gscale=F):
    qm.moe_quantize(NV, x, 0, 256, 1, gscale, ROWS, STREAM)


def routed(x=X, ids=I, inv_perm=I, offsets=I):
    qm.moe_quantize_routed(M8, x, 0, 256, 2, 8, 1, ids, inv_perm, offsets, ROWS, U, STREAM)


def tiles(src=U, dst=U):
    qm.moe_tile_scales(M8, src, 0, 1, 256, dst, STREAM)


def gemm(offsets=I, y=X):
    qm.moe_scaled_gemm(M8, ROWS, MAT, 0, 256, 256, 1, offsets, y, U, STREAM)


def swiglu(offsets=I, h_scale=F):
    qm.moe_scaled_swiglu(NV, ROWS, MAT, MAT, 0, 256, 256, 1, offsets, h_scale, ROWS, U, STREAM)


def forward(x=X, router_bias=F, logits_in=F, y=X, ids_out=I, p_out=X, w_shared_out=Y):
    ws = dense(qm.moe_scaled_workspace_size(CFG, M8, 0), torch.uint8)
    qm.moe_scaled_forward(CFG, W, x, 0, router_bias, logits_in, y, ids_out, p_out, w_shared_out, ws, STREAM)


BITS = (torch.bfloat16, torch.int16, torch.uint16)
TENSORS = [(norm, n, BITS) for n in ("x", "residual", "weight", "sum_out", "y_out")]
TENSORS += [(quantize, "x", BITS + (torch.float32,)), (quantize, "gscale", (torch.float32,)), (routed, "x", BITS)]
TENSORS += [(routed, n, (torch.int32,)) for n in ("ids", "inv_perm", "offsets")]
TENSORS += [(tiles, n, (torch.uint8, torch.int8, torch.float8_e4m3fn)) for n in ("src", "dst")]
TENSORS += [(gemm, "offsets", (torch.int32,)), (gemm, "y", BITS + (torch.float32,))]
TENSORS += [(swiglu, "offsets", (torch.int32,)), (swiglu, "h_scale", (torch.float32,))]
TENSORS += [(forward, n, BITS) for n in ("x", "y", "p_out", "w_shared_out")]
TENSORS += [(forward, "router_bias", (torch.float32,)), (forward, "logits_in", (torch.float32,)), (forward, "ids_out", (torch.int32,))]
ALL = BITS + (torch.float16, torch.float32, torch.float64, torch.int32, torch.int64, torch.uint8, torch.int8, torch.float8_e4m3fn)


@pytest.mark.parametrize("call,name,types", TENSORS, ids=[f"{c.__name__}-{n}" for c, n, _ in TENSORS])
def test_element_types_and_strides(call, name, types):
    call()
    for dtype in ALL:
        if dtype in types:
            call(**{name: dense(256, dtype)})
            bad = strided(256, dtype)
        else:
            bad = dense(256, dtype)
        with pytest.raises(qm.MoeError) as e:
            call(**{name: bad})
        assert e.value.status == qm.MOE_ERR_INVALID_ARG and "moe_" in str(e.value)


@pytest.mark.parametrize("make", [qm.scaled_rows, qm.scaled_mat])
def test_descriptors(make):
    make(U, U), make(U, U, F), make(U.view(torch.float8_e4m3fn), U, None)
    for bad in ((U[::2], U, F), (U, U[::2], F), (U, U, F[::2]), (U, U, F.double()), (U, U, F.bfloat16()), (U.view(64, 64).t(), U, F)):
        with pytest.raises(qm.MoeError) as e:
            make(*bad)
        assert e.value.status == qm.MOE_ERR_INVALID_ARG


SHAPE = synth.LayerShape(hidden=128, inter=64, n_experts=4, top_k=2, fmt="nvfp4")


@pytest.mark.parametrize("h_scale", [torch.full((5,), 0.5, dtype=torch.float16), torch.full((5,), 0.5, dtype=torch.float64),
                                     torch.tensor([0.5]).expand(5), torch.full((5,), 0.5)], ids=["fp16", "fp64", "expanded", "fp32"])
def test_quantized_layer_takes_any_calibration(monkeypatch, h_scale):
    """The kernels read fp32 factors of h, one after the other, whatever the calibration came in."""
    monkeypatch.setattr(qm, "moe_quantize", lambda *a: None)
    G, H, I = 5, SHAPE.hidden, SHAPE.inter
    gen = torch.Generator().manual_seed(0)
    gate, up, down = (torch.randn(s, generator=gen) for s in ((G, I, H), (G, I, H), (G, H, I)))
    layer = qm.ScaledLayer.quantized(synth.make_weights(SHAPE, 1), NV, gate, up, down, h_scale, device="cpu")
    held = layer.tensors[5]
    assert held.dtype == torch.float32 and held.is_contiguous() and torch.equal(held, torch.full((G,), 0.5))
    assert layer.w.h_scale == held.data_ptr()
    assert torch.equal(layer.tensors[4].tensors[2], (down.abs().amax((1, 2)) / 2688) * 0.5)


def test_layer_refuses_factors_it_would_misread():
    router = [U, Y, Y]
    five = F[:5]
    qm.ScaledLayer(SHAPE, NV, router, Y, MAT, MAT, MAT, five)
    for v, h_scale in ((Y, five.double()), (Y, F[:10:2]), (F, five), (Y[::2], five), (Y, F[:4]), (Y, F[:1])):
        with pytest.raises(qm.MoeError) as e:
            qm.ScaledLayer(SHAPE, NV, router, v, MAT, MAT, MAT, h_scale)
        assert e.value.status == qm.MOE_ERR_INVALID_ARG
