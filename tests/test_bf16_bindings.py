"""The Python bindings of the 16-bit operators refuse tensors whose addresses the library would misread: another element type,
or elements that are not dense.  No call here has rows, and none reaches a GPU."""
import pytest
import torch

import quantised_moe_expert_gb300 as qm
from tests.test_scaled_bindings import ALL, BITS, dense, strided

STREAM = 0
X, F, I = dense(256, torch.bfloat16), dense(64, torch.float32), dense(64, torch.int32)
WS = dense(1 << 16, torch.uint8)


def gemm(a=X, w=X, a2=X, w2=X, offsets=I, bias=X, residual=X, pre_out=X, y=X):
    qm.moe_gemm(a, w, a2, w2, 0, 0, 16, 16, 1, offsets, bias, qm.MOE_ACT_SILU, residual, pre_out, y, WS, STREAM)


def glu(a=X, gate=X, up=X, gate_bias=X, up_bias=X, offsets=I, gate_out=X, up_out=X, h=X):
    qm.moe_gemm_glu(a, gate, up, gate_bias, up_bias, qm.MOE_ACT_SILU, 0, 16, 16, 1, offsets, gate_out, up_out, h, WS, STREAM)


def wgrad(dy=X, x=X, offsets=I, dw=F, db=F):
    qm.moe_gemm_wgrad(dy, x, 0, 8, 8, 1, offsets, 1, dw, db, WS, STREAM)


def act_grad(dy=X, pre=X, up=X, dpre=X, dup=dense(256, torch.bfloat16)):
    qm.moe_act_grad(qm.MOE_ACT_SILU, dy, pre, up, 0, 16, dpre, dup, STREAM)


def dispatch(x=X, inv_perm=I, y=X):
    qm.moe_dispatch(x, 0, 16, 2, 1, inv_perm, y, WS, STREAM)


def weighted(rows=X, inv_perm=I, p=X, w_shared=X, y=X):
    qm.moe_weighted_sum(rows, 0, 16, 2, 1, inv_perm, p, w_shared, y, WS, STREAM)


def weighted_grad(dy=X, rows=X, inv_perm=I, p=X, w_shared=X, drows=X, dp=F, dw_shared=F):
    qm.moe_weighted_sum_grad(dy, rows, 0, 16, 2, 1, inv_perm, p, w_shared, drows, dp, dw_shared, WS, STREAM)


def norm(x=X, residual=X, gate=X, post_weight=X, pre_weight=X, sum_out=X, y_out=X):
    qm.moe_gated_norm(x, residual, gate, qm.MOE_GATE_FULL, qm.MOE_ACT_SILU, 1.0, 1, post_weight, pre_weight, 0.0, 1e-6, 0, 16, sum_out,
                      y_out, STREAM)


def norm_grad(x=X, sum=X, gate=X, post_weight=X, pre_weight=X, dy=X, dsum=X, dx=X, dresidual=X, dgate=X):
    qm.moe_gated_norm_grad(x, sum, gate, qm.MOE_GATE_FULL, qm.MOE_ACT_SILU, 1.0, 1, post_weight, pre_weight, 0.0, 1e-6, 0, 16, dy, dsum, dx,
                           dresidual, dgate, None, None, WS, STREAM)


TENSORS = [(gemm, n, BITS) for n in ("a", "w", "a2", "w2", "bias", "residual", "pre_out")] + [(gemm, "y", BITS + (torch.float32,))]
TENSORS += [(glu, n, BITS) for n in ("a", "gate", "up", "gate_bias", "up_bias", "gate_out", "up_out", "h")]
TENSORS += [(c, "offsets", (torch.int32,)) for c in (gemm, glu, wgrad)]
TENSORS += [(wgrad, n, BITS) for n in ("dy", "x")] + [(wgrad, "db", (torch.float32,))]
TENSORS += [(act_grad, n, BITS) for n in ("dy", "pre", "up", "dpre", "dup")]
TENSORS += [(c, "inv_perm", (torch.int32,)) for c in (dispatch, weighted, weighted_grad)]
TENSORS += [(dispatch, n, BITS) for n in ("x", "y")] + [(weighted, n, BITS) for n in ("rows", "p", "w_shared", "y")]
TENSORS += [(weighted_grad, n, BITS) for n in ("dy", "rows", "p", "w_shared", "drows")]
TENSORS += [(weighted_grad, n, (torch.float32,)) for n in ("dp", "dw_shared")]
TENSORS += [(norm, n, BITS) for n in ("x", "residual", "gate", "post_weight", "pre_weight", "sum_out", "y_out")]
TENSORS += [(norm_grad, n, BITS) for n in ("x", "sum", "gate", "post_weight", "pre_weight", "dy", "dsum", "dx", "dresidual", "dgate")]


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


def test_gradients_of_one_type():
    """dw and db are both fp32 or both bf16; sums that are added to are fp32."""
    for dw, db in ((F, X), (X, F), (F.double(), None), (F[::2], None)):
        with pytest.raises(qm.MoeError):
            wgrad(dw=dw, db=db)
    with pytest.raises(qm.MoeError) as e:
        wgrad(dw=X, db=X)
    assert e.value.status == qm.MOE_ERR_UNSUPPORTED


def test_a_gate_s_gradient_has_its_type():
    for shape, bad in ((qm.MOE_GATE_ROW, X), (qm.MOE_GATE_CHANNEL, X), (qm.MOE_GATE_FULL, F)):
        with pytest.raises(qm.MoeError):
            qm.moe_gated_norm_grad(X, X, X, shape, 0, 1.0, 0, None, None, 0.0, 1e-6, 0, 16, X, X, X, None, bad, None, None, WS, STREAM)
