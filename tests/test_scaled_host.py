"""Host-side checks of the block-scaled operators: bad arguments are refused before any GPU work.

Every call below fails validation or has no rows; the fake device pointers are never dereferenced.
"""
import ctypes

import pytest

import quantised_moe_expert_gb300 as qm

FAKE = 0x7f0000010000
ODD = FAKE + 8
NV, M8, M4 = qm.MOE_SCALED_NVFP4, qm.MOE_SCALED_MXFP8, qm.MOE_SCALED_MXFP4
OK, INVALID, UNSUPPORTED, WS = qm.MOE_OK, qm.MOE_ERR_INVALID_ARG, qm.MOE_ERR_UNSUPPORTED, qm.MOE_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    return qm.load()


def rows(codes=FAKE, scales=FAKE, row_scale=None):
    return qm.moe_scaled_rows(codes, scales, row_scale)


def mat(codes=FAKE, scales=FAKE, alpha=None):
    return qm.moe_scaled_mat(codes, scales, alpha)


def norm(lib, x=FAKE, residual=FAKE, weight=FAKE, eps=1e-6, T=0, n=2048, sum_out=FAKE, y_out=FAKE, fmt=M8, q=None, none=False):
    q = None if none else (q or rows())
    return lib.moe_add_rmsnorm(x, residual, weight, 0.0, eps, T, n, sum_out, y_out, fmt, q, None)


@pytest.mark.parametrize("kw,expect", [
    ({}, OK),
    (dict(fmt=NV, q=rows(row_scale=FAKE)), OK),
    (dict(fmt=0, none=True, n=8), OK),
    (dict(residual=None, weight=None, sum_out=None, y_out=None), OK),
    (dict(eps=0.0), OK),
    (dict(n=16384), OK),
    (dict(x=None), INVALID), (dict(x=ODD), INVALID), (dict(residual=ODD), INVALID), (dict(weight=ODD), INVALID),
    (dict(sum_out=ODD), INVALID), (dict(y_out=ODD), INVALID),
    (dict(T=-1), INVALID), (dict(n=0), INVALID), (dict(n=-32), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID),
    (dict(n=2056), UNSUPPORTED), (dict(n=16416), UNSUPPORTED), (dict(fmt=NV, n=2056, q=rows(row_scale=FAKE)), UNSUPPORTED),
    (dict(fmt=0, none=True, n=12), UNSUPPORTED),
    (dict(fmt=M4), UNSUPPORTED), (dict(fmt=7), UNSUPPORTED), (dict(fmt=-1), UNSUPPORTED),
    (dict(none=True), INVALID), (dict(fmt=0), INVALID),
    (dict(fmt=NV), INVALID),                              # NVFP4 rows need room for their factors
    (dict(q=rows(row_scale=FAKE)), INVALID),              # MXFP8 rows have none
    (dict(q=rows(codes=ODD)), INVALID), (dict(q=rows(scales=None)), INVALID),
])
def test_norm_arguments(lib, kw, expect):
    assert norm(lib, **kw) == expect


def quantize(lib, fmt=M8, x=FAKE, x_f32=0, T=0, n=256, groups=1, gscale=None, q=None):
    return lib.moe_quantize(fmt, x, x_f32, T, n, groups, gscale, q or rows(), None)


@pytest.mark.parametrize("kw,expect", [
    ({}, OK), (dict(fmt=M4), OK), (dict(x_f32=1), OK), (dict(n=1 << 20), OK), (dict(groups=3), OK),
    (dict(fmt=NV, q=rows(row_scale=FAKE)), OK), (dict(fmt=NV, gscale=FAKE), OK),
    (dict(x_f32=2), INVALID), (dict(T=-1), INVALID), (dict(n=0), INVALID), (dict(groups=0), INVALID),
    (dict(T=4, groups=3), INVALID), (dict(x=ODD), INVALID),
    (dict(n=48), UNSUPPORTED), (dict(fmt=NV, n=24, gscale=FAKE), UNSUPPORTED), (dict(fmt=9), UNSUPPORTED),
    (dict(fmt=NV, n=16400, q=rows(row_scale=FAKE)), UNSUPPORTED),
    (dict(fmt=NV), INVALID),                                             # neither a factor nor room for one
    (dict(fmt=NV, gscale=FAKE, q=rows(row_scale=FAKE)), INVALID),        # both
    (dict(gscale=FAKE), INVALID), (dict(fmt=NV, gscale=FAKE + 2), INVALID),
])
def test_quantize_arguments(lib, kw, expect):
    assert quantize(lib, **kw) == expect


def routed(lib, fmt=M8, x=FAKE, T=0, n=256, k=2, E=16, shared=1, ids=FAKE, inv=FAKE, offsets=FAKE, q=None, ws=FAKE,
           ws_bytes=512):
    return lib.moe_quantize_routed(fmt, x, T, n, k, E, shared, ids, inv, offsets, q or rows(), ws, ws_bytes, None)


@pytest.mark.parametrize("kw,expect", [
    ({}, OK), (dict(fmt=NV, q=rows(row_scale=FAKE)), OK), (dict(shared=0), OK),
    (dict(fmt=M4), UNSUPPORTED), (dict(k=17), UNSUPPORTED), (dict(n=100), UNSUPPORTED), (dict(E=1024), UNSUPPORTED),
    (dict(fmt=NV), INVALID), (dict(k=0), INVALID), (dict(E=0), INVALID), (dict(shared=2), INVALID), (dict(T=65537), INVALID),
    (dict(ids=None), INVALID), (dict(inv=None), INVALID), (dict(offsets=FAKE + 2), INVALID), (dict(x=ODD), INVALID),
    (dict(ws=None), INVALID), (dict(ws=ODD), INVALID), (dict(ws_bytes=511), WS),
])
def test_quantize_routed_arguments(lib, kw, expect):
    assert routed(lib, **kw) == expect


def gemm(lib, fmt=NV, a=None, w=None, R=0, N=512, K=256, G=1, offsets=None, y=FAKE, f32=0, ws=FAKE, ws_bytes=512):
    return lib.moe_scaled_gemm(fmt, a or rows(row_scale=FAKE if fmt == NV else None), w or mat(), R, N, K, G, offsets, y, f32,
                               ws, ws_bytes, None)


@pytest.mark.parametrize("kw,expect", [
    ({}, OK), (dict(fmt=M8), OK), (dict(G=256, offsets=FAKE), OK), (dict(N=8, K=64), OK), (dict(f32=1), OK), (dict(a=rows()), OK),
    (dict(fmt=M4), UNSUPPORTED), (dict(fmt=0), UNSUPPORTED), (dict(K=96), UNSUPPORTED), (dict(fmt=M8, K=192), UNSUPPORTED),
    (dict(N=12), UNSUPPORTED), (dict(K=65600), UNSUPPORTED), (dict(G=1025, offsets=FAKE), UNSUPPORTED),
    (dict(N=(1 << 20) + 8), UNSUPPORTED),
    (dict(R=-1), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(G=0), INVALID), (dict(G=2), INVALID),
    (dict(G=2, offsets=FAKE + 1), INVALID), (dict(y=ODD), INVALID), (dict(y=None), INVALID), (dict(f32=3), INVALID),
    (dict(a=rows(codes=ODD)), INVALID), (dict(w=mat(codes=ODD)), INVALID), (dict(w=mat(scales=None)), INVALID),
    (dict(w=mat(alpha=FAKE + 2)), INVALID), (dict(fmt=M8, w=mat(codes=FAKE + 16)), INVALID),
    (dict(fmt=M8, a=rows(row_scale=FAKE)), INVALID),
    (dict(ws=None), INVALID), (dict(ws_bytes=0), WS),
])
def test_gemm_arguments(lib, kw, expect):
    assert gemm(lib, **kw) == expect


def swiglu(lib, fmt=NV, a=None, gate=None, up=None, R=0, inter=128, K=256, G=1, offsets=None, h_scale="auto", h=None, ws=FAKE,
           ws_bytes=512):
    hs = (FAKE if fmt == NV else None) if h_scale == "auto" else h_scale
    return lib.moe_scaled_swiglu(fmt, a or rows(), gate or mat(), up or mat(), R, inter, K, G, offsets, hs, h or rows(), ws,
                                 ws_bytes, None)


@pytest.mark.parametrize("kw,expect", [
    ({}, OK), (dict(fmt=M8), OK), (dict(inter=64), OK),
    (dict(inter=96), UNSUPPORTED), (dict(fmt=M8, inter=64), UNSUPPORTED), (dict(fmt=M4), UNSUPPORTED), (dict(K=32), UNSUPPORTED),
    (dict(h_scale=None), INVALID), (dict(fmt=M8, h_scale=FAKE), INVALID), (dict(h=rows(row_scale=FAKE)), INVALID),
    (dict(gate=mat(codes=None)), INVALID), (dict(up=mat(scales=ODD)), INVALID), (dict(h=rows(codes=ODD)), INVALID),
    (dict(G=3), INVALID), (dict(ws=ODD), INVALID), (dict(ws_bytes=100), WS),
])
def test_swiglu_arguments(lib, kw, expect):
    assert swiglu(lib, **kw) == expect


@pytest.mark.parametrize("args,expect", [
    ((NV, FAKE, 0, 128, 256, FAKE), OK), ((M4, FAKE, 0, 1, 32, FAKE), OK),
    ((9, FAKE, 0, 128, 256, FAKE), UNSUPPORTED), ((M4, FAKE, 0, 128, 48, FAKE), UNSUPPORTED),
    ((NV, FAKE, -1, 128, 256, FAKE), INVALID), ((NV, None, 0, 128, 256, FAKE), INVALID), ((NV, FAKE, 0, 128, 256, ODD), INVALID),
    ((NV, FAKE, 0, 0, 256, FAKE), INVALID),
])
def test_tile_scales_arguments(lib, args, expect):
    assert lib.moe_tile_scales(*args, None) == expect


def test_errors_reach_python():
    with pytest.raises(qm.MoeError) as e:
        qm._check("moe_scaled_gemm", gemm(qm.load(), K=96))
    assert e.value.status == UNSUPPORTED and "moe_scaled_gemm" in str(e.value)


@pytest.mark.parametrize("fmt,kw,expect", [
    (NV, {}, OK), (M8, {}, OK), (M4, {}, UNSUPPORTED), (0, {}, UNSUPPORTED),
    (M8, dict(hidden=2112), UNSUPPORTED), (NV, dict(hidden=2112), OK), (NV, dict(top_k=17), UNSUPPORTED), (NV, dict(hidden=0), INVALID),
])
def test_layer_workspace_size(lib, fmt, kw, expect):
    d = dict(hidden=2048, inter=512, n_experts=256, top_k=8, group=64, bits=4, router_bits=8, has_shared=1, wait_polls=0)
    cfg, n, plain = qm.moe_config(**{**d, **kw}), ctypes.c_size_t(), ctypes.c_size_t()
    assert lib.moe_scaled_workspace_size(ctypes.byref(cfg), fmt, 16, ctypes.byref(n)) == expect
    if expect == OK:
        assert lib.moe_workspace_size(ctypes.byref(cfg), 16, ctypes.byref(plain)) == OK and n.value > plain.value
        assert lib.moe_scaled_workspace_size(ctypes.byref(cfg), fmt, -1, ctypes.byref(n)) == INVALID
        assert lib.moe_scaled_workspace_size(ctypes.byref(cfg), fmt, 16, None) == INVALID


@pytest.mark.parametrize("n,expect", [(16400, OK), (65536, OK), (1 << 20, OK), ((1 << 20) + 16, UNSUPPORTED)])
def test_quantize_long_rows_with_a_given_factor(lib, n, expect):
    """Only rows whose factor comes from the whole row are limited to what a kernel keeps of one."""
    assert quantize(lib, fmt=NV, gscale=FAKE, n=n) == expect
    assert quantize(lib, fmt=NV, q=rows(row_scale=FAKE), n=n) == UNSUPPORTED


@pytest.mark.parametrize("fmt,n,expect", [(M8, 16416, OK), (M8, 1 << 20, OK), (M8, (1 << 20) + 32, UNSUPPORTED), (NV, 16384, OK),
                                          (NV, 16400, UNSUPPORTED)])
def test_quantize_routed_row_lengths(lib, fmt, n, expect):
    assert routed(lib, fmt=fmt, q=rows(row_scale=FAKE if fmt == NV else None), n=n) == expect
