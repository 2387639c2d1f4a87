"""Host-side checks of the 16-bit operators: bad arguments are refused before any GPU work.

Every call below fails validation or has no rows; the fake device pointers are never dereferenced.
"""
import ctypes

import pytest

import quantised_moe_expert_gb300 as qm

FAKE = 0x7f0000010000
ODD = FAKE + 8
OK, INVALID, UNSUPPORTED, WS = qm.MOE_OK, qm.MOE_ERR_INVALID_ARG, qm.MOE_ERR_UNSUPPORTED, qm.MOE_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    return qm.load()


def gemm(lib, a=FAKE, w=FAKE, a2=None, w2=None, transposed=0, R=0, N=64, K=128, G=1, offsets=FAKE, bias=FAKE, act=1, residual=FAKE,
         pre=FAKE, y=FAKE, y_f32=0, ws=FAKE, ws_bytes=512):
    return lib.moe_gemm(a, w, a2, w2, transposed, R, N, K, G, offsets, bias, act, residual, pre, y, y_f32, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,expect", [
    ({}, OK), (dict(offsets=None), OK), (dict(G=1024), OK), (dict(transposed=1), OK), (dict(y_f32=1), OK), (dict(a2=FAKE, w2=FAKE), OK),
    (dict(bias=None, residual=None, pre=None), OK), (dict(a=None, y=None), OK), (dict(a=None, a2=None, w2=FAKE, y=None), OK),
    (dict(N=1 << 20, K=65536), OK), (dict(N=8, K=8), OK), (dict(act=0), OK), (dict(act=3), OK),
    (dict(R=-1), INVALID), (dict(R=(1 << 21) + 1), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(G=0), INVALID),
    (dict(N=-8), INVALID), (dict(R=4, a=None), INVALID), (dict(R=4, y=None), INVALID), (dict(w=None), INVALID), (dict(w=ODD), INVALID),
    (dict(R=4, a=ODD), INVALID), (dict(a2=FAKE), INVALID), (dict(R=4, w2=FAKE), INVALID), (dict(a2=ODD, w2=FAKE), INVALID),
    (dict(G=2, offsets=None), INVALID), (dict(offsets=FAKE + 2), INVALID), (dict(bias=ODD), INVALID), (dict(residual=ODD), INVALID),
    (dict(pre=ODD), INVALID), (dict(y=ODD), INVALID), (dict(transposed=2), INVALID), (dict(y_f32=2), INVALID),
    (dict(act=-1), INVALID), (dict(act=9), INVALID), (dict(act=4), UNSUPPORTED),
    (dict(N=12), UNSUPPORTED), (dict(K=12), UNSUPPORTED), (dict(K=65544), UNSUPPORTED), (dict(N=(1 << 20) + 8), UNSUPPORTED),
    (dict(G=1025), UNSUPPORTED), (dict(ws=None), INVALID), (dict(ws=ODD), INVALID), (dict(ws_bytes=511), WS),
])
def test_gemm_arguments(lib, kw, expect):
    assert gemm(lib, **kw) == expect


def glu(lib, a=FAKE, gate=FAKE, up=FAKE, gb=FAKE, ub=FAKE, act=1, R=0, I=64, K=128, G=1, offsets=None, g=FAKE, u=FAKE, h=FAKE, ws=FAKE,
        ws_bytes=512):
    return lib.moe_gemm_glu(a, gate, up, gb, ub, act, R, I, K, G, offsets, g, u, h, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,expect", [
    ({}, OK), (dict(gb=None, ub=None, g=None, u=None), OK), (dict(gb=None), OK), (dict(a=None, h=None), OK), (dict(act=2), OK),
    (dict(g=None), INVALID), (dict(u=None), INVALID), (dict(gate=None), INVALID), (dict(up=ODD), INVALID), (dict(gb=ODD), INVALID),
    (dict(ub=ODD), INVALID), (dict(g=ODD), INVALID), (dict(u=ODD), INVALID), (dict(R=2, h=None), INVALID), (dict(R=2, a=None), INVALID),
    (dict(act=4), UNSUPPORTED), (dict(act=5), INVALID), (dict(I=100), UNSUPPORTED), (dict(K=4), UNSUPPORTED), (dict(G=3), INVALID),
    (dict(ws=ODD), INVALID), (dict(ws_bytes=0), WS),
])
def test_glu_arguments(lib, kw, expect):
    assert glu(lib, **kw) == expect


def wgrad(lib, dy=FAKE, x=FAKE, R=0, N=64, K=128, G=1, offsets=None, accumulate=1, dw=FAKE, db=FAKE, f32=1, ws=FAKE, ws_bytes=512):
    # with accumulate == 1 a call without rows enqueues nothing
    return lib.moe_gemm_wgrad(dy, x, R, N, K, G, offsets, accumulate, dw, db, f32, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,expect", [
    ({}, OK), (dict(db=None), OK), (dict(dy=None, x=None), OK), (dict(G=4, offsets=FAKE), OK),
    (dict(f32=0), UNSUPPORTED),                           # sums are added to in 32 bits
    (dict(accumulate=2), INVALID), (dict(f32=2), INVALID), (dict(dw=None), INVALID), (dict(dw=ODD), INVALID), (dict(db=ODD), INVALID),
    (dict(R=3, dy=None), INVALID), (dict(R=3, x=ODD), INVALID), (dict(G=4), INVALID), (dict(N=4), UNSUPPORTED), (dict(K=65544), UNSUPPORTED),
    (dict(G=1024, offsets=FAKE, N=1 << 20, K=65536), UNSUPPORTED),       # tiles past 2^30
    (dict(R=-1), INVALID), (dict(ws=None), INVALID), (dict(ws_bytes=511), WS),
])
def test_wgrad_arguments(lib, kw, expect):
    assert wgrad(lib, **kw) == expect


def act_grad(lib, act=1, dy=FAKE, pre=FAKE, up=None, R=0, N=64, dpre=FAKE, dup=None):
    return lib.moe_act_grad(act, dy, pre, up, R, N, dpre, dup, None)


@pytest.mark.parametrize("kw,expect", [
    ({}, OK), (dict(up=FAKE, dup=FAKE + 64), OK), (dict(dy=None, pre=None, dpre=None), OK),
    (dict(act=4), UNSUPPORTED), (dict(act=7), INVALID), (dict(N=60), UNSUPPORTED), (dict(N=0), INVALID), (dict(R=-1), INVALID),
    (dict(R=(1 << 24) + 1), INVALID), (dict(R=2, up=FAKE), INVALID), (dict(R=2, dup=FAKE + 64), INVALID), (dict(R=2, up=FAKE, dup=FAKE), INVALID),
    (dict(R=2, dy=None), INVALID), (dict(pre=ODD), INVALID), (dict(up=ODD), INVALID), (dict(dpre=ODD), INVALID), (dict(dup=ODD), INVALID),
])
def test_act_grad_arguments(lib, kw, expect):
    assert act_grad(lib, **kw) == expect


def dispatch(lib, x=FAKE, T=0, n=64, k=2, shared=1, inv=FAKE, y=FAKE, ws=FAKE, ws_bytes=512):
    return lib.moe_dispatch(x, T, n, k, shared, inv, y, ws, ws_bytes, None)


def weighted(lib, rows=FAKE, T=0, n=64, k=2, shared=1, inv=FAKE, p=FAKE, w_s=FAKE, y=FAKE, ws=FAKE, ws_bytes=512):
    return lib.moe_weighted_sum(rows, T, n, k, shared, inv, p, w_s, y, ws, ws_bytes, None)


def weighted_grad(lib, dy=FAKE, rows=FAKE, T=0, n=64, k=2, shared=1, inv=FAKE, p=FAKE, w_s=FAKE, drows=FAKE, dp=FAKE, dws=FAKE, ws=FAKE,
                  ws_bytes=512):
    return lib.moe_weighted_sum_grad(dy, rows, T, n, k, shared, inv, p, w_s, drows, dp, dws, ws, ws_bytes, None)


COMMON = [({}, OK), (dict(n=1 << 20), OK), (dict(k=16), OK), (dict(inv=None), OK), (dict(T=-1), INVALID), (dict(T=65537), INVALID),
          (dict(n=0), INVALID), (dict(k=0), INVALID), (dict(shared=2), INVALID), (dict(k=17), UNSUPPORTED), (dict(n=12), UNSUPPORTED),
          (dict(n=(1 << 20) + 8), UNSUPPORTED), (dict(T=1, inv=None), INVALID), (dict(inv=FAKE + 2), INVALID), (dict(ws=None), INVALID),
          (dict(ws=ODD), INVALID), (dict(ws_bytes=511), WS)]


@pytest.mark.parametrize("call", [dispatch, weighted, weighted_grad])
@pytest.mark.parametrize("kw,expect", COMMON)
def test_routed_arguments(lib, call, kw, expect):
    assert call(lib, **kw) == expect


@pytest.mark.parametrize("call,kw", [
    (dispatch, dict(T=1, x=None)), (dispatch, dict(T=1, y=ODD)),
    (weighted, dict(T=1, rows=None)), (weighted, dict(T=1, y=None)), (weighted, dict(p=ODD)), (weighted, dict(w_s=ODD)),
    (weighted, dict(T=1, w_s=None)), (weighted, dict(T=1, p=None)), (weighted, dict(T=1, shared=0)),
    (weighted_grad, dict(T=1, dy=None)), (weighted_grad, dict(T=1, p=None)), (weighted_grad, dict(T=1, drows=None)),
    (weighted_grad, dict(T=1, w_s=None)), (weighted_grad, dict(T=1, shared=0, dws=None)), (weighted_grad, dict(shared=0, w_s=None)),
    (weighted_grad, dict(T=1, rows=None)), (weighted_grad, dict(T=1, rows=None, dp=None)), (weighted_grad, dict(dp=ODD)),
    (weighted_grad, dict(dws=ODD)), (weighted_grad, dict(rows=ODD)),
])
def test_routed_refusals(lib, call, kw):
    assert call(lib, **kw) == INVALID


def norm(lib, x=FAKE, residual=FAKE, gate=FAKE, shape=3, act=1, scale=0.5, post=1, w_post=FAKE, w_pre=FAKE, off=0.0, eps=1e-6, T=0, n=64,
         s=FAKE, y=FAKE):
    return lib.moe_gated_norm(x, residual, gate, shape, act, scale, post, w_post, w_pre, off, eps, T, n, s, y, None)


def norm_grad(lib, x=FAKE, s=FAKE, gate=FAKE, shape=3, act=1, scale=0.5, post=1, w_post=FAKE, w_pre=FAKE, off=0.0, eps=1e-6, T=0, n=64,
              dy=FAKE, ds=FAKE, dx=FAKE, dres=FAKE + 64, dgate=None, dpost=None, dpre=None, ws=FAKE, ws_bytes=1 << 20):
    return lib.moe_gated_norm_grad(x, s, gate, shape, act, scale, post, w_post, w_pre, off, eps, T, n, dy, ds, dx, dres, dgate, dpost, dpre,
                                   ws, ws_bytes, None)


@pytest.mark.parametrize("call", [norm, norm_grad])
@pytest.mark.parametrize("kw,expect", [
    ({}, OK), (dict(shape=0, act=0, gate=None), OK), (dict(shape=1, act=4), OK), (dict(shape=2, act=0), OK), (dict(n=8192), OK), (dict(n=8), OK),
    (dict(x=None, gate=None), OK), (dict(post=0, w_post=None), OK), (dict(w_post=None, w_pre=None), OK), (dict(eps=0.0), OK),
    (dict(T=-1), INVALID), (dict(n=0), INVALID), (dict(T=(1 << 24) + 1), INVALID), (dict(eps=-1e-6), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(post=2), INVALID), (dict(shape=4), INVALID), (dict(shape=-1), INVALID),
    (dict(shape=0), INVALID), (dict(shape=0, gate=None), INVALID),                 # no gate, but a gate or a function
    (dict(post=0), INVALID),                                                        # a weight of no norm
    (dict(shape=2, gate=None), INVALID), (dict(T=2, gate=None), INVALID), (dict(T=2, x=None), INVALID), (dict(x=ODD), INVALID),
    (dict(w_post=ODD), INVALID), (dict(w_pre=ODD), INVALID), (dict(gate=ODD, T=2), INVALID),
    (dict(act=2), UNSUPPORTED), (dict(act=3), UNSUPPORTED), (dict(n=12), UNSUPPORTED), (dict(n=8200), UNSUPPORTED),
])
def test_norm_arguments(lib, call, kw, expect):
    assert call(lib, **kw) == expect


@pytest.mark.parametrize("call,kw,expect", [
    (norm, dict(residual=ODD), INVALID), (norm, dict(s=ODD), INVALID), (norm, dict(y=ODD), INVALID), (norm, dict(s=None, y=None), OK),
    (norm_grad, dict(T=2, s=None), INVALID), (norm_grad, dict(T=2, dx=None), INVALID), (norm_grad, dict(dy=ODD), INVALID),
    (norm_grad, dict(ds=ODD), INVALID), (norm_grad, dict(dres=ODD), INVALID), (norm_grad, dict(dgate=ODD), INVALID),
    (norm_grad, dict(dpost=ODD), INVALID), (norm_grad, dict(dpre=ODD), INVALID), (norm_grad, dict(T=2, dy=None, ds=None), INVALID),
    (norm_grad, dict(T=2, dy=None, dpre=FAKE), INVALID), (norm_grad, dict(T=2, dres=FAKE), INVALID),
    (norm_grad, dict(shape=0, act=0, gate=None, dgate=FAKE), INVALID), (norm_grad, dict(post=0, w_post=None, dpost=FAKE), INVALID),
    (norm_grad, dict(ws=None), INVALID), (norm_grad, dict(ws=ODD), INVALID), (norm_grad, dict(ws_bytes=511), WS),
    (norm_grad, dict(T=100, ws_bytes=512 + 100 * 3 * 64 * 4 - 1), WS),
])
def test_norm_refusals(lib, call, kw, expect):
    assert call(lib, **kw) == expect


def test_norm_workspace(lib):
    size = ctypes.c_size_t(0)
    call = lambda T, n: lib.moe_gated_norm_workspace_size(T, n, ctypes.byref(size))
    assert call(0, 64) == OK and size.value >= qm.MOE_SCALED_WS_BYTES
    assert call(100, 64) == OK and size.value == 512 + 100 * 3 * 64 * 4
    assert call(1 << 24, 8192) == OK and size.value < 64 << 20
    assert call(-1, 64) == INVALID and call(1, 0) == INVALID and call(1, 12) == UNSUPPORTED and call(1, 8200) == UNSUPPORTED
    assert lib.moe_gated_norm_workspace_size(1, 64, None) == INVALID
