"""Products of few block-scaled rows, which run a row at a time: sizes on both sides of every choice that the launch makes,
against 64 bits with the tolerances of the other products."""
import numpy as np
import pytest
import torch

import quantised_moe_expert_gb300 as qm

from . import scaled_ref as S
from . import test_gpu_scaled as T
from .test_gpu_scaled import M4, M8, NV, Out, gpu, grouped, operand, product_error, weights, workspace

pytestmark = pytest.mark.gpu

SIZES = {
    "one": [1], "two": [2], "five": [5], "apart": [1] * 9, "holes": [0, 0, 1, 0, 3, 0, 0, 0, 2, 0],
}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


@pytest.mark.parametrize("fmt,K", [(NV, 320), (NV, 512), (NV, 576), (NV, 1024), (NV, 1088), (NV, 2112), (NV, 8256),
                                   (M8, 384), (M8, 512), (M8, 896), (M8, 1152), (M8, 2176), (M8, 4224)])
@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("N", [8, 40, 136])
def test_gemm_few(monkeypatch, fmt, K, sizes, N):
    monkeypatch.setitem(T.GROUPS, "few", SIZES[sizes])
    T.test_gemm(fmt, "few", N, K)


@pytest.mark.parametrize("fmt", [NV, M8])
@pytest.mark.parametrize("K", [384, 1152])
def test_gemm_few_many_groups(monkeypatch, fmt, K):
    monkeypatch.setitem(T.GROUPS, "few", [0] * 300 + [1] + [0] * 600 + [2, 1] + [0] * 100)
    T.test_gemm(fmt, "few", 8, K)


@pytest.mark.parametrize("fmt", [NV, M8])
@pytest.mark.parametrize("R,G,N", [(1, 1, 4864), (1, 1, 4872), (1, 1, 10240), (1, 1, 10248), (2, 1, 5120), (3, 1, 3416), (10, 10, 2048),
                                   (10, 10, 2056), (1, 3, 20480), (10, 10, 4096), (10, 10, 4104)])
@pytest.mark.parametrize("K", [384, 640, 1152])
def test_gemm_around_the_limits(fmt, R, G, N, K):
    """A CTA for every SM and more; as many outputs as run a row at a time and a few more."""
    rng = np.random.default_rng(N + K)
    off = [min(g, R) for g in range(G)]
    a, av = operand(rng, fmt, R, K, off)
    w, wv, alpha = weights(rng, fmt, G, N, K)
    want, mag = grouped(av, wv, off, alpha)
    y, ws = Out((R, N), torch.float32), workspace()
    qm.moe_scaled_gemm(fmt, a, w, R, N, K, G, gpu(np.array(off, np.int32)) if G > 1 else None, y.t, ws)
    assert qm.moe_get_device_status(ws) == 0
    assert (np.abs(y.check() - want) <= product_error(K) * mag).all()


@pytest.mark.parametrize("fmt,K", [(NV, 320), (NV, 512), (NV, 960), (NV, 2112), (NV, 6144), (M8, 384), (M8, 1024), (M8, 2176)])
@pytest.mark.parametrize("sizes", ["one", "two", "apart", "holes"])
@pytest.mark.parametrize("inter", [128, 640])
def test_swiglu_few(monkeypatch, fmt, K, sizes, inter):
    monkeypatch.setitem(T.GROUPS, "few", SIZES[sizes])
    T.test_swiglu(fmt, "few", inter, K)


@pytest.mark.parametrize("fmt,K", [(NV, 3840), (M8, 2176)])
@pytest.mark.parametrize("sizes", [[32], [29, 3]])
def test_swiglu_long_sums(monkeypatch, fmt, K, sizes):
    """Too many rows for a row at a time, few enough to share the K steps between two CTAs."""
    monkeypatch.setitem(T.GROUPS, "few", sizes)
    T.test_swiglu(fmt, "few", 512, K)


@pytest.mark.parametrize("fmt,K", [(NV, 3648), (NV, 6208), (M8, 1920), (M8, 3200)])
@pytest.mark.parametrize("sizes", [[33], [64], [60, 4], [301], [130, 0, 3]])
def test_long_sums_of_more_rows(monkeypatch, fmt, K, sizes):
    """K steps shared by two CTAs for every number of rows in a tile, and groups of several tiles."""
    monkeypatch.setitem(T.GROUPS, "few", sizes)
    T.test_gemm(fmt, "few", 328, K)
    if K > 3648 or fmt == M8:
        T.test_swiglu(fmt, "few", 256, K)


@pytest.mark.parametrize("fmt", [NV, M8])
def test_few_rows_before_the_first_group(fmt):
    """Rows before the first group belong to none and are left as they are."""
    rng = np.random.default_rng(5)
    R, N, K = 4, 72, 640
    a, av = operand(rng, fmt, R, K, [0, 1, 1])
    w, wv, alpha = weights(rng, fmt, 3, N, K)
    want, mag = grouped(av, wv, [0, 1, 1], alpha)
    pad = lambda t: None if t is None else torch.cat([t[:2], t])                                       # noqa: E731
    codes, scales, factors = (list(a.tensors) + [None])[:3]
    a = qm.scaled_rows(pad(codes), scales, pad(factors))
    y, ws = torch.full((R + 2, N), 7.0, device="cuda"), workspace()
    qm.moe_scaled_gemm(fmt, a, w, R + 2, N, K, 3, gpu(np.array([2, 3, 3], np.int32)), y, ws)
    assert qm.moe_get_device_status(ws) == 0
    got = y.cpu().numpy().astype(np.float64)
    assert (got[:2] == 7).all() and (np.abs(got[2:] - want) <= product_error(K) * mag).all()


@pytest.mark.parametrize("off", [[0, 5, 4], [-3, 2, 4], [0, 2, 900], [0, 0, 7]])
@pytest.mark.parametrize("K", [512, 2048])
def test_few_rows_report_bad_offsets(off, K):
    rng = np.random.default_rng(3)
    R, N, G = 6, 64, 3
    a, _ = operand(rng, NV, R, K, [0, 2, 4])
    w, _, _ = weights(rng, NV, G, N, K)
    y, ws = torch.full((R, N), 7.0, device="cuda"), workspace()
    qm.moe_scaled_gemm(NV, a, w, R, N, K, G, gpu(np.array(off, np.int32)), y, ws)
    assert qm.moe_get_device_status(ws) == qm.MOE_ERR_DEVICE
    assert (y == 7).all()


@pytest.mark.parametrize("fmt", [NV, M8])
@pytest.mark.parametrize("K", [384, 2176])
def test_few_rows_nan_stay_apart(fmt, K):
    """A NaN scale reaches its own row (or, in a weight, its own column) and no other."""
    rng = np.random.default_rng(3)
    R, N = 4, 64
    a, _ = operand(rng, fmt, R, K, [0])
    w, _, _ = weights(rng, fmt, 1, N, K)
    w.alpha = None
    nan = 0x7F if fmt == NV else 0xFF
    a.tensors[1][int(S.scale_index(fmt, K, [2])[0, 3])] = nan
    w.tensors[1][int(S.scale_index(NV if fmt == NV else M4, K, [50])[0, 1])] = nan
    y, ws = Out((R, N), torch.float32), workspace()
    qm.moe_scaled_gemm(fmt, a, w, R, N, K, 1, None, y.t, ws)
    got = np.isnan(y.check())
    assert got[2].all() and got[:, 50].all() and got.sum() == N + R - 1


def test_few_rows_extreme_scales():
    """Power-of-two scales whose product is moderate although either alone would leave fp32's range with the sums."""
    R, N, K = 2, 32, 512
    rng = np.random.default_rng(11)
    ac, wc = rng.integers(0, 126, (R, K)).astype(np.uint8), rng.integers(0, 16, (N, K)).astype(np.uint8)
    sa, sw = np.full((R, K // 32), 247, np.uint8), np.full((N, K // 32), 7, np.uint8)       # 2^120, 2^-120
    a = qm.scaled_rows(gpu(S.pack(M8, ac)), gpu(S.tile(M8, sa, S.scale_rows([0], R), R // 128 + 1, 0xFF)), None)
    w = qm.scaled_mat(gpu(S.pack(M4, wc).reshape(1, N, -1)), gpu(S.weight_tiles(M4, sw.reshape(1, N, -1))), None)
    av, wv = S.dequantise(M8, ac, sa, None), S.dequantise(M4, wc, sw, None)
    want, mag = av @ wv.T, np.abs(av) @ np.abs(wv).T
    y, ws = Out((R, N), torch.float32), workspace()
    qm.moe_scaled_gemm(M8, a, w, R, N, K, 1, None, y.t, ws)
    assert (np.abs(y.check() - want) <= product_error(K) * mag).all()


def test_few_rows_weights_past_32_bits():
    """Weights and their scales beyond 2^32 bytes, by the last of many groups."""
    G, N, K = 40, 16384, 16384
    gen = torch.Generator(device="cuda").manual_seed(1)
    wc = torch.randint(0, 256, (G, N, K // 2), dtype=torch.uint8, device="cuda", generator=gen)
    wsc = torch.randint(0x30, 0x40, (G * (N // 128) * (K // 64) * 512,), dtype=torch.uint8, device="cuda", generator=gen)
    ac = torch.randint(0, 256, (1, K // 2), dtype=torch.uint8, device="cuda", generator=gen)
    asc = torch.randint(0x30, 0x40, (G * (K // 64) * 512,), dtype=torch.uint8, device="cuda", generator=gen)
    y, ws = torch.empty((1, N), device="cuda"), workspace()
    qm.moe_scaled_gemm(NV, qm.scaled_rows(ac, asc), qm.scaled_mat(wc, wsc), 1, N, K, G, gpu(np.zeros(G, np.int32)), y, ws)
    assert qm.moe_get_device_status(ws) == 0
    cols = np.array([0, 127, 128, 8191, N - 1])
    sr = np.array([(G - 1) * 128])
    av = S.dequantise(NV, S.unpack(NV, ac.cpu().numpy()), asc[gpu(S.scale_index(NV, K, sr).reshape(-1))].cpu().numpy().reshape(1, -1))
    wr = (G - 1) * N + cols
    wv = S.dequantise(NV, S.unpack(NV, wc[G - 1][cols].cpu().numpy()), wsc[gpu(S.scale_index(NV, K, wr).reshape(-1))].cpu().numpy().reshape(len(cols), -1))
    want, mag = av @ wv.T, np.abs(av) @ np.abs(wv).T
    assert (np.abs(y[:, cols].cpu().numpy() - want) <= product_error(K) * mag).all()


@pytest.mark.parametrize("ea,ew,small", [(120, 20, False), (127, 127, False), (10, 118, False), (120, 8, True), (64, 64, True), (-127, -24, False),
                                         (-100, -45, False), (-127, 127, False), (127, -127, True)])
def test_few_rows_scales_past_fp32(ea, ew, small):
    """Power-of-two scales whose product leaves fp32's range although the sums stay within it: blocks of zero codes give zero,
    small codes (or the smallest sums) their value, but for the rounding of subnormal
    sums, one step of 2^-149 a block."""
    R, N, K = 2, 40, 512
    rng = np.random.default_rng(abs(ea + ew))
    ac, wc = np.zeros((R, K), np.uint8), rng.integers(0, 16, (N, K)).astype(np.uint8)
    if small:
        ac[:, 64:96] = rng.integers(0, 3, (R, 32)) + 128 * rng.integers(0, 2, (R, 32))          # 0, 2^-9, 2^-8 and their negatives
    elif ea + ew < 100:
        ac[:] = rng.integers(0, 127, (R, K))
    sa, sw = np.full((R, K // 32), ea + 127, np.uint8), np.full((N, K // 32), ew + 127, np.uint8)
    a = qm.scaled_rows(gpu(S.pack(M8, ac)), gpu(S.tile(M8, sa, S.scale_rows([0], R), R // 128 + 1, 0xFF)), None)
    w = qm.scaled_mat(gpu(S.pack(M4, wc).reshape(1, N, -1)), gpu(S.weight_tiles(M4, sw.reshape(1, N, -1))), None)
    av, wv = S.dequantise(M8, ac, sa, None), S.dequantise(M4, wc, sw, None)
    want, mag = av @ wv.T, np.abs(av) @ np.abs(wv).T
    assert mag.max() < 3e38 and (mag.max() > 0) == bool(ac.any())
    y, ws = Out((R, N), torch.float32), workspace()
    qm.moe_scaled_gemm(M8, a, w, R, N, K, 1, None, y.t, ws)
    assert (np.abs(y.check() - want) <= product_error(K) * mag + K // 32 * 2.0 ** -149).all()


@pytest.mark.parametrize("fmt,K", [(NV, 64), (NV, 128), (NV, 192), (NV, 256), (M8, 128), (M8, 256)])
@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("N", [8, 136, 2056])
def test_gemm_few_of_a_single_step(monkeypatch, fmt, K, sizes, N):
    """Sums that one step of a tile would hold, and steps that end inside a warp's."""
    monkeypatch.setitem(T.GROUPS, "few", SIZES[sizes])
    T.test_gemm(fmt, "few", N, K)


@pytest.mark.parametrize("fmt,K", [(NV, 64), (NV, 256), (M8, 128), (M8, 256)])
@pytest.mark.parametrize("R,G,N", [(1, 1, 10240), (1, 1, 10248), (20, 1, 512), (20, 1, 520), (40, 33, 1024), (40, 33, 1032)])
def test_single_steps_around_the_limits(fmt, K, R, G, N):
    """As many outputs as run a row at a time and a few more."""
    test_gemm_around_the_limits(fmt, R, G, N, K)


@pytest.mark.parametrize("fmt", [NV, M8])
@pytest.mark.parametrize("sizes", ["one", "apart", "holes"])
@pytest.mark.parametrize("inter", [128, 640])
def test_swiglu_few_of_a_single_step(monkeypatch, fmt, sizes, inter):
    monkeypatch.setitem(T.GROUPS, "few", SIZES[sizes])
    for K in (128, 256):
        T.test_swiglu(fmt, "few", inter, K)


@pytest.mark.parametrize("fmt,K", [(NV, 64), (NV, 256), (M8, 128)])
@pytest.mark.parametrize("R,G,N", [(20, 33, 2048), (20, 33, 2056), (20, 19, 1024), (20, 19, 1032), (640, 3, 32), (640, 3, 40)])
def test_single_steps_of_more_and_fewer_groups_than_rows(fmt, K, R, G, N):
    """The limit is another where rows must share groups."""
    test_gemm_around_the_limits(fmt, R, G, N, K)
