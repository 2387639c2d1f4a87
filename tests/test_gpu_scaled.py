"""GPU checks of the block-scaled operators against plain implementations in 64 bits.

Tolerances (set before any run):
  quantisation  scale bytes, factors and codes equal the definition's, bit for bit
  norm          bf16 outputs within half a bf16 step (2^-9 of the value; 2^-8 allows for a power of two between)
                and 2^-20 of it for the fp32 steps; codes within half an E4M3 or E2M1 step and the same 2^-20
  products      every instruction adds a block of products to an fp32 accumulator and may drop what is below its
                last bit once more on aligning them: (2 K / 32 + 4) 2^-23 of sum |a w|, plus the output's rounding
  SwiGLU        that error through silu(g) u (|silu'| <= 1.1), plus half a step of the code
"""
import numpy as np
import pytest
import torch

import quantised_moe_expert_gb300 as qm

from . import scaled_ref as S

pytestmark = pytest.mark.gpu

NV, M8, M4 = S.NV, S.M8, S.M4
GUARD = 4096


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    qm.load()


def gpu(a):
    a = np.ascontiguousarray(a)
    return torch.tensor(a.view(np.int16) if a.dtype == np.uint16 else a).cuda()


class Out:
    """A device buffer of `shape` between two guard regions, which check() reads back unchanged."""

    def __init__(self, shape, dtype):
        n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
        self.raw = torch.full((GUARD + (n + 15) // 16 * 16 + GUARD,), 0xA5, dtype=torch.uint8, device="cuda")
        self.n, self.t = n, self.raw[GUARD:GUARD + n].view(dtype).view(shape)

    def check(self):
        raw = self.raw.cpu().numpy()
        assert (raw[:GUARD] == 0xA5).all() and (raw[GUARD + self.n:] == 0xA5).all(), "write outside the output"
        return self.t.float().cpu().numpy() if self.t.dtype == torch.bfloat16 else self.t.cpu().numpy()


class Rows:
    """Room for R block-scaled rows of n elements in `groups` groups, guarded."""

    def __init__(self, fmt, R, n, groups=1, factors=True):
        self.fmt, self.R, self.n = fmt, R, n
        self.codes = Out((R, n if fmt == M8 else n // 2), torch.uint8)
        self.scales = Out(((R // 128 + groups) * S.col_tiles(fmt, n) * 512,), torch.uint8)
        self.factor = Out((R,), torch.float32) if fmt == NV and factors else None
        self.c = qm.scaled_rows(self.codes.t, self.scales.t, None if self.factor is None else self.factor.t)

    def read(self, srows=None):
        """Codes [R, n], scale bytes [R, n / block], factors."""
        srows = np.arange(self.R) if srows is None else srows
        return (S.unpack(self.fmt, self.codes.check()), self.scales.check()[S.scale_index(self.fmt, self.n, srows)],
                None if self.factor is None else self.factor.check())


def workspace():
    return torch.zeros(512, dtype=torch.uint8, device="cuda")


def random_rows(rng, T, n, wide=False):
    x = rng.standard_normal((T, n)) * np.exp(0.5 * rng.standard_normal((T, 1)))
    if wide:
        x *= np.exp2(rng.integers(-40, 40, (T, n // 16)).repeat(16, axis=1))
    return S.bf16(x)


def bits(x):
    return (x.view(np.uint32) >> 16).astype(np.uint16)


# ---------------------------------------------------------------- quantisation

@pytest.mark.parametrize("fmt", [NV, M8, M4])
@pytest.mark.parametrize("T,n", [(1, 32), (1, 2048), (3, 96), (5, 8192), (127, 160), (129, 1056), (300, 2048), (700, 1344), (2, 16384)])
@pytest.mark.parametrize("f32", [0, 1])
def test_quantize(fmt, T, n, f32):
    rng = np.random.default_rng(T * n + fmt)
    x = random_rows(rng, T, n, wide=True)
    if f32:
        x = (x * (1 + rng.random((T, n), np.float32) * 2 ** -8)).astype(np.float32)
    x[T // 2, :n // 2] = 0
    x[0] = 0 if T > 2 else x[0]                                    # a row of zeros
    q = Rows(fmt, T, n)
    qm.moe_quantize(fmt, gpu(x) if f32 else gpu(bits(x)), T, n, 1, None, q.c)
    codes, scales, g = q.read()
    want_c, want_s, want_g = S.quantise(fmt, x)
    assert np.array_equal(scales, want_s)
    if fmt == NV:
        assert np.array_equal(g, want_g)
    zero = S.decode(fmt, want_c) == 0
    assert np.array_equal(codes[~zero], want_c[~zero])
    assert (S.decode(fmt, codes[zero]) == 0).all()


@pytest.mark.parametrize("fmt", [NV, M4])
@pytest.mark.parametrize("G,N,n", [(3, 40, 64), (2, 128, 256), (5, 136, 128)])
def test_quantize_weight_stack(fmt, G, N, n):
    """Groups start at a row tile of their own; NVFP4 with a given factor per matrix."""
    rng = np.random.default_rng(G * N)
    w = S.bf16(rng.standard_normal((G * N, n)))
    g = (np.abs(w).reshape(G, -1).max(1) / 2688 * np.array([1, 4, .25, 1, 2])[:G]).astype(np.float32)
    codes = Out((G * N, n // 2), torch.uint8)
    scales = Out((G * -(-N // 128) * S.col_tiles(fmt, n) * 512,), torch.uint8)
    qm.moe_quantize(fmt, gpu(bits(w)), G * N, n, G, gpu(g) if fmt == NV else None, qm.scaled_rows(codes.t, scales.t))
    want_c, want_s, _ = S.quantise(fmt, w, g.repeat(N) if fmt == NV else None)
    assert np.array_equal(S.unpack(fmt, codes.check()), want_c)
    rows = (np.arange(G)[:, None] * -(-N // 128) * 128 + np.arange(N)[None]).reshape(-1)
    assert np.array_equal(scales.check()[S.scale_index(fmt, n, rows)], want_s)


@pytest.mark.parametrize("fmt", [NV, M8, M4])
def test_quantize_nonfinite(fmt):
    """A non-finite element makes its block's scale NaN (NVFP4 rows with their own factor: the whole row)."""
    x = S.bf16(np.random.default_rng(0).standard_normal((4, 128)))
    x[1, 37], x[2, 5], x[3, 127] = np.inf, np.nan, -np.inf
    q = Rows(fmt, 4, 128)
    qm.moe_quantize(fmt, gpu(bits(x)), 4, 128, 1, None, q.c)
    codes, scales, g = q.read()
    v = S.dequantise(fmt, codes, scales, g)
    assert np.isfinite(v[0]).all()
    for r, j in ((1, 37), (2, 5), (3, 127)):
        b = j // S.block(fmt)
        blocks = np.isnan(v[r]).reshape(-1, S.block(fmt))
        assert blocks[b].all()
        assert blocks.all() if fmt == NV else blocks.sum() == S.block(fmt)


@pytest.mark.parametrize("fmt", [NV, M8])
@pytest.mark.parametrize("T,n,E,k,shared", [(1, 256, 16, 2, 1), (16, 2048, 256, 8, 1), (150, 160, 8, 3, 0), (600, 512, 64, 16, 1),
                                            (130, 64, 1, 1, 0), (5, 9216, 16, 2, 1)])
def test_quantize_routed(fmt, T, n, E, k, shared):
    rng = np.random.default_rng(T + n)
    x = random_rows(rng, T, n)
    ids = np.stack([rng.permutation(max(E, k))[:k] % E for _ in range(T)]).astype(np.int32) if E > 1 else np.zeros((T, k), np.int32)
    ids[rng.random(ids.shape) < 0.3] = E - 1                       # a crowded expert (a pick may repeat)
    flat = ids.reshape(-1)
    perm = np.argsort(flat, kind="stable")
    inv = np.empty(T * k, np.int32)
    inv[perm] = np.arange(T * k)
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat, minlength=E))]).astype(np.int32)
    R, G = T * (k + shared), E + shared
    q, ws = Rows(fmt, R, n, G), workspace()
    qm.moe_quantize_routed(fmt, gpu(bits(x)), T, n, k, E, shared, gpu(ids), gpu(inv), gpu(offsets), q.c, ws)
    assert qm.moe_get_device_status(ws) == 0
    srows = S.scale_rows(list(offsets[:G]), R)
    codes, scales, g = q.read(srows)
    token = np.concatenate([perm // k, np.arange(T)[:T * shared]])
    want_c, want_s, want_g = S.quantise(fmt, x[token])
    assert np.array_equal(scales, want_s) and np.array_equal(S.decode(fmt, codes), S.decode(fmt, want_c))
    if fmt == NV:
        assert np.array_equal(g, want_g)


def test_quantize_routed_reports_bad_routing():
    T, n, E, k = 4, 128, 8, 2
    x = gpu(bits(random_rows(np.random.default_rng(0), T, n)))
    good = dict(ids=np.arange(8, dtype=np.int32).reshape(4, 2), inv=np.arange(8, dtype=np.int32), off=np.arange(9, dtype=np.int32))
    for key, at, v in (("ids", (1, 1), 8), ("ids", (0, 0), -1), ("inv", 3, 8), ("inv", 3, -5), ("off", 5, 7), ("off", 2, -1)):
        a = {m: t.copy() for m, t in good.items()}
        a[key][at] = v
        q, ws = Rows(M8, T * k, n, E), workspace()
        qm.moe_quantize_routed(M8, x, T, n, k, E, 0, gpu(a["ids"]), gpu(a["inv"]), gpu(a["off"]), q.c, ws)
        assert qm.moe_get_device_status(ws) == qm.MOE_ERR_DEVICE, (key, at)
        q.codes.check(), q.scales.check()


@pytest.mark.parametrize("fmt,G,N,n", [(NV, 3, 200, 192), (M4, 2, 64, 160), (M8, 1, 129, 32)])
def test_tile_scales(fmt, G, N, n):
    s = np.random.default_rng(1).integers(0, 256, (G, N, n // S.block(fmt)), dtype=np.uint8)
    out = Out((G * -(-N // 128) * S.col_tiles(fmt, n) * 512,), torch.uint8)
    qm.moe_tile_scales(fmt, gpu(s), G, N, n, out.t)
    assert np.array_equal(out.check(), S.weight_tiles(fmt, s))


# ---------------------------------------------------------------- norm

def norm_ref(x, r, w, off, eps):
    s = S.bf16(x if r is None else x + r).astype(np.float64)
    y = s / np.sqrt((s * s).mean(1, keepdims=True) + eps)
    return s, y if w is None else y * (off + w.astype(np.float64))


def half_step(fmt, v, unit):
    """Half the distance between neighbouring codes at v (in units of the scale), an upper bound."""
    a = np.abs(v) / unit
    if fmt == M8:
        return unit * np.maximum(2.0 ** -10, np.exp2(np.floor(np.log2(np.maximum(a, 1e-30))) - 4)) * (1 + 1e-9)
    return unit * np.where(a < 2, 0.25, np.where(a < 4, 0.5, 1.0)) * (1 + 1e-9)


def check_codes(fmt, codes, scales, g, y, slack):
    """Each block's scale is the one for y (or for a y within slack of it), each code's value a nearest one.
    `slack`: how far the kernel's fp32 y may be from the fp64 y."""
    R, n = y.shape
    blk = S.block(fmt)
    amax, sl = np.abs(y).reshape(R, -1, blk).max(2), np.broadcast_to(slack, y.shape).reshape(R, -1, blk).max(2)
    if fmt == NV:
        lim = amax / g.astype(np.float64)[:, None] / 6
        e = sl / g.astype(np.float64)[:, None] / 6 + lim * 2.0 ** -21
        lo, hi = S.E4M3[S.nearest(S.E4M3, np.maximum(lim - e, 0))], S.E4M3[S.nearest(S.E4M3, lim + e)]
        sv = S.scale_value(NV, scales)
        assert ((sv >= lo) & (sv <= hi)).all()
        unit = np.repeat(sv * g.astype(np.float64)[:, None], blk, 1)
        clip = 6.0
    else:
        top = 448.0 if fmt == M8 else 6.0
        unit = S.scale_value(fmt, scales)
        assert (amax - sl <= top * unit).all() and ((amax + sl > top * unit / 2) | (scales == 0)).all()
        unit, clip = np.repeat(unit, blk, 1), top
    v = S.decode(fmt, codes) * unit
    inside = np.clip(y, -clip * unit, clip * unit)
    assert (np.abs(v - inside) <= np.where(unit > 0, half_step(fmt, inside, np.maximum(unit, 1e-300)), np.inf) + slack).all()
    assert (v[unit == 0] == 0).all()


@pytest.mark.parametrize("fmt", [0, NV, M8])
@pytest.mark.parametrize("T,n", [(1, 2048), (1, 32), (2, 96), (7, 5120), (129, 1024), (300, 1056), (513, 2048), (600, 1696), (3, 16384)])
def test_norm(fmt, T, n):
    rng = np.random.default_rng(T * n + fmt)
    x, r = random_rows(rng, T, n), S.bf16(3 * random_rows(rng, T, n))
    w = S.bf16(1 + 0.3 * rng.standard_normal(n))
    if T > 2:
        x[1] = r[1] = 0                                            # a row of zeros
    q = Rows(fmt, T, n) if fmt else None
    so, yo = Out((T, n), torch.bfloat16), Out((T, n), torch.bfloat16)
    qm.moe_add_rmsnorm(gpu(bits(x)), gpu(bits(r)), gpu(bits(w)), 0.0, 1e-6, T, n, so.t, yo.t, fmt, q.c if q else None)
    s, y = norm_ref(x, r, w, 0.0, 1e-6)
    assert np.array_equal(so.check(), s)
    assert (np.abs(yo.check() - y) <= (2.0 ** -8 + 2.0 ** -20) * np.abs(y)).all()
    if fmt:
        codes, scales, g = q.read()
        if fmt == NV:
            assert (np.abs(g - np.maximum(np.abs(y).max(1) / 2688, 2.0 ** -110)) <= 2.0 ** -20 * g).all()
        check_codes(fmt, codes, scales, g, y, 2.0 ** -20 * np.abs(y))


def test_norm_options():
    """No residual, no weight, weight_offset, in-place sums, only codes."""
    rng = np.random.default_rng(5)
    T, n = 37, 1280
    x, r, w = random_rows(rng, T, n), random_rows(rng, T, n), S.bf16(0.2 * rng.standard_normal(n))
    for res, wt, off in ((None, w, 1.0), (r, None, 0.0), (r, w, 1.0), (None, None, 0.0)):
        yo = Out((T, n), torch.bfloat16)
        qm.moe_add_rmsnorm(gpu(bits(x)), None if res is None else gpu(bits(res)), None if wt is None else gpu(bits(wt)), off, 1e-5,
                           T, n, None, yo.t, 0, None)
        _, y = norm_ref(x, res, wt, off, 1e-5)
        assert (np.abs(yo.check() - y) <= (2.0 ** -8 + 2.0 ** -20) * np.abs(y)).all()
    s, y = norm_ref(x, r, w, 0.0, 1e-5)
    outs = []
    for which in ("x", "residual"):
        dx, dr, q = gpu(bits(x)), gpu(bits(r)), Rows(M8, T, n)
        qm.moe_add_rmsnorm(dx, dr, gpu(bits(w)), 0.0, 1e-5, T, n, dx if which == "x" else dr, None, M8, q.c)
        got = (dx if which == "x" else dr).view(torch.bfloat16).float().cpu().numpy()
        assert np.array_equal(got, s)
        outs.append(q.read())
    assert np.array_equal(outs[0][0], outs[1][0]) and np.array_equal(outs[0][1], outs[1][1])
    check_codes(M8, *outs[0], y, 2.0 ** -20 * np.abs(y))


def test_norm_nonfinite_rows_stay_apart():
    x = random_rows(np.random.default_rng(2), 5, 256)
    x[1, 3], x[3, 200] = np.nan, np.inf
    q, yo = Rows(NV, 5, 256), Out((5, 256), torch.bfloat16)
    qm.moe_add_rmsnorm(gpu(bits(x)), None, None, 0.0, 1e-6, 5, 256, None, yo.t, NV, q.c)
    y = yo.check()
    codes, scales, g = q.read()
    v = S.dequantise(NV, codes, scales, g)
    for r in range(5):
        if r in (1, 3):
            assert not np.isfinite(y[r]).all() and np.isnan(v[r]).any()
        else:
            assert np.isfinite(y[r]).all() and np.isfinite(v[r]).all()


# ---------------------------------------------------------------- products

def weights(rng, fmt, G, N, K):
    """A stack of G matrices: device tensors and fp64 values [G, N, K] (factors apart)."""
    wf = NV if fmt == NV else M4
    codes = rng.integers(0, 16, (G, N, K), dtype=np.uint8)
    s = rng.integers(1, 0x7F, (G, N, K // S.block(wf)), dtype=np.uint8) if wf == NV else \
        rng.integers(110, 140, (G, N, K // S.block(wf)), dtype=np.uint8)
    if wf == NV:
        s[rng.random(s.shape) < 0.05] = 0
    alpha = rng.uniform(.5, 2, G).astype(np.float32) / np.float32(64)
    dev = qm.scaled_mat(gpu(S.pack(wf, codes)), gpu(S.weight_tiles(wf, s, fill=0xFF if wf == M4 else 0x7F)), gpu(alpha))
    return dev, S.dequantise(wf, codes, s), alpha


def operand(rng, fmt, R, K, offsets):
    """Activation rows with arbitrary codes and scales: device rows and fp64 values."""
    G = len(offsets)
    codes = rng.integers(0, 16, (R, K), dtype=np.uint8)
    if fmt == M8:
        codes = rng.integers(0, 256, (R, K), dtype=np.uint8)
        codes[(codes & 127) == 127] = 0
    s = rng.integers(1, 0x7F, (R, K // S.block(fmt)), dtype=np.uint8) if fmt == NV else \
        rng.integers(112, 136, (R, K // S.block(fmt)), dtype=np.uint8)
    g = rng.uniform(.5, 2, R).astype(np.float32) if fmt == NV else None
    # unused scale rows hold NaN: they must not reach any output
    tiles = S.tile(fmt, s, S.scale_rows(offsets, R), R // 128 + G, fill=0x7F if fmt == NV else 0xFF)
    dev = qm.scaled_rows(gpu(S.pack(fmt, codes)), gpu(tiles), None if g is None else gpu(g))
    return dev, S.dequantise(fmt, codes, s, g)


def bounds_of(offsets, R):
    return list(zip(offsets, list(offsets[1:]) + [R]))


def grouped(a, w, offsets, alpha):
    """fp64 product and sum of magnitudes, group by group."""
    y, m = np.zeros((a.shape[0], w.shape[1])), np.zeros((a.shape[0], w.shape[1]))
    for g, (lo, hi) in enumerate(bounds_of(offsets, a.shape[0])):
        y[lo:hi] = a[lo:hi] @ w[g].T * float(alpha[g])
        m[lo:hi] = np.abs(a[lo:hi]) @ np.abs(w[g]).T * float(alpha[g])
    return y, m


def product_error(K):
    return (2 * K / 32 + 4) * 2.0 ** -23


GROUPS = {                                                          # group sizes
    "one_row": [1], "full_tile": [128], "over_a_tile": [129], "two_tiles": [256], "ragged": [300],
    "empty_groups": [0, 5, 0, 0, 130, 1, 0], "small": [1, 2, 3, 31, 32, 33, 64, 96, 97], "many": [3] * 70 + [0] * 30 + [140],
}


@pytest.mark.parametrize("fmt", [NV, M8])
@pytest.mark.parametrize("groups", GROUPS)
@pytest.mark.parametrize("N,K", [(8, 128), (72, 384), (136, 640), (520, 256)])
def test_gemm(fmt, groups, N, K):
    sizes = GROUPS[groups]
    G, R = len(sizes), sum(sizes)
    offsets = np.concatenate([[0], np.cumsum(sizes)[:-1]]).astype(np.int32)
    rng = np.random.default_rng(N * K + R + fmt)
    a, av = operand(rng, fmt, R, K, list(offsets))
    w, wv, alpha = weights(rng, fmt, G, N, K)
    want, mag = grouped(av, wv, list(offsets), alpha)
    for dt in (torch.float32, torch.bfloat16):
        y, ws = Out((R, N), dt), workspace()
        qm.moe_scaled_gemm(fmt, a, w, R, N, K, G, gpu(offsets) if G > 1 else None, y.t, ws)
        assert qm.moe_get_device_status(ws) == 0
        tol = product_error(K) * mag + (2.0 ** -8 * np.abs(want) if dt == torch.bfloat16 else 0)
        got = y.check()
        assert (np.abs(got - want) <= tol).all(), np.abs((got - want) / np.maximum(tol, 1e-300)).max()


@pytest.mark.parametrize("fmt,K", [(NV, 64), (NV, 192), (NV, 320), (NV, 2112), (M8, 128), (M8, 2176), (NV, 8192), (M8, 4096)])
@pytest.mark.parametrize("R,N", [(1, 4096), (17, 200), (200, 2000)])
def test_gemm_depths(fmt, K, R, N):
    """K steps that end inside a tile, long sums, and the launch shapes for few and many tiles."""
    rng = np.random.default_rng(K + R)
    a, av = operand(rng, fmt, R, K, [0])
    w, wv, alpha = weights(rng, fmt, 1, N, K)
    want, mag = grouped(av, wv, [0], alpha)
    y, ws = Out((R, N), torch.float32), workspace()
    qm.moe_scaled_gemm(fmt, a, w, R, N, K, 1, None, y.t, ws)
    assert qm.moe_get_device_status(ws) == 0
    assert (np.abs(y.check() - want) <= product_error(K) * mag).all()


@pytest.mark.parametrize("fmt,K", [(NV, 3584), (NV, 3776), (NV, 12288), (M8, 1792), (M8, 4224)])
@pytest.mark.parametrize("sizes,N", [([1], 72), ([32], 1000), ([3, 0, 1, 7, 0], 264), ([31, 1], 64)])
def test_gemm_few_rows_long_sums(fmt, K, sizes, N):
    """Few rows and many K steps (the launch shape that halves them), both output types; the same bits every time."""
    rng = np.random.default_rng(K + N)
    G, R = len(sizes), sum(sizes)
    offsets = np.concatenate([[0], np.cumsum(sizes)[:-1]]).astype(np.int32)
    a, av = operand(rng, fmt, R, K, list(offsets))
    w, wv, alpha = weights(rng, fmt, G, N, K)
    want, mag = grouped(av, wv, list(offsets), alpha)
    for dt in (torch.float32, torch.bfloat16):
        y, ws = Out((R, N), dt), workspace()
        first = None
        for _ in range(3):
            qm.moe_scaled_gemm(fmt, a, w, R, N, K, G, gpu(offsets) if G > 1 else None, y.t, ws)
            first = y.t.clone() if first is None else first
            assert torch.equal(first, y.t)
        assert qm.moe_get_device_status(ws) == 0
        tol = product_error(K) * mag + (2.0 ** -8 * np.abs(want) if dt == torch.bfloat16 else 0)
        assert (np.abs(y.check() - want) <= tol).all()


@pytest.mark.parametrize("fmt", [NV, M8])
def test_gemm_many_tiles(fmt):
    """More tiles than SMs, several row tiles a group: spot rows and columns."""
    rng = np.random.default_rng(8)
    offsets, R, N, K = [0, 700, 701], 2300, 3000, 256
    a, av = operand(rng, fmt, R, K, offsets)
    w, wv, alpha = weights(rng, fmt, 3, N, K)
    want, mag = grouped(av, wv, offsets, alpha)
    y, ws = Out((R, N), torch.float32), workspace()
    for _ in range(2):
        qm.moe_scaled_gemm(fmt, a, w, R, N, K, 3, gpu(np.array(offsets, np.int32)), y.t, ws)
    assert qm.moe_get_device_status(ws) == 0
    first = y.check()
    assert (np.abs(first - want) <= product_error(K) * mag).all()


@pytest.mark.parametrize("fmt,K", [(NV, 2112), (M8, 1408), (NV, 4416), (M8, 2304)])
@pytest.mark.parametrize("offsets", [None, [0, 0, 257, 1500]])
def test_gemm_large_groups(fmt, K, offsets):
    """Groups of many row tiles (the launch shape for them), rows and outputs that end inside a tile."""
    rng = np.random.default_rng(K)
    off = offsets or [0]
    R, N, G = 3001, 2008, len(off)
    a, av = operand(rng, fmt, R, K, off)
    w, wv, alpha = weights(rng, fmt, G, N, K)
    want, mag = grouped(av, wv, off, alpha)
    for dt in (torch.bfloat16, torch.float32):
        y, ws = Out((R, N), dt), workspace()
        qm.moe_scaled_gemm(fmt, a, w, R, N, K, G, None if offsets is None else gpu(np.array(off, np.int32)), y.t, ws)
        assert qm.moe_get_device_status(ws) == 0
        tol = product_error(K) * mag + (2.0 ** -8 * np.abs(want) if dt == torch.bfloat16 else 0)
        assert (np.abs(y.check() - want) <= tol).all()


@pytest.mark.parametrize("fmt", [NV, M8])
def test_gemm_nan_rows_stay_apart(fmt):
    """A NaN scale reaches its own row (or, in a weight, its own column) and no other."""
    rng = np.random.default_rng(3)
    R, N, K = 40, 64, 256
    a, av = operand(rng, fmt, R, K, [0])
    w, wv, _ = weights(rng, fmt, 1, N, K)
    w.alpha = None
    a.tensors[1][int(S.scale_index(fmt, K, [7])[0, 3])] = 0x7F if fmt == NV else 0xFF
    wf = NV if fmt == NV else M4
    w.tensors[1][int(S.scale_index(wf, K, [50])[0, 1])] = 0x7F if fmt == NV else 0xFF
    y, ws = Out((R, N), torch.float32), workspace()
    qm.moe_scaled_gemm(fmt, a, w, R, N, K, 1, None, y.t, ws)
    nan = np.isnan(y.check())
    assert nan[7].all() and nan[:, 50].all() and nan.sum() == N + R - 1


@pytest.mark.parametrize("off", [[0, 50, 40], [-3, 20, 40], [0, 20, 900]])
def test_gemm_reports_bad_offsets(off):
    rng = np.random.default_rng(3)
    R, N, K, G = 64, 64, 128, 3
    a, _ = operand(rng, NV, R, K, [0, 20, 40])
    w, _, _ = weights(rng, NV, G, N, K)
    y, ws = Out((R, N), torch.bfloat16), workspace()
    qm.moe_scaled_gemm(NV, a, w, R, N, K, G, gpu(np.array(off, np.int32)), y.t, ws)
    assert qm.moe_get_device_status(ws) == qm.MOE_ERR_DEVICE
    y.check()


@pytest.mark.parametrize("fmt", [NV, M8])
@pytest.mark.parametrize("groups", ["one_row", "over_a_tile", "empty_groups", "small", "many"])
@pytest.mark.parametrize("inter,K", [(128, 256), (384, 128), (256, 640), (128, 3840)])
def test_swiglu(fmt, groups, inter, K):
    inter = inter + 64 if fmt == NV else inter
    sizes = GROUPS[groups]
    G, R = len(sizes), sum(sizes)
    offsets = np.concatenate([[0], np.cumsum(sizes)[:-1]]).astype(np.int32)
    rng = np.random.default_rng(inter * K + R + fmt)
    # operands of ordinary size: gate and up products of order one
    x = random_rows(rng, R, K)
    c, s, g = S.quantise(fmt, x)
    a = qm.scaled_rows(gpu(S.pack(fmt, c)), gpu(S.tile(fmt, s, S.scale_rows(list(offsets), R), R // 128 + G, 0x7F if fmt == NV else 0xFF)),
                       None if g is None else gpu(g))
    av = S.dequantise(fmt, c, s, g)
    wf = NV if fmt == NV else M4
    mats, vals = [], []
    for _ in range(2):
        v = (rng.standard_normal((G * inter, K)) / np.sqrt(K)).astype(np.float32)
        f = np.float32(np.abs(v).max() / 2688)
        c, s, _ = S.quantise(wf, v, f if wf == NV else None)
        s = s.reshape(G, inter, -1)
        alpha = np.full(G, f if wf == NV else 1, np.float32)
        mats.append(qm.scaled_mat(gpu(S.pack(wf, c).reshape(G, inter, -1)), gpu(S.weight_tiles(wf, s)), gpu(alpha)))
        vals.append((S.dequantise(wf, c.reshape(G, inter, K), s), alpha))
    gate, gm = grouped(av, vals[0][0], list(offsets), vals[0][1])
    up, um = grouped(av, vals[1][0], list(offsets), vals[1][1])
    h = S.silu(gate) * up
    err = product_error(K) * (1.1 * gm * np.abs(up) + um * np.abs(S.silu(gate))) + 2.0 ** -18 * np.abs(h) * (1 + np.abs(gate))
    hs = np.full(G, 1 / 256, np.float32)
    q, ws = Rows(fmt, R, inter, G, factors=False), workspace()
    qm.moe_scaled_swiglu(fmt, a, mats[0], mats[1], R, inter, K, G, gpu(offsets) if G > 1 else None, gpu(hs) if fmt == NV else None,
                         q.c, ws)
    assert qm.moe_get_device_status(ws) == 0
    codes, scales, _ = q.read(S.scale_rows(list(offsets), R))
    check_codes(fmt, codes, scales, np.full(R, 1 / 256, np.float32) if fmt == NV else None, h, err)


@pytest.mark.parametrize("fmt", [NV, M8])
def test_swiglu_zero_and_large_gates(fmt):
    """Rows of zeros give zeros; gates far below zero give zeros, not NaN."""
    R, inter, K = 3, 128, 128
    x = np.zeros((R, K), np.float32)
    x[1], x[2] = 100, -100
    c, s, g = S.quantise(fmt, x)
    a = qm.scaled_rows(gpu(S.pack(fmt, c)), gpu(S.tile(fmt, s, np.arange(R), 1)), None if g is None else gpu(g))
    wf = NV if fmt == NV else M4
    c, s, _ = S.quantise(wf, np.full((inter, K), 1.0, np.float32), np.float32(1 / 2688) if wf == NV else None)
    one = qm.scaled_mat(gpu(S.pack(wf, c)), gpu(S.weight_tiles(wf, s[None])), gpu(np.full(1, 1 / 2688 if wf == NV else 1, np.float32)))
    q, ws = Rows(fmt, R, inter, 1, factors=False), workspace()
    # h of row 1 is the square of 12800, which the scale has to hold
    qm.moe_scaled_swiglu(fmt, a, one, one, R, inter, K, 1, None, gpu(np.full(1, 2.0 ** 28 / 2688, np.float32)) if fmt == NV else None, q.c, ws)
    codes, scales, _ = q.read()
    v = S.dequantise(fmt, codes, scales, np.full(R, 2.0 ** 28 / 2688) if fmt == NV else None)
    assert (v[0] == 0).all() and (v[2] == 0).all()
    assert (np.abs(v[1] - 12800.0 ** 2) <= 12800.0 ** 2 / 8).all()


def test_products_on_another_stream_and_graph():
    """The operators run on the stream they are given, and replay from a graph."""
    rng = np.random.default_rng(11)
    T, K, N = 9, 512, 256
    x = random_rows(rng, T, K)
    w, wv, alpha = weights(rng, NV, 1, N, K)
    dx, q, ws = gpu(bits(x)), Rows(NV, T, K), workspace()
    y = Out((T, N), torch.float32)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    qm.moe_quantize(NV, dx, T, K, 1, None, q.c, stream=side)
    qm.moe_scaled_gemm(NV, q.c, w, T, N, K, 1, None, y.t, ws, stream=side)
    side.synchronize()
    first = y.check().copy()
    c, s, g = S.quantise(NV, x)
    want, mag = grouped(S.dequantise(NV, c, s, g), wv, [0], alpha)
    assert (np.abs(first - want) <= product_error(K) * mag).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qm.moe_quantize(NV, dx, T, K, 1, None, q.c)
        qm.moe_scaled_gemm(NV, q.c, w, T, N, K, 1, None, y.t, ws)
    x2 = random_rows(rng, T, K)
    dx.copy_(gpu(bits(x2)))
    graph.replay()
    torch.cuda.synchronize()
    c, s, g = S.quantise(NV, x2)
    want, mag = grouped(S.dequantise(NV, c, s, g), wv, [0], alpha)
    got = y.check()
    assert (np.abs(got - want) <= product_error(K) * mag).all() and not np.array_equal(got, first)


def test_gemm_offsets_past_32_bits():
    """Code and output offsets beyond 2^32 bytes and 2^31 elements."""
    G, N, K, R = 70, 65536, 2048, 40000
    sizes = np.zeros(G, np.int64)
    sizes[0], sizes[-1] = R - 300, 300
    offsets = np.concatenate([[0], np.cumsum(sizes)[:-1]]).astype(np.int32)
    gen = torch.Generator(device="cuda").manual_seed(1)
    wc = torch.randint(0, 256, (G, N, K // 2), dtype=torch.uint8, device="cuda", generator=gen)
    wsc = torch.randint(0x30, 0x40, (G * (N // 128) * (K // 64) * 512,), dtype=torch.uint8, device="cuda", generator=gen)
    ac = torch.randint(0, 256, (R, K // 2), dtype=torch.uint8, device="cuda", generator=gen)
    asc = torch.randint(0x30, 0x40, ((R // 128 + G) * (K // 64) * 512,), dtype=torch.uint8, device="cuda", generator=gen)
    y = torch.empty((R, N), dtype=torch.bfloat16, device="cuda")
    ws = workspace()
    qm.moe_scaled_gemm(NV, qm.scaled_rows(ac, asc), qm.scaled_mat(wc, wsc), R, N, K, G, gpu(offsets), y, ws)
    assert qm.moe_get_device_status(ws) == 0
    cols = np.array([0, 127, 128, 255, 256, 40000, N - 1])
    for rows, g in ((np.array([0, 128, 20001, R - 301]), 0), (np.array([R - 300, R - 1]), G - 1)):
        lo = int(offsets[g])
        sr = (lo // 128 + g) * 128 + rows - lo
        av = S.dequantise(NV, S.unpack(NV, ac[rows].cpu().numpy()), asc[gpu(S.scale_index(NV, K, sr).reshape(-1))].cpu().numpy().reshape(len(rows), -1))
        wr = g * N + cols
        wv = S.dequantise(NV, S.unpack(NV, wc[g][cols].cpu().numpy()), wsc[gpu(S.scale_index(NV, K, wr).reshape(-1))].cpu().numpy().reshape(len(cols), -1))
        want, mag = av @ wv.T, np.abs(av) @ np.abs(wv).T
        got = y[rows][:, cols].float().cpu().numpy()
        assert (np.abs(got - want) <= product_error(K) * mag + 2.0 ** -8 * np.abs(want)).all()


@pytest.mark.parametrize("T,G,n", [(2, 2, 16400), (3, 1, 20496), (260, 2, 24592), (1, 1, 65536)])
@pytest.mark.parametrize("f32", [0, 1])
def test_quantize_long_rows_with_a_given_factor(T, G, n, f32):
    """NVFP4 rows longer than a block of threads holds, as a product's K or a weight matrix may be."""
    rng = np.random.default_rng(n + T)
    x = random_rows(rng, T, n, wide=False)
    if f32:
        x = (x * (1 + rng.random((T, n), np.float32) * 2 ** -8)).astype(np.float32)
    x[0, n // 2:n // 2 + 32] = 0
    g = (np.abs(x).reshape(G, -1).max(1) / 2688 * np.array([1, 3])[:G]).astype(np.float32)
    codes = Out((T, n // 2), torch.uint8)
    scales = Out((G * -(-(T // G) // 128) * S.col_tiles(NV, n) * 512,), torch.uint8)
    qm.moe_quantize(NV, gpu(x) if f32 else gpu(bits(x)), T, n, G, gpu(g), qm.scaled_rows(codes.t, scales.t))
    want_c, want_s, _ = S.quantise(NV, x, g.repeat(T // G))
    r = np.arange(T)
    srows = r // (T // G) * -(-(T // G) // 128) * 128 + r % (T // G)
    assert np.array_equal(scales.check()[S.scale_index(NV, n, srows)], want_s)
    got = S.unpack(NV, codes.check())
    zero = S.decode(NV, want_c) == 0
    assert np.array_equal(got[~zero], want_c[~zero]) and (S.decode(NV, got[zero]) == 0).all()


@pytest.mark.parametrize("T,n,E,k,shared", [(1, 16416, 8, 2, 1), (7, 20480, 16, 3, 0), (40, 32768, 8, 2, 1)])
def test_quantize_routed_long_rows(T, n, E, k, shared):
    """MXFP8 rows of more than one panel, each of them into all of the row's copies."""
    test_quantize_routed(M8, T, n, E, k, shared)
