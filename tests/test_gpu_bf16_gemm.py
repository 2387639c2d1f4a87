"""Grouped products of 16-bit rows and their gradients against their definition in 64 bits."""
import pytest
import torch

import quantised_moe_expert_gb300 as qm
from tests.bf16_ref import BF16, FUNCTION, SLOPE, act, bf16, groups, offsets_of, outer, product, within

pytestmark = pytest.mark.gpu

ACTS = {"none": qm.MOE_ACT_NONE, "silu": qm.MOE_ACT_SILU, "gelu": qm.MOE_ACT_GELU, "relu": qm.MOE_ACT_RELU}
MARK = -7.0                                            # what rows of no group keep


@pytest.fixture()
def ws():
    w = torch.zeros(qm.MOE_SCALED_WS_BYTES, dtype=torch.uint8, device="cuda")
    yield w
    assert qm.moe_get_device_status(w) == 0


def marked(*shape, dtype=torch.bfloat16):
    return torch.full(shape, MARK, dtype=dtype, device="cuda")


def round_tol(v):
    return BF16 * v.abs()


def sum_tol(K, s):
    return K * 2.0 ** -23 * s


# sizes on both sides of every tile edge; one row to many; groups without rows, with one, with several tiles
SIZES = [
    ([1], 8, 8), ([1], 4096, 2048), ([2], 72, 520), ([5], 64, 64), ([7], 264, 72), ([9], 2048, 512), ([16], 1000, 200), ([33], 256, 128),
    ([64], 512, 256), ([129], 136, 328), ([301], 1000, 2184), ([700], 520, 136), ([1500], 768, 192),
    ([0, 3, 0, 130, 1, 0], 200, 136), ([1, 1, 1, 1], 512, 2048), ([40, 0, 0, 257], 72, 64), ([0, 0, 5], 8, 1032),
    ([128, 128, 64], 256, 320), ([300, 500, 1, 700], 512, 264),
    # widths of whole blocks of 64: a tile that ends inside the blocks of a copy
    ([50], 64, 64), ([300], 320, 128), ([90, 200], 192, 200), ([20, 700], 576, 192),
    # a tile's steps shared out to 2, 4 and 8 CTAs, of one group and of several
    ([12], 1000, 520), ([140], 520, 1032), ([20], 264, 1096), ([9, 0, 14], 136, 1032), ([30, 90], 1000, 456),
    # pairs of CTAs: row tiles of 256, whole and partial
    ([6660], 2312, 136), ([2560], 2048, 2056), ([1500, 1, 0, 3300, 1557, 900], 2312, 72), ([20000], 520, 72),
]


def case(counts, N, K, transposed=False, pairs=1, first=0, seed=0):
    """Rows of the groups and one more at the front for each of `first`."""
    offsets, R = offsets_of(counts, first=first)
    shape = (len(counts), K, N) if transposed else (len(counts), N, K)
    a = [bf16(R, K, seed=seed + i) for i in range(pairs)]
    w = [bf16(*shape, seed=seed + 10 + i, size=K ** -0.5) for i in range(pairs)]
    y = s = 0
    for i in range(pairs):
        d = product(a[i], w[i], counts, first, transposed)
        y, s = y + d[0], s + d[1]
    return a, w, offsets if len(counts) > 1 or first else None, R, y, s


@pytest.mark.parametrize("transposed", [0, 1])
@pytest.mark.parametrize("counts,N,K", SIZES)
def test_product(ws, counts, N, K, transposed):
    (a,), (w,), offsets, R, want, s = case(counts, N, K, bool(transposed))
    y, y32 = marked(R + 3, N), marked(R + 3, N, dtype=torch.float32)
    for out in (y, y32):
        qm.moe_gemm(a, w, None, None, transposed, R, N, K, len(counts), offsets, None, 0, None, None, out[:R], ws)
    within(y32[:R], want, sum_tol(K, s))
    within(y[:R], want, round_tol(want) + 2 * sum_tol(K, s))
    assert bool((y[R:] == MARK).all()) and bool((y32[R:] == MARK).all())


@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("counts,N,K", [([1], 264, 136), ([3], 1024, 512), ([301], 1000, 200), ([20, 0, 150], 136, 72), ([2, 0, 1], 512, 512),
                                        ([20], 264, 1096), ([100, 0, 30], 136, 1032), ([300], 1000, 584)])
def test_epilogue(ws, counts, N, K, name):
    """Bias, activation and residual, with and without the product before the activation; the residual in place."""
    (a,), (w,), offsets, R, want, s = case(counts, N, K, seed=3)
    bias, res = bf16(len(counts), N, seed=30), bf16(R, N, seed=31, size=2.0)
    pre = want.clone()
    for g, r in groups(counts):
        pre[r] += bias[g].double()
    value = act(name, pre)[0]
    tol = sum_tol(K + 1, s + pre.abs())
    out_tol = SLOPE * tol + FUNCTION * pre.abs()
    y, p, inplace = marked(R, N), marked(R, N), res.clone()
    call = lambda residual, pre_out, y: qm.moe_gemm(a, w, None, None, 0, R, N, K, len(counts), offsets, bias, ACTS[name], residual,
                                                    pre_out, y, ws)
    call(res, p, y)
    call(inplace, None, inplace)
    within(p, pre, round_tol(pre) + 2 * tol)
    within(y, value + res.double(), round_tol(value + res.double()) + 2 * out_tol + 2.0 ** -23 * res.double().abs())
    assert torch.equal(y, inplace)
    y32 = marked(R, N, dtype=torch.float32)
    call(None, None, y32)
    within(y32, value, out_tol)
    # the parts one by one
    qm.moe_gemm(a, w, None, None, 0, R, N, K, len(counts), offsets, None, 0, res, None, y, ws)
    within(y, want + res.double(), round_tol(want + res.double()) + 2 * tol + 2.0 ** -23 * res.double().abs())


@pytest.mark.parametrize("transposed", [0, 1])
@pytest.mark.parametrize("counts,N,K", [([1], 512, 264), ([150], 264, 72), ([60, 0, 200, 1], 128, 136), ([600], 768, 512),
                                        ([6700], 2312, 72), ([2900, 3900], 2312, 136), ([2600], 2048, 1032), ([20], 264, 584)])
def test_two_pairs(ws, counts, N, K, transposed):
    """The sum of two products, rounded once."""
    a, w, offsets, R, want, s = case(counts, N, K, bool(transposed), pairs=2, seed=5)
    y = marked(R, N)
    qm.moe_gemm(a[0], w[0], a[1], w[1], transposed, R, N, K, len(counts), offsets, None, 0, None, None, y, ws)
    within(y, want, round_tol(want) + 2 * sum_tol(2 * K, s))


@pytest.mark.parametrize("name,biased", [("silu", False), ("gelu", True), ("none", True), ("relu", False)])
@pytest.mark.parametrize("counts,I,K", [([1], 512, 2048), ([4], 264, 136), ([200], 136, 72), ([0, 3, 0, 130, 1, 0], 200, 136),
                                        ([1] * 9, 512, 512), ([300, 280], 264, 520),
                                        ([6570], 1160, 72), ([3000, 0, 5, 3900], 1168, 136),
                                        ([20], 136, 1096), ([30, 0, 110], 264, 584), ([200], 520, 456)])
def test_gated_pair(ws, counts, I, K, name, biased):
    offsets, R = offsets_of(counts)
    G = len(counts)
    a, gate, up = bf16(R, K, seed=1), bf16(G, I, K, seed=2, size=K ** -0.5), bf16(G, I, K, seed=3, size=K ** -0.5)
    bias = [bf16(G, I, seed=4 + i) if biased else None for i in range(2)]
    v, tol = [], []
    for m, b in ((gate, bias[0]), (up, bias[1])):
        p, s = product(a, m, counts)
        if biased:
            for g, r in groups(counts):
                p[r] += b[g].double()
        v.append(p)
        tol.append(sum_tol(K + 1, s + p.abs()))
    f = act(name, v[0])[0]
    want = f * v[1]
    out_tol = (SLOPE * tol[0] + FUNCTION * v[0].abs()) * (v[1].abs() + tol[1]) + f.abs() * tol[1]
    h, h2, g_out, u_out = (marked(R + 1, I) for _ in range(4))
    call = lambda g, u, out: qm.moe_gemm_glu(a, gate, up, bias[0], bias[1], ACTS[name], R, I, K, G, offsets if G > 1 else None, g, u,
                                             out[:R], ws)
    call(None, None, h)
    call(g_out[:R], u_out[:R], h2)
    assert torch.equal(h, h2)
    within(h[:R], want, round_tol(want) + 2 * out_tol)
    within(g_out[:R], v[0], round_tol(v[0]) + 2 * tol[0])
    within(u_out[:R], v[1], round_tol(v[1]) + 2 * tol[1])
    for t in (h, g_out, u_out):
        assert bool((t[R:] == MARK).all())


WSIZES = [([1], 8, 8), ([1], 264, 72), ([15], 64, 64), ([64], 128, 256), ([100], 136, 328), ([700], 520, 264), ([0, 3, 0, 130, 1, 0], 200, 136),
          ([17, 16, 1, 64, 65, 128], 256, 512), ([300, 0, 500], 72, 1032), ([2] * 40, 64, 136), ([2000], 384, 256),
          # one group of many rows among many of few: its tiles first
          ([2000] + [3] * 100, 264, 264), ([3] * 60 + [2000] + [5] * 40, 264, 264), ([70] * 100 + [3000], 264, 264), ([0] * 500 + [900] + [1] * 9, 72, 136),
          # widths of whole blocks of 64
          ([90, 0, 200, 3], 192, 320), ([70], 448, 64), ([20, 700], 200, 576), ([300] * 5, 64, 192),
          # a tile's steps shared out
          ([2000], 64, 72), ([700, 0, 900, 40], 72, 136), ([530], 264, 328), ([1, 515, 510], 200, 264), ([500, 3, 0], 520, 200),
          # pairs of CTAs
          ([400], 2048, 2560), ([448], 2056, 2632), ([516, 0, 1777, 1, 900], 1000, 1288), ([15 * 64 + 9, 300, 15 * 64], 1288, 1544)]


@pytest.mark.parametrize("counts,N,K", WSIZES)
def test_weight_gradient(ws, counts, N, K):
    offsets, R = offsets_of(counts)
    G = len(counts)
    dy, x = bf16(R, N, seed=7), bf16(R, K, seed=8)
    w, s, b, t = outer(dy, x, counts)
    n = max(counts)
    for dtype in (torch.bfloat16, torch.float32):
        dw, db = marked(G + 1, N, K, dtype=dtype), marked(G + 1, N, dtype=dtype)
        qm.moe_gemm_wgrad(dy, x, R, N, K, G, offsets if G > 1 else None, 0, dw[:G], db[:G], ws)
        step = BF16 if dtype == torch.bfloat16 else 0.0
        within(dw[:G], w, step * w.abs() + 2 * sum_tol(n, s))
        within(db[:G], b, step * b.abs() + 2 * sum_tol(n, t))
        assert bool((dw[G:] == MARK).all()) and bool((db[G:] == MARK).all())
        only = torch.zeros_like(dw[:G])
        qm.moe_gemm_wgrad(dy, x, R, N, K, G, offsets if G > 1 else None, 0, only, None, ws)
        assert torch.equal(only, dw[:G])
    # added to what is there
    base, bbase = torch.randn(G, N, K, device="cuda"), torch.randn(G, N, device="cuda")
    dw, db = base.clone(), bbase.clone()
    qm.moe_gemm_wgrad(dy, x, R, N, K, G, offsets if G > 1 else None, 1, dw, db, ws)
    within(dw, base.double() + w, 2 * sum_tol(n, s) + 2.0 ** -23 * (base.double() + w).abs())
    within(db, bbase.double() + b, 2 * sum_tol(n, t) + 2.0 ** -23 * (bbase.double() + b).abs())


def test_weight_gradient_without_rows(ws):
    G, N, K = 3, 24, 40
    none = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    offsets = torch.zeros(G, dtype=torch.int32, device="cuda")
    dw, db = marked(G, N, K), marked(G, N)
    qm.moe_gemm_wgrad(none, none, 0, N, K, G, offsets, 0, dw, db, ws)
    assert bool((dw == 0).all()) and bool((db == 0).all())
    dw, db = marked(G, N, K, dtype=torch.float32), marked(G, N, dtype=torch.float32)
    qm.moe_gemm_wgrad(none, none, 0, N, K, G, offsets, 1, dw, db, ws)
    assert bool((dw == MARK).all()) and bool((db == MARK).all())
    y = marked(1, N)
    qm.moe_gemm(none, bf16(G, N, K), None, None, 0, 0, N, K, G, offsets, None, 0, None, None, y, ws)
    assert bool((y == MARK).all())


@pytest.mark.parametrize("counts,N,K", [([3, 4], 136, 72), ([100, 300], 136, 72), ([0, 600], 136, 72), ([3000, 3700], 2312, 72),
                                        ([300, 700], 2056, 1288)])
def test_rows_of_no_group(ws, counts, N, K):
    """Rows before the first group: not written, and what they hold (NaN) reaches nothing."""
    first = 5
    offsets, R = offsets_of(counts, first=first)
    a, w = bf16(R, K, seed=1), bf16(2, N, K, seed=2, size=K ** -0.5)
    a[:first] = float("nan")
    want, s = product(a, w, counts, first)
    y = marked(R, N)
    qm.moe_gemm(a, w, None, None, 0, R, N, K, 2, offsets, None, 0, None, None, y, ws)
    assert bool((y[:first] == MARK).all())
    within(y[first:], want[first:], round_tol(want[first:]) + 2 * sum_tol(K, s[first:]))
    dy = bf16(R, N, seed=3)
    dy[:first] = float("inf")
    d, t, _, _ = outer(dy[first:], a[first:], counts)
    dw = marked(2, N, K, dtype=torch.float32)
    qm.moe_gemm_wgrad(dy, a, R, N, K, 2, offsets, 0, dw, None, ws)
    within(dw, d, 2 * sum_tol(max(counts), t))


@pytest.mark.parametrize("transposed", [0, 1])
@pytest.mark.parametrize("counts,N,K", [([1, 2, 1], 136, 72), ([70, 30, 90], 136, 72), ([260, 300, 10], 136, 72),
                                        ([9, 20, 12], 136, 1096), ([300, 700, 90], 72, 136),
                                        ([2290, 2300, 1300], 2568, 72), ([900, 300, 99], 1288, 1288)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_non_finite_values_stay_apart(ws, counts, N, K, transposed, bad):
    """A group whose rows and matrix hold no finite value next to groups that do: tiles, panels and steps end inside one."""
    offsets, R = offsets_of(counts)
    a, w = bf16(R, K, seed=1), bf16(3, *((K, N) if transposed else (N, K)), seed=2, size=K ** -0.5)
    rows = list(groups(counts))
    a[rows[1][1]] = bad
    w[1] = bad
    want, s = product(a, w, counts, transposed=bool(transposed))
    y = marked(R, N)
    qm.moe_gemm(a, w, None, None, transposed, R, N, K, 3, offsets, None, 0, None, None, y, ws)
    for g in (0, 2):
        r = rows[g][1]
        within(y[r], want[r], round_tol(want[r]) + 2 * sum_tol(K, s[r]))
    assert not bool(y[rows[1][1]].isfinite().any())
    dy = bf16(R, N, seed=3)
    dy[rows[1][1]] = bad
    d, t, b, u = outer(dy, a, counts)
    dw, db = marked(3, N, K, dtype=torch.float32), marked(3, N, dtype=torch.float32)
    qm.moe_gemm_wgrad(dy, a, R, N, K, 3, offsets, 0, dw, db, ws)
    for g in (0, 2):
        within(dw[g], d[g], 2 * sum_tol(max(counts), t[g]))
        within(db[g], b[g], 2 * sum_tol(max(counts), u[g]))
    assert not bool(dw[1].isfinite().any()) and not bool(db[1].isfinite().any())


@pytest.mark.parametrize("bad_offsets", [[0, 9, 4], [0, 4, 99], [-1, 3, 4], [1 << 30, 2, 3]])
@pytest.mark.parametrize("R,N,K", [(6, 72, 64), (30, 72, 1032), (700, 72, 64), (2600, 2048, 2048)])
def test_malformed_offsets_are_reported(bad_offsets, R, N, K):
    w = torch.zeros(512, dtype=torch.uint8, device="cuda")
    bad_offsets = [o if o != 9 else R - 1 for o in bad_offsets] if R > 10 else bad_offsets
    bad_offsets = [o if o != 99 else R + 1 for o in bad_offsets]
    offsets = torch.tensor(bad_offsets, dtype=torch.int32, device="cuda")
    a, m = bf16(R, K), bf16(3, N, K)
    y, dw, db = marked(R, N), marked(3, N, K), marked(3, N)
    calls = [lambda: qm.moe_gemm(a, m, None, None, 0, R, N, K, 3, offsets, None, 0, None, None, y, w),
             lambda: qm.moe_gemm(a, m.view(3, K, N), None, None, 1, R, N, K, 3, offsets, None, 0, None, None, y, w),
             lambda: qm.moe_gemm_glu(a, m, m, None, None, 1, R, N, K, 3, offsets, None, None, y, w),
             lambda: qm.moe_gemm_wgrad(y, a, R, N, K, 3, offsets, 0, dw, db, w)]
    for call in calls:
        call()
        assert qm.moe_get_device_status(w) == qm.MOE_ERR_DEVICE
        for t in (y, dw, db):
            assert bool((t == MARK).all())


def test_same_call_same_bits(ws):
    counts, N, K = [50, 300, 2], 520, 264
    offsets, R = offsets_of(counts)
    a, w, dy = bf16(R, K, seed=1), bf16(3, N, K, seed=2), bf16(R, N, seed=3)
    outs = []
    for _ in range(3):
        y, dw, db = marked(R, N), marked(3, N, K), marked(3, N)
        qm.moe_gemm(a, w, None, None, 0, R, N, K, 3, offsets, None, 0, None, None, y, ws)
        qm.moe_gemm_wgrad(dy, a, R, N, K, 3, offsets, 0, dw, db, ws)
        outs.append((y, dw, db))
    for o in outs[1:]:
        assert all(torch.equal(p, q) for p, q in zip(o, outs[0]))


@pytest.mark.parametrize("terms,N,K", [(500, 200, 136), (4096, 1000, 72), (8192, 64, 72), (5000, 2056, 2632), (4100, 264, 1032)])
def test_fp32_sums(ws, terms, N, K):
    """Long sums in fp32: the error in the 2-norm stays that of sums of 768 terms.  An addition is truncated by at most 2^-23 of the
    sum so far, half of that in the mean, and the sums so far are half of the last one in the mean: 768 / 4 times 2^-23 of a sum, if all point
    one way; the sums of 768 are then rounded as they are added."""
    dy, x = bf16(terms, N, seed=1), bf16(terms, K, seed=2)
    want = dy.double().t() @ x.double()
    dw, y = marked(1, N, K, dtype=torch.float32), marked(N, K, dtype=torch.float32)
    qm.moe_gemm_wgrad(dy, x, terms, N, K, 1, None, 0, dw, None, ws)
    outs = [dw[0]]
    if terms % 8 == 0:
        qm.moe_gemm(dy.t().contiguous(), x, None, None, 1, N, K, terms, 1, None, None, 0, None, None, y, ws)
        outs.append(y)
    most = min(terms, 768) / 4 * 2.0 ** -23 + (terms / 768) ** 0.5 * 2.0 ** -24
    for got in outs:
        assert float((got.double() - want).norm() / want.norm()) < most


def test_past_32_bits(ws):
    """Outputs of more than 2^31 elements: the last rows, columns and matrices are where they belong (exact: small whole numbers)."""
    R, N, K = (1 << 17) + 3, 16392, 8
    a = torch.zeros(R, K, dtype=torch.bfloat16, device="cuda")
    a[:, 0] = (torch.arange(R, device="cuda") % 251).bfloat16()
    w = torch.zeros(1, N, K, dtype=torch.bfloat16, device="cuda")
    w[0, :, 0] = (torch.arange(N, device="cuda") % 5 - 2).bfloat16()
    y = torch.empty(R, N, dtype=torch.bfloat16, device="cuda")
    assert y.numel() > 1 << 31
    want = lambda r: (a[r, 0].float()[:, None] * w[0, :, 0].float()).bfloat16()
    for transposed in (0, 1):
        y.fill_(MARK)
        qm.moe_gemm(a, w.transpose(1, 2).contiguous() if transposed else w, None, None, transposed, R, N, K, 1, None, None, 0, None, None, y, ws)
        for r in (slice(0, 5), slice(R // 2, R // 2 + 5), slice(R - 200, R)):
            assert torch.equal(y[r], want(r))
    d = torch.empty(R, N, dtype=torch.bfloat16, device="cuda")
    qm.moe_act_grad(qm.MOE_ACT_NONE, y, y, None, R, N, d, None)
    assert torch.equal(d[-200:], y[-200:])
    del d
    # gradients of many matrices
    G, N, K = 520, 2048, 2056
    off = torch.arange(G, dtype=torch.int32, device="cuda")
    dy, x = torch.zeros(G, N, dtype=torch.bfloat16, device="cuda"), torch.ones(G, K, dtype=torch.bfloat16, device="cuda")
    dy[:] = (torch.arange(G, device="cuda") % 200).bfloat16()[:, None]
    del y
    dw = torch.empty(G, N, K, dtype=torch.bfloat16, device="cuda")
    assert dw.numel() > 1 << 31
    qm.moe_gemm_wgrad(dy, x, G, N, K, G, off, 0, dw, None, ws)
    for g in (0, 255, 511, G - 1):
        assert bool((dw[g] == g % 200).all())
