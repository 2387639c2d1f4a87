"""Expert-sorted copies of rows, weighted sums of them, and gradients through activations, against 64 bits."""
import pytest
import torch

import quantised_moe_expert_gb300 as qm
from tests.bf16_ref import BF16, FUNCTION, act, bf16, within

pytestmark = pytest.mark.gpu
MARK = -7.0


@pytest.fixture()
def ws():
    w = torch.zeros(qm.MOE_SCALED_WS_BYTES, dtype=torch.uint8, device="cuda")
    yield w
    assert qm.moe_get_device_status(w) == 0


def routing(T, k, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randperm(T * k, generator=g, device="cuda").int()


SIZES = [(1, 8, 1, 0), (1, 2048, 8, 1), (3, 72, 16, 1), (65, 1032, 3, 0), (300, 256, 5, 1), (17, 8200, 2, 1)]


@pytest.mark.parametrize("T,n,k,shared", SIZES)
def test_dispatch(ws, T, n, k, shared):
    x, inv = bf16(T, n), routing(T, k)
    R = T * (k + shared)
    y = torch.full((R + 2, n), MARK, dtype=torch.bfloat16, device="cuda")
    qm.moe_dispatch(x, T, n, k, shared, inv, y[:R], ws)
    want = torch.empty_like(y[:R])
    want[inv.long()] = x.repeat_interleave(k, 0)
    want[T * k:] = x[:T * shared]
    assert torch.equal(y[:R], want) and bool((y[R:] == MARK).all())


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("T,n,k,shared", SIZES)
def test_weighted_sum_and_gradient(ws, T, n, k, shared, weighted):
    R, inv = T * (k + shared), routing(T, k, 1)
    rows, p = bf16(R, n, seed=1), bf16(T, k, seed=2)
    w_s = bf16(T, seed=3) if shared else None
    at = inv.long().view(T, k)
    pd = p.double() if weighted else torch.ones(T, k, dtype=torch.float64, device="cuda")
    sd = None if not shared else w_s.double() if weighted else torch.ones(T, dtype=torch.float64, device="cuda")
    terms = pd[:, :, None] * rows.double()[at]
    if shared:
        terms = torch.cat([terms, (sd[:, None] * rows.double()[T * k:])[:, None]], 1)
    y = torch.full((T + 2, n), MARK, dtype=torch.bfloat16, device="cuda")
    qm.moe_weighted_sum(rows, T, n, k, shared, inv, p if weighted else None, w_s if weighted else None, y[:T], ws)
    want = terms.sum(1)
    within(y[:T], want, BF16 * want.abs() + 2 * (k + 1) * 2.0 ** -23 * terms.abs().sum(1))
    assert bool((y[T:] == MARK).all())
    if not weighted:
        return
    dy = bf16(T, n, seed=4)
    drows = torch.full((R + 2, n), MARK, dtype=torch.bfloat16, device="cuda")
    dp, dw_s = torch.full((T, k), MARK, device="cuda"), torch.full((T,), MARK, device="cuda") if shared else None
    qm.moe_weighted_sum_grad(dy, rows, T, n, k, shared, inv, p, w_s, drows[:R], dp, dw_s, ws)
    want = torch.zeros(R, n, dtype=torch.float64, device="cuda")
    want[at] = pd[:, :, None] * dy.double()[:, None]
    if shared:
        want[T * k:] = sd[:, None] * dy.double()
    within(drows[:R], want, BF16 * want.abs())                           # a product of two bf16 is exact in fp32
    assert bool((drows[R:] == MARK).all())
    each = rows.double()[at] * dy.double()[:, None]
    within(dp, each.sum(2), n * 2.0 ** -24 * each.abs().sum(2))
    if shared:
        each = rows.double()[T * k:] * dy.double()
        within(dw_s, each.sum(1), n * 2.0 ** -24 * each.abs().sum(1))
    # the gradient of the rows alone, and in the rows' place
    again = torch.full_like(drows, MARK)
    qm.moe_weighted_sum_grad(dy, None, T, n, k, shared, inv, p, w_s, again[:R], None, None, ws)
    assert torch.equal(again, drows)
    place, dp2 = rows.clone(), torch.empty_like(dp)
    qm.moe_weighted_sum_grad(dy, place, T, n, k, shared, inv, p, w_s, place, dp2, None, ws)
    assert torch.equal(place, drows[:R]) and torch.equal(dp, dp2)


def test_dispatch_and_sum_are_each_others_gradients(ws):
    """<dispatch(x), r> = <x, sum of r's rows> in exact arithmetic: small whole numbers."""
    T, n, k = 40, 64, 3
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    whole = lambda *s: torch.randint(-3, 4, s, generator=g, device="cuda").bfloat16()
    x, r, inv = whole(T, n), whole(T * 4, n), routing(T, k)
    y, dx = torch.empty_like(r), torch.empty_like(x)
    qm.moe_dispatch(x, T, n, k, 1, inv, y, ws)
    qm.moe_weighted_sum(r, T, n, k, 1, inv, None, None, dx, ws)
    assert float((y.double() * r.double()).sum()) == float((x.double() * dx.double()).sum())


def test_places_outside_the_rows_are_reported():
    ws = torch.zeros(512, dtype=torch.uint8, device="cuda")
    T, n, k = 4, 64, 2
    inv = torch.tensor([0, 1, 2, 3, 4, 8, -1, 1 << 30], dtype=torch.int32, device="cuda")
    x, rows = bf16(T, n), bf16(T * k, n, seed=1)
    y = torch.full((T * k, n), MARK, dtype=torch.bfloat16, device="cuda")
    qm.moe_dispatch(x, T, n, k, 0, inv, y, ws)
    assert qm.moe_get_device_status(ws) == qm.MOE_ERR_DEVICE
    assert torch.equal(y[:5], x.repeat_interleave(2, 0)[:5]) and bool((y[5:] == MARK).all())
    out, p = torch.empty(T, n, dtype=torch.bfloat16, device="cuda"), torch.ones(T, k, dtype=torch.bfloat16, device="cuda")
    qm.moe_weighted_sum(rows, T, n, k, 0, inv, p, None, out, ws)
    assert qm.moe_get_device_status(ws) == qm.MOE_ERR_DEVICE
    assert torch.equal(out[2], rows[4]) and bool((out[3] == 0).all())
    y.fill_(MARK)
    dp = torch.empty(T, k, device="cuda")
    qm.moe_weighted_sum_grad(x, rows, T, n, k, 0, inv, p, None, y, dp, None, ws)
    assert qm.moe_get_device_status(ws) == qm.MOE_ERR_DEVICE
    assert bool((y[5:] == MARK).all()) and dp[2, 1] == 0 and bool((dp[3] == 0).all())


ACTS = {"none": qm.MOE_ACT_NONE, "silu": qm.MOE_ACT_SILU, "gelu": qm.MOE_ACT_GELU, "relu": qm.MOE_ACT_RELU}


@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("R,N", [(1, 8), (3, 72), (301, 1000)])
def test_act_grad(name, R, N):
    dy, pre, up = bf16(R, N, seed=1), bf16(R, N, seed=2, size=3.0), bf16(R, N, seed=3)
    pre[0, :8] = torch.tensor([0.0, -0.0, 30.0, -30.0, 1e30, -1e30, 100.0, -100.0])
    v, d = act(name, pre.double().clamp(-1e4, 1e4))          # the slopes are flat there, and v^3 leaves no range
    v = torch.where(pre.double() > 1e4, pre.double(), torch.where((pre.double() < -1e4) & (name != "none"), torch.zeros_like(v), v))
    if name == "none":
        v = pre.double()
    # slopes: sums of two terms of at most |pre| + 1, each off by the function's error
    off = FUNCTION * (1 + pre.double().abs().clamp_max(30))
    dpre, dup = torch.empty_like(dy), torch.empty_like(dy)
    qm.moe_act_grad(ACTS[name], dy, pre, None, R, N, dpre, None)
    want = dy.double() * d
    tiny = 2.0 ** -126
    within(dpre, want, BF16 * want.abs() + dy.double().abs() * off + tiny)
    qm.moe_act_grad(ACTS[name], dy, pre, up, R, N, dpre, dup)
    want = dy.double() * up.double() * d
    within(dpre, want, BF16 * want.abs() + (dy.double() * up.double()).abs() * off + tiny)
    want = dy.double() * v
    within(dup, want, BF16 * want.abs() + dy.double().abs() * off + tiny)
    a, b = dpre.clone(), dup.clone()
    in_pre, in_up = pre.clone(), up.clone()
    qm.moe_act_grad(ACTS[name], dy, in_pre, in_up, R, N, in_pre, in_up)
    assert torch.equal(in_pre, a) and torch.equal(in_up, b)


def test_act_grad_against_differences():
    """The slopes that the gradient uses against differences of the function that the product's epilogue uses."""
    n, step = 512, 2.0 ** -5
    pre = torch.linspace(-6, 6, n, device="cuda").bfloat16().view(1, n)
    ones, ws = torch.ones_like(pre), torch.zeros(512, dtype=torch.uint8, device="cuda")
    eye = torch.eye(n, device="cuda").bfloat16()[None]
    def value(v, a):
        y = torch.empty(1, n, device="cuda")
        zero = torch.zeros_like(v)
        qm.moe_gemm(zero, eye, None, None, 0, 1, n, n, 1, None, v, a, None, None, y, ws)
        return y.double()
    for name, a in ACTS.items():
        if name == "relu":
            continue
        lo, hi = (pre.double() - step).bfloat16(), (pre.double() + step).bfloat16()
        got = torch.empty_like(pre)
        qm.moe_act_grad(a, ones, pre, None, 1, n, got, None)
        want = (value(hi, a) - value(lo, a)) / (hi.double() - lo.double()).clamp_min(1e-9)
        # a difference over [lo, hi] is the slope somewhere in it: off by at most 1.2 (largest second derivative, about 1.1 for
        # these functions) times its width; the values' fp32 errors (2^-20 of up to 6) over that width
        width = hi.double() - lo.double()
        ok = width > 0
        tol = BF16 * want.abs() + 1.2 * width + 6 * 2.0 ** -20 / width.clamp_min(1e-9)
        within(got[ok], want[ok], tol[ok])


@pytest.mark.parametrize("name", ACTS)
def test_act_grad_at_the_ends_of_the_range(name):
    """Values and slopes at the largest arguments and around the point past which GELU's slope is held; the value is the one that the
    products' epilogue gives."""
    v = torch.tensor([3e38, -3e38, 1e38, -1e38, 1e20, -1e20, 300.0, -300.0, 12.0, -12.0, 10.0, -10.0, 10.25, -10.25, 9.75, -9.75], device="cuda").bfloat16()
    n = v.numel()
    ones, up, d, dup = torch.ones(1, n, dtype=torch.bfloat16, device="cuda"), torch.full((1, n), 2.0, dtype=torch.bfloat16, device="cuda"), *(
        torch.empty(1, n, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    qm.moe_act_grad(ACTS[name], ones, v.view(1, n), up, 1, n, d, dup)
    c = v.double().clamp(-1e4, 1e4)                          # v^3 of the 64-bit form stays in range
    value, slope = act(name, c)
    if name != "none":
        value = torch.where(v.double() > 1e4, v.double(), value)
    else:
        value = v.double()
    # past +-9 a function is v or 0, and its slope 1 or 0, to fewer than 2^-20 of 12
    within(dup[0], value, BF16 * value.abs() + 2.0 ** -16)
    within(d[0], 2 * slope, BF16 * 2 * slope.abs() + 2.0 ** -16)
    ws = torch.zeros(512, dtype=torch.uint8, device="cuda")
    zero, y = torch.zeros(1, n, dtype=torch.bfloat16, device="cuda"), torch.empty(1, n, device="cuda")
    qm.moe_gemm(zero, torch.zeros(1, n, n, dtype=torch.bfloat16, device="cuda"), None, None, 0, 1, n, n, 1, None, v, ACTS[name], None, None, y, ws)
    within(dup, y.double(), BF16 * y.double().abs())


@pytest.mark.parametrize("name", ["silu", "gelu", "relu"])
def test_nan_reaches_the_gradients(name):
    """Of an element whose pre is NaN, and of no other, value and slope are NaN, plain and as a gated pair."""
    pre = torch.linspace(-3, 3, 16, device="cuda").bfloat16().view(2, 8)
    dy, up, odd = torch.ones_like(pre), torch.full_like(pre, 2.0), pre.clone()
    odd[1, 3] = float("nan")
    outs = []
    for v in (pre, odd):
        plain, d, dup = (torch.empty_like(pre) for _ in range(3))
        qm.moe_act_grad(ACTS[name], dy, v, None, 2, 8, plain, None)
        qm.moe_act_grad(ACTS[name], dy, v, up, 2, 8, d, dup)
        outs.append((plain, d, dup))
    for a, b in zip(*outs):
        assert bool(b[1, 3].isnan()) and int(b.isnan().sum()) == 1
        assert torch.equal(torch.where(odd.isnan(), 0.0, a), torch.where(odd.isnan(), 0.0, b))
