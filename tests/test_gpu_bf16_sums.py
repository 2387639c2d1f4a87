"""Long sums of the 16-bit products in 32 bits: few rows, tiles, and sums that are rounded to bf16 at their end.

An instruction adds 16 terms and truncates the sum so far by at most 2^-23 of it, half of that in the mean.  Over a sum of
random terms the sums so far are 2/3 of the last one in the mean.  768 terms, 48 instructions: 48 / 3 times 2^-23 of a sum if all
truncations point one way; then those sums are added up with a rounding (2^-24 of the sum so far) each."""
import pytest
import torch

import quantised_moe_expert_gb300 as qm
from tests.bf16_ref import bf16

pytestmark = pytest.mark.gpu
SEGMENT = 48 / 3 * 2.0 ** -23


@pytest.fixture()
def ws():
    w = torch.zeros(qm.MOE_SCALED_WS_BYTES, dtype=torch.uint8, device="cuda")
    yield w
    assert qm.moe_get_device_status(w) == 0


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


def most(terms):
    return SEGMENT + (terms / 768) ** 0.5 * 2.0 ** -24


# rows that run without tiles (up to 8, 16 and more of groups), and rows that do not
@pytest.mark.parametrize("pairs", [1, 2])
@pytest.mark.parametrize("R,N,K,G", [(1, 264, 65536, 1), (8, 64, 65536, 1), (8, 1000, 8192, 1), (30, 72, 65528, 3), (17, 200, 30000, 2),
                                     (9, 64, 65536, 1), (300, 136, 65536, 1), (300, 136, 8192, 1)])
def test_products(ws, R, N, K, G, pairs):
    """The same bound at any number of rows and any length."""
    a, w = [bf16(R, K, seed=i) for i in range(pairs)], [bf16(G, N, K, seed=5 + i) for i in range(pairs)]
    first = [g * R // G for g in range(G)] + [R]
    offsets = torch.tensor(first[:G], dtype=torch.int32, device="cuda") if G > 1 else None
    y = torch.empty(R, N, device="cuda")
    two = lambda t: t[1] if pairs == 2 else None
    qm.moe_gemm(a[0], w[0], two(a), two(w), 0, R, N, K, G, offsets, None, 0, None, None, y, ws)
    for g in range(G):
        r = slice(first[g], first[g + 1])
        want = sum(m[r].double() @ v[g].double().t() for m, v in zip(a, w))
        assert off(y[r], want) < most(pairs * K)


@pytest.mark.parametrize("terms,N,K", [(4096, 1000, 72), (8192, 64, 72), (65536, 64, 72), (65536, 264, 1032), (8192, 2560, 2560)])
def test_gradients(ws, terms, N, K):
    dy, x = bf16(terms, N, seed=1), bf16(terms, K, seed=2)
    want = dy.double().t() @ x.double()
    dw, y = torch.empty(1, N, K, device="cuda"), torch.empty(N, K, device="cuda")
    qm.moe_gemm_wgrad(dy, x, terms, N, K, 1, None, 0, dw, None, ws)
    qm.moe_gemm(dy.t().contiguous(), x, None, None, 1, N, K, terms, 1, None, None, 0, None, None, y, ws)
    assert off(dw[0], want) < most(terms) and off(y, want) < most(terms)


def nearest(got, want, terms):
    """bf16 values that are what 64 bits round to, but for what fp32 sums may be off by.  Sums of one sign, so far half of the last one
    in the mean: in segments of 8192 terms an instruction's truncation is off by at most 2^-23 of that, 512 times, and every
    segment, and every part of a sum, is added with a rounding of at most 2^-24 of it.  512 2^-24 = 2^-15 is 1/64 of the smallest half
    step of bf16, 2^-9."""
    half = torch.exp2(torch.floor(torch.log2(want)) - 8)
    tol = half + (512 * 2.0 ** -24 + (terms / 8192 + 8) * 2.0 ** -25) * want
    bad = (got.double() - want).abs() > tol
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()}, by {float(((got.double() - want).abs() / want).max()):.2e}"


# a tile's steps shared out to CTAs, tiles of one CTA, pairs of CTAs; with the end of a sum inside a step, beside a group of a few rows
@pytest.mark.parametrize("counts,N,K", [([1 << 21], 64, 64), ([3, (1 << 18) + 5], 1032, 1032), ([1 << 18], 2560, 2560), ([40, (1 << 18) - 3], 2568, 2560)])
def test_bf16_gradients_of_very_long_groups(ws, counts, N, K):
    """Sums of one sign, where what an addition loses grows with the number of terms: it must not reach the rounding to bf16."""
    R = sum(counts)
    u = 0.5 + bf16(R, seed=1).float().abs().bfloat16()
    x = bf16(R, K, seed=2).abs_().add_(0.25)
    dy = u[:, None].expand(R, N).contiguous()
    first = [sum(counts[:g]) for g in range(len(counts))]
    dw = torch.empty(len(counts), N, K, dtype=torch.bfloat16, device="cuda")
    qm.moe_gemm_wgrad(dy, x, R, N, K, len(counts), torch.tensor(first, dtype=torch.int32, device="cuda"), 0, dw, None, ws)
    for g, c in enumerate(counts):
        want = torch.zeros(K, dtype=torch.float64, device="cuda")
        for r in range(first[g], first[g] + c, 1 << 16):
            r = slice(r, min(r + (1 << 16), first[g] + c))
            want += u[r].double() @ x[r].double()
        nearest(dw[g], want.expand(N, K), c)


@pytest.mark.parametrize("transposed", [0, 1])
@pytest.mark.parametrize("R,N", [(300, 136), (1024, 8192)])
def test_bf16_products_of_two_long_pairs(ws, R, N, transposed):
    """The longest sums of a product: two pairs of 65536 terms."""
    K = 65536
    a = [bf16(1, K, seed=i).abs_().add_(0.25).expand(R, K).contiguous() for i in range(2)]
    w = [bf16(N, K, seed=5 + i).abs_().add_(0.25) for i in range(2)]
    want = sum(torch.cat([w[i][n:n + 1024].double() @ a[i][0].double() for n in range(0, N, 1024)]) for i in range(2))
    m = [(v.t().contiguous() if transposed else v)[None] for v in w]
    y = torch.empty(R, N, dtype=torch.bfloat16, device="cuda")
    qm.moe_gemm(a[0], m[0], a[1], m[1], transposed, R, N, K, 1, None, None, 0, None, None, y, ws)
    nearest(y, want.expand(R, N), 2 * K)


@pytest.mark.parametrize("R,N", [(300, 72), (1024, 5120)])
def test_long_gated_pairs(ws, R, N):
    """A gated pair of 65536 terms each, whose up products are kept: those, and h where the gate is one."""
    K = 65536
    a = bf16(1, K, seed=1).abs_().add_(0.25).expand(R, K).contiguous()
    gate, up = torch.zeros(1, N, K, dtype=torch.bfloat16, device="cuda"), bf16(1, N, K, seed=3).abs_().add_(0.25)
    bias = torch.ones(1, N, dtype=torch.bfloat16, device="cuda")
    g, u, h = (torch.empty(R, N, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    qm.moe_gemm_glu(a, gate, up, bias, None, qm.MOE_ACT_RELU, R, N, K, 1, None, g, u, h, ws)
    want = torch.cat([up[0, n:n + 1024].double() @ a[0].double() for n in range(0, N, 1024)]).expand(R, N)
    nearest(u, want, K)
    assert bool((g == 1).all()) and torch.equal(h, u)
