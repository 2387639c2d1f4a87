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
