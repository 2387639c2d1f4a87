"""Block-scaled products whose in-kernel waits run out: reported, the kernels return, and what they leave serves the next
call.  Sizes reach every launch shape that waits (tiles, halves of the K steps on two CTAs, pairs of CTAs); limits from a
single poll up end the roles of a CTA at different places.  Nothing here traps, faults or hangs the GPU."""
import numpy as np
import pytest
import torch

import quantised_moe_expert_gb300 as qm
from quantised_moe_expert_gb300 import synth

from . import scaled_ref as S

pytestmark = pytest.mark.gpu

NV, M8 = S.NV, S.M8
# tokens, hidden, inter (two experts, one pick each): both products in tiles; the SwiGLU's K steps on two CTAs each; the down
# products by pairs of CTAs (512 rows a group)
SIZES = {
    "tiles": {NV: (700, 512, 192), M8: (700, 512, 256)},
    "split": {NV: (64, 4096, 256), M8: (64, 4096, 256)},
    "pairs": {NV: (1024, 8192, 2048), M8: (1024, 8192, 1024)},
}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    qm.load()


def layer(fmt, hidden, inter):
    """Two experts of random codes, no shared one, routed by given logits."""
    gen = torch.Generator(device="cuda").manual_seed(hidden + inter)
    lo, hi = (0x30, 0x40) if fmt == NV else (118, 122)

    def mat(N, K):
        codes = torch.randint(0, 256, (2, N, K // 2), dtype=torch.uint8, device="cuda", generator=gen)
        tiles = 2 * -(-N // 128) * qm.scaled_col_tiles(fmt, K)
        scales = torch.randint(lo, hi, (tiles * 512,), dtype=torch.uint8, device="cuda", generator=gen)
        return qm.scaled_mat(codes, scales, torch.full((2,), 1 / 64, device="cuda") if fmt == NV else None)

    shape = synth.LayerShape(hidden=hidden, inter=inter, n_experts=2, top_k=1, has_shared=0)
    h_scale = torch.full((2,), 16.0, device="cuda") if fmt == NV else None
    router = [torch.zeros(16, device="cuda")] * 3
    return shape, qm.ScaledLayer(shape, fmt, router, None, mat(inter, hidden), mat(inter, hidden), mat(hidden, inter), h_scale)


@pytest.mark.parametrize("fmt", [NV, M8])
@pytest.mark.parametrize("size", SIZES)
def test_waits_that_run_out(fmt, size):
    T, hidden, inter = SIZES[size][fmt]
    shape, lay = layer(fmt, hidden, inter)
    gen = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn(T, hidden, generator=gen, device="cuda").bfloat16()
    logits = torch.randn(T, 2, generator=gen, device="cuda")
    y, ws = torch.empty_like(x), qm.scaled_workspace(lay.cfg, fmt, T)

    def call(cfg):
        qm.moe_scaled_forward(cfg, lay.w, x, T, None, logits, y, None, None, None, ws)
        return qm.moe_get_device_status(ws)

    assert call(lay.cfg) == 0
    want = y.clone()
    assert torch.isfinite(want.float()).all() and want.float().abs().max() > 0
    assert call(qm.config_of(shape, wait_polls=1)) == qm.MOE_ERR_TIMEOUT
    for polls in (2, 3, 5, 8, 13, 30, 100):
        status = call(qm.config_of(shape, wait_polls=polls))
        assert status == qm.MOE_ERR_TIMEOUT or (status == 0 and torch.equal(y, want))
    assert call(lay.cfg) == 0 and torch.equal(y, want)


@pytest.mark.parametrize("fmt", [NV, M8])
@pytest.mark.parametrize("R,N,K", [(300, 520, 128), (64, 512, 3840), (3001, 2008, 2304)])
@pytest.mark.parametrize("bad", [(0, 0.5, 0.4), (-3, 0.2, 0.4), (0, 0.2, 1.5)])
def test_bad_offsets_in_every_launch_shape(fmt, R, N, K, bad):
    """Offsets that decrease or leave the rows: reported, nothing is computed."""
    G, n = 3, qm.scaled_col_tiles(fmt, K) * 512
    codes = torch.zeros((R, K if fmt == M8 else K // 2), dtype=torch.uint8, device="cuda")
    a = qm.scaled_rows(codes, torch.full(((R // 128 + G) * n,), 0x38, dtype=torch.uint8, device="cuda"))
    w = qm.scaled_mat(torch.zeros((G, N, K // 2), dtype=torch.uint8, device="cuda"),
                      torch.full((G * -(-N // 128) * n,), 0x38, dtype=torch.uint8, device="cuda"))
    off = np.array([bad[0], int(bad[1] * R), int(bad[2] * R)], np.int32)
    y, ws = torch.full((R, N), 7.0, device="cuda"), torch.zeros(512, dtype=torch.uint8, device="cuda")
    qm.moe_scaled_gemm(fmt, a, w, R, N, K, G, torch.from_numpy(off).cuda(), y, ws)
    assert qm.moe_get_device_status(ws) == qm.MOE_ERR_DEVICE
    assert (y == 7).all()
    qm.moe_scaled_gemm(fmt, a, w, R, N, K, G, torch.tensor([0, R // 3, R // 2], dtype=torch.int32, device="cuda"), y, ws)
    assert qm.moe_get_device_status(ws) == 0 and (y == 0).all()
