"""The block-scaled operators and the layer's other kernels behind one another on one stream.  Each of the former lets its
successor start early, and some of the latter may be started early; what they write for one another must be there all the
same: a chain called without waits, and replayed from a graph, gives the bits of the chain with a wait after every call."""
import numpy as np
import pytest
import torch

import quantised_moe_expert_gb300 as qm
from quantised_moe_expert_gb300 import synth

pytestmark = pytest.mark.gpu

NV, M8 = qm.MOE_SCALED_NVFP4, qm.MOE_SCALED_MXFP8
LAYERS = 3


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    qm.load()


@pytest.mark.parametrize("T", [1, 16, 40])
@pytest.mark.parametrize("kind", ["affine", "nvfp4"])
def test_norm_layer_projection_chain(kind, T):
    """norm -> moe_forward (16 bits) -> norm to codes -> product -> norm -> block-scaled layer, layer after layer."""
    shape = synth.LayerShape(hidden=512, inter=256, n_experts=16, top_k=4, fmt=kind)
    nvshape = synth.LayerShape(hidden=512, inter=256, n_experts=16, top_k=4, fmt="nvfp4")
    H = shape.hidden
    plain = [qm.DeviceLayer(synth.make_weights(shape, 50 + i)) for i in range(LAYERS)]
    host = [synth.make_weights(nvshape, 60 + i) for i in range(LAYERS)]
    x0 = torch.from_numpy(synth.make_x(shape, T, 3).view(np.int16)).cuda()
    scaled = [qm.ScaledLayer.from_nvfp4(h, torch.full((17,), 0.02)) for h in host]
    gen = torch.Generator(device="cuda").manual_seed(7)
    codes = torch.randint(0, 256, (1, H, H // 2), dtype=torch.uint8, generator=gen, device="cuda")
    tiles = torch.randint(0x30, 0x40, (H // 128 * qm.scaled_col_tiles(NV, H) * 512,), dtype=torch.uint8, generator=gen, device="cuda")
    w = qm.scaled_mat(codes, tiles, torch.full((1,), 1 / (3.3 * H ** 0.5), device="cuda"))
    ws, ws_s, ws_g = qm.workspace(plain[0].cfg, T), qm.scaled_workspace(scaled[0].cfg, NV, T), torch.zeros(512, dtype=torch.uint8, device="cuda")
    s, x, y, z = (torch.empty_like(x0) for _ in range(4))
    q = qm.scaled_rows_empty(NV, T, H)
    kept = [[torch.empty_like(x0) for _ in range(4)] for _ in range(LAYERS)]
    torch.cuda.synchronize()

    def chain(wait):
        s.copy_(x0)
        y.zero_()
        for i in range(LAYERS):
            steps = [
                lambda: qm.moe_add_rmsnorm(s, y, None, 0.0, 1e-6, T, H, s, x, 0, None),
                lambda: qm.moe_forward(plain[i].cfg, plain[i].w, x, T, None, None, y, None, None, None, qm.MOE_PATH_AUTO, ws),
                lambda: qm.moe_add_rmsnorm(s, y, None, 0.0, 1e-6, T, H, s, None, NV, q),
                lambda: qm.moe_scaled_gemm(NV, q, w, T, H, H, 1, None, z, ws_g),
                lambda: qm.moe_add_rmsnorm(s, z, None, 0.0, 1e-6, T, H, s, x, 0, None),
                lambda: qm.moe_scaled_forward(scaled[i].cfg, scaled[i].w, x, T, None, None, y, None, None, None, ws_s),
            ]
            for step in steps:
                step()
                if wait:
                    torch.cuda.synchronize()
            for k, t in zip(kept[i], (s, x, y, z)):
                k.copy_(t)

    def result():
        torch.cuda.synchronize()
        assert all(qm.moe_get_device_status(v) == 0 for v in (ws, ws_s, ws_g))
        return [k.clone() for row in kept for k in row]

    chain(True)
    want = result()
    assert all(torch.isfinite(t.view(torch.bfloat16).float()).all() and (t != 0).any() for t in want)
    for _ in range(5):
        chain(False)
        assert all(torch.equal(a, b) for a, b in zip(want, result()))
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        chain(False)
    for _ in range(5):
        for row in kept:
            for k in row:
                k.zero_()
        torch.cuda.synchronize()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(want, result()))
