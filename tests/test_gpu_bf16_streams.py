"""Experts16 on a stream that is given, beside a current stream that goes on allocating and writing."""
import pytest
import torch

import quantised_moe_expert_gb300 as qm
from tests.bf16_ref import bf16
from tests.test_gpu_bf16_layer import layer, routing

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("by_handle", [False, True])
def test_a_given_stream(by_handle):
    """Memory of the sizes that the layer works in is allocated and filled on the current stream right behind each call, while the
    given stream is still busy with earlier work: values and gradients are those of the current stream alone."""
    T, E, I, H, k = 300, 6, 136, 264, 2
    e, x, dy = layer(E, I, H, k, 1), bf16(T, H, seed=5), bf16(T, H, seed=8)
    _, inv, offsets = routing(T, E, k)
    p, w_s = torch.softmax(bf16(T, k, seed=6).float(), 1).bfloat16(), torch.sigmoid(bf16(T, seed=7).float()).bfloat16()
    ws, ws2 = (torch.zeros(512, dtype=torch.uint8, device="cuda") for _ in range(2))
    y, kept = e.forward(x, inv, offsets, p, w_s, ws, keep=True)
    want = [y.clone()] + [t.clone() for t in e.backward(dy, kept, ws)]
    del y, kept
    side = torch.cuda.Stream()
    stream = side.cuda_stream if by_handle else side
    big = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    R = T * (k + 1)
    sizes = [(R, H), (R, I), (T, H), (R, H), (R, I), (R, I), (R, I), tuple(e.gate.shape), tuple(e.up.shape), tuple(e.down.shape)]
    for _ in range(5):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for _ in range(4):
                big @ big                                    # what the layer's kernels wait behind
        y, kept = e.forward(x, inv, offsets, p, w_s, ws2, keep=True, stream=stream)
        written = [torch.full(s, float("nan"), dtype=torch.bfloat16, device="cuda") for s in sizes]
        got = [y, *e.backward(dy, kept, ws2, stream=stream)]
        del kept
        written += [torch.full(s, float("nan"), dtype=torch.bfloat16, device="cuda") for s in sizes]
        torch.cuda.current_stream().wait_stream(side)
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        assert all(bool(t.isnan().all()) for t in written)
        y = got = None
    assert qm.moe_get_device_status(ws2) == 0


@pytest.mark.parametrize("forked", [False, True])
def test_a_given_stream_captured(forked):
    """The same in a captured graph, on the capturing stream and on one that it forks to and joins, replayed with other inputs."""
    T, E, I, H, k = 90, 6, 136, 264, 2
    e = layer(E, I, H, k, 1)
    _, inv, offsets = routing(T, E, k)
    p, w_s = torch.softmax(bf16(T, k, seed=6).float(), 1).bfloat16(), torch.sigmoid(bf16(T, seed=7).float()).bfloat16()
    ws = torch.zeros(512, dtype=torch.uint8, device="cuda")
    xs, dys = [bf16(T, H, seed=20 + i) for i in range(3)], [bf16(T, H, seed=30 + i) for i in range(3)]

    def both(x, dy, stream=None):
        y, kept = e.forward(x, inv, offsets, p, w_s, ws, keep=True, stream=stream)
        return (y, *e.backward(dy, kept, ws, stream=stream))

    want = [[t.clone() for t in both(x, dy)] for x, dy in zip(xs, dys)]
    main, other, graph = torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    x, dy = xs[0].clone(), dys[0].clone()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=main):
        if forked:
            other.wait_stream(main)
        out = both(x, dy, other if forked else main)
        if forked:
            main.wait_stream(other)
    for i in (0, 1, 2, 1):
        x.copy_(xs[i])
        dy.copy_(dys[i])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want[i]))
    assert qm.moe_get_device_status(ws) == 0
