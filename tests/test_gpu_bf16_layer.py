"""The 16-bit operators together, as a layer and a training step use them: values and gradients, one stream without
synchronisation, other streams, captured graphs, and the operators of the framework that they stand beside."""
import os
import sys

import numpy as np
import pytest
import torch

import quantised_moe_expert_gb300 as qm
from quantised_moe_expert_gb300 import synth
from tests.bf16_ref import BF16, act, bf16

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import train_experts  # noqa: E402

pytestmark = pytest.mark.gpu


def routing(T, E, k, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    ids = torch.rand(T, E, generator=g, device="cuda").topk(k, dim=1).indices
    order = torch.argsort(ids.reshape(-1), stable=True)
    inv = torch.empty_like(order)
    inv[order] = torch.arange(T * k, device="cuda")
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.bincount(ids.reshape(-1), minlength=E).cumsum(0)
    return ids, inv.int(), offsets


def layer(E, I, H, k, shared, seed=0):
    G = E + shared
    return qm.Experts16(bf16(G, I, H, seed=seed, size=H ** -0.5), bf16(G, I, H, seed=seed + 1, size=H ** -0.5),
                        bf16(G, H, I, seed=seed + 2, size=I ** -0.5), k, bool(shared))


def reference(e, x, ids, p, w_s):
    """The layer in 64 bits, differentiable."""
    leaves = [t.double().detach().requires_grad_() for t in (x, p, e.gate, e.up, e.down)]
    x, p, gate, up, down = leaves
    w = None if w_s is None else w_s.double().detach().requires_grad_()
    y = torch.zeros_like(x)
    for g in range(gate.shape[0]):
        if g < e.n_experts:
            t, j = (ids == g).nonzero(as_tuple=True)
            c = p[t, j]
        else:
            t, c = torch.arange(x.shape[0], device=x.device), w
        h = act("silu", x[t] @ gate[g].t())[0] * (x[t] @ up[g].t())
        y = y.index_add(0, t, c[:, None] * (h @ down[g].t()))
    return y, leaves[:2] + ([w] if w is not None else []) + leaves[2:]


def off(got, want):
    return float((got.double() - want.double()).norm() / want.double().norm().clamp_min(1e-300))


SHAPES = [(1, 8, 64, 128, 2, 1), (17, 16, 72, 136, 3, 0), (65, 12, 264, 200, 4, 1), (400, 5, 128, 256, 2, 1), (900, 3, 256, 264, 1, 0)]


@pytest.mark.parametrize("T,E,I,H,k,shared", SHAPES)
def test_layer_and_gradients(T, E, I, H, k, shared):
    e, x = layer(E, I, H, k, shared), bf16(T, H, seed=5)
    ids, inv, offsets = routing(T, E, k)
    p = torch.softmax(bf16(T, k, seed=6).float(), 1).bfloat16()
    w_s = torch.sigmoid(bf16(T, seed=7).float()).bfloat16() if shared else None
    ws = torch.zeros(512, dtype=torch.uint8, device="cuda")
    want, leaves = reference(e, x, ids, p, w_s)
    y, kept = e.forward(x, inv, offsets, p, w_s, ws, keep=True)
    assert torch.equal(y, e.forward(x, inv, offsets, p, w_s, ws))
    # in the 2-norm, a rounding of a tensor to bf16 is off by at most 2^-8 of its size, and so is (about) what follows from it: h,
    # the experts' outputs and y; backward also g, u, dslots, dh, dg and du, dx_rows
    assert off(y, want) < 3 * BF16
    dy = bf16(T, H, seed=8)
    grads = torch.autograd.grad(want, leaves, dy.double())
    dx, dp, dw_s, dgate, dup, ddown = e.backward(dy, kept, ws)
    got = [dx, dp] + ([dw_s] if shared else []) + [dgate, dup, ddown]
    for a, b in zip(got, grads):
        assert off(a, b) < 8 * BF16
    # fp32 gradients, and added twice
    f = [torch.zeros_like(m, dtype=torch.float32) for m in (e.gate, e.up, e.down)]
    e.backward(dy, kept, ws, dgate=f[0], dup=f[1], ddown=f[2])
    once = [t.clone() for t in f]
    e.backward(dy, kept, ws, dgate=f[0], dup=f[1], ddown=f[2], accumulate=True)
    for a, b, c in zip(f, once, (dgate, dup, ddown)):
        assert torch.equal(a, b + b) and torch.equal(b.bfloat16(), c)
    assert qm.moe_get_device_status(ws) == 0


def test_block_gradients():
    """The example's block against autograd in 64 bits through the same picks."""
    T, (H, I, E, k) = 50, (136, 72, 6, 2)
    block, ws = train_experts.Block(H, I, E, k), train_experts.workspace(50, 136)
    s0 = bf16(T, H, seed=1, size=2.0)
    out, saved = block.forward(s0, ws)
    dout = bf16(T, H, seed=2)
    ds0, grads = block.backward(dout, saved, ws)
    inv, offsets, p, w_s = saved[3][5:]
    ids = torch.searchsorted(offsets.long(), inv.long(), right=True).view(T, k) - 1
    w = {n: v.double().requires_grad_() for n, v in block.w.items()}
    s = s0.double().requires_grad_()
    unit = lambda v: v * torch.rsqrt(v.square().mean(1, keepdim=True) + train_experts.EPS)
    x = unit(s) * w["norm_in"]
    y = torch.zeros_like(x)
    for g in range(E + 1):
        t, j = (ids == g).nonzero(as_tuple=True) if g < E else (torch.arange(T, device="cuda"), None)
        c = p.double()[t, j] if g < E else w_s.double()
        h = act("silu", x[t] @ w["gate"][g].t())[0] * (x[t] @ w["up"][g].t())
        y = y.index_add(0, t, c[:, None] * (h @ w["down"][g].t()))
    s1 = s + block.scale * act("silu", w["channel_gate"])[0] * unit(y) * w["norm_post"]
    want = unit(s1) * w["norm_out"]
    assert off(out, want.detach()) < 6 * BF16                        # as the layer, and x, s1 and out
    names = list(w)
    ref = torch.autograd.grad(want, [s] + [w[n] for n in names], dout.double())
    assert off(ds0, ref[0]) < 12 * BF16
    for n, r in zip(names, ref[1:]):
        assert off(grads[n], r) < 12 * BF16, n
    assert qm.moe_get_device_status(ws) == 0


def test_example_runs():
    losses = train_experts.run(tokens=70, steps=2, hidden=136, inter=72, n_experts=6, top_k=2)
    assert len(losses) == 2 and all(np.isfinite(losses))


def test_routed_by_the_framework():
    """moe_route and moe_permute give what the 16-bit experts take: against moe_forward on the same (dequantised) matrices."""
    shape = synth.LayerShape(hidden=256, inter=128, n_experts=16, top_k=4)
    host = synth.make_weights(shape, 3)
    T = 33
    x = torch.from_numpy(synth.make_x(shape, T, 3).view(np.int16)).cuda()
    plain = qm.DeviceLayer(host)
    ws = qm.workspace(plain.cfg, T)

    def matrix(m, s, N, n):
        parts = []
        for q in (m, s):
            c = torch.from_numpy(np.ascontiguousarray(q.codes)).cuda().view(-1, N, n // 2)
            c = torch.stack([c & 15, c >> 4], -1).flatten(-2).double()
            t = lambda a: torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).cuda().view(torch.bfloat16).double().view(-1, N, n // 64, 1)
            parts.append((c.view(-1, N, n // 64, 64) * t(q.scales) + t(q.biases)).view(-1, N, n))
        return torch.cat(parts).bfloat16()

    H, I = shape.hidden, shape.inter
    e = qm.Experts16(matrix(host.gate, host.s_gate, I, H), matrix(host.up, host.s_up, I, H), matrix(host.down, host.s_down, H, I), 4, True)
    i32 = lambda *n: torch.empty(n, dtype=torch.int32, device="cuda")
    ids, p, w_s = i32(T, 4), torch.empty(T, 4, dtype=torch.int16, device="cuda"), torch.empty(T, dtype=torch.int16, device="cuda")
    counts, offsets, perm, inv = i32(16), i32(17), i32(T * 4), i32(T * 4)
    qm.moe_route(plain.cfg, plain.w, x, T, None, None, None, ids, p, w_s, ws)
    qm.moe_permute(plain.cfg, ids, T, counts, offsets, perm, inv, ws)
    y = e.forward(x.view(torch.bfloat16), inv, offsets, p, w_s, ws)
    want = qm.forward(plain, x, ws).view(torch.bfloat16)
    # the matrices' rounding to bf16 (three products deep), x's and h's to fp16 there, h, slots and y here
    assert off(y, want) < 7 * BF16
    assert qm.moe_get_device_status(ws) == 0


def chain(block, s0, dout, ws, sync=False):
    out, saved = block.forward(s0, ws)
    if sync:
        torch.cuda.synchronize()
    ds0, grads = block.backward(dout, saved, ws)
    return [out, ds0] + [grads[n] for n in sorted(grads)]


def test_one_stream_without_synchronisation():
    """Every kernel starts under its predecessor's tail: the same bits as with the device idle between the calls."""
    T, H = 200, 264
    block, ws = train_experts.Block(H, 136, 8, 2), train_experts.workspace(200, 264)
    s0, dout = bf16(T, H, seed=1), bf16(T, H, seed=2)
    want = None
    names = [n for n in qm.EXPORTED if n.startswith(("moe_gemm", "moe_act", "moe_disp", "moe_weighted", "moe_gated_norm")) and "size" not in n]
    saved = {n: getattr(qm, n) for n in names}
    try:
        for n in names:
            def idle(*a, call=saved[n], **k):
                torch.cuda.synchronize()
                call(*a, **k)
                torch.cuda.synchronize()
            setattr(qm, n, idle)
        want = chain(block, s0, dout, ws)
    finally:
        for n in names:
            setattr(qm, n, saved[n])
    for _ in range(10):
        for a, b in zip(chain(block, s0, dout, ws), want):
            assert torch.equal(a, b)


def test_other_streams_and_captured_graphs():
    """The layer, forward and backward, on a stream of its own and from a captured graph replayed with other inputs, beside an
    eager pass on the current stream with a workspace of its own."""
    T, E, I, H, k = 90, 8, 136, 264, 2
    e = layer(E, I, H, k, 1)
    _, inv, offsets = routing(T, E, k)
    p, w_s = torch.softmax(bf16(T, k, seed=6).float(), 1).bfloat16(), torch.sigmoid(bf16(T, seed=7).float()).bfloat16()
    ws, ws2 = (torch.zeros(512, dtype=torch.uint8, device="cuda") for _ in range(2))
    xs, dys = [bf16(T, H, seed=20 + i) for i in range(3)], [bf16(T, H, seed=30 + i) for i in range(3)]

    def both(x, dy, ws):
        y, kept = e.forward(x, inv, offsets, p, w_s, ws, keep=True)
        return (y, *e.backward(dy, kept, ws))

    want = [both(x, dy, ws) for x, dy in zip(xs, dys)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = both(xs[1], dys[1], ws2)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want[1]))
    x, dy, graph = xs[0].clone(), dys[0].clone(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        out = both(x, dy, ws2)
    for i in (0, 1, 2, 1):
        x.copy_(xs[i])
        dy.copy_(dys[i])
        graph.replay()
        eager = both(xs[2], dys[2], ws)                              # the same kernels and leaves, between replays
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want[i]))
        assert all(torch.equal(a, b) for a, b in zip(eager, want[2]))
    assert qm.moe_get_device_status(ws) == 0 and qm.moe_get_device_status(ws2) == 0


def test_two_calls_at_once():
    """Products of two streams on the device together, each with its workspace."""
    a, w = bf16(700, 520, seed=1), bf16(1, 1000, 520, seed=2)
    ws = [torch.zeros(512, dtype=torch.uint8, device="cuda") for _ in range(2)]
    ys = [torch.empty(700, 1000, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    dw = [torch.empty(1, 1000, 520, device="cuda") for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, s in enumerate(streams):
            qm.moe_gemm(a, w, None, None, 0, 700, 1000, 520, 1, None, None, 0, None, None, ys[i], ws[i], s)
            qm.moe_gemm_wgrad(ys[i], a, 700, 1000, 520, 1, None, 0, dw[i], None, ws[i], s)
    torch.cuda.synchronize()
    assert torch.equal(ys[0], ys[1]) and torch.equal(dw[0], dw[1])
    assert off(ys[0], a.double() @ w[0].double().t()) < BF16
    assert all(qm.moe_get_device_status(v) == 0 for v in ws)
