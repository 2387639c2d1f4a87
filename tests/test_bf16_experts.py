"""Experts16 on the host: whose memory it works in.  The library's calls are replaced by recorders; no call reaches a GPU."""
import contextlib
import inspect

import pytest
import torch

import quantised_moe_expert_gb300 as qm

CALLS = ("moe_dispatch", "moe_gemm_glu", "moe_gemm", "moe_weighted_sum", "moe_weighted_sum_grad", "moe_gemm_wgrad", "moe_act_grad")
T, E, K, H, I = 3, 4, 2, 16, 8
HERE, SIDE = "the current stream", 0x5000


def rows(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def experts(shared=True):
    G = E + shared
    return qm.Experts16(rows(G, I, H), rows(G, I, H), rows(G, H, I), K, shared)


def arguments():
    return torch.arange(T * K, dtype=torch.int32), torch.zeros(E + 1, dtype=torch.int32), rows(T, K), rows(T)


WS = torch.zeros(512, dtype=torch.uint8)


@pytest.fixture()
def world(monkeypatch):
    """Streams without a GPU: which one is current, whose memory each tensor is, which streams its memory waits for, and the
    library's calls."""
    class World:
        current, owner, uses, calls = HERE, {}, {}, []
        kept = []                                            # (keeps the tensors alive, and so their addresses apart)

    w = World()
    w.owner, w.uses, w.calls, w.kept = {}, {}, [], []

    @contextlib.contextmanager
    def stream(s):
        before, w.current = w.current, s
        yield
        w.current = before

    make = torch.empty

    def empty(*a, **k):
        t = make(*a, **k)
        w.owner[t.data_ptr()] = w.current
        w.kept.append(t)
        return t

    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch, "empty_like", lambda t, **k: empty(t.shape, dtype=k.get("dtype", t.dtype)))
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: w.current)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda *a: "the default stream")
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, *a: handle)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: w.uses.setdefault(t.data_ptr(), set()).add(s))
    for name in CALLS:
        names = list(inspect.signature(getattr(qm, name)).parameters)

        def call(*a, _name=name, _names=names, **k):
            given = dict(zip(_names, a), **k)
            on = given.pop("stream", None)
            w.calls.append((_name, w.current if on is None else on, given))

        monkeypatch.setattr(qm, name, call)
    return w


def both(e, **how):
    y, kept = e.forward(rows(T, H), *arguments(), WS, keep=True, **how)
    return (y, *kept[:5]), e.backward(rows(T, H), kept, WS, **how)


@pytest.mark.parametrize("stream,expect", [(None, HERE), (SIDE, SIDE), (0, "the default stream")])
def test_memory_belongs_to_the_stream_of_the_call(world, stream, expect):
    """Everything that a call makes and works in is memory of the stream that it runs on: with memory of another stream, what is
    dropped when the call returns would be handed out again under its kernels."""
    out, grads = both(experts(), stream=stream)
    assert [c[0] for c in world.calls] == list(CALLS[:4]) + ["moe_weighted_sum_grad", "moe_gemm_wgrad", "moe_gemm", "moe_act_grad",
                                                             "moe_gemm_wgrad", "moe_gemm_wgrad", "moe_gemm", "moe_weighted_sum"]
    assert world.current == HERE
    made = 0
    for name, on, given in world.calls:
        assert on in (expect, stream)
        for t in given.values():
            if isinstance(t, torch.Tensor) and t.data_ptr() in world.owner:
                made += 1
                assert world.owner[t.data_ptr()] == expect, name
    assert made >= 20
    if stream is not None:                                   # what the caller gets may be used, and dropped, on the stream it called from
        for t in (*out, *grads):
            assert HERE in world.uses.get(t.data_ptr(), ())
        for t in out[1:]:                                    # and what forward kept is read by backward's stream
            assert expect in world.uses[t.data_ptr()]


def test_memory_belongs_to_the_stream_without_keeping(world):
    y = experts().forward(rows(T, H), *arguments(), WS, stream=SIDE)
    assert world.owner[y.data_ptr()] == SIDE and HERE in world.uses[y.data_ptr()]
    assert all(owner == SIDE for owner in world.owner.values())


@pytest.mark.parametrize("default", [torch.float64, torch.bfloat16])
def test_gradients_of_pick_weights_are_fp32(world, default):
    """Whatever torch's default element type is: the library would refuse the call half way through the pass."""
    torch.set_default_dtype(default)
    try:
        _, (dx, dp, dw_shared, *_) = both(experts())
    finally:
        torch.set_default_dtype(torch.float32)
    assert dp.dtype == dw_shared.dtype == torch.float32 and dx.dtype == torch.bfloat16


def short(t):
    return t.reshape(-1)[:-1].contiguous()


@pytest.mark.parametrize("name,bad", [
    ("x", rows(T, H - 8)), ("x", rows(T, H + 8)), ("x", rows(T * H)), ("inv_perm", short(arguments()[0])), ("offsets", arguments()[1][:E]),
    ("p", short(rows(T, K))), ("w_shared", rows(T - 1)), ("w_shared", None)])
def test_sizes_that_do_not_fit_are_refused_forward(world, name, bad):
    """The library sees addresses and the sizes that follow from x and the matrices: a tensor that holds less would be read past its end."""
    e, given = experts(), dict(zip(("x", "inv_perm", "offsets", "p", "w_shared"), (rows(T, H), *arguments())))
    e.forward(**given, ws=WS)
    count = len(world.calls)
    with pytest.raises(qm.MoeError) as err:
        e.forward(**{**given, name: bad}, ws=WS)
    assert err.value.status == qm.MOE_ERR_INVALID_ARG and len(world.calls) == count


def f32(*shape):
    return torch.zeros(shape)


@pytest.mark.parametrize("bad", [
    dict(dy=rows(T, H - 8)), dict(dy=rows(T + 1, H)), dict(dy=rows(T - 1, H)), dict(dy=rows(T * H)), dict(dgate=short(f32(E + 1, I, H))),
    dict(dup=f32(E, I, H)), dict(ddown=f32(E + 2, H, I)),
    # added to: only what the caller holds, in 32 bits, and none of the three before all of them are known to be
    dict(accumulate=True), dict(accumulate=True, dgate=f32(E + 1, I, H), ddown=f32(E + 1, H, I)),
    dict(accumulate=True, dgate=f32(E + 1, I, H), dup=rows(E + 1, I, H), ddown=f32(E + 1, H, I))])
def test_what_does_not_fit_is_refused_backward(world, bad):
    e = experts()
    _, kept = e.forward(rows(T, H), *arguments(), WS, keep=True)
    given = dict(dy=rows(T, H), dgate=f32(E + 1, I, H), dup=f32(E + 1, I, H), ddown=f32(E + 1, H, I))
    e.backward(**given, kept=kept, ws=WS, accumulate=True)
    count = len(world.calls)
    with pytest.raises(qm.MoeError) as err:
        e.backward(**({"dy": given["dy"], **bad} if "accumulate" in bad else {**given, **bad}), kept=kept, ws=WS)
    assert err.value.status in (qm.MOE_ERR_INVALID_ARG, qm.MOE_ERR_UNSUPPORTED) and len(world.calls) == count


def test_longer_routing_buffers_and_no_tokens(world):
    """Routing buffers may hold more than the tokens need; there may be no tokens."""
    inv, offsets, p, w_s = arguments()
    for shared in (True, False):
        e, longer = experts(shared), lambda t: torch.cat([t.reshape(-1), t.reshape(-1)])
        for n in (T, 0):
            y, kept = e.forward(rows(n, H), longer(inv), longer(offsets), longer(p), longer(w_s) if shared else None, WS, keep=True)
            assert y.shape == (n, H) and e.backward(rows(n, H), kept, WS)[0].shape == (n, H)
