"""Norms around a block with its gate and residual, forward and backward, against 64 bits."""
import pytest
import torch

import quantised_moe_expert_gb300 as qm
from tests.bf16_ref import BF16, FUNCTION, act, bf16, within

pytestmark = pytest.mark.gpu
MARK = -7.0
EPS = 1e-6
GATES = {"none": qm.MOE_GATE_NONE, "row": qm.MOE_GATE_ROW, "channel": qm.MOE_GATE_CHANNEL, "full": qm.MOE_GATE_FULL}
ACTS = {"none": qm.MOE_ACT_NONE, "silu": qm.MOE_ACT_SILU, "sigmoid": qm.MOE_ACT_SIGMOID}


def inputs(T, n, gate, seed=0):
    shape = {"none": None, "row": (T,), "channel": (n,), "full": (T, n)}[gate]
    return {"x": bf16(T, n, seed=seed, size=2.0), "residual": bf16(T, n, seed=seed + 1, size=3.0),
            "gate": None if shape is None else bf16(*shape, seed=seed + 2),
            "post": (1 + 0.2 * bf16(n, seed=seed + 3).float()).bfloat16(), "pre": (1 + 0.2 * bf16(n, seed=seed + 4).float()).bfloat16(),
            "dy": bf16(T, n, seed=seed + 5), "ds": bf16(T, n, seed=seed + 6)}


def rstd(v):
    return torch.rsqrt((v * v).mean(1, keepdim=True) + EPS)


def gate_of(i, gate, fn):
    if gate == "none":
        return torch.ones((), dtype=torch.float64, device="cuda"), None
    g = i["gate"].double()
    return act(fn, g[:, None] if gate == "row" else g)


CASES = [(1, 8, "none", "none", 0), (1, 2048, "row", "sigmoid", 1), (3, 264, "channel", "none", 1), (7, 1000, "full", "silu", 1),
         (33, 72, "full", "none", 0), (301, 520, "row", "silu", 0), (5, 8192, "full", "sigmoid", 1), (700, 256, "channel", "sigmoid", 1),
         (2000, 5120, "channel", "silu", 1), (1300, 1024, "row", "none", 1)]


@pytest.mark.parametrize("offset,scale", [(0.0, 1.0), (1.0, -0.375)])
@pytest.mark.parametrize("T,n,gate,fn,post", CASES)
def test_forward(T, n, gate, fn, post, offset, scale):
    i = inputs(T, n, gate)
    x, f = i["x"].double(), gate_of(i, gate, fn)[0]
    w_post = i["post"] if post else None
    b = x * rstd(x) * (offset + i["post"].double()) if post else x
    branch = scale * f * b
    want = i["residual"].double() + branch
    s, y = (torch.full((T + 1, n), MARK, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    call = lambda residual, s_out, y_out: qm.moe_gated_norm(i["x"], residual, i["gate"], GATES[gate], ACTS[fn], scale, post, w_post,
                                                           i["pre"], offset, EPS, T, n, s_out, y_out)
    call(i["residual"], s[:T], y[:T])
    # the branch: a few fp32 roundings, a mean of n squares (n 2^-24, halved by the root), the fast exponential (of gates up to 5)
    off = (8 * 2.0 ** -24 + n * 2.0 ** -25 + 6 * FUNCTION) * branch.abs()
    within(s[:T], want, BF16 * want.abs() + 2 * off)
    got = s[:T].double()                                   # y is the norm of the s that was written
    want = got * rstd(got) * (offset + i["pre"].double())
    within(y[:T], want, (BF16 + 8 * 2.0 ** -24 + n * 2.0 ** -25) * want.abs())
    assert bool((s[T:] == MARK).all()) and bool((y[T:] == MARK).all())
    # in the residual's place, one output at a time, without a residual
    place, only = i["residual"].clone(), torch.empty_like(y[:T])
    call(place, place, None)
    call(i["residual"], None, only)
    assert torch.equal(place, s[:T]) and torch.equal(only, y[:T])
    call(None, place, None)
    within(place, branch, BF16 * branch.abs() + 2 * off)


def test_norm_alone_is_the_framework_s_norm():
    """Without gate and post norm, s and y are those of moe_add_rmsnorm."""
    T, n = 9, 2048
    i = inputs(T, n, "none")
    s, y, s2, y2 = (torch.empty(T, n, dtype=torch.bfloat16, device="cuda") for _ in range(4))
    qm.moe_gated_norm(i["x"], i["residual"], None, 0, 0, 1.0, 0, None, i["pre"], 0.5, EPS, T, n, s, y)
    qm.moe_add_rmsnorm(i["x"], i["residual"], i["pre"], 0.5, EPS, T, n, s2, y2, 0, None)
    assert torch.equal(s, s2)
    within(y, y2.double(), 2 * BF16 * y2.double().abs())


def backward(i, s, gate, fn, post, scale, offset, use_dy=True, use_ds=True):
    """The formulas in 64 bits: outputs and, for each, the size of the terms it sums."""
    n = s.shape[1]
    s, x = s.double(), i["x"].double()
    pre, w_post = offset + i["pre"].double(), (offset + i["post"].double()) if post else torch.ones(n, dtype=torch.float64, device="cuda")
    D = i["ds"].double() if use_ds else torch.zeros_like(s)
    size = D.abs()
    out = {}
    if use_dy:
        rs = rstd(s)
        sh, d = s * rs, i["dy"].double() * pre
        m = (d * sh).mean(1, keepdim=True)
        D = D + rs * (d - sh * m)
        size = size + rs * (d.abs() + sh.abs() * (d * sh).abs().mean(1, keepdim=True))
        out["dpre"] = ((i["dy"].double() * sh).sum(0), (i["dy"].double() * sh).abs().sum(0))
    out["dres"] = (D, size)
    f, slope = gate_of(i, gate, fn)
    rx = rstd(x) if post else 1.0
    xh = x * rx
    b = xh * w_post
    if gate != "none":
        each, mag = scale * D * b * slope, abs(scale) * size * (b * slope).abs()
        dim = {"row": 1, "channel": 0, "full": None}[gate]
        out["dgate"] = (each, mag) if dim is None else (each.sum(dim), mag.sum(dim))
    e, esize = scale * f * D, (scale * f).abs() * size
    if post:
        out["dpost"] = ((e * xh).sum(0), (esize * xh.abs()).sum(0))
        d, dsize = e * w_post, esize * w_post.abs()
        e = rx * (d - xh * (d * xh).mean(1, keepdim=True))
        esize = rx * (dsize + xh.abs() * (dsize * xh.abs()).mean(1, keepdim=True))
    out["dx"] = (e, esize)
    return out


def run_grad(i, s, gate, fn, post, scale, offset, use_dy=True, use_ds=True):
    T, n = s.shape
    ws = torch.zeros(qm.moe_gated_norm_workspace_size(T, n), dtype=torch.uint8, device="cuda")
    out = {"dx": torch.empty_like(s), "dres": torch.empty_like(s)}
    if gate != "none":
        out["dgate"] = torch.empty_like(i["gate"], dtype=torch.bfloat16 if gate == "full" else torch.float32)
    if post:
        out["dpost"] = torch.empty(n, device="cuda")
    if use_dy:
        out["dpre"] = torch.empty(n, device="cuda")
    qm.moe_gated_norm_grad(i["x"], s, i["gate"], GATES[gate], ACTS[fn], scale, post, i["post"] if post else None, i["pre"], offset, EPS, T, n,
                           i["dy"] if use_dy else None, i["ds"] if use_ds else None, out["dx"], out["dres"], out.get("dgate"),
                           out.get("dpost"), out.get("dpre"), ws)
    return out


@pytest.mark.parametrize("use", ["both", "dy", "ds"])
@pytest.mark.parametrize("T,n,gate,fn,post", CASES)
def test_backward(T, n, gate, fn, post, use):
    i, scale, offset = inputs(T, n, gate, seed=20), 0.75, 0.5
    s = bf16(T, n, seed=40, size=3.0)
    how = dict(use_dy=use != "ds", use_ds=use != "dy")
    want, got = backward(i, s, gate, fn, post, scale, offset, **how), run_grad(i, s, gate, fn, post, scale, offset, **how)
    assert set(want) == set(got)
    # fp32 throughout: two means of n terms, the fast exponential, and a sum of T terms where rows are summed
    each = 32 * 2.0 ** -24 + 2 * n * 2.0 ** -24 + 6 * FUNCTION
    for name, (v, size) in want.items():
        summed = T * 2.0 ** -24 if name in ("dpost", "dpre") or (name == "dgate" and gate == "channel") else 0.0
        step = BF16 * v.abs() if got[name].dtype == torch.bfloat16 else 0.0
        within(got[name], v, step + 2 * (each + summed) * size)
    again = run_grad(i, s, gate, fn, post, scale, offset, **how)
    assert all(torch.equal(got[k], again[k]) for k in got)


# every width of block of the backward pass, each with more rows than the blocks hold at once
@pytest.mark.parametrize("T,n,gate,fn,post", [(1500, 64, "row", "silu", 1), (1111, 512, "full", "silu", 1), (1900, 1032, "full", "none", 1),
                                              (1400, 2048, "row", "sigmoid", 1), (1100, 2056, "none", "none", 1), (1003, 2560, "full", "silu", 0),
                                              (801, 3320, "channel", "sigmoid", 1), (997, 4096, "row", "silu", 1), (900, 5000, "full", "sigmoid", 1),
                                              (620, 6144, "none", "none", 0), (457, 8184, "channel", "none", 1)])
def test_backward_of_many_rows(T, n, gate, fn, post):
    test_backward(T, n, gate, fn, post, "both")


@pytest.mark.parametrize("gate,fn", [("full", "silu"), ("row", "sigmoid"), ("channel", "none")])
def test_backward_against_differences(gate, fn):
    """The formulas' gradients against differences of the formulas (in 64 bits), for the loss <dy, y> + <ds, s>."""
    T, n = 3, 16
    i, scale, offset = inputs(T, n, gate, seed=60), 0.75, 0.5
    i = {k: v.double() for k, v in i.items()}

    def loss(i):
        x, f = i["x"], gate_of(i, gate, fn)[0]
        s = i["residual"] + scale * f * x * rstd(x) * (offset + i["post"])
        return (i["ds"] * s).sum() + (i["dy"] * s * rstd(s) * (offset + i["pre"])).sum(), s

    want = backward(i, loss(i)[1], gate, fn, 1, scale, offset)
    for name, key in (("x", "dx"), ("residual", "dres"), ("gate", "dgate"), ("post", "dpost"), ("pre", "dpre")):
        h = 1e-4
        for at in range(0, i[name].numel(), 5):
            d = []
            for sign in (1, -1):
                j = dict(i)
                j[name] = i[name].clone()
                j[name].view(-1)[at] += sign * h
                d.append(loss(j)[0])
            slope = float((d[0] - d[1]) / (2 * h))
            # third derivatives of a few tens at most: h^2 times that
            assert abs(slope - float(want[key][0].reshape(-1)[at])) < 1e-5


def test_rows_apart_and_in_place():
    """A row without finite values leaves the others alone; outputs in their inputs' places."""
    T, n = 40, 264
    i = inputs(T, n, "full", seed=80)
    s = bf16(T, n, seed=90)
    clean = run_grad(i, s, "full", "silu", 1, 1.0, 0.0)
    j = {k: (v.clone() if v is not None else v) for k, v in i.items()}
    j["x"][5], j["dy"][5] = float("nan"), float("inf")
    got = run_grad(j, s, "full", "silu", 1, 1.0, 0.0)
    keep = torch.arange(T, device="cuda") != 5
    for k in ("dx", "dres", "dgate"):
        assert torch.equal(got[k][keep], clean[k][keep])
    ws = torch.zeros(qm.moe_gated_norm_workspace_size(T, n), dtype=torch.uint8, device="cuda")
    x, ds = i["x"].clone(), i["ds"].clone()
    qm.moe_gated_norm_grad(x, s, i["gate"], 3, 1, 1.0, 1, i["post"], i["pre"], 0.0, EPS, T, n, i["dy"], ds, x, ds, None, None, None, ws)
    assert torch.equal(x, clean["dx"]) and torch.equal(ds, clean["dres"])


def test_zero_rows_and_no_rows():
    """Rows of zeros divide by sqrt(eps); sums over no rows are zero."""
    n = 64
    i = inputs(2, n, "none")
    z = torch.zeros(2, n, dtype=torch.bfloat16, device="cuda")
    y = torch.empty_like(z)
    qm.moe_gated_norm(z, None, None, 0, 0, 1.0, 1, i["post"], i["pre"], 0.0, EPS, 2, n, None, y)
    assert bool((y == 0).all())
    i["x"] = z
    out = run_grad(i, z, "none", "none", 1, 1.0, 0.0)
    assert all(bool(v.isfinite().all()) for v in out.values())
    e = z[:0]
    dpost, dpre = torch.full((n,), MARK, device="cuda"), torch.full((n,), MARK, device="cuda")
    ws = torch.zeros(qm.moe_gated_norm_workspace_size(0, n), dtype=torch.uint8, device="cuda")
    qm.moe_gated_norm_grad(e, e, None, 0, 0, 1.0, 1, i["post"], i["pre"], 0.0, EPS, 0, n, e, e, e, None, None, dpost, dpre, ws)
    assert bool((dpost == 0).all()) and bool((dpre == 0).all())


@pytest.mark.parametrize("T,n,gate", [(40, 264, "row"), (40, 264, "full"), (40, 264, "channel"), (600, 2048, "full"), (600, 2056, "row")])
@pytest.mark.parametrize("fn", ["sigmoid", "silu"])
def test_saturated_gates(T, n, gate, fn):
    """Gates of -30 to 30: where the function is next to 0 or 1, its slope is small and not 0, and as exact, relative to itself, as
    others (SiLU's between its zero and 0 is left out: a difference of two terms)."""
    i, scale = inputs(T, n, gate, seed=70), 0.75
    g = torch.linspace(-30, 30, i["gate"].numel(), dtype=torch.float64, device="cuda").view(i["gate"].shape)
    if fn == "silu":
        g = torch.where((g > -4) & (g < 0), -g, g)
    i["gate"] = g.bfloat16()
    s = bf16(T, n, seed=71, size=3.0)
    # what the gate multiplies, times the slope without 1 - s, which is off by 2^-53 of 1 in 64 bits too (1e-3 of itself at 30)
    g = i["gate"].double()
    up, down = torch.sigmoid(g), torch.sigmoid(-g)
    slope = up * down if fn == "sigmoid" else up * (1 + g * down)
    v, size = (t * (slope if k == 0 else slope.abs()) for k, t in enumerate(backward(i, s, gate, "none", 1, scale, 0.0)["dgate"]))
    got = run_grad(i, s, gate, fn, 1, scale, 0.0)["dgate"]
    # as test_backward; the exponential of up to 30 is off by 2^-23 of 2 + 1.2 x 30 units
    each = 32 * 2.0 ** -24 + 2 * n * 2.0 ** -24 + 40 * 2.0 ** -23
    summed = T * 2.0 ** -24 if gate == "channel" else 0.0
    within(got, v, (BF16 * v.abs() if gate == "full" else 0.0) + 2 * (each + summed) * size)


# dsum and a gate per element come a row ahead through registers past 5120 columns: several rows a block, with and without each
@pytest.mark.parametrize("use", ["both", "dy", "ds"])
@pytest.mark.parametrize("T,n,gate,fn,post", [(700, 5640, "full", "silu", 1), (500, 8192, "full", "sigmoid", 1), (613, 6152, "full", "none", 0),
                                              (470, 8192, "row", "silu", 1), (613, 5128, "channel", "sigmoid", 1)])
def test_backward_of_many_wide_rows(T, n, gate, fn, post, use):
    test_backward(T, n, gate, fn, post, use)


@pytest.mark.parametrize("n", [2048, 5120, 8192])
def test_rows_apart_and_in_place_of_many_rows(n):
    """As test_rows_apart_and_in_place, with several rows a block: what a row leaves in shared memory does not reach the next."""
    T = 1000
    i = inputs(T, n, "full", seed=80)
    s = bf16(T, n, seed=90)
    clean = run_grad(i, s, "full", "silu", 1, 1.0, 0.0)
    j = {k: (v.clone() if v is not None else v) for k, v in i.items()}
    for r, bad in ((5, float("nan")), (400, float("inf")), (T - 200, -float("inf"))):
        j["x"][r], j["dy"][r, 3], j["gate"][r, n - 1] = bad, bad, bad
    got = run_grad(j, s, "full", "silu", 1, 1.0, 0.0)
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[[5, 400, T - 200]] = False
    for k in ("dx", "dres", "dgate"):
        assert torch.equal(got[k][keep], clean[k][keep])
    ws = torch.zeros(qm.moe_gated_norm_workspace_size(T, n), dtype=torch.uint8, device="cuda")
    for dx, dres in (("x", "ds"), ("dy", "s"), ("ds", "dy")):    # outputs in the inputs' places
        b = {"x": i["x"].clone(), "dy": i["dy"].clone(), "ds": i["ds"].clone(), "s": s.clone()}
        qm.moe_gated_norm_grad(b["x"], b["s"], i["gate"], 3, 1, 1.0, 1, i["post"], i["pre"], 0.0, EPS, T, n, b["dy"], b["ds"], b[dx], b[dres],
                               None, None, None, ws)
        assert torch.equal(b[dx], clean["dx"]) and torch.equal(b[dres], clean["dres"])
    assert qm.moe_get_device_status(ws) == 0
