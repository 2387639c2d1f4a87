"""The 16-bit operators of the framework, forward and backward, as measured cases.

Rows are bf16 and dense.  Grouped rows are sorted by expert: group g owns rows offsets[g] .. offsets[g + 1] - 1 and multiplies
matrix g of a stack.  What a user sees between two calls (h, gate and up products, expert outputs, their gradients) is bf16
and rounded there; sums are 32 bits.

Operators ("op" of a case):
  linear        y = act(x w^T + bias) + residual, one group; with "pre" also the product before the activation
  linear_grad   of y = x w^T + bias: dx = dy w, dw = dy^T x and dbias, the latter two in fp32
  experts       tokens to expert-sorted rows, h = silu(x gate^T) (x up^T), h down^T, the weighted sum of a token's picks
  experts_grad  its backward pass from what the forward pass keeps: gradients of x, of the pick weights and of all matrices
  norm          s = residual + scale f(gate) norm(x) w_post, y = norm(s) w_pre
  norm_grad     its backward pass from dy and ds: gradients of x, residual, gate and both weights
`own` selects the framework's kernels; without it `run` computes the same in elementary torch operations in 32 bits.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
WS_BYTES = 64 << 20


def listed():
    return [
        # one token of a decode step through a projection: weight streaming, launch latency
        dict(name="linear_decode", op="linear", R=1, N=4096, K=2048, act="silu", pre=False),
        # odd sizes: rows, outputs and inputs that end inside a tile, and what a backward pass needs
        dict(name="linear_odd", op="linear", R=301, N=1000, K=2184, act="gelu", pre=True),
        # a large prompt through a projection: tensor-core rate
        dict(name="linear_prompt", op="linear", R=8192, N=8192, K=4096, act="gelu", pre=False),
        # a training batch's gradients of a projection, in the precision in which an optimiser adds them up
        dict(name="linear_grad", op="linear_grad", R=4096, N=4096, K=2048),
        # the repository's layer at its token counts: one token, a prompt
        dict(name="experts_t1", op="experts", T=1, H=2048, I=512, E=256, k=8, shared=True, skew=0.0),
        dict(name="experts_t512", op="experts", T=512, H=2048, I=512, E=256, k=8, shared=True, skew=0.0),
        # a fine-tuning step: few tokens (some experts have none) of a small layer, and a batch of the repository's layer
        dict(name="experts_grad_t64", op="experts_grad", T=65, H=1032, I=264, E=64, k=3, shared=False, skew=0.3),
        dict(name="experts_grad_t4096", op="experts_grad", T=4096, H=2048, I=512, E=256, k=8, shared=True, skew=0.3),
        # one token behind a block whose output has a gate per token (as the shared expert's): launch latency
        dict(name="norm_decode", op="norm", T=1, n=2048, gate="row", act="sigmoid", scale=1.0, post=True),
        # a prompt batch behind a block with a gate per element: bandwidth
        dict(name="norm_prompt", op="norm", T=16384, n=2048, gate="full", act="silu", scale=0.5, post=True),
        # an odd number of rows of a wider model with a learned scale per channel
        dict(name="norm_grad_odd", op="norm_grad", T=777, n=5120, gate="channel", act="none", scale=0.5, post=True),
        # a training batch
        dict(name="norm_grad_batch", op="norm_grad", T=16384, n=2048, gate="full", act="silu", scale=0.5, post=True),
    ]


def _odd(rng, lo, hi, step=1):
    """An odd multiple of step in [lo, hi], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    m = int(v / step) | 1
    return step * (m if m * step <= hi else m - 2)


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_grad", "experts", "experts_grad", "norm", "norm_grad"])
    if op == "linear":
        return dict(op=op, R=_odd(rng, 1, 8192), N=_odd(rng, 64, 8192, 8), K=_odd(rng, 64, 4096, 8),
                    act=rng.choice(["none", "silu", "gelu", "relu"]), pre=rng.random() < 0.5)
    if op == "linear_grad":
        return dict(op=op, R=_odd(rng, 16, 8192), N=_odd(rng, 64, 4096, 8), K=_odd(rng, 64, 4096, 8))
    if op in ("experts", "experts_grad"):
        return dict(op=op, T=_odd(rng, 1, 4096), H=_odd(rng, 256, 2048, 8), I=_odd(rng, 64, 512, 8),
                    E=rng.choice([16, 64, 256]), k=rng.randint(1, 8), shared=rng.random() < 0.5,
                    skew=round(rng.uniform(0.0, 0.3), 2))
    n = _odd(rng, 64, 8192, 8)
    gate = rng.choice(["none", "row", "channel", "full"])
    return dict(op=op, T=_odd(rng, 1, min(16384, 16384 * 2048 // n)), n=n, gate=gate,
                act="none" if gate == "none" else rng.choice(["none", "silu", "sigmoid"]),
                scale=rng.choice([1.0, 0.5]), post=rng.random() < 0.7)


def work(case):
    op = case["op"]
    if op == "linear":
        R, N, K = case["R"], case["N"], case["K"]
        return {"bytes": 2 * (R * K + N * K + N + (3 if case["pre"] else 2) * R * N), "flops": 2 * R * N * K}
    if op == "linear_grad":
        R, N, K = case["R"], case["N"], case["K"]
        return {"bytes": 2 * (R * N + 2 * R * K + N * K) + 4 * (N * K + N), "flops": 4 * R * N * K}
    if op in ("experts", "experts_grad"):
        T, H, I, E, k = case["T"], case["H"], case["I"], case["E"], case["k"]
        rows = T * (k + case["shared"])
        active = E * (1.0 - (1.0 - k / E) ** T) + case["shared"]    # expected number of experts with a token
        if op == "experts":
            return {"bytes": 6 * active * H * I + 4 * T * H + 6 * T * k, "flops": 6 * rows * H * I}
        stack = 6 * H * I
        return {"bytes": active * stack + (E + case["shared"]) * stack + rows * (4 * H + 6 * I) + 4 * T * H + 10 * T * k,
                "flops": 12 * rows * H * I}
    T, n = case["T"], case["n"]
    gate = {"none": 0, "row": 2 * T, "channel": 2 * n, "full": 2 * T * n}[case["gate"]]
    if op == "norm":
        return {"bytes": 8 * T * n + gate + 4 * n, "flops": 12 * T * n}
    return {"bytes": 12 * T * n + 2 * gate + 12 * n, "flops": 30 * T * n}


# ---------------------------------------------------------------- inputs


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _activations(T, n, g):
    """Rows of different size with a few large channels, as hidden states have them."""
    x = torch.randn(T, n, generator=g, device=DEV)
    x *= torch.exp(0.5 * torch.randn(T, 1, generator=g, device=DEV))
    x *= 1 + 15 * (torch.rand(1, n, generator=g, device=DEV) > 0.995)
    return x.bfloat16()


def _normal(shape, g, size=1.0):
    return (size * torch.randn(shape, generator=g, device=DEV)).bfloat16()


def _stack(G, N, K, g):
    """G matrices [N, K] whose products are of the inputs' size."""
    w = torch.empty(G, N, K, dtype=torch.bfloat16, device=DEV)
    for i in range(0, G, 32):
        w[i:i + 32] = torch.randn(min(32, G - i), N, K, generator=g, device=DEV) * K ** -0.5
    return w


def _routing(T, E, k, skew, g):
    """Picks, their order by expert and their weights (normalised over the picks)."""
    logits = torch.randn(T, E, generator=g, device=DEV) + skew * torch.randn(1, E, generator=g, device=DEV)
    top = logits.topk(k, dim=1)
    flat = top.indices.reshape(-1)
    perm = torch.argsort(flat, stable=True)
    inv = torch.empty_like(perm)
    inv[perm] = torch.arange(T * k, device=DEV)
    counts = torch.bincount(flat, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = counts.cumsum(0)
    return {"inv_perm": inv.int(), "offsets": offsets, "cap": int(counts.max()),
            "p": torch.softmax(top.values, 1).bfloat16().contiguous(),
            "w_s": torch.sigmoid(torch.randn(T, generator=g, device=DEV)).bfloat16()}


def prepare(case, seed):
    op, g = case["op"], _gen(seed)
    empty = lambda *n, dtype=torch.bfloat16: torch.empty(n, dtype=dtype, device=DEV)
    st = {"case": dict(case), "ws": torch.zeros(WS_BYTES, dtype=torch.uint8, device=DEV)}
    if op in ("linear", "linear_grad"):
        R, N, K = case["R"], case["N"], case["K"]
        st["x"] = _activations(R, K, g)
        st["w"] = _stack(1, N, K, g)
        if op == "linear":
            st["bias"] = _normal((1, N), g, 0.5)
            st["residual"] = _activations(R, N, g)
            st["y"] = empty(R, N)
            st["pre"] = empty(R, N) if case["pre"] else None
        else:
            st["dy"] = _normal((R, N), g, 0.1)
            st["dx"] = empty(R, K)
            st["dw"], st["db"] = empty(1, N, K, dtype=torch.float32), empty(1, N, dtype=torch.float32)
    if op in ("experts", "experts_grad"):
        T, H, I, E, k, sh = case["T"], case["H"], case["I"], case["E"], case["k"], int(case["shared"])
        G, R = E + sh, T * (k + sh)
        r = st["routing"] = _routing(T, E, k, case["skew"], g)
        if not sh:
            r["w_s"] = None
        st["gate"], st["up"], st["down"] = _stack(G, I, H, g), _stack(G, I, H, g), _stack(G, H, I, g)
        x = _activations(T, H, g)
        if op == "experts":
            st |= {"x": x, "y": empty(T, H), "rows": empty(R, H), "h": empty(R, I), "slots": empty(R, H)}
        else:
            # what the forward pass keeps: sorted rows of x, gate and up products, h, the experts' outputs
            st["x_rows"] = empty(R, H)
            st["x_rows"][_slot_rows(r, T, k, sh)] = x[_slot_tokens(T, k, sh)]
            st["g"], st["u"] = _normal((R, I), g), _normal((R, I), g)
            st["h"] = (torch.nn.functional.silu(st["g"].float()) * st["u"].float()).bfloat16()
            st["slots"] = _normal((R, H), g, 0.5)
            st["dy"] = _normal((T, H), g, 0.1)
            st |= {"dslots": empty(R, H), "dh": empty(R, I), "dg": empty(R, I), "du": empty(R, I), "dx_rows": empty(R, H)}
            st |= {"dx": empty(T, H), "dp": empty(T, k, dtype=torch.float32), "dw_s": empty(T, dtype=torch.float32) if sh else None}
            st |= {"dgate": torch.empty_like(st["gate"]), "dup": torch.empty_like(st["up"]), "ddown": torch.empty_like(st["down"])}
    if op in ("norm", "norm_grad"):
        T, n = case["T"], case["n"]
        st["x"] = _activations(T, n, g)
        res = 3 * _activations(T, n, g)
        shape = {"none": None, "row": (T,), "channel": (n,), "full": (T, n)}[case["gate"]]
        st["gate"] = None if shape is None else _normal(shape, g)
        st["w_post"] = (1 + 0.2 * torch.randn(n, generator=g, device=DEV)).bfloat16() if case["post"] else None
        st["w_pre"] = (1 + 0.2 * torch.randn(n, generator=g, device=DEV)).bfloat16()
        if op == "norm":
            st |= {"residual": res, "s": empty(T, n), "y": empty(T, n)}
        else:
            st |= {"s": res, "dy": _normal((T, n), g, 0.1), "ds": _normal((T, n), g, 0.1)}
            st |= {"dx": empty(T, n), "dres": empty(T, n), "dw_pre": empty(n, dtype=torch.float32)}
            st["dw_post"] = empty(n, dtype=torch.float32) if case["post"] else None
            st["dgate"] = None if shape is None else empty(*shape, dtype=torch.bfloat16 if case["gate"] == "full" else torch.float32)
    return st


# ---------------------------------------------------------------- plain form


def _slot_rows(r, T, k, sh):
    """Row of each slot: routed picks in token order, then the shared expert's."""
    return torch.cat([r["inv_perm"].long(), T * k + torch.arange(T * sh, device=DEV)])


def _slot_tokens(T, k, sh):
    t = torch.arange(T, device=DEV)
    return torch.cat([t.repeat_interleave(k), t[:T * sh]])


def _act(name, v):
    if name == "silu":
        return v * torch.sigmoid(v)
    if name == "sigmoid":
        return torch.sigmoid(v)
    if name == "gelu":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    return v.clamp_min(0) if name == "relu" else v


def _act_slope(name, v):
    """Derivative of the gates' and experts' functions."""
    s = torch.sigmoid(v)
    if name == "silu":
        return s * (1 + v * (1 - s))
    return s * (1 - s) if name == "sigmoid" else torch.ones_like(v)


def _padded(a, r, E):
    """The routed rows as [E, most rows of an expert, n], and where they are in it."""
    p = torch.arange(r["inv_perm"].numel(), device=DEV)
    start = r["offsets"][:E].long()
    gid = torch.searchsorted(start, p, right=True) - 1
    at = gid * r["cap"] + p - start[gid]
    pad = torch.zeros(E * r["cap"], a.shape[1], device=DEV)
    pad[at] = a[:p.numel()].float()
    return pad.view(E, r["cap"], -1), at


def _grouped(a, w, r, E, transpose):
    """Each row times its group's matrix, w [G, N, K] (transpose) or [G, K, N]."""
    Tk = r["inv_perm"].numel()
    f = w.float()
    if transpose:
        f = f.transpose(1, 2)
    pad, at = _padded(a, r, E)
    y = torch.bmm(pad, f[:E]).flatten(0, 1)[at]
    return y if a.shape[0] == Tk else torch.cat([y, a[Tk:].float() @ f[E]])


def _grouped_outer(dy, x, r, E):
    """dy_g^T x_g of each group."""
    Tk = r["inv_perm"].numel()
    w = torch.bmm(_padded(dy, r, E)[0].transpose(1, 2), _padded(x, r, E)[0])
    return (w if dy.shape[0] == Tk else torch.cat([w, (dy[Tk:].float().t() @ x[Tk:].float())[None]])).bfloat16()


def _gate_rows(case, gate):
    """The gate to multiply rows with, before its function."""
    return gate.float()[:, None] if case["gate"] == "row" else gate.float()


def _rstd(v):
    return torch.rsqrt(v.square().mean(1, keepdim=True) + EPS)


def _plain_norm(c, st):
    x = st["x"].float()
    p = x * _rstd(x) * st["w_post"].float() if c["post"] else x
    if c["gate"] != "none":
        p = p * _act(c["act"], _gate_rows(c, st["gate"]))
    s = (st["residual"].float() + c["scale"] * p).bfloat16()
    f = s.float()
    return {"s": s, "y": (f * _rstd(f) * st["w_pre"].float()).bfloat16()}


def _plain_norm_grad(c, st):
    s, dy, x = st["s"].float(), st["dy"].float(), st["x"].float()
    sh = s * _rstd(s)
    d = dy * st["w_pre"].float()
    ds = st["ds"].float() + _rstd(s) * (d - sh * (d * sh).mean(1, keepdim=True))
    xh = x * _rstd(x) if c["post"] else x
    p = xh * st["w_post"].float() if c["post"] else x
    out = {"dres": ds.bfloat16(), "dw_pre": (dy * sh).sum(0)}
    dp = c["scale"] * ds
    if c["gate"] != "none":
        gate = _gate_rows(c, st["gate"])
        dgate = dp * p
        if c["gate"] == "row":
            dgate = dgate.sum(1, keepdim=True)
        if c["gate"] == "channel":
            dgate = dgate.sum(0)
        dgate = dgate * _act_slope(c["act"], gate)
        out["dgate"] = dgate.bfloat16() if c["gate"] == "full" else dgate.flatten()
        dp = dp * _act(c["act"], gate)
    if c["post"]:
        out["dw_post"] = (dp * xh).sum(0)
        d = dp * st["w_post"].float()
        dp = _rstd(x) * (d - xh * (d * xh).mean(1, keepdim=True))
    return {**out, "dx": dp.bfloat16()}


def _plain(st):
    c = st["case"]
    op = c["op"]
    if op == "linear":
        pre = st["x"].float() @ st["w"][0].float().t() + st["bias"].float()
        y = (_act(c["act"], pre) + st["residual"].float()).bfloat16()
        return {"y": y, "pre": pre.bfloat16()} if c["pre"] else {"y": y}
    if op == "linear_grad":
        dy = st["dy"].float()
        return {"dx": (dy @ st["w"][0].float()).bfloat16(), "dw": (dy.t() @ st["x"].float())[None], "db": dy.sum(0)[None]}
    if op == "norm":
        return _plain_norm(c, st)
    if op == "norm_grad":
        return _plain_norm_grad(c, st)
    T, E, k, sh, r = c["T"], c["E"], c["k"], int(c["shared"]), st["routing"]
    rows, token = _slot_rows(r, T, k, sh), _slot_tokens(T, k, sh)
    weight = torch.cat([r["p"].flatten()] + ([r["w_s"]] if sh else [])).float()
    if op == "experts":
        x = torch.empty_like(st["rows"])
        x[rows] = st["x"][token]
        g = _grouped(x, st["gate"], r, E, True)
        h = (_act("silu", g) * _grouped(x, st["up"], r, E, True)).bfloat16()
        slots = _grouped(h, st["down"], r, E, True).bfloat16()
        v = weight[:, None] * slots[rows].float()
        y = v[:T * k].view(T, k, -1).sum(1)
        return (y + v[T * k:] if sh else y).bfloat16()
    dy = st["dy"].float()[token]
    dslots = torch.empty_like(st["slots"])
    dslots[rows] = (weight[:, None] * dy).bfloat16()
    dp = (dy * st["slots"][rows].float()).sum(1)
    dh = _grouped(dslots, st["down"], r, E, False).bfloat16().float()
    g, u = st["g"].float(), st["u"].float()
    dg, du = (dh * u * _act_slope("silu", g)).bfloat16(), (dh * _act("silu", g)).bfloat16()
    dx_rows = (_grouped(dg, st["gate"], r, E, False) + _grouped(du, st["up"], r, E, False)).bfloat16()
    v = dx_rows[rows].float()
    dx = v[:T * k].view(T, k, -1).sum(1)
    out = {"dx": (dx + v[T * k:] if sh else dx).bfloat16(), "dp": dp[:T * k].view(T, k),
           "dgate": _grouped_outer(dg, st["x_rows"], r, E), "dup": _grouped_outer(du, st["x_rows"], r, E),
           "ddown": _grouped_outer(dslots, st["h"], r, E)}
    return {**out, "dw_s": dp[T * k:]} if sh else out


# ---------------------------------------------------------------- the framework's kernels


def _own(st):
    import quantised_moe_expert_gb300 as qm
    c, ws = st["case"], st["ws"]
    op = c["op"]
    act = {"none": qm.MOE_ACT_NONE, "silu": qm.MOE_ACT_SILU, "gelu": qm.MOE_ACT_GELU, "relu": qm.MOE_ACT_RELU,
           "sigmoid": qm.MOE_ACT_SIGMOID}
    if op == "linear":
        qm.moe_gemm(st["x"], st["w"], None, None, 0, c["R"], c["N"], c["K"], 1, None, st["bias"], act[c["act"]], st["residual"],
                    st["pre"], st["y"], ws)
        return {"y": st["y"], "pre": st["pre"]} if c["pre"] else {"y": st["y"]}
    if op == "linear_grad":
        qm.moe_gemm(st["dy"], st["w"], None, None, 1, c["R"], c["K"], c["N"], 1, None, None, qm.MOE_ACT_NONE, None, None,
                    st["dx"], ws)
        qm.moe_gemm_wgrad(st["dy"], st["x"], c["R"], c["N"], c["K"], 1, None, 0, st["dw"], st["db"], ws)
        return {"dx": st["dx"], "dw": st["dw"], "db": st["db"]}
    if op in ("norm", "norm_grad"):
        shape = {"none": qm.MOE_GATE_NONE, "row": qm.MOE_GATE_ROW, "channel": qm.MOE_GATE_CHANNEL, "full": qm.MOE_GATE_FULL}
        how = (shape[c["gate"]], act[c["act"]], c["scale"], int(c["post"]), st["w_post"], st["w_pre"], 0.0, EPS, c["T"], c["n"])
        if op == "norm":
            qm.moe_gated_norm(st["x"], st["residual"], st["gate"], *how, st["s"], st["y"])
            return {"s": st["s"], "y": st["y"]}
        qm.moe_gated_norm_grad(st["x"], st["s"], st["gate"], *how, st["dy"], st["ds"], st["dx"], st["dres"], st["dgate"],
                               st["dw_post"], st["dw_pre"], ws)
        out = {"dres": st["dres"], "dw_pre": st["dw_pre"]}
        if c["gate"] != "none":
            out["dgate"] = st["dgate"]
        if c["post"]:
            out["dw_post"] = st["dw_post"]
        return {**out, "dx": st["dx"]}
    T, H, I, E, k, sh, r = c["T"], c["H"], c["I"], c["E"], c["k"], int(c["shared"]), st["routing"]
    G, R, inv, offsets = E + sh, T * (k + sh), r["inv_perm"], r["offsets"]
    if op == "experts":
        qm.moe_dispatch(st["x"], T, H, k, sh, inv, st["rows"], ws)
        qm.moe_gemm_glu(st["rows"], st["gate"], st["up"], None, None, qm.MOE_ACT_SILU, R, I, H, G, offsets, None, None, st["h"], ws)
        qm.moe_gemm(st["h"], st["down"], None, None, 0, R, H, I, G, offsets, None, qm.MOE_ACT_NONE, None, None, st["slots"], ws)
        qm.moe_weighted_sum(st["slots"], T, H, k, sh, inv, r["p"], r["w_s"], st["y"], ws)
        return st["y"]
    qm.moe_weighted_sum_grad(st["dy"], st["slots"], T, H, k, sh, inv, r["p"], r["w_s"], st["dslots"], st["dp"], st["dw_s"], ws)
    qm.moe_gemm(st["dslots"], st["down"], None, None, 1, R, I, H, G, offsets, None, qm.MOE_ACT_NONE, None, None, st["dh"], ws)
    qm.moe_gemm_wgrad(st["dslots"], st["h"], R, H, I, G, offsets, 0, st["ddown"], None, ws)
    qm.moe_act_grad(qm.MOE_ACT_SILU, st["dh"], st["g"], st["u"], R, I, st["dg"], st["du"])
    qm.moe_gemm(st["dg"], st["gate"], st["du"], st["up"], 1, R, H, I, G, offsets, None, qm.MOE_ACT_NONE, None, None, st["dx_rows"],
                ws)
    qm.moe_gemm_wgrad(st["dg"], st["x_rows"], R, I, H, G, offsets, 0, st["dgate"], None, ws)
    qm.moe_gemm_wgrad(st["du"], st["x_rows"], R, I, H, G, offsets, 0, st["dup"], None, ws)
    qm.moe_weighted_sum(st["dx_rows"], T, H, k, sh, inv, None, None, st["dx"], ws)
    out = {n: st[n] for n in ("dx", "dp", "dgate", "dup", "ddown")}
    return {**out, "dw_s": st["dw_s"]} if sh else out


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- the definition in 64 bits


def _x_sigmoid(v):
    return 1 / (1 + torch.exp(-v))


def _x_fn(name, v):
    """A function's value and derivative."""
    if name == "silu":
        s = _x_sigmoid(v)
        return v * s, s + v * s * (1 - s)
    if name == "sigmoid":
        s = _x_sigmoid(v)
        return s, s * (1 - s)
    if name == "gelu":                                   # v times the logistic function of twice the tanh's argument
        return v * _x_sigmoid(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)), None
    if name == "relu":
        return torch.where(v > 0, v, torch.zeros_like(v)), None
    return v, torch.ones_like(v)


def _x16(v):
    """The value that 16 bits hold of v."""
    return v.to(torch.bfloat16).double()


def _x_norm(v):
    """v / rms(v), and 1 / rms(v)."""
    inv = 1 / torch.sqrt((v * v).sum(1, keepdim=True) / v.shape[1] + EPS)
    return v * inv, inv


def _x_norm_back(d, unit, inv):
    """Gradient of v from the gradient d of v / rms(v)."""
    return inv * (d - unit * ((d * unit).sum(1, keepdim=True) / d.shape[1]))


def _x_gate(case, st):
    if case["gate"] == "none":
        return None, None
    gate = st["gate"].double()
    return _x_fn(case["act"], gate.view(-1, 1) if case["gate"] == "row" else gate)


def _x_bounds(st, E, R, sh):
    at = st["routing"]["offsets"].tolist()
    return [(i, at[i], at[i + 1]) for i in range(E) if at[i + 1] > at[i]] + ([(E, at[E], R)] if sh else [])


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "linear":
        pre = torch.einsum("rk,nk->rn", st["x"].double(), st["w"][0].double()) + st["bias"].double()
        y = _x_fn(case["act"], pre)[0] + st["residual"].double()
        return {"y": y, "pre": pre} if case["pre"] else {"y": y}
    if op == "linear_grad":
        dy = st["dy"].double()
        return {"dx": torch.einsum("rn,nk->rk", dy, st["w"][0].double()),
                "dw": torch.einsum("rn,rk->nk", dy, st["x"].double())[None], "db": dy.sum(0, keepdim=True)}
    if op in ("norm", "norm_grad"):
        x, scale = st["x"].double(), case["scale"]
        a, slope = _x_gate(case, st)
        unit, inv = _x_norm(x) if case["post"] else (x, None)
        w_post = st["w_post"].double() if case["post"] else torch.ones(case["n"], dtype=torch.float64, device=DEV)
        branch = unit * w_post
        if op == "norm":
            s = _x16(st["residual"].double() + scale * (branch if a is None else a * branch))
            return {"s": s, "y": _x_norm(s)[0] * st["w_pre"].double()}
        s_unit, s_inv = _x_norm(st["s"].double())
        dy = st["dy"].double()
        ds = st["ds"].double() + _x_norm_back(dy * st["w_pre"].double(), s_unit, s_inv)
        out = {"dres": ds, "dw_pre": (dy * s_unit).sum(0)}
        d = scale * ds
        if a is not None:
            each = d * branch * slope
            out["dgate"] = each.sum(1) if case["gate"] == "row" else each.sum(0) if case["gate"] == "channel" else each
            d = d * a
        if case["post"]:
            out["dw_post"] = (d * unit).sum(0)
            d = _x_norm_back(d * w_post, unit, inv)
        return {**out, "dx": d}
    T, H, E, k, sh, r = case["T"], case["H"], case["E"], case["k"], int(case["shared"]), st["routing"]
    R, inv_perm = T * (k + sh), r["inv_perm"].long().view(T, k)
    p = r["p"].double()
    if op == "experts":
        x = torch.zeros(R, H, dtype=torch.float64, device=DEV)
        for j in range(k):
            x[inv_perm[:, j]] = st["x"].double()
        x[T * k:] = st["x"].double()[:T * sh]
        slots = torch.zeros_like(x)
        for i, lo, hi in _x_bounds(st, E, R, sh):
            g, u = x[lo:hi] @ st["gate"][i].double().t(), x[lo:hi] @ st["up"][i].double().t()
            slots[lo:hi] = _x16(_x_fn("silu", g)[0] * u) @ st["down"][i].double().t()
        slots = _x16(slots)
        y = r["w_s"].double()[:, None] * slots[T * k:] if sh else 0.0
        for j in range(k):
            y = y + p[:, j, None] * slots[inv_perm[:, j]]
        return y
    dy, slots = st["dy"].double(), st["slots"].double()
    dslots = torch.zeros_like(slots)
    dp = torch.zeros(T, k, dtype=torch.float64, device=DEV)
    for j in range(k):
        dslots[inv_perm[:, j]] = _x16(p[:, j, None] * dy)
        dp[:, j] = torch.einsum("th,th->t", dy, slots[inv_perm[:, j]])
    out = {"dp": dp}
    if sh:
        dslots[T * k:] = _x16(r["w_s"].double()[:, None] * dy)
        out["dw_s"] = torch.einsum("th,th->t", dy, slots[T * k:])
    dx_rows = torch.zeros_like(slots)
    for name in ("gate", "up", "down"):
        out["d" + name] = torch.zeros(st[name].shape, dtype=torch.float64, device=DEV)
    x, h, g, u = st["x_rows"], st["h"], st["g"], st["u"]
    for i, lo, hi in _x_bounds(st, E, R, sh):
        d = dslots[lo:hi]
        dh = _x16(d @ st["down"][i].double())
        a, slope = _x_fn("silu", g[lo:hi].double())
        dg, du = _x16(dh * u[lo:hi].double() * slope), _x16(dh * a)
        dx_rows[lo:hi] = dg @ st["gate"][i].double() + du @ st["up"][i].double()
        out["ddown"][i] = d.t() @ h[lo:hi].double()
        out["dgate"][i], out["dup"][i] = dg.t() @ x[lo:hi].double(), du.t() @ x[lo:hi].double()
    dx_rows = _x16(dx_rows)
    dx = dx_rows[T * k:] if sh else 0.0
    for j in range(k):
        dx = dx + dx_rows[inv_perm[:, j]]
    order = ("dx", "dp", "dgate", "dup", "ddown") + (("dw_s",) if sh else ())
    out["dx"] = dx
    return {n: out[n] for n in order}
