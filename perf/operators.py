"""The block-scaled operators of the framework as measured cases.

A block-scaled row holds narrow codes and one scale per block of consecutive elements:
  nvfp4  E2M1 codes, an E4M3 scale per 16 elements, an fp32 factor per row (activations) or matrix (weights)
  mxfp8  E4M3 codes, a power-of-two scale (E8M0) per 32 elements; its products take mxfp4 weights
  mxfp4  E2M1 codes, a power-of-two scale (E8M0) per 32 elements
Scales are stored in tiles of 128 rows x 4 blocks, 512 bytes each: byte (r % 32) * 16 + (r // 32) * 4 + b of a tile.

Operators ("op" of a case):
  norm         s = bf16(x + residual), y = s * rsqrt(mean(s^2) + eps) * w, out as bf16 and as mxfp8
  quant        rows of x as mxfp8, written into the expert-sorted rows of their k picks and of the shared expert
  gemm         y = a w^T, both operands block-scaled (one group)
  linear       bf16 rows quantised, then the product (one group)
  norm_linear  norm with block-scaled output only, then the product
  experts      expert-sorted rows: gate/up products, h = silu(g) u quantised, down product
`own` selects the framework's kernels; without it `run` computes the same in elementary torch operations in 32 bits.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
WS_BYTES = 16 << 20


def listed():
    return [
        # one token of a decode step, hidden size of the repository's layer: launch latency
        dict(name="norm_decode", op="norm", T=1, H=2048, fmt="mxfp8"),
        # an odd number of rows of a wider model
        dict(name="norm_odd", op="norm", T=777, H=5120, fmt="mxfp8"),
        # a prompt batch: bandwidth
        dict(name="norm_prefill", op="norm", T=32768, H=2048, fmt="mxfp8"),
        # the norm of a 16-token decode batch straight into a 4-bit projection
        dict(name="norm_linear_t16", op="norm_linear", T=16, H=2048, N=8192, fmt="nvfp4"),
        # token rows into expert-sorted rows, the repository's prefill of 512 tokens
        dict(name="quant_prefill", op="quant", T=512, H=2048, E=256, k=8, shared=True, fmt="mxfp8"),
        # the same for a decode batch
        dict(name="quant_decode", op="quant", T=16, H=2048, E=256, k=8, shared=True, fmt="mxfp8"),
        # one token through a 4-bit projection: weight streaming
        dict(name="linear_decode", op="linear", T=1, N=4096, K=2048, fmt="nvfp4"),
        # odd sizes: rows that end inside a tile, outputs that end inside a tile
        dict(name="linear_odd", op="linear", T=301, N=1000, K=2176, fmt="mxfp8"),
        # a large prompt through a projection: tensor-core rate
        dict(name="gemm_prefill", op="gemm", T=8192, N=8192, K=4096, fmt="nvfp4"),
        # the repository's layer at its token counts: one token, a prompt, a long prompt
        dict(name="experts_t1", op="experts", T=1, H=2048, I=512, E=256, k=8, shared=True, fmt="nvfp4", skew=0.0),
        dict(name="experts_t512", op="experts", T=512, H=2048, I=512, E=256, k=8, shared=True, fmt="nvfp4", skew=0.0),
        dict(name="experts_t4096", op="experts", T=4096, H=2048, I=512, E=256, k=8, shared=True, fmt="mxfp8", skew=0.3),
    ]


def _odd(rng, lo, hi, step=1):
    """An odd multiple of step in [lo, hi], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    m = int(v / step) | 1
    return step * (m if m * step <= hi else m - 2)


def draw(rng):
    op = rng.choice(["norm", "norm_linear", "quant", "linear", "gemm", "experts", "experts"])
    fmt = rng.choice(["nvfp4", "mxfp8"])
    unit = 64 if fmt == "nvfp4" else 128
    if op == "norm":
        H = _odd(rng, 256, 8192, 32)
        return dict(op=op, T=_odd(rng, 1, (32768 * 2048) // H), H=H, fmt="mxfp8")
    if op == "quant":
        return dict(op=op, T=_odd(rng, 1, 2048), H=_odd(rng, 256, 4096, 32), E=rng.choice([16, 64, 256]),
                    k=rng.randint(1, 8), shared=rng.random() < 0.5, fmt="mxfp8")
    if op == "experts":
        return dict(op=op, T=_odd(rng, 1, 4096), H=_odd(rng, 256, 2048, unit), I=_odd(rng, 128, 512, unit),
                    E=rng.choice([16, 64, 256]), k=rng.randint(1, 8), shared=rng.random() < 0.5, fmt=fmt,
                    skew=round(rng.uniform(0.0, 0.3), 2))
    T, N, K = _odd(rng, 1, 8192), _odd(rng, 64, 8192, 8), _odd(rng, 256, 4096, unit)
    if op == "norm_linear":
        return dict(op=op, T=T, H=K, N=N, fmt=fmt)
    return dict(op=op, T=T, N=N, K=K, fmt=fmt)


# ---------------------------------------------------------------- sizes


def _block(fmt):
    return 16 if fmt == "nvfp4" else 32


def _row_bytes(fmt, n):
    """Codes and scales of a row."""
    return n * (1 if fmt == "mxfp8" else 0.5) + n / _block(fmt) + (4 if fmt == "nvfp4" else 0)


def _weight_fmt(fmt):
    return "mxfp4" if fmt == "mxfp8" else fmt


def _tiles(n, fmt):
    return -(-(n // _block(fmt)) // 4)


def work(case):
    op, T, fmt = case["op"], case["T"], case["fmt"]
    wf = _weight_fmt(fmt)
    if op == "norm":
        H = case["H"]
        return {"bytes": T * (8 * H + _row_bytes(fmt, H)) + 2 * H, "flops": 6 * T * H}
    if op == "quant":
        H, copies = case["H"], case["k"] + case["shared"]
        return {"bytes": T * (2 * H + copies * _row_bytes(fmt, H) + 8 * case["k"]), "flops": 3 * T * H}
    if op == "norm_linear":
        H, N = case["H"], case["N"]
        return {"bytes": T * (6 * H + 2 * N) + N * _row_bytes(wf, H), "flops": 2 * T * N * H}
    if op in ("linear", "gemm"):
        N, K = case["N"], case["K"]
        return {"bytes": T * ((2 * K if op == "linear" else _row_bytes(fmt, K)) + 2 * N) + N * _row_bytes(wf, K),
                "flops": 2 * T * N * K}
    H, I, E, k = case["H"], case["I"], case["E"], case["k"]
    rows = T * (k + case["shared"])
    active = E * (1.0 - (1.0 - k / E) ** T) + case["shared"]        # expected number of experts with a token
    return {"bytes": active * (2 * I * _row_bytes(wf, H) + H * _row_bytes(wf, I)) + rows * (_row_bytes(fmt, H) + 2 * H),
            "flops": 6 * rows * H * I}


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


def _weights(G, N, K, fmt, g):
    """A stack of G matrices [N, K]: codes, scale tiles and a factor per matrix, so that outputs are of the inputs' size."""
    w = {"codes": torch.randint(0, 256, (G, N, K // 2), dtype=torch.uint8, generator=g, device=DEV)}
    n = G * -(-N // 128) * _tiles(K, fmt) * 512
    if fmt == "nvfp4":
        w["scales"] = torch.randint(0x30, 0x40, (n,), dtype=torch.uint8, generator=g, device=DEV)
        w["alpha"] = (0.8 + 0.4 * torch.rand(G, generator=g, device=DEV)) / (3.3 * math.sqrt(K))
    else:
        e = 127 - round(math.log2(2.9 * math.sqrt(K)))
        w["scales"] = torch.randint(e - 1, e + 2, (n,), dtype=torch.uint8, generator=g, device=DEV)
        w["alpha"] = None
    return w


def _routing(T, E, k, skew, g):
    logits = torch.randn(T, E, generator=g, device=DEV) + skew * torch.randn(1, E, generator=g, device=DEV)
    ids = logits.topk(k, dim=1).indices.int().contiguous()
    flat = ids.reshape(-1).long()
    perm = torch.argsort(flat, stable=True)
    inv = torch.empty_like(perm)
    inv[perm] = torch.arange(T * k, device=DEV)
    counts = torch.bincount(flat, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = counts.cumsum(0)
    return {"ids": ids, "perm": perm.int(), "inv_perm": inv.int(), "offsets": offsets, "cap": int(counts.max())}


def _rows(R, n, groups, fmt):
    """Room for R rows of n elements in block-scaled form, the rows in `groups` groups."""
    return {"codes": torch.zeros(R, n if fmt == "mxfp8" else n // 2, dtype=torch.uint8, device=DEV),
            "scales": torch.zeros((R // 128 + groups) * _tiles(n, fmt) * 512, dtype=torch.uint8, device=DEV),
            "row_scale": torch.zeros(R, device=DEV) if fmt == "nvfp4" else None}


def prepare(case, seed):
    op, T, fmt, g = case["op"], case["T"], case["fmt"], _gen(seed)
    wf = _weight_fmt(fmt)
    st = {"case": dict(case), "ws": torch.zeros(WS_BYTES, dtype=torch.uint8, device=DEV)}
    if op in ("norm", "norm_linear"):
        H = case["H"]
        st["x"] = _activations(T, H, g)
        st["residual"] = 3 * _activations(T, H, g)
        st["weight"] = (1 + 0.2 * torch.randn(H, generator=g, device=DEV)).bfloat16()
        st["sum"] = torch.empty_like(st["x"])
        st["q"] = _rows(T, H, 1, fmt)
        st["y"] = torch.empty_like(st["x"]) if op == "norm" else None
    if op == "norm_linear":
        st["w"] = _weights(1, case["N"], case["H"], wf, g)
        st["out"] = torch.empty(T, case["N"], dtype=torch.bfloat16, device=DEV)
    if op == "quant":
        st["x"] = _activations(T, case["H"], g)
        st["routing"] = _routing(T, case["E"], case["k"], 0.3, g)
        st["q"] = _rows(T * (case["k"] + case["shared"]), case["H"], case["E"] + case["shared"], fmt)
    if op in ("linear", "gemm"):
        N, K = case["N"], case["K"]
        st["x"] = _activations(T, K, g)
        st["q"] = _rows(T, K, 1, fmt)
        if op == "gemm":
            _plain_quantise_into(st["x"].float(), fmt, st["q"], torch.arange(T, device=DEV), torch.arange(T, device=DEV))
        st["w"] = _weights(1, N, K, wf, g)
        st["out"] = torch.empty(T, N, dtype=torch.bfloat16, device=DEV)
    if op == "experts":
        H, I, E, k, sh = case["H"], case["I"], case["E"], case["k"], int(case["shared"])
        G, R = E + sh, T * (k + sh)
        r = st["routing"] = _routing(T, E, k, case["skew"], g)
        x = _activations(T, H, g).float()
        st["q"] = _rows(R, H, G, fmt)
        token = torch.cat([r["perm"].long() // k, torch.arange(T, device=DEV)[:T * sh]])
        _plain_quantise_into(x[token], fmt, st["q"], torch.arange(R, device=DEV), _scale_rows(r["offsets"], R, G))
        st["gate"], st["up"] = _weights(G, I, H, wf, g), _weights(G, I, H, wf, g)
        st["down"] = _weights(G, H, I, wf, g)
        # the calibrated size of h: a row's largest value near 2688 h_scale
        st["h_scale"] = torch.full((G,), 1.0 / 256, device=DEV) if fmt == "nvfp4" else None
        if fmt == "nvfp4":
            st["down"]["alpha"] *= 1.0 / 256                         # a program folds it into the matrices' factor
        st["h"] = _rows(R, I, G, fmt)
        st["h"]["row_scale"] = None
        st["out"] = torch.empty(R, H, dtype=torch.bfloat16, device=DEV)
    return st


# ---------------------------------------------------------------- plain form


def _scale_rows(offsets, R, G):
    """Row of the scale tiles for each of R grouped rows: group g starts at row tile offsets[g] // 128 + g."""
    p = torch.arange(R, device=DEV)
    start = offsets[:G].long()
    gid = torch.searchsorted(start, p, right=True) - 1
    return (start[gid] // 128 + gid) * 128 + p - start[gid]


def _e2m1_code(v):
    a = v.abs()
    c = (a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte()
    c = c + (a > 2.5).byte() + (a >= 3.5).byte() + (a > 5.0).byte()
    return c + 8 * torch.signbit(v).byte()


def _e2m1_value(codes):
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0.0, -.5, -1, -1.5, -2, -3, -4, -6], device=DEV)
    return table[codes.long()]


def _pow2(e):
    """2^e in 32 bits, exactly, for integers -127 <= e <= 127."""
    return torch.where(e > -127, (e.clamp_min(-126) + 127).int() << 23, torch.full_like(e, 1 << 22, dtype=torch.int32)).view(torch.float32)


def _pow2_exponent(amax, top, top_exp):
    """Smallest e with amax <= top * 2^e (top = m * 2^top_exp, 1 <= m < 2), within what E8M0 holds."""
    m, e = torch.frexp(amax)                                         # amax = m 2^e, 0.5 <= m < 1
    e = e - 1 - top_exp + (2 * m > top / 2 ** top_exp).int()
    return torch.where(amax > 0, e.clamp(-127, 127), torch.full_like(e, -127))


def _plain_quantise(v, fmt, g=None):
    """Codes, scale bytes [R, n / block] and the fp32 factor per row of rows v (32 bits).  g: a given factor per row."""
    R, n = v.shape
    b = v.reshape(R, n // _block(fmt), _block(fmt))
    amax = b.abs().amax(2)
    if fmt == "nvfp4":
        if g is None:
            g = (v.abs().amax(1) / 2688).clamp_min(2.0 ** -110)
        ginv = (1 / g)[:, None]
        s = (amax * ginv * torch.tensor(1 / 6, dtype=torch.float32, device=DEV)).clamp_max(448).to(torch.float8_e4m3fn)
        sf = s.float()
        inv = torch.where(sf > 0, ginv / sf, torch.zeros_like(sf))
        return _e2m1_code(b * inv[:, :, None]).reshape(R, n), s.view(torch.uint8), g
    top, top_exp = (448.0, 8) if fmt == "mxfp8" else (6.0, 2)
    e = _pow2_exponent(amax, top, top_exp)
    q = (b * _pow2(-e)[:, :, None]).reshape(R, n)
    if fmt == "mxfp8":
        return q.to(torch.float8_e4m3fn).view(torch.uint8), (e + 127).byte(), None
    return _e2m1_code(q), (e + 127).byte(), None


def _plain_quantise_into(v, fmt, q, rows, scale_rows):
    """Row i of v into row rows[i] of q, its scales into row scale_rows[i] of the tiles."""
    codes, s, g = _plain_quantise(v, fmt)
    q["codes"][rows] = codes if fmt == "mxfp8" else codes[:, 0::2] | (codes[:, 1::2] << 4)
    tiles = q["scales"].view(-1, _tiles(v.shape[1], fmt), 32, 4, 4)
    full = torch.zeros(tiles.shape[0] * 128, tiles.shape[1] * 4, dtype=torch.uint8, device=DEV)
    full[scale_rows, :s.shape[1]] = s
    tiles.copy_(full.view(tiles.shape[0], 4, 32, tiles.shape[1], 4).permute(0, 3, 2, 1, 4))
    if fmt == "nvfp4":
        q["row_scale"][rows] = g


def _scale_value(s, fmt):
    if fmt == "nvfp4":
        return s.view(torch.float8_e4m3fn).float()
    return _pow2(s.int() - 127)


def _untile(scales, fmt, n):
    """[row tiles * 128, n / block] scale bytes from the tiles."""
    t = scales.view(-1, _tiles(n, fmt), 32, 4, 4)
    return t.permute(0, 3, 2, 1, 4).reshape(t.shape[0] * 128, -1)[:, :n // _block(fmt)]


def _values(codes, scale, fmt):
    """codes [..., n or n / 2] times scale values [..., n / block], in 32 bits."""
    v = codes.view(torch.float8_e4m3fn).float() if fmt == "mxfp8" else \
        _e2m1_value(torch.stack([codes & 15, codes >> 4], -1).flatten(-2))
    return (v.view(*v.shape[:-1], -1, _block(fmt)) * scale[..., None]).view(v.shape)


def _plain_rows(q, fmt, n, scale_rows):
    v = _values(q["codes"], _scale_value(_untile(q["scales"], fmt, n)[scale_rows], fmt), fmt)
    return v if q["row_scale"] is None else v * q["row_scale"][:, None]


def _plain_weights(w, fmt, n):
    G, N = w["codes"].shape[:2]
    s = _untile(w["scales"], fmt, n).view(G, -1, n // _block(fmt))[:, :N]
    v = _values(w["codes"], _scale_value(s, fmt), fmt)
    return v if w["alpha"] is None else v * w["alpha"][:, None, None]


def _plain_grouped(a, w, r, E):
    """a [R, K] in expert-sorted rows, w [G, N, K]: a's rows times their group's matrix."""
    Tk = r["ids"].numel()
    p = torch.arange(Tk, device=DEV)
    start = r["offsets"][:E].long()
    gid = torch.searchsorted(start, p, right=True) - 1
    pad = torch.zeros(E, r["cap"], a.shape[1], device=DEV)
    pad[gid, p - start[gid]] = a[:Tk]
    y = torch.bmm(pad, w[:E].transpose(1, 2))[gid, p - start[gid]]
    return y if a.shape[0] == Tk else torch.cat([y, a[Tk:] @ w[E].t()])


def _plain_norm(st):
    s = (st["x"].float() + st["residual"].float()).bfloat16()
    f = s.float()
    return s, f * torch.rsqrt(f.square().mean(1, keepdim=True) + EPS) * st["weight"].float()


def _plain(st):
    c = st["case"]
    op, T, fmt = c["op"], c["T"], c["fmt"]
    wf = _weight_fmt(fmt)
    if op in ("norm", "norm_linear"):
        s, y = _plain_norm(st)
        rows = torch.arange(T, device=DEV)
        _plain_quantise_into(y, fmt, st["q"], rows, rows)
        if op == "norm":
            return {"sum": s, "y": y.bfloat16(), **_codes_out(st["q"])}
        a = _plain_rows(st["q"], fmt, c["H"], rows)
        return {"sum": s, "out": (a @ _plain_weights(st["w"], wf, c["H"])[0].t()).bfloat16()}
    if op == "quant":
        r, k, sh = st["routing"], c["k"], int(c["shared"])
        R, G = T * (k + sh), c["E"] + sh
        token = torch.cat([r["perm"].long() // k, torch.arange(T, device=DEV)[:T * sh]])
        _plain_quantise_into(st["x"].float()[token], fmt, st["q"], torch.arange(R, device=DEV),
                             _scale_rows(r["offsets"], R, G))
        return _codes_out(st["q"])
    if op in ("linear", "gemm"):
        rows = torch.arange(T, device=DEV)
        if op == "linear":
            _plain_quantise_into(st["x"].float(), fmt, st["q"], rows, rows)
        a = _plain_rows(st["q"], fmt, c["K"], rows)
        return (a @ _plain_weights(st["w"], wf, c["K"])[0].t()).bfloat16()
    r, E, G, R = st["routing"], c["E"], c["E"] + int(c["shared"]), st["out"].shape[0]
    a = _plain_rows(st["q"], fmt, c["H"], _scale_rows(r["offsets"], R, G))
    gate = _plain_grouped(a, _plain_weights(st["gate"], wf, c["H"]), r, E)
    up = _plain_grouped(a, _plain_weights(st["up"], wf, c["H"]), r, E)
    h = gate / (1 + torch.exp(-gate)) * up
    g = None if st["h_scale"] is None else st["h_scale"][0].expand(R)
    codes, s, g = _plain_quantise(h, fmt, g)
    packed = codes if fmt == "mxfp8" else codes[:, 0::2] | (codes[:, 1::2] << 4)
    h = _values(packed.contiguous(), _scale_value(s, fmt), fmt)
    return _plain_grouped(h, _plain_weights(st["down"], wf, c["I"]), r, E).bfloat16()


def _codes_out(q):
    return {"codes": q["codes"].view(torch.float8_e4m3fn), "scales": q["scales"].view(torch.float8_e8m0fnu)}


# ---------------------------------------------------------------- the framework's kernels


def _handles(qm, st):
    """The descriptors of block-scaled rows and weights that a program makes once for its buffers."""
    d = {n: qm.scaled_rows(st[n]["codes"], st[n]["scales"], st[n]["row_scale"]) for n in ("q", "h") if n in st}
    d |= {n: qm.scaled_mat(st[n]["codes"], st[n]["scales"], st[n]["alpha"]) for n in ("w", "gate", "up", "down") if n in st}
    return d


def _own(st):
    import quantised_moe_expert_gb300 as qm
    if "handles" not in st:
        st["handles"] = _handles(qm, st)
    c, ws, d = st["case"], st["ws"], st["handles"]
    op, T = c["op"], c["T"]
    fmt = qm.MOE_SCALED_NVFP4 if c["fmt"] == "nvfp4" else qm.MOE_SCALED_MXFP8
    if op in ("norm", "norm_linear"):
        qm.moe_add_rmsnorm(st["x"], st["residual"], st["weight"], 0.0, EPS, T, c["H"], st["sum"], st["y"], fmt, d["q"])
        if op == "norm":
            return {"sum": st["sum"], "y": st["y"], **_codes_out(st["q"])}
        qm.moe_scaled_gemm(fmt, d["q"], d["w"], T, c["N"], c["H"], 1, None, st["out"], ws)
        return {"sum": st["sum"], "out": st["out"]}
    if op == "quant":
        r = st["routing"]
        qm.moe_quantize_routed(fmt, st["x"], T, c["H"], c["k"], c["E"], int(c["shared"]), r["ids"], r["inv_perm"],
                               r["offsets"], d["q"], ws)
        return _codes_out(st["q"])
    if op in ("linear", "gemm"):
        if op == "linear":
            qm.moe_quantize(fmt, st["x"], T, c["K"], 1, None, d["q"])
        qm.moe_scaled_gemm(fmt, d["q"], d["w"], T, c["N"], c["K"], 1, None, st["out"], ws)
        return st["out"]
    G, R, offsets = c["E"] + int(c["shared"]), st["out"].shape[0], st["routing"]["offsets"]
    qm.moe_scaled_swiglu(fmt, d["q"], d["gate"], d["up"], R, c["I"], c["H"], G, offsets, st["h_scale"], d["h"], ws)
    qm.moe_scaled_gemm(fmt, d["h"], d["down"], R, c["H"], c["I"], G, offsets, st["out"], ws)
    return st["out"]


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- the definition in 64 bits


def _x_pow2(e):
    """2^e in 64 bits, exactly, for integers e held as floating-point numbers."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _x_round(v, mant, min_exp, top):
    """v to the nearest value with `mant` fraction bits and no exponent below min_exp, ties to even, at most top."""
    e = torch.floor(torch.log2(v.abs().clamp_min(1e-300))).clamp_min(min_exp)
    step = _x_pow2(e - mant)
    return (torch.round(v / step) * step).clamp(-top, top)


def _x_quantise(v, fmt, g=None):
    """Element values, scale values and row factors, all in 64 bits."""
    R, n = v.shape
    b = v.reshape(R, -1, _block(fmt))
    top = b.abs().max(2).values
    if fmt == "nvfp4":
        g = (v.abs().max(1).values / 2688).clamp_min(2.0 ** -110) if g is None else g
        s = _x_round(top / g[:, None] / 6, 3, -6, 448.0)
        q = torch.where(s[:, :, None] > 0, b / (g[:, None] * s).clamp_min(1e-300)[:, :, None], torch.zeros_like(b))
        return _x_round(q, 1, 0, 6.0), s, g
    limit = 448.0 if fmt == "mxfp8" else 6.0
    e = torch.ceil(torch.log2(top.clamp_min(1e-300) / limit)).clamp(-1000, 1000)
    e = torch.where(top > limit * _x_pow2(e), e + 1, e)
    e = torch.where(top <= limit * _x_pow2(e - 1), e - 1, e).clamp(-127, 127)
    s = _x_pow2(e)
    q = b / s[:, :, None]
    return (_x_round(q, 3, -6, 448.0) if fmt == "mxfp8" else _x_round(q, 1, 0, 6.0)), s, None


def _x_dequant(v, fmt):
    q, s, g = _x_quantise(v, fmt)
    q = (q * s[:, :, None]).reshape(v.shape)
    return q if g is None else q * g[:, None]


def _x_scales(raw, row0, rows, n, fmt):
    """Scale values of `rows` rows from row row0 on, read from the tiles one byte at a time."""
    nb = n // _block(fmt)
    r = row0 + torch.arange(rows, device=DEV)[:, None]
    b = torch.arange(nb, device=DEV)[None, :]
    at = ((r // 128) * _tiles(n, fmt) + b // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4
    s = raw[at].long()
    if fmt != "nvfp4":
        return _x_pow2(s - 127)
    e, m = s >> 3, (s & 7).double()
    return torch.where(e > 0, (8 + m) * _x_pow2(e - 10), m * 2.0 ** -9)


def _x_codes(c, fmt):
    if fmt == "mxfp8":
        c = c.long()
        e, m = (c >> 3) & 15, (c & 7).double()
        v = torch.where(e > 0, (8 + m) * _x_pow2(e - 10), m * 2.0 ** -9)
        return torch.where(c >= 128, -v, v)
    c = torch.stack([c & 15, c >> 4], -1).flatten(-2).long()
    e, m = (c >> 1) & 3, (c & 1).double()
    v = torch.where(e > 0, (2 + m) * _x_pow2(e - 2), m * 0.5)
    return torch.where(c >= 8, -v, v)


def _x_matrix(w, i, fmt, n):
    N = w["codes"].shape[1]
    s = _x_scales(w["scales"], i * -(-N // 128) * 128, N, n, fmt)
    v = _x_codes(w["codes"][i], fmt).view(N, -1, _block(fmt)) * s[:, :, None]
    return v.view(N, n) * (1.0 if w["alpha"] is None else w["alpha"][i].double())


def _x_tiled(s, scale_rows, row_tiles, col_tiles):
    """Scale values in tile order, the value of a zero byte (2^-127) where there is no row."""
    out = torch.full((row_tiles * col_tiles * 512,), 2.0 ** -127, dtype=torch.float64, device=DEV)
    r, b = scale_rows[:, None], torch.arange(s.shape[1], device=DEV)[None, :]
    out[((r // 128) * col_tiles + b // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4] = s
    return out


def exact(case, seed):
    st = prepare(case, seed)
    op, T, fmt = case["op"], case["T"], case["fmt"]
    wf = _weight_fmt(fmt)
    if op in ("norm", "norm_linear"):
        s = (st["x"].double() + st["residual"].double()).to(torch.bfloat16).double()
        y = s / torch.sqrt((s * s).mean(1, keepdim=True) + EPS) * st["weight"].double()
        if op == "norm_linear":
            return {"sum": s, "out": _x_dequant(y, fmt) @ _x_matrix(st["w"], 0, wf, case["H"]).t()}
        q, sc, _ = _x_quantise(y, fmt)
        return {"sum": s, "y": y, "codes": q.reshape(T, -1),
                "scales": _x_tiled(sc, torch.arange(T, device=DEV), T // 128 + 1, _tiles(case["H"], fmt))}
    if op == "quant":
        r, k, E = st["routing"], case["k"], case["E"]
        q, sc, _ = _x_quantise(st["x"].double(), fmt)
        R = T * (k + case["shared"])
        codes = torch.zeros(R, case["H"], dtype=torch.float64, device=DEV)
        at = r["inv_perm"].long()
        group = r["ids"].reshape(-1).long()
        start = r["offsets"].long()
        tok = torch.arange(T, device=DEV).repeat_interleave(k)
        srow = (start[group] // 128 + group) * 128 + at - start[group]
        if case["shared"]:
            at = torch.cat([at, T * k + torch.arange(T, device=DEV)])
            srow = torch.cat([srow, (T * k // 128 + E) * 128 + torch.arange(T, device=DEV)])
            tok = torch.cat([tok, torch.arange(T, device=DEV)])
        codes[at] = q.reshape(T, -1)[tok]
        return {"codes": codes, "scales": _x_tiled(sc[tok], srow, R // 128 + E + int(case["shared"]), _tiles(case["H"], fmt))}
    if op in ("linear", "gemm"):
        K = case["K"]
        if op == "linear":
            a = _x_dequant(st["x"].double(), fmt)
        else:
            a = _x_codes(st["q"]["codes"], fmt).view(T, -1, _block(fmt)) * _x_scales(st["q"]["scales"], 0, T, K, fmt)[:, :, None]
            a = a.view(T, K) * (1.0 if fmt != "nvfp4" else st["q"]["row_scale"].double()[:, None])
        return a @ _x_matrix(st["w"], 0, wf, K).t()
    H, I, E = case["H"], case["I"], case["E"]
    R, q = st["out"].shape[0], st["q"]
    out = torch.zeros(R, H, dtype=torch.float64, device=DEV)
    starts = st["routing"]["offsets"].tolist()
    bounds = [(i, starts[i], starts[i + 1]) for i in range(E)] + ([(E, starts[E], R)] if case["shared"] else [])
    for i, lo, hi in bounds:
        if lo == hi:
            continue
        a = _x_codes(q["codes"][lo:hi], fmt).view(hi - lo, -1, _block(fmt))
        a = (a * _x_scales(q["scales"], (lo // 128 + i) * 128, hi - lo, H, fmt)[:, :, None]).view(hi - lo, H)
        if fmt == "nvfp4":
            a = a * q["row_scale"][lo:hi].double()[:, None]
        g, u = a @ _x_matrix(st["gate"], i, wf, H).t(), a @ _x_matrix(st["up"], i, wf, H).t()
        h = g * torch.sigmoid(g) * u
        hs = None if st["h_scale"] is None else st["h_scale"][i].double().expand(hi - lo)
        qv, sc, _ = _x_quantise(h, fmt, hs)
        h = (qv * sc[:, :, None]).reshape(h.shape)
        out[lo:hi] = h @ _x_matrix(st["down"], i, wf, I).t()
    return out
