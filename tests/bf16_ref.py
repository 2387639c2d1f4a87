"""The 16-bit operators' definitions in 64 bits, and inputs for their tests.

A rounding to bf16 is off by at most 2^-8 of the value (BF16), one to fp32 by 2^-24.  A product of K terms, summed in fp32 in
any order and with each addition rounded or truncated, is off by at most K 2^-23 of the sum of the terms' magnitudes."""
import math

import torch

BF16 = 2.0 ** -8


def bf16(*shape, seed=0, size=1.0, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return (size * torch.randn(*shape, generator=g, device=device)).bfloat16()


def act(name, v):
    """Value and derivative."""
    if name == "none":
        return v, torch.ones_like(v)
    if name == "relu":
        return v.clamp_min(0), (v > 0).to(v.dtype)
    if name == "gelu":
        c = math.sqrt(2 / math.pi)
        th = torch.tanh(c * (v + 0.044715 * v ** 3))
        return 0.5 * v * (1 + th), 0.5 * (1 + th) + 0.5 * v * (1 - th * th) * c * (1 + 3 * 0.044715 * v * v)
    s = torch.sigmoid(v)
    return (v * s, s * (1 + v * (1 - s))) if name == "silu" else (s, s * (1 - s))


#: The largest slope of a function, and how far its value is off where the fast exponential is (of the argument's size).
SLOPE, FUNCTION = 1.13, 2.0 ** -20


def offsets_of(counts, device="cuda", first=0):
    at, out = first, []
    for c in counts:
        out.append(at)
        at += c
    return torch.tensor(out, dtype=torch.int32, device=device), at


def groups(counts, first=0):
    at = first
    for g, c in enumerate(counts):
        yield g, slice(at, at + c)
        at += c


def product(a, w, counts, first=0, transposed=False):
    """Grouped product and the sum of its terms' magnitudes; rows of no group are zero."""
    N = w.shape[2] if transposed else w.shape[1]
    y = torch.zeros(a.shape[0], N, dtype=torch.float64, device=a.device)
    s = torch.zeros_like(y)
    for g, r in groups(counts, first):
        m = w[g].double() if transposed else w[g].double().t()
        y[r] = a[r].double() @ m
        s[r] = a[r].double().abs() @ m.abs()
    return y, s


def outer(dy, x, counts, first=0):
    w = torch.zeros(len(counts), dy.shape[1], x.shape[1], dtype=torch.float64, device=dy.device)
    s = torch.zeros_like(w)
    b = torch.zeros(len(counts), dy.shape[1], dtype=torch.float64, device=dy.device)
    t = torch.zeros_like(b)
    for g, r in groups(counts, first):
        d, v = dy[r].double(), x[r].double()
        w[g], s[g] = d.t() @ v, d.abs().t() @ v.abs()
        b[g], t[g] = d.sum(0), d.abs().sum(0)
    return w, s, b, t


def within(got, want, tol):
    """Every element of `got` within `tol` of `want`."""
    err = (got.double() - want).abs() - tol
    assert bool((err <= 0).all()), f"largest excess {float(err.max())}, {int((err > 0).sum())} of {err.numel()} elements"
