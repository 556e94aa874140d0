"""Reference of the gated linear recurrence in fp64 numpy, with elementwise
error bounds, for its tests.

Bounds.  Write u = 2^-24 (half a step of fp32).  Whatever order the affine
maps h -> g h + x are composed in, the computed h_t is a sum over j <= t of
x_j g_{j+1} ... g_t in which every term has passed a number of roundings: at
most two per token on its way (one for the running state or B, one for the
product A), plus one each where a wave's, a tile's and the chain's maps are
applied and where x itself is folded in.  With the count 2 (t - j) + 6 the
error is at most 1.01 u W_t, where
    M_t = |g_t| M_{t-1} + |x_t|                        (sum of magnitudes)
    W_t = |g_t| (W_{t-1} + 2 M_{t-1}) + 6 |x_t|        (weighted by the count)
and the initial state enters like an x before the first token.  The backward
recurrence d_t = dy_t + g_{t+1} d_{t+1} has the same bound in reverse.  Storing
in a type of half step r adds r |value| (r = 2^-8 bf16, 2^-11 fp16), and half
the smallest subnormal.
"""
from __future__ import annotations

import numpy as np
import torch

U32 = 2.0 ** -24
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11,
             torch.float8_e4m3fn: 2.0 ** -4, torch.float8_e5m2: 2.0 ** -3}
TINY = {torch.float32: 2.0 ** -126, torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -25,
        torch.float8_e4m3fn: 2.0 ** -10, torch.float8_e5m2: 2.0 ** -17}


def f64(t):
    return None if t is None else t.detach().to("cpu").to(torch.float32).numpy().astype(np.float64)


def stored(value, err, dtype):
    """Bound of a value with error err once it is stored in dtype."""
    return err + HALF_STEP[dtype] * (np.abs(value) + err) + TINY[dtype]


def wide(g, shape):
    """Gate [T, H] or [T, H, D] as [T, H, D]."""
    return np.broadcast_to(g[..., None] if g.ndim == 2 else g, shape)


def forward(x, g, lens, h0=None, begin=0):
    """(h, err, final, final_err) of sequences of the given lengths from row
    ``begin`` on; rows outside are NaN."""
    g = wide(g, x.shape)
    h, err = np.full(x.shape, np.nan), np.full(x.shape, np.nan)
    final = np.zeros((len(lens),) + x.shape[1:])
    ferr = np.zeros_like(final)
    t = begin
    for i, n in enumerate(lens):
        s = np.zeros(x.shape[1:]) if h0 is None else h0[i].copy()
        m, w = np.abs(s), 6 * np.abs(s)
        if n == 0:
            w = np.zeros_like(m)
        for _ in range(n):
            a = np.abs(g[t])
            s = g[t] * s + x[t]
            w = a * (w + 2 * m) + 6 * np.abs(x[t])
            m = a * m + np.abs(x[t])
            h[t], err[t] = s, 1.01 * U32 * w
            t += 1
        final[i], ferr[i] = s, 1.01 * U32 * w
    return h, err, final, ferr


def backward(dy, x, g, lens, h0=None, dfinal=None, begin=0):
    """dict of dx, dg, dh0 as (value, err); rows outside are zero."""
    per_head = g.ndim == 2
    gw = wide(g, x.shape)
    h, herr, _, _ = forward(x, g, lens, h0, begin)
    dx, dxe = np.zeros_like(x), np.zeros_like(x)
    dg, dge = np.zeros_like(x), np.zeros_like(x)
    dh0 = np.zeros((len(lens),) + x.shape[1:])
    dh0e = np.zeros_like(dh0)
    zero = np.zeros(x.shape[1:])
    t = begin
    for i, n in enumerate(lens):
        k = zero if dfinal is None else dfinal[i].copy()
        m, w = np.abs(k), (6 if n else 0) * np.abs(k)
        kerr = 1.01 * U32 * w
        for j in range(t + n - 1, t - 1, -1):
            d = dy[j] + k
            m = m + np.abs(dy[j])
            w = w + 6 * np.abs(dy[j])
            dx[j], dxe[j] = d, 1.01 * U32 * (w + m)
            if j > t:
                before, be = h[j - 1], herr[j - 1]
            else:
                before, be = (zero if h0 is None else h0[i]), zero
            dg[j] = d * before
            dge[j] = np.abs(d) * be + dxe[j] * (np.abs(before) + be) + U32 * np.abs(dg[j])
            a = np.abs(gw[j])
            k = gw[j] * d
            w = a * (w + 2 * m)
            m = a * m
            kerr = 1.01 * U32 * (w + m)
        dh0[i], dh0e[i] = k, kerr
        t += n
    if per_head:
        # at most 4 in-lane and 5 cross-lane additions: 9 roundings of partial sums
        dge = dge.sum(-1) + 9 * U32 * (np.abs(dg) + dge).sum(-1)
        dg = dg.sum(-1)
    return {"dx": (dx, dxe), "dg": (dg, dge), "dh0": (dh0, dh0e)}


def check(name, got, want, err, dtype):
    """Every element within the bound of a value of error err stored in dtype."""
    got = f64(got)
    lim = stored(want, err, dtype)
    bad = ~(np.abs(got - want) <= lim)
    if bad.any():
        at = np.unravel_index(np.argmax(np.where(bad, np.abs(got - want) / lim, 0)), got.shape)
        raise AssertionError("%s: %d of %d outside the bound, worst at %s: got %r want %r limit %r"
                             % (name, bad.sum(), bad.size, at, got[at], want[at], lim[at]))


def make(seed, lens, H, D, dtype=torch.float32, gate=torch.float32, per_head=False, h0=True,
         tail=0, device="cuda"):
    """Inputs of a packed batch with ``tail`` rows behind the last sequence."""
    gen = torch.Generator().manual_seed(seed)
    T, N = sum(lens) + tail, len(lens)
    x = torch.randn((T, H, D), generator=gen).to(dtype)
    shape = (H,) if per_head else (H, D)
    rate = torch.exp(-7.0 * torch.rand(shape, generator=gen))
    z = torch.randn((T,) + shape, generator=gen)
    g = torch.exp(-rate * torch.nn.functional.softplus(z)).to(gate)
    d = {"x": x, "g": g, "cu": torch.tensor([0] + lens).cumsum(0).to(torch.int32),
         "h0": torch.randn((N, H, D), generator=gen) if h0 else None,
         "dy": torch.randn((T, H, D), generator=gen).to(dtype),
         "dfinal": torch.randn((N, H, D), generator=gen)}
    return {k: v if v is None else v.to(device) for k, v in d.items()}
