"""References of the short convolution and the selective scan in fp64 numpy,
with a bound for every element, for their tests.

Bounds.  Every value is carried with a bound of the error that fp32 arithmetic
can have made on it (class E): u = 2^-24 is half a step relative to a result,
and a product or sum adds u of its own result to what its operands bring.
exp2, log2 and 1 / x of the GPU are off by at most one step (2 u); an exponent
that is itself off by d makes its power relatively off by d (of the natural
one).  A sum of n terms, in whatever order, is off by at most n u of the sum of
their magnitudes.  The scan composes up to 256 tokens' decays as exp(A sum d):
the sum's own roundings move the exponent by at most 256 u of itself, which is
added to every token's decay (TILE).  Storing in a type of half step r adds
r |value| and half its smallest subnormal.  A value beyond fp32's range, 2^128,
is infinite there or not by the order of its products (h exp(a) exp(b) against
h exp(a + b)), so that it and what is formed from it have no bound.
"""
from __future__ import annotations

import numpy as np
import torch

from tests.recurrence_testlib import HALF_STEP, TINY, f64

U = 2.0 ** -24
MOST = 2.0 ** 128
TILE = 256


class E:
    """Values and bounds of their errors."""

    def __init__(self, v, e=None):
        self.v = np.array(v, dtype=np.float64)
        self.e = np.zeros_like(self.v) if e is None else np.array(np.broadcast_to(e, self.v.shape))
        beyond = ~(np.abs(self.v) + self.e < MOST) | np.isnan(self.v)
        if beyond.any():  # (a finite stand-in: it is its bound that says so)
            self.e = np.where(beyond, np.inf, self.e)
            self.v = np.where(beyond, 0.0, self.v)

    @property
    def known(self):
        return np.isfinite(self.e)

    def __getitem__(self, i):
        return E(self.v[i], self.e[i])

    def __mul__(self, o):
        o = o if isinstance(o, E) else E(o)
        v = self.v * o.v
        with np.errstate(invalid="ignore"):
            e = np.abs(self.v) * o.e + np.abs(o.v) * self.e + self.e * o.e
        return E(v, np.where(self.known & o.known, e + U * (np.abs(v) + e), np.inf))

    def __add__(self, o):
        o = o if isinstance(o, E) else E(o)
        v, e = self.v + o.v, self.e + o.e
        return E(v, e + U * (np.abs(v) + e))

    def sum(self, axis, extra=0):
        """A sum in any order, with ``extra`` further roundings of partial sums."""
        mag = (np.abs(self.v) + self.e).sum(axis)
        e = self.e.sum(axis) + (self.v.shape[axis] + extra) * U * mag
        # partial sums, formed of terms with a factor log2(e) < 2, stay in range too
        return E(self.v.sum(axis), np.where(2 * mag < MOST, e, np.inf))


def same(a, b):
    """Equal bit for bit, NaN as well."""
    return a.shape == b.shape and torch.equal(a.contiguous().view(torch.uint8),
                                              b.contiguous().view(torch.uint8))


def power(x, tile=0):
    """e^x, formed as 2^(log2(e) x): the exponent is off by what x is, by its two
    roundings and by ``tile`` of its sum's; one step of the result."""
    with np.errstate(over="ignore", invalid="ignore"):
        v = np.exp(x.v)
        d = x.e + (3 + tile) * U * (np.abs(x.v) + x.e)
        e = v * np.expm1(d) + 2 * U * v * np.exp(d)
    return E(v, np.where(np.isnan(e), np.inf, e))


def sigmoid(x):
    """1 / (1 + e^-x): the sum's rounding and the reciprocal's step."""
    with np.errstate(over="ignore"):
        v = 1 / (1 + np.exp(-x.v))
    # e^-x off by a factor (1 + r) moves the result by at most (1 - v) r of itself
    r = np.expm1(x.e + 3 * U * (np.abs(x.v) + x.e)) + 2 * U
    return E(v, v * ((1 - v) * r + 4 * U))


def silu(x):
    return x * sigmoid(x)


def silu_slope(x):
    """s (1 + x (1 - s))."""
    s = sigmoid(x)
    rest = E(1 - s.v, s.e + U * (1 - s.v))
    return s * (E(np.ones_like(x.v)) + x * rest)


def softplus(x):
    """max(x, 0) + log(1 + e^-|x|); the logarithm's quotient form adds 8 half
    steps at most (logarithm 2, ln 2, three products, a reciprocal 2)."""
    a = E(-np.abs(x.v), x.e)
    p = power(a)
    tail = E(np.log1p(p.v), p.e + 8 * U * np.log1p(p.v))
    return E(np.maximum(x.v, 0), x.e * (x.v > 0)) + tail


def check(name, got, want, dtype):
    """Every element of got within the bound of want once it is stored in dtype."""
    got = f64(got)
    lim = want.e + HALF_STEP[dtype] * (np.abs(want.v) + want.e) + TINY[dtype]
    assert got.shape == want.v.shape, (name, got.shape, want.v.shape)
    bad = ~(np.abs(got - want.v) <= lim) & want.known
    # beyond the type's range: its infinity
    bad &= ~(np.isinf(got) & (np.sign(got) == np.sign(want.v)) &
             (np.abs(want.v) + lim > torch.finfo(dtype).max))
    if bad.any():
        at = np.unravel_index(np.argmax(np.where(bad, np.abs(got - want.v) / lim, 0)), got.shape)
        raise AssertionError("%s: %d of %d outside the bound, worst at %s: got %r want %r limit %r"
                             % (name, bad.sum(), bad.size, at, got[at], want.v[at], lim[at]))


def _starts(lens, begin):
    return [(i, begin + sum(lens[:i]), n) for i, n in enumerate(lens)]


# ---------------------------------------------------------------- convolution

def conv_make(seed, lens, C, W, dtype=torch.float32, wtype=torch.float32, tail=0, device="cuda"):
    gen = torch.Generator().manual_seed(seed)
    T, N = sum(lens) + tail, len(lens)
    d = {"x": torch.randn((T, C), generator=gen).to(dtype),
         "w": (torch.randn((C, W), generator=gen) * W ** -0.5).to(wtype),
         "bias": (0.3 * torch.randn(C, generator=gen)).to(wtype),
         "cu": torch.tensor([0] + lens).cumsum(0).to(torch.int32),
         "h0": torch.randn((N, W - 1, C), generator=gen),
         "dy": torch.randn((T, C), generator=gen).to(dtype),
         "dfinal": torch.randn((N, W - 1, C), generator=gen)}
    return {k: v.to(device) for k, v in d.items()}


def conv_forward(x, w, bias, lens, h0, act, begin=0):
    """(output rows of each sequence as E, final states, pre-activations, windows)."""
    W = w.shape[1]
    out, final, pres, seen = [], [], [], []
    for i, t, n in _starts(lens, begin):
        s = np.concatenate([h0[i] if h0 is not None else np.zeros((W - 1,) + x.shape[1:]),
                            x[t:t + n]])
        terms = np.stack([s[j:j + n] * w[:, j] for j in range(W)] +
                         [np.broadcast_to(0 if bias is None else bias, (n,) + x.shape[1:])])
        pre = E(terms).sum(0)
        out.append(silu(pre) if act else pre)
        final.append(s[n:])
        pres.append(pre)
        seen.append(s)
    return out, final, pres, seen


def conv_backward(dy, x, w, bias, lens, h0, dfinal, act, begin=0):
    """dx [T, C], dw, dbias, dh0 as E; rows outside are zero."""
    W, C = w.shape[1], x.shape[1]
    _, _, pres, seen = conv_forward(x, w, bias, lens, h0, act, begin)
    dx, dh0 = E(np.zeros_like(x)), E(np.zeros((len(lens), W - 1, C)))
    dws, dbs = [], []
    for i, t, n in _starts(lens, begin):
        d = E(dy[t:t + n])
        if act:
            d = d * silu_slope(pres[i])
        v, e, m = (np.zeros((n + W - 1, C)) for _ in range(3))
        for j in range(W):
            p = d * E(np.broadcast_to(w[:, j], d.v.shape))
            v[j:j + n] += p.v
            e[j:j + n] += p.e
            m[j:j + n] += np.abs(p.v)
        if dfinal is not None:
            v[n:] += dfinal[i]
            m[n:] += np.abs(dfinal[i])
        e += (W + 1) * U * (m + e)
        dh0.v[i], dh0.e[i] = v[:W - 1], e[:W - 1]
        dx.v[t:t + n], dx.e[t:t + n] = v[W - 1:], e[W - 1:]
        dws.append([d * E(seen[i][j:j + n]) for j in range(W)])
        dbs.append(d)
    every = lambda parts: E(np.concatenate([p.v for p in parts]), np.concatenate([p.e for p in parts]))  # noqa: E731
    dw = [every([s[j] for s in dws]).sum(0) for j in range(W)]
    return {"dx": dx, "dw": E(np.stack([q.v for q in dw], 1), np.stack([q.e for q in dw], 1)),
            "dbias": every(dbs).sum(0), "dh0": dh0}


# ----------------------------------------------------------------------- scan

def scan_make(seed, lens, C, N, G=1, dtype=torch.float32, plus=True, tail=0, device="cuda"):
    """Step sizes from a few hundredths to one, decay rates from 0.1 to 4."""
    gen = torch.Generator().manual_seed(seed)
    T, n = sum(lens) + tail, len(lens)
    rnd = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    raw = rnd(T, C)
    d = {"x": rnd(T, C).to(dtype), "z": rnd(T, C).to(dtype),
         "delta": (raw if plus else 0.05 + 0.3 * raw.abs()).to(dtype),
         "A": -torch.exp(-2.3 + 3.7 * torch.rand((C, N), generator=gen)),
         "B": rnd(T, G, N).to(dtype), "C": rnd(T, G, N).to(dtype), "D": rnd(C),
         "dbias": -2 + rnd(C), "cu": torch.tensor([0] + lens).cumsum(0).to(torch.int32),
         "h0": rnd(n, C, N), "dy": rnd(T, C).to(dtype), "dfinal": rnd(n, C, N)}
    return {k: v.to(device) for k, v in d.items()}


class Scan:
    """The scan and its gradients; d: fp64 arrays of scan_make's names (None: not
    given)."""

    def __init__(self, d, lens, plus, begin=0):
        self.d, self.lens, self.plus, self.begin = d, lens, plus, begin
        self.T, self.C = d["x"].shape
        self.N, self.G = d["A"].shape[1], d["B"].shape[1]
        self.of = np.arange(self.C) // (self.C // self.G)
        raw = E(d["delta"])
        self.raw = raw if d["dbias"] is None else raw + E(d["dbias"])
        self.dt = softplus(self.raw) if plus else self.raw
        self.u = self.dt * E(d["x"])
        self.forward()

    def decay(self, t):
        return power(self.dt[t][:, None] * E(self.d["A"]), TILE)

    def forward(self):
        d = self.d
        self.h, self.final = {}, []
        y, ye = np.zeros((self.T, self.C)), np.zeros((self.T, self.C))
        for i, t0, n in _starts(self.lens, self.begin):
            h = E(np.zeros((self.C, self.N)) if d["h0"] is None else d["h0"][i])
            self.h[t0 - 1, i] = h
            for t in range(t0, t0 + n):
                h = self.decay(t) * h + self.u[t][:, None] * E(d["B"][t][self.of])
                self.h[t, i] = h
                s = (h * E(d["C"][t][self.of])).sum(-1, 2)
                if d["D"] is not None:
                    s = s + E(d["D"]) * E(d["x"][t])
                y[t], ye[t] = s.v, s.e
            self.final.append(h)
        self.y = E(y, ye)
        self.out = self.y if d["z"] is None else self.y * silu(E(d["z"]))

    def backward(self):
        d, C, N, T = self.d, self.C, self.N, self.T
        dy = E(d["dy"])
        dz = None
        if d["z"] is not None:
            z = E(d["z"])
            dz = dy * self.y * silu_slope(z)
            dy = dy * silu(z)
        dx, dd = E(np.zeros((T, C))), E(np.zeros((T, C)))
        dB, dC = E(np.zeros((T, self.G, N))), E(np.zeros((T, self.G, N)))
        dh0 = E(np.zeros((len(self.lens), C, N)))
        inside = np.zeros(T, dtype=bool)
        dA, dAe, dAm = (np.zeros((C, N)) for _ in range(3))
        P = C // self.G

        def put(to, at, val):
            to.v[at], to.e[at] = val.v, val.e

        def by_group(val):  # [C, N] -> sums over the channels of a group
            return E(val.v.reshape(self.G, P, N), val.e.reshape(self.G, P, N)).sum(1)

        for i, t0, n in _starts(self.lens, self.begin):
            inside[t0:t0 + n] = True
            g = E(np.zeros((C, N)) if d["dfinal"] is None else d["dfinal"][i])
            for t in range(t0 + n - 1, t0 - 1, -1):
                before = self.h[t - 1, i]
                g = E(d["C"][t][self.of]) * dy[t][:, None] + g
                put(dC, t, by_group(self.h[t, i] * dy[t][:, None]))
                put(dB, t, by_group(g * self.u[t][:, None]))
                du = (g * E(d["B"][t][self.of])).sum(-1, 2)
                g = g * self.decay(t)
                r = g * before
                step = du * E(d["x"][t]) + (r * E(d["A"])).sum(-1, 4)
                put(dd, t, step)
                q = du * self.dt[t]
                put(dx, t, q if d["D"] is None else q + dy[t] * E(d["D"]))
                r = r * self.dt[t][:, None]
                dA += r.v
                dAe += r.e
                dAm += np.abs(r.v) + r.e
            put(dh0, i, g)
        if self.plus:
            dd = dd * sigmoid(self.raw)
        for a in (dd,) + ((dz,) if dz is not None else ()):
            a.v, a.e = a.v * inside[:, None], a.e * inside[:, None]
        res = {"dx": dx, "ddelta": dd, "dA": E(dA, dAe + T * U * dAm), "dB": dB, "dC": dC, "dh0": dh0,
               "dz": dz}
        only = lambda a: E(a.v * inside[:, None], a.e * inside[:, None])  # noqa: E731
        if d["D"] is not None:
            res["dD"] = only(dy * E(d["x"])).sum(0)
        if d["dbias"] is not None:
            res["dbias"] = dd.sum(0)
        return res
