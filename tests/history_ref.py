"""The click-history operators by their definitions, in 64 bits on the CPU, with the error bounds of
the kernels' arithmetic beside the results.

U32 is half a step of binary32.  A sum of L fp32 terms is within (L + 2) U32 of the exact sum,
relative to the sum of the terms' magnitudes, whatever the order.  The sigmoid of x costs at most
(10 + 2 |x|) U32 relative: the exponential's argument x log2(e) is rounded once (|x| 1.45 U32),
exp2 and the reciprocal are within a unit of the last place, and three more operations are rounded.
"""
import math

import torch

from tests.experts_ref import U32, assert_near, floor_of, step, stored  # noqa: F401

F8_MAX, F8_TINY = 448.0, 2.0 ** -100


# ------------------------------------------------------------------------------- tokens
def embed_fwd(table, ids, scale):
    V = table.shape[0]
    at = ids.clamp(0, V - 1).long()
    y = table.double()[at] * float(torch.tensor(scale, dtype=torch.float32))
    y[ids < 0] = 0.0
    y[ids >= V] = float("nan")
    return y


def embed_bwd(dY, ids, V, scale):
    """(dtable, sum of the terms' magnitudes, terms of each row)"""
    s = float(torch.tensor(scale, dtype=torch.float32))
    here = (ids >= 0) & (ids < V)
    at, x = ids[here].long(), dY.double()[here] * s
    d = torch.zeros((V, dY.shape[1]), dtype=torch.float64).index_add_(0, at, x)
    m = torch.zeros_like(d).index_add_(0, at, x.abs())
    return d, m, torch.bincount(at, minlength=V).double()[:, None]


# --------------------------------------------------------------------------------- norm
def norm_fwd(S, weight, eps):
    """(y, rstd, relative error bound of both)"""
    x = S.double()
    D = x.shape[1]
    rstd = 1.0 / torch.sqrt((x * x).sum(1, keepdim=True) / D + eps)
    y = x * rstd * (1.0 if weight is None else weight.double())
    # the squares' sum within (D + 2) U32, half of that in its root; the division by D, the
    # addition of eps, root, inverse and two products
    return y, rstd, (D / 2 + 10) * U32


def norm_bwd(dY, S, rstd, weight, dS):
    """(dX, bound, dweight, bound); rstd as the kernel has it."""
    x, dy, r = S.double(), dY.double(), rstd.double()[:, None]
    n, D = x.shape
    dn = dy if weight is None else dy * weight.double()
    t = (dn * x).sum(1, keepdim=True) / D * r * r
    m = (dn * x).abs().sum(1, keepdim=True) / D * r * r
    dx = r * (dn - x * t)
    err = (D + 14) * U32 * (r * (dn.abs() + x.abs() * m))
    if dS is not None:
        dx = dx + dS.double()
        err = err + U32 * dS.double().abs()
    dw = (dy * x * r).sum(0)
    return dx, err, dw, (n + 6) * U32 * (dy * x * r).abs().sum(0)


def e4m3(x):
    """x to the nearest e4m3 number, ties to even."""
    _, e = torch.frexp(x)
    unit = torch.ldexp(torch.ones_like(x), (e - 1).clamp(min=-6) - 3)
    return torch.round(x / unit) * unit


def assert_codes(codes, scale, y, rel, what):
    """8-bit rows that stand for y, which the kernel knows within rel of its magnitude."""
    n, D = y.shape
    assert codes.shape == (n, (D + 15) // 16 * 16) and codes.dtype == torch.float8_e4m3fn
    c, s = codes.cpu().float().double(), scale.cpu().double()
    bad = ~torch.isfinite(y).all(1)
    assert (c[:, D:] == 0).all(), what
    assert torch.isnan(c[bad, :D] * s[bad, None]).all(), what
    y, c, s = y[~bad], c[~bad, :D], s[~bad]
    top = y.abs().amax(1).clamp(min=F8_TINY) if D else s
    assert_near(s, top / F8_MAX, (rel + 2 * U32) * top / F8_MAX, what + " scale")
    # half a step of e4m3: 2^-4 of the value, 2^-10 of the scale below the normal range
    err = (2.0 ** -4 * y.abs() + 2.0 ** -10 * s[:, None]) * (1 + 2 * rel + 8 * U32)
    assert_near(c * s[:, None], y, err + (rel + 4 * U32) * y.abs(), what)


# --------------------------------------------------------------------------------- scan
def _sig(x):
    return torch.sigmoid(x), torch.sigmoid(-x)


def scan(gate, value, offsets, out=None, h0=None, dY=None, dhN=None):
    """Results and bounds by name: Y, hN, and with dY dgate, dvalue, dout, dh0.  Rows in no
    sequence are NaN."""
    g, v = gate.double(), value.double()
    n, D = g.shape
    B = len(offsets) - 1
    f, i = _sig(g)
    eps = (24 + 4 * g.abs()) * U32                 # sigmoid, product, sum, joined maps
    o = None if out is None else out.double()
    nan = torch.full((n, D), float("nan"), dtype=torch.float64)
    h, eh, mh = nan.clone(), nan.clone(), nan.clone()
    before, eb, mb = nan.clone(), nan.clone(), nan.clone()
    hN, ehN = torch.zeros((B, D), dtype=torch.float64), torch.zeros((B, D), dtype=torch.float64)
    for b in range(B):
        s = h0[b].double() if h0 is not None else torch.zeros(D, dtype=torch.float64)
        m, e = s.abs(), torch.zeros(D, dtype=torch.float64)
        for t in range(offsets[b], offsets[b + 1]):
            before[t], eb[t], mb[t] = s, e, m
            s = f[t] * s + i[t] * v[t]
            m = f[t] * m + i[t] * v[t].abs()
            e = f[t] * e + eps[t] * m
            h[t], eh[t], mh[t] = s, e, m
        hN[b], ehN[b] = s, e
    res = {"hN": (hN, ehN)}
    q, eq = None, None
    if o is None:
        res["Y"] = (h, eh)
    else:
        z, zi = _sig(o)
        eo = (24 + 4 * o.abs()) * U32
        res["Y"] = (h * o * z, (eh + eo * mh) * (o * z).abs())
    if dY is None:
        return res
    dy = dY.double()
    if o is None:
        q, eq = dy, torch.zeros_like(dy)
    else:
        slope = z * (1 + o * zi)
        most = z * (1 + o.abs() * zi)
        res["dout"] = (dy * h * slope, dy.abs() * (eh * slope.abs() + 2 * eo * mh * most))
        q, eq = dy * o * z, (dy * o * z).abs() * eo
    dh, ed, md = nan.clone(), nan.clone(), nan.clone()
    dh0, edh0 = torch.zeros((B, D), dtype=torch.float64), torch.zeros((B, D), dtype=torch.float64)
    for b in range(B):
        s = dhN[b].double() if dhN is not None else torch.zeros(D, dtype=torch.float64)
        m, e = s.abs(), torch.zeros(D, dtype=torch.float64)
        for t in range(offsets[b + 1] - 1, offsets[b] - 1, -1):
            s, m = q[t] + s, q[t].abs() + m
            e = e + eq[t] + 4 * U32 * m
            dh[t], ed[t], md[t] = s, e, m
            s, m, e = f[t] * s, f[t] * m, f[t] * e + eps[t] * f[t] * m
        dh0[b], edh0[b] = s, e
    res["dh0"] = (dh0, edh0)
    res["dvalue"] = (i * dh, i * (ed + eps * md))
    res["dgate"] = (dh * (before - v) * f * i,
                    f * i * (ed * (before - v).abs() + md * eb + 3 * eps * md * (mb + v.abs())))
    return res


def scan_step(gate, value, state, index, out=None):
    """(Y, state after, bounds) row by row."""
    g, v = gate.double(), value.double()
    f, i = _sig(g)
    s = state.double().clone()
    m, e = s.abs(), torch.zeros_like(s)
    Y, E = torch.zeros_like(g), torch.zeros_like(g)
    for r in range(g.shape[0]):
        k = r if index is None else int(index[r])
        if not 0 <= k < s.shape[0]:
            continue
        eps = (24 + 4 * g[r].abs()) * U32
        s[k] = f[r] * s[k] + i[r] * v[r]
        m[k] = f[r] * m[k] + i[r] * v[r].abs()
        e[k] = f[r] * e[k] + eps * m[k]
        Y[r], E[r] = s[k], e[k]
        if out is not None:
            o = out[r].double()
            w = o * torch.sigmoid(o)
            Y[r], E[r] = s[k] * w, (e[k] + (24 + 4 * o.abs()) * U32 * m[k]) * w.abs()
    return Y, E, s, e


# -------------------------------------------------------------------------------- dense
def act(x, name):
    if name == "relu":
        return x.clamp(min=0)
    if name == "silu":
        return x * torch.sigmoid(x)
    if name == "gelu":
        return 0.5 * x * (1 + torch.erf(x * math.sqrt(0.5)))
    return x


def dense(X, xs, W, ws, b, name, R, dtype):
    """(Y, bound).  Products of codes are exact, sums of them fp32.  Where Y is of 16 bits, the 8-bit
    matrix instructions cut what of eight neighbouring products lies below 2^-13 of the largest of
    them: at most 8 * 2^-13 of it for each eight."""
    x, w = X.float().double(), W.float().double()
    by = xs.double()[:, None] * ws.double()
    z, m = x @ w.t() * by, x.abs() @ w.abs().t() * by
    err = (x.shape[1] + 8) * U32 * m
    if dtype != torch.float32:
        for k in range(0, x.shape[1], 8):
            most = (x[:, None, k:k + 8] * w[None, :, k:k + 8]).abs().amax(2)
            err = err + 8 * 2.0 ** -13 * most * by
    if b is not None:
        z = z + b.double()
        err = err + U32 * (b.double().abs() + z.abs())
    y = act(z, name)
    # the slope of silu and gelu is at most 1.13; the function's own error as the sigmoid's
    err = 1.13 * err + (0 if name in ("none", "relu") else (16 + 4 * z.abs()) * U32 * z.abs())
    if R is not None:
        y = y + R.double()
        err = err + U32 * (R.double().abs() + y.abs())
    return y, err
