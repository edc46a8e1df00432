"""The expert operators and the gradient clipping by their definitions, in 64 bits on the CPU,
and the error bounds of the kernels' arithmetic."""
import math

import torch

NINF = float("-inf")
U32 = 2.0 ** -24                     # half a step of binary32, relative


def step(dtype):
    """Half a step of a stored result, relative to its value."""
    return torch.finfo(dtype).eps / 2


def floor_of(dtype):
    """Half the distance of the type's subnormals: what rounding costs near zero."""
    return 2.0 ** -25 if dtype == torch.float16 else 2.0 ** -133 if dtype == torch.bfloat16 else 0.0


def assert_near(got, want, err, what):
    """|got - want| <= err elementwise; err is a bound of the arithmetic, and infinities and NaN
    have to be in the same places."""
    got = got.detach().cpu().double()
    want, err = want.double(), torch.as_tensor(err, dtype=torch.float64).expand(want.shape)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    fine = torch.isfinite(want)
    assert torch.equal(torch.isfinite(got), fine), what
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what
    bad = fine & ~((got - want).abs() <= err)
    if bad.any():
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError("%s: %d of %d beyond the bound, first at %s: %r, want %r, bound %.3g"
                             % (what, int(bad.sum()), bad.numel(), i, float(got[i]),
                                float(want[i]), float(err[i])))


def stored(want, err, dtype):
    """The bound of a result stored in dtype that was computed to within err."""
    return err + step(dtype) * (want.abs() + err) + floor_of(dtype)


# ------------------------------------------------------------------------------- router
def route_fwd(logits, k, renorm):
    x = logits.double()
    T, E = x.shape
    experts = torch.full((T, k), -1, dtype=torch.int32)
    weights = torch.zeros((T, k), dtype=torch.float64)
    for t in range(T):
        row = [float(v) for v in x[t]]
        open_ = [e for e in range(E) if row[e] > NINF]
        chosen = sorted(open_, key=lambda e: (-row[e], e))[:k]
        over = chosen if renorm else open_
        if not chosen:
            continue
        most = max(row[e] for e in over)
        ex = {e: 1.0 if row[e] == most else math.exp(row[e] - most) for e in over}
        total = sum(ex.values())
        for j, e in enumerate(chosen):
            experts[t, j] = e
            weights[t, j] = ex[e] / total
    return experts, weights


def route_bwd(logits, experts, dweights, renorm):
    """The formula's gradient, from the softmax q in 64 bits."""
    x = logits.double()
    T, E = x.shape
    k = experts.shape[1]
    out = torch.zeros((T, E), dtype=torch.float64)
    for t in range(T):
        chosen = [int(e) for e in experts[t] if e >= 0]
        over = chosen if renorm else [e for e in range(E) if float(x[t, e]) > NINF]
        if not chosen:
            continue
        most = max(float(x[t, e]) for e in over)
        ex = {e: 1.0 if float(x[t, e]) == most else math.exp(float(x[t, e]) - most) for e in over}
        total = sum(ex.values())
        q = {e: v / total for e, v in ex.items()}
        dw = {int(experts[t, j]): float(dweights[t, j]) for j in range(k) if experts[t, j] >= 0}
        s = sum(q[e] * dw[e] for e in chosen)
        for e in over:
            out[t, e] = q[e] * (dw.get(e, 0.0) - s)
    return out


# --------------------------------------------------------------------------------- rows
def sort(experts, E):
    flat = experts.reshape(-1).tolist()
    groups = [[] for _ in range(E)]
    for i, e in enumerate(flat):
        if 0 <= e < E:
            groups[e].append(i)
    offsets, order = [0], []
    for g in groups:
        order += g
        offsets.append(len(order))
    slots = torch.full((len(flat),), -1, dtype=torch.int32)
    seq = torch.tensor(order, dtype=torch.int64)
    slots[seq] = torch.arange(len(order), dtype=torch.int32)
    full = torch.full((len(flat),), -1, dtype=torch.int32)
    full[:len(order)] = seq.int()
    return torch.tensor(offsets, dtype=torch.int32), slots.view(experts.shape), full


def dispatch(X, slots):
    T, k = slots.shape
    P = torch.zeros((T * k, X.shape[1]), dtype=torch.float64)
    t, j = (slots >= 0).nonzero(as_tuple=True)
    P[slots[t, j].long()] = X.double()[t]
    return P


def combine_fwd(P, slots, weights):
    """(Y, sum of the terms' magnitudes)"""
    T, k = slots.shape
    Y = torch.zeros((T, P.shape[1]), dtype=torch.float64)
    M = torch.zeros_like(Y)
    t, j = (slots >= 0).nonzero(as_tuple=True)
    w = torch.ones(len(t), dtype=torch.float64) if weights is None else weights.double()[t, j]
    term = w[:, None] * P.double()[slots[t, j].long()]
    Y.index_add_(0, t, term)
    M.index_add_(0, t, term.abs())
    return Y, M


def combine_bwd(dY, P, slots, weights):
    """(dP, dweights, sum of the dots' magnitudes)"""
    T, k = slots.shape
    dP = torch.zeros((T * k, dY.shape[1]), dtype=torch.float64)
    dw = torch.zeros((T, k), dtype=torch.float64)
    mag = torch.zeros((T, k), dtype=torch.float64)
    t, j = (slots >= 0).nonzero(as_tuple=True)
    p = slots[t, j].long()
    w = torch.ones(len(t), dtype=torch.float64) if weights is None else weights.double()[t, j]
    dP[p] = w[:, None] * dY.double()[t]
    prod = dY.double()[t] * P.double()[p]
    dw[t, j] = prod.sum(1)
    mag[t, j] = prod.abs().sum(1)
    return dP, dw, mag


# ----------------------------------------------------------------------------- products
def x_of(X, order, k, n):
    """The rows that the positions read; a position without a slot reads zeros."""
    if order is None:
        return X.double()[:n]
    i = order.long()
    row = torch.where(i >= 0, i // k, X.shape[0])
    there = row < X.shape[0]
    return torch.where(there[:, None], X.double()[row.clamp(max=max(X.shape[0] - 1, 0))], 0.0)


def dense_fwd(X, W, b, offsets, relu, order, k, n):
    """(Y, sum of the terms' magnitudes)"""
    E, N, K = W.shape
    x = x_of(X, order, k, n)
    Y = torch.zeros((n, N), dtype=torch.float64)
    M = torch.zeros_like(Y)
    for e in range(E):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        y = x[lo:hi] @ W[e].double().T
        m = x[lo:hi].abs() @ W[e].double().abs().T
        if b is not None:
            y, m = y + b[e].double(), m + b[e].double().abs()
        Y[lo:hi], M[lo:hi] = y, m
    return (Y.clamp(min=0) if relu else Y), M


def dense_bwd(X, W, offsets, dY, order, k, x_relu):
    """{name: (value, sum of the terms' magnitudes, terms)}"""
    E, N, K = W.shape
    n = dY.shape[0]
    x = x_of(X, order, k, n)
    g = dY.double()
    dX = torch.zeros((n, K), dtype=torch.float64)
    mX = torch.zeros_like(dX)
    dW = torch.zeros((E, N, K), dtype=torch.float64)
    mW = torch.zeros_like(dW)
    db = torch.zeros((E, N), dtype=torch.float64)
    mb = torch.zeros_like(db)
    for e in range(E):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        dX[lo:hi] = g[lo:hi] @ W[e].double()
        mX[lo:hi] = g[lo:hi].abs() @ W[e].double().abs()
        dW[e] = g[lo:hi].T @ x[lo:hi]
        mW[e] = g[lo:hi].abs().T @ x[lo:hi].abs()
        db[e], mb[e] = g[lo:hi].sum(0), g[lo:hi].abs().sum(0)
    if x_relu:
        dX = torch.where(x > 0, dX, 0.0)
    most = int((offsets[1:] - offsets[:-1]).max())
    return {"dX": (dX, mX, N), "dW": (dW, mW, most), "db": (db, mb, most)}
