"""The expert operators on the GPU against their definitions in 64 bits (tests/experts_ref.py).

Bounds: a sum of L fp32 terms is within (L + 2) half steps of binary32 of the exact sum,
relative to the sum of the terms' magnitudes, whatever the order (products of 16-bit operands
are exact in binary32, those of binary32 operands cost the one half step in the 2); a stored
result adds half a step of its type.  Choices, positions and copies are equal bit for bit.
"""
import ctypes

import numpy as np
import pytest
import torch

from sparse_embedding_lookup_amd import ctr
from tests import experts_ref as ref
from tests.experts_ref import NINF, U32, assert_near, stored

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

DEV = "cuda"
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
TYPES = [F32, BF16, F16]


def say(*a):
    print(*a, flush=True)


def gen(seed):
    return torch.Generator().manual_seed(seed)


def strided(a, pad, offset=0):
    """a on the GPU in rows `pad` elements wider, starting `offset` elements into its memory; NaN
    around it."""
    rows, width = a.shape
    buf = torch.full((offset + rows * (width + pad) + 8,), float("nan"), dtype=a.dtype, device=DEV)
    out = buf[offset:offset + rows * (width + pad)].view(rows, width + pad)[:, :width]
    out.copy_(a)
    return out


def canvas(rows, width, pad, offset, dtype):
    """An output with padded rows, filled with -3 all around: (view, check of the padding)."""
    buf = torch.full((offset + rows * (width + pad) + 8,), -3.0, dtype=dtype, device=DEV)
    full = buf[offset:offset + rows * (width + pad)].view(rows, width + pad)

    def untouched():
        assert (buf[:offset] == -3).all() and (full[:, width:] == -3).all()
        assert (buf[offset + rows * (width + pad):] == -3).all()
    return full[:, :width], untouched


def choose(g, T, E, k, skew=1.0, drop=0.1):
    like = torch.randn((T, E), generator=g) + skew * torch.randn((1, E), generator=g)
    experts = torch.argsort(like, 1, descending=True)[:, :k].to(torch.int32)
    lost = torch.rand((T, k), generator=g) < drop
    return torch.where(lost, -1, experts).contiguous()


# ------------------------------------------------------------------------------- router
# (T, E, k, row padding)
ROUTES = [(1, 1, 1, 0), (1, 8, 2, 0), (37, 8, 2, 0), (5, 3, 3, 1), (64, 64, 4, 0),
          (130, 61, 4, 3), (33, 16, 16, 0), (9, 200, 8, 0), (7, 513, 2, 0), (4, 1024, 64, 5),
          (0, 8, 2, 0)]
MASKS = ["none", "some", "rows", "few", "lowest", "ties", "nan", "inf"]


def _logits(T, E, k, dtype, mask):
    g = gen(T * 7 + E + k)
    x = torch.randn((T, E), generator=g) * 3
    low = torch.finfo(dtype).min
    hide = torch.rand((T, E), generator=g)
    if mask == "some":
        x[hide < 0.3] = NINF
    elif mask == "rows":
        x[::2] = NINF
    elif mask == "few":                     # fewer open experts than choices
        x[:, k // 2:] = NINF
    elif mask == "lowest":
        x[hide < 0.7] = low
        x[::3] = low
    elif mask == "ties":
        x = torch.round(x / 3)
    elif mask == "nan":
        x[hide < 0.2] = float("nan")
    elif mask == "inf":
        x[hide < 0.2] = float("inf")
    return x.to(dtype)


@pytest.mark.parametrize("mask", MASKS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,E,k,pad", ROUTES)
def test_route(T, E, k, pad, dtype, mask):
    say("route", T, E, k, pad, dtype, mask)
    x = _logits(T, E, k, dtype, mask)
    xd = strided(x, pad)
    dw = torch.randn((T, k), generator=gen(3))
    for renorm in (True, False):
        experts, weights = ctr.ctr_expert_route_fwd(xd, k, renorm)
        we, ww = ref.route_fwd(x, k, renorm)
        assert torch.equal(experts.cpu(), we)
        # exp within 2 units of its last place of an argument rounded once (its magnitude is
        # the logits' difference, where the result is not negligible below 64), E + 2 additions,
        # one division
        assert_near(weights, ww, (64 + E + 10) * 2 * U32 * ww + 1e-30, "weights")
        dl, untouched = canvas(T, E, pad, 0, dtype)
        ctr.ctr_expert_route_bwd(xd, experts, weights, dw.to(DEV), renorm, dl)
        want = ref.route_bwd(x, we, dw, renorm)
        # each of q and the sum carries the weights' error; magnitudes at most |dw|
        most = dw.abs().sum(1, keepdim=True).double()
        assert_near(dl, want, stored(want, (64 + E + k + 20) * 4 * U32 * most, dtype), "dlogits")
        untouched()


@pytest.mark.parametrize("renorm", [True, False])
def test_route_gradient_against_differences(renorm):
    say("route differences", renorm)
    T, E, k, h = 40, 24, 3, 2.0 ** -12
    g = gen(5)
    x = torch.randn((T, E), generator=g)
    dw = torch.randn((T, k), generator=g)
    d = torch.randn((T, E), generator=g).double()
    experts, weights = ctr.ctr_expert_route_fwd(x.to(DEV), k, renorm)
    got = ctr.ctr_expert_route_bwd(x.to(DEV), experts, weights, dw.to(DEV), renorm).cpu().double()
    at = experts.cpu().long()

    def loss(y):                            # the choice held fixed
        z = y.gather(1, at) if renorm else y
        w = torch.exp(y.gather(1, at) - torch.logsumexp(z, 1, keepdim=True))
        return (w * dw.double()).sum(1)
    diff = (loss(x.double() + h * d) - loss(x.double() - h * d)) / (2 * h)
    # the difference is off by h^2/6 of the third derivative, at most 26 |dw| |d|^3
    bound = h * h / 6 * 26 * dw.double().abs().sum(1) * d.abs().max() ** 3 + 1e-5
    assert_near((got * d).sum(1), diff, bound, "directional derivative")


# --------------------------------------------------------------------------------- sort
SORTS = [(0, 2, 4), (1, 1, 1), (1, 2, 16), (63, 1, 5), (64, 1, 1), (257, 2, 8), (2048, 2, 61),
         (2049, 2, 16), (5000, 3, 64), (8192, 2, 1024), (33333, 4, 33), (150000, 2, 7)]


@pytest.mark.parametrize("T,k,E", SORTS)
def test_sort(T, k, E):
    say("sort", T, k, E)
    g = gen(T + E)
    for kind in ("spread", "one", "none", "strange"):
        experts = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32)
        if kind == "one":
            experts.fill_(E - 1)
        elif kind == "none":
            experts.fill_(-1)
        elif kind == "strange":             # dropped, out of range, the extremes
            r = torch.rand((T, k), generator=g)
            experts[r < 0.2] = -1
            experts[(r >= 0.2) & (r < 0.3)] = E
            experts[(r >= 0.3) & (r < 0.4)] = 2 ** 31 - 1
            experts[(r >= 0.4) & (r < 0.5)] = -2 ** 31
        got = ctr.ctr_expert_sort(experts.to(DEV), E)
        for a, b, name in zip(got, ref.sort(experts, E), ("offsets", "slots", "order")):
            assert torch.equal(a.cpu(), b), (kind, name)


# --------------------------------------------------------------------------------- rows
# (T, k, E, D, padding, offset in elements)
ROWS = [(1, 1, 1, 1, 0, 0), (1, 2, 4, 128, 0, 0), (37, 2, 8, 128, 0, 0), (50, 3, 5, 7, 2, 1),
        (20, 2, 4, 8, 8, 0), (33, 4, 16, 136, 0, 1), (129, 2, 7, 1024, 0, 0),
        (65, 2, 64, 2208, 0, 8), (30, 1, 3, 2209, 0, 0), (0, 2, 4, 64, 0, 0), (3, 64, 64, 40, 8, 8)]


@pytest.mark.parametrize("drop", [0.0, 0.2, 1.0])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,k,E,D,pad,off", ROWS)
def test_rows(T, k, E, D, pad, off, dtype, drop):
    say("rows", T, k, E, D, pad, off, dtype, drop)
    g = gen(T + D)
    experts = choose(g, T, E, k, drop=drop)
    offsets, slots, order = ref.sort(experts, E)
    X, dY = (torch.randn((T, D), generator=g).to(dtype) for _ in range(2))
    Q = torch.randn((T * k, D), generator=g).to(dtype)
    Q[int(offsets[E]):] = float("nan")      # positions of no slot are not read
    w = torch.rand((T, k), generator=g)
    so, ss = offsets.to(DEV), slots.to(DEV)

    P, untouched = canvas(T * k, D, pad, off, dtype)
    ctr.ctr_expert_dispatch(strided(X, pad, off), ss, so, P)
    assert torch.equal(P.cpu().double(), ref.dispatch(X, slots))
    untouched()

    for weights in (w, None):
        wd = None if weights is None else weights.to(DEV)
        Y, untouched = canvas(T, D, pad, off, dtype)
        ctr.ctr_expert_combine_fwd(strided(Q, pad, off), ss, wd, Y)
        want, mag = ref.combine_fwd(torch.nan_to_num(Q), slots, weights)
        assert_near(Y, want, stored(want, (k + 2) * U32 * mag, dtype), "Y")
        untouched()

        dP, untouched = canvas(T * k, D, pad, off, dtype)
        _, dwt = ctr.ctr_expert_combine_bwd(strided(dY, pad, off), strided(Q, pad, off), ss, so,
                                            wd, dP)
        wP, wdw, mdw = ref.combine_bwd(dY, torch.nan_to_num(Q), slots, weights)
        assert_near(dP, wP, stored(wP, U32 * wP.abs(), dtype), "dP")
        assert_near(dwt, wdw, (D + 2) * U32 * mdw, "dweights")
        untouched()
        alone, none = ctr.ctr_expert_combine_bwd(dY.to(DEV), None, ss, so, wd)
        assert none is None and torch.equal(alone, dP)


# ----------------------------------------------------------------------------- products
# (T, k, E, K, N, padding, offset, drop): widths around the tiles and vectors, experts without
# rows, few rows, many
PRODUCTS = [(1, 1, 1, 1, 1, 0, 0, 0.0), (1, 2, 16, 128, 64, 0, 0, 0.0),
            (5, 2, 4, 32, 48, 0, 0, 0.0), (48, 2, 16, 256, 128, 0, 0, 0.0),
            (64, 1, 1, 64, 64, 0, 0, 0.0), (200, 2, 3, 136, 72, 8, 8, 0.2),
            (150, 2, 5, 61, 33, 3, 1, 0.1), (40, 2, 70, 96, 80, 0, 0, 0.1),
            (700, 2, 4, 264, 520, 0, 0, 0.1), (513, 1, 2, 512, 256, 0, 0, 0.0),
            (300, 2, 2, 257, 300, 0, 0, 1.0), (3000, 2, 6, 320, 192, 0, 0, 0.05),
            (0, 2, 4, 64, 64, 0, 0, 0.0)]


@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,k,E,K,N,pad,off,drop", PRODUCTS)
def test_products(T, k, E, K, N, pad, off, drop, dtype, gather):
    say("products", T, k, E, K, N, pad, off, drop, dtype, gather)
    g = gen(T + K + N)
    offsets, slots, order = ref.sort(choose(g, T, E, k, 2.0, drop), E)
    n = T * k
    m = int(offsets[E])
    X = torch.randn((T if gather else n, K), generator=g).to(dtype)
    W = (torch.randn((E, N, K), generator=g) * K ** -0.5).to(dtype)
    b = torch.randn((E, N), generator=g)
    dY = torch.randn((n, N), generator=g).to(dtype)
    dY[m:] = float("nan")                   # rows of no expert are not read
    x_relu = not gather
    if not gather:
        X = torch.relu(X)
        X[m:] = float("nan")
    at = order.to(DEV) if gather else None
    fd, Wd = offsets.to(DEV), W.to(DEV)
    Xd, dYd = strided(X, pad, off), strided(dY, pad, off)
    X, dY = torch.nan_to_num(X), torch.nan_to_num(dY)
    o = order if gather else None

    for relu, bias in ((True, b), (False, None)):
        Y, untouched = canvas(n, N, pad, off, dtype)
        ctr.ctr_expert_dense_fwd(Xd, Wd, None if bias is None else bias.to(DEV), fd, relu, at, k, Y)
        want, mag = ref.dense_fwd(X, W, bias, offsets, relu, o, k, n)
        assert_near(Y, want, stored(want, (K + 3) * U32 * mag, dtype), "Y")
        untouched()

    dX, untouched = canvas(n, K, pad, off, dtype)
    _, dW, db = ctr.ctr_expert_dense_bwd(Xd, Wd, fd, dYd, at, k, x_relu=x_relu, dX=dX)
    want = ref.dense_bwd(X, W, offsets, dY, o, k, x_relu)
    v, mag, L = want["dX"]
    assert_near(dX, v, stored(v, (L + 2) * U32 * mag, dtype), "dX")
    untouched()
    for got, name in ((dW, "dW"), (db, "db")):
        v, mag, L = want[name]
        assert_near(got, v, (L + 2) * U32 * mag, name)
    # one gradient at a time gives the same
    only = dict(x_relu=x_relu, bias=False, want_dx=False, want_dw=False)
    a, _, _ = ctr.ctr_expert_dense_bwd(Xd, Wd, fd, dYd, at, k, **dict(only, want_dx=True))
    _, c, _ = ctr.ctr_expert_dense_bwd(Xd, Wd, fd, dYd, at, k, **dict(only, want_dw=True))
    _, _, d = ctr.ctr_expert_dense_bwd(Xd, Wd, fd, dYd, at, k, **dict(only, bias=True))
    assert torch.equal(a, dX) and torch.equal(c, dW) and torch.equal(d, db)


@pytest.mark.parametrize("dtype", TYPES)
def test_product_gradients_against_differences(dtype):
    """<dX, d> and <dW, d> against central differences of the forward's definition."""
    say("product differences", dtype)
    T, k, E, K, N, h = 60, 2, 4, 40, 24, 2.0 ** -10
    g = gen(11)
    offsets, slots, order = ref.sort(choose(g, T, E, k), E)
    n = T * k
    X = torch.relu(torch.randn((n, K), generator=g)).to(dtype)
    W = torch.randn((E, N, K), generator=g).to(dtype)
    dY = torch.randn((n, N), generator=g).to(dtype)
    m = int(offsets[E])
    dX, dW, db = ctr.ctr_expert_dense_bwd(X.to(DEV), W.to(DEV), offsets.to(DEV), dY.to(DEV))
    eX, eW = (torch.randn(a.shape, generator=g).double() for a in (X, W))
    eX[m:] = 0

    def loss(x, w):
        y = ref.dense_fwd(x, w, None, offsets, False, None, k, n)[0]
        return (y[:m] * dY.double()[:m]).sum()
    x, w = X.double(), W.double()
    num = (loss(x + h * eX, w + h * eW) - loss(x - h * eX, w - h * eW)) / (2 * h)
    got = (dX.cpu().double() * eX).sum() + (dW.cpu().double() * eW).sum()
    # bilinear: the central difference is exact but for the rounding of 64 bits; the stored
    # gradients are off by half a step each, the sums by their fp32 bounds
    v = ref.dense_bwd(X, W, offsets, dY, None, k, False)
    bound = 1e-9 * (abs(num) + 1) / h
    bound += float((stored(v["dX"][0], (N + 2) * U32 * v["dX"][1], dtype) * eX.abs()).sum())
    bound += float((((v["dW"][2] + 2) * U32 * v["dW"][1]) * eW.abs()).sum())
    assert abs(float(got - num)) <= bound


@pytest.mark.parametrize("dtype", TYPES)
def test_products_masked_nan_and_infinity_stay_in_their_rows(dtype):
    """A NaN or an infinity in one row of X reaches that row of Y only, and only its expert's dW."""
    T, E, K, N = 96, 3, 64, 48
    g = gen(2)
    X = torch.randn((T, K), generator=g).to(dtype)
    X[40, 3] = float("nan")
    X[41, 5] = float("inf")
    W = torch.randn((E, N, K), generator=g).to(dtype)
    offsets = torch.tensor([0, 32, 64, 96], dtype=torch.int32)
    Y = ctr.ctr_expert_dense_fwd(X.to(DEV), W.to(DEV), None, offsets.to(DEV), False).cpu()
    assert torch.isnan(Y[40]).all() and not torch.isfinite(Y[41]).any()
    rest = torch.ones(T, dtype=torch.bool)
    rest[40:42] = False
    assert torch.isfinite(Y[rest]).all()
    dY = torch.randn((T, N), generator=g).to(dtype)
    dX, dW, db = ctr.ctr_expert_dense_bwd(X.to(DEV), W.to(DEV), offsets.to(DEV), dY.to(DEV))
    assert torch.isfinite(dX).all() and torch.isfinite(db).all()
    assert torch.isfinite(dW[0]).all() and torch.isfinite(dW[2]).all()
    bad = ~torch.isfinite(dW[1].cpu())
    assert bad[:, 3].all() and bad[:, 5].all() and int(bad.sum()) == 2 * N


def test_products_bad_offsets_and_order_stay_inside():
    """Offsets beyond n, falling offsets and slots outside X give numbers, not faults."""
    say("bad offsets")
    T, E, K, N = 100, 4, 64, 64
    X = torch.randn((T, K), device=DEV).to(BF16)
    W = torch.randn((E, N, K), device=DEV).to(BF16)
    dY = torch.randn((T, N), device=DEV).to(BF16)
    order = torch.arange(T, dtype=torch.int32, device=DEV)
    order[7], order[8], order[9] = -1, T + 5, 2 ** 31 - 1
    for off in ([0, 500, 20, -3, 90], [-5, 10, 10, 10, 2 ** 31 - 1], [90, 80, 70, 60, 50]):
        f = torch.tensor(off, dtype=torch.int32, device=DEV)
        ctr.ctr_expert_dense_fwd(X, W, None, f, True, order, 1)
        ctr.ctr_expert_dense_bwd(X, W, f, dY, order, 1)
    torch.cuda.synchronize()
    good = torch.tensor([0, 25, 50, 75, 100], dtype=torch.int32, device=DEV)
    Y = ctr.ctr_expert_dense_fwd(X, W, None, good, False, order, 1)
    assert (Y[7:10] == 0).all() and torch.isfinite(Y).all()


# ------------------------------------------------------- streams, graphs, repeated calls
def _layer_pass(c):
    """One pass through every operator, forward and backward: all its outputs."""
    experts, weights = ctr.ctr_expert_route_fwd(c["logits"], c["k"])
    offsets, slots, order = ctr.ctr_expert_sort(experts, c["E"])
    H = ctr.ctr_expert_dense_fwd(c["X"], c["W"], c["b"], offsets, True, order, c["k"])
    Y = ctr.ctr_expert_combine_fwd(H, slots, weights)
    dH, dw = ctr.ctr_expert_combine_bwd(c["dY"], H, slots, offsets, weights)
    dP, dW, db = ctr.ctr_expert_dense_bwd(c["X"], c["W"], offsets, dH, order, c["k"])
    dX = ctr.ctr_expert_combine_fwd(dP, slots, None)
    dl = ctr.ctr_expert_route_bwd(c["logits"], experts, weights, dw)
    outs = [torch.empty_like(g) for g in (dW, db)]
    stats = ctr.ctr_grad_clip([dW, db], 0.5, outs)
    return [experts, weights, offsets, slots, order, H, Y, dH, dw, dP, dW, db, dX, dl, stats] + outs


def _layer_case(T=3000, E=12, k=2, K=256, N=320, dtype=BF16):
    g = gen(1)
    return dict(k=k, E=E, logits=torch.randn((T, E), generator=g).to(dtype).to(DEV),
                X=torch.randn((T, K), generator=g).to(dtype).to(DEV),
                W=(torch.randn((E, N, K), generator=g) * 0.1).to(dtype).to(DEV),
                b=torch.randn((E, N), generator=g).to(DEV),
                dY=torch.randn((T, N), generator=g).to(dtype).to(DEV))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_same_bits_in_every_run_and_on_another_stream(dtype):
    say("same bits", dtype)
    c = _layer_case(dtype=dtype)
    first = _layer_pass(c)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = _layer_pass(c)
    torch.cuda.current_stream().wait_stream(side)
    third = _layer_pass(c)
    for a, b, d in zip(first, second, third):
        assert torch.equal(a, b) and torch.equal(a, d)


def test_captured_pass_replays_like_the_eager_one():
    say("capture")
    c = _layer_case()
    want = [t.clone() for t in _layer_pass(c)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _layer_pass(c)
    for _ in range(4):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        again = _layer_pass(c)               # eager work between the replays
        torch.cuda.synchronize()
        for a, b in zip(again, want):
            assert torch.equal(a, b)


# --------------------------------------------------------------------- gradient clipping
SIZES = [[1], [7], [1, 3, 0, 5], [8192], [8191, 8193], [100000, 1, 16384, 33], [5] * 230,
         [1 << 20, 3, (1 << 18) + 1], [0], [8192 * 1500 + 5]]


def _norm(grads):
    return float(torch.sqrt(sum((g.double() ** 2).sum() for g in grads)))


@pytest.mark.parametrize("packed", [True, False])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("which", range(len(SIZES)))
def test_grad_clip(which, dtype, packed):
    sizes = SIZES[which]
    say("clip", which, dtype, packed)
    g = gen(which)
    total = sum(sizes)
    flat = (torch.randn(total + 1, generator=g) * 0.1).to(dtype)
    # packed: views of one buffer, one element in, so hardly one is aligned
    dev = flat.to(DEV)
    grads = list(torch.split(dev[1:], sizes))
    if not packed:
        grads = [t.clone() for t in grads]
    host = [t.cpu() for t in grads]
    norm = _norm(host)
    for max_norm in (norm * 2 + 1, norm / 3, 0.0):
        scale = 1.0 if not norm > max_norm else max_norm / norm
        outs = [torch.full_like(t, -3.0) for t in grads]
        stats = ctr.ctr_grad_clip(grads, max_norm, outs).cpu().double()
        # binary64 sums: the error is that of the fp32 result and of max_norm's own rounding
        assert abs(float(stats[0]) - norm) <= 2 * U32 * norm
        assert abs(float(stats[1]) - scale) <= 4 * U32 * scale
        for a, b in zip(outs, host):
            want = b.double() * scale
            assert_near(a, want, stored(want, 6 * U32 * want.abs(), dtype), "clipped")
        inplace = [t.clone() for t in grads]
        ctr.ctr_grad_clip(inplace, max_norm)
        for a, b in zip(inplace, outs):
            assert torch.equal(a, b)
    for a, b in zip(grads, host):
        assert torch.equal(a.cpu(), b)      # the gradients are kept


@pytest.mark.parametrize("ptype", TYPES)
@pytest.mark.parametrize("gtype", TYPES)
def test_grad_clip_sgd(gtype, ptype):
    say("clip sgd", gtype, ptype)
    g = gen(9)
    sizes = [20000, 1, 513, 8192, 8191, 3]
    grads = [torch.randn(s, generator=g).to(gtype).to(DEV) for s in sizes]
    buf = torch.randn(sum(sizes), generator=g).to(ptype).to(DEV)
    params = list(torch.split(buf, sizes))  # of another alignment than the gradients
    before = [p.cpu().clone() for p in params]
    norm, max_norm, lr = _norm([t.cpu() for t in grads]), 2.0, 0.3
    stats = ctr.ctr_grad_clip_sgd(grads, params, lr, max_norm)
    c = np.float32(lr) * (max_norm / norm)
    assert abs(float(stats[0]) - norm) <= 2 * U32 * norm
    for p, b, t in zip(params, before, grads):
        step = c * t.cpu().double()
        want = b.double() - step
        assert_near(p, want, stored(want, U32 * want.abs() + 4 * U32 * step.abs(), ptype), "param")


def test_grad_clip_large_and_strange_values():
    say("clip values")
    big = torch.full((3000,), 1e30, device=DEV)           # squares beyond binary32
    out = torch.empty_like(big)
    stats = ctr.ctr_grad_clip([big], 1.0, [out]).cpu()
    assert abs(float(stats[0]) / (1e30 * 3000 ** 0.5) - 1) < 1e-6
    assert torch.allclose(out.cpu(), torch.full((3000,), 3000 ** -0.5), rtol=1e-6, atol=0)
    tiny = torch.full((4,), 1e-30, device=DEV)            # squares below binary32
    assert abs(float(ctr.ctr_grad_clip([tiny], 1.0)[0]) / 2e-30 - 1) < 1e-6
    nan = torch.tensor([1.0, float("nan")], device=DEV)
    stats = ctr.ctr_grad_clip([nan], 1.0, [torch.empty_like(nan)]).cpu()
    assert torch.isnan(stats).all()
    inf = torch.tensor([1.0, float("inf")], device=DEV)
    out = torch.empty_like(inf)
    stats = ctr.ctr_grad_clip([inf], 1.0, [out]).cpu()
    assert float(stats[0]) == float("inf") and float(stats[1]) == 0.0
    assert float(out[0]) == 0.0 and bool(torch.isnan(out[1]))


def test_grad_clip_mixed_types():
    say("clip mixed")
    g = gen(4)
    grads = [torch.randn(9000, generator=g).to(t).to(DEV) for t in (F32, BF16, F16)]
    norm = _norm([t.cpu() for t in grads])
    outs = [torch.empty_like(t) for t in grads]
    ctr.ctr_grad_clip(grads, norm / 2, outs)
    for a, b in zip(outs, grads):
        want = b.cpu().double() / 2
        assert_near(a, want, stored(want, 6 * U32 * want.abs(), b.dtype), "mixed")


# ------------------------------------------------------------------- nothing beside an output
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N", [1, 33, 64, 257])
def test_gradients_of_no_rows_stay_in_their_arrays(N, dtype):
    """Without rows dW and db are zero, and what lies beside them in one buffer is kept."""
    say("no rows", N, dtype)
    E, K = 8, 24
    X, dY = (torch.empty((0, c), dtype=dtype, device=DEV) for c in (K, N))
    W = torch.ones((E, N, K), dtype=dtype, device=DEV)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    for shift in (64, 65):                  # aligned and not
        flat = torch.full((E * N * K + E * N + 256,), 7.0, device=DEV)
        dW = flat[shift:shift + E * N * K].view(E, N, K)
        at = shift + E * N * K + 64
        db = flat[at:at + E * N].view(E, N)
        dX, _, _ = ctr.ctr_expert_dense_bwd(X, W, offsets, dY, dW=dW, db=db)
        assert dX.shape == (0, K) and (dW == 0).all() and (db == 0).all()
        dW.fill_(7.0)
        db.fill_(7.0)
        assert (flat == 7).all()


# (rows, E, K, N): the last tile across has fewer columns than a 16-byte piece, the reductions end
# with whole rounds, and the last expert's last row is the arrays' last
EDGES = [(128, 2, 65, 64), (256, 2, 64, 257), (256, 1, 129, 131), (192, 3, 71, 128),
         (640, 1, 135, 66), (7168, 2, 1027, 640), (128, 2, 67, 3), (128, 1, 5, 64)]


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,E,K,N", EDGES)
def test_products_to_the_last_row_of_every_array(n, E, K, N, dtype, gather):
    say("edges", n, E, K, N, dtype, gather)
    g = gen(n + K + N)
    X = torch.randn((n, K), generator=g).to(dtype)
    W = (torch.randn((E, N, K), generator=g) * K ** -0.5).to(dtype)
    dY = torch.randn((n, N), generator=g).to(dtype)
    offsets = torch.arange(E + 1, dtype=torch.int32) * (n // E)
    offsets[E] = n
    order = torch.randperm(n, generator=g).int() if gather else None
    at = None if order is None else order.to(DEV)
    Xd, Wd, fd, dYd = X.to(DEV), W.to(DEV), offsets.to(DEV), dY.to(DEV)
    Y = ctr.ctr_expert_dense_fwd(Xd, Wd, None, fd, False, at, 1)
    dX, dW, db = ctr.ctr_expert_dense_bwd(Xd, Wd, fd, dYd, at, 1)
    v, mag = ref.dense_fwd(X, W, None, offsets, False, order, 1, n)
    assert_near(Y, v, stored(v, (K + 3) * U32 * mag, dtype), "Y")
    want = ref.dense_bwd(X, W, offsets, dY, order, 1, False)
    v, mag, L = want["dX"]
    assert_near(dX, v, stored(v, (L + 2) * U32 * mag, dtype), "dX")
    for got, name in ((dW, "dW"), (db, "db")):
        v, mag, L = want[name]
        assert_near(got, v, (L + 2) * U32 * mag, name)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,K,N", [(40, 64, 48), (40, 65, 33), (1500, 64, 128), (1500, 67, 130)])
def test_products_of_an_input_without_rows(n, K, N, dtype):
    """Slots, but no row of X: every slot is outside, and nothing is read at X's address (here
    the end of what is allocated)."""
    say("no input rows", n, K, N, dtype)
    E, lib = 3, ctr.load()
    g = gen(n + K)
    W = torch.randn((E, N, K), generator=g).to(dtype).to(DEV)
    b = torch.randn((E, N), generator=g).to(DEV)
    dY = torch.randn((n, N), generator=g).to(dtype).to(DEV)
    order = torch.arange(n, dtype=torch.int32, device=DEV)
    offsets = torch.tensor([0, n // 4, n // 2, n], dtype=torch.int32, device=DEV)
    block = torch.zeros(4096, dtype=torch.uint8, device=DEV)
    X = block.data_ptr() + block.numel()
    Y, dX = (torch.full((n, c), -3.0, dtype=dtype, device=DEV) for c in (N, K))
    dW = torch.full((E, N, K), -3.0, device=DEV)
    code, stream = ctr._dtype_code(W), torch.cuda.current_stream().cuda_stream
    assert lib.ctr_expert_dense_fwd(X, code, K, 0, order.data_ptr(), 1, offsets.data_ptr(), n, E,
                                    K, W.data_ptr(), b.data_ptr(), N, 1, Y.data_ptr(), N,
                                    stream) == ctr.CTR_OK
    bytes_ = ctypes.c_size_t(ctr.expert_dense_bwd_workspace_bytes(n, E, K, N, code))
    room = torch.empty(bytes_.value, dtype=torch.uint8, device=DEV)
    assert lib.ctr_expert_dense_bwd(X, code, K, 0, order.data_ptr(), 1, offsets.data_ptr(), n, E,
                                    K, W.data_ptr(), N, 1, dY.data_ptr(), N, dX.data_ptr(), K,
                                    dW.data_ptr(), None, room.data_ptr(), ctypes.byref(bytes_),
                                    stream) == ctr.CTR_OK
    expert = torch.bucketize(order, offsets[1:], right=True)
    assert torch.equal(Y, torch.relu(b[expert.long()]).to(dtype))
    assert (dX == 0).all() and (dW == 0).all()


def test_clipping_no_gradients():
    """A step without gradients has norm 0 and scale 1, where there are stats to write them to."""
    say("no gradients")
    for call in (lambda s: ctr.ctr_grad_clip([], 1.0, stats=s),
                 lambda s: ctr.ctr_grad_clip([], 1.0, [], stats=s),
                 lambda s: ctr.ctr_grad_clip_sgd([], [], 0.1, 0.0, stats=s)):
        stats = torch.full((2,), -3.0, device=DEV)
        assert call(stats) is stats and stats.tolist() == [0.0, 1.0]
    with pytest.raises(ValueError):
        ctr.ctr_grad_clip([], 1.0)
    with pytest.raises(ValueError):
        ctr.ctr_grad_clip_sgd([], [torch.zeros(3, device=DEV)], 0.1, 1.0,
                              stats=torch.zeros(2, device=DEV))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", [65, 129, 192, 300])
def test_few_rows_with_most_of_them_in_one_expert(rows, dtype):
    """A request small enough for the few-rows kernel, one of whose experts has more rows than the
    kernel takes at a time."""
    say("few rows", rows, dtype)
    E, n, K, N = 16, 300, 136, 72
    g = gen(rows)
    left, tail = n - rows, (n - rows) // 4      # tail: positions of no expert
    counts = torch.zeros(E, dtype=torch.int32)
    counts[3] = rows
    counts[4:8] = (left - tail) // 4
    counts[11] = left - tail - 4 * ((left - tail) // 4)
    offsets = torch.cat([torch.zeros(1, dtype=torch.int32), counts.cumsum(0).int()])
    X = torch.randn((n, K), generator=g).to(dtype)
    W = (torch.randn((E, N, K), generator=g) * K ** -0.5).to(dtype)
    b = torch.randn((E, N), generator=g)
    order = torch.randperm(n, generator=g).int()
    for o, relu, bias in ((None, True, b), (order, False, None)):
        Y, untouched = canvas(n, N, 8, 0, dtype)
        ctr.ctr_expert_dense_fwd(X.to(DEV), W.to(DEV), None if bias is None else bias.to(DEV),
                                 offsets.to(DEV), relu, None if o is None else o.to(DEV), 1, Y)
        want, mag = ref.dense_fwd(X, W, bias, offsets, relu, o, 1, n)
        assert_near(Y, want, stored(want, (K + 3) * U32 * mag, dtype), "Y")
        untouched()


# the tiles of both kernels: 128 and 256 wide, 64 and 128 at any width
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,k,E,K,N,pad,off", [(150, 2, 5, 136, 72, 8, 8), (150, 2, 5, 61, 33, 3, 1),
                                               (4000, 2, 4, 2048, 96, 0, 0),
                                               (4000, 2, 4, 1031, 40, 0, 0)])
def test_gradient_of_rectified_rows_read_in_place(T, k, E, K, N, pad, off, dtype):
    """x_relu with an order: dX of a position is masked by its token's row."""
    say("rectified rows in place", T, k, E, K, N, pad, off, dtype)
    g = gen(T + K)
    offsets, slots, order = ref.sort(choose(g, T, E, k, 1.0, 0.1), E)
    X = torch.relu(torch.randn((T, K), generator=g)).to(dtype)
    W = (torch.randn((E, N, K), generator=g) * K ** -0.5).to(dtype)
    dY = torch.randn((T * k, N), generator=g).to(dtype)
    dX, untouched = canvas(T * k, K, pad, off, dtype)
    _, dW, db = ctr.ctr_expert_dense_bwd(strided(X, pad, off), W.to(DEV), offsets.to(DEV),
                                         strided(dY, pad, off), order.to(DEV), k, x_relu=True,
                                         dX=dX)
    want = ref.dense_bwd(X, W, offsets, dY, order, k, True)
    v, mag, L = want["dX"]
    assert_near(dX, v, stored(v, (L + 2) * U32 * mag, dtype), "dX")
    untouched()
    for got, name in ((dW, "dW"), (db, "db")):
        v, mag, L = want[name]
        assert_near(got, v, (L + 2) * U32 * mag, name)
