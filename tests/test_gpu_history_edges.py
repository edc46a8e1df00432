"""The click-history operators at the calls their documentation allows that the sweeps of sizes do
not reach: rows far apart in memory, calls at the same time, slots left alone, derivatives of what
the GPU itself computes."""
import pytest
import torch

from sparse_embedding_lookup_amd import ctr
from sparse_embedding_lookup_amd.history import HistoryEncoder, HistoryServer
from tests import history_ref as ref
from tests.history_ref import assert_near, stored

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

DEV = "cuda"
F32, BF16, F8 = torch.float32, torch.bfloat16, torch.float8_e4m3fn


def say(*a):
    print(*a, flush=True)


def normal(seed, *shape, dtype=F32, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def far(a, stride):
    """a on the GPU, its rows `stride` elements apart."""
    buf = torch.empty(((a.shape[0] - 1) * stride + a.shape[1],), dtype=a.dtype, device=DEV)
    out = buf.as_strided(a.shape, (stride, 1))
    out.copy_(a)
    return out


def test_rows_past_32_bits():
    """Rows whose last lies beyond 2^32 bytes, and 2^31 elements, of the first: as close ones."""
    n, D, stride = 70, 40, (1 << 25) + 8
    assert (n - 1) * stride > 1 << 31
    say("far rows", n, D, stride)
    x, y = normal(1, n, D, dtype=BF16), normal(2, n, D, dtype=BF16)
    w, off = normal(3, D).to(DEV), torch.tensor([0, 33, n], device=DEV)
    near = ctr.ctr_gated_scan_fwd(x.to(DEV), y.to(DEV), off, want_states=True)
    back = ctr.ctr_gated_scan_bwd(x.to(DEV), y.to(DEV), off, x.to(DEV), near[2])
    step = ctr.ctr_gated_scan_step(x.to(DEV), y.to(DEV), torch.ones(n, D, device=DEV))
    norm = ctr.ctr_rms_norm_fwd(x.to(DEV), w, want_rstd=True)
    norm_back = ctr.ctr_rms_norm_bwd(y.to(DEV), x.to(DEV), norm[3], w)
    codes = ctr.ctr_quantize_rows(x.to(DEV))
    fx, out = far(x, stride), far(y, stride)
    got = ctr.ctr_gated_scan_fwd(fx, y.to(DEV), off, want_states=True, Y=out)
    assert all(torch.equal(a, b) for a, b in zip(near, got))
    got = ctr.ctr_gated_scan_bwd(fx, y.to(DEV), off, x.to(DEV), near[2], dgate=out)
    assert torch.equal(back[0], got[0]) and torch.equal(back[1], got[1])
    got = ctr.ctr_gated_scan_step(fx, y.to(DEV), torch.ones(n, D, device=DEV), Y=out)
    assert torch.equal(step[0], got[0])
    got = ctr.ctr_rms_norm_fwd(fx, w, want_rstd=True, Y=out)
    assert torch.equal(norm[0], got[0]) and torch.equal(norm[3], got[3])
    got = ctr.ctr_rms_norm_bwd(y.to(DEV), fx, norm[3], w, dX=out)
    assert torch.equal(norm_back[0], got[0]) and torch.equal(norm_back[1], got[1])
    got = ctr.ctr_quantize_rows(fx)
    assert torch.equal(codes[0].float(), got[0].float()) and torch.equal(codes[1], got[1])
    ids = torch.randint(0, 9, (n,), generator=torch.Generator().manual_seed(4)).to(DEV)
    assert torch.equal(ctr.ctr_token_embed_bwd(fx, ids, 9),
                       ctr.ctr_token_embed_bwd(x.to(DEV), ids, 9))
    table = normal(5, 9, D, dtype=BF16).to(DEV)
    assert torch.equal(ctr.ctr_token_embed_fwd(table, ids, 2.0, out),
                       ctr.ctr_token_embed_fwd(table, ids, 2.0))


@pytest.mark.parametrize("M,N", [(1100, 96), (60, 96), (96, 1100)])
def test_codes_past_32_bits(M, N):
    """Rows of codes that lie as far apart as is allowed."""
    K, stride = 80, (1 << 22) - 16
    say("far codes", M, N)
    X, W = normal(1, M, K).to(DEV), normal(2, N, K).to(DEV)
    (Xq, xs), (Wq, ws) = ctr.ctr_quantize_rows(X), ctr.ctr_quantize_rows(W)
    want = ctr.ctr_quant_dense_fwd(Xq, xs, Wq, ws)
    if M > N:
        Xq = far(Xq, stride)
    else:
        Wq = far(Wq, stride)
    assert torch.equal(ctr.ctr_quant_dense_fwd(Xq, xs, Wq, ws), want)


def test_calls_at_the_same_time():
    """Scans, sorts and products on four streams at once, each with its own memory: as one by
    one."""
    say("at the same time")
    n, D, V = 20000, 256, 5000
    streams = [torch.cuda.Stream() for _ in range(4)]
    sets, want = [], []
    for i in range(4):
        g, v, o = (normal(10 * i + j, n, D, dtype=BF16).to(DEV) for j in range(3))
        off = torch.tensor([0, 1000 * i, 9000 + i, n], device=DEV)
        ids = torch.randint(-1, V, (n,), generator=torch.Generator().manual_seed(i)).to(DEV)
        sets.append((g, v, o, off, ids))

    def run(g, v, o, off, ids, **s):
        Y, hN, st = ctr.ctr_gated_scan_fwd(g, v, off, o, want_states=True, **s)
        back = ctr.ctr_gated_scan_bwd(g, v, off, Y, st, o, **s)
        d = ctr.ctr_token_embed_bwd(back[0], ids, V, **s)
        Q, q = ctr.ctr_quantize_rows(back[1], **s)
        return Y, hN, *back, d, ctr.ctr_quant_dense_fwd(Q, q, Q[:D], q[:D], **s)
    for x in sets:
        want.append(run(*x))
        torch.cuda.synchronize()
    for _ in range(3):
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
        got = [run(*x, stream=s) for x, s in zip(sets, streams)]
        for s in streams:
            torch.cuda.current_stream().wait_stream(s)
        for a, b in zip(want, got):
            for x, y in zip(a, b):
                assert torch.equal(x, y)


def test_slots_that_no_row_names_stay():
    """A step into other memory, with slots named twice and slots that are not there."""
    say("slots")
    B, D, slots = 40, 66, 30
    g, v = normal(1, B, D), normal(2, B, D)
    state = normal(3, slots, D)
    index = torch.randint(-3, 20, (B,), generator=torch.Generator().manual_seed(4)).int()
    index[7] = slots + 5
    keep, new = state.to(DEV), torch.full((slots, D), -3.0, device=DEV)
    Y, to = ctr.ctr_gated_scan_step(g.to(DEV), v.to(DEV), keep, index.to(DEV), new_state=new)
    want, err, s, es = ref.scan_step(g, v, state, index)
    assert to is new and torch.equal(keep.cpu(), state)
    assert_near(Y, want, stored(want, err, F32), "Y")
    named = torch.zeros(slots, dtype=torch.bool)
    named[index[(index >= 0) & (index < slots)].long()] = True
    assert_near(new[named.to(DEV)], s[named], es[named] + 1e-30, "new state")
    assert (new[~named.to(DEV)] == -3).all()
    assert (Y[((index < 0) | (index >= slots)).to(DEV)] == 0).all()


def slope(loss, x, move, h=2.0 ** -7):
    """The derivative of loss (64 bits) along move, from four values: h^4 beside it."""
    f = [loss(x + k * h * move) for k in (-2, -1, 1, 2)]
    return float((f[0] - 8 * f[1] + 8 * f[2] - f[3]) / (12 * h))


def test_scan_gradients_are_the_forwards_differences():
    """The kernels' gradients against differences of the kernels' own forward in fp32.  Some twenty
    roundings of 2^-24 in each value, 18 / 12 h of them in the difference: 2.3e-4 of the terms; its
    own error, h^4 / 30 of the fifth derivative, is below 1e-8 of them for moves of one."""
    say("scan differences")
    n, D = 150, 5
    off = torch.tensor([0, 70, 70, 139, 150], device=DEV)
    x = [normal(i, n, D).to(DEV) for i in range(3)] + [normal(3, 4, D).to(DEV)]
    dY, dhN = normal(4, n, D).to(DEV), normal(5, 4, D).to(DEV)

    def forward(g, v, o, h0):
        Y, hN, st = ctr.ctr_gated_scan_fwd(g, v, off, o, h0, want_states=True)
        return (Y.double() * dY).sum() + (hN.double() * dhN).sum(), st
    st = forward(*x)[1]
    got = ctr.ctr_gated_scan_bwd(x[0], x[1], off, dY, st, x[2], x[3], dhN)
    for i in range(4):
        move = normal(6 + i, *x[i].shape).to(DEV)
        want = slope(lambda y: forward(*[y if j == i else x[j] for j in range(4)])[0], x[i], move)
        terms = (got[i].double() * move)
        assert abs(want - float(terms.sum())) <= 1e-3 * float(terms.abs().sum()), i


def test_norm_gradients_are_the_forwards_differences():
    say("norm differences")
    n, D = 60, 33
    X, w = normal(1, n, D).to(DEV), (1 + 0.2 * normal(2, D)).to(DEV)
    dY = normal(3, n, D).to(DEV)

    def loss(x, w):
        return (ctr.ctr_rms_norm_fwd(x, w)[0].double() * dY).sum()
    _, _, S, rstd = ctr.ctr_rms_norm_fwd(X, w, want_rstd=True)
    dX, dw = ctr.ctr_rms_norm_bwd(dY, S, rstd, w)
    for x, g, f in ((X, dX, lambda y: loss(y, w)), (w, dw, lambda y: loss(X, y))):
        move = normal(4, *x.shape).to(DEV)
        terms = g.double() * move
        assert abs(slope(f, x, move) - float(terms.sum())) <= 1e-3 * float(terms.abs().sum())


def test_many_empty_sequences():
    """More sequences than rows, and more than the marks' search holds in LDS."""
    n, B, D = 700, 9000, 6
    say("many sequences", n, B, D)
    g = torch.Generator().manual_seed(1)
    off = torch.cat([torch.zeros(1, dtype=torch.int64),
                     torch.randint(0, n + 1, (B - 1,), generator=g).sort().values,
                     torch.tensor([n])])
    gate, value, dY = (normal(i, n, D) for i in (2, 3, 4))
    h0, dhN = normal(5, B, D), normal(6, B, D)
    want = ref.scan(gate, value, off.tolist(), None, h0, dY, dhN)
    offd = off.to(DEV)
    Y, hN, st = ctr.ctr_gated_scan_fwd(gate.to(DEV), value.to(DEV), offd, None, h0.to(DEV),
                                       want_states=True)
    back = ctr.ctr_gated_scan_bwd(gate.to(DEV), value.to(DEV), offd, dY.to(DEV), st, h0=h0.to(DEV),
                                  dhN=dhN.to(DEV))
    for name, got in (("Y", Y), ("hN", hN), ("dgate", back[0]), ("dvalue", back[1]),
                      ("dh0", back[3])):
        right, err = want[name]
        assert_near(got, right, stored(right, err, F32), name)


@pytest.mark.parametrize("dtype,D", [(F32, 37), (torch.float16, 50), (BF16, 129)])
def test_server_of_odd_widths(dtype, D):
    """Widths that are no whole 16-byte pieces, users without clicks, a step in a graph: what the
    training side and eager calls give.  (Each 8-bit operand is 2^-4 off at most, eight products.)"""
    say("server", dtype, D)
    B, V, n = 5, 30, 61
    E = HistoryEncoder(n, B, V, D, 2, dtype, seed=3)
    ids = torch.randint(0, V, (n,), generator=torch.Generator().manual_seed(4)).to(DEV)
    off = torch.tensor([0, 20, 20, 21, 50, n], device=DEV)
    E.ids.copy_(ids)
    E.offsets.copy_(off)
    want = E.forward()
    server, other = HistoryServer(E, 8), HistoryServer(E, 8)
    users = [6, 1, 0, 7, 3]
    for s in (server, other):
        U = s.prefill(ids, off, users)
        assert (U.float() - want).norm() <= 8 * 2.0 ** -4 * want.norm()
        assert not U[1].any() and not s.state[0][1].any()
    click = torch.tensor([3, 9, 3], device=DEV)
    index = torch.tensor([6, 1, 6], dtype=torch.int32, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = server.step(click, index)
    for t in range(4):
        click.fill_(t)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, other.step(click, index))
        for a, b in zip(server.state, other.state):
            assert torch.equal(a, b)


@pytest.mark.parametrize("n,V,D,dtype", [(300001, 5000, 8, BF16), (270000, 3000001, 4, F32),
                                         (1000003, 60, 12, torch.float16)])
def test_embed_bwd_of_many_tokens(n, V, D, dtype):
    """Sorts of many tiles, of one to three digits, with a quarter of all tokens the same."""
    say("many tokens", n, V, D, dtype)
    g = torch.Generator().manual_seed(1)
    ids = torch.randint(-1, V + 1, (n,), generator=g)
    ids[torch.rand(n, generator=g) < 0.25] = V // 3
    dY = normal(2, n, D, dtype=dtype)
    want, m, terms = ref.embed_bwd(dY, ids, V, 1.5)
    for kind in (torch.int64, torch.int32):
        got = ctr.ctr_token_embed_bwd(dY.to(DEV), ids.to(kind).to(DEV), V, 1.5)
        assert_near(got, want, (terms + 4) * 2.0 ** -24 * m, "dtable")


@pytest.mark.parametrize("K", [1152, 1168, 1280, 1424, 1600, 1664])
@pytest.mark.parametrize("out", [F32, BF16, torch.float16])
def test_dense_large_tiles_of_any_depth(K, out):
    """The largest tiles at every number of rounds that their loop ends with, ragged ones too."""
    M, N = 4100, 4099
    say("large tiles", K, out)
    Xq, xs = ctr.ctr_quantize_rows(normal(1, M, K, dtype=BF16, scale=2.0).to(DEV))
    Wq, ws = ctr.ctr_quantize_rows(normal(2, N, K, dtype=BF16, scale=K ** -0.5).to(DEV))
    b, R = normal(3, N), normal(4, M, N, dtype=out)
    rows = torch.cat([torch.arange(0, M, 331), torch.arange(M - 5, M)])
    for act, bias, res in (("silu", True, True), ("relu", False, False)):
        Y = ctr.ctr_quant_dense_fwd(Xq, xs, Wq, ws, b.to(DEV) if bias else None, act,
                                    R.to(DEV) if res else None, out_dtype=out)
        want, err = ref.dense(Xq.cpu()[rows], xs.cpu()[rows], Wq.cpu(), ws.cpu(),
                              b if bias else None, act, R[rows] if res else None, out)
        assert_near(Y.cpu()[rows], want, stored(want, err, out), act)
