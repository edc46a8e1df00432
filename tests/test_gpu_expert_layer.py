"""ExpertLayer and ExpertClicks: every stage against its definition in 64 bits on the stage's own
inputs (so the bounds are those of the single operators), graph replays against eager steps,
training; and the products at sizes that take the largest tiles, with several tiles a block,
cut reductions and odd widths."""
import numpy as np
import pytest
import torch

from sparse_embedding_lookup_amd import ctr
from sparse_embedding_lookup_amd.experts import ExpertClicks, ExpertLayer, synthetic_clicks
from tests import experts_ref as ref
from tests.experts_ref import U32, assert_near, stored

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

DEV = "cuda"
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def say(*a):
    print(*a, flush=True)


def _fill(layer, seed):
    g = torch.Generator().manual_seed(seed)
    layer.X.copy_(torch.randn(layer.X.shape, generator=g))
    layer.dY.copy_(torch.randn(layer.dY.shape, generator=g))
    layer.b1.copy_(torch.randn(layer.b1.shape, generator=g) * 0.1)
    layer.b2.copy_(torch.randn(layer.b2.shape, generator=g) * 0.1)


# (tokens, dim, hidden, out, experts, k, renormalize, gather)
LAYERS = [(1, 8, 16, 8, 4, 2, True, True), (37, 40, 24, 16, 8, 2, True, False),
          (300, 61, 33, 7, 5, 3, False, True), (1200, 96, 136, 64, 4, 1, False, False),
          (513, 128, 256, 1, 16, 2, True, True)]


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("T,D,N1,N2,E,k,renorm,gather", LAYERS)
def test_layer_stages(T, D, N1, N2, E, k, renorm, gather, dtype):
    say("layer", T, D, N1, N2, E, k, renorm, gather, dtype)
    L = ExpertLayer(T, D, N1, N2, E, k, dtype, renorm, gather)
    _fill(L, T + D)
    before = [p.cpu().clone() for p in L.params]
    L.forward()
    L.backward()
    h = {n: getattr(L, n).cpu() for n in ("X", "logits", "experts", "weights", "offsets", "slots",
                                          "order", "H", "Q", "Y", "dY", "dQ", "dweights", "dH",
                                          "dP", "dlogits", "dXg", "dX", "P")}
    n, m = T * k, int(h["offsets"][E])
    Wg, W1, b1, W2, b2 = before
    all_rows = torch.tensor([0, T])

    def near(name, v, mag, terms):
        assert_near(h[name], v, stored(v, (terms + 3) * U32 * mag, dtype), name)
    near("logits", *ref.dense_fwd(h["X"], Wg, None, all_rows, False, None, 1, T), D)
    we, ww = ref.route_fwd(h["logits"], k, renorm)
    assert torch.equal(h["experts"], we)
    assert_near(h["weights"], ww, (64 + E + 10) * 2 * U32 * ww + 1e-30, "weights")
    for a, b in zip((h["offsets"], h["slots"], h["order"]), ref.sort(we, E)):
        assert torch.equal(a, b)
    order = h["order"] if gather else None
    near("H", *ref.dense_fwd(h["P"], W1, b1, h["offsets"], True, order, k, n), D)
    near("Q", *ref.dense_fwd(h["H"], W2, b2, h["offsets"], False, None, 1, n), N1)
    near("Y", *ref.combine_fwd(h["Q"], h["slots"], h["weights"]), k)
    dQ, dw, mag = ref.combine_bwd(h["dY"], h["Q"], h["slots"], h["weights"])
    near("dQ", dQ, dQ.abs(), 0)
    assert_near(h["dweights"], dw, (N2 + 2) * U32 * mag, "dweights")
    second = ref.dense_bwd(h["H"], W2, h["offsets"], h["dQ"], None, 1, True)
    near("dH", *second["dX"])
    first = ref.dense_bwd(h["P"], W1, h["offsets"], h["dH"], order, k, False)
    near("dP", *first["dX"])
    want = ref.route_bwd(h["logits"], we, h["dweights"], renorm)
    most = h["dweights"].abs().sum(1, keepdim=True).double()
    assert_near(h["dlogits"], want, stored(want, (64 + E + k + 20) * 4 * U32 * most, dtype), "dlogits")
    gate = ref.dense_bwd(h["X"], Wg, all_rows, h["dlogits"], None, 1, False)
    near("dXg", *gate["dX"])
    # the sum of the slots' rows, rounded, plus the gate's part, rounded
    back, bmag = ref.combine_fwd(h["dP"], h["slots"], None)
    half = stored(back, (k + 2) * U32 * bmag, dtype)
    total = back + h["dXg"].double()
    assert_near(h["dX"], total, stored(total, half, dtype), "dX")
    grads = [g.cpu() for g in L.grads]
    for g, (v, mag, terms), name in zip(grads, (gate["dW"], first["dW"], first["db"], second["dW"],
                                                second["db"]), ("dWg", "dW1", "db1", "dW2", "db2")):
        assert_near(g, v, (terms + 2) * U32 * mag, name)
    norm = float(torch.sqrt(sum((g.double() ** 2).sum() for g in grads)))
    lr, max_norm = 0.25, norm / 2
    stats = L.update(lr, max_norm).cpu()
    assert abs(float(stats[0]) - norm) <= 2 * U32 * norm
    c = float(np.float32(lr)) * (float(np.float32(max_norm)) / norm)
    for p, b, g in zip(L.params, before, grads):
        move = c * g.double()
        want = b.double() - move
        assert_near(p, want, stored(want, U32 * want.abs() + 4 * U32 * move.abs(), p.dtype), "param")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_layer_in_a_graph(dtype):
    """Steps replayed from a graph leave the parameters that eager steps leave."""
    say("layer graph", dtype)
    pair = [ExpertLayer(700, 64, 128, 32, 6, 2, dtype) for _ in range(2)]
    for L in pair:
        _fill(L, 5)

    def step(L):
        L.forward()
        L.backward()
        L.update(0.1, 1.0)
    for L in pair:
        step(L)                                 # also marshals the update's call
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(pair[0])
    for _ in range(4):
        graph.replay()
        step(pair[1])
        torch.cuda.synchronize()
        for a, b in zip(pair[0].params + [pair[0].dX, pair[0].Y],
                        pair[1].params + [pair[1].dX, pair[1].Y]):
            assert torch.equal(a, b)


def test_clicks_learn():
    """Training lowers the normalized entropy well below that of the click rate alone (1)."""
    m = ExpertClicks(2048, 32, 64, 8)
    last = []
    for i in range(150):
        x, y = synthetic_clicks(2048, 32, DEV, i)
        m.layer.X.copy_(x)
        m.labels.copy_(y)
        m.step(1.0, 1.0)
        if i >= 140:
            last.append(float(m.ne[2]))
    say("NE", last)
    assert max(last) < 0.8 and all(np.isfinite(last))


# (rows, experts, K, N, dtype): the largest tiles and more of them than blocks for Y, dX and dW;
# odd widths at the same sizes
LARGE = [(9000, 4, 96, 2048, BF16), (9000, 4, 2048, 96, F16), (600, 4, 2048, 2048, BF16),
         (5000, 4, 2048, 2056, BF16), (9000, 5, 97, 2049, F32), (9000, 5, 2049, 97, BF16),
         (3000, 3, 1031, 1027, F16), (40000, 3, 72, 64, BF16), (40000, 3, 33, 65, F32)]


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("n,E,K,N,dtype", LARGE)
def test_large_products(n, E, K, N, dtype, gather):
    say("large", n, E, K, N, dtype, gather)
    g = torch.Generator().manual_seed(n + K)
    share = torch.softmax(1.5 * torch.randn(E, generator=g), 0).cumsum(0)
    offsets = torch.cat([torch.zeros(1), (share * n).floor()]).int()
    offsets[E] = n - 13                         # a few positions of no expert
    order = torch.randperm(n, generator=g).int() if gather else None
    X = torch.randn((n, K), generator=g).to(dtype)
    W = (torch.randn((E, N, K), generator=g) * K ** -0.5).to(dtype)
    dY = torch.randn((n, N), generator=g).to(dtype)
    at = None if order is None else order.to(DEV)
    Xd, Wd, fd, dYd = X.to(DEV), W.to(DEV), offsets.to(DEV), dY.to(DEV)
    Y = ctr.ctr_expert_dense_fwd(Xd, Wd, None, fd, False, at, 1)
    dX, dW, db = ctr.ctr_expert_dense_bwd(Xd, Wd, fd, dYd, at, 1)
    v, mag = ref.dense_fwd(X, W, None, offsets, False, order, 1, n)
    assert_near(Y, v, stored(v, (K + 3) * U32 * mag, dtype), "Y")
    want = ref.dense_bwd(X, W, offsets, dY, order, 1, False)
    v, mag, terms = want["dX"]
    assert_near(dX, v, stored(v, (terms + 2) * U32 * mag, dtype), "dX")
    for got, name in ((dW, "dW"), (db, "db")):
        v, mag, terms = want[name]
        assert_near(got, v, (terms + 2) * U32 * mag, name)


def test_memory_of_a_call_on_another_stream():
    """What the binding allocates for a call on a given stream is not reused by the current
    stream before that call has run."""
    side = torch.cuda.Stream()
    g = torch.Generator().manual_seed(3)
    experts = torch.randint(0, 7, (60000, 2), generator=g, dtype=torch.int32)
    want = ref.sort(experts, 7)
    e = experts.to(DEV)
    a = torch.randn(4096, 4096, device=DEV)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(10):
            a = a @ a * 1e-3                    # the sort waits behind these
    got = ctr.ctr_expert_sort(e, 7, stream=side)
    for _ in range(8):                          # the workspace's memory, were it free
        torch.empty(200 * 7 * 4 + 512, dtype=torch.uint8, device=DEV).fill_(255)
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x.cpu(), y)


def test_gpu_tensors_are_required():
    with pytest.raises(ValueError):
        ctr.ctr_expert_route_fwd(torch.zeros(4, 8), 2)
    with pytest.raises(ValueError):
        ctr.ctr_grad_clip([torch.zeros(4)], 1.0)


# offsets that are not ctr_expert_sort's: every second expert claims all rows
@pytest.mark.parametrize("n,E,K,N,dtype", [(4096, 16, 64, 40, BF16), (4096, 16, 61, 33, BF16),
                                           (2048, 64, 32, 24, F32), (16384, 8, 512, 512, F16)])
def test_offsets_out_of_order_stay_inside(n, E, K, N, dtype):
    say("out of order", n, E, K, N, dtype)
    X = torch.ones(n, K, device=DEV, dtype=dtype)
    dY = torch.ones(n, N, device=DEV, dtype=dtype)
    W = torch.ones(E, N, K, device=DEV, dtype=dtype)
    offsets = torch.tensor([0, n] * (E // 2) + [0], device=DEV, dtype=torch.int32)
    size = ctr.expert_dense_bwd_workspace_bytes(n, E, K, N, ctr._dtype_code(X))
    guard = 1 << 20
    room = torch.full((size + guard,), 0x5A, device=DEV, dtype=torch.uint8)
    ctr.ctr_expert_dense_bwd(X, W, offsets, dY, workspace=room[:size])
    ctr.ctr_expert_dense_fwd(X, W, None, offsets, False)
    torch.cuda.synchronize()
    assert bool((room[size:] == 0x5A).all())
    # and in order again, in the same workspace
    offsets = torch.arange(E + 1, device=DEV, dtype=torch.int32) * (n // E)
    _, dW, db = ctr.ctr_expert_dense_bwd(X, W, offsets, dY, workspace=room[:size])
    assert bool((dW == n // E).all()) and bool((db == n // E).all())


def test_memory_of_a_prepared_call_on_another_stream():
    """The same of a prepared call that is gone before its work has run."""
    say("prepared on another stream")
    side = torch.cuda.Stream()
    g = torch.Generator().manual_seed(4)
    experts = torch.randint(0, 7, (60000, 2), generator=g, dtype=torch.int32)
    want = ref.sort(experts, 7)
    e = experts.to(DEV)
    a = torch.randn(4096, 4096, device=DEV)
    call = ctr.ctr_expert_sort(e, 7, prepare=True)
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(10):
            a = a @ a * 1e-3                    # the sort waits behind these
    got = call(stream=side)
    del call
    for _ in range(8):                          # the workspace's memory, were it free
        torch.empty(200 * 7 * 4 + 512, dtype=torch.uint8, device=DEV).fill_(255)
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x.cpu(), y)
    # the outputs of a call that nobody keeps
    call = ctr.ctr_expert_sort(e, 7, prepare=True)
    places = [t.data_ptr() for t in call.result]
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(10):
            a = a @ a * 1e-3
        call()
    del call
    taken = [torch.empty_like(t) for t in got]
    assert not set(places) & {t.data_ptr() for t in taken}
    torch.cuda.synchronize()


def _operators(stream=None):
    """One small call of every operator: names and calls that take the stream."""
    g = torch.Generator().manual_seed(6)
    T, E, k, K, N = 300, 5, 2, 72, 40
    logits = torch.randn((T, E), generator=g).to(DEV)
    X, Q = (torch.randn((r, K), generator=g).to(DEV) for r in (T, T * k))
    W, dY = torch.randn((E, N, K), generator=g).to(DEV), torch.randn((T * k, N), generator=g).to(DEV)
    dw = torch.randn((T, k), generator=g).to(DEV)
    experts, weights = ctr.ctr_expert_route_fwd(logits, k)
    offsets, slots, order = ctr.ctr_expert_sort(experts, E)
    return [
        ("route_fwd", lambda **a: ctr.ctr_expert_route_fwd(logits, k, **a)),
        ("route_bwd", lambda **a: ctr.ctr_expert_route_bwd(logits, experts, weights, dw, **a)),
        ("sort", lambda **a: ctr.ctr_expert_sort(experts, E, **a)),
        ("dispatch", lambda **a: ctr.ctr_expert_dispatch(X, slots, offsets, **a)),
        ("combine_fwd", lambda **a: ctr.ctr_expert_combine_fwd(Q, slots, weights, **a)),
        ("combine_bwd", lambda **a: ctr.ctr_expert_combine_bwd(X, Q, slots, offsets, weights, **a)),
        ("dense_fwd", lambda **a: ctr.ctr_expert_dense_fwd(X, W, None, offsets, True, order, k, **a)),
        ("dense_bwd", lambda **a: ctr.ctr_expert_dense_bwd(X, W, offsets, dY, order, k, **a)),
        ("clip", lambda **a: ctr.ctr_grad_clip([dw, X], 0.5, [torch.empty_like(dw),
                                                             torch.empty_like(X)], **a)),
        ("clip_sgd", lambda **a: ctr.ctr_grad_clip_sgd([dw], [dw.clone()], 0.1, 0.5, **a))]


@pytest.mark.parametrize("prepare", [False, True])
def test_calls_on_another_stream_take_none_of_the_current_streams_memory(prepare):
    """Memory that was freed while the current stream still writes to it is not given to a call on
    another stream, which does not wait for that."""
    say("memory under way", prepare)
    side = torch.cuda.Stream()
    calls = _operators()
    want = [tuple(ctr._tensors(call())) for _, call in calls]
    sizes = sorted({t.numel() * t.element_size() for w in want for t in w})
    torch.cuda.synchronize()
    a = torch.randn(4096, 4096, device=DEV)
    for (name, call), right in zip(calls, want):
        torch.cuda.synchronize()
        for _ in range(10):
            a = a @ a * 1e-3
        places = set()
        for size in sizes + [256, 16384, 1 << 20]:
            for _ in range(4):
                held = torch.empty(size, dtype=torch.uint8, device=DEV)
                held.fill_(255)                 # waits behind the products
                places.add(held.untyped_storage().data_ptr())
                del held
        got = call(stream=side, prepare=prepare)
        if prepare:
            got = got(stream=side)
        got = tuple(ctr._tensors(got))
        assert not places & {t.untyped_storage().data_ptr() for t in got}, name
        torch.cuda.synchronize()
        assert len(got) == len(right) > 0
        for x, y in zip(got, right):
            assert torch.equal(x, y), name


def test_a_captured_step_after_updates_of_other_rates():
    """Steps replayed from a graph do not depend on what eager updates of other rates, and memory
    allocated after them, hold."""
    say("captured step, other rates")
    pair = [ExpertLayer(200, 32, 48, 16, 4, 2, F32) for _ in range(2)]
    for L in pair:
        _fill(L, 8)

    def step(L, lr):
        L.forward()
        L.backward()
        L.update(lr, 0.5)
    for L in pair:
        step(L, 0.1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(pair[0], 0.1)
    size = ctr.grad_clip_workspace_bytes(len(pair[0].grads))
    for lr in (0.3, 0.05, 0.2):
        for L in pair:
            step(L, lr)
        held = [torch.full((size,), 255, dtype=torch.uint8, device=DEV) for _ in range(8)]
        graph.replay()
        step(pair[1], 0.1)
        torch.cuda.synchronize()
        assert all(bool((h == 255).all()) for h in held)
        for a, b in zip(pair[0].params, pair[1].params):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("gather", [True, False])
def test_layer_without_tokens(gather, dtype):
    """An empty batch: gradients of zero, norm 0, parameters as they were."""
    say("layer without tokens", gather, dtype)
    L = ExpertLayer(0, 16, 24, 1, 4, 2, dtype, gather=gather)
    before = [p.clone() for p in L.params]
    for g in L.grads:
        g.fill_(-3.0)
    assert L.forward().shape == (0, 1) and L.backward().shape == (0, 16)
    assert all(bool((g == 0).all()) for g in L.grads)
    assert L.update(0.1, 1.0).tolist() == [0.0, 1.0]
    assert all(torch.equal(a, b) for a, b in zip(L.params, before))


def test_calls_on_another_stream_inside_a_capture():
    """stream= in a captured pass: forked, joined, and replayed like the eager one."""
    say("another stream, captured")
    side = torch.cuda.Stream()
    calls = [c for name, c in _operators() if not name.startswith("clip")]
    want = [tuple(ctr._tensors(call())) for call in calls]
    torch.cuda.synchronize()

    def forked():
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        got = [tuple(ctr._tensors(call(stream=side))) for call in calls]
        here.wait_stream(side)
        return got
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = forked()
    for _ in range(3):
        for t in [t for g in got for t in g]:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for passed in (got, forked()):
            torch.cuda.synchronize()
            for a, b in zip([t for g in passed for t in g], [t for w in want for t in w]):
                assert torch.equal(a, b)
