"""Cases of the click-history operators: a sequence of a user's clicks looked up, normalised,
projected and folded into a state.

Each case is one pass through one operator as a training or serving program calls it.  With
``own`` false the pass is computed in plain form (elementary torch operations in 32 bits);
with ``own`` true by the entry points of ``sparse_embedding_lookup_amd.ctr``.

    embed  rows of a table by token, scaled; training adds the table's whole gradient
    norm   root-mean-square norm with the residual's addition; the output in 8 bits with a scale
           a row ("quant"), or with the gradients of the input and the weight (training)
    scan   a gated linear recurrence over packed sequences with an output gate; training adds
           all gradients; "step" is one token of each of many users
    dense  a product of 8-bit rows with scales, with bias, activation and residual in the
           epilogue
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
F8 = torch.float8_e4m3fn
F8_MAX = 448.0
F8_TINY = 2.0 ** -100               # rows whose largest value is below this take its scale
EPS = 1e-6


def _embed(name, n, V, D, dtype, train, pad):
    return {"name": name, "op": "embed", "n": n, "V": V, "D": D, "dtype": dtype, "train": train,
            "pad": pad}


def _norm(name, n, D, dtype, mode, residual):
    return {"name": name, "op": "norm", "n": n, "D": D, "dtype": dtype, "mode": mode,
            "residual": residual}


def _scan(name, n, B, D, dtype, mode, out_gate):
    return {"name": name, "op": "scan", "n": n, "B": B, "D": D, "dtype": dtype, "mode": mode,
            "out_gate": out_gate}


def _dense(name, M, K, N, out, act, bias, residual):
    return {"name": name, "op": "dense", "M": M, "K": K, "N": N, "dtype": out, "act": act,
            "bias": bias, "residual": residual}


def listed():
    return [
        # one request: a user's last 64 clicks looked up in a table of a million fp32 rows
        _embed("embed_serve", 64, 1000000, 64, "f32", False, 0.0),
        # an ordinary training batch over a bf16 table whose gradient is clipped with the others
        _embed("embed_train", 65536, 100003, 128, "bf16", True, 0.1),
        # the large batch: 32768 histories of 32 clicks over a million rows
        _embed("embed_large", 1048576, 1000000, 128, "bf16", True, 0.0),
        # a small request on its way into the 8-bit product
        _norm("norm_serve", 48, 1024, "bf16", "quant", True),
        # an ordinary training batch of a residual stream
        _norm("norm_train", 65536, 1024, "bf16", "train", True),
        # fp32 training at an odd width, no residual
        _norm("norm_f32", 16387, 479, "f32", "train", False),
        # one click of each of 64 users
        _scan("scan_step", 64, 64, 1024, "bf16", "step", True),
        # one long history: few rows, much of one axis
        _scan("scan_long", 65537, 1, 512, "bf16", "forward", False),
        # a training batch of ragged histories
        _scan("scan_train", 131072, 512, 1024, "bf16", "train", True),
        # one token through one layer: the time to read its weights
        _dense("dense_one", 1, 1024, 1024, "bf16", "none", False, True),
        # a prefill of a few hundred clicks
        _dense("dense_serve", 777, 1024, 1024, "bf16", "silu", True, True),
        # scoring at the width of the large model's interaction
        _dense("dense_large", 32768, 2208, 2048, "bf16", "relu", True, False),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["embed", "norm", "scan", "scan", "dense"])
    dtype = rng.choice(["f32", "bf16", "bf16", "f16"])
    if op == "embed":
        # widths in whole 16-byte vectors mostly, as table rows are; odd ones too
        D = _log(rng, 8, 1024)
        D = D if rng.random() < 0.3 else max(8, D // 8 * 8)
        V = _log(rng, 8, min(1000000, 64000000 // D))
        c = _embed("", _log(rng, 1, min(1000000, 64000000 // D)), V, D, dtype,
                   rng.random() < 0.6, rng.choice([0.0, 0.1]))
    elif op == "norm":
        D = _log(rng, 8, 2208)
        D = D if rng.random() < 0.3 else max(8, D // 8 * 8)
        c = _norm("", _log(rng, 1, min(65536, 32000000 // D)), D, dtype,
                  rng.choice(["train", "train", "quant", "forward"]), rng.random() < 0.6)
    elif op == "scan":
        D = _log(rng, 16, 1024)
        D = D if rng.random() < 0.3 else max(8, D // 8 * 8)
        mode = rng.choice(["train", "forward", "step"])
        if mode == "step":
            n = B = _log(rng, 1, 4096)
        else:
            n = _log(rng, 1, min(131072, 64000000 // D))
            B = _log(rng, 1, n)
        c = _scan("", n, B, D, dtype, mode, rng.random() < 0.6)
    else:
        K = _log(rng, 16, 2208)
        N = _log(rng, 8, 2208)
        if rng.random() < 0.7:
            K, N = max(16, K // 16 * 16), max(8, N // 8 * 8)
        c = _dense("", _log(rng, 1, 32768), K, N, dtype, rng.choice(["none", "relu", "silu", "gelu"]),
                   rng.random() < 0.6, rng.random() < 0.4)
    del c["name"]
    return c


# ------------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(DTYPES[dtype])


def _tokens(g, n, V, pad):
    """Tokens whose frequency falls as one over their rank; `pad` of them no token (-1)."""
    u = torch.rand(n, generator=g, device=DEV, dtype=torch.float64)
    ids = torch.exp(u * math.log(V + 1)).long().sub_(1).clamp_(0, V - 1)
    return torch.where(torch.rand(n, generator=g, device=DEV) < pad, -1, ids)


def _codes(x):
    """8-bit rows of x and the scale of each, padded with zeros to a multiple of 16."""
    x = x.float()
    most = x.abs().amax(1, keepdim=True).clamp(min=F8_TINY)
    q = (x * (F8_MAX / most)).clamp(-F8_MAX, F8_MAX)
    q = torch.nn.functional.pad(q, (0, -x.shape[1] % 16))
    return q.to(F8), (most / F8_MAX).squeeze(1)


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    dt = case["dtype"]
    if case["op"] == "embed":
        n, V, D = case["n"], case["V"], case["D"]
        s["scale"] = math.sqrt(D)
        s["ids"] = _tokens(g, n, V, case["pad"])
        s["table"] = _normal(g, (V, D), dt, D ** -0.5)
        if case["train"]:
            s["dY"] = _normal(g, (n, D), dt)
    elif case["op"] == "norm":
        n, D = case["n"], case["D"]
        s["X"] = _normal(g, (n, D), dt)
        s["R"] = _normal(g, (n, D), dt, 2.0) if case["residual"] else None
        s["weight"] = 1.0 + 0.2 * torch.randn(D, generator=g, device=DEV)
        if case["mode"] == "train":
            s["dY"] = _normal(g, (n, D), dt)
            s["dS"] = _normal(g, (n, D), dt) if case["residual"] else None
    elif case["op"] == "scan":
        n, B, D = case["n"], case["B"], case["D"]
        # gate, value and output gate come side by side out of one projection; channels
        # remember between a few and a few hundred tokens
        P = torch.randn((n, 3 * D), generator=g, device=DEV)
        P[:, :D] += 5.0 * torch.rand(D, generator=g, device=DEV)
        P = P.to(DTYPES[dt])
        s["gate"], s["value"] = P[:, :D], P[:, D:2 * D]
        s["out"] = P[:, 2 * D:] if case["out_gate"] else None
        s["h0"] = torch.randn((B, D), generator=g, device=DEV)
        if case["mode"] == "step":
            return s
        cut = torch.randint(0, n + 1, (B - 1,), generator=g, device=DEV).sort().values
        s["offsets"] = torch.nn.functional.pad(torch.nn.functional.pad(cut, (1, 0)), (0, 1), value=n)
        s["longest"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())
        if case["mode"] == "train":
            s["dY"] = _normal(g, (n, D), dt)
            s["dhN"] = torch.randn((B, D), generator=g, device=DEV)
    else:
        M, K, N = case["M"], case["K"], case["N"]
        s["X8"], s["xs"] = _codes(torch.randn((M, K), generator=g, device=DEV))
        s["W8"], s["ws"] = _codes(torch.randn((N, K), generator=g, device=DEV) * K ** -0.5)
        s["b"] = torch.randn(N, generator=g, device=DEV) * 0.5 if case["bias"] else None
        s["R"] = _normal(g, (M, N), dt) if case["residual"] else None
    return s


# --------------------------------------------------------------------------- plain forms
def _plain_embed(s):
    ids, scale, dt = s["ids"], s["scale"], s["table"].dtype
    here = ids >= 0
    at = ids.clamp(min=0)
    out = {"Y": torch.where(here[:, None], s["table"][at].float() * scale, 0.0).to(dt)}
    if s["train"]:
        d = torch.zeros((s["V"], s["D"]), device=DEV)
        d.index_add_(0, at, torch.where(here[:, None], s["dY"].float() * scale, 0.0))
        out["dtable"] = d
    return out


def _plain_norm(s):
    dt, w = s["X"].dtype, s["weight"]
    out = {}
    S = s["X"]
    if s["R"] is not None:
        out["S"] = S = (S.float() + s["R"].float()).to(dt)
    x = S.float()
    rstd = torch.rsqrt(x.square().mean(1, keepdim=True) + EPS)
    y = x * rstd * w
    if s["mode"] == "quant":
        q, scale = _codes(y)
        # the values that the codes stand for, in the type of what they come from
        out["Y"] = (q[:, :s["D"]].float() * scale[:, None]).to(torch.bfloat16)
        out["y_scale"] = scale
        return out
    out["Y"] = y.to(dt)
    if s["mode"] == "train":
        dy = s["dY"].float()
        out["dweight"] = (dy * x * rstd).sum(0)
        dn = dy * w
        dx = rstd * (dn - x * rstd * rstd * (dn * x).mean(1, keepdim=True))
        if s["dS"] is not None:
            dx = dx + s["dS"].float()
        out["dX"] = dx.to(dt)
    return out


def _affine_scan(a, b, longest):
    """h_t = a_t h_{t-1} + b_t down the first axis, in ceil(log2(longest)) doublings; a is 0
    where a sequence begins."""
    d = 1
    while d < longest:
        b = torch.cat([b[:d], torch.addcmul(b[d:], a[d:], b[:-d])])
        if 2 * d < longest:
            a = torch.cat([a[:d], a[d:] * a[:-d]])
        d *= 2
    return b


def _plain_scan(s):
    dt, o = s["value"].dtype, s["out"]
    f, i, v = torch.sigmoid(s["gate"].float()), torch.sigmoid(-s["gate"].float()), s["value"].float()
    z = None
    if o is not None:
        z = torch.sigmoid(o.float())
    if s["mode"] == "step":
        h = f * s["h0"] + i * v
        y = h if z is None else h * (o.float() * z)
        return {"Y": y.to(dt), "state": h}
    lo, hi = s["offsets"][:-1], s["offsets"][1:]
    there = hi > lo
    first, last = lo[there], hi[there] - 1
    b = i * v
    b[first] += f[first] * s["h0"][there]
    a = f.clone()
    a[first] = 0.0
    h = _affine_scan(a, b, s["longest"])
    del a, b
    y = h if z is None else h * (o.float() * z)
    hN = s["h0"].clone()
    hN[there] = h[last]
    out = {"Y": y.to(dt), "hN": hN}
    del y
    if s["mode"] == "train":
        dy = s["dY"].float()
        if z is not None:
            of = o.float()
            out["dout"] = (dy * h * z * (1.0 + of * (1.0 - z))).to(dt)
            dy = dy * (of * z)
        before = torch.cat([h[:1], h[:-1]])
        before[first] = s["h0"][there]
        # backwards in time: dh_t = dy_t + f_{t+1} dh_{t+1}
        g = dy.clone()
        g[last] += s["dhN"][there]
        a = torch.cat([f[1:], f[:1]])
        a[last] = 0.0
        dh = _affine_scan(a.flip(0), g.flip(0), s["longest"]).flip(0)
        out["dvalue"] = (dh * i).to(dt)
        out["dgate"] = (dh * (before - v) * f * i).to(dt)
        out["dh0"] = s["dhN"].clone()
        out["dh0"][there] = f[first] * dh[first]
    return out


def _act(x, act):
    if act == "relu":
        return torch.relu(x)
    if act == "silu":
        return x * torch.sigmoid(x)
    if act == "gelu":
        return 0.5 * x * (1.0 + torch.erf(x * math.sqrt(0.5)))
    return x


def _plain_dense(s):
    y = (s["X8"].float() @ s["W8"].float().t()) * s["xs"][:, None] * s["ws"]
    if s["b"] is not None:
        y = y + s["b"]
    y = _act(y, s["act"])
    if s["R"] is not None:
        y = y + s["R"].float()
    return {"Y": y.to(DTYPES[s["dtype"]])}


# ----------------------------------------------------------------------- the framework's
def _own_embed(s):
    from sparse_embedding_lookup_amd import ctr
    out = {"Y": ctr.ctr_token_embed_fwd(s["table"], s["ids"], s["scale"])}
    if s["train"]:
        out["dtable"] = ctr.ctr_token_embed_bwd(s["dY"], s["ids"], s["V"], s["scale"])
    return out


def _own_norm(s):
    from sparse_embedding_lookup_amd import ctr
    out = {}
    train = s["mode"] == "train"
    Y, scale, S, rstd = ctr.ctr_rms_norm_fwd(s["X"], s["weight"], s["R"], EPS,
                                             quantize=s["mode"] == "quant", want_rstd=train)
    if s["R"] is not None:
        out["S"] = S
    if s["mode"] == "quant":
        out["Y"] = (Y[:, :s["D"]].float() * scale[:, None]).to(torch.bfloat16)
        out["y_scale"] = scale
        return out
    out["Y"] = Y
    if train:
        out["dX"], out["dweight"] = ctr.ctr_rms_norm_bwd(s["dY"], S, rstd, s["weight"], s["dS"])
    return out


def _own_scan(s):
    from sparse_embedding_lookup_amd import ctr
    if s["mode"] == "step":
        Y, state = ctr.ctr_gated_scan_step(s["gate"], s["value"], s["h0"], out_gate=s["out"],
                                           new_state=True)
        return {"Y": Y, "state": state}
    train = s["mode"] == "train"
    Y, hN, states = ctr.ctr_gated_scan_fwd(s["gate"], s["value"], s["offsets"], s["out"], s["h0"],
                                           want_states=train)
    out = {"Y": Y, "hN": hN}
    if train:
        dgate, dvalue, dout, dh0 = ctr.ctr_gated_scan_bwd(
            s["gate"], s["value"], s["offsets"], s["dY"], states, s["out"], s["h0"], s["dhN"])
        out.update(dgate=dgate, dvalue=dvalue, dh0=dh0)
        if dout is not None:
            out["dout"] = dout
    return out


def _own_dense(s):
    from sparse_embedding_lookup_amd import ctr
    return {"Y": ctr.ctr_quant_dense_fwd(s["X8"], s["xs"], s["W8"], s["ws"], s["b"], s["act"],
                                         s["R"], out_dtype=DTYPES[s["dtype"]])}


def run(state):
    op = state["op"]
    if own:
        return {"embed": _own_embed, "norm": _own_norm, "scan": _own_scan,
                "dense": _own_dense}[op](state)
    return {"embed": _plain_embed, "norm": _plain_norm, "scan": _plain_scan,
            "dense": _plain_dense}[op](state)


# -------------------------------------------------------------------- what a pass cannot spare
def _distinct(n, V):
    """Expected distinct tokens among n of _tokens(): the sum over ranks of 1 - (1 - p)^n, by
    stretches of ranks that grow."""
    got, r = 0.0, 1
    while r <= V:
        to = min(V + 1, max(r + 1, int(r * 1.05)))
        p = math.log(to / r) / math.log(V + 1) / (to - r)
        got += (to - r) * -math.expm1(n * math.log1p(-min(p, 1 - 1e-12)))
        r = to
    return got


def work(case):
    z = BYTES[case["dtype"]]
    if case["op"] == "embed":
        n, V, D = case["n"], case["V"], case["D"]
        kept = n * (1 - case["pad"])
        b, f = n * 8 + _distinct(kept, V) * D * z + n * D * z, 1.0 * n * D
        if case["train"]:
            b, f = b + kept * D * z + V * D * 4, f + 2.0 * n * D
        return {"bytes": b, "flops": f}
    if case["op"] == "norm":
        n, D = case["n"], case["D"]
        b, f = n * D * z * (1 + 2 * case["residual"]) + D * 4, 5.0 * n * D
        b += n * (D + 4) if case["mode"] == "quant" else n * D * z
        if case["mode"] == "train":
            b, f = b + n * D * z * (2 + case["residual"]) + D * 4, f + 10.0 * n * D
        return {"bytes": b, "flops": f}
    if case["op"] == "scan":
        n, B, D, o = case["n"], case["B"], case["D"], case["out_gate"]
        b, f = n * D * z * (3 + o) + 2 * B * D * 4, 12.0 * n * D
        if case["mode"] == "train":
            b, f = b + n * D * z * (3 + o) + 2 * B * D * 4, f + 24.0 * n * D
        return {"bytes": b, "flops": f}
    M, K, N = case["M"], case["K"], case["N"]
    b = M * K + N * K + (M + N) * 4 + M * N * z * (1 + case["residual"]) + N * 4 * case["bias"]
    return {"bytes": b, "flops": 2.0 * M * N * K}


# --------------------------------------------------------------------- the definitions, 64 bits
def _e4m3(x):
    """x to the nearest number of 3 fraction bits and exponents -6 to 8, ties to even."""
    _, e = torch.frexp(x)                          # x = m 2^e, 1/2 <= |m| < 1
    step = torch.ldexp(torch.ones_like(x), (e - 1).clamp(min=-6) - 3)
    return (torch.round(x / step) * step).clamp(-F8_MAX, F8_MAX)


def _exact_scan(s, case):
    lo, hi = s["offsets"][:-1], s["offsets"][1:]
    f, v = torch.sigmoid(s["gate"].double()), s["value"].double()
    h, before = torch.zeros_like(f), torch.zeros_like(f)
    state = s["h0"].double().clone()
    order = torch.argsort(hi - lo, descending=True)
    longest = int((hi - lo).max())
    alive = torch.bincount(hi - lo, minlength=longest + 1).flip(0).cumsum(0).flip(0).tolist()
    lo_by, hi_by = lo[order], hi[order]
    state = state[order]
    for j in range(longest):                       # one token of every history that has one
        m = alive[j + 1]
        rows = lo_by[:m] + j
        before[rows] = state[:m]
        state[:m] = f[rows] * state[:m] + (1 - f[rows]) * v[rows]
        h[rows] = state[:m]
    back = torch.argsort(order)
    out = {"hN": state[back]}
    o = s["out"].double() if s["out"] is not None else None
    gate = o * torch.sigmoid(o) if o is not None else None
    out["Y"] = h * gate if o is not None else h
    if case["mode"] == "train":
        dy = s["dY"].double()
        if o is not None:
            z = torch.sigmoid(o)
            out["dout"] = dy * h * (z + o * z * (1 - z))
            dy = dy * gate
        carry = s["dhN"].double()[order]
        dh = torch.zeros_like(f)
        for j in range(longest):                   # the j-th token from the end
            m = alive[j + 1]
            rows = hi_by[:m] - 1 - j
            got = dy[rows] + carry[:m]
            dh[rows] = got
            carry[:m] = f[rows] * got
        out["dh0"] = carry[back]
        out["dvalue"] = dh * (1 - f)
        out["dgate"] = dh * (before - v) * f * (1 - f)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "embed":
        here = (s["ids"] >= 0).double()[:, None]
        ids = s["ids"] % case["V"]                 # any row in the place of none
        out = {"Y": s["table"].double()[ids] * s["scale"] * here}
        if case["train"]:
            d = torch.zeros((case["V"], case["D"]), dtype=torch.float64, device=DEV)
            order = torch.argsort(ids, stable=True)
            rows, counts = torch.unique_consecutive(ids[order], return_counts=True)
            ends = counts.cumsum(0)
            for c in range(0, case["D"], 64):      # sums of runs as differences of running sums
                x = (s["dY"][:, c:c + 64].double() * here * s["scale"])[order].cumsum(0)
                upto = x[ends - 1]
                upto[1:] = upto[1:] - upto[:-1].clone()
                d[rows, c:c + 64] = upto
            out["dtable"] = d
        return out
    if case["op"] == "norm":
        x = s["X"].double()
        out = {}
        if case["residual"]:
            out["S"] = x + s["R"].double()
            x = (s["X"].float() + s["R"].float()).to(s["X"].dtype).double()   # what is stored
        w, D = s["weight"].double(), case["D"]
        rms = torch.sqrt(torch.linalg.vector_norm(x, dim=1, keepdim=True) ** 2 / D + EPS)
        n = x / rms
        y = n * w
        if case["mode"] == "quant":
            most = torch.clamp(y.abs().max(1, keepdim=True).values, min=F8_TINY)
            out["y_scale"] = (most / F8_MAX).squeeze(1)
            out["Y"] = _e4m3(y * F8_MAX / most) * (most / F8_MAX)
            return out
        out["Y"] = y
        if case["mode"] == "train":
            dn = s["dY"].double() * w
            out["dweight"] = torch.einsum("nd,nd->d", s["dY"].double(), n)
            dx = (dn - n * torch.linalg.vecdot(dn, n)[:, None] / D) / rms
            out["dX"] = dx + s["dS"].double() if case["residual"] else dx
        return out
    if case["op"] == "scan":
        if case["mode"] != "step":
            return _exact_scan(s, case)
        f = 1 / (1 + torch.exp(-s["gate"].double()))
        h = f * s["h0"].double() + (1 - f) * s["value"].double()
        o = s["out"].double() if s["out"] is not None else None
        return {"Y": h if o is None else h * o / (1 + torch.exp(-o)), "state": h}
    X = s["X8"].double() * s["xs"].double()[:, None]
    W = s["W8"].double() * s["ws"].double()[:, None]
    y = X @ W.t()
    if s["b"] is not None:
        y += s["b"].double()
    if case["act"] == "relu":
        y = y.clamp(min=0)
    elif case["act"] == "silu":
        y = y / (1 + torch.exp(-y))
    elif case["act"] == "gelu":
        y = y * torch.special.ndtr(y)
    return {"Y": y + s["R"].double() if s["R"] is not None else y}
