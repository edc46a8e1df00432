"""A mixture of two-layer perceptrons as a layer of the click model, as a chain of libctr calls.

    logits = X Wg^T, the k experts of each token and their weights   gate and router
    slots sorted by expert                                          sort
    H = relu(W1[e] x + b1[e]),  Q = W2[e] H + b2[e]                 the experts' two products
    Y = sum_j w_j Q[slot j]                                         weighted sum back

The backward pass gives dX and the gradients of every parameter (fp32), and `update` clips them
by their global norm and takes the SGD step.  Parameters and rows are of one type (fp32, bf16 or
fp16), biases fp32.  The first product reads the tokens' rows in place, or with
``gather=False`` rows copied into the experts' order.

What passes from call to call is of the rows' type too, as the calls take it: each result is
rounded to it once, from fp32 sums.  So are the gate's logits, which the experts are chosen by,
and the two parts of dX, the experts' and the gate's, whose sum is rounded again.  A layer that
has to choose by fp32 logits is an fp32 layer.

Every call is marshalled once on buffers that stay, so a step allocates nothing and can be
captured into a HIP graph.  Torch adds the gate's part of dX; everything else is libctr.

    python -m sparse_embedding_lookup_amd.experts          # trains on synthetic clicks
"""
from __future__ import annotations

import argparse
from typing import List, Optional

import torch

from . import ctr


class ExpertLayer:
    """Device state of the layer for batches of `tokens` rows: parameters, activations,
    gradients.  Write the rows into ``X`` before forward(), which fills ``Y``; write the
    gradient of Y into ``dY`` before backward(), which fills ``dX`` and ``grads``."""

    def __init__(self, tokens: int, dim: int, hidden: int, out: int, num_experts: int, k: int = 2,
                 dtype: torch.dtype = torch.bfloat16, renormalize: bool = True,
                 gather: bool = True, device="cuda", seed: int = 0):
        T, E, n = tokens, num_experts, tokens * k
        dev = self.device = torch.device(device)
        g = torch.Generator(device=dev).manual_seed(seed)

        def weights(*shape):
            return (torch.randn(shape, generator=g, device=dev) * shape[-1] ** -0.5).to(dtype)

        def rows(r, c, t=dtype):
            return torch.zeros((r, c), dtype=t, device=dev)

        f32, i32 = torch.float32, torch.int32
        self.k, self.num_experts, self.gather = k, E, gather
        self.Wg = weights(1, E, dim)
        self.W1, self.b1 = weights(E, hidden, dim), rows(E, hidden, f32)
        self.W2, self.b2 = weights(E, out, hidden), rows(E, out, f32)
        self.X, self.Y, self.dX, self.dY = rows(T, dim), rows(T, out), rows(T, dim), rows(T, out)
        self.logits, self.dlogits = rows(T, E), rows(T, E)
        self.experts, self.weights, self.dweights = rows(T, k, i32), rows(T, k, f32), rows(T, k, f32)
        self.offsets = torch.zeros(E + 1, dtype=i32, device=dev)
        self.slots, self.order = rows(T, k, i32), torch.zeros(n, dtype=i32, device=dev)
        self.all_rows = torch.tensor([0, T], dtype=i32, device=dev)      # the gate: one "expert"
        self.P = self.X if gather else rows(n, dim)
        self.H, self.dH = rows(n, hidden), rows(n, hidden)
        self.Q, self.dQ = rows(n, out), rows(n, out)
        self.dP, self.dXg = rows(n, dim), rows(T, dim)
        self.params: List[torch.Tensor] = [self.Wg, self.W1, self.b1, self.W2, self.b2]
        self.grads = [torch.zeros(p.shape, dtype=f32, device=dev) for p in self.params]
        self.stats = torch.zeros(2, dtype=f32, device=dev)
        # a graph that holds an update uses this memory after the call itself has gone
        self.clip_room = torch.empty(ctr.grad_clip_workspace_bytes(len(self.grads)),
                                     dtype=torch.uint8, device=dev)
        self._update = {}

        p = dict(prepare=True)
        order = dict(order=self.order, k=k) if gather else {}
        dWg, dW1, db1, dW2, db2 = self.grads
        self._forward = [
            ctr.ctr_expert_dense_fwd(self.X, self.Wg, None, self.all_rows, False, Y=self.logits, **p),
            ctr.ctr_expert_route_fwd(self.logits, k, renormalize, self.experts, self.weights, **p),
            ctr.ctr_expert_sort(self.experts, E, self.offsets, self.slots, self.order, **p),
            ctr.ctr_expert_dense_fwd(self.P, self.W1, self.b1, self.offsets, True, Y=self.H,
                                     **order, **p),
            ctr.ctr_expert_dense_fwd(self.H, self.W2, self.b2, self.offsets, False, Y=self.Q, **p),
            ctr.ctr_expert_combine_fwd(self.Q, self.slots, self.weights, self.Y, **p)]
        if not gather:
            self._forward.insert(3, ctr.ctr_expert_dispatch(self.X, self.slots, self.offsets,
                                                            self.P, **p))
        self._backward = [
            ctr.ctr_expert_combine_bwd(self.dY, self.Q, self.slots, self.offsets, self.weights,
                                       self.dQ, self.dweights, **p),
            ctr.ctr_expert_dense_bwd(self.H, self.W2, self.offsets, self.dQ, x_relu=True,
                                     dX=self.dH, dW=dW2, db=db2, **p),
            ctr.ctr_expert_dense_bwd(self.P, self.W1, self.offsets, self.dH, dX=self.dP, dW=dW1,
                                     db=db1, **order, **p),
            ctr.ctr_expert_combine_fwd(self.dP, self.slots, None, self.dX, **p),
            ctr.ctr_expert_route_bwd(self.logits, self.experts, self.weights, self.dweights,
                                     renormalize, self.dlogits, **p),
            ctr.ctr_expert_dense_bwd(self.X, self.Wg, self.all_rows, self.dlogits, bias=False,
                                     dX=self.dXg, dW=dWg, **p)]

    def forward(self) -> torch.Tensor:
        for call in self._forward:
            call()
        return self.Y

    def backward(self) -> torch.Tensor:
        for call in self._backward:
            call()
        return self.dX.add_(self.dXg)

    def update(self, lr: float, max_norm: float) -> torch.Tensor:
        """The SGD step with gradients clipped to `max_norm`; returns [norm, scale] (device).  A
        captured step keeps the lr and max_norm it was captured with."""
        call = self._update.get((lr, max_norm))
        if call is None:
            self._update.clear()
            call = ctr.ctr_grad_clip_sgd(self.grads, self.params, lr, max_norm, self.stats,
                                         self.clip_room, prepare=True)
            self._update[lr, max_norm] = call
        return call()


class ExpertClicks:
    """Training of click probabilities by experts with one output: the layer's Y is the logit."""

    def __init__(self, tokens: int, dim: int, hidden: int, num_experts: int, k: int = 2, **layer):
        self.layer = L = ExpertLayer(tokens, dim, hidden, 1, num_experts, k, torch.float32, **layer)
        self.labels = torch.zeros(tokens, device=L.device)
        self.ne = torch.zeros(3, device=L.device)
        self._head = ctr.ctr_logistic_ne(L.Y, self.labels, None, L.dY, self.ne, prepare=True)

    def step(self, lr: float, max_norm: float) -> None:
        """forward, head, backward and update on the batch in layer.X and labels; the batch's
        normalized entropy is ne[2]."""
        self.layer.forward()
        self._head()
        self.layer.backward()
        self.layer.update(lr, max_norm)


def synthetic_clicks(rows: int, dim: int, device, seed: int, kinds: int = 4):
    """Rows of `kinds` kinds, each kind with a rule of its own for its clicks: (X, labels)."""
    g = torch.Generator(device=device).manual_seed(1234)             # the rules
    centre = torch.randn((kinds, dim), generator=g, device=device)
    rule = torch.randn((kinds, dim), generator=g, device=device) * (4.0 * dim ** -0.5)
    g = torch.Generator(device=device).manual_seed(seed)
    kind = torch.randint(0, kinds, (rows,), generator=g, device=device)
    x = torch.randn((rows, dim), generator=g, device=device)
    p = torch.sigmoid((x * rule[kind]).sum(1))
    return x + centre[kind], (torch.rand(rows, generator=g, device=device) < p).float()


def main(argv: Optional[list] = None) -> None:
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in (("tokens", 4096), ("dim", 64), ("hidden", 128), ("experts", 8), ("k", 2),
                        ("steps", 200)):
        ap.add_argument("--" + name, type=int, default=value)
    ap.add_argument("--lr", type=float, default=1.0)
    ap.add_argument("--max-norm", type=float, default=1.0)
    a = ap.parse_args(argv)
    m = ExpertClicks(a.tokens, a.dim, a.hidden, a.experts, a.k)
    for i in range(a.steps):
        x, y = synthetic_clicks(a.tokens, a.dim, m.layer.device, i)
        m.layer.X.copy_(x)
        m.labels.copy_(y)
        m.step(a.lr, a.max_norm)
        if i % 20 == 0 or i == a.steps - 1:
            norm, scale = m.layer.stats.tolist()
            print("step %4d  NE %.4f  gradient norm %.3f  scale %.3f"
                  % (i, float(m.ne[2]), norm, scale), flush=True)


if __name__ == "__main__":
    main()
