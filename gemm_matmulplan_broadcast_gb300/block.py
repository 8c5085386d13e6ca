"""The layer plans at work together: a pre-norm gated feed-forward block with
a vocabulary product behind it, scored by the log probabilities of given
tokens, and its gradient.

    n1 = layer_norm(x);  h = act(n1 Wg) * (n1 Wu);  y = x + h Wdown
    n2 = layer_norm(y);  z = n2 Whead;              logprob, entropy = score(z, tokens)

Every product and every reduction runs in the library's kernels (the down
projection adds the residual in its epilogue); torch holds the tensors and
adds the two gradients that meet at each residual.

    python -m gemm_matmulplan_broadcast_gb300.block

trains one block for a few steps on fixed tokens, then scores a single token
with its most likely alternatives.
"""

from __future__ import annotations

from .binding import GemmPlan, Plan
from .layers import ROW_DTYPES, GatedPlan, LayerNormPlan, TokenLogProbsPlan

PARAMETERS = ("gamma1", "beta1", "wg", "wu", "wdown", "gamma2", "beta2", "whead")


class ScoredBlock:
    """Plans and activations for ``rows`` tokens.  ``forward`` takes x [rows,
    d_model], int64 tokens [rows] and a dict of PARAMETERS; ``backward`` gives
    a dict of their gradients (and x's, as ``x``) from the gradients of the
    log probabilities and entropies."""

    def __init__(self, rows: int, d_model: int, d_hidden: int, vocab: int, dtype: str = "bfloat16", act: str = "silu",
                 top: int = 0, device="cuda"):
        import torch
        if dtype not in ROW_DTYPES:
            raise ValueError("unsupported dtype %r" % (dtype,))
        t = getattr(torch, dtype)
        self.shape, self.dtype = (rows, d_model, d_hidden, vocab), dtype
        new = lambda *s, of=t: torch.empty(s, dtype=of, device=device)  # noqa: E731
        self.norm1, self.norm2 = LayerNormPlan(rows, d_model, dtype), LayerNormPlan(rows, d_model, dtype)
        self.gate = GatedPlan(rows, d_model, d_hidden, dtype, act)
        self.down = Plan((rows, d_hidden), (d_hidden, d_model), dtype).set_epilogue(residual=True)
        self.head = Plan((rows, d_model), (d_model, vocab), dtype)
        self.score = TokenLogProbsPlan(rows, vocab, dtype, top)
        f32 = torch.float32
        self.n1, self.n2, self.y = (new(rows, d_model) for _ in range(3))
        self.h, self.g, self.u = (new(rows, d_hidden) for _ in range(3))
        self.z = new(rows, vocab)
        self.stats = [new(rows, of=f32) for _ in range(4)]          # mean and rstd of both norms
        self.logprob, self.entropy, self.lse = (new(rows, of=f32) for _ in range(3))
        self.top_logprob = new(rows, top, of=f32) if top else None
        self.top_index = new(rows, top, of=torch.int64) if top else None
        self._back = None

    def forward(self, x, tokens, p):
        """(logprob, entropy), float32 [rows]."""
        m1, r1, m2, r2 = self.stats
        self.x, self.tokens, self.p = x, tokens, p
        self.norm1.forward(x, p["gamma1"], p["beta1"], self.n1, mean=m1, rstd=r1)
        self.gate.forward(self.n1, p["wg"], p["wu"], self.h, G=self.g, U=self.u)
        self.down.execute_fused(self.h, p["wdown"], self.y, R=x)
        self.norm2.forward(self.y, p["gamma2"], p["beta2"], self.n2, mean=m2, rstd=r2)
        self.head.execute(self.n2, p["whead"], self.z)
        self.score.forward(self.z, tokens, self.logprob, entropy=self.entropy, lse=self.lse,
                           top_logprob=self.top_logprob, top_index=self.top_index)
        return self.logprob, self.entropy

    def _backward_plans(self):
        if self._back is None:
            rows, d, f, v = self.shape
            self._back = {
                "n2": GemmPlan((rows, v), (d, v), self.dtype, trans_b=True),          # dz Whead'
                "whead": GemmPlan((rows, d), (rows, v), self.dtype, trans_a=True),    # n2' dz
                "h": GemmPlan((rows, d), (f, d), self.dtype, trans_b=True),           # dy Wdown'
                "wdown": GemmPlan((rows, f), (rows, d), self.dtype, trans_a=True),    # h' dy
            }
        return self._back

    def backward(self, dlogprob, dentropy=None):
        """Gradients of x and of every parameter of the last ``forward``."""
        import torch
        p, plans = self.p, self._backward_plans()
        m1, r1, m2, r2 = self.stats
        like = torch.empty_like
        g = {k: like(p[k]) for k in PARAMETERS}
        dz, dn2, dy, dh, dn1, dx = like(self.z), like(self.n2), like(self.y), like(self.h), like(self.n1), like(self.x)
        self.score.backward(self.z, self.tokens, self.lse, self.entropy, dlogprob, dz, dentropy=dentropy)
        plans["n2"].execute(dz, p["whead"], dn2)
        plans["whead"].execute(self.n2, dz, g["whead"])
        self.norm2.backward(dn2, self.y, p["gamma2"], m2, r2, dy, g["gamma2"], g["beta2"])
        plans["h"].execute(dy, p["wdown"], dh)
        plans["wdown"].execute(self.h, dy, g["wdown"])
        self.gate.backward(dh, self.n1, p["wg"], p["wu"], self.g, self.u, dX=dn1, dWg=g["wg"], dWu=g["wu"])
        self.norm1.backward(dn1, self.x, p["gamma1"], m1, r1, dx, g["gamma1"], g["beta1"])
        g["x"] = dx.add_(dy)                                         # the residual's branch
        return g


def parameters(d_model: int, d_hidden: int, vocab: int, dtype: str = "bfloat16", seed: int = 0, device="cuda"):
    """Random parameters of a block (drawn on the CPU)."""
    import torch
    gen = torch.Generator().manual_seed(seed)
    draw = lambda *s, scale: (torch.randn(s, generator=gen) * scale).to(getattr(torch, dtype)).to(device)  # noqa: E731
    p = {"wg": draw(d_model, d_hidden, scale=d_model ** -0.5), "wu": draw(d_model, d_hidden, scale=d_model ** -0.5),
         "wdown": draw(d_hidden, d_model, scale=d_hidden ** -0.5), "whead": draw(d_model, vocab, scale=d_model ** -0.5)}
    for i in ("1", "2"):
        p["gamma" + i], p["beta" + i] = draw(d_model, scale=0.1) + 1, draw(d_model, scale=0.1)
    return p


def main(rows=512, d_model=1024, d_hidden=2816, vocab=8192, steps=12, rate=0.5, dtype="bfloat16"):
    import torch
    p = parameters(d_model, d_hidden, vocab, dtype)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(rows, d_model, generator=gen, device="cuda").to(p["wg"].dtype)
    tokens = torch.randint(0, vocab, (rows,), generator=gen, device="cuda")
    block = ScoredBlock(rows, d_model, d_hidden, vocab, dtype)
    # the loss: minus the mean log probability, minus a little entropy
    dlogprob = torch.full((rows,), 1.0 / rows, device="cuda")
    for step in range(steps):
        logprob, entropy = block.forward(x, tokens, p)
        print("step %2d  mean log probability %.4f  entropy %.4f" % (step, float(logprob.mean()), float(entropy.mean())))
        grads = block.backward(dlogprob, dentropy=dlogprob * 0.01)
        for k in PARAMETERS:
            p[k].add_(grads[k], alpha=rate)
    one = ScoredBlock(1, d_model, d_hidden, vocab, dtype, top=5)
    one.forward(x[:1], tokens[:1], p)
    print("token %d: log probability %.4f; the likeliest: %s" % (
        int(tokens[0]), float(one.logprob[0]),
        ", ".join("%d (%.4f)" % (i, v) for i, v in zip(one.top_index[0].tolist(), one.top_logprob[0].tolist()))))


if __name__ == "__main__":
    main()
