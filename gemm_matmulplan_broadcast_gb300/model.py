"""A small language model made of the library's plans, from token ids to token
ids: rows of a table, pre-norm gated blocks with a norm and a learned scale
of each channel behind every block, a vocabulary product, log probabilities for
training and sampled tokens for generation.  (Tokens do not see one another:
what follows a token depends on that token alone.)

    x = scale table[ids];  n = norm(x)
    for each block:  f = (act(n Wg) * (n Wu)) Wdown
                     x, n = x + gate * norm(f), norm of that
    z = n Whead;  logprob, entropy = score(z, targets)  or  ids = sample(z)

Every product, norm, lookup, reduction and choice runs in the library's
kernels; torch holds the tensors and adds the two gradients that meet at the
first norm.

    python -m gemm_matmulplan_broadcast_gb300.model

trains one on a made-up language and lets it write.
"""

from __future__ import annotations

import math

from .binding import GemmPlan, Plan
from .layers import ROW_DTYPES, EmbeddingPlan, GatedPlan, LayerNormPlan, ResidualNormPlan, SamplePlan, TokenLogProbsPlan

#: of a block, before the number of the block; gamma and beta also of the norm in front of the first one
BLOCK_PARAMETERS = ("wg", "wu", "wdown", "gate", "after_gamma", "after_beta", "gamma", "beta")


def parameter_names(layers: int):
    names = ["table", "gamma0", "beta0"]
    for i in range(layers):
        names += [k + str(i + 1 if k in ("gamma", "beta") else i) for k in BLOCK_PARAMETERS]
    return names + ["whead"]


class TokenModel:
    """Plans and activations for ``rows`` ids.  ``forward`` takes int64 ids and
    targets [rows] (negative: ignored) and a dict of parameters; ``backward``
    gives a dict of their gradients; ``next_tokens`` draws a token for each id
    from one uniform number each.  All use the same activations: after
    ``logits`` or ``next_tokens``, ``backward`` raises until the next
    ``forward``."""

    def __init__(self, rows: int, layers: int, d_model: int, d_hidden: int, vocab: int, dtype: str = "bfloat16",
                 act: str = "silu", device="cuda"):
        import torch
        if dtype not in ROW_DTYPES:
            raise ValueError("unsupported dtype %r" % (dtype,))
        t, f32 = getattr(torch, dtype), torch.float32
        self.rows, self.layers, self.dtype = rows, layers, dtype
        self.shape = (rows, d_model, d_hidden, vocab)
        new = lambda *s, of=t: torch.empty(s, dtype=of, device=device)  # noqa: E731
        self.embed = EmbeddingPlan(rows, vocab, d_model, dtype, scale=math.sqrt(d_model))
        self.norm = LayerNormPlan(rows, d_model, dtype)
        self.gate = GatedPlan(rows, d_model, d_hidden, dtype, act)
        self.down = Plan((rows, d_hidden), (d_hidden, d_model), dtype)
        self.join = ResidualNormPlan(rows, d_model, dtype, after=True)
        self.head = Plan((rows, d_model), (d_model, vocab), dtype)
        self.score = TokenLogProbsPlan(rows, vocab, dtype)
        self.sample = SamplePlan(rows, vocab, dtype)
        self.x, self.n = ([new(rows, d_model) for _ in range(layers + 1)] for _ in range(2))
        self.h, self.g, self.u = ([new(rows, d_hidden) for _ in range(layers)] for _ in range(3))
        self.f = [new(rows, d_model) for _ in range(layers)]
        self.stats = [new(4, rows, of=f32) for _ in range(layers)]
        self.mean, self.rstd, self.logprob, self.entropy, self.lse, self.drawn = (new(rows, of=f32) for _ in range(6))
        self.z = new(rows, vocab)
        self.targets = self._back = None

    def logits(self, ids, p):
        """[rows, vocab], from the ids alone."""
        self.ids, self.p, self.targets = ids, p, None
        self.embed.forward(p["table"], ids, self.x[0])
        self.norm.forward(self.x[0], p["gamma0"], p["beta0"], self.n[0], mean=self.mean, rstd=self.rstd)
        for i in range(self.layers):
            self.gate.forward(self.n[i], p["wg%d" % i], p["wu%d" % i], self.h[i], G=self.g[i], U=self.u[i])
            self.down.execute(self.h[i], p["wdown%d" % i], self.f[i])
            self.join.forward(self.x[i], self.f[i], self.x[i + 1], Z=self.n[i + 1], gate=p["gate%d" % i],
                              gamma=p["gamma%d" % (i + 1)], beta=p["beta%d" % (i + 1)], stats=self.stats[i],
                              after_gamma=p["after_gamma%d" % i], after_beta=p["after_beta%d" % i])
        self.head.execute(self.n[-1], p["whead"], self.z)
        return self.z

    def forward(self, ids, targets, p):
        """(logprob, entropy) of the targets behind the ids, float32 [rows]."""
        self.score.forward(self.logits(ids, p), targets, self.logprob, entropy=self.entropy, lse=self.lse)
        self.targets = targets
        return self.logprob, self.entropy

    def next_tokens(self, ids, uniforms, p, temperature=None, top_k=None, top_p=None, min_p=None):
        """(tokens, their log probabilities among those the settings leave)."""
        import torch
        tokens = torch.empty_like(ids)
        self.sample.forward(self.logits(ids, p), uniforms, tokens, temperature=temperature, top_k=top_k, top_p=top_p,
                            min_p=min_p, logprob=self.drawn)
        return tokens, self.drawn

    def _backward_plans(self):
        if self._back is None:
            rows, d, f, v = self.shape
            self._back = {
                "n": GemmPlan((rows, v), (d, v), self.dtype, trans_b=True),          # dz Whead'
                "whead": GemmPlan((rows, d), (rows, v), self.dtype, trans_a=True),   # n' dz
                "h": GemmPlan((rows, d), (f, d), self.dtype, trans_b=True),          # df Wdown'
                "wdown": GemmPlan((rows, f), (rows, d), self.dtype, trans_a=True),   # h' df
            }
        return self._back

    def backward(self, dlogprob, dentropy=None):
        """Gradients of every parameter of the last ``forward``."""
        import torch
        if self.targets is None:
            raise RuntimeError("backward follows forward: the activations are another call's")
        p, plans = self.p, self._backward_plans()
        like = torch.empty_like
        grads = {k: like(p[k]) for k in parameter_names(self.layers)}
        dz, dn, dx, df, dh = like(self.z), like(self.n[0]), None, like(self.x[0]), like(self.h[0]) if self.h else None
        self.score.backward(self.z, self.targets, self.lse, self.entropy, dlogprob, dz, dentropy=dentropy)
        plans["n"].execute(dz, p["whead"], dn)
        plans["whead"].execute(self.n[-1], dz, grads["whead"])
        for i in reversed(range(self.layers)):
            passed = like(self.x[0]) if dx is None else dx
            self.join.backward(dx, dn, self.f[i], self.x[i + 1], self.stats[i], gate=p["gate%d" % i],
                               gamma=p["gamma%d" % (i + 1)], after_gamma=p["after_gamma%d" % i],
                               after_beta=p["after_beta%d" % i], dX=passed, dF=df, dgate=grads["gate%d" % i],
                               dgamma=grads["gamma%d" % (i + 1)], dbeta=grads["beta%d" % (i + 1)],
                               dafter_gamma=grads["after_gamma%d" % i], dafter_beta=grads["after_beta%d" % i])
            dx = passed
            plans["h"].execute(df, p["wdown%d" % i], dh)
            plans["wdown"].execute(self.h[i], df, grads["wdown%d" % i])
            self.gate.backward(dh, self.n[i], p["wg%d" % i], p["wu%d" % i], self.g[i], self.u[i], dX=dn,
                               dWg=grads["wg%d" % i], dWu=grads["wu%d" % i])
        first = like(self.x[0])
        self.norm.backward(dn, self.x[0], p["gamma0"], self.mean, self.rstd, first, grads["gamma0"], grads["beta0"])
        if dx is not None:
            first.add_(dx)                                   # the residual's branch
        self.embed.backward(first, self.ids, grads["table"])
        return grads


def parameters(layers: int, d_model: int, d_hidden: int, vocab: int, dtype: str = "bfloat16", seed: int = 0, device="cuda"):
    """Random parameters of a model (drawn on the CPU)."""
    import torch
    gen = torch.Generator().manual_seed(seed)

    def draw(*s, scale, shift=0.0):
        return (torch.randn(s, generator=gen) * scale + shift).to(getattr(torch, dtype)).to(device)

    p = {"table": draw(vocab, d_model, scale=d_model ** -0.5), "whead": draw(d_model, vocab, scale=d_model ** -0.5)}
    for i in range(layers + 1):
        p["gamma%d" % i], p["beta%d" % i] = draw(d_model, scale=0.1, shift=1.0), draw(d_model, scale=0.1)
    for i in range(layers):
        p["wg%d" % i], p["wu%d" % i] = (draw(d_model, d_hidden, scale=d_model ** -0.5) for _ in range(2))
        p["wdown%d" % i] = draw(d_hidden, d_model, scale=d_hidden ** -0.5)
        p["gate%d" % i] = draw(d_model, scale=0.1, shift=0.5)
        p["after_gamma%d" % i], p["after_beta%d" % i] = draw(d_model, scale=0.1, shift=1.0), draw(d_model, scale=0.1)
    return {k: p[k] for k in parameter_names(layers)}


def main(rows=1024, layers=2, d_model=512, d_hidden=1408, vocab=1024, steps=40, rate=0.5, dtype="bfloat16"):
    import torch
    p = parameters(layers, d_model, d_hidden, vocab, dtype)
    gen = torch.Generator(device="cuda").manual_seed(1)
    follows = torch.randperm(vocab, generator=gen, device="cuda")       # the language: what follows each token
    model = TokenModel(rows, layers, d_model, d_hidden, vocab, dtype)
    dlogprob = torch.full((rows,), 1.0 / rows, device="cuda")
    for step in range(steps):
        ids = torch.randint(0, vocab, (rows,), generator=gen, device="cuda")
        logprob, entropy = model.forward(ids, follows[ids], p)
        if step % 8 == 0 or step == steps - 1:
            print("step %2d  mean log probability %.4f  entropy %.4f" % (step, float(logprob.mean()), float(entropy.mean())))
        grads = model.backward(dlogprob)
        for k in p:
            p[k].add_(grads[k], alpha=rate)
    writer = TokenModel(4, layers, d_model, d_hidden, vocab, dtype)
    ids = torch.arange(4, device="cuda")
    temperature, top_p = torch.full((4,), 0.7, device="cuda"), torch.full((4,), 0.9, device="cuda")
    text = [ids]
    for _ in range(10):
        ids, _ = writer.next_tokens(ids, torch.rand(4, generator=gen, device="cuda"), p, temperature=temperature, top_p=top_p)
        text.append(ids)
    for line in torch.stack(text, 1).tolist():
        right = sum(int(follows[a]) == b for a, b in zip(line, line[1:]))
        print("%s  (%d of %d follow)" % (" ".join(map(str, line)), right, len(line) - 1))


if __name__ == "__main__":
    main()
