"""What is measured of the operators that stand around a language model's matrix products:

  norm   layer norm over the last axis, forward (with its row statistics) and backward (with the gradients of
         the weight and the bias, reduced over the rows)
  gate   the gated feed-forward product h = act(x Wg) * (x Wu), forward (with g = x Wg and u = x Wu kept for
         training, or not) and backward (from dh, g and u to dx, dWg and dWu)
  score  log probabilities of given tokens from the vocabulary product's logits, with the entropy and the most
         likely alternatives, forward and backward

`run` computes them in plain torch operations (32-bit arithmetic, one rounding at the end) or, where `own` is
true, through the package's plans.  `exact` gives the same results from the definitions in 64 bits.
"""

import math

import torch

own = False

TYPES = {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16}
EPS = 1e-5


def listed():
    return [
        # one decoding step of four sequences: a few rows, where the call itself is the cost
        {"name": "norm_token", "op": "norm", "dir": "forward", "dtype": "float16", "rows": 4, "cols": 4096},
        # the norm in front of a projection of 8 x 2048 tokens
        {"name": "norm_prompt", "op": "norm", "dir": "forward", "dtype": "bfloat16", "rows": 16384, "cols": 4096},
        # its gradient in a training step
        {"name": "norm_grad", "op": "norm", "dir": "backward", "dtype": "bfloat16", "rows": 16384, "cols": 4096},
        # a small 32-bit model with a width that no vector load divides
        {"name": "norm_grad_odd", "op": "norm", "dir": "backward", "dtype": "float32", "rows": 2049, "cols": 1001},
        # one token through the 4096 -> 14336 projections: the weights' bytes
        {"name": "gate_token", "op": "gate", "dir": "forward", "dtype": "bfloat16", "rows": 1, "d_in": 4096,
         "d_hidden": 14336, "act": "silu", "trans_w": False, "keep": False},
        # a short batch with odd widths, weights stored [out, in]
        {"name": "gate_odd", "op": "gate", "dir": "forward", "dtype": "float16", "rows": 333, "d_in": 1000,
         "d_hidden": 2730, "act": "gelu", "trans_w": True, "keep": False},
        # a 32-bit model's block
        {"name": "gate_float", "op": "gate", "dir": "forward", "dtype": "float32", "rows": 1024, "d_in": 1024,
         "d_hidden": 2816, "act": "silu", "trans_w": False, "keep": True},
        # the forward pass of a training step over 8 x 2048 tokens
        {"name": "gate_train", "op": "gate", "dir": "forward", "dtype": "bfloat16", "rows": 16384, "d_in": 4096,
         "d_hidden": 14336, "act": "silu", "trans_w": False, "keep": True},
        # the backward pass of half as many tokens: the same number of operations
        {"name": "gate_grad", "op": "gate", "dir": "backward", "dtype": "bfloat16", "rows": 8192, "d_in": 4096,
         "d_hidden": 14336, "act": "silu", "trans_w": False, "keep": True},
        # one decoding step that reports its twenty best alternatives
        {"name": "score_token", "op": "score", "dir": "forward", "dtype": "float16", "rows": 1, "vocab": 50257,
         "pitch": 50264, "top": 20, "masked": True},
        # scoring 4096 tokens of a prompt
        {"name": "score_prompt", "op": "score", "dir": "forward", "dtype": "bfloat16", "rows": 4096,
         "vocab": 50257, "pitch": 50264, "top": 5, "masked": False},
        # the gradient of a policy's log probabilities and entropy
        {"name": "score_grad", "op": "score", "dir": "backward", "dtype": "bfloat16", "rows": 4096,
         "vocab": 50257, "pitch": 50264, "top": 0, "masked": False},
    ]


def _log_int(rng, low, high):
    n = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    return min(high, max(low, n))


def _width(rng, low, high):
    """A width: half of the time a multiple of 64, else anything."""
    n = _log_int(rng, low, high)
    return max(64, n // 64 * 64) + (64 if n // 64 * 64 == 3072 else 0) if rng.random() < 0.5 else n + (n == 3072)


def draw(rng):
    op = rng.choice(("norm", "gate", "score"))
    way = rng.choice(("forward", "forward", "backward"))
    dtype = rng.choice(("bfloat16", "float16", "float32", "bfloat16"))
    if op == "norm":
        cols = _width(rng, 128, 16384)
        rows = _log_int(rng, 1, min(32768, 16384 * 4096 // cols))
        return {"op": op, "dir": way, "dtype": dtype, "rows": rows, "cols": cols}
    if op == "gate":
        wide = dtype != "float32"
        d_in = _width(rng, 256, 4096 if wide else 2048)
        d_hidden = _width(rng, 512, 14336 if wide else 5632)
        most = (8192 if way == "backward" else 16384) if wide else 2048
        return {"op": op, "dir": way, "dtype": dtype, "rows": _log_int(rng, 1, most), "d_in": d_in,
                "d_hidden": d_hidden, "act": rng.choice(("silu", "gelu", "relu", "sigmoid")),
                "trans_w": rng.random() < 0.5, "keep": way == "backward" or rng.random() < 0.5}
    vocab = _log_int(rng, 1000, 200000)
    rows = _log_int(rng, 1, min(16384, 4096 * 50257 * (1 if dtype != "float32" else 0.5) // vocab))
    return {"op": op, "dir": way, "dtype": dtype, "rows": int(rows), "vocab": vocab,
            "pitch": vocab if rng.random() < 0.5 else (vocab + 7) // 8 * 8,
            "top": rng.choice((0, 1, 5, 20)) if way == "forward" else 0, "masked": rng.random() < 0.5}


# ---- inputs -----------------------------------------------------------------


def _inputs(case, seed):
    dev, dt = "cuda", TYPES[case["dtype"]]
    gen = torch.Generator(device=dev).manual_seed(int(seed))

    def normal(*shape, scale=1.0, shift=0.0):
        return (torch.randn(shape, generator=gen, device=dev) * scale + shift).to(dt)

    if case["op"] == "norm":
        rows, cols = case["rows"], case["cols"]
        s = {"x": normal(rows, cols, scale=1.5, shift=0.25), "gamma": normal(cols, scale=0.2, shift=1.0),
             "beta": normal(cols, scale=0.2)}
        if case["dir"] == "backward":
            s["dy"] = normal(rows, cols)
            x = s["x"].float()
            mean = x.mean(-1)
            s["mean"], s["rstd"] = mean, torch.rsqrt((x - mean[:, None]).square().mean(-1) + EPS)
        return s
    if case["op"] == "gate":
        rows, d, f = case["rows"], case["d_in"], case["d_hidden"]
        shape = (f, d) if case["trans_w"] else (d, f)
        s = {"x": normal(rows, d), "wg": normal(*shape, scale=d ** -0.5), "wu": normal(*shape, scale=d ** -0.5)}
        if case["dir"] == "backward":
            s["g"], s["u"], s["dh"] = normal(rows, f), normal(rows, f), normal(rows, f, scale=0.1)
        return s
    rows, vocab, pitch = case["rows"], case["vocab"], case["pitch"]
    # the vocabulary product's output: rows padded to the pitch, of which the first `vocab` columns count
    logits = normal(rows, pitch, scale=2.5)[:, :vocab]
    if case["masked"]:      # constrained decoding: about half of the vocabulary is forbidden
        logits[:, torch.rand(vocab, generator=gen, device=dev) < 0.5] = -math.inf
    tokens = logits.argmax(-1)                      # a token that no mask forbids; some of them the best one
    if not case["masked"]:
        tokens = torch.where(torch.rand(rows, generator=gen, device=dev) < 0.3, tokens,
                             torch.randint(0, vocab, (rows,), generator=gen, device=dev))
    s = {"logits": logits, "tokens": tokens}
    if case["dir"] == "backward":
        z = logits.float()
        s["lse"] = torch.logsumexp(z, -1)
        p = torch.exp(z - s["lse"][:, None])
        s["entropy"] = s["lse"] - torch.where(p > 0, p * z, 0.0).sum(-1)
        s["dlogprob"] = torch.randn(rows, generator=gen, device=dev)
        s["dentropy"] = torch.randn(rows, generator=gen, device=dev) * 0.01
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    s["plan"] = _plan(case) if own else None        # what a program makes once for its sizes
    dev, back = "cuda", case["dir"] == "backward"
    if case["op"] == "norm":
        out = {"dx": torch.empty_like(s["x"]), "dgamma": torch.empty_like(s["gamma"]),
               "dbeta": torch.empty_like(s["beta"])} if back else {
            "y": torch.empty_like(s["x"]), "mean": torch.empty(case["rows"], device=dev),
            "rstd": torch.empty(case["rows"], device=dev)}
    elif case["op"] == "gate":
        h = (case["rows"], case["d_hidden"])
        if back:
            out = {"dx": torch.empty_like(s["x"]), "dwg": torch.empty_like(s["wg"]), "dwu": torch.empty_like(s["wu"])}
        else:
            out = {k: torch.empty(h, dtype=s["x"].dtype, device=dev) for k in (("h", "g", "u") if case["keep"] else ("h",))}
    elif back:
        padded = torch.empty(case["rows"], case["pitch"], dtype=s["logits"].dtype, device=dev)
        out = {"dlogits": padded[:, :case["vocab"]]}    # laid out as the logits are
    else:
        out = {"logprob": torch.empty(case["rows"], device=dev), "entropy": torch.empty(case["rows"], device=dev),
               "lse": torch.empty(case["rows"], device=dev)}
        if case["top"]:
            out["top_logprob"] = torch.empty(case["rows"], case["top"], device=dev)
            out["top_index"] = torch.empty(case["rows"], case["top"], dtype=torch.int64, device=dev)
    s["out"] = out
    return s


# ---- the framework's calls ----------------------------------------------------


def _plan(case):
    import gemm_matmulplan_broadcast_gb300 as olc
    if case["op"] == "norm":
        return olc.LayerNormPlan(case["rows"], case["cols"], case["dtype"], eps=EPS)
    if case["op"] == "gate":
        return olc.GatedPlan(case["rows"], case["d_in"], case["d_hidden"], case["dtype"], act=case["act"],
                             trans_w=case["trans_w"])
    return olc.TokenLogProbsPlan(case["rows"], case["vocab"], case["dtype"], top=case["top"])


def _run_own(s):
    case, plan, out = s["case"], s["plan"], s["out"]
    if case["op"] == "norm":
        if case["dir"] == "forward":
            plan.forward(s["x"], s["gamma"], s["beta"], out["y"], mean=out["mean"], rstd=out["rstd"])
        else:
            plan.backward(s["dy"], s["x"], s["gamma"], s["mean"], s["rstd"], out["dx"], dgamma=out["dgamma"],
                          dbeta=out["dbeta"])
    elif case["op"] == "gate":
        if case["dir"] == "forward":
            plan.forward(s["x"], s["wg"], s["wu"], out["h"], G=out.get("g"), U=out.get("u"))
        else:
            plan.backward(s["dh"], s["x"], s["wg"], s["wu"], s["g"], s["u"], dX=out["dx"], dWg=out["dwg"],
                          dWu=out["dwu"])
    elif case["dir"] == "forward":
        plan.forward(s["logits"], s["tokens"], out["logprob"], entropy=out["entropy"], lse=out["lse"],
                     top_logprob=out.get("top_logprob"), top_index=out.get("top_index"))
    else:
        plan.backward(s["logits"], s["tokens"], s["lse"], s["entropy"], s["dlogprob"], out["dlogits"],
                      dentropy=s["dentropy"])
    return out


# ---- the plain form -------------------------------------------------------------


def _act(name, g):
    if name == "silu":
        return g * torch.sigmoid(g)
    if name == "gelu":
        return g * 0.5 * (1 + torch.erf(g * math.sqrt(0.5)))
    return torch.relu(g) if name == "relu" else torch.sigmoid(g)


def _act_slope(name, g):
    s = torch.sigmoid(g)
    if name == "silu":
        return s * (1 + g * (1 - s))
    if name == "gelu":
        return 0.5 * (1 + torch.erf(g * math.sqrt(0.5))) + g * torch.exp(-0.5 * g * g) * (1 / math.sqrt(2 * math.pi))
    return (g > 0).to(g.dtype) if name == "relu" else s * (1 - s)


def _norm(s, case, dt):
    x, gamma = s["x"].float(), s["gamma"].float()
    if case["dir"] == "forward":
        mean = x.mean(-1)
        d = x - mean[:, None]
        rstd = torch.rsqrt((d * d).mean(-1) + EPS)
        return {"y": (d * rstd[:, None] * gamma + s["beta"].float()).to(dt), "mean": mean, "rstd": rstd}
    dy = s["dy"].float()
    xh = (x - s["mean"][:, None]) * s["rstd"][:, None]
    dxh = dy * gamma
    dx = s["rstd"][:, None] * (dxh - dxh.mean(-1)[:, None] - xh * (dxh * xh).mean(-1)[:, None])
    return {"dx": dx.to(dt), "dgamma": (dy * xh).sum(0).to(dt), "dbeta": dy.sum(0).to(dt)}


def _gate(s, case, dt):
    x, wg, wu = s["x"].float(), s["wg"].float(), s["wu"].float()
    if case["trans_w"]:
        wg, wu = wg.t(), wu.t()
    if case["dir"] == "forward":
        g, u = x @ wg, x @ wu
        out = {"h": (_act(case["act"], g) * u).to(dt)}
        return dict(out, g=g.to(dt), u=u.to(dt)) if case["keep"] else out
    g, u, dh = s["g"].float(), s["u"].float(), s["dh"].float()
    dg, du = dh * u * _act_slope(case["act"], g), dh * _act(case["act"], g)
    dx = dg @ wg.t() + du @ wu.t()
    dwg, dwu = (dg.t() @ x, du.t() @ x) if case["trans_w"] else (x.t() @ dg, x.t() @ du)
    return {"dx": dx.to(dt), "dwg": dwg.to(dt), "dwu": dwu.to(dt)}


def _score(s, case, dt):
    z, tokens = s["logits"].float(), s["tokens"]
    if case["dir"] == "backward":
        p = torch.exp(z - s["lse"][:, None])
        slope = torch.where(p > 0, p * (z - (s["lse"] - s["entropy"])[:, None]), 0.0)
        d = -s["dlogprob"][:, None] * p - s["dentropy"][:, None] * slope
        d.scatter_add_(1, tokens[:, None], s["dlogprob"][:, None])
        return {"dlogits": d.to(dt)}
    m = z.amax(-1)
    e = torch.exp(z - m[:, None])
    total = e.sum(-1)
    lse = m + torch.log(total)
    mean = torch.where(e > 0, e * (z - m[:, None]), 0.0).sum(-1) / total
    out = {"logprob": z.gather(1, tokens[:, None])[:, 0] - lse, "entropy": torch.log(total) - mean, "lse": lse}
    if case["top"]:
        # one 64-bit key for each value and place: the value's order first, then the lower index
        i = (z + 0.0).view(torch.int32)
        key = torch.where(i < 0, i ^ 0x7FFFFFFF, i).to(torch.int64) << 32
        key += case["vocab"] - 1 - torch.arange(case["vocab"], device=z.device)
        top = case["vocab"] - 1 - (key.topk(case["top"], -1).values & 0xFFFFFFFF)
        out.update(top_logprob=z.gather(1, top) - lse[:, None], top_index=top)
    return out


def run(state):
    if own:
        return _run_own(state)
    case = state["case"]
    return {"norm": _norm, "gate": _gate, "score": _score}[case["op"]](state, case, TYPES[case["dtype"]])


# ---- what it has to move and compute ------------------------------------------------


def work(case):
    size = 4 if case["dtype"] == "float32" else 2
    back = case["dir"] == "backward"
    rows = case["rows"]
    if case["op"] == "norm":
        n = rows * case["cols"]
        # forward: x in, y out; backward: x and dy in, dx out; the weights and the row statistics once
        return {"bytes": (3 if back else 2) * n * size + (3 if back else 2) * case["cols"] * size + 8 * rows,
                "flops": (14 if back else 8) * n}
    if case["op"] == "gate":
        d, f = case["d_in"], case["d_hidden"]
        if back:        # dh, g, u, x and the weights in; dx and the weights' gradients out
            return {"bytes": size * (3 * rows * f + 2 * rows * d + 4 * d * f), "flops": 8 * rows * d * f}
        return {"bytes": size * (rows * d + 2 * d * f + (3 if case["keep"] else 1) * rows * f),
                "flops": 4 * rows * d * f}
    n = rows * case["vocab"]
    return {"bytes": (2 if back else 1) * n * size + rows * (32 + 12 * case["top"]), "flops": (8 if back else 6) * n}


# ---- the definitions in 64 bits --------------------------------------------------------


def exact(case, seed):
    s = {k: v.double() if v.is_floating_point() else v for k, v in _inputs(case, seed).items()}
    back = case["dir"] == "backward"
    if case["op"] == "norm":
        x, gamma, beta = (s[k].requires_grad_(back) for k in ("x", "gamma", "beta"))
        var, mean = torch.var_mean(x, -1, correction=0, keepdim=True)
        y = (x - mean) / torch.sqrt(var + EPS) * gamma + beta
        if not back:
            return {"y": y, "mean": mean[:, 0], "rstd": 1 / torch.sqrt(var[:, 0] + EPS)}
        dx, dgamma, dbeta = torch.autograd.grad(y, (x, gamma, beta), s["dy"])
        return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}
    if case["op"] == "gate":
        act = {"silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu, "relu": torch.relu,
               "sigmoid": torch.sigmoid}[case["act"]]
        product = "mk,nk->mn" if case["trans_w"] else "mk,kn->mn"
        if not back:
            g, u = (torch.einsum(product, s["x"], s[w]) for w in ("wg", "wu"))
            return {"h": act(g) * u, "g": g, "u": u} if case["keep"] else {"h": act(g) * u}
        g, u = s["g"].requires_grad_(), s["u"].requires_grad_()
        dg, du = torch.autograd.grad(act(g) * u, (g, u), s["dh"])
        x, wg, wu = (s[k].requires_grad_() for k in ("x", "wg", "wu"))
        products = (torch.einsum(product, x, wg), torch.einsum(product, x, wu))
        dx, dwg, dwu = torch.autograd.grad(products, (x, wg, wu), (dg, du))
        return {"dx": dx, "dwg": dwg, "dwu": dwu}
    z, tokens = s["logits"], s["tokens"]
    logp = torch.log_softmax(z, -1)
    p = torch.exp(logp)
    plogp = torch.where(p > 0, p * logp, torch.zeros_like(p))
    entropy = -plogp.sum(-1)
    if back:
        one = torch.nn.functional.one_hot(tokens, case["vocab"])
        return {"dlogits": s["dlogprob"][:, None] * (one - p) - s["dentropy"][:, None] * (plogp + p * entropy[:, None])}
    picked = torch.arange(len(tokens), device=z.device)
    out = {"logprob": logp[picked, tokens], "entropy": entropy, "lse": torch.logsumexp(z, -1)}
    if case["top"]:
        order = torch.sort(z, dim=-1, descending=True, stable=True).indices[:, :case["top"]]
        out.update(top_logprob=torch.gather(logp, 1, order), top_index=order)
    return out
