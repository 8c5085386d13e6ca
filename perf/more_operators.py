"""What is measured of the operators that lead from token ids into a language model's blocks, from block to block,
and from the last product to the next token ids:

  embed     rows of a table by token id, scaled (negative ids mark padding: rows of zeros), and the table's gradient:
            the sum over the places of each token, zeros for tokens that do not occur
  residual  the residual step between two blocks: y = x + scale gate after_norm(f), z = norm(y), with layer or RMS
            norms, the norm of the block's output f optional, the gate absent, one for each channel or one for each
            element; and its gradient down to x, f, the gate and the norms' weights
  sample    one token for each row of logits, from one given uniform number a row: temperature, then the top_k
            largest, then the shortest prefix of those that holds top_p of their weight, without tokens below min_p of
            the largest; and the token's log probability among the ones that were left

`run` computes them in plain torch operations (32-bit arithmetic with one rounding at the end; sampling in 64 bits,
because its choices lie next to borders) or, where `own` is true, through the package's plans.  `exact` gives the same
results from the definitions in 64 bits.
"""

import math

import numpy as np
import torch

own = False

TYPES = {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16}
EPS = 1e-5


def listed():
    return [
        # one decoding step of eight sequences: eight rows of the table
        {"name": "embed_token", "op": "embed", "dir": "forward", "dtype": "float16", "tokens": 8, "vocab": 50257,
         "cols": 4096, "scale": 1.0, "padded": False},
        # the tokens of 8 x 2048, with the scale by sqrt(cols) that some models put here
        {"name": "embed_prompt", "op": "embed", "dir": "forward", "dtype": "bfloat16", "tokens": 16384, "vocab": 50257,
         "cols": 4096, "scale": 64.0, "padded": True},
        # the table's gradient in a training step over 8 x 2048 tokens, frequent tokens among them
        {"name": "embed_grad", "op": "embed", "dir": "backward", "dtype": "bfloat16", "tokens": 16384, "vocab": 50257,
         "cols": 4096, "scale": 1.0, "padded": True},
        # a small 32-bit model: few tokens of a small vocabulary many times each, a width that no vector load divides
        {"name": "embed_grad_odd", "op": "embed", "dir": "backward", "dtype": "float32", "tokens": 9001, "vocab": 1001,
         "cols": 333, "scale": 18.25, "padded": False},
        # one decoding step of four sequences between two blocks
        {"name": "residual_token", "op": "residual", "dir": "forward", "dtype": "float16", "rows": 4, "cols": 4096,
         "norm": "rms", "after": True, "gate": "none", "scale": 1.0, "bias": False},
        # the same over a prompt of 8 x 2048 tokens
        {"name": "residual_prompt", "op": "residual", "dir": "forward", "dtype": "bfloat16", "rows": 16384,
         "cols": 4096, "norm": "rms", "after": True, "gate": "none", "scale": 1.0, "bias": False},
        # its gradient in a training step
        {"name": "residual_grad", "op": "residual", "dir": "backward", "dtype": "bfloat16", "rows": 16384,
         "cols": 4096, "norm": "rms", "after": True, "gate": "none", "scale": 1.0, "bias": False},
        # a small 32-bit model with layer norms and a learned scale of each channel; odd sizes
        {"name": "residual_grad_odd", "op": "residual", "dir": "backward", "dtype": "float32", "rows": 2049,
         "cols": 1001, "norm": "layer", "after": False, "gate": "channel", "scale": 0.5, "bias": True},
        # one decoding step of one sequence, everything switched on
        {"name": "sample_token", "op": "sample", "dir": "forward", "dtype": "float16", "rows": 1, "vocab": 50257,
         "pitch": 50264, "filter": "mixed", "masked": False},
        # one decoding step of a batch in which every request has settings of its own
        {"name": "sample_batch", "op": "sample", "dir": "forward", "dtype": "bfloat16", "rows": 256, "vocab": 50257,
         "pitch": 50264, "filter": "mixed", "masked": True},
        # a 32-bit batch over a large vocabulary with nothing but a temperature
        {"name": "sample_full", "op": "sample", "dir": "forward", "dtype": "float32", "rows": 64, "vocab": 131072,
         "pitch": 131072, "filter": "none", "masked": False},
        # many rollouts of one step, cut by their weight alone
        {"name": "sample_rollouts", "op": "sample", "dir": "forward", "dtype": "bfloat16", "rows": 1024,
         "vocab": 50257, "pitch": 50264, "filter": "top_p", "masked": False},
    ]


def _log_int(rng, low, high):
    n = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    return min(high, max(low, n))


def _width(rng, low, high):
    """A width: half of the time a multiple of 64, else anything."""
    n = _log_int(rng, low, high)
    return max(64, n // 64 * 64) if rng.random() < 0.5 else n


def draw(rng):
    op = rng.choice(("embed", "residual", "sample"))
    way = rng.choice(("forward", "backward"))
    dtype = rng.choice(("bfloat16", "float16", "float32", "bfloat16"))
    size = 4 if dtype == "float32" else 2
    if op == "embed":
        cols = _width(rng, 64, 8192)
        vocab = _log_int(rng, 256, min(200000, (16384 + 50257) * 4096 * 2 // (cols * size) * 3 // 4))
        most = (16384 + 50257) * 4096 * 2 // (cols * size) - (vocab if way == "backward" else 0)
        return {"op": op, "dir": way, "dtype": dtype, "tokens": _log_int(rng, 1, max(1, min(131072, most))),
                "vocab": vocab, "cols": cols, "scale": rng.choice((1.0, math.sqrt(cols))), "padded": rng.random() < 0.3}
    if op == "residual":
        cols = _width(rng, 128, 8192)
        gate = rng.choice(("none", "none", "channel", "element"))
        rows = _log_int(rng, 1, min(32768, 16384 * 4096 * 2 // (cols * size) * (3 if gate == "element" else 4) // 4))
        return {"op": op, "dir": way, "dtype": dtype, "rows": rows, "cols": cols, "norm": rng.choice(("layer", "rms")),
                "after": rng.random() < 0.6, "gate": gate, "scale": rng.choice((1.0, 0.5)), "bias": rng.random() < 0.5}
    vocab = _log_int(rng, 1000, 200000)
    rows = _log_int(rng, 1, min(2048, 1024 * 50257 * 2 // (vocab * size)))
    return {"op": op, "dir": "forward", "dtype": dtype, "rows": rows, "vocab": vocab,
            "pitch": vocab if rng.random() < 0.5 else (vocab + 7) // 8 * 8,
            "filter": rng.choice(("none", "top_k", "top_p", "mixed", "mixed")), "masked": rng.random() < 0.4}


# ---- inputs -----------------------------------------------------------------


def _inputs(case, seed):
    dev, dt = "cuda", TYPES[case["dtype"]]
    gen = torch.Generator(device=dev).manual_seed(int(seed))

    def normal(*shape, scale=1.0, shift=0.0, of=dt):
        return (torch.randn(shape, generator=gen, device=dev) * scale + shift).to(of)

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device=dev)

    back = case["dir"] == "backward"
    if case["op"] == "embed":
        n, vocab, cols = case["tokens"], case["vocab"], case["cols"]
        # ids as a tokenizer's: the r-th most frequent one with a probability of about 1 / r
        rank = torch.exp(uniform(n).double() * math.log(vocab + 1)).long() - 1
        tokens = rank.clamp(0, vocab - 1)
        if case["padded"]:      # one place in ten holds no token
            tokens = torch.where(uniform(n) < 0.1, -1, tokens)
        return {"ids": tokens, "dy": normal(n, cols)} if back else {"ids": tokens, "table": normal(vocab, cols, scale=0.02)}
    if case["op"] == "residual":
        rows, cols = case["rows"], case["cols"]
        s = {"f": normal(rows, cols, scale=0.7, shift=0.1), "gamma": normal(cols, scale=0.2, shift=1.0)}
        if case["bias"]:
            s["beta"] = normal(cols, scale=0.2)
        if case["after"]:
            s["after_gamma"] = normal(cols, scale=0.2, shift=1.0)
            if case["bias"]:
                s["after_beta"] = normal(cols, scale=0.2)
        if case["gate"] != "none":
            s["gate"] = normal(*((cols,) if case["gate"] == "channel" else (rows, cols)), scale=0.3, shift=0.5)
        if not back:
            s["x"] = normal(rows, cols, scale=1.5, shift=0.25)
            return s
        s["y"], s["dy"], s["dz"] = normal(rows, cols, scale=1.7, shift=0.25), normal(rows, cols), normal(rows, cols)
        s["stats"] = torch.stack(_stats(case, s["y"].float()) + (_stats(case, s["f"].float()) if case["after"] else []))
        return s
    rows, vocab, pitch = case["rows"], case["vocab"], case["pitch"]
    # the vocabulary product's output: a broad background, and a few dozen tokens that the context makes likely
    logits = normal(rows, pitch, scale=2.0, of=torch.float32)
    likely = torch.randint(0, vocab, (rows, 48), generator=gen, device=dev)
    logits.scatter_reduce_(1, likely, normal(rows, 48, scale=2.5, shift=9.0, of=torch.float32), "amax")
    logits = logits.to(dt)[:, :vocab]
    if case["masked"]:          # constrained decoding: about half of the vocabulary is forbidden
        logits[:, uniform(vocab) < 0.5] = -math.inf
    s = {"logits": logits, "uniforms": uniform(rows), "temperature": uniform(rows) * 0.7 + 0.5}
    which = case["filter"]
    if which in ("top_k", "mixed"):
        s["top_k"] = torch.randint(1, min(200, vocab), (rows,), generator=gen, device=dev, dtype=torch.int32)
    if which in ("top_p", "mixed"):
        s["top_p"] = uniform(rows) * 0.3 + 0.69
    if which == "mixed" and rows > 1:
        s["min_p"] = uniform(rows) * 0.05
        # every request its own way: some of them without a limit, some greedy
        s["top_k"][uniform(rows) < 0.3] = 0
        s["top_p"][uniform(rows) < 0.2] = 1.0
        s["min_p"][uniform(rows) < 0.5] = 0.0
        s["temperature"][uniform(rows) < 0.1] = 0.0
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    s["plan"] = _plan(case) if own else None        # what a program makes once for its sizes
    dev, dt, back = "cuda", TYPES[case["dtype"]], case["dir"] == "backward"

    def like(*names, to="d"):
        return {to + k: torch.empty_like(s[k]) for k in names if k in s}

    if case["op"] == "embed":
        shape = (case["vocab"] if back else case["tokens"], case["cols"])
        s["out"] = {"dtable" if back else "y": torch.empty(shape, dtype=dt, device=dev)}
    elif case["op"] == "residual":
        if back:
            s["out"] = dict({"dx": torch.empty_like(s["y"])},
                            **like("f", "gate", "gamma", "beta", "after_gamma", "after_beta"))
        else:
            s["out"] = {"y": torch.empty_like(s["x"]), "z": torch.empty_like(s["x"]),
                        "stats": torch.empty(4 if case["after"] else 2, case["rows"], device=dev)}
    else:
        s["out"] = {"tokens": torch.empty(case["rows"], dtype=torch.int64, device=dev),
                    "logprob": torch.empty(case["rows"], device=dev)}
    return s


# ---- the framework's calls ----------------------------------------------------


def _plan(case):
    import gemm_matmulplan_broadcast_gb300 as olc
    if case["op"] == "embed":
        return olc.EmbeddingPlan(case["tokens"], case["vocab"], case["cols"], case["dtype"], scale=case["scale"])
    if case["op"] == "residual":
        return olc.ResidualNormPlan(case["rows"], case["cols"], case["dtype"], eps=EPS, scale=case["scale"],
                                    norm=case["norm"], after=case["after"])
    return olc.SamplePlan(case["rows"], case["vocab"], case["dtype"])


def _run_own(s):
    case, plan, out = s["case"], s["plan"], s["out"]
    if case["op"] == "embed":
        if case["dir"] == "forward":
            plan.forward(s["table"], s["ids"], out["y"])
        else:
            plan.backward(s["dy"], s["ids"], out["dtable"])
    elif case["op"] == "residual":
        weights = {k: s.get(k) for k in ("gate", "gamma", "after_gamma")}
        if case["dir"] == "forward":
            plan.forward(s["x"], s["f"], out["y"], Z=out["z"], beta=s.get("beta"), after_beta=s.get("after_beta"),
                         stats=out["stats"], **weights)
        else:
            plan.backward(s["dy"], s["dz"], s["f"], s["y"], s["stats"], after_beta=s.get("after_beta"),
                          dX=out["dx"], dF=out["df"], dgate=out.get("dgate"), dgamma=out["dgamma"],
                          dbeta=out.get("dbeta"), dafter_gamma=out.get("dafter_gamma"),
                          dafter_beta=out.get("dafter_beta"), **weights)
    else:
        plan.forward(s["logits"], s["uniforms"], out["tokens"], temperature=s["temperature"], top_k=s.get("top_k"),
                     top_p=s.get("top_p"), min_p=s.get("min_p"), logprob=out["logprob"])
    return out


# ---- the plain form -------------------------------------------------------------


def _embed(s, case, dt):
    ids, real = s["ids"], (s["ids"] >= 0)[:, None]
    if case["dir"] == "forward":
        rows = s["table"][ids.clamp(min=0)].float() * case["scale"]
        return {"y": torch.where(real, rows, 0.0).to(dt)}
    total = torch.zeros(case["vocab"], case["cols"], device=ids.device)
    total.index_add_(0, ids.clamp(min=0), torch.where(real, s["dy"].float(), 0.0))
    return {"dtable": (total * case["scale"]).to(dt)}


def _stats(case, v):
    mean = v.mean(-1) if case["norm"] == "layer" else torch.zeros_like(v[:, 0])
    return [mean, torch.rsqrt((v - mean[:, None]).square().mean(-1) + EPS)]


def _norm_grad(case, d, hat, rstd):
    """From the gradient of the normalised rows to that of the rows."""
    d_mean = d.mean(-1)[:, None] if case["norm"] == "layer" else 0.0
    return rstd[:, None] * (d - d_mean - hat * (d * hat).mean(-1)[:, None])


def _residual(s, case, dt):
    w = {k: s[k].float() for k in ("gate", "gamma", "beta", "after_gamma", "after_beta") if k in s}
    f, scale = s["f"].float(), case["scale"]
    gate = w.get("gate", 1.0)
    if case["dir"] == "forward":
        n, of_f = f, []
        if case["after"]:
            of_f = _stats(case, f)
            n = (f - of_f[0][:, None]) * of_f[1][:, None] * w["after_gamma"] + w.get("after_beta", 0.0)
        y = s["x"].float() + scale * gate * n
        mean, rstd = _stats(case, y)
        z = (y - mean[:, None]) * rstd[:, None] * w["gamma"] + w.get("beta", 0.0)
        return {"y": y.to(dt), "z": z.to(dt), "stats": torch.stack([mean, rstd] + of_f)}
    mean, rstd = s["stats"][:2]
    dz, hat = s["dz"].float(), (s["y"].float() - mean[:, None]) * rstd[:, None]
    dy = s["dy"].float() + _norm_grad(case, dz * w["gamma"], hat, rstd)
    dn = scale * gate * dy
    out = {"dx": dy.to(dt), "dgamma": (dz * hat).sum(0).to(dt)}
    if case["bias"]:
        out["dbeta"] = dz.sum(0).to(dt)
    n, df = f, dn
    if case["after"]:
        mean_f, rstd_f = s["stats"][2:]
        hat = (f - mean_f[:, None]) * rstd_f[:, None]
        n = hat * w["after_gamma"] + w.get("after_beta", 0.0)
        df = _norm_grad(case, dn * w["after_gamma"], hat, rstd_f)
        out["dafter_gamma"] = (dn * hat).sum(0).to(dt)
        if case["bias"]:
            out["dafter_beta"] = dn.sum(0).to(dt)
    out["df"] = df.to(dt)
    if "gate" in w:
        dgate = scale * n * dy
        out["dgate"] = (dgate.sum(0) if case["gate"] == "channel" else dgate).to(dt)
    return {k: out[k] for k in s["out"]}


def _sample(s, case, dt):
    z, vocab = s["logits"].double(), case["vocab"]
    heat = s["temperature"].double()
    greedy = heat == 0
    top_p = s["top_p"].double()[:, None] if "top_p" in s else 1.0
    min_p = s["min_p"].double()[:, None] if "min_p" in s else 0.0
    z, order = torch.sort(z, dim=-1, descending=True, stable=True)     # by value, then by the lower index
    weight = torch.exp((z - z[:, :1]) / torch.where(greedy, 1.0, heat)[:, None])
    place = torch.arange(vocab, device=z.device)
    if "top_k" in s:
        top_k = torch.where(s["top_k"] > 0, s["top_k"], vocab)[:, None]
        weight = torch.where(place < top_k, weight, 0.0)
    before = torch.cumsum(weight, -1) - weight
    total = weight.sum(-1, keepdim=True)
    keep = (before < top_p * total) & (weight >= min_p) & ~greedy[:, None] | (place == 0)
    left = torch.zeros_like(weight).scatter_(1, order, torch.where(keep, weight, 0.0))
    reach = torch.cumsum(left, -1)
    total = reach[:, -1:]
    tokens = (reach > s["uniforms"].double()[:, None] * total).to(torch.uint8).argmax(-1)
    chosen = torch.log(left.gather(1, tokens[:, None]) / total)[:, 0]
    return {"tokens": tokens, "logprob": chosen.float()}


def run(state):
    if own:
        return _run_own(state)
    case = state["case"]
    return {"embed": _embed, "residual": _residual, "sample": _sample}[case["op"]](state, case, TYPES[case["dtype"]])


# ---- what it has to move and compute ------------------------------------------------


def work(case):
    size = 4 if case["dtype"] == "float32" else 2
    back = case["dir"] == "backward"
    if case["op"] == "embed":
        n, vocab, cols = case["tokens"], case["vocab"], case["cols"]
        if back:        # the gradient of every place in, every row of the table out
            return {"bytes": (n + vocab) * cols * size + 8 * n, "flops": n * cols + vocab * cols}
        # the rows that occur, each of them once, and a row for every place
        r = np.arange(1, vocab + 1, dtype=np.float64)
        p = np.log1p(1 / r) / math.log(vocab + 1)
        real = n * (0.9 if case["padded"] else 1.0)
        rows = float(-np.expm1(real * np.log1p(-p)).sum())
        return {"bytes": int((rows + n) * cols * size) + 8 * n, "flops": n * cols}
    if case["op"] == "residual":
        rows, cols = case["rows"], case["cols"]
        n = rows * cols
        gates = {"none": 0, "channel": 0, "element": 2 if back else 1}[case["gate"]]
        norms = 2 if case["after"] else 1
        weights = norms * (2 if case["bias"] else 1) + (case["gate"] == "channel")
        # forward: x and f in, y and z out; backward: dy, dz, y and f in, dx and df out; statistics and weights once
        return {"bytes": ((6 if back else 4) + gates) * n * size + weights * cols * size * (2 if back else 1) + 16 * rows,
                "flops": n * ((14 if back else 8) * norms + 4)}
    n = case["rows"] * case["vocab"]
    return {"bytes": n * size + 32 * case["rows"], "flops": 6 * n}


# ---- the definitions in 64 bits --------------------------------------------------------


def exact(case, seed):
    s = {k: v.double() if v.is_floating_point() else v for k, v in _inputs(case, seed).items()}
    back = case["dir"] == "backward"
    if case["op"] == "embed":
        known = s["ids"] >= 0
        if not back:
            y = torch.zeros(case["tokens"], case["cols"], dtype=torch.float64, device=known.device)
            y[known] = torch.index_select(s["table"], 0, s["ids"][known]) * case["scale"]
            return {"y": y}
        # the places in the order of their tokens, and the sums of what lies between two changes
        ids, order = torch.sort(s["ids"][known], stable=True)
        runs, lengths = torch.unique_consecutive(ids, return_counts=True)
        dtable = torch.zeros(case["vocab"], case["cols"], dtype=torch.float64, device=known.device)
        if len(runs):
            dtable[runs] = torch.segment_reduce(s["dy"][known][order] * case["scale"], "sum", lengths=lengths)
        return {"dtable": dtable}
    if case["op"] == "residual":
        cols = case["cols"]
        leaves = {k: s[k].requires_grad_(back) for k in ("f", "gate", "gamma", "beta", "after_gamma", "after_beta")
                  if k in s}

        def norm(v, weight, bias):
            if case["norm"] == "layer":
                return torch.nn.functional.layer_norm(v, (cols,), weight, bias, EPS)
            return v / torch.sqrt((v * v).sum(-1, keepdim=True) / cols + EPS) * weight + (0 if bias is None else bias)

        def added():
            n = norm(s["f"], s["after_gamma"], s.get("after_beta")) if case["after"] else s["f"]
            return case["scale"] * n * s["gate"] if "gate" in s else case["scale"] * n

        def statistics(v):
            mean = v.sum(-1) / cols if case["norm"] == "layer" else torch.zeros_like(v[:, 0])
            return [mean, 1 / torch.sqrt(((v - mean[:, None]) ** 2).sum(-1) / cols + EPS)]

        if not back:
            y = s["x"] + added()
            of_f = statistics(s["f"]) if case["after"] else []
            return {"y": y, "z": norm(y, s["gamma"], s.get("beta")), "stats": torch.stack(statistics(y) + of_f)}
        y = s["y"].requires_grad_()
        before = [k for k in ("gamma", "beta") if k in s]
        rest = [k for k in leaves if k not in before]
        grads = torch.autograd.grad(norm(y, s["gamma"], s.get("beta")), [y] + [s[k] for k in before], s["dz"])
        dx = s["dy"] + grads[0]
        out = dict({"dx": dx}, **{"d" + k: g for k, g in zip(before, grads[1:])})
        out.update(("d" + k, g) for k, g in zip(rest, torch.autograd.grad(added(), [s[k] for k in rest], dx)))
        return {k: out[k] for k in ["dx"] + ["d" + k for k in leaves]}
    rows, vocab = case["rows"], case["vocab"]
    logits, tokens, logprob = s["logits"], [], []
    for r in range(rows):
        z, heat = logits[r], float(s["temperature"][r])
        if heat == 0:
            tokens.append(torch.nonzero(z == z.max())[0])
            logprob.append(torch.zeros(1, dtype=torch.float64, device=z.device))
            continue
        p = torch.softmax(z / heat, -1)
        ids = torch.argsort(z, descending=True, stable=True)       # equal logits by the lower index
        if "top_k" in s and 0 < int(s["top_k"][r]) < vocab:
            ids = ids[:int(s["top_k"][r])]
        if "top_p" in s and float(s["top_p"][r]) < 1:
            share = torch.cumsum(p[ids] / p[ids].sum(), 0)
            ids = ids[:int((share < s["top_p"][r]).sum()) + 1]
        if "min_p" in s:
            ids = ids[p[ids] >= s["min_p"][r] * p.max()]
        ids = torch.sort(ids).values
        share = torch.cumsum(p[ids], 0)
        at = torch.searchsorted(share, s["uniforms"][r] * share[-1], right=True).clamp(max=len(ids) - 1)
        tokens.append(ids[at].view(1))
        logprob.append(torch.log(p[ids[at]] / share[-1]).view(1))
    return {"tokens": torch.cat(tokens), "logprob": torch.cat(logprob)}
