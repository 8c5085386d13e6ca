"""The token model, the plans together from ids to ids: log probabilities,
entropy and every gradient against autograd in 64 bits, and what it draws against
its own logits.

Tolerances as for the block of test_block_gpu.py: FLOAT, each of the chain's stages
(seven a block, four around them) is off by a few times sqrt(K) 2^-24 of its scale
(K <= 96 terms) and the products of the stages' slopes stay below 100 a block, two
blocks at most: 1e-3 of a tensor's largest value covers the chain.  FLOAT16 / BFLOAT16: every
stage rounds to 2^-11 / 2^-8 as well: 5e-2 / 4e-1 of a tensor's root mean
square, in the 2-norm over the tensor."""

import pytest
import torch

from gemm_matmulplan_broadcast_gb300.model import TokenModel, parameter_names, parameters
from test_sample_gpu import reference as sampled

pytestmark = pytest.mark.gpu


def reference(ids, targets, p, layers, dlp, dh, act):
    q = {k: v.double().cpu().requires_grad_() for k, v in p.items()}
    d = q["table"].shape[1]
    norm = lambda t, g, b: torch.nn.functional.layer_norm(t, t.shape[-1:], q[g], q[b])  # noqa: E731
    fn = {"silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu}[act]
    known = (ids.cpu() >= 0).double()[:, None]
    x = q["table"][ids.cpu().clamp(min=0)] * d ** 0.5 * known
    n = norm(x, "gamma0", "beta0")
    for i in range(layers):
        f = (fn(n @ q["wg%d" % i]) * (n @ q["wu%d" % i])) @ q["wdown%d" % i]
        x = x + q["gate%d" % i] * norm(f, "after_gamma%d" % i, "after_beta%d" % i)
        n = norm(x, "gamma%d" % (i + 1), "beta%d" % (i + 1))
    logp = torch.log_softmax(n @ q["whead"], -1)
    lp = logp[torch.arange(len(ids)), targets.cpu()]
    entropy = -(logp.exp() * logp).sum(-1)
    loss = (lp * dlp.double().cpu()).sum() + (entropy * dh.double().cpu()).sum()
    names = parameter_names(layers)
    return lp.detach(), entropy.detach(), dict(zip(names, torch.autograd.grad(loss, [q[k] for k in names])))


@pytest.mark.parametrize("dtype,act", [("float32", "silu"), ("float32", "gelu"), ("float16", "silu"), ("bfloat16", "gelu")])
@pytest.mark.parametrize("rows,layers,d,f,vocab", [(40, 2, 64, 96, 101), (17, 1, 56, 80, 96), (9, 0, 64, 8, 50)])
def test_gradients(rows, layers, d, f, vocab, dtype, act):
    p = parameters(layers, d, f, vocab, dtype, seed=3)
    gen = torch.Generator().manual_seed(4)
    ids, targets = (torch.randint(0, vocab, (rows,), generator=gen).cuda() for _ in range(2))
    ids[rows // 2] = ids[0]                                  # the same token twice
    dlp, dh = torch.randn(rows, generator=gen).cuda(), torch.randn(rows, generator=gen).cuda() * 0.1
    model = TokenModel(rows, layers, d, f, vocab, dtype, act)
    lp, entropy = model.forward(ids, targets, p)
    grads = model.backward(dlp, dentropy=dh)
    want_lp, want_entropy, want = reference(ids, targets, p, layers, dlp, dh, act)
    assert list(grads) == parameter_names(layers)
    for name, got, ref in [("logprob", lp, want_lp), ("entropy", entropy, want_entropy)] + [(k, grads[k], want[k]) for k in want]:
        got = got.double().cpu()
        if dtype == "float32":
            assert float((got - ref).abs().max()) <= 1e-3 * float(ref.abs().max()), name
        else:
            assert float((got - ref).norm()) <= (5e-2 if dtype == "float16" else 4e-1) * float(ref.norm()), name


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_tokens_are_drawn_from_the_logits(dtype):
    rows, vocab = 12, 4096
    p = parameters(1, 64, 128, vocab, dtype, seed=1)
    model = TokenModel(rows, 1, 64, 128, vocab, dtype)
    gen = torch.Generator().manual_seed(2)
    ids, u = torch.randint(0, vocab, (rows,), generator=gen), torch.rand(rows, generator=gen)
    heat, top_k = torch.rand(rows, generator=gen) + 0.5, torch.randint(1, 200, (rows,), generator=gen, dtype=torch.int32)
    heat[3] = 0
    tokens, logprob = model.next_tokens(ids.cuda(), u.cuda(), p, temperature=heat.cuda(), top_k=top_k.cuda())
    for r in range(rows):
        token, lp, border = sampled(model.z[r].double().cpu().numpy(), float(u[r]), float(heat[r]), int(top_k[r]))
        assert border > 2.0 ** -32 and int(tokens[r]) == token
        assert abs(float(logprob[r]) - lp) <= 4 * 2.0 ** -24 * (1 + abs(lp))


def test_a_captured_step_of_generation():
    """Ids fed back through a graph: the same tokens as call by call."""
    rows, vocab, steps = 5, 1000, 6
    p = parameters(2, 64, 128, vocab, "bfloat16", seed=7)
    model = TokenModel(rows, 2, 64, 128, vocab, "bfloat16")
    us = torch.rand(steps, rows, generator=torch.Generator().manual_seed(3)).cuda()
    top_p = torch.full((rows,), 0.9, device="cuda")
    ids, want = torch.arange(rows, device="cuda"), []
    for k in range(steps):
        ids = model.next_tokens(ids, us[k], p, top_p=top_p)[0]
        want.append(ids)
    torch.cuda.synchronize()
    ids, u = torch.arange(rows, device="cuda"), us[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ids.copy_(model.next_tokens(ids, u, p, top_p=top_p)[0])
    for k in range(steps):
        u.copy_(us[k])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(ids, want[k]), k


def test_a_captured_training_step():
    rows, vocab = 64, 300
    p = parameters(2, 64, 96, vocab, "bfloat16", seed=9)
    model = TokenModel(rows, 2, 64, 96, vocab, "bfloat16")
    gen = torch.Generator().manual_seed(5)
    ids, targets = (torch.randint(0, vocab, (rows,), generator=gen).cuda() for _ in range(2))
    dlp = torch.full((rows,), 1.0 / rows, device="cuda")
    model.forward(ids, targets, p)
    want = model.backward(dlp)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        model.forward(ids, targets, p)
        got = model.backward(dlp)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(got[k], want[k]) for k in want)
