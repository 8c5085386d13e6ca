"""The layer plans together: the example block's log probabilities, entropy
and every gradient against autograd in 64 bits, a few steps of training, and
the form for one token.

Tolerances, FLOAT: each of the chain's seven stages is off by a few times
sqrt(K) 2^-24 of its scale (K <= 96 terms); with unit-variance activations the
products of the stages' slopes stay below 100, so 2e-4 of a tensor's largest
value covers the chain.  FLOAT16 / BFLOAT16: every stage rounds to 2^-11 / 2^-8
as well; eight stages with the same slopes: 3e-2 / 2.5e-1 of a tensor's
root mean square, in the 2-norm over the tensor."""

import pytest
import torch

from gemm_matmulplan_broadcast_gb300.block import PARAMETERS, ScoredBlock, parameters

pytestmark = pytest.mark.gpu


def reference(x, tokens, p, dlp, dh, act):
    x = x.double().cpu().requires_grad_()
    q = {k: v.double().cpu().requires_grad_() for k, v in p.items()}
    norm = lambda t, g, b: torch.nn.functional.layer_norm(t, t.shape[-1:], g, b)  # noqa: E731
    n1 = norm(x, q["gamma1"], q["beta1"])
    fn = {"silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu}[act]
    y = x + (fn(n1 @ q["wg"]) * (n1 @ q["wu"])) @ q["wdown"]
    logp = torch.log_softmax(norm(y, q["gamma2"], q["beta2"]) @ q["whead"], -1)
    lp = logp[torch.arange(len(tokens)), tokens.cpu()]
    entropy = -(logp.exp() * logp).sum(-1)
    loss = (lp * dlp.double().cpu()).sum() + (entropy * dh.double().cpu()).sum()
    grads = torch.autograd.grad(loss, [x] + [q[k] for k in PARAMETERS])
    return lp.detach(), entropy.detach(), dict(zip(("x",) + PARAMETERS, grads))


@pytest.mark.parametrize("dtype,act", [("float32", "silu"), ("float32", "gelu"), ("float16", "silu"), ("bfloat16", "gelu")])
@pytest.mark.parametrize("rows,d,f,vocab", [(40, 64, 96, 101), (17, 56, 80, 96)])
def test_block_and_gradients(rows, d, f, vocab, dtype, act):
    p = parameters(d, f, vocab, dtype, seed=3)
    gen = torch.Generator().manual_seed(4)
    t = p["wg"].dtype
    x = torch.randn(rows, d, generator=gen).to(t).cuda()
    tokens = torch.randint(0, vocab, (rows,), generator=gen).cuda()
    dlp, dh = torch.randn(rows, generator=gen).cuda(), torch.randn(rows, generator=gen).cuda() * 0.1
    block = ScoredBlock(rows, d, f, vocab, dtype, act)
    lp, entropy = block.forward(x, tokens, p)
    grads = block.backward(dlp, dentropy=dh)
    want_lp, want_entropy, want = reference(x, tokens, p, dlp, dh, act)
    for name, got, ref in [("logprob", lp, want_lp), ("entropy", entropy, want_entropy)] + [(k, grads[k], want[k]) for k in want]:
        got = got.double().cpu()
        if dtype == "float32":
            assert float((got - ref).abs().max()) <= 2e-4 * float(ref.abs().max()), name
        else:
            assert float((got - ref).norm()) <= (3e-2 if dtype == "float16" else 2.5e-1) * float(ref.norm()), name


def test_training_raises_the_log_probability_and_one_token_agrees():
    rows, d, f, vocab = 96, 128, 320, 512
    p = parameters(d, f, vocab, "bfloat16", seed=5)
    gen = torch.Generator().manual_seed(6)
    x = torch.randn(rows, d, generator=gen).bfloat16().cuda()
    tokens = torch.randint(0, vocab, (rows,), generator=gen).cuda()
    block = ScoredBlock(rows, d, f, vocab, "bfloat16")
    seen = []
    for _ in range(6):
        lp, _ = block.forward(x, tokens, p)
        seen.append(float(lp.mean()))
        grads = block.backward(torch.full((rows,), 1.0 / rows, device="cuda"))
        for k in PARAMETERS:
            p[k].add_(grads[k], alpha=0.5)
    assert all(b > a for a, b in zip(seen, seen[1:])), seen
    lp, entropy = (t.clone() for t in block.forward(x, tokens, p))
    one = ScoredBlock(1, d, f, vocab, "bfloat16", top=3)
    one.forward(x[7:8], tokens[7:8], p)
    # other kernels, the same roundings to bfloat16 at each stage: a few of them apart
    assert abs(float(one.logprob[0]) - float(lp[7])) <= 0.05 and abs(float(one.entropy[0]) - float(entropy[7])) <= 0.05
    best = one.top_logprob[0].tolist()
    assert best == sorted(best, reverse=True) and float(one.z[0, int(one.top_index[0, 0])]) == float(one.z.max())
