"""Quantise a block, run it from its packed codes, and tune what is left of it.

    python examples/tune_quantized_block.py

The block is a layer norm, a linear layer and a mixture of experts.  Its
weights are quantised by the solver (bakron_factors, bakron_prepare,
bakron_quantize_grid), packed (bakron_pack), and from then on only the codes
are used:

1. the norm's gamma and beta are tuned so that the layer after it (P) sees of the
   quantised linear layer what it saw of the original one: forward through bakron_layernorm and
   bakron_linear, back through bakron_linear_grad and
   bakron_layernorm_grad; the loss is quadratic in (gamma, beta), so each
   step goes to the minimum along the gradient;
2. the samples of that pass, activations and gradients, are what a two-sided
   quantisation of the layer takes (bakron_factors, B from the gradients);
3. the block answers single tokens: bakron_layernorm, bakron_linear and bakron_moe,
   with outputs and workspaces kept from token to token.
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from kronecker_factored_gptq_gb300 import bakron as kb  # noqa: E402

EPS = 1e-5


def quantize(W, X, group, G=None, bits=3):
    """Codes of W and their grid, for samples X (and output gradients G)."""
    A, B = kb.bakron_factors(X.float(), None if G is None else G.float(), want_B=G is not None)
    UA, UB, _, _, _ = kb.bakron_prepare(A, 0.01, B, 0.01)
    scale, zero, qmin, qmax = kb.bakron_grid_params(W, bits, asymmetric=True, group=group)
    _, codes, _ = kb.bakron_quantize_grid(W, UA, UB, scale, zero, group, qmin, qmax)
    return codes, scale, zero, qmin, qmax


def pack(parts, group):
    """One packed weight of one matrix, or of several (experts)."""
    codes, scale, zero = (torch.stack([p[i] for p in parts]) if len(parts) > 1 else parts[0][i] for i in range(3))
    return kb.bakron_pack(codes, scale, parts[0][3], parts[0][4], zero=zero, group=group)


def silu(v):
    return v * torch.sigmoid(v)


def run(tokens=1024, d=512, m=768, experts=8, f=256, top_k=2, group=64, steps=6, dtype=torch.bfloat16, seed=0):
    """Returns the losses of the tuning steps, the error tr(B E A E^T) of the one-sided
    and of the two-sided quantisation, and the block's answers for eight tokens: one by
    one, and at once."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")
    x = (rand(tokens, d) * torch.exp(rand(d)) + 0.5 * rand(d)).to(dtype)
    gamma, beta = 1 + 0.2 * rand(d), 0.1 * rand(d)
    W, P = rand(m, d) / d ** 0.5, rand(m // 4, m) / m ** 0.5

    # the linear layer, one-sided, and what the original one answers
    h, mean, rstd = kb.bakron_layernorm(x, gamma, beta, EPS)
    want = h.float() @ W.T
    w = pack([quantize(W, h, group)], group)

    # 1. tune gamma and beta
    gamma, beta = gamma.clone(), beta.clone()
    losses = []
    for _ in range(steps + 1):
        h, mean, rstd = kb.bakron_layernorm(x, gamma, beta, EPS)
        error = (kb.bakron_linear(h, w).float() - want) @ P.T
        losses.append(0.5 * error.square().sum().item() / tokens)
        dz = (error @ P / tokens).to(dtype)
        dh = kb.bakron_linear_grad(dz, w)
        _, dgamma, dbeta = kb.bakron_layernorm_grad(dh, x, gamma, mean, rstd)
        # the outputs move along the gradient as those of a norm with its parameters do
        along, _, _ = kb.bakron_layernorm(x, dgamma, dbeta, EPS, want_stats=False)
        move = kb.bakron_linear(along, w).float() @ P.T
        step = (error * move).sum() / move.square().sum()
        gamma -= step * dgamma
        beta -= step * dbeta

    # 2. the same layer again, two-sided, for the samples of the last pass
    two = pack([quantize(W, h, group, G=dz)], group)
    A, B = kb.bakron_factors(h.float(), dz.float())

    def weighted(packed):
        E = packed.unpack() - W
        return ((E @ A) * (B @ E)).sum().item()

    sides = weighted(w), weighted(two)

    # 3. experts behind the layer, and tokens one by one
    h, _, _ = kb.bakron_layernorm(x, gamma, beta, EPS)
    z = kb.bakron_linear(h, w)
    router = (rand(experts, m) / m ** 0.5).to(dtype)
    w_in, w_out = [], []
    for _ in range(experts):
        I, O = rand(2 * f, m) / m ** 0.5, rand(m, f) / f ** 0.5
        u = z.float() @ I.T
        w_in.append(quantize(I, z, group, bits=4))
        w_out.append(quantize(O, silu(u[:, :f]) * u[:, f:], group, bits=4))
    w_in, w_out = pack(w_in, group), pack(w_out, group)

    n = min(8, tokens)
    h1 = torch.empty((1, d), dtype=dtype, device="cuda")
    rows = torch.empty((n, m), dtype=dtype, device="cuda")
    answers = torch.empty_like(rows)
    ws1, ws2 = kb.linear_workspace(w, 1, dtype), kb.moe_workspace(w_in, w_out, 1, top_k, dtype)
    for t in range(n):
        kb.bakron_layernorm(x[t:t + 1], gamma, beta, EPS, out=h1, want_stats=False)
        kb.bakron_linear(h1, w, out=rows[t:t + 1], workspace=ws1)
        kb.bakron_moe(rows[t:t + 1], router, w_in, w_out, top_k, out=answers[t:t + 1], workspace=ws2)
    together = kb.bakron_moe(rows, router, w_in, w_out, top_k)
    kb.bakron_async_status()
    return losses, sides, answers, together


def main():
    losses, sides, answers, together = run()
    print("loss per token while gamma and beta are tuned: " + " ".join("%.5f" % v for v in losses))
    print("weighted error of the layer: one-sided %.4g, two-sided %.4g" % sides)
    print("largest answer %.3f; one by one against together: %.5f"
          % (together.float().abs().max().item(), (answers.float() - together.float()).abs().max().item()))


if __name__ == "__main__":
    main()
