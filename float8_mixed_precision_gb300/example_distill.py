"""Example: a head distilled from a teacher's head, on a Float8 linear.

    python -m float8_mixed_precision_gb300.example_distill [--tokens 4096] [--steps 20]

The teacher's pass: its head linear (f8_linear_fwd), then f8_token_logprobs,
which keeps the 64 most likely tokens of each position.  The student's step:
RMS norm with its output's amax and E4M3 cast (f8_quantize_norm), the head GEMM,
loss and logit gradient in one pass over the logits and in their place, with
the gradient's amax (f8_distill_fwd_bwd), the cast on that amax, dgrad and wgrad
(f8_gemm_grouped), and the norm's backward (f8_norm_bwd).  No pass over the
logits only takes a maximum.  The same step runs through the modules of
float8_mixed_precision_gb300.nn under autograd, as a user's model would have it,
and both are timed.  Sizes are those of the Llama-3.1-8B head: 4096 features,
128256 tokens.
"""
from __future__ import annotations

import argparse

import torch

from . import binding as f8
from . import nn as f8nn
from . import ops


def teacher_top(hidden: torch.Tensor, weight: torch.Tensor, k: int, vocab: int | None = None):
    """(ids, log probabilities), both [tokens, k], of the teacher's most likely
    tokens."""
    logits, _ = f8.f8_linear_fwd(hidden, weight)
    _, _, _, ids, logp = ops.f8_token_logprobs(logits[:, :vocab], top_k=k)
    return ids, logp


def student_step(x: torch.Tensor, gain: torch.Tensor, weight: torch.Tensor, ids: torch.Tensor,
                 values: torch.Tensor, dloss: torch.Tensor, vocab: int | None = None,
                 tail: bool = True):
    """(loss per token, dx, dgain, dweight) of the head's distillation loss for
    the gradient dloss [tokens] of each token's loss."""
    xq, xq_t, xs, _, _, _, rstd = ops.f8_quantize_norm(x, gain, kind=f8.F8_RMS_NORM)
    wq, wq_t, ws, _ = f8.f8_quantize(weight)
    logits = f8.f8_gemm(xq, wq, xs, ws)
    amax = torch.empty((), dtype=torch.float32, device=x.device)
    loss, dlogits = ops.f8_distill_fwd_bwd(logits[:, :vocab], ids, values, dloss, tail=tail,
                                           dlogits=logits, amax_out=amax)
    dq, dq_t, ds = f8.f8_cast_transpose(dlogits, amax)
    dy, dweight = f8.f8_gemm_grouped([(dq, wq_t, ds, ws), (dq_t, xq_t, ds, xs)])
    dx, dgain, _ = ops.f8_norm_bwd(dy, x, gain, None, rstd, kind=f8.F8_RMS_NORM)
    return loss, dx, dgain, dweight


def main(argv=None) -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--features", type=int, default=4096)
    ap.add_argument("--vocab", type=int, default=128256)
    ap.add_argument("--top", type=int, default=64)
    args = ap.parse_args(argv)
    dev = torch.device("cuda", 0)
    M, D, V = args.tokens, args.features, args.vocab
    width = (V + 15) // 16 * 16
    gen = torch.Generator(device=dev).manual_seed(0)

    def rnd(shape, std):
        return (torch.randn(shape, generator=gen, device=dev) * std).to(torch.bfloat16)

    x = rnd((M, D), 1.0)
    teacher, weight = rnd((width, D), 4.0 * D ** -0.5), rnd((width, D), D ** -0.5)
    gain = torch.ones(D, dtype=torch.bfloat16, device=dev)
    dloss = torch.full((M,), 1.0 / M, device=dev)

    def timed(fn):
        for _ in range(3):
            fn()
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(args.steps):
            fn()
        b.record()
        b.synchronize()
        return a.elapsed_time(b) / args.steps

    ids, values = teacher_top(x, teacher, args.top, V)
    ms = timed(lambda: teacher_top(x, teacher, args.top, V))
    print(f"teacher: {ms:.3f} ms, top {args.top} tokens hold {values.exp().sum(1).mean().item():.3f}")

    ms = timed(lambda: student_step(x, gain, weight, ids, values, dloss, V))
    print(f"student step, loss and gradient in one pass: {ms:.3f} ms")

    norm = f8nn.RMSNorm(D, device=dev)
    head = f8nn.Float8Linear(D, width, weight=torch.nn.Parameter(weight.clone()))
    leaf = x.clone().requires_grad_(True)

    def module_step():
        for p in (leaf, norm.weight, head.weight):
            p.grad = None
        f8nn.distill_loss(head(norm(leaf)), ids, values, tail=True, vocab=V).mean().backward()

    ms = timed(module_step)
    print(f"student step, modules under autograd:        {ms:.3f} ms")

    losses = []
    for _ in range(args.steps):
        loss, _, dgain, dweight = student_step(x, gain, weight, ids, values, dloss, V)
        weight.sub_(dweight, alpha=10.0)
        gain.sub_(dgain, alpha=0.1)
        losses.append(loss.mean())
    print(f"loss over {args.steps} steps: {losses[0].item():.4f} -> {losses[-1].item():.4f}")
    status = f8.f8_last_device_status()
    if status != 0:
        raise RuntimeError(f8.f8_status_string(status))


if __name__ == "__main__":
    main()
