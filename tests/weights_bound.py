"""Bound of outputs whose softmax weights are the sum of two bf16, and what breaks it."""
import torch


def bound(o, mass, score, half):
    """Half a step of the result, each weight within half a step (2^-8) of what half a step (2^-8) of bf16 leaves of it, a
    score's error for the weights above and below the line."""
    return half * o.abs() + (2.0 ** -16 + 2 * score) * mass * 1.01 + 1e-30


def outputs(x, v, parts):
    """Softmax of scores x [row, position] over values v [position, D] with weights cut to `parts` bf16, rounded to bf16."""
    w = torch.exp(x - x.amax(1, keepdim=True))
    kept, rest = torch.zeros_like(w), w.clone()
    for _ in range(parts):
        step = rest.bfloat16().double()
        kept, rest = kept + step, rest - step
    return ((kept @ v) / w.sum(1, keepdim=True)).bfloat16().double()
