"""Operands whose products have exact fp32 sums: integer activations and
weights that are multiples of 1/2, small enough that every partial sum, in any
order, is a multiple of 1/2 below 2^23.  A product has then one right answer,
the bf16 nearest to the sum, and a missing, doubled or misplaced block of k
shows in it."""
import torch

X_MAX, W_MAX = 3, 12  # 3 * 12 * 2 halves * K < 2^24 for K up to 233,016


def integers(shape, g, hi=X_MAX, device="cuda"):
    return torch.randint(-hi, hi + 1, shape, generator=g, device=device).to(torch.bfloat16)


def product(a, B):
    """bf16 nearest to the exact a B."""
    want = a.double() @ B.double()
    assert a.shape[1] < 233_016 and a.abs().max() <= X_MAX and B.abs().max() <= W_MAX
    return want.float().to(torch.bfloat16)  # the sum is exact in fp32: one rounding
