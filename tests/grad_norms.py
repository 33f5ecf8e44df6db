"""Bounds on a gradient's error in the norm, for tests.

Per element a bf16 dW may be off by 2^-8 of the sum of its products' magnitudes, which
over many tokens is far more than its error and hides a token left out.  In the norm
the roundings average.  A rounding to nearest of a value with mantissa 1 <= f < 2 is
off by at most 2^-8 / f of it (bf16), evenly spread: an rms of at most 2^-8 / sqrt(3).
Roundings of different values are independent, so that
  dX (bf16)  exact products, one rounding of the output:     2^-8 / sqrt(3)
  dW (bf16)  one rounding of q / s a product, which the sum over the tokens passes on
             with the same share of the norm, and one of the output:
                                                             2^-8 sqrt(2 / 3)
  dW (fp32)  two bf16 a product: at most 2^-16 each, 2^-16 / sqrt(3) in the mean, and
             the sums of up to 2048 tokens (twice as many products) are added with 2^-24
The tensor core truncates its fp32 accumulator: every addition of 16 products takes at
most two fp32 steps, 2^-22, of it.
A token (or an output row) left out or taken twice, of L of the same size, makes an error
of 1 / sqrt(L) of the norm: ten times the bound at 1024 and still three at 10240.
"""

import torch

F64 = torch.float64
BF16 = 2.0**-8


def rel_norm(got, want):
    return ((got.to(F64) - want).norm() / want.norm()).item()


def dx_bound(L):
    return BF16 / 3**0.5 + 2.0**-22 * L / 16


def dw_bound(dtype, L):
    if dtype == torch.bfloat16:
        return BF16 * (2 / 3) ** 0.5 + 2.0**-22 * L / 16
    return 2.0**-16 / 3**0.5 + 2.0**-22 * 2 * min(L, 2048) / 16 + 2.0**-24 * (L / 2048 + 1)


def even_grads(M, N, seed, device="cpu"):
    """Output gradients of the same size in every row and column."""
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(M, N, generator=g) * 1e-3).to(torch.bfloat16).to(device)
