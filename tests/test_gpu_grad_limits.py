"""The weight gradient at the limits of the scales it takes.

Per product an fp32 dW takes q / s as two bf16: off by at most 2^-16 |q / s| (half a
step of half a step, 2^-8 each), as long as the second one is a normal number or what
is flushed is below that: 2^-126 <= 2^-16 / s, s <= 2^110.  A bf16 dW takes one bf16,
2^-8.  With one token there is one product an element: no sums.  The reciprocal is off
by 2^-23.  The outputs are rounded once more (fp32: hi and lo are added, 2^-24 twice at
most; bf16 2^-8)."""

import pytest
import torch

from bitlinear_bl_forward_b200 import bl

pytestmark = pytest.mark.gpu

F64 = torch.float64
BF16_MAX = torch.finfo(torch.bfloat16).max


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def check(scale, q, size):
    K, N = q.numel(), 40
    dY = (torch.randn(1, N, generator=torch.Generator().manual_seed(1)) * size).to(torch.bfloat16).cuda()
    s = torch.full((1,), scale, dtype=torch.float32, device="cuda")
    want = dY.to(F64).t() @ (q.to(F64) / s.to(F64))[None, :]
    assert torch.isfinite(want.to(torch.bfloat16)).all()   # the case itself stays in range
    for dtype, step in ((torch.float32, 2.0**-16 + 2.0**-22), (torch.bfloat16, 2.0**-8 + 2.0**-8 + 2.0**-16 + 2.0**-22)):
        got = bl.bl_backward_weight(dY, q[None, :].contiguous(), s, dtype=dtype)
        assert got.shape == (N, K)
        err = (got.to(F64) - want).abs()
        assert bool((err <= step * want.abs()).all()), (scale, dtype, (err / want.abs().clamp_min(1e-300)).max().item())


@pytest.mark.parametrize("scale", [2.0**110, 1.7 * 2.0**109, 2.0**100, 2.0**23.6, 1.0, 2.0**-100])
def test_all_codes(scale):
    q = torch.arange(-128, 128, dtype=torch.int32).to(torch.int8).cuda()
    check(scale, q, scale * 1e-3 if scale > 1 else 1e-3)


@pytest.mark.parametrize("bits,top", [(8, 127), (4, 7)])
def test_scales_of_the_largest_activations(bits, top):
    # what the forward writes for a token with the largest finite bf16
    X = torch.zeros(1, 64, dtype=torch.bfloat16, device="cuda")
    X[0, :3] = torch.tensor([BF16_MAX, -BF16_MAX, BF16_MAX / 2], dtype=torch.bfloat16)
    q, s = bl.bl_quant_act(X, bits)
    assert q.max().item() == top and q.min().item() == -top
    check(s.item(), q[0], 1e-3)


def test_smallest_activations():
    # below 1e-5 the scale stays at Q / 1e-5: the largest that the forward writes
    X = torch.full((1, 64), 1e-6, dtype=torch.bfloat16, device="cuda")
    q, s = bl.bl_quant_act(X)
    assert s.item() <= 2.0**23.6
    check(s.item(), q[0], 1.0)


@pytest.mark.parametrize("norm", [bl.BL_NORM_RMS, bl.BL_NORM_LAYER])
@pytest.mark.parametrize("K", [64, 2560, 8256])
def test_norm_rows_beyond_the_sums_range(K, norm):
    # squares whose sum passes 2^128 leave an infinite statistic in their row; the
    # largest row that the limit allows, and every other row, are as without them
    g = torch.Generator().manual_seed(K)
    X = torch.randn(6, K, generator=g).to(torch.bfloat16)
    X[4] = (torch.rand(K, generator=g) - 0.5).to(torch.bfloat16) * (2.0**64 / K**0.5)
    bad = X.clone()
    bad[2, K // 2] = 1e30
    X, bad = X.cuda(), bad.cuda()
    Y, mean, stat = bl.bl_norm_forward(X, norm)
    Yb, meanb, statb = bl.bl_norm_forward(bad, norm)
    others = [0, 1, 3, 4, 5]
    assert torch.isinf(statb[2]) and torch.isfinite(stat).all() and torch.isfinite(Y.float()).all()
    assert torch.equal(Y[others], Yb[others]) and torch.equal(stat[others], statb[others])
    if mean is not None:
        assert torch.equal(mean[others], meanb[others])
    # the large row's values: mean 0, statistic far above eps
    x = X[4].to(F64)
    d = x - x.mean() if norm == bl.BL_NORM_LAYER else x
    want = d / d.square().mean().sqrt()
    # 2^-8 of the output; sums of K fp32 terms, at most K / 32 + 16 additions deep, of
    # the statistic (half of it in the root) and of the mean; 2^-20 for the rest
    depth = 2.0**-24 * (K / 32 + 16)
    spread = x.abs().mean() / d.square().mean().sqrt()
    tol = (2.0**-8 + depth + 2.0**-20) * want.abs() + depth * spread
    assert bool(((Y[4].to(F64) - want).abs() <= tol).all())
