"""GPU tests of the training entry points against plain 64-bit formulas.

Half a step of a rounding, relative: bf16 2^-8, fp32 2^-24.  Tolerances, per
element, with P the sum of the magnitudes of the products that are added:

  dX   2^-8 |v|                     the bf16 output
       + 2^-22 (L/16 + 4) P         fp32 sums of L products: the tensor core
                                    adds 16 products and the running sum at
                                    once, each step off by at most two steps
                                    of the largest (2^-22 P)
  dW   the same sums, plus per product what q / s loses as operand:
         fp32 out  2^-16 P  (two bf16: 2^-8 of 2^-8), twice as many steps
         bf16 out  2^-8 P   (one bf16), and 2^-8 |v| of the output
  norm rows of K elements, at most K/32 + 16 additions deep (the sums are
       formed by at least 32 lanes): a relative 2^-24 (K/32 + 16) of the sum
       of magnitudes for every statistic; written out at each test.
"""

import numpy as np
import pytest
import torch

from bitlinear_bl_forward_b200 import bl
from bitlinear_bl_forward_b200.inputs import random_case
from tests.gpu_helpers import x_to_dev
from tests.test_gpu_canary import Guarded

pytestmark = pytest.mark.gpu

EPS = 1e-5
F64 = torch.float64


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    bl.lib()
    bl.bl_device_status(clear=True)
    yield
    assert bl.bl_device_status(clear=True) == (0, 0)


def grads(M, N, seed):
    g = torch.Generator().manual_seed(seed)
    d = torch.randn(M, N, generator=g) * 1e-3 * torch.exp(torch.randn(M, 1, generator=g))
    return d.to(torch.bfloat16).cuda()


def layer(M, K, N, seed, bits=8):
    """X, packed weights, gamma, dense codes, and the forward's checkpoint."""
    X, W = random_case(M, K, N, seed)
    Wp, gamma = bl.bl_quantize_weights(torch.from_numpy(W).cuda())
    C = bl.bl_unpack_weights(Wp, N, K).to(F64)
    X = x_to_dev(X)
    q, s = bl.bl_quant_act(X, bits)
    return X, Wp, gamma, C, q, s


def worst(got, want, tol):
    r = ((got.to(F64) - want).abs() / tol).max().item() if got.numel() else 0.0
    assert np.isfinite(r), "not finite"
    return r


def check_dx(dX, dY, C, gamma):
    w = gamma.to(F64)
    want = (dY.to(F64) @ C) * w
    P = (dY.to(F64).abs() @ C.abs()) * w
    tol = 2.0**-8 * want.abs() + 2.0**-22 * (dY.shape[1] / 16 + 4) * P + 1e-300
    assert worst(dX, want, tol) <= 1.0


def check_dw(dW, dY, q, s, base=None):
    xh = q.to(F64) / s.to(F64)[:, None]
    want = dY.to(F64).t() @ xh
    P = dY.to(F64).abs().t() @ xh.abs()
    L = dY.shape[0]
    steps = 2.0**-22 * (2 * L / 16 + 4) * P
    if base is not None:
        want = want + base.to(F64)
    if dW.dtype == torch.float32:
        tol = 2.0**-16 * P + steps + 2.0**-23 * want.abs()
    else:
        tol = 2.0**-8 * P + steps + 2.0**-8 * want.abs()
    # a value whose products all vanish is exact
    assert worst(dW, want, tol + 1e-300) <= 1.0


# sizes: one token; tiles of 32, 64, 128 and 256 tokens and one more; N that is
# not a multiple of 8 (rows of dY off 16-byte boundaries) or 64; one and many
# k tiles, the last one whole or half; sums long enough to be split
SHAPES = [(1, 64, 1), (1, 2560, 6912), (2, 64, 8), (3, 128, 7), (16, 256, 512), (17, 320, 130), (32, 192, 64),
          (33, 256, 65), (64, 448, 1000), (65, 64, 129), (128, 512, 4096), (129, 576, 258), (255, 192, 33),
          (257, 1344, 1003), (300, 256, 72), (513, 320, 700), (1000, 128, 256), (2049, 256, 264)]


@pytest.mark.parametrize("M,K,N", SHAPES)
def test_backward_input(M, K, N):
    _, Wp, gamma, C, _, _ = layer(M, K, N, M + K + N)
    dY = grads(M, N, 3 * M + N)
    check_dx(bl.bl_backward_input(dY, Wp, gamma, K), dY, C, gamma)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_backward_weight(M, K, N, bits):
    *_, q, s = layer(M, K, N, M + K + N, bits)
    dY = grads(M, N, 5 * M + N)
    g = torch.Generator().manual_seed(N)
    base = (torch.randn(N, K, generator=g) * 1e-2).cuda()
    for dtype in (torch.float32, torch.bfloat16):
        check_dw(bl.bl_backward_weight(dY, q, s, dtype=dtype), dY, q, s)
        b = base.to(dtype)
        out = b.clone()
        assert bl.bl_backward_weight(dY, q, s, out=out, accumulate=True) is out
        check_dw(out, dY, q, s, base=b)


def test_long_sums():
    # contraction far longer than the output is large
    M, K, N = 20000, 64, 24
    *_, q, s = layer(M, K, N, 4)
    dY = grads(M, N, 9)
    check_dw(bl.bl_backward_weight(dY, q, s), dY, q, s)
    M, K, N = 5, 64, 30001
    _, Wp, gamma, C, _, _ = layer(M, K, N, 5)
    dY = grads(M, N, 10)
    check_dx(bl.bl_backward_input(dY, Wp, gamma, K), dY, C, gamma)


def test_weight_gradient_accuracy_over_many_tokens():
    # the fp32 gradient keeps fp32-like accuracy: two bf16 a product leave at
    # most 2^-16 each, in the mean (independent errors, a uniform half step has
    # an rms of 1/sqrt(3)) below 2^-16 of the gradient's norm; the same again
    # is left for the sums
    M, K, N = 8192, 256, 264
    *_, q, s = layer(M, K, N, 11)
    dY = grads(M, N, 12)
    want = dY.to(F64).t() @ (q.to(F64) / s.to(F64)[:, None])
    rel = ((bl.bl_backward_weight(dY, q, s).to(F64) - want).norm() / want.norm()).item()
    assert rel <= 2.0**-16, rel


def test_rows_of_zeros_and_zero_gradients():
    # a token of zeros has s = Q / 1e-5 and codes 0; a zero gradient gives zeros
    M, K, N = 37, 128, 40
    X = torch.randn(M, K).to(torch.bfloat16).cuda()
    X[3] = 0
    X[36] = 0
    _, Wp, gamma, C, _, _ = layer(4, K, N, 1)
    Y, q, s, stat = bl.bl_forward_checkpoint(X, Wp, gamma, N)
    assert stat is None and not q[3].any() and not Y[3].any()
    dY = grads(M, N, 2)
    dY[:, 5] = 0
    dY[7] = 0
    dW = bl.bl_backward_weight(dY, q, s)
    check_dw(dW, dY, q, s)
    assert not dW[5].any()
    dX = bl.bl_backward_input(dY, Wp, gamma, K)
    check_dx(dX, dY, C, gamma)
    assert not dX[7].any()


def test_extreme_scales():
    # tokens from the smallest normal to near the largest bf16
    M, K, N = 24, 64, 16
    X = torch.randn(M, K, generator=torch.Generator().manual_seed(0))
    X = (X * torch.logspace(-36, 36, M)[:, None]).to(torch.bfloat16).cuda()
    _, Wp, gamma, C, _, _ = layer(4, K, N, 1)
    Y, q, s, _ = bl.bl_forward_checkpoint(X, Wp, gamma, N)
    for m in range(0, M, 5):   # one token at a time: the products stay in range
        dY = grads(1, N, m)
        check_dw(bl.bl_backward_weight(dY, q[m:m + 1].clone(), s[m:m + 1].clone()), dY, q[m:m + 1], s[m:m + 1])


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("norm", [None, bl.BL_NORM_RMS, bl.BL_NORM_LAYER])
@pytest.mark.parametrize("M,K,N", [(1, 2560, 700), (2, 64, 9), (3, 192, 130), (16, 256, 512), (65, 320, 136),
                                   (300, 2560, 264), (1300, 256, 64)])
def test_forward_checkpoint_is_the_forward(M, K, N, norm, bits):
    X, Wp, gamma, _, q0, s0 = layer(M, K, N, M + N, bits)
    Y, q, s, stat = bl.bl_forward_checkpoint(X, Wp, gamma, N, bits, norm=norm, eps=EPS)
    if norm is None:
        want, st = bl.bl_forward(X, Wp, gamma, N, bits), None
    elif norm == bl.BL_NORM_RMS:
        want = bl.bl_forward_rmsnorm(X, Wp, gamma, N, bits, eps=EPS)
        q0, s0, st = bl.bl_quant_act_rmsnorm(X, bits, eps=EPS)
    else:
        want = bl.bl_forward_layernorm(X, Wp, gamma, N, bits, eps=EPS)
        q0, s0, _, st = bl.bl_quant_act_layernorm(X, bits, eps=EPS)
    assert torch.equal(Y.view(torch.int16), want.view(torch.int16))
    assert torch.equal(q, q0) and torch.equal(s, s0)
    assert stat is None if st is None else torch.equal(stat, st)


def norm_ref(x, norm):
    x = x.to(F64)
    mu = x.mean(1) if norm == bl.BL_NORM_LAYER else torch.zeros_like(x[:, 0])
    d = x - mu[:, None]
    return mu, d.square().mean(1), d


def fp32_err(K):
    return 2.0**-24 * (K / 32 + 16)


# widths: one chunk of a warp; ragged; each number of chunks a thread holds;
# beyond what stays in registers; the widest
NORMS = [(1, 64), (1, 2560), (3, 192), (7, 2048), (5, 2112), (33, 2560), (301, 1344), (4, 4096), (9, 4160), (6, 8192),
         (257, 8192), (10, 8256), (40, 16448), (2, 65536), (700, 512), (1999, 128)]


@pytest.mark.parametrize("norm", [bl.BL_NORM_RMS, bl.BL_NORM_LAYER])
@pytest.mark.parametrize("M,K", NORMS)
def test_norm_forward_and_backward(M, K, norm):
    g = torch.Generator().manual_seed(M * 7 + K)
    X = (torch.randn(M, K, generator=g) * torch.exp(torch.randn(M, 1, generator=g)) + 0.5).to(torch.bfloat16).cuda()
    w = (1 + 0.2 * torch.randn(K, generator=g)).to(torch.bfloat16).cuda()
    b = (0.2 * torch.randn(K, generator=g)).to(torch.bfloat16).cuda()
    dY = grads(M, K, K)
    la = norm == bl.BL_NORM_LAYER
    e = fp32_err(K)
    mu, var, d = norm_ref(X, norm)
    mag = X.to(F64).abs().mean(1)
    for ww, bb in ((w, b), (None, None), (w, None), (None, b)):
        Y, mean, stat = bl.bl_norm_forward(X, norm, weight=ww, bias=bb, eps=EPS)
        e_mu = e * mag if la else torch.zeros_like(mag)
        assert (mean is not None) == la
        if la:
            assert worst(mean, mu, e_mu + 1e-300) <= 1.0
        # the squares: a relative e, and twice the mean's error times the deviations (their mean vanishes)
        e_var = (e + 2.0**-20) * var + 2 * e_mu.square()
        assert worst(stat, var, e_var) <= 1.0
        rs = (var + EPS).rsqrt()
        xh = d * rs[:, None]
        wd = ww.to(F64) if ww is not None else torch.ones(K, dtype=F64, device="cuda")
        want = xh * wd + (bb.to(F64) if bb is not None else 0.0)
        # rounding of y; x - mu (its mean's error), the statistic's half error, and four fp32 steps
        rel = (0.5 * e_var / (var + EPS) + 2.0**-22)[:, None]
        tol = 2.0**-8 * want.abs() + (e_mu * rs)[:, None] * wd.abs() + rel * (xh * wd).abs() + 2.0**-23 * want.abs()
        assert worst(Y, want, tol * (1 + 2.0**-7) + 1e-300) <= 1.0
    # gradients, with the forward's statistics as inputs
    for ww, need_b in ((w, True), (None, False), (w, False), (None, True)):
        dX, dw, db = bl.bl_norm_backward(dY, X, norm, stat, mean=mean, weight=ww, need_bias=need_b, eps=EPS)
        m64 = mean.to(F64) if la else torch.zeros_like(mag)
        rs = (stat.to(F64) + EPS).rsqrt()[:, None]
        xh = (X.to(F64) - m64[:, None]) * rs
        dy = dY.to(F64)
        gg = dy * ww.to(F64) if ww is not None else dy
        want = (gg - xh * (gg * xh).mean(1, keepdim=True) - (gg.mean(1, keepdim=True) if la else 0.0)) * rs
        terms = (gg.abs() + xh.abs() * (gg * xh).abs().mean(1, keepdim=True) + gg.abs().mean(1, keepdim=True)) * rs
        assert worst(dX, want, 2.0**-8 * want.abs() + (e + 2.0**-20) * terms + 1e-300) <= 1.0
        assert (dw is None) == (ww is None) and (db is None) == (not need_b)
        # sums over M rows: at most M additions deep
        em = 2.0**-24 * (M + 16)
        if dw is not None:
            assert worst(dw, (dy * xh).sum(0), em * (dy * xh).abs().sum(0) + 1e-300) <= 1.0
        if db is not None:
            assert worst(db, dy.sum(0), em * dy.abs().sum(0) + 1e-300) <= 1.0


@pytest.mark.parametrize("norm", [bl.BL_NORM_RMS, bl.BL_NORM_LAYER])
@pytest.mark.parametrize("M,K", [(1, 64), (5, 320), (129, 2560), (17, 4160), (3, 8256), (2, 65536), (4100, 128)])
def test_norm_backward_from_the_checkpoint(M, K, norm):
    X = x_to_dev(random_case(M, K, 8, M + K)[0])
    q, s, stat = (bl.bl_quant_act_rmsnorm(X, 8, eps=EPS) if norm == bl.BL_NORM_RMS else
                  [bl.bl_quant_act_layernorm(X, 8, eps=EPS)[i] for i in (0, 1, 3)])
    g = grads(M, K, 1)
    xh = q.to(F64) / s.to(F64)[:, None]
    rs = (stat.to(F64) + EPS).rsqrt()[:, None]
    gd = g.to(F64)
    la = norm == bl.BL_NORM_LAYER
    want = (gd - xh * (gd * xh).mean(1, keepdim=True) - (gd.mean(1, keepdim=True) if la else 0.0)) * rs
    terms = (gd.abs() + xh.abs() * (gd * xh).abs().mean(1, keepdim=True) + gd.abs().mean(1, keepdim=True)) * rs
    tol = 2.0**-8 * want.abs() + (fp32_err(K) + 2.0**-20) * terms + 1e-300
    dX = bl.bl_norm_backward_checkpoint(g, q, s, norm, stat, eps=EPS)
    assert worst(dX, want, tol) <= 1.0
    # in place
    g2 = g.clone()
    assert torch.equal(bl.bl_norm_backward_checkpoint(g2, q, s, norm, stat, eps=EPS, out=g2), dX)


def test_norm_in_place_and_accumulate():
    for M, K in ((40, 320), (9, 8256)):
        X = torch.randn(M, K).to(torch.bfloat16).cuda()
        w = torch.randn(K).to(torch.bfloat16).cuda()
        dY = grads(M, K, 1)
        Y, mean, stat = bl.bl_norm_forward(X, bl.BL_NORM_LAYER, weight=w)
        dX, dw, db = bl.bl_norm_backward(dY, X, bl.BL_NORM_LAYER, stat, mean=mean, weight=w, need_bias=True)
        X2 = X.clone()
        assert torch.equal(bl.bl_norm_forward(X2, bl.BL_NORM_LAYER, weight=w, out=X2)[0], Y)
        d2, dw2, db2 = dY.clone(), torch.ones(K, device="cuda"), torch.full((K,), 2.0, device="cuda")
        bl.bl_norm_backward(d2, X, bl.BL_NORM_LAYER, stat, mean=mean, weight=w, out=d2, dweight=dw2, dbias=db2,
                            accumulate=True)
        assert torch.equal(d2, dX) and torch.equal(dw2, 1 + dw) and torch.equal(db2, 2 + db)
        x3 = X.clone()
        assert torch.equal(bl.bl_norm_backward(dY, x3, bl.BL_NORM_LAYER, stat, mean=mean, weight=w, out=x3)[0], dX)


def test_no_tokens():
    K, N = 64, 24
    Wp = torch.zeros(N, K // 4, dtype=torch.uint8, device="cuda")
    one = torch.ones(1, device="cuda")
    X = torch.empty(0, K, dtype=torch.bfloat16, device="cuda")
    dY = torch.empty(0, N, dtype=torch.bfloat16, device="cuda")
    Y, q, s, stat = bl.bl_forward_checkpoint(X, Wp, one, N, norm=bl.BL_NORM_RMS)
    assert Y.shape == (0, N) and q.shape == (0, K) and stat.shape == (0,)
    assert bl.bl_backward_input(dY, Wp, one, K).shape == (0, K)
    for dtype in (torch.float32, torch.bfloat16):
        out = torch.full((N, K), 3.0, dtype=dtype, device="cuda")
        bl.bl_backward_weight(dY, q, s, out=out, accumulate=True)
        assert bool((out == 3).all())
        bl.bl_backward_weight(dY, q, s, out=out)
        assert not out.any()
    dw, db = torch.ones(K, device="cuda"), torch.ones(K, device="cuda")
    bl.bl_norm_backward(X, X, bl.BL_NORM_LAYER, s, mean=s, dweight=dw, dbias=db)
    assert not dw.any() and not db.any()
    assert bl.bl_norm_forward(X, bl.BL_NORM_LAYER)[0].shape == (0, K)


def test_gradients_against_differences():
    # Y = X^ (gamma C)^T is linear in X^ and in the weights, the norm is not:
    # central differences of 64-bit forwards along random directions
    M, K, N = 19, 192, 50
    X, Wp, gamma, C, q, s = layer(M, K, N, 7)
    dY = grads(M, N, 8)
    dy = dY.to(F64)
    W = C * gamma.to(F64)
    xh = q.to(F64) / s.to(F64)[:, None]
    loss = lambda x, w: ((x @ w.t()) * dy).sum()  # noqa: E731
    g = torch.Generator(device="cuda").manual_seed(5)
    dX, dW = bl.bl_backward_input(dY, Wp, gamma, K), bl.bl_backward_weight(dY, q, s)
    for grad, f, x, half in ((dX, lambda t: loss(t, W), xh, 2.0**-8), (dW, lambda t: loss(xh, t), W, 2.0**-16)):
        u = torch.randn(x.shape, generator=g, device="cuda", dtype=F64)
        num = (f(x + 1e-3 * u) - f(x - 1e-3 * u)) / 2e-3
        ana = (grad.to(F64) * u).sum()
        # what the roundings of the gradient's elements may add up to
        assert abs(num - ana) <= (half * 1.5 * (grad.to(F64).abs() * u.abs()).sum() + 1e-9).item()
    # the norm
    w = (1 + 0.2 * torch.randn(K, generator=g, device="cuda")).to(torch.bfloat16)
    dyn = grads(M, K, 3)
    for norm in (bl.BL_NORM_RMS, bl.BL_NORM_LAYER):
        _, mean, stat = bl.bl_norm_forward(X, norm, weight=w)
        dx, dw, db = bl.bl_norm_backward(dyn, X, norm, stat, mean=mean, weight=w, need_bias=True)

        def f(x, ww, bb):
            mu, var, d = norm_ref(x, norm)
            return ((d * (var + EPS).rsqrt()[:, None] * ww + bb) * dyn.to(F64)).sum()

        x0, w0, b0 = X.to(F64), w.to(F64), torch.zeros(K, device="cuda", dtype=F64)
        for grad, at in ((dx, 0), (dw, 1), (db, 2)):
            args = [x0, w0, b0]
            u = torch.randn(args[at].shape, generator=g, device="cuda", dtype=F64)
            h = 1e-5
            hi, lo = list(args), list(args)
            hi[at], lo[at] = args[at] + h * u, args[at] - h * u
            num = (f(*hi) - f(*lo)) / (2 * h)
            ana = (grad.to(F64) * u).sum()
            bound = (2.0**-8 if at == 0 else 2.0**-18) * 1.5 * (grad.to(F64).abs() * u.abs()).sum() + 1e-8
            assert abs(num - ana) <= bound.item(), (norm, at)


@pytest.mark.parametrize("norm", [None, bl.BL_NORM_RMS, bl.BL_NORM_LAYER])
def test_a_training_step(norm):
    """The calls of one step together, as they are used: two micro-batches
    through norm + BitLinear and back, gradients added up."""
    K, N = 320, 130
    g = torch.Generator().manual_seed(0)
    Wl = torch.randn(N, K, generator=g) * 0.02
    Wp, gamma = bl.bl_quantize_weights(Wl.cuda())
    C = bl.bl_unpack_weights(Wp, N, K).to(F64)
    dW = torch.zeros(N, K, device="cuda")
    want = torch.zeros(N, K, device="cuda", dtype=F64)
    P = torch.zeros(N, K, device="cuda", dtype=F64)
    for i, M in enumerate((33, 70)):
        X = torch.randn(M, K, generator=g).to(torch.bfloat16).cuda()
        Y, q, s, stat = bl.bl_forward_checkpoint(X, Wp, gamma, N, norm=norm, eps=EPS)
        xh = q.to(F64) / s.to(F64)[:, None]
        # the 64-bit sum of whole numbers is exact (rounded factors would leave 1e-17 where it is zero)
        y = (q.to(F64) @ C.t()) * (gamma.to(F64) / s.to(F64))[:, None]
        # fp32(acc) exact, gamma / s, the product: three roundings, then bf16
        assert worst(Y, y, (2.0**-8 + 2.0**-22) * y.abs() + 1e-300) <= 1.0
        dY = (Y.float() - 1.0).mul(1e-2).to(torch.bfloat16)
        dXn = bl.bl_backward_input(dY, Wp, gamma, K)
        check_dx(dXn, dY, C, gamma)
        bl.bl_backward_weight(dY, q, s, out=dW, accumulate=True)
        want += dY.to(F64).t() @ xh
        P += dY.to(F64).abs().t() @ xh.abs()
        if norm is not None:
            dX = bl.bl_norm_backward_checkpoint(dXn, q, s, norm, stat, eps=EPS)
            assert torch.isfinite(dX.float()).all()
            # the bf16 input's own backward differs by the codes' half steps only
            mean = X.float().mean(1) if norm == bl.BL_NORM_LAYER else None
            dX2, _, _ = bl.bl_norm_backward(dXn, X, norm, stat, mean=mean, eps=EPS)
            d, r = (dX.to(F64) - dX2.to(F64)), dX2.to(F64)
            # |xh error| <= half a code step, 1 / (2 s); it enters twice, times mean(g xh) and g / sqrt(K)
            assert (d.norm() / r.norm()).item() <= 2 * (0.5 / s.to(F64)).max().item() + 2.0**-7
    assert worst(dW, want, (2.0**-16 + 2.0**-22 * 30) * P + 2.0**-22 * want.abs() + 1e-300) <= 1.0


@pytest.mark.parametrize("M,K,N", [(5, 320, 130), (130, 192, 72), (257, 1344, 1003), (300, 64, 264)])
def test_writes_stay_in_bounds_and_repeat(M, K, N):
    X, Wp, gamma, _, q, s = layer(M, K, N, 3)
    dY = grads(M, N, 4)
    dX = Guarded((M, K), torch.bfloat16)
    ws = Guarded((max(16, bl.bl_backward_input_workspace_bytes(M, K, N)),), torch.uint8)
    bl.bl_backward_input(dY, Wp, gamma, K, out=dX.t, workspace=ws.t)
    assert dX.intact() and ws.intact()
    assert torch.equal(dX.t, bl.bl_backward_input(dY, Wp, gamma, K))
    for dtype in (torch.float32, torch.bfloat16):
        flags = bl.BL_GRAD_BF16 if dtype == torch.bfloat16 else 0
        for acc in (False, True):
            dW = Guarded((N, K), dtype)
            dW.t.zero_()
            ws = Guarded((max(16, bl.bl_backward_weight_workspace_bytes(M, K, N, flags | acc)),), torch.uint8)
            bl.bl_backward_weight(dY, q, s, out=dW.t, accumulate=acc, workspace=ws.t)
            assert dW.intact() and ws.intact()
            assert torch.equal(dW.t, bl.bl_backward_weight(dY, q, s, dtype=dtype))
    Y = Guarded((M, N), torch.bfloat16)
    ws = Guarded((bl.bl_forward_checkpoint_workspace_bytes(M, K, N),), torch.uint8)
    bl.bl_forward_checkpoint(X, Wp, gamma, N, out=Y.t, workspace=ws.t)
    assert Y.intact() and ws.intact()
    for norm in (bl.BL_NORM_RMS, bl.BL_NORM_LAYER):
        o = Guarded((M, K), torch.bfloat16)
        _, mean, stat = bl.bl_norm_forward(X, norm, out=o.t)
        assert o.intact()
        dw, db = Guarded((K,), torch.float32), Guarded((K,), torch.float32)
        ws = Guarded((bl.bl_norm_backward_workspace_bytes(M, K),), torch.uint8)
        dYn = grads(M, K, 6)
        a = bl.bl_norm_backward(dYn, X, norm, stat, mean=mean, out=o.t, dweight=dw.t, dbias=db.t, workspace=ws.t)
        assert o.intact() and dw.intact() and db.intact() and ws.intact()
        b = bl.bl_norm_backward(dYn, X, norm, stat, mean=mean, dweight=torch.empty(K, device="cuda"), need_bias=True)
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_streams_and_graphs():
    """Another stream than the default one; a captured step replayed on new
    contents of the same buffers."""
    M, K, N = 70, 320, 200
    X, Wp, gamma, C, _, _ = layer(M, K, N, 2)
    dY = grads(M, N, 1)

    def step(x, dy):
        Y, q, s, stat = bl.bl_forward_checkpoint(x, Wp, gamma, N, norm=bl.BL_NORM_LAYER)
        dXn = bl.bl_backward_input(dy, Wp, gamma, K)
        dW = bl.bl_backward_weight(dy, q, s)
        dX = bl.bl_norm_backward_checkpoint(dXn, q, s, bl.BL_NORM_LAYER, stat)
        return Y, dXn, dW, dX

    want = step(X, dY)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = step(X, dY)
    torch.cuda.current_stream().wait_stream(st)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    x2, dy2 = X.clone(), dY.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(x2, dy2)
    for seed in (3, 4):
        x2.copy_(x_to_dev(random_case(M, K, N, seed)[0]))
        dy2.copy_(grads(M, N, seed))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, step(x2, dy2)))


def test_binding_refuses():
    M, K, N = 8, 64, 24
    X, Wp, gamma, _, q, s = layer(M, K, N, 1)
    dY = grads(M, N, 1)
    with pytest.raises(ValueError):
        bl.bl_backward_input(dY, Wp[:-1].clone(), gamma, K)
    with pytest.raises(ValueError):
        bl.bl_backward_input(dY.t(), Wp, gamma, K)
    with pytest.raises(TypeError):
        bl.bl_backward_input(dY.float(), Wp, gamma, K)
    with pytest.raises(ValueError):
        bl.bl_backward_weight(dY, q[:-1].clone(), s)
    with pytest.raises(ValueError):
        bl.bl_backward_weight(dY, q, s, accumulate=True)
    with pytest.raises(TypeError):
        bl.bl_backward_weight(dY, q, s, dtype=torch.float16)
    with pytest.raises(ValueError):
        bl.bl_backward_weight(dY, q, s, out=torch.empty(N, K + 64, device="cuda"))
    with pytest.raises(ValueError):
        bl.bl_norm_forward(X, bl.BL_NORM_RMS, weight=torch.ones(K - 1, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(bl.BLError):
        bl.bl_norm_forward(X, 7)
    with pytest.raises(bl.BLError):
        bl.bl_norm_backward(X, X, bl.BL_NORM_LAYER, s)      # LayerNorm's mean is missing
    with pytest.raises(bl.BLError):
        bl.bl_forward_checkpoint(X, Wp, gamma, N, norm=bl.BL_NORM_RMS, eps=0.0)
    with pytest.raises(ValueError):
        bl.bl_norm_backward(X, X, bl.BL_NORM_RMS, s, weight=torch.ones(K, dtype=torch.bfloat16, device="cuda"),
                            accumulate=True)


# One shape for every tile width (32..256 rows of the output) with whole tiles,
# tiles in equal parts, and stages dealt out to the pairs, as the cost model
# chooses them.
REACH_INPUT = [(33, 64, 1003), (33, 64, 6001), (2500, 64, 33), (640, 64, 1500), (6000, 64, 33), (1030, 64, 2050),
               (640, 1088, 6001), (6000, 320, 33), (130, 2560, 6001), (520, 4160, 6001), (6000, 1088, 33),
               (2500, 64, 6001), (2049, 2112, 4100)]
REACH_WEIGHT = [(640, 64, 33), (6000, 64, 33), (33, 320, 6001), (2049, 64, 4100), (6000, 1088, 520),
                (260, 1088, 6001), (1500, 64, 6001), (6000, 1088, 1003), (770, 64, 33), (1500, 64, 4100),
                (4100, 2112, 520), (33, 4160, 3001), (2500, 64, 3001), (6000, 576, 2050)]


@pytest.mark.parametrize("M,K,N", REACH_INPUT)
def test_backward_input_tiles(M, K, N):
    _, Wp, gamma, C, _, _ = layer(M, K, N, 1)
    dY = grads(M, N, 2)
    dX = Guarded((M, K), torch.bfloat16)
    ws = Guarded((max(16, bl.bl_backward_input_workspace_bytes(M, K, N)),), torch.uint8)
    bl.bl_backward_input(dY, Wp, gamma, K, out=dX.t, workspace=ws.t)
    assert dX.intact() and ws.intact()
    check_dx(dX.t, dY, C, gamma)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,K,N", REACH_WEIGHT)
def test_backward_weight_tiles(M, K, N, dtype):
    *_, q, s = layer(M, K, N, 1)
    dY = grads(M, N, 2)
    flags = bl.BL_GRAD_BF16 if dtype == torch.bfloat16 else 0
    for acc in (False, True):
        dW = Guarded((N, K), dtype)
        base = None
        if acc:
            base = (torch.randn(N, K, generator=torch.Generator().manual_seed(3)) * 1e-2).to(dtype).cuda()
            dW.t.copy_(base)
        ws = Guarded((max(16, bl.bl_backward_weight_workspace_bytes(M, K, N, flags | acc)),), torch.uint8)
        bl.bl_backward_weight(dY, q, s, out=dW.t, accumulate=acc, workspace=ws.t)
        assert dW.intact() and ws.intact()
        check_dw(dW.t, dY, q, s, base=base)


def test_positive_products_over_many_tokens():
    # sums that only grow show what the accumulator truncates
    M, K, N = 16384, 64, 136
    q = torch.randint(1, 128, (M, K), generator=torch.Generator().manual_seed(1)).to(torch.int8).cuda()
    s = (torch.rand(M, generator=torch.Generator().manual_seed(2)) + 0.5).cuda()
    dY = grads(M, N, 3).abs()
    want = dY.to(F64).t() @ (q.to(F64) / s.to(F64)[:, None])
    got = bl.bl_backward_weight(dY, q, s)
    check_dw(got, dY, q, s)
    assert ((got.to(F64) - want).norm() / want.norm()).item() <= 2.0**-16


def test_norm_backward_captured_and_concurrent():
    """The backward with weight gradients in a graph, replayed on new contents;
    and two different calls at once on two streams with their own workspaces."""
    M, K = 300, 2560
    w = torch.randn(K).to(torch.bfloat16).cuda()
    X, dY = torch.randn(M, K).to(torch.bfloat16).cuda(), grads(M, K, 1)

    def both(x, dy):
        Y, mean, stat = bl.bl_norm_forward(x, bl.BL_NORM_LAYER, weight=w)
        return (Y, *bl.bl_norm_backward(dy, x, bl.BL_NORM_LAYER, stat, mean=mean, weight=w, need_bias=True))

    both(X, dY)
    x2, dy2 = X.clone(), dY.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both(x2, dy2)
    for seed in (5, 6):
        x2.copy_(torch.randn(M, K).to(torch.bfloat16))
        dy2.copy_(grads(M, K, seed))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, both(x2, dy2)))
    _, Wp, gamma, _, q, s = layer(200, 320, 1003, 1)
    dz = grads(200, 1003, 2)
    want = (both(X, dY), bl.bl_backward_weight(dz, q, s), bl.bl_backward_input(dz, Wp, gamma, 320))
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(a):
            r1 = both(X, dY)
            r3 = bl.bl_backward_input(dz, Wp, gamma, 320)
        with torch.cuda.stream(b):
            r2 = bl.bl_backward_weight(dz, q, s)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(r1, want[0]))
        assert torch.equal(r2, want[1]) and torch.equal(r3, want[2])


def test_one_tokens_training_step_and_reused_rows():
    # rows of a larger buffer (16-byte aligned rows are enough), the same buffer twice
    K, N = 192, 72
    _, Wp, gamma, C, _, _ = layer(4, K, N, 1)
    big = torch.randn(9, K).to(torch.bfloat16).cuda()
    for m in (0, 5, 8):
        X = big[m:m + 1]
        Y, q, s, stat = bl.bl_forward_checkpoint(X, Wp, gamma, N, norm=bl.BL_NORM_RMS)
        dY = grads(1, N, m)
        dXn = bl.bl_backward_input(dY, Wp, gamma, K)
        check_dx(dXn, dY, C, gamma)
        check_dw(bl.bl_backward_weight(dY, q, s), dY, q, s)
    # X as its own gradient: the same tensor as both arguments
    X = torch.randn(6, K).to(torch.bfloat16).cuda()
    _, _, stat = bl.bl_norm_forward(X, bl.BL_NORM_RMS)
    dX, _, _ = bl.bl_norm_backward(X, X, bl.BL_NORM_RMS, stat)
    x = X.to(F64)
    rs = (stat.to(F64) + EPS).rsqrt()[:, None]
    xh = x * rs
    want = (x - xh * (x * xh).mean(1, keepdim=True)) * rs
    terms = (x.abs() + xh.abs() * (x * xh).abs().mean(1, keepdim=True)) * rs
    assert worst(dX, want, 2.0**-8 * want.abs() + (fp32_err(K) + 2.0**-20) * terms) <= 1.0


@pytest.mark.parametrize("M,K", [(1, 64), (37, 2560), (40, 4160), (9, 8192), (11, 8256)])
def test_norm_weight_gradients_alone(M, K):
    # the C entry with dX not wanted, and each of dweight and dbias alone
    L = bl.lib()
    X, dY = torch.randn(M, K).to(torch.bfloat16).cuda(), grads(M, K, 1)
    w = torch.randn(K).to(torch.bfloat16).cuda()
    _, mean, stat = bl.bl_norm_forward(X, bl.BL_NORM_LAYER, weight=w)
    _, dw, db = bl.bl_norm_backward(dY, X, bl.BL_NORM_LAYER, stat, mean=mean, weight=w, need_bias=True)
    need = bl.bl_norm_backward_workspace_bytes(M, K)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    st = torch.cuda.current_stream().cuda_stream
    for want_w, want_b in ((1, 1), (1, 0), (0, 1)):
        gw, gb = Guarded((K,), torch.float32), Guarded((K,), torch.float32)
        assert L.bl_norm_backward(dY.data_ptr(), X.data_ptr(), w.data_ptr(), bl.BL_NORM_LAYER, EPS, mean.data_ptr(),
                                  stat.data_ptr(), M, K, 0, None, gw.t.data_ptr() if want_w else None,
                                  gb.t.data_ptr() if want_b else None, ws.data_ptr(), need, st) == 0
        assert gw.intact() and gb.intact()
        assert not want_w or torch.equal(gw.t, dw)
        assert not want_b or torch.equal(gb.t, db)


def test_widest_rows_and_offsets_past_32_bits():
    # K = 65536; outputs and inputs of more than 2^31 elements, checked at both ends
    K = 65536
    g = torch.Generator(device="cuda").manual_seed(0)
    M, N = 70, 33001
    q = torch.randint(-127, 128, (M, K), generator=g, device="cuda").to(torch.int8)
    s = torch.rand(M, generator=g, device="cuda") + 1
    dY = (torch.randn(M, N, generator=g, device="cuda") * 1e-3).to(torch.bfloat16)
    for dtype in (torch.float32, torch.bfloat16):
        out = torch.zeros(N, K, dtype=dtype, device="cuda")
        bl.bl_backward_weight(dY, q, s, out=out, accumulate=True)
        for a, b in ((0, 40), (N - 40, N)):
            check_dw(out[a:b], dY[:, a:b], q, s)
        del out
    del q, dY
    M, N = 33001, 24
    Wp = torch.randint(0, 256, (N, K // 4), generator=g, device="cuda").to(torch.uint8)
    Wp = torch.where((Wp & (Wp >> 1) & 0x55) != 0, Wp & 0x55, Wp)   # no field is 3
    gamma = torch.full((1,), 0.02, device="cuda")
    C = bl.bl_unpack_weights(Wp, N, K).to(F64)
    dY = (torch.randn(M, N, generator=g, device="cuda") * 1e-3).to(torch.bfloat16)
    dX = bl.bl_backward_input(dY, Wp, gamma, K)
    for a, b in ((0, 40), (M - 40, M)):
        check_dx(dX[a:b], dY[a:b], C, gamma)
    # the norm of those 33001 rows, forward and back
    Y, mean, stat = bl.bl_norm_forward(dX, bl.BL_NORM_LAYER)
    b = slice(M - 20, M)
    mu, var, d = norm_ref(dX[b], bl.BL_NORM_LAYER)
    e = fp32_err(K)
    mag = dX[b].to(F64).abs().mean(1)
    assert worst(stat[b], var, (e + 2.0**-20) * var + 2 * (e * mag).square()) <= 1.0
    dZ, _, db = bl.bl_norm_backward(Y, dX, bl.BL_NORM_LAYER, stat, mean=mean, need_bias=True, out=Y)
    assert dZ is Y and torch.isfinite(dZ[b].float()).all() and torch.isfinite(db).all()


@pytest.mark.parametrize("norm", [bl.BL_NORM_RMS, bl.BL_NORM_LAYER])
def test_a_step_behind_a_norm_with_parameters(norm):
    """Norm with weight (and bias), checkpointed linear, and back: the chain of
    calls, its norm part against 64 bits from the calls' own dXn."""
    M, K, N = 67, 320, 130
    g = torch.Generator().manual_seed(4)
    X = torch.randn(M, K, generator=g).to(torch.bfloat16).cuda()
    w = (1 + 0.2 * torch.randn(K, generator=g)).to(torch.bfloat16).cuda()
    la = norm == bl.BL_NORM_LAYER
    b = (0.2 * torch.randn(K, generator=g)).to(torch.bfloat16).cuda() if la else None
    _, Wp, gamma, C, _, _ = layer(4, K, N, 1)
    Xn, mean, stat = bl.bl_norm_forward(X, norm, weight=w, bias=b, eps=EPS)
    Y, q, s, _ = bl.bl_forward_checkpoint(Xn, Wp, gamma, N)
    assert torch.equal(Y, bl.bl_forward(Xn, Wp, gamma, N))
    dY = grads(M, N, 5)
    dXn = bl.bl_backward_input(dY, Wp, gamma, K)
    check_dx(dXn, dY, C, gamma)
    check_dw(bl.bl_backward_weight(dY, q, s), dY, q, s)
    dX, dw, db = bl.bl_norm_backward(dXn, X, norm, stat, mean=mean, weight=w, need_bias=la, eps=EPS)
    rs = (stat.to(F64) + EPS).rsqrt()[:, None]
    xh = (X.to(F64) - (mean.to(F64)[:, None] if la else 0.0)) * rs
    dy = dXn.to(F64)
    gg = dy * w.to(F64)
    want = (gg - xh * (gg * xh).mean(1, keepdim=True) - (gg.mean(1, keepdim=True) if la else 0.0)) * rs
    terms = (gg.abs() + xh.abs() * (gg * xh).abs().mean(1, keepdim=True) + gg.abs().mean(1, keepdim=True)) * rs
    assert worst(dX, want, 2.0**-8 * want.abs() + (fp32_err(K) + 2.0**-20) * terms + 1e-300) <= 1.0
    em = 2.0**-24 * (M + 16)
    assert worst(dw, (dy * xh).sum(0), em * (dy * xh).abs().sum(0) + 1e-300) <= 1.0
    assert (db is not None) == la and (db is None or worst(db, dy.sum(0), em * dy.abs().sum(0) + 1e-300) <= 1.0)


@pytest.mark.parametrize("M,K,N", [(1, 1024, 4096), (16, 2560, 6912), (192, 2048, 4100), (256, 2048, 8192),
                                   (260, 4160, 9001), (320, 8192, 8192), (256, 8192, 28672)])
def test_accumulating_over_many_tiles(M, K, N):
    # many tiles a pair with few stages each: the epilogue, with loads and stores
    # of the whole output, is what the others wait for
    g = torch.Generator(device="cuda").manual_seed(M)
    q = torch.randint(-127, 128, (M, K), generator=g, device="cuda").to(torch.int8)
    s = torch.rand(M, generator=g, device="cuda") + 1
    dY = (torch.randn(M, N, generator=g, device="cuda") * 1e-3).to(torch.bfloat16)
    for dtype in (torch.float32, torch.bfloat16):
        plain = bl.bl_backward_weight(dY, q, s, out=torch.empty(N, K, dtype=dtype, device="cuda"))
        base = (torch.randn(N, K, generator=g, device="cuda") * 1e-2).to(dtype)
        out = base.clone()
        bl.bl_backward_weight(dY, q, s, out=out, accumulate=True)
        for a in (0, N // 2, N - 24):
            b = slice(a, a + 24)
            check_dw(plain[b], dY[:, b], q, s)
            check_dw(out[b], dY[:, b], q, s, base=base[b])
        if dtype == torch.float32:   # one rounding, of the same sum
            assert torch.equal(out, base + plain)
        out.zero_()
        for _ in range(3):
            bl.bl_backward_weight(dY, q, s, out=out.zero_(), accumulate=True)
        assert torch.equal(out, plain)


@pytest.mark.parametrize("M,K,N", [(10240, 2048, 1280), (6200, 1088, 1400), (4500, 2112, 4100)])
def test_several_accumulators_a_tile(M, K, N):
    # sums longer than one accumulator takes, whole and in parts
    *_, q, s = layer(M, K, N, 1)
    dY = grads(M, N, 2)
    base = (torch.randn(N, K, generator=torch.Generator().manual_seed(3)) * 1e-2).cuda()
    for acc in (False, True):
        runs = []
        for _ in range(2):
            dW = Guarded((N, K), torch.float32)
            dW.t.copy_(base)
            bl.bl_backward_weight(dY, q, s, out=dW.t, accumulate=acc)
            assert dW.intact()
            runs.append(dW.t.clone())
        assert torch.equal(runs[0], runs[1])
        check_dw(runs[0], dY, q, s, base=base if acc else None)


def test_runs_repeat_bit_for_bit():
    # long rings of stages whose loads may land out of order; a stage expanded
    # from rows that are not its own shows in some runs only
    g = torch.Generator(device="cuda").manual_seed(5)
    for M, K, N in ((10240, 2048, 1280), (4500, 2112, 4100), (4096, 512, 2048)):
        q = torch.randint(-127, 128, (M, K), generator=g, device="cuda").to(torch.int8)
        s = torch.rand(M, generator=g, device="cuda") + 1
        dY = (torch.randn(M, N, generator=g, device="cuda") * 1e-3).to(torch.bfloat16)
        for dtype in (torch.float32, torch.bfloat16):
            first = bl.bl_backward_weight(dY, q, s, dtype)
            check_dw(first, dY, q, s)
            out = torch.empty_like(first)
            for _ in range(60):
                assert torch.equal(bl.bl_backward_weight(dY, q, s, out=out), first)
    for M, K, N in ((4096, 2048, 6912), (400, 2112, 9000), (128, 2560, 20000), (33, 1088, 20000), (17, 1088, 9000)):
        Wp = torch.randint(0, 256, (N, K // 4), generator=g, device="cuda").to(torch.uint8)
        Wp = torch.where((Wp & (Wp >> 1) & 0x55) != 0, Wp & 0x55, Wp)   # no field is 3
        gamma = torch.full((1,), 0.02, device="cuda")
        dY = (torch.randn(M, N, generator=g, device="cuda") * 1e-3).to(torch.bfloat16)
        first = bl.bl_backward_input(dY, Wp, gamma, K)
        check_dx(first, dY, bl.bl_unpack_weights(Wp, N, K).to(F64), gamma)
        out = torch.empty_like(first)
        for _ in range(60):
            assert torch.equal(bl.bl_backward_input(dY, Wp, gamma, K, out=out), first)


# a full wave of whole tiles and a few more, whose stages are dealt out: their first
# row of tiles is whole in part, the last tiles end past K and past the last row
REACH_REST = [(1030, 4160, 4100), (4100, 1088, 4100), (2049, 2112, 2050), (2500, 2112, 2050), (2500, 1088, 4100)]


@pytest.mark.parametrize("M,K,N", REACH_REST)
def test_tiles_behind_whole_waves(M, K, N):
    test_backward_input_tiles(M, K, N)
    test_backward_weight_tiles(M, K, N, torch.float32)
    test_backward_weight_tiles(M, K, N, torch.bfloat16)


@pytest.mark.parametrize("M,K,N", [(1, 64, 9), (70, 320, 130), (257, 1344, 1003), (4200, 192, 260)])
def test_values_that_are_not_finite_stay_in_their_rows(M, K, N):
    _, Wp, gamma, C, q, s = layer(M, K, N, 1)
    q[q == 0] = 1   # (Inf times a zero code is NaN; times any other it is not finite)
    dY = grads(M, N, 2)
    bad = dY.clone()
    ms, ns = sorted({0, M // 2, M - 1}), sorted({0, N // 2, N - 1})
    for i, (m, n) in enumerate(zip(ms, ns)):
        bad[m, n] = (float("nan"), float("inf"), float("-inf"))[i]
    ms, ns = ms[:len(ns)], ns[:len(ms)]
    rest = torch.ones(M, dtype=torch.bool, device="cuda")
    rest[ms] = False
    a, b = bl.bl_backward_input(dY, Wp, gamma, K), bl.bl_backward_input(bad, Wp, gamma, K)
    assert torch.equal(a[rest], b[rest]) and not torch.isfinite(b[ms].float()).any()
    rest = torch.ones(N, dtype=torch.bool, device="cuda")
    rest[ns] = False
    for dtype in (torch.float32, torch.bfloat16):
        a, b = bl.bl_backward_weight(dY, q, s, dtype), bl.bl_backward_weight(bad, q, s, dtype)
        assert torch.equal(a[rest], b[rest]) and not torch.isfinite(b[ns].float()).any()
