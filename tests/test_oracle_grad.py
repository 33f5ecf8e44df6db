"""Pins for the oracle's gradients: hand-worked values, float64 autograd of the
straight-through forward, and central differences; and the CUDA library's
training step against the oracle."""

import numpy as np
import pytest
import torch

from oracle import bitlinear_oracle as o


def test_grads_by_hand():
    # two tokens, two outputs, three inputs; gamma = 1/2
    codes = np.array([[1, 0, -1], [-1, 1, 0]])
    dy = np.array([[2.0, 4.0], [-1.0, 3.0]])
    assert np.array_equal(o.grad_input(dy, codes, np.float32(0.5)), [[-1.0, 2.0, -1.0], [-2.0, 1.5, 0.5]])
    q = np.array([[10, -20, 0], [4, 8, 127]])
    s = np.array([10.0, 4.0])
    # x^ = [[1, -2, 0], [1, 2, 31.75]]
    assert np.array_equal(o.grad_weight(dy, q, s), [[1.0, -6.0, -31.75], [7.0, -2.0, 95.25]])


def test_norm_by_hand():
    # a row (3, -1): mean 1, deviations (2, -2), variance 4; eps = 0
    y, mean, stat = o.norm_plain([[3.0, -1.0]], True, weight=[2.0, 3.0], bias=[0.5, 0.0], eps=0.0)
    assert mean[0] == 1 and stat[0] == 4 and np.array_equal(y, [[2.5, -3.0]])
    # RMSNorm of (1, 7): mean of squares 25
    y, mean, stat = o.norm_plain([[1.0, 7.0]], False, eps=0.0)
    assert mean is None and stat[0] == 25 and np.allclose(y, [[0.2, 1.4]], rtol=1e-15, atol=0)
    # two elements leave LayerNorm no freedom: its gradient vanishes
    dx, dw, db = o.norm_grad([[5.0, 1.0]], [[1.0, -1.0]], [4.0], True, eps=0.0)
    assert np.array_equal(dx, [[0.0, 0.0]]) and np.array_equal(dw, [5.0, -1.0]) and np.array_equal(db, [5.0, 1.0])


def test_straight_through_autograd():
    """x + (x^ - x).detach() and w + (w^ - w).detach() in float64 autograd."""
    rng = np.random.default_rng(0)
    M, K, N = 7, 64, 10
    x = rng.standard_normal((M, K)).astype(np.float32)
    xb = o.round_to_bf16_bits(x)
    W = (rng.standard_normal((N, K)) * 0.02).astype(np.float32)
    gamma = o.absmean_scale(W)
    codes = o.ternary_codes(W, gamma)
    q, s = o.act_quant(xb, 8)[:2]
    X = torch.tensor(o.bf16_bits_to_f32(xb).astype(np.float64), requires_grad=True)
    L = torch.tensor(W.astype(np.float64), requires_grad=True)
    xh = torch.tensor(q.astype(np.float64) / s.astype(np.float64)[:, None])
    wh = torch.tensor(codes.astype(np.float64) * float(gamma))
    y = (X + (xh - X).detach()) @ (L + (wh - L).detach()).t()
    dy = torch.tensor(rng.standard_normal((M, N)))
    y.backward(dy)
    assert np.allclose(o.grad_input(dy.numpy(), codes, gamma), X.grad.numpy(), rtol=1e-12, atol=1e-15)
    assert np.allclose(o.grad_weight(dy.numpy(), q, s), L.grad.numpy(), rtol=1e-12, atol=1e-15)


@pytest.mark.parametrize("layer", [False, True])
def test_norm_autograd_and_differences(layer):
    rng = np.random.default_rng(1)
    M, K, eps = 5, 12, 1e-5
    x = torch.tensor(rng.standard_normal((M, K)) + 0.3, requires_grad=True)
    w = torch.tensor(rng.standard_normal(K), requires_grad=True)
    b = torch.tensor(rng.standard_normal(K), requires_grad=True)
    dy = rng.standard_normal((M, K))
    if layer:
        y = torch.nn.functional.layer_norm(x, (K,), w, b, eps)
    else:
        y = x * (x.square().mean(1, keepdim=True) + eps).rsqrt() * w + b
    y.backward(torch.tensor(dy))
    xn, wn, bn = x.detach().numpy(), w.detach().numpy(), b.detach().numpy()
    got, mean, stat = o.norm_plain(xn, layer, wn, bn, eps)
    assert np.allclose(got, y.detach().numpy(), rtol=1e-12, atol=1e-14)
    xh = (xn - mean[:, None] if layer else xn) / np.sqrt(stat + eps)[:, None]
    dx, dw, db = o.norm_grad(dy, xh, stat, layer, wn, eps)
    assert np.allclose(dx, x.grad.numpy(), rtol=1e-11, atol=1e-13)
    assert np.allclose(dw, w.grad.numpy(), rtol=1e-11, atol=1e-13)
    assert np.allclose(db, b.grad.numpy(), rtol=1e-11, atol=1e-13)
    u, h = rng.standard_normal((M, K)), 1e-6
    f = lambda t: (o.norm_plain(t, layer, wn, bn, eps)[0] * dy).sum()  # noqa: E731
    assert abs((f(xn + h * u) - f(xn - h * u)) / (2 * h) - (dx * u).sum()) < 1e-7


@pytest.mark.gpu
@pytest.mark.parametrize("norm", [None, 0, 1])
@pytest.mark.parametrize("M,K,N", [(1, 64, 24), (33, 320, 130), (140, 256, 72)])
def test_library_step_against_the_oracle(M, K, N, norm):
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from bitlinear_bl_forward_b200 import bl
    from bitlinear_bl_forward_b200.inputs import random_case
    from tests.gpu_helpers import x_to_dev

    xb, W = random_case(M, K, N, seed=M)
    rng = np.random.default_rng(M)
    dyb = o.round_to_bf16_bits((rng.standard_normal((M, N)) * 1e-2).astype(np.float32))
    dy = o.bf16_bits_to_f32(dyb).astype(np.float64)
    Wp, gd = bl.bl_quantize_weights(torch.from_numpy(W).cuda())
    gamma = o.absmean_scale(W)
    codes = o.ternary_codes(W, gamma)
    Y, q, s, stat = bl.bl_forward_checkpoint(x_to_dev(xb), Wp, gd, N, norm=norm)
    dXn = bl.bl_backward_input(x_to_dev(dyb), Wp, gd, K)
    dW = bl.bl_backward_weight(x_to_dev(dyb), q, s)
    q, s = q.cpu().numpy(), s.cpu().numpy()
    if norm is None:
        q0, s0 = o.act_quant(xb, 8)[:2]
        assert np.array_equal(q, q0) and np.array_equal(s, s0)
    want = o.grad_input(dy, codes, gamma)
    P = np.abs(dy) @ np.abs(codes.astype(np.float64)) * float(gamma)
    # the bf16 output's half step, and fp32 sums of N products (two steps per 16)
    tol = 2.0**-8 * np.abs(want) + 2.0**-22 * (N / 16 + 4) * P + 1e-300
    dx = dXn.float().cpu().numpy().astype(np.float64)
    assert (np.abs(dx - want) <= tol).all()
    want = o.grad_weight(dy, q, s)
    P = np.abs(dy).T @ np.abs(q.astype(np.float64) / s.astype(np.float64)[:, None])
    # q / s as two bf16 (2^-16), twice as many steps
    tol = (2.0**-16 + 2.0**-22 * (M / 8 + 4)) * P + 2.0**-23 * np.abs(want) + 1e-300
    assert (np.abs(dW.cpu().numpy() - want) <= tol).all()
    if norm is not None:
        dX = bl.bl_norm_backward_checkpoint(dXn, torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda(), norm, stat)
        st = stat.cpu().numpy().astype(np.float64)
        xh = q.astype(np.float64) / s.astype(np.float64)[:, None]
        want, _, _ = o.norm_grad(dx, xh, st, norm == 1)
        terms = (np.abs(dx) + np.abs(xh) * np.abs(dx * xh).mean(1, keepdims=True)
                 + np.abs(dx).mean(1, keepdims=True)) / np.sqrt(st + 1e-5)[:, None]
        tol = 2.0**-8 * np.abs(want) + (2.0**-24 * (K / 32 + 16) + 2.0**-20) * terms + 1e-300
        assert (np.abs(dX.float().cpu().numpy() - want) <= tol).all()
