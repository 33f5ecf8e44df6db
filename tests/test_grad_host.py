"""Host-side checks of the training entry points that need no GPU: sizes, and
argument validation (every call carries an invalid argument or no rows, so
nothing is launched; the pointers are fake)."""

import pytest
import torch

from bitlinear_bl_forward_b200 import bl
from bitlinear_bl_forward_b200 import build as blbuild

OK, INVALID, SHAPE, ALIGN, UNSUP, CUDA, TIMEOUT, WS = range(8)
A = 0x10000      # fake, 16-byte aligned
U = 0x10001      # fake, misaligned
BIG = 1 << 30


@pytest.fixture(scope="module")
def L():
    blbuild.build()
    return bl.lib()


def test_sizes(L):
    assert L.bl_forward_checkpoint_workspace_bytes(300, 256, 64, 8) >= 4 * 300
    assert L.bl_forward_checkpoint_workspace_bytes(300, 250, 64, 8) == 0
    assert L.bl_backward_input_workspace_bytes(4, 100, 8) == 0      # bad shapes
    assert L.bl_backward_weight_workspace_bytes(4, 64, 0, 0) == 0
    assert L.bl_norm_backward_workspace_bytes(0, 64) == 0
    assert L.bl_norm_backward_workspace_bytes(4, 60) == 0
    for M in (1, 3, 4096, 100000):
        for K in (64, 2560, 8192, 8256, 65536):
            assert L.bl_norm_backward_workspace_bytes(M, K) >= 8 * K
    # the whole range gives sizes without a device
    for M in (1, 2, 17, 128, 4096, 1 << 20):
        for N in (1, 7, 130, 28672):
            L.bl_backward_input_workspace_bytes(M, 8192, N)
            for f in (0, 1, 2, 3):
                L.bl_backward_weight_workspace_bytes(M, 8192, N, f)


@pytest.mark.parametrize("args,want", [
    # (X, norm, eps, M, K, N, Wp, gamma, bits, Y, Xq, scale, stat, ws, ws_bytes)
    ((A, 2, 1e-5, 4, 100, 8, A, A, 8, A, A, A, None, A, BIG), SHAPE),
    ((A, 2, 1e-5, -1, 64, 8, A, A, 8, A, A, A, None, A, BIG), SHAPE),
    ((A, 2, 1e-5, 4, 64, 8, A, A, 3, A, A, A, None, A, BIG), UNSUP),
    ((A, 3, 1e-5, 4, 64, 8, A, A, 8, A, A, A, A, A, BIG), UNSUP),
    ((A, -1, 1e-5, 4, 64, 8, A, A, 8, A, A, A, A, A, BIG), UNSUP),
    ((A, 0, 0.0, 4, 64, 8, A, A, 8, A, A, A, A, A, BIG), INVALID),
    ((A, 1, float("inf"), 4, 64, 8, A, A, 8, A, A, A, A, A, BIG), INVALID),
    ((A, 1, 1e-5, 4, 64, 8, A, A, 8, A, A, A, None, A, BIG), INVALID),     # the statistic is needed
    ((None, 2, 1e-5, 4, 64, 8, A, A, 8, A, A, A, None, A, BIG), INVALID),
    ((A, 2, 1e-5, 4, 64, 8, A, A, 8, A, None, A, None, A, BIG), INVALID),
    ((A, 2, 1e-5, 4, 64, 8, A, A, 8, A, A, None, None, A, BIG), INVALID),
    ((U, 2, 1e-5, 4, 64, 8, A, A, 8, A, A, A, None, A, BIG), ALIGN),
    ((A, 2, 1e-5, 4, 64, 8, A, A, 8, A, U, A, None, A, BIG), ALIGN),
    ((A, 2, 1e-5, 4, 64, 8, A, A, 8, A, A, U, None, A, BIG), ALIGN),
    ((A, 2, 1e-5, 4, 64, 8, A, A, 8, A, A, A, None, None, 0), WS),
    ((A, 2, 1e-5, 4, 64, 8, A, A, 8, A, A, A, None, A, 15), WS),
    ((A, 2, 1e-5, 4, 64, 8, A, A, 8, A, A, A, None, U, BIG), ALIGN),
    ((None, 2, 1e-5, 0, 64, 8, None, None, 8, None, None, None, None, None, 0), OK),
])
def test_forward_checkpoint_validation(L, args, want):
    assert L.bl_forward_checkpoint(*args, None) == want


@pytest.mark.parametrize("args,want", [
    # (dY, M, K, N, Wp, gamma, dX)
    ((A, 4, 100, 8, A, A, A), SHAPE),
    ((A, 4, 64, 0, A, A, A), SHAPE),
    ((A, -4, 64, 8, A, A, A), SHAPE),
    ((A, 1 << 30, 64, 1 << 20, A, A, A), SHAPE),      # M*N >= 2^40
    ((None, 4, 64, 8, A, A, A), INVALID),
    ((A, 4, 64, 8, None, A, A), INVALID),
    ((A, 4, 64, 8, A, None, A), INVALID),
    ((A, 4, 64, 8, A, A, None), INVALID),
    ((U, 4, 64, 8, A, A, A), ALIGN),
    ((A, 4, 64, 8, U, A, A), ALIGN),
    ((A, 4, 64, 8, A, U, A), ALIGN),
    ((A, 4, 64, 8, A, A, U), ALIGN),
    ((None, 0, 64, 8, None, None, None), OK),
])
def test_backward_input_validation(L, args, want):
    assert L.bl_backward_input(*args, A, BIG, None) == want


@pytest.mark.parametrize("args,want", [
    # (dY, Xq, scale, M, K, N, flags, dW)
    ((A, A, A, 4, 100, 8, 0, A), SHAPE),
    ((A, A, A, 4, 64, 0, 0, A), SHAPE),
    ((A, A, A, -1, 64, 8, 0, A), SHAPE),
    ((A, A, A, 4, 64, 8, 4, A), UNSUP),
    ((None, A, A, 4, 64, 8, 0, A), INVALID),
    ((A, None, A, 4, 64, 8, 0, A), INVALID),
    ((A, A, None, 4, 64, 8, 0, A), INVALID),
    ((A, A, A, 4, 64, 8, 0, None), INVALID),
    ((None, None, None, 0, 64, 8, 0, None), INVALID),  # no tokens still writes zeros
    ((None, None, None, 0, 64, 8, 1, A), OK),          # ... unless they are added
    ((U, A, A, 4, 64, 8, 0, A), ALIGN),
    ((A, U, A, 4, 64, 8, 0, A), ALIGN),
    ((A, A, U, 4, 64, 8, 0, A), ALIGN),
    ((A, A, A, 4, 64, 8, 0, U), ALIGN),
])
def test_backward_weight_validation(L, args, want):
    assert L.bl_backward_weight(*args, A, BIG, None) == want


def test_workspace_validation(L):
    # a row of dY that is not a multiple of 16 bytes needs a padded copy
    for M, K, N in ((5, 64, 130), (300, 128, 1003)):
        need = L.bl_backward_input_workspace_bytes(M, K, N)
        if need:
            assert L.bl_backward_input(A, M, K, N, A, A, A, None, 0, None) == WS
            assert L.bl_backward_input(A, M, K, N, A, A, A, A, need - 1, None) == WS
            assert L.bl_backward_input(A, M, K, N, A, A, A, U, need, None) == ALIGN
        need = L.bl_backward_weight_workspace_bytes(M, K, N, 0)
        if need:
            assert L.bl_backward_weight(A, A, A, M, K, N, 0, A, None, 0, None) == WS
            assert L.bl_backward_weight(A, A, A, M, K, N, 0, A, A, need - 1, None) == WS
            assert L.bl_backward_weight(A, A, A, M, K, N, 0, A, U, need, None) == ALIGN


@pytest.mark.parametrize("args,want", [
    # (X, weight, bias, norm, eps, M, K, Y, mean, stat)
    ((A, A, A, 1, 1e-5, 4, 60, A, A, A), SHAPE),
    ((A, A, A, 1, 1e-5, 4, 131072, A, A, A), SHAPE),
    ((A, A, A, 1, 1e-5, -1, 64, A, A, A), SHAPE),
    ((A, A, A, 2, 1e-5, 4, 64, A, A, A), UNSUP),
    ((A, A, A, 1, 0.0, 4, 64, A, A, A), INVALID),
    ((A, A, A, 1, float("nan"), 4, 64, A, A, A), INVALID),
    ((A, A, A, 0, 1e-5, 4, 64, A, A, A), INVALID),      # RMSNorm has no mean
    ((None, A, A, 1, 1e-5, 4, 64, A, A, A), INVALID),
    ((A, A, A, 1, 1e-5, 4, 64, None, A, A), INVALID),
    ((U, A, A, 1, 1e-5, 4, 64, A, A, A), ALIGN),
    ((A, U, A, 1, 1e-5, 4, 64, A, A, A), ALIGN),
    ((A, A, U, 1, 1e-5, 4, 64, A, A, A), ALIGN),
    ((A, A, A, 1, 1e-5, 4, 64, U, A, A), ALIGN),
    ((A, A, A, 1, 1e-5, 4, 64, A, U, A), ALIGN),
    ((A, A, A, 1, 1e-5, 4, 64, A, A, U), ALIGN),
    ((None, None, None, 1, 1e-5, 0, 64, None, None, None), OK),
])
def test_norm_forward_validation(L, args, want):
    assert L.bl_norm_forward(*args, None) == want


@pytest.mark.parametrize("args,want", [
    # (dY, X, weight, norm, eps, mean, stat, M, K, flags, dX, dweight, dbias, ws, ws_bytes)
    ((A, A, A, 1, 1e-5, A, A, 4, 60, 0, A, A, A, A, BIG), SHAPE),
    ((A, A, A, 2, 1e-5, A, A, 4, 64, 0, A, A, A, A, BIG), UNSUP),
    ((A, A, A, 1, 1e-5, A, A, 4, 64, 2, A, A, A, A, BIG), UNSUP),
    ((A, A, A, 1, -1.0, A, A, 4, 64, 0, A, A, A, A, BIG), INVALID),
    ((A, A, A, 0, 1e-5, A, A, 4, 64, 0, A, A, A, A, BIG), INVALID),
    ((A, A, A, 1, 1e-5, None, A, 4, 64, 0, A, A, A, A, BIG), INVALID),
    ((A, A, A, 1, 1e-5, A, None, 4, 64, 0, A, A, A, A, BIG), INVALID),
    ((None, A, A, 1, 1e-5, A, A, 4, 64, 0, A, A, A, A, BIG), INVALID),
    ((A, None, A, 1, 1e-5, A, A, 4, 64, 0, A, A, A, A, BIG), INVALID),
    ((A, A, A, 1, 1e-5, A, A, 4, 64, 0, None, None, None, A, BIG), INVALID),   # nothing wanted
    ((U, A, A, 1, 1e-5, A, A, 4, 64, 0, A, A, A, A, BIG), ALIGN),
    ((A, U, A, 1, 1e-5, A, A, 4, 64, 0, A, A, A, A, BIG), ALIGN),
    ((A, A, U, 1, 1e-5, A, A, 4, 64, 0, A, A, A, A, BIG), ALIGN),
    ((A, A, A, 1, 1e-5, A, A, 4, 64, 0, U, A, A, A, BIG), ALIGN),
    ((A, A, A, 1, 1e-5, A, A, 4, 64, 0, A, U, A, A, BIG), ALIGN),
    ((A, A, A, 1, 1e-5, A, A, 4, 64, 0, A, A, U, A, BIG), ALIGN),
    ((A, A, A, 1, 1e-5, A, A, 4, 64, 0, A, A, A, None, 0), WS),
    ((A, A, A, 1, 1e-5, A, A, 4, 64, 0, A, A, A, A, 64), WS),
    ((None, None, None, 1, 1e-5, None, None, 0, 64, 1, A, A, A, None, 0), OK),
])
def test_norm_backward_validation(L, args, want):
    assert L.bl_norm_backward(*args, None) == want


@pytest.mark.parametrize("args,want", [
    # (dXn, Xq, scale, norm, eps, stat, M, K, dX)
    ((A, A, A, 1, 1e-5, A, 4, 60, A), SHAPE),
    ((A, A, A, 2, 1e-5, A, 4, 64, A), UNSUP),
    ((A, A, A, 1, 0.0, A, 4, 64, A), INVALID),
    ((None, A, A, 1, 1e-5, A, 4, 64, A), INVALID),
    ((A, None, A, 1, 1e-5, A, 4, 64, A), INVALID),
    ((A, A, None, 1, 1e-5, A, 4, 64, A), INVALID),
    ((A, A, A, 1, 1e-5, None, 4, 64, A), INVALID),
    ((A, A, A, 1, 1e-5, A, 4, 64, None), INVALID),
    ((U, A, A, 1, 1e-5, A, 4, 64, A), ALIGN),
    ((A, U, A, 1, 1e-5, A, 4, 64, A), ALIGN),
    ((A, A, U, 1, 1e-5, A, 4, 64, A), ALIGN),
    ((A, A, A, 1, 1e-5, U, 4, 64, A), ALIGN),
    ((None, None, None, 1, 1e-5, None, 0, 64, None), OK),
])
def test_norm_backward_checkpoint_validation(L, args, want):
    assert L.bl_norm_backward_checkpoint(*args, None) == want


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.zeros(8, 16, dtype=torch.uint8)
    g = torch.ones(1)
    q = torch.zeros(4, 64, dtype=torch.int8)
    with pytest.raises(TypeError):
        bl.bl_forward_checkpoint(x, w, g, 8)
    with pytest.raises(TypeError):
        bl.bl_backward_input(x, w, g, 64)
    with pytest.raises(TypeError):
        bl.bl_backward_weight(x, q, g)
    with pytest.raises(TypeError):
        bl.bl_norm_forward(x, bl.BL_NORM_RMS)
    with pytest.raises(TypeError):
        bl.bl_norm_backward(x, x, bl.BL_NORM_RMS, g)
    with pytest.raises(TypeError):
        bl.bl_norm_backward_checkpoint(x, q, g, bl.BL_NORM_RMS, g)
    with pytest.raises(TypeError):
        bl.bl_norm_forward(torch.zeros(64), bl.BL_NORM_RMS)


def test_overlaps_are_refused(L):
    B = 0x1000000
    # dX over dY or the weights; dW over dY or the codes
    assert L.bl_backward_input(B, 4, 64, 64, A, A, B, A, BIG, None) == INVALID
    assert L.bl_backward_input(B, 4, 64, 64, A, A, B + 4 * 64 * 2 - 16, A, BIG, None) == INVALID
    assert L.bl_backward_input(A, 4, 64, 64, B, A, B - 16, A, BIG, None) == INVALID
    assert L.bl_backward_weight(B, A, A, 4, 64, 8, 0, B + 16, A, BIG, None) == INVALID
    assert L.bl_backward_weight(A, B, A, 4, 64, 8, 2, B - 8 * 64 * 2 + 16, A, BIG, None) == INVALID
    # a norm's rows in place only as a whole
    assert L.bl_norm_forward(B, None, None, 1, 1e-5, 4, 64, B + 128, None, None, None) == INVALID
    assert L.bl_norm_backward(B, A, None, 0, 1e-5, None, A, 4, 64, 0, B + 16, None, None, None, 0, None) == INVALID
    assert L.bl_norm_backward(A, B, None, 0, 1e-5, None, A, 4, 64, 0, B - 16, None, None, None, 0, None) == INVALID
    assert L.bl_norm_backward(A, B, None, 0, 1e-5, None, A, 4, 64, 0, None, B, B, A, BIG, None) == INVALID
    assert L.bl_norm_backward_checkpoint(B, A, A, 1, 1e-5, A, 4, 64, B + 16, None) == INVALID
    assert L.bl_norm_backward_checkpoint(A, B, A, 1, 1e-5, A, 4, 64, B, None) == INVALID
    # the checkpoint's outputs over its input or over one another
    for Y, q in ((B, A), (A, B + 16), (B + 4096, B + 4112)):
        assert L.bl_forward_checkpoint(B, 2, 1e-5, 4, 64, 8, A, A, 8, Y, q, A, None, A, BIG, None) == INVALID
