"""Out-features beyond what the kernels count in 32 bits are refused, by every entry
point that forms [M, N] outputs or takes base-3 rows.  (They used to be cut to their
low 32 bits: N = 2^32 + 8 computed 8 columns and returned BL_OK.)  Nothing is
launched: every call lacks a pointer besides."""

import ctypes

import pytest

from bitlinear_bl_forward_b200 import bl
from bitlinear_bl_forward_b200 import build as blbuild

OK, INVALID, SHAPE = 0, 1, 2
A = 0x10000
BIG = 1 << 40
LAST = 2**31 - 65537   # the largest N
WIDE = [LAST + 1, 2**31 - 1, 2**31 + 8, 2**32 + 8, 2**33 + 130]


@pytest.fixture(scope="module")
def L():
    blbuild.build()
    return bl.lib()


def problem(n):
    return (bl.BLLinear * 1)(bl.BLLinear(None, 1, 64, n, A, A, A))


# entry point -> the call with N = n and a null input
CALLS = {
    "bl_forward": lambda L, n: L.bl_forward(None, 1, 64, n, A, A, 8, A, A, BIG, None),
    "bl_forward_f32": lambda L, n: L.bl_forward_f32(None, 4, 64, n, A, A, 8, A, A, BIG, None),
    "bl_forward_noalloc": lambda L, n: L.bl_forward_noalloc(None, 4, 64, n, A, A, 8, A, None),
    "bl_forward_grouped": lambda L, n: L.bl_forward_grouped(1, problem(n), 8, A, BIG, None),
    "bl_forward_relu2": lambda L, n: L.bl_forward_relu2(None, A, 1, 64, n, A, A, 8, A, A, BIG, None),
    "bl_forward_ex": lambda L, n: L.bl_forward_ex(None, 1, 64, n, A, A, 8, 0, None, A, A, BIG, None),
    "bl_forward_rmsnorm": lambda L, n: L.bl_forward_rmsnorm(None, None, 1e-5, 1, 64, n, A, A, 8, A, A, BIG, None),
    "bl_forward_layernorm": lambda L, n: L.bl_forward_layernorm(None, 1e-5, 1, 64, n, A, A, 8, A, A, BIG, None),
    "bl_forward_norm_grouped": lambda L, n: L.bl_forward_norm_grouped(1, problem(n), 1, None, 1e-5, 8, A, BIG, None),
    "bl_forward_checkpoint": lambda L, n: L.bl_forward_checkpoint(None, 2, 0.0, 1, 64, n, A, A, 8, A, A, A, None, A,
                                                                  BIG, None),
    "bl_backward_input": lambda L, n: L.bl_backward_input(None, 1, 64, n, A, A, A, A, BIG, None),
    "bl_backward_weight": lambda L, n: L.bl_backward_weight(None, A, A, 1, 64, n, 0, A, A, BIG, None),
    "bl_matmul_i32": lambda L, n: L.bl_matmul_i32(None, 1, 64, n, A, A, A, BIG, None),
    "bl_quantize_weights_b3": lambda L, n: L.bl_quantize_weights_b3(None, n, 64, A, A, A, BIG, None),
    "bl_unpack_weights_b3": lambda L, n: L.bl_unpack_weights_b3(None, n, 64, A, None),
    "bl_forward_b3": lambda L, n: L.bl_forward_b3(None, 1, 64, n, A, A, 8, A, None),
    "bl_matmul_i32_b3": lambda L, n: L.bl_matmul_i32_b3(None, 1, 64, n, A, A, None),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_wide_outputs_are_refused(L, name):
    for n in WIDE:
        assert CALLS[name](L, n) == SHAPE, n
    # the last one that fits is looked at further: its input is missing
    assert CALLS[name](L, LAST) == INVALID


def test_workspace_queries_agree(L):
    for n in WIDE:
        p = problem(n)
        p[0].M = 300
        assert L.bl_forward_workspace_bytes(300, 64, n, 8) == 0
        assert L.bl_forward_checkpoint_workspace_bytes(300, 64, n, 8) == 0
        assert L.bl_forward_grouped_workspace_bytes(1, ctypes.byref(p), 8) == 0
        assert L.bl_forward_rmsnorm_workspace_bytes(300, 64, n, 8) == 0
        assert L.bl_matmul_i32_workspace_bytes(300, 64, n) == 0
        assert L.bl_backward_input_workspace_bytes(300, 64, n) == 0
    assert L.bl_forward_checkpoint_workspace_bytes(300, 64, LAST, 8) > 0


def test_the_checkpoints_forward_takes_what_its_backward_takes(L):
    # M*N of 2^40 and more
    assert L.bl_forward_checkpoint(None, 2, 0.0, 1 << 30, 64, 1 << 20, A, A, 8, A, A, A, None, A, BIG, None) == SHAPE
    assert L.bl_forward_checkpoint_workspace_bytes(1 << 30, 64, 1 << 20, 8) == 0


def test_packing_itself_counts_in_64_bits(L):
    # the 2-bit packer and its inverse go over N*K weights in a row: no limit but N*K
    assert L.bl_quantize_weights_workspace_bytes(2**32 + 8, 64) > 0
    assert L.bl_quantize_weights(None, 2**32 + 8, 64, A, A, A, BIG, None) == INVALID
    assert L.bl_unpack_weights(None, 2**32 + 8, 64, A, None) == INVALID
