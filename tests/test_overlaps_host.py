"""Training calls whose outputs or workspace share a byte with an input, or with one
another, are refused; the rows that a norm takes in place and ranges that only touch
are not.  Fake pointers, no GPU: a call that is not refused ends with a CUDA error."""

import itertools

import pytest
import torch

from bitlinear_bl_forward_b200 import bl
from bitlinear_bl_forward_b200 import build as blbuild

INVALID, CUDA = 1, 5
M, K, N = 300, 128, 1003   # N off 16 bytes: the gradients take a workspace

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="fake pointers: only where nothing can be launched")


@pytest.fixture(scope="module")
def L():
    blbuild.build()
    return bl.lib()


def up(n):
    return (n + 255) // 256 * 256


def calls(L):
    """name -> (call of {argument: pointer}, {argument: bytes} of the outputs, the
    same of the inputs, pairs that may be exactly the same range)"""
    rows, codes, col, vec = 2 * M * K, M * K, 4 * M, 2 * K
    ws_i = L.bl_backward_input_workspace_bytes(M, K, N)
    ws_w = L.bl_backward_weight_workspace_bytes(M, K, N, 0)
    ws_b = L.bl_backward_weight_workspace_bytes(M, K, N, 2)
    ws_n = L.bl_norm_backward_workspace_bytes(M, K)
    ws_c = L.bl_forward_checkpoint_workspace_bytes(M, K, N, 8)
    assert min(ws_i, ws_w, ws_b, ws_n, ws_c) > 0
    c = {}
    for norm, tag in ((2, "plain"), (1, "norm")):
        out = {"Y": 2 * M * N, "Xq": codes, "scale": col, "ws": ws_c}
        if norm == 1:
            out["stat"] = col
        c[f"forward_checkpoint_{tag}"] = (
            lambda a, norm=norm: L.bl_forward_checkpoint(a["X"], norm, 1e-5, M, K, N, a["Wp"], a["gamma"], 8, a["Y"],
                                                         a["Xq"], a["scale"], a.get("stat"), a["ws"], ws_c, None),
            out, {"X": rows, "Wp": N * K // 4, "gamma": 4}, ())
    c["backward_input"] = (
        lambda a: L.bl_backward_input(a["dY"], M, K, N, a["Wp"], a["gamma"], a["dX"], a["ws"], ws_i, None),
        {"dX": rows, "ws": ws_i}, {"dY": 2 * M * N, "Wp": N * K // 4, "gamma": 4}, ())
    for flags, size, ws, tag in ((0, 4, ws_w, "fp32"), (3, 2, ws_b, "bf16")):
        c[f"backward_weight_{tag}"] = (
            lambda a, flags=flags, ws=ws: L.bl_backward_weight(a["dY"], a["Xq"], a["scale"], M, K, N, flags, a["dW"],
                                                               a["ws"], ws, None),
            {"dW": size * N * K, "ws": ws}, {"dY": 2 * M * N, "Xq": codes, "scale": col}, ())
    c["norm_forward"] = (
        lambda a: L.bl_norm_forward(a["X"], a["weight"], a["bias"], 1, 1e-5, M, K, a["Y"], a["mean"], a["stat"], None),
        {"Y": rows, "mean": col, "stat": col}, {"X": rows, "weight": vec, "bias": vec}, (("Y", "X"),))
    c["norm_backward"] = (
        lambda a: L.bl_norm_backward(a["dY"], a["X"], a["weight"], 1, 1e-5, a["mean"], a["stat"], M, K, 1, a["dX"],
                                     a["dweight"], a["dbias"], a["ws"], ws_n, None),
        {"dX": rows, "dweight": 4 * K, "dbias": 4 * K, "ws": ws_n},
        {"dY": rows, "X": rows, "weight": vec, "mean": col, "stat": col}, (("dX", "dY"), ("dX", "X")))
    c["norm_backward_checkpoint"] = (
        lambda a: L.bl_norm_backward_checkpoint(a["dXn"], a["Xq"], a["scale"], 1, 1e-5, a["stat"], M, K, a["dX"], None),
        {"dX": rows}, {"dXn": rows, "Xq": codes, "scale": col, "stat": col}, (("dX", "dXn"),))
    return c


NAMES = ["forward_checkpoint_plain", "forward_checkpoint_norm", "backward_input", "backward_weight_fp32",
         "backward_weight_bf16", "norm_forward", "norm_backward", "norm_backward_checkpoint"]


def spread(sizes):
    return {name: (i + 1) << 32 for i, name in enumerate(sizes)}


@pytest.mark.parametrize("name", NAMES)
def test_overlapping_outputs_are_refused(L, name):
    call, out, inp, in_place = calls(L)[name]
    sizes = {**out, **inp}
    assert call(spread(sizes)) == CUDA   # apart: not refused
    for o, other in itertools.chain(itertools.product(out, inp), itertools.combinations(out, 2)):
        at = spread(sizes)
        base = at[other]
        # the output begins with the other range, holds its last bytes, or ends in it
        starts = [base, base + (sizes[other] - 1) // 16 * 16, base - (sizes[o] - 1) // 16 * 16]
        for start in starts:
            at[o] = start
            want = CUDA if (o, other) in in_place and start == base else INVALID
            assert call(at) == want, (o, other, start - base)


@pytest.mark.parametrize("name", NAMES)
def test_ranges_that_touch_are_not_refused(L, name):
    call, out, inp, _ = calls(L)[name]
    at, p = {}, 1 << 32
    for arg, size in {**out, **inp}.items():
        at[arg] = p
        p += (size + 15) // 16 * 16
    assert call(at) == CUDA


def test_inputs_may_share_bytes(L):
    # a norm's rows as their own gradient; one buffer for the weight and the bias
    call, out, inp, _ = calls(L)["norm_backward"]
    at = spread({**out, **inp})
    at["dY"] = at["X"]
    assert call(at) == CUDA
    call, out, inp, _ = calls(L)["norm_forward"]
    at = spread({**out, **inp})
    at["bias"] = at["weight"]
    assert call(at) == CUDA


def test_a_workspace_that_is_not_needed_may_be_anywhere(L):
    # 8 columns: rows of dY on 16 bytes, one tile; no byte of the workspace is used
    assert L.bl_backward_input_workspace_bytes(4, 64, 8) == 0
    dY, Wp, gamma, dX = ((i + 1) << 32 for i in range(4))
    for ws in (dY + 16, Wp, dX + 32, None):
        assert L.bl_backward_input(dY, 4, 64, 8, Wp, gamma, dX, ws, 1 << 20, None) == CUDA
    # nor without weight gradients
    assert L.bl_norm_backward(dY, Wp, None, 0, 1e-5, None, gamma, 4, 64, 0, dX, None, None, dY + 16, 1 << 20,
                              None) == CUDA
