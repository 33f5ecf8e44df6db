"""The gradients in the norm, and one token (or one output row) at a time at the ends
of stages, parts, accumulators and tiles: what an element's tolerance over a long sum
cannot show (grad_norms.py derives the bounds)."""

import pytest
import torch

from bitlinear_bl_forward_b200 import bl
from tests.grad_norms import F64, dw_bound, dx_bound, even_grads, rel_norm
from tests.test_gpu_grad import REACH_INPUT, REACH_REST, REACH_WEIGHT, layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    bl.bl_device_status(clear=True)
    yield
    assert bl.bl_device_status(clear=True) == (0, 0)


LONG = [(10240, 2048, 1280), (6200, 1088, 1400), (4096, 512, 2048), (4097, 2560, 264)]


@pytest.mark.parametrize("M,K,N", [s for s in REACH_WEIGHT + REACH_REST + LONG if s[0] >= 260])
def test_weight_gradient(M, K, N):
    *_, q, s = layer(M, K, N, 1)
    dY = even_grads(M, N, 2, "cuda")
    want = dY.to(F64).t() @ (q.to(F64) / s.to(F64)[:, None])
    for dtype in (torch.float32, torch.bfloat16):
        got = bl.bl_backward_weight(dY, q, s, dtype=dtype)
        assert rel_norm(got, want) <= dw_bound(dtype, M)


@pytest.mark.parametrize("M,K,N", [s for s in REACH_INPUT + REACH_REST + [(400, 2112, 9000), (128, 2560, 20000),
                                                                          (33, 1088, 20000), (17, 1088, 9000)]])
def test_input_gradient(M, K, N):
    _, Wp, gamma, C, _, _ = layer(M, K, N, 1)
    dY = even_grads(M, N, 2, "cuda")
    want = dY.to(F64) @ C * gamma.to(F64)
    assert rel_norm(bl.bl_backward_input(dY, Wp, gamma, K), want) <= dx_bound(N)


def ends(length, stage, per):
    """Indices around the ends of stages, parts and accumulators of a sum."""
    at = {0, length - 1, length // 2}
    for edge in (stage, 2 * stage, per * stage, 2 * per * stage, 2048, 4096, length // stage * stage):
        at |= {edge - 1, edge}
    return sorted(i for i in at if 0 <= i < length)


@pytest.mark.parametrize("M,K,N", [(6200, 1088, 1400), (2500, 2112, 2050), (1500, 64, 6001), (300, 2560, 264),
                                   (6000, 64, 33)])
def test_weight_gradient_one_token_at_a_time(M, K, N):
    # all other rows of dY are zero: an element is one product
    *_, q, s = layer(M, K, N, 1)
    full = even_grads(M, N, 3, "cuda")
    for dtype, flags, step in ((torch.float32, 0, 2.0**-16 + 2.0**-22), (torch.bfloat16, 2, 2.0**-7 + 2.0**-16)):
        plan = bl.bl_gradient_plan(True, M, K, N, flags)
        for m in ends(M, 64, plan[4]):
            dY = torch.zeros_like(full)
            dY[m] = full[m]
            want = dY[m].to(F64)[:, None] * (q[m].to(F64) / s[m].to(F64))[None, :]
            err = (bl.bl_backward_weight(dY, q, s, dtype=dtype).to(F64) - want).abs()
            assert bool((err <= step * want.abs()).all()), (dtype, m)


@pytest.mark.parametrize("M,K,N", [(130, 2560, 6001), (33, 64, 6001), (2049, 2112, 4100), (640, 1088, 6001),
                                   (17, 1088, 9000)])
def test_input_gradient_one_output_row_at_a_time(M, K, N):
    # all other columns of dY are zero: an element is one product
    _, Wp, gamma, C, _, _ = layer(M, K, N, 1)
    full = even_grads(M, N, 3, "cuda")
    plan = bl.bl_gradient_plan(False, M, K, N)
    stage = 128 if plan[0] <= 128 else 64
    assert plan[3] == -(-N // stage)
    for n in ends(N, stage, plan[4]):
        dY = torch.zeros_like(full)
        dY[:, n] = full[:, n]
        want = dY[:, n].to(F64)[:, None] * C[n][None, :] * gamma.to(F64)
        err = (bl.bl_backward_input(dY, Wp, gamma, K).to(F64) - want).abs()
        assert bool((err <= (2.0**-8 + 2.0**-22) * want.abs()).all()), n
