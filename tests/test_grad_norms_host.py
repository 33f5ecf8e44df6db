"""The norm bounds of the gradients' tests, on the CPU: roundings as the kernels make
them keep to the bound, and a token left out, or taken twice, does not."""

import pytest
import torch

from tests.grad_norms import F64, dw_bound, dx_bound, even_grads, rel_norm


def codes(M, K, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=g)
    s = 127 / x.abs().amax(1)
    return torch.round(x * s[:, None]).to(torch.int8), s


@pytest.mark.parametrize("M", [260, 2049, 4100, 10240])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_weight_gradient(M, dtype):
    K, N = 64, 40
    q, s = codes(M, K, M)
    dY = even_grads(M, N, 1)
    want = dY.to(F64).t() @ (q.to(F64) / s.to(F64)[:, None])
    x = q.float() / s[:, None]
    hi = x.to(torch.bfloat16).to(F64)
    operand = hi if dtype == torch.bfloat16 else hi + (x.to(F64) - hi).to(torch.bfloat16).to(F64)

    def run(rows):
        return (dY.to(F64)[rows].t() @ operand[rows]).to(dtype)

    every = torch.arange(M)
    assert rel_norm(run(every), want) <= dw_bound(dtype, M)
    for m in (0, 63, 64, M // 2, M - 1):
        assert rel_norm(run(every[every != m]), want) > 2 * dw_bound(dtype, M)
        assert rel_norm(run(torch.cat([every, every[m:m + 1]])), want) > 2 * dw_bound(dtype, M)


@pytest.mark.parametrize("N", [260, 2050, 9001, 20000])
def test_input_gradient(N):
    M, K = 24, 64
    g = torch.Generator().manual_seed(N)
    C = torch.randint(-1, 2, (N, K), generator=g).to(F64)
    dY = even_grads(M, N, 2).to(F64)
    want = dY @ C
    assert rel_norm(want.to(torch.bfloat16), want) <= dx_bound(N)
    for n in (0, 127, 128, N // 2, N - 1):
        lost = want - dY[:, n:n + 1] @ C[n:n + 1]
        twice = want + dY[:, n:n + 1] @ C[n:n + 1]
        assert rel_norm(lost.to(torch.bfloat16), want) > 2 * dx_bound(N)
        assert rel_norm(twice.to(torch.bfloat16), want) > 2 * dx_bound(N)
