"""Stacks that are worked off in chunks. 83 matrices of 2048 x 2112 take 51.1 MB of workspace each (6 bytes per
padded element of X and of A), 4.2 GB together, twice the 2 GiB that the workspace may fill: chunks of 28, 28 and 27."""
import pytest
import torch

import sparse_moe_layer_biased_b200 as moe
from sparse_moe_layer_biased_b200 import _abi
from test_gpu_orthogonalize import check, gauss, reference

pytestmark = pytest.mark.gpu
N, ROWS, COLS = 83, 2048, 2112
CHUNKS = ((0, 28), (28, 56), (56, 83))


@pytest.fixture(scope="module", autouse=True)
def cuda_ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    _abi.lib()
    yield
    _abi.moe_check_device()


@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_stack_in_three_chunks(dtype, nesterov):
    """Each chunk's updates and momenta are those of a stack of that chunk alone, bit for bit, and right at its borders."""
    def plan(n):
        return moe.Orthogonalizer(n, ROWS, COLS, grad_dtype=dtype, beta=0.9, nesterov=nesterov)

    o, one = plan(N), plan(1)
    assert 28 * one.ws.numel() > 0.99 * o.ws.numel() > 27 * 0.99 * one.ws.numel()  # 28 matrices' workspace, not 83
    g = gauss(N, ROWS, COLS, 21).to(dtype)
    m = gauss(N, ROWS, COLS, 22)
    before = m.clone()
    out = torch.full((N, ROWS, COLS), 7.0, dtype=torch.bfloat16, device="cuda")
    assert o.orthogonalize(g, momentum=m, out=out) is out
    beta = float(torch.tensor(0.9))  # as the descriptor holds it
    for first, last in CHUNKS:
        alone = before[first:last].clone()
        assert torch.equal(plan(last - first).orthogonalize(g[first:last], momentum=alone), out[first:last])
        assert torch.equal(alone, m[first:last])
        for i in (first, last - 1):
            m64 = beta * before[i:i + 1].double() + g[i:i + 1].double()
            size = before[i:i + 1].double().abs() + g[i:i + 1].double().abs()
            assert bool(((m[i:i + 1].double() - m64).abs() <= 2.0**-24 * 3 * size).all())
            check(out[i:i + 1], reference(g[i:i + 1].double() + beta * m64 if nesterov else m64))
