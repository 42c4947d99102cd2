"""Expired waits of the orthogonalised update's products.

The lowest limit is 1 us: a tile's first operands take longer from HBM (L2 is flushed first), and an accumulator takes its whole K
loop, so a call's waits run out. The results of such a call are void; it has to report the timeout, end
with its own loads landed, and leave nothing behind."""
import pytest
import torch

import sparse_moe_layer_biased_b200 as moe
from sparse_moe_layer_biased_b200 import _abi

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def cuda_ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    _abi.lib()
    yield
    _abi.moe_check_device()


def expired_calls(n, rows, cols, calls=6):
    """Statuses and times (us) of calls at the lowest limit; the calls before and after them give the same bits."""
    o = moe.Orthogonalizer(n, rows, cols)
    g = torch.randn((n, rows, cols), device="cuda", generator=torch.Generator(device="cuda").manual_seed(20))
    want = o.orthogonalize(g).clone()
    _abi.moe_check_device()
    flush = torch.empty(64 << 20, dtype=torch.float32, device="cuda")  # 256 MB > L2
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    statuses, times = [], []
    old = _abi.moe_set_wait_limit_ns(1000)
    try:
        for _ in range(calls):
            flush.fill_(1.0)
            begin.record()
            o.orthogonalize(g)
            end.record()
            try:
                _abi.moe_check_device()
                statuses.append("ok")
            except _abi.MoeError as e:
                assert e.status == 5, e
                statuses.append("timeout")
            times.append(begin.elapsed_time(end) * 1e3)
    finally:
        _abi.moe_set_wait_limit_ns(old)
    assert torch.equal(o.orthogonalize(g), want)
    _abi.moe_check_device()
    return statuses, times


@pytest.mark.parametrize("n,rows,cols", [(4, 1280, 1536), (4, 1536, 1280)])
def test_a_pair_waits_for_its_loads_not_for_a_time(n, rows, cols):
    """CTA pairs: 15 launches whose waits run out. A pair that left after a fixed time in place of its last load's
    arrival would be either too early or, at 200 us a launch, 3 ms late; an undisturbed call takes 0.36 ms."""
    statuses, times = expired_calls(n, rows, cols)
    assert set(statuses) == {"timeout"}
    assert min(times) < 1500, times


@pytest.mark.parametrize("n,rows,cols", [
    (64, 300, 900), (64, 900, 300),                  # single CTAs
    (16, 768, 2048),                                 # CTA pairs
    (1, 256, 1100), (1, 1100, 256), (1, 256, 4096),  # every product split over K
])
def test_every_form_of_the_products_reports_expired_waits(n, rows, cols):
    statuses, _ = expired_calls(n, rows, cols)
    assert "timeout" in statuses


@pytest.mark.parametrize("n,rows,cols", [(40, 100, 700), (40, 700, 100), (3, 128, 2048)])
def test_short_matrices_at_the_lowest_limit(n, rows, cols):
    """The one-launch form waits for nothing but its own products, of at most 16 MMAs: less than the lowest limit, so
    its waits do not have to run out; a call that reports no timeout has to be right."""
    o = moe.Orthogonalizer(n, rows, cols)
    g = torch.randn((n, rows, cols), device="cuda", generator=torch.Generator(device="cuda").manual_seed(23))
    want = o.orthogonalize(g).clone()
    old = _abi.moe_set_wait_limit_ns(1000)
    try:
        for _ in range(4):
            got = o.orthogonalize(g)
            try:
                _abi.moe_check_device()
            except _abi.MoeError as e:
                assert e.status == 5, e
                continue
            assert torch.equal(got, want)
    finally:
        _abi.moe_set_wait_limit_ns(old)
    assert torch.equal(o.orthogonalize(g), want)
