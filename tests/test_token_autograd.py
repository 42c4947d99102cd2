"""TokenSorter and autograd: a call that autograd would silently leave out of its graph is refused."""
import pytest
import torch

import sparse_moe_layer_biased_b200 as moe
from sparse_moe_layer_biased_b200 import _abi

T, H, E, K = 6, 16, 4, 2
CALLS = {"sort": 5, "sort_backward": 3, "unsort": 5, "unsort_backward": 6}  # tensors of each


@pytest.mark.parametrize("name", list(CALLS))
def test_the_module_refuses_tensors_that_require_a_gradient(name):
    """Host tensors: without one that requires a gradient the call is refused for their memory (-1)."""
    fn = getattr(_abi.calls(), name)
    spec = (T, H, E, K, 0, 0, 1 << 20, 1 << 20)
    plain = [torch.zeros(T, H) for _ in range(CALLS[name])]
    assert fn(spec, 0, *plain) == -1
    for i in range(CALLS[name]):
        args = list(plain)
        args[i] = torch.zeros(T, H, requires_grad=True)
        assert fn(spec, 0, *args) == -2
        args[i] = args[i] * 2  # neither a leaf
        assert fn(spec, 0, *args) == -2
        with torch.no_grad():
            assert fn(spec, 0, *args) == -1
        args[i] = args[i].detach()
        assert fn(spec, 0, *args) == -1


def cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn((T, H), generator=gen, device="cuda")
    idx = torch.randint(-1, E + 1, (T, K), generator=gen, device="cuda", dtype=torch.int32)
    w = torch.rand((T, K), generator=gen, device="cuda")
    return moe.TokenSorter(T, H, E, K, dtype=torch.float32), x, idx, w


@pytest.mark.gpu
def test_methods_name_the_tensor():
    s, x, idx, w = cuda()
    rows, offsets, slot = s.sort(x, idx)
    keep = rows.clone()
    need = lambda t: t.clone().requires_grad_()  # noqa: E731
    for call, name in (
            (lambda: s.sort(need(x), idx), "x"), (lambda: s.sort_backward(need(rows), slot), "dx_sorted"),
            (lambda: s.sort(x, idx, out=(need(rows), offsets, slot)), "x_sorted"),
            (lambda: s.unsort(need(rows), slot, w), "y_sorted"), (lambda: s.unsort(rows, slot, need(w)), "topk_w"),
            (lambda: s.unsort(rows, slot, w, add=need(x) * 2), "add"), (lambda: s.unsort_backward(need(x), rows, slot), "dy"),
            (lambda: s.unsort_backward(x, need(rows), slot, need(w)), "y_sorted, topk_w")):
        with pytest.raises(ValueError, match=f"_tokens(_backward)?: {name}: requires a gradient"):
            call()
        with torch.no_grad():
            call()
    assert torch.equal(s.unsort(rows, slot, w, add=x), s.unsort(need(rows).detach(), slot, w, add=x))
    n = int(offsets[-1])
    assert torch.equal(rows[:n], keep[:n])


@pytest.mark.gpu
def test_gradients_through_autograd_functions():
    """The documented way: the calls inside autograd.Function, against the same formulas in torch. Everything but the
    order of sums of K or H fp32 terms is the same: off by at most (K + H) 2^-24 of the terms' magnitudes, twice."""
    s, x, idx, w = cuda()

    class Sort(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, idx):
            rows, offsets, slot = s.sort(x, idx, out=(torch.zeros((T * K, H), device="cuda"), torch.empty(
                E + 1, dtype=torch.int32, device="cuda"), torch.empty((T, K), dtype=torch.int32, device="cuda")))
            ctx.save_for_backward(slot)
            ctx.mark_non_differentiable(offsets, slot)
            return rows, offsets, slot

        @staticmethod
        def backward(ctx, drows, *_):
            return s.sort_backward(drows.contiguous(), *ctx.saved_tensors), None

    class Unsort(torch.autograd.Function):
        @staticmethod
        def forward(ctx, rows, slot, w):
            ctx.save_for_backward(rows, slot, w)
            return s.unsort(rows, slot, w)

        @staticmethod
        def backward(ctx, dy):
            rows, slot, w = ctx.saved_tensors
            drows, dw = s.unsort_backward(dy.contiguous(), rows, slot, w, out=(torch.zeros_like(rows), torch.empty_like(w)))
            return drows, None, dw

    leaves = [x.clone().requires_grad_(), w.clone().requires_grad_()]
    rows, _, slot = Sort.apply(leaves[0], idx)
    Unsort.apply(rows * rows, slot, leaves[1]).sin().sum().backward()
    plain = [x.double().requires_grad_(), w.double().requires_grad_()]
    kept = ((idx >= 0) & (idx < E)).double()
    y = torch.einsum("tk,th->th", plain[1] * kept, plain[0] * plain[0])
    y.sin().sum().backward()
    big = (K + H) * 2.0**-24 * 2
    # the argument of the cosine is off by that share of |y|, at most K x^2, and carries into both gradients
    size = K * (x.double() ** 2 + 1) ** 2 * 4
    assert bool(((leaves[0].grad.double() - plain[0].grad).abs() <= big * size).all())
    assert bool(((leaves[1].grad.double() - plain[1].grad).abs() <= big * size.sum(1, keepdim=True)).all())
