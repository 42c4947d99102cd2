"""The training operators through the binding's functions (the C entry points' names), as a caller with memory of
its own uses them, against TokenSorter and Orthogonalizer."""
import pytest
import torch

import sparse_moe_layer_biased_b200 as moe

BF = torch.bfloat16


@pytest.mark.gpu
@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("T,H,E,k,dtype", [(50, 96, 9, 4, BF), (900, 33, 40, 6, torch.float32), (9000, 16, 40, 8, torch.float16)])
def test_token_functions(T, H, E, k, dtype, given):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    gen = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn((T, H), generator=gen, device="cuda").to(dtype)
    idx = torch.randint(-1, E + 1, (T, k), generator=gen, device="cuda", dtype=torch.int32)
    w = torch.rand((T, k), generator=gen, device="cuda")
    s = moe.TokenSorter(T, H, E, k, dtype=dtype)
    rows, offsets, slot = s.sort(x, idx)
    n = int(offsets[-1])
    d = moe.TokenDesc(T, H, E, k, moe.DTYPES[dtype])
    ws = torch.empty(moe.moe_sort_workspace_size(d), dtype=torch.uint8, device="cuda")
    stream = torch.cuda.Stream() if given else None
    got = torch.empty_like(rows), torch.empty_like(offsets), torch.empty_like(slot)
    y, dx, dx2, drows, dw = (torch.empty_like(t) for t in (x, x, x, rows, w))
    torch.cuda.synchronize()
    moe.moe_sort_tokens(d, x, idx, *got, ws, stream=stream)
    moe.moe_unsort_tokens(d, got[0], got[2], w, x, y, stream=stream)
    moe.moe_unsort_tokens_backward(d, y, got[0], got[2], w, drows, dw, stream=stream)
    moe.moe_sort_tokens_backward(d, got[0], got[2], dx, stream=stream)
    moe.moe_unsort_tokens(d, got[0], got[2], None, None, dx2, stream=stream)
    torch.cuda.synchronize()
    assert torch.equal(got[0][:n], rows[:n]) and torch.equal(got[1], offsets) and torch.equal(got[2], slot)
    assert torch.equal(y, s.unsort(rows, slot, w, add=x))
    want = s.unsort_backward(y, rows, slot, w)
    assert torch.equal(drows[:n], want[0][:n]) and torch.equal(dw, want[1])
    assert torch.equal(dx, s.sort_backward(rows, slot)) and torch.equal(dx, dx2)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols", [(100, 180), (300, 200)])
def test_orthogonalize_function(rows, cols):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    n = 3
    g = torch.randn((n, rows, cols), device="cuda")
    m = torch.randn((n, rows, cols), device="cuda")
    o = moe.Orthogonalizer(n, rows, cols, beta=0.9, scale=0.5)
    m2 = m.clone()
    want = o.orthogonalize(g, momentum=m2)
    d = moe.OrthogonalizeDesc(n, rows, cols, moe.DTYPES[torch.float32], 5, 3.4445, -4.7750, 2.0315, 1e-7, 0.5, 0.9, 1)
    ws = torch.empty(moe.moe_orthogonalize_workspace_size(d), dtype=torch.uint8, device="cuda")
    out = torch.empty((n, rows, cols), dtype=BF, device="cuda")
    moe.moe_orthogonalize(d, g, m, out, ws)
    assert torch.equal(out, want) and torch.equal(m, m2)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    moe.moe_orthogonalize(d, g, None, out, ws, stream=side)
    side.synchronize()
    assert torch.equal(out, o.orthogonalize(g))


def test_functions_raise_on_refused_calls():
    """Host only: refusals come before anything is launched."""
    host = torch.zeros(16, 16)
    d = moe.TokenDesc(8, 16, 4, 33, 0)
    for call in (lambda: moe.moe_sort_workspace_size(d), lambda: moe.moe_sort_tokens(d, *[host] * 6, stream=0),
                 lambda: moe.moe_sort_tokens_backward(d, host, host, host, stream=0),
                 lambda: moe.moe_unsort_tokens(d, host, host, None, None, host, stream=0),
                 lambda: moe.moe_unsort_tokens_backward(d, host, host, host, None, host, host, stream=0)):
        with pytest.raises(moe.MoeError) as e:
            call()
        assert e.value.status == 1
    d = moe.TokenDesc(8, 16, 4, 2, 0)
    with pytest.raises(moe.MoeError) as e:
        moe.moe_sort_tokens(d, host, host, host, host, host, host[:1, :2].contiguous(), stream=0)
    assert e.value.status in (2, 3)  # 8 bytes of workspace, at whatever address
    o = moe.OrthogonalizeDesc(2, 8, 16, 0, 0, 3.4445, -4.7750, 2.0315, 1e-7, 1.0, 0.95, 1)
    for call in (lambda: moe.moe_orthogonalize_workspace_size(o), lambda: moe.moe_orthogonalize(o, host, None, host, host, stream=0)):
        with pytest.raises(moe.MoeError) as e:
            call()
        assert e.value.status == 1
