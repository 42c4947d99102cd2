"""Host-only checks of the token sort and orthogonalisation entry points: refusals happen before
anything touches the device."""
import ctypes

import pytest
import torch

import sparse_moe_layer_biased_b200 as moe
from sparse_moe_layer_biased_b200 import _abi

FAKE = 1 << 20  # non-null, 256-byte aligned; never dereferenced because validation fails first
BIG = 1 << 40


def tok(**kw):
    d = dict(T=64, H=256, E=16, k=4, dtype=1)
    d.update(kw)
    return _abi.TokenDesc(d["T"], d["H"], d["E"], d["k"], d["dtype"])


def orth(**kw):
    d = dict(n=2, rows=128, cols=256, dtype=0, steps=5, a=3.4445, b=-4.7750, c=2.0315, eps=1e-7, scale=1.0, beta=0.95,
             nesterov=1)
    d.update(kw)
    return _abi.OrthogonalizeDesc(*[d[f] for f, _ in _abi.OrthogonalizeDesc._fields_])


def token_calls(d):
    """Status of every token entry point for descriptor d (fake pointers)."""
    L, r = moe.lib(), ctypes.byref(d)
    out = ctypes.c_size_t(0)
    return [L.moe_sort_workspace_size(r, ctypes.byref(out)),
            L.moe_sort_tokens(r, *[FAKE] * 6, BIG, None),
            L.moe_sort_tokens_backward(r, FAKE, FAKE, FAKE, None),
            L.moe_unsort_tokens(r, *[FAKE] * 5, None),
            L.moe_unsort_tokens_backward(r, *[FAKE] * 6, None)]


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), 1), (dict(H=0), 1), (dict(E=0), 1), (dict(k=0), 1), (dict(k=33), 1), (dict(dtype=3), 1),
    (dict(dtype=-1), 1), (dict(E=1025), 2), (dict(H=(1 << 22) + 1), 2), (dict(T=1 << 28, k=8), 2),
])
def test_bad_token_descriptors_rejected(kw, status):
    assert token_calls(tok(**kw)) == [status] * 5


def test_token_pointers():
    L, r = moe.lib(), ctypes.byref(tok())
    for i in range(6):
        a = [FAKE] * 6
        a[i] = None
        assert L.moe_sort_tokens(r, *a, BIG, None) == 1
    for i, off in ((0, 1), (1, 2), (2, 1), (3, 2), (4, 2), (5, 8)):  # below each array's alignment
        a = [FAKE] * 6
        a[i] += off
        assert L.moe_sort_tokens(r, *a, BIG, None) == 2
    assert L.moe_sort_tokens(r, *[FAKE] * 6, moe.moe_sort_workspace_size(tok()) - 1, None) == 3
    for i in (0, 1, 4):  # topk_w and add may be NULL
        a = [FAKE] * 5
        a[i] = None
        assert L.moe_unsort_tokens(r, *a, None) == 1
    for i in range(5):
        a = [FAKE] * 5
        a[i] += 1
        assert L.moe_unsort_tokens(r, *a, None) == 2
    for missing in ((0,), (2,), (4, 5), (1,)):  # dy, slot_of, both outputs, rows with dtopk_w wanted
        a = [FAKE] * 6
        for i in missing:
            a[i] = None
        assert L.moe_unsort_tokens_backward(r, *a, None) == 1
    for i in range(6):
        a = [FAKE] * 6
        a[i] += 1
        assert L.moe_unsort_tokens_backward(r, *a, None) == 2
    f32 = ctypes.byref(tok(dtype=0))
    assert L.moe_unsort_tokens(f32, FAKE + 2, FAKE, None, None, FAKE, None) == 2
    assert L.moe_sort_tokens_backward(f32, FAKE, FAKE, FAKE + 2, None) == 2


def test_no_tokens_is_a_no_op():
    L, r = moe.lib(), ctypes.byref(tok(T=0))
    assert L.moe_sort_tokens(r, *[None] * 6, 0, None) == 0
    assert L.moe_sort_tokens(r, None, None, None, FAKE + 2, None, None, 0, None) == 2
    assert L.moe_sort_tokens_backward(r, None, None, None, None) == 0
    assert L.moe_unsort_tokens(r, *[None] * 5, None) == 0
    assert L.moe_unsort_tokens_backward(r, *[None] * 6, None) == 0


def test_sort_workspace_covers_every_smaller_call():
    # a sorter's workspace, sized for its largest call, serves each smaller one
    for E, k in ((16, 4), (1024, 32), (1, 1)):
        sizes = [moe.moe_sort_workspace_size(tok(T=T, E=E, k=k)) for T in (0, 1, 100, 5000, 70000)]
        assert sizes == sorted(sizes)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), 1), (dict(rows=0), 1), (dict(cols=-3), 1), (dict(steps=0), 1), (dict(steps=33), 1),
    (dict(dtype=5), 1), (dict(eps=-1e-8), 1), (dict(eps=float("nan")), 1), (dict(a=float("inf")), 1),
    (dict(scale=float("nan")), 1), (dict(beta=float("inf")), 1), (dict(nesterov=2), 1),
    (dict(dtype=2), 2), (dict(rows=16385), 2), (dict(cols=16385), 2), (dict(n=65536), 2),
    # singular values would leave the operands' range: 9 s in the first step; growth over the steps; b s^2
    (dict(a=9.0, b=0.0, c=0.0, steps=2), 2), (dict(a=2.0, b=0.0, c=0.0), 2), (dict(a=1.0, b=-40.0, c=39.0), 2),
])
def test_bad_orthogonalize_descriptors_rejected(kw, status):
    L, d = moe.lib(), orth(**kw)
    out = ctypes.c_size_t(0)
    assert L.moe_orthogonalize_workspace_size(ctypes.byref(d), ctypes.byref(out)) == status
    assert L.moe_orthogonalize(ctypes.byref(d), FAKE, FAKE, FAKE, FAKE, BIG, None) == status


def test_coefficients_in_range_are_accepted():
    for kw in (dict(), dict(a=1.5, b=-0.5, c=0.0, steps=32), dict(a=2.0, b=-1.5, c=0.5, steps=12),
               dict(a=9.0, b=0.0, c=0.0, steps=1)):  # the last X is not an operand
        assert moe.moe_orthogonalize_workspace_size(orth(**kw)) > 0


def test_orthogonalize_pointers():
    L, d = moe.lib(), orth()
    need = moe.moe_orthogonalize_workspace_size(d)
    r = ctypes.byref(d)
    assert L.moe_orthogonalize(r, FAKE, None, FAKE, FAKE, need - 1, None) == 3
    for i in (0, 2, 3):
        a = [FAKE] * 4
        a[i] = None
        assert L.moe_orthogonalize(r, *a, need, None) == 1
    for i, off in ((0, 2), (1, 2), (2, 1), (3, 128)):
        a = [FAKE] * 4
        a[i] += off
        assert L.moe_orthogonalize(r, *a, need, None) == 2
    assert L.moe_orthogonalize(ctypes.byref(orth(n=0)), None, None, None, None, 0, None) == 0


def test_orthogonalize_workspace_is_bounded():
    # more matrices than fit 2 GiB are worked off in chunks
    big = moe.moe_orthogonalize_workspace_size(orth(n=4000, rows=1280, cols=4096))
    assert big <= (2 << 30) + (1 << 16)
    assert moe.moe_orthogonalize_workspace_size(orth(n=1, rows=16384, cols=16384)) > 2 << 30


def test_wrappers_refuse_on_the_host():
    s = moe.TokenSorter(8, 16, 4, 2, dtype=torch.float32, device="cpu")
    x, idx = torch.zeros(8, 16), torch.zeros(8, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="topk_idx"):
        s.sort(x, idx.long())
    with pytest.raises(ValueError, match="exceed"):
        s.sort(torch.zeros(9, 16), torch.zeros(9, 2, dtype=torch.int32))
    with pytest.raises(ValueError, match="x:"):
        s.sort(x.bfloat16(), idx)
    with pytest.raises(ValueError, match="not contiguous"):
        s.sort(torch.zeros(16, 8).t(), idx)
    with pytest.raises(ValueError, match="y_sorted"):
        s.unsort(torch.zeros(8, 16), idx)
    with pytest.raises(ValueError, match="topk_w"):
        s.unsort(torch.zeros(16, 16), idx, idx)
    with pytest.raises(ValueError, match="add"):
        s.unsort(torch.zeros(16, 16), idx, add=torch.zeros(7, 16))
    with pytest.raises(ValueError, match="dy:"):
        s.unsort_backward(torch.zeros(7, 16), torch.zeros(16, 16), idx)
    with pytest.raises(ValueError, match="slot_of"):
        s.sort_backward(torch.zeros(16, 16), torch.zeros(16, dtype=torch.int32))
    with pytest.raises(ValueError, match="float64"):
        moe.TokenSorter(8, 16, 4, 2, dtype=torch.float64, device="cpu")
    with pytest.raises(moe.MoeError):
        moe.TokenSorter(8, 16, 4, 33, device="cpu")
    o = moe.Orthogonalizer(2, 8, 16, device="cpu")
    g = torch.zeros(2, 8, 16)
    with pytest.raises(ValueError, match="grad"):
        o.orthogonalize(g.bfloat16())
    with pytest.raises(ValueError, match="momentum"):
        o.orthogonalize(g, momentum=g.bfloat16())
    with pytest.raises(ValueError, match="out"):
        o.orthogonalize(g, out=g)
    with pytest.raises(moe.MoeError):
        moe.Orthogonalizer(2, 8, 16, grad_dtype=torch.float16, device="cpu")


def test_tensors_in_host_memory_never_reach_the_library():
    """Calls that are right in all but the memory they are in."""
    s = moe.TokenSorter(8, 16, 4, 2, dtype=torch.float32, device="cpu")
    x, idx, rows = torch.zeros(8, 16), torch.zeros(8, 2, dtype=torch.int32), torch.zeros(16, 16)
    w = torch.zeros(8, 2)
    for call in (lambda: s.sort(x, idx), lambda: s.sort_backward(rows, idx), lambda: s.unsort(rows, idx, w, add=x),
                 lambda: s.unsort_backward(x, rows, idx, w),
                 lambda: moe.Orthogonalizer(2, 8, 16, device="cpu").orthogonalize(torch.zeros(2, 8, 16))):
        with pytest.raises(ValueError, match="CUDA device"):
            call()
