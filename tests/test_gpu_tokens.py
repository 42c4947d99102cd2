"""Token sort, unsort and their gradients against the definition in 64 bits.

Tolerances. A result is a sum of n fp32 terms (any order: off by at most n 2^-24 of the sum of
magnitudes, counting each term's own product rounding) rounded once to the row type (half a step,
finfo.eps / 2 of the value, or half the smallest subnormal step). The sort itself is exact."""
import pytest
import torch

import sparse_moe_layer_biased_b200 as moe
from sparse_moe_layer_biased_b200 import _abi

pytestmark = pytest.mark.gpu
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32

# T, H, E, k, dtype, share of dropped entries
CASES = [
    (1, 4096, 288, 8, BF, 0.0), (1, 1, 1, 1, FP, 0.0), (3, 7, 5, 2, HF, 0.3), (64, 4096, 288, 8, BF, 0.0),
    (64, 256, 16, 4, BF, 0.2), (33, 1290, 60, 6, HF, 0.2), (5, 24, 1024, 32, FP, 0.1), (128, 40, 1, 32, HF, 0.4),
    (512, 72, 352, 8, BF, 0.0), (513, 72, 352, 8, BF, 0.1),
    (256, 40, 352, 8, BF, 0.1), (257, 40, 352, 8, BF, 0.1),          # 2048 entries: the last sort of one launch
    (1024, 16, 33, 8, HF, 0.1), (1025, 16, 33, 8, HF, 0.1),          # 8192: one round a warp
    (4096, 8, 1024, 8, BF, 0.1), (4097, 8, 1024, 8, BF, 0.1),        # 32768: the last sort of two launches
    (1500, 1023, 40, 3, FP, 0.2), (777, 514, 16, 7, FP, 0.1), (2001, 100, 1024, 9, HF, 0.0),
    (4096, 513, 3, 4, BF, 1.0), (200, 64, 7, 5, FP, 1.0), (9000, 32, 288, 8, BF, 0.05), (700, 8200, 11, 8, BF, 0.5),
    (40000, 8, 1000, 8, HF, 0.02),
]
IDS = [f"T{c[0]}-H{c[1]}-E{c[2]}-k{c[3]}-{str(c[4])[6:]}-d{c[5]}" for c in CASES]


@pytest.fixture(scope="module", autouse=True)
def cuda_ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    _abi.lib()
    yield
    _abi.moe_check_device()


def routing(T, E, k, drop, gen):
    """Skewed ids with repeats within a token; dropped ones as -1, E and far outside."""
    idx = (torch.rand((T, k), generator=gen) ** 2 * E).to(torch.int32).clamp_(max=E - 1)
    gone = torch.rand((T, k), generator=gen) < drop
    if T > 2 and drop > 0:
        gone[T // 2] = True  # a token without any entry
    outside = torch.tensor([-1, E, 2**31 - 1, -(2**31)], dtype=torch.int32)[torch.randint(0, 4, (T, k), generator=gen)]
    return torch.where(gone, outside, idx)


def places(idx, E):
    """slot_of and offsets from the definition."""
    flat = idx.flatten().tolist()
    kept = sorted((e, n) for n, e in enumerate(flat) if 0 <= e < E)
    slot = torch.full((len(flat),), -1, dtype=torch.int32)
    for s, (_, n) in enumerate(kept):
        slot[n] = s
    count = torch.zeros(E + 1, dtype=torch.int64)
    for e, _ in kept:
        count[e + 1] += 1
    return slot.view(idx.shape), count.cumsum(0).to(torch.int32)


def setup(T, H, E, k, dtype, drop, seed=0):
    gen = torch.Generator().manual_seed(seed + T + H)
    idx = routing(T, E, k, drop, gen)
    slot, offsets = places(idx, E)
    return gen, idx, slot, offsets, moe.TokenSorter(T, H, E, k, dtype=dtype)


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def assert_close(got, want, magnitude, terms, dtype):
    slack = terms * 2.0**-24 * magnitude
    tol = slack + half_step(dtype) * (want.abs() + slack) + torch.finfo(dtype).smallest_normal * half_step(dtype) * 2
    off = (got.double().cpu() - want).abs()
    assert bool((off <= tol).all()), f"off by {(off - tol).max().item():.3e} more than allowed"


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_sort(case):
    T, H, E, k, dtype, drop = case
    gen, idx, slot, offsets, s = setup(*case)
    x = torch.randn((T, H), generator=gen).to(dtype)
    out = (torch.full((T * k, H), 7.0, dtype=dtype, device="cuda"), torch.full((E + 1,), -5, dtype=torch.int32,
           device="cuda"), torch.full((T, k), -5, dtype=torch.int32, device="cuda"))
    got = s.sort(x.cuda(), idx.cuda(), out=out)
    assert all(a is b for a, b in zip(got, out))
    assert torch.equal(got[2].cpu(), slot) and torch.equal(got[1].cpu(), offsets)
    want = torch.full((T * k, H), 7.0, dtype=dtype)  # rows that no entry owns stay as they were
    at = slot.flatten().long()
    want[at[at >= 0]] = x.repeat_interleave(k, 0)[at >= 0]
    assert torch.equal(got[0].cpu(), want)


@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_unsort(case, weighted, add):
    T, H, E, k, dtype, drop = case
    gen, idx, slot, offsets, s = setup(*case)
    rows = torch.randn((T * k, H), generator=gen).to(dtype)
    rows[offsets[-1]:] = float("nan")  # what no entry owns is not read
    w = torch.randn((T, k), generator=gen)
    w[slot < 0] = float("inf")
    shared = torch.randn((T, H), generator=gen).to(dtype)
    y = s.unsort(rows.cuda(), slot.cuda(), w.cuda() if weighted else None, add=shared.cuda() if add else None)
    want, size = torch.zeros((T, H), dtype=torch.float64), torch.zeros((T, H), dtype=torch.float64)
    for j in range(k):
        on = slot[:, j] >= 0
        r = rows[slot[on, j].long()].double() * (w[on, j].double()[:, None] if weighted else 1.0)
        want[on] += r
        size[on] += r.abs()
    if add:
        want += shared.double()
        size += shared.double().abs()
    assert y.dtype == dtype
    assert_close(y, want, size, k + 1, dtype)
    if not weighted and not add:  # the sort's gradient is the same sum
        assert torch.equal(s.sort_backward(rows.cuda(), slot.cuda()), y)


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_unsort_backward(case, weighted):
    T, H, E, k, dtype, drop = case
    gen, idx, slot, offsets, s = setup(*case)
    rows = torch.randn((T * k, H), generator=gen).to(dtype)
    rows[offsets[-1]:] = float("nan")
    dy = torch.randn((T, H), generator=gen).to(dtype)
    w = torch.randn((T, k), generator=gen)
    w[slot < 0] = float("nan")
    out = (torch.full((T * k, H), 7.0, dtype=dtype, device="cuda"),
           torch.full((T, k), 7.0, dtype=torch.float32, device="cuda"))
    drows, dw = s.unsort_backward(dy.cuda(), rows.cuda(), slot.cuda(), w.cuda() if weighted else None, out=out)
    n = int(offsets[-1])
    assert torch.equal(drows[n:].cpu(), torch.full((T * k - n, H), 7.0, dtype=dtype))
    want, want_w, size_w = torch.zeros((n, H), dtype=torch.float64), torch.zeros((T, k)).double(), torch.zeros((T, k)).double()
    for j in range(k):
        on = slot[:, j] >= 0
        at = slot[on, j].long()
        want[at] = dy[on].double() * (w[on, j].double()[:, None] if weighted else 1.0)
        p = dy[on].double() * rows[at].double()
        want_w[on, j], size_w[on, j] = p.sum(1), p.abs().sum(1)
    assert_close(drows[:n], want, want.abs(), 1, dtype)
    assert_close(dw, want_w, size_w, H, torch.float32)
    assert bool((dw.cpu()[slot < 0] == 0).all())
    # one output alone
    desc = _abi.TokenDesc(T, H, E, k, _abi.DTYPES[dtype])
    only = torch.full_like(out[0], 7.0), torch.full_like(out[1], 7.0)
    wc = w.cuda() if weighted else None
    _abi.moe_unsort_tokens_backward(desc, dy.cuda(), None, slot.cuda(), wc, only[0], None)
    _abi.moe_unsort_tokens_backward(desc, dy.cuda(), rows.cuda(), slot.cuda(), wc, None, only[1])
    assert torch.equal(only[0].view(torch.uint8), drows.view(torch.uint8)) and torch.equal(only[1], dw)


def test_gradients_against_differences():
    """The unsort is linear in the rows and in the weights: its derivative along a direction is the
    difference quotient with a step that fp32 holds exactly, off by the two values' roundings."""
    T, H, E, k = 37, 64, 9, 3
    gen, idx, slot, offsets, s = setup(T, H, E, k, FP, 0.2, seed=3)
    rows, dirs = torch.randn((T * k, H), generator=gen), torch.randn((T * k, H), generator=gen)
    w, dirw = torch.randn((T, k), generator=gen), torch.randn((T, k), generator=gen)
    dy = torch.randn((T, H), generator=gen)
    cu = lambda *ts: [t.cuda() for t in ts]  # noqa: E731
    drows, dw = s.unsort_backward(*cu(dy, rows, slot, w),
                                  out=(torch.zeros((T * k, H), device="cuda"), torch.zeros((T, k), device="cuda")))
    step = 0.5

    def loss(r, ww):
        return (s.unsort(*cu(r, slot, ww)).double().cpu() * dy.double()).sum().item()

    size = 8 * (T * k * H) * 2.0**-24 * 4  # terms of the two losses x unit rounding x magnitude of a term
    got = (loss(rows + step * dirs, w) - loss(rows, w)) / step
    assert abs(got - (drows.double().cpu() * dirs.double()).sum().item()) <= size
    got = (loss(rows, w + step * dirw) - loss(rows, w)) / step
    assert abs(got - (dw.double().cpu() * dirw.double()).sum().item()) <= size
    # and of the sort: <sort(x), g> = <x, sort_backward(g)>
    x, g = torch.randn((T, H), generator=gen), torch.randn((T * k, H), generator=gen)
    xs, off, sl = s.sort(x.cuda(), idx.cuda())
    n = int(off[-1])
    left = (xs[:n].double().cpu() * g[:n].double()).sum().item()
    right = (s.sort_backward(g.cuda(), sl).double().cpu() * x.double()).sum().item()
    assert abs(left - right) <= size


@pytest.mark.parametrize("dtype", [BF, FP])
def test_arrays_that_start_off_their_alignment(dtype):
    """Rows that start one element behind a 16-byte boundary take a narrower access."""
    T, H, E, k = 70, 64, 9, 3
    gen, idx, slot, offsets, s = setup(T, H, E, k, dtype, 0.1)

    def shifted(*shape):
        n = 1
        for v in shape:
            n *= v
        return torch.zeros(n + 1, dtype=dtype, device="cuda")[1:].view(*shape)

    x, xs = shifted(T, H), shifted(T * k, H)
    x.copy_(torch.randn((T, H), generator=gen))
    a = s.sort(x, idx.cuda(), out=(xs, torch.empty(E + 1, dtype=torch.int32, device="cuda"),
                                   torch.empty((T, k), dtype=torch.int32, device="cuda")))
    b = s.sort(x.clone(), idx.cuda())
    n = int(b[1][-1])
    assert torch.equal(a[0][:n], b[0][:n]) and torch.equal(a[2], b[2])
    w = torch.rand((T, k), generator=gen).cuda()
    y = shifted(T, H)
    s.unsort(xs, a[2], w, add=x, out=y)
    assert torch.equal(y, s.unsort(xs.clone(), a[2], w, add=x.clone()))
    d = shifted(T * k, H)
    dw = torch.empty((T, k), device="cuda")
    s.unsort_backward(x, xs, a[2], w, out=(d, dw))
    e, ew = s.unsort_backward(x.clone(), xs.clone(), a[2], w)
    assert torch.equal(d[:n], e[:n])
    assert_close(dw, ew.double().cpu(), (x.double().abs().sum(1, keepdim=True) * 5).cpu().expand(T, k), 2 * H, FP)


@pytest.mark.slow
def test_row_offsets_past_32_bits():
    """T k H = 2.3e9 elements: rows sampled at both ends."""
    T, H, E, k = 70000, 4096, 64, 8
    gen = torch.Generator().manual_seed(5)
    idx = routing(T, E, k, 0.01, gen).cuda()
    s = moe.TokenSorter(T, H, E, k)
    x = torch.randn((T, H), device="cuda").to(BF)
    xs, offsets, slot = s.sort(x, idx)
    n = int(offsets[-1])
    key = torch.where((idx >= 0) & (idx < E), idx, E).flatten()
    order = torch.argsort(key, stable=True)
    want = torch.full_like(order, -1)
    want[order[:n]] = torch.arange(n, device="cuda")
    assert torch.equal(slot.flatten().long(), want)
    for a, b in ((0, 200), (n // 2, n // 2 + 200), (n - 200, n)):
        assert torch.equal(xs[a:b], x[order[a:b] // k])
    w = torch.rand((T, k), device="cuda")
    y = s.unsort(xs, slot, w)
    tail = slice(T - 50, T)
    kept = slot[tail] >= 0
    total = (w[tail] * kept).double().sum(1, keepdim=True)
    assert_close(y[tail], (total * x[tail].double()).cpu(), (total * x[tail].double().abs()).cpu(), 9, BF)
    dxs, dw = s.unsort_backward(x, xs, slot, w)
    at = slot[tail][kept].long()
    t = torch.arange(T - 50, T, device="cuda")[:, None].expand(50, k)[kept]
    assert_close(dxs[at], (w[tail][kept].double()[:, None] * x[t].double()).cpu(), (3 * x[t].double().abs()).cpu(), 1, BF)
    dots = x[t].double().square().sum(1)
    assert_close(dw[tail][kept], dots.cpu(), dots.cpu(), H, FP)


def test_another_stream_and_a_replayed_graph():
    """The whole run on a side stream and replayed from a graph, for a small and a large sort."""
    for T, H, E, k in ((24, 512, 40, 8), (1200, 264, 40, 8)):
        gen, idx, slot, offsets, s = setup(T, H, E, k, BF, 0.1)
        x = torch.randn((T, H), generator=gen).to(BF).cuda()
        ids, w = idx.cuda(), torch.rand((T, k), generator=gen).cuda()

        def run():
            xs, off, sl = s.sort(x, ids)
            y = s.unsort(xs, sl, w, add=x)
            d, dw = s.unsort_backward(y, xs, sl, w, out=(torch.zeros_like(xs), torch.empty_like(w)))
            return [off, sl, y, dw, s.sort_backward(d, sl)]

        want = [t.clone() for t in run()]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got = run()
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = run()
        ids.copy_(routing(T, E, k, 0.4, gen))
        x.copy_(torch.randn((T, H), generator=gen))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        assert all(torch.equal(a, b) for a, b in zip(got, run()))


def test_no_tokens():
    s = moe.TokenSorter(16, 64, 5, 2)
    x = torch.empty((0, 64), dtype=BF, device="cuda")
    xs, offsets, slot = s.sort(x, torch.empty((0, 2), dtype=torch.int32, device="cuda"))
    assert xs.shape == (0, 64) and slot.shape == (0, 2) and offsets.tolist() == [0] * 6
    assert s.unsort(xs, slot).shape == (0, 64) and s.sort_backward(xs, slot).shape == (0, 64)
    d, dw = s.unsort_backward(x, xs, slot)
    assert d.shape == (0, 64) and dw.shape == (0, 2)


def test_infinities_and_nan_stay_in_their_tokens():
    T, H, E, k = 20, 32, 4, 2
    gen, idx, slot, offsets, s = setup(T, H, E, k, FP, 0.0)
    rows = torch.randn((T * k, H), generator=gen)
    rows[slot[3, 1], 5], rows[slot[7, 0], 6] = float("inf"), float("nan")
    y = s.unsort(rows.cuda(), slot.cuda(), torch.ones((T, k)).cuda()).cpu()
    bad = ~torch.isfinite(y)
    assert bad.nonzero().tolist() == [[3, 5], [7, 6]]
    assert y[3, 5] == float("inf") and torch.isnan(y[7, 6])


# widths around those where rows share a block, a warp or a few lanes; token counts that leave a block's last ones empty
NARROW = [
    (2403, 1064, 40, 5, BF, 0.1), (2403, 1064, 40, 12, BF, 0.1), (403, 1064, 40, 5, BF, 0.1), (2501, 264, 7, 9, HF, 0.2),
    (1003, 90, 9, 4, BF, 0.1), (777, 45, 9, 3, BF, 0.1), (301, 64, 40, 8, HF, 0.3), (301, 64, 40, 8, FP, 0.3),
    (2405, 130, 5, 2, FP, 0.1), (2405, 255, 40, 1, BF, 0.2), (4099, 520, 40, 1, BF, 0.0), (605, 512, 40, 4, BF, 0.1),
    (605, 513, 40, 6, HF, 0.1), (2369, 1280, 16, 8, BF, 0.1), (2369, 1288, 16, 8, BF, 0.1), (305, 2, 3, 20, FP, 0.5),
]


@pytest.mark.parametrize("case", NARROW, ids=[f"T{c[0]}-H{c[1]}-k{c[3]}-{str(c[4])[6:]}" for c in NARROW])
def test_rows_that_share_a_block(case):
    test_sort(case)
    for weighted in (True, False):
        test_unsort(case, weighted, weighted)
        test_unsort_backward(case, weighted)


def test_refusals_on_the_device():
    """What the host tests refuse, with tensors on the device: no call is made, the error names the tensor."""
    T, H, E, k = 12, 64, 5, 2
    s = moe.TokenSorter(T, H, E, k)
    x = torch.ones((T, H), dtype=BF, device="cuda")
    idx = torch.zeros((T, k), dtype=torch.int32, device="cuda")
    xs, offsets, slot = s.sort(x, idx)
    w = torch.ones((T, k), device="cuda")
    keep = xs.clone()
    for bad in (x.half(), x.cpu(), x[:, :32], x.t().contiguous().t(), x[0]):
        with pytest.raises(ValueError, match="x:"):
            s.sort(bad, idx, out=(xs, offsets, slot))
        if bad.dim() == 2:
            with pytest.raises(ValueError, match="dy:"):
                s.unsort_backward(bad, xs, slot, w)
            with pytest.raises(ValueError, match="add:"):
                s.unsort(xs, slot, w, add=bad)
            with pytest.raises(ValueError, match="dx:"):
                s.sort_backward(xs, slot, out=bad)
    for bad in (idx.long(), idx.cpu(), idx[:-1], idx.flatten()):
        with pytest.raises(ValueError, match="topk_idx"):
            s.sort(x, bad)
    for bad in (w.double(), w.bfloat16(), w.cpu(), w[:, :1], slot):
        with pytest.raises(ValueError, match="topk_w"):
            s.unsort(xs, slot, bad)
        with pytest.raises(ValueError, match="topk_w"):
            s.unsort_backward(x, xs, slot, bad)
    with pytest.raises(ValueError, match="offsets"):
        s.sort(x, idx, out=(xs, offsets[:-1], slot))
    with pytest.raises(ValueError, match="exceed"):
        s.sort(torch.cat([x, x]), torch.cat([idx, idx]))
    calls = _abi.calls()
    spec = s._spec
    for args in ((), (spec, 0), (spec, 0, xs, slot), ((1, 2), 0, xs, slot, x), (spec, "stream", xs, slot, x)):
        with pytest.raises(TypeError):
            calls.sort_backward(*args)
    assert calls.sort_backward(spec, 0, xs, slot, None) == -1 and calls.sort_backward(spec, 0, xs, x, x) == -1
    meta = torch.empty((T, H), dtype=BF, device="meta")
    assert calls.sort_backward(spec, 0, xs, slot, meta) == -1
    torch.cuda.synchronize()
    assert torch.equal(xs, keep)


@pytest.mark.parametrize("T,E", [(2048, 31), (2049, 32), (6144, 1024), (6145, 7), (8192, 300), (8193, 300)])
def test_sort_at_the_borders_of_its_rounds(T, E):
    """16384, 49152 and 65536 entries, and a token more."""
    test_sort((T, 8, E, 8, BF, 0.1))
