"""The training operators at the ends of their stated ranges, and several of them at once."""
import pytest
import torch

import sparse_moe_layer_biased_b200 as moe
from sparse_moe_layer_biased_b200 import _abi
from test_gpu_orthogonalize import check, gauss, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def cuda_ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    _abi.lib()
    yield
    _abi.moe_check_device()
    torch.cuda.empty_cache()


@pytest.mark.slow
@pytest.mark.parametrize("T,E,k,dtype", [(268_000_000, 5, 7, torch.float16), (2_100_000_000, 3, 1, torch.bfloat16)])
def test_entry_counts_near_2_to_31(T, E, k, dtype):
    """1.9e9 and 2.1e9 entries of rows of one element: places by their definition, the rest sampled at both ends."""
    idx = torch.randint(-1, E + 1, (T, k), device="cuda", dtype=torch.int32)
    x = torch.randn((T, 1), device="cuda").to(dtype)
    s = moe.TokenSorter(T, 1, E, k, dtype=dtype)
    rows, offsets, slot = s.sort(x, idx)
    ids, places = idx.view(-1), slot.view(-1)
    kept = (ids >= 0) & (ids < E)
    counts = torch.stack([(ids == e).sum() for e in range(E)])
    assert int(offsets[0]) == 0 and torch.equal(offsets[1:].long(), counts.cumsum(0))
    assert bool((places[~kept] == -1).all())
    for e in range(E):
        want = torch.arange(int(offsets[e]), int(offsets[e + 1]), device="cuda", dtype=torch.int32)
        assert torch.equal(places[ids == e], want)
        del want
    w = torch.rand((T, k), device="cuda")
    y = s.unsort(rows, slot, w)
    dx = s.sort_backward(rows, slot)
    drows, dw = s.unsort_backward(x, rows, slot, w)
    half = torch.finfo(dtype).eps / 2
    tiny = torch.finfo(dtype).smallest_normal * half * 2
    for part in (slice(0, 50_000), slice(T - 50_000, T)):
        on = kept.view(T, k)[part]
        at, xp = slot[part][on].long(), x[part].double()
        assert torch.equal(rows[at], x[part][:, None].expand(-1, k, 1)[on])
        for got, weight in ((y, w[part].double() * on), (dx, on.double())):
            want = weight.sum(1, keepdim=True) * xp  # k + 1 fp32 operations on terms of one sign, one rounding
            tol = want.abs() * (half + (k + 1) * 2.0**-24 * (1 + half)) + tiny
            assert bool(((got[part].double() - want).abs() <= tol).all())
        want = (w[part].double()[:, :, None] * xp[:, None])[on]
        assert bool(((drows[at].double() - want).abs() <= want.abs() * (half + 2.0**-24 * (1 + half)) + tiny).all())
        assert bool((dw[part][~on] == 0).all())
        want = (xp**2).expand(-1, k)[on]
        assert bool(((dw[part][on].double() - want).abs() <= want * 2.0**-24 + 2.0**-149).all())


@pytest.mark.parametrize("n,rows,cols", [(65535, 16, 24), (65535, 1, 2049), (65535, 1, 1), (1, 16384, 1), (1, 1, 16384),
                                         (2, 16384, 130), (3, 100, 16384)])
def test_the_most_matrices_and_the_longest_sides(n, rows, cols):
    g = gauss(n, rows, cols, 24)
    out = moe.Orthogonalizer(n, rows, cols).orthogonalize(g)
    pick = sorted({0, n // 2, n - 1})
    check(out[pick], reference(g[pick]))


@pytest.mark.slow
def test_the_largest_matrix():
    g = gauss(1, 16384, 16384, 25)
    check(moe.Orthogonalizer(1, 16384, 16384).orthogonalize(g), reference(g))


def test_several_calls_at_once():
    """Updates on CTA pairs, on single CTAs, split over K and in one launch, and a sorter's round trip, each on a stream of
    its own and with its own plan: the same bits as one after the other."""
    work = []
    for i, (n, rows, cols) in enumerate([(12, 768, 2048), (12, 2048, 768), (40, 300, 500), (1, 256, 2100), (60, 128, 1000)]):
        o, g = moe.Orthogonalizer(n, rows, cols), gauss(n, rows, cols, 30 + i)
        work.append(lambda o=o, g=g: (o.orthogonalize(g),))
    T, H, E, k = 9000, 520, 40, 8
    s = moe.TokenSorter(T, H, E, k)
    gen = torch.Generator(device="cuda").manual_seed(31)
    x = torch.randn((T, H), generator=gen, device="cuda").bfloat16()
    idx = torch.randint(0, E, (T, k), generator=gen, device="cuda", dtype=torch.int32)
    w = torch.rand((T, k), generator=gen, device="cuda")

    def round_trip():
        rows, offsets, slot = s.sort(x, idx)
        y = s.unsort(rows, slot, w, add=x)
        drows, dw = s.unsort_backward(y, rows, slot, w)
        return rows, offsets, slot, y, drows, dw, s.sort_backward(drows, slot)

    work.append(round_trip)
    want = [[t.clone() for t in f()] for f in work]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in work]
    for _ in range(5):
        got = []
        for f, stream in zip(work, streams):
            with torch.cuda.stream(stream):
                got.append(f())
        torch.cuda.synchronize()
        _abi.moe_check_device()
        for a, b in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(a, b, strict=True))
