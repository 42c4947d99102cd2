"""Orthogonalised updates against the iteration in 64 bits.

Tolerance (2-norm of the difference over that of the result), before the first run: a step rounds its
operands X, A and B to fp16, 2^-12 of each element in the root mean square. B = bA + cAA is at most 2.8 near
orthogonality, so X's and B's roundings move the next X by 2.8 2^-12 each; A's enters cAA twice,
4 2^-12. Together 5.6 2^-12 a step; the polynomial's slope where singular values settle is about one, so
s steps add to sqrt(s) 5.6 2^-12, and the bf16 result adds 2^-8 / sqrt(3): sqrt(2.3e-3^2 + 3.1e-3^2) = 3.8e-3 for five
steps. Root mean squares hold for many elements; of few, each can be at its worst, where the bf16 half step
alone is 2^-8 of the value (it is at least 2^-9 of it) and adds to the products' part. Element by element eight
times the product part's root mean square on top of the half step."""
import math

import pytest
import torch

import sparse_moe_layer_biased_b200 as moe
from sparse_moe_layer_biased_b200 import _abi

pytestmark = pytest.mark.gpu
COEFFS = (3.4445, -4.7750, 2.0315)


@pytest.fixture(scope="module", autouse=True)
def cuda_ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    _abi.lib()
    yield
    _abi.moe_check_device()


def reference(u, steps=5, coeffs=COEFFS, eps=1e-7, scale=1.0):
    a, b, c = coeffs
    X = u.double()
    X = X / (torch.linalg.matrix_norm(X, keepdim=True) + eps)
    tall = X.shape[1] > X.shape[2]
    for _ in range(steps):
        A = X.mT @ X if tall else X @ X.mT
        B = b * A + c * A @ A
        X = a * X + (X @ B if tall else B @ X)
    return scale * X


def check(got, want, steps=5):
    part = math.sqrt(steps) * 5.6 * 2.0**-12
    for i in range(want.shape[0]):
        d, w = got[i].double() - want[i], want[i]
        norm = w.norm().item()
        most = math.hypot(part, 2.0**-8 / math.sqrt(3)) if w.numel() >= 256 else part + 2.0**-8
        assert d.norm().item() <= most * norm, f"matrix {i}: {d.norm().item() / norm:.3e}"
        rms = norm / math.sqrt(w.numel())
        assert bool((d.abs() <= 2.0**-8 * w.abs() + 8 * part * rms).all()), f"matrix {i}"


def gauss(n, rows, cols, seed=0):
    return torch.randn((n, rows, cols), generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


SIZES = [(3, 128, 256), (2, 256, 128), (1, 1, 1), (2, 1, 77), (2, 77, 1), (3, 33, 40), (2, 40, 33), (2, 130, 129),
         (1, 129, 131), (4, 64, 64), (1, 200, 1000), (1, 1000, 200), (2, 384, 257), (1, 513, 640), (1, 640, 513),
         (1, 1281, 700), (1, 700, 1281), (150, 16, 24),
         # short sides up to 128: a cluster per matrix, up to 2048 on the long side; beyond, the products
         (3, 100, 256), (2, 100, 257), (2, 600, 100), (1, 128, 2048), (1, 2047, 127), (2, 17, 1100), (1, 128, 2049),
         (1, 2100, 64)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size", SIZES, ids=["x".join(map(str, s)) for s in SIZES])
def test_random_matrices(size, dtype):
    g = gauss(*size).mul_(1e-3).to(dtype)
    o = moe.Orthogonalizer(*size, grad_dtype=dtype)
    keep = g.clone()
    check(o.orthogonalize(g), reference(g))
    assert torch.equal(g, keep)


@pytest.mark.parametrize("rows,cols", [(1280, 4096), (4096, 1536)])
def test_layer_sizes(rows, cols):
    g = gauss(2, rows, cols, 3)
    check(moe.Orthogonalizer(2, rows, cols, scale=0.7).orthogonalize(g), reference(g, scale=0.7))


@pytest.mark.parametrize("rank", [1, 5, 40])
@pytest.mark.parametrize("rows,cols", [(160, 416), (416, 160), (1280, 1408), (60, 200), (700, 128)])
def test_gradients_of_few_tokens(rows, cols, rank):
    """A gradient of few tokens has a low rank: nothing may grow outside its range."""
    g = gauss(2, rows, rank, 1) @ gauss(2, rank, cols, 2)
    check(moe.Orthogonalizer(2, rows, cols).orthogonalize(g), reference(g))


@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,cols", [(96, 200), (131, 77), (131, 177), (600, 96)])
def test_momentum(rows, cols, dtype, nesterov):
    o = moe.Orthogonalizer(3, rows, cols, grad_dtype=dtype, beta=0.9, nesterov=nesterov)
    m = gauss(3, rows, cols, 4)
    m64 = m.double()
    beta = float(torch.tensor(0.9))  # as the descriptor holds it
    for step in range(3):
        g = gauss(3, rows, cols, 5 + step).to(dtype)
        out = o.orthogonalize(g, momentum=m)
        m64 = beta * m64 + g.double()
        # one rounding a step, the earlier ones decayed by beta
        assert bool(((m.double() - m64).abs() <= 2.0**-24 * 3 * (m64.abs() + g.double().abs())).all())
        check(out, reference(g.double() + beta * m64 if nesterov else m64))
        m64 = m.double()


@pytest.mark.parametrize("steps,coeffs", [(1, COEFFS), (2, COEFFS), (8, (2.0, -1.5, 0.5)), (6, (1.5, -0.5, 0.0))])
def test_other_iterations(steps, coeffs):
    g = gauss(2, 100, 180, 8)
    check(moe.Orthogonalizer(2, 100, 180, steps=steps, coeffs=coeffs).orthogonalize(g), reference(g, steps, coeffs), steps)


def test_result_is_nearly_orthogonal():
    """The customary coefficients bring every singular value of a well-conditioned matrix into
    [0.68, 1.21] (the polynomial's values on the interval it settles in), here with the tolerance above."""
    q, _ = torch.linalg.qr(gauss(1, 256, 192, 9).double())
    g = (q * torch.linspace(0.2, 1.0, 192, device="cuda", dtype=torch.float64)).float().contiguous()
    s = torch.linalg.svdvals(moe.Orthogonalizer(1, 256, 192).orthogonalize(g)[0].double())
    slack = 2.0**-8 * math.sqrt(192)
    assert 0.68 - slack <= s.min().item() and s.max().item() <= 1.21 + slack


@pytest.mark.parametrize("rows,cols", [(72, 200), (150, 216), (330, 150)])
def test_zero_tiny_huge_and_broken_matrices(rows, cols):
    """Each matrix by itself: a zero one gives zero, sizes of 1e-30 and 1e30 change nothing but by eps, a NaN or
    an infinity spoils its own matrix only."""
    g = gauss(7, rows, cols, 10)
    g[0] = 0
    g[2] *= 1e30
    g[3, 5, 6] = float("nan")
    g[4, 1, 2] = float("inf")
    g[6] *= 1e-30
    out = moe.Orthogonalizer(7, rows, cols, eps=1e-36).orthogonalize(g)
    assert bool((out[0] == 0).all())
    assert bool(torch.isnan(out[3]).all()) and bool(torch.isnan(out[4]).all())
    ok = [1, 2, 5, 6]
    check(out[ok], reference(g[ok], eps=1e-36))
    # eps counts against the norm
    g = gauss(1, rows, cols, 11) * 1e-9
    check(moe.Orthogonalizer(1, rows, cols, eps=1e-7).orthogonalize(g), reference(g, eps=1e-7))


@pytest.mark.parametrize("rows,cols", [(136, 264), (40, 700), (900, 520)])
def test_same_bits_on_a_side_stream_and_from_a_graph(rows, cols):
    o = moe.Orthogonalizer(5, rows, cols)
    g, m = gauss(5, rows, cols, 12), gauss(5, rows, cols, 13)
    want = o.orthogonalize(g, momentum=m.clone()).clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = o.orthogonalize(g, momentum=m.clone())
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    gg, mm = torch.zeros_like(g), torch.zeros_like(m)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = o.orthogonalize(gg, momentum=mm)
    gg.copy_(g)
    mm.copy_(m)
    graph.replay()
    assert torch.equal(held, want)
    mm.copy_(m)
    graph.replay()
    assert torch.equal(held, want)


def test_chunks_give_the_same_bits():
    """A stack too large for the workspace is worked off in chunks: 40 matrices of 2048 x 2112 are over 2 GiB."""
    n, rows, cols = 40, 2048, 2112
    o = moe.Orthogonalizer(n, rows, cols, grad_dtype=torch.bfloat16)
    assert o.ws.numel() < n * rows * cols * 12
    g = gauss(n, rows, cols, 14).bfloat16()
    out = o.orthogonalize(g)
    for i in (0, n // 2, n - 1):
        one = moe.Orthogonalizer(1, rows, cols, grad_dtype=torch.bfloat16).orthogonalize(g[i:i + 1])
        assert torch.equal(one[0], out[i])
    check(out[-1:], reference(g[-1:]))


def test_misaligned_inputs():
    """Views one element behind a 16-byte boundary, of widths that are and are not multiples of eight."""
    for rows, cols in ((40, 64), (40, 61)):
        n = 2 * rows * cols
        shift = lambda dt: torch.zeros(n + 1, dtype=dt, device="cuda")[1:].view(2, rows, cols)  # noqa: E731
        g, m, out = shift(torch.float32), shift(torch.float32), shift(torch.bfloat16)
        g.copy_(gauss(2, rows, cols, 15))
        m.copy_(gauss(2, rows, cols, 16))
        o = moe.Orthogonalizer(2, rows, cols)
        m2 = m.clone()
        want = o.orthogonalize(g.clone(), momentum=m2).clone()
        o.orthogonalize(g, momentum=m, out=out)
        assert torch.equal(m, m2)
        # the norm's partial sums differ in their grouping, so not bit for bit: two results, each of them in tolerance
        check(out, want.double())


def test_no_matrices():
    o = moe.Orthogonalizer(0, 16, 32)
    assert o.orthogonalize(torch.empty((0, 16, 32), device="cuda")).shape == (0, 16, 32)


@pytest.mark.parametrize("rows,cols", [(300, 337), (600, 340), (340, 600), (200, 2000)])
def test_many_tiles_a_cta_with_short_ones_among_them(rows, cols):
    """More matrices than CTAs, tiles of one to four (or eight) column blocks in turn."""
    n = 170
    g = gauss(n, rows, cols, 17)
    check(moe.Orthogonalizer(n, rows, cols).orthogonalize(g), reference(g))


@pytest.mark.parametrize("tall", [False, True])
@pytest.mark.parametrize("n,p,q", [(1, 129, 140), (1, 256, 1100), (2, 130, 560), (3, 260, 2049), (8, 256, 1000), (30, 200, 500),
                                   (1, 900, 1000), (80, 200, 260), (1, 100, 4001)])
def test_few_tiles(n, p, q, tall):
    """Products whose K is split over clusters of two to eight CTAs, some of them without a slice, beside ones that are not."""
    rows, cols = (q, p) if tall else (p, q)
    g = gauss(n, rows, cols, 18)
    o = moe.Orthogonalizer(n, rows, cols)
    out = o.orthogonalize(g)
    check(out, reference(g))
    assert torch.equal(out, o.orthogonalize(g))
