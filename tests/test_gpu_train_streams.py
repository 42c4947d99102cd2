"""TokenSorter and Orthogonalizer on a stream that is given and is not the current one."""
import pytest
import torch

import sparse_moe_layer_biased_b200 as moe
from sparse_moe_layer_biased_b200 import _abi

pytestmark = pytest.mark.gpu
T, H, E, K = 700, 512, 24, 4


@pytest.fixture(scope="module", autouse=True)
def cuda_ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    _abi.lib()
    yield
    _abi.moe_check_device()


class Handle:
    """A stream of another library: nothing but its handle."""

    def __init__(self, stream):
        self.cuda_stream = stream.cuda_stream


@pytest.fixture(scope="module")
def calls():
    """The five calls, each call(stream) -> its results."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((T, H), generator=gen, device="cuda").bfloat16()
    idx = torch.randint(0, E, (T, K), generator=gen, device="cuda", dtype=torch.int32)
    w = torch.rand((T, K), generator=gen, device="cuda")
    grad = torch.randn((2, 160, 200), generator=gen, device="cuda")
    s, o = moe.TokenSorter(T, H, E, K), moe.Orthogonalizer(2, 160, 200)
    rows, _, slot = s.sort(x, idx)
    torch.cuda.synchronize()
    return {
        "sort": lambda stream: s.sort(x, idx, stream=stream),
        "sort_backward": lambda stream: (s.sort_backward(rows, slot, stream=stream),),
        "unsort": lambda stream: (s.unsort(rows, slot, w, add=x, stream=stream),),
        "unsort_backward": lambda stream: s.unsort_backward(x, rows, slot, w, stream=stream),
        "orthogonalize": lambda stream: (o.orthogonalize(grad, stream=stream),),
    }


@pytest.mark.parametrize("form", ["stream", "handle", "object"])
@pytest.mark.parametrize("name", ["sort", "sort_backward", "unsort", "unsort_backward", "orthogonalize"])
def test_results_are_not_in_memory_that_the_current_stream_still_writes(calls, name, form):
    """Tensors of the results' sizes are freed while the current stream has yet to fill them: PyTorch hands their memory to
    the next allocation for that stream, which a call on another one must not be."""
    call = calls[name]
    want = [t.clone() for t in call(None)]
    side = torch.cuda.Stream()
    given = {"stream": side, "handle": side.cuda_stream, "object": Handle(side)}[form]
    # memory for the other stream and the kernels used below: to get them from the driver later would wait for the current stream
    call(given)
    held = [torch.empty_like(t).fill_(1) for t in want for _ in range(3)]
    torch.cuda._sleep(1)
    torch.cuda.synchronize()
    torch.cuda._sleep(800_000_000)  # 0.4 s of the current stream
    for t in held:
        t.fill_(77)
    del held, t
    got = call(given)
    side.synchronize()
    assert not torch.cuda.current_stream().query()  # the fills are still to come
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want, strict=True))


@pytest.mark.parametrize("name", ["sort", "sort_backward", "unsort", "unsort_backward", "orthogonalize"])
def test_the_default_stream_by_its_handles_from_another(calls, name):
    call = calls[name]
    want = [t.clone() for t in call(None)]
    torch.cuda.synchronize()
    for stream in (0, 1, torch.cuda.default_stream()):
        with torch.cuda.stream(torch.cuda.Stream()):
            got = call(stream)
        assert all(torch.equal(a, b) for a, b in zip(got, want, strict=True))


def test_a_call_with_out_on_a_given_stream(calls):
    side = torch.cuda.Stream()
    o = moe.Orthogonalizer(2, 40, 64)
    g = torch.randn((2, 40, 64), device="cuda")
    want = o.orthogonalize(g).clone()
    out = torch.empty_like(want)
    torch.cuda.synchronize()
    assert o.orthogonalize(g, out=out, stream=side) is out
    side.synchronize()
    assert torch.equal(out, want)
