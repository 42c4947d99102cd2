"""MoeLayer on a stream that is given and is not the current one."""
import pytest
import torch

from sparse_moe_layer_biased_b200 import _abi
from sparse_moe_layer_biased_b200.inputs import WORKLOADS, draw
from sparse_moe_layer_biased_b200.layer import MoeLayer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("handle", [False, True])
def test_results_are_not_in_memory_that_the_current_stream_still_writes(handle):
    """Tensors of the results' sizes are freed while the current stream has yet to fill them: PyTorch hands their memory to
    the next allocation for that stream, which a call on another one must not be."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    sh = WORKLOADS["tiny"]
    inp = {k: v.cuda() for k, v in draw(sh).items()}
    layer = MoeLayer(sh, inp, deterministic=True)
    want = [t.clone() for t in layer.forward(inp["x"], routing=True)]
    side = torch.cuda.Stream()
    given = side.cuda_stream if handle else side
    # memory for the other stream and the kernels used below: to get them from the driver later would wait for the current stream
    layer.forward(inp["x"], routing=True, stream=given)
    held = [torch.empty_like(t).fill_(1) for t in want for _ in range(3)]
    torch.cuda._sleep(1)
    torch.cuda.synchronize()
    torch.cuda._sleep(800_000_000)  # 0.4 s of the current stream
    for t in held:
        t.fill_(77)
    del held, t
    got = layer.forward(inp["x"], routing=True, stream=given)
    side.synchronize()
    assert not torch.cuda.current_stream().query()  # the fills are still to come
    torch.cuda.synchronize()
    _abi.moe_check_device()
    assert all(torch.equal(a, b) for a, b in zip(got, want, strict=True))


def test_host_batches_on_a_given_stream():
    """The workspace of host batches is made by the first such call: the same, for the stream of that call."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    sh = WORKLOADS["tiny"]
    inp = {k: v.cuda() for k, v in draw(sh).items()}
    layer = MoeLayer(sh, inp, deterministic=True)
    x = inp["x"].cpu().expand(3, -1, -1).contiguous().pin_memory()
    want = layer.forward_host(x)
    torch.cuda.synchronize()
    size = layer.ws_host.numel()
    side = torch.cuda.Stream()
    y = torch.empty_like(want).pin_memory()
    layer.ws_host = None
    layer.forward_host(x, y, stream=side)  # memory for that stream (see above)
    layer.ws_host = None
    held = [torch.empty(size, dtype=torch.uint8, device="cuda").fill_(1) for _ in range(3)]
    torch.cuda._sleep(1)
    torch.cuda.synchronize()
    torch.cuda._sleep(800_000_000)
    for t in held:
        t.fill_(77)
    del held, t
    y.zero_()
    layer.forward_host(x, y, stream=side)
    side.synchronize()
    assert not torch.cuda.current_stream().query()
    torch.cuda.synchronize()
    _abi.moe_check_device()
    assert torch.equal(y, want)
