"""moe_backward on a workspace whose bytes spell NaN: the rows that pad a group to 64 must not reach
the gradients (zeros times what the workspace held before)."""
import pytest
import torch

from sparse_moe_layer_biased_b200 import _abi
from sparse_moe_layer_biased_b200.inputs import LayerShape, draw
from sparse_moe_layer_biased_b200.layer import MoeLayer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,E,k", [(40, 24, 2), (300, 3, 2), (600, 3, 2), (700, 16, 4)])
def test_the_workspace_holds_nan(T, E, k):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    sh = LayerShape("bwd_ws", T=T, H=256, E=E, k=k, I=128, Is=256, limit_routed=0.5, seed=75, weight_std=0.05)
    inp = {n: t.cuda() for n, t in draw(sh).items()}
    _, idx, w = MoeLayer(sh, inp).forward(inp["x"], routing=True)
    d = _abi.desc_of(sh)
    dy = torch.randn((T, sh.H), device="cuda", generator=torch.Generator(device="cuda").manual_seed(2))
    names = ("Wr", "W_gate_up", "W_down", "Wsh_gate_up", "Wsh_down")
    got = []
    for fill in (0, 255):  # 0xffff is a bf16 NaN, 0xffffffff an fp32 one
        ws = torch.full((_abi.moe_backward_workspace_size(d),), fill, dtype=torch.uint8, device="cuda")
        out = [torch.full((T, sh.H), float("nan"), device="cuda")]
        out += [torch.full(inp[n].shape, float("nan"), device="cuda") for n in names]
        _abi.moe_backward(d, inp["x"], *(inp[n] for n in names), idx, w, dy, *out, ws)
        got.append(out)
    _abi.moe_check_device()
    for name, a, b in zip(("x",) + names, *got):
        assert bool(torch.isfinite(b).all()), name
        # dx and dWr are summed with atomics, whose order changes from run to run: fp32 roundings apart
        assert (a - b).abs().max().item() <= 1e-4 * a.abs().max().item(), name
