"""The training operators together, as a training step uses them: route, sort, experts, unsort; the gradients
back; the experts' weight gradients into updates. The layer's own forward and backward give the values to meet.

Tolerance: the layer's (relative Frobenius error 1e-2): both sides round rows to bf16 in several places."""
import pytest
import torch

import sparse_moe_layer_biased_b200 as moe
from sparse_moe_layer_biased_b200 import _abi
from sparse_moe_layer_biased_b200.inputs import LayerShape, draw
from sparse_moe_layer_biased_b200.layer import MoeLayer

pytestmark = pytest.mark.gpu


def rel(a, b):
    return ((a.double() - b.double()).norm() / b.double().norm()).item()


@pytest.mark.parametrize("T", [48, 700])
def test_a_training_step(T):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    sh = LayerShape("train", T=T, H=256, E=16, k=4, I=128, Is=128, seed=31, weight_std=0.05)
    inp = {k: v.cuda() for k, v in draw(sh).items()}
    x, E, I, H = inp["x"], sh.E, sh.I, sh.H
    y_layer, idx, w = MoeLayer(sh, inp).forward(x, routing=True)
    d = _abi.desc_of(sh)

    sorter = moe.TokenSorter(T, H, E, sh.k)
    x_sorted, offsets, slot_of = sorter.sort(x, idx)
    wgu = [inp["W_gate_up"][e].float().requires_grad_() for e in range(E)]
    wd = [inp["W_down"][e].float().requires_grad_() for e in range(E)]
    rows = x_sorted.float().requires_grad_()

    def expert(h, gu, down):
        a = h @ gu.t()
        return (torch.nn.functional.silu(a[:, :gu.shape[0] // 2]) * a[:, gu.shape[0] // 2:]) @ down.t()

    off = offsets.tolist()
    out = torch.cat([expert(rows[off[e]:off[e + 1]], wgu[e], wd[e]) for e in range(E)])
    shared = expert(x.float(), inp["Wsh_gate_up"].float(), inp["Wsh_down"].float()).bfloat16()
    y_sorted = out.detach().bfloat16()
    y = sorter.unsort(y_sorted, slot_of, w, add=shared)
    assert rel(y, y_layer) < 1e-2

    dy = torch.randn((T, H), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    dy_sorted, dw = sorter.unsort_backward(dy.bfloat16(), y_sorted, slot_of, w)
    out.backward(dy_sorted.float())
    dx = sorter.sort_backward(rows.grad.bfloat16(), slot_of)

    # the layer's backward: weight gradients, and dx less the router's and the shared expert's parts
    g = {n: torch.empty(inp[n].shape, device="cuda") for n in ("Wr", "W_gate_up", "W_down", "Wsh_gate_up", "Wsh_down")}
    dx_layer = torch.empty((T, H), device="cuda")
    ws = torch.empty(_abi.moe_backward_workspace_size(d), dtype=torch.uint8, device="cuda")
    _abi.moe_backward(d, x, inp["Wr"], inp["W_gate_up"], inp["W_down"], inp["Wsh_gate_up"], inp["Wsh_down"], idx, w, dy,
                      dx_layer, g["Wr"], g["W_gate_up"], g["W_down"], g["Wsh_gate_up"], g["Wsh_down"], ws)
    assert rel(torch.stack([t.grad if t.grad is not None else torch.zeros_like(t) for t in wgu]), g["W_gate_up"]) < 2e-2
    assert rel(torch.stack([t.grad if t.grad is not None else torch.zeros_like(t) for t in wd]), g["W_down"]) < 2e-2
    xs = x.float().requires_grad_()
    expert(xs, inp["Wsh_gate_up"].float(), inp["Wsh_down"].float()).backward(dy)
    logits = x.float() @ inp["Wr"].float().t()
    s = torch.sigmoid(logits.gather(1, idx.long())).requires_grad_()
    (sh.scale * s / s.sum(1, keepdim=True)).backward(dw)
    dlogit = s.grad * s.detach() * (1 - s.detach())
    dx_router = torch.einsum("tk,tkh->th", dlogit, inp["Wr"].float()[idx.long()])
    assert rel(dx.float() + xs.grad + dx_router, dx_layer) < 2e-2
    dwr = torch.zeros_like(g["Wr"]).index_put_((idx.long().flatten(),), (dlogit[:, :, None] * x.float()[:, None]).view(-1, H),
                                               accumulate=True)
    assert rel(dwr, g["Wr"]) < 2e-2

    # and the update of the experts' weights: singular values of matrices with gradients end near one
    muon = moe.Orthogonalizer(2 * E, I, H)
    m = torch.zeros((2 * E, I, H), device="cuda")
    update = muon.orthogonalize(g["W_gate_up"].view(2 * E, I, H), momentum=m)
    assert torch.equal(m, g["W_gate_up"].view(2 * E, I, H))
    counts = (offsets[1:] - offsets[:-1]).tolist()
    top = torch.linalg.matrix_norm(update.float(), ord=2)
    for e in range(E):
        for half in range(2):
            v = top[2 * e + half].item()
            assert 0.6 < v < 1.3 if counts[e] else v == 0.0
    # applied to bf16 weights: off by half a step (2^-8) of the step taken and of the weight it ends at, no
    # smaller a bound holds, since a step of 1e-4 is itself less than half a step of a weight of 0.05
    before = inp["W_gate_up"].double()
    inp["W_gate_up"].view(2 * E, I, H).sub_(0.01 * update)
    step = 0.01 * update.double().view(E, 2 * I, H)
    after = inp["W_gate_up"].double()
    assert bool(((after - (before - step)).abs() <= 2.0**-8 * (after.abs() + step.abs())).all())


@pytest.mark.parametrize("n,rows,cols", [(40, 100, 700), (20, 200, 600), (4, 1280, 1536)])
def test_short_wait_limit_reports_timeout_and_recovers(n, rows, cols):
    """The waits of the cluster form, of single CTAs and of CTA pairs run out without a hang."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    o = moe.Orthogonalizer(n, rows, cols)
    g = torch.randn((n, rows, cols), device="cuda")
    want = o.orthogonalize(g).clone()
    _abi.moe_check_device()
    flush = torch.empty(64 << 20, dtype=torch.float32, device="cuda")  # 256 MB > L2
    statuses = []
    old = _abi.moe_set_wait_limit_ns(1000)
    try:
        for _ in range(4):
            flush.fill_(1.0)
            o.orthogonalize(g)
            try:
                _abi.moe_check_device()
                statuses.append("ok")
            except _abi.MoeError as e:
                assert e.status == 5, e
                statuses.append("timeout")
    finally:
        _abi.moe_set_wait_limit_ns(old)
    assert set(statuses) <= {"ok", "timeout"}
    assert torch.equal(o.orthogonalize(g), want)
    _abi.moe_check_device()
