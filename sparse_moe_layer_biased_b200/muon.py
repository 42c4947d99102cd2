"""Orthogonalizer: orthogonalised updates of a stack of weight matrices (the Muon optimiser's rule).

For the layer's expert weights, whose fp32 gradients moe_backward writes: dW_gate_up [E, 2I, H] is a
stack of 2E matrices [I, H] (gate and up are separate matrices), dW_down [E, H, I] one of E:

    muon = Orthogonalizer(2 * E, I, H, scale=..., beta=0.95, nesterov=True)
    update = muon.orthogonalize(dW_gate_up.view(2 * E, I, H), momentum=m)    # bf16; m updated in place
    W_gate_up.view(2 * E, I, H).sub_(lr * update)

PyTorch only allocates device memory and supplies the stream; the arithmetic runs in libmoe_b200.so.
"""
from __future__ import annotations

import ctypes

import torch

from . import _abi
from .tokens import Caller, check_tensor


def _orthogonalize(desc, stream, *args) -> int:
    return _abi.lib().moe_orthogonalize(desc, *args, stream)


class Orthogonalizer(Caller):
    """n matrices [rows, cols]: u = grad, or with momentum m <- beta m + grad and u = grad + beta m
    (nesterov) or m; X = u / (|u|_F + eps); `steps` times X <- a X + (b A + c A A) X with A = X X^T
    (of the shorter side), coeffs = (a, b, c); the update is bf16(scale X). Autograd does not record it.

    The workspace (up to 2 GiB, more if one matrix needs it, none to speak of for sides up to 128 x 2048) serves one call at a time: calls
    that may overlap on the GPU (two streams, two graphs replayed at once) need an Orthogonalizer
    each. It belongs to the stream that was current when the Orthogonalizer was made, which outlives its calls in flight
    on other streams and the graphs captured from it."""

    def __init__(self, n: int, rows: int, cols: int, grad_dtype: torch.dtype = torch.float32, steps: int = 5,
                 coeffs=(3.4445, -4.7750, 2.0315), eps: float = 1e-7, scale: float = 1.0, beta: float = 0.95,
                 nesterov: bool = True, device="cuda"):
        if grad_dtype not in _abi.DTYPES:
            raise ValueError(f"gradients of {grad_dtype} are not supported")
        self.shape, self.grad_dtype = (n, rows, cols), grad_dtype
        self.desc = _abi.OrthogonalizeDesc(n, rows, cols, _abi.DTYPES[grad_dtype], steps, *coeffs, eps, scale, beta,
                                           int(bool(nesterov)))
        nbytes = _abi.moe_orthogonalize_workspace_size(self.desc)
        super().__init__(device)
        self.ws = torch.empty(nbytes, dtype=torch.uint8, device=device)

    def orthogonalize(self, grad: torch.Tensor, momentum: torch.Tensor | None = None, out: torch.Tensor | None = None,
                      stream=None) -> torch.Tensor:
        """grad [n, rows, cols] of grad_dtype, momentum [n, rows, cols] fp32 (updated in place) or
        None -> the update [n, rows, cols] bf16, in `out` if given (else allocated on the stream that the call runs on).
        Runs on the current stream of the tensors' device, or on `stream`."""
        check_tensor(grad, "grad", self.shape, self.grad_dtype, self._dev)
        if momentum is not None:
            check_tensor(momentum, "momentum", self.shape, torch.float32, self._dev)
        if out is None:
            with _abi._allocating_on(stream, self.device):
                out = torch.empty(self.shape, dtype=torch.bfloat16, device=self.device)
        check_tensor(out, "out", self.shape, torch.bfloat16, self._dev)
        status = self._call(_orthogonalize, stream, ctypes.byref(self.desc), grad.data_ptr(),
                            None if momentum is None else momentum.data_ptr(), out.data_ptr(), self.ws.data_ptr(),
                            self.ws.numel())
        if status < 0:
            raise ValueError("moe_orthogonalize: tensors in the memory of a CUDA device are wanted")
        if status:
            raise _abi.MoeError("moe_orthogonalize", status)
        return out
