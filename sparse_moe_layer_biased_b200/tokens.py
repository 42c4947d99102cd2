"""TokenSorter: token rows sorted by expert and back, with the gradients of both.

The differentiable form of an expert-parallel dispatch and return, for training: EPMoeLayer's
moe_ep_pack and moe_combine are its forward-only counterparts inside the layer. A training step of a
layer whose experts are computed elsewhere:

    x_sorted, offsets, slot_of = sorter.sort(x, topk_idx)      # expert e: rows offsets[e]:offsets[e+1]
    y_sorted = experts(x_sorted, offsets)
    y = sorter.unsort(y_sorted, slot_of, topk_w, add=shared)
    ...
    dy_sorted, dtopk_w = sorter.unsort_backward(dy, y_sorted, slot_of, topk_w)   # dshared = dy
    dx_sorted = experts_backward(dy_sorted, offsets)
    dx = sorter.sort_backward(dx_sorted, slot_of)

Autograd does not record these calls: inside torch.autograd.Function (or under torch.no_grad()) they take any tensor,
while autograd is recording they refuse one that requires a gradient.

PyTorch only allocates device memory and supplies the stream; the arithmetic runs in libmoe_b200.so. A small call's
kernel is over in 2.5 us, so the extension module _calls checks the tensors and makes the call: 3 us of host time, of which
the launch takes 2.3; the checks in Python and ctypes took 6.5.
"""
from __future__ import annotations

import torch

from . import _abi


def check_tensor(t, name: str, shape, dtype, index) -> None:
    """ValueError unless t is a contiguous tensor of this shape and type on CUDA device `index` (-1: the host)."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous {dtype} tensor of shape {tuple(shape)} on "
                         f"{'the host' if index < 0 else f'cuda:{index}'} is wanted, got {t.dtype} {tuple(t.shape)} on "
                         f"{t.device}{'' if t.is_contiguous() else ' (not contiguous)'}")


def device_index(device) -> int:
    """Index of a CUDA device (the current one if `device` names none), -1 for the host."""
    device = torch.device(device)
    if device.type != "cuda":
        return -1
    return torch.cuda.current_device() if device.index is None else device.index


class Caller:
    """Calls of the library for tensors of one device."""

    def __init__(self, device):
        self._dev = device_index(device)
        self.device = torch.device("cpu") if self._dev < 0 else torch.device("cuda", self._dev)
        self._several = torch.cuda.device_count() > 1

    def _call(self, fn, stream, plan, *args) -> int:
        """Status of fn(plan, stream handle, *args) with the device current, on `stream` or the device's current stream;
        -1 on the host."""
        if self._dev < 0:
            return -1
        if self._several and torch.cuda.current_device() != self._dev:
            with torch.cuda.device(self._dev):
                return self._call(fn, stream, plan, *args)
        return fn(plan, _abi._raw_stream(self._dev) if stream is None else _abi._stream(stream), *args)


class TokenSorter(Caller):
    """Sorts rows [T, H] of `dtype` (bf16, fp16 or fp32) of up to max_tokens tokens with k
    entries each over E experts. An entry whose id is outside [0, E) is dropped: it has no row, adds
    nothing and gets no gradient (a padded token; with expert parallelism an expert held
    elsewhere, so k may exceed E).

    Every method runs on the current stream of the tensors' device, or on `stream`. `out` gives
    the results' tensors, else they are allocated on the stream that the method runs on; rows of a sorted array
    that no entry owns are not written. The sorter's workspace serves one sort at a time: sorts that may overlap on
    the GPU (two streams, two graphs replayed at once) need a sorter each. It belongs to the stream that was current
    when the sorter was made: a sorter outlives its sorts in flight on other streams and the graphs captured from it."""

    def __init__(self, max_tokens: int, H: int, E: int, k: int, dtype: torch.dtype = torch.bfloat16, device="cuda"):
        if dtype not in _abi.DTYPES:
            raise ValueError(f"rows of {dtype} are not supported")
        self.max_tokens, self.H, self.E, self.k, self.dtype = max_tokens, H, E, k, dtype
        super().__init__(device)
        nbytes = _abi.moe_sort_workspace_size(self._desc(max_tokens))
        self.ws = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
        self._spec = (max_tokens, H, E, k, _abi.DTYPES[dtype], self._dev, self.ws.data_ptr(), nbytes)
        self._calls = _abi.calls()

    def _desc(self, T: int) -> _abi.TokenDesc:
        return _abi.TokenDesc(T, self.H, self.E, self.k, _abi.DTYPES[self.dtype])

    def _refuse(self, name: str, status: int, wanted, sorted_tokens: int = 0) -> None:
        """The error of a call: for status -1 that of the tensor which is not as wanted, (tensor, name, shape, dtype); for -2
        that of the one which requires a gradient."""
        if status == -2:
            names = ", ".join(what for tensor, what, _, _ in wanted if tensor is not None and tensor.requires_grad)
            raise ValueError(f"{name}: {names}: requires a gradient, but autograd does not record this call; make it inside "
                             "torch.autograd.Function or under torch.no_grad(), and take gradients with the _backward methods")
        if status < 0:
            for tensor, what, shape, dtype in wanted:
                if tensor is not None:
                    check_tensor(tensor, what, shape, dtype, self._dev)
            if sorted_tokens > self.max_tokens:
                raise ValueError(f"{sorted_tokens} tokens exceed the workspace size of {self.max_tokens}")
            raise ValueError(f"{name}: tensors in the memory of a CUDA device are wanted")
        raise _abi.MoeError(name, status)

    def sort(self, x: torch.Tensor, topk_idx: torch.Tensor, out=None, stream=None):
        """x [T, H], topk_idx [T, k] int32 -> (x_sorted [T*k, H], offsets [E+1], slot_of [T, k] int32)."""
        T, H, k, dt = x.shape[0], self.H, self.k, self.dtype
        if out is None:
            with _abi._allocating_on(stream, self.device):
                out = (torch.empty((T * k, H), dtype=dt, device=self.device),
                       torch.empty(self.E + 1, dtype=torch.int32, device=self.device),
                       torch.empty((T, k), dtype=torch.int32, device=self.device))
        x_sorted, offsets, slot_of = out
        status = self._call(self._calls.sort, stream, self._spec, x, topk_idx, x_sorted, offsets, slot_of)
        if status:
            self._refuse("moe_sort_tokens", status, (
                (x, "x", (T, H), dt), (topk_idx, "topk_idx", (T, k), torch.int32), (x_sorted, "x_sorted", (T * k, H), dt),
                (offsets, "offsets", (self.E + 1,), torch.int32), (slot_of, "slot_of", (T, k), torch.int32)), T)
        return out

    def sort_backward(self, dx_sorted: torch.Tensor, slot_of: torch.Tensor, out=None, stream=None):
        """dx_sorted [T*k, H] -> dx [T, H], the sum of each token's rows."""
        T, H, k, dt = slot_of.shape[0], self.H, self.k, self.dtype
        if out is None:
            with _abi._allocating_on(stream, self.device):
                out = torch.empty((T, H), dtype=dt, device=self.device)
        status = self._call(self._calls.sort_backward, stream, self._spec, dx_sorted, slot_of, out)
        if status:
            self._refuse("moe_sort_tokens_backward", status, (
                (slot_of, "slot_of", (T, k), torch.int32), (dx_sorted, "dx_sorted", (T * k, H), dt), (out, "dx", (T, H), dt)))
        return out

    def unsort(self, y_sorted: torch.Tensor, slot_of: torch.Tensor, topk_w=None, add=None, out=None, stream=None):
        """y_sorted [T*k, H] -> y [T, H]: each token's rows weighted by topk_w [T, k] fp32 (None: 1)
        and summed, plus add [T, H] (None: 0)."""
        T, H, k, dt = slot_of.shape[0], self.H, self.k, self.dtype
        if out is None:
            with _abi._allocating_on(stream, self.device):
                out = torch.empty((T, H), dtype=dt, device=self.device)
        status = self._call(self._calls.unsort, stream, self._spec, y_sorted, slot_of, topk_w, add, out)
        if status:
            self._refuse("moe_unsort_tokens", status, (
                (slot_of, "slot_of", (T, k), torch.int32), (y_sorted, "y_sorted", (T * k, H), dt),
                (topk_w, "topk_w", (T, k), torch.float32), (add, "add", (T, H), dt), (out, "y", (T, H), dt)))
        return out

    def unsort_backward(self, dy: torch.Tensor, y_sorted: torch.Tensor, slot_of: torch.Tensor, topk_w=None, out=None,
                        stream=None):
        """dy [T, H] -> (dy_sorted [T*k, H], dtopk_w [T, k] fp32). The gradient of unsort's `add` is dy."""
        T, H, k, dt = slot_of.shape[0], self.H, self.k, self.dtype
        if out is None:
            with _abi._allocating_on(stream, self.device):
                out = (torch.empty((T * k, H), dtype=dt, device=self.device),
                       torch.empty((T, k), dtype=torch.float32, device=self.device))
        dy_sorted, dtopk_w = out
        status = self._call(self._calls.unsort_backward, stream, self._spec, dy, y_sorted, slot_of, topk_w, dy_sorted,
                            dtopk_w)
        if status:
            self._refuse("moe_unsort_tokens_backward", status, (
                (slot_of, "slot_of", (T, k), torch.int32), (dy, "dy", (T, H), dt), (y_sorted, "y_sorted", (T * k, H), dt),
                (topk_w, "topk_w", (T, k), torch.float32), (dy_sorted, "dy_sorted", (T * k, H), dt),
                (dtopk_w, "dtopk_w", (T, k), torch.float32)))
        return out
