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

PyTorch only allocates device memory and supplies the stream; the arithmetic runs in libmoe_b200.so.
"""
from __future__ import annotations

import ctypes

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
    """Calls of the library for tensors of one device, with little host time: a small call's kernel is
    over in 3 us, and a call through _abi's functions costs 2 us more than this."""

    def __init__(self, device):
        self._dev = device_index(device)
        self.device = torch.device("cpu") if self._dev < 0 else torch.device("cuda", self._dev)
        self._several = torch.cuda.device_count() > 1

    def _run(self, fn, stream, *args) -> None:
        """fn(*args, stream handle) with the device current, on `stream` or the device's current stream."""
        if self._several and torch.cuda.current_device() != self._dev:
            with torch.cuda.device(self._dev):
                return self._run(fn, stream, *args)
        status = fn(*args, _abi._raw_stream(self._dev) if stream is None else _abi._stream(stream))
        if status:
            raise _abi.MoeError(fn.__name__, status)


class TokenSorter(Caller):
    """Sorts rows [T, H] of `dtype` (bf16, fp16 or fp32) of up to max_tokens tokens with k
    entries each over E experts. An entry whose id is outside [0, E) is dropped: it has no row, adds
    nothing and gets no gradient (a padded token; with expert parallelism an expert held
    elsewhere, so k may exceed E).

    Every method runs on the current stream of the tensors' device, or on `stream`. `out` gives
    the results' tensors, else they are allocated on the current stream; rows of a sorted array that no
    entry owns are not written. The sorter's workspace serves one sort at a time: sorts that may overlap on
    the GPU (two streams, two graphs replayed at once) need a sorter each, and a sorter outlives the
    graphs captured from it."""

    def __init__(self, max_tokens: int, H: int, E: int, k: int, dtype: torch.dtype = torch.bfloat16, device="cuda"):
        if dtype not in _abi.DTYPES:
            raise ValueError(f"rows of {dtype} are not supported")
        self.max_tokens, self.H, self.E, self.k, self.dtype = max_tokens, H, E, k, dtype
        super().__init__(device)
        nbytes = _abi.moe_sort_workspace_size(self._desc(max_tokens))
        self.ws = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
        self._last = (-1, None)  # the latest call's token count, and its descriptor by reference
        self._lib = _abi.lib()

    def _desc(self, T: int) -> _abi.TokenDesc:
        return _abi.TokenDesc(T, self.H, self.E, self.k, _abi.DTYPES[self.dtype])

    def _ref(self, T: int):
        last = self._last
        if last[0] != T:
            last = self._last = (T, ctypes.byref(self._desc(T)))
        return last[1]

    def sort(self, x: torch.Tensor, topk_idx: torch.Tensor, out=None, stream=None):
        """x [T, H], topk_idx [T, k] int32 -> (x_sorted [T*k, H], offsets [E+1], slot_of [T, k] int32)."""
        T, H, k, dt, dev = x.shape[0], self.H, self.k, self.dtype, self._dev
        check_tensor(x, "x", (T, H), dt, dev)
        check_tensor(topk_idx, "topk_idx", (T, k), torch.int32, dev)
        if T > self.max_tokens:
            raise ValueError(f"{T} tokens exceed the workspace size of {self.max_tokens}")
        if out is None:
            out = (torch.empty((T * k, H), dtype=dt, device=self.device),
                   torch.empty(self.E + 1, dtype=torch.int32, device=self.device),
                   torch.empty((T, k), dtype=torch.int32, device=self.device))
        x_sorted, offsets, slot_of = out
        check_tensor(x_sorted, "x_sorted", (T * k, H), dt, dev)
        check_tensor(offsets, "offsets", (self.E + 1,), torch.int32, dev)
        check_tensor(slot_of, "slot_of", (T, k), torch.int32, dev)
        self._run(self._lib.moe_sort_tokens, stream, self._ref(T), x.data_ptr(), topk_idx.data_ptr(), x_sorted.data_ptr(),
                  offsets.data_ptr(), slot_of.data_ptr(), self.ws.data_ptr(), self.ws.numel())
        return out

    def sort_backward(self, dx_sorted: torch.Tensor, slot_of: torch.Tensor, out=None, stream=None):
        """dx_sorted [T*k, H] -> dx [T, H], the sum of each token's rows."""
        T, H, dt, dev = slot_of.shape[0], self.H, self.dtype, self._dev
        check_tensor(slot_of, "slot_of", (T, self.k), torch.int32, dev)
        check_tensor(dx_sorted, "dx_sorted", (T * self.k, H), dt, dev)
        if out is None:
            out = torch.empty((T, H), dtype=dt, device=self.device)
        check_tensor(out, "dx", (T, H), dt, dev)
        self._run(self._lib.moe_sort_tokens_backward, stream, self._ref(T), dx_sorted.data_ptr(), slot_of.data_ptr(),
                  out.data_ptr())
        return out

    def unsort(self, y_sorted: torch.Tensor, slot_of: torch.Tensor, topk_w=None, add=None, out=None, stream=None):
        """y_sorted [T*k, H] -> y [T, H]: each token's rows weighted by topk_w [T, k] fp32 (None: 1)
        and summed, plus add [T, H] (None: 0)."""
        T, H, dt, dev = slot_of.shape[0], self.H, self.dtype, self._dev
        check_tensor(slot_of, "slot_of", (T, self.k), torch.int32, dev)
        check_tensor(y_sorted, "y_sorted", (T * self.k, H), dt, dev)
        if topk_w is not None:
            check_tensor(topk_w, "topk_w", (T, self.k), torch.float32, dev)
        if add is not None:
            check_tensor(add, "add", (T, H), dt, dev)
        if out is None:
            out = torch.empty((T, H), dtype=dt, device=self.device)
        check_tensor(out, "y", (T, H), dt, dev)
        self._run(self._lib.moe_unsort_tokens, stream, self._ref(T), y_sorted.data_ptr(), slot_of.data_ptr(),
                  None if topk_w is None else topk_w.data_ptr(), None if add is None else add.data_ptr(), out.data_ptr())
        return out

    def unsort_backward(self, dy: torch.Tensor, y_sorted: torch.Tensor, slot_of: torch.Tensor, topk_w=None, out=None,
                        stream=None):
        """dy [T, H] -> (dy_sorted [T*k, H], dtopk_w [T, k] fp32). The gradient of unsort's `add` is dy."""
        T, H, k, dt, dev = slot_of.shape[0], self.H, self.k, self.dtype, self._dev
        check_tensor(slot_of, "slot_of", (T, k), torch.int32, dev)
        check_tensor(dy, "dy", (T, H), dt, dev)
        check_tensor(y_sorted, "y_sorted", (T * k, H), dt, dev)
        if topk_w is not None:
            check_tensor(topk_w, "topk_w", (T, k), torch.float32, dev)
        if out is None:
            out = (torch.empty((T * k, H), dtype=dt, device=self.device),
                   torch.empty((T, k), dtype=torch.float32, device=self.device))
        dy_sorted, dtopk_w = out
        check_tensor(dy_sorted, "dy_sorted", (T * k, H), dt, dev)
        check_tensor(dtopk_w, "dtopk_w", (T, k), torch.float32, dev)
        self._run(self._lib.moe_unsort_tokens_backward, stream, self._ref(T), dy.data_ptr(), y_sorted.data_ptr(),
                  slot_of.data_ptr(), None if topk_w is None else topk_w.data_ptr(), dy_sorted.data_ptr(),
                  dtopk_w.data_ptr())
        return out
