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

import torch

from . import _abi


def check_tensor(t, name: str, shape, dtype, device) -> None:
    """ValueError unless t is a contiguous tensor of this shape, type and device."""
    if t.shape != shape or t.dtype is not dtype or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous {dtype} tensor of shape {tuple(shape)} on {device} is wanted, got "
                         f"{t.dtype} {tuple(t.shape)} on {t.device}"
                         f"{'' if t.is_contiguous() else ' (not contiguous)'}")


class TokenSorter:
    """Sorts rows [T, H] of `dtype` (bf16, fp16 or fp32) of up to max_tokens tokens with k
    entries each over E experts. An entry whose id is outside [0, E) is dropped: it has no row, adds
    nothing and gets no gradient (a padded token; with expert parallelism an expert held
    elsewhere, so k may exceed E).

    Every method runs on the current stream of the tensors' device, or on `stream`. `out` gives
    the results' tensors, else they are allocated; rows of a sorted array that no entry owns are
    not written. The sorter's workspace serves one sort at a time: sorts that may overlap on
    the GPU (two streams, two graphs replayed at once) need a sorter each, and a sorter outlives the
    graphs captured from it."""

    def __init__(self, max_tokens: int, H: int, E: int, k: int, dtype: torch.dtype = torch.bfloat16, device="cuda"):
        if dtype not in _abi.DTYPES:
            raise ValueError(f"rows of {dtype} are not supported")
        self.max_tokens, self.H, self.E, self.k, self.dtype = max_tokens, H, E, k, dtype
        self._code = _abi.DTYPES[dtype]
        self._last = None  # the latest call's descriptor
        nbytes = _abi.moe_sort_workspace_size(self._desc(max_tokens))
        device = torch.device(device)
        if device.type == "cuda" and device.index is None:
            device = torch.device("cuda", torch.cuda.current_device())
        self.device = device
        self.ws = torch.empty(nbytes, dtype=torch.uint8, device=device)

    def _desc(self, T: int) -> _abi.TokenDesc:
        d = self._last
        if d is None or d.T != T:
            d = self._last = _abi.TokenDesc(T, self.H, self.E, self.k, self._code)
        return d

    def _rows(self, t: torch.Tensor, name: str, rows: int) -> None:
        check_tensor(t, name, (rows, self.H), self.dtype, self.device)

    def _table(self, t: torch.Tensor, name: str, dtype, T=None) -> int:
        if T is None:
            T = t.shape[0] if t.dim() == 2 else -1
        check_tensor(t, name, (T, self.k), dtype, self.device)
        return T

    def _call(self, fn, *args, stream=None):
        if torch.cuda.current_device() == self.device.index:
            fn(*args, stream=stream)
        else:
            with torch.cuda.device(self.device):
                fn(*args, stream=stream)

    def sort(self, x: torch.Tensor, topk_idx: torch.Tensor, out=None, stream=None):
        """x [T, H], topk_idx [T, k] int32 -> (x_sorted [T*k, H], offsets [E+1], slot_of [T, k] int32)."""
        T, dev = self._table(topk_idx, "topk_idx", torch.int32), self.device
        if T > self.max_tokens:
            raise ValueError(f"{T} tokens exceed the workspace size of {self.max_tokens}")
        self._rows(x, "x", T)
        if out is None:
            out = (torch.empty((T * self.k, self.H), dtype=self.dtype, device=dev),
                   torch.empty(self.E + 1, dtype=torch.int32, device=dev),
                   torch.empty((T, self.k), dtype=torch.int32, device=dev))
        x_sorted, offsets, slot_of = out
        self._rows(x_sorted, "x_sorted", T * self.k)
        check_tensor(offsets, "offsets", (self.E + 1,), torch.int32, dev)
        self._table(slot_of, "slot_of", torch.int32, T)
        self._call(_abi.moe_sort_tokens, self._desc(T), x, topk_idx, x_sorted, offsets, slot_of, self.ws,
                   stream=stream)
        return out

    def sort_backward(self, dx_sorted: torch.Tensor, slot_of: torch.Tensor, out=None, stream=None):
        """dx_sorted [T*k, H] -> dx [T, H], the sum of each token's rows."""
        T = self._table(slot_of, "slot_of", torch.int32)
        self._rows(dx_sorted, "dx_sorted", T * self.k)
        if out is None:
            out = torch.empty((T, self.H), dtype=self.dtype, device=self.device)
        self._rows(out, "dx", T)
        self._call(_abi.moe_sort_tokens_backward, self._desc(T), dx_sorted, slot_of, out, stream=stream)
        return out

    def unsort(self, y_sorted: torch.Tensor, slot_of: torch.Tensor, topk_w=None, add=None, out=None, stream=None):
        """y_sorted [T*k, H] -> y [T, H]: each token's rows weighted by topk_w [T, k] fp32 (None: 1)
        and summed, plus add [T, H] (None: 0)."""
        T = self._table(slot_of, "slot_of", torch.int32)
        self._rows(y_sorted, "y_sorted", T * self.k)
        if topk_w is not None:
            self._table(topk_w, "topk_w", torch.float32, T)
        if add is not None:
            self._rows(add, "add", T)
        if out is None:
            out = torch.empty((T, self.H), dtype=self.dtype, device=self.device)
        self._rows(out, "y", T)
        self._call(_abi.moe_unsort_tokens, self._desc(T), y_sorted, slot_of, topk_w, add, out, stream=stream)
        return out

    def unsort_backward(self, dy: torch.Tensor, y_sorted: torch.Tensor, slot_of: torch.Tensor, topk_w=None, out=None,
                        stream=None):
        """dy [T, H] -> (dy_sorted [T*k, H], dtopk_w [T, k] fp32). The gradient of unsort's `add` is dy."""
        T = self._table(slot_of, "slot_of", torch.int32)
        self._rows(dy, "dy", T)
        self._rows(y_sorted, "y_sorted", T * self.k)
        if topk_w is not None:
            self._table(topk_w, "topk_w", torch.float32, T)
        if out is None:
            out = (torch.empty((T * self.k, self.H), dtype=self.dtype, device=self.device),
                   torch.empty((T, self.k), dtype=torch.float32, device=self.device))
        dy_sorted, dtopk_w = out
        self._rows(dy_sorted, "dy_sorted", T * self.k)
        self._table(dtopk_w, "dtopk_w", torch.float32, T)
        self._call(_abi.moe_unsort_tokens_backward, self._desc(T), dy, y_sorted, slot_of, topk_w, dy_sorted, dtopk_w,
                   stream=stream)
        return out
