"""TokenSorter and Orthogonalizer on the host with a stream given: refused as without one (nothing asks for a device)."""
import pytest
import torch

import sparse_moe_layer_biased_b200 as moe


@pytest.mark.parametrize("stream", [None, 0, 1 << 40])
def test_host_tensors_with_a_stream(stream):
    s = moe.TokenSorter(8, 16, 4, 2, dtype=torch.float32, device="cpu")
    o = moe.Orthogonalizer(2, 8, 16, device="cpu")
    x, idx, rows = torch.zeros(8, 16), torch.zeros(8, 2, dtype=torch.int32), torch.zeros(16, 16)
    for call in (lambda: s.sort(x, idx, stream=stream), lambda: s.sort_backward(rows, idx, stream=stream),
                 lambda: s.unsort(rows, idx, add=x, stream=stream), lambda: s.unsort_backward(x, rows, idx, stream=stream),
                 lambda: o.orthogonalize(torch.zeros(2, 8, 16), stream=stream)):
        with pytest.raises(ValueError, match="CUDA device"):
            call()
    with pytest.raises(ValueError, match="topk_idx"):
        s.sort(x, idx.long(), stream=stream)
