"""Sizes that do not fit the library's 32 bits are refused by the binding, not cut (no GPU, no memory behind them)."""
import pytest
import torch

import linear_attention_recurrence_06_b200 as kda

BIG = (1 << 32) + 2  # 2 when cut to 32 bits


class Cuda(torch.Tensor):  # a host tensor that says it is on a GPU
    is_cuda = True


def of(*shape, dtype=torch.float32):
    return torch.zeros([1] * len(shape), dtype=dtype).expand(*shape).as_subclass(Cuda)


def refused(call):
    with pytest.raises(kda.KdaError) as e:
        call()
    assert e.value.status == -2


@pytest.mark.parametrize("shape", [(BIG, 1, 1), (1, 1, BIG), (1, 1, 1 << 16, 1 << 16)])
def test_scan(shape):
    x = of(*shape)
    refused(lambda: kda.scan_fwd(x, x))
    refused(lambda: kda.scan_bwd(x, x, x))


def test_workspace_and_lists():
    refused(lambda: kda.scan_bwd_workspace_size(BIG, 1, 8))
    refused(lambda: kda.scan_bwd_workspace_size(1, 1, BIG))
    x, slots = of(1, 4, 8), of(BIG, dtype=torch.int32)
    refused(lambda: kda.scan_fwd(x, x, cu_seqlens=slots))
    refused(lambda: kda.state_copy(of(4, 8), slots, None, slots))
    live = torch.zeros(8, dtype=torch.uint8).as_subclass(Cuda)
    refused(lambda: kda.state_alloc(live, BIG))
    refused(lambda: kda.state_free(live, slots))
