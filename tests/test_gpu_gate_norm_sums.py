"""The gate norm's weight gradient and its ends: sums over more rows than one turn of the kernel's loop, eps = 0, gates
next to open (tests/scan_ref.py derives the bounds that are not derived here)."""
import pytest
import torch

import linear_attention_recurrence_06_b200 as kda
import scan_ref
from test_gpu_gate_norm_bwd import check, inputs

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows", [1, 3, 15, 301, 9473])
def test_eps_of_zero(dtype, rows):
    """Rows that no half warp has beside it: 1 / sqrt(0 + 0) of nothing must not reach the weight's sum."""
    o, ga, dy, w = inputs(rows + 100, rows, dtype)
    check(o, ga, dy, w, kda.gate_norm_bwd(o, ga, dy, w, eps=0.0), eps=0.0)
