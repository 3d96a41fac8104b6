"""The backward's reverse walk waits for every consumer's part of its operands: gradients do not depend on what ran on an
SM before or on how the consumers' loads are staggered."""
import pytest

import oracle
from kda_testutil import D, assert_rel_l2, dev, host, make_prefill
from linear_attention_recurrence_06_b200 import synth

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [6, 65, 70, 90, 127, 128, 134])
@pytest.mark.parametrize("bf16", [True, False])
def test_backward_gives_the_same_back_to_back(T, bf16):
    """Every call against the first, with large products in between that leave other data in shared memory."""
    import torch
    import linear_attention_recurrence_06_b200 as kda
    H = 2
    d = make_prefill(77, [T], H, bf16=bf16)
    dt = torch.bfloat16 if bf16 else torch.float32
    up = lambda x, *s: dev(x, dt).view(1, T, H, *s)  # noqa: E731
    args = [up(d[k], D) for k in ("q", "k", "v", "log_alpha")] + [up(d["beta"])]
    dy = synth.normal(78, synth.TAG_V, (T, H, D), 1.0, bf16)
    d_o = up(dy, D)
    big = torch.randn(4096, 4096, device="cuda")
    first = kda.chunk_bwd(*args, d_o)
    ref = oracle.kda_recurrent_bwd(d["q"], d["k"], d["v"], d["log_alpha"], d["beta"], dy, None, None, d["cu"])
    for name in ("dq", "dk", "dv", "dlog_alpha"):
        assert_rel_l2(host(first[name]).reshape(T, H, D), ref[name].reshape(T, H, D), name)
    for _ in range(8):
        big @ big
        got = kda.chunk_bwd(*args, d_o)
        for name in ("dq", "dk", "dv", "dlog_alpha", "d_initial_state"):
            assert torch.equal(got[name], first[name]), name
