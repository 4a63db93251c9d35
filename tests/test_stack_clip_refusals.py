"""stack_bwd(max_norm=...) refuses a norm that the clip would refuse before it
has consumed anything: the same state then serves a call with a good one."""
import math

import pytest
import torch

import blockwise_attention_ffn_gb300 as bpt
from blockwise_attention_ffn_gb300 import stack
from tests.test_stack_schedule import CFG, OracleOps, _stack


@pytest.fixture(scope="module", autouse=True)
def lib():
    from blockwise_attention_ffn_gb300 import build
    build.build()


@pytest.mark.parametrize("bad", [0.0, -1.0, math.nan, -math.inf, 1e-60])
def test_a_bad_norm_leaves_the_state_whole(bad):
    x, Ws, dy = _stack(3)
    ops = OracleOps()
    y, st = stack.stack_fwd(CFG, Ws, torch.from_numpy(x), 2, ops=ops)
    with pytest.raises(bpt.BptError) as e:
        stack.stack_bwd(CFG, Ws, st, torch.from_numpy(dy), ops=ops, max_norm=bad)
    assert e.value.status == bpt.BPT_EINVAL
    assert sorted(st.ckpt) == [0, 2] and not ops.bwd_calls
    dx, grads = stack.stack_bwd(CFG, Ws, st, torch.from_numpy(dy), ops=ops)
    _, again = stack.stack_fwd(CFG, Ws, torch.from_numpy(x), 2, ops=OracleOps())
    want, _ = stack.stack_bwd(CFG, Ws, again, torch.from_numpy(dy), ops=OracleOps())
    assert torch.equal(dx, want)
