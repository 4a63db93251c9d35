"""Edges of the distillation loss on the GPU: padding of the stored
log-probabilities, large teacher logits, rows whose entries all have
probability 0.  References and tolerances as in test_gpu_distill.py."""
import math

import pytest
import torch

import blockwise_attention_ffn_gb300 as bpt
from blockwise_attention_ffn_gb300.presets import DistillConfig
from tests.test_gpu_distill import LOGPROBS, inputs, loss_of, near, run

pytestmark = pytest.mark.gpu
DET = bpt.BPT_FLAG_DETERMINISTIC


@pytest.mark.parametrize("teacher", [0, LOGPROBS])
@pytest.mark.parametrize("value", [89.0, 1e4, 3e38])
@pytest.mark.parametrize("grads", [0, 1])
def test_padding_may_hold_any_finite_value(teacher, value, grads):
    """A row of weight 0 leaves no trace, also where exp of its stored values
    is beyond fp32."""
    cfg = DistillConfig(n=200, h=128, vocab=900, top_k=9, teacher=teacher, grads_dtype=grads, flags=DET)
    x, w, ids, v, weight = inputs(cfg, True)
    once = run(cfg, x, w, ids, v, weight)
    assert all(t.isfinite().all() for t in once)
    v[weight == 0] = value
    for a, b in zip(once, run(cfg, x, w, ids, v, weight)):
        assert torch.equal(a, b)
