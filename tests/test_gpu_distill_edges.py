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


def test_teacher_logits_are_taken_from_their_maximum():
    """p = softmax(values / T) goes by the values' differences: at an offset of
    2^20 (whose fp32 neighbours are 2^-3 away) as without it, and where values / T
    are beyond fp32.  Differences of multiples of 2^-3 are exact in fp32."""
    cfg = DistillConfig(n=120, h=64, vocab=500, top_k=6, temperature=3.0, flags=DET)
    x, w, ids, v, _ = inputs(cfg)
    v = (v * 8).round() / 8
    want, off = loss_of(cfg, x.double(), w.double(), ids, v, None)
    loss, dx, dw = run(cfg, x, w, ids, v, None)
    far, fx, fw = run(cfg, x, w, ids, v + 2.0 ** 20, None)
    assert abs(float(loss) - float(want)) <= off + 2.0 ** -23 * float(want)
    assert torch.equal(far, loss) and torch.equal(fx, dx) and torch.equal(fw, dw)
    # values / T beyond fp32: the largest alone
    cold = cfg.with_(temperature=2.0 ** -8)
    v[::2] = torch.tensor([1e38, 3e38, 2e38, -3e38, 2.9e38, 0.0], device="cuda")
    sure = ids.clone()
    sure[::2, [0, 2, 3, 4, 5]] = -1
    got, want = run(cold, x, w, ids, v, None), run(cold, x, w, sure, v, None)
    exact, off = loss_of(cold, x.double(), w.double(), sure, v, None)
    assert abs(float(got[0]) - float(exact)) <= off + 2.0 ** -23 * float(exact)
    assert torch.equal(got[0], want[0])
    near(got[1], want[1].double(), 2, "dx")
    near(got[2], want[2].double(), 2, "dw")


def test_rows_of_probability_zero_give_nothing():
    """Entries that are there but all of probability 0 (-inf): no loss and no
    gradient, whatever the row's logits are (infinite here)."""
    cfg = DistillConfig(n=70, h=64, vocab=500, top_k=6, vocab_block=256, flags=DET)
    for teacher in (0, LOGPROBS):
        c = cfg.with_(teacher=teacher)
        x, w, ids, v, _ = inputs(c)
        v[::2] = -math.inf
        once = run(c, x, w, ids, v, None)
        assert all(t.isfinite().all() for t in once) and bool((once[1][::2] == 0).all())
        x[::2] = 3e38
        for a, b in zip(once, run(c, x, w, ids, v, None)):
            assert torch.equal(a, b)
