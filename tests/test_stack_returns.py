"""What the stack returns when it runs on a stream of its own: every tensor that
the caller gets is marked as used by the caller's current stream, so that the
caller, having waited for the stack's stream, may use and drop it."""
import pytest
import torch

import blockwise_attention_ffn_gb300 as bpt
from blockwise_attention_ffn_gb300 import stack
from blockwise_attention_ffn_gb300.presets import LayerConfig
from tests.test_stack_streams import FakeCuda


@pytest.mark.parametrize("max_norm", [None, 1.0])
def test_results_are_marked_for_the_callers_stream(monkeypatch, max_norm):
    cuda = FakeCuda(monkeypatch)
    cuda.current, marked = "caller", cuda.marked
    x = torch.zeros(4, 8)
    Ws = [{"w1": torch.zeros(3, 8), "b1": None} for _ in range(3)]
    ops = stack.LibOps("side")
    y, st = stack.stack_fwd(None, Ws, x, 2, ops=ops)
    assert marked == [(y.data_ptr(), "caller")]
    marked.clear()
    dx, grads, *norm = stack.stack_bwd(None, Ws, st, torch.zeros(4, 8), ops=ops, max_norm=max_norm)
    assert len(norm) == (max_norm is not None)
    want = [dx, *norm, *(g["w1"] for g in grads)]
    assert sorted(marked) == sorted((t.data_ptr(), "caller") for t in want)
    # on the current stream there is nothing to mark
    marked.clear()
    y, st = stack.stack_fwd(None, Ws, x, 2, ops=stack.LibOps())
    stack.stack_bwd(None, Ws, st, torch.zeros(4, 8), ops=stack.LibOps(), max_norm=max_norm)
    assert not marked


@pytest.mark.gpu
def test_a_result_dropped_while_the_caller_still_reads_it():
    """The caller's stream, held up, reads y after it was dropped; the stack's
    stream meanwhile allocates and fills as much again."""
    from blockwise_attention_ffn_gb300.synth import make_layer_inputs
    cfg = LayerConfig(b=1, s=200, h=256, n_heads=4, n_kv_heads=4, head_dim=64, ffn_dim=512, ffn_block=128,
                      flags=bpt.BPT_FLAG_DETERMINISTIC)
    inp = make_layer_inputs(cfg, seed=1, device="cuda")
    Ws = [make_layer_inputs(cfg, seed=i, device="cuda", with_dy=False)["weights"] for i in range(2)]
    want, _ = stack.stack_fwd(cfg, Ws, inp["x"], 1)
    got = torch.empty_like(want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y, st = stack.stack_fwd(cfg, Ws, inp["x"], 1, ops=stack.LibOps(side))
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(200_000_000)  # a tenth of a second
    got.copy_(y)
    del y, st
    with torch.cuda.stream(side):
        junk = [torch.full_like(want, 7.0) for _ in range(8)]
    torch.cuda.synchronize()
    assert torch.equal(got, want) and len(junk) == 8
    assert bpt.bpt_last_device_error() == (bpt.BPT_OK, 0)
