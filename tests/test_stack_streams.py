"""The stack's buffers on a stream of their own.  What LibOps allocates is used
on its stream, so it has to be allocated there too: the allocator hands a freed
block to the next tensor of the stream it came from, and a block of another
stream may be in that one's hands again while this one's kernels still use it.

On the CPU the library and the allocator are watched: every allocation made by
the stack must happen with the ops' stream current.  On the GPU the stack runs on
a stream that is held up while the current one allocates and writes."""
import contextlib

import pytest
import torch

import blockwise_attention_ffn_gb300 as bpt
from blockwise_attention_ffn_gb300 import stack
from blockwise_attention_ffn_gb300.presets import LayerConfig


class FakeCuda:
    """torch.cuda's notion of the current stream, the streams on which buffers
    were allocated and given to the library, and those they were marked for."""

    def __init__(self, monkeypatch):
        self.current, self.where, self.used, self.marked = "default", {}, [], []
        monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: self.current)
        monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: self.marked.append((t.data_ptr(), s)))
        monkeypatch.setattr(torch.cuda, "stream", self.stream)
        monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: handle)
        for name in ("empty", "empty_like"):
            monkeypatch.setattr(torch, name, self.watched(getattr(torch, name)))
        for name in ("bpt_layer_fwd", "bpt_layer_bwd"):
            monkeypatch.setattr(bpt, name, self.layer)
        monkeypatch.setattr(bpt, "bpt_clip_grads", self.clip)
        for name in ("bpt_workspace_bytes", "bpt_saved_bytes", "bpt_clip_workspace_bytes"):
            monkeypatch.setattr(bpt, name, lambda *a: 512)

    @contextlib.contextmanager
    def stream(self, s):
        before, self.current = self.current, s
        yield
        self.current = before

    def watched(self, make):
        def alloc(*a, **kw):
            t = make(*a, **kw)
            self.where[t.data_ptr()] = (self.current, t)
            return t
        return alloc

    def use(self, *ts):
        for t in ts:
            for v in t.values() if isinstance(t, dict) else t if isinstance(t, (list, tuple)) else [t]:
                if torch.is_tensor(v) and v.data_ptr() in self.where:
                    self.used.append(self.where[v.data_ptr()][0])

    def layer(self, cfg, *a):
        *ts, stream = a
        self.use(*ts)

    def clip(self, grads, max_norm, norm, ws, out=None, flags=0, stream=None):
        self.use(grads, norm, ws)


@pytest.mark.parametrize("stream", ["side", 1234])
def test_buffers_are_allocated_on_the_stream_that_uses_them(monkeypatch, stream):
    cuda = FakeCuda(monkeypatch)
    x = torch.zeros(4, 8)
    Ws = [{"w1": torch.zeros(3, 8), "b1": None} for _ in range(3)]
    ops = stack.LibOps(stream)
    y, st = stack.stack_fwd(None, Ws, x, 2, ops=ops)
    stack.stack_bwd(None, Ws, st, torch.zeros(4, 8), ops=ops, max_norm=1.0)
    # workspaces, outputs, log-sum-exps, gradients, the clip's norm and workspace
    assert len(cuda.used) > 20 and set(cuda.used) == {stream}
    assert cuda.current == "default"
    # without a stream everything stays on the current one
    cuda.used.clear()
    y, st = stack.stack_fwd(None, Ws, x, 2, ops=stack.LibOps())
    stack.stack_bwd(None, Ws, st, torch.zeros(4, 8), ops=stack.LibOps(), max_norm=1.0)
    assert set(cuda.used) == {"default"}


@pytest.mark.gpu
def test_stack_on_a_stream_that_is_held_up():
    """Forward, backward and clipping queued behind a long wait on a side
    stream, while the current stream frees, allocates and fills buffers of the
    same sizes: bitwise what the same calls give on the current stream."""
    from blockwise_attention_ffn_gb300.synth import make_layer_inputs
    cfg = LayerConfig(b=1, s=200, h=256, n_heads=4, n_kv_heads=4, head_dim=64, ffn_dim=512, ffn_block=128,
                      flags=bpt.BPT_FLAG_DETERMINISTIC)
    inp = make_layer_inputs(cfg, seed=1, device="cuda")
    Ws = [make_layer_inputs(cfg, seed=i, device="cuda", with_dy=False)["weights"] for i in range(2)]

    def run(ops):
        y, st = stack.stack_fwd(cfg, Ws, inp["x"], 1, ops=ops)
        return y, stack.stack_bwd(cfg, Ws, st, inp["dy"], ops=ops, max_norm=0.7)

    want, (wdx, wgrads, wnorm) = run(None)
    torch.cuda.synchronize()
    for handle in (False, True):
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            torch.cuda._sleep(200_000_000)  # a tenth of a second
        y, (dx, grads, norm) = run(stack.LibOps(side.cuda_stream if handle else side))
        for n in (256, 4096, 9728, 65536, 262144, 1 << 20, 1 << 24):
            junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for _ in range(8)]
            del junk
        torch.cuda.synchronize()
        assert bpt.bpt_last_device_error() == (bpt.BPT_OK, 0)
        assert torch.equal(y, want) and torch.equal(dx, wdx) and torch.equal(norm, wnorm)
        for a, b in zip(grads, wgrads):
            for k in a:
                assert a[k] is None or torch.equal(a[k], b[k]), k
