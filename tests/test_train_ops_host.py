"""Host side of the modified attention, the head norm with rotation and the
gradient clipping: every refusal comes before anything is launched, so all of
it runs without a GPU (addresses that are never read stand in for device
memory)."""
import ctypes

import numpy as np
import pytest
import torch

import blockwise_attention_ffn_gb300 as bpt
from blockwise_attention_ffn_gb300 import stack
from blockwise_attention_ffn_gb300.presets import C3, C4, LayerConfig
from oracle import train_ops as T
from tests.test_stack_schedule import CFG, OracleOps, _stack

A = 1 << 40  # a 16-byte aligned address nothing lives at


@pytest.fixture(scope="module")
def lib():
    from blockwise_attention_ffn_gb300 import build
    build.build()
    return bpt.lib()


def cfg(**kw):
    base = dict(b=2, s=200, h=256, n_heads=4, n_kv_heads=2, head_dim=64, ffn_dim=64, rope_base=10000.0)
    return bpt.make_config(LayerConfig(**{**base, **kw}))


def far(i):
    """Addresses far apart."""
    return A + (i << 34)


def fwd(lib, c=None, mod=None, **kw):
    a = dict(qkv=far(1), o=far(2), lse=far(3), stream=0, **{}) | kw
    mod = bpt.BptScoreMod(None, None, None, 0.0) if mod is None else mod
    return lib.bpt_attention_mod_fwd(c if c is not None else cfg(), mod, a["qkv"], a["o"], a["lse"], a["stream"])


def bwd(lib, c=None, mod=None, **kw):
    c = cfg() if c is None else c
    a = dict(qkv=far(1), o=far(2), lse=far(3), dout=far(4), dqkv=far(5), ws=far(6),
             n=lib.bpt_attention_mod_bwd_workspace_bytes(c)) | kw
    mod = bpt.BptScoreMod(None, None, None, 0.0) if mod is None else mod
    return lib.bpt_attention_mod_bwd(c, mod, a["qkv"], a["o"], a["lse"], a["dout"], a["dqkv"], a["ws"], a["n"], None)


def test_structs_match_the_header():
    assert ctypes.sizeof(bpt.BptScoreMod) == 32
    assert ctypes.sizeof(bpt.BptClipTensor) == 32


@pytest.mark.parametrize("kw", [dict(qkv=None), dict(o=None), dict(qkv=far(1) + 8), dict(o=far(2) + 2),
                                dict(lse=far(3) + 4), dict(o=far(1)), dict(lse=far(1) + 64), dict(lse=far(2) + 16)])
def test_attention_forward_rejects_pointers(lib, kw):
    assert fwd(lib, **kw) == bpt.BPT_EINVAL


@pytest.mark.parametrize("kw", [dict(qkv=None), dict(o=None), dict(lse=None), dict(dout=None), dict(dqkv=None),
                                dict(ws=None), dict(dqkv=far(1)), dict(dqkv=far(4) + 32), dict(dqkv=far(2)),
                                dict(ws=far(5)), dict(ws=far(1) + 256), dict(dqkv=far(3)), dict(dout=far(4) + 8)])
def test_attention_backward_rejects_pointers(lib, kw):
    assert bwd(lib, **kw) == bpt.BPT_EINVAL


def test_attention_rejects_shapes_modifiers_and_workspace(lib):
    for cap in (-1.0, float("nan"), float("inf"), 1e-4, 3e6):
        mod = bpt.BptScoreMod(None, None, None, cap)
        assert fwd(lib, mod=mod) == bpt.BPT_EINVAL and bwd(lib, mod=mod) == bpt.BPT_EINVAL
    for i in range(3):
        mod = bpt.BptScoreMod(*[far(7) + 2 if j == i else None for j in range(3)], 0.0)
        assert fwd(lib, mod=mod) == bpt.BPT_EINVAL and bwd(lib, mod=mod) == bpt.BPT_EINVAL
    assert lib.bpt_attention_mod_fwd(cfg(), None, far(1), far(2), None, None) == bpt.BPT_EINVAL
    assert fwd(lib, c=cfg(head_dim=72)) == bpt.BPT_EUNSUPPORTED
    assert fwd(lib, c=cfg(n_kv_heads=3)) == bpt.BPT_EINVAL
    assert fwd(lib, c=cfg(causal=2)) == bpt.BPT_EINVAL
    assert fwd(lib, c=cfg(b=4096, s=131072 * 2, n_heads=4)) == bpt.BPT_EUNSUPPORTED
    n = lib.bpt_attention_mod_bwd_workspace_bytes(cfg())
    assert bwd(lib, n=n - 1) == bpt.BPT_ENOSPC
    # dO.O sums, -LSE log2(e) and extra rows: 24 bytes a row and head; windows
    # 1056 + 8 bytes a query tile; five regions, each rounded up to 256 bytes
    for c in (C3, C4):
        rows = c.b * c.n_heads * bpt.s_pad(c)
        tiles = c.b * bpt.s_pad(c) // 128
        got = bpt.bpt_attention_mod_bwd_workspace_bytes(c)
        assert 24 * rows + 1064 * tiles <= got < 24 * rows + 1064 * tiles + 5 * 256
    assert lib.bpt_attention_mod_bwd_workspace_bytes(cfg(head_dim=72)) == 0


@pytest.mark.parametrize("i", range(3))
def test_attention_rejects_outputs_over_the_modifiers(lib, i):
    """o, lse, dqkv and ws may not share bytes with the windows or slopes."""
    mod = bpt.BptScoreMod(*[far(7) if j == i else None for j in range(3)], 0.0)
    for kw in (dict(o=far(7)), dict(lse=far(7)), dict(o=far(7) - 512)):
        assert fwd(lib, mod=mod, **kw) == bpt.BPT_EINVAL, kw
    for kw in (dict(dqkv=far(7)), dict(ws=far(7)), dict(ws=far(7) - 4096)):
        assert bwd(lib, mod=mod, **kw) == bpt.BPT_EINVAL, kw


def norm_fwd(lib, c=None, **kw):
    a = dict(qkv=far(1), wq=far(2), wk=far(3), pos=None, out=far(4)) | kw
    return lib.bpt_qk_norm_rope_fwd(cfg() if c is None else c, a["qkv"], a["wq"], a["wk"], a["pos"], a["out"], None)


def norm_bwd(lib, c=None, **kw):
    c = cfg() if c is None else c
    a = dict(qkv=far(1), wq=far(2), wk=far(3), pos=None, dout=far(4), dqkv=far(5), dwq=far(6), dwk=far(7), ws=far(8),
             n=lib.bpt_qk_norm_rope_workspace_bytes(c)) | kw
    return lib.bpt_qk_norm_rope_bwd(c, a["qkv"], a["wq"], a["wk"], a["pos"], a["dout"], a["dqkv"], a["dwq"], a["dwk"],
                                    a["ws"], a["n"], None)


def test_norm_rope_rejects(lib):
    for kw in (dict(qkv=None), dict(out=None), dict(wq=None), dict(wk=None), dict(out=far(1) + 512), dict(wq=far(2) + 2),
               dict(pos=far(9) + 2), dict(qkv=far(1) + 8)):
        assert norm_fwd(lib, **kw) == bpt.BPT_EINVAL, kw
    assert norm_fwd(lib, c=cfg(rope_base=0.0), wq=None, wk=None) == bpt.BPT_EINVAL
    assert norm_fwd(lib, c=cfg(head_dim=48)) == bpt.BPT_EUNSUPPORTED
    for kw in (dict(qkv=None), dict(dout=None), dict(dqkv=None), dict(dwq=None), dict(dwk=None), dict(ws=None),
               dict(dqkv=far(1)), dict(dqkv=far(4) + 64), dict(dqkv=far(1) + 64), dict(wq=None), dict(dwq=far(6) + 2)):
        assert norm_bwd(lib, **kw) == bpt.BPT_EINVAL, kw
    assert norm_bwd(lib, n=16) == bpt.BPT_ENOSPC


def test_norm_rope_rejects_outputs_over_other_buffers(lib):
    for kw in (dict(out=far(2)), dict(out=far(3) - 4096), dict(out=far(9), pos=far(9)), dict(pos=far(4) + 4096)):
        assert norm_fwd(lib, **kw) == bpt.BPT_EINVAL, kw
    for kw in (dict(dqkv=far(2)), dict(dqkv=far(9), pos=far(9)), dict(dwq=far(7)), dict(dwk=far(6) + 128),
               dict(dwq=far(5) + 64), dict(dwk=far(4)), dict(dwq=far(1)), dict(dwq=far(2)), dict(ws=far(5)),
               dict(ws=far(6)), dict(ws=far(1) + 256), dict(ws=far(3) - 256), dict(dwk=far(9), pos=far(9))):
        assert norm_bwd(lib, **kw) == bpt.BPT_EINVAL, kw


def test_clip_rejects_tensors_over_norm_and_workspace(lib):
    for bad in ([(far(20), far(2), 100, 0)], [(far(1), far(20) - 4, 2, 0)], [(far(21) + 64, far(2), 100, 0)],
                [(far(1), far(21), 100, 1)]):
        assert clip(lib, bad) == bpt.BPT_EINVAL, bad
    assert clip(lib, [], norm=far(21)) == bpt.BPT_EINVAL


def clip(lib, tensors, max_norm=1.0, flags=0, norm=far(20), ws=far(21), n=None, size=None):
    t = (bpt.BptClipTensor * max(1, len(tensors)))(*tensors)
    return lib.bpt_clip_grads(len(tensors) if size is None else size, ctypes.addressof(t), max_norm, flags, norm, ws,
                              lib.bpt_clip_workspace_bytes() if n is None else n, None)


def test_clip_rejects(lib):
    ok = (far(1), far(2), 100, 0)
    for bad in ([(None, far(2), 100, 0)], [(far(1), None, 100, 0)], [(far(1), far(2), -1, 0)], [(far(1), far(2), 10, 2)],
                [(far(1) + 2, far(2), 10, 0)], [(far(1), far(2) + 1, 10, 1)],
                [ok, ok], [ok, (far(3), far(2) + 396, 5, 0)], [(far(1), far(1) + 4, 100, 0)],
                [ok, (far(2) + 4, far(3), 2, 0)], [(far(1), far(1), 100, 0), (far(1), far(1), 100, 0)],
                [(far(1), far(1), 100, 0), (far(1) + 200, far(3), 10, 1)]):
        assert clip(lib, bad) == bpt.BPT_EINVAL, bad
    for m in (0.0, -1.0, float("nan")):
        assert clip(lib, [ok], m) == bpt.BPT_EINVAL
    assert clip(lib, [ok], flags=1) == bpt.BPT_EINVAL
    assert clip(lib, [ok], norm=None) == bpt.BPT_EINVAL and clip(lib, [ok], ws=None) == bpt.BPT_EINVAL
    assert clip(lib, [ok], size=-1) == bpt.BPT_EINVAL
    assert clip(lib, [ok], n=8) == bpt.BPT_ENOSPC


def test_binding_checks_tensors_before_the_call(lib):
    """CPU tensors, wrong types and short tensors never reach the library."""
    x = torch.zeros(10, dtype=torch.bfloat16)
    for t in (x, x.float(), None):
        with pytest.raises(bpt.BptError) as e:
            bpt._want("call", "x", t, torch.bfloat16, 10, 0)
        assert e.value.status == bpt.BPT_EINVAL
    assert bpt._may("call", "x", None, torch.bfloat16, 10, 0) is None


@pytest.mark.parametrize("limit", [0.05, 1e9])
def test_stack_backward_clips(limit):
    """stack_bwd(max_norm=...) hands every layer's gradients to the clip and
    returns the norm; without it nothing changes."""

    class Ops(OracleOps):
        def clip(self, grads, max_norm, like):
            ts = [g for d in grads for g in d.values() if g is not None]
            norm, out = T.clip([t.numpy() for t in ts], max_norm)
            for t, o in zip(ts, out):
                t.copy_(torch.from_numpy(np.asarray(o)).view(t.shape))
            return torch.tensor([norm])

    x, Ws, dy = _stack(3)
    runs = []
    for max_norm in (None, limit):
        ops = Ops()
        y, st = stack.stack_fwd(CFG, Ws, torch.from_numpy(x), 2, ops=ops)
        runs.append(stack.stack_bwd(CFG, Ws, st, torch.from_numpy(dy), ops=ops, max_norm=max_norm))
    (dx, grads), (dx2, grads2, norm) = runs
    assert torch.equal(dx, dx2)
    want = sum(float((g ** 2).sum()) for d in grads for g in d.values() if g is not None) ** 0.5
    assert abs(float(norm) - want) < 1e-9 * want
    for d, e in zip(grads, grads2):
        for k in d:
            if d[k] is not None:
                torch.testing.assert_close(e[k], d[k] * min(1.0, limit / (want + 1e-6)), rtol=1e-12, atol=0)
