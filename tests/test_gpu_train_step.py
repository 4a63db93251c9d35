"""The training operators together, as a step uses them: a projection whose
query and key heads are normalised and rotated, attention over packed documents
with capped scores and a distance bias, the way back through both, and the
clipping of the weight gradients; against PyTorch autograd in fp64 on the same
bf16 inputs, and against differences of the loss.

Tolerances: each bf16 tensor that passes from one call to the next (the
normalised heads, O, dO, dqkv) is rounded once, 2^-8 relative, as are P and dx
inside the attention; the result carries six such roundings, most of which add
in random signs, and none is amplified by more than the sums it enters (the
norms are taken over whole tensors): 6 * 2^-8 covers the worst case of the
2-norm."""
import math

import pytest
import torch

import blockwise_attention_ffn_gb300 as bpt
from blockwise_attention_ffn_gb300 import stack
from blockwise_attention_ffn_gb300.presets import LayerConfig
from blockwise_attention_ffn_gb300.synth import make_layer_inputs

pytestmark = pytest.mark.gpu

BOUND = 6 * 2.0 ** -8


def rel(a, b):
    return float((a.double() - b).norm() / b.norm())


@pytest.mark.parametrize("d,cap,causal", [(64, 20.0, 1), (80, 0.0, 1), (128, 30.0, 0)])
def test_attention_block(d, cap, causal):
    b, s, H, K = 2, 330, 4, 2
    cfg = LayerConfig(b=b, s=s, h=H * d, n_heads=H, n_kv_heads=K, head_dim=d, ffn_dim=64, causal=causal, rope_base=10000.0)
    g = torch.Generator(device="cuda").manual_seed(d)
    rows, width = b * s, (H + 2 * K) * d
    qkv = torch.randn(rows, width, generator=g, device="cuda").bfloat16()
    wq, wk = ((1 + 0.3 * torch.randn(d, generator=g, device="cuda")).bfloat16() for _ in range(2))
    dout = torch.randn(rows, H * d, generator=g, device="cuda").bfloat16()
    begin = torch.tensor([0] * 100 + [100] * 57 + [157] * (s - 157), dtype=torch.int32, device="cuda").repeat(b)
    end = torch.tensor([100] * 100 + [157] * 57 + [s] * (s - 157), dtype=torch.int32, device="cuda").repeat(b)
    pos = (torch.arange(s, device="cuda").repeat(b) - begin).int()
    slopes = torch.tensor([0.3, 0.1, 0.03, 0.01], device="cuda")
    mod = bpt.ScoreMod(begin, end, slopes, cap)

    normed, o, lse = torch.empty_like(qkv), torch.empty_like(dout), torch.empty(b, H, bpt.s_pad(cfg), device="cuda")
    bpt.bpt_qk_norm_rope_fwd(cfg, qkv, wq, wk, pos, normed)
    bpt.bpt_attention_mod_fwd(cfg, mod, normed, o, lse)
    dqkv = torch.empty_like(qkv)
    ws = bpt.alloc_bytes(max(bpt.bpt_attention_mod_bwd_workspace_bytes(cfg), bpt.bpt_qk_norm_rope_workspace_bytes(cfg)))
    bpt.bpt_attention_mod_bwd(cfg, mod, normed, o, lse, dout, dqkv, ws)
    dwq, dwk = torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    bpt.bpt_qk_norm_rope_bwd(cfg, qkv, wq, wk, pos, dqkv, dqkv, dwq, dwk, ws)  # in place
    grads = [dwq, dwk]
    before = [t.clone() for t in grads]
    norm = torch.empty(1, device="cuda")
    limit = 0.5 * float(sum(t.double().square().sum() for t in grads).sqrt())
    bpt.bpt_clip_grads(grads, limit, norm, ws)
    torch.cuda.synchronize()
    assert bpt.bpt_last_device_error() == (bpt.BPT_OK, 0)

    def forward(x, a, c):
        u = x.view(rows, H + 2 * K, d)
        z = u[:, :H + K]
        z = z * torch.rsqrt(z.square().mean(-1, keepdim=True) + cfg.norm_eps)
        z = z * torch.cat((a.expand(H, d), c.expand(K, d)))
        t = pos.double()[:, None] * 10000.0 ** (-2 * torch.arange(d // 2, device="cuda").double() / d)
        z = torch.complex(z[..., :d // 2], z[..., d // 2:]) * torch.polar(torch.ones_like(t), t)[:, None]
        z = torch.cat((z.real, z.imag), -1).view(b, s, H + K, d).transpose(1, 2)
        q, k = z[:, :H], z[:, H:].repeat_interleave(H // K, 1)
        v = u[:, H + K:].view(b, s, K, d).transpose(1, 2).repeat_interleave(H // K, 1)
        y = q @ k.transpose(-1, -2) / math.sqrt(d)
        y = cap * torch.tanh(y / cap) if cap else y
        i = torch.arange(s, device="cuda")
        y = y - slopes.double()[:, None, None] * (i[:, None] - i).abs()
        off = (i < begin.view(b, s, 1)) | (i >= end.view(b, s, 1))
        if causal:
            off = off | (i > i[:, None])
        p = torch.softmax(y.masked_fill(off[:, None], -math.inf), -1)
        return (p @ v).transpose(1, 2).reshape(rows, H * d)

    x, a, c = (t.double().requires_grad_() for t in (qkv, wq, wk))
    want = forward(x, a, c)
    want.backward(dout.double())
    assert rel(o, want.detach()) < BOUND
    assert rel(dqkv, x.grad) < BOUND
    assert rel(before[0], a.grad) < BOUND and rel(before[1], c.grad) < BOUND
    total = math.sqrt(sum(float(t.double().square().sum()) for t in before))
    assert abs(float(norm) - total) < 2.0 ** -20 * total
    for t, u in zip(grads, before):
        torch.testing.assert_close(t, u * (limit / (total + 1e-6)), rtol=2.0 ** -18, atol=0)
    # differences of <O, dO> along a direction of each input
    with torch.no_grad():
        for i, got in ((0, dqkv), (1, before[0]), (2, before[1])):
            e = torch.randn((x, a, c)[i].shape, generator=g, device="cuda", dtype=torch.float64)
            h = 1e-5
            hi = [t + h * e if j == i else t for j, t in enumerate((x, a, c))]
            lo = [t - h * e if j == i else t for j, t in enumerate((x, a, c))]
            diff = float(((forward(*hi) - forward(*lo)) * dout.double()).sum() / (2 * h))
            assert abs(diff - float((got.double() * e).sum())) < BOUND * float(got.double().norm() * e.norm())


@pytest.mark.parametrize("limit", [0.7, math.inf])
def test_stack_clips_its_gradients(limit):
    """stack_bwd(max_norm=...): the gradients of the plain call, scaled, bitwise
    the clip's own (fixed-order mode)."""
    cfg = LayerConfig(b=1, s=200, h=256, n_heads=4, n_kv_heads=4, head_dim=64, ffn_dim=512, ffn_block=128,
                      flags=bpt.BPT_FLAG_DETERMINISTIC)
    inp = make_layer_inputs(cfg, seed=1, device="cuda")
    Ws = [make_layer_inputs(cfg, seed=i, device="cuda", with_dy=False)["weights"] for i in range(2)]
    runs = []
    for max_norm in (None, limit):
        y, st = stack.stack_fwd(cfg, Ws, inp["x"], 1)
        runs.append(stack.stack_bwd(cfg, Ws, st, inp["dy"], max_norm=max_norm))
    (dx, grads), (dx2, grads2, norm) = runs
    torch.cuda.synchronize()
    flat = [g for d in grads for g in d.values() if g is not None]
    total = math.sqrt(sum(float(g.double().square().sum()) for g in flat))
    assert torch.equal(dx, dx2) and abs(float(norm) - total) < 2.0 ** -20 * total
    want = torch.empty(1, device="cuda")
    bpt.bpt_clip_grads(flat, limit, want, bpt.alloc_bytes(bpt.bpt_clip_workspace_bytes()))
    assert torch.equal(want, norm)
    for g, e in zip(flat, (g for d in grads2 for g in d.values() if g is not None)):
        assert torch.equal(g, e)
