"""The modified attention over the whole range of caps and scores: caps up to
the largest accepted, scores at and beyond the cap, values of any size, and
masked rows holding anything finite.

Every score here is one product: a query has a single nonzero column, so q.k is
exact in fp32 and a score's error comes from its modification alone.  That is
2^-20 of its size: the scale, the tanh (an error of at most 2^-21.5 relative to
its own value), the fp32 steps of the score, of the bias and of the
log-sum-exp.  A probability rebuilt from both moves by expm1 of it; one below
2^-126, the least normal fp32 number, is 0 instead.  The other terms are those of
the roundings to bf16 (h = 2^-8) as in the tests of ordinary scores."""
import math

import numpy as np
import pytest
import torch

import blockwise_attention_ffn_gb300 as bpt
from blockwise_attention_ffn_gb300.presets import LayerConfig
from oracle import train_ops as T
from tests.gpu_helpers import to64
from tests.test_gpu_attention_mod import as_int32, check, make, run

pytestmark = pytest.mark.gpu

H8 = 2.0 ** -8 * 1.02
P0 = 2.0 ** -126


def inputs(s, d, levels, seed, v_scale=1.0, block=128, signs="both"):
    """One head of s rows.  Row i of Q: levels[i // block] * sqrt(d) in one
    column; K: magnitudes between 15/16 and 1 of each sign, so that the scores
    of the row lie just below its level."""
    g = torch.Generator().manual_seed(seed)
    q = torch.zeros(s, d)
    lev = torch.tensor([levels[(i // block) % len(levels)] for i in range(s)], dtype=torch.float64)
    q[torch.arange(s), torch.randint(0, d, (s,), generator=g)] = (lev * math.sqrt(d)).float()
    k = 1 - torch.randint(0, 9, (s, d), generator=g) / 128
    if signs == "both":
        k *= torch.randint(0, 2, (s, d), generator=g) * 2 - 1
    elif signs == "minus":
        k = -k
    v = torch.randn(s, d, generator=g) * v_scale
    return torch.cat((q, k, v), 1).to(torch.bfloat16), torch.randn(s, d, generator=g).to(torch.bfloat16)


def check_head(s, d, causal, cap, slope, qkv, dout, o, lse, dqkv, begin=None, end=None):
    q, k, v = np.split(to64(qkv), 3, axis=1)
    do, dO = to64(dout), np.abs(to64(dout))
    o, lse, dx = to64(o), to64(lse)[0, 0], to64(dqkv)
    ok = T.allowed(s, causal, begin, end)
    wo, wl, wq, wk, wv = T.attention_mod_head(q, k, v, ok, slope, cap, do)
    raw = q @ k.T / math.sqrt(d)
    u = np.tanh(raw / cap) if cap else np.zeros_like(raw)
    far = abs(slope) * np.abs(np.arange(s)[:, None] - np.arange(s)[None])
    y = (cap * u if cap else raw) - np.sign(slope) * far
    fin = np.where(np.isfinite(wl), wl, 0.0)[:, None]
    p = np.where(ok, np.exp(np.minimum(y - fin, 0.0)), 0.0)
    e = np.where(ok, 2.0 ** -20 * (np.abs(cap * u if cap else raw) + far + np.abs(fin) + 8), 0.0)
    E = np.expm1(e)
    # the row's own sum divides by what the same errors moved
    pe = np.where(ok, (H8 + E) * p + P0, 0.0)  # the error of a probability
    bo = pe @ np.abs(v) + (H8 + E.max(1, keepdims=True)) * np.abs(wo) + P0
    check("O", o, wo, bo)
    check("LSE", lse[:s], wl, e.max(1) + 2.0 ** -20)
    check("dV", dx[:, 2 * d:], wv, pe.T @ dO + H8 * np.abs(wv) + P0)
    dP = do @ v.T - (do * wo).sum(1, keepdims=True)
    f = 1 - u * u
    # dP: D from the rounded O, and d terms of the products with V^T
    eD = (dO * bo).sum(1, keepdims=True) + d * 2.0 ** -22 * (dO @ np.abs(v).T)
    # and u to 2^-22, which counts twice in 1 - u^2
    edx = (pe * f * (np.abs(dP) + eD) + p * f * eD + 2.0 ** -21 * (p + pe) * (np.abs(dP) + eD)) / math.sqrt(d)
    check("dQ", dx[:, :d], wq, edx @ np.abs(k) + H8 * np.abs(wq) + P0)
    check("dK", dx[:, d:2 * d], wk, edx.T @ np.abs(q) + H8 * np.abs(wk) + P0)


def one_head(s, d, causal, cap, slope, x, do, end=None):
    cfg = LayerConfig(b=1, s=s, h=d, n_heads=1, n_kv_heads=1, head_dim=d, ffn_dim=64, causal=causal)
    mod = bpt.ScoreMod(None, as_int32(end), None if not slope else torch.tensor([slope], device="cuda"), cap)
    got = run(cfg, mod, x, do, bpt.BPT_FLAG_DETERMINISTIC)
    check_head(s, d, causal, cap, slope, x, do, *got, end=end)


LEVELS = [0.2, 0.3, 0.45, 0.59, 0.8, 1.0, 2.0, 0.05]  # of the cap, per tile of 128 rows


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("slope", [0.0, 0.01])
@pytest.mark.parametrize("cap", [2.0 ** -10, 1.0, 60.0, 100.0, 1000.0, 8192.0, 65536.0, 2.0 ** 20])
def test_caps_of_every_size(cap, slope, d):
    """Scores from a twentieth of the cap to twice it, a tile of rows at each."""
    s = 128 * len(LEVELS)
    x, do = inputs(s, d, [f * cap for f in LEVELS], seed=int(math.log2(cap)) + d)
    one_head(s, d, 0, cap, slope, x, do)


@pytest.mark.parametrize("cap", [20.0, 50.0, 64.0, 65.0, 8192.0, 2.0 ** 20])
def test_small_scores_beside_large_ones(cap):
    """Rows of a few units among rows beyond the cap: a row's scores keep their
    own accuracy whatever its neighbours in the tile are."""
    s, d = 384, 80
    x, do = inputs(s, d, [3.0, 1.5 * cap, 0.5], seed=3, block=1)
    one_head(s, d, 0, cap, 0.0, x, do)


@pytest.mark.parametrize("v_scale", [2.0 ** 55, 1.0, 2.0 ** -60])
@pytest.mark.parametrize("signs", ["plus", "minus", "both"])
@pytest.mark.parametrize("slope", [0.0, 0.02, -0.02, 2.0])
@pytest.mark.parametrize("cap", [60.0, 30.0])
def test_saturated_scores(cap, slope, signs, v_scale):
    """Whole rows at +cap and at -cap, beside rows in the cap's nearly linear
    range, with values far from 1."""
    s, d = 640, 64
    x, do = inputs(s, d, [3 * cap, 0.55 * cap, 0.1 * cap, cap], seed=4, v_scale=v_scale, block=96, signs=signs)
    one_head(s, d, 1, cap, slope, x, do)


@pytest.mark.parametrize("slope", [0.0, 0.02, 1.5])
@pytest.mark.parametrize("level", [300.0, 3000.0])
def test_large_scores_without_a_cap(level, slope):
    s, d = 400, 112
    x, do = inputs(s, d, [level, -0.3 * level, 2.0], seed=5)
    one_head(s, d, 1, 0.0, slope, x, do, end=[max(q + 1, 150) for q in range(s)])


@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("cap,biased", [(20.0, True), (50.0, False), (100.0, False), (100.0, True)])
def test_masked_rows_leave_no_trace_with_a_cap(d, cap, biased):
    """What (finite) lies in rows that no window reaches changes no bit of any
    output: the largest bf16 values, and values near the scores' own size."""
    b, s, H, K = 3, 300, 4, 2
    cfg = LayerConfig(b=b, s=s, h=H * d, n_heads=H, n_kv_heads=K, head_dim=d, ffn_dim=64, causal=0)
    n = [300, 131, 0]
    end = as_int32([n[i] if q < n[i] else 0 for i in range(b) for q in range(s)])
    qkv, dout = make(b, s, H, K, d, seed=2)
    mod = bpt.ScoreMod(None, end, torch.tensor([0.5, 0.1, 0.01, 0.0], device="cuda") if biased else None, cap)
    clean = [t.clone() for t in run(cfg, mod, qkv, dout, bpt.BPT_FLAG_DETERMINISTIC)]
    for fill in (3.3e38, 6.0, -40.0):
        dirty, ddirty = qkv.clone().view(b, s, -1), dout.clone().view(b, s, -1)
        for i in range(b):
            dirty[i, n[i]:] = fill
            dirty[i, n[i]:, ::2] = -fill
            ddirty[i, n[i]:] = fill
        got = run(cfg, mod, dirty.view(b * s, -1), ddirty.view(b * s, -1), bpt.BPT_FLAG_DETERMINISTIC)
        for what, a, c in zip(("o", "lse", "dqkv"), got, clean):
            assert torch.equal(a, c), (what, fill)
