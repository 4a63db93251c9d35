"""Attention with key windows, capped scores and a distance bias, forward and
backward, on the GPU against the fp64 definition.

Tolerances, entry by entry, from the roundings the method makes (h = 2^-8, half
a bf16 step relative to the value):
  score   fp32 sums of d exact products: at most d 2^-23 |q|.|k| / sqrt(d), then
          fp32 steps of the modified score's and the log-sum-exp's size; a
          probability moves by e = that, relative (worst case, so small against h)
  O       bf16 P against an fp32 row sum: (h + e) P|V|, and its own rounding h |O|
  LSE     e and fp32 steps of its size
  dV      (h + e) P^T|dO| + h |dV|
  D       |dO| . (error of O), as O is stored in bf16
  dx      = P (dP - D)(1 - u^2): (h + e) |dx| + P (1 - u^2) err(D) + fp32 steps of
          |dO|.|V|
  dQ, dK  err(dx) times |K|, |Q| / sqrt(d), and their own rounding
fp32 sums over the keys or queries add under s 2^-24 of the terms' sizes, inside
the margin h leaves (s 2^-24 < h / 100 here)."""
import math

import numpy as np
import pytest
import torch

import blockwise_attention_ffn_gb300 as bpt
from blockwise_attention_ffn_gb300.presets import LayerConfig
from oracle import train_ops as T
from tests.gpu_helpers import to64

pytestmark = pytest.mark.gpu

H8 = 2.0 ** -8 * 1.02  # and the fp32 sums


def windows(kind, b, s, seed=0):
    """(causal, row_begin, row_end) as int lists of b*s, or None."""
    rng = np.random.default_rng(seed)
    begin, end = [], []
    for i in range(b):
        cuts = sorted({0, s, *rng.integers(0, s + 1, 1 + s // 90).tolist()})
        doc = [(a, e) for a, e in zip(cuts, cuts[1:]) for _ in range(a, e)]
        n = max(0, s - i * (s // 3 + 1))
        if kind == "docs":
            begin += [a for a, _ in doc]
        elif kind == "docs_both":
            begin += [a for a, _ in doc]
            end += [e for _, e in doc]
        elif kind == "prefix":
            end += [max(q + 1, min(s // 3, n)) if q < n else 0 for q in range(s)]
        elif kind == "window":
            begin += [q - 20 for q in range(s)]
        elif kind == "padded":
            end += [n] * s
        elif kind == "holes":  # rows of every kind: empty, reversed, far outside
            lo, hi = rng.integers(-5, s + 5, (2, s))
            lo[rng.random(s) < 0.1], hi[rng.random(s) < 0.1] = -2 ** 31, 2 ** 31 - 1
            begin += lo.tolist()
            end += hi.tolist()
        elif kind == "none":
            end += [0] * s
    return int(kind in ("causal", "docs", "window")), begin or None, end or None


def as_int32(v):
    return None if v is None else torch.tensor(v, dtype=torch.int64).to(torch.int32).cuda()


def make(b, s, H, K, d, seed, qscale=1.5):
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn(b * s, (H + 2 * K) * d, generator=g)
    qkv[:, :H * d] *= qscale
    return qkv.to(torch.bfloat16), torch.randn(b * s, H * d, generator=g).to(torch.bfloat16)


def run(cfg, mod, qkv, dout, flags=0):
    cfg = cfg.with_(flags=flags)
    rows = cfg.b * cfg.s
    x = qkv.cuda()
    o = torch.full((rows, cfg.n_heads * cfg.head_dim), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((cfg.b, cfg.n_heads, bpt.s_pad(cfg)), float("nan"), device="cuda")
    bpt.bpt_attention_mod_fwd(cfg, mod, x, o, lse)
    dqkv = torch.full_like(x, float("nan"))
    ws = bpt.alloc_bytes(bpt.bpt_attention_mod_bwd_workspace_bytes(cfg))
    ws.fill_(255)
    bpt.bpt_attention_mod_bwd(cfg, mod, x, o, lse, dout.cuda(), dqkv, ws)
    torch.cuda.synchronize()
    assert bpt.bpt_last_device_error() == (bpt.BPT_OK, 0)
    return o, lse, dqkv


def check(what, got, want, bound):
    assert np.array_equal(np.isfinite(got), np.isfinite(want)), f"{what}: finite entries differ"
    ok = np.isfinite(want)
    assert np.array_equal(got[~ok], want[~ok])
    over = np.abs(got[ok] - want[ok]) - bound[ok]
    assert not over.size or over.max() <= 0, f"{what}: {over.max():.3e} over its bound, {np.mean(over > 0):.2e} of the entries"


def check_all(cfg, causal, begin, end, slopes, cap, qkv, dout, o, lse, dqkv):
    b, s, H, K, d = cfg.b, cfg.s, cfg.n_heads, cfg.n_kv_heads, cfg.head_dim
    G = H // K
    x, do = to64(qkv).reshape(b, s, H + 2 * K, d), to64(dout).reshape(b, s, H, d)
    o, lse, dx = to64(o).reshape(b, s, H, d), to64(lse), to64(dqkv).reshape(x.shape)
    assert np.all(lse[:, :, s:] == 0)
    for bi in range(b):
        rows = slice(bi * s, (bi + 1) * s)
        ok = T.allowed(s, causal, None if begin is None else begin[rows], None if end is None else end[rows])
        for g in range(K):
            k, v = x[bi, :, H + g], x[bi, :, H + K + g]
            dk, dv, ek, ev = (np.zeros((s, d)) for _ in range(4))
            for n in range(g * G, (g + 1) * G):
                q, a = x[bi, :, n], 0.0 if slopes is None else float(slopes[n])
                wo, wl, wq, wk, wv = T.attention_mod_head(q, k, v, ok, a, cap, do[bi, :, n])
                raw = q @ k.T / math.sqrt(d)
                u = np.tanh(raw / cap) if cap else np.zeros_like(raw)
                far = a * np.abs(np.arange(s)[:, None] - np.arange(s)[None])
                y = (cap * u if cap else raw) - far
                fin = np.where(np.isfinite(wl), wl, 0.0)
                p = np.where(ok, np.exp(np.minimum(y - fin[:, None], 0.0)), 0.0)
                e = (d * 2.0 ** -23 * (np.abs(q) @ np.abs(k).T) / math.sqrt(d)
                     + 2.0 ** -20 * (np.abs(raw if not cap else cap * u) + far + np.abs(fin)[:, None] + 8))
                e = np.where(ok, e, 0.0)
                bo = ((H8 + e) * p) @ np.abs(v) + H8 * np.abs(wo) + 1e-30
                check(f"O[{bi}, {n}]", o[bi, :, n], wo, bo)
                check(f"LSE[{bi}, {n}]", lse[bi, n, :s], wl, e.max(1) + 2.0 ** -21 * np.abs(fin) + 2.0 ** -21)
                dk, dv = dk + wk, dv + wv
                dO = np.abs(do[bi, :, n])
                ev += ((H8 + e) * p).T @ dO
                size = dO @ np.abs(v).T
                dP = do[bi, :, n] @ v.T - (do[bi, :, n] * wo).sum(1, keepdims=True)
                f = p * (1 - u * u)
                edx = ((H8 + e) * f * np.abs(dP) + f * ((dO * bo).sum(1, keepdims=True) + d * 2.0 ** -22 * size)
                       + 2.0 ** -21 * p * np.abs(dP)) / math.sqrt(d)
                check(f"dQ[{bi}, {n}]", dx[bi, :, n], wq, edx @ np.abs(k) + H8 * np.abs(wq) + 1e-30)
                ek += edx.T @ np.abs(q)
            check(f"dK[{bi}, {g}]", dx[bi, :, H + g], dk, ek + H8 * np.abs(dk) + 1e-30)
            check(f"dV[{bi}, {g}]", dx[bi, :, H + K + g], dv, ev + H8 * np.abs(dv) + 1e-30)


CASES = [
    # b, s, H, K, d, windows, cap, slopes
    (1, 1, 1, 1, 64, "causal", 0.0, False),
    (1, 2, 2, 1, 128, "docs", 30.0, True),
    (1, 1, 1, 1, 80, "none", 30.0, True),
    (2, 63, 2, 2, 80, "docs", 0.0, True),
    (1, 64, 2, 1, 96, "docs_both", 20.0, False),
    (3, 65, 2, 2, 112, "padded", 0.0, False),
    (1, 127, 2, 2, 128, "window", 50.0, True),
    (2, 128, 2, 1, 64, "prefix", 0.0, True),
    (1, 129, 2, 2, 80, "holes", 10.0, True),
    (2, 200, 4, 2, 112, "holes", 0.0, False),
    (1, 300, 4, 1, 96, "docs", 5.0, False),
    (2, 257, 3, 1, 128, "docs_both", 0.0, True),
    (1, 513, 4, 2, 128, "docs", 30.0, False),
    (1, 640, 2, 2, 64, "window", 0.0, False),
    (2, 385, 2, 1, 80, "prefix", 20.0, True),
    (1, 600, 2, 2, 96, "causal", 0.0, False),
    (1, 600, 2, 2, 128, "all", 1.0, True),
    (3, 390, 2, 2, 64, "padded", 60.0, False),
    (1, 500, 2, 1, 112, "causal", 2.0, False),
    (2, 300, 2, 2, 128, "none", 0.0, False),
    (1, 300, 4, 2, 64, "causal", 0.0, "mixed"),
    (1, 300, 4, 2, 80, "docs_both", 0.0, "mixed"),
    (1, 200, 4, 2, 128, "window", 30.0, "mixed"),
    (1, 260, 4, 2, 96, "all", 100.0, "mixed"),
    # few key/value heads with many query heads: clusters share a key tile
    (1, 513, 8, 1, 64, "docs", 0.0, False),
    (1, 900, 8, 1, 128, "causal", 30.0, False),
    (1, 1000, 16, 1, 96, "prefix", 20.0, True),
    (1, 1030, 16, 1, 80, "none", 0.0, False),
]


@pytest.mark.parametrize("flags", [0, bpt.BPT_FLAG_DETERMINISTIC])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_against_the_definition(case, flags):
    b, s, H, K, d, kind, cap, biased = case
    causal, begin, end = windows(kind, b, s, seed=s + d)
    slopes = [2.0 ** -(1 + 3 * n) for n in range(H)] if biased else None
    if biased == "mixed":  # steep, gentle and negative ones
        slopes = [(3.0, -0.02, 0.3, -2.0)[n % 4] for n in range(H)]
    cfg = LayerConfig(b=b, s=s, h=H * d, n_heads=H, n_kv_heads=K, head_dim=d, ffn_dim=64, causal=causal)
    mod = bpt.ScoreMod(as_int32(begin), as_int32(end), None if slopes is None else torch.tensor(slopes, device="cuda"), cap)
    qkv, dout = make(b, s, H, K, d, seed=s)
    got = run(cfg, mod, qkv, dout, flags)
    check_all(cfg, causal, begin, end, slopes, cap, qkv, dout, *got)
    if flags:
        again = run(cfg, mod, qkv, dout, flags)
        assert all(torch.equal(a, c) for a, c in zip(got, again))


def docs_mod(s, n, b=1):
    i = torch.arange(s, dtype=torch.int32, device="cuda")
    return bpt.ScoreMod(row_begin=(i // n * n).int().repeat(b), softcap=30.0)


def test_equals_the_plain_attention_without_modifiers():
    """No modifier: the plain calls' definition; O and the gradients agree to
    their own roundings (each side within them), the log-sum-exp to the plain
    one's bf16 row sums."""
    b, s, H, K, d = 2, 333, 4, 2, 128
    cfg = LayerConfig(b=b, s=s, h=H * d, n_heads=H, n_kv_heads=K, head_dim=d, ffn_dim=64)
    qkv, dout = make(b, s, H, K, d, seed=1)
    o, lse, dqkv = run(cfg, bpt.ScoreMod(), qkv, dout)
    o2, lse2, dqkv2 = torch.empty_like(o), torch.empty_like(lse), torch.empty_like(dqkv)
    bpt.bpt_attention_fwd(cfg, qkv.cuda(), o2, lse2)
    ws = bpt.alloc_bytes(bpt.bpt_attention_bwd_workspace_bytes(cfg))
    bpt.bpt_attention_bwd(cfg, qkv.cuda(), o2, lse2, dout.cuda(), dqkv2, ws)
    torch.cuda.synchronize()
    assert float((lse - lse2)[:, :, :s].abs().max()) <= 2.0 ** -8 * 1.02
    for a, c in ((o, o2), (dqkv, dqkv2)):
        assert float((a.float() - c.float()).norm() / c.float().norm()) < 5e-3


def test_masked_rows_leave_no_trace():
    """Whatever (finite) lies in rows that no window reaches changes nothing:
    the largest bf16 values in the padding of each sequence."""
    b, s, H, K, d = 3, 300, 4, 2, 64
    cfg = LayerConfig(b=b, s=s, h=H * d, n_heads=H, n_kv_heads=K, head_dim=d, ffn_dim=64, causal=0)
    n = [300, 131, 0]
    end = as_int32([n[i] if q < n[i] else 0 for i in range(b) for q in range(s)])
    qkv, dout = make(b, s, H, K, d, seed=2)
    slopes = torch.tensor([0.5, 0.1, 0.01, 0.0], device="cuda")
    for mod in (bpt.ScoreMod(None, end), bpt.ScoreMod(None, end, slopes, 20.0), bpt.ScoreMod(None, end, None, 100.0)):
        clean = [t.clone() for t in run(cfg, mod, qkv, dout, bpt.BPT_FLAG_DETERMINISTIC)]
        dirty, ddirty = qkv.clone().view(b, s, -1), dout.clone().view(b, s, -1)
        for i in range(b):
            dirty[i, n[i]:] = 3.3e38
            dirty[i, n[i]:, ::2] = -3.3e38
            ddirty[i, n[i]:] = 3.3e38
        got = run(cfg, mod, dirty.view(b * s, -1), ddirty.view(b * s, -1), bpt.BPT_FLAG_DETERMINISTIC)
        for a, c in zip(got, clean):
            fin = c.isfinite()
            assert torch.equal(fin, a.isfinite())
            if mod.softcap == 0.0:
                assert torch.equal(a, c)
            else:
                # a tile's scores, masked ones too, choose the form of tanh its
                # warp takes: within 1e-6 of each other, so a rounding to bf16
                # may fall to the other side, one step of 2^-7
                a, c = a[fin].double(), c[fin].double()
                assert float((a - c).norm()) <= 2.0 ** -7 * float(c.norm())
        o, lse, dqkv = (t.view(b, s, -1) if t.dim() == 2 else t for t in got)
        for i in range(b):
            assert not o[i, n[i]:].any() and not dqkv[i, n[i]:].any()
            assert bool((lse[i, :, n[i]:s] == -math.inf).all()) and not lse[i, :, s:].any()


def test_streams_and_graphs():
    """Two calls at once on two streams with workspaces of their own, and a
    captured forward and backward replayed on new inputs, give bitwise what
    the calls give alone (fixed-order mode)."""
    s, H, K, d = 700, 8, 2, 128
    cfg = LayerConfig(b=1, s=s, h=H * d, n_heads=H, n_kv_heads=K, head_dim=d, ffn_dim=64, flags=bpt.BPT_FLAG_DETERMINISTIC)
    mod = docs_mod(s, 150)
    ins = [make(1, s, H, K, d, seed=10 + i) for i in range(3)]
    want = [[t.clone() for t in run(cfg, mod, *x, flags=cfg.flags)] for x in ins]

    def buffers(x, do):
        return dict(x=x.cuda(), do=do.cuda(), o=torch.empty(s, H * d, dtype=torch.bfloat16, device="cuda"),
                    lse=torch.empty(1, H, bpt.s_pad(cfg), device="cuda"), dx=torch.empty(s, (H + 2 * K) * d, dtype=torch.bfloat16, device="cuda"),
                    ws=bpt.alloc_bytes(bpt.bpt_attention_mod_bwd_workspace_bytes(cfg)))

    def call(z, stream=None):
        bpt.bpt_attention_mod_fwd(cfg, mod, z["x"], z["o"], z["lse"], stream)
        bpt.bpt_attention_mod_bwd(cfg, mod, z["x"], z["o"], z["lse"], z["do"], z["dx"], z["ws"], stream)

    zs = [buffers(*x) for x in ins]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for z, st in zip(zs, streams):
            call(z, st)
    torch.cuda.synchronize()
    for z, w in zip(zs[:2], want):
        assert torch.equal(z["o"], w[0]) and torch.equal(z["lse"], w[1]) and torch.equal(z["dx"], w[2])
    graph = torch.cuda.CUDAGraph()
    z = zs[2]
    with torch.cuda.graph(graph):
        call(z)
    for x, w in zip(ins, want):
        z["x"].copy_(x[0])
        z["do"].copy_(x[1])
        z["o"].zero_(), z["dx"].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(z["o"], w[0]) and torch.equal(z["lse"], w[1]) and torch.equal(z["dx"], w[2])
    assert bpt.bpt_last_device_error() == (bpt.BPT_OK, 0)


@pytest.mark.parametrize("d,cap,biased", [(64, 0.0, False), (64, 30.0, True), (80, 0.0, True), (80, 20.0, False), (96, 0.0, False),
                                          (96, 50.0, True), (112, 30.0, False), (128, 0.0, True), (128, 50.0, False),
                                          (128, 0.0, False)])
def test_many_items_per_block(d, cap, biased):
    """Far more query and key tiles than blocks, some of them seen by nothing:
    every sequence of a batch gets bitwise what it gets alone (fixed-order mode),
    again and again, and within the roundings' size in the default mode."""
    b, s, H, K = 40, 391, 8, 4
    cfg = LayerConfig(b=b, s=s, h=H * d, n_heads=H, n_kv_heads=K, head_dim=d, ffn_dim=64, causal=0)
    gen = torch.Generator().manual_seed(d)
    begin, end = torch.zeros(b, s, dtype=torch.int32), torch.zeros(b, s, dtype=torch.int32)
    q = torch.arange(s, dtype=torch.int32)
    for i in range(b):
        n = [s, 0, 130, 257, 1][i % 5]  # the sequence's length
        size = int(torch.randint(1, s, (1,), generator=gen))
        if i % 3:  # documents
            begin[i] = q // size * size
        end[i] = torch.where(q < n, torch.clamp(q + 1, min=min(n, 40)) if i % 2 else torch.clamp(begin[i] + size, max=n), 0)
    slopes = torch.linspace(0.0, 0.3, H, device="cuda") if biased else None
    qkv, dout = make(b, s, H, K, d, seed=3)
    flag = bpt.BPT_FLAG_DETERMINISTIC
    mod = bpt.ScoreMod(begin.view(-1).cuda(), end.view(-1).cuda(), slopes, cap)
    got = [t.clone() for t in run(cfg, mod, qkv, dout, flag)]
    for i in range(b):
        rows = slice(i * s, (i + 1) * s)
        part = bpt.ScoreMod(begin[i].cuda(), end[i].cuda(), slopes, cap)
        o, lse, dx = run(cfg.with_(b=1), part, qkv[rows], dout[rows], flag)
        assert torch.equal(o, got[0][rows]) and torch.equal(lse[0], got[1][i]) and torch.equal(dx, got[2][rows]), i
    for _ in range(5):
        for a, c in zip(run(cfg, mod, qkv, dout, flag), got):
            assert torch.equal(a, c)
    # the forward has one order of sums in every mode; the backward's fp32 sums
    # differ in their last bits, so a rounding to bf16 may go the other way
    o, lse, dx = run(cfg, mod, qkv, dout)
    assert torch.equal(o, got[0]) and torch.equal(lse, got[1])
    assert float((dx.double() - got[2].double()).norm()) <= 2.0 ** -8 * float(got[2].double().norm())


def test_far_offsets():
    """A packed buffer of more than 2^31 elements: documents at its end equal
    the same documents alone, within both sides' roundings (their tiles differ)."""
    b, s, H, K, d, n = 3, 131072, 32, 8, 128, 128
    cfg = LayerConfig(b=b, s=s, h=H * d, n_heads=H, n_kv_heads=K, head_dim=d, ffn_dim=64, flags=bpt.BPT_FLAG_DETERMINISTIC)
    mod = docs_mod(s, n, b)
    g = torch.Generator(device="cuda").manual_seed(4)
    qkv = torch.randn(b * s, (H + 2 * K) * d, generator=g, device="cuda", dtype=torch.bfloat16)
    dout = torch.randn(b * s, H * d, generator=g, device="cuda", dtype=torch.bfloat16)
    assert qkv.numel() > 2 ** 31
    o, dqkv = torch.empty_like(dout), torch.empty_like(qkv)
    lse = torch.empty(b, H, s, device="cuda")
    ws = bpt.alloc_bytes(bpt.bpt_attention_mod_bwd_workspace_bytes(cfg))
    bpt.bpt_attention_mod_fwd(cfg, mod, qkv, o, lse)
    bpt.bpt_attention_mod_bwd(cfg, mod, qkv, o, lse, dout, dqkv, ws)
    torch.cuda.synchronize()
    assert bpt.bpt_last_device_error() == (bpt.BPT_OK, 0)
    # documents of one tile: the call on four of them alone runs the same tiles
    small = cfg.with_(b=1, s=4 * n)
    for at in (0, s - 4 * n, 2 * s - 4 * n, 3 * s - 4 * n):
        e = at + 4 * n
        so, sx = torch.empty(4 * n, H * d, dtype=torch.bfloat16, device="cuda"), torch.empty_like(qkv[at:e])
        sl = torch.empty(1, H, 4 * n, device="cuda")
        sws = bpt.alloc_bytes(bpt.bpt_attention_mod_bwd_workspace_bytes(small))
        part = bpt.ScoreMod(row_begin=(torch.arange(4 * n, device="cuda") // n * n).int(), softcap=30.0)
        bpt.bpt_attention_mod_fwd(small, part, qkv[at:e], so, sl)
        bpt.bpt_attention_mod_bwd(small, part, qkv[at:e], so, sl, dout[at:e].contiguous(), sx, sws)
        torch.cuda.synchronize()
        assert torch.equal(so, o[at:e]) and torch.equal(sl[0], lse[at // s, :, at % s:at % s + 4 * n])
        assert float((sx.float() - dqkv[at:e].float()).norm() / sx.float().norm()) < 1e-3


def test_lse_is_optional_and_debug_checks():
    s, H, K, d = 200, 2, 2, 80
    cfg = LayerConfig(b=1, s=s, h=H * d, n_heads=H, n_kv_heads=K, head_dim=d, ffn_dim=64)
    qkv, dout = make(1, s, H, K, d, seed=5)
    mod = docs_mod(s, 60)
    want = run(cfg, mod, qkv, dout, bpt.BPT_FLAG_DETERMINISTIC)
    o = torch.empty_like(want[0])
    bpt.bpt_attention_mod_fwd(cfg, mod, qkv.cuda(), o, None)
    torch.cuda.synchronize()
    assert torch.equal(o, want[0])
    got = run(cfg, mod, qkv, dout, bpt.BPT_FLAG_DETERMINISTIC | bpt.BPT_FLAG_DEBUG_CHECKS)
    assert all(torch.equal(a, c) for a, c in zip(got, want))


def test_refusals():
    s, H, K, d = 200, 2, 2, 64
    cfg = LayerConfig(b=1, s=s, h=H * d, n_heads=H, n_kv_heads=K, head_dim=d, ffn_dim=64)
    qkv, dout = (t.cuda() for t in make(1, s, H, K, d, seed=6))
    o, lse = torch.empty_like(dout), torch.empty(1, H, 256, device="cuda")
    dx, ws = torch.empty_like(qkv), bpt.alloc_bytes(bpt.bpt_attention_mod_bwd_workspace_bytes(cfg))
    plain = bpt.ScoreMod()
    lo = torch.zeros(s, dtype=torch.int32, device="cuda")
    bad = [
        lambda: bpt.bpt_attention_mod_fwd(cfg, bpt.ScoreMod(lo[:-1]), qkv, o, lse),
        lambda: bpt.bpt_attention_mod_fwd(cfg, bpt.ScoreMod(lo.long()), qkv, o, lse),
        lambda: bpt.bpt_attention_mod_fwd(cfg, bpt.ScoreMod(None, lo.cpu()), qkv, o, lse),
        lambda: bpt.bpt_attention_mod_fwd(cfg, bpt.ScoreMod(None, None, torch.zeros(1, device="cuda")), qkv, o, lse),
        lambda: bpt.bpt_attention_mod_fwd(cfg, bpt.ScoreMod(softcap=-3.0), qkv, o, lse),
        lambda: bpt.bpt_attention_mod_fwd(cfg, plain, qkv[:, ::2], o, lse),
        lambda: bpt.bpt_attention_mod_fwd(cfg, plain, qkv.half(), o, lse),
        lambda: bpt.bpt_attention_mod_fwd(cfg, plain, qkv, o[:-1], lse),
        lambda: bpt.bpt_attention_mod_fwd(cfg, plain, qkv, o, lse[:, :, :s].contiguous()),
        lambda: bpt.bpt_attention_mod_fwd(cfg, plain, qkv, qkv.view(-1)[:o.numel()].view_as(o), lse),
        lambda: bpt.bpt_attention_mod_bwd(cfg, plain, qkv, o, lse, dout, qkv, ws),
        lambda: bpt.bpt_attention_mod_bwd(cfg, plain, qkv, o, None, dout, dx, ws),
        lambda: bpt.bpt_attention_mod_bwd(cfg, plain, qkv, o, lse, dout, dx, ws[:1024]),
    ]
    for call in bad:
        with pytest.raises(bpt.BptError):
            call()
    torch.cuda.synchronize()
    assert bpt.bpt_last_device_error() == (bpt.BPT_OK, 0)
