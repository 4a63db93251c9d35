"""The head norm with rotation and the gradient clipping on the GPU against
their fp64 definitions.

Tolerances.  A bf16 output is one rounding of an fp32 value: off by at most
2^-8 of its size from the fp32 value (2^-8 |y| covers half a step), whose own
error is a few fp32 roundings: norm_rope's outputs are sums of two products
with |sin|, |cos| <= 1 of values that carry about 8 roundings (sum of d
squares, rsqrt at 2 units, the products), under 32 * 2^-24 of the pair's size.
An angle's argument is rounded to 2^-25 half turns, under 2^-23 rad.  A weight
gradient is a sum of N fp32 terms in fp32 (per lane, then tree): its error is
bounded by 2^-24 (chain + 16) sum |term| with the longest chain of additions,
rows * heads / lanes + lanes + blocks, under 2^12 for every size here."""
import math

import numpy as np
import pytest
import torch

import blockwise_attention_ffn_gb300 as bpt
from blockwise_attention_ffn_gb300.presets import LayerConfig
from oracle import train_ops as T
from tests.gpu_helpers import to64

pytestmark = pytest.mark.gpu


def cfg_of(b, s, H, K, d, **kw):
    return LayerConfig(b=b, s=s, h=H * d, n_heads=H, n_kv_heads=K, head_dim=d, ffn_dim=64, **kw)


def sync():
    torch.cuda.synchronize()
    assert bpt.bpt_last_device_error() == (bpt.BPT_OK, 0)


# ------------------------------------------------------------------ head norm and rotation

NR = [
    # b, s, H, K, d, base, norm, positions
    (1, 1, 1, 1, 64, 10000.0, True, None),
    (2, 37, 4, 4, 80, 10000.0, True, None),
    (3, 50, 6, 2, 96, 500000.0, True, "random"),
    (1, 129, 7, 1, 112, 500.0, True, "random"),
    (1, 300, 32, 8, 128, 500000.0, True, "random"),
    (2, 65, 3, 3, 128, 0.0, True, None),
    (1, 77, 5, 5, 80, 10000.0, False, "random"),
    (1, 2000, 2, 1, 64, 10000.0, True, "far"),
]


def nr_inputs(b, s, H, K, d, norm, positions, seed=0):
    g = torch.Generator().manual_seed(seed + s + d)
    rows, width = b * s, (H + 2 * K) * d
    qkv = (2 * torch.randn(rows, width, generator=g)).to(torch.bfloat16)
    qkv[0, :d] = 0  # a head of zeros: r = eps^(-1/2)
    qkv[-1, -3 * d:] *= 1e4
    dout = torch.randn(rows, width, generator=g).to(torch.bfloat16)
    w = [(1 + 0.2 * torch.randn(d, generator=g)).to(torch.bfloat16) if norm else None for _ in range(2)]
    top = 2 ** 31 - 1 if positions == "far" else 200000
    pos = None if positions is None else torch.randint(-top, top, (rows,), generator=g, dtype=torch.int64).to(torch.int32)
    return qkv, dout, w, pos


def cu(t):
    return None if t is None else t.cuda()


def pair_size(y, rows, n, d):
    """|(u, v)| of every element's rotation pair."""
    y = np.abs(y.reshape(rows, n, d))
    m = np.hypot(y[..., :d // 2], y[..., d // 2:])
    return np.concatenate((m, m), -1).reshape(rows, -1)


@pytest.mark.parametrize("case", NR)
@pytest.mark.parametrize("in_place", [False, True])
def test_norm_rope_forward(case, in_place):
    b, s, H, K, d, base, norm, positions = case
    cfg = cfg_of(b, s, H, K, d, rope_base=base)
    qkv, _, w, pos = nr_inputs(b, s, H, K, d, norm, positions)
    x = qkv.cuda()
    out = x if in_place else torch.full_like(x, float("nan"))
    bpt.bpt_qk_norm_rope_fwd(cfg, x, cu(w[0]), cu(w[1]), cu(pos), out)
    sync()
    want = T.norm_rope(to64(qkv), s, H, K, d, *(None if v is None else to64(v) for v in w), base, cfg.norm_eps,
                       None if pos is None else pos.numpy())
    size = pair_size(want, b * s, H + 2 * K, d)
    err = np.abs(to64(out) - want)
    # the angle's argument (2^-23 rad, plus the oracle's own double product at
    # positions up to 2^31: 2^-21 rad) turns the pair by that much of its size
    bound = 2.0 ** -8 * np.abs(want) + (32 * 2.0 ** -24 + 2.0 ** -20) * size
    assert np.all(err <= bound), float(np.max(err - bound))
    assert torch.equal(out.cpu()[:, (H + K) * d:], qkv[:, (H + K) * d:])  # V passes through


@pytest.mark.parametrize("case", NR)
@pytest.mark.parametrize("in_place", [False, True])
def test_norm_rope_backward(case, in_place):
    b, s, H, K, d, base, norm, positions = case
    cfg = cfg_of(b, s, H, K, d, rope_base=base)
    qkv, dout, w, pos = nr_inputs(b, s, H, K, d, norm, positions, seed=1)
    dy = dout.cuda()
    dqkv = dy if in_place else torch.full_like(dy, float("nan"))
    dw = [torch.full((d,), float("nan"), device="cuda") for _ in range(2)] if norm else [None, None]
    ws = bpt.alloc_bytes(bpt.bpt_qk_norm_rope_workspace_bytes(cfg)) if norm else None
    ws.fill_(255) if norm else None
    bpt.bpt_qk_norm_rope_bwd(cfg, cu(qkv) if norm else None, cu(w[0]), cu(w[1]), cu(pos), dy, dqkv, *dw, ws)
    sync()
    w64 = [None if v is None else to64(v) for v in w]
    p = None if pos is None else pos.numpy()
    want, dwq, dwk = T.norm_rope(to64(qkv), s, H, K, d, *w64, base, cfg.norm_eps, p, to64(dout))
    err = np.abs(to64(dqkv) - want).reshape(b * s, H + 2 * K, d)
    want3 = want.reshape(b * s, H + 2 * K, d)
    # dx = r (g - n mean(g n)): both terms are at most r |g|_2-sized before
    # they cancel, and each carries about 12 fp32 roundings and the angle's
    # (2^-20 as above)
    x3 = to64(qkv).reshape(b * s, H + 2 * K, d)
    r = 1 / np.sqrt((x3 * x3).mean(-1, keepdims=True) + cfg.norm_eps) if norm else np.ones((b * s, H + 2 * K, 1))
    g = np.abs(to64(dout)).reshape(x3.shape)
    big = 1.0 if not norm else max(np.abs(v).max() for v in w64)
    term = r * big * np.sqrt((g * g).sum(-1, keepdims=True)) * (1 + np.abs(x3 * r) if norm else 1)
    bound = 2.0 ** -8 * np.abs(want3) + (64 * 2.0 ** -24 + 2.0 ** -20) * term
    assert np.all(err <= bound), float(np.max(err - bound))
    assert torch.equal(dqkv.cpu()[:, (H + K) * d:], dout[:, (H + K) * d:])
    if norm:
        # sum of |dn n| over the rows and heads: dn's pair size times |n|
        dn = pair_size(to64(dout), b * s, H + 2 * K, d).reshape(x3.shape)
        for at, n, got, ref in ((0, H, dw[0], dwq), (H, K, dw[1], dwk)):
            terms = (dn * np.abs(x3 * r))[:, at:at + n].sum((0, 1))
            # random-order error grows like the square root of the 2^12 chain;
            # the bound below is the worst case of it
            bound = (2.0 ** -24 * 2.0 ** 12 + 2.0 ** -20) * terms
            assert np.all(np.abs(to64(got) - ref) <= bound)
        # accumulation adds to what is there, in the same fixed order
        acc = [v.clone() for v in dw]
        bpt.bpt_qk_norm_rope_bwd(cfg.with_(flags=bpt.BPT_FLAG_ACCUM_GRADS), cu(qkv), cu(w[0]), cu(w[1]), cu(pos),
                                 cu(dout), torch.empty_like(dqkv), *acc, ws)
        sync()
        for a, v in zip(acc, dw):
            assert torch.equal(a, v + v)


@pytest.mark.parametrize("H,K,d", [(4, 2, 80), (2, 1, 64), (32, 8, 128), (6, 6, 112), (3, 1, 96), (40, 40, 128)])
@pytest.mark.parametrize("in_place", [False, True])
def test_norm_rope_many_rows(H, K, d, in_place):
    """More rows than the SMs take at once, against calls on a few rows each
    (bitwise: a row's result does not depend on the rest), with a norm and
    without."""
    s = 20011
    cfg = cfg_of(1, s, H, K, d, rope_base=10000.0)
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(s, (H + 2 * K) * d, generator=g, device="cuda").to(torch.bfloat16)
    dy = torch.randn(s, (H + 2 * K) * d, generator=g, device="cuda").to(torch.bfloat16)
    norm = [(1 + 0.1 * torch.randn(d, generator=g, device="cuda")).to(torch.bfloat16) for _ in range(2)]
    pos = torch.arange(s, dtype=torch.int32, device="cuda")
    ws = bpt.alloc_bytes(bpt.bpt_qk_norm_rope_workspace_bytes(cfg))
    rng = np.random.default_rng(5)
    for w in (norm, [None, None]):
        out, dx = (x.clone(), dy.clone()) if in_place else (torch.empty_like(x), torch.empty_like(x))
        bpt.bpt_qk_norm_rope_fwd(cfg, out if in_place else x, *w, None, out)
        dw = [torch.zeros(d, device="cuda") for _ in range(2)]
        bpt.bpt_qk_norm_rope_bwd(cfg, x, *w, None, dx if in_place else dy, dx, *dw, ws)
        sync()
        for a in (0, s - 9, *rng.integers(9, s - 18, 6).tolist()):
            e = a + 9
            part, dpart = torch.empty_like(x[a:e]), torch.empty_like(x[a:e])
            small = cfg.with_(s=e - a)
            bpt.bpt_qk_norm_rope_fwd(small, x[a:e], *w, pos[a:e].clone(), part)
            bpt.bpt_qk_norm_rope_bwd(small, x[a:e], *w, pos[a:e].clone(), dy[a:e], dpart,
                                     *[torch.zeros(d, device="cuda") for _ in range(2)], ws)
            sync()
            assert torch.equal(part, out[a:e]) and torch.equal(dpart, dx[a:e])
        if w[0] is None:
            continue
        # the weights' gradients of all rows against fp64
        u = x.double().view(s, H + 2 * K, d)[:, :H + K]
        n = u * torch.rsqrt(u.square().mean(-1, keepdim=True) + cfg.norm_eps)
        a = pos.double()[:, None] * 10000.0 ** (-2 * torch.arange(d // 2, device="cuda").double() / d)
        z = dy.double().view(s, H + 2 * K, d)[:, :H + K]
        z = torch.complex(z[..., :d // 2].contiguous(), z[..., d // 2:].contiguous()) * torch.polar(torch.ones_like(a), -a)[:, None]
        terms = torch.cat((z.real, z.imag), -1) * n
        for got, part in zip(dw, (terms[:, :H], terms[:, H:])):
            # chains of at most rows * heads / lanes additions per lane, under
            # 2^10, and angles' 2^-20: both of the terms' sum of sizes
            bound = (2.0 ** -24 * 2 ** 10 + 2.0 ** -20) * part.abs().sum((0, 1))
            assert bool(((got.double() - part.sum((0, 1))).abs() <= bound).all())


@pytest.mark.parametrize("b,s,H,K,d", [(23, 1291, 2, 1, 64), (5000, 7, 2, 1, 64), (30001, 1, 1, 1, 80), (9, 555, 32, 8, 128),
                                       (7, 901, 12, 12, 96), (2, 30011, 1, 1, 112)])
def test_norm_rope_rows_of_many_sequences(b, s, H, K, d):
    """Without positions a row's is its index in its sequence, whatever part of
    how many sequences a block takes at once (bitwise the call with them)."""
    cfg = cfg_of(b, s, H, K, d, rope_base=10000.0)
    g = torch.Generator(device="cuda").manual_seed(b)
    x, dy = (torch.randn(b * s, (H + 2 * K) * d, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    w = [(1 + 0.1 * torch.randn(d, generator=g, device="cuda")).to(torch.bfloat16) for _ in range(2)]
    ws = bpt.alloc_bytes(bpt.bpt_qk_norm_rope_workspace_bytes(cfg))
    got = []
    for pos in (None, (torch.arange(b * s, device="cuda") % s).to(torch.int32)):
        out, dx, dw = torch.empty_like(x), torch.empty_like(x), [torch.empty(d, device="cuda") for _ in range(2)]
        bpt.bpt_qk_norm_rope_fwd(cfg, x, *w, pos, out)
        bpt.bpt_qk_norm_rope_bwd(cfg, x, *w, pos, dy, dx, *dw, ws)
        sync()
        got.append([out, dx, *dw])
    for a, c in zip(*got):
        assert torch.equal(a, c)
    # and the first row of the last sequences against a call on one row each
    one = cfg.with_(b=3, s=1)
    rows = torch.arange(b - min(b, 3), b, device="cuda") * s
    part = torch.empty_like(x[:3])
    bpt.bpt_qk_norm_rope_fwd(one.with_(b=len(rows)), x[rows], *w, None, part[:len(rows)])
    sync()
    assert torch.equal(part[:len(rows)], got[0][0][rows])


def test_norm_rope_refusals():
    cfg = cfg_of(1, 8, 2, 1, 64, rope_base=10000.0)
    x = torch.zeros(8, 256, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(x)
    f = torch.empty(64, device="cuda")
    ws = bpt.alloc_bytes(bpt.bpt_qk_norm_rope_workspace_bytes(cfg))
    big = torch.zeros(16 * 256, dtype=torch.bfloat16, device="cuda")
    bad = [
        lambda: bpt.bpt_qk_norm_rope_fwd(cfg, x, w, None, None, out),
        lambda: bpt.bpt_qk_norm_rope_fwd(cfg.with_(rope_base=0.0), x, None, None, None, out),
        lambda: bpt.bpt_qk_norm_rope_fwd(cfg, x.float(), w, w, None, out),
        lambda: bpt.bpt_qk_norm_rope_fwd(cfg, x.cpu(), w, w, None, out),
        lambda: bpt.bpt_qk_norm_rope_fwd(cfg, x[:7], w, w, None, out),
        lambda: bpt.bpt_qk_norm_rope_fwd(cfg, x, w[:32], w, None, out),
        lambda: bpt.bpt_qk_norm_rope_fwd(cfg, x, w, w, torch.zeros(8, device="cuda"), out),
        lambda: bpt.bpt_qk_norm_rope_fwd(cfg, x, w, w, torch.zeros(7, dtype=torch.int32, device="cuda"), out),
        lambda: bpt.bpt_qk_norm_rope_fwd(cfg, big[:2048], w, w, None, big[1024:]),
        lambda: bpt.bpt_qk_norm_rope_bwd(cfg, x, w, w, None, out, x, f, f.clone(), ws),
        lambda: bpt.bpt_qk_norm_rope_bwd(cfg, x, w, w, None, out, out, f, None, ws),
        lambda: bpt.bpt_qk_norm_rope_bwd(cfg, x, w, w, None, out, out, f, f.clone(), ws[:256]),
        lambda: bpt.bpt_qk_norm_rope_fwd(cfg.with_(head_dim=72), x, w, w, None, out),
    ]
    for call in bad:
        with pytest.raises(bpt.BptError):
            call()
    sync()


# ------------------------------------------------------------------ clipping

def clip_call(grads, limit, out=None, flags=0):
    norm = torch.full((1,), float("nan"), device="cuda")
    ws = bpt.alloc_bytes(bpt.bpt_clip_workspace_bytes())
    ws.fill_(255)
    bpt.bpt_clip_grads(grads, limit, norm, ws, out=out, flags=flags)
    sync()
    return float(norm)


def clip_check(grads, limit, norm, out):
    """norm: at most 32 squares in fp32 (5 roundings deep per unit, 8 more),
    the rest in fp64, halved by the root, plus its own rounding: 2^-20.  An
    output: the factor's rounding and the norm's, one product, one rounding."""
    want, scaled = T.clip([to64(g) for g in grads], limit)
    assert abs(norm - want) <= 2.0 ** -20 * want
    for g, o, w in zip(grads, out, scaled):
        tol = (2.0 ** -8 if g.dtype == torch.bfloat16 else 0.0) + 2.0 ** -18
        assert np.all(np.abs(to64(o) - w) <= tol * np.abs(w))


SIZES = [[1], [3, 8, 0, 5], [8192], [8193, 16384, 7], [100000, 3, 250001], [1] * 70, [1000 + 17 * i for i in range(80)]]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{s[0]}")
@pytest.mark.parametrize("limit", [0.25, 1e9, math.inf])
@pytest.mark.parametrize("kind", ["fp32", "bf16", "mixed"])
def test_clip(sizes, limit, kind):
    g = torch.Generator().manual_seed(len(sizes) + sizes[0])
    types = {"fp32": [torch.float32], "bf16": [torch.bfloat16], "mixed": [torch.float32, torch.bfloat16]}[kind]
    grads = [torch.randn(n, generator=g).to(types[i % len(types)]).cuda() for i, n in enumerate(sizes)]
    out = [torch.full_like(t, float("nan")) for t in grads]
    norm = clip_call(grads, limit, out)
    clip_check(grads, limit, norm, out)
    before = [t.clone() for t in grads]
    assert clip_call(grads, limit) == norm  # in place: the same bits
    for t, o, b in zip(grads, out, before):
        assert torch.equal(t, o)
        assert limit == 0.25 or torch.equal(t, b)


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
def test_clip_unaligned(kind):
    """Gradients and outputs that start anywhere, together and apart."""
    g = torch.Generator().manual_seed(5)
    grads, outs = [], []
    for n in (1, 5, 8200, 20001):
        for a, c in ((0, 0), (1, 1), (3, 3), (1, 2), (0, 5)):
            grads.append(torch.randn(n + 8, generator=g).to(kind).cuda()[a:a + n])
            outs.append(torch.zeros(n + 8, device="cuda", dtype=kind)[c:c + n])
    norm = clip_call(grads, 1.0, outs)
    clip_check(grads, 1.0, norm, outs)
    for t in outs:  # nothing beside the outputs was written
        base = t._base
        at = t.storage_offset()
        assert not base[:at].any() and not base[at + t.numel():].any()


def test_clip_many_tensors():
    """More tensors than one table holds (1000)."""
    g = torch.Generator(device="cuda").manual_seed(6)
    flat = torch.randn(2300 * 40, generator=g, device="cuda")
    grads = [flat[40 * i:40 * i + 1 + i % 40] for i in range(2300)]
    outs = [torch.empty_like(t) for t in grads]
    norm = clip_call(grads, 2.0, outs)
    clip_check(grads, 2.0, norm, outs)


@pytest.mark.parametrize("scale", [1e-30, 1e-42, 1e25, 3e37])
def test_clip_range(scale):
    """Norms whose squares leave fp32."""
    x = torch.rand(5000, generator=torch.Generator().manual_seed(7), dtype=torch.float64).add(0.5)
    grads = [(x * scale).float().cuda(), torch.zeros(3000, device="cuda")]
    out = [torch.empty_like(t) for t in grads]
    norm = clip_call(grads, 1.0, out)
    want, _ = T.clip([to64(t) for t in grads], 1.0)
    if want > 3.4e38:
        assert norm == math.inf
    else:
        # below 2^-126 the norm itself has fewer bits
        assert abs(norm - want) <= 2.0 ** -20 * want + 2.0 ** -149
        assert torch.isfinite(out[0]).all()


def test_clip_special_values():
    one = torch.ones(9000, device="cuda")
    for bad, want in ((math.inf, math.inf), (-math.inf, math.inf), (math.nan, math.nan)):
        t = one.clone()
        t[4097] = bad
        out = [torch.empty_like(t)]
        norm = clip_call([t], 1.0, out)
        assert math.isnan(norm) if math.isnan(want) else norm == want
        o = out[0].cpu()
        if math.isnan(want):
            assert o.isnan().all()
        else:  # a factor of 0: 0 * inf is NaN
            assert o[4097].isnan() and (o[:4097] == 0).all()
    assert clip_call([], 1.0) == 0.0
    assert clip_call([torch.zeros(0, device="cuda")], 1.0) == 0.0
    z = torch.zeros(100, device="cuda")
    assert clip_call([z], 1.0) == 0.0 and not z.any()


def test_clip_is_repeatable_and_captures():
    g = torch.Generator(device="cuda").manual_seed(8)
    grads = [torch.randn(n, generator=g, device="cuda") for n in (3000001, 77, 500000)]
    outs = [torch.empty_like(t) for t in grads]
    norms = {clip_call(grads, 1.0, outs) for _ in range(5)}
    assert len(norms) == 1
    want = [o.clone() for o in outs]
    norm = torch.zeros(1, device="cuda")
    ws = bpt.alloc_bytes(bpt.bpt_clip_workspace_bytes())
    st = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=st):
        bpt.bpt_clip_grads(grads, 1.0, norm, ws, out=outs)
    for o in outs:
        o.zero_()
    grads[1].mul_(4)
    graph.replay()
    sync()
    clip_check(grads, 1.0, float(norm), outs)
    grads[1].div_(4)
    graph.replay()
    sync()
    assert {float(norm)} == norms and all(torch.equal(a, b) for a, b in zip(outs, want))


def test_clip_far_offsets():
    """A gradient of more than 2^31 elements: its squares and its last element."""
    n = 2 ** 31 + 12345
    t = torch.full((n,), 2.0 ** -10, dtype=torch.bfloat16, device="cuda")
    t[-1] = 64.0
    norm = clip_call([t], 1.0)
    want = math.sqrt((n - 1) * 2.0 ** -20 + 64.0 ** 2)
    assert abs(norm - want) <= 2.0 ** -20 * want
    for i, v in ((0, 2.0 ** -10), (n // 2, 2.0 ** -10), (n - 2, 2.0 ** -10), (n - 1, 64.0)):
        assert abs(float(t[i]) - v / want) <= 2.0 ** -8 * v / want + 2.0 ** -18 * v


def test_norm_rope_streams_and_graphs():
    """Two calls at once on two streams, and captured calls replayed on other
    inputs, both forms (few rows and many)."""
    H, K, d = 8, 4, 64
    for s in (50, 12000):
        cfg = cfg_of(1, s, H, K, d, rope_base=10000.0)
        g = torch.Generator(device="cuda").manual_seed(s)
        mk = lambda: torch.randn(s, (H + 2 * K) * d, generator=g, device="cuda").bfloat16()  # noqa: E731
        w = torch.ones(d, device="cuda", dtype=torch.bfloat16)
        zs = [dict(x=mk(), dy=mk(), out=mk(), dx=mk(), a=torch.zeros(d, device="cuda"), c=torch.zeros(d, device="cuda"),
                   ws=bpt.alloc_bytes(bpt.bpt_qk_norm_rope_workspace_bytes(cfg))) for _ in range(3)]

        def call(z, stream=None):
            bpt.bpt_qk_norm_rope_fwd(cfg, z["x"], w, w, None, z["out"], stream)
            bpt.bpt_qk_norm_rope_bwd(cfg, z["x"], w, w, None, z["dy"], z["dx"], z["a"], z["c"], z["ws"], stream)

        want = []
        for z in zs:
            call(z)
            sync()
            want.append({k: v.clone() for k, v in z.items() if k != "ws"})
        streams = [torch.cuda.Stream() for _ in range(2)]
        for _ in range(20):
            for z, st in zip(zs, streams):
                call(z, st)
        sync()
        for z, v in zip(zs, want):
            assert all(torch.equal(z[k], v[k]) for k in v)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(zs[2])
        for v in want:
            zs[2]["x"].copy_(v["x"])
            zs[2]["dy"].copy_(v["dy"])
            graph.replay()
            sync()
            assert all(torch.equal(zs[2][k], v[k]) for k in v)


def test_clip_refusals():
    a = torch.ones(64, device="cuda")
    norm = torch.full((1,), 7.0, device="cuda")
    ws = bpt.alloc_bytes(bpt.bpt_clip_workspace_bytes())
    call = lambda gs, limit=1.0, n=norm, w=ws, **kw: bpt.bpt_clip_grads(gs, limit, n, w, **kw)  # noqa: E731
    bad = [
        lambda: call([a], 0.0), lambda: call([a], -1.0), lambda: call([a], math.nan), lambda: call([a.double()]),
        lambda: call([a.cpu()]), lambda: call([a[::2]]), lambda: call([a, a]), lambda: call([a[:40], a[32:]]),
        lambda: call([a], out=[]), lambda: call([a], out=[a.bfloat16()]), lambda: call([a[:32]], out=[a[16:48]]),
        lambda: call([a, a.clone()], out=[a.clone(), a]), lambda: call([a], w=ws[:128]),
        lambda: call([a], n=norm.double()), lambda: call([a], flags=1),
    ]
    for c in bad:
        with pytest.raises(bpt.BptError):
            c()
    sync()
    assert float(norm) == 7.0 and bool((a == 1).all())
    # the same gradient read by two outputs is not a conflict
    o = [torch.empty_like(a), torch.empty_like(a)]
    assert abs(clip_call([a, a], 1.0, o) - math.sqrt(128)) < 1e-4
    # the debug flag: the call reports for itself
    clip_call([a], math.inf, flags=bpt.BPT_FLAG_DEBUG_CHECKS)
