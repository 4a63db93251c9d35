"""Pins of the fp64 definitions in oracle/train_ops.py: PyTorch autograd in
fp64, finite differences and closed forms."""
import numpy as np
import pytest
import torch

from oracle import ref
from oracle import train_ops as T


def _rand(seed, *shape):
    return np.random.default_rng(seed).standard_normal(shape)


CASES = [
    dict(causal=1),
    dict(causal=0),
    dict(causal=1, begin=[0, 0, 0, 3, 3, 3, 3, 7, 7]),
    dict(causal=0, end=[4, 4, 4, 4, 5, 6, 7, 0, 0]),
    dict(causal=1, begin=[0, 1, 1, 2, 3, 4, 9, 6, 8], cap=2.0, slope=0.3),
    dict(causal=0, begin=[0, 0, 2, 2, 2, 5, 5, 5, 5], end=[2, 2, 5, 5, 5, 9, 9, 9, 9], cap=0.7, slope=0.1),
]


@pytest.mark.parametrize("case", CASES)
def test_attention_head_matches_autograd_and_differences(case):
    s, d = 9, 6
    q, k, v, do = (_rand(i, s, d) for i in range(4))
    begin, end, cap, slope = case.get("begin"), case.get("end"), case.get("cap", 0.0), case.get("slope", 0.0)
    ok = T.allowed(s, case["causal"], begin, end)
    o, lse, dq, dk, dv = T.attention_mod_head(q, k, v, ok, slope, cap, do)
    tq, tk, tv = (torch.tensor(a, requires_grad=True) for a in (q, k, v))
    y = tq @ tk.T / d ** 0.5
    if cap:
        y = cap * torch.tanh(y / cap)
    i = torch.arange(s)
    y = y - slope * (i[:, None] - i).abs().double()
    y = y.masked_fill(~torch.tensor(ok), -1e300)
    p = torch.softmax(y, -1) * torch.tensor(ok)
    to = p @ tv
    to.backward(torch.tensor(do))
    for got, want in ((o, to.detach()), (dq, tq.grad), (dk, tk.grad), (dv, tv.grad)):
        np.testing.assert_allclose(got, want.numpy(), atol=1e-12)
    some = ok.any(1)
    assert np.all(lse[~some] == -np.inf) and np.all(o[~some] == 0) and np.all(dq[~some] == 0)
    np.testing.assert_allclose(lse[some], torch.logsumexp(y, -1).detach().numpy()[some], atol=1e-12)
    # differences of sum(o * do) along one direction per input
    h = 1e-6
    for a, g, at in ((q, dq, 0), (k, dk, 1), (v, dv, 2)):
        e = _rand(9 + at, s, d)
        hi = [x + h * e if j == at else x for j, x in enumerate((q, k, v))]
        lo = [x - h * e if j == at else x for j, x in enumerate((q, k, v))]
        diff = ((T.attention_mod_head(*hi, ok, slope, cap)[0] - T.attention_mod_head(*lo, ok, slope, cap)[0]) * do).sum()
        assert abs(diff / (2 * h) - (g * e).sum()) < 1e-7


def test_plain_attention_is_the_layers():
    q, k, v, do = (_rand(20 + i, 11, 8) for i in range(4))
    for causal in (True, False):
        o, lse, *g = T.attention_mod_head(q, k, v, T.allowed(11, causal), do=do)
        o2, lse2 = ref.attention_head(q, k, v, causal)
        np.testing.assert_allclose(o, o2, atol=1e-13)
        np.testing.assert_allclose(lse, lse2, atol=1e-13)
        for a, b in zip(g, ref.attention_head_backward(q, k, v, do, causal)):
            np.testing.assert_allclose(a, b, atol=1e-13)


def test_documents_are_separate_sequences():
    """Packed documents give what each gives alone, heads grouped."""
    H, K, d, cuts = 4, 2, 6, [0, 3, 4, 10]
    qkv, do = _rand(30, 10, (H + 2 * K) * d), _rand(31, 10, H * d)
    begin = np.repeat(cuts[:-1], np.diff(cuts))
    slopes = [0.5, 0.25, 0.125, 0.0625]
    o, lse, dx = T.attention_mod(qkv, 1, 10, H, K, d, 1, begin, None, slopes, 3.0, do)
    for a, e in zip(cuts, cuts[1:]):
        o1, lse1, dx1 = T.attention_mod(qkv[a:e], 1, e - a, H, K, d, 1, None, None, slopes, 3.0, do[a:e])
        np.testing.assert_allclose(o[a:e], o1, atol=1e-13)
        np.testing.assert_allclose(lse[:, :, a:e], lse1, atol=1e-13)
        np.testing.assert_allclose(dx[a:e], dx1, atol=1e-13)


@pytest.mark.parametrize("norm,base", [(True, 10000.0), (True, 0.0), (False, 500.0)])
def test_norm_rope_matches_autograd(norm, base):
    H, K, d, s = 3, 1, 8, 5
    rows, eps = 10, 1e-5
    x, dy = _rand(40, rows, (H + 2 * K) * d), _rand(41, rows, (H + 2 * K) * d)
    wq, wk = (1 + 0.1 * _rand(42, d), 1 + 0.1 * _rand(43, d)) if norm else (None, None)
    pos = np.random.default_rng(44).integers(-5, 200, rows)
    for positions in (None, pos):
        tx = torch.tensor(x, requires_grad=True)
        tw = [torch.tensor(w, requires_grad=True) for w in (wq, wk)] if norm else None
        p = torch.arange(rows) % s if positions is None else torch.tensor(positions)
        u = tx.view(rows, H + 2 * K, d)
        z = u[:, :H + K]
        if norm:
            w = torch.cat((tw[0].expand(H, d), tw[1].expand(K, d)))
            z = z * torch.rsqrt(z.square().mean(-1, keepdim=True) + eps) * w
        if base:
            a = p[:, None].double() * base ** (-2 * torch.arange(d // 2).double() / d)
            c = torch.polar(torch.ones(1, dtype=torch.float64), a)[:, None]
            c = torch.complex(z[..., :d // 2], z[..., d // 2:]) * c
            z = torch.cat((c.real, c.imag), -1)
        y = torch.cat((z, u[:, H + K:]), 1).reshape(rows, -1)
        y.backward(torch.tensor(dy))
        np.testing.assert_allclose(T.norm_rope(x, s, H, K, d, wq, wk, base, eps, positions), y.detach().numpy(), atol=1e-12)
        dx, dwq, dwk = T.norm_rope(x, s, H, K, d, wq, wk, base, eps, positions, dy)
        np.testing.assert_allclose(dx, tx.grad.numpy(), atol=1e-12)
        if norm:
            np.testing.assert_allclose(dwq, tw[0].grad.numpy(), atol=1e-12)
            np.testing.assert_allclose(dwk, tw[1].grad.numpy(), atol=1e-12)


def test_clip_matches_torch():
    gs = [_rand(50, 7, 3), _rand(51, 5), _rand(52, 1)]
    for limit in (0.5, 100.0, float("inf")):
        ps = [torch.nn.Parameter(torch.zeros(g.shape, dtype=torch.float64)) for g in gs]
        for p, g in zip(ps, gs):
            p.grad = torch.tensor(g)
        norm = torch.nn.utils.clip_grad_norm_(ps, limit)
        n, out = T.clip(gs, limit)
        assert abs(n - float(norm)) < 1e-12
        for p, o in zip(ps, out):
            np.testing.assert_allclose(p.grad.numpy(), o, atol=1e-12)
