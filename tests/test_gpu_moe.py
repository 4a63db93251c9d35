"""The router and the experts' network on the GPU against fp64.

Whole numbers (ids, offsets, order, slot) are equal.  The router's fp32 values
come from expf, sums over at most E values and a division: below 64 roundings
of 2^-24 of the value; a gradient is a difference of terms of size
q (|g| + sum |g| q), each with as many; losses add an fp32 sum over the rows of
a block (at most n / 256 + 64 of them, all positive).

The experts' network rounds to bf16, at 2^-8 of the value at most, what passes
from one product to the next.  y: act, the choice's row, y; dx: the saved pair
twice, its slope's product, the choice's row, dx; the matrices: the saved pair
twice, the operand, the result; dweights: the saved pair twice, the result.
The errors enter sums in which none is amplified beyond the sum itself, so in
the 2-norm of a whole tensor the count of roundings times 2^-8 covers them."""
import math

import pytest
import torch

import blockwise_attention_ffn_gb300 as bpt
from blockwise_attention_ffn_gb300.presets import MoeConfig

pytestmark = pytest.mark.gpu

F32, BF16 = bpt.BPT_DTYPE_F32, bpt.BPT_DTYPE_BF16
KIND = {F32: torch.float32, BF16: torch.bfloat16}
U = 2.0 ** -24


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def sync():
    torch.cuda.synchronize()
    assert bpt.bpt_last_device_error() == (bpt.BPT_OK, 0)


# ------------------------------------------------------------------ the router

def routes_of(z, k, norm):
    """ids, weights, offsets, order, slot of fp64 logits, one choice at a time."""
    n, E = z.shape
    left, ids, tops = z.clone(), [], []
    for _ in range(k):
        top = left.max(-1, keepdim=True).values
        first = (left == top).int().argmax(-1, keepdim=True)
        ids.append(torch.where(top > -math.inf, first, -1))
        tops.append(top)
        left.scatter_(-1, first, -math.inf)
    ids, tops = torch.cat(ids, -1), torch.cat(tops, -1)
    live = ids[:, 0] >= 0
    # from the maximum: beside the type's lowest value a logarithm of the sum has no digits left
    m = torch.where(live, z.amax(-1), 0.0)[:, None]
    total = torch.exp((tops if norm else z) - m).sum(-1, keepdim=True)
    w = torch.where(ids >= 0, torch.exp(tops - m) / torch.where(live[:, None], total, 1.0), 0.0)
    flat = ids.flatten()
    order = torch.full_like(flat, -1)
    slot = torch.full_like(flat, -1)
    at, offsets = 0, [0]
    for e in range(E):
        rows = (flat == e).nonzero()[:, 0]
        order[at:at + len(rows)] = rows
        slot[rows] = torch.arange(at, at + len(rows), device=z.device)
        at += len(rows)
        offsets.append(at)
    return ids, w, torch.tensor(offsets + [int(live.sum())], device=z.device), order, slot


def loss_of(z, ids, offsets, k, balance, zc):
    """The losses as a differentiable function of z."""
    E = z.shape[1]
    live = ids[:, 0] >= 0
    nv = max(1, int(live.sum()))
    zl = z[live]
    if not len(zl):
        return (z * 0).nan_to_num().sum()
    p = torch.softmax(zl, -1)
    counts = offsets[1:E + 1] - offsets[:E]
    return balance * E / (nv * k) * (counts * p.sum(0) / nv).sum() + zc * torch.logsumexp(zl, -1).square().sum() / nv


ROUTES = [
    # n, E, k, logits, weights, norm, balance, z, how
    (1, 1, 1, F32, F32, 1, 0.0, 0.0, ""),
    (1, 8, 2, F32, BF16, 0, 0.1, 0.01, ""),
    (7, 5, 5, BF16, F32, 1, 0.1, 0.0, "masked"),
    (33, 16, 3, F32, F32, 0, 0.0, 0.0, "ties"),
    (256, 60, 6, BF16, BF16, 1, 0.01, 0.001, "ties"),
    (257, 64, 8, F32, F32, 0, 0.01, 0.001, "masked"),
    (300, 100, 20, F32, F32, 1, 0.01, 0.001, "masked"),
    (32, 64, 6, F32, F32, 0, 0.01, 0.001, "masked"),
    (24, 300, 8, F32, F32, 0, 0.01, 0.001, "ties"),
    (33, 64, 6, BF16, BF16, 0, 0.01, 0.0, "ties"),
    (1000, 9, 9, F32, F32, 1, 0.0, 0.5, "lowest"),
    (5000, 160, 6, F32, F32, 0, 0.02, 0.0, "masked"),
    (777, 256, 32, BF16, F32, 1, 0.01, 0.001, "masked"),
    (300, 16, 16, F32, BF16, 1, 0.01, 0.001, "masked"),
    (130, 500, 8, F32, F32, 0, 0.01, 0.001, "far"),
    (65, 1024, 32, F32, F32, 1, 0.01, 0.001, "masked"),
    (20000, 64, 4, F32, F32, 0, 0.01, 0.001, "one"),
]


def logits_for(n, E, dtype, how):
    g = gen(n + E)
    z = 2 * torch.randn(n, E, generator=g, device="cuda")
    if how == "ties":
        z = z.round()
    if how == "masked":
        z[torch.rand(n, E, generator=g, device="cuda") < 0.5] = -math.inf
        z[torch.rand(n, generator=g, device="cuda") < 0.2] = -math.inf
    if how == "lowest":  # the type's lowest value is a value: chosen last, with weight 0
        z[torch.rand(n, E, generator=g, device="cuda") < 0.5] = torch.finfo(KIND[dtype]).min
    if how == "far":
        z *= 1e4
    if how == "one":  # every position to the same experts
        z = torch.linspace(3, -3, E, device="cuda").repeat(n, 1)
    return z.to(KIND[dtype])


@pytest.mark.parametrize("case", ROUTES, ids=lambda c: f"n{c[0]}e{c[1]}k{c[2]}{c[8]}")
def test_route(case):
    n, E, k, lt, wt, norm, balance, zc, how = case
    cfg = MoeConfig(n=n, h=8, ffn_dim=8, n_experts=E, top_k=k, logits_dtype=lt, weights_dtype=wt, norm_topk=norm,
                    balance_coef=balance, z_coef=zc)
    z = logits_for(n, E, lt, how)
    r = bpt.alloc_moe_route(cfg)
    for t in (r.ids, r.offsets, r.order, r.slot):
        t.fill_(12345)
    loss = torch.full((1,), float("nan"), device="cuda")
    ws = bpt.alloc_bytes(bpt.bpt_moe_route_workspace_bytes(cfg)).fill_(255)
    bpt.bpt_moe_route_fwd(cfg, z, r, loss, ws)
    sync()
    z64 = z.double()
    ids, w, offsets, order, slot = routes_of(z64, k, norm)
    for got, want in ((r.ids, ids), (r.offsets, offsets), (r.order, order), (r.slot, slot)):
        assert torch.equal(got.long(), want)
    # an exponent z - max of size up to D is off by D 2^-24: relative to the value
    spread = torch.where(ids >= 0, z64.amax(-1, keepdim=True) - z64.gather(-1, ids.clamp(min=0)), 0.0)
    wb = (64 + E / 4 + spread.clamp(max=200)) * U * w + (2.0 ** -8 * w if wt == BF16 else 1e-44)
    assert bool(((r.weights.double() - w).abs() <= wb).all())
    if how != "lowest":
        zr = z64.clone().requires_grad_()
        want = loss_of(zr, ids, offsets, k, balance, zc).detach()
        rows = n / 256 + 64 + 64 + E / 4
        assert abs(float(loss) - float(want)) <= (rows + 64) * U * abs(float(want)) + 1e-30
    else:
        assert not math.isnan(float(loss))


@pytest.mark.parametrize("case", [c for c in ROUTES if c[8] != "lowest"], ids=lambda c: f"n{c[0]}e{c[1]}k{c[2]}{c[8]}")
def test_route_backward(case):
    n, E, k, lt, wt, norm, balance, zc, how = case
    cfg = MoeConfig(n=n, h=8, ffn_dim=8, n_experts=E, top_k=k, logits_dtype=lt, weights_dtype=wt, norm_topk=norm,
                    balance_coef=balance, z_coef=zc)
    z = logits_for(n, E, lt, how)
    ids, w, offsets, order, slot = routes_of(z.double(), k, norm)
    r = bpt.MoeRoute(ids.int(), w.to(KIND[wt]), offsets.int(), order.int(), slot.int())
    dw = torch.randn(n, k, generator=gen(n), device="cuda").to(KIND[wt])
    dz = torch.full_like(z, float("nan"))
    bpt.bpt_moe_route_bwd(cfg, z, r, dw, -1.5, dz)
    sync()
    live = ids[:, 0] >= 0
    zr = z.double()[live].requires_grad_()
    li, g = ids[live], dw.double()[live]
    top = zr.gather(-1, li.clamp(min=0)).masked_fill(li < 0, -math.inf)
    q = torch.softmax(top, -1) if norm else torch.exp(top - torch.logsumexp(zr, -1, keepdim=True))
    total = (q * g.masked_fill(li < 0, 0.0)).sum() - 1.5 * loss_of(zr, li, offsets, k, balance, zc)
    want = torch.zeros_like(z, dtype=torch.float64)
    want[live] = torch.autograd.grad(total, zr)[0].nan_to_num()
    # each term is at most |g| q, q sum |g| q, or the losses' p (c + sum c p + 2 z lse / nv)
    nv = max(1, int(live.sum()))
    p = torch.zeros_like(want)
    p[live] = torch.softmax(z.double()[live], -1)
    c = balance * E / (nv * nv * k) * (offsets[1:E + 1] - offsets[:E])
    lse = torch.zeros(n, 1, dtype=torch.float64, device="cuda")
    lse[live] = torch.logsumexp(z.double()[live], -1, keepdim=True)
    size = p * (c + (p * c).sum(-1, keepdim=True) + 2 * zc / nv * lse.abs()) * 1.5
    gq = dw.double().abs().masked_fill(ids < 0, 0.0) * (w if norm else p.gather(-1, ids.clamp(min=0)))
    size.scatter_add_(-1, ids.clamp(min=0), gq)
    one = torch.zeros_like(size).scatter_add_(-1, ids.clamp(min=0), w.masked_fill(ids < 0, 0.0)) if norm else p
    size += one * gq.sum(-1, keepdim=True)
    # exponents z - max off by their size times 2^-24; beyond 200 the values vanish
    bound = (64 + E / 4 + 200 * (how == "far") + 2 * 16) * 2 * U * size + (2.0 ** -8 * want.abs() if lt == BF16 else 0.0) + 1e-38
    err = (dz.double() - want).abs()
    assert bool((err <= bound).all()), float((err - bound).max())


def test_route_records_bad_logits():
    """NaN and +inf count as -inf; the error word says so, once."""
    cfg = MoeConfig(n=40, h=8, ffn_dim=8, n_experts=12, top_k=3)
    z = logits_for(40, 12, F32, "")
    bad = z.clone()
    bad[3, 4], bad[7, 0], bad[9] = float("nan"), math.inf, float("nan")
    clean = bad.clone()
    clean[3, 4] = clean[7, 0] = -math.inf
    clean[9] = -math.inf
    r = bpt.alloc_moe_route(cfg)
    ws = bpt.alloc_bytes(bpt.bpt_moe_route_workspace_bytes(cfg))
    bpt.bpt_moe_route_fwd(cfg, bad, r, None, ws)
    assert bpt.bpt_last_device_error() == (bpt.BPT_EINVAL, bpt.BPT_MOE_BAD_LOGIT_SITE)
    assert bpt.bpt_last_device_error() == (bpt.BPT_OK, 0)
    ids, w, offsets, order, slot = routes_of(clean.double(), 3, 1)
    for got, want in ((r.ids, ids), (r.offsets, offsets), (r.order, order), (r.slot, slot)):
        assert torch.equal(got.long(), want)
    assert torch.allclose(r.weights.double(), w, rtol=64 * U, atol=0)


# ------------------------------------------------------------------ the experts' network

FFN = [
    # n, h, f, E, k, act, masked
    (1, 64, 64, 8, 2, 2, False),
    (1, 264, 136, 4, 4, 0, False),
    (5, 40, 72, 64, 3, 2, False),
    (1, 264, 136, 16, 4, 0, False),     # rows one by one (inference)
    (3, 1000, 520, 96, 6, 1, True),
    (4, 72, 2056, 32, 2, 2, True),
    (7, 40, 104, 28, 1, 2, False),
    (2, 2056, 1032, 128, 8, 2, False),
    (2, 136, 104, 14, 3, 2, True),      # few, but not so few
    (70, 256, 200, 12, 2, 1, True),
    (90, 392, 136, 16, 3, 2, True),     # 32-row tiles, several an expert
    (90, 136, 392, 16, 3, 0, False),
    (300, 136, 264, 4, 2, 2, True),     # one-SM tiles
    (333, 512, 328, 3, 3, 0, False),
    (1300, 72, 520, 2, 1, 2, False),    # 256-row tiles
    (2500, 264, 136, 4, 2, 2, True),
    (1200, 200, 72, 2, 2, 1, True),
]


def ffn_inputs(n, h, f, E, k, act, masked, wt, seed=0):
    g = gen(seed + n + h)
    z = torch.randn(n, E, generator=g, device="cuda") + torch.linspace(1, -1, E, device="cuda")
    if masked:
        z[torch.rand(n, E, generator=g, device="cuda") < 0.3] = -math.inf
        z[torch.rand(n, generator=g, device="cuda") < 0.2] = -math.inf
    ids, w, offsets, order, slot = routes_of(z.double(), k, 1)
    r = bpt.MoeRoute(ids.int(), w.to(KIND[wt]), offsets.int(), order.int(), slot.int())
    rnd = lambda *s, sc=1.0: (sc * torch.randn(*s, generator=g, device="cuda")).bfloat16()  # noqa: E731
    return r, rnd(n, h), rnd(E, f, h, sc=1.5 * h ** -0.5), rnd(E, f, h, sc=h ** -0.5) if act == 2 else None, \
        rnd(E, h, f, sc=f ** -0.5), rnd(n, h)


def network(r, act, x, w, w1, w3, w2):
    """y of fp64 tensors, pair by pair of each expert."""
    y = torch.zeros_like(x)
    for e in range(len(w1)):
        t, j = (r.ids == e).nonzero(as_tuple=True)
        g = x[t] @ w1[e].T
        a = torch.nn.functional.silu(g) * (x[t] @ w3[e].T) if act == 2 else \
            torch.nn.functional.gelu(g, approximate="tanh" if act == 1 else "none")
        y = y.index_add(0, t, (a @ w2[e].T) * w[t, j, None])
    return y


def near(got, want, roundings, what):
    assert got.shape == want.shape and got.isfinite().all(), what
    norm = float(want.norm())
    err = float((got.double() - want).norm())
    print(f"  {what}: {err / max(norm, 1e-30):.2e} (bound {roundings * 2.0 ** -8:.2e})")
    assert err <= roundings * 2.0 ** -8 * norm, what


@pytest.mark.parametrize("case", FFN, ids=lambda c: f"n{c[0]}h{c[1]}f{c[2]}e{c[3]}k{c[4]}a{c[5]}")
@pytest.mark.parametrize("wt,gt", [(F32, F32), (BF16, BF16)])
def test_experts(case, wt, gt):
    n, h, f, E, k, act, masked = case
    cfg = MoeConfig(n=n, h=h, ffn_dim=f, n_experts=E, top_k=k, act=act, weights_dtype=wt, grads_dtype=gt)
    r, x, w1, w3, w2, dy = ffn_inputs(n, h, f, E, k, act, masked, wt)
    y = torch.full_like(x, float("nan"))
    ws = bpt.alloc_bytes(bpt.bpt_moe_ffn_workspace_bytes(cfg, bpt.BPT_PASS_FWD)).fill_(255)
    saved = bpt.alloc_bytes(bpt.bpt_moe_saved_bytes(cfg)).fill_(255)
    bpt.bpt_moe_ffn_fwd(cfg, r, x, w1, w3, w2, y, saved, ws)
    plain = torch.full_like(x, float("nan"))
    ws.fill_(255)
    bpt.bpt_moe_ffn_fwd(cfg, r, x, w1, w3, w2, plain, None, ws)
    dx, dwt = torch.full_like(x, float("nan")), torch.full((n, k), float("nan"), device="cuda", dtype=KIND[wt])
    dm = [None if m is None else torch.full(m.shape, float("nan"), device="cuda", dtype=KIND[gt]) for m in (w1, w3, w2)]
    ws = bpt.alloc_bytes(bpt.bpt_moe_ffn_workspace_bytes(cfg, bpt.BPT_PASS_BWD)).fill_(255)
    bpt.bpt_moe_ffn_bwd(cfg, r, x, w1, w3, w2, saved, dy, dx, dwt, *dm, ws)
    sync()
    if 4 * n * k > E:  # fewer rows: inference takes them one by one
        assert torch.equal(y, plain)
    leaves = [t.double().requires_grad_() for t in (x, r.weights, w1, w3, w2) if t is not None]
    if w3 is None:
        leaves.insert(3, None)
    want = network(r, act, *leaves)
    grads = iter(torch.autograd.grad(want, [t for t in leaves if t is not None], dy.double()))
    near(y, want.detach(), 3, "y")
    near(plain, want.detach(), 3, "y without saved")
    near(dx, next(grads), 5, "dx")
    near(dwt, next(grads), 3, "dweights")
    for name, got in zip(("dw1", "dw3", "dw2"), dm):
        if got is not None:
            near(got, next(grads), 4, name)
    gone = r.ids[:, 0] < 0
    assert bool((y[gone] == 0).all()) and bool((plain[gone] == 0).all()) and bool((dx[gone] == 0).all()) and bool((dwt[r.ids < 0] == 0).all())
    empty = (r.offsets[1:E + 1] == r.offsets[:E]).nonzero()[:, 0]
    assert all(bool((m[empty] == 0).all()) for m in dm if m is not None)


@pytest.mark.parametrize("n,E", [(40, 6), (900, 2)])
def test_accumulated_gradients_and_repeats(n, E):
    h, f, k = 136, 72, 2
    cfg = MoeConfig(n=n, h=h, ffn_dim=f, n_experts=E, top_k=k)
    r, x, w1, w3, w2, dy = ffn_inputs(n, h, f, E, k, 2, True, F32)
    saved = bpt.alloc_bytes(bpt.bpt_moe_saved_bytes(cfg))
    ws = bpt.alloc_bytes(max(bpt.bpt_moe_ffn_workspace_bytes(cfg, p) for p in (0, 1)))
    y = torch.empty_like(x)
    runs = []
    for flags, fill in ((0, 3.0), (0, 5.0), (bpt.BPT_FLAG_ACCUM_GRADS, 1.0)):
        c = cfg.with_(flags=flags)
        dx, dwt = torch.empty_like(x), torch.empty(n, k, device="cuda")
        dm = [torch.full(m.shape, fill, device="cuda") for m in (w1, w3, w2)]
        bpt.bpt_moe_ffn_fwd(c, r, x, w1, w3, w2, y, saved, ws)
        bpt.bpt_moe_ffn_bwd(c, r, x, w1, w3, w2, saved, dy, dx, dwt, *dm, ws)
        sync()
        runs.append([y.clone(), dx, dwt, *dm])
    assert all(torch.equal(a, b) for a, b in zip(runs[0], runs[1]))
    for a, b in zip(runs[0][3:], runs[2][3:]):
        assert torch.allclose(b, a + 1.0, rtol=0, atol=float(a.abs().max() + 1) * 2.0 ** -23)


def test_gradients_against_differences():
    """The loss sum(y dy) of the fp64 network at x + t v against the kernel's
    <dx, v>, and the same for every matrix."""
    n, h, f, E, k = 64, 40, 48, 5, 2
    cfg = MoeConfig(n=n, h=h, ffn_dim=f, n_experts=E, top_k=k)
    r, x, w1, w3, w2, dy = ffn_inputs(n, h, f, E, k, 2, False, F32)
    saved = bpt.alloc_bytes(bpt.bpt_moe_saved_bytes(cfg))
    ws = bpt.alloc_bytes(max(bpt.bpt_moe_ffn_workspace_bytes(cfg, p) for p in (0, 1)))
    y, dx, dwt = torch.empty_like(x), torch.empty_like(x), torch.empty(n, k, device="cuda")
    dm = [torch.empty(m.shape, device="cuda") for m in (w1, w3, w2)]
    bpt.bpt_moe_ffn_fwd(cfg, r, x, w1, w3, w2, y, saved, ws)
    bpt.bpt_moe_ffn_bwd(cfg, r, x, w1, w3, w2, saved, dy, dx, dwt, *dm, ws)
    sync()
    at = [t.double() for t in (x, r.weights, w1, w3, w2)]
    for i, got in enumerate((dx, dwt, *dm)):
        v = got.double() / got.double().norm()  # along the gradient: the slope is its norm
        t = 1e-4 * float(at[i].norm())
        plus, minus = ([a + s * t * v if j == i else a for j, a in enumerate(at)] for s in (1, -1))
        slope = float(((network(r, 2, *plus) - network(r, 2, *minus)) * dy.double()).sum()) / (2 * t)
        want = float((got.double() * v).sum())
        assert abs(slope - want) <= 5 * 2.0 ** -8 * abs(want), i


def test_bad_order_and_slots_are_taken_as_none():
    """Entries outside their range: those pairs add nothing, nothing faults."""
    n, h, f, E, k = 50, 64, 72, 4, 2
    cfg = MoeConfig(n=n, h=h, ffn_dim=f, n_experts=E, top_k=k)
    r, x, w1, w3, w2, dy = ffn_inputs(n, h, f, E, k, 2, False, F32)
    lost = torch.tensor([3, 40, 77], device="cuda")  # pairs, and the row each one has
    at = r.slot[lost].long()
    slot, order, weights = r.slot.clone(), r.order.clone(), r.weights.clone().view(-1)
    slot[lost] = torch.tensor([-7, n * k, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    order[at] = torch.tensor([n * k, -2, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    weights[lost] = 0.0
    bad = bpt.MoeRoute(r.ids, r.weights, r.offsets, order, slot)
    zero = bpt.MoeRoute(r.ids, weights.view(n, k), r.offsets, r.order, r.slot)
    ws = bpt.alloc_bytes(max(bpt.bpt_moe_ffn_workspace_bytes(cfg, p) for p in (0, 1)))
    got = []
    for route in (bad, zero):
        saved = bpt.alloc_bytes(bpt.bpt_moe_saved_bytes(cfg))
        y, dx, dwt = torch.empty_like(x), torch.empty_like(x), torch.empty(n, k, device="cuda")
        dm = [torch.empty(m.shape, device="cuda") for m in (w1, w3, w2)]
        bpt.bpt_moe_ffn_fwd(cfg, route, x, w1, w3, w2, y, saved, ws)
        bpt.bpt_moe_ffn_bwd(cfg, route, x, w1, w3, w2, saved, dy, dx, dwt, *dm, ws)
        sync()
        got.append([y, dx, *dm])
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_refusals():
    n, h, f, E, k = 20, 64, 72, 4, 2
    cfg = MoeConfig(n=n, h=h, ffn_dim=f, n_experts=E, top_k=k)
    r, x, w1, w3, w2, dy = ffn_inputs(n, h, f, E, k, 2, False, F32)
    ws = bpt.alloc_bytes(bpt.bpt_moe_ffn_workspace_bytes(cfg, 0))
    y = torch.empty_like(x)
    a = dict(cfg=cfg, r=r, x=x, w1=w1, w3=w3, w2=w2, y=y, saved=None, ws=ws)
    for kw in (dict(x=x.float()), dict(x=x[:10]), dict(w1=w1[:3]), dict(w3=None), dict(w1=w1.transpose(1, 2)), dict(y=x),
               dict(ws=ws[:256]), dict(saved=ws[:64]), dict(cfg=cfg.with_(act=1)), dict(cfg=cfg.with_(weights_dtype=1)),
               dict(cfg=cfg.with_(top_k=5)), dict(cfg=cfg.with_(h=60)), dict(cfg=cfg.with_(grads_dtype=1, flags=1)),
               dict(r=bpt.MoeRoute(r.ids, r.weights, r.offsets[:E], r.order, r.slot)),
               dict(r=bpt.MoeRoute(r.ids, r.weights, r.offsets, r.order.long(), r.slot)),
               dict(r=bpt.MoeRoute(r.ids, r.weights, r.offsets, r.order, None))):
        v = a | kw
        with pytest.raises(bpt.BptError):
            bpt.bpt_moe_ffn_fwd(v["cfg"], v["r"], v["x"], v["w1"], v["w3"], v["w2"], v["y"], v["saved"], v["ws"])
    z = torch.randn(n, E, device="cuda")
    rw = bpt.alloc_bytes(bpt.bpt_moe_route_workspace_bytes(cfg))
    for c, logits, loss in ((cfg, z.bfloat16(), None), (cfg, z[:5], None), (cfg.with_(z_coef=0.1), z, None), (cfg, None, None),
                            (cfg.with_(balance_coef=float("nan")), z, torch.empty(1, device="cuda")),
                            (cfg.with_(n_experts=1025), z, None), (cfg.with_(norm_topk=2), z, None)):
        with pytest.raises(bpt.BptError):
            bpt.bpt_moe_route_fwd(c, logits, r, loss, rw)
    for d in (float("nan"), math.inf):
        with pytest.raises(bpt.BptError):
            bpt.bpt_moe_route_bwd(cfg, z, r, torch.empty(n, k, device="cuda"), d, torch.empty_like(z))
