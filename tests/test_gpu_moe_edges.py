"""Edges of the router and the experts' network on the GPU: zeros of both
signs, products beyond fp32, malformed offsets, a route of which only what a
call reads is given.  References and tolerances as in test_gpu_moe.py."""
import pytest
import torch

import blockwise_attention_ffn_gb300 as bpt
from blockwise_attention_ffn_gb300.presets import MoeConfig
from tests.test_gpu_moe import BF16, F32, KIND, U, ffn_inputs, gen, near, network, routes_of, sync

pytestmark = pytest.mark.gpu


def spaces(cfg):
    """A workspace for both passes and what the forward saves, full of NaN."""
    ws = bpt.alloc_bytes(max(bpt.bpt_moe_ffn_workspace_bytes(cfg, p) for p in (0, 1))).fill_(255)
    return ws, bpt.alloc_bytes(bpt.bpt_moe_saved_bytes(cfg)).fill_(255)


# a router in one launch and in two for each number of lanes a row is held by
@pytest.mark.parametrize("n,E,k", [(16, 9, 8), (200, 16, 11), (20, 32, 20), (300, 24, 15), (31, 64, 32), (500, 60, 32), (15, 128, 32),
                                   (300, 100, 32), (9, 256, 32), (200, 200, 32), (9, 400, 32), (100, 512, 32), (7, 1000, 32),
                                   (100, 1024, 32)])
@pytest.mark.parametrize("lt", [F32, BF16])
def test_zeros_of_both_signs_are_equal(n, E, k, lt):
    """-0.0 and +0.0 are equal logits: the lowest index goes first.  Every
    logit is one of the zeros or below them."""
    cfg = MoeConfig(n=n, h=8, ffn_dim=8, n_experts=E, top_k=k, logits_dtype=lt)
    kind = torch.randint(0, 3, (n, E), generator=gen(E + n), device="cuda")
    z = torch.tensor([0.0, -0.0, -1.0], device="cuda")[kind].to(KIND[lt])
    assert bool((z.float().signbit() & (z == 0)).any())
    r = bpt.alloc_moe_route(cfg)
    ws = bpt.alloc_bytes(bpt.bpt_moe_route_workspace_bytes(cfg)).fill_(255)
    bpt.bpt_moe_route_fwd(cfg, z, r, None, ws)
    sync()
    ids, w, offsets, order, slot = routes_of(z.double(), k, 1)
    for got, want in ((r.ids, ids), (r.offsets, offsets), (r.order, order), (r.slot, slot)):
        assert torch.equal(got.long(), want)
    assert torch.allclose(r.weights.double(), w, rtol=(64 + E / 4) * U, atol=0)


# few rows (rows one by one in inference), 32-row tiles, one SM a tile, a pair
SIZES = [(5, 64), (40, 8), (300, 4), (1000, 2)]


def outlying(n, h, f, E, k, act):
    """Inputs of which every third position alone has a first column, 2^60."""
    r, x, w1, w3, w2, dy = ffn_inputs(n, h, f, E, k, act, False, F32)
    big = torch.arange(n, device="cuda") % 3 == 1
    x[:, 0] = 0
    x[big, 0] = 2.0 ** 60
    return r, x, w1, w3, w2, dy, big


def both_passes(cfg, r, x, w1, w3, w2, dy):
    ws, saved = spaces(cfg)
    y, plain, dx = (torch.full_like(x, float("nan")) for _ in range(3))
    dwt = torch.full_like(r.weights, float("nan"))
    dm = [None if m is None else torch.full(m.shape, float("nan"), device="cuda") for m in (w1, w3, w2)]
    bpt.bpt_moe_ffn_fwd(cfg, r, x, w1, w3, w2, plain, None, ws)
    ws.fill_(255)
    bpt.bpt_moe_ffn_fwd(cfg, r, x, w1, w3, w2, y, saved, ws)
    ws.fill_(255)
    bpt.bpt_moe_ffn_bwd(cfg, r, x, w1, w3, w2, saved, dy, dx, dwt, *dm, ws)
    sync()
    return y, plain, dx, dwt, dm


@pytest.mark.parametrize("n,E", SIZES)
def test_a_closed_gate_closes_any_up_product(n, E):
    """silu(g) u is 0 for g far below zero, also where g u is beyond fp32
    (2^130 here), and so are the gradients, also where dy u is beyond it."""
    h, f, k = 72, 136, 2
    cfg = MoeConfig(n=n, h=h, ffn_dim=f, n_experts=E, top_k=k)
    r, x, w1, w3, w2, dy, big = outlying(n, h, f, E, k, 2)
    w1[:, :, 0], w3[:, :, 0] = -2.0 ** 10, 1.0  # g = -2^70, u = 2^60
    dy[big] *= 2.0 ** 70
    y, plain, dx, dwt, dm = both_passes(cfg, r, x, w1, w3, w2, dy)
    for t in (y, plain, dx, dwt):
        assert bool((t[big] == 0).all())
    leaves = [t.double().requires_grad_() for t in (x, r.weights, w1, w3, w2)]
    want = network(r, 2, *leaves)
    grads = torch.autograd.grad(want, leaves, dy.double())
    near(y, want.detach(), 3, "y")
    near(plain, want.detach(), 3, "y without saved")
    for name, got, g, c in zip(("dx", "dweights", "dw1", "dw3", "dw2"), (dx, dwt, *dm), grads, (5, 3, 4, 4, 4)):
        near(got, g, c, name)


@pytest.mark.parametrize("n,E", SIZES)
@pytest.mark.parametrize("act", [0, 1])
def test_far_out_gelu(n, E, act):
    """Far out the GeLU is z or 0 and its slope 1 or 0, also where z^2 is
    beyond fp32 (z = 2^70 and -2^70 here).  The other positions' results are
    looked at by themselves: beside 2^70 they would not count."""
    h, f, k = 72, 136, 2
    cfg = MoeConfig(n=n, h=h, ffn_dim=f, n_experts=E, top_k=k, act=act)
    r, x, w1, _, w2, dy, big = outlying(n, h, f, E, k, act)
    w1[:, :, 0] = 2.0 ** 10
    w1[:, 1::2, 0] = -2.0 ** 10
    y, plain, dx, dwt, (dw1, _, dw2) = both_passes(cfg, r, x, w1, None, w2, dy)
    leaves = [t.double().requires_grad_() for t in (x, r.weights, w1, w2)]
    want = network(r, act, *leaves[:3], None, leaves[3])
    gx, gwt, gw1, gw2 = torch.autograd.grad(want, leaves, dy.double())
    for rows in (big, ~big):
        near(y[rows], want.detach()[rows], 3, "y")
        near(plain[rows], want.detach()[rows], 3, "y without saved")
        near(dx[rows], gx[rows], 5, "dx")
        near(dwt[rows], gwt[rows], 3, "dweights")
    near(dw1[:, :, 0], gw1[:, :, 0], 4, "dw1's first column")
    near(dw1[:, :, 1:], gw1[:, :, 1:], 4, "dw1's others")
    near(dw2, gw2, 4, "dw2")


def rows_of(offsets, pairs):
    """The rows of each group as the products take them: none for a group whose
    offsets fall, leave [0, pairs] or start before an earlier one's end."""
    rows, end = [], 0
    for lo, hi in zip(offsets, offsets[1:]):
        inside = 0 <= lo <= hi <= pairs
        rows.append(range(lo, hi) if inside and lo >= end else range(0))
        end = max(end, hi if inside else 0)
    return rows


def malformed(how, offsets, pairs):
    """Offsets of which some rows are in no group, and whether that is an error."""
    E = len(offsets) - 2
    o, used = list(offsets), [e for e in range(E) if offsets[e + 1] > offsets[e]]
    if how == "cut":        # the last rows are in no group
        last = used[-1]
        o[last + 1:E + 1] = [o[last]] * (E - last)
        return o, False
    if how == "late":       # nor are the first
        first = used[0]
        o[:first + 1] = [o[first + 1]] * (first + 1)
        return o, False
    mid = len(used) // 2
    e, after = used[mid], used[mid + 1]
    if how == "far":        # a group ends behind the last row
        o[e + 1] = pairs + 1000
    if how == "negative":   # the first one begins before the first row
        o[used[0]] = -5
    if how == "falling":    # a later one begins before the end of an earlier one
        o[e] = offsets[e + 1]
        o[e + 1:after + 1] = [offsets[e]] * (after - e)
    return o, True


@pytest.mark.parametrize("n,E", [(3, 64), (9, 96), (40, 8), (300, 4), (1600, 4)])
@pytest.mark.parametrize("how", ["cut", "late", "far", "negative", "falling"])
@pytest.mark.parametrize("act", [2, 0])
def test_pairs_in_no_group_add_nothing(n, E, how, act):
    """Rows that no expert's offsets hold: their pairs add nothing to y, dx and
    dweights, whatever the workspace holds and by which path the rows go."""
    h, f, k = 72, 136, 2
    cfg = MoeConfig(n=n, h=h, ffn_dim=f, n_experts=E, top_k=k, act=act)
    r, x, w1, w3, w2, dy = ffn_inputs(n, h, f, E, k, act, False, F32)
    offsets, error = malformed(how, r.offsets.tolist(), n * k)
    bad = bpt.MoeRoute(r.ids, r.weights, torch.tensor(offsets, dtype=torch.int32, device="cuda"), r.order, r.slot)
    # the same network with the pairs of the rows that are left
    ids = torch.full((n * k,), -1, device="cuda")
    for e, rows in enumerate(rows_of(offsets[:E + 1], n * k)):
        ids[r.order[list(rows)].long()] = e
    ids = ids.view(n, k)
    assert bool((ids < 0).any()) and bool((ids >= 0).any())
    left = bpt.MoeRoute(ids, r.weights, None, None, None)
    ws, saved = spaces(cfg)
    y, plain, dx, dwt = *(torch.full_like(x, float("nan")) for _ in range(3)), torch.full_like(r.weights, float("nan"))
    dm = [None if m is None else torch.full(m.shape, float("nan"), device="cuda") for m in (w1, w3, w2)]
    for call in (lambda: bpt.bpt_moe_ffn_fwd(cfg, bad, x, w1, w3, w2, plain, None, ws),
                 lambda: bpt.bpt_moe_ffn_fwd(cfg, bad, x, w1, w3, w2, y, saved, ws),
                 lambda: bpt.bpt_moe_ffn_bwd(cfg, bad, x, w1, w3, w2, saved, dy, dx, dwt, *dm, ws)):
        ws.fill_(255)
        call()
        torch.cuda.synchronize()
        assert bpt.bpt_last_device_error() == ((bpt.BPT_EINVAL, bpt.BPT_GROUPED_BAD_OFFSET_SITE) if error else (bpt.BPT_OK, 0))
    leaves = [t.double().requires_grad_() for t in (x, r.weights, w1, w3, w2) if t is not None]
    if w3 is None:
        leaves.insert(3, None)
    want = network(left, act, leaves[0], *leaves[1:])
    grads = iter(torch.autograd.grad(want, [t for t in leaves if t is not None], dy.double()))
    near(y, want.detach(), 3, "y")
    near(plain, want.detach(), 3, "y without saved")
    near(dx, next(grads), 5, "dx")
    near(dwt, next(grads), 3, "dweights")
    for name, got in zip(("dw1", "dw3", "dw2"), dm):
        if got is not None:
            near(got, next(grads), 4, name)
    assert bool((dwt[ids < 0] == 0).all())
    gone = (ids < 0).all(-1)
    assert bool((y[gone] == 0).all()) and bool((plain[gone] == 0).all()) and bool((dx[gone] == 0).all())


def test_route_backward_takes_what_it_reads():
    """ids and offsets: the other tensors of a route may be gone by then."""
    cfg = MoeConfig(n=70, h=8, ffn_dim=8, n_experts=12, top_k=3, balance_coef=0.1, z_coef=0.01)
    g = gen(5)
    z, dw = torch.randn(70, 12, generator=g, device="cuda"), torch.randn(70, 3, generator=g, device="cuda")
    r, loss = bpt.alloc_moe_route(cfg), torch.empty(1, device="cuda")
    bpt.bpt_moe_route_fwd(cfg, z, r, loss, bpt.alloc_bytes(bpt.bpt_moe_route_workspace_bytes(cfg)))
    want, got = torch.empty_like(z), torch.empty_like(z)
    bpt.bpt_moe_route_bwd(cfg, z, r, dw, 1.0, want)
    bpt.bpt_moe_route_bwd(cfg, z, bpt.MoeRoute(r.ids, None, r.offsets, None, None), dw, 1.0, got)
    sync()
    assert torch.equal(got, want)
    for bad in (bpt.MoeRoute(None, r.weights, r.offsets, r.order, r.slot), bpt.MoeRoute(r.ids, r.weights, None, r.order, r.slot),
                bpt.MoeRoute(r.ids.long(), None, r.offsets, None, None), bpt.MoeRoute(r.ids, None, r.offsets[:13], None, None)):
        with pytest.raises(bpt.BptError):
            bpt.bpt_moe_route_bwd(cfg, z, bad, dw, 1.0, got)
