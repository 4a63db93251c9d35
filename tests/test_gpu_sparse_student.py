"""The router, the experts' network and the distillation loss together, as a
training step of a layer with experts uses them: the router's logits by a
grouped product, the routes, the experts' network with its residual, the loss
against a teacher's entries, and the way back through all of it to every weight,
then the clipping; against PyTorch autograd in fp64 on the same bf16 inputs and
the same choices.

Tolerances: every tensor that passes from one call to the next in bf16 (logits,
weights, activations, rows, y, the logits' gradient) is off by at most 2^-8 of
its values, and enters sums in which nothing is amplified beyond the sum: in the
2-norm the count of roundings on the way to a tensor times 2^-8.  The longest way
(to x through the router: y and its three, the loss's two, the experts' five, the
weights' and logits' gradients) has twelve."""
import math

import pytest
import torch

import blockwise_attention_ffn_gb300 as bpt
from blockwise_attention_ffn_gb300.presets import DistillConfig, GroupedConfig, MoeConfig

pytestmark = pytest.mark.gpu

BOUND = 12 * 2.0 ** -8
NT, NN, TN = bpt.BPT_GROUPED_NT, bpt.BPT_GROUPED_NN, bpt.BPT_GROUPED_TN


def rel(a, b):
    return float((a.double() - b).norm() / b.norm())


class Step:
    """One training step's buffers and calls."""

    def __init__(self, n, h, f, E, k, V, K, seed=0, norm=0):
        g = torch.Generator(device="cuda").manual_seed(seed + n)
        rnd = lambda *s, sc=1.0: (sc * torch.randn(*s, generator=g, device="cuda")).bfloat16()  # noqa: E731
        self.moe = MoeConfig(n=n, h=h, ffn_dim=f, n_experts=E, top_k=k, logits_dtype=1, weights_dtype=1, norm_topk=norm,
                             balance_coef=0.01, z_coef=0.001)
        self.kd = DistillConfig(n=n, h=h, vocab=V, top_k=K, temperature=2.0, flags=bpt.BPT_FLAG_DETERMINISTIC)
        self.gate = GroupedConfig(rows=n, n=E, k=h, groups=1, form=NT, out_dtype=1)
        self.x, self.wr, self.w = rnd(n, h), rnd(E, h, sc=h ** -0.5), rnd(V, h, sc=2 * h ** -0.5)
        self.w1, self.w3, self.w2 = rnd(E, f, h, sc=h ** -0.5), rnd(E, f, h, sc=h ** -0.5), rnd(E, h, f, sc=f ** -0.5)
        self.ids = torch.rand(n, V, generator=g, device="cuda").argsort(-1)[:, :K].int().contiguous()
        self.v = 2 * torch.randn(n, K, generator=g, device="cuda")
        self.one = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        self.route = bpt.alloc_moe_route(self.moe)
        self.logits, self.dlogits = (torch.empty(n, E, device="cuda", dtype=torch.bfloat16) for _ in range(2))
        self.y, self.dx, self.dxr, self.dz = (torch.empty_like(self.x) for _ in range(4))
        self.dweights = torch.empty_like(self.route.weights)
        self.aux, self.loss = torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
        self.dw = [torch.empty(t.shape, device="cuda") for t in (self.w1, self.w3, self.w2, self.wr, self.w)]
        size = max(bpt.bpt_moe_route_workspace_bytes(self.moe), bpt.bpt_clip_workspace_bytes(),
                   *(bpt.bpt_moe_ffn_workspace_bytes(self.moe, p) for p in (0, 1)),
                   *(bpt.bpt_lm_distill_workspace_bytes(self.kd, p) for p in (0, 1)))
        self.ws = bpt.alloc_bytes(size)
        self.saved = bpt.alloc_bytes(bpt.bpt_moe_saved_bytes(self.moe))
        self.kept = bpt.alloc_bytes(bpt.bpt_lm_distill_saved_bytes(self.kd))
        self.norm = torch.empty(1, device="cuda")

    def run(self, stream=None):
        s, m = dict(stream=stream), self.moe
        bpt.bpt_grouped_gemm(self.gate, self.x, self.wr, self.one, self.logits, **s)
        bpt.bpt_moe_route_fwd(m, self.logits, self.route, self.aux, self.ws, **s)
        bpt.bpt_moe_ffn_fwd(m, self.route, self.x, self.w1, self.w3, self.w2, self.y, self.saved, self.ws, **s)
        bpt.bpt_lm_distill_fwd(self.kd, self.y, self.w, self.ids, self.v, None, self.loss, self.kept, self.ws, **s)
        d1, d3, d2, dr, dv = self.dw
        bpt.bpt_lm_distill_bwd(self.kd, self.y, self.w, None, self.kept, 1.0, self.dz, dv, self.ws, **s)
        bpt.bpt_moe_ffn_bwd(m, self.route, self.x, self.w1, self.w3, self.w2, self.saved, self.dz, self.dx, self.dweights, d1, d3, d2,
                            self.ws, **s)
        bpt.bpt_moe_route_bwd(m, self.logits, self.route, self.dweights, 1.0, self.dlogits, **s)
        c = self.gate.with_(n=m.h, k=m.n_experts)
        bpt.bpt_grouped_gemm(c.with_(form=NN), self.dlogits, self.wr, self.one, self.dxr, **s)
        bpt.bpt_grouped_gemm(c.with_(form=TN, out_dtype=0), self.dlogits, self.x, self.one, dr, **s)
        bpt.bpt_clip_grads(self.dw, 1e30, self.norm, self.ws, **s)  # measures, scales nothing

    def results(self):
        return [t.clone() for t in (self.logits, self.route.ids, self.route.weights, self.route.offsets, self.route.order,
                                    self.route.slot, self.y, self.aux, self.loss, self.dz, self.dx, self.dxr, self.dlogits,
                                    self.dweights, self.norm, *self.dw)]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("n,h,f,E,k,norm", [(300, 128, 200, 8, 2, 0), (1500, 64, 136, 16, 3, 1), (40, 264, 72, 64, 4, 0)])
def test_step(n, h, f, E, k, norm):
    t = Step(n, h, f, E, k, 1000, 9, norm=norm)
    t.run()
    torch.cuda.synchronize()
    assert bpt.bpt_last_device_error() == (bpt.BPT_OK, 0)
    ids = t.route.ids.long()
    x, wr, w, w1, w3, w2 = (v.double().requires_grad_() for v in (t.x, t.wr, t.w, t.w1, t.w3, t.w2))
    z = x @ wr.T
    # where the fp64 logits' order differs from the rounded ones' the choice is the calls'
    p = torch.softmax(z, -1)
    top = z.gather(-1, ids)
    q = torch.softmax(top, -1) if norm else p.gather(-1, ids)
    y = torch.zeros_like(x)
    for e in range(E):
        r, j = (ids == e).nonzero(as_tuple=True)
        a = torch.nn.functional.silu(x[r] @ w1[e].T) * (x[r] @ w3[e].T)
        y = y.index_add(0, r, (a @ w2[e].T) * q[r, j, None])
    counts = torch.bincount(ids.flatten(), minlength=E)
    aux = 0.01 * E / (n * k) * (counts * p.mean(0)).sum() + 0.001 * torch.logsumexp(z, -1).square().mean()
    pt = torch.softmax(t.v.double() / 2, -1)
    lq = torch.log_softmax(y @ w.T / 2, -1).gather(-1, t.ids.long())
    loss = 4 * (pt * (pt.log() - lq)).sum(-1).mean()
    (loss + aux).backward()
    assert abs(float(t.aux) - float(aux.detach())) <= 2.0 ** -8 * 4 * float(aux.detach())
    assert abs(float(t.loss) - float(loss.detach())) <= 2.0 ** -8 * 4 * float(loss.detach())
    assert rel(t.y, y.detach()) < BOUND
    assert rel(t.dx.double() + t.dxr.double(), x.grad) < BOUND
    for name, got, want in zip(("w1", "w3", "w2", "wr", "w"), t.dw, (w1, w3, w2, wr, w)):
        assert rel(got, want.grad) < BOUND, name
    total = math.sqrt(sum(float(g.double().square().sum()) for g in t.dw))
    assert abs(float(t.norm) - total) < 2.0 ** -20 * total


def test_repeats_captures_and_streams():
    """The same bits again, replayed from a graph with new inputs in place, and
    from two streams at once with buffers of their own."""
    t, u = Step(500, 128, 264, 8, 2, 900, 7), Step(700, 64, 136, 16, 2, 1200, 5, seed=3)
    t.run(), u.run()
    torch.cuda.synchronize()
    want, other = t.results(), u.results()
    t.run()
    torch.cuda.synchronize()
    assert same(t.results(), want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        t.run()
    for b in (t.y, t.dx, t.loss, *t.dw):
        b.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    assert same(t.results(), want)
    fresh = Step(500, 128, 264, 8, 2, 900, 7, seed=11)
    fresh.run()
    torch.cuda.synchronize()
    for name in ("x", "wr", "w", "w1", "w3", "w2", "ids", "v"):
        getattr(t, name).copy_(getattr(fresh, name))
    graph.replay()
    torch.cuda.synchronize()
    assert same(t.results(), fresh.results())
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(4):
        with torch.cuda.stream(a):
            fresh.run()
        u.run(stream=b)
    torch.cuda.synchronize()
    assert same(u.results(), other) and same(t.results(), fresh.results())
    assert bpt.bpt_last_device_error() == (bpt.BPT_OK, 0)


def test_debug_checks():
    """BPT_FLAG_DEBUG_CHECKS: the same results, every pointer looked at first."""
    t = Step(200, 64, 136, 8, 2, 500, 5)
    t.run()
    torch.cuda.synchronize()
    want = t.results()
    f = bpt.BPT_FLAG_DEBUG_CHECKS
    t.moe, t.kd, t.gate = t.moe.with_(flags=f), t.kd.with_(flags=t.kd.flags | f), t.gate.with_(flags=f)
    t.run()
    assert same(t.results(), want)
    short = t.saved[:1024]  # a device tensor, but the call keeps more than its allocation may hold
    with pytest.raises(bpt.BptError):
        bpt.bpt_moe_ffn_fwd(t.moe, t.route, t.x, t.w1, t.w3, t.w2, t.y, short, t.ws)


@pytest.mark.parametrize("n,E", [(90, 16), (1300, 2), (3, 64)])
def test_padded_positions_leave_no_trace(n, E):
    """Positions without a route may hold anything, NaN too, in x and in dy."""
    cfg = MoeConfig(n=n, h=136, ffn_dim=200, n_experts=E, top_k=2)
    g = torch.Generator(device="cuda").manual_seed(n)
    rnd = lambda *s, sc=1.0: (sc * torch.randn(*s, generator=g, device="cuda")).bfloat16()  # noqa: E731
    z = torch.randn(n, E, generator=g, device="cuda")
    gone = torch.arange(n, device="cuda") % 3 == 1
    z[gone] = -math.inf
    x, dy, w1, w3, w2 = rnd(n, 136), rnd(n, 136), rnd(E, 200, 136, sc=0.1), rnd(E, 200, 136, sc=0.1), rnd(E, 136, 200, sc=0.1)
    r = bpt.alloc_moe_route(cfg)
    ws = bpt.alloc_bytes(max(bpt.bpt_moe_route_workspace_bytes(cfg), *(bpt.bpt_moe_ffn_workspace_bytes(cfg, p) for p in (0, 1))))
    bpt.bpt_moe_route_fwd(cfg, z, r, None, ws)
    saved = bpt.alloc_bytes(bpt.bpt_moe_saved_bytes(cfg))
    runs = []
    for fill in (0.0, float("nan")):
        x[gone] = dy[gone] = fill
        ws.fill_(255), saved.fill_(255)
        y, plain, dx, dwt = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x), torch.empty(n, 2, device="cuda")
        dm = [torch.empty(m.shape, device="cuda") for m in (w1, w3, w2)]
        bpt.bpt_moe_ffn_fwd(cfg, r, x, w1, w3, w2, plain, None, ws)
        bpt.bpt_moe_ffn_fwd(cfg, r, x, w1, w3, w2, y, saved, ws)
        bpt.bpt_moe_ffn_bwd(cfg, r, x, w1, w3, w2, saved, dy, dx, dwt, *dm, ws)
        torch.cuda.synchronize()
        runs.append([y, plain, dx, dwt, *dm])
    assert all(torch.equal(a, b) and a.isfinite().all() for a, b in zip(*runs))
    assert bool((runs[0][0][gone] == 0).all()) and bool((runs[0][2][gone] == 0).all())


def test_offsets_beyond_31_bits():
    """200000 rows of a network 16384 wide: 3.3e9 values in every tensor between
    the products."""
    n, h, f, E = 200000, 64, 16384, 2
    cfg = MoeConfig(n=n, h=h, ffn_dim=f, n_experts=E, top_k=1)
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s, sc=1.0: (sc * torch.randn(*s, generator=g, device="cuda")).bfloat16()  # noqa: E731
    x, w1, w3, w2, dy = rnd(n, h), rnd(E, f, h, sc=0.125), rnd(E, f, h, sc=0.125), rnd(E, h, f, sc=f ** -0.5), rnd(n, h)
    r = bpt.alloc_moe_route(cfg)
    loss = torch.empty(1, device="cuda")
    ws = bpt.alloc_bytes(max(bpt.bpt_moe_route_workspace_bytes(cfg), *(bpt.bpt_moe_ffn_workspace_bytes(cfg, p) for p in (0, 1))))
    bpt.bpt_moe_route_fwd(cfg, torch.randn(n, E, generator=g, device="cuda"), r, loss, ws)
    saved = bpt.alloc_bytes(bpt.bpt_moe_saved_bytes(cfg))
    y, dx, dwt = torch.empty_like(x), torch.empty_like(x), torch.empty(n, 1, device="cuda")
    dm = [torch.empty(m.shape, device="cuda") for m in (w1, w3, w2)]
    bpt.bpt_moe_ffn_fwd(cfg, r, x, w1, w3, w2, y, saved, ws)
    bpt.bpt_moe_ffn_bwd(cfg, r, x, w1, w3, w2, saved, dy, dx, dwt, *dm, ws)
    torch.cuda.synchronize()
    assert bpt.bpt_last_device_error() == (bpt.BPT_OK, 0)
    rows = torch.cat((torch.arange(40), torch.arange(n - 40, n), torch.arange(n // 2, n // 2 + 40))).cuda()
    for e in range(E):
        s = rows[r.ids[rows, 0] == e]
        xs = x[s].double().requires_grad_()
        want = (torch.nn.functional.silu(xs @ w1[e].double().T) * (xs @ w3[e].double().T)) @ w2[e].double().T
        assert rel(y[s], want.detach()) <= 3 * 2.0 ** -8
        want.backward(dy[s].double())
        assert rel(dx[s], xs.grad) <= 5 * 2.0 ** -8
        assert rel(dwt[s, 0], (want.detach() * dy[s].double()).sum(-1)) <= 3 * 2.0 ** -8
    # a few rows of the last expert's gradients over all its rows
    s = (r.ids[:, 0] == E - 1).nonzero()[:, 0]
    cols = torch.tensor([0, 1, f // 2, f - 1], device="cuda")
    xs, g1, u1 = x[s].double(), x[s].double() @ w1[-1][cols].double().T, x[s].double() @ w3[-1][cols].double().T
    da, sg = dy[s].double() @ w2[-1][:, cols].double(), torch.sigmoid(g1)
    assert rel(dm[1][-1][cols], (da * g1 * sg).T @ xs) <= 4 * 2.0 ** -8
    assert rel(dm[0][-1][cols], (da * u1 * sg * (1 + g1 * (1 - sg))).T @ xs) <= 4 * 2.0 ** -8
    assert rel(dm[2][-1][:, cols], dy[s].double().T @ (g1 * sg * u1)) <= 4 * 2.0 ** -8


def test_products_and_loss_beyond_31_bits():
    rows, n, k = 140000, 16384, 64
    g = torch.Generator(device="cuda").manual_seed(2)
    a, b = torch.randn(rows, k, generator=g, device="cuda").bfloat16(), torch.randn(3, n, k, generator=g, device="cuda").bfloat16()
    offsets = torch.tensor([0, 50000, 139000, rows], dtype=torch.int32, device="cuda")
    out = torch.empty(rows, n, device="cuda")
    bpt.bpt_grouped_gemm(GroupedConfig(rows=rows, n=n, k=k, groups=3, form=NT, out_dtype=0), a, b, offsets, out)
    for r, e in ((slice(49990, 50000), 0), (slice(138990, 139000), 1), (slice(rows - 10, rows), 2)):
        torch.testing.assert_close(out[r].double(), a[r].double() @ b[e].double().T, rtol=1e-5, atol=1e-4)
    del out
    cfg = DistillConfig(n=270000, h=64, vocab=9000, top_k=3)
    x = torch.randn(cfg.n, 64, generator=g, device="cuda").bfloat16()
    w = (0.25 * torch.randn(cfg.vocab, 64, generator=g, device="cuda")).bfloat16()
    ids = torch.randint(0, 3000, (cfg.n, 1), generator=g, device="cuda") + torch.tensor([0, 3000, 6000], device="cuda")
    v = torch.randn(cfg.n, 3, generator=g, device="cuda")
    loss, dx, dw = torch.empty(1, device="cuda"), torch.empty_like(x), torch.empty(cfg.vocab, 64, device="cuda")
    saved = bpt.alloc_bytes(bpt.bpt_lm_distill_saved_bytes(cfg))
    ws = bpt.alloc_bytes(max(bpt.bpt_lm_distill_workspace_bytes(cfg, p) for p in (0, 1)))
    bpt.bpt_lm_distill_fwd(cfg, x, w, ids.int(), v, None, loss, saved, ws)
    bpt.bpt_lm_distill_bwd(cfg, x, w, None, saved, 1.0, dx, dw, ws)
    torch.cuda.synchronize()
    assert bpt.bpt_last_device_error() == (bpt.BPT_OK, 0)
    total, want = 0.0, torch.zeros(cfg.vocab, 64, dtype=torch.float64, device="cuda")
    for r0 in range(0, cfg.n, 30000):
        r = slice(r0, r0 + 30000)
        p, lq = torch.softmax(v[r].double(), -1), torch.log_softmax(x[r].double() @ w.double().T, -1)
        total += float((p * (p.log() - lq.gather(-1, ids[r]))).sum())
        dz = lq.exp().scatter_add_(-1, ids[r], -p) / cfg.n
        want += dz.T @ x[r].double()
        got = dz[-8:] @ w.double()
        assert rel(dx[r][-8:], got) <= 2 * 2.0 ** -8
    assert abs(float(loss) - total / cfg.n) <= 2.0 ** -16 * total / cfg.n
    assert rel(dw, want) <= 1.01 * 2.0 ** -8
