"""Every entry of the experts' network's results, and of the distillation
loss's gradients, against fp64: a lost row, a wrong tail word or the last block
of a group would not show in the 2-norm of a whole tensor.

Bounds, entry by entry, by running the error through the formulas in absolute
values.  R = 2^-8 is a rounding to bf16, relative to the value; a sum of K
products in fp32 is off by at most (K + 1) 2^-23 of the sum of the absolute
values (the tensor core may cut); exponentials, reciprocals and the erf
polynomial, in fp32, by F = 2^-18 of what they are multiplied by.
  g, u: their sums' errors; the backward takes them rounded to bf16 besides.
  |silu'| <= 1.1 and |silu''| <= 0.5, |gelu'| <= 1.13 and |gelu''| <= 0.8 (at 0).
  y: act (rounded), the choice's row (rounded), the sum (rounded)
  dg, du, w act: from the kept g and u, rounded; dx their products' sum,
  rounded as a choice's row and as dx; the matrices' gradients and dweights
  sums of them, rounded where they are bf16.
Products of two errors are covered by 1.02."""
import pytest
import torch

import blockwise_attention_ffn_gb300 as bpt
from blockwise_attention_ffn_gb300.presets import MoeConfig
from tests.test_gpu_distill import CASES as DISTILL
from tests.test_gpu_distill import inputs as distill_inputs
from tests.test_gpu_distill import run as distill
from tests.test_gpu_distill import teacher_of
from tests.test_gpu_moe import BF16, F32, FFN, KIND, ffn_inputs, sync

pytestmark = pytest.mark.gpu

R, S, F = 2.0 ** -8, 2.0 ** -23, 2.0 ** -18


def inside(got, want, bound, what):
    err = (got.double() - want).abs()
    over = err > 1.02 * bound + 1e-30
    print(f"  {what}: at most {float((err / (bound + 1e-30)).max()):.2f} of the bound")
    assert got.isfinite().all() and not over.any(), (what, over.nonzero()[:4].tolist())


def activation(act, g, u):
    """act, dact/dg, dact/du, and the bounds of their slopes by g."""
    if act == 2:
        s = torch.sigmoid(g)
        si = g * s
        return si * u, u * (s + si * (1 - s)), si, 1.1 * u.abs(), 0.5 * u.abs()
    gd = g.clone().requires_grad_()
    a = torch.nn.functional.gelu(gd, approximate="tanh" if act == 1 else "none")
    slope = torch.autograd.grad(a.sum(), gd)[0]
    one = torch.ones_like(g)
    return a.detach(), slope, None, 1.13 * one, 0.8 * one


@pytest.mark.parametrize("case", FFN, ids=lambda c: f"n{c[0]}h{c[1]}f{c[2]}e{c[3]}k{c[4]}a{c[5]}")
@pytest.mark.parametrize("wt,gt", [(F32, F32), (BF16, BF16)])
def test_experts_entry_by_entry(case, wt, gt):
    n, h, f, E, k, act, masked = case
    cfg = MoeConfig(n=n, h=h, ffn_dim=f, n_experts=E, top_k=k, act=act, weights_dtype=wt, grads_dtype=gt)
    r, x, w1, w3, w2, dy = ffn_inputs(n, h, f, E, k, act, masked, wt)
    ws = bpt.alloc_bytes(max(bpt.bpt_moe_ffn_workspace_bytes(cfg, p) for p in (0, 1))).fill_(255)
    saved = bpt.alloc_bytes(bpt.bpt_moe_saved_bytes(cfg)).fill_(255)
    y, plain, dx = (torch.full_like(x, float("nan")) for _ in range(3))
    dwt = torch.full((n, k), float("nan"), device="cuda", dtype=KIND[wt])
    dm = [None if m is None else torch.full(m.shape, float("nan"), device="cuda", dtype=KIND[gt]) for m in (w1, w3, w2)]
    bpt.bpt_moe_ffn_fwd(cfg, r, x, w1, w3, w2, plain, None, ws)
    bpt.bpt_moe_ffn_fwd(cfg, r, x, w1, w3, w2, y, saved, ws)
    bpt.bpt_moe_ffn_bwd(cfg, r, x, w1, w3, w2, saved, dy, dx, dwt, *dm, ws)
    sync()
    z = lambda t: torch.zeros(t.shape, dtype=torch.float64, device="cuda")  # noqa: E731
    wy, by, wdx, bdx, wdw, bdw = z(x), z(x), z(x), z(x), z(dwt), z(dwt)
    for e in range(E):
        t, j = (r.ids == e).nonzero(as_tuple=True)
        xe, de, w = x[t].double(), dy[t].double(), r.weights[t, j, None].double()
        a1, a2 = w1[e].double(), w2[e].double()
        a3 = None if w3 is None else w3[e].double()
        g, eg = xe @ a1.T, (h + 1) * S * (xe.abs() @ a1.abs().T)
        u, eu = (xe @ a3.T, (h + 1) * S * (xe.abs() @ a3.abs().T)) if act == 2 else (torch.ones_like(g), 0 * eg)
        a, slope, by_u, l1, l2 = activation(act, g, u)
        by_u = torch.zeros_like(g) if by_u is None else by_u
        ea = l1 * eg + by_u.abs() * eu + F * g.abs() * u.abs() + R * a.abs()
        row = a @ a2.T
        erow = ea @ a2.abs().T + (f + 1) * S * (a.abs() @ a2.abs().T) + R * row.abs()
        wy.index_add_(0, t, w * row)
        by.index_add_(0, t, w * erow + k * S * w * row.abs())
        # backward, from what was kept
        kg, ku = eg + R * g.abs(), eu + (R * u.abs() if act == 2 else 0)
        da, eda = de @ a2, (h + 1) * S * (de.abs() @ a2.abs())
        dg, du, aw = w * da * slope, w * da * by_u, w * a
        off_u = ku * (slope / u).abs() if act == 2 else 0  # the slope by g is u times one of g
        edg = w * (eda * slope.abs() + da.abs() * (off_u + l2 * kg + F * (1 + g.abs()) * u.abs())) + R * dg.abs()
        edu = w * (eda * by_u.abs() + da.abs() * (1.1 * kg + F * g.abs())) + R * du.abs() if act == 2 else 0 * edg
        ea = l1 * kg + by_u.abs() * ku + F * g.abs() * u.abs()
        eaw = w * ea + R * aw.abs()
        wdw[t, j] = (a * da).sum(-1)
        bdw[t, j] = (ea * da.abs() + a.abs() * eda + (f + 1) * S * (a * da).abs()).sum(-1)
        dr, size, er = dg @ a1, dg.abs() @ a1.abs(), edg @ a1.abs()
        if act == 2:
            dr, size, er = dr + du @ a3, size + du.abs() @ a3.abs(), er + edu @ a3.abs()
        wdx.index_add_(0, t, dr)
        bdx.index_add_(0, t, er + (2 * f + 1) * S * size + R * dr.abs() + k * S * dr.abs())
        for got, left, off, right, what in ((dm[0], dg, edg, xe, "dw1"), (dm[1], du, edu, xe, "dw3"), (dm[2], de, None, aw, "dw2")):
            if got is None:
                continue
            want = left.T @ right
            bound = (len(t) + 1) * S * (left.abs().T @ right.abs()) + (de.abs().T @ eaw if off is None else off.T @ right.abs())
            inside(got[e], want, bound + (R * want.abs() if gt == BF16 else 0), f"{what} of expert {e}")
    inside(y, wy, by + R * wy.abs(), "y")
    inside(plain, wy, by + R * wy.abs(), "y without saved")
    inside(dx, wdx, bdx + R * wdx.abs(), "dx")
    inside(dwt, wdw, bdw + (R * wdw.abs() if wt == BF16 else 0), "dweights")


@pytest.mark.parametrize("cfg", DISTILL, ids=lambda c: c.name)
@pytest.mark.parametrize("masked", [False, True])
def test_distill_entry_by_entry(cfg, masked):
    """dz = T c (P q - p): q's exponent is off by the logit's and the
    log-sum-exp's errors, p by its own exponential's; then one rounding."""
    x, w, ids, v, weight = distill_inputs(cfg, masked)
    _, dx, dw = distill(cfg, x, w, ids, v, weight)
    T, p = cfg.temperature, teacher_of(cfg, ids, v)
    x64, w64 = x.double(), w.double()
    zt = x64 @ w64.T / T
    off = (cfg.h + 1) * S * (x64.abs() @ w64.abs().T) / T + S * zt.abs()
    lse = torch.logsumexp(zt, -1, keepdim=True)
    q = torch.exp(zt - lse)
    eq = q * (off + off.amax(-1, keepdim=True) + F * (1 + lse.abs()))
    c = (torch.full((cfg.n, 1), 1.0 / cfg.n, device="cuda", dtype=torch.float64) if weight is None else weight.double()[:, None]) * T
    mass = p.sum(-1, keepdim=True)
    at = torch.zeros_like(q).scatter_add_(-1, ids.long().clamp(min=0), p)
    dz = c * (mass * q - at)
    ez = c * (mass * eq + F * (mass * q + at) * (1 + v.clamp(min=-100).abs().amax(-1, keepdim=True) / T)) + R * dz.abs()
    inside(dx, dz @ w64, ez @ w64.abs() + (cfg.vocab + 1) * S * (dz.abs() @ w64.abs()) + R * (dz @ w64).abs(), "dx")
    inside(dw, dz.T @ x64, ez.T @ x64.abs() + (cfg.n + 1) * S * (dz.abs().T @ x64.abs()) + (R * (dz.T @ x64).abs() if cfg.grads_dtype else 0),
           "dw")
