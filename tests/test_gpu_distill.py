"""The distillation loss from a teacher's stored top logits on the GPU against
fp64.

Tolerances.  A logit is a sum of h exact products in fp32: off by at most
h 2^-23 S, S = sum |x w| (the tensor core may cut), and so is the log-sum-exp,
which besides carries the exponentials' and the sum's own roundings, under
2^-18 of it and of one.  A row's divergence is sum p (log p - z + lse): off by
2 P (h 2^-23 S / T + 2^-18 (1 + |lse|)); its gradient by the logits the same
times q or p, which is far below the rounding to bf16.  That rounding, 2^-8 of
each value, enters sums in which nothing is amplified beyond the sum itself:
in the 2-norm dw in fp32 is off by one of them, a bf16 result by two."""
import math

import pytest
import torch

import blockwise_attention_ffn_gb300 as bpt
from blockwise_attention_ffn_gb300.presets import DistillConfig

pytestmark = pytest.mark.gpu

LOGITS, LOGPROBS = bpt.BPT_TEACHER_LOGITS, bpt.BPT_TEACHER_LOGPROBS

CASES = [
    DistillConfig(n=1, h=8, vocab=1, top_k=1, name="one of one"),
    DistillConfig(n=1, h=64, vocab=300, top_k=5, temperature=2.0, name="one row"),
    DistillConfig(n=100, h=72, vocab=1000, top_k=33, temperature=1.5, name="ragged"),
    DistillConfig(n=300, h=256, vocab=1000, top_k=7, vocab_block=512, temperature=3.0, name="two blocks"),
    DistillConfig(n=257, h=136, vocab=257, top_k=128, name="dense entries"),
    DistillConfig(n=1000, h=512, vocab=8191, top_k=64, teacher=LOGPROBS, vocab_block=2048, name="four blocks"),
    DistillConfig(n=129, h=128, vocab=300, top_k=16, teacher=LOGPROBS, temperature=4.0, grads_dtype=1, name="bf16 grads"),
    DistillConfig(n=300, h=2560, vocab=5000, top_k=16, vocab_block=1024, name="K in slabs"),
    DistillConfig(n=640, h=384, vocab=3000, top_k=20, vocab_block=768, flags=bpt.BPT_FLAG_DETERMINISTIC, name="fixed order"),
]


def inputs(cfg, masked=False, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + cfg.n + cfg.vocab)
    x = torch.randn(cfg.n, cfg.h, generator=g, device="cuda").bfloat16()
    w = (2 * torch.randn(cfg.vocab, cfg.h, generator=g, device="cuda") * cfg.h ** -0.5).bfloat16()
    # k distinct ids where there are as many, in no order
    ids = torch.rand(cfg.n, cfg.vocab, generator=g, device="cuda").argsort(-1)[:, :cfg.top_k]
    if cfg.top_k > cfg.vocab:
        ids = torch.randint(0, cfg.vocab, (cfg.n, cfg.top_k), generator=g, device="cuda")
    v = 2 * torch.randn(cfg.n, cfg.top_k, generator=g, device="cuda")
    if cfg.teacher == LOGPROBS:
        v = torch.log_softmax(v, -1) + math.log(0.8)
    weight = None
    if masked:
        ids = ids.masked_fill(torch.rand(cfg.n, cfg.top_k, generator=g, device="cuda") < 0.3, -1)
        ids[torch.rand(cfg.n, generator=g, device="cuda") < 0.2] = -5
        v = v.masked_fill(torch.rand(cfg.n, cfg.top_k, generator=g, device="cuda") < 0.1, -math.inf)
        weight = torch.rand(cfg.n, generator=g, device="cuda") / cfg.n
        weight[torch.rand(cfg.n, generator=g, device="cuda") < 0.2] = 0.0
    return x, w, ids.int().contiguous(), v, weight


def run(cfg, x, w, ids, v, weight, dloss=1.0, dw=None):
    loss = torch.full((1,), float("nan"), device="cuda")
    saved = bpt.alloc_bytes(bpt.bpt_lm_distill_saved_bytes(cfg)).fill_(255)
    ws = bpt.alloc_bytes(max(bpt.bpt_lm_distill_workspace_bytes(cfg, p) for p in (0, 1))).fill_(255)
    bpt.bpt_lm_distill_fwd(cfg, x, w, ids, v, weight, loss, saved, ws)
    dx = torch.full_like(x, float("nan"))
    if dw is None:
        dw = torch.full((cfg.vocab, cfg.h), float("nan"), device="cuda", dtype=torch.bfloat16 if cfg.grads_dtype else torch.float32)
    ws.fill_(255)
    bpt.bpt_lm_distill_bwd(cfg, x, w, weight, saved, dloss, dx, dw, ws)
    torch.cuda.synchronize()
    assert bpt.bpt_last_device_error() == (bpt.BPT_OK, 0)
    return loss, dx, dw


def teacher_of(cfg, ids, v):
    t = v.double()
    gone = ids < 0
    if cfg.teacher == LOGPROBS:
        return torch.where(gone, 0.0, t.exp())
    t = (t / cfg.temperature).masked_fill(gone, -math.inf)
    none = (t == -math.inf).all(-1, keepdim=True)
    return torch.where(gone | none, 0.0, torch.softmax(torch.where(none, 0.0, t), -1))


def loss_of(cfg, x, w, ids, v, weight):
    """The loss of fp64 x and w, and the bound of its error."""
    p, T = teacher_of(cfg, ids, v), cfg.temperature
    z = x @ w.T / T
    lse = torch.logsumexp(z, -1, keepdim=True)
    rows = (torch.special.xlogy(p, p) - p * (z - lse).gather(-1, ids.long().clamp(min=0))).sum(-1)
    c = torch.full_like(rows, 1.0 / cfg.n) if weight is None else weight.double()
    size = (x.detach().abs() @ w.detach().abs().T).amax(-1)
    off = 2 * p.sum(-1) * (cfg.h * 2.0 ** -23 * size / T + 2.0 ** -18 * (1 + lse.detach()[:, 0].abs()))
    return T * T * (c * rows).sum(), float(T * T * (c * off).sum())


def near(got, want, roundings, what):
    assert got.isfinite().all(), what
    norm, err = float(want.norm()), float((got.double() - want).norm())
    print(f"  {what}: {err / max(norm, 1e-30):.2e} (bound {roundings * 2.0 ** -8:.2e})")
    assert err <= roundings * 2.0 ** -8 * norm + 1e-9, what


@pytest.mark.parametrize("cfg", CASES, ids=lambda c: c.name)
@pytest.mark.parametrize("masked", [False, True])
def test_distill(cfg, masked):
    x, w, ids, v, weight = inputs(cfg, masked)
    loss, dx, dw = run(cfg, x, w, ids, v, weight, dloss=-2.0)
    x64, w64 = x.double().requires_grad_(), w.double().requires_grad_()
    want, off = loss_of(cfg, x64, w64, ids, v, weight)
    print(f"{cfg.name}: loss {float(loss):.8f}, {float(want.detach()):.8f} +- {off:.1e}")
    assert abs(float(loss) - float(want.detach())) <= off + 2.0 ** -23 * abs(float(want.detach()))
    gx, gw = torch.autograd.grad(-2.0 * want, (x64, w64))
    if cfg.vocab > 1:
        near(dx, gx, 2, "dx")
        near(dw, gw, 2 if cfg.grads_dtype else 1.01, "dw")
    else:  # one word: q = 1 and the gradient is a rounding of zero
        assert float(dx.abs().max()) <= 1e-5 and float(dw.abs().max()) <= 1e-5
    if masked:
        assert bool((dx[weight == 0] == 0).all()) and bool((dx[(ids < 0).all(-1)] == 0).all())


def test_the_same_id_twice():
    """An id given twice (and often) counts with both its values."""
    cfg = DistillConfig(n=50, h=64, vocab=400, top_k=12)
    x, w, ids, v, _ = inputs(cfg)
    ids[:, 1] = ids[:, 0]
    ids[10:20, 2:] = ids[10:20, :1]
    loss, dx, dw = run(cfg, x, w, ids, v, None)
    x64, w64 = x.double().requires_grad_(), w.double().requires_grad_()
    want, off = loss_of(cfg, x64, w64, ids, v, None)
    assert abs(float(loss) - float(want.detach())) <= off + 2.0 ** -23 * abs(float(want.detach()))
    gx, gw = torch.autograd.grad(want, (x64, w64))
    near(dx, gx, 2, "dx")
    near(dw, gw, 1.01, "dw")


def test_one_entry_is_the_cross_entropy():
    """A teacher sure of one token at T = 1: the library's own loss."""
    from blockwise_attention_ffn_gb300.presets import LmConfig
    cfg = DistillConfig(n=333, h=128, vocab=2000, top_k=1)
    x, w, ids, v, _ = inputs(cfg)
    loss, dx, dw = run(cfg, x, w, ids, v, None)
    lm = LmConfig(n=cfg.n, h=cfg.h, vocab=cfg.vocab)
    ws = bpt.alloc_bytes(max(bpt.bpt_lm_workspace_bytes(lm, p) for p in (0, 1)))
    want, lse = torch.empty(1, device="cuda"), torch.empty(cfg.n, device="cuda")
    t = ids.view(-1)
    bpt.bpt_lm_loss_fwd(lm, x, w, t, want, lse, ws)
    gx, gw = torch.empty_like(x), torch.empty(cfg.vocab, cfg.h, device="cuda")
    bpt.bpt_lm_loss_bwd(lm, x, w, t, lse, 1.0, gx, gw, ws)
    torch.cuda.synchronize()
    assert abs(float(loss) - float(want)) <= 2.0 ** -16 * abs(float(want))
    near(dx, gx.double(), 4, "dx")
    near(dw, gw.double(), 2, "dw")


def test_a_row_of_weight_zero_leaves_no_trace():
    cfg = DistillConfig(n=200, h=128, vocab=900, top_k=9, flags=bpt.BPT_FLAG_DETERMINISTIC)
    x, w, ids, v, weight = inputs(cfg, True)
    once = run(cfg, x, w, ids, v, weight)
    gone = weight == 0
    x[gone] = 3e30
    v[gone] = 50.0
    again = run(cfg, x, w, ids, v, weight)
    for a, b in zip(once, again):
        assert torch.equal(a, b)


def test_extreme_rows():
    """A row without entries gives nothing whatever its logits are (infinite
    here); a teacher value beyond fp32 over T is as good as certain."""
    cfg = DistillConfig(n=70, h=64, vocab=500, top_k=6, temperature=2.0 ** -8, flags=bpt.BPT_FLAG_DETERMINISTIC)
    x, w, ids, v, _ = inputs(cfg)
    ids[::2] = -1
    v[1] = torch.tensor([1.0, -3e38, 3e38, 5.0, -math.inf, 0.0], device="cuda")
    once = run(cfg, x, w, ids, v, None)
    assert all(t.isfinite().all() for t in once)
    x64, w64 = x.double(), w.double()
    sure = ids[1].clone()
    sure[[0, 1, 3, 4, 5]] = -1
    same = ids.clone()
    same[1] = sure
    want, off = loss_of(cfg, x64, w64, same, v.clamp(max=1e30), None)
    assert abs(float(once[0]) - float(want)) <= off + 2.0 ** -23 * abs(float(want))
    big = x.clone()
    big[::2] = 3e38
    loss, dx, dw = run(cfg, big, w, ids, v, None)
    assert torch.equal(loss, once[0]) and torch.equal(dx, once[1])


def test_accumulated_and_repeated():
    cfg = CASES[8]
    x, w, ids, v, weight = inputs(cfg, True)
    one, two = run(cfg, x, w, ids, v, weight), run(cfg, x, w, ids, v, weight)
    assert all(torch.equal(a, b) for a, b in zip(one, two))
    acc = torch.full((cfg.vocab, cfg.h), 2.0, device="cuda")
    run(cfg.with_(flags=cfg.flags | bpt.BPT_FLAG_ACCUM_GRADS), x, w, ids, v, weight, dw=acc)
    assert torch.allclose(acc, one[2] + 2.0, rtol=0, atol=2.0 ** -22)


def test_gradient_against_differences():
    cfg = DistillConfig(n=40, h=64, vocab=300, top_k=8, temperature=2.0)
    x, w, ids, v, _ = inputs(cfg)
    _, dx, dw = run(cfg, x, w, ids, v, None)
    for i, got in enumerate((dx.double(), dw.double())):
        at = [x.double(), w.double()]
        d = got / got.norm()
        t = 1e-4 * float(at[i].norm())
        side = []
        for s in (1, -1):
            moved = list(at)
            moved[i] = at[i] + s * t * d
            side.append(float(loss_of(cfg, *moved, ids, v, None)[0]))
        assert abs((side[0] - side[1]) / (2 * t) - float(got.norm())) <= 2 * 2.0 ** -8 * float(got.norm())


def test_bad_entries_are_recorded_and_left_out():
    cfg = DistillConfig(n=60, h=64, vocab=500, top_k=6)
    x, w, ids, v, _ = inputs(cfg)
    bad, clean, vb = ids.clone(), ids.clone(), v.clone()
    bad[3, 2], bad[9, 0], vb[11, 4], vb[12, 1] = 500, 2 ** 31 - 1, float("nan"), math.inf
    clean[3, 2] = clean[9, 0] = clean[11, 4] = clean[12, 1] = -1
    loss = torch.empty(1, device="cuda")
    saved = bpt.alloc_bytes(bpt.bpt_lm_distill_saved_bytes(cfg))
    ws = bpt.alloc_bytes(bpt.bpt_lm_distill_workspace_bytes(cfg, 0))
    bpt.bpt_lm_distill_fwd(cfg, x, w, bad, vb, None, loss, saved, ws)
    assert bpt.bpt_last_device_error() == (bpt.BPT_EINVAL, bpt.BPT_DISTILL_BAD_ENTRY_SITE)
    want = torch.empty(1, device="cuda")
    bpt.bpt_lm_distill_fwd(cfg, x, w, clean, v, None, want, saved, ws)
    assert bpt.bpt_last_device_error() == (bpt.BPT_OK, 0)
    assert torch.equal(loss, want)


def test_refusals():
    cfg = DistillConfig(n=30, h=64, vocab=300, top_k=4)
    x, w, ids, v, _ = inputs(cfg)
    loss = torch.empty(1, device="cuda")
    saved = bpt.alloc_bytes(bpt.bpt_lm_distill_saved_bytes(cfg))
    ws = bpt.alloc_bytes(bpt.bpt_lm_distill_workspace_bytes(cfg, 0))
    ok = dict(cfg=cfg, x=x, w=w, ids=ids, v=v, rw=None, loss=loss, saved=saved, ws=ws)
    for kw in (dict(x=x.float()), dict(w=w[:299]), dict(ids=ids.long()), dict(v=v.bfloat16()), dict(rw=loss), dict(loss=None),
               dict(saved=saved[:64]), dict(ws=ws[:64]), dict(cfg=cfg.with_(top_k=129)), dict(cfg=cfg.with_(temperature=0.0)),
               dict(cfg=cfg.with_(temperature=float("nan"))), dict(cfg=cfg.with_(teacher=2)), dict(cfg=cfg.with_(vocab_block=100)),
               dict(cfg=cfg.with_(grads_dtype=1, flags=1)), dict(cfg=cfg.with_(flags=2)), dict(ws=saved)):
        a = ok | kw
        with pytest.raises(bpt.BptError):
            bpt.bpt_lm_distill_fwd(a["cfg"], a["x"], a["w"], a["ids"], a["v"], a["rw"], a["loss"], a["saved"], a["ws"])
    dx, dw = torch.empty_like(x), torch.empty(300, 64, device="cuda")
    for d, gx, gw in ((float("inf"), dx, dw), (1.0, x, dw), (1.0, dx, dw.bfloat16()), (1.0, dx, None)):
        with pytest.raises(bpt.BptError):
            bpt.bpt_lm_distill_bwd(cfg, x, w, None, saved, d, gx, gw, ws)
