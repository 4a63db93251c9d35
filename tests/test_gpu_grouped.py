"""Products over ragged groups of rows on the GPU against the same sums in
fp64.

Tolerance: products of two bf16 values are exact in fp32 and K of them are
added in fp32, each addition off by at most 2^-23 of the partial sum (the
tensor core may cut instead of rounding), which is at most S = sum |a b|: so
K 2^-23 S bounds an fp32 result, and a bf16 result is off by half a step,
2^-8 of its value, besides.  BPT_FLAG_ACCUM_GRADS adds one fp32 rounding of the
sum, 2^-24 of |out| + |old|."""
import pytest
import torch

import blockwise_attention_ffn_gb300 as bpt
from blockwise_attention_ffn_gb300.presets import GroupedConfig

pytestmark = pytest.mark.gpu

NT, NN, TN = bpt.BPT_GROUPED_NT, bpt.BPT_GROUPED_NN, bpt.BPT_GROUPED_TN
F32, BF16 = bpt.BPT_DTYPE_F32, bpt.BPT_DTYPE_BF16

# rows, n, k, sizes of the groups (rows behind them are in none), rows before the first
CASES = [
    (1, 8, 8, [1], 0),
    (1, 264, 72, [0, 1, 0], 0),
    (5, 64, 64, [0, 0, 0], 0),
    (70, 96, 40, [3, 0, 64, 1], 2),
    (300, 520, 136, [129, 1, 0, 63, 65], 7),
    (1000, 256, 64, [128, 256, 1, 0, 300, 17], 0),
    (1500, 328, 1000, [700, 0, 513, 255], 3),
    (4000, 776, 264, [3000, 900], 11),   # 256-row tiles of a pair of SMs
    (2600, 1288, 72, [40] * 64, 0),
    (400, 328, 456, [5] * 36 + [70, 0, 33, 97], 4),  # 32-row tiles of 64 columns
    (300, 24, 16, [1] * 300, 0),
    (1100, 16, 24, [1] * 1000 + [0] * 20 + [3, 0, 90, 0], 3),
]


def inputs(rows, n, k, sizes, first, form, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + rows + n)
    a = torch.randn(rows, k, generator=g, device="cuda").bfloat16()
    shape = {NT: (len(sizes), n, k), NN: (len(sizes), k, n), TN: (rows, n)}[form]
    b = torch.randn(*shape, generator=g, device="cuda").bfloat16()
    offsets = torch.tensor([first] + sizes, device="cuda").cumsum(0).int()
    out = torch.full((len(sizes), k, n) if form == TN else (rows, n), 7.0, device="cuda")
    return a, b, offsets, out


def reference(a, b, offsets, out, form):
    """fp64 result over a copy of out, and sum |a b|."""
    want, size = out.double(), torch.zeros_like(out, dtype=torch.float64)
    at = offsets.tolist()
    for e in range(len(at) - 1):
        r = slice(at[e], at[e + 1])
        x = a[r].double()
        y = b[r].double() if form == TN else b[e].double().T if form == NT else b[e].double()
        x, where = (x.T, e) if form == TN else (x, r)
        want[where] = x @ y
        size[where] = x.abs() @ y.abs()
    return want, size


def run(cfg, a, b, offsets, out):
    bpt.bpt_grouped_gemm(cfg, a, b, offsets, out)
    torch.cuda.synchronize()
    assert bpt.bpt_last_device_error() == (bpt.BPT_OK, 0)


def close(got, want, size, terms, bf16):
    err = (got.double() - want).abs()
    bound = terms * 2.0 ** -23 * size + (2.0 ** -8 * want.abs() if bf16 else 0.0)
    assert bool((err <= bound).all()), float((err - bound).max())


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0]}x{c[1]}x{c[2]}g{len(c[3])}")
@pytest.mark.parametrize("form", [NT, NN, TN])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_grouped_products(case, form, dtype):
    rows, n, k, sizes, first = case
    a, b, offsets, out = inputs(rows, n, k, sizes, first, form)
    out = out.bfloat16() if dtype == BF16 else out
    want, size = reference(a, b, offsets, out, form)
    cfg = GroupedConfig(rows=rows, n=n, k=k, groups=len(sizes), form=form, out_dtype=dtype)
    run(cfg, a, b, offsets, out)
    close(out, want, size, (max(sizes) if form == TN else k) + 1, dtype == BF16)


@pytest.mark.parametrize("form", [NT, NN, TN])
@pytest.mark.parametrize("sizes", [[100, 31, 0, 150], [700, 0, 601], [3] * 30])
def test_other_rows_and_matrices_leave_no_trace(form, sizes):
    """NaN in the rows of no group, and in the rows and the matrix of one
    group: the others' results are the same bits as without."""
    rows, n, k, first = sum(sizes) + 40, 136, 200, 5
    a, b, offsets, out = inputs(rows, n, k, sizes, first, form)
    cfg = GroupedConfig(rows=rows, n=n, k=k, groups=len(sizes), form=form, out_dtype=F32)
    clean = out.clone()
    run(cfg, a, b, offsets, clean)
    lo, hi = int(offsets[0]), int(offsets[1])
    a[:lo] = a[lo:hi] = a[sum(sizes) + first:] = float("nan")
    if form == TN:
        b[:lo] = b[lo:hi] = b[sum(sizes) + first:] = float("nan")
    else:
        b[0] = float("nan")
    run(cfg, a, b, offsets, out)
    if form == TN:
        assert out[0].isnan().all() and torch.equal(out[1:], clean[1:])
    else:
        assert out[lo:hi].isnan().all() and torch.equal(out[hi:], clean[hi:]) and bool((out[:lo] == 7.0).all())


@pytest.mark.parametrize("form", [NT, NN, TN])
@pytest.mark.parametrize("case", [CASES[3], CASES[6]], ids=["small", "large"])
def test_accumulate_and_repeat(form, case):
    rows, n, k, sizes, first = case
    a, b, offsets, out = inputs(rows, n, k, sizes, first, form)
    cfg = GroupedConfig(rows=rows, n=n, k=k, groups=len(sizes), form=form, out_dtype=F32)
    once = out.clone()
    run(cfg, a, b, offsets, once)
    again = out.clone()
    run(cfg, a, b, offsets, again)
    assert torch.equal(once, again)
    acc = out.clone()
    run(cfg.with_(flags=bpt.BPT_FLAG_ACCUM_GRADS), a, b, offsets, acc)
    want, size = reference(a, b, offsets, torch.zeros_like(out), form)
    terms = (max(sizes) if form == TN else k) + 1
    err = (acc.double() - (want + 7.0)).abs()
    assert bool((err <= terms * 2.0 ** -23 * size + 2.0 ** -23 * (want.abs() + 7.0)).all())


@pytest.mark.parametrize("form", [NT, NN, TN])
def test_bad_offsets_are_recorded_and_empty(form):
    """Falling, negative, too large and overlapping offsets: those groups are
    empty, the others right, the error word says so."""
    rows, n, k = 200, 64, 72
    offs = torch.tensor([0, 50, 40, 90, rows + 1, -3, 100, 150], dtype=torch.int32, device="cuda")
    good = [(0, 0, 50), (6, 100, 150)]
    a, b, _, _ = inputs(rows, n, k, [1] * 7, 0, form)
    out = torch.full((7, k, n) if form == TN else (rows, n), 7.0, device="cuda")
    want = torch.zeros_like(out).double() if form == TN else out.double()
    for e, lo, hi in good:
        x = a[lo:hi].double()
        if form == TN:
            want[e] = x.T @ b[lo:hi].double()
        else:
            want[lo:hi] = x @ (b[e].double().T if form == NT else b[e].double())
    bpt.bpt_grouped_gemm(GroupedConfig(rows=rows, n=n, k=k, groups=7, form=form, out_dtype=F32), a, b, offs, out)
    assert bpt.bpt_last_device_error() == (bpt.BPT_EINVAL, bpt.BPT_GROUPED_BAD_OFFSET_SITE)
    assert torch.allclose(out.double(), want, rtol=1e-4, atol=1e-3)


def test_refusals():
    cfg = GroupedConfig(rows=64, n=64, k=64, groups=2, out_dtype=F32)
    a, b, offsets, out = inputs(64, 64, 64, [30, 34], 0, NT)
    for t in (dict(a=a[:, :32]), dict(a=a.float()), dict(b=b[:1]), dict(offsets=offsets[:2]), dict(offsets=offsets.long()),
              dict(out=out.bfloat16()), dict(out=out[:32]), dict(a=a.cpu()), dict(out=None)):
        x = dict(a=a, b=b, offsets=offsets, out=out) | t
        with pytest.raises(bpt.BptError):
            bpt.bpt_grouped_gemm(cfg, x["a"], x["b"], x["offsets"], x["out"])
