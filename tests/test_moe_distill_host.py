"""Host side of the router, the experts' network, the products over ragged
groups and the distillation loss: every refusal comes before anything is
launched, so all of it runs without a GPU (addresses that are never read stand
in for device memory)."""
import ctypes
import os
import re

import pytest

import blockwise_attention_ffn_gb300 as bpt
from blockwise_attention_ffn_gb300.presets import DistillConfig, GroupedConfig, MoeConfig

A = 1 << 40  # a 16-byte aligned address nothing lives at


@pytest.fixture(scope="module")
def lib():
    from blockwise_attention_ffn_gb300 import build
    build.build()
    return bpt.lib()


def far(i):
    """Addresses far apart."""
    return A + (i << 36)


@pytest.mark.parametrize("struct,name", [(bpt.BptMoeConfig, "bpt_moe_config"), (bpt.BptMoeRoute, "bpt_moe_route"),
                                         (bpt.BptGroupedConfig, "bpt_grouped_config"), (bpt.BptDistillConfig, "bpt_distill_config")])
def test_structs_match_the_header(struct, name):
    hdr = open(os.path.join(os.path.dirname(__file__), "..", "include", "bpt.h")).read()
    end = hdr.index("} %s;" % name)
    body = hdr[hdr.rindex("typedef struct {", 0, end) + len("typedef struct {"):end]
    body = re.sub(r"\b(int32_t|float|void)\b", "", body)
    assert re.findall(r"\b([a-z_0-9]+)\b", body) == [f for f, _ in struct._fields_]


def test_sites_match_the_header():
    hdr = open(os.path.join(os.path.dirname(__file__), "..", "include", "bpt.h")).read()
    for n in ("BPT_MOE_BAD_LOGIT_SITE", "BPT_DISTILL_BAD_ENTRY_SITE", "BPT_GROUPED_BAD_OFFSET_SITE"):
        assert int(re.search(r"#define %s (\d+)" % n, hdr).group(1)) == getattr(bpt, n)


def moe(**kw):
    return bpt.make_moe_config(MoeConfig(**{**dict(n=50, h=64, ffn_dim=72, n_experts=8, top_k=2), **kw}))


def route(i=20, **kw):
    a = dict(ids=far(i), weights=far(i + 1), offsets=far(i + 2), order=far(i + 3), slot=far(i + 4)) | kw
    return bpt.BptMoeRoute(*[a[f] for f, _ in bpt.BptMoeRoute._fields_])


BAD_MOE = [dict(n=0), dict(n=-1), dict(h=0), dict(h=60), dict(ffn_dim=4), dict(ffn_dim=100), dict(n_experts=0), dict(n_experts=1025),
           dict(top_k=0), dict(top_k=9), dict(n_experts=64, top_k=33), dict(act=3), dict(act=-1), dict(logits_dtype=2),
           dict(weights_dtype=-1), dict(grads_dtype=2), dict(norm_topk=2), dict(balance_coef=float("nan")), dict(z_coef=float("inf")),
           dict(flags=2), dict(flags=16), dict(grads_dtype=1, flags=1)]


@pytest.mark.parametrize("kw", BAD_MOE, ids=str)
def test_moe_configs_are_refused(lib, kw):
    c = moe(**kw)
    assert lib.bpt_moe_route_workspace_bytes(c) == 0 and lib.bpt_moe_saved_bytes(c) == 0
    assert lib.bpt_moe_ffn_workspace_bytes(c, 0) == 0 and lib.bpt_moe_ffn_workspace_bytes(c, 1) == 0
    assert lib.bpt_moe_route_fwd(c, far(1), route(), far(2), far(3), 1 << 40, None) == bpt.BPT_EINVAL
    assert lib.bpt_moe_route_bwd(c, far(1), route(), far(2), 1.0, far(3), None) == bpt.BPT_EINVAL
    assert lib.bpt_moe_ffn_fwd(c, route(), *map(far, range(1, 8)), 1 << 40, None) == bpt.BPT_EINVAL
    assert lib.bpt_moe_ffn_bwd(c, route(), *map(far, range(1, 13)), 1 << 40, None) == bpt.BPT_EINVAL


def test_too_many_rows(lib):
    c = moe(n=1 << 26, top_k=2)
    assert lib.bpt_moe_route_fwd(c, far(1), route(), far(2), far(3), 1 << 40, None) == bpt.BPT_EUNSUPPORTED
    assert lib.bpt_moe_ffn_fwd(c, route(), *map(far, range(1, 8)), 1 << 40, None) == bpt.BPT_EUNSUPPORTED
    g = bpt.BptGroupedConfig((1 << 29) + 1, 64, 64, 4, 0, 0, 0)
    assert lib.bpt_grouped_gemm(g, far(1), far(2), far(3), far(4), None) == bpt.BPT_EUNSUPPORTED


def test_route_pointers(lib):
    c = moe(balance_coef=0.1)
    n = lib.bpt_moe_route_workspace_bytes(c)

    def call(c=c, logits=far(1), r=None, loss=far(2), ws=far(3), n=n):
        return lib.bpt_moe_route_fwd(c, logits, route() if r is None else r, loss, ws, n, None)

    assert call(n=n - 1) == bpt.BPT_ENOSPC
    for kw in (dict(logits=None), dict(loss=None), dict(ws=None), dict(logits=far(1) + 8), dict(loss=far(2) + 2), dict(ws=far(3) + 4),
               dict(ws=far(1)), dict(loss=far(1) + 64), dict(loss=far(3) + 16), dict(r=route(ids=None)), dict(r=route(weights=None)),
               dict(r=route(offsets=None)), dict(r=route(order=None)), dict(r=route(slot=None)), dict(r=route(ids=far(20) + 2)),
               dict(r=route(weights=far(1))), dict(r=route(order=far(20) + 8)), dict(r=route(slot=far(3)))):
        assert call(**kw) == bpt.BPT_EINVAL, kw
    assert lib.bpt_moe_route_fwd(c, far(1), None, far(2), far(3), n, None) == bpt.BPT_EINVAL

    def back(logits=far(1), r=None, dw=far(2), d=1.0, dz=far(3)):
        return lib.bpt_moe_route_bwd(c, logits, route() if r is None else r, dw, d, dz, None)

    for kw in (dict(logits=None), dict(dw=None), dict(dz=None), dict(d=float("nan")), dict(d=float("inf")), dict(dz=far(1)),
               dict(dz=far(2) + 16), dict(dz=far(3) + 8), dict(r=route(ids=None)), dict(r=route(offsets=None)), dict(dz=far(20))):
        assert back(**kw) == bpt.BPT_EINVAL, kw


def test_experts_pointers(lib):
    c = moe()
    n = lib.bpt_moe_ffn_workspace_bytes(c, 0)
    names = ("x", "w1", "w3", "w2", "y", "saved", "ws")

    def call(c=c, r=None, n=n, **kw):
        a = {k: far(i + 1) for i, k in enumerate(names)} | kw
        return lib.bpt_moe_ffn_fwd(c, route() if r is None else r, *[a[k] for k in names], n, None)

    assert call(n=n - 1) == bpt.BPT_ENOSPC
    bad = [{k: None} for k in names if k != "saved"] + [{k: far(9) + 8} for k in names] + [dict(y=far(1)), dict(y=far(2)), dict(saved=far(1)),
           dict(ws=far(6)), dict(ws=far(5) + 64), dict(y=far(21)), dict(c=moe(act=1)), dict(r=route(slot=None)), dict(r=route(weights=None))]
    for kw in bad:
        assert call(**kw) == bpt.BPT_EINVAL, kw
    assert call(c=moe(act=0), w3=None, n=0) == bpt.BPT_ENOSPC  # fine but for the workspace
    names = ("x", "w1", "w3", "w2", "saved", "dy", "dx", "dweights", "dw1", "dw3", "dw2", "ws")
    m = lib.bpt_moe_ffn_workspace_bytes(c, 1)

    def back(c=c, n=m, **kw):
        a = {k: far(i + 1) for i, k in enumerate(names)} | kw
        return lib.bpt_moe_ffn_bwd(c, route(), *[a[k] for k in names], n, None)

    assert back(n=m - 1) == bpt.BPT_ENOSPC
    for kw in [{k: None} for k in names] + [dict(dx=far(6)), dict(dx=far(1)), dict(dw1=far(2)), dict(dw3=far(9)), dict(dw2=far(5)),
                                           dict(ws=far(7)), dict(dweights=far(21)), dict(dw1=far(9) + 8)]:
        assert back(**kw) == bpt.BPT_EINVAL, kw


def test_moe_sizes(lib):
    c = moe(n=1000, h=256, ffn_dim=512)
    rows = 2000
    assert 2 * rows * 512 * 2 <= lib.bpt_moe_saved_bytes(c) < 2 * rows * 512 * 2 + 512
    assert rows * 512 * 2 <= lib.bpt_moe_saved_bytes(moe(n=1000, h=256, ffn_dim=512, act=0)) < rows * 512 * 2 + 256
    need = 2 * rows * (512 + 256)
    assert need <= lib.bpt_moe_ffn_workspace_bytes(c, 0) < need + 512
    need = 2 * rows * (3 * 512 + 256) + 4 * rows * 2 * 2
    assert need <= lib.bpt_moe_ffn_workspace_bytes(c, 1) < need + 5 * 256
    assert lib.bpt_moe_ffn_workspace_bytes(c, 2) == 0


@pytest.mark.parametrize("kw", [dict(rows=0), dict(n=0), dict(n=12), dict(k=4), dict(k=20), dict(groups=0), dict(groups=1025),
                                dict(form=3), dict(form=-1), dict(out_dtype=2), dict(flags=2), dict(out_dtype=1, flags=1)], ids=str)
def test_grouped_configs_are_refused(lib, kw):
    g = GroupedConfig(**{**dict(rows=100, n=64, k=72, groups=4, out_dtype=0), **kw})
    c = bpt.BptGroupedConfig(g.rows, g.n, g.k, g.groups, g.form, g.out_dtype, g.flags)
    assert lib.bpt_grouped_gemm(c, far(1), far(2), far(3), far(4), None) == bpt.BPT_EINVAL


def test_grouped_pointers(lib):
    for form in range(3):
        c = bpt.BptGroupedConfig(100, 64, 72, 4, form, 0, 0)
        for a in ((None, far(2), far(3), far(4)), (far(1), None, far(3), far(4)), (far(1), far(2), None, far(4)),
                  (far(1), far(2), far(3), None), (far(1) + 8, far(2), far(3), far(4)), (far(1), far(2) + 8, far(3), far(4)),
                  (far(1), far(2), far(3) + 2, far(4)), (far(1), far(2), far(3), far(4) + 8), (far(1), far(2), far(3), far(1)),
                  (far(1), far(2), far(3), far(2) + 64), (far(1), far(2), far(3), far(3))):
            assert lib.bpt_grouped_gemm(c, *a, None) == bpt.BPT_EINVAL, a
    assert lib.bpt_grouped_gemm(None, far(1), far(2), far(3), far(4), None) == bpt.BPT_EINVAL


def distill(**kw):
    return bpt.make_distill_config(DistillConfig(**{**dict(n=50, h=64, vocab=1000, top_k=8), **kw}))


@pytest.mark.parametrize("kw", [dict(n=0), dict(h=4), dict(h=60), dict(vocab=0), dict(vocab_block=100), dict(vocab_block=-256),
                                dict(top_k=0), dict(top_k=129), dict(teacher=2), dict(grads_dtype=2), dict(temperature=0.0),
                                dict(temperature=-1.0), dict(temperature=float("nan")), dict(temperature=float("inf")),
                                dict(temperature=2000.0), dict(flags=2), dict(grads_dtype=1, flags=1)], ids=str)
def test_distill_configs_are_refused(lib, kw):
    c = distill(**kw)
    assert lib.bpt_lm_distill_saved_bytes(c) == 0
    assert lib.bpt_lm_distill_workspace_bytes(c, 0) == 0 and lib.bpt_lm_distill_workspace_bytes(c, 1) == 0
    assert lib.bpt_lm_distill_fwd(c, *map(far, range(1, 9)), 1 << 40, None) == bpt.BPT_EINVAL
    assert lib.bpt_lm_distill_bwd(c, *map(far, range(1, 5)), 1.0, *map(far, range(5, 8)), 1 << 40, None) == bpt.BPT_EINVAL


def test_distill_pointers_and_sizes(lib):
    c = distill(n=300, vocab=20000)
    names = ("x", "w", "ids", "values", "row_weight", "loss", "saved", "ws")
    n = lib.bpt_lm_distill_workspace_bytes(c, 0)

    def call(n=n, **kw):
        a = {k: far(i + 1) for i, k in enumerate(names)} | kw
        return lib.bpt_lm_distill_fwd(c, *[a[k] for k in names], n, None)

    assert call(n=n - 1) == bpt.BPT_ENOSPC
    for kw in [{k: None} for k in names if k != "row_weight"] + [dict(x=far(1) + 8), dict(row_weight=far(5) + 2), dict(saved=far(7) + 8),
               dict(loss=far(3)), dict(saved=far(1)), dict(ws=far(7) + 256), dict(loss=far(8) + 16)]:
        assert call(**kw) == bpt.BPT_EINVAL, kw
    names2 = ("x", "w", "row_weight", "saved", "dx", "dw", "ws")
    m = lib.bpt_lm_distill_workspace_bytes(c, 1)

    def back(n=m, d=1.0, **kw):
        a = {k: far(i + 1) for i, k in enumerate(names2)} | kw
        return lib.bpt_lm_distill_bwd(c, *[a[k] for k in names2[:4]], d, *[a[k] for k in names2[4:]], n, None)

    assert back(n=m - 1) == bpt.BPT_ENOSPC
    for kw in [{k: None} for k in names2 if k != "row_weight"] + [dict(d=float("nan")), dict(dx=far(1)), dict(dw=far(2)), dict(dw=far(5)),
                                                                 dict(ws=far(4)), dict(dx=far(3)), dict(ws=far(7) + 8)]:
        assert back(**kw) == bpt.BPT_EINVAL, kw
    # the block of n x c_v gradients, dx's accumulator and its K ranges (two tiles: 8)
    need = 300 * 8192 * 2 + 300 * 64 * 4 * 9
    assert need <= m < need + 3 * 256
    parts = (20000 + 255) // 256 * 2
    need = 300 * 8 * 12 + 300 * 12 + (parts + 1) * 300
    assert need <= lib.bpt_lm_distill_saved_bytes(c) < need + 7 * 256
    assert ctypes.sizeof(bpt.BptDistillConfig) == 36
