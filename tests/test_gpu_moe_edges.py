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
