"""The modified attention's backward where clusters of two, four and eight CTAs
share a key tile, and where none does: shapes on all sides of the choice, with
masks that leave parts of a cluster without a pair, against the definition (the
bounds of the ordinary cases), repeatable bit by bit in the fixed-order mode."""
import pytest
import torch

import blockwise_attention_ffn_gb300 as bpt
from blockwise_attention_ffn_gb300.presets import LayerConfig
from tests.test_gpu_attention_mod import as_int32, check_all, make, run, windows

pytestmark = pytest.mark.gpu

CASES = [
    # b, s, H, K, d, windows, cap, slopes
    (2, 600, 16, 4, 64, "causal", 0.0, False),    # 40 items of up to 20 tiles
    (2, 600, 16, 4, 80, "padded", 20.0, True),
    (1, 600, 20, 5, 128, "docs", 0.0, True),      # 25 items of up to 20 tiles
    (1, 600, 20, 5, 96, "prefix", 30.0, False),
    (1, 385, 16, 2, 112, "causal", 0.0, False),   # 8 items of up to 32 tiles
    (1, 385, 16, 2, 64, "holes", 50.0, True),
    (3, 1111, 12, 4, 96, "prefix", 30.0, True),   # 108 items of up to 27 tiles
    (2, 1155, 24, 4, 80, "causal", 0.0, False),   # 80 items of up to 60 tiles
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_against_the_definition(case):
    b, s, H, K, d, kind, cap, biased = case
    causal, begin, end = windows(kind, b, s, seed=s + d)
    slopes = [2.0 ** -(1 + n % 8) for n in range(H)] if biased else None
    cfg = LayerConfig(b=b, s=s, h=H * d, n_heads=H, n_kv_heads=K, head_dim=d, ffn_dim=64, causal=causal)
    mod = bpt.ScoreMod(as_int32(begin), as_int32(end), None if slopes is None else torch.tensor(slopes, device="cuda"), cap)
    qkv, dout = make(b, s, H, K, d, seed=s)
    got = run(cfg, mod, qkv, dout, bpt.BPT_FLAG_DETERMINISTIC)
    check_all(cfg, causal, begin, end, slopes, cap, qkv, dout, *got)
    again = run(cfg, mod, qkv, dout, bpt.BPT_FLAG_DETERMINISTIC)
    assert all(torch.equal(a, c) for a, c in zip(got, again))
    check_all(cfg, causal, begin, end, slopes, cap, qkv, dout, *run(cfg, mod, qkv, dout))
