"""Chunks with more pairs of query tiles than the GPU has multiprocessors: every CTA walks
over several, of lengths from none to many key tiles."""
import pytest
import torch

from tests.scored_reference import Case
from tests.test_gpu_scored import expand, run

pytestmark = pytest.mark.gpu

# 45 sequences x 4 KV heads x 2 pairs of tiles (the second pair's second tile is empty)
LENS = [0, 70, 1, 200, 69, 333, 64, 71, 128, 30, 0, 500, 70, 3, 65, 64 * 7, 99, 0, 0, 150, 321, 7,
        70, 641, 12, 192, 90, 35, 0, 256, 77, 70, 400, 2, 0, 0, 0, 129, 100, 110, 300, 44, 59, 64, 710]


@pytest.mark.parametrize("kv,rules", [
    ("bf16", {"cap": 12.0, "docs": True}), ("f16", {"slopes": True, "prefix": True, "window": 150}),
    ("e4m3", {"window": 40}), ("scaled", {})])
def test_many_items(kv, rules):
    case = Case(LENS, 16, 4, 128, "e4m3" if kv == "scaled" else kv, 16, 70, seed=11,
                block_scales=kv == "scaled")
    r = expand(case, rules)
    want = case.reference(**r)
    got = run(case, torch.float32, **r)
    case.check(got, want)
    again = run(case, torch.float32, **r)
    for _ in range(10):                      # the same bits, whoever is late
        assert torch.equal(run(case, torch.float32, **r), again)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_many_items_over_stale_heads(kv):
    window, q_len = 33, 70
    case = Case(LENS, 16, 4, 128, kv, 16, q_len, seed=12)
    want = case.reference(window=window)
    for b, n in enumerate(LENS):
        first = max(0, n - q_len + 1 - window)
        case.hide(b, 0, first)
        case.tables[b, :first // 16] = -1
    case.check(run(case, window=window), want)


@pytest.mark.parametrize("hq,hkv", [(64, 64), (64, 1)])
def test_every_group_size_with_many_items(hq, hkv):
    # 128 tokens a tile, and 2
    case = Case([300, 0, 140, 257, 66], hq, hkv, 128, "f16", 16, 140, seed=13)
    case.check(run(case, window=100), case.reference(window=100))
