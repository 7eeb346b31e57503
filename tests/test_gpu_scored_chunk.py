"""Chunks (many query rows per KV head) under score rules against the 64-bit reference."""
import pytest
import torch

from tests.scored_reference import Case, slopes
from tests.test_gpu_scored import expand, run

pytestmark = pytest.mark.gpu

RULES = {
    "none": {},
    "cap": dict(cap=20.0),
    "window": dict(window=50),
    "slopes": dict(slopes=True),
    "prefix": dict(prefix=True),
    "docs": dict(docs=True),
    "all": dict(cap=10.0, window=90, slopes=True, prefix=True, docs=True),
}


@pytest.mark.parametrize("rules", RULES)
@pytest.mark.parametrize("kv,hq,hkv,bs,q_len", [
    ("bf16", 8, 2, 16, 40), ("f16", 8, 1, 32, 130), ("e4m3", 8, 2, 16, 65), ("bf16", 2, 2, 64, 300),
    ("e4m3", 4, 2, 64, 33), ("f16", 4, 1, 16, 5)])
def test_chunk(kv, hq, hkv, bs, q_len, rules):
    lens = [q_len + 200, q_len, q_len // 2, 0, q_len + 1, 321]
    case = Case(lens, hq, hkv, 128, kv, bs, q_len, seed=hq + q_len)
    r = expand(case, RULES[rules])
    want = case.reference(**r)
    case.check(run(case, torch.float32, **r), want)
    case.check(run(case, **r), want)


def test_e4m3_block_scales():
    case = Case([150, 64, 333], 8, 2, 128, "e4m3", 16, 48, seed=3, block_scales=True)
    r = expand(case, RULES["all"])
    case.check(run(case, torch.float32, **r), case.reference(**r))


@pytest.mark.parametrize("scale", [-0.3, 0.0, 1.5])
def test_scale_sign_and_size(scale):
    case = Case([90, 217], 8, 2, 128, "bf16", 16, 20, seed=4, q_gain=1.0)
    for r in ({}, {"cap": 30.0}, {"window": 33}):
        case.check(run(case, torch.float32, scale=scale, **r), case.reference(scale=scale, **r))


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "scaled"])
@pytest.mark.parametrize("bs", [16, 64])
def test_unseen_keys_hold_anything(kv, bs):
    # ahead of the first query's window: stale table entries, NaN in the live block's slots
    lens, q_len, window = [400, 43, 290], 40, 70
    case = Case(lens, 8, 2, 128, "e4m3" if kv == "scaled" else kv, bs, q_len, seed=5,
                block_scales=kv == "scaled")
    want = case.reference(window=window)
    for b, n in enumerate(lens):
        first = max(0, n - q_len + 1 - window)
        if kv == "scaled":
            stale = case.tables[b, :first // bs].long()
            case.block_scales[stale] = float("nan")
        case.hide(b, 0, first)
        case.tables[b, :first // bs] = -1
    case.check(run(case, torch.float32, window=window), want)


def test_rows_that_see_nothing():
    lens, q_len = [300, 100, 64], 64
    case = Case(lens, 8, 2, 128, "bf16", 16, q_len, seed=6)
    docs = [[n] * q_len for n in lens]                     # sequence 0: nobody sees anything
    docs[1] = [36 + i if i % 3 else 2 ** 31 - 1 for i in range(q_len)]
    docs[2] = [-1] * 32 + [64] * 32                        # the second half sees nothing
    case.check(run(case, torch.float32, docs=docs), case.reference(docs=docs))


def test_far_documents_start_in_later_tiles():
    # rows of one tile whose keys begin hundreds of keys apart
    q_len = 90
    case = Case([700, 90], 4, 2, 128, "f16", 16, q_len, seed=7)
    docs = [[610 + i if i % 2 else 3 * i for i in range(q_len)], [0] * 45 + [45] * 45]
    case.check(run(case, torch.float32, docs=docs, cap=15.0), case.reference(docs=docs, cap=15.0))


def test_layer_of_a_deeper_pool_and_a_long_context():
    case = Case([3001], 8, 2, 128, "bf16", 32, 35, seed=8, layers=2, layer=1)
    r = dict(cap=25.0, slopes=slopes(8), window=2500)
    case.check(run(case, torch.float32, **r), case.reference(**r))
