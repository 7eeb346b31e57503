"""Documents of one query token that start at any number, behind the query too: such a query
sees nothing, whatever kernel serves it."""
import pytest
import torch

from tests.scored_reference import Case
from tests.test_gpu_scored import run

pytestmark = pytest.mark.gpu

TOP = 2 ** 31 - 1


@pytest.mark.parametrize("prefix", [False, True])
@pytest.mark.parametrize("kv,hq,hkv,dim", [
    ("bf16", 8, 2, 128), ("e4m3", 16, 1, 128), ("f16", 16, 1, 64), ("bf16", 8, 2, 96), ("f32", 4, 2, 128),
    ("f32", 32, 2, 256), ("e4m3", 2, 2, 16)])
def test_one_query(kv, hq, hkv, dim, prefix):
    starts = [TOP, TOP - 1, TOP - 200, 2 ** 30, -TOP - 1, -1, 0]
    lens = [300, 1, 64, 33, 20, 0, 17]
    lens, docs = lens + [120, 119, 50, 51, 5], starts + [120, 118, TOP, 50, 4]
    case = Case(lens, hq, hkv, dim, kv, 16, seed=61)
    r = dict(docs=[[d] for d in docs])
    if prefix:
        r["prefix"] = [n if i % 2 else TOP for i, n in enumerate(lens)]
    want = case.reference(**r)
    w = torch.full((len(lens), hkv, 300), -5.0, device="cuda")
    before = torch.rand(len(lens), hkv, 300).cuda()
    case.check(run(case, torch.float32, w, before, **r), want, w, before)
    case.check(run(case, **r), want)


@pytest.mark.parametrize("kv,hq,hkv,q_len", [("bf16", 4, 2, 4), ("e4m3", 2, 1, 16), ("f16", 8, 1, 40)])
def test_chunks(kv, hq, hkv, q_len):
    lens = [300, q_len, 3, 90]
    case = Case(lens, hq, hkv, 128, kv, 16, q_len, seed=62)
    docs = [[[TOP, TOP - 3, n, n - 1, 0, -TOP - 1][i % 6] for i in range(q_len)] for n in lens]
    case.check(run(case, torch.float32, docs=docs), case.reference(docs=docs))
