"""The bits of a scored call go by what its queries see: what lies in the slots around, of
any size, changes none (a cap's polynomial is chosen by the scores of a warp)."""
import pytest
import torch

from tests.scored_reference import Case
from tests.test_gpu_scored import run

pytestmark = pytest.mark.gpu


def fill_unseen(case, seen, value):
    """`value` in every slot of the pool that no sequence's queries see."""
    fill = torch.tensor([value]).to(torch.float8_e4m3fn if case.kv == "e4m3" else case.pool.dtype)
    fill = fill.view(torch.uint8) if case.kv == "e4m3" else fill
    keep = torch.zeros(case.nb, case.bs, dtype=torch.bool)
    for b, ranges in enumerate(seen):
        for lo, hi in ranges:
            t = torch.arange(lo, hi)
            keep[case.tables[b].cpu()[t // case.bs].long(), t % case.bs] = True
    blocks, slots = (~keep).nonzero(as_tuple=True)
    case.pool[blocks.cuda(), :, case.layer, :, slots.cuda()] = fill.cuda()


@pytest.mark.parametrize("rules", [dict(cap=30.0), dict(cap=30.0, window=29), dict(cap=30.0, slopes=True),
                                   dict(cap=30.0, docs=True)])
@pytest.mark.parametrize("kv,hq,hkv,dim,bs,q_len", [
    ("bf16", 8, 2, 128, 16, 1), ("e4m3", 8, 2, 128, 64, 1), ("f16", 16, 1, 128, 32, 1),
    ("bf16", 8, 2, 128, 64, 4), ("e4m3", 4, 2, 128, 16, 7), ("f32", 4, 2, 64, 16, 1),
    ("bf16", 8, 2, 128, 16, 40), ("f16", 8, 1, 128, 16, 150), ("e4m3", 8, 2, 128, 64, 70)])
def test_unseen_slots_change_no_bit(kv, hq, hkv, dim, bs, q_len, rules):
    lens = [300, q_len, 77, 5 * bs + 1]
    # scores small beside the cap, so that the shortest polynomial serves them
    case = Case(lens, hq, hkv, dim, kv, bs, q_len, seed=51, q_gain=0.5)
    r = dict(rules)
    if r.pop("slopes", None):
        r["slopes"] = torch.tensor([2.0 ** -(h + 1) for h in range(hq)])
    if r.pop("docs", None):
        r["docs"] = [[max(0, n - q_len + i - 9) for i in range(q_len)] for n in lens]
    seen = [case.ranges(b, r.get("window", 0), 0, r.get("docs")) for b in range(len(lens))]
    record = (q_len * hq // hkv) <= 16
    results = []
    for value in (0.0, 7.0, 300.0, -40.0, float("nan")):
        fill_unseen(case, seen, value)
        w = torch.zeros(len(lens), hkv, max(lens), device="cuda") if record else None
        results.append((run(case, torch.float32, w, **r), w))
    case.check(results[0][0], case.reference(**r))
    for out, w in results[1:]:
        assert torch.equal(out, results[0][0])
        assert not record or torch.equal(w, results[0][1])
