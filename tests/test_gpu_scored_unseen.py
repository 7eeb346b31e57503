"""Keys that no query of a sequence sees may hold anything, wherever they lie: ahead of the
seen ones, behind them (queries that see nothing at a chunk's end, as padding has them) and
between them, and the table entries of blocks without a seen key may be stale."""
import random

import pytest
import torch

from tests.scored_reference import Case, slopes
from tests.test_gpu_scored import run

pytestmark = pytest.mark.gpu

NOTHING = 2 ** 31 - 1                # the start of a document behind every query


def documents(kind, lens, q_len, seed=0):
    """doc_starts [B][q_len] whose queries leave keys unseen."""
    rng = random.Random(seed)
    docs = []
    for n in lens:
        at = [n - q_len + i for i in range(q_len)]             # the queries' positions
        if kind == "behind":
            docs.append([max(0, at[0]) // 2] * (q_len // 2) + [NOTHING] * (q_len - q_len // 2))
        elif kind == "between":
            a, b = q_len // 4 + 1, q_len - q_len // 3
            docs.append([0] * a + [NOTHING] * (b - a) + [at[b]] * (q_len - b))
        elif kind == "every third":
            docs.append([at[i] if i % 3 == 0 else NOTHING for i in range(q_len)])
        else:
            row = []
            while len(row) < q_len:
                run_of = rng.choice([1, 2, 5, 17, 40])
                start = rng.choice([NOTHING, at[min(len(row), q_len - 1)], rng.randrange(max(n, 1))])
                row += [start] * run_of
            docs.append(row[:q_len])
    return docs


def hide_unseen(case, **rules):
    """NaN in every slot that no query sees, -1 in the entries of blocks without a seen
    key, and scales there that would spoil what they meet."""
    for b, n in enumerate(case.lens):
        seen = set()
        prefix = rules["prefix"][b] if rules.get("prefix") else 0
        for lo, hi in case.ranges(b, rules.get("window", 0), prefix, rules.get("docs")):
            seen.update(range(max(lo, 0), hi))
        table = case.tables[b].tolist()
        at = [(table[j // case.bs], j % case.bs) for j in range(n) if j not in seen]
        if at:
            at = torch.tensor(at, device="cuda")
            case.pool[at[:, 0], :, case.layer, :, at[:, 1]] = case.nan
        blocks = {j // case.bs for j in seen}
        stale = [j for j in range(-(-n // case.bs)) if j not in blocks]
        if stale:
            if case.block_scales is not None:
                unseen = torch.tensor([table[j] for j in stale], device="cuda")
                case.block_scales[unseen, 0] = float("nan")
                case.block_scales[unseen, 1] = 1e30
            case.tables[b, torch.tensor(stale, device="cuda")] = -1


RULES = {"docs": {}, "cap": dict(cap=9.0), "slopes": dict(cap=12.0, slopes=True),
         "window": dict(window=21), "prefix": dict(prefix=True)}


def rules_of(case, kind, rules, seed=0):
    r = dict(RULES[rules], docs=documents(kind, case.lens, case.q_len, seed))
    if r.get("slopes"):
        r["slopes"] = slopes(case.hq)
    if r.get("prefix"):
        r["prefix"] = [n // 2 for n in case.lens]
    return r


@pytest.mark.parametrize("kind", ["behind", "between", "every third", "any"])
@pytest.mark.parametrize("rules", RULES)
@pytest.mark.parametrize("kv,hq,hkv,bs,q_len", [
    ("bf16", 8, 2, 16, 150), ("f16", 8, 1, 32, 64), ("e4m3", 8, 2, 64, 150), ("scaled", 8, 2, 16, 150),
    ("f16", 2, 2, 16, 300)])
def test_chunk(kv, hq, hkv, bs, q_len, rules, kind):
    lens = [q_len, q_len + 171, q_len // 3, 0]
    case = Case(lens, hq, hkv, 128, "e4m3" if kv == "scaled" else kv, bs, q_len, seed=31,
                block_scales=kv == "scaled")
    r = rules_of(case, kind, rules, seed=q_len)
    want = case.reference(**r)
    hide_unseen(case, **r)
    case.check(run(case, torch.float32, **r), want)


@pytest.mark.parametrize("kind", ["behind", "between", "every third", "any"])
@pytest.mark.parametrize("rules", RULES)
@pytest.mark.parametrize("kv,hq,hkv,bs,q_len", [
    ("bf16", 4, 2, 16, 8), ("f16", 2, 2, 32, 16), ("e4m3", 2, 1, 16, 7), ("scaled", 8, 2, 64, 4),
    ("bf16", 6, 2, 64, 5)])
def test_drafts(kv, hq, hkv, bs, q_len, rules, kind):
    lens = [q_len, 150, 2 * bs + 3, 0, bs + q_len - 1]
    case = Case(lens, hq, hkv, 128, "e4m3" if kv == "scaled" else kv, bs, q_len, seed=32,
                block_scales=kv == "scaled")
    r = rules_of(case, kind, rules, seed=q_len)
    want = case.reference(**r)
    hide_unseen(case, **r)
    before = torch.rand(len(lens), hkv, 160).cuda()
    w = torch.full((len(lens), hkv, 160), -5.0, device="cuda")
    case.check(run(case, torch.float32, w, before, **r), want, w, before)
    for b, n in enumerate(lens):                           # columns behind the sequence
        assert (w[b, :, n:] == -5.0).all()
    case.check(run(case, torch.float32, **r), want)


@pytest.mark.parametrize("kv,hq,rules,kind", [
    ("bf16", 16, "cap", "between"), ("bf16", 16, "prefix", "any"), ("f16", 16, "docs", "any"),
    ("e4m3", 16, "docs", "between"), ("e4m3", 16, "cap", "any"), ("scaled", 16, "docs", "any")])
def test_many_items(kv, hq, rules, kind):
    # more pairs of query tiles than multiprocessors: gaps of one item beside the next one's
    lens = [0, 70, 1, 200, 69, 333, 64, 71, 128, 30, 0, 500, 70, 3, 65, 448, 99, 0, 150, 321, 7, 70,
            641, 12, 192, 90, 35, 256, 77, 400, 129, 100, 110, 300, 44, 59]
    case = Case(lens, hq, 4, 128, "e4m3" if kv == "scaled" else kv, 16, 70, seed=33,
                block_scales=kv == "scaled")
    r = rules_of(case, kind, rules, seed=hq)
    want = case.reference(**r)
    hide_unseen(case, **r)
    got = run(case, torch.float32, **r)
    case.check(got, want)
    for _ in range(5):                                     # the same bits, whoever is late
        assert torch.equal(run(case, torch.float32, **r), got)
