"""Scored attention and eviction at the ends of their arguments, and chunks on two streams
and in a graph."""
import pytest
import torch

from tests.scored_reference import Case
from tests.test_gpu_scored import run

pytestmark = pytest.mark.gpu

SHAPES = [("bf16", 8, 2, 128, 1), ("e4m3", 8, 2, 128, 2), ("f32", 4, 2, 64, 1), ("bf16", 8, 2, 128, 40),
          ("e4m3", 16, 1, 128, 20)]


@pytest.mark.parametrize("kv,hq,hkv,dim,q_len", SHAPES)
def test_no_tokens_at_all(kv, hq, hkv, dim, q_len):
    case = Case([0, 0, 0], hq, hkv, dim, kv, 16, q_len, seed=1)
    for rules in ({}, dict(window=3), dict(cap=5.0)):
        assert torch.equal(run(case, torch.float32, max_len=0, **rules),
                           torch.zeros_like(case.q, dtype=torch.float32))


@pytest.mark.parametrize("kv,hq,hkv,dim,q_len", SHAPES)
def test_rules_at_the_ends_of_their_types_change_nothing(kv, hq, hkv, dim, q_len):
    lens, top = [150, 1, 40, 0], 2 ** 31 - 1
    case = Case(lens, hq, hkv, dim, kv, 16, q_len, seed=2)
    want = case.reference()
    for rules in (dict(window=top), dict(prefix=[-top - 1, -1, 0, 5]),
                  dict(docs=[[-top - 1] * q_len] * 4)):
        case.check(run(case, torch.float32, **rules), want)
    # a prefix longer than the sequence: every query sees every key
    whole = case.reference(prefix=lens)
    case.check(run(case, torch.float32, prefix=[top] * 4), whole)
    # a cap far above every score
    case.check(run(case, torch.float32, cap=1e20), case.reference(cap=1e20))


def test_evicting_nothing_from_nothing():
    from paged_kv_cache_215_gb300 import pkv  # noqa: F401
    case = Case([0, 0], 8, 2, 128, "bf16", 16, seed=3, width=2)
    pool = case.handle()
    before = case.pool.clone()
    lens = torch.full((2,), -9, dtype=torch.int32, device="cuda")
    w, new_w = torch.ones(2, 2, 4, device="cuda"), torch.full((2, 2, 5), -9.0, device="cuda")
    fresh = torch.zeros(2, 1, dtype=torch.int32, device="cuda")
    pool.evict(0, fresh, case.tables, case.seq_lens, 0, torch.full_like(lens, 7), 3, w, new_w, lens)
    torch.cuda.synchronize()
    assert lens.tolist() == [0, 0] and not new_w.any() and pool.check_status() == 0
    assert torch.equal(case.pool.view(torch.int16), before.view(torch.int16))


def chunk(case, pool, out, window, stream=None):
    from paged_kv_cache_215_gb300 import pkv
    ws = torch.empty(max(16, pkv.scored_workspace_bytes(pool.geom, case.batch, case.q_len, 2000)),
                     dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    return lambda: pkv.paged_decode_attention_scored(
        out, case.q, pool, 0, case.tables, case.seq_lens, 2000, case.scale,
        scores=pkv.Scores(window=window), k_scale=case.k_scale, v_scale=case.v_scale, workspace=ws,
        stream=stream)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_chunks_on_two_streams_at_once(kv):
    cases = [Case([1000, 300, 999], 16, 4, 128, kv, 16, 200, seed=s, width=125) for s in (4, 5)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [torch.empty(c.q.shape, device="cuda") for c in cases]
    pools = [c.handle() for c in cases]
    calls = [chunk(c, p, o, 170, s) for c, p, o, s in zip(cases, pools, outs, streams)]
    for _ in range(20):
        for call in calls:
            call()
    torch.cuda.synchronize()
    for c, p, o in zip(cases, pools, outs):
        assert p.check_status() == 0
        c.check(o, c.reference(window=170))


def test_a_captured_chunk_goes_by_the_lengths_it_finds():
    case = Case([700, 90, 1200], 8, 2, 128, "bf16", 16, 64, seed=6, width=125)
    pool, out = case.handle(), torch.empty(case.q.shape, device="cuda")
    call = chunk(case, pool, out, 100)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for lens in ([700, 90, 1200], [3, 64, 0], [650, 1, 65]):
        case.lens = lens
        case.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        assert pool.check_status() == 0
        case.check(out, case.reference(window=100))
