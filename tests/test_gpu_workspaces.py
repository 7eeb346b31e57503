"""Calls on a given stream that get no workspace take one from that stream's memory: a block
of the current stream's may still be in use by what was launched there."""
import pytest
import torch

from tests.scored_reference import Case

pytestmark = pytest.mark.gpu


def calls(case, pool):
    """Every call that takes a workspace, by name: f(stream=...)."""
    from paged_kv_cache_215_gb300 import pkv
    q1 = case.q[:, 0].contiguous()
    out, outq = torch.zeros_like(q1), torch.zeros_like(case.q)
    o32, lse = torch.zeros(q1.shape, device="cuda"), torch.zeros(q1.shape[:2], device="cuda")
    n, top = case.seq_lens, max(case.lens)
    kv = torch.zeros(case.batch, case.hkv, case.dim, dtype=q1.dtype, device="cuda")
    common = (pool, 0, case.tables, n, top, case.scale)
    w = torch.rand(case.batch, case.hkv, top).cuda()
    prefix = case.tables[0, :2].contiguous()
    shared = torch.zeros(case.batch, dtype=torch.int32, device="cuda")
    fresh = case.tables[:, :1].contiguous()
    keep, lens = torch.zeros_like(n), torch.zeros_like(n)
    return {
        "attention": lambda **k: pkv.paged_decode_attention(out, q1, *common, **k),
        "partial": lambda **k: pkv.paged_decode_attention_partial(o32, lse, q1, *common, **k),
        "step": lambda **k: pkv.paged_decode_step(out, q1, kv, kv, *common, **k),
        "mq": lambda **k: pkv.paged_decode_attention_mq(outq, case.q, *common, **k),
        "cascade": lambda **k: pkv.paged_decode_attention_cascade(
            out, q1, pool, 0, prefix, 32, shared, case.tables, n, top, case.scale, **k),
        "scored": lambda **k: pkv.paged_decode_attention_scored(outq, case.q, *common, **k),
        # (nothing is kept: the old blocks stand in for new ones)
        "evict": lambda **k: pool.evict(0, fresh, case.tables, n, top, keep, 0, w,
                                        torch.zeros_like(w), lens, **k),
    }


@pytest.mark.parametrize("name", ["attention", "partial", "step", "mq", "cascade", "scored", "evict"])
def test_workspaces_come_from_the_stream_of_the_call(name, monkeypatch):
    case = Case([90, 64], 8, 2, 128, "bf16", 16, 2, seed=1)
    pool = case.handle()
    call = calls(case, pool)[name]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    taken, empty = [], torch.empty

    def recorded(*a, **k):
        t = empty(*a, **k)
        if k.get("dtype") == torch.uint8:
            taken.append(torch.cuda.current_stream())
        return t
    monkeypatch.setattr(torch, "empty", recorded)
    call(stream=side)
    call()
    torch.cuda.synchronize()
    assert taken == [side, torch.cuda.current_stream()] and pool.check_status() == 0
    assert torch.cuda.current_stream() != side


def test_a_call_behind_one_on_another_stream_leaves_its_scratch_alone():
    # calls without workspaces in turn on the current stream, where each one's scratch is free
    # again while its launches still wait, and on another
    from paged_kv_cache_215_gb300 import pkv
    cases = [Case([6000, 4000], 8, 2, 128, "bf16", 16, seed=s) for s in (2, 3)]
    pools = [c.handle() for c in cases]
    outs = [torch.zeros(c.q.shape, device="cuda") for c in cases]
    weights = [torch.zeros(2, 2, 6000, device="cuda") for _ in cases]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)                          # what is launched here runs later
    for _ in range(10):
        for c, p, o, w, s in zip(cases, pools, outs, weights, (None, side)):
            pkv.paged_decode_attention_scored(o, c.q, p, 0, c.tables, c.seq_lens, 6000, c.scale,
                                              scores=pkv.Scores(cap=20.0), weights=w, stream=s)
    torch.cuda.synchronize()
    for c, p, o, w in zip(cases, pools, outs, weights):
        assert p.check_status() == 0
        c.check(o, c.reference(cap=20.0), w)


def test_evictions_on_two_streams_leave_each_others_scratch_alone():
    from tests.test_gpu_evict import weights_of
    from tests.scored_reference import evicted
    side = torch.cuda.Stream()
    sets = []
    for seed in (4, 5):
        case = Case([5000], 4, 2, 16, "f16", 16, seed=seed, spare=130)
        used = set(case.tables[0][case.tables[0] >= 0].tolist())
        fresh = torch.tensor([[b for b in range(case.nb) if b not in used][:125]]).int().cuda()
        sets.append((case, case.handle(), fresh, weights_of("random", 1, 2, 5000, seed).cuda(),
                     torch.zeros(1, 2, 2000, device="cuda"),
                     torch.zeros(1, dtype=torch.int32, device="cuda"),
                     torch.full((1,), 2000, dtype=torch.int32, device="cuda")))
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)
    for _ in range(5):
        for (case, pool, fresh, w, new_w, lens, keep), s in zip(sets, (None, side)):
            pool.evict(0, fresh, case.tables, case.seq_lens, 5000, keep, 100, w, new_w, lens, stream=s)
    torch.cuda.synchronize()
    for case, pool, fresh, w, new_w, lens, _ in sets:
        assert pool.check_status() == 0 and lens.tolist() == [2000]
        for h in range(2):
            j = torch.tensor(evicted(w[0, h].cpu(), 5000, 2000, 100))
            assert torch.equal(new_w[0, h].cpu(), w[0, h].cpu()[j])
            t = torch.arange(2000)
            at = lambda table, x: case.pool[table[0].cpu().long()[x // 16].cuda(), :, 0, h, (x % 16).cuda()]
            assert torch.equal(at(fresh, t), at(case.tables, j))


def test_scales_are_read_back_behind_their_stream():
    from paged_kv_cache_215_gb300 import pkv
    x = [torch.randn(1000, device="cuda") for _ in range(3)]
    want = pkv.fp8_scales(x[:2], x[2:])
    pkv.fp8_scales([9 * x[0]], [7 * x[1]])                 # what is free now holds other scales
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)                      # what is launched there runs later
    assert pkv.fp8_scales(x[:2], x[2:], stream=side) == want and min(want) > 0
