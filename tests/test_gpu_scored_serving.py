"""Scored attention, its record and eviction together, as a serving loop uses them: behind
and ahead of work that writes their inputs and reads their outputs, captured and replayed,
on another stream, and a cache that is appended to, attended, evicted and goes on."""
import pytest
import torch

from tests.scored_reference import Case, evicted, slopes
from tests.test_gpu_scored import expand, run

pytestmark = pytest.mark.gpu


def calls(case, pool, rules, out, weights, ws, q, lens, tables, **kw):
    from paged_kv_cache_215_gb300 import pkv
    pkv.paged_decode_attention_scored(out, q, pool, 0, tables, lens, max(case.lens), case.scale,
                                      scores=rules, weights=weights, weights_in=weights,
                                      workspace=ws, **kw)


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_calls_in_a_row_see_what_was_written_ahead(graph, kv):
    # every input (pool, q, lengths, tables, weights) is overwritten by the launch just ahead
    from paged_kv_cache_215_gb300 import pkv
    case = Case([700, 350, 90], 8, 2, 128, kv, 16, seed=1)
    rules = pkv.Scores(cap=12.0)
    pool = case.handle()
    zero = dict(pool=torch.zeros_like(case.pool), q=torch.zeros_like(case.q),
                lens=torch.zeros_like(case.seq_lens), tables=torch.zeros_like(case.tables))
    data = dict(pool=case.pool.clone(), q=case.q.clone(), lens=case.seq_lens.clone(),
                tables=case.tables.clone())
    live = dict(pool=case.pool, q=case.q, lens=case.seq_lens, tables=case.tables)
    out = torch.zeros(case.q.shape, device="cuda")
    weights = torch.zeros(3, 2, 700, device="cuda")
    copies = torch.zeros(2, *out.shape, device="cuda")
    kw = dict(k_scale=case.k_scale, v_scale=case.v_scale)
    ws = torch.empty(pkv.scored_workspace_bytes(pool.geom, 3, 1, 700, True), dtype=torch.uint8,
                     device="cuda")

    def step():
        weights.zero_()
        for turn, source in enumerate((data, zero, data)):
            for name in live:
                live[name].copy_(source[name])
            calls(case, pool, rules, out, weights, ws, case.q, case.seq_lens, case.tables, **kw)
            if source is data:
                copies[turn // 2].copy_(out)
            out.fill_(float("nan"))
    if graph:
        step()
        torch.cuda.synchronize()
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            step()
        for _ in range(3):
            captured.replay()
    else:
        for _ in range(3):
            step()
    torch.cuda.synchronize()
    assert pool.check_status() == 0
    want = case.reference(cap=12.0)
    assert torch.equal(copies[0], copies[1])
    half = [(o, b, 2 * w, 2 * e) for o, b, w, e in want]     # two of the three calls saw tokens
    case.check(copies[0], half, weights)


def test_two_graphs_share_a_workspace_and_replay_in_turn():
    from paged_kv_cache_215_gb300 import pkv
    cases = [Case([500, 33], 8, 2, 128, "bf16", 16, seed=2),
             Case([64, 450], 8, 2, 128, "bf16", 16, 2, seed=3)]
    pools = [c.handle() for c in cases]
    ws = torch.empty(max(pkv.scored_workspace_bytes(p.geom, 2, c.q_len, 500, True)
                         for c, p in zip(cases, pools)), dtype=torch.uint8, device="cuda")
    outs = [torch.zeros(c.q.shape, device="cuda") for c in cases]
    weights = [torch.zeros(2, 2, 500, device="cuda") for _ in cases]
    graphs = []
    for c, p, o, w in zip(cases, pools, outs, weights):
        def call():
            w.zero_()
            calls(c, p, pkv.Scores(window=100), o, w, ws, c.q, c.seq_lens, c.tables)
        call()
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            call()
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for c, o, w in zip(cases, outs, weights):
        c.check(o, c.reference(window=100), w)


def test_two_streams_at_once():
    from paged_kv_cache_215_gb300 import pkv
    cases = [Case([900, 100], 8, 2, 128, "bf16", 16, seed=4), Case([40, 800], 4, 4, 64, "f16", 16, seed=5),
             Case([600], 8, 2, 128, "e4m3", 16, 40, seed=6)]
    pools = [c.handle() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [torch.zeros(c.q.shape, device="cuda") for c in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, p, s, o in zip(cases, pools, streams, outs):
            pkv.paged_decode_attention_scored(o, c.q, p, 0, c.tables, c.seq_lens, max(c.lens),
                                              c.scale, scores=pkv.Scores(cap=9.0),
                                              k_scale=c.k_scale, v_scale=c.v_scale, stream=s)
    torch.cuda.synchronize()
    for c, o in zip(cases, outs):
        c.check(o, c.reference(cap=9.0))


def test_outputs_count_as_written():
    case = Case([30], 4, 2, 128, "bf16", 16, seed=7)
    w = torch.zeros(1, 2, 30, device="cuda")
    v = w._version
    run(case, weights=w)
    assert w._version > v


def append(case, pool, k, v, tables, positions):
    ids = torch.arange(len(positions), dtype=torch.int32, device="cuda")
    pool.append_tokens(0, k, v, tables, ids, positions)


@pytest.mark.parametrize("kv,bs,graph", [("bf16", 16, False), ("f16", 32, True)])
def test_a_cache_under_a_budget(kv, bs, graph):
    """Steps of append, scored attention with its record and, every few tokens, eviction
    into fresh blocks, against the same steps on the host in 64 bits: the record decides
    what stays, so every step's weights matter to the next."""
    from paged_kv_cache_215_gb300 import pkv
    B, hq, hkv, D, budget, slack, recent = 3, 8, 2, 128, 48, 8, 12
    lens = [budget, budget - 5, budget - 1]
    case = Case(lens, hq, hkv, D, kv, bs, seed=8)
    dt = case.q.dtype
    gen = torch.Generator().manual_seed(9)
    width = budget + slack
    per = -(-width // bs)
    geom_blocks = case.nb + 2 * B * per
    pool_t = torch.zeros((geom_blocks,) + case.pool.shape[1:], dtype=dt, device="cuda")
    pool_t[:case.nb] = case.pool
    case.pool, case.nb = pool_t, geom_blocks
    pool = case.handle()
    pool.reserve(list(range(case.nb - 2 * B * per)))        # the prompts' and the spare blocks
    tables = torch.zeros(B, per, dtype=torch.int32, device="cuda")
    tables[:, :case.tables.shape[1]] = case.tables[:, :per].clamp(min=0)
    ids = pool.alloc(2 * B * per)
    sets = [torch.tensor(ids[i * B * per:(i + 1) * B * per]).view(B, per).int().cuda()
            for i in range(2)]
    # the first tables are too short for the slack: begin in a set of their own
    weights = [torch.zeros(B, hkv, width, device="cuda") for _ in range(2)]
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    keep = torch.full((B,), budget, dtype=torch.int32, device="cuda")
    pool.evict(0, sets[0], tables, n, budget, keep, 10 ** 6, weights[1], weights[0], n.clone())
    now = 0
    # the host's cache: per sequence and head K, V [n, D] and weights [n]
    host = []
    for b in range(B):
        k, v = case.kv_of(b)
        host.append([[k[:, h], v[:, h], torch.zeros(lens[b], dtype=torch.float64)]
                     for h in range(hkv)])
    out = torch.zeros(B, hq, D, device="cuda")
    q = torch.zeros(B, hq, D, dtype=dt, device="cuda")
    kn = torch.zeros(B, hkv, D, dtype=dt, device="cuda")
    vn = torch.zeros(B, hkv, D, dtype=dt, device="cuda")
    rules = pkv.Scores(cap=20.0)
    ws = torch.empty(pkv.scored_workspace_bytes(pool.geom, B, 1, width, True), dtype=torch.uint8,
                     device="cuda")
    lens_d, pos_d = n.clone(), n.clone()
    graphs = {}

    def attend(which):
        append(case, pool, kn, vn, sets[which], pos_d)
        pkv.paged_decode_attention_scored(out, q, pool, 0, sets[which], lens_d, width, D ** -0.5,
                                          scores=rules, weights=weights[which],
                                          weights_in=weights[which], workspace=ws)
    lens = list(lens)
    for step in range(40):
        kk, vv, qq = (torch.randn(B, h, D, generator=gen).to(dt) for h in (hkv, hkv, hq))
        qq = (2 * qq.float()).to(dt)
        kn.copy_(kk), vn.copy_(vv), q.copy_(qq)
        pos_d.copy_(torch.tensor(lens, dtype=torch.int32))
        lens = [x + 1 for x in lens]
        lens_d.copy_(torch.tensor(lens, dtype=torch.int32))
        if graph and now not in graphs:
            before = weights[now].clone()
            attend(now)                                      # warm up, then put back
            torch.cuda.synchronize()
            weights[now].copy_(before)
            graphs[now] = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graphs[now]):
                attend(now)
        graphs[now].replay() if graph else attend(now)
        torch.cuda.synchronize()
        got, gw = out.double().cpu(), weights[now].double().cpu()
        for b in range(B):
            for h in range(hkv):
                K, V, W = host[b][h]
                K = torch.cat([K, kk[b, h].double()[None]])
                V = torch.cat([V, vv[b, h].double()[None]])
                W = torch.cat([W, torch.zeros(1, dtype=torch.float64)])
                for g in range(h * hq // hkv, (h + 1) * hq // hkv):
                    x = 20.0 * torch.tanh(K @ qq[b, g].double() * D ** -0.5 / 20.0)
                    p = torch.softmax(x, 0)
                    # scores within 2^-13 (128 products summed in 32 bits), weights' rounding
                    # 2^-11 (f16) and fp32 sums
                    bound = (2 ** -12 + 2 ** -11) * (p @ V.abs()) + 1e-6
                    assert ((got[b, g] - p @ V).abs() <= bound).all(), (step, b, g)
                    W = W + p
                assert ((gw[b, h, :lens[b]] - W).abs() <= 2 ** -12 * (W + 1e-3)).all()
                host[b][h] = [K, V, W]
        if max(lens) == width:
            nxt = 1 - now
            new_lens = torch.zeros(B, dtype=torch.int32, device="cuda")
            index = torch.full((B, hkv, budget), -1, dtype=torch.int32, device="cuda")
            pool.evict(0, sets[nxt], sets[now], lens_d, width, keep, recent, weights[now],
                       weights[nxt], new_lens, index=index)
            torch.cuda.synchronize()
            w32 = weights[now].cpu()
            for b in range(B):
                for h in range(hkv):
                    # by the device's own weights: near ties go either way in 64 bits
                    j = evicted(w32[b, h], lens[b], budget, recent)
                    assert index[b, h, :len(j)].tolist() == j
                    host[b][h] = [t[j] for t in host[b][h][:2]] + [w32[b, h, j].double()]
            lens = [min(x, budget) for x in lens]
            assert new_lens.tolist() == lens
            assert (weights[nxt][:, :, budget:] == 0).all()
            now = nxt
    assert pool.check_status() == 0


def test_eviction_behind_a_call_and_ahead_of_one():
    # the weights are written by the call just ahead, the new cache read by the next one
    from paged_kv_cache_215_gb300 import pkv
    case = Case([400, 130], 8, 2, 128, "bf16", 16, seed=10)
    keep, recent = [64, 100], 16
    first = case.nb
    case.pool = torch.cat([case.pool, torch.full((16,) + case.pool.shape[1:], float("nan"),
                                                 dtype=case.pool.dtype, device="cuda")])
    case.nb += 16
    fresh = torch.arange(first, first + 16).view(2, 8).int().cuda()
    pool = case.handle()
    out, after = torch.zeros(2, 8, 128, device="cuda"), torch.zeros(2, 8, 128, device="cuda")
    w, new_w = torch.zeros(2, 2, 400, device="cuda"), torch.full((2, 2, 128), -1.0, device="cuda")
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    index = torch.zeros(2, 2, 100, dtype=torch.int32, device="cuda")
    k = torch.tensor(keep, dtype=torch.int32, device="cuda")
    q = case.q[:, 0].contiguous()
    for _ in range(3):
        new_w.fill_(-1.0)
        lens.zero_()
        pkv.paged_decode_attention_scored(out, q, pool, 0, case.tables, case.seq_lens, 400,
                                          case.scale, weights=w)
        pool.evict(0, fresh, case.tables, case.seq_lens, 400, k, recent, w, new_w, lens,
                   index=index)
        pkv.paged_decode_attention_scored(after, q, pool, 0, fresh, lens, 128, case.scale,
                                          weights=new_w, weights_in=new_w)
    torch.cuda.synchronize()
    assert pool.check_status() == 0 and lens.tolist() == keep
    case.check(out, case.reference(), w)
    for b in range(2):
        K, V = case.kv_of(b)
        for h in range(2):
            j = evicted(w[b, h].cpu(), case.lens[b], keep[b], recent)
            assert index[b, h, :keep[b]].tolist() == j
            for g in range(4 * h, 4 * h + 4):
                p = torch.softmax(K[j, h] @ q[b, g].double().cpu() * case.scale, 0)
                bound = 2.0 ** -11 * (p @ V[j, h].abs()) + 1e-6
                assert ((after[b, g].double().cpu() - p @ V[j, h]).abs() <= bound).all()
