"""The rotary, append and verification calls between other work: behind a decode step
whose inputs they overwrite, and in a captured graph behind joins of streams, copies
and fills."""
import pytest
import torch

from tests import rotary_reference as ref
from tests.test_gpu_append_rope import Step
from tests.test_gpu_verify import _case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_215_gb300 import pkv as mod
    return mod


@pytest.mark.parametrize("n", [40, 70000])
@pytest.mark.parametrize("graph", [False, True])
def test_what_a_decode_call_reads_is_overwritten_behind_it(pkv, n, graph):
    """Twelve steps: decode, rotate its queries in place, overwrite the slot of the last
    token; the same, bit for bit, as with a wait on the host between all calls."""
    D, bs, hq, hk = 128, 16, 8, 2
    g = torch.Generator().manual_seed(n)
    blocks = -(-n // bs)
    geom = pkv.geometry(1, hq, hk, D, bs, blocks, "bf16")
    start = torch.randn(blocks, 2, 1, hk, bs, D, generator=g).bfloat16().cuda()
    q0, k0, v0 = (torch.randn(1, h, D, generator=g).bfloat16().cuda() for h in (hq, hk, hk))
    tables = torch.randperm(blocks, generator=g).int().view(1, -1).cuda()
    lens, pos = (torch.tensor([x], dtype=torch.int32, device="cuda") for x in (n, n - 1))
    rope, opts = pkv.Rope(D), pkv.launch_opts(pdl=1)
    ws = torch.empty(max(16, pkv.workspace_bytes(geom, 1, n, 0)), dtype=torch.uint8,
                     device="cuda")

    def steps(wait):
        storage = start.clone().view(torch.uint8).view(-1)
        pool = pkv.KVPool(geom, storage=storage)
        q, k, outs = q0.clone(), k0.clone(), torch.zeros(12, 1, hq, D, device="cuda")

        def run():
            for i in range(12):
                pkv.paged_decode_attention(outs[i], q, pool, 0, tables, lens, n, D ** -0.5,
                                           workspace=ws)
                wait()
                pkv.rope_apply(q, q, pos, rope, k_out=k, k=k)
                wait()
                pool.append_rope(0, None, None, k, v0, rope, tables, pos)
                wait()
                if i % 3 == 2:
                    pkv.paged_decode_attention(outs[i], q0, pool, 0, tables, lens, n, D ** -0.5,
                                               workspace=ws)
                    wait()
                    # reads the pool alone while the next kernel may be scheduled
                    pkv.paged_decode_attention(outs[i], q0, pool, 0, tables, lens, n, D ** -0.5,
                                               workspace=ws, opts=opts)
                    wait()
        return run, (outs, q, k, storage), pool

    run, want, keep = steps(torch.cuda.synchronize)
    run()
    torch.cuda.synchronize()
    run, got, keep2 = steps(lambda: None)
    if graph:
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            run()
        captured.replay()
    else:
        torch.cuda.synchronize()
        run()
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def test_captured_behind_joins_copies_and_fills(pkv):
    s = Step(pkv, [20, 3, 700], [4, 1, 9], seed=90)
    freqs, m = ref.frequencies(64)
    rope, side = pkv.Rope(64), torch.cuda.Stream()
    src = [t.clone() for t in (s.q, s.k, s.v)]
    q, k, v = (torch.zeros_like(t) for t in src)
    first, out = torch.zeros_like(q), torch.zeros_like(q)
    case = _case(3, 2, 9001, seed=91)
    given = [t.clone() for t in case]
    tokens = torch.zeros(3, 3, dtype=torch.int32, device="cuda")
    acc = torch.zeros(3, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            q.copy_(src[0])
            for a, b in zip(given, case):
                a.copy_(b)
        k.copy_(src[1])
        first.fill_(7.0)
        s.q_out.fill_(7.0)
        main.wait_stream(side)                               # two predecessors
        pkv.rope_apply(first, q, s.pos, rope)
        with torch.cuda.stream(side):
            tokens.zero_()
            pkv.verify_drafts(tokens, acc, *given)           # beside what follows
        v.copy_(src[2])                                      # a copy right ahead
        s.pool.append_rope(0, s.q_out, q, k, v, rope, s.tables, s.pos, seq_ids=s.seq)
        main.wait_stream(side)
        pkv.rope_apply(out, first, s.pos, rope, backward=True)
    for turn in range(3):
        for t, seed in zip(src, (1, 2, 3)):
            t.copy_(torch.randn(t.shape, generator=torch.Generator().manual_seed(10 * turn + seed)))
        for a, b in zip(case, _case(3, 2, 9001, seed=92 + turn)):
            a.copy_(b)
        for t in (q, k, v, first, out, s.q_out):
            t.fill_(9.0)
        s.pool.storage.copy_(s.before)
        graph.replay()
        torch.cuda.synchronize()
        assert s.pool.check_status() == 0
        s.q, s.k, s.v = (t.clone() for t in src)
        s.check(0, freqs, m, 64, False)
        assert torch.equal(first, s.q_out)
        ref.check_rotated(out, first, s.pos, freqs, m, 64, False, backward=True)
        assert (tokens.tolist(), acc.tolist()) == ref.verify(*case)
