"""A step of speculative decoding as a user runs it: the new and drafted tokens'
queries and keys rotated and appended (append_rope), the drafts attended
(paged_decode_attention_mq), verified (verify_drafts), twice in a row, against the
same steps in 64 bits."""
import numpy as np
import pytest
import torch

import oracle
from tests import rotary_reference as ref
from tests.gpu_harness import TOL
from tests.helpers import np_raw

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("graph", [False, True])
def test_two_speculative_steps(kv, graph):
    from paged_kv_cache_215_gb300 import pkv
    B, K, hq, hk, D, bs, V = 3, 3, 8, 2, 128, 16, 300
    g = torch.Generator().manual_seed(5)
    rand = lambda *s: torch.randn(*s, generator=g)
    lens = [37, 0, 120]
    width, nb = 10, 33
    tables = torch.randperm(nb, generator=g)[:B * width].view(B, width).int()
    geom = pkv.geometry(1, hq, hk, D, bs, nb, kv)
    pool = pkv.KVPool(geom, storage=torch.zeros(pkv.kv_pool_bytes(geom), dtype=torch.uint8,
                                                device="cuda"))
    rope = pkv.Rope(D, scaling="ntk", factor=2.0)
    freqs, m = ref.frequencies(D, scaling="ntk", factor=2.0)
    ks = vs = 0.02 if kv == "e4m3" else 1.0
    opool = np.zeros(pool.nbytes, dtype=np.uint8)
    gdict = dict(num_blocks=nb, num_layers=1, num_kv_heads=hk, block_size=bs, head_dim=D,
                 num_q_heads=hq)
    head = (rand(hq * D, V) * 0.5).cuda()
    dev = tables.cuda()

    def ints(values):
        return torch.tensor(values, dtype=torch.int32, device="cuda")

    # the cached prompts
    seq = [s for s in range(B) for _ in range(lens[s])]
    pos = [i for s in range(B) for i in range(lens[s])]
    kk, vv = rand(len(seq), hk, D).bfloat16(), rand(len(seq), hk, D).bfloat16()
    pool.append_rope(0, None, None, kk.cuda(), vv.cuda(), rope, dev, ints(pos), seq_ids=ints(seq),
                     k_scale=ks, v_scale=vs)

    # one step's buffers, captured or eager
    T = B * (K + 1)
    qkv = torch.zeros(T, (hq + 2 * hk) * D, dtype=torch.bfloat16, device="cuda")
    q, k, v = (t.view(T, -1, D) for t in qkv.split([hq * D, hk * D, hk * D], 1))
    q_out = torch.zeros(T, hq, D, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros(B, K + 1, hq, D, device="cuda")
    positions, total = ints([0] * T), ints([0] * B)
    ids = ints([s for s in range(B) for _ in range(K + 1)])
    draft = torch.zeros(B, K, V, device="cuda")
    drafts = torch.zeros(B, K, dtype=torch.int32, device="cuda")
    ua, us = torch.zeros(B, K, device="cuda"), torch.zeros(B, device="cuda")
    target = torch.zeros(B, K + 1, V, device="cuda")
    tokens = torch.zeros(B, K + 1, dtype=torch.int32, device="cuda")
    acc = torch.zeros(B, dtype=torch.int32, device="cuda")
    maxlen = width * bs
    ws = torch.empty(int(pkv.lib().paged_decode_workspace_bytes_mq(geom, B, K + 1, maxlen, 0)),
                     dtype=torch.uint8, device="cuda")

    def step():
        pool.append_rope(0, q_out, q, k, v, rope, dev, positions, seq_ids=ids, k_scale=ks,
                         v_scale=vs)
        pkv.paged_decode_attention_mq(out, q_out.view(B, K + 1, hq, D), pool, 0, dev, total,
                                      maxlen, D ** -0.5, ks, vs, workspace=ws)
        torch.softmax(out.view(B, K + 1, hq * D) @ head, -1, out=target)
        pkv.verify_drafts(tokens, acc, target, draft, drafts, ua, us)

    if graph:
        positions.fill_(-1)                                  # warm-up and capture store nothing
        step()
        torch.cuda.synchronize()
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            step()
    for turn in range(2):
        qkv.copy_(rand(*qkv.shape).bfloat16())
        positions.copy_(ints([n + i for n in lens for i in range(K + 1)]))
        total.copy_(ints([n + K + 1 for n in lens]))
        draft.copy_(torch.softmax(rand(B, K, V), -1))
        drafts.copy_(torch.randint(0, V, (B, K), generator=g).int())
        ua.copy_(torch.rand(B, K, generator=g) * 0.7)
        us.copy_(torch.rand(B, generator=g))
        captured.replay() if graph else step()
        torch.cuda.synchronize()
        assert pool.check_status() == 0
        ref.check_rotated(q_out, q, positions, freqs, m, D, False)
        # attention over the pool's bytes (checked against the reference in the append's
        # own tests) with the rotated queries, in 64 bits
        want, _ = oracle.decode_mq(np_raw(q_out.cpu().view(B, K + 1, hq, D)), "bf16",
                                   pool.storage.cpu().numpy(), kv, gdict, 0, tables.numpy(),
                                   total.cpu().numpy(), K + 1, D ** -0.5, ks, vs)
        values = oracle.to_f64(pool.storage.cpu().numpy(), kv, vs).reshape(nb, 2, -1)[:, 1]
        assert np.abs(out.cpu().double().numpy() - want).max() <= TOL[kv] * np.abs(values).max()
        assert (tokens.tolist(), acc.tolist()) == ref.verify(target, draft, drafts, ua, us)
        lens = [n + 1 + int(a) for n, a in zip(lens, acc.tolist())]
