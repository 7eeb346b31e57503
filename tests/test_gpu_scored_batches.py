"""Scored decode of more sequences than a warp has lanes (their run of blocks is found by
another loop), and chunks into outputs that start on a 16-byte boundary only."""
import random

import pytest
import torch

from tests.scored_reference import Case
from tests.test_gpu_scored import expand, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rules", [{}, dict(cap=15.0, window=70), dict(slopes=True, docs=True)])
@pytest.mark.parametrize("kv,hq,hkv,dim,bs,q_len,batch", [
    ("bf16", 8, 2, 128, 16, 1, 33), ("bf16", 4, 1, 128, 32, 4, 64), ("e4m3", 8, 8, 128, 16, 1, 70),
    ("f16", 16, 1, 128, 16, 1, 100), ("f32", 4, 2, 64, 16, 1, 40), ("e4m3", 4, 2, 128, 64, 3, 257)])
def test_many_sequences(kv, hq, hkv, dim, bs, q_len, batch, rules):
    rng = random.Random(batch)
    lens = [rng.choice([0, 1, 7, bs, rng.randrange(90), rng.randrange(400)]) for _ in range(batch)]
    lens[0], lens[-1], lens[31] = 0, 333, 0                # nothing at a warp's ends
    case = Case(lens, hq, hkv, dim, kv, bs, q_len, seed=batch)
    r = expand(case, rules)
    want = case.reference(**r)
    before = torch.rand(batch, hkv, 400).cuda()
    w = torch.full((batch, hkv, 400), -5.0, device="cuda")
    case.check(run(case, torch.float32, w, before, **r), want, w, before)
    case.check(run(case, **r), want)


def test_no_sequence_holds_a_token():
    case = Case([0] * 50, 8, 2, 128, "bf16", 16, seed=1)
    w = torch.full((50, 2, 9), -5.0, device="cuda")
    out = run(case, torch.float32, w, max_len=9)
    assert not out.any() and (w == -5.0).all()


@pytest.mark.parametrize("rules", [{}, dict(cap=20.0), dict(slopes=True)])
@pytest.mark.parametrize("out_dtype", [torch.float32, None])
@pytest.mark.parametrize("kv", ["bf16", "f16", "e4m3"])
def test_outputs_on_16_byte_boundaries(kv, out_dtype, rules):
    from paged_kv_cache_215_gb300 import pkv
    case = Case([300, 33, 0, 90], 8, 2, 128, kv, 16, 50, seed=2)
    r = expand(case, rules)
    dtype = out_dtype or case.q.dtype
    ahead = 16 // torch.tensor([], dtype=dtype).element_size()
    store = torch.full((ahead + case.q.numel() + 64,), -3.0, dtype=dtype, device="cuda")
    out = store[ahead:ahead + case.q.numel()].view(case.q.shape)
    assert out.data_ptr() % 32 == 16
    pool = case.handle()
    sc = pkv.Scores(cap=r.get("cap", 0.0),
                    slopes=r["slopes"].float().cuda() if r.get("slopes") is not None else None)
    pkv.paged_decode_attention_scored(out, case.q, pool, 0, case.tables, case.seq_lens, 300,
                                      case.scale, scores=sc, k_scale=case.k_scale,
                                      v_scale=case.v_scale)
    torch.cuda.synchronize()
    assert pool.check_status() == 0
    case.check(out, case.reference(**r))
    assert (store[:ahead] == -3.0).all() and (store[ahead + case.q.numel():] == -3.0).all()
