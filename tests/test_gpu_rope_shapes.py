"""The shapes of the rotary kernel that long calls take (four heads a thread, token
groups or, above 64 MiB of rows, head groups next to one another), alone and into a pool: every row equals
what a call of a few tokens gives, bit for bit, and a sample of them the 64-bit
reference.  Sizes are stated for 152 SMs: a call takes four heads a thread above 152 x 8
blocks of 128 threads (152 x 10 for an E4M3 pool) with one part of one head each."""
import pytest
import torch

from tests import rotary_reference as ref
from tests.test_gpu_append_rope import Step

pytestmark = pytest.mark.gpu
DT = [torch.float32, torch.float16, torch.bfloat16]


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_215_gb300 import pkv as mod
    return mod


def _x(shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


ROWS = [  # tokens, q heads, k heads, head_dim, rotary_dim
    (3001, 13, 3, 128, 128),      # token groups next to one another
    (1501, 33, 9, 128, 128),
    (6401, 33, 9, 128, 128),      # more than 64 MiB of rows: head groups
    (4003, 13, 5, 80, 20),        # a part whose half is no vector; 60 elements behind it
    (2503, 30, 11, 144, 132),     # a part that ends inside a vector
    (3001, 14, 2, 96, 48),
]


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", DT, ids=str)
@pytest.mark.parametrize("shape", ROWS, ids=str)
def test_long_calls(pkv, shape, dtype, interleaved, backward):
    T, hq, hk, D, rd = shape
    freqs, m = ref.frequencies(rd, scaling="yarn", factor=4.0, original=2048.0)
    rope = pkv.Rope(rd, scaling="yarn", factor=4.0, original_positions=2048,
                    interleaved=interleaved)
    x = _x((T, hq + hk, D), dtype, T + rd)                  # q and k side by side
    q, k = x.split([hq, hk], 1)
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 37 % 100003
    pos[5::11] = -1
    out, ko = (torch.full_like(t.contiguous(), 7.0) for t in (q, k))
    pkv.rope_apply(out, q, pos, rope, k_out=ko, k=k, backward=backward)
    few, few_k = (torch.full_like(t.contiguous(), 7.0) for t in (q, k))
    for t in range(0, T, 50):
        at = slice(t, min(t + 50, T))
        pkv.rope_apply(few[at], q[at], pos[at], rope, k_out=few_k[at], k=k[at], backward=backward)
    assert torch.equal(out, few) and torch.equal(ko, few_k)
    assert bool((out[5::11] == 7.0).all()) and bool((ko[5::11] == 7.0).all())
    rows = torch.tensor([r for r in [*range(0, T, 997), T - 1] if r % 11 != 5])
    ref.check_rotated(out[rows], q[rows], pos[rows], freqs, m, rd, interleaved, backward)
    ref.check_rotated(ko[rows], k[rows], pos[rows], freqs, m, rd, interleaved, backward)
    # in place, through the views
    pkv.rope_apply(q, q, pos, rope, k_out=k, k=k, backward=backward)
    live = pos >= 0
    assert torch.equal(q[live], out[live]) and torch.equal(k[live], ko[live])


APPENDS = [  # (cached, new) per sequence, q heads, kv heads, head_dim, rotary_dim, block size
    dict(lens=[0, 777, 30], new=[1100, 501, 400], hq=15, hk=5, D=96, rd=96, bs=16),
    dict(lens=[5, 0], new=[1203, 800], hq=36, hk=6, D=128, rd=128, bs=64),
    dict(lens=[100], new=[2001], hq=21, hk=3, D=112, rd=36, bs=5),
    dict(lens=[5, 0], new=[3203, 2600], hq=36, hk=6, D=128, rd=128, bs=64),   # head groups
]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("kv,dt,scaled", [("bf16", "bf16", False), ("f16", "f16", False),
                                          ("f32", "f32", False), ("e4m3", "bf16", False),
                                          ("e4m3", "f16", True), ("e4m3", "f32", True)])
@pytest.mark.parametrize("i", range(len(APPENDS)))
def test_long_appends(pkv, i, kv, dt, scaled, interleaved):
    c = dict(APPENDS[i])
    rd = c.pop("rd")
    s = Step(pkv, kv=kv, dt=dt, layers=2, seed=60 + i, **c)
    s.pos[7::13] = -1
    freqs, m = ref.frequencies(rd)
    rope = pkv.Rope(rd, interleaved=interleaved)
    other = pkv.KVPool(s.geom, storage=s.before.clone())
    scales = None
    if scaled:
        g = torch.Generator().manual_seed(3)
        scales = (torch.rand(s.nb, 2, 2, c["hk"], generator=g) * 0.02 + 0.004).cuda()
        s.pool.set_block_scales(scales)
        other.set_block_scales(scales)
    how = dict(k_scale=0.0131, v_scale=0.0097)
    s.pool.append_rope(1, s.q_out, s.q, s.k, s.v, rope, s.tables, s.pos, seq_ids=s.seq, **how)
    few = torch.full_like(s.q_out, 7.0)
    for t in range(0, s.T, 50):
        at = slice(t, min(t + 50, s.T))
        other.append_rope(1, few[at], s.q[at], s.k[at], s.v[at], rope, s.tables, s.pos[at],
                          seq_ids=s.seq[at], **how)
    assert s.pool.check_status() == 0 and other.check_status() == 0
    assert torch.equal(few, s.q_out)
    assert torch.equal(other.storage, s.pool.storage)
    # a sample against the reference, as a step of those tokens alone
    rows = torch.tensor([r for r in range(0, s.T, 151) if r % 13 != 7])
    whole = s.pool.view().clone()
    for name in ("q", "k", "v", "q_out", "seq", "pos"):
        setattr(s, name, getattr(s, name)[rows])
    s.T = len(rows)
    s.pool.storage.copy_(s.before)
    for t in range(s.T):
        blk, off = s.slots(t)
        s.pool.view()[blk, :, 1, :, off] = whole[blk, :, 1, :, off]
    s.check(1, freqs, m, rd, interleaved, 0.0131, 0.0097, scales=scales)
