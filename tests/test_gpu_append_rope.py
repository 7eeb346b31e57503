"""Append with rotation on the GPU (kv_append_rope): rotated keys in their slots,
values as kv_append stores them, rotated queries, in every pool type, against the
64-bit reference; padding, bad ids, block scales, layers, streams and graphs."""
import numpy as np
import pytest
import torch

import oracle
from tests import rotary_reference as ref
from tests.helpers import np_raw

pytestmark = pytest.mark.gpu
IN = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_215_gb300 import pkv as mod
    return mod


def _x(shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


class Step:
    """Tokens for `lens` cached tokens and `new` new ones per sequence."""

    def __init__(self, pkv, lens, new, hq=4, hk=2, D=64, bs=16, kv="bf16", dt="bf16", layers=1,
                 seed=0, joint=True):
        self.kv, self.dt, self.bs, self.D, self.layers = kv, IN[dt], bs, D, layers
        g = torch.Generator().manual_seed(seed + 100)
        need = [-(-(n + k) // bs) for n, k in zip(lens, new)]
        self.nb = sum(need) + 3
        ids = torch.randperm(self.nb, generator=g).tolist()
        width = max(max(need), 1)
        tab = torch.full((len(lens), width), -1, dtype=torch.int32)
        for s, c in enumerate(need):
            for j in range(c):
                tab[s, j] = ids.pop()
        self.tables = tab.cuda()
        self.seq = torch.tensor([s for s, k in enumerate(new) for _ in range(k)],
                                dtype=torch.int32).cuda()
        self.pos = torch.tensor([n + i for n, k in zip(lens, new) for i in range(k)],
                                dtype=torch.int32).cuda()
        T = self.T = int(self.pos.numel())
        if joint:
            x = _x((T, (hq + 2 * hk) * D), self.dt, seed)
            q, k, v = x.split([hq * D, hk * D, hk * D], 1)
            self.q, self.k, self.v = (t.view(T, -1, D) for t in (q, k, v))
        else:
            self.q, self.k, self.v = (_x((T, h, D), self.dt, seed + i)
                                      for i, h in enumerate((hq, hk, hk)))
        self.q_out = torch.full((T, hq, D), 7.0, dtype=self.dt, device="cuda")
        self.geom = pkv.geometry(layers, hq, hk, D, bs, self.nb, kv)
        nbytes = pkv.kv_pool_bytes(self.geom)
        self.before = torch.randint(0, 120, (nbytes,), generator=g, dtype=torch.uint8).cuda()
        self.pool = pkv.KVPool(self.geom, storage=self.before.clone())

    def slots(self, t):
        return int(self.tables[int(self.seq[t]), int(self.pos[t]) // self.bs]), \
            int(self.pos[t]) % self.bs

    def check(self, layer, freqs, m, rd, inter, ks=1.0, vs=1.0, scales=None, tokens=None,
              q=True):
        """q_out, the tokens' slots, and every other byte of the pool."""
        tokens = list(range(self.T)) if tokens is None else tokens
        if q:
            ref.check_rotated(self.q_out[tokens], self.q[tokens], self.pos[tokens], freqs, m, rd,
                              inter)
        want = self.before.clone().view(self.pool.view().dtype).view(self.pool.view().shape)
        got = self.pool.view()
        kref, size = ref.rotate(self.k, self.pos, freqs, m, rd, inter)
        if self.kv == "e4m3":
            err = ref.compute_bound(size, m, self.dt, self.pos)
        for t in tokens:
            blk, off = self.slots(t)
            k_got, v_got = got[blk, 0, layer, :, off], got[blk, 1, layer, :, off]
            if self.kv == "e4m3":
                hk = self.k.shape[1]
                sk = np.full((hk, 1), ks, np.float32) if scales is None else \
                    scales[blk, 0, layer].cpu().numpy()[:, None]
                sv = np.full((hk, 1), vs, np.float32) if scales is None else \
                    scales[blk, 1, layer].cpu().numpy()[:, None]
                for h in range(hk):
                    codes = k_got[h].cpu().numpy()
                    # encoding is monotone: the code lies between those of the value's bounds
                    e = np.where(np.arange(self.D) < rd, err[t, h], 0.0)
                    lo = oracle.e4m3_encode(np.float32(kref[t, h] - e - 1e-30), float(sk[h, 0]))
                    hi = oracle.e4m3_encode(np.float32(kref[t, h] + e + 1e-30), float(sk[h, 0]))
                    d = oracle.e4m3_decode
                    assert np.all((d(lo) <= d(codes)) & (d(codes) <= d(hi)))
                    vw = oracle.e4m3_encode(self.v[t, h].float().cpu().numpy(), float(sv[h, 0]))
                    assert np.array_equal(v_got[h].cpu().numpy(), vw)
            else:
                assert torch.equal(v_got, self.v[t])
                lim = ref.bound(kref[t:t + 1], size[t:t + 1], m, self.dt, self.pos[t:t + 1])[0]
                e = np.abs(k_got.double().cpu().numpy() - kref[t])
                assert np.all(e[:, :rd] <= lim[:, :rd])
                assert torch.equal(k_got[:, rd:], self.k[t][:, rd:])
            want[blk, 0, layer, :, off], want[blk, 1, layer, :, off] = k_got, v_got
        assert torch.equal(want.view(torch.uint8), got.view(torch.uint8)), "another slot changed"


CASES = [
    dict(lens=[2000], new=[1], hq=64, hk=8, D=128),
    dict(lens=[0], new=[1], hq=1, hk=1, D=8),
    dict(lens=[15, 16, 17, 0, 31], new=[1, 1, 1, 1, 1]),
    dict(lens=[7, 0, 30], new=[40, 1, 19], hq=7, hk=1, D=80, bs=5),
    dict(lens=[3, 500], new=[4, 4], hq=8, hk=8, D=256, bs=64),
    dict(lens=[100, 0], new=[300, 211], hq=16, hk=2, D=96, bs=256),
]


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("kv,dt", [("bf16", "bf16"), ("f16", "f16"), ("f32", "f32"),
                                   ("e4m3", "bf16"), ("e4m3", "f16"), ("e4m3", "f32")])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_append_rope(pkv, i, kv, dt, inter):
    c = dict(CASES[i])
    if kv == "e4m3" and c.get("D", 64) % 16:
        c["D"] = 16
    s = Step(pkv, kv=kv, dt=dt, seed=i, **c)
    for rd in sorted({s.D, max(2, s.D // 4 // 2 * 2)}):
        s.pool.storage.copy_(s.before)
        freqs, m = ref.frequencies(rd, scaling="yarn", factor=2.0, original=1024.0)
        rope = pkv.Rope(rd, scaling="yarn", factor=2.0, original_positions=1024,
                        interleaved=inter)
        s.pool.append_rope(0, s.q_out, s.q, s.k, s.v, rope, s.tables, s.pos, seq_ids=s.seq,
                           k_scale=0.0131, v_scale=0.0097)
        assert s.pool.check_status() == 0
        s.check(0, freqs, m, rd, inter, 0.0131, 0.0097)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_layers_keys_only_and_default_sequence_ids(pkv, kv):
    s = Step(pkv, [5, 0, 33], [1, 1, 1], kv=kv, layers=3, seed=40, joint=False)
    freqs, m = ref.frequencies(64)
    s.pool.append_rope(1, None, None, s.k, s.v, pkv.Rope(64), s.tables, s.pos, k_scale=0.01,
                       v_scale=0.02)
    assert s.pool.check_status() == 0
    s.check(1, freqs, m, 64, False, 0.01, 0.02, q=False)
    assert bool((s.q_out == 7.0).all())


def test_rotated_once_equals_rope_then_append(pkv):
    """bf16: the fused call stores what rope_apply and append_tokens store."""
    s = Step(pkv, [9, 100], [30, 21], hq=8, hk=4, D=128, seed=41)
    rope = pkv.Rope(128)
    s.pool.append_rope(0, s.q_out, s.q, s.k, s.v, rope, s.tables, s.pos, seq_ids=s.seq)
    other = pkv.KVPool(s.geom, storage=s.before.clone())
    k, q = torch.empty(s.T, 4, 128, dtype=s.dt, device="cuda"), torch.empty_like(s.q_out)
    pkv.rope_apply(q, s.q, s.pos, rope, k_out=k, k=s.k)
    other.append_tokens(0, k, s.v.contiguous(), s.tables, s.seq, s.pos)
    assert torch.equal(q, s.q_out) and torch.equal(other.storage, s.pool.storage)


@pytest.mark.parametrize("kv,dt", [("bf16", "bf16"), ("f32", "f32"), ("e4m3", "f16")])
@pytest.mark.parametrize("inter", [False, True])
def test_odd_bases_and_strides(pkv, kv, dt, inter):
    """k one element off, v with an odd token stride, q as [heads, tokens] in memory."""
    s = Step(pkv, [13, 60], [7, 4], hq=4, hk=2, D=48, kv=kv, dt=dt, seed=50, joint=False)
    s.k = _x((s.T * 2 * 48 + 1,), s.dt, 51)[1:].view(s.T, 2, 48)
    s.v = _x((s.T, 2 * 48 + 1), s.dt, 52)[:, :96].unflatten(1, (2, 48))
    s.q = _x((4, s.T, 48), s.dt, 53).transpose(0, 1)
    for rd in (48, 20):
        s.pool.storage.copy_(s.before)
        freqs, m = ref.frequencies(rd)
        s.pool.append_rope(0, s.q_out, s.q, s.k, s.v, pkv.Rope(rd, interleaved=inter), s.tables,
                           s.pos, seq_ids=s.seq, k_scale=0.01, v_scale=0.02)
        assert s.pool.check_status() == 0
        s.check(0, freqs, m, rd, inter, 0.01, 0.02)


def test_two_streams_at_once(pkv):
    a = Step(pkv, [100, 3], [900, 800], hq=16, hk=4, D=128, seed=54)
    b = Step(pkv, [7], [1500], hq=16, hk=4, D=128, kv="e4m3", seed=55)
    rope = pkv.Rope(128)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, st in zip((a, b), streams):
            s.pool.append_rope(0, s.q_out, s.q, s.k, s.v, rope, s.tables, s.pos, seq_ids=s.seq,
                               k_scale=0.01, v_scale=0.01, stream=st)
    torch.cuda.synchronize()
    freqs, m = ref.frequencies(128)
    for s in (a, b):
        assert s.pool.check_status() == 0
        other = pkv.KVPool(s.geom, storage=s.before.clone())
        q = torch.empty_like(s.q_out)
        other.append_rope(0, q, s.q, s.k, s.v, rope, s.tables, s.pos, seq_ids=s.seq,
                          k_scale=0.01, v_scale=0.01)
        assert torch.equal(q, s.q_out) and torch.equal(other.storage, s.pool.storage)
        ref.check_rotated(s.q_out[::113], s.q[::113], s.pos[::113], freqs, m, 128, False)


def test_in_place_queries(pkv):
    s = Step(pkv, [50], [20], seed=42)
    q0 = s.q.clone()
    freqs, m = ref.frequencies(32)
    s.pool.append_rope(0, s.q, s.q, s.k, s.v, pkv.Rope(32), s.tables, s.pos, seq_ids=s.seq)
    s.q_out, s.q = s.q, q0
    s.check(0, freqs, m, 32, False)


def test_padding_and_bad_ids(pkv):
    s = Step(pkv, [20, 3, 40, 8, 9, 1], [1] * 6, seed=43)
    freqs, m = ref.frequencies(64)
    rope = pkv.Rope(64)
    s.pos[1] = -1                                            # padding
    s.pool.append_rope(0, s.q_out, s.q, s.k, s.v, rope, s.tables, s.pos, seq_ids=s.seq)
    assert s.pool.check_status() == 0
    assert bool((s.q_out[1] == 7.0).all())
    s.check(0, freqs, m, 64, False, tokens=[0, 2, 3, 4, 5])
    # a sequence id, a position past the table, and block ids out of range: no store,
    # the error is recorded, the query still turns
    for bad in ("seq", "seq_negative", "position", "block", "block_negative"):
        s = Step(pkv, [20, 3, 40, 8, 9, 1], [1] * 6, seed=44)
        if bad == "seq":
            s.seq[2] = 6
        elif bad == "seq_negative":
            s.seq[2] = -1
        elif bad == "position":
            s.pos[2] = s.tables.shape[1] * s.bs
        else:
            s.tables[2, 2] = s.nb if bad == "block" else -5
        s.pool.append_rope(0, s.q_out, s.q, s.k, s.v, rope, s.tables, s.pos, seq_ids=s.seq)
        assert s.pool.check_status() == pkv.PKV_EBOUNDS, bad
        ref.check_rotated(s.q_out, s.q, s.pos, freqs, m, 64, False)
        s.check(0, freqs, m, 64, False, tokens=[0, 1, 3, 4, 5], q=False)


def test_attached_block_scales(pkv):
    s = Step(pkv, [10, 40], [9, 30], hq=8, hk=2, D=64, kv="e4m3", layers=2, seed=45)
    scales = (torch.rand(s.nb, 2, 2, 2, generator=torch.Generator().manual_seed(1)) * 0.02 +
              0.004).cuda()
    s.pool.set_block_scales(scales)
    freqs, m = ref.frequencies(64)
    s.pool.append_rope(1, s.q_out, s.q, s.k, s.v, pkv.Rope(64, interleaved=True), s.tables, s.pos,
                       seq_ids=s.seq, k_scale=-1.0)          # ignored while scales are attached
    assert s.pool.check_status() == 0
    s.check(1, freqs, m, 64, True, scales=scales)


def test_e4m3_saturation_and_non_finite_values(pkv):
    s = Step(pkv, [0], [2], hq=2, hk=1, D=16, kv="e4m3", seed=46, joint=False)
    s.k[0, 0], s.v[0, 0] = 1e4, -1e4
    s.v[1, 0, 0], s.v[1, 0, 1], s.v[1, 0, 2] = float("nan"), float("inf"), float("-inf")
    s.pool.append_rope(0, s.q_out, s.q, s.k, s.v, pkv.Rope(16), s.tables, s.pos, seq_ids=s.seq)
    blk, off = s.slots(0)
    got = s.pool.view()
    assert bool((got[blk, 0, 0, 0, off] == 0x7E).all())      # position 0: 10000 -> 448
    assert bool((got[blk, 1, 0, 0, off] == 0xFE).all())
    assert got[blk, 1, 0, 0, off + 1, :3].tolist() == [0x7F, 0x7E, 0xFE]


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_e4m3_codes_equal_those_of_append(pkv, dt):
    """Every 16-bit value (and fp32 values around the boundaries between codes) under
    scales that put them anywhere: the same bytes as append_tokens stores, values in
    any position, keys at position 0 (angle 0)."""
    hk, D, bs = 4, 128, 16
    if dt == "f32":
        # quotients within a few steps of the midpoint between two codes, times the scale
        codes = np.arange(0x08, 0x7E, dtype=np.uint8)
        mid = (oracle.e4m3_decode(codes) + oracle.e4m3_decode(codes + 1)) / 2
        u = mid.astype(np.float32).view(np.uint32).astype(np.int64)[:, None] + np.arange(-24, 25)
        base = torch.from_numpy(u.astype(np.uint32).view(np.float32).reshape(-1).copy())
    else:
        base = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(IN[dt])
    for scale in (1.0, 1.0 / 448, 0.0123456, 3.7e-5, 55.5, 2.0 ** -130, 2.0 ** 110):
        x = base if dt != "f32" else (base.double() * scale).float()
        T = -(-x.numel() // (hk * D))
        v = torch.zeros(T * hk * D, dtype=x.dtype)
        v[:x.numel()] = x
        v = v.view(T, hk, D).cuda()
        k = torch.where(torch.isfinite(v), v, torch.zeros_like(v))
        geom = pkv.geometry(1, hk, hk, D, bs, T, "e4m3")
        a, b = (pkv.KVPool(geom, storage=torch.zeros(pkv.kv_pool_bytes(geom), dtype=torch.uint8,
                                                     device="cuda")) for _ in range(2))
        # every token at position 0 of a sequence of its own
        tab = torch.arange(T, dtype=torch.int32, device="cuda").view(T, 1)
        pos = torch.zeros(T, dtype=torch.int32, device="cuda")
        seq = torch.arange(T, dtype=torch.int32, device="cuda")
        a.append_tokens(0, k, v, tab, seq, pos, scale, scale)
        b.append_rope(0, None, None, k, v, pkv.Rope(D), tab, pos, k_scale=scale, v_scale=scale)
        got, want = b.view(), a.view()
        assert torch.equal(got[:, 1], want[:, 1]), scale
        # x * 1 - y * 0: a zero's sign may differ
        zero = (got[:, 0] & 0x7F) == 0
        assert torch.equal(got[:, 0][~zero], want[:, 0][~zero])
        assert bool(((want[:, 0] & 0x7F) == 0)[zero].all())


def test_many_tokens_in_a_long_pool(pkv):
    """More than 2^31 elements between a pool's ends: 64-bit slot offsets."""
    nb, hk, D, bs = 20000, 8, 128, 64                        # 2.6e9 elements of one byte
    geom = pkv.geometry(1, 8, hk, D, bs, nb, "e4m3")
    pool = pkv.KVPool(geom, storage=torch.zeros(pkv.kv_pool_bytes(geom), dtype=torch.uint8,
                                                device="cuda"))
    assert pool.nbytes > 2 ** 31
    tables = torch.tensor([[nb - 1, 0]], dtype=torch.int32, device="cuda")
    pos = torch.tensor([63, 64], dtype=torch.int32, device="cuda")
    seq = torch.zeros(2, dtype=torch.int32, device="cuda")
    k = torch.ones(2, hk, D, dtype=torch.bfloat16, device="cuda")
    pool.append_rope(0, None, None, k, k, pkv.Rope(D), tables, pos, seq_ids=seq)
    assert pool.check_status() == 0
    view = pool.view()
    one = 0x38
    assert bool((view[nb - 1, 1, 0, :, 63] == one).all())
    assert bool((view[0, 1, 0, :, 0] == one).all())
    assert int((view[nb - 1] != 0).sum()) <= 2 * hk * D and int((view[1:nb - 1] != 0).sum()) == 0
    pool.close()


def test_another_stream_and_graph_replay(pkv):
    s = Step(pkv, [20, 3], [1, 1], seed=47)
    rope = pkv.Rope(64)
    freqs, m = ref.frequencies(64)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    s.pool.append_rope(0, s.q_out, s.q, s.k, s.v, rope, s.tables, s.pos, seq_ids=s.seq,
                       stream=side)
    side.synchronize()
    s.check(0, freqs, m, 64, False)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.pool.append_rope(0, s.q_out, s.q, s.k, s.v, rope, s.tables, s.pos, seq_ids=s.seq)
    for step in (1, 2):
        s.pos += 1                                           # the next token of each sequence
        s.pool.storage.copy_(s.before)
        graph.replay()
        torch.cuda.synchronize()
        assert s.pool.check_status() == 0
        s.check(0, freqs, m, 64, False)


def test_binding_refusals(pkv):
    s = Step(pkv, [20, 3], [1, 1], seed=48, joint=False)
    rope = pkv.Rope(64)
    good = dict(layer=0, q_out=s.q_out, q=s.q, k=s.k, v=s.v, rope=rope, tables=s.tables,
                positions=s.pos, seq_ids=s.seq)
    s.pool.append_rope(**good)
    for bad in (dict(q=None), dict(k=s.k[:1]), dict(v=s.v[:, :1]), dict(v=s.v.float()),
                dict(tables=s.tables.long()), dict(tables=s.tables[0]),
                dict(positions=s.pos.long()), dict(seq_ids=s.seq[:1]),
                dict(tables=s.tables[:1], seq_ids=None), dict(k=s.k.cpu()),
                dict(q=s.q.transpose(1, 2))):
        with pytest.raises(ValueError):
            s.pool.append_rope(**dict(good, **bad))
    for bad in (dict(layer=1), dict(rope=pkv.Rope(128))):
        with pytest.raises(pkv.PkvError):
            s.pool.append_rope(**dict(good, **bad))
