"""Eviction by accumulated weight against a plain reading of its rule; every byte and
bit of the results is compared."""
import pytest
import torch

from tests.scored_reference import Case, evicted

pytestmark = pytest.mark.gpu


def weights_of(kind, batch, hkv, width, seed=0):
    g = torch.Generator().manual_seed(seed)
    if kind == "random":
        return torch.rand(batch, hkv, width, generator=g)
    if kind == "ties":                                     # a handful of values
        return torch.randint(0, 4, (batch, hkv, width), generator=g).float() * 0.25
    if kind == "equal":
        return torch.full((batch, hkv, width), 0.125)
    if kind == "zero":
        return torch.zeros(batch, hkv, width)
    if kind == "wide":                                     # every exponent, subnormals too
        return torch.exp2(torch.rand(batch, hkv, width, generator=g) * 270 - 148).float()
    w = torch.randn(batch, hkv, width, generator=g)        # odd: signs, NaN, infinities
    at = torch.rand(batch, hkv, width, generator=g)
    w[at < 0.1] = float("nan")
    w[at > 0.95] = float("inf")
    w[(at > 0.9) & (at < 0.95)] = -float("inf")
    w[(at > 0.5) & (at < 0.6)] = -0.0
    return w


def evict(case, w, keep, recent, new_width=None, want_index=True, capacity=None, fill=None):
    """Run into blocks that hold NaN; returns (pool handle, new tables, lens, index, weights)."""
    from paged_kv_cache_215_gb300 import pkv
    kept = [min(n, k) for n, k in zip(case.lens, keep)]
    bs, most = case.bs, max(max(kept), 1) if capacity is None else capacity
    per = -(-most // bs)
    extra = per * case.batch
    blank = torch.full((extra,) + case.pool.shape[1:], case.nan, dtype=case.pool.dtype,
                       device="cuda")
    case.pool = torch.cat([case.pool, blank])
    first, case.nb = case.nb, case.nb + extra
    fresh = (first + torch.randperm(extra, generator=torch.Generator().manual_seed(1))).view(
        case.batch, per).int().cuda()
    pool = case.handle()
    width = most if new_width is None else new_width
    new_w = torch.full((case.batch, case.hkv, width), -9.0, device="cuda")
    lens = torch.full((case.batch,), -9, dtype=torch.int32, device="cuda")
    index = torch.full((case.batch, case.hkv, most), -9, dtype=torch.int32, device="cuda") \
        if want_index else None
    pool.evict(case.layer, fresh, case.tables, case.seq_lens, max(case.lens),
               torch.tensor(keep, dtype=torch.int32, device="cuda"), recent, w, new_w, lens,
               index=index)
    torch.cuda.synchronize()
    return pool, fresh, lens, index, new_w


def check(case, before, w, keep, recent, result):
    pool, fresh, lens, index, new_w = result
    bs = case.bs
    assert lens.tolist() == [min(n, k) for n, k in zip(case.lens, keep)]
    want = case.pool.clone()
    want[:before.shape[0]] = before
    want[before.shape[0]:] = case.nan
    host = w.cpu()
    for b, n in enumerate(case.lens):
        k = min(n, keep[b])
        for h in range(case.hkv):
            j = torch.tensor(evicted(host[b, h], n, keep[b], recent), dtype=torch.long)
            t = torch.arange(k)
            if index is not None:
                assert index[b, h].tolist() == j.tolist() + [-9] * (index.shape[2] - k), (b, h)
            got = new_w[b, h].cpu()
            assert torch.equal(got[:k].view(torch.int32), host[b, h, j].view(torch.int32))
            assert (got[k:] == 0).all()
            src = case.tables[b].cpu().long()[j // bs].cuda()
            dst = fresh[b].cpu().long()[t // bs].cuda()
            want[dst, :, case.layer, h, (t % bs).cuda()] = \
                before[src, :, case.layer, h, (j % bs).cuda()]
    raw = lambda x: x.view(torch.uint8)
    assert torch.equal(raw(case.pool), raw(want))          # every other slot as it was
    assert pool.check_status() == 0


@pytest.mark.parametrize("kind", ["random", "ties", "equal", "zero", "wide", "odd"])
@pytest.mark.parametrize("kv,dim,bs,hkv", [("bf16", 128, 16, 2), ("f16", 64, 32, 3),
                                           ("e4m3", 16, 64, 1), ("f32", 8, 5, 2),
                                           ("e4m3", 256, 1, 4)])
def test_against_the_rule(kv, dim, bs, hkv, kind):
    lens, keep, recent = [100, 0, 1, 37, 64, 250], [40, 5, 1, 36, 64, 0], 17
    case = Case(lens, hkv, hkv, dim, kv, bs, seed=dim + bs)
    w = weights_of(kind, len(lens), hkv, 260).cuda()
    before = case.pool.clone()
    check(case, before, w, keep, recent, evict(case, w, keep, recent))


@pytest.mark.parametrize("recent", [0, 1, 39, 40, 41, 10 ** 9])
def test_recent(recent):
    case = Case([100, 39], 2, 2, 32, "bf16", 16, seed=1)
    w = weights_of("ties", 2, 2, 100).cuda()
    before = case.pool.clone()
    check(case, before, w, [40, 40], recent, evict(case, w, [40, 40], recent, want_index=False))


@pytest.mark.parametrize("n,keep,recent,kind", [
    (1023, 1, 0, "random"), (1024, 1023, 5, "ties"), (1025, 700, 100, "equal"),
    (5000, 1234, 77, "ties"), (70001, 4096, 512, "ties"), (70001, 65536, 0, "wide"),
    (200000, 100000, 1, "random")])
def test_long_rows(n, keep, recent, kind):
    case = Case([n], 2, 2, 16, "bf16", 64, seed=2, q_gain=1.0)
    w = weights_of(kind, 1, 2, n, seed=n).cuda()
    before = case.pool.clone()
    check(case, before, w, [keep], recent, evict(case, w, [keep], recent))


def test_strided_weights_wider_rows_and_a_layer():
    case = Case([90, 33, 60], 4, 4, 64, "bf16", 16, seed=3, layers=3, layer=2)
    store = weights_of("random", 4, 3, 120).cuda()
    w = store.transpose(0, 1)[:, :, 7:100]
    before = case.pool.clone()
    keep = [20, 20, 59]
    check(case, before, w, keep, 8, evict(case, w, keep, 8, new_width=77))


def test_what_does_not_fit_is_recorded():
    from paged_kv_cache_215_gb300 import pkv
    case = Case([60, 30], 2, 2, 32, "bf16", 16, seed=4)
    w = weights_of("random", 2, 2, 60).cuda()
    before = case.pool.clone()
    pool, fresh, lens, index, new_w = evict(case, w, [50, 20], 4, capacity=32, new_width=32)
    assert pool.check_status() == pkv.PKV_EBOUNDS and lens.tolist() == [32, 20]
    check(case, before, w, [32, 20], 4, (pool, fresh, lens, index, new_w))


def test_bad_blocks_lengths_and_budgets_are_recorded():
    from paged_kv_cache_215_gb300 import pkv
    case = Case([60, 30, 40], 2, 2, 32, "bf16", 16, seed=5)
    w = weights_of("random", 3, 2, 60).cuda()
    case.tables[0, 1] = 10 ** 6
    pool, fresh, lens, index, new_w = evict(case, w, [60, -3, 40], 4)
    assert pool.check_status() == pkv.PKV_EBOUNDS and lens.tolist() == [60, 0, 40]
    got = case.pool[fresh[0].long()][:, :, 0].cpu()
    assert got[1].isnan().all() and not got[0].isnan().any()
    case.seq_lens[:] = torch.tensor([-1, 10 ** 9, 3])
    pool.evict(0, fresh, case.tables, case.seq_lens, 60, torch.tensor([1, 1, 1]).int().cuda(), 0, w,
               new_w, lens)
    torch.cuda.synchronize()
    assert pool.check_status() == pkv.PKV_EBOUNDS and lens.tolist() == [0, 1, 1]


def test_refusals():
    from paged_kv_cache_215_gb300 import pkv
    case = Case([40, 20], 2, 2, 64, "e4m3", 16, seed=6, spare=8)
    pool = case.handle()
    f = lambda *s: torch.zeros(*s, device="cuda")
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    w = f(2, 2, 64)

    def call(**kw):
        a = dict(new_tables=i(2, 2), tables=case.tables, seq_lens=case.seq_lens, max_seq_len=40,
                 keep=i(2), recent=4, weights=w, new_weights=f(2, 2, 32), new_lens=i(2))
        a.update(kw)
        return pool.evict(0, **a)
    call()
    for bad in (dict(max_seq_len=-1), dict(max_seq_len=65, weights=f(2, 2, 80)), dict(recent=-1),
                dict(new_weights=w), dict(new_weights=f(1, 2, 32).expand(2, 2, 32))):
        with pytest.raises(pkv.PkvError) as e:
            call(**bad)
        assert e.value.code == pkv.PKV_EINVAL, bad
    with pytest.raises(pkv.PkvError) as e:
        call(workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.code == pkv.PKV_ENOMEM
    for bad in (dict(new_tables=i(3, 2)), dict(new_tables=i(2, 2).long()), dict(tables=i(2)),
                dict(seq_lens=i(3)), dict(keep=i(2, 1)), dict(keep=f(2)), dict(weights=f(2, 2, 39)),
                dict(weights=w.double()), dict(new_weights=f(2, 3, 32)), dict(new_lens=i(1)),
                dict(index=i(2, 2)), dict(index=f(2, 2, 40)), dict(index=i(2, 2, 40)[:, :, ::2]),
                dict(workspace=f(64)), dict(weights=w.cpu())):
        with pytest.raises(ValueError):
            call(**bad)
    pool.set_block_scales(torch.ones(case.nb, 2, 1, 2, device="cuda"))
    with pytest.raises(pkv.PkvError) as e:
        call()
    assert e.value.code == pkv.PKV_EUNSUPPORTED
