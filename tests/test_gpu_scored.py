"""Decode attention under score rules, and the record of its weights, against the 64-bit
reference."""
import pytest
import torch

from tests.scored_reference import Case, slopes

pytestmark = pytest.mark.gpu


def run(case, out_dtype=None, weights=None, weights_in=None, scale=None, max_len=None, **rules):
    from paged_kv_cache_215_gb300 import pkv
    pool = case.handle()
    out = torch.full(case.q.shape, float("nan"), dtype=out_dtype or case.q.dtype, device="cuda")
    t = {}
    if rules.get("slopes") is not None:
        t["slopes"] = rules["slopes"].float().cuda()
    if rules.get("prefix") is not None:
        t["prefix_lens"] = torch.tensor(rules["prefix"], dtype=torch.int32, device="cuda")
    if rules.get("docs") is not None:
        t["doc_starts"] = torch.tensor(rules["docs"], dtype=torch.int32, device="cuda")
    sc = pkv.Scores(cap=rules.get("cap", 0.0), window=rules.get("window", 0), **t)
    pkv.paged_decode_attention_scored(
        out, case.q, pool, case.layer, case.tables, case.seq_lens,
        max(case.lens) if max_len is None else max_len,
        case.scale if scale is None else scale, scores=sc, k_scale=case.k_scale,
        v_scale=case.v_scale, weights=weights, weights_in=weights_in)
    torch.cuda.synchronize()
    assert pool.check_status() == 0
    return out


RULES = {
    "none": {},
    "cap": dict(cap=20.0),
    "small-cap": dict(cap=1.5),
    "window": dict(window=37),
    "window-1": dict(window=1),
    "slopes": dict(slopes=True),
    "all": dict(cap=10.0, window=100, slopes=True, prefix=True, docs=True),
}


def expand(case, rules):
    r = dict(rules)
    if r.get("slopes"):
        r["slopes"] = slopes(case.hq)
    if r.get("prefix"):
        r["prefix"] = [(n * 2) // 3 for n in case.lens]
    if r.get("docs"):
        r["docs"] = [[max(0, n - case.q_len + i) // 3 for i in range(case.q_len)]
                     for n in case.lens]
    return r


@pytest.mark.parametrize("rules", RULES)
@pytest.mark.parametrize("kv,hq,hkv,dim,bs,q_len", [
    ("bf16", 8, 2, 128, 16, 1), ("bf16", 8, 2, 128, 16, 4), ("f16", 4, 4, 128, 32, 1),
    ("f16", 14, 2, 128, 32, 2), ("e4m3", 8, 1, 128, 16, 1), ("e4m3", 8, 2, 128, 64, 2),
    ("bf16", 7, 1, 128, 64, 1), ("bf16", 16, 1, 128, 16, 1), ("f32", 4, 2, 64, 16, 1),
    ("bf16", 12, 4, 96, 16, 1), ("e4m3", 4, 2, 64, 32, 1), ("f16", 5, 1, 256, 8, 1),
    ("f16", 3, 1, 40, 16, 1), ("e4m3", 2, 2, 16, 1, 1), ("f32", 16, 1, 8, 4, 1),
    ("f32", 32, 2, 256, 16, 1), ("bf16", 16, 1, 128, 64, 1), ("f16", 32, 2, 128, 64, 1),
    ("e4m3", 10, 2, 128, 64, 3)])
def test_decode(kv, hq, hkv, dim, bs, q_len, rules):
    lens = [300, 1, bs, bs + 1, 0, 2 * bs - 1, 77]
    case = Case(lens, hq, hkv, dim, kv, bs, q_len, seed=hq + dim + q_len)
    r = expand(case, RULES[rules])
    want = case.reference(**r)
    before = torch.rand(len(lens), hkv, 301).cuda()
    weights = torch.full((len(lens), hkv, 333), -5.0).cuda()
    out = run(case, torch.float32, weights, before, **r)
    case.check(out, want, weights, before)
    for b, n in enumerate(lens):                           # columns behind the sequence
        assert (weights[b, :, n:] == -5.0).all()
    plain = run(case, **r)                                 # without the record, its own type
    case.check(plain, want)


@pytest.mark.parametrize("scaled", [False, True])
def test_e4m3_block_scales(scaled):
    case = Case([130, 64, 3], 8, 2, 128, "e4m3", 16, 2, seed=3, block_scales=scaled)
    r = expand(case, RULES["all"])
    weights = torch.zeros(3, 2, 130, device="cuda")
    out = run(case, torch.float32, weights, **r)
    case.check(out, case.reference(**r), weights)


@pytest.mark.parametrize("scale", [-0.3, 0.0, 3.0])
@pytest.mark.parametrize("kv", ["bf16", "f32"])
def test_scale_sign_and_size(kv, scale):
    case = Case([90, 17], 8, 2, 128 if kv == "bf16" else 64, kv, 16, seed=4, q_gain=1.0)
    for r in ({}, {"cap": 30.0}):
        out = run(case, torch.float32, scale=scale, **r)
        case.check(out, case.reference(scale=scale, **r))


@pytest.mark.parametrize("kv,dim", [("bf16", 128), ("e4m3", 128), ("f32", 64)])
def test_unseen_keys_hold_anything(kv, dim):
    # what lies ahead of the window or the document, and stale table entries there
    lens = [200, 33, 129]
    case = Case(lens, 8, 2, dim, kv, 16, seed=5)
    want = case.reference(window=40)
    for b, n in enumerate(lens):
        case.hide(b, 0, max(0, n - 40))
        case.tables[b, :max(0, n - 40) // 16] = -1
    w = torch.zeros(3, 2, 200, device="cuda")
    case.check(run(case, torch.float32, w, window=40), want, w)
    docs = [[n - 7] for n in lens]
    want = case.reference(docs=docs)
    for b, n in enumerate(lens):
        case.hide(b, 0, n - 7)
        case.tables[b, :(n - 7) // 16] = -1
    case.check(run(case, torch.float32, docs=docs), want)


def test_rows_that_see_nothing():
    lens = [50, 20, 3]
    for q_len in (1, 4):
        case = Case(lens, 8, 2, 128, "bf16", 16, q_len, seed=6)
        # a document that starts behind its query: sequence 0 throughout, 1 in part
        docs = [[n for _ in range(q_len)] for n in lens]
        docs[1] = [20 - q_len + i if i % 2 == 0 else 2 ** 31 - 1 for i in range(q_len)]
        docs[2] = [-3] * q_len
        w = torch.zeros(3, 2, 50, device="cuda")
        case.check(run(case, torch.float32, w, docs=docs), case.reference(docs=docs), w)


def test_more_queries_than_tokens():
    case = Case([2, 0, 1, 30], 4, 2, 128, "f16", 16, 5, seed=7)
    r = dict(cap=5.0, prefix=[2, 0, 1, 28], window=9)
    w = torch.zeros(4, 2, 30, device="cuda")
    case.check(run(case, torch.float32, w, **r), case.reference(**r), w)


def test_weights_accumulate_in_place_in_strided_rows_and_repeat():
    case = Case([100, 40], 8, 4, 128, "bf16", 16, seed=8)
    store = torch.zeros(4, 2, 256, device="cuda")
    rows = store.transpose(0, 1)[:, :, 16:]                # [2, 4, 240]
    for turn in range(3):
        run(case, weights=rows, weights_in=rows if turn else None)
    want = case.reference()
    for b, (_, _, w, err) in enumerate(want):
        n = case.lens[b]
        got = rows[b, :, :n].double().cpu()
        assert ((got - 3 * w).abs() <= 3 * err + 2.0 ** -21 * w + 1e-30).all()
    assert (store[:, :, :16] == 0).all() and (rows[0, :, 100:] == 0).all()
    once = torch.zeros(2, 4, 100, device="cuda")
    again = torch.zeros_like(once)
    run(case, weights=once)
    run(case, weights=again)
    assert torch.equal(once, again)


def test_layer_of_a_deeper_pool():
    case = Case([70, 5], 8, 2, 128, "bf16", 16, seed=9, layers=3, layer=1)
    w = torch.zeros(2, 2, 70, device="cuda")
    case.check(run(case, torch.float32, w, cap=9.0), case.reference(cap=9.0), w)


def test_long_sequence():
    case = Case([20001], 8, 2, 128, "bf16", 16, seed=10)
    r = dict(cap=20.0, slopes=slopes(8))
    w = torch.zeros(1, 2, 20001, device="cuda")
    case.check(run(case, torch.float32, w, **r), case.reference(**r), w)


def test_lengths_beyond_the_limit_are_recorded():
    from paged_kv_cache_215_gb300 import pkv
    case = Case([64, 40], 8, 2, 128, "bf16", 16, seed=11)
    want = case.reference()
    pool = case.handle()
    lens = torch.tensor([70, -4], dtype=torch.int32, device="cuda")
    out = torch.zeros(2, 8, 128, device="cuda")
    w = torch.zeros(2, 2, 64, device="cuda")
    pkv.paged_decode_attention_scored(out, case.q[:, 0].contiguous(), pool, 0, case.tables, lens,
                                      64, case.scale, weights=w)
    assert pool.check_status() == pkv.PKV_EBOUNDS
    o, bound, ww, err = want[0]                              # 70 is taken as 64
    assert ((out[0].double().cpu() - o[0]).abs() <= bound[0] + 2.0 ** -22 * o[0].abs()).all()
    assert (out[1] == 0).all() and (w[1] == 0).all()


def test_refusals():
    from paged_kv_cache_215_gb300 import pkv
    case = Case([40, 20], 8, 2, 128, "bf16", 16, seed=12)
    pool = case.handle()
    out = torch.zeros(2, 8, 128, dtype=torch.bfloat16, device="cuda")
    q = case.q[:, 0].contiguous()

    def call(o=out, qq=q, n=40, sc=None, **kw):
        pkv.paged_decode_attention_scored(o, qq, pool, 0, kw.pop("tables", case.tables),
                                          kw.pop("lens", case.seq_lens), n,
                                          kw.pop("scale", 0.1), scores=sc, **kw)
    call()
    f = lambda *s: torch.zeros(*s, device="cuda")
    for sc in (pkv.Scores(cap=-1.0), pkv.Scores(window=-2), pkv.Scores(cap=float("inf")),
               pkv.Scores(cap=float("nan")), pkv.Scores(cap=1e-44)):
        with pytest.raises(pkv.PkvError) as e:
            call(sc=sc)
        assert e.value.code == pkv.PKV_EINVAL
    with pytest.raises(pkv.PkvError) as e:
        call(n=100)                                        # longer than the table
    assert e.value.code == pkv.PKV_EINVAL
    with pytest.raises(pkv.PkvError) as e:
        call(workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert e.value.code == pkv.PKV_ENOMEM
    with pytest.raises(pkv.PkvError) as e:                 # rows of weights on one another
        call(weights=f(2, 1, 64).expand(2, 2, 64))
    assert e.value.code == pkv.PKV_EINVAL
    with pytest.raises(pkv.PkvError) as e:                 # the input's rows in another order
        w = f(2, 2, 64)
        call(weights=w, weights_in=w.flatten()[:256].view(2, 2, 64).transpose(0, 1))
    assert e.value.code == pkv.PKV_EINVAL
    with pytest.raises(pkv.PkvError) as e:                 # an input alone
        call(weights_in=f(2, 2, 64))
    assert e.value.code == pkv.PKV_EINVAL
    for bad in (dict(weights=f(2, 2, 39)), dict(weights=f(2, 3, 64)),
                dict(weights=f(2, 2, 64).half()), dict(weights=f(2, 64, 2).transpose(1, 2)),
                dict(weights=torch.zeros(2, 2, 64)), dict(weights=f(2, 2, 64), weights_in=f(1, 2, 64)),
                dict(sc=pkv.Scores(slopes=f(7))), dict(sc=pkv.Scores(slopes=f(8).double())),
                dict(sc=pkv.Scores(prefix_lens=f(2))),
                dict(sc=pkv.Scores(doc_starts=f(2, 2).int())),
                dict(qq=q[:, ::2]), dict(qq=q[:1]), dict(o=out[:, :, ::2]), dict(o=out[:1]),
                dict(qq=q.double()), dict(lens=case.seq_lens.long()), dict(tables=case.tables[0]),
                dict(tables=case.tables[:1]), dict(qq=q.cpu()),
                dict(qq=q.clone().requires_grad_())):
        with pytest.raises(ValueError):
            call(**bad)
    big = Case([90], 8, 2, 128, "bf16", 16, 5, seed=13)    # 20 query rows: no record
    h = big.handle()
    with pytest.raises(pkv.PkvError) as e:
        pkv.paged_decode_attention_scored(torch.zeros_like(big.q), big.q, h, 0, big.tables,
                                          big.seq_lens, 90, 0.1, weights=f(1, 2, 90))
    assert e.value.code == pkv.PKV_EUNSUPPORTED
    h.close()
    with pytest.raises(ValueError):
        pkv.paged_decode_attention_scored(torch.zeros_like(big.q), big.q, h, 0, big.tables,
                                          big.seq_lens, 90, 0.1)
