"""Draft verification on the GPU (verify_drafts) against the 64-bit reference:
accepted counts and tokens are whole numbers and must be equal."""
import pytest
import torch

from tests import rotary_reference as ref

pytestmark = pytest.mark.gpu
DT = [torch.float32, torch.float16, torch.bfloat16]


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_215_gb300 import pkv as mod
    return mod


def _case(B, K, V, dtype=torch.float32, seed=0, noise=0.5, sharp=2.0):
    g = torch.Generator().manual_seed(seed)
    logits = sharp * torch.randn(B, K + 1, V, generator=g)
    target = torch.softmax(logits, -1).to(dtype)
    q = torch.softmax(logits[:, :K] + noise * torch.randn(B, K, V, generator=g), -1).to(dtype)
    drafts = torch.multinomial(q.float().reshape(B * K, V).clamp(min=1e-9), 1,
                               generator=g).view(B, K).int() if K else \
        torch.zeros(B, 0, dtype=torch.int32)
    return [t.cuda() for t in (target, q, drafts, torch.rand(B, K, generator=g),
                               torch.rand(B, generator=g))]


def _run(pkv, target, draft, drafts, ua, us, num=None, status=None, **kw):
    B, K = drafts.shape
    tokens = torch.full((B, K + 1), 12345, dtype=torch.int32, device="cuda")
    acc = torch.full((B,), 12345, dtype=torch.int32, device="cuda")
    pkv.verify_drafts(tokens, acc, target, draft, drafts, ua, us, num_drafts=num, status=status,
                      **kw)
    torch.cuda.synchronize()
    return tokens, acc


def _check(pkv, target, draft, drafts, ua, us, num=None):
    tokens, acc = _run(pkv, target, draft, drafts, ua, us, num)
    want, n = ref.verify(target, draft, drafts, ua, us, None if num is None else num.tolist())
    assert acc.tolist() == n
    assert tokens.tolist() == want
    return n


@pytest.mark.parametrize("lookup", [False, True])
@pytest.mark.parametrize("dtype", DT, ids=str)
@pytest.mark.parametrize("B,K,V", [(1, 4, 131072), (3, 2, 100003), (1, 1, 1), (5, 3, 2),
                                   (7, 8, 33), (40, 5, 4099), (2, 3, 524289), (300, 1, 511),
                                   (16, 600, 64), (1, 7, 8192)])
def test_verify(pkv, B, K, V, dtype, lookup):
    t, q, x, ua, us = _case(B, K, V, dtype, seed=V)
    _check(pkv, t, None if lookup else q, x, ua, us)


@pytest.mark.parametrize("dtype", DT, ids=str)
def test_different_numbers_of_drafts(pkv, dtype):
    t, q, x, ua, us = _case(12, 6, 5003, dtype, seed=2)
    num = torch.tensor([0, 1, 2, 3, 4, 5, 6, 0, 6, 3, 1, 2], dtype=torch.int32, device="cuda")
    x[0] = x[7] = -77                                        # behind the last draft: never read
    t[0, 1:], q[0] = float("nan"), float("nan")
    n = _check(pkv, t, q, x, ua, us, num)
    assert n[0] == 0 and max(n) > 0


def test_no_drafts_is_sampling(pkv):
    t, q, x, ua, us = _case(9, 0, 3001, seed=3)
    assert _check(pkv, t, None, x, ua, us) == [0] * 9
    assert _check(pkv, t, q, x, ua, us) == [0] * 9


@pytest.mark.parametrize("lookup", [False, True])
def test_every_draft_accepted_or_refused(pkv, lookup):
    t, q, x, ua, us = _case(6, 4, 2048, seed=4, noise=0.0)
    d = None if lookup else q
    if not lookup:
        assert _check(pkv, t, d, x, torch.zeros_like(ua), us) == [4] * 6
    # u = 1: accepted only where p exceeds q; with p == q the residual has no mass, and
    # the token is drawn from the target
    n = _check(pkv, t, d, x, torch.ones_like(ua), us)
    assert n == [0] * 6


def test_random_numbers_at_their_ends(pkv):
    t, q, x, ua, us = _case(8, 3, 1000, seed=5)
    t[:, :, :7] = 0                                          # mass starts and ends inside the row
    t[:, :, 990:] = 0
    ends = torch.tensor([0.0, 1 - 2.0 ** -24, 1.0, 2.0 ** -149, float("nan"), -1.0, float("inf"),
                         0.5], device="cuda")
    for u in (0.0, 1 - 2.0 ** -24, float("nan")):
        _check(pkv, t, q, x, torch.full_like(ua, u), ends)
        _check(pkv, t, None, x, torch.full_like(ua, u), ends)


def test_zeros_nan_and_values_above_one(pkv):
    t, q, x, ua, us = _case(6, 3, 999, seed=6)
    t[0, :, ::2] = float("nan")
    t[1, :, 5:] = -0.25
    t[2, :, 100] = 7.0
    q[3] = float("nan")
    q[4, 0] = 0.0
    t[5, :, :] = 0.0
    t[5, :, 998] = 1e-3                                      # a row with one token
    _check(pkv, t, q, x, ua, us)


@pytest.mark.parametrize("V", [200, 100000])
def test_a_sum_above_16_saturates(pkv, V):
    t, q, x, ua, us = _case(7, 2, V, seed=20)
    t[:4] = 1.0
    t[4:6, :, V // 2] = 1.0
    _check(pkv, t, q, x, ua, us)
    _check(pkv, t, None, x, ua, us)


@pytest.mark.parametrize("V", [1000, 131072])
def test_rows_without_mass_give_no_token_and_report_it(pkv, V):
    t, q, x, ua, us = _case(3, 2, V, seed=7)
    t[1] = 0.0
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    tokens, acc = _run(pkv, t, q, x, ua, us, status=status)
    want, n = ref.verify(t, q, x, ua, us)
    assert tokens.tolist() == want and acc.tolist() == n
    assert tokens[1].tolist() == [-1, -1, -1] and int(acc[1]) == 0
    assert int(status) == pkv.PKV_EINVAL


def test_drafts_and_counts_out_of_range_are_refused_and_reported(pkv):
    for bad in (-1, 1000, 2 ** 31 - 1):
        t, q, x, ua, us = _case(4, 3, 1000, seed=8, noise=0.0)
        ua.zero_()
        x[2, 1] = bad
        for d in (q, None):
            status = torch.zeros(1, dtype=torch.int32, device="cuda")
            tokens, acc = _run(pkv, t, d, x, ua, us, status=status)
            want, n = ref.verify(t, d, x, ua, us)
            assert tokens.tolist() == want and acc.tolist() == n and n[2] == 1
            assert int(status) == pkv.PKV_EBOUNDS
    t, q, x, ua, us = _case(4, 3, 1000, seed=9)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    num = torch.tensor([3, 4, -1, 2], dtype=torch.int32, device="cuda")
    tokens, acc = _run(pkv, t, q, x, ua, us, num=num, status=status)
    want, n = ref.verify(t, q, x, ua, us, num.tolist())
    assert tokens.tolist() == want and acc.tolist() == n and int(status) == pkv.PKV_EBOUNDS


def test_strides_and_odd_bases(pkv):
    B, K, V = 5, 3, 1001
    t, q, x, ua, us = _case(B, K, V, seed=10)
    wide = torch.full((B, K + 1, V + 23), 9.0, device="cuda")     # a padded vocabulary
    wide[..., :V] = t
    odd = torch.zeros(B * K * V + 1, device="cuda")[1:].view(B, K, V)
    odd.copy_(q)
    _check(pkv, wide[..., :V], odd, x, ua, us)
    rows_first = t.transpose(0, 1).contiguous().transpose(0, 1)   # [K + 1, B, V] in memory
    _check(pkv, rows_first, q, x, ua, us)
    _check(pkv, t[:1].expand(B, K + 1, V), q[:1].expand(B, K, V), x, ua, us)


def test_more_than_2_31_elements(pkv):
    """The last sequences of 4096 x 5 rows of 131072; the rows ahead have no mass."""
    B, K, V = 4096, 4, 131072
    t = torch.zeros(B, K + 1, V, dtype=torch.float16, device="cuda")
    q = torch.zeros(B, K, V, dtype=torch.float16, device="cuda")
    x = torch.zeros(B, K, dtype=torch.int32, device="cuda")
    ua, us = torch.zeros(B, K, device="cuda"), torch.zeros(B, device="cuda")
    few = _case(3, K, V, torch.float16, seed=30)
    for a, b in zip((t, q, x, ua, us), few):
        a[-3:] = b
    tokens, acc = _run(pkv, t, q, x, ua, us)
    want, n = ref.verify(*few)
    assert tokens[-3:].tolist() == want and acc[-3:].tolist() == n
    assert bool((tokens[:-3] == -1).all()) and int(acc[:-3].sum()) == 0


def test_the_same_answer_in_any_batch(pkv):
    """One sequence's row is cut differently in a batch of another size."""
    t, q, x, ua, us = _case(400, 2, 20000, seed=11)
    tokens, acc = _run(pkv, t, q, x, ua, us)
    for lo, hi in ((0, 1), (17, 40), (100, 230)):
        a, b = _run(pkv, t[lo:hi], q[lo:hi], x[lo:hi], ua[lo:hi], us[lo:hi])
        assert torch.equal(a, tokens[lo:hi]) and torch.equal(b, acc[lo:hi])


def test_kept_tokens_follow_the_target(pkv):
    """First token over 2^18 sequences drawn from one pair of distributions: each
    frequency within 5 standard deviations, sqrt(p (1 - p) / N), of the target's."""
    N, V = 1 << 18, 12
    g = torch.Generator().manual_seed(12)
    p = torch.softmax(torch.randn(V, generator=g), 0)
    q = torch.softmax(torch.randn(V, generator=g), 0)
    x = torch.multinomial(q, N, replacement=True, generator=g).int().view(N, 1).cuda()
    ua, us = torch.rand(N, 1, generator=g).cuda(), torch.rand(N, generator=g).cuda()
    tokens, _ = _run(pkv, p.cuda().expand(N, 2, V), q.cuda().expand(N, 1, V), x, ua, us)
    freq = torch.bincount(tokens[:, 0].long().cpu(), minlength=V).double() / N
    sd = (p.double() * (1 - p.double()) / N).sqrt()
    assert bool(((freq - p.double()).abs() <= 5 * sd).all())


def test_two_streams_at_once(pkv):
    cases = [_case(20, 3, 50000, seed=40), _case(1, 4, 131072, seed=41)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [(torch.empty(c[2].shape[0], c[2].shape[1] + 1, dtype=torch.int32, device="cuda"),
             torch.empty(c[2].shape[0], dtype=torch.int32, device="cuda")) for c in cases]
    torch.cuda.synchronize()
    for _ in range(10):
        for c, o, st in zip(cases, outs, streams):
            pkv.verify_drafts(*o, *c, stream=st)
    torch.cuda.synchronize()
    for c, o in zip(cases, outs):
        want, n = ref.verify(*c)
        assert o[0].tolist() == want and o[1].tolist() == n


@pytest.mark.parametrize("lookup", [False, True])
@pytest.mark.parametrize("sharp", [6.0, 30.0])
def test_peaked_rows(pkv, sharp, lookup):
    """Most of the mass on a few tokens, among them ones above 2^-8 next to one another."""
    t, q, x, ua, us = _case(30, 4, 40001, seed=42, sharp=sharp, noise=1.0)
    t[:10, :, 500:530] += 0.5 / 30
    q[:10, :, 505:520] += 0.1
    _check(pkv, t, None if lookup else q, x, ua, us)


def test_another_stream_and_graph_replay(pkv):
    args = _case(4, 3, 9000, seed=13)
    t, q, x, ua, us = args
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    tokens = torch.empty(4, 4, dtype=torch.int32, device="cuda")
    acc = torch.empty(4, dtype=torch.int32, device="cuda")
    pkv.verify_drafts(tokens, acc, t, q, x, ua, us, stream=side)
    side.synchronize()
    want, n = ref.verify(t, q, x, ua, us)
    assert tokens.tolist() == want and acc.tolist() == n
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.verify_drafts(tokens, acc, t, q, x, ua, us)
    for seed in (14, 15):
        for a, b in zip(args, _case(4, 3, 9000, seed=seed)):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        want, n = ref.verify(t, q, x, ua, us)
        assert tokens.tolist() == want and acc.tolist() == n


@pytest.mark.parametrize("B,V", [(1, 131072), (90, 20000), (400, 700)])
def test_calls_in_a_row_see_each_other(pkv, B, V):
    """Consecutive calls overlap on the device but each waits for the one before: the
    same buffers take another step's inputs between two calls, and each call's outputs
    are copied before the next overwrites them."""
    steps = [_case(B, 2, V, seed=s) for s in (21, 22, 23)]
    bufs = [t.clone() for t in steps[0]]
    tokens = torch.empty(B, 3, dtype=torch.int32, device="cuda")
    acc = torch.empty(B, dtype=torch.int32, device="cuda")
    got = []
    for i in range(9):
        for b, t in zip(bufs, steps[i % 3]):
            b.copy_(t)
        pkv.verify_drafts(tokens, acc, *bufs)
        pkv.verify_drafts(tokens, acc, *bufs)
        got.append((tokens.clone(), acc.clone()))
    torch.cuda.synchronize()
    for i in range(3):
        want, n = ref.verify(*steps[i])
        for j in range(i, 9, 3):
            assert got[j][0].tolist() == want and got[j][1].tolist() == n


def test_binding_refusals(pkv):
    t, q, x, ua, us = _case(3, 2, 100, seed=16)
    tok = torch.empty(3, 3, dtype=torch.int32, device="cuda")
    acc = torch.empty(3, dtype=torch.int32, device="cuda")
    good = dict(tokens=tok, num_accepted=acc, target=t, draft=q, drafts=x, u_accept=ua,
                u_sample=us)
    pkv.verify_drafts(**good)
    for bad in (dict(tokens=tok[:, :2]), dict(num_accepted=acc.long()), dict(target=t[:, :2]),
                dict(draft=q.half()), dict(draft=t), dict(drafts=x.long()),
                dict(u_accept=ua.double()), dict(u_sample=us[:2]), dict(target=t.cpu()),
                dict(num_drafts=acc[:2]), dict(status=us),
                dict(target=t.transpose(1, 2).contiguous().transpose(1, 2)),
                dict(target=t.double(), draft=None)):
        with pytest.raises(ValueError):
            pkv.verify_drafts(**dict(good, **bad))
