"""Rotary positions on the GPU (rope_apply): both layouts, part of the head, every
type, strides, odd sizes, far positions, padding, gradients, streams and graphs
against the 64-bit reference (bounds derived in rotary_reference)."""
import numpy as np
import pytest
import torch

from tests import rotary_reference as ref

pytestmark = pytest.mark.gpu
DT = [torch.float32, torch.float16, torch.bfloat16]


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_215_gb300 import pkv as mod
    return mod


def _x(shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def _pos(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _check(pkv, x, positions, rope, freqs, m, k=None, backward=False, in_place=False):
    """One call on x (and k), checked; the inputs stay as they were unless in place."""
    keep = [t.clone() for t in (x, k) if t is not None]
    if in_place:
        out, k_out = x, k
    else:
        out = torch.full(x.shape, float("nan"), dtype=x.dtype, device="cuda")
        k_out = None if k is None else torch.full(k.shape, float("nan"), dtype=k.dtype,
                                                  device="cuda")
    pkv.rope_apply(out, x, positions, rope, k_out=k_out, k=k, backward=backward)
    torch.cuda.synchronize()
    for got, src, inp in zip((out, k_out), keep, (x, k)):
        ref.check_rotated(got, src, positions, freqs, m, rope.rotary_dim, rope.interleaved,
                          backward)
        if not in_place:
            assert torch.equal(inp, src)


SHAPES = [  # tokens, q heads, k heads, head_dim, rotary_dim
    (1, 32, 8, 128, 128), (1, 1, 1, 2, 2), (5, 4, 2, 64, 64), (33, 7, 1, 80, 20),
    (17, 3, 3, 96, 48), (9, 2, 1, 65, 64), (4, 2, 2, 512, 512), (3, 2, 1, 511, 2),
    (257, 16, 4, 128, 32), (6, 5, 2, 72, 24), (2, 3, 1, 256, 128),
]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", DT, ids=str)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_rotation(pkv, shape, dtype, interleaved):
    T, hq, hk, D, rd = shape
    freqs, m = ref.frequencies(rd)
    rope = pkv.Rope(rd, interleaved=interleaved)
    q, k = _x((T, hq, D), dtype, 1), _x((T, hk, D), dtype, 2)
    positions = _pos([(i * 37) % 5000 for i in range(T)])
    _check(pkv, q, positions, rope, freqs, m, k=k)
    _check(pkv, q, positions, rope, freqs, m)
    _check(pkv, q.clone(), positions, rope, freqs, m, k=k.clone(), in_place=True)


@pytest.mark.parametrize("dtype", DT, ids=str)
def test_many_tokens_visit_several_heads_per_thread(pkv, dtype):
    T, hq, hk, D = 1500, 33, 5, 64          # heads that do not divide by the thread's share
    freqs, m = ref.frequencies(D)
    rope = pkv.Rope(D)
    q, k = _x((T, hq, D), dtype, 3), _x((T, hk, D), dtype, 4)
    out, ko = torch.empty_like(q), torch.empty_like(k)
    # long enough for the widest share of heads a thread takes
    big_q, big_k = q.repeat(12, 1, 1), k.repeat(12, 1, 1)
    pos = _pos([i % 1500 for i in range(12 * T)])
    bo, bk = torch.empty_like(big_q), torch.empty_like(big_k)
    pkv.rope_apply(bo, big_q, pos, rope, k_out=bk, k=big_k)
    pkv.rope_apply(out, q, pos[:T].contiguous(), rope, k_out=ko, k=k)
    torch.cuda.synchronize()
    assert torch.equal(bo, out.repeat(12, 1, 1)) and torch.equal(bk, ko.repeat(12, 1, 1))
    ref.check_rotated(out[::97], q[::97], pos[:T:97], freqs, m, D, False)
    ref.check_rotated(ko[::97], k[::97], pos[:T:97], freqs, m, D, False)


@pytest.mark.parametrize("scaling", ["linear", "ntk", "yarn"])
@pytest.mark.parametrize("dtype", DT, ids=str)
def test_scaled_for_long_contexts(pkv, dtype, scaling):
    freqs, m = ref.frequencies(128, scaling=scaling, factor=8.0, original=4096.0)
    rope = pkv.Rope(128, scaling=scaling, factor=8.0, original_positions=4096)
    q, k = _x((6, 4, 128), dtype, 5), _x((6, 2, 128), dtype, 6)
    _check(pkv, q, _pos([0, 1, 4095, 32768, 131071, 1048575]), rope, freqs, m, k=k)


@pytest.mark.parametrize("dtype", DT, ids=str)
def test_far_positions_and_given_frequencies(pkv, dtype):
    freqs = np.array([1.0, 0.75, 1e-3, 0.0])
    rope = pkv.Rope(8, frequencies=freqs, attn_scale=-1.5)
    _check(pkv, _x((5, 3, 16), dtype, 7), _pos([2 ** 20, 2 ** 24 + 1, 2 ** 28 + 3, 2 ** 31 - 1,
                                                0]), rope, freqs, -1.5)


def _views(kind, T, hq, hk, D, dtype):
    if kind == "joint":                     # parts of one projection's output
        x = _x((T, (hq + 2 * hk) * D), dtype, 8)
        q, k, _ = x.split([hq * D, hk * D, hk * D], 1)
        return q.view(T, hq, D), k.view(T, hk, D)
    if kind == "heads_first":
        return _x((hq, T, D), dtype, 9).transpose(0, 1), _x((hk, T, D), dtype, 10).transpose(0, 1)
    if kind == "odd_base":                  # rows that start one element off
        return (_x((T * hq * D + 1,), dtype, 11)[1:].view(T, hq, D),
                _x((T * hk * D + 1,), dtype, 12)[1:].view(T, hk, D))
    if kind == "odd_stride":
        return _x((T, hq, D + 1), dtype, 13)[..., :D], _x((T, hk, D + 3), dtype, 14)[..., :D]
    assert kind == "broadcast"              # one row read for every token
    return (_x((1, hq, D), dtype, 15).expand(T, hq, D), _x((T, 1, D), dtype, 16).expand(T, hk, D))


@pytest.mark.parametrize("kind", ["joint", "heads_first", "odd_base", "odd_stride", "broadcast"])
@pytest.mark.parametrize("dtype", DT, ids=str)
@pytest.mark.parametrize("interleaved", [False, True])
def test_strides(pkv, kind, dtype, interleaved):
    T, hq, hk, D = 11, 4, 2, 64
    q, k = _views(kind, T, hq, hk, D, dtype)
    freqs, m = ref.frequencies(D)
    rope = pkv.Rope(D, interleaved=interleaved)
    positions = _pos(list(range(100, 100 + T)))
    _check(pkv, q, positions, rope, freqs, m, k=k)
    if kind in ("joint", "heads_first", "odd_stride"):
        # into rows of another order, and in place through the views
        out = torch.full((hq, T, D), float("nan"), dtype=dtype, device="cuda").transpose(0, 1)
        pkv.rope_apply(out, q, positions, rope)
        ref.check_rotated(out, q, positions, freqs, m, D, interleaved)
        _check(pkv, q, positions, rope, freqs, m, k=k, in_place=True)


def test_in_place_leaves_what_lies_between_the_rows(pkv):
    x = _x((5, 6 * 64), torch.bfloat16, 17)
    keep = x.clone()
    q = x[:, :4 * 64].view(5, 4, 64)
    pkv.rope_apply(q, q, _pos([3, 4, 5, 6, 7]), pkv.Rope(32))
    torch.cuda.synchronize()
    assert torch.equal(x[:, 4 * 64:], keep[:, 4 * 64:])
    freqs, m = ref.frequencies(32)
    ref.check_rotated(q, keep[:, :4 * 64].view(5, 4, 64), _pos([3, 4, 5, 6, 7]), freqs, m, 32,
                      False)


def test_padding_rows_are_left_as_they_were(pkv):
    q, k = _x((5, 4, 64), torch.bfloat16, 18), _x((5, 2, 64), torch.bfloat16, 19)
    out, ko = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
    positions = _pos([10, -1, 12, -2147483648, 14])
    pkv.rope_apply(out, q, positions, pkv.Rope(64), k_out=ko, k=k)
    torch.cuda.synchronize()
    freqs, m = ref.frequencies(64)
    for got, src in ((out, q), (ko, k)):
        assert bool((got[[1, 3]] == 7.0).all())
        ref.check_rotated(got[[0, 2, 4]], src[[0, 2, 4]], positions[[0, 2, 4]], freqs, m, 64,
                          False)


def test_non_finite_values_stay_in_their_pairs(pkv):
    q = _x((1, 1, 8), torch.float32, 20)
    q[0, 0, 1], q[0, 0, 6] = float("inf"), float("nan")
    out = torch.empty_like(q)
    pkv.rope_apply(out, q, _pos([3]), pkv.Rope(8))
    bad = ~torch.isfinite(out[0, 0])
    assert bad.tolist() == [False, True, True, False, False, True, True, False]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T", [9, 4000])
@pytest.mark.parametrize("rd", [2, 20, 36, 78])
@pytest.mark.parametrize("dtype", DT, ids=str)
def test_the_rest_of_a_head_is_copied_bit_for_bit(pkv, dtype, rd, T, interleaved):
    """Any bits behind the rotated part (NaN payloads, infinities, -0), also where it ends
    inside a vector; out of place, and untouched in place."""
    bits = torch.int32 if dtype == torch.float32 else torch.int16
    info = torch.iinfo(bits)
    g = torch.Generator().manual_seed(rd)
    raw = torch.randint(info.min, info.max, (T, 5, 80), generator=g).to(bits).cuda()
    raw[..., :rd] = _x((T, 5, rd), dtype, 33).view(bits)
    x = raw.view(dtype)
    out = torch.zeros_like(x)
    positions = _pos([i % 1000 for i in range(T)])
    rope = pkv.Rope(rd, interleaved=interleaved)
    pkv.rope_apply(out, x, positions, rope)
    assert torch.equal(out.view(bits)[..., rd:], raw[..., rd:])
    freqs, m = ref.frequencies(rd)
    rows = slice(None, None, max(1, T // 9))
    ref.check_rotated(out[rows, :, :rd], x[rows, :, :rd], positions[rows], freqs, m, rd,
                      interleaved)
    keep = raw.clone()
    pkv.rope_apply(x, x, positions, rope)
    assert torch.equal(raw[..., rd:], keep[..., rd:])
    assert torch.equal(x[..., :rd], out[..., :rd])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", DT, ids=str)
def test_gradient_against_the_formula(pkv, dtype, interleaved):
    freqs, m = ref.frequencies(48, scaling="yarn", factor=4.0, original=2048.0)
    rope = pkv.Rope(48, scaling="yarn", factor=4.0, original_positions=2048,
                    interleaved=interleaved)
    gq, gk = _x((9, 6, 64), dtype, 21), _x((9, 2, 64), dtype, 22)
    _check(pkv, gq, _pos([i * 1111 for i in range(9)]), rope, freqs, m, k=gk, backward=True)


@pytest.mark.parametrize("interleaved", [False, True])
def test_gradient_against_differences(pkv, interleaved):
    """L(x) = <g, rope(x)> is linear: (L(x + d) - L(x - d)) / 2 = <grad, d>.  Each
    output is off by at most 2^-21 (|a| + |b|) m plus half an fp32 step (2^-24), so
    both sides are within the summed bounds."""
    T, H, D, rd = 4, 3, 32, 24
    rope = pkv.Rope(rd, scaling="yarn", factor=2.0, original_positions=512,
                    interleaved=interleaved)
    m = rope.attn_scale
    x, g, d = (_x((T, H, D), torch.float32, s) for s in (23, 24, 25))
    positions = _pos([0, 5, 700, 90001])
    up, down, grad = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    plus, minus = x + d, x - d
    pkv.rope_apply(up, plus, positions, rope)
    pkv.rope_apply(down, minus, positions, rope)
    pkv.rope_apply(grad, g, positions, rope, backward=True)
    dd = (plus.double() - minus.double()) / 2
    left = (g.double() * (up.double() - down.double())).sum() / 2
    right = (grad.double() * dd).sum()
    freqs, _ = ref.frequencies(rd, scaling="yarn", factor=2.0, original=512.0)
    lim = 0.0
    for t, w in ((plus, g), (minus, g), (g, dd)):
        r, size = ref.rotate(t, positions, freqs, m, rd, interleaved)
        lim += float((ref.bound(r, size, m, torch.float32, positions) *
                      np.abs(w.double().cpu().numpy())).sum()) * (0.5 if w is g else 1.0)
    assert abs(float(left - right)) <= lim


def test_backward_then_forward_is_the_identity(pkv):
    q = _x((7, 4, 128), torch.float32, 26)
    rope, positions = pkv.Rope(128), _pos([i * 99991 for i in range(7)])
    y, z = torch.empty_like(q), torch.empty_like(q)
    pkv.rope_apply(y, q, positions, rope)
    pkv.rope_apply(z, y, positions, rope, backward=True)
    # two rotations' errors on pairs of |a| + |b| <= 2 sqrt(2) max|q|
    assert float((z - q).abs().max()) <= 2 * (2.0 ** -21 + 2.0 ** -24) * 2 * 2 ** 0.5 * \
        float(q.abs().max())


def test_another_stream_and_graph_replay(pkv):
    T = 6
    q = _x((T, 4, 64), torch.bfloat16, 27)
    positions, out, rope = _pos([0] * T), torch.zeros_like(q), pkv.Rope(64)
    freqs, m = ref.frequencies(64)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        pkv.rope_apply(out, q, positions, rope)            # the current stream
    side.synchronize()
    ref.check_rotated(out, q, positions, freqs, m, 64, False)
    out.zero_()
    torch.cuda.synchronize()
    pkv.rope_apply(out, q, positions, rope, stream=side)   # a given one
    side.synchronize()
    ref.check_rotated(out, q, positions, freqs, m, 64, False)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.rope_apply(out, q, positions, rope)
    for first in (5, 77777):
        positions.copy_(_pos(list(range(first, first + T))))
        q.copy_(_x((T, 4, 64), torch.bfloat16, first))
        graph.replay()
        torch.cuda.synchronize()
        ref.check_rotated(out, q, positions, freqs, m, 64, False)


@pytest.mark.parametrize("T,H", [(3, 2), (1500, 40)])
def test_calls_in_a_row_see_each_other(pkv, T, H):
    """Consecutive calls overlap on the device but each waits for the one before: 40
    rotations in place, a copy in between, equal one by 40 times the position.  A step
    is off by at most (2^-21 + 2^-24) (|a| + |b|) an element, (|a| + |b|) at most sqrt 2
    times the pair's norm, and rotations keep the norm of what is off: 40 steps of two
    elements each give 80 (2^-21 + 2^-24) (|a| + |b|)."""
    D, n = 32, 40
    x0 = _x((T, H, D), torch.float32, 30)
    x, y = x0.clone(), torch.empty_like(x0)
    positions = _pos([i % 91 for i in range(T)])
    rope = pkv.Rope(D)
    for i in range(n // 2):
        pkv.rope_apply(x, x, positions, rope)
        pkv.rope_apply(y, x, positions, rope)
        x.copy_(y)
    torch.cuda.synchronize()
    freqs, m = ref.frequencies(D)
    rows = slice(None, None, max(1, T // 40))
    want, size = ref.rotate(x0[rows], positions[rows] * n, freqs, m, D, False)
    lim = 2 * n * (2.0 ** -21 + 2.0 ** -24) * size
    assert np.all(np.abs(x[rows].double().cpu().numpy() - want) <= lim)


def test_more_than_2_31_elements(pkv):
    T, H, D = 131200, 128, 128
    x = torch.zeros(T, H, D, dtype=torch.bfloat16, device="cuda")
    x[-3:] = _x((3, H, D), torch.bfloat16, 31)
    assert x.numel() > 2 ** 31
    out = torch.empty_like(x)
    positions = torch.arange(T, dtype=torch.int32, device="cuda")
    pkv.rope_apply(out, x, positions, pkv.Rope(D))
    freqs, m = ref.frequencies(D)
    ref.check_rotated(out[-3:], x[-3:], positions[-3:], freqs, m, D, False)
    assert int(torch.count_nonzero(out[:-3])) == 0


def test_copies_of_a_rotation(pkv):
    import copy
    import pickle
    rope = pkv.Rope(16, scaling="yarn", factor=2.0, original_positions=100, interleaved=True)
    copies = [copy.copy(rope), copy.deepcopy(rope), pickle.loads(pickle.dumps(rope))]
    q = _x((4, 2, 16), torch.float32, 32)
    want = torch.empty_like(q)
    pkv.rope_apply(want, q, _pos([1, 2, 3, 4]), rope)
    del rope
    for r in copies:
        out = torch.empty_like(q)
        pkv.rope_apply(out, q, _pos([1, 2, 3, 4]), r)
        assert torch.equal(out, want)


def test_no_tokens(pkv):
    q = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    pkv.rope_apply(q, q, _pos([]), pkv.Rope(64))


def test_binding_refusals(pkv):
    q = _x((3, 4, 64), torch.bfloat16, 28)
    out, pos, rope = torch.empty_like(q), _pos([0, 1, 2]), pkv.Rope(64)
    for args, kw in (((out[:2], q, pos, rope), {}), ((out.float(), q, pos, rope), {}),
                     ((out, q, pos.long(), rope), {}), ((out, q, pos[:2], rope), {}),
                     ((out, q, _pos([0, 0, 1, 1, 2, 2])[::2], rope), {}),
                     ((out, q.transpose(1, 2), pos, rope), {}),
                     ((out, q.cpu(), pos, rope), {}), ((out, q, pos.cpu(), rope), {}),
                     ((out, q, pos, rope), dict(k=q)),
                     ((out, q.double(), pos, rope), {})):
        with pytest.raises(ValueError):
            pkv.rope_apply(*args, **kw)
    with pytest.raises(ValueError, match="gradient"):
        pkv.rope_apply(out, q.clone().requires_grad_(), pos, rope)
    with pytest.raises(pkv.PkvError):                        # every token in one row
        pkv.rope_apply(out[:1].expand(3, 4, 64), q, pos, rope)
    with pytest.raises(pkv.PkvError):
        pkv.rope_apply(out, q, pos, pkv.Rope(128))           # wider than the head
