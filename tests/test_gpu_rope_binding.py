"""What torch knows of the rotary, append and verification calls: the rotation that
they are given, tensors that carry a tangent, and outputs that a graph has saved."""
import pytest
import torch
import torch.autograd.forward_ad as fwd

from tests import rotary_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_215_gb300 import pkv as mod
    return mod


def _x(*shape, dtype=torch.float32):
    g = torch.Generator().manual_seed(sum(shape))
    return torch.randn(shape, generator=g).to(dtype).cuda()


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _pool(pkv, blocks=4, heads=2, dim=64):
    geom = pkv.geometry(1, heads, heads, dim, 16, blocks, "f32")
    return pkv.KVPool(geom, storage=torch.zeros(pkv.kv_pool_bytes(geom), dtype=torch.uint8,
                                                device="cuda"))


def _verify_args(B=2, K=2, V=50):
    p = torch.softmax(_x(B, K + 1, V), -1)
    q = torch.softmax(_x(B, K, V), -1)
    return [torch.empty(B, K + 1, dtype=torch.int32, device="cuda"),
            torch.empty(B, dtype=torch.int32, device="cuda"), p, q,
            torch.zeros(B, K, dtype=torch.int32, device="cuda"),
            torch.full((B, K), 0.5, device="cuda"), torch.full((B,), 0.5, device="cuda")]


def test_a_rotation_changed_after_it_was_made(pkv):
    """Each call goes by what the rotation holds then."""
    q, pos = _x(5, 3, 64), _ints([3, 9, 27, 81, 243])
    rope, other = pkv.Rope(64), pkv.Rope(64, base=500.0)
    out, pool, table = torch.empty_like(q), _pool(pkv, 5, 3), _ints([[0], [1], [2], [3], [4]])
    kept = rope.freqs                       # stays alive
    for change, base, m, inter in (
            (lambda: setattr(rope, "attn_scale", 0.25), 10000.0, 0.25, False),
            (lambda: setattr(rope, "interleaved", True), 10000.0, 0.25, True),
            (lambda: setattr(rope, "freqs", other.freqs), 500.0, 0.25, True)):
        change()
        freqs, _ = ref.frequencies(64, base=base)
        pkv.rope_apply(out, q, pos, rope)
        ref.check_rotated(out, q, pos, freqs, m, 64, inter)
        pool.append_rope(0, None, None, q, q, rope, table, pos % 16)
        for t, p in enumerate((pos % 16).tolist()):
            ref.check_rotated(pool.view()[t, 0, 0, :, p][None], q[t:t + 1],
                              (pos % 16)[t:t + 1], freqs, m, 64, inter)
    assert kept is not rope.freqs
    with pytest.raises(AttributeError):
        pkv.rope_apply(out, q, pos, None)


def test_a_table_that_does_not_fit_is_refused(pkv):
    q, pos = _x(2, 3, 64), _ints([3, 9])
    out, pool, table = torch.empty_like(q), _pool(pkv, heads=3), _ints([[0], [1]])
    good = pkv.Rope(64).freqs
    for bad in (good[:31], good.float(), good.cpu(), good.view(2, 16), good.repeat(2)[::2], None):
        rope = pkv.Rope(64)
        rope.freqs = bad
        with pytest.raises(ValueError, match="rope"):
            pkv.rope_apply(out, q, pos, rope)
        with pytest.raises(ValueError, match="rope"):
            pool.append_rope(0, None, None, q, q, rope, table, pos)


def test_tangents_are_refused(pkv):
    """A forward-mode tangent would be lost, as a recorded gradient would."""
    q, pos, rope = _x(2, 3, 64), _ints([3, 9]), pkv.Rope(64)
    out, pool, table = torch.empty_like(q), _pool(pkv, heads=3), _ints([[0], [1]])
    with fwd.dual_level():
        dual = fwd.make_dual(q, torch.ones_like(q))
        with pytest.raises(ValueError, match="gradient"):
            pkv.rope_apply(out, dual, pos, rope)
        with pytest.raises(ValueError, match="gradient"):
            pool.append_rope(0, out, q, dual, q, rope, table, pos)
        args = _verify_args()
        args[2] = fwd.make_dual(args[2], torch.ones_like(args[2]))
        with pytest.raises(ValueError, match="gradient"):
            pkv.verify_drafts(*args)
        primal, _ = fwd.unpack_dual(dual)
        pkv.rope_apply(out, primal, pos, rope)
    pkv.rope_apply(out, q, pos, rope)


def test_a_graph_notices_that_its_saved_tensor_was_overwritten(pkv):
    q, pos, rope = _x(4, 2, 64), _ints([1, 2, 3, 4]), pkv.Rope(64)
    pool, table = _pool(pkv), _ints([[0], [1], [2], [3]])
    stored = pool.storage.view(torch.float32)
    out, ko = torch.zeros_like(q), torch.zeros_like(q)

    def apply():
        pkv.rope_apply(out, q, pos, rope, k_out=ko, k=q)

    def append():
        pool.append_rope(0, out, q, q, q, rope, table, pos)

    for call, saved in ((apply, out), (apply, ko), (append, out), (append, stored)):
        w = torch.ones_like(saved, requires_grad=True)
        loss = (w * saved).sum()
        call()
        with pytest.raises(RuntimeError, match="inplace"):
            loss.backward()
        loss = (w * saved).sum()                 # saved behind the call: still good
        loss.backward()
        assert torch.equal(w.grad, saved)
    inputs = [t._version for t in (q, pos, rope.freqs, table)]
    apply(), append()
    assert inputs == [t._version for t in (q, pos, rope.freqs, table)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = _verify_args()
    before = [t._version for t in (*args, status)]
    pkv.verify_drafts(*args, status=status)
    after = [t._version for t in (*args, status)]
    assert [b > a for a, b in zip(before, after)] == [True, True] + [False] * 5 + [True]


def test_inference_mode(pkv):
    """Tensors without a version counter, and ordinary ones."""
    q, pos, rope = _x(4, 2, 64), _ints([1, 2, 3, 4]), pkv.Rope(64)
    want, ordinary = torch.empty_like(q), torch.empty_like(q)
    pkv.rope_apply(want, q, pos, rope)
    with torch.inference_mode():
        out = torch.empty_like(q)
        pkv.rope_apply(out, q, pos, rope)
        pkv.rope_apply(ordinary, q, pos, rope)
        assert torch.equal(out, want) and torch.equal(ordinary, want)
