"""What the rotary calls hand on, without a GPU: the rotation as it is at the call."""
import copy
import pickle
import types

import pytest
import torch

from paged_kv_cache_215_gb300 import build as pkv_build


@pytest.fixture(scope="module")
def pkv():
    pkv_build.build()
    from paged_kv_cache_215_gb300 import pkv as mod
    return mod


def _recorded(pkv, monkeypatch):
    calls = []

    def record(*args):
        calls.append(args)
        return 0

    monkeypatch.setattr(pkv, "_tensors", types.SimpleNamespace(rope_apply=record,
                                                               append_rope=record))
    return calls


def _holds(args, rope):
    """freqs, rotary_dim, interleaved and attn_scale stand in the call, nothing older."""
    at = next(i for i, a in enumerate(args) if a is rope.freqs)
    return args[at + 1:at + 4] == (rope.rotary_dim, rope.interleaved, rope.attn_scale)


def test_a_changed_rotation_reaches_the_call(pkv, monkeypatch):
    calls = _recorded(pkv, monkeypatch)
    rope = pkv.Rope(16, scaling="yarn", factor=2.0, original_positions=100, device="cpu")
    pool = object.__new__(pkv.KVPool)
    pool.handle = pool.storage = None
    changes = (("attn_scale", 0.5), ("interleaved", True),
               ("freqs", pkv.Rope(16, base=77.0, device="cpu").freqs),
               ("rotary_dim", 8), ("freqs", rope.freqs[:4].clone()))
    for name, value in changes:
        setattr(rope, name, value)
        pkv.rope_apply(None, None, None, rope)
        pool.append_rope(0, None, None, None, None, rope, None, None)
        assert _holds(calls[-2], rope) and _holds(calls[-1], rope)
    pool.handle = None


def test_copies_hold_their_own(pkv, monkeypatch):
    calls = _recorded(pkv, monkeypatch)
    rope = pkv.Rope(16, interleaved=True, attn_scale=3.0, device="cpu")
    for other in (copy.copy(rope), copy.deepcopy(rope), pickle.loads(pickle.dumps(rope))):
        rope.attn_scale = 2.0
        assert other.attn_scale == 3.0 and torch.equal(other.freqs, rope.freqs)
        pkv.rope_apply(None, None, None, other)
        assert _holds(calls[-1], other)
        rope.attn_scale = 3.0
