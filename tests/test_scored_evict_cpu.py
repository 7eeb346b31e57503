"""Scored attention and eviction without a GPU: what the C entries refuse before any
device work, workspace sizes, and what the Python calls hand on."""
import ctypes

import pytest

from paged_kv_cache_215_gb300 import build as pkv_build
from tests.test_abi import FakePool


@pytest.fixture(scope="module")
def pkv():
    pkv_build.build()
    from paged_kv_cache_215_gb300 import pkv as mod
    return mod


X = ctypes.c_void_p(1 << 20)


def scored(pkv, pool, scores=None, weights=None, weights_in=None, **kw):
    a = dict(out=X, od=pkv.PKV_BF16, q=X, qd=pkv.PKV_BF16, q_len=1, layer=0, tab=X, mb=4, lens=X,
             B=2, most=64, scale=0.125, ks=1.0, vs=1.0, ws=X, wsb=1 << 30)
    a.update(kw)
    ref = lambda x: None if x is None else ctypes.byref(x)
    return pkv.lib().paged_decode_attention_scored(
        a["out"], a["od"], a["q"], a["qd"], a["q_len"], pool, a["layer"], a["tab"], a["mb"],
        a["lens"], a["B"], a["most"], a["scale"], a["ks"], a["vs"], ref(scores), ref(weights),
        ref(weights_in), a["ws"], a["wsb"], None)


def rules(pkv, cap=0.0, window=0):
    return pkv.ScoreRules(cap, window, None, None, None)


def rows(pkv, at=1 << 20, seq=128, head=64):
    return pkv.WeightRows(at, seq, head)


def test_scored_refusals(pkv):
    p = FakePool(pkv, nb=8)                                 # bf16, 4 + 2 heads of 64, bs 16
    bad = pkv.PKV_EINVAL
    assert scored(pkv, p.h, B=0) == 0                       # nothing to do
    assert scored(pkv, None) == bad
    for kw in (dict(B=-1), dict(layer=1), dict(q_len=0), dict(most=-1), dict(most=65),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(od=pkv.PKV_FP8_E4M3),
               dict(qd=7), dict(out=None), dict(q=None), dict(tab=None), dict(lens=None),
               dict(mb=0), dict(q=ctypes.c_void_p((1 << 20) + 2)),
               dict(out=ctypes.c_void_p((1 << 20) + 8)), dict(ws=ctypes.c_void_p((1 << 20) + 4))):
        assert scored(pkv, p.h, **kw) == bad, kw
    for cap, window in ((-1.0, 0), (float("nan"), 0), (float("inf"), 0), (1e-44, 0), (0.0, -1)):
        assert scored(pkv, p.h, rules(pkv, cap, window)) == bad, (cap, window)
    # weights: rows that overlap, misalignment, an input alone, the same rows in another order
    for w in (rows(pkv, head=63), rows(pkv, seq=64, head=64), rows(pkv, seq=-1),
              rows(pkv, at=(1 << 20) + 2), rows(pkv, at=None)):
        assert scored(pkv, p.h, None, w) == bad
    assert scored(pkv, p.h, None, None, rows(pkv)) == bad
    assert scored(pkv, p.h, None, rows(pkv), rows(pkv, seq=64, head=128)) == bad
    p.close()
    g = pkv.geometry(1, 4, 2, 64, 16, 8, "e4m3")
    h = ctypes.c_void_p()
    assert pkv.lib().kv_pool_create(ctypes.byref(g), X, pkv.kv_pool_bytes(g), None,
                                    ctypes.byref(h)) == 0
    for ks in (0.0, -1.0, float("nan"), float("inf")):
        assert scored(pkv, h, ks=ks) == bad and scored(pkv, h, vs=ks) == bad
    pkv.lib().kv_pool_destroy(h)


def evict(pkv, pool, **kw):
    a = dict(layer=0, new=X, nb=2, tab=X, mb=4, lens=X, B=2, most=64, keep=X, recent=3,
             w=rows(pkv), o=rows(pkv, at=1 << 24), width=32, out=X, index=None, iw=0, ws=X,
             wsb=1 << 20)
    a.update(kw)
    ref = lambda x: None if x is None else ctypes.byref(x)
    return pkv.lib().kv_evict(pool, a["layer"], a["new"], a["nb"], a["tab"], a["mb"], a["lens"],
                              a["B"], a["most"], a["keep"], a["recent"], ref(a["w"]), ref(a["o"]),
                              a["width"], a["out"], a["index"], a["iw"], a["ws"], a["wsb"], None)


def test_evict_refusals(pkv):
    p = FakePool(pkv, nb=8)
    bad = pkv.PKV_EINVAL
    assert evict(pkv, p.h, B=0) == 0
    assert evict(pkv, None) == bad
    for kw in (dict(layer=-1), dict(layer=1), dict(B=-1), dict(most=-1), dict(most=65),
               dict(recent=-1), dict(nb=-1), dict(width=-1), dict(new=None), dict(tab=None),
               dict(mb=0), dict(lens=None), dict(keep=None), dict(out=None), dict(w=None),
               dict(o=None), dict(o=rows(pkv)), dict(o=rows(pkv, at=1 << 24, head=31)),
               dict(w=rows(pkv, at=(1 << 20) + 1)), dict(index=X, iw=-1),
               dict(ws=ctypes.c_void_p((1 << 20) + 4))):
        assert evict(pkv, p.h, **kw) == bad, kw
    assert evict(pkv, p.h, wsb=64) == pkv.PKV_ENOMEM
    assert evict(pkv, p.h, ws=None) == pkv.PKV_ENOMEM
    p.close()


def test_evict_workspace_bytes(pkv):
    g = pkv.geometry(1, 8, 4, 64, 16, 8, "bf16")
    need = pkv.evict_workspace_bytes(g, 3, 1000)
    assert 3 * 4 * 1000 * 4 <= need < 3 * 4 * 1000 * 4 + 256
    assert pkv.evict_workspace_bytes(g, 1, 1 << 30) >= 4 * (1 << 32)      # past 32 bits
    assert pkv.evict_workspace_bytes(g, -1, 5) == 0


def test_scores_hand_on_what_they_hold_at_the_call(pkv, monkeypatch):
    seen = []

    class Fake:
        @staticmethod
        def attend_scored(*a):
            seen.append(a)
            return 0
    monkeypatch.setattr(pkv, "_tensors", Fake)

    class Pool:
        handle, storage = ctypes.c_void_p(7), "storage"
    rules = pkv.Scores(cap=3.0, window=5)
    rules.cap, rules.slopes = 4.0, "slopes"
    pkv.paged_decode_attention_scored("out", "q", Pool, 2, "tables", "lens", 9, 0.5, scores=rules,
                                      weights="w", weights_in="w0", workspace="ws")
    pkv.paged_decode_attention_scored("out", "q", Pool, 2, "tables", "lens", 9, 0.5,
                                      workspace="ws")
    assert seen[0] == ("out", "q", 7, "storage", 2, "tables", "lens", 9, 0.5, 4.0, 5, "slopes",
                       None, None, 1.0, 1.0, "w", "w0", "ws", None)
    assert seen[1][9:14] == (0.0, 0, None, None, None)


def test_caps_at_the_ends_of_fp32(pkv):
    p = FakePool(pkv, nb=8)
    bad = pkv.PKV_EINVAL
    assert scored(pkv, p.h, rules(pkv, 3e38)) == bad          # cap * log2(e) overflows
    assert scored(pkv, p.h, rules(pkv, 1e38), scale=0.125) == bad     # scale / cap is subnormal
    assert scored(pkv, p.h, rules(pkv, 1e30), scale=1e-9) == bad
    for cap, scale in ((1e30, 0.125), (1e30, 0.0), (1e-30, 0.125)):
        # (without a workspace: nothing is launched where there is a GPU)
        assert scored(pkv, p.h, rules(pkv, cap), scale=scale, ws=None) in (pkv.PKV_ECUDA,
                                                                           pkv.PKV_ENOMEM)
    p.close()


def test_evict_refuses_lengths_written_over_read_ones(pkv):
    p = FakePool(pkv, nb=8)
    bad, far = pkv.PKV_EINVAL, lambda d: ctypes.c_void_p((1 << 22) + d)
    assert evict(pkv, p.h, out=far(0), lens=far(0)) == bad
    assert evict(pkv, p.h, out=far(0), lens=far(4)) == bad    # two sequences: one apart
    assert evict(pkv, p.h, out=far(4), keep=far(0)) == bad
    # more than a sequence may keep: refused too, but for another reason where they are apart
    big = dict(most=1 << 23, mb=1 << 20, nb=1 << 20, width=1 << 23, index=X, iw=1 << 23,
               o=rows(pkv, 1 << 40, 1 << 24, 1 << 23), out=far(0))
    assert evict(pkv, p.h, lens=far(8), keep=far(-8), **big) == pkv.PKV_EUNSUPPORTED
    assert evict(pkv, p.h, lens=far(7), keep=far(-8), **big) == bad
    assert evict(pkv, p.h, lens=far(8), keep=far(-4), **big) == bad
    p.close()


def test_evict_refuses_new_weights_that_meet_the_weights(pkv):
    """Against every pair of rows: 2 sequences, 2 heads, 40 columns read, 8 written."""
    p = FakePool(pkv, nb=8)
    at, most, width = 1 << 24, 40, 8
    met = apart = 0
    for seq_in, head_in in ((80, 40), (200, 100), (50, 130), (0, 0), (400, 0), (0, 48)):
        for seq_out, head_out in ((16, 8), (200, 100), (100, 200), (8, 60), (43, 9), (60, 52)):
            for d in range(-260, 420, 13):
                read = {d + s * seq_in + h * head_in + j
                        for s in range(2) for h in range(2) for j in range(most)}
                written = {s * seq_out + h * head_out + j
                           for s in range(2) for h in range(2) for j in range(width)}
                w, o = rows(pkv, at + 4 * d, seq_in, head_in), rows(pkv, at, seq_out, head_out)
                # (a workspace too small: nothing is launched where there is a GPU)
                got = evict(pkv, p.h, w=w, o=o, most=most, width=width, wsb=0)
                assert got == (pkv.PKV_EINVAL if read & written else pkv.PKV_ENOMEM), \
                    (seq_in, head_in, seq_out, head_out, d)
                met += bool(read & written)
                apart += not read & written
    assert met > 300 and apart > 300
    far = (1 << 62) - 1                                       # strides whose sums pass 64 bits
    assert evict(pkv, p.h, w=rows(pkv, at, far, far), o=rows(pkv, at + 156, far, 16),
                 width=8, most=40, wsb=0) == pkv.PKV_EINVAL
    assert evict(pkv, p.h, w=rows(pkv, at, far, far), o=rows(pkv, at - 512, far, 16),
                 width=8, most=40, wsb=0) == pkv.PKV_ENOMEM
    one = lambda a, b: evict(pkv, p.h, B=1, w=rows(pkv, a, 0, 64), o=rows(pkv, b, 0, 64), wsb=0)
    assert one(at, at + 4 * 127) == pkv.PKV_EINVAL and one(at, at + 4 * 128) == pkv.PKV_ENOMEM
    p.close()


def test_sequences_whose_slots_leave_32_bits_are_refused(pkv):
    p = FakePool(pkv, nb=8)
    most = 2 ** 31 - 2 ** 16                                  # (no workspace: nothing is launched)
    for n, codes in ((most, (pkv.PKV_ECUDA, pkv.PKV_ENOMEM)), (most + 1, (pkv.PKV_EUNSUPPORTED,)),
                     (2 ** 31 - 1, (pkv.PKV_EUNSUPPORTED,))):
        assert scored(pkv, p.h, most=n, mb=1 << 27, ws=None) in codes
        w = rows(pkv, 1 << 40, 1 << 32, 1 << 31)
        assert scored(pkv, p.h, None, w, most=n, mb=1 << 27, ws=None) in codes
        codes = tuple(c for c in codes if c != pkv.PKV_ECUDA)
        assert evict(pkv, p.h, w=w, most=n, mb=1 << 27, ws=None) in codes
        wide = rows(pkv, 1 << 44, 1 << 32, 1 << 31)
        assert evict(pkv, p.h, o=wide, width=n, ws=None) in codes
    p.close()
