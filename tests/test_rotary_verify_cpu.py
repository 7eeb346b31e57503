"""Rotary positions and draft verification without a GPU: the frequency tables
against their formulas, and every refusal before any device work."""
import ctypes
import math

import numpy as np
import pytest

from paged_kv_cache_215_gb300 import build as pkv_build
from tests import rotary_reference as ref
from tests.test_abi import FakePool


@pytest.fixture(scope="module")
def pkv():
    pkv_build.build()
    from paged_kv_cache_215_gb300 import pkv as mod
    return mod


def _table(pkv, rotary, scaling="none", base=10000.0, factor=1.0, original=4096.0, fast=32.0,
           slow=1.0):
    n = max(rotary // 2, 1)
    t, m = (ctypes.c_uint64 * n)(), ctypes.c_float(0)
    cfg = pkv.RopeConfig(rotary, pkv.ROPE_SCALING.get(scaling, 9), base, factor, original, fast,
                         slow)
    rc = pkv.lib().pkv_rope_freqs(ctypes.byref(cfg), t, ctypes.byref(m))
    return rc, np.array(t[:], dtype=np.uint64), m.value


@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "yarn"])
@pytest.mark.parametrize("rotary", [2, 20, 64, 128])
def test_frequency_table(pkv, rotary, scaling):
    """Turns per position within 2^-52 of the formula (two roundings of the frequency
    and the division, 2^-53 each, of values up to 0.16 turns; 2^-48 allows for pow)."""
    factor = 1.0 if scaling == "none" else 8.0
    rc, table, m = _table(pkv, rotary, scaling, factor=factor)
    f, want = ref.frequencies(rotary, scaling=scaling, factor=factor, original=4096.0)
    assert rc == 0 and abs(m - want) <= 2.0 ** -24 * want
    got = table.astype(np.float64) / 2.0 ** 64
    assert np.all(np.abs(got - f / (2 * math.pi)) <= 2.0 ** -48 * f + 2.0 ** -63)


def test_table_follows_the_given_frequency_to_the_last_bits(pkv):
    """The table against f / (2 pi) in 60-digit arithmetic: within two units of 2^-64 of
    a turn (two truncations)."""
    from fractions import Fraction
    pi = Fraction(3141592653589793238462643383279502884197169399375105820974944592307816406286,
                  10 ** 75)
    x = [1.0, 0.7498942093324559, 1e-4, 3.3e-9, 5.0, 123456.789, -0.1, -2e-7]
    t = (ctypes.c_uint64 * len(x))()
    assert pkv.lib().pkv_rope_freqs_from((ctypes.c_double * len(x))(*x), len(x), t) == 0
    for f, got in zip(x, t):
        want = Fraction(f) / (2 * pi) % 1 * 2 ** 64
        off = abs(Fraction(got) - want)
        assert min(off, 2 ** 64 - off) <= 2, f


def test_given_frequencies_wrap_to_one_turn(pkv):
    t = (ctypes.c_uint64 * 4)()
    x = (ctypes.c_double * 4)(0.0, 2 * math.pi * 1.25, -2 * math.pi * 0.25, math.pi)
    assert pkv.lib().pkv_rope_freqs_from(x, 4, t) == 0
    got = np.array(t[:], dtype=np.float64) / 2.0 ** 64
    assert np.allclose(got, [0.0, 0.25, 0.75, 0.5], atol=2.0 ** -50)


def test_frequency_refusals(pkv):
    for kw in (dict(rotary=0), dict(rotary=3), dict(rotary=-2), dict(scaling="other"),
               dict(base=0.0), dict(base=float("nan")), dict(scaling="linear", factor=0.5),
               dict(scaling="ntk", factor=float("inf")), dict(scaling="yarn", original=0.0),
               dict(scaling="yarn", fast=1.0, slow=1.0),
               dict(scaling="yarn", fast=float("nan"))):
        rc, _, _ = _table(pkv, **dict(dict(rotary=8), **kw))
        assert rc == pkv.PKV_EINVAL, kw
    t = (ctypes.c_uint64 * 1)()
    for f in (float("inf"), float("nan"), 1e10, -1e10):
        assert pkv.lib().pkv_rope_freqs_from((ctypes.c_double * 1)(f), 1, t) == pkv.PKV_EINVAL
    assert pkv.lib().pkv_rope_freqs_from((ctypes.c_double * 1)(1.0), 0, t) == pkv.PKV_EINVAL


BASE = 1 << 20


def _rows(pkv, heads=4, dim=64, data=BASE, ts=None, hs=None):
    return pkv.Rows(data, heads * dim if ts is None else ts, dim if hs is None else hs)


def _rope(pkv, rotary=64, **kw):
    d = dict(d_freqs=BASE, rotary_dim=rotary, interleaved=0, attn_scale=1.0)
    d.update(kw)
    return pkv.RopeRef(d["d_freqs"], d["rotary_dim"], d["interleaved"], d["attn_scale"])


def test_rope_apply_refusals(pkv):
    L = pkv.lib()

    def call(**kw):
        a = dict(qo=_rows(pkv, data=2 * BASE), q=_rows(pkv), H=4, ko=None, k=None, Hk=0,
                 dt=pkv.PKV_BF16, D=64, pos=BASE, T=5, rope=_rope(pkv), back=0)
        a.update(kw)
        ref_ = lambda r: None if r is None else ctypes.byref(r)
        return L.rope_apply(ref_(a["qo"]), ref_(a["q"]), a["H"], ref_(a["ko"]), ref_(a["k"]),
                            a["Hk"], a["dt"], a["D"], a["pos"], a["T"], ref_(a["rope"]),
                            a["back"], None)

    assert call(T=0) == 0                                    # no tokens: no work
    bad = [dict(T=-1), dict(H=0), dict(Hk=-1), dict(dt=pkv.PKV_FP8_E4M3), dict(D=513), dict(D=0),
           dict(pos=None), dict(back=2), dict(rope=None), dict(q=None), dict(qo=None),
           dict(q=_rows(pkv, data=None)), dict(q=_rows(pkv, data=BASE + 1)),
           dict(q=_rows(pkv, ts=-256)), dict(Hk=2),
           dict(rope=_rope(pkv, rotary=66)), dict(rope=_rope(pkv, rotary=3)),
           dict(rope=_rope(pkv, rotary=0)), dict(rope=_rope(pkv, d_freqs=None)),
           dict(rope=_rope(pkv, d_freqs=BASE + 4)), dict(rope=_rope(pkv, interleaved=2)),
           dict(rope=_rope(pkv, attn_scale=float("nan"))),
           dict(qo=_rows(pkv, data=2 * BASE, ts=0)),         # every token in one row
           dict(qo=_rows(pkv, data=2 * BASE, hs=0)),
           dict(qo=_rows(pkv, data=2 * BASE, ts=255)),       # a token's last head overlaps
           dict(qo=_rows(pkv, data=2 * BASE, ts=64, hs=319)),   # heads outermost, overlapping
           dict(qo=_rows(pkv, ts=512)),                      # in place with other strides
           dict(T=1 << 31), dict(H=65536, qo=_rows(pkv, heads=65536, data=2 * BASE)),
           dict(H=65535, Hk=1, qo=_rows(pkv, heads=65535, data=2 * BASE))]
    for kw in bad:
        assert call(**kw) == pkv.PKV_EINVAL, kw


def test_append_rope_refusals(pkv):
    p = FakePool(pkv, nb=8)                                  # bf16, 4 / 2 heads of 64, bs 16
    L = pkv.lib()

    def call(**kw):
        a = dict(pool=p.h, layer=0, qo=_rows(pkv, data=2 * BASE), q=_rows(pkv),
                 k=_rows(pkv, heads=2), v=_rows(pkv, heads=2), dt=pkv.PKV_BF16, rope=_rope(pkv),
                 tab=BASE, mb=4, B=2, ids=BASE, pos=BASE, T=2)
        a.update(kw)
        ref_ = lambda r: None if r is None else ctypes.byref(r)
        return L.kv_append_rope(a["pool"], a["layer"], ref_(a["qo"]), ref_(a["q"]), ref_(a["k"]),
                                ref_(a["v"]), a["dt"], ref_(a["rope"]), a["tab"], a["mb"],
                                a["B"], a["ids"], a["pos"], a["T"], 1.0, 1.0, None)

    assert call(T=0) == 0
    bad = [dict(pool=None), dict(layer=1), dict(layer=-1), dict(B=-1), dict(B=0), dict(T=-1),
           dict(dt=pkv.PKV_F16), dict(dt=pkv.PKV_F32), dict(tab=None), dict(mb=0),
           dict(pos=None), dict(k=None), dict(v=None), dict(q=None), dict(qo=None),
           dict(k=_rows(pkv, heads=2, data=BASE + 1)), dict(rope=None),
           dict(rope=_rope(pkv, rotary=128)), dict(qo=_rows(pkv, data=2 * BASE, ts=1))]
    for kw in bad:
        assert call(**kw) == pkv.PKV_EINVAL, kw
    p.close()


def test_append_rope_refuses_bad_e4m3_scales(pkv):
    g = pkv.geometry(1, 4, 2, 64, 16, 8, "e4m3")
    h = ctypes.c_void_p()
    assert pkv.lib().kv_pool_create(ctypes.byref(g), ctypes.c_void_p(BASE), pkv.kv_pool_bytes(g),
                                    None, ctypes.byref(h)) == 0
    r, k = _rope(pkv), _rows(pkv, heads=2)
    for ks, vs in ((0.0, 1.0), (1.0, -1.0), (float("nan"), 1.0), (1.0, float("inf"))):
        assert pkv.lib().kv_append_rope(h, 0, None, None, ctypes.byref(k), ctypes.byref(k),
                                        pkv.PKV_BF16, ctypes.byref(r), BASE, 4, 2, BASE, BASE, 2,
                                        ks, vs, None) == pkv.PKV_EINVAL
    pkv.lib().kv_pool_destroy(h)


def test_verify_refusals(pkv):
    L = pkv.lib()

    def call(**kw):
        a = dict(tok=BASE, acc=BASE, t=pkv.Probs(BASE, 300, 100), d=pkv.Probs(BASE, 200, 100),
                 dt=pkv.PKV_F32, x=BASE, n=None, ua=BASE, us=BASE, B=3, K=2, V=100)
        a.update(kw)
        ref_ = lambda r: None if r is None else ctypes.byref(r)
        return L.verify_drafts(a["tok"], a["acc"], ref_(a["t"]), ref_(a["d"]), a["dt"], a["x"],
                               a["n"], a["ua"], a["us"], a["B"], a["K"], a["V"], None, None)

    assert call(B=0) == 0
    bad = [dict(B=-1), dict(K=-1), dict(V=0), dict(dt=pkv.PKV_FP8_E4M3), dict(tok=None),
           dict(acc=None), dict(t=None), dict(t=pkv.Probs(None, 300, 100)),
           dict(t=pkv.Probs(BASE + 2, 300, 100)), dict(t=pkv.Probs(BASE, -300, 100)),
           dict(d=pkv.Probs(BASE + 1, 200, 100)), dict(d=pkv.Probs(BASE, 200, -1)),
           dict(x=None), dict(ua=None), dict(us=None)]
    for kw in bad:
        assert call(**kw) == pkv.PKV_EINVAL, kw


def test_binding_refuses_host_tensors_and_wrong_shapes(pkv):
    import torch
    rope = pkv.Rope(64, device="cpu")
    q, pos = torch.zeros(3, 4, 64), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA device"):
        pkv.rope_apply(q, q, pos, rope)
    with pytest.raises(ValueError, match="k_out"):
        pkv.rope_apply(q, q, pos, rope, k=q)
    with pytest.raises(ValueError, match="rotary_dim"):
        pkv.Rope(7, device="cpu")
    with pytest.raises(ValueError, match="frequencies"):
        pkv.Rope(8, frequencies=[1.0], device="cpu")
    with pytest.raises(ValueError, match="scaling"):
        pkv.Rope(8, scaling="other", device="cpu")
    with pytest.raises(pkv.PkvError):
        pkv.Rope(8, scaling="yarn", factor=4.0, device="cpu")     # no original_positions
