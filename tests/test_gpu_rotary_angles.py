"""Accuracy of rotated values near the zeros of sine and cosine, where a value is far
smaller than its pair: each output is held to the products it is made of.

Bound.  With the angle t reduced to [-pi, pi], the output a cos t - b sin t is off by
  (|a cos t| + |b sin t|) m times 2^-22.8 (sine and cosine) + 2^-24 (times m)
                                  + 2^-24 (the product) + 2^-24 (the sum): below 2^-21;
  (|a sin t| + |b cos t|) m times what t is off: two fp32 roundings of it, |t| 2^-23,
                                  and 2^-51 radians a position (see rotary_reference);
then one rounding to the output's type.  a sin t + b cos t likewise."""
import math

import numpy as np
import pytest
import torch

import oracle
from tests import rotary_reference as ref

pytestmark = pytest.mark.gpu
DT = [torch.float32, torch.float16, torch.bfloat16]
POSITIONS = [0, 1, 2, 3, 7, 22, 100, 355, 1000, 4097, 65537, 120000, 710 * 1477, 2 ** 24 + 1]


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_215_gb300 import pkv as mod
    return mod


def _rows(T, heads, D, dtype, interleaved):
    """Pairs (0, 1), (1, 0), (0, -0.75), (random, random), one kind a head."""
    g = torch.Generator().manual_seed(D + heads)
    a, b = torch.randn(T, heads, D // 2, generator=g), torch.randn(T, heads, D // 2, generator=g)
    for h in range(heads):
        if h % 4 < 3:
            a[:, h], b[:, h] = [(0.0, 1.0), (1.0, 0.0), (0.0, -0.75)][h % 4]
    x = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return x.to(dtype).cuda()


def _exact(x, positions, freqs, m, interleaved, backward=False):
    """(rotated, largest error ahead of the rounding) in fp64."""
    x = x.detach().cpu().double().numpy()
    n = x.shape[2] // 2
    p = np.array(positions, dtype=np.float64)[:, None, None]
    t = np.fmod(p * np.asarray(freqs, dtype=np.float64), 2 * math.pi)
    t = (t - 2 * math.pi * np.round(t / (2 * math.pi))) * (-1 if backward else 1)
    first, second = (slice(0, None, 2), slice(1, None, 2)) if interleaved else \
        (slice(0, n), slice(n, None))
    a, b, c, s = x[..., first], x[..., second], np.cos(t), np.sin(t)
    out, err = np.empty_like(x), np.empty_like(x)
    off = np.abs(t) * 2.0 ** -23 + p * 2.0 ** -51
    out[..., first], out[..., second] = m * (a * c - b * s), m * (a * s + b * c)
    for at, u, v in ((first, a * c, b * s), (second, a * s, b * c)):
        w = (b * c, a * s) if at is first else (b * s, a * c)
        err[..., at] = abs(m) * ((np.abs(u) + np.abs(v)) * 2.0 ** -21 +
                                 (np.abs(w[0]) + np.abs(w[1])) * off)
    return out, err


def _check(got, x, positions, freqs, m, interleaved, backward=False):
    want, err = _exact(x, positions, freqs, m, interleaved, backward)
    fi = torch.finfo(x.dtype)
    lim = err + fi.eps / 2 * (np.abs(want) + err) + fi.smallest_normal * fi.eps / 2
    off = np.abs(got.detach().cpu().double().numpy() - want)
    worst = float((off / lim).max())
    assert worst <= 1.0, f"worst error / bound {worst:.3f}"


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", DT, ids=str)
@pytest.mark.parametrize("repeat", [1, 400])           # one and several heads a thread
def test_small_results_keep_their_digits(pkv, dtype, interleaved, backward, repeat):
    H, D = 5, 128
    positions = POSITIONS * repeat
    freqs, m = ref.frequencies(D)
    rope = pkv.Rope(D, interleaved=interleaved)
    x = _rows(len(POSITIONS), H, D, dtype, interleaved)
    big = x.repeat(repeat, 1, 1)
    out = torch.empty_like(big)
    pkv.rope_apply(out, big, torch.tensor(positions, dtype=torch.int32, device="cuda"), rope,
                   backward=backward)
    _check(out[:len(POSITIONS)], x, POSITIONS, freqs, m, interleaved, backward)
    assert torch.equal(out, out[:len(POSITIONS)].repeat(repeat, 1, 1))


@pytest.mark.parametrize("dtype", DT, ids=str)
def test_slow_frequencies(pkv, dtype):
    """Turns of 1e-3 to 1e-12 radians a position, either direction."""
    freqs = np.array([1e-3, -1e-5, 3e-7, -2e-9, 1e-12, -0.4, 0.0, 1e-8])
    rope = pkv.Rope(16, frequencies=freqs, attn_scale=1.25)
    x = _rows(len(POSITIONS), 4, 16, dtype, False)
    out = torch.empty_like(x)
    pkv.rope_apply(out, x, torch.tensor(POSITIONS, dtype=torch.int32, device="cuda"), rope)
    _check(out, x, POSITIONS, freqs, 1.25, False)


@pytest.mark.parametrize("kv,dtype", [("f32", torch.float32), ("f16", torch.float16),
                                      ("bf16", torch.bfloat16), ("e4m3", torch.float32),
                                      ("e4m3", torch.float16), ("e4m3", torch.bfloat16)])
def test_small_results_in_the_pool(pkv, kv, dtype):
    """Keys (0, 1) and the like stored; for E4M3 under a scale that gives the small
    results codes of their own (the large ones saturate)."""
    hk, D, bs, scale = 4, 64, 16, 2.0 ** -20
    freqs, m = ref.frequencies(D)
    T = len(POSITIONS)
    k = _rows(T, hk, D, dtype, False)
    positions = torch.tensor([p % 128 for p in POSITIONS], dtype=torch.int32, device="cuda")
    geom = pkv.geometry(1, hk, hk, D, bs, 8 * T, kv)
    pool = pkv.KVPool(geom, storage=torch.zeros(pkv.kv_pool_bytes(geom), dtype=torch.uint8,
                                                device="cuda"))
    tables = torch.arange(8 * T, dtype=torch.int32, device="cuda").view(T, 8)
    pool.append_rope(0, None, None, k, k, pkv.Rope(D), tables, positions, k_scale=scale,
                     v_scale=1.0)
    assert pool.check_status() == 0
    at = positions.tolist()
    view = pool.view()
    got = torch.stack([view[8 * t + p // bs, 0, 0, :, p % bs] for t, p in enumerate(at)])
    if kv != "e4m3":
        _check(got, k, at, freqs, m, False)
        return
    want, err = _exact(k, at, freqs, m, False)
    # encoding is monotone: the code lies between those of the value's bounds
    below, above = (np.nextafter((want + e).astype(np.float32), np.float32(s * np.inf))
                    for e, s in ((-err, -1), (err, 1)))
    lo, hi = (oracle.e4m3_encode(v.reshape(-1), scale) for v in (below, above))
    code = oracle.e4m3_decode(got.cpu().numpy().reshape(-1))
    assert np.all((oracle.e4m3_decode(lo) <= code) & (code <= oracle.e4m3_decode(hi)))
