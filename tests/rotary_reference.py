"""Plain 64-bit implementations of the rotary positions, the append with rotation
and the verification of drafts, and the error bounds the GPU tests hold them to.

Bound of a rotated pair.  The kernel's sine and cosine of an angle are off by at
most: pi * 2^-25 (the angle in half turns rounded to fp32) + 2^-33 turns (the phase
cut to 32 bits) + one ulp of sincospif (2^-24 for results up to 1); times the
attention scale (2^-24 of the product) and the value (2^-24), plus the final
addition (2^-24 of a sum up to |a| + |b|): below 2^-21 (|a| + |b|) m together.
The angle itself is off by the roundings of the frequency, of its quotient by 2 pi
and of this reference's product, 2^-53 of it each: 2^-51 radians per position in all
(frequencies up to 1).  16-bit outputs may take the special-function unit's sine, off
by up to 2^-20.9 in [-pi, pi], so 2^-19 is allowed there.  Storing rounds once: half a step,
torch.finfo(dtype).eps / 2 of the value, and half the smallest subnormal."""
import math

import numpy as np
import torch

COMPUTE = {torch.float32: 2.0 ** -21, torch.float16: 2.0 ** -19, torch.bfloat16: 2.0 ** -19}


def frequencies(rotary, base=10000.0, scaling="none", factor=1.0, original=0.0, fast=32.0,
                slow=1.0):
    """([rotary / 2] radians per position, attention scale), one pair at a time."""
    out = []
    for i in range(rotary // 2):
        b = base * factor ** (rotary / (rotary - 2)) if scaling == "ntk" and rotary > 2 else base
        f = b ** (-2 * i / rotary)
        if scaling == "linear":
            f /= factor
        if scaling == "yarn":
            g = (original * f / (2 * math.pi) - slow) / (fast - slow)
            g = min(max(g, 0.0), 1.0)
            f = (1 - g) * f / factor + g * f
        out.append(f)
    return np.array(out), (0.1 * math.log(factor) + 1 if scaling == "yarn" else 1.0)


def rotate(x, positions, freqs, m, rotary, interleaved, backward=False):
    """x [T, H, D] (any dtype) in fp64: (rotated, |a| + |b| of each element's pair)."""
    x = x.detach().cpu().double().numpy()
    out, size = x.copy(), np.abs(x)
    for t, p in enumerate(positions.cpu().tolist()):
        for i, f in enumerate(freqs):
            j, k = (2 * i, 2 * i + 1) if interleaved else (i, i + rotary // 2)
            angle = math.fmod(p * float(f), 2 * math.pi) * (-1 if backward else 1)
            a, b = x[t, :, j], x[t, :, k]
            out[t, :, j] = m * (a * math.cos(angle) - b * math.sin(angle))
            out[t, :, k] = m * (a * math.sin(angle) + b * math.cos(angle))
            size[t, :, j] = size[t, :, k] = np.abs(a) + np.abs(b)
    return out, size


def compute_bound(size, m, dtype, positions):
    angle = positions.cpu().double().numpy().reshape(-1, 1, 1) * 2.0 ** -51
    return (COMPUTE[dtype] + angle) * size * abs(m)


def bound(ref, size, m, dtype, positions):
    """Largest error of a stored value: computing and one rounding."""
    fi = torch.finfo(dtype)
    c = compute_bound(size, m, dtype, positions)
    return c + fi.eps / 2 * (np.abs(ref) + c) + fi.smallest_normal * fi.eps / 2


def check_rotated(got, x, positions, freqs, m, rotary, interleaved, backward=False):
    """Rotated rows within the bound; the unrotated elements bit for bit."""
    ref, size = rotate(x, positions, freqs, m, rotary, interleaved, backward)
    g = got.detach().cpu().double().numpy()
    err = np.abs(g - ref)[..., :rotary]
    lim = bound(ref, size, m, x.dtype, positions)[..., :rotary]
    worst = float((err / lim).max()) if err.size else 0.0
    assert worst <= 1.0, f"worst error / bound {worst:.3f}"
    assert torch.equal(got[..., rotary:].cpu(), x[..., rotary:].cpu())
    return worst


def verify(target, draft, drafts, u_accept, u_sample, num_drafts=None):
    """(tokens, accepted) as lists, sequence by sequence in fp64."""
    def clean(row):
        row = np.nan_to_num(row.detach().cpu().double().numpy(), nan=0.0, posinf=1.0)
        return np.clip(row, 0.0, 1.0)

    B, K = drafts.shape
    x, ua, us = drafts.cpu().numpy(), u_accept.cpu().numpy(), u_sample.cpu().numpy()
    tokens, accepted = [], []
    for s in range(B):
        n = K if num_drafts is None else int(min(max(int(num_drafts[s]), 0), K))
        a = 0
        while a < n:
            t = int(x[s, a])
            if not 0 <= t < target.shape[2]:
                break
            p = clean(target[s, a])[t]
            q = 1.0 if draft is None else clean(draft[s, a])[t]
            if not (p > 0 and float(ua[s, a]) * q < p):
                break
            a += 1
        row = clean(target[s, a])
        w = row
        if a < n:
            if draft is None:
                w = row.copy()
                if 0 <= int(x[s, a]) < len(w):
                    w[int(x[s, a])] = 0.0
            else:
                w = np.maximum(row - clean(draft[s, a]), 0.0)
            if w.sum() == 0:
                w = row
        u = float(us[s])
        u = 0.0 if not u > 0 else min(u, 1 - 2.0 ** -53)
        total = np.minimum(np.cumsum(w), 16.0)
        if total[-1] == 0:
            new = -1
        else:
            new = int(np.searchsorted(total, u * total[-1], side="right"))
            new = min(new, int(np.flatnonzero(w)[-1]))
        tokens.append(list(map(int, x[s, :a])) + [new] + [-1] * (K - a))
        accepted.append(a)
    return tokens, accepted
