"""Attention under score rules and the record of its weights, in 64 bits and written
from the formulas, with bounds on what a kernel in 32 bits may be off by; and paged pools
for it whose unseen places hold NaN."""
import math

import torch

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
# rounding of a softmax weight to the matrix instructions' operand: two bf16 terms,
# one f16, none (CUDA cores); an E4M3 pool's weights are f16
P_ROUND = {"f32": 0.0, "f16": 2.0 ** -11, "bf16": 2.0 ** -16, "e4m3": 2.0 ** -11}
NAN = {"f32": float("nan"), "f16": float("nan"), "bf16": float("nan")}


class Case:
    """Random q and a paged pool of the given lengths; everything on `device`."""

    def __init__(self, lens, hq, hkv, dim, kv, bs, q_len=1, seed=0, layers=1, layer=0, device="cuda",
                 q_gain=2.0, block_scales=False, q_dtype=None, spare=2, width=None):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.hq, self.hkv, self.dim, self.kv, self.bs = lens, hq, hkv, dim, kv, bs
        self.q_len, self.layers, self.layer, self.batch = q_len, layers, layer, len(lens)
        self.scale = dim ** -0.5
        act = DT[q_dtype or ("bf16" if kv == "e4m3" else kv)]
        self.q = (q_gain * torch.randn(self.batch, q_len, hq, dim, generator=g)).to(act).to(device)
        widths = [-(-n // bs) for n in lens]
        nb = sum(widths) + spare
        ids = torch.randperm(nb, generator=g).to(torch.int32)
        # entries behind a sequence's blocks are outside the pool
        self.tables = torch.full((self.batch, width or max(max(widths), 1) + 1), -7,
                                 dtype=torch.int32)
        at = 0
        for b, w in enumerate(widths):
            self.tables[b, :w] = ids[at:at + w]
            at += w
        shape = (nb, 2, layers, hkv, bs, dim)
        values = torch.randn(shape, generator=g)
        values[:, 0] *= 1.0 + 2.0 * (torch.rand(nb, 1, 1, bs, 1, generator=g) < 0.02)
        self.k_scale = self.v_scale = 1.0
        self.block_scales = None
        if kv == "e4m3":
            if block_scales:
                sc = torch.rand(nb, 2, layers, hkv, generator=g) * 0.02 + 0.005
                self.block_scales = sc.to(device)
                values = values / sc[..., None, None]
            else:
                self.k_scale, self.v_scale = 10.0 / 448, 5.0 / 448
                values[:, 0] /= self.k_scale
                values[:, 1] /= self.v_scale
            pool = values.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            self.nan = 0x7F
        else:
            pool = values.to(DT[kv])
            self.nan = float("nan")
        # only the sequences' tokens hold values
        keep = torch.zeros(nb, bs, dtype=torch.bool)
        for b, n in enumerate(lens):
            t = torch.arange(n)
            keep[self.tables[b, t // bs].long(), t % bs] = True
        pool = torch.where(keep[:, None, None, None, :, None], pool,
                           torch.full((), self.nan, dtype=pool.dtype))
        if layers > 1:
            other = [i for i in range(layers) if i != layer]
            pool[:, :, other] = self.nan
        self.nb, self.pool = nb, pool.to(device)
        self.tables = self.tables.to(device)
        self.seq_lens = torch.tensor(lens, dtype=torch.int32, device=device)

    def handle(self):
        from paged_kv_cache_215_gb300 import pkv
        geom = pkv.geometry(self.layers, self.hq, self.hkv, self.dim, self.bs, self.nb, self.kv)
        pool = pkv.KVPool(geom, storage=self.pool.view(torch.uint8).view(-1))
        if self.block_scales is not None:
            pool.set_block_scales(self.block_scales)
        return pool

    def hide(self, b, lo, hi=None):
        """NaN in the sequence's slots [lo, hi), as if another had reused them."""
        t = torch.arange(lo, self.lens[b] if hi is None else hi, device=self.tables.device)
        t = t[self.tables[b].long()[t // self.bs] >= 0]      # entries may be stale already
        self.pool[self.tables[b].long()[t // self.bs], :, self.layer, :, t % self.bs] = self.nan

    def kv_of(self, b):
        """K and V of the sequence's tokens in 64 bits: [n, hkv, dim] each."""
        t = torch.arange(self.lens[b], device=self.tables.device)
        block = self.tables[b].long()[t // self.bs]
        out = []
        for i, scale in ((0, self.k_scale), (1, self.v_scale)):
            x = self.pool[block, i, self.layer, :, t % self.bs]
            x = x.view(torch.float8_e4m3fn).double() if self.kv == "e4m3" else x.double()
            if self.block_scales is not None:
                x = x * self.block_scales[block, i, self.layer].double()[..., None]
            else:
                x = x * scale
            out.append(x.cpu())
        return out

    def ranges(self, b, window=0, prefix=0, docs=None):
        """[(lo, hi)] of each query token."""
        n, rows = self.lens[b], []
        for i in range(self.q_len):
            p = n - self.q_len + i
            if p < 0:
                rows.append((0, 0))
                continue
            lo = max(0, p - window + 1 if window else 0, docs[b][i] if docs else 0)
            rows.append((lo, max(p + 1, min(prefix, n))))
        return rows

    def reference(self, cap=0.0, window=0, slopes=None, prefix=None, docs=None, scale=None):
        """Per sequence (out, bound, weights, weight bound) in 64 bits: [q_len, hq, dim],
        [hkv, n]."""
        scale = self.scale if scale is None else scale
        g = self.hq // self.hkv
        result = []
        for b, n in enumerate(self.lens):
            out = torch.zeros(self.q_len, self.hq, self.dim, dtype=torch.float64)
            bound = torch.zeros_like(out)
            w_sum = torch.zeros(self.hkv, n, dtype=torch.float64)
            w_err = torch.zeros_like(w_sum)
            k, v = self.kv_of(b)
            for i, (lo, hi) in enumerate(self.ranges(b, window, prefix[b] if prefix else 0, docs)):
                if lo >= hi:
                    continue
                p = n - self.q_len + i
                far = (p - torch.arange(lo, hi)).abs().double()
                for h in range(self.hq):
                    q = self.q[b, i, h].double().cpu()
                    kk, vv = k[lo:hi, h // g], v[lo:hi, h // g]
                    x = kk @ q * scale
                    # 128 products summed in 32 bits, 16 at a time and truncated: each of
                    # 8 x 17 additions off by 2^-23 of the sum of magnitudes
                    size = (kk.abs() @ q.abs()).max() * abs(scale)
                    if cap:
                        x = cap * torch.tanh(x / cap)
                    if slopes is not None:
                        x = x - float(slopes[h]) * far
                    lse = torch.logsumexp(x, 0)
                    w = torch.exp(x - lse)
                    # scores in 32 bits: the sum above, tanh within 2^-22, and roundings of
                    # values as large as the ones that count (and as their log-sum-exp)
                    counts = x[w > 1e-30]
                    large = max(float(counts.abs().max()), abs(float(lse)))
                    if slopes is not None:
                        large += float((abs(float(slopes[h])) * far[w > 1e-30]).max())
                    eps = 2.0 ** -16 * float(size) + 2.0 ** -20 * (large + 1.0)
                    # scores off by eps: each weight, normalised, by a factor within
                    # e^(2 eps) either way
                    off = math.expm1(2 * eps)
                    mass = w @ vv.abs()
                    steps = 2.0 ** -23 * ((hi - lo) / 8 + 64)
                    out[i, h] = w @ vv
                    bound[i, h] = (off + P_ROUND[self.kv] + steps) * mass + 1e-30
                    w_sum[h // g, lo:hi] += w
                    w_err[h // g, lo:hi] += off * w + 1e-30
            result.append((out, bound, w_sum, w_err))
        return result

    def check(self, out, want, weights=None, before=None):
        """out [B, q_len, hq, dim] (or [B, hq, dim]) and weights [B, hkv, width] against
        `want`; returns the largest error over its bound."""
        worst = 0.0
        half = torch.finfo(out.dtype).eps / 2
        got = out.double().cpu().view(self.batch, self.q_len, self.hq, self.dim)
        for b, (o, bound, w, w_err) in enumerate(want):
            limit = bound + half * (o.abs() + bound)
            if out.dtype == torch.float16:
                limit = limit + 2.0 ** -25                 # subnormal results
            err = (got[b] - o).abs()
            assert torch.isfinite(got[b]).all(), f"sequence {b}: non-finite output"
            nothing = bound.amax(-1) == 0
            assert (got[b][nothing] == 0).all(), f"sequence {b}: a query that sees nothing"
            live = ~nothing
            if live.any():
                worst = max(worst, float((err / limit.clamp(min=1e-300))[live].max()))
            assert (err <= limit).all(), f"sequence {b}: off by {float((err - limit).max())}"
            if weights is not None:
                n = self.lens[b]
                old = before[b, :, :n].double().cpu() if before is not None else torch.zeros_like(w)
                total = old + w
                g = self.hq // self.hkv * self.q_len
                limit = w_err + 2.0 ** -23 * (g + 1) * total.abs() + 1e-30
                err = (weights[b, :, :n].double().cpu() - total).abs()
                assert (err <= limit).all(), \
                    f"sequence {b}: weights off by {float((err / limit).max())} bounds"
                if n:
                    worst = max(worst, float((err / limit).max()))
        return worst


def slopes(hq):
    """The usual distance biases: a geometric series of slopes."""
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / hq) for h in range(hq)])


def evicted(weights, n, keep, recent):
    """Slots that stay of a row's n tokens, in order."""
    k = min(n, keep)
    r = min(recent, k)
    w = [x if x > 0 and not math.isnan(x) else 0.0 for x in weights[:n - r].tolist()]
    heavy = sorted(range(n - r), key=lambda j: (-w[j], j))[:k - r]
    return sorted(heavy) + list(range(n - r, n))
