"""Attention with the score rules of released models, the record of where it went,
and the eviction that reads the record: what is measured.

    attend   paged attention with capped scores, a distance bias, a sliding window,
             packed documents or a bidirectional prefix
    weigh    the same, and each cached token's accumulated attention weight
    evict    the heaviest and the most recent tokens of every head copied into fresh
             blocks

``listed()`` gives the cases, ``prepare`` what a serving program has in hand
before the call, ``run`` one call.  With ``own`` false, ``run`` computes the
operator in elementary torch operations; with ``own`` true it calls the library.

Formulas.  Query i of a sequence of n tokens sits at p = n - q_len + i.  It sees key
j if (j <= p or j < prefix) and p - j < window and j >= the start of its document.
A score x = scale <q, k> becomes cap tanh(x / cap), then loses slope |p - j|; softmax
over the visible keys, and the sum of the values.  A token's weight grows by the
softmax weights that the query heads of its KV head gave it.  Eviction keeps the last
``recent`` tokens and the heaviest of the others (the lowest slot first among
equals), in their order.
"""
import math
import random

import torch

own = False

_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_BYTES = {"f32": 4, "f16": 2, "bf16": 2, "e4m3": 1}


# ---------------------------------------------------------------- cases

def _attend(name, batch, q_len, n, hq, hkv, dim, kv, bs, cap=0.0, window=0, alibi=False, prefix=0,
            docs=0, ragged=False, weights=False):
    return {"name": name, "op": "weigh" if weights else "attend", "batch": batch, "q_len": q_len,
            "n": n, "hq": hq, "hkv": hkv, "dim": dim, "kv": kv, "bs": bs, "cap": cap,
            "window": window, "alibi": alibi, "prefix": prefix, "docs": docs, "ragged": ragged}


def _evict(name, batch, n, keep, recent, hkv, dim, kv, bs, ragged=False):
    return {"name": name, "op": "evict", "batch": batch, "n": n, "keep": keep, "recent": recent,
            "hq": hkv, "hkv": hkv, "dim": dim, "kv": kv, "bs": bs, "ragged": ragged}


def listed():
    return [
        # the latency of one request's decode step with capped scores
        _attend("attend_decode_1", 1, 1, 2048, 32, 8, 128, "bf16", 16, cap=50.0),
        # a sliding-window layer of 32 requests far into their contexts
        _attend("attend_window_32", 32, 1, 32768, 32, 8, 128, "bf16", 16, cap=50.0, window=4096),
        # distance biases, a KV head for each query head, ragged lengths
        _attend("attend_alibi_8_f16", 8, 1, 8192, 32, 32, 128, "f16", 32, alibi=True,
                ragged=True),
        # one request of 128K tokens on the 8-bit cache
        _attend("attend_128k_e4m3", 1, 1, 131072, 32, 8, 128, "e4m3", 16, cap=30.0),
        # a token and three drafts of 16 requests, sliding window
        _attend("attend_drafts_16", 16, 4, 8192, 32, 8, 128, "bf16", 32, cap=50.0, window=2048),
        # a chunk of two prompts that pack several documents
        _attend("attend_chunk_docs", 2, 2048, 8192, 32, 8, 128, "bf16", 16, cap=50.0, docs=3000),
        # a sliding-window chunk of four long prompts on the 8-bit cache
        _attend("attend_chunk_window_e4m3", 4, 2048, 16384, 32, 8, 128, "e4m3", 16, window=4096),
        # a whole prompt of odd length whose first part sees itself both ways
        _attend("attend_prefix_f16", 3, 1001, 1001, 64, 8, 128, "f16", 16, prefix=257),
        # a few requests with the record of their weights: latency
        _attend("weigh_decode_4", 4, 1, 2048, 32, 8, 128, "bf16", 16, weights=True),
        # a decode batch with the record, ragged lengths
        _attend("weigh_decode_32", 32, 1, 8192, 32, 8, 128, "bf16", 16, cap=50.0, ragged=True,
                weights=True),
        # 32 requests that have grown past their budget
        _evict("evict_grown_32", 32, 2304, 2048, 256, 8, 128, "bf16", 16),
        # eight long prompts brought down to an eighth, ragged lengths
        _evict("evict_prompt_8", 8, 32768, 4096, 512, 8, 128, "bf16", 16, ragged=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


_HEADS = [(32, 8), (64, 8), (16, 2), (8, 8), (32, 32), (4, 2), (7, 1)]


def draw(rng):
    op = rng.choice(["attend", "attend", "weigh", "evict"])
    hq, hkv = rng.choice(_HEADS)
    kv = rng.choice(["bf16", "f16", "e4m3"])
    bs = rng.choice([16, 32, 64])
    if op == "evict":
        batch = _log_int(rng, 1, 32)
        kv = rng.choice(["bf16", "f16", "e4m3", "f32"])
        n = _log_int(rng, 16, min(131072, 1048576 // (batch * hkv * _BYTES[kv])))
        keep = max(1, int(n * rng.uniform(0.05, 0.9)))
        case = _evict("", batch, n, keep, rng.randint(0, keep), hkv, rng.choice([64, 128]), kv, bs,
                      rng.random() < 0.5)
        del case["name"]
        return case
    rules = dict(cap=rng.choice([0.0, 30.0, 50.0]), window=0, alibi=rng.random() < 0.25)
    if rng.random() < 0.4:
        rules["window"] = _log_int(rng, 16, 8192)
    dim = 128
    if op == "attend" and hq != 7 and rng.random() < 0.35:       # chunks
        q_len = _log_int(rng, 33, 2048)
        batch = rng.randint(1, max(1, min(4, 4096 // q_len)))
        n = q_len + rng.choice([0, _log_int(rng, 1, 8192)])
        rule = rng.choice(["none", "docs", "prefix"])
        if rule == "docs":
            rules["docs"] = _log_int(rng, 16, n)
        if rule == "prefix":
            rules["prefix"] = rng.randint(1, n)
    else:
        q_len = rng.choice([1, 1, 1, rng.randint(2, 5)])
        most = 8 if bs == 64 else 16
        if q_len * (hq // hkv) > most:
            q_len = 1
        if q_len == 1 and rng.random() < 0.15:
            dim = 64
        batch = _log_int(rng, 1, 32)
        n = q_len + _log_int(rng, 1, min(131072, 1048576 // (batch * hkv)))
        if rng.random() < 0.2:
            rules["docs"] = _log_int(rng, 16, n)
    case = _attend("", batch, q_len, n, hq, hkv, dim, kv, bs, ragged=rng.random() < 0.5,
                   weights=op == "weigh", **rules)
    del case["name"]
    return case


# ---------------------------------------------------------------- what a case fixes

def _lengths(case):
    n, least = case["n"], case.get("q_len", 1)
    if not case["ragged"]:
        return [n] * case["batch"]
    rng = random.Random(f"lengths {n} {case['batch']}")
    return [n] + [rng.randint(max(least, n // 2), n) for _ in range(case["batch"] - 1)]


def _doc_starts(case, lens):
    """The first position of each query token's document: [batch][q_len]."""
    rng = random.Random(f"documents {case['docs']} {lens}")
    rows = []
    for n in lens:
        cuts = [0]
        while cuts[-1] < n:
            cuts.append(cuts[-1] + rng.randint(1, 2 * case["docs"]))
        row, c = [], 0
        for p in range(n - case["q_len"], n):
            while cuts[c + 1] <= p:
                c += 1
            row.append(cuts[c])
        rows.append(row)
    return rows


def _ranges(case):
    """Per sequence the visible keys [lo, hi) of each query token."""
    lens = _lengths(case)
    docs = _doc_starts(case, lens) if case["docs"] else None
    out = []
    for b, n in enumerate(lens):
        row = []
        for i in range(case["q_len"]):
            p = n - case["q_len"] + i
            lo = max(0, p - case["window"] + 1) if case["window"] else 0
            if docs:
                lo = max(lo, docs[b][i])
            row.append((lo, max(p + 1, min(case["prefix"], n))))
        out.append(row)
    return out


# ---------------------------------------------------------------- inputs

def _normal(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda").to(dtype)


def _pool(gen, blocks, case):
    """Cached keys and values [blocks, 2, 1, hkv, bs, dim], one key in a hundred four
    times as large (tokens that draw the attention)."""
    shape = (blocks, 2, 1, case["hkv"], case["bs"], case["dim"])
    dtype = _DT.get(case["kv"], torch.bfloat16)
    pool = torch.empty(shape, dtype=torch.float8_e4m3fn if case["kv"] == "e4m3" else dtype,
                       device="cuda")
    for at in range(0, blocks, 8192):
        part = torch.randn((min(8192, blocks - at),) + shape[1:], generator=gen, device="cuda")
        heavy = torch.rand(part.shape[0], 1, 1, case["bs"], 1, generator=gen, device="cuda") < 0.01
        part[:, 0] *= 1.0 + 3.0 * heavy
        if case["kv"] == "e4m3":
            part[:, 0] /= _SCALES[0]
            part[:, 1] /= _SCALES[1]
            part = part.clamp(-448, 448)
        pool[at:at + part.shape[0]] = part.to(pool.dtype)
    return pool


_SCALES = (24.0 / 448, 6.0 / 448)        # of E4M3 keys and values


def _handle(s):
    from paged_kv_cache_215_gb300 import pkv
    c = s["case"]
    geom = pkv.geometry(1, c["hq"], c["hkv"], c["dim"], c["bs"], s["pool"].shape[0], c["kv"])
    s["handle"] = pkv.KVPool(geom, storage=s["pool"].view(torch.uint8).view(-1))
    return pkv, geom


def _tables(gen, blocks, first, widths):
    """A table of random blocks of [first, first + blocks), one row for each width."""
    ids = (torch.randperm(blocks, generator=gen, device="cuda") + first).to(torch.int32)
    tables = torch.zeros(len(widths), max(widths), dtype=torch.int32, device="cuda")
    at = 0
    for b, w in enumerate(widths):
        tables[b, :w] = ids[at:at + w]
        at += w
    return tables


def _weights(gen, lens, hkv, width):
    """Accumulated weights of some steps: most tokens next to none, a few a lot; coarse,
    so that equal ones occur."""
    w = torch.randn(len(lens), hkv, width, generator=gen, device="cuda").mul_(2.0).exp_()
    w = (w / 64.0).to(torch.bfloat16).float()
    for b, n in enumerate(lens):
        w[b, :, n:] = 0.0
    return w


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    lens, bs = _lengths(case), case["bs"]
    s = {"case": case, "lens": lens}
    s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    widths = [-(-n // bs) for n in lens]
    if case["op"] == "evict":
        kept = [min(n, case["keep"]) for n in lens]
        new = [-(-k // bs) for k in kept]
        s["pool"] = _pool(gen, sum(new) + sum(widths), case)
        s["new_blocks"] = sum(new)
        s["new_tables"] = _tables(gen, sum(new), 0, new)
        s["tables"] = _tables(gen, sum(widths), sum(new), widths)
        s["weights"] = _weights(gen, lens, case["hkv"], case["n"])
        s["keep"] = torch.full((len(lens),), case["keep"], dtype=torch.int32, device="cuda")
        s["new_weights"] = torch.zeros_like(s["weights"])
        s["new_lens"] = torch.zeros_like(s["seq_lens"])
        s["index"] = torch.full((len(lens), case["hkv"], max(kept)), -1, dtype=torch.int32,
                                device="cuda")
        if own:
            pkv, geom = _handle(s)
            s["workspace"] = torch.empty(
                pkv.evict_workspace_bytes(geom, len(lens), case["n"]), dtype=torch.uint8,
                device="cuda")
        return s
    dtype = _DT.get(case["kv"], torch.bfloat16)
    s["pool"] = _pool(gen, sum(widths), case)
    s["tables"] = _tables(gen, sum(widths), 0, widths)
    s["scale"] = case["dim"] ** -0.5
    s["k_scale"], s["v_scale"] = _SCALES if case["kv"] == "e4m3" else (1.0, 1.0)
    shape = (case["batch"], case["q_len"], case["hq"], case["dim"])
    s["q"] = (2.0 * torch.randn(shape, generator=gen, device="cuda")).to(dtype)
    s["out"] = torch.empty_like(s["q"])
    s["slopes"] = s["docs"] = s["prefix"] = s["weights"] = None
    if case["alibi"]:
        s["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / case["hq"])
                                    for h in range(case["hq"])], device="cuda")
    if case["docs"]:
        s["docs"] = torch.tensor(_doc_starts(case, lens), dtype=torch.int32, device="cuda")
    if case["prefix"]:
        s["prefix"] = torch.full((case["batch"],), case["prefix"], dtype=torch.int32,
                                 device="cuda")
    # the first key that a sequence's queries see, on the host and on the device
    s["first"] = [min(lo for lo, _ in row) for row in _ranges(case)]
    s["first_key"] = torch.tensor(s["first"], device="cuda")
    if case["op"] == "weigh":
        s["weights"] = _weights(gen, lens, case["hkv"], case["n"])
        s["new_weights"] = torch.zeros_like(s["weights"])
    if own:
        pkv, geom = _handle(s)
        s["scores"] = pkv.Scores(cap=case["cap"], window=case["window"], slopes=s["slopes"],
                                 prefix_lens=s["prefix"], doc_starts=s["docs"])
        s["workspace"] = torch.empty(
            pkv.scored_workspace_bytes(geom, case["batch"], case["q_len"], case["n"],
                                       weights=case["op"] == "weigh"),
            dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    return _run_evict(s) if s["case"]["op"] == "evict" else _run_attend(s)


def _run_attend(s):
    c = s["case"]
    if own:
        from paged_kv_cache_215_gb300 import pkv
        pkv.paged_decode_attention_scored(
            s["out"], s["q"], s["handle"], 0, s["tables"], s["seq_lens"], c["n"], s["scale"],
            scores=s["scores"], k_scale=s["k_scale"], v_scale=s["v_scale"],
            weights=s["new_weights"] if c["op"] == "weigh" else None, weights_in=s["weights"],
            workspace=s["workspace"])
        return s["out"] if c["op"] == "attend" else (s["out"], s["new_weights"])
    out = torch.empty_like(s["q"])
    new = s["weights"].clone() if c["op"] == "weigh" else None
    g = c["hq"] // c["hkv"]
    span = [n - f for n, f in zip(s["lens"], s["first"])]
    # as many sequences at a time as fit some gigabytes in 32 bits
    per_seq = max(span) * (4 * c["hq"] * c["q_len"] + 2 * c["hkv"] * c["dim"]) * 4
    step = max(1, min(c["batch"], (8 << 30) // per_seq))
    for b0 in range(0, c["batch"], step):
        b1 = min(c["batch"], b0 + step)
        rows = slice(b0, b1)
        n = s["seq_lens"][rows].long()[:, None]
        pos = s["first_key"][rows, None] + torch.arange(max(span[rows]), device="cuda")
        at = torch.minimum(pos, n - 1)
        block = s["tables"][rows].long().gather(1, at // c["bs"])
        k = s["pool"][block, 0, 0, :, at % c["bs"]].float() * s["k_scale"]
        v = s["pool"][block, 1, 0, :, at % c["bs"]].float() * s["v_scale"]
        q = s["q"][rows].float().view(b1 - b0, c["q_len"], c["hkv"], g, c["dim"])
        x = torch.einsum("bqhgd,bkhd->bhgqk", q, k) * s["scale"]
        if c["cap"]:
            x = torch.tanh(x / c["cap"]) * c["cap"]
        p = n - c["q_len"] + torch.arange(c["q_len"], device="cuda")
        back = p[:, :, None] - pos[:, None, :]                       # [b, q, k]
        if s["slopes"] is not None:
            x = x - s["slopes"].view(1, c["hkv"], g, 1, 1) * back.abs()[:, None, None].float()
        ahead = pos < torch.minimum(s["prefix"][rows].long()[:, None], n) \
            if s["prefix"] is not None else torch.zeros_like(pos, dtype=torch.bool)
        seen = ((back >= 0) | ahead[:, None]) & (pos < n)[:, None]
        if c["window"]:
            seen &= back < c["window"]
        if s["docs"] is not None:
            seen &= pos[:, None] >= s["docs"][rows].long()[:, :, None]
        x = x.masked_fill(~seen[:, None, None], -math.inf)
        e = torch.exp(x - x.amax(-1, keepdim=True).clamp(min=-1e30))
        e = e / e.sum(-1, keepdim=True).clamp(min=1e-30)
        o = torch.einsum("bhgqk,bkhd->bqhgd", e, v)
        out[rows] = o.reshape(b1 - b0, c["q_len"], c["hq"], c["dim"]).to(out.dtype)
        if new is not None:
            w = e.sum((2, 3)) * (pos < n)[:, None]
            new[rows].scatter_add_(2, at[:, None].expand_as(w), w)
    return out if new is None else (out, new)


def _run_evict(s):
    c = s["case"]
    if own:
        s["handle"].evict(0, s["new_tables"], s["tables"], s["seq_lens"], c["n"], s["keep"],
                          c["recent"], s["weights"], s["new_weights"], s["new_lens"],
                          index=s["index"], workspace=s["workspace"])
        return s["new_lens"], s["index"], s["new_weights"], s["pool"][:s["new_blocks"]]
    n = s["seq_lens"].long()
    kept = torch.minimum(n, s["keep"].long())
    recent = kept.clamp(max=c["recent"])
    slot = torch.arange(c["n"], device="cuda")
    w = s["weights"]
    key = torch.where(w > 0, w, torch.zeros_like(w))
    last = (slot >= (n - recent)[:, None]) & (slot < n[:, None])
    key = key.masked_fill(last[:, None], math.inf).masked_fill((slot >= n[:, None])[:, None], -1.0)
    order = torch.sort(key, dim=2, descending=True, stable=True).indices
    rank = torch.arange(c["n"], device="cuda")
    picked = order.masked_fill((rank >= kept[:, None])[:, None], c["n"])
    index = torch.sort(picked, dim=2).values[:, :, :s["index"].shape[2]]
    live = (rank[:index.shape[2]] < kept[:, None])[:, None].expand_as(index)
    from_slot = index.clamp(max=c["n"] - 1)
    new_weights = torch.zeros_like(w)
    new_weights[:, :, :index.shape[2]] = torch.where(live, w.gather(2, from_slot),
                                                     torch.zeros_like(index, dtype=w.dtype))
    b, h, t = live.nonzero(as_tuple=True)
    j = from_slot[b, h, t]
    src, dst = s["tables"].long()[b, j // c["bs"]], s["new_tables"].long()[b, t // c["bs"]]
    pool = s["pool"].view(torch.uint8) if c["kv"] == "e4m3" else s["pool"]
    for kv in (0, 1):
        pool[dst, kv, 0, h, t % c["bs"]] = pool[src, kv, 0, h, j % c["bs"]]
    return (kept.to(torch.int32), torch.where(live, index, -torch.ones_like(index)).to(torch.int32),
            new_weights, s["pool"][:s["new_blocks"]])


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    lens = _lengths(case)
    row = case["hkv"] * case["dim"] * _BYTES[case["kv"]]          # K (or V) of a token
    if case["op"] == "evict":
        kept = [min(n, case["keep"]) for n in lens]
        return {"bytes": 4 * case["hkv"] * (sum(lens) + case["n"] * len(lens) + sum(kept))
                + 4 * row * sum(kept) + 4 * sum(-(-n // case["bs"]) for n in lens + kept)
                + 12 * len(lens),
                "flops": case["hkv"] * sum(lens)}
    ranges = _ranges(case)
    tokens = sum(max(hi for _, hi in r) - min(lo for lo, _ in r) for r in ranges)
    pairs = sum(hi - lo for r in ranges for lo, hi in r)
    act = 4 if case["kv"] == "f32" else 2
    need = 2 * row * tokens + 4 * tokens // case["bs"] + 4 * len(lens) \
        + 2 * act * case["batch"] * case["q_len"] * case["hq"] * case["dim"]
    if case["docs"]:
        need += 4 * case["batch"] * case["q_len"]
    if case["op"] == "weigh":
        need += 8 * case["hkv"] * sum(lens)
    return {"bytes": need, "flops": 4 * case["dim"] * case["hq"] * pairs}


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    return _exact_evict(prepare(case, seed)) if case["op"] == "evict" else \
        _exact_attend(prepare(case, seed))


def _exact_attend(s):
    """Sequence by sequence and head by head, from the visible ranges."""
    c, bs = s["case"], s["case"]["bs"]
    g = c["hq"] // c["hkv"]
    ranges = torch.tensor(_ranges(c), device="cuda")                 # [b, q, 2]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    weights = s["weights"].double() if c["op"] == "weigh" else None
    for b, n in enumerate(s["lens"]):
        f = s["first"][b]
        slot = torch.arange(f, n, device="cuda")
        block, off = s["tables"][b].long()[slot // bs], slot % bs
        lo, hi = ranges[b, :, :1], ranges[b, :, 1:]
        hidden = (slot < lo) | (slot >= hi)                          # [q, k]
        at = torch.arange(n - c["q_len"], n, device="cuda")[:, None]
        far = (at - slot).abs().double()
        for h in range(c["hq"]):
            kv = h // g
            k = s["pool"][block, 0, 0, kv, off].double() * s["k_scale"]
            v = s["pool"][block, 1, 0, kv, off].double() * s["v_scale"]
            x = s["q"][b, :, h].double() @ k.T * s["scale"]
            if c["cap"]:
                x = c["cap"] * torch.tanh(x / c["cap"])
            if c["alibi"]:
                x = x - float(s["slopes"][h].item()) * far
            x = torch.where(hidden, -math.inf, x)
            total = torch.logsumexp(x, 1, keepdim=True)
            w = torch.where(hidden, 0.0, torch.exp(x - torch.where(total > -math.inf, total, 0.0)))
            out[b, :, h] = w @ v
            if weights is not None:
                weights[b, kv, f:n] += w.sum(0)
    return out if weights is None else (out, weights)


def _exact_evict(s):
    """On the host, row by row."""
    c, bs = s["case"], s["case"]["bs"]
    pool = s["pool"][:s["new_blocks"]].double().cpu()
    tables, fresh = s["tables"].cpu().long(), s["new_tables"].cpu().long()
    old = (s["pool"].view(torch.uint8) if c["kv"] == "e4m3" else s["pool"]).cpu()
    w = s["weights"].cpu()
    index = torch.full(s["index"].shape, -1, dtype=torch.int32)
    weights = torch.zeros(w.shape, dtype=torch.float64)
    lens = []
    for b, n in enumerate(s["lens"]):
        k = min(n, c["keep"])
        r = min(k, c["recent"])
        lens.append(k)
        t = torch.arange(k)
        for h in range(c["hkv"]):
            others = w[b, h, :n - r].tolist()
            heavy = sorted(range(n - r), key=lambda j: (-others[j], j))[:k - r]
            j = torch.tensor(sorted(heavy) + list(range(n - r, n)), dtype=torch.long)
            index[b, h, :k] = j.int()
            weights[b, h, :k] = w[b, h, j].double()
            for kv in (0, 1):
                rows = old[tables[b, j // bs], kv, 0, h, j % bs].view(s["pool"].dtype)
                pool[fresh[b, t // bs], kv, 0, h, t % bs] = rows.double()
    return torch.tensor(lens, dtype=torch.int32), index, weights, pool
