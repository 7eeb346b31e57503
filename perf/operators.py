"""The operators around the paged attention that turn a step's projections into
cached, rotated tokens and a step's probabilities into tokens: what is measured.

    rotate   rotary positions of queries and keys (and the gradients of it)
    append   the same rotation fused with the store of k and v into the paged pool
    verify   drafted tokens checked against the target's probabilities

``listed()`` gives the cases, ``prepare`` what a serving program has in hand
before the call, ``run`` one call.  With ``own`` false, ``run`` computes the
operator in elementary torch operations; with ``own`` true it calls the library.

Formulas.  Rotary pair i of a row at position p turns by the angle p * f_i:
    (a, b) -> m * (a cos - b sin, a sin + b cos)
with (a, b) = (x[i], x[i + r/2]) in the half layout and (x[2i], x[2i+1]) in the
interleaved one, r the rotated part of the head; f_i = base^(-2i/r), scaled for
long contexts (``_scaled_frequencies``); m = 1 except with "yarn".  The gradient
turns by -p * f_i.  Verification accepts draft j of a sequence while
u_j q_j(x_j) < p_j(x_j); the next token is the lowest i whose running sum of
w exceeds u * sum(w), with w = max(p - q, 0) at the first refused draft, or
w = p behind the last one when all were accepted.
"""
import math

import numpy as np
import torch

own = False

_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_BYTES = {"f32": 4, "f16": 2, "bf16": 2, "e4m3": 1}
BASE = 10000.0


# ---------------------------------------------------------------- cases

def _rotate_case(name, tokens, hq, hkv, dim, rotary, dtype, layout, scaling, factor, packed,
                 backward, first):
    return {"name": name, "op": "rotate", "tokens": tokens, "hq": hq, "hkv": hkv, "dim": dim,
            "rotary": rotary, "dtype": dtype, "interleaved": layout == "interleaved",
            "scaling": scaling, "factor": factor, "packed": packed, "backward": backward,
            "first": first}


def _append_case(name, batch, new, prefix, hq, hkv, dim, rotary, dtype, kv, bs, layout, scaling,
                 factor):
    return {"name": name, "op": "append", "batch": batch, "new": new, "prefix": prefix, "hq": hq,
            "hkv": hkv, "dim": dim, "rotary": rotary, "dtype": dtype, "kv": kv, "bs": bs,
            "interleaved": layout == "interleaved", "scaling": scaling, "factor": factor}


def _verify_case(name, batch, drafts, vocab, one_hot, ragged):
    return {"name": name, "op": "verify", "batch": batch, "drafts": drafts, "vocab": vocab,
            "one_hot": one_hot, "ragged": ragged}


def listed():
    return [
        # a decode step of eight requests far into a long context
        _rotate_case("rotate_decode_8", 8, 32, 8, 128, 128, "bf16", "half", "yarn", 8.0, True,
                     False, 120000),
        # a prompt of 8K tokens, q and k as views of the projections' joint output
        _rotate_case("rotate_prompt_8k", 8192, 32, 8, 128, 128, "bf16", "half", "ntk", 4.0, True,
                     False, 0),
        # gradients of a training batch in 32 bits
        _rotate_case("rotate_backward_f32", 4099, 16, 4, 64, 64, "f32", "interleaved", "none",
                     1.0, False, True, 0),
        # a quarter of an odd-sized head rotated, positions near a million
        _rotate_case("rotate_partial_f16", 1003, 7, 1, 80, 20, "f16", "interleaved", "linear",
                     8.0, False, False, 1000000),
        # the latency of one request's decode step
        _append_case("append_decode_1", 1, 1, 2000, 64, 8, 128, 128, "bf16", "bf16", 16, "half",
                     "none", 1.0),
        # a decode step of 32 requests over one shared document
        _append_case("append_decode_32", 32, 1, 8192, 32, 8, 128, 128, "bf16", "bf16", 16, "half",
                     "ntk", 4.0),
        # 64 requests with a token and three drafts each, 8-bit cache
        _append_case("append_drafts_e4m3", 64, 4, 1024, 64, 8, 128, 128, "bf16", "e4m3", 32,
                     "half", "yarn", 4.0),
        # a chunk of five requests' prompts, half of each head rotated
        _append_case("append_chunk_f16", 5, 1001, 37, 16, 2, 96, 48, "f16", "f16", 16,
                     "interleaved", "linear", 2.0),
        # prompts of 16K tokens in all
        _append_case("append_prompt_16k", 4, 4096, 0, 64, 8, 128, 128, "bf16", "bf16", 16, "half",
                     "none", 1.0),
        # one request, four drafts
        _verify_case("verify_1", 1, 4, 131072, False, False),
        # a batch with different numbers of drafts, rows of odd length
        _verify_case("verify_32_ragged", 32, 5, 131071, False, True),
        # drafts looked up in the prompt: no draft probabilities
        _verify_case("verify_128_lookup", 128, 3, 32768, True, False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotate", "append", "verify"])
    layout = rng.choice(["half", "interleaved"])
    scaling = rng.choice(["none", "linear", "ntk", "yarn"])
    factor = 1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0])
    if op == "verify":
        vocab = _log_int(rng, 1000, 131072)
        batch = min(_log_int(rng, 1, 256), 4194304 // vocab)
        c = _verify_case("", batch, rng.randint(1, 8), vocab, rng.random() < 0.3,
                         rng.random() < 0.5)
    else:
        hq, hkv = rng.choice([(32, 8), (64, 8), (16, 2), (8, 8), (4, 2), (7, 1)])
        dim = rng.choice([64, 80, 96, 128, 256])
        rotary = rng.choice([dim, dim, dim // 2, dim // 4])
        if op == "rotate":
            most = max(1, 8192 * 48 * 128 // ((hq + 2 * hkv) * dim * 2))
            c = _rotate_case("", _log_int(rng, 1, most), hq, hkv, dim, rotary,
                             rng.choice(["f32", "f16", "bf16"]), layout, scaling, factor,
                             rng.random() < 0.5, rng.random() < 0.3, _log_int(rng, 1, 1000000))
        else:
            kv = rng.choice(["bf16", "f16", "f32", "e4m3"])
            batch = _log_int(rng, 1, 64)
            most = max(1, 8192 * 48 * 128 // ((hq + 2 * hkv) * dim * 2 * batch))
            c = _append_case("", batch, _log_int(rng, 1, most), _log_int(rng, 1, 8192), hq, hkv,
                             dim, rotary, "bf16" if kv == "e4m3" else kv, kv,
                             rng.choice([16, 32, 64]), layout, scaling, factor)
    del c["name"]
    return c


# ---------------------------------------------------------------- inputs

ORIGINAL = 16384      # positions of training, which the scalings stretch


def _scaled_frequencies(rotary, scaling, factor):
    """(f [r/2], m) as a float64 array and a number."""
    i = np.arange(0, rotary, 2, dtype=np.float64) / rotary
    if scaling == "ntk" and rotary > 2:
        return (BASE * factor ** (rotary / (rotary - 2))) ** -i, 1.0
    f = BASE ** -i
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "yarn":
        turns = ORIGINAL * f / (2 * np.pi)
        keep = np.clip((turns - 1.0) / (32.0 - 1.0), 0.0, 1.0)
        return f / factor * (1 - keep) + f * keep, 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _normal(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda").to(dtype)


def _rows(gen, tokens, heads, dim, dtype, packed):
    """q, k (and v) as views of one projection's output, or as tensors of their own."""
    if packed:
        x = _normal(gen, (tokens, sum(heads) * dim), dtype)
        return [t.view(tokens, -1, dim) for t in x.split([h * dim for h in heads], dim=1)]
    return [_normal(gen, (tokens, h, dim), dtype) for h in heads]


def _rope(case):
    from paged_kv_cache_215_gb300 import pkv
    return pkv.Rope(case["rotary"], base=BASE, interleaved=case["interleaved"],
                    scaling=case["scaling"], factor=case["factor"], original_positions=ORIGINAL)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    if case["op"] == "verify":
        b, n, v = case["batch"], case["drafts"], case["vocab"]
        logits = 2.0 * torch.randn(b, n + 1, v, generator=gen, device="cuda")
        s["target"] = torch.softmax(logits, -1)
        if case["one_hot"]:
            s["draft"], source = None, s["target"][:, :n]
        else:
            logits = logits[:, :n] + 0.5 * torch.randn(b, n, v, generator=gen, device="cuda")
            s["draft"] = source = torch.softmax(logits, -1)
        s["tokens"] = torch.multinomial(source.reshape(b * n, v), 1, generator=gen).view(
            b, n).to(torch.int32)
        if case["one_hot"]:       # a lookup hits the likeliest token about half of the time
            hit = torch.rand(b, n, generator=gen, device="cuda") < 0.5
            s["tokens"] = torch.where(hit, source.argmax(-1).to(torch.int32), s["tokens"])
        s["u_accept"] = torch.rand(b, n, generator=gen, device="cuda")
        s["u_sample"] = torch.rand(b, generator=gen, device="cuda")
        s["count"] = torch.randint(0, n + 1, (b,), generator=gen, device="cuda").to(
            torch.int32) if case["ragged"] else None
        s["out"] = torch.empty(b, n + 1, dtype=torch.int32, device="cuda")
        s["accepted"] = torch.empty(b, dtype=torch.int32, device="cuda")
        return s
    dtype, hq, hkv, dim = _DT[case["dtype"]], case["hq"], case["hkv"], case["dim"]
    f, s["m"] = _scaled_frequencies(case["rotary"], case["scaling"], case["factor"])
    s["f"] = torch.from_numpy(f).cuda()
    if own:
        s["rope"] = _rope(case)
    if case["op"] == "rotate":
        n = case["tokens"]
        heads = [hq, hkv, hkv] if case["packed"] else [hq, hkv]
        s["q"], s["k"] = _rows(gen, n, heads, dim, dtype, case["packed"])[:2]
        s["positions"] = (torch.arange(n, device="cuda") + case["first"]).to(torch.int32)
        s["q_out"] = torch.empty(n, hq, dim, dtype=dtype, device="cuda")
        s["k_out"] = torch.empty(n, hkv, dim, dtype=dtype, device="cuda")
        return s
    b, new, bs = case["batch"], case["new"], case["bs"]
    s["q"], s["k"], s["v"] = _rows(gen, b * new, [hq, hkv, hkv], dim, dtype, True)
    # every sequence shares the blocks of one document, then has blocks of its own
    shared = case["prefix"] // bs
    private = -(-(case["prefix"] % bs + new) // bs)
    blocks = shared + b * private
    ids = torch.randperm(blocks, generator=gen, device="cuda").to(torch.int32)
    s["tables"] = torch.cat([ids[:shared].expand(b, shared), ids[shared:].view(b, private)],
                            1).contiguous()
    tok = torch.arange(b * new, device="cuda")
    s["seq_ids"] = (tok // new).to(torch.int32)
    s["positions"] = (case["prefix"] + tok % new).to(torch.int32)
    s["q_out"] = torch.empty(b * new, hq, dim, dtype=dtype, device="cuda")
    shape = (blocks, 2, 1, hkv, bs, dim)
    pool = _normal(gen, shape, torch.float32)
    s["scales"] = (6.0 / 448, 5.0 / 448) if case["kv"] == "e4m3" else (1.0, 1.0)
    pool = (pool * 100).clamp(-448, 448).to(torch.float8_e4m3fn) if case["kv"] == "e4m3" else \
        pool.to(dtype)
    s["pool"] = pool
    if own:
        from paged_kv_cache_215_gb300 import pkv
        geom = pkv.geometry(1, hq, hkv, dim, bs, blocks, case["kv"])
        s["handle"] = pkv.KVPool(geom, storage=pool.view(torch.uint8).view(-1))
    return s


# ---------------------------------------------------------------- one pass

def _turn(x, positions, f, m, rotary, interleaved, backward=False):
    angle = positions.double()[:, None] * f
    cos = (m * angle.cos()).float()[:, None, :]
    sin = (m * angle.sin()).float()[:, None, :]
    if backward:
        sin = -sin
    x = x.float()
    r = x[..., :rotary]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else r.chunk(2, -1)
    a, b = a * cos - b * sin, a * sin + b * cos
    r = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([r, x[..., rotary:]], -1)


def _encode(x, scale):
    return (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn)


def run(s):
    return {"rotate": _run_rotate, "append": _run_append, "verify": _run_verify}[
        s["case"]["op"]](s)


def _run_rotate(s):
    c = s["case"]
    if own:
        from paged_kv_cache_215_gb300 import pkv
        return pkv.rope_apply(s["q_out"], s["q"], s["positions"], s["rope"], k_out=s["k_out"],
                              k=s["k"], backward=c["backward"])
    how = (s["positions"], s["f"], s["m"], c["rotary"], c["interleaved"], c["backward"])
    return _turn(s["q"], *how).to(s["q"].dtype), _turn(s["k"], *how).to(s["k"].dtype)


def _run_append(s):
    c = s["case"]
    if own:
        s["handle"].append_rope(0, s["q_out"], s["q"], s["k"], s["v"], s["rope"], s["tables"],
                                s["positions"], seq_ids=s["seq_ids"], k_scale=s["scales"][0],
                                v_scale=s["scales"][1])
        return s["q_out"], s["pool"]
    how = (s["positions"], s["f"], s["m"], c["rotary"], c["interleaved"])
    q = _turn(s["q"], *how).to(s["q"].dtype)
    k, v, pool = _turn(s["k"], *how), s["v"], s["pool"]
    if c["kv"] == "e4m3":
        k = _encode(k, s["scales"][0]).view(torch.uint8)
        v = _encode(v.float(), s["scales"][1]).view(torch.uint8)
        pool = pool.view(torch.uint8)
    at = s["positions"].long()
    block = s["tables"][s["seq_ids"].long(), at // c["bs"]].long()
    pool[block, 0, 0, :, at % c["bs"]] = k.to(pool.dtype)
    pool[block, 1, 0, :, at % c["bs"]] = v.to(pool.dtype)
    return q, s["pool"]


def _run_verify(s):
    if own:
        from paged_kv_cache_215_gb300 import pkv
        return pkv.verify_drafts(s["out"], s["accepted"], s["target"], s["draft"], s["tokens"],
                                 s["u_accept"], s["u_sample"], num_drafts=s["count"])
    target, draft, tokens = s["target"], s["draft"], s["tokens"].long()
    b, n = tokens.shape
    seq, at = torch.arange(b, device="cuda"), torch.arange(n, device="cuda")
    count = s["count"].long() if s["count"] is not None else torch.full_like(seq, n)
    p = target[:, :n].gather(2, tokens[..., None])[..., 0].double()
    q = torch.ones_like(p) if draft is None else \
        draft.gather(2, tokens[..., None])[..., 0].double()
    ok = (s["u_accept"].double() * q < p) & (at < count[:, None])
    accepted = ok.long().cumprod(1).sum(1)
    refused = accepted < count
    last = accepted.clamp(max=n - 1)
    row = target[seq, accepted].double()
    if draft is None:
        w = row.scatter(1, tokens[seq, last][:, None], 0.0)
    else:
        w = (row - draft[seq, last].double()).clamp(min=0)
    w = torch.where(refused[:, None] & (w.sum(1) > 0)[:, None], w, row)
    total = w.cumsum(1)
    new = (total <= s["u_sample"].double()[:, None] * total[:, -1:]).sum(1)
    new = new.clamp(max=target.shape[2] - 1)
    steps = torch.arange(n + 1, device="cuda")
    out = torch.cat([tokens, tokens[:, :1]], 1)
    out = torch.where(steps < accepted[:, None], out, -1)
    out = torch.where(steps == accepted[:, None], new[:, None], out)
    return out.to(torch.int32), accepted.to(torch.int32)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    if case["op"] == "verify":
        # one row of the target for each sequence, and the draft's row beside it where a
        # draft was refused (about half of them)
        b, n, v = case["batch"], case["drafts"], case["vocab"]
        rows = 1.0 if case["one_hot"] else 1.5
        return {"bytes": b * (4 * v * rows + 16 * n + 4 * (n + 1) + 12), "flops": 3 * b * v}
    hq, hkv, dim, e = case["hq"], case["hkv"], case["dim"], _BYTES[case["dtype"]]
    if case["op"] == "rotate":
        n = case["tokens"]
        return {"bytes": n * (2 * (hq + hkv) * dim * e + 4) + 4 * case["rotary"],
                "flops": 3 * n * (hq + hkv) * case["rotary"]}
    n = case["batch"] * case["new"]
    return {"bytes": n * (2 * hq * dim * e + 2 * hkv * dim * (e + _BYTES[case["kv"]]) + 12)
            + 4 * case["rotary"],
            "flops": 3 * n * (hq + hkv) * case["rotary"]}


# ---------------------------------------------------------------- in 64 bits

def _exact_turn(x, positions, case, sign=1.0):
    """Each pair as a complex number, multiplied by m * exp(i angle)."""
    r, t, factor = case["rotary"], case["scaling"], case["factor"]
    speeds, m = [], 1.0
    for i in range(r // 2):
        base = BASE * factor ** (r / (r - 2)) if t == "ntk" and r > 2 else BASE
        speed = base ** (-2.0 * i / r)
        if t == "linear":
            speed = speed / factor
        if t == "yarn":
            m = 1.0 + math.log(factor) / 10
            ramp = min(max((ORIGINAL * speed / math.tau - 1.0) / 31.0, 0.0), 1.0)
            speed = speed * (ramp + (1.0 - ramp) / factor)
        speeds.append(speed)
    angle = positions.double()[:, None] * torch.tensor(speeds, dtype=torch.float64, device="cuda")
    factor = torch.polar(torch.full_like(angle, m), sign * angle)[:, None]
    out = x.double().clone()
    first = slice(0, r, 2) if case["interleaved"] else slice(0, r // 2)
    second = slice(1, r, 2) if case["interleaved"] else slice(r // 2, r)
    z = torch.complex(out[..., first].contiguous(), out[..., second].contiguous()) * factor
    out[..., first], out[..., second] = z.real, z.imag
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotate":
        sign = -1.0 if case["backward"] else 1.0
        return tuple(_exact_turn(s[x], s["positions"], case, sign) for x in ("q", "k"))
    if case["op"] == "append":
        pool, bs = s["pool"].double(), case["bs"]
        at = s["positions"].long()
        page = s["tables"][s["seq_ids"].long()].gather(1, (at // bs)[:, None])[:, 0].long()
        kv = torch.stack([_exact_turn(s["k"], s["positions"], case) / s["scales"][0],
                          s["v"].double() / s["scales"][1]], 1)
        if case["kv"] == "e4m3":
            kv = kv.clamp(-448, 448)
        # [blocks, slots, ...]: a token's slot is one row
        rows = pool.permute(0, 4, 1, 2, 3, 5).reshape(-1, 2, 1, case["hkv"], case["dim"])
        rows[page * bs + at % bs] = kv[:, :, None]
        pool = rows.view(-1, bs, 2, 1, case["hkv"], case["dim"]).permute(0, 2, 3, 4, 1, 5)
        return _exact_turn(s["q"], s["positions"], case), pool.contiguous()
    b, n = case["batch"], case["drafts"]
    tokens, count = s["tokens"].tolist(), s["count"].tolist() if case["ragged"] else [n] * b
    u, last = s["u_accept"].tolist(), s["u_sample"].tolist()
    out, accepted = [], []
    for j in range(b):
        row, k = s["target"][j].double().cpu().numpy(), 0
        other = None if s["draft"] is None else s["draft"][j].double().cpu().numpy()
        while k < count[j] and u[j][k] * (1.0 if other is None else other[k][tokens[j][k]]) < \
                row[k][tokens[j][k]]:
            k += 1
        w = row[k].copy()
        if k < count[j]:
            if other is None:
                w[tokens[j][k]] = 0.0
            else:
                w = np.maximum(w - other[k], 0.0)
            if not w.sum() > 0:
                w = row[k]
        sums = np.cumsum(w)
        new = min(int(np.searchsorted(sums, last[j] * sums[-1], side="right")), len(w) - 1)
        out.append(tokens[j][:k] + [new] + [-1] * (n - k))
        accepted.append(k)
    return (torch.tensor(out, dtype=torch.int32), torch.tensor(accepted, dtype=torch.int32))
