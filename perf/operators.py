"""Cases and plain forms of the serving operators around the compressed key/value cache.

Three operators, each computed here in a plain form (elementary torch operations in 32 bits) or, where ``own`` is
true, by the library's own calls:

* ``rope``    rotary positions on the query and key heads of a fused projection;
* ``cache``   new keys and values written to a paged compressed cache (rotate, scale by the group's RMS, snap, pack)
              and the context read back (unpack, scale, rotate back);
* ``attend``  attention of a tree of drafted tokens: every sequence's compressed context out of its pages, and the
              drafted tokens themselves through an ancestor mask.

Head length 128, 32 query over 8 key/value heads, groups of 32, 8-bit keys with 3-bit values and 131072 cached tokens
are the sizes of the library's own cache workload; the rest spreads around them.
"""
from __future__ import annotations

import functools
import math

import numpy as np
import torch

own = False

D = 128  # head length of the cache


# ---------------------------------------------------------------- cases

def _rope(name, tokens, hq, hkv, dim, rotary, layout, dtype, scaling="none", base=10000.0, start=0, inverse=False):
    return dict(name=name, op="rope", tokens=tokens, hq=hq, hkv=hkv, dim=dim, rotary=rotary, layout=layout, dtype=dtype,
                scaling=scaling, base=base, start=start, inverse=inverse)


def _cache(name, new, history, hkv, klevels, vlevels, group, page, dtype, out, rope=False, dropped=0.0):
    return dict(name=name, op="cache", new=new, history=history, hkv=hkv, klevels=klevels, vlevels=vlevels, group=group,
                page=page, dtype=dtype, out=out, rope=rope, dropped=dropped)


def _attend(name, batch, drafted, hq, hkv, context, klevels=256, vlevels=8, group=32, page=64, ragged=False,
            tree="random"):
    return dict(name=name, op="attend", batch=batch, drafted=drafted, hq=hq, hkv=hkv, context=context, klevels=klevels,
                vlevels=vlevels, group=group, page=page, ragged=ragged, tree=tree)


def listed():
    return [
        # one decode step of 8 sequences deep in their contexts: launch latency is everything
        _rope("rope step", 8, 32, 8, 128, 128, "half", "bfloat16", start=100000),
        # a prompt whose heads rotate their first half only, neighbouring elements paired, 32-bit activations
        _rope("rope prompt partial", 2049, 24, 8, 128, 64, "interleaved", "float32"),
        # a long prompt with frequencies scaled by parts for 131072 positions
        _rope("rope long prompt", 32768, 32, 8, 128, 128, "half", "bfloat16", scaling="parts", base=500000.0),
        # one token joins a short context, which is read back: the smallest update-and-fetch
        _cache("cache step", 1, 99, 8, 256, 8, 32, 16, "bfloat16", "bfloat16"),
        # 13 drafted tokens of which some were rejected, keys rotated on the way, 4-bit books, 32-bit activations
        _cache("cache accepted drafts", 13, 4000, 8, 16, 16, 64, 32, "float32", "float16", rope=True, dropped=0.4),
        # a whole prompt written and read back once
        _cache("cache prompt", 65536, 0, 8, 256, 8, 32, 64, "bfloat16", "bfloat16", rope=True),
        # one token of one sequence over the library's longest cache: plain decoding
        _attend("attend decode 131072", 1, 1, 32, 8, 131072, tree="chain"),
        # four sequences just begun, five drafts each, contexts of 0 to 300 tokens: latency
        _attend("attend short", 4, 5, 32, 8, 300, page=16, ragged=True),
        # a serving batch: 16 sequences of very different lengths, eight drafts each
        _attend("attend batch", 16, 8, 32, 8, 8192, ragged=True),
        # a tree of 16 drafts over a long context
        _attend("attend tree 16", 1, 16, 32, 8, 32768),
        # three query heads to a key/value head, 4-bit keys and values in whole-row groups, odd everything
        _attend("attend odd", 3, 23, 24, 8, 5003, klevels=16, vlevels=16, group=128, page=128, ragged=True),
        # the largest: a tree of 64 drafts over the longest cache, 256 rows to a key/value head
        _attend("attend tree 64", 1, 64, 32, 8, 131072),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "cache", "attend", "attend"])
    if op == "rope":
        hkv = rng.choice([1, 2, 4, 8])
        dim = rng.choice([64, 96, 128, 256])
        rotary = rng.choice([dim, dim, dim // 2, dim // 4])
        per = 2 * dim * (hkv * 5)
        return {k: v for k, v in _rope("", min(_log(rng, 1, 32768), 32768 * 40 * 128 * 2 // per // 2), hkv * 4, hkv, dim, rotary,
                                       rng.choice(["half", "interleaved"]), rng.choice(["bfloat16", "float16", "float32"]),
                                       scaling=rng.choice(["none", "linear", "base", "parts"]),
                                       start=rng.choice([0, _log(rng, 1, 1 << 20)]), inverse=rng.random() < 0.25).items()
                if k != "name"}
    hkv = rng.choice([1, 2, 4, 8])
    klevels, vlevels = rng.choice([(256, 8), (256, 8), (256, 16), (16, 16), (16, 8)])
    group, page = rng.choice([16, 32, 32, 64, 128]), rng.choice([16, 32, 64, 128])
    if op == "cache":
        new = _log(rng, 1, 60000)
        history = rng.choice([0, _log(rng, 1, 65000)])
        history = min(history, 65536 - new)
        rope = rng.random() < 0.5
        return {k: v for k, v in _cache("", new, history, hkv, klevels, vlevels, group, page,
                                        rng.choice(["bfloat16", "bfloat16", "float32"]),
                                        rng.choice(["bfloat16", "float16"]), rope=rope,
                                        dropped=rng.choice([0.0, 0.0, 0.3])).items() if k != "name"}
    ratio = rng.choice([1, 2, 3, 4, 4, 6, 8])
    batch, drafted = _log(rng, 1, 48), rng.choice([1, _log(rng, 2, 64)])
    context = _log(rng, 16, 131072)
    context = max(1, min(context, 131072 * 8 // (batch * hkv), 131072 * 8 * 256 // (batch * hkv * drafted * ratio)))
    return {k: v for k, v in _attend("", batch, drafted, hkv * ratio, hkv, context, klevels, vlevels, group, page,
                                     rng.random() < 0.6, rng.choice(["random", "random", "chain", "bushy"])).items()
            if k != "name"}


# ---------------------------------------------------------------- books, rotation, frequencies (what a model file holds)

@functools.lru_cache(None)
def _book(levels):
    """A Gaussian codebook (centroids, midpoint thresholds), 64-bit numpy: companded start, then Lloyd's iteration."""
    p = (np.arange(levels) + 0.5) / levels
    c = math.sqrt(3.0) * math.sqrt(2.0) * torch.erfinv(torch.from_numpy(2 * p - 1)).numpy()
    for _ in range(200):
        t = np.concatenate(([-40.0], 0.5 * (c[1:] + c[:-1]), [40.0]))
        upper = torch.special.erfc(torch.from_numpy(np.abs(t) / math.sqrt(2.0))).numpy() / 2  # mass beyond |t|
        cdf = np.where(t > 0, 1 - upper, upper)
        mass = np.where(t[:-1] > 0, upper[:-1] - upper[1:], cdf[1:] - cdf[:-1])
        pdf = np.exp(-0.5 * t * t) / math.sqrt(2 * math.pi)
        c = (pdf[:-1] - pdf[1:]) / mass
        c = 0.5 * (c - c[::-1])
    return c, 0.5 * (c[1:] + c[:-1])


@functools.lru_cache(None)
def _signs():
    return np.random.Generator(np.random.PCG64(11)).integers(0, 2, D).astype(np.int8) * 2 - 1


@functools.lru_cache(None)
def _frequencies(rotary, base, scaling):
    """Angle per position of each rotated pair (64-bit), and the factor on the rotated elements.

    linear: positions a quarter as far apart; base: a base that stretches the slowest pair fourfold; parts: pairs that
    turn less than once in 8192 positions slowed sixteenfold, those that turn over 32 times kept, a ramp between."""
    i = np.arange(0, rotary, 2) / rotary
    f = base ** -i
    if scaling == "linear":
        return f / 4.0, 1.0
    if scaling == "base":
        return (base * 4.0 ** (rotary / max(rotary - 2, 1))) ** -i, 1.0
    if scaling == "parts":
        turns = 8192 * f / (2 * math.pi)
        keep = np.clip((turns - 1.0) / (32.0 - 1.0), 0.0, 1.0)
        return f * (keep + (1 - keep) / 16.0), 0.1 * math.log(16.0) + 1.0
    return f, 1.0


def _steps(freq):
    """Phase per position in 2^-64 turns: the product with a position wraps by itself."""
    return np.array([int(f / (2 * math.pi) * 2 ** 64) for f in freq], dtype=np.uint64).view(np.int64)


# ---------------------------------------------------------------- inputs

_DT = {"bfloat16": torch.bfloat16, "float16": torch.float16, "float32": torch.float32}


def _bits(levels):
    return levels.bit_length() - 1


def _per_word(levels):
    return 32 // _bits(levels)


def _words(levels):
    return -(-D // _per_word(levels))


def _pack(codes, levels):
    """[..., 128] codes to [..., words] 32-bit words, 32 // bits codes to a word."""
    bits, per, n = _bits(levels), _per_word(levels), _words(levels)
    codes = torch.nn.functional.pad(codes.to(torch.int32), (0, n * per - D)).unflatten(-1, (n, per))
    return (codes << (torch.arange(per, device=codes.device, dtype=torch.int32) * bits)).sum(-1, dtype=torch.int32)


def _unpack(words, levels):
    """[..., words] to [..., 128] codes."""
    bits, per = _bits(levels), _per_word(levels)
    return ((words[..., None] >> (torch.arange(per, device=words.device, dtype=torch.int32) * bits)) & (levels - 1)).flatten(-2)[..., :D]


def _filled(gen, shape, levels, group, spread):
    """Codes and scales as a quantized Gaussian cache holds them: codes of N(0, 1) values, scales around `spread`."""
    t = torch.tensor(_book(levels)[1], dtype=torch.float32, device="cuda")
    flat = max(1, math.prod(shape))
    words = torch.empty((flat, _words(levels)), dtype=torch.int32, device="cuda")
    for lo in range(0, flat, 1 << 18):
        n = min(1 << 18, flat - lo)
        u = torch.randn((n, D), generator=gen, device="cuda")
        words[lo:lo + n] = _pack(torch.bucketize(u, t, out_int32=True), levels)
    scales = torch.exp(0.3 * torch.randn((*shape, D // group), generator=gen, device="cuda")) * spread
    return words.view(*shape, _words(levels)), scales.to(torch.float16)


def _pool(gen, case, pages, used):
    """A pool of pages [pages, hkv, page, ...] and its handle's parts. Slots that hold no token hold whatever was there."""
    shape = (pages, case["hkv"], case["page"])
    kc, ks = _filled(gen, shape, case["klevels"], case["group"], 1.5)
    vc, vs = _filled(gen, shape, case["vlevels"], case["group"], 0.8)
    free = torch.ones(pages * case["page"], dtype=torch.bool, device="cuda")
    free[used] = False
    free = free.view(pages, 1, case["page"], 1)
    ks.masked_fill_(free, float("nan"))
    vs.masked_fill_(free, float("inf"))
    book = lambda n: tuple(torch.tensor(x, dtype=torch.float32, device="cuda") for x in _book(n))  # noqa: E731
    sign = torch.tensor(_signs(), device="cuda")
    r = torch.ones((1, 1), device="cuda")
    while r.shape[0] < D:
        r = torch.cat([torch.cat([r, r], 1), torch.cat([r, -r], 1)], 0)
    return dict(kcodes=kc, kscales=ks, vcodes=vc, vscales=vs, kbook=book(case["klevels"]), vbook=book(case["vlevels"]),
                signs=sign, rotation=r * sign.float()[None, :] / math.sqrt(D), group=case["group"], page=case["page"],
                klevels=case["klevels"], vlevels=case["vlevels"])


def _heavy(gen, shape):
    """N(0, 1) with a scale of its own for each head and channel, as keys and values have them."""
    s = torch.exp(torch.randn((1, *shape[1:]), generator=gen, device="cuda").clamp(-2, 2) * 0.7)
    return torch.randn(shape, generator=gen, device="cuda") * s


def _tree_mask(rng, case):
    """Ancestor bits [batch, drafted, words] and the drafts in use [batch]."""
    b, n = case["batch"], case["drafted"]
    see = np.zeros((b, n, -(-n // 64) * 64), dtype=bool)
    count = np.full(b, n, dtype=np.int32)
    for s in range(b):
        if case["ragged"]:
            count[s] = rng.integers(1, n + 1)
        for i in range(count[s]):
            if case["tree"] == "chain":
                parent = i - 1
            elif case["tree"] == "bushy":
                parent = (i - 1) // 4 if i else -1
            else:
                parent = int(rng.integers(max(-1, i - 6), i))
            if parent >= 0:
                see[s, i] = see[s, parent]
            see[s, i, i] = True
        if case["ragged"] and s == b - 1:
            see[s, count[s] - 1] = False  # a row that sees no draft, and no context where that is empty
    words = np.packbits(see, axis=-1, bitorder="little").view(np.int64)
    return see[:, :, :n], words, count


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rng = np.random.Generator(np.random.PCG64(seed))
    if case["op"] == "rope":
        t, hq, hkv, dim = case["tokens"], case["hq"], case["hkv"], case["dim"]
        x = torch.randn((t, hq + 2 * hkv, dim), generator=gen, device="cuda").to(_DT[case["dtype"]])
        freq, factor = _frequencies(case["rotary"], case["base"], case["scaling"])
        if t <= 64:  # a step: each sequence is somewhere else
            pos = rng.integers(0, 4096, t) + case["start"]
        else:
            pos = np.arange(t) + case["start"]
        return dict(op="rope", q=x[:, :hq], k=x[:, hq:hq + hkv], factor=factor, rotary=case["rotary"], layout=case["layout"],
                    inverse=case["inverse"], positions=torch.tensor(pos, dtype=torch.int32, device="cuda"),
                    steps=torch.tensor(_steps(freq), device="cuda"))
    if case["op"] == "cache":
        t, h, hkv, page = case["new"], case["history"], case["hkv"], case["page"]
        pages = -(-(t + h) // page) + 1
        order = rng.permutation(pages)
        slots = (order[np.arange(t + h) // page] * page + np.arange(t + h) % page).astype(np.int32)
        state = _pool(gen, case, pages, torch.tensor(slots[:h], dtype=torch.int64, device="cuda"))
        new = slots[h:].copy()
        new[rng.random(t) < case["dropped"]] = -1
        qkv = _heavy(gen, (t, 2 * hkv, D)).to(_DT[case["dtype"]])
        state |= dict(op="cache", k=qkv[:, :hkv], v=qkv[:, hkv:], new=torch.tensor(new, device="cuda"),
                      slots=torch.tensor(np.concatenate([slots[:h], new]), device="cuda"), out=_DT[case["out"]], steps=None)
        if case["rope"]:
            state |= dict(positions=torch.arange(h, h + t, dtype=torch.int32, device="cuda"),
                          steps=torch.tensor(_steps(_frequencies(D, 10000.0, "none")[0]), device="cuda"))
        return state
    b, n, hq, hkv, page, most = (case[k] for k in ("batch", "drafted", "hq", "hkv", "page", "context"))
    lens = rng.integers(0, most + 1, b) if case["ragged"] else np.full(b, most)
    if case["ragged"]:
        lens[0] = most
        lens[-1] = 0 if b > 1 else most
    need = -(-lens // page)
    order, at = rng.permutation(int(need.sum()) + 2), 0
    table = np.full((b, max(1, -(-most // page))), -1, dtype=np.int32)
    used = []
    for s in range(b):
        table[s, :need[s]] = order[at:at + need[s]]
        at += need[s]
        i = np.arange(lens[s])
        used.append(table[s, i // page].astype(np.int64) * page + i % page)
    state = _pool(gen, case, len(order), torch.tensor(np.concatenate(used), device="cuda"))
    see, words, count = _tree_mask(rng, case)
    qkv = _heavy(gen, (b * n, hq + 2 * hkv, D)).to(torch.bfloat16).view(b, n, hq + 2 * hkv, D)
    dev = lambda a: torch.tensor(a, device="cuda")  # noqa: E731
    state |= dict(op="attend", q=qkv[:, :, :hq], k=qkv[:, :, hq:hq + hkv], v=qkv[:, :, hq + hkv:], table=dev(table),
                  lens=dev(lens.astype(np.int32)), mask=dev(words), see=dev(see), count=dev(count), context=most)
    return state


# ---------------------------------------------------------------- plain forms

def _turn(x, positions, steps, rotary, layout, factor, inverse):
    """Rotary positions on x [tokens, heads, dim] in 32 bits."""
    phase = (positions.to(torch.int64)[:, None] * steps[None, :]) >> 32  # the product wraps: whole turns drop out
    angle = phase.to(torch.float32) * (math.pi / 2 ** 31)
    cos, sin = torch.cos(angle)[:, None] * factor, torch.sin(angle)[:, None] * (-factor if inverse else factor)
    x = x.to(torch.float32)
    r, rest = x[..., :rotary], x[..., rotary:]
    if layout == "half":
        a, b = r[..., :rotary // 2], r[..., rotary // 2:]
        r = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    else:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return torch.cat([r, rest], -1)


def _encode(x, state, levels, book):
    """Rotated vectors [..., 128] to (words, fp16 scales)."""
    g = (x @ state["rotation"].T).unflatten(-1, (D // state["group"], state["group"]))
    rms = torch.sqrt((g * g).sum(-1, keepdim=True) / state["group"])
    u = torch.where(rms > 0, g / rms, torch.zeros_like(g))
    return _pack(torch.bucketize(u.flatten(-2), book[1], out_int32=True), levels), rms[..., 0].to(torch.float16)


def _decode(words, scales, state, levels, book):
    """(words, scales) to the vectors they stand for, rotated back, in 32 bits."""
    c = book[0][_unpack(words, levels)].unflatten(-1, (D // state["group"], state["group"]))
    return (c * scales.to(torch.float32)[..., None]).flatten(-2) @ state["rotation"]


def _plain_cache(s):
    k, v = s["k"].to(torch.float32), s["v"].to(torch.float32)
    if s["steps"] is not None:
        k = _turn(k, s["positions"], s["steps"], D, "half", 1.0, False)
    kept = s["new"] >= 0
    slot = s["new"][kept].to(torch.int64)
    page, at = slot // s["page"], slot % s["page"]
    for name, x in (("k", k), ("v", v)):
        words, scales = _encode(x[kept], s, s[name + "levels"], s[name + "book"])
        s[name + "codes"][page, :, at] = words
        s[name + "scales"][page, :, at] = scales
    got = s["slots"] >= 0
    slot = s["slots"].clamp(min=0).to(torch.int64)
    page, at = slot // s["page"], slot % s["page"]
    back = lambda n: torch.where(got[:, None, None], _decode(s[n + "codes"][page, :, at], s[n + "scales"][page, :, at],  # noqa: E731
                                                             s, s[n + "levels"], s[n + "book"]), 0.0).to(s["out"])
    return {"k": back("k"), "v": back("v")}


def _plain_attend(s):
    b, n, hq, _ = s["q"].shape
    hkv, most = s["k"].shape[2], s["context"]
    table = s["table"].clamp(min=0).to(torch.int64)
    flat = lambda x: x[table].transpose(1, 2).flatten(2, 3)[:, :, :most]  # noqa: E731  [b, hkv, most, ...]
    inside = torch.arange(most, device="cuda")[None] < s["lens"][:, None]  # [b, most]
    cached = lambda n: torch.where(inside[:, None, :, None], _decode(flat(s[n + "codes"]), flat(s[n + "scales"]), s,  # noqa: E731
                                                                     s[n + "levels"], s[n + "book"]), 0.0)
    heads = lambda x: x.to(torch.float32).transpose(1, 2)  # noqa: E731  [b, heads, n, 128]
    k = torch.cat([cached("k"), heads(s["k"])], 2)
    live = torch.arange(n, device="cuda")[None] < s["count"][:, None]
    see = torch.cat([inside[:, None].expand(b, n, most), s["see"]], 2) & live[:, :, None]  # [b, n, most + n]
    q = heads(s["q"]).unflatten(1, (hkv, hq // hkv)).flatten(2, 3)  # [b, hkv, ratio * n, 128]
    score = (q @ k.transpose(-1, -2)) * (1.0 / math.sqrt(D))
    score = score.unflatten(2, (hq // hkv, n)).masked_fill_(~see[:, None, None], float("-inf"))
    del k
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top > float("-inf"), top, 0.0))
    del score
    total = p.sum(-1, keepdim=True)
    p = (p / torch.where(total > 0, total, 1.0)).flatten(2, 3)
    v = torch.cat([cached("v"), heads(s["v"])], 2)
    o = (p @ v).unflatten(2, (hq // hkv, n)).flatten(1, 2)  # [b, hq, n, 128]
    return o.transpose(1, 2).to(torch.bfloat16)


# ---------------------------------------------------------------- the library's calls

def _handles(s):
    """The handles that a program keeps beside its pool, made on a state's first pass."""
    import rotated_codebook_quantized_gb300 as tq

    if "handles" not in s:
        if s["op"] == "rope":
            s["handles"] = tq.Rope(s["q"].shape[-1], s["rotary"], layout=s["layout"], steps=s["steps"], factor=s["factor"])
        else:
            book = lambda n: tq.Codebook(s[n + "levels"], centroids=s[n + "book"][0].cpu(), thresholds=s[n + "book"][1].cpu())  # noqa: E731
            cache = tq.PagedKVCache(s["kcodes"].shape[0], s["page"], s["kcodes"].shape[1], D, s["group"], book("k"), book("v"),
                                    tq.Rotation(D, D, signs=s["signs"].cpu()),
                                    storage=(s["kcodes"], s["kscales"], s["vcodes"], s["vscales"]))
            rope = tq.Rope(D, D, steps=s["steps"]) if s.get("steps") is not None else None
            s["handles"] = cache, rope
    return tq, s["handles"]


def run(s):
    if own:
        tq, h = _handles(s)
        if s["op"] == "rope":
            q, k = tq.rope(s["q"], s["positions"], h, k=s["k"], inverse=s["inverse"])
            return {"q": q, "k": k}
        if s["op"] == "cache":
            tq.kv_append(h[0], s["k"], s["v"], s["new"], rope=h[1], positions=s.get("positions"))
            k, v = tq.kv_fetch(h[0], s["slots"], out_dtype=s["out"])
            return {"k": k, "v": v}
        return {"o": tq.kv_attend_tree(h[0], s["q"], s["table"], s["lens"], k_new=s["k"], v_new=s["v"], mask=s["mask"],
                                       n_tok=s["count"], max_len=s["context"])}
    if s["op"] == "rope":
        turn = lambda x: _turn(x, s["positions"], s["steps"], s["rotary"], s["layout"], s["factor"], s["inverse"]).to(x.dtype)  # noqa: E731
        return {"q": turn(s["q"]), "k": turn(s["k"])}
    if s["op"] == "cache":
        return _plain_cache(s)
    return {"o": _plain_attend(s)}


# ---------------------------------------------------------------- what a pass cannot do without

def _row_bytes(case):
    """A cached token of one head: key and value words and scales."""
    return 4 * (_words(case["klevels"]) + _words(case["vlevels"])) + 2 * 2 * (D // case["group"])


def work(case):
    size = lambda d: 4 if d == "float32" else 2  # noqa: E731
    if case["op"] == "rope":
        heads = case["tokens"] * (case["hq"] + case["hkv"])
        return {"bytes": 2 * heads * case["dim"] * size(case["dtype"]) + 4 * case["tokens"], "flops": 3 * heads * case["rotary"]}
    if case["op"] == "cache":
        kept = case["new"] * (1 - case["dropped"])
        new, back = kept * case["hkv"], (case["history"] + kept) * case["hkv"]
        every = (case["history"] + case["new"]) * case["hkv"]
        return {"bytes": new * (2 * D * size(case["dtype"]) + _row_bytes(case)) + back * _row_bytes(case)
                + every * 2 * D * size(case["out"]) + 4 * (case["history"] + 2 * case["new"]),
                "flops": (new + back) * 2 * (D * 7 + 4 * D)}
    b, n = case["batch"], case["drafted"]
    mean = case["context"] * (1.0 if not case["ragged"] else 0.5 + 0.5 / b if b > 1 else 1.0)
    rows = b * n * (0.5 + 0.5 / n if case["ragged"] else 1.0)
    return {"bytes": b * mean * case["hkv"] * _row_bytes(case) + rows * 2 * D * (2 * case["hq"] + 2 * case["hkv"]),
            "flops": 4 * D * rows * case["hq"] * (mean + n / 2)}


# ---------------------------------------------------------------- the same from the definitions, in 64 bits

def _exact_turn(x, pos, freq, rotary, layout, factor, inverse):
    a = pos.double()[:, None] * torch.tensor(freq, dtype=torch.float64, device="cuda")[None]
    z = torch.polar(torch.full_like(a, factor), -a if inverse else a)[:, None]
    y = x.double().clone()
    if layout == "half":
        w = torch.complex(y[..., :rotary // 2].contiguous(), y[..., rotary // 2:rotary].contiguous()) * z
        y[..., :rotary // 2], y[..., rotary // 2:rotary] = w.real, w.imag
    else:
        w = torch.complex(y[..., 0:rotary:2].contiguous(), y[..., 1:rotary:2].contiguous()) * z
        y[..., 0:rotary:2], y[..., 1:rotary:2] = w.real, w.imag
    return y


def _exact_hadamard(x):
    """The order-128 Walsh-Hadamard transform over the square root of 128, by halves."""
    h, shape = 1, x.shape
    while h < D:
        y = x.reshape(-1, D // (2 * h), 2, h)
        x = torch.stack([y[:, :, 0] + y[:, :, 1], y[:, :, 0] - y[:, :, 1]], 2).reshape(shape)
        h *= 2
    return x / math.sqrt(D)


def _exact_values(words, scales, levels, group, c):
    """The vectors that rows of words [rows, words] and scales stand for, one code position at a time."""
    bits, per = _bits(levels), _per_word(levels)
    out = torch.empty((words.shape[0], D), dtype=torch.float64, device="cuda")
    book = torch.tensor(c, dtype=torch.float32, device="cuda").double()
    for d in range(D):
        code = torch.bitwise_and(torch.div(words[:, d // per].to(torch.int64) % (1 << 32), 1 << (bits * (d % per)),
                                           rounding_mode="floor"), levels - 1)
        out[:, d] = book[code] * scales[:, d // group].double()
    return _exact_hadamard(out) * torch.tensor(_signs(), device="cuda").double()


def _exact_cache(case, s):
    found = {}
    sign = torch.tensor(_signs(), device="cuda").double()
    for name in ("k", "v"):
        x = s[name].double()
        if name == "k" and case["rope"]:
            x = _exact_turn(x, s["positions"], _frequencies(D, 10000.0, "none")[0], D, "half", 1.0, False)
        c, t = _book(case[name + "levels"])
        # the books are 32-bit numbers of the model; everything computed from them is in 64 bits
        c, t = (torch.tensor(a, dtype=torch.float32, device="cuda").double() for a in (c, t))
        y = _exact_hadamard(x * sign).reshape(-1, case["group"])
        rms = y.square().mean(1, keepdim=True).sqrt()
        code = torch.searchsorted(t, torch.where(rms > 0, y / rms, 0.0).contiguous())
        new = (c[code] * rms.to(torch.float16).double()).reshape(case["new"], case["hkv"], D)
        new = _exact_hadamard(new) * sign
        new[s["new"] < 0] = 0.0
        old = s["slots"][:case["history"]].to(torch.int64)
        at = (old // case["page"], slice(None), old % case["page"])
        words, scales = s[name + "codes"][at], s[name + "scales"][at]
        old = _exact_values(words.flatten(0, 1), scales.flatten(0, 1), case[name + "levels"], case["group"], _book(case[name + "levels"])[0])
        found[name] = torch.cat([old.reshape(-1, case["hkv"], D), new], 0)
    return found


def _exact_attend(case, s):
    b, n, hq, hkv, page = (case[k] for k in ("batch", "drafted", "hq", "hkv", "page"))
    out = torch.zeros((b, n, hq, D), dtype=torch.float64, device="cuda")
    lens, count = s["lens"].tolist(), s["count"].tolist()
    for i in range(b):
        m, length = count[i], lens[i]
        pages = s["table"][i, :-(-length // page)].to(torch.int64)
        for h in range(hkv):
            kept = {}
            for name in ("k", "v"):
                w = s[name + "codes"][pages, h].reshape(-1, _words(case[name + "levels"]))[:length]
                z = s[name + "scales"][pages, h].reshape(-1, D // case["group"])[:length]
                old = _exact_values(w, z, case[name + "levels"], case["group"], _book(case[name + "levels"])[0])
                kept[name] = torch.cat([old, s[name][i, :m, h].double()], 0)
            block = torch.cat([torch.zeros((m, length), dtype=torch.bool, device="cuda"), ~s["see"][i, :m, :m]], 1)
            for g in range(h * (hq // hkv), (h + 1) * (hq // hkv)):
                score = (s["q"][i, :m, g].double() @ kept["k"].T / math.sqrt(D)).masked_fill(block, float("-inf"))
                out[i, :m, g] = torch.nan_to_num(torch.softmax(score, 1)) @ kept["v"]  # a row that sees nothing is zero
    return {"o": out}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        freq, factor = _frequencies(case["rotary"], case["base"], case["scaling"])
        turn = lambda x: _exact_turn(x, s["positions"], freq, case["rotary"], case["layout"], factor, case["inverse"])  # noqa: E731
        return {"q": turn(s["q"]), "k": turn(s["k"])}
    return _exact_cache(case, s) if case["op"] == "cache" else _exact_attend(case, s)
