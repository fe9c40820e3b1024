"""Cases and plain forms of the operators around a serving step with drafted tokens and latent attention.

Five operators, each computed here in a plain form (elementary torch operations) or, where ``own`` is true, by the
library's own calls:

* ``plan``    pages taken from and given back to a pool on the GPU, with the slot and position of every new token;
* ``verify``  drafted trees accepted or rejected against the target's probabilities, from given uniform numbers;
* ``write``   latent vectors and their rotary keys written to a paged cache;
* ``absorb``  attention of drafted tokens over the latent cache itself: keys and values are the latent vectors;
* ``expand``  attention of prompts over keys and values expanded from the latents, with one rotary key for all heads.

Latent vectors of 512, rotary keys of 64, heads of 128 and 64 heads are the layout of the model whose expert layer is the
library's headline workload; 131072 tokens are its longest cache; the rest spreads around them.
"""
from __future__ import annotations

import functools
import math

import numpy as np
import torch

own = False

C, R, W = 512, 64, 576  # latent vector, rotary key, a cached row of both
N, V = 128, 128         # a head's expanded key (without its rotary part) and value
SCALE = 1.0 / math.sqrt(N + R)


# ---------------------------------------------------------------- cases

def _plan(name, batch, context, new, page, packed=False, path=False, tight=False):
    return dict(name=name, op="plan", batch=batch, context=context, new=new, page=page, packed=packed, path=path, tight=tight)


def _verify(name, batch, nodes, vocab, dtype="float32", proposal=True, tree="random", ragged=False):
    return dict(name=name, op="verify", batch=batch, nodes=nodes, vocab=vocab, dtype=dtype, proposal=proposal, tree=tree,
                ragged=ragged)


def _write(name, tokens, page, dtype, cache, rope=False, dropped=0.0):
    return dict(name=name, op="write", tokens=tokens, page=page, dtype=dtype, cache=cache, rope=rope, dropped=dropped)


def _absorb(name, batch, drafted, heads, context, page=64, dtype="bfloat16", ragged=False, tree="random"):
    return dict(name=name, op="absorb", batch=batch, drafted=drafted, heads=heads, context=context, page=page, dtype=dtype,
                ragged=ragged, tree=tree)


def _expand(name, batch, tokens, history, heads, dtype="bfloat16", ragged=False):
    return dict(name=name, op="expand", batch=batch, tokens=tokens, history=history, heads=heads, dtype=dtype, ragged=ragged)


def listed():
    return [
        # a decode step of 64 sequences, up to 4 accepted tokens each out of trees of 8: launch latency is everything
        _plan("plan step", 64, 8192, 8, 64, path=True),
        # prompts of 300 sequences packed one after another, a pool that runs out before the last ones
        _plan("plan prompts", 300, 0, 400, 16, packed=True, tight=True),
        # eight sequences with chains of five drafts sampled from a draft model, a vocabulary of 131072
        _verify("verify chains", 8, 6, 131072, tree="chain"),
        # a batch of 48 trees of up to 23 drafts, an odd vocabulary, bf16 probabilities
        _verify("verify trees", 48, 24, 50001, dtype="bfloat16", ragged=True),
        # the accepted tokens of a decode step, some drafts rejected
        _write("write step", 48, 64, "bfloat16", "bfloat16", rope=True, dropped=0.5),
        # a whole prompt written once, keys turned to their positions on the way
        _write("write prompt", 65536, 64, "bfloat16", "bfloat16", rope=True),
        # three sequences just begun, five drafts each, 24 heads, contexts of 0 to 300 tokens: latency
        _absorb("absorb short", 3, 5, 24, 300, page=16, dtype="float16", ragged=True),
        # plain decoding of a serving batch: 32 sequences of very different lengths, one token each
        _absorb("absorb batch", 32, 1, 64, 16384, ragged=True, tree="chain"),
        # trees of 8 drafts over two long contexts, 512 rows to a sequence
        _absorb("absorb trees", 2, 8, 64, 65536),
        # a first prompt of a few words
        _expand("expand short", 1, 77, 0, 16),
        # chunks of prompts of seven sequences, each with what came before it, odd lengths
        _expand("expand chunks", 7, 701, 2500, 32, dtype="float16", ragged=True),
        # the largest: a prompt of 8192 tokens over all 64 heads
        _expand("expand prompt", 1, 8192, 0, 64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "verify", "write", "absorb", "absorb", "absorb", "expand", "expand"])
    page = rng.choice([16, 32, 64, 64, 128, 256])
    if op == "plan":
        packed = rng.random() < 0.5
        batch = _log(rng, 1, 2000)
        new = _log(rng, 1, max(2, min(65536, 131072 // batch))) if packed else rng.randint(1, 64)
        case = _plan("", batch, rng.choice([0, _log(rng, 1, max(2, min(131072, 4000000 // batch)))]), new, page, packed=packed,
                     path=not packed and rng.random() < 0.6, tight=rng.random() < 0.3)
    elif op == "verify":
        vocab, nodes = _log(rng, 50, 163840), rng.choice([1, rng.randint(2, 8), _log(rng, 2, 64)])
        batch = min(_log(rng, 1, 256), max(1, (48 * 24 * 50001 * 2) // (vocab * nodes)))
        case = _verify("", batch, nodes, vocab, rng.choice(["float32", "float32", "bfloat16", "float16"]), rng.random() < 0.7,
                       rng.choice(["chain", "chain", "random", "bushy"]), rng.random() < 0.5)
    elif op == "write":
        case = _write("", _log(rng, 1, 65536), page, rng.choice(["bfloat16", "bfloat16", "float16", "float32"]),
                      rng.choice(["bfloat16", "bfloat16", "float16"]), rng.random() < 0.7, rng.choice([0.0, 0.0, 0.4]))
    elif op == "absorb":
        batch, drafted = _log(rng, 1, 48), rng.choice([1, 1, _log(rng, 2, 64)])
        heads = rng.choice([8, 16, 24, 32, 64, 64, 128])
        context = min(_log(rng, 16, 131072), (1 << 19) // batch, (1 << 28) // (batch * drafted * heads))
        case = _absorb("", batch, drafted, heads, max(1, context), page, rng.choice(["bfloat16", "bfloat16", "float16"]),
                       rng.random() < 0.6, rng.choice(["random", "random", "chain", "bushy"]))
    else:
        batch, heads = _log(rng, 1, 16), rng.choice([4, 8, 16, 32, 64, 64])
        tokens = max(1, min(_log(rng, 1, 8192), 16384 // batch))
        history = rng.choice([0, _log(rng, 1, 8192)])
        history = min(history, (8192 * 8192 * 64 // 2) // (batch * heads * tokens), 32768 // batch)
        tokens = max(1, min(tokens, int(math.sqrt(8192 * 8192 * 64 // 2 / (batch * heads)))))
        case = _expand("", batch, tokens, history, heads, rng.choice(["bfloat16", "bfloat16", "float16"]), rng.random() < 0.6)
    del case["name"]
    return case


# ---------------------------------------------------------------- inputs

_DT = {"bfloat16": torch.bfloat16, "float16": torch.float16, "float32": torch.float32}


def _dev(a, dtype=None):
    return torch.tensor(np.ascontiguousarray(a), dtype=dtype, device="cuda")


@functools.lru_cache(None)
def _frequencies():
    return 50000.0 ** (-np.arange(0, R, 2) / R)


def _steps():
    """Phase per position in 2^-64 turns: the product with a position wraps by itself."""
    return np.array([int(f / (2 * math.pi) * 2 ** 64) for f in _frequencies()], dtype=np.uint64).view(np.int64)


def _parents(rng, kind, nodes):
    """Parents of a tree's nodes 1, 2, ... in an order that puts parents first; node 0 is the root."""
    if kind == "chain":
        return [-1] + list(range(nodes - 1))
    if kind == "bushy":
        return [-1] + [(i - 1) // 4 for i in range(1, nodes)]
    return [-1] + [int(rng.integers(max(0, i - 6), i)) for i in range(1, nodes)]


def _pairs(rng, b, low, most):
    """b numbers spread over low..most whose sum does not depend on the generator's state: each pair adds up to low + most."""
    x = rng.integers(low, most + 1, (b + 1) // 2)
    return rng.permutation(np.concatenate([x, low + most - x])[:b]) if b % 2 == 0 else np.concatenate(
        [rng.permutation(np.concatenate([x[1:], low + most - x[1:]])), [(low + most + 1) // 2]])


def _prepare_plan(case, rng):
    b, page, packed = case["batch"], case["page"], case["packed"]
    lens = rng.integers(0, case["context"] + 1, b)
    if packed:
        new = _pairs(rng, b, 0, case["new"])
    else:
        new = rng.integers(1, (case["new"] + 1) // 2 + 1 if case["path"] else case["new"] + 1, b)
    held = -(-lens // page)
    most = -(-(case["context"] + case["new"]) // page) + 2
    take = int((-(-(lens + new) // page) - held).sum())
    spare = int(take * 0.8) if case["tight"] else take + 5
    pages = b * most  # some of them with other pools' users
    order, at = rng.permutation(pages).astype(np.int32), 0
    table = np.full((b, most), -1, dtype=np.int32)
    for s in range(b):
        table[s, :held[s]] = order[at:at + held[s]]
        at += held[s]
    free = np.full(pages, -1, dtype=np.int32)
    free[:spare] = order[at:at + spare]
    path = None
    if case["path"]:  # the accepted nodes of a tree of `new` nodes: the root and some after it
        path = np.full((b, case["new"]), -1, dtype=np.int32)
        for s in range(b):
            path[s, :new[s]] = np.concatenate([[0], 1 + np.sort(rng.permutation(case["new"] - 1)[:new[s] - 1])])
    return dict(op="plan", page=page, packed=packed, n=case["new"], tokens=int(new.sum()) + 7, pages=pages,
                lens=_dev(lens, torch.int32), new=_dev(new, torch.int32), none=torch.zeros(b, dtype=torch.int32, device="cuda"),
                table=_dev(table), held=_dev(held, torch.int32), free=_dev(free),
                n_free=torch.full((1,), spare, dtype=torch.int32, device="cuda"), path=None if path is None else _dev(path))


def _prepare_verify(case, rng, gen):
    b, n, vocab, dt = case["batch"], case["nodes"], case["vocab"], _DT[case["dtype"]]
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    logits = rand(b, n, vocab) * 2.5
    p = torch.softmax(logits + 0.7 * rand(b, n, vocab), -1).to(dt)
    q = torch.softmax(logits, -1).to(dt)
    del logits
    parent = np.stack([_parents(rng, case["tree"], n) for _ in range(b)]).astype(np.int32)
    count = rng.integers(1, n + 1, b) if case["ragged"] else np.full(b, n)
    up = _dev(parent).long()
    tokens = torch.zeros((b, n), dtype=torch.int32, device="cuda")
    rows = torch.arange(b, device="cuda")
    for i in range(1, n):  # drafts come from the proposal at their parent (the likeliest of a few where it is not kept)
        at = q[rows, up[:, i]].float()
        some = torch.multinomial(at, 1 if case["proposal"] else min(4, vocab), replacement=case["proposal"], generator=gen)
        tokens[:, i] = some.gather(1, at.gather(1, some).argmax(1, keepdim=True))[:, 0].int()
    return dict(op="verify", p=p, q=q if case["proposal"] else None, tokens=tokens, parent=_dev(parent),
                u=torch.rand((b, n), generator=gen, device="cuda"),
                count=_dev(count, torch.int32) if case["ragged"] else None)


def _prepare_write(case, rng, gen):
    t, page = case["tokens"], case["page"]
    pages = -(-t // page) + 2
    order = rng.permutation(pages)
    slots = (order[np.arange(t) // page] * page + np.arange(t) % page).astype(np.int32)
    slots[rng.random(t) < case["dropped"]] = -1
    x = torch.randn((t, 3 * C + W), generator=gen, device="cuda").to(_DT[case["dtype"]])  # beside the queries' own projection
    return dict(op="write", c=x[:, 3 * C:3 * C + C], k=x[:, 3 * C + C:], slots=_dev(slots),
                rows=torch.zeros((pages, page, W), dtype=_DT[case["cache"]], device="cuda"),
                positions=torch.arange(17, 17 + t, dtype=torch.int32, device="cuda") if case["rope"] else None,
                steps=_dev(_steps()) if case["rope"] else None)


def _tree_mask(rng, case):
    """Ancestor bits [batch, drafted, words] and the drafts in use [batch]."""
    b, n = case["batch"], case["drafted"]
    see = np.zeros((b, n, -(-n // 64) * 64), dtype=bool)
    count = np.full(b, n, dtype=np.int32)
    for s in range(b):
        if case["ragged"]:
            count[s] = rng.integers(1, n + 1)
        parent = _parents(rng, case["tree"], n)
        for i in range(count[s]):
            if i:
                see[s, i] = see[s, parent[i]]
            see[s, i, i] = True
        if case["ragged"] and s == b - 1 and n > 1:
            see[s, count[s] - 1] = False  # a row that sees no draft, and no context where that is empty
    return see[:, :, :n], np.packbits(see, axis=-1, bitorder="little").view(np.int64), count


def _spread(gen, *shape):
    """N(0, 1) with a scale of its own for each channel, as normalised latents have them."""
    s = torch.exp(torch.randn(shape[-1], generator=gen, device="cuda").clamp(-2, 2) * 0.4)
    return torch.randn(shape, generator=gen, device="cuda") * s


def _prepare_absorb(case, rng, gen):
    b, n, h, page, most = (case[k] for k in ("batch", "drafted", "heads", "page", "context"))
    dt = _DT[case["dtype"]]
    lens = rng.integers(0, most + 1, b) if case["ragged"] else np.full(b, most)
    if case["ragged"]:
        lens[0] = most
        lens[-1] = 0 if b > 1 else most
    need = -(-lens // page)
    order, at = rng.permutation(int(need.sum()) + 2), 0
    table = np.full((b, max(1, -(-most // page))), -1, dtype=np.int32)
    for s in range(b):
        table[s, :need[s]] = order[at:at + need[s]]
        at += need[s]
    rows = _spread(gen, len(order), page, W).to(dt)
    rows[_dev(order[at:]).long()] = float("nan")  # pages that no sequence owns, and what lies past a sequence's end
    for s in range(b):
        if lens[s] % page:
            rows[int(table[s, need[s] - 1]), int(lens[s] % page):] = float("nan")
    see, words, count = _tree_mask(rng, case)
    return dict(op="absorb", rows=rows, page=page, table=_dev(table), lens=_dev(lens, torch.int32), most=most,
                q=(_spread(gen, b, n, h, W) * 1.2).to(dt), new=_spread(gen, b, n, W).to(dt), mask=_dev(words), see=_dev(see),
                count=_dev(count))


def _prepare_expand(case, rng, gen):
    b, t, past, h, dt = case["batch"], case["tokens"], case["history"], case["heads"], _DT[case["dtype"]]
    ql = _pairs(rng, b, 1, t) if case["ragged"] else np.full(b, t)
    kl = ql + (_pairs(rng, b, 0, past) if case["ragged"] else past)
    qs, ks = np.concatenate([[0], np.cumsum(ql)]), np.concatenate([[0], np.cumsum(kl)])
    q = (torch.randn((int(qs[-1]), h, N + R), generator=gen, device="cuda") * 1.3).to(dt)
    kv = _spread(gen, int(ks[-1]), h, N + V).to(dt)  # the expansion's own layout: a head's key, then its value
    return dict(op="expand", q=q, k=kv[..., :N], v=kv[..., N:], shared=torch.randn((int(ks[-1]), R), generator=gen, device="cuda").to(dt),
                q_starts=_dev(qs, torch.int32), kv_starts=_dev(ks, torch.int32), spans=list(zip(qs[:-1].tolist(), qs[1:].tolist(),
                                                                                               ks[:-1].tolist(), ks[1:].tolist())))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rng = np.random.Generator(np.random.PCG64(seed))
    if case["op"] == "plan":
        return _prepare_plan(case, rng)
    return {"verify": _prepare_verify, "write": _prepare_write, "absorb": _prepare_absorb,
            "expand": _prepare_expand}[case["op"]](case, rng, gen)


# ---------------------------------------------------------------- plain forms

def _plain_pages(s, new, n, path, packed):
    """One plan: the pool's tensors are changed in place; whole numbers throughout."""
    table, held, free, n_free, lens, page = s["table"], s["held"].long(), s["free"], s["n_free"].long(), s["lens"].long(), s["page"]
    b, width = table.shape
    new = new.long()
    need = (lens + new + page - 1) // page
    index = torch.arange(width, device="cuda")[None]
    back = (index >= need[:, None]) & (index < held[:, None])
    rank, given = back.flatten().cumsum(0).view(b, width) - 1, back.sum()
    stack = torch.cat([free, free.new_zeros(1)])  # the last place takes what is not moved
    stack[torch.where(back, n_free + given - 1 - rank, free.numel())] = table
    stack, top = stack[:-1], n_free + given
    take = (need - held).clamp(min=0)
    upto = take.cumsum(0)
    served = (upto <= top) | (take == 0)
    fresh = (index >= held[:, None]) & (index < need[:, None]) & served[:, None]
    source = top - 1 - ((upto - take)[:, None] + index - held[:, None])
    got = stack[torch.where(fresh, source, 0)]
    table.copy_(torch.where(fresh, got, torch.where(back, -1, table)))
    free.copy_(stack)
    s["held"].copy_(torch.where(served, need, held))
    s["n_free"].copy_(top - torch.where(served, take, 0).sum())
    out = {"lens": torch.where(served, lens + new, lens).int()}
    if packed:
        starts = torch.cat([new.new_zeros(1), new.cumsum(0)])
        t = torch.arange(s["tokens"], device="cuda")
        row = torch.searchsorted(starts, t, right=True) - 1
        live, row = row < b, row.clamp(max=b - 1)
        at = lens[row] + t - starts[row]
        out["starts"] = starts.int()
    else:
        row = torch.arange(b, device="cuda")[:, None]
        i = torch.arange(n, device="cuda")[None]
        live, at = i < new[:, None], lens[:, None] + i
    live = live & served[row]
    at = torch.where(live, at, 0)
    slot = table[row, (at // page).clamp(max=width - 1)].long() * page + at % page
    slot, at = torch.where(live, slot, -1).int(), at.int()
    if path is not None:  # the k-th new token is the tree's node path[k]
        column = torch.where(live, path.long(), n)
        slot, at = (torch.full((b, n + 1), none, dtype=torch.int32, device="cuda").scatter_(1, column, x)[:, :n]
                    for x, none in ((slot, -1), (at, 0)))
    return out | {"slots": slot, "positions": at}


def _plain_verify(s):
    """The walk over all sequences at once, in 64 bits: an acceptance or a sampled token can hang on a last digit."""
    p, q, tokens, parent, u = s["p"], s["q"], s["tokens"].long(), s["parent"].long(), s["u"].double()
    b, n, vocab = p.shape
    rows = torch.arange(b, device="cuda")
    used = torch.full((b,), n, device="cuda") if s["count"] is None else s["count"].long()
    at, length = torch.zeros(b, dtype=torch.long, device="cuda"), torch.ones(b, dtype=torch.long, device="cuda")
    path = torch.full((b, n + 1), -1, dtype=torch.long, device="cuda")
    path[:, 0] = 0
    r, total = p[:, 0].double(), torch.ones(b, dtype=torch.float64, device="cuda")
    for i in range(1, n):
        x = tokens[:, i]
        tested = (parent[:, i] == at) & (i < used)
        share = r[rows, x]
        if q is None:
            proposed = torch.zeros_like(r).scatter_(1, x[:, None], 1.0)
        else:
            proposed = q[rows, at].double()
        yes = tested & (u[:, i] * proposed[rows, x] * total < share)
        no = tested & ~yes
        if q is None:
            left = torch.where(proposed > 0, 0.0, r)
            rest = total - share
        else:
            left = (r - total[:, None] * proposed).clamp(min=0)
            rest = left.sum(1)
        r = torch.where(no[:, None], left, r)
        total = torch.where(no, rest, total)
        r = torch.where(yes[:, None], p[:, i].double(), r)
        total = torch.where(yes, 1.0, total)
        path[rows, torch.where(yes, length, n)] = i
        at, length = torch.where(yes, i, at), length + yes
    r = torch.where(r.sum(1, keepdim=True) > 0, r, p[rows, at].double())  # nothing left: the target's own
    cum = r.cumsum(1)
    above = cum > u[:, :1] * cum[:, -1:]
    none = ~above.any(1)
    last = vocab - 1 - (r.flip(1) > 0).int().argmax(1)
    return {"path": path[:, :n].int(), "count": length.int(), "next": torch.where(none, last, above.int().argmax(1)).int()}


def _plain_write(s):
    kept = s["slots"] >= 0
    slot = s["slots"][kept].long()
    k = s["k"].float()
    if s["steps"] is not None:
        phase = (s["positions"].long()[:, None] * s["steps"][None]) >> 32  # the product wraps: whole turns drop out
        angle = phase.float() * (math.pi / 2 ** 31)
        a, b, cos, sin = k[:, 0::2], k[:, 1::2], torch.cos(angle), torch.sin(angle)
        k = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(1)
    s["rows"].view(-1, W)[slot] = torch.cat([s["c"].float(), k], 1)[kept].to(s["rows"].dtype)
    return {"rows": s["rows"]}


def _plain_absorb(s):
    b, n, h, _ = s["q"].shape
    most = s["most"]
    inside = torch.arange(most, device="cuda")[None] < s["lens"][:, None]
    live = torch.arange(n, device="cuda")[None] < s["count"][:, None]
    cached = s["rows"][s["table"].clamp(min=0).long()].flatten(1, 2)[:, :most]
    rows = torch.cat([torch.where(inside[:, :, None], cached, 0.0).float(), torch.where(live[:, :, None], s["new"], 0.0).float()], 1)
    see = torch.cat([inside[:, None].expand(b, n, most), s["see"]], 2) & live[:, :, None]
    score = (s["q"].float().flatten(1, 2) @ rows.transpose(1, 2)) * SCALE
    score = score.view(b, n, h, most + n).masked_fill_(~see[:, :, None], float("-inf"))
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top > float("-inf"), top, 0.0))
    del score
    total = p.sum(-1, keepdim=True)
    o = p.flatten(1, 2) @ rows[..., :C]
    return {"o": (o.view(b, n, h, C) / torch.where(total > 0, total, 1.0)).to(s["q"].dtype)}


def _plain_expand(s):
    out = torch.empty((s["q"].shape[0], s["q"].shape[1], V), dtype=s["q"].dtype, device="cuda")
    for q0, q1, k0, k1 in s["spans"]:
        see = torch.arange(k1 - k0, device="cuda")[None] <= torch.arange(q1 - q0, device="cuda")[:, None] + (k1 - k0 - q1 + q0)
        shared = s["shared"][k0:k1].float()
        for h in range(out.shape[1]):
            q = s["q"][q0:q1, h].float()
            score = (q[:, :N] @ s["k"][k0:k1, h].float().T + q[:, N:] @ shared.T) * SCALE
            score.masked_fill_(~see, float("-inf"))
            top = score.amax(-1, keepdim=True)
            p = torch.exp(score - torch.where(top > float("-inf"), top, 0.0))
            total = p.sum(-1, keepdim=True)
            out[q0:q1, h] = ((p @ s["v"][k0:k1, h].float()) / torch.where(total > 0, total, 1.0)).to(out.dtype)
    return {"o": out}


# ---------------------------------------------------------------- the library's calls

def _handle(s):
    """The handle that a program keeps beside its tensors, made on a state's first pass."""
    import rotated_codebook_quantized_gb300 as tq

    if "handle" not in s:
        if s["op"] == "plan":
            s["handle"] = tq.PagePool(s["pages"], s["page"], *s["table"].shape, storage=(s["table"], s["held"], s["free"], s["n_free"]))
        elif s["op"] in ("write", "absorb"):
            cache = tq.LatentCache(s["rows"].shape[0], s["rows"].shape[1], dtype=s["rows"].dtype, storage=s["rows"])
            s["handle"] = cache, tq.Rope(R, R, layout="interleaved", steps=s["steps"]) if s.get("steps") is not None else None
        else:
            s["handle"] = None
    return tq, s["handle"]


def run(s):
    if s["op"] == "plan":
        # a step is planned and, its drafts all rejected or its requests ended, taken back: the pool is as it was
        if own:
            tq, pool = _handle(s)
            if s["packed"]:
                plan = tq.kv_plan(pool, s["lens"], s["new"], tokens=s["tokens"])
            else:
                plan = tq.kv_plan(pool, s["lens"], s["new"], n=s["n"], path=s["path"])
            undone = tq.kv_plan(pool, s["lens"], s["none"], n=1)
            out = {"slots": plan.slots, "positions": plan.positions, "lens": plan.lens, "undone": undone.lens}
            if s["packed"]:
                out["starts"] = plan.starts
        else:
            out = _plain_pages(s, s["new"], s["n"], s["path"], s["packed"])
            out["undone"] = _plain_pages(s, s["none"], 1, None, False)["lens"]
        return out | {"table": s["table"], "held": s["held"], "free": s["free"], "n_free": s["n_free"]}
    if not own:
        return {"verify": _plain_verify, "write": _plain_write, "absorb": _plain_absorb, "expand": _plain_expand}[s["op"]](s)
    tq, h = _handle(s)
    if s["op"] == "verify":
        path, count, token = tq.verify_tree(s["p"], s["tokens"], s["parent"], s["u"], q=s["q"], n_tok=s["count"])
        return {"path": path, "count": count, "next": token}
    if s["op"] == "write":
        tq.latent_append(h[0], s["c"], s["k"], s["slots"], rope=h[1], positions=s["positions"])
        return {"rows": s["rows"]}
    if s["op"] == "absorb":
        return {"o": tq.latent_attend_tree(h[0], s["q"], s["table"], s["lens"], SCALE, new=s["new"], mask=s["mask"], n_tok=s["count"],
                                           max_len=s["most"])}
    return {"o": tq.latent_attend_prompt(s["q"], s["k"], s["v"], s["shared"], s["q_starts"], s["kv_starts"], SCALE)}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    size = lambda d: 4 if d == "float32" else 2  # noqa: E731
    if case["op"] == "plan":
        b = case["batch"]
        new = b * case["new"] * (0.5 if case["packed"] or not case["path"] else 0.25)
        # lengths, counts and pages held in and out, both ways; a page that is taken and given back; the new tokens
        return {"bytes": 2 * b * 20 + new / case["page"] * 16 + (new if case["packed"] else b * case["new"]) * 8
                + (4 * b * case["new"] if case["path"] else 0), "flops": 0}
    if case["op"] == "verify":
        # the distributions at the node where the walk ends, every node's token, parent and number, two probabilities each
        rows = 2 if case["proposal"] else 1
        nodes = case["batch"] * case["nodes"] * (0.5 if case["ragged"] else 1.0)
        return {"bytes": case["batch"] * case["vocab"] * size(case["dtype"]) * rows + nodes * (12 + 4 + size(case["dtype"]) * rows),
                "flops": case["batch"] * case["vocab"] * (rows + 1)}
    if case["op"] == "write":
        kept = case["tokens"] * (1 - case["dropped"])
        return {"bytes": kept * W * (size(case["dtype"]) + 2) + case["tokens"] * 4 + (kept * 4 if case["rope"] else 0),
                "flops": kept * R * 3 if case["rope"] else 0}
    if case["op"] == "absorb":
        b, n = case["batch"], case["drafted"]
        mean = case["context"] * (1.0 if not case["ragged"] else 0.5 + 0.5 / b if b > 1 else 1.0)
        rows = b * n * (0.5 + 0.5 / n if case["ragged"] else 1.0)
        return {"bytes": 2 * (b * mean * W + rows * (W + case["heads"] * (W + C))), "flops": 2 * (W + C) * rows * case["heads"] * (mean + n / 2)}
    b, h = case["batch"], case["heads"]
    t = case["tokens"] * (0.5 if case["ragged"] else 1.0)
    past = case["history"] * (0.5 if case["ragged"] else 1.0)
    # the square of a length spread evenly up to `tokens` is a third of it on average
    pairs = t * past + case["tokens"] ** 2 * (1 / 3 if case["ragged"] else 1.0) / 2
    return {"bytes": 2 * b * (t * h * (N + R + V) + (t + past) * (h * (N + V) + R)), "flops": 2 * (N + R + V) * b * h * pairs}


# ---------------------------------------------------------------- the same from the definitions, in 64 bits

def _exact_plan(case, s):
    """One list of pages after another, on the host."""
    page, b = s["page"], case["batch"]
    lens, new, table, stack = s["lens"].tolist(), s["new"].tolist(), s["table"].tolist(), s["free"].tolist()
    n_free = int(s["n_free"])
    own_pages = [[p for p in row if p >= 0] for row in table]
    pool = stack[:n_free]
    n = case["new"]
    starts, slots, positions, after = [0], [], [], []
    asked, blocked, top = 0, n_free, n_free
    taken = []
    for i in range(b):
        more = max(0, -(-(lens[i] + new[i]) // page) - len(own_pages[i]))
        asked += more
        ok = more == 0 or asked <= blocked
        mine = own_pages[i] + ([pool[top - 1 - (asked - more) - k] for k in range(more)] if ok else [])
        taken += mine[len(own_pages[i]):]
        after.append(lens[i] + new[i] if ok else lens[i])
        a = [mine[t // page] * page + t % page if ok else -1 for t in range(lens[i], lens[i] + new[i])]
        z = [t if ok else 0 for t in range(lens[i], lens[i] + new[i])]
        if case["packed"]:
            slots += a
            positions += z
            starts.append(starts[-1] + new[i])
        else:
            where = s["path"][i, :new[i]].tolist() if s["path"] is not None else range(new[i])
            row, at = [-1] * n, [0] * n
            for k, w in enumerate(where):
                row[w], at[w] = a[k], z[k]
            slots.append(row)
            positions.append(at)
    if case["packed"]:
        slots += [-1] * (s["tokens"] - len(slots))
        positions += [0] * (s["tokens"] - len(positions))
    whole = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    # what is taken back lies on the stack again as it lay before, and the tables end where they ended
    out = {"slots": whole(slots), "positions": whole(positions), "lens": whole(after), "undone": s["lens"]}
    if case["packed"]:
        out["starts"] = whole(starts)
    return out | {"table": s["table"], "held": s["held"], "free": s["free"], "n_free": s["n_free"]}


def _exact_verify(case, s):
    """One sequence after another, normalised at every step."""
    b, n = case["batch"], case["nodes"]
    tokens, parent, u = s["tokens"].tolist(), s["parent"].tolist(), s["u"].tolist()
    used = s["count"].tolist() if s["count"] is not None else [n] * b
    paths, counts, following = [], [], []
    for i in range(b):
        node, walked, r = 0, [0], None  # r: the residual distribution, the target's own until a child is rejected
        child = 1
        while child < used[i]:
            if parent[i][child] == node:
                x = tokens[i][child]
                have = float(s["p"][i, node, x]) if r is None else float(r[x])
                offered = 1.0 if s["q"] is None else float(s["q"][i, node, x])
                if u[i][child] * offered < have:
                    node, r = child, None
                    walked.append(child)
                else:
                    r = s["p"][i, node].double() if r is None else r
                    if s["q"] is None:
                        whole = 1.0 - have  # what is left of a distribution whose sum is one
                        r = r.clone()
                        r[x] = 0.0
                    else:
                        r = torch.relu(r - s["q"][i, node].double())
                        whole = float(r.sum())
                    r = r / whole if whole > 0 else r
            child += 1
        if r is None or float(r.sum()) <= 0:
            r = s["p"][i, node].double()
        edge = torch.cumsum(r, 0)
        at = int(torch.searchsorted(edge, u[i][0] * edge[-1], right=True))
        following.append(at if at < case["vocab"] else int(torch.nonzero(r).max()))
        paths.append(walked + [-1] * (n - len(walked)))
        counts.append(len(walked))
    whole = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    return {"path": whole(paths), "count": whole(counts), "next": whole(following)}


def _exact_write(case, s):
    rows = s["rows"].double().flatten(0, 1)
    k = s["k"].double()
    if case["rope"]:
        turn = s["positions"].double()[:, None] * torch.tensor(_frequencies(), device="cuda")[None]
        k = torch.view_as_real(torch.view_as_complex(k.unflatten(1, (R // 2, 2)).contiguous()) * torch.polar(torch.ones_like(turn), turn)).flatten(1)
    for part, lo, hi in ((s["c"].double(), 0, C), (k, C, W)):
        rows[:, lo:hi].index_copy_(0, s["slots"].long()[s["slots"] >= 0], part[s["slots"] >= 0])
    return {"rows": rows.view(s["rows"].shape)}


def _exact_absorb(case, s):
    b, n, h, page = (case[k] for k in ("batch", "drafted", "heads", "page"))
    out = torch.zeros((b, n, h, C), dtype=torch.float64, device="cuda")
    lens, count = s["lens"].tolist(), s["count"].tolist()
    for i in range(b):
        pages = s["table"][i, :-(-lens[i] // page)].long()
        old = s["rows"][pages].reshape(-1, W)[:lens[i]].double()
        for d in range(count[i]):
            seen = torch.nonzero(s["see"][i, d])[:, 0]
            rows = torch.cat([old, s["new"][i, seen].double()])
            if len(rows):
                out[i, d] = torch.softmax(s["q"][i, d].double() @ rows.T / math.sqrt(N + R), 1) @ rows[:, :C]
    return {"o": out}


def _exact_expand(case, s):
    out = torch.zeros((*s["q"].shape[:2], V), dtype=torch.float64, device="cuda")
    for q0, q1, k0, k1 in s["spans"]:
        for h in range(case["heads"]):
            k = torch.cat([s["k"][k0:k1, h], s["shared"][k0:k1]], 1).double()
            v = s["v"][k0:k1, h].double()
            for lo in range(q0, q1, 2048):  # a block of rows sees nothing past its last row's position
                hi = min(lo + 2048, q1)
                upto = hi - q1 + k1 - k0
                score = (s["q"][lo:hi, h].double() @ k[:upto].T) / math.sqrt(N + R)
                late = torch.arange(upto, device="cuda")[None] > torch.arange(lo, hi, device="cuda")[:, None] - q1 + (k1 - k0)
                out[lo:hi, h] = torch.softmax(score.masked_fill(late, float("-inf")), 1) @ v[:upto]
    return {"o": out}


def exact(case, seed):
    s = prepare(case, seed)
    return {"plan": _exact_plan, "verify": _exact_verify, "write": _exact_write, "absorb": _exact_absorb,
            "expand": _exact_expand}[case["op"]](case, s)
