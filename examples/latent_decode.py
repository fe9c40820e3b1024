"""Serving two requests of a model with latent attention: one attention layer, planned on the GPU from end to end.

The requests' prompts are packed one after another.  Their pages come from a pool on the device, their latent vectors go to the paged
cache, and their attention runs in the expanded form (keys and values of each head out of the latents).  Then every step drafts a
tree of tokens for each request, attends over the cache in the absorbed form (queries through the key projection, results through the
value projection), verifies the drafts against the target's probabilities, plans pages for the accepted path alone and writes its
latents.  Lengths, slots and accepted paths never leave the GPU.  The last step is checked against the expanded form over everything
that is cached.

Run on a GPU, after the library is built:  python examples/latent_decode.py
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import rotated_codebook_quantized_gb300 as tq

HEADS, LATENT, ROPE, KEY, VALUE = 16, 512, 64, 128, 128
PAGE, PAGES, NODES, VOCAB, STEPS = 64, 40, 8, 1000, 5
SCALE = (KEY + ROPE) ** -0.5
PROMPTS = [300, 77]


def main():
    dev, dt = "cuda", torch.bfloat16
    gen = torch.Generator().manual_seed(0)
    rand = lambda *shape: torch.randn(shape, generator=gen).to(dev)  # noqa: E731
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    B = len(PROMPTS)
    wk, wv = rand(HEADS, KEY, LATENT) * LATENT ** -0.5, rand(HEADS, VALUE, LATENT) * LATENT ** -0.5  # of the layer
    rope = tq.Rope(ROPE, ROPE, base=50000.0, layout="interleaved")
    pool, cache = tq.PagePool(PAGES, PAGE, B, 16), tq.LatentCache(PAGES, PAGE)

    def expanded(c):
        return (torch.einsum("tc,hdc->thd", c.float(), w).to(dt) for w in (wk, wv))

    def projected(*lead):
        """What the layer's projections give: latent and rotary key (one row), and the heads' queries."""
        return rand(*lead, LATENT + ROPE).to(dt), rand(*lead, HEADS, KEY + ROPE).to(dt)

    # ---- prompts
    T = sum(PROMPTS)
    row, q = projected(T)
    plan = tq.kv_plan(pool, ints([0] * B), ints(PROMPTS), tokens=T, err=err)
    lens = plan.lens
    tq.latent_append(cache, row[:, :LATENT], row[:, LATENT:], plan.slots, rope=rope, positions=plan.positions, err=err)
    qr, kr = tq.rope(q[..., KEY:].contiguous(), plan.positions, rope, k=row[:, None, LATENT:].contiguous())
    k, v = expanded(row[:, :LATENT])
    out = tq.latent_attend_prompt(torch.cat([q[..., :KEY], qr], -1), k, v, kr[:, 0], plan.starts, plan.starts, SCALE, err=err)

    worst, accepted = 0.0, 0
    for step in range(STEPS):
        # ---- a tree a request: node 0 is the last token that came out, each other one hangs on one before it
        parent = torch.full((B, NODES), -1)
        see = torch.zeros((B, NODES, NODES), dtype=torch.bool)
        for b in range(B):
            for i in range(NODES):
                if i:
                    parent[b, i] = torch.randint(max(0, i - 3), i, (1,), generator=gen)
                    see[b, i] = see[b, parent[b, i]]
                see[b, i, i] = True
        words = (see.long() << torch.arange(NODES)).sum(-1, keepdim=True).to(dev)
        positions = lens[:, None] + (see.sum(-1).int() - 1).to(dev)
        # ---- attention over the cache and the tree
        row, q = projected(B, NODES)
        turned = row.clone()
        qr = tq.rope(q[..., KEY:].contiguous(), positions, rope)
        tq.rope(turned[..., None, LATENT:], positions, rope, inplace=True)
        absorbed = torch.cat([torch.einsum("bnhd,hdc->bnhc", q[..., :KEY].float(), wk).to(dt), qr], -1)
        o = tq.latent_attend_tree(cache, absorbed, pool.table, lens, SCALE, new=turned, mask=words, err=err)
        out = torch.einsum("bnhc,hdc->bnhd", o.float(), wv)
        if step == STEPS - 1:
            break
        # ---- what the rest of the model makes of it: the target's distributions; the draft model's are near them
        logits = rand(B, NODES, VOCAB) * 2
        target, draft = torch.softmax(logits, -1), torch.softmax(logits + 0.5 * rand(B, NODES, VOCAB), -1)
        at = parent.clamp(min=0).to(dev)
        tokens = torch.multinomial(draft.gather(1, at[..., None].expand(-1, -1, VOCAB)).flatten(0, 1).cpu(), 1, generator=gen)
        path, count, following = tq.verify_tree(target, tokens.view(B, NODES).int().to(dev), parent.int().to(dev),
                                                torch.rand((B, NODES), generator=gen).to(dev), q=draft, err=err)
        # ---- pages and slots of the accepted path; rejected drafts are never written
        plan = tq.kv_plan(pool, lens, count, n=NODES, path=path, err=err)
        tq.latent_append(cache, row[..., :LATENT], row[..., LATENT:], plan.slots, rope=rope, positions=plan.positions, err=err)
        lens = plan.lens
        accepted += int(count.sum())

    # ---- the last step's first rows in the expanded form over all that is cached
    for b, n in enumerate(lens.tolist()):
        at = torch.arange(n, device=dev)
        cached = cache.rows.view(-1, LATENT + ROPE)[pool.table[b, at // PAGE].long() * PAGE + at % PAGE]
        rows = torch.cat([cached, turned[b, :1]])
        k, v = expanded(rows[:, :LATENT])
        qb = torch.cat([q[b, :1, :, :KEY], qr[b, :1]], -1)
        ref = tq.latent_attend_prompt(qb, k, v, rows[:, LATENT:], ints([0, 1]), ints([0, n + 1]), SCALE, err=err)[0].float()
        worst = max(worst, float((out[b, 0] - ref).norm() / ref.norm()))
    bits = tq.check_error(err)
    print(f"{STEPS} steps, {accepted} tokens accepted, contexts of {lens.tolist()} tokens, error word {bits}, absorbed and expanded "
          f"forms {worst:.2e} apart (relative 2-norm)")
    return worst, bits, lens.tolist(), accepted


if __name__ == "__main__":
    tq.load()
    worst, bits, _, _ = main()
    sys.exit(0 if worst < 1.2e-2 and bits == 0 else 1)
