"""Decoding with drafted trees over a paged compressed cache: the serving path of one attention layer.

Two sequences share a pool of pages.  Their prompts are written with rotary positions on the way; then every step drafts a
small tree of tokens for each sequence, turns the drafts' queries and keys, attends (context out of the compressed pages,
drafts through their ancestor mask), accepts the path that a stand-in for sampling picks, and appends that path alone.  At the
end the cache is read back and the last step is checked against a plain computation over it.

Run on a GPU, after the library is built:  python examples/drafted_decode.py
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import rotated_codebook_quantized_gb300 as tq

HEADS, KV_HEADS, DIM, GROUP, PAGE = 32, 8, 128, 32, 64
BATCH, DRAFTS, STEPS = 2, 8, 6


def draft_tree(gen):
    """Parents of DRAFTS nodes (-1: the last accepted token) as an ancestor matrix, itself included, and the depths."""
    see = torch.zeros((BATCH, DRAFTS, DRAFTS), dtype=torch.bool)
    for b in range(BATCH):
        for i in range(DRAFTS):
            parent = int(torch.randint(-1, i, (1,), generator=gen)) if i else -1
            if parent >= 0:
                see[b, i] = see[b, parent]
            see[b, i, i] = True
    return see, see.sum(-1).int() - 1


def main():
    dev = "cuda"
    gen = torch.Generator().manual_seed(0)
    rand = lambda *shape: torch.randn(shape, generator=gen).to(dev, torch.bfloat16)  # noqa: E731
    rope = tq.Rope(DIM, base=500000.0, scaling={"kind": "parts", "factor": 16.0, "original": 8192})
    cache = tq.PagedKVCache(64, PAGE, KV_HEADS, DIM, GROUP, tq.Codebook(256), tq.Codebook(8), tq.Rotation(DIM, DIM, seed=5000))
    table = torch.randperm(64, generator=gen).int().view(BATCH, 32).to(dev)  # 32 pages to a sequence
    lens = torch.tensor([700, 45], dtype=torch.int32, device=dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)

    def slots(b, positions):
        return (table[b, positions // PAGE] * PAGE + positions % PAGE).int()

    for b, n in enumerate(lens.tolist()):  # prompts
        at = torch.arange(n, device=dev)
        kv = rand(n, 2 * KV_HEADS, DIM)
        tq.kv_append(cache, kv[:, :KV_HEADS], kv[:, KV_HEADS:], slots(b, at), rope=rope, positions=at.int(), err=err)

    for step in range(STEPS):
        see, depth = draft_tree(gen)
        words = torch.zeros((BATCH, DRAFTS), dtype=torch.int64)
        for j in range(DRAFTS):
            words |= see[:, :, j].long() << j
        qkv = rand(BATCH, DRAFTS, HEADS + 2 * KV_HEADS, DIM)  # what the layer's projection would give
        positions = lens[:, None] + depth.to(dev)
        q, k = tq.rope(qkv[:, :, :HEADS], positions, rope, k=qkv[:, :, HEADS:HEADS + KV_HEADS])
        v = qkv[:, :, HEADS + KV_HEADS:]
        out = tq.kv_attend_tree(cache, q, table, lens, k_new=k, v_new=v, mask=words[..., None].to(dev), err=err)
        if step == STEPS - 1:
            break
        # the deepest leaf stands for the path that sampling accepts; rejected drafts are never written
        leaf = depth.argmax(-1)
        taken = torch.stack([see[b, leaf[b]] for b in range(BATCH)]).to(dev)
        page = table.gather(1, (positions // PAGE).long())
        tq.kv_append(cache, k, v, torch.where(taken, page * PAGE + positions % PAGE, -1).int(), err=err)
        lens += taken.sum(-1).int()

    worst = 0.0
    for b in range(BATCH):  # the last step over what the cache stands for
        ck, cv = tq.kv_fetch(cache, slots(b, torch.arange(int(lens[b]), device=dev)), out_dtype=torch.float32, err=err)
        kk, vv = torch.cat([ck, k[b].float()]), torch.cat([cv, v[b].float()])
        kk, vv = (x.repeat_interleave(HEADS // KV_HEADS, 1).transpose(0, 1) for x in (kk, vv))
        s = q[b].float().transpose(0, 1) @ kk.transpose(1, 2) * DIM ** -0.5
        s[:, :, int(lens[b]):].masked_fill_(~see[b].to(dev), float("-inf"))
        ref = (torch.softmax(s, -1) @ vv).transpose(0, 1)
        worst = max(worst, float((out[b].float() - ref).norm() / ref.norm()))
    bits = tq.check_error(err)
    print(f"{STEPS} steps, contexts of {lens.tolist()} tokens, error word {bits}, last step off by {worst:.2e} (relative 2-norm)")
    return worst, bits


if __name__ == "__main__":
    tq.load()
    worst, bits = main()
    sys.exit(0 if worst < 4e-3 and bits == 0 else 1)
