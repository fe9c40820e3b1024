"""Attention of drafted trees over batches of very different lengths, where a CTA's run crosses many short contexts, against
the definition in 64 bits.

Tolerances: those of tests/test_gpu_paged_cache.py, for the same reasons.
"""
import numpy as np
import pytest

from tests import test_gpu_paged_cache as base

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

D, H, PAGE = base.D, 8, 64


@pytest.fixture(scope="module")
def pool(lib):
    """8 kv heads by 10240 tokens, and what they stand for in 64 bits, [tokens, heads, D]."""
    g = base._rng(100)
    pages = 160
    c = base._cache(lib, pages, PAGE, H, 32, 256, 8)
    slots = np.arange(pages * PAGE, dtype=np.int32)
    lib.kv_append(c, *(base._dev(base._heavy(g, len(slots), H), torch.float32) for _ in range(2)), base._dev(slots))
    return c, *(torch.tensor(x, device="cuda") for x in base._values(c, slots))


def _batch(g, lens, n, Hq, pages):
    """Tables of shuffled pages (sequences may share pages), trees, and a fused projection's heads."""
    B, most = len(lens), -(-max(lens) // PAGE)
    table = np.stack([g.permutation(pages)[:most] for _ in range(B)]).astype(np.int32)
    see = base._tree(g, B, n)
    qkv = base._dev(g.normal(size=(B, n, Hq + 2 * H, D)), torch.bfloat16)
    return table, see, qkv[:, :, :Hq], qkv[:, :, Hq:Hq + H], qkv[:, :, Hq + H:]


def _definition(pool, lens, table, see, q, kn, vn):
    _, pk, pv = pool
    B, n, Hq, _ = q.shape
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    for b, x in enumerate(lens):
        i = np.arange(x)
        at = torch.tensor(table[b, i // PAGE].astype(np.int64) * PAGE + i % PAGE, device="cuda")
        k = torch.cat([pk[at], kn[b].double()]).transpose(0, 1)  # [H, x + n, D]
        v = torch.cat([pv[at], vn[b].double()]).transpose(0, 1)
        r = q[b].double().unflatten(1, (H, Hq // H)).permute(1, 0, 2, 3).flatten(1, 2)  # [H, n * ratio, D]
        s = (r @ k.transpose(1, 2)) * D ** -0.5
        hide = ~base._dev(see[b]).repeat_interleave(Hq // H, 0)
        s[:, :, x:].masked_fill_(hide, float("-inf"))
        out[b] = (torch.softmax(s, -1) @ v).unflatten(1, (n, Hq // H)).permute(1, 0, 2, 3).flatten(1, 2)
    return out.cpu().numpy()


SHORT_AND_LONG = {
    "one_short_first": [50] + [8192] * 15,
    "two_of_one_step": [20, 20] + [8192] * 14,
    "short_in_the_middle": [8192] * 5 + [33, 64] + [8192] * 8,
    "short_last_and_empty": [8192] * 7 + [0, 1, 31, 0, 65, 32, 100, 7],
    "odd_steps": [5 * 32, 8192, 8 * 32 - 1, 8192, 3 * 32, 7 * 32, 8192, 8192 - 33, 8192, 33, 8192],
}


@pytest.mark.parametrize("n", [1, 4, 8, 32, 64])  # 4, 16, 32, 128 and 256 rows to a kv head
@pytest.mark.parametrize("lens", SHORT_AND_LONG.values(), ids=SHORT_AND_LONG.keys())
def test_short_contexts_beside_long_ones(lib, pool, lens, n):
    g = base._rng(101, n, *lens)
    c = pool[0]
    table, see, q, kn, vn = _batch(g, lens, n, 4 * H, c.pages)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = [lib.kv_attend_tree(c, q, base._dev(table), base._dev(lens, torch.int32), k_new=kn, v_new=vn,
                              mask=base._dev(base._pack_mask(see)), err=err) for _ in range(2)]
    assert lib.check_error(err) == 0
    assert torch.equal(*got)
    base._check(got[0], _definition(pool, lens, table, see, q, kn, vn))


@pytest.mark.parametrize("n", [2, 6, 20, 40])  # 8, 24, 80 and 160 rows to a kv head
def test_hundreds_of_ragged_contexts(lib, pool, n):
    g = base._rng(102, n)
    lens = [int(x) for x in g.integers(1, 301, 300)]
    for b in g.integers(0, 300, 12):
        lens[b] = int(g.integers(2000, 9000))
    c = pool[0]
    table, see, q, kn, vn = _batch(g, lens, n, 4 * H, c.pages)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = lib.kv_attend_tree(c, q, base._dev(table), base._dev(lens, torch.int32), k_new=kn, v_new=vn,
                             mask=base._dev(base._pack_mask(see)), err=err)
    assert lib.check_error(err) == 0
    base._check(got, _definition(pool, lens, table, see, q, kn, vn))


@pytest.mark.parametrize("n", [8, 64])
def test_nothing_of_a_call_is_left_running(lib, n):
    """No sequence holds a token: the workspace is the caller's again when the call's last launch is done."""
    g = base._rng(103, n)
    B, Hq = 512 // n, 4 * H
    c = base._cache(lib, 4, PAGE, H, 32, 256, 8)
    table, lens = torch.zeros((B, 4), dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    q, kn, vn = (base._dev(g.normal(size=(B, n, h, D)), torch.bfloat16) for h in (Hq, H, H))
    ws = torch.empty(c.tree_bytes(B, n, Hq, 256), dtype=torch.uint8, device="cuda")
    ref = lib.kv_attend_tree(c, q, table, lens, k_new=kn, v_new=vn)
    base._check(ref, base._attend(base._f64(q), [(np.zeros((0, H, D)),) * 2] * B, base._f64(kn), base._f64(vn),
                                  np.broadcast_to(np.tril(np.ones((n, n), bool)), (B, n, n)), None))
    for _ in range(20):
        got = lib.kv_attend_tree(c, q, table, lens, ws=ws)
        ws.fill_(0x5A)
        torch.cuda.synchronize()
        assert bool((ws == 0x5A).all())
        assert not bool(got.any())
        assert torch.equal(ref, lib.kv_attend_tree(c, q, table, lens, k_new=kn, v_new=vn, ws=ws))


@pytest.mark.parametrize("n", [1, 4, 16, 64])  # 4, 16, 64 and 256 rows to a kv head
def test_many_small_weights_beside_a_large_one(lib, n):
    """One token far above 32767 equal ones, whose values are 4000 times as large: their weights, 2^-20 to 2^-28 of its own,
    decide the result.  A weight is off by 2^-32 of the largest at most, beside the usual roundings."""
    g = base._rng(104)
    T, B, page, at = 32768, 152, 256, 5
    c = base._cache(lib, T // page, page, 1, 32, 256, 8)
    k, v = (torch.empty((T, 1, D), device="cuda") for _ in range(2))
    k[:] = base._dev(g.normal(size=D), torch.float32)
    v[:] = base._dev(g.normal(size=D) * 4000, torch.float32)
    k[at], v[at] = (base._dev(g.normal(size=(1, D)), torch.float32) for _ in range(2))
    lib.kv_append(c, k, v, torch.arange(T, dtype=torch.int32, device="cuda"))
    (k1, k0), (v1, v0) = ((x[0, 0], x[1, 0]) for x in base._values(c, np.array([at, 0])))
    q = torch.stack([base._dev((k1 - k0) * w, torch.bfloat16) for w in (20, 24.4, 25.1, 28)])
    q64 = base._f64(q)
    scale = np.log(2.0) / ((k1 - k0) @ (k1 - k0))
    weight = np.exp(-scale * (q64 @ (k1 - k0)))[:, None]  # of the others
    assert np.all(weight < 2.0 ** -19) and np.all(weight > 2.0 ** -29)
    ref = (v1 + (T - 1) * weight * v0) / (1 + (T - 1) * weight)
    table = torch.arange(T // page, dtype=torch.int32, device="cuda").repeat(B, 1)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = lib.kv_attend_tree(c, q.expand(B, n, 4, D).contiguous(), table, torch.full((B,), T, dtype=torch.int32, device="cuda"),
                             scale=float(scale), err=err)
    assert lib.check_error(err) == 0
    bound = base.ATTEND_ROW * np.linalg.norm(ref, axis=-1) + T * 2.0 ** -32 * np.linalg.norm(v0)
    off = np.linalg.norm(base._f64(got) - ref, axis=-1)
    assert np.all(off <= bound), (off / bound).max()
