"""Refusals of the page plan, the verification and the latent calls: decided on the host, before any CUDA call."""
import ctypes

import pytest

F = 0x1000  # an aligned address that is never read


@pytest.fixture(scope="module")
def tq():
    from rotated_codebook_quantized_gb300 import _build

    _build.build()
    import rotated_codebook_quantized_gb300 as tq

    tq.load()
    return tq


def test_plan_refusals(tq):
    lib, ref = tq.load(), ctypes.byref

    def call(pool=None, n=4, tokens=0, path=None, slots=F, starts=None, lens=F, **kw):
        p = dict(table=F, held=F, free=F, n_free=F, batch=3, width=8, page=64, pages=100)
        p.update(kw)
        return lib.tq_kv_plan(ref(tq.tq_page_pool_t(**p)), lens, F, path, n, tokens, slots, F, F, starts, None, None)

    assert lib.tq_kv_plan(None, F, F, None, 4, 0, F, F, F, None, None, None) == tq.TQ_ERR_INVALID
    for kw in (dict(page=48), dict(page=8), dict(page=512), dict(batch=-1), dict(width=-1), dict(pages=-1), dict(n=-1), dict(tokens=-1),
               dict(n=0, tokens=5), dict(n=0, tokens=5, starts=F, path=F), dict(starts=F), dict(held=None), dict(table=None),
               dict(free=None), dict(n_free=None), dict(lens=None), dict(slots=None), dict(slots=F + 2), dict(lens=F + 1)):
        assert call(**kw) == tq.TQ_ERR_INVALID, kw
    for kw in (dict(pages=(2 ** 31) // 64 + 1), dict(batch=2 ** 20 + 1), dict(batch=2 ** 20, n=2 ** 11), dict(n=0, tokens=2 ** 30 + 1, starts=F)):
        assert call(**kw) == tq.TQ_ERR_UNSUPPORTED, kw
    assert call(batch=0) == tq.TQ_OK  # nothing to do


def test_verify_refusals(tq):
    lib = tq.load()

    def call(p=F, ps=1000, q=None, qs=0, dt=tq.TQ_F32, B=2, n=3, V=1000, tokens=F, parent=F, u=F, path=F):
        return lib.tq_verify_tree(p, ps, q, qs, dt, B, n, V, tokens, parent, u, None, path, F, F, None, None)

    for kw in (dict(p=None), dict(ps=999), dict(q=F, qs=999), dict(dt=7), dict(B=-1), dict(n=-1), dict(V=-1), dict(n=0), dict(V=0),
               dict(tokens=None), dict(parent=None), dict(u=None), dict(path=None), dict(p=F + 2), dict(tokens=F + 2)):
        assert call(**kw) == tq.TQ_ERR_INVALID, kw
    for kw in (dict(n=1025), dict(V=2 ** 20 + 1, ps=2 ** 21), dict(B=2 ** 20 + 1)):
        assert call(**kw) == tq.TQ_ERR_UNSUPPORTED, kw
    assert call(B=0) == tq.TQ_OK


def _cache(tq, **kw):
    c = dict(rows=F, dt=tq.TQ_BF16, latent=512, rope=64, page=64, pages=10, page_stride=64)
    c.update(kw)
    return ctypes.byref(tq.tq_latent_pages_t(**c))


def test_latent_cache_refusals(tq):
    lib = tq.load()
    bytes_ = lambda **kw: lib.tq_latent_attend_tree_workspace_bytes(_cache(tq, **kw), 1, 1, 64, 640)  # noqa: E731
    assert bytes_() > 0
    for kw, want in ((dict(page=24), tq.TQ_ERR_INVALID), (dict(page=512), tq.TQ_ERR_INVALID), (dict(dt=tq.TQ_F32), tq.TQ_ERR_UNSUPPORTED),
                     (dict(dt=9), tq.TQ_ERR_INVALID), (dict(latent=256), tq.TQ_ERR_UNSUPPORTED), (dict(rope=32), tq.TQ_ERR_UNSUPPORTED),
                     (dict(page_stride=63), tq.TQ_ERR_INVALID), (dict(pages=-1), tq.TQ_ERR_INVALID), (dict(rows=None), tq.TQ_ERR_INVALID),
                     (dict(rows=F + 8), tq.TQ_ERR_INVALID), (dict(pages=2 ** 31 // 64 + 1), tq.TQ_ERR_UNSUPPORTED),
                     (dict(page_stride=2 ** 40), tq.TQ_ERR_UNSUPPORTED)):
        assert bytes_(**kw) == 0, kw
        assert lib.tq_latent_append(_cache(tq, **kw), F, 512, F, 64, tq.TQ_BF16, 4, F, None, None, None, None) == want, kw
        assert lib.tq_latent_attend_tree(_cache(tq, **kw), F, 64 * 576, 1, 1, 64, F, 10, F, 640, None, 0, None, None, 0.1, F, F, 1 << 40,
                                         None, None) == want, kw


def test_latent_append_refusals(tq):
    lib = tq.load()
    rope = lambda **kw: ctypes.byref(tq.tq_rope_t(**dict(dict(dim=64, rotary=64, layout=1, factor=1.0, steps=F), **kw)))  # noqa: E731

    def call(c=F, cs=512, k=F, ks=64, dt=tq.TQ_BF16, T=4, slots=F, rope=None, positions=None):
        return lib.tq_latent_append(_cache(tq), c, cs, k, ks, dt, T, slots, rope, positions, None, None)

    for kw in (dict(c=None), dict(cs=504), dict(cs=516), dict(k=None), dict(ks=60), dict(ks=68), dict(dt=5), dict(T=-1), dict(slots=None),
               dict(c=F + 8), dict(slots=F + 2), dict(rope=rope(), positions=None), dict(rope=rope(dim=128), positions=F),
               dict(rope=rope(rotary=63), positions=F), dict(rope=rope(steps=None), positions=F), dict(dt=tq.TQ_F32, cs=514)):
        assert call(**kw) == tq.TQ_ERR_INVALID, kw
    assert call(T=2 ** 41) == tq.TQ_ERR_UNSUPPORTED
    assert call(T=0, c=None, k=None, slots=None) == tq.TQ_OK


def test_latent_attend_tree_refusals(tq):
    lib = tq.load()

    def call(q=F, qs=64 * 576, B=2, n=3, H=64, table=F, ts=10, lens=F, most=640, fresh=F, fs=576, mask=None, scale=0.1, o=F, ws=F, nb=1 << 50):
        return lib.tq_latent_attend_tree(_cache(tq), q, qs, B, n, H, table, ts, lens, most, fresh, fs, mask, None, scale, o, ws, nb, None,
                                         None)

    for kw in (dict(q=None), dict(qs=64 * 576 - 8), dict(qs=64 * 576 + 4), dict(B=-1), dict(n=-1), dict(H=0), dict(H=65536), dict(table=None),
               dict(most=641), dict(most=-1), dict(lens=None), dict(fs=568), dict(fs=580), dict(scale=float("nan")), dict(scale=float("inf")),
               dict(o=None), dict(ws=None), dict(nb=8), dict(q=F + 2), dict(fresh=F + 2), dict(o=F + 8), dict(ws=F + 8), dict(mask=F + 4)):
        assert call(**kw) == tq.TQ_ERR_INVALID, kw
    for kw in (dict(B=2 ** 20, n=2 ** 10), dict(B=2 ** 16), dict(B=60000, n=400), dict(qs=2 ** 41), dict(fs=2 ** 41)):
        assert call(**kw) == tq.TQ_ERR_UNSUPPORTED, kw
    assert call(B=0) == tq.TQ_OK and call(n=0) == tq.TQ_OK


def test_latent_attend_prompt_refusals(tq):
    lib = tq.load()

    def call(q=F, qs=16 * 192, k=F, v=F, kvs=16 * 256, kvh=256, kr=F, krs=64, dt=tq.TQ_BF16, B=2, H=16, Tq=9, Tkv=9, starts=F, scale=0.1, o=F, ws=F, nb=1 << 30):
        return lib.tq_latent_attend_prompt(q, qs, k, v, kvs, kvh, kr, krs, dt, B, H, Tq, Tkv, starts, F, 1, scale, o, ws, nb, None, None)

    for kw in (dict(q=None), dict(qs=16 * 192 - 8), dict(qs=16 * 192 + 4), dict(k=None), dict(v=None), dict(kr=None), dict(kvs=15 * 256),
               dict(kvh=120), dict(kvh=252), dict(krs=56), dict(krs=68), dict(dt=5), dict(B=-1), dict(H=0), dict(H=65536), dict(Tq=-1),
               dict(Tkv=-1), dict(starts=None), dict(scale=float("nan")), dict(o=None), dict(q=F + 8), dict(k=F + 8), dict(v=F + 8),
               dict(kr=F + 8), dict(o=F + 8), dict(starts=F + 2), dict(ws=None),
               dict(ws=F + 2), dict(nb=3)):
        assert call(**kw) == tq.TQ_ERR_INVALID, kw
    for kw in (dict(dt=tq.TQ_F32), dict(Tq=2 ** 30 + 1), dict(Tkv=2 ** 30 + 1), dict(kvs=2 ** 33), dict(kvs=2 ** 32, kvh=2 ** 28)):
        assert call(**kw) == tq.TQ_ERR_UNSUPPORTED, kw
    need = lib.tq_latent_attend_prompt_workspace_bytes(2, 16, 9, 9000)  # (few tiles, many keys: partial results)
    assert need > 1 << 20 and call(Tkv=9000, nb=need - 1) == tq.TQ_ERR_INVALID
    assert call(B=0) == tq.TQ_OK and call(Tq=0) == tq.TQ_OK
