"""Host side of the rotary positions and the paged cache: frequencies against 64-bit numpy, and every refusal that the
C entry points make before any CUDA call (the pointers here are made up; nothing is launched)."""
import ctypes
import math

import numpy as np
import pytest

import rotated_codebook_quantized_gb300 as tq

FAKE = ctypes.c_void_p(0x1000)


@pytest.fixture(scope="module")
def lib():
    from rotated_codebook_quantized_gb300 import _build

    _build.build()
    return tq.load()


@pytest.mark.parametrize("rotary,base", [(2, 10000.0), (6, 10000.0), (64, 500000.0), (128, 10000.0), (128, 1.5)])
@pytest.mark.parametrize("scaling", [None, {"kind": "linear", "factor": 4.0}, {"kind": "base", "factor": 2.0},
                                     {"kind": "parts", "factor": 16.0, "original": 8192, "fast_turns": 24.0}])
def test_rope_steps(lib, rotary, base, scaling):
    steps, factor = tq.rope_steps(rotary, base, scaling)
    i = np.arange(0, rotary, 2, dtype=np.float64) / rotary
    w, f = base ** -i, 1.0
    if scaling and scaling["kind"] == "linear":
        w = w / 4
    if scaling and scaling["kind"] == "base":
        w = (base * 2.0 ** (rotary / max(rotary - 2, 1))) ** -i
        if rotary > 2:  # the slowest pair is slowed by exactly the factor
            assert abs(w[-1] * 2.0 / base ** -i[-1] - 1) < 1e-12
    if scaling and scaling["kind"] == "parts":
        keep = np.clip((8192 * w / (2 * math.pi) - 1) / 23.0, 0, 1)
        w, f = w * keep + w / 16 * (1 - keep), 0.1 * math.log(16) + 1
    turns = steps.view(np.uint64).astype(np.float64) / 2.0 ** 64
    # pow and the divisions: a few ulps of 2^-53; and the step is a whole number of 2^-64 turns
    np.testing.assert_allclose(turns, w / (2 * math.pi), rtol=1e-14, atol=2.0 ** -64)
    assert factor == np.float32(f)


def test_rope_steps_refusals(lib):
    out = (ctypes.c_uint64 * 64)()
    ok = lambda rotary=8, base=1e4, sc=None: lib.tq_rope_steps(rotary, base, sc, out, None)  # noqa: E731
    s = lambda *a: ctypes.byref(tq.tq_rope_scaling_t(*a))  # noqa: E731
    assert ok() == tq.TQ_OK and ok(sc=s(0, 0, 0, 0, 0)) == tq.TQ_OK and ok(sc=s(3, 2.0, 4096, 1, 32)) == tq.TQ_OK
    for bad in (ok(7), ok(0), ok(base=1.0), ok(base=float("nan")), ok(base=float("inf")), ok(sc=s(4, 2.0, 1, 1, 2)),
                ok(sc=s(1, 0.5, 0, 0, 0)), ok(sc=s(1, float("nan"), 0, 0, 0)), ok(sc=s(3, 2.0, 0.0, 1, 32)),
                ok(sc=s(3, 2.0, 4096, 32, 1)), ok(base=1e300, sc=s(2, 1e300, 0, 0, 0)),
                lib.tq_rope_steps(8, 1e4, None, None, None)):
        assert bad == tq.TQ_ERR_INVALID


def _rope(dim=128, rotary=128, layout=0, steps=0x1000):
    return tq.tq_rope_t(dim, rotary, layout, 1.0, steps)


def test_rope_refusals(lib):
    def call(rope=None, pos=FAKE, T=4, dt=tq.TQ_BF16, q=FAKE, qs=1024, hq=8, yq=FAKE, yqs=1024, k=None, ks=0, hk=0,
             yk=None, yks=0):
        r = rope if rope is not None else _rope()
        return lib.tq_rope(ctypes.byref(r), pos, T, dt, 0, q, qs, hq, yq, yqs, k, ks, hk, yk, yks, None)

    for bad in (call(_rope(rotary=3)), call(_rope(rotary=130)), call(_rope(layout=2)), call(_rope(steps=0)), call(T=-1),
                call(dt=3), call(qs=1023), call(yqs=1023), call(hq=-1), call(pos=None), call(q=None), call(yq=None),
                call(hk=1, ks=128, yks=128), call(qs=2048), call(q=ctypes.c_void_p(0x1001)),
                call(hk=1, k=FAKE, yk=FAKE, ks=127, yks=128), lib.tq_rope(None, FAKE, 1, 1, 0, FAKE, 1024, 8, FAKE, 1024,
                                                                         None, 0, 0, None, 0, None)):
        assert bad == tq.TQ_ERR_INVALID
    assert call(T=0, q=None) == tq.TQ_OK and call(hq=0, q=None) == tq.TQ_OK


def _pages(kl=256, vl=8, page=64, group=32, D=128, Hkv=8, pages=10, ps=512, hs=64, ptr=0x1000, signs=0x1000, block=128):
    cb = lambda n: tq.tq_codebook_t(n, 0x1000, 0x1000)  # noqa: E731
    return tq.tq_kv_pages_t(ptr, ptr, ptr, ptr, Hkv, D, group, page, pages, ps, hs, cb(kl), cb(vl),
                            tq.tq_rotation_t(D, block, signs))


BAD_POOLS = [(dict(D=64), 2), (dict(group=48), 1), (dict(page=8), 1), (dict(page=48), 1), (dict(page=512), 1), (dict(kl=8), 2),
             (dict(vl=256), 2), (dict(kl=5), 1), (dict(Hkv=0), 1), (dict(pages=-1), 1), (dict(ps=500), 1), (dict(hs=32), 1),
             (dict(ptr=0x1008), 1), (dict(ptr=0), 1), (dict(signs=0), 1), (dict(signs=0x1004), 1), (dict(block=64), 1), (dict(pages=1 << 26), 2)]


@pytest.mark.parametrize("change,status", BAD_POOLS)
def test_every_call_checks_the_pool(lib, change, status):
    c = ctypes.byref(_pages(**change))
    assert lib.tq_kv_append(c, FAKE, 1024, FAKE, 1024, 1, 4, FAKE, None, None, None, None) == status
    assert lib.tq_kv_fetch(c, FAKE, 4, FAKE, FAKE, 1, None, None) == status
    assert lib.tq_kv_attend_tree(c, FAKE, 1024, 1, 1, 1, 8, FAKE, 4, FAKE, 256, None, 0, None, 0, None, None, 1.0, FAKE,
                                 FAKE, 1 << 30, None, None) == status
    assert lib.tq_kv_attend_tree_workspace_bytes(c, 1, 1, 8, 256) == 0


def test_append_and_fetch_refusals(lib):
    c = ctypes.byref(_pages())

    def app(k=FAKE, ks=1024, v=FAKE, vs=1024, dt=tq.TQ_BF16, T=4, slots=FAKE, rope=None, pos=None):
        return lib.tq_kv_append(c, k, ks, v, vs, dt, T, slots, ctypes.byref(rope) if rope else None, pos, None, None)

    odd = ctypes.c_void_p(0x1004)
    for bad in (app(ks=1016), app(vs=1028), app(dt=tq.TQ_F16), app(T=-1), app(k=None), app(v=None), app(slots=None),
                app(k=odd), app(v=odd), app(rope=_rope()), app(rope=_rope(dim=64, rotary=64), pos=FAKE)):
        assert bad == tq.TQ_ERR_INVALID
    assert app(rope=_rope(rotary=96), pos=FAKE) == tq.TQ_ERR_UNSUPPORTED
    assert app(T=0, k=None) == tq.TQ_OK

    def get(slots=FAKE, T=4, k=FAKE, v=FAKE, dt=tq.TQ_BF16):
        return lib.tq_kv_fetch(c, slots, T, k, v, dt, None, None)

    for bad in (get(slots=None), get(T=-1), get(k=odd), get(v=odd), get(dt=3)):
        assert bad == tq.TQ_ERR_INVALID
    assert get(T=0) == tq.TQ_OK and get(k=None, v=None) == tq.TQ_OK


def test_tree_refusals(lib):
    c = ctypes.byref(_pages())
    big = lib.tq_kv_attend_tree_workspace_bytes(c, 2, 3, 16, 200)
    assert big > 0
    for zero in ((0, 3, 16, 200), (2, 0, 16, 200), (2, 3, 0, 200), (2, 3, 16, -1)):
        assert lib.tq_kv_attend_tree_workspace_bytes(c, *zero) == 0

    def call(q=FAKE, qs=2048, dt=tq.TQ_BF16, B=2, n=3, hq=16, table=FAKE, ts=4, lens=FAKE, most=200, k=FAKE, ks=1024, v=FAKE,
             vs=1024, mask=None, scale=0.1, o=FAKE, ws=FAKE, nb=big):
        return lib.tq_kv_attend_tree(c, q, qs, dt, B, n, hq, table, ts, lens, most, k, ks, v, vs, mask, None, scale, o, ws,
                                     nb, None, None)

    odd = ctypes.c_void_p(0x1008)
    for bad in (call(qs=2047), call(qs=2052), call(dt=7), call(B=-1), call(n=-1), call(hq=12), call(hq=0), call(table=None),
                call(ts=3), call(lens=None), call(most=-1), call(most=257), call(k=None), call(v=None), call(ks=1000),
                call(vs=1028), call(scale=float("nan")), call(o=None), call(ws=None), call(nb=big - 16), call(q=odd),
                call(o=odd), call(k=odd), call(ws=odd), call(mask=ctypes.c_void_p(0x1004)), call(q=None)):
        assert bad == tq.TQ_ERR_INVALID
    assert call(dt=tq.TQ_F32) == tq.TQ_ERR_UNSUPPORTED and call(dt=tq.TQ_F16) == tq.TQ_ERR_UNSUPPORTED
    assert call(B=0, q=None) == tq.TQ_OK and call(n=0, q=None) == tq.TQ_OK


@pytest.mark.parametrize("streams_share_steps", [False, True])
def test_wide_kernel_places_are_never_taken_early(streams_share_steps):
    """The hand-over of decoded steps in csrc/kv_tree_wide.cu, played with its own constants and every order of the roles
    that a slow stream allows: decoder warps wait for a place by its barrier's parity, the two streams free places out of
    order (each takes every other step) or together (each takes all).  No unit may be written before its place is free,
    and no step be read before it is whole."""
    import os
    import random
    import re

    src = open(os.path.join(os.path.dirname(tq.__file__), "csrc", "kv_tree_wide.cu")).read()
    const = lambda n: int(re.search(rf"constexpr int {n} = (\d+);", src).group(1))  # noqa: E731
    decoders, places = const("kDec"), const("kStages")
    per_step = const("kTok") // const("kUnit")
    steps, need = 40, 2 if streams_share_steps else 1
    for seed in range(40):
        rnd = random.Random(seed)
        freed, frees, wrote, whole = [0] * places, [0] * places, [0] * places, [0] * places
        unit, at = list(range(decoders)), [0, 0] if streams_share_steps else [0, 1]
        while min(at) < steps:
            moves = []
            for d in range(decoders):
                step, k = unit[d] // per_step % places, unit[d] // per_step // places
                if unit[d] < steps * per_step and freed[step] % 2 != (k - 1) % 2:
                    moves.append(("write", d))
            for s in range(2):
                if at[s] < steps and whole[at[s] % places] % 2 != at[s] // places % 2:
                    moves.append(("read", s))
            assert moves, "every role waits"
            kind, who = rnd.choice(moves)
            if kind == "read" and who == seed % 2 and len(moves) > 1 and rnd.random() < 0.95:
                continue  # one stream is slow
            if kind == "write":
                place, k = unit[who] // per_step % places, unit[who] // per_step // places
                assert freed[place] == k, "a place was written before it was free"
                unit[who] += decoders
                wrote[place] += 1
                if wrote[place] == per_step:
                    wrote[place], whole[place] = 0, whole[place] + 1
            else:
                place = at[who] % places
                assert whole[place] == at[who] // places + 1, "a step was read before it was whole"
                at[who] += 1 if streams_share_steps else 2
                frees[place] += 1
                if frees[place] == need:
                    frees[place], freed[place] = 0, freed[place] + 1


@pytest.mark.parametrize("change", [dict(pages=1 << 58), dict(pages=1 << 57, page=128, hs=128), dict(ps=1 << 60, pages=16), dict(ps=1 << 48),
                                    dict(hs=1 << 61), dict(hs=1 << 48)], ids=str)
def test_pools_past_64_bits_are_refused(lib, change):
    """Products of page counts, pages and strides that wrap around."""
    c = ctypes.byref(_pages(**change))
    assert lib.tq_kv_append(c, FAKE, 1024, FAKE, 1024, 1, 4, FAKE, None, None, None, None) == tq.TQ_ERR_UNSUPPORTED
    assert lib.tq_kv_fetch(c, FAKE, 4, FAKE, FAKE, 1, None, None) == tq.TQ_ERR_UNSUPPORTED
    assert lib.tq_kv_attend_tree(c, FAKE, 1024, 1, 1, 1, 8, FAKE, 4, FAKE, 64, None, 0, None, 0, None, None, 1.0, FAKE,
                                 FAKE, 1 << 30, None, None) == tq.TQ_ERR_UNSUPPORTED


@pytest.mark.parametrize("T", [1 << 61, (1 << 61) + 1, 1 << 60])
def test_token_counts_past_64_bits_are_refused(lib, T):
    """Eight heads to a token: the count of (token, head) pairs wraps around to a small one."""
    c = ctypes.byref(_pages())
    assert lib.tq_kv_append(c, FAKE, 1024, FAKE, 1024, 1, T, FAKE, None, None, None, None) == tq.TQ_ERR_UNSUPPORTED
    assert lib.tq_kv_fetch(c, FAKE, T, FAKE, FAKE, 1, None, None) == tq.TQ_ERR_UNSUPPORTED
    assert lib.tq_rope(ctypes.byref(_rope()), FAKE, T, tq.TQ_BF16, 0, FAKE, 1024, 8, FAKE, 1024, None, 0, 0, None, 0,
                       None) == tq.TQ_ERR_UNSUPPORTED


@pytest.mark.parametrize("B,n,hq,most", [(1 << 30, 1 << 20, 8, 64), (1 << 30, 1 << 30, 8, 64), (2 ** 31 - 1, 64, 65528, 0), (1, 1 << 30, 65528, 256),
                                         (1 << 28, 16, 8, 256), (1, 1, 8, 2 ** 31 - 1), (1 << 24, 1, 8, 1 << 20)])
def test_trees_past_the_counters_are_refused(lib, B, n, hq, most):
    """Rows, tiles or steps that the kernels' 32-bit counters do not hold, some of which wrap 64 bits too."""
    c = ctypes.byref(_pages())
    assert lib.tq_kv_attend_tree_workspace_bytes(c, B, n, hq, most) == 0
    assert lib.tq_kv_attend_tree(c, FAKE, hq * 128, 1, B, n, hq, FAKE, 1 << 26, FAKE, most, None, 0, None, 0, None, None, 1.0, FAKE,
                                 FAKE, 2 ** 63, None, None) == tq.TQ_ERR_UNSUPPORTED


def test_integer_arrays_are_aligned(lib):
    """Positions, slots, tables, lengths, counts and the error word are read as 32-bit numbers."""
    odd, c, r = ctypes.c_void_p(0x1002), ctypes.byref(_pages()), ctypes.byref(_rope())
    nb = lib.tq_kv_attend_tree_workspace_bytes(c, 1, 1, 8, 64)
    app = lambda slots=FAKE, pos=FAKE, err=None: lib.tq_kv_append(c, FAKE, 1024, FAKE, 1024, 1, 4, slots, r, pos, err, None)  # noqa: E731
    get = lambda slots=FAKE, err=None: lib.tq_kv_fetch(c, slots, 4, FAKE, FAKE, 1, err, None)  # noqa: E731
    tree = lambda table=FAKE, lens=FAKE, n_tok=None, err=None: lib.tq_kv_attend_tree(  # noqa: E731
        c, FAKE, 1024, 1, 1, 1, 8, table, 4, lens, 64, None, 0, None, 0, None, n_tok, 1.0, FAKE, FAKE, nb, err, None)
    for bad in (app(slots=odd), app(pos=odd), app(err=odd), get(slots=odd), get(err=odd), tree(table=odd), tree(lens=odd), tree(n_tok=odd),
                tree(err=odd), lib.tq_rope(r, odd, 4, 1, 0, FAKE, 1024, 8, FAKE, 1024, None, 0, 0, None, 0, None)):
        assert bad == tq.TQ_ERR_INVALID
