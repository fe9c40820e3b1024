"""Rotary positions, the paged compressed cache and the attention of drafted tokens over it, against 64-bit numpy.

Tolerances.  Rotary angles carry at most pi 2^-25 from the 24-bit phase and an ulp of sin and cos, so 4e-7 of the pair's
length; 16-bit results add half an ulp of their type (2^-8 bf16, 2^-11 fp16).  Codes and scales: bit-exact but for
counted ties (tests/helpers.py), the tie window 4e-6 where rotary positions come first (4e-7 of the vector's length,
up to sqrt(128) of its RMS in one rotated value).  Attention: the bf16 output's rounding (2^-9 / sqrt(3) to 2^-8 / sqrt(3) rms),
fp16 weights, values, keys and queries (2^-11 / sqrt(3) each; a score of deviation s moves a weight by about
2^-11 sqrt(2/3) s, s <= 4 here): 2.5e-3 together, 4e-3 allowed over a tensor and 1.2e-2 on a single row.
"""
import math

import numpy as np
import pytest

from oracle import tq_oracle as o
from tests import helpers

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

D = 128
ATTEND, ATTEND_ROW = 4e-3, 1.2e-2
ULP = {"float32": 0.0, "bfloat16": 2.0 ** -8, "float16": 2.0 ** -11}


def _rng(*key):
    return np.random.Generator(np.random.PCG64(list(key)))


def _dev(a, dtype=None):
    return torch.tensor(np.ascontiguousarray(a), device="cuda", dtype=dtype)


def _f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


# ---------------------------------------------------------------- rotary positions

def _freq(rotary, base=10000.0, scaling=None):
    w = base ** (-np.arange(0, rotary, 2, dtype=np.float64) / rotary)
    if not scaling:
        return w, 1.0
    f = scaling["factor"]
    if scaling["kind"] == "linear":
        return w / f, 1.0
    if scaling["kind"] == "base":
        return (base * f ** (rotary / (rotary - 2))) ** (-np.arange(0, rotary, 2, dtype=np.float64) / rotary), 1.0
    r = scaling["original"] * w / (2 * np.pi)
    keep = np.clip((r - scaling.get("slow_turns", 1.0)) / (scaling.get("fast_turns", 32.0) - scaling.get("slow_turns", 1.0)), 0, 1)
    return w * keep + w / f * (1 - keep), 0.1 * math.log(f) + 1.0


def _turn(x, pos, w, rotary, layout, factor=1.0, inverse=False):
    a = np.asarray(pos, np.float64)[:, None] * w[None] * (-1 if inverse else 1)
    c, s = np.cos(a)[:, None] * factor, np.sin(a)[:, None] * factor
    y = np.array(x, np.float64)
    if layout == "half":
        p, q = x[..., :rotary // 2], x[..., rotary // 2:rotary]
        y[..., :rotary // 2], y[..., rotary // 2:rotary] = p * c - q * s, p * s + q * c
    else:
        p, q = x[..., 0:rotary:2], x[..., 1:rotary:2]
        y[..., 0:rotary:2], y[..., 1:rotary:2] = p * c - q * s, p * s + q * c
    return y


def _pair_length(x, rotary, layout):
    """Length of the pair that each element belongs to (the element's own size past the rotated part)."""
    n = np.abs(np.array(x, np.float64))
    if layout == "half":
        m = np.hypot(x[..., :rotary // 2], x[..., rotary // 2:rotary])
        n[..., :rotary // 2] = n[..., rotary // 2:rotary] = m
    else:
        n[..., 0:rotary:2] = n[..., 1:rotary:2] = np.hypot(x[..., 0:rotary:2], x[..., 1:rotary:2])
    return n


def _check_turn(got, x, ref, rotary, layout, factor=1.0):
    ulp = ULP[str(got.dtype).split(".")[1]]
    bound = ulp * np.abs(ref) * 1.01 + 4e-7 * factor * _pair_length(x, rotary, layout) + 1e-12
    if ulp == 2.0 ** -11:
        bound += 2.0 ** -25  # fp16's subnormals
    assert np.all(np.abs(_f64(got) - ref) <= bound)


@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("T,hq,hkv,dim,rotary,start", [
    (1, 1, 1, 128, 128, 0), (1, 32, 8, 128, 128, 131071), (7, 3, 1, 128, 64, 1 << 20), (33, 5, 2, 96, 24, 4000),
    (130, 4, 4, 64, 64, 0), (5, 2, 1, 256, 256, 77), (9, 6, 3, 80, 80, 5), (3, 1, 1, 10, 6, 1 << 30), (4, 2, 2, 2, 2, 9),
    (1000, 8, 2, 128, 32, 0)])
def test_rope_matches_the_definition(lib, dtype, layout, T, hq, hkv, dim, rotary, start):
    g = _rng(1, T, hq, dim, rotary)
    dt = getattr(torch, dtype)
    qkv = _dev(g.normal(size=(T, hq + 2 * hkv, dim)) * 3, torch.float32).to(dt)
    q, k = qkv[:, :hq], qkv[:, hq:hq + hkv]  # views of a fused projection
    before = qkv.clone()
    pos = (g.integers(-3, 4096, T) + start).clip(max=2 ** 31 - 1)
    r = lib.Rope(dim, rotary, layout=layout)
    w, _ = _freq(rotary)
    yq, yk = lib.rope(q, _dev(pos, torch.int32), r, k=k)
    assert yq.shape == q.shape and yk.shape == k.shape and yq.dtype == dt and yq.is_contiguous()
    for y, x in ((yq, q), (yk, k)):
        _check_turn(y, _f64(x), _turn(_f64(x), pos, w, rotary, layout), rotary, layout)
    assert torch.equal(before, qkv)
    # the query heads alone, and the same in place on the strided views
    assert torch.equal(lib.rope(q, _dev(pos, torch.int32), r), yq)
    lib.rope(q, _dev(pos, torch.int32), r, k=k, inplace=True)
    assert torch.equal(q, yq) and torch.equal(k, yk) and torch.equal(qkv[:, hq + hkv:], before[:, hq + hkv:])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_inverse_is_the_transpose(lib, layout):
    """<rope(x), y> = <x, inverse(y)> (its gradient), and inverse(rope(x)) = x for a factor of 1."""
    g = _rng(2)
    T, H = 37, 6
    x, y = (_dev(g.normal(size=(T, H, D)), torch.float32) for _ in range(2))
    pos = _dev(g.integers(0, 100000, T), torch.int32)
    r = lib.Rope(D, 96, layout=layout)
    fx, gy = lib.rope(x, pos, r), lib.rope(y, pos, r, inverse=True)
    w, _ = _freq(96)
    _check_turn(gy, _f64(y), _turn(_f64(y), pos.cpu().numpy(), w, 96, layout, inverse=True), 96, layout)
    a, b = float((fx.double() * y.double()).sum()), float((x.double() * gy.double()).sum())
    assert abs(a - b) <= 8e-7 * float(x.double().norm() * y.double().norm())
    assert float((lib.rope(fx, pos, r, inverse=True) - x).abs().max()) < 8e-7 * 8


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_gradient_against_differences(lib, layout):
    """L(x) = <rope(x), y> is linear: its differences in each of 24 directions are <direction, inverse(y)>, whatever the step."""
    g = _rng(21)
    T, H = 5, 3
    x, y = (_dev(g.normal(size=(T, H, D)), torch.float32) for _ in range(2))
    pos = _dev(g.integers(0, 100000, T), torch.int32)
    r = lib.Rope(D, 64, layout=layout, scaling={"kind": "parts", "factor": 16.0, "original": 8192})
    grad = lib.rope(y, pos, r, inverse=True)
    for _ in range(24):
        d = _dev(g.normal(size=(T, H, D)), torch.float32)
        up, down = (float((lib.rope(z, pos, r).double() * y.double()).sum()) for z in (x + d, x - d))
        # six fp32 roundings of 2^-24 a result, of sums of |x| + |d| over the norm of y; x + d itself another two
        assert abs((up - down) / 2 - float((d.double() * grad.double()).sum())) <= 8 * 2 ** -24 * r.factor * float(
            (x.double().abs() + d.double().abs()).norm() * y.double().norm())


@pytest.mark.parametrize("scaling", [None, {"kind": "linear", "factor": 4.0}, {"kind": "base", "factor": 8.0},
                                     {"kind": "parts", "factor": 16.0, "original": 8192},
                                     {"kind": "parts", "factor": 4.0, "original": 4096, "slow_turns": 2.0, "fast_turns": 20.0}])
def test_rope_scaled_frequencies(lib, scaling):
    g = _rng(3)
    T = 65
    pos = np.concatenate([[0, 1, 8191, 8192, 131071], g.integers(0, 131072, T - 5)])
    x = _dev(g.normal(size=(T, 2, D)), torch.float32)
    r = lib.Rope(D, base=500000.0, scaling=scaling)
    w, factor = _freq(D, 500000.0, scaling)
    assert abs(r.factor - factor) < 1e-6
    ref = _turn(_f64(x), pos, w, D, "half", r.factor)
    _check_turn(lib.rope(x, _dev(pos, torch.int32), r), _f64(x), ref, D, "half", factor)


def test_rope_odd_alignment_and_nothing(lib):
    """Rows that start at an odd element, and calls with no tokens."""
    g = _rng(4)
    T, H, dim = 11, 3, 64
    buf = torch.zeros(T * (H * dim + 3) + 5, device="cuda", dtype=torch.bfloat16)
    x = buf[1:1 + T * (H * dim + 3)].view(T, H * dim + 3)[:, 1:1 + H * dim].unflatten(1, (H, dim))
    x.copy_(_dev(g.normal(size=(T, H, dim)), torch.float32))
    pos = g.integers(0, 9999, T)
    w, _ = _freq(dim)
    r = lib.Rope(dim)
    _check_turn(lib.rope(x, _dev(pos, torch.int32), r), _f64(x), _turn(_f64(x), pos, w, dim, "half"), dim, "half")
    empty = torch.zeros((0, H, dim), device="cuda")
    assert lib.rope(empty, torch.zeros(0, dtype=torch.int32, device="cuda"), r).shape == (0, H, dim)


def test_rope_refusals(lib):
    x = torch.zeros((4, 2, 64), device="cuda")
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    r = lib.Rope(64)
    for bad in (lambda: lib.Rope(64, 7), lambda: lib.Rope(64, 66), lambda: lib.Rope(64, layout="spiral"),
                lambda: lib.Rope(64, scaling={"kind": "no", "factor": 2}),
                lambda: lib.Rope(64, steps=torch.zeros(31, dtype=torch.int64)),
                lambda: lib.rope(x, pos[:3], r), lambda: lib.rope(x, pos.long(), r), lambda: lib.rope(x[..., :32], pos, r),
                lambda: lib.rope(x.transpose(0, 1), pos[:2], r), lambda: lib.rope(x, pos, r, k=x.half()),
                lambda: lib.rope(x.cpu(), pos, r)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: lib.Rope(64, base=0.5), lambda: lib.Rope(64, scaling={"kind": "linear", "factor": 0.5}),
                lambda: lib.Rope(64, scaling={"kind": "parts", "factor": 2.0})):
        with pytest.raises(lib.TQError):
            bad()


# ---------------------------------------------------------------- the paged cache

def _cache(lib, pages, page, heads, group, kl, vl, poison=True):
    rot = lib.Rotation(D, D, seed=77)
    c = lib.PagedKVCache(pages, page, heads, D, group, lib.Codebook(kl), lib.Codebook(vl), rot)
    if poison:  # what free slots hold must never matter
        c.kcodes.fill_(-1)
        c.vcodes.fill_(-1)
        c.kscales.fill_(0x7E00)  # fp16 NaN
        c.vscales.fill_(0x7C00)  # fp16 infinity
    return c


def _signs():
    return o.rotation_signs(77, D)


def _slots(g, T, page, pages, spare=0):
    """Slots of T consecutive tokens on shuffled pages, and the page list."""
    order = g.permutation(pages)[:-(-T // page)]
    i = np.arange(T)
    return (order[i // page] * page + i % page).astype(np.int32), order.astype(np.int32)


def _rows(t, slots, page):
    """[T, heads, words] of a pool tensor [pages, heads, page, words]."""
    s = torch.as_tensor(np.asarray(slots, np.int64), device=t.device)
    return t[s // page, :, s % page]


def _values(cache, slots):
    """What the cache holds at the slots, in 64 bits, de-rotated: k, v [T, heads, D]."""
    if not len(slots):
        return [np.zeros((0, cache.heads, D))] * 2
    out = []
    for codes, scales, cb in ((cache.kcodes, cache.kscales, cache.kcb), (cache.vcodes, cache.vscales, cache.vcb)):
        w = helpers.u32(_rows(codes, slots, cache.page))
        T, H = w.shape[:2]
        c = o.unpack(w.reshape(T * H, -1), cb.levels, D)
        s = helpers.f16_from_bits(_rows(scales, slots, cache.page)).reshape(T * H, -1)
        v = o.dequantize(c, s, cb.centroids.cpu().numpy().astype(np.float64), cache.group)
        out.append((v @ o.rotation_matrix(_signs(), D)).reshape(T, H, D))
    return out


BOOKS = [(256, 8), (256, 16), (16, 16), (16, 8)]


def _heavy(g, T, H):
    return g.normal(size=(T, H, D)) * np.exp(0.7 * g.normal(size=(1, H, D)).clip(-2, 2))


@pytest.mark.parametrize("kl,vl", BOOKS)
@pytest.mark.parametrize("group", [16, 32, 64, 128])
@pytest.mark.parametrize("T,H,page,dtype", [(1, 1, 16, "bfloat16"), (37, 3, 32, "float32"), (131, 8, 64, "bfloat16")])
def test_append_writes_the_codes_of_the_definition(lib, kl, vl, group, T, H, page, dtype):
    g = _rng(5, T, H, group, kl, vl)
    pages = -(-T // page) + 2
    c = _cache(lib, pages, page, H, group, kl, vl)
    slots, _ = _slots(g, T, page, pages)
    kv = _dev(np.concatenate([_heavy(g, T, H), _heavy(g, T, H)], 1), torch.float32).to(getattr(torch, dtype))
    kv[T // 2, 0] = 0  # an all-zero vector
    k, v = kv[:, :H], kv[:, H:]
    lib.kv_append(c, k, v, _dev(slots))
    R = o.rotation_matrix(_signs(), D)
    for x, codes, scales, levels in ((k, c.kcodes, c.kscales, kl), (v, c.vcodes, c.vscales, vl)):
        _, thr = o.lloyd_max_gaussian(levels)
        y = _f64(x).reshape(T * H, D) @ R.T
        u, rms = helpers.oracle_u(y, group)
        oc, os16 = o.encode_rotated(y, group, thr)
        helpers.compare_codes(helpers.u32(_rows(codes, slots, page)).reshape(T * H, -1), o.pack(oc, levels), levels, D, u, thr)
        helpers.compare_scales(helpers.f16_from_bits(_rows(scales, slots, page)).reshape(T * H, -1), os16, rms)
    untouched = np.setdiff1d(np.arange(pages * page), slots)
    assert bool((_rows(c.kcodes, untouched, page) == -1).all()) and bool((_rows(c.vscales, untouched, page) == 0x7C00).all())


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("rotary", [32, 64, 128])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_append_turns_keys_on_the_way(lib, layout, rotary, dtype):
    g = _rng(6, rotary)
    T, H, page = 45, 4, 16
    c = _cache(lib, 4, page, H, 32, 256, 8)
    slots, _ = _slots(g, T, page, 4)
    k, v = (_dev(_heavy(g, T, H), torch.float32).to(getattr(torch, dtype)) for _ in range(2))
    pos = g.integers(0, 131072, T)
    r = lib.Rope(D, rotary, layout=layout, scaling={"kind": "parts", "factor": 4.0, "original": 4096})
    lib.kv_append(c, k, v, _dev(slots), rope=r, positions=_dev(pos, torch.int32))
    w, _ = _freq(rotary, scaling={"kind": "parts", "factor": 4.0, "original": 4096})
    y = _turn(_f64(k), pos, w, rotary, layout, r.factor).reshape(T * H, D) @ o.rotation_matrix(_signs(), D).T
    cent, thr = o.lloyd_max_gaussian(256)
    u, rms = helpers.oracle_u(y, 32)
    oc, os16 = o.encode_rotated(y, 32, thr)
    gc = o.unpack(helpers.u32(_rows(c.kcodes, slots, page)).reshape(T * H, -1), 256, D)
    off = np.argwhere(gc != oc)
    for i, j in off:
        assert abs(int(gc[i, j]) - int(oc[i, j])) == 1
        assert abs(u[i, j] - thr[min(gc[i, j], oc[i, j])]) <= 4e-6 * max(1.0, abs(u[i, j]))
    plain = _cache(lib, 4, page, H, 32, 256, 8)
    lib.kv_append(plain, k, v, _dev(slots))
    assert torch.equal(_rows(plain.vcodes, slots, page), _rows(c.vcodes, slots, page))  # values do not turn


def _compare_written(c, x, codes, scales, levels, thr, slots, group, tie=None):
    """Codes and scales of tokens x (64 bits) against the definition; tie: the bar on a mismatched u, if not the helpers' own."""
    T, H = x.shape[:2]
    y = x.reshape(T * H, D) @ o.rotation_matrix(_signs(), D).T
    u, rms = helpers.oracle_u(y, group)
    oc, os16 = o.encode_rotated(y, group, thr)
    words = helpers.u32(_rows(codes, slots, c.page)).reshape(T * H, -1)
    if tie is None:
        helpers.compare_codes(words, o.pack(oc, levels), levels, D, u, thr)
        helpers.compare_scales(helpers.f16_from_bits(_rows(scales, slots, c.page)).reshape(T * H, -1), os16, rms)
        return
    gc = o.unpack(words, levels, D)
    for i, j in np.argwhere(gc != oc):
        assert abs(int(gc[i, j]) - int(oc[i, j])) == 1
        assert abs(u[i, j] - thr[min(gc[i, j], oc[i, j])]) <= tie * max(1.0, abs(u[i, j]))


# more (token, head) pairs than the calls above, which another kernel takes: whole tables, eight tokens to a warp
@pytest.mark.parametrize("kl,vl", BOOKS)
@pytest.mark.parametrize("group", [16, 32, 64, 128])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("close", [False, True])
def test_append_of_many_tokens(lib, kl, vl, group, dtype, close):
    """close: books whose thresholds lie a quarter as far apart, several to a bin of the lookup."""
    if close and (group, dtype) not in ((32, "bfloat16"), (128, "float32")):
        pytest.skip("the search does not depend on them")
    g = _rng(25, group, kl, vl)
    T, H, page = 605, 7, 64
    pages = -(-T // page) + 2
    c = _cache(lib, pages, page, H, group, kl, vl)
    thrs = []
    for name, levels in (("kcb", kl), ("vcb", vl)):
        cent, thr = o.lloyd_max_gaussian(levels)
        if close:
            cent, thr = np.float32(cent * 0.25).astype(np.float64), np.float32(thr * 0.25).astype(np.float64)
            for t, v in ((getattr(c, name).centroids, cent), (getattr(c, name).thresholds, thr)):
                t.copy_(_dev(v, torch.float32))
        thrs.append(thr)
    slots, _ = _slots(g, T, page, pages)
    slots[[5, 300]] = -1  # skipped
    kv = _dev(np.concatenate([_heavy(g, T, H), _heavy(g, T, H)], 1), torch.float32).to(getattr(torch, dtype))
    kv[T // 2, 0] = 0  # an all-zero vector
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    lib.kv_append(c, kv[:, :H], kv[:, H:], _dev(slots), err=err)
    assert lib.check_error(err) == 0
    kept = slots >= 0
    for x, codes, scales, levels, thr in ((kv[:, :H], c.kcodes, c.kscales, kl, thrs[0]), (kv[:, H:], c.vcodes, c.vscales, vl, thrs[1])):
        _compare_written(c, _f64(x)[kept], codes, scales, levels, thr, slots[kept], group)
    untouched = np.setdiff1d(np.arange(pages * page), slots)
    assert bool((_rows(c.kcodes, untouched, page) == -1).all()) and bool((_rows(c.vscales, untouched, page) == 0x7C00).all())
    slots[7] = pages * page  # outside the pool
    lib.kv_append(c, kv[:, :H], kv[:, H:], _dev(slots), err=err)
    assert lib.check_error(err) == lib.TQ_DEVERR_BAD_PAGE
    assert bool((_rows(c.kcodes, untouched, page) == -1).all())


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("rotary", [32, 64, 128])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("T,H", [(841, 5), (9800, 5)])  # one head to a warp, and four (and the fifth)
def test_append_turns_keys_of_many_tokens(lib, layout, rotary, dtype, T, H):
    g = _rng(26, rotary, T)
    page = 64
    pages = -(-T // page)
    c, plain = (_cache(lib, pages, page, H, 32, 256, 8) for _ in range(2))
    slots, _ = _slots(g, T, page, pages)
    k, v = (_dev(_heavy(g, T, H), torch.float32).to(getattr(torch, dtype)) for _ in range(2))
    pos = g.integers(0, 131072, T)
    scaling = {"kind": "parts", "factor": 4.0, "original": 4096}
    r = lib.Rope(D, rotary, layout=layout, scaling=scaling)
    lib.kv_append(c, k, v, _dev(slots), rope=r, positions=_dev(pos, torch.int32))
    lib.kv_append(plain, k, v, _dev(slots))
    assert torch.equal(_rows(plain.vcodes, slots, page), _rows(c.vcodes, slots, page))  # values do not turn
    at = g.permutation(T)[:800]  # of which the definition is computed
    w, _ = _freq(rotary, scaling=scaling)
    y = _turn(_f64(k)[at], pos[at], w, rotary, layout, r.factor)
    _compare_written(c, y, c.kcodes, c.kscales, 256, o.lloyd_max_gaussian(256)[1], slots[at], 32, tie=4e-6)


def test_append_equals_the_contiguous_cache(lib):
    """The same tokens through kv_quantize and through pages over the same storage, but for counted ties."""
    g = _rng(7)
    T, H, cap = 200, 8, 256
    rot = lib.Rotation(D, D, seed=77)
    a, b = (lib.KVCache(cap, H, D, 32, lib.Codebook(256), lib.Codebook(8), rot) for _ in range(2))
    k, v = (_dev(_heavy(g, T, H), torch.float32).to(torch.bfloat16) for _ in range(2))
    lib.kv_quantize(a, k, v)
    lib.kv_append(lib.PagedKVCache.of(b), k, v, torch.arange(T, dtype=torch.int32, device="cuda"))
    for x, y in ((a.kcodes, b.kcodes), (a.vcodes, b.vcodes)):
        assert float((x != y).float().mean()) < 1e-4
    assert float((a.kscales.int() - b.kscales.int()).abs().max()) <= 1 and int((a.kscales != b.kscales).sum()) <= 8


def test_append_and_fetch_skip_and_flag_slots(lib):
    g = _rng(8)
    T, H, page = 40, 2, 16
    c = _cache(lib, 4, page, H, 32, 256, 8)
    k, v = (_dev(_heavy(g, T, H), torch.float32) for _ in range(2))
    slots = g.permutation(4 * page)[:T].astype(np.int32)
    slots[[3, 17]] = -1
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    lib.kv_append(c, k, v, _dev(slots), err=err)
    assert lib.check_error(err) == 0
    free = np.setdiff1d(np.arange(4 * page), slots)
    assert bool((_rows(c.kcodes, free, page) == -1).all())
    fk, fv = lib.kv_fetch(c, _dev(slots), out_dtype=torch.float32, err=err)
    assert lib.check_error(err) == 0
    assert bool((fk[[3, 17]] == 0).all()) and bool((fv[[3, 17]] == 0).all())
    live = slots >= 0
    for got, ref in zip((fk, fv), _values(c, slots[live])):
        np.testing.assert_allclose(_f64(got)[live], ref, rtol=0, atol=2e-6 * np.abs(ref).max())
    past = slots.copy()
    past[5], past[6] = 4 * page, 2 ** 31 - 1
    keep = c.kcodes.clone()
    lib.kv_append(c, k, v, _dev(past), err=err)
    assert lib.check_error(err) == lib.TQ_DEVERR_BAD_PAGE
    assert torch.equal(keep, c.kcodes)
    fk, _ = lib.kv_fetch(c, _dev(past), out_dtype=torch.float32, err=err)
    assert lib.check_error(err) == lib.TQ_DEVERR_BAD_PAGE and bool((fk[5:7] == 0).all())


@pytest.mark.parametrize("kl,vl", BOOKS)
@pytest.mark.parametrize("group", [16, 32, 64, 128])
@pytest.mark.parametrize("T,H,page,out", [(1, 8, 16, "bfloat16"), (53, 3, 64, "float16"), (300, 1, 128, "float32")])
def test_fetch_reads_what_the_codes_stand_for(lib, kl, vl, group, T, H, page, out):
    g = _rng(9, T, group, kl, vl)
    pages = -(-T // page) + 1
    c = _cache(lib, pages, page, H, group, kl, vl)
    slots, _ = _slots(g, T, page, pages)
    lib.kv_append(c, *(_dev(_heavy(g, T, H), torch.float32) for _ in range(2)), _dev(slots))
    order = g.permutation(T)  # any order, and slots read twice
    ask = np.concatenate([slots[order], slots[:1]])
    k, v = lib.kv_fetch(c, _dev(ask), out_dtype=getattr(torch, out))
    assert k.shape == (T + 1, H, D) and k.dtype == getattr(torch, out)
    for got, ref in zip((k, v), _values(c, ask)):
        # fp32 products and seven levels of sums: 8 roundings of values up to the vector's length
        bound = ULP[out] * np.abs(ref) * 1.01 + 8 * 2.0 ** -24 * np.linalg.norm(ref, axis=-1, keepdims=True) + 1e-12
        assert np.all(np.abs(_f64(got) - ref) <= bound)


def test_cache_rows_past_32_bit_offsets(lib):
    """A pool whose code words do not fit a signed 32-bit index: written, read and attended at its far end."""
    g = _rng(10)
    H, page, pages = 8, 128, 70000
    assert pages * H * page * 32 > 2 ** 31
    rot = lib.Rotation(D, D, seed=77)
    kw, vw = lib.row_words(256, D), lib.row_words(8, D)
    store = tuple(torch.empty((pages, H, page, n), dtype=t, device="cuda")
                  for n, t in ((kw, torch.int32), (4, torch.int16), (vw, torch.int32), (4, torch.int16)))
    c = lib.PagedKVCache(pages, page, H, D, 32, lib.Codebook(256), lib.Codebook(8), rot, storage=store)
    T = 200
    table = np.array([[pages - 1, pages - 3]], np.int32)
    i = np.arange(T)
    slots = (table[0, i // page].astype(np.int64) * page + i % page).astype(np.int32)
    k, v = (_dev(_heavy(g, T, H), torch.float32) for _ in range(2))
    lib.kv_append(c, k, v, _dev(slots))
    fk, fv = lib.kv_fetch(c, _dev(slots), out_dtype=torch.float32)
    rk, rv = _values(c, slots)
    np.testing.assert_allclose(_f64(fk), rk, rtol=0, atol=2e-6 * np.abs(rk).max())
    assert helpers.rel_l2(_f64(fk), _f64(k)) < 0.02 and helpers.rel_l2(_f64(fv), _f64(v)) < 0.25
    q = _dev(g.normal(size=(1, 1, 16, D)), torch.bfloat16)
    got = lib.kv_attend_tree(c, q, _dev(table), _dev([T], torch.int32))
    ref = _attend(_f64(q), [(rk, rv)], None, None, None, None)
    assert helpers.rel_l2(_f64(got), ref) < ATTEND


# ---------------------------------------------------------------- attention of drafted tokens

def _attend(q, contexts, kn, vn, see, n_tok, scale=None):
    """64-bit reference.  contexts: (k, v) [len, heads, D] of each sequence; see: bool [B, n, n]."""
    B, n, Hq, _ = q.shape
    out = np.zeros_like(q)
    for b in range(B):
        k, v = contexts[b]
        m = n if n_tok is None else n_tok[b]
        H = k.shape[1]
        for i in range(m):
            kk, vv = k, v
            if kn is not None:
                j = np.nonzero(see[b, i, :m])[0]
                kk, vv = np.concatenate([k, kn[b, j]]), np.concatenate([v, vn[b, j]])
            if not len(kk):
                continue
            for h in range(Hq):
                s = kk[:, h // (Hq // H)] @ q[b, i, h] * (D ** -0.5 if scale is None else scale)
                p = np.exp(s - s.max())
                out[b, i, h] = (p / p.sum()) @ vv[:, h // (Hq // H)]
    return out


def _pack_mask(see):
    B, n, _ = see.shape
    full = np.zeros((B, n, -(-n // 64) * 64), bool)
    full[:, :, :n] = see
    return np.packbits(full, axis=-1, bitorder="little").view(np.int64)


def _tree(g, B, n):
    see = np.zeros((B, n, n), bool)
    for b in range(B):
        for i in range(n):
            p = int(g.integers(-1, i)) if i else -1
            if p >= 0:
                see[b, i] = see[b, p]
            see[b, i, i] = True
    return see


def _setup(lib, key, lens, n, Hq, H, page=16, group=32, kl=256, vl=8, spread=1.0):
    g = _rng(11, *key)
    B = len(lens)
    need = [-(-x // page) for x in lens]
    order = g.permutation(sum(need) + 1).astype(np.int32)
    c = _cache(lib, len(order), page, H, group, kl, vl)
    table = np.full((B, max(1, max(need))), 2 ** 31 - 1, np.int32)  # entries past a sequence's pages are not read
    at, contexts = 0, []
    for b, x in enumerate(lens):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
        i = np.arange(x)
        slots = (table[b, i // page] * page + i % page).astype(np.int32)
        if x:
            lib.kv_append(c, *(_dev(_heavy(g, x, H) * spread, torch.float32) for _ in range(2)), _dev(slots))
        contexts.append(_values(c, slots))
    qkv = _dev(_heavy(g, B * n, Hq + 2 * H), torch.bfloat16).view(B, n, Hq + 2 * H, D)
    return g, c, _dev(table), _dev(lens, torch.int32), contexts, qkv[:, :, :Hq], qkv[:, :, Hq:Hq + H], qkv[:, :, Hq + H:]


def _check(got, ref):
    got = _f64(got)
    assert np.all(np.isfinite(got))
    assert helpers.rel_l2(got, ref) < ATTEND
    norm = np.linalg.norm(ref, axis=-1)
    off = np.linalg.norm(got - ref, axis=-1)
    assert np.all(off <= ATTEND_ROW * norm + 1e-30), (off / np.maximum(norm, 1e-30)).max()


@pytest.mark.parametrize("lens,n,Hq,H,page", [
    ([1], 1, 1, 1, 16), ([0], 1, 4, 1, 16), ([17], 1, 8, 2, 16), ([300], 4, 32, 8, 64), ([0, 5, 64, 65], 5, 8, 2, 32),
    ([1000], 16, 8, 2, 64), ([257, 0, 31], 13, 6, 2, 16), ([128, 511], 33, 4, 1, 128), ([90], 64, 16, 2, 256),
    ([700], 70, 4, 2, 64), ([40, 1], 129, 3, 1, 16), ([2048], 3, 20, 4, 32), ([63], 7, 12, 1, 16), ([1025], 2, 64, 2, 64)])
def test_tree_matches_the_definition(lib, lens, n, Hq, H, page):
    g, c, table, dlens, ctx, q, kn, vn = _setup(lib, (1, *lens, n, Hq), lens, n, Hq, H, page)
    see = _tree(g, len(lens), n)
    got = lib.kv_attend_tree(c, q, table, dlens, k_new=kn, v_new=vn, mask=_dev(_pack_mask(see)), max_len=max(lens))
    assert got.shape == q.shape and got.dtype == torch.bfloat16
    _check(got, _attend(_f64(q), ctx, _f64(kn), _f64(vn), see, None))


@pytest.mark.parametrize("kl,vl", BOOKS)
@pytest.mark.parametrize("group", [16, 32, 64, 128])
@pytest.mark.parametrize("n,Hq,H", [(1, 4, 1), (9, 6, 2), (40, 4, 1)])
def test_tree_books_and_groups(lib, kl, vl, group, n, Hq, H):
    lens = [333, 70]
    g, c, table, dlens, ctx, q, kn, vn = _setup(lib, (2, kl, vl, group, n), lens, n, Hq, H, 32, group, kl, vl)
    see = _tree(g, 2, n)
    got = lib.kv_attend_tree(c, q, table, dlens, k_new=kn, v_new=vn, mask=_dev(_pack_mask(see)))
    _check(got, _attend(_f64(q), ctx, _f64(kn), _f64(vn), see, None))


@pytest.mark.parametrize("length", [4095, 20000])
@pytest.mark.parametrize("n", [1, 6])
def test_tree_long_context(lib, length, n):
    g, c, table, dlens, ctx, q, kn, vn = _setup(lib, (3, length, n), [length, length // 3], n, 4, 1, 64)
    see = _tree(g, 2, n)
    got = lib.kv_attend_tree(c, q, table, dlens, k_new=kn, v_new=vn, mask=_dev(_pack_mask(see)))
    _check(got, _attend(_f64(q), ctx, _f64(kn), _f64(vn), see, None))


@pytest.mark.parametrize("n", [1, 5, 64, 100, 300])
def test_tree_without_a_mask_is_a_chain(lib, n):
    g, c, table, dlens, ctx, q, kn, vn = _setup(lib, (4, n), [50], n, 4, 2)
    see = np.tril(np.ones((1, n, n), bool))
    got = lib.kv_attend_tree(c, q, table, dlens, k_new=kn, v_new=vn)
    _check(got, _attend(_f64(q), ctx, _f64(kn), _f64(vn), see, None))
    assert torch.equal(got, lib.kv_attend_tree(c, q, table, dlens, k_new=kn, v_new=vn, mask=_dev(_pack_mask(see))))


def test_tree_over_the_context_alone(lib):
    """No drafts' keys: every row sees the context only, as kv_attend does for one token of a contiguous cache."""
    g, c, table, dlens, ctx, q, _, _ = _setup(lib, (5,), [120, 0, 33], 3, 8, 2)
    got = lib.kv_attend_tree(c, q, table, dlens)
    _check(got, _attend(_f64(q), ctx, None, None, None, None))
    assert bool((got[1] == 0).all())
    rot = lib.Rotation(D, D, seed=77)
    kv = lib.KVCache(2048, 8, D, 32, lib.Codebook(256), lib.Codebook(8), rot)
    lib.kv_quantize(kv, *(_dev(_heavy(g, 1999, 8), torch.bfloat16) for _ in range(2)))
    q1 = _dev(g.normal(size=(1, 1, 32, D)), torch.bfloat16)
    pages = lib.PagedKVCache.of(kv)
    table = torch.arange(pages.pages, dtype=torch.int32, device="cuda")[None]
    a = lib.kv_attend_tree(pages, q1, table, _dev([1999], torch.int32))
    assert helpers.rel_l2(_f64(a)[0, 0], _f64(lib.kv_attend(kv, q1[0, 0]))) < ATTEND


def test_tree_rows_that_see_nothing_and_rows_not_in_use(lib):
    lens, n = [0, 20, 0], 6
    g, c, table, dlens, ctx, q, kn, vn = _setup(lib, (6,), lens, n, 4, 2)
    see = _tree(g, 3, n)
    see[0, 3] = False  # no context and no draft
    see[1, 2] = False  # the context only
    n_tok = np.array([6, 4, 0], np.int32)
    got = lib.kv_attend_tree(c, q, table, dlens, k_new=kn, v_new=vn, mask=_dev(_pack_mask(see)), n_tok=_dev(n_tok))
    _check(got, _attend(_f64(q), ctx, _f64(kn), _f64(vn), see, n_tok))
    assert bool((got[0, 3] == 0).all()) and bool((got[1, 4:] == 0).all()) and bool((got[2] == 0).all())


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 3e38])
def test_tree_what_a_row_does_not_see_never_reaches_it(lib, bad):
    """Non-finite and enormous keys and values of drafts that rows do not see, and of drafts not in use."""
    n = 10
    g, c, table, dlens, ctx, q, kn, vn = _setup(lib, (7,), [45], n, 8, 2)
    see = _tree(g, 1, n)
    see[0, :, 4] = False
    see[0, 6, 4] = True  # one row sees the bad draft
    n_tok = np.array([9], np.int32)
    clean = lib.kv_attend_tree(c, q, table, dlens, k_new=kn, v_new=vn, mask=_dev(_pack_mask(see)), n_tok=_dev(n_tok))
    kn, vn = kn.clone(), vn.clone()
    kn[0, 4], vn[0, 4], vn[0, 9], kn[0, 9] = bad, bad, bad, bad
    got = lib.kv_attend_tree(c, q, table, dlens, k_new=kn, v_new=vn, mask=_dev(_pack_mask(see)), n_tok=_dev(n_tok))
    rows = [i for i in range(n) if i != 6]
    assert torch.equal(got[:, rows], clean[:, rows])
    if bad != bad:
        assert bool(torch.isnan(got[0, 6]).all())


def test_tree_one_bad_value_stays_in_its_place(lib):
    """An infinity in one value element of a draft reaches that element of the rows that see it, and no other."""
    n = 4
    g, c, table, dlens, ctx, q, kn, vn = _setup(lib, (8,), [30], n, 2, 1)
    see = np.tril(np.ones((1, n, n), bool))
    see[0, 3, 2] = False
    clean = lib.kv_attend_tree(c, q, table, dlens, k_new=kn, v_new=vn, mask=_dev(_pack_mask(see)))
    vn = vn.clone()
    vn[0, 2, 0, 77] = float("inf")
    got = lib.kv_attend_tree(c, q, table, dlens, k_new=kn, v_new=vn, mask=_dev(_pack_mask(see)))
    assert torch.equal(got[0, [0, 1, 3]], clean[0, [0, 1, 3]])
    assert bool(torch.isinf(got[0, 2, :, 77]).all())
    other = [d for d in range(D) if d != 77]
    assert torch.equal(got[0, 2][:, other], clean[0, 2][:, other])


def test_tree_a_bad_query_stays_in_its_row(lib):
    n = 5
    g, c, table, dlens, ctx, q, kn, vn = _setup(lib, (9,), [100], n, 8, 2)
    clean = lib.kv_attend_tree(c, q, table, dlens, k_new=kn, v_new=vn)
    q = q.clone()
    q[0, 2, 3, 5] = float("nan")
    got = lib.kv_attend_tree(c, q, table, dlens, k_new=kn, v_new=vn)
    assert bool(torch.isnan(got[0, 2, 3]).all())
    got[0, 2, 3] = clean[0, 2, 3]
    assert torch.equal(got, clean)


@pytest.mark.parametrize("factor", [1e-3, 50.0])
def test_tree_flat_and_sharp_scores(lib, factor):
    """Weights all but equal, and weights on one token: the maximum and sum are carried across splits."""
    g, c, table, dlens, ctx, q, kn, vn = _setup(lib, (10,), [3000], 3, 4, 1, 64)
    see = _tree(g, 1, 3)
    got = lib.kv_attend_tree(c, q, table, dlens, k_new=kn, v_new=vn, mask=_dev(_pack_mask(see)), scale=factor * D ** -0.5)
    ref = _attend(_f64(q), ctx, _f64(kn), _f64(vn), see, None, factor * D ** -0.5)
    if factor < 1:
        _check(got, ref)
    else:
        # a score of deviation 150 is off by about 2^-11 sqrt(2/3) 150 = 0.06: weights of near ties move by that much
        assert helpers.rel_l2(_f64(got), ref) < 0.1


@pytest.mark.parametrize("scale", [0.0, -0.05])
@pytest.mark.parametrize("n,Hq,H", [(1, 4, 1), (2, 4, 1), (3, 4, 1), (33, 4, 1), (70, 4, 1)])
def test_tree_scales_of_zero_and_below(lib, scale, n, Hq, H):
    """All weights equal, and the order of the scores turned round; also past the end of a step and where nothing is cached."""
    lens = [75, 0, 16]
    g, c, table, dlens, ctx, q, kn, vn = _setup(lib, (22, n), lens, n, Hq, H, 32)
    see = _tree(g, 3, n)
    got = lib.kv_attend_tree(c, q, table, dlens, k_new=kn, v_new=vn, mask=_dev(_pack_mask(see)), scale=scale)
    _check(got, _attend(_f64(q), ctx, _f64(kn), _f64(vn), see, None, scale))


@pytest.mark.parametrize("n,Hq,H", [(1, 4, 1), (3, 4, 1), (33, 4, 1), (70, 4, 1)])
def test_tree_scores_that_vanish(lib, n, Hq, H):
    """The smallest queries times a small scale: all weights equal, and what lies past a context's end stays out."""
    g, c, table, dlens, ctx, q, kn, vn = _setup(lib, (24, n), [75], n, Hq, H, 32)
    see = _tree(g, 1, n)
    q = (q.float() * 2.0 ** -125).bfloat16()
    got = lib.kv_attend_tree(c, q, table, dlens, k_new=kn, v_new=vn, mask=_dev(_pack_mask(see)), scale=1e-9)
    _check(got, _attend(_f64(q), ctx, _f64(kn), _f64(vn), see, None, 1e-9))


@pytest.mark.parametrize("n,Hq,H", [(1, 8, 1), (2, 4, 1), (1, 16, 1), (5, 4, 1), (20, 8, 1)])
def test_tree_a_bad_query_stays_in_its_row_of_each_form(lib, n, Hq, H):
    g, c, table, dlens, ctx, q, kn, vn = _setup(lib, (23, n, Hq), [333, 40], n, Hq, H, 32)
    clean = lib.kv_attend_tree(c, q, table, dlens, k_new=kn, v_new=vn)
    for bad in (float("nan"), float("inf")):
        b = q.clone()
        b[0, n - 1, 3, 5] = bad
        got = lib.kv_attend_tree(c, b, table, dlens, k_new=kn, v_new=vn)
        assert bool(torch.isnan(got[0, n - 1, 3]).all())
        got[0, n - 1, 3] = clean[0, n - 1, 3]
        assert torch.equal(got, clean)


@pytest.mark.parametrize("size", [3e-4, 3e3])
def test_tree_small_and_large_caches(lib, size):
    """Group scales far from one: fp16 scales of 3e-4 (still 11 bits of precision) and of 3e3."""
    g, c, table, dlens, ctx, q, kn, vn = _setup(lib, (12,), [500], 2, 4, 1, 64, spread=size)
    got = lib.kv_attend_tree(c, q / size, table, dlens, scale=D ** -0.5)
    ref = _attend(_f64(q / size), ctx, None, None, None, None)
    # decoded values are multiples of 2^-24 below 2^-14: 3e-4 * 2^-1 in steps of 2^-24 is 2e-4 of a value
    _check(got, ref)


def test_tree_flags_bad_pages_and_lengths(lib):
    g, c, table, dlens, ctx, q, kn, vn = _setup(lib, (13,), [40, 25], 3, 4, 2)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    good = lib.kv_attend_tree(c, q, table, dlens, k_new=kn, v_new=vn, err=err)
    assert lib.check_error(err) == 0
    for value in (-1, c.pages, 2 ** 31 - 1):
        t = table.clone()
        t[0, 1] = value
        got = lib.kv_attend_tree(c, q, t, dlens, k_new=kn, v_new=vn, err=err)
        assert lib.check_error(err) == lib.TQ_DEVERR_BAD_PAGE
        assert torch.equal(got[1], good[1])
        left = [(np.delete(ctx[0][0], np.s_[16:32], 0), np.delete(ctx[0][1], np.s_[16:32], 0)), ctx[1]]
        see = np.tril(np.ones((2, 3, 3), bool))
        _check(got, _attend(_f64(q), left, _f64(kn), _f64(vn), see, None))
    for value in (-5, 41):
        d = dlens.clone()
        d[0] = value
        got = lib.kv_attend_tree(c, q, table, d, k_new=kn, v_new=vn, max_len=40, err=err)
        assert lib.check_error(err) == lib.TQ_DEVERR_BAD_PAGE
        assert torch.equal(got[1], good[1])
        if value > 0:  # clamped to 40
            assert torch.equal(got[0], lib.kv_attend_tree(c, q, table, dlens, k_new=kn, v_new=vn, max_len=40)[0])


def test_tree_repeats_bit_for_bit_and_on_another_stream(lib):
    lens, n = [4000, 77], 8
    g, c, table, dlens, ctx, q, kn, vn = _setup(lib, (14,), lens, n, 8, 2, 64)
    a = lib.kv_attend_tree(c, q, table, dlens, k_new=kn, v_new=vn)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        b = lib.kv_attend_tree(c, q, table, dlens, k_new=kn, v_new=vn)
    side.synchronize()
    assert torch.equal(a, b)
    assert torch.equal(a, lib.kv_attend_tree(c, q.contiguous(), table, dlens, k_new=kn.contiguous(), v_new=vn.contiguous()))


def test_tree_in_a_graph_follows_the_lengths(lib):
    """Captured once, replayed as the context grows: nothing of a call depends on the lengths on the host."""
    lens, n = [500], 4
    g, c, table, dlens, ctx, q, kn, vn = _setup(lib, (15,), lens, n, 8, 2, 64)
    q, kn, vn = q.contiguous(), kn.contiguous(), vn.contiguous()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        lib.kv_attend_tree(c, q, table, dlens, k_new=kn, v_new=vn)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = lib.kv_attend_tree(c, q, table, dlens, k_new=kn, v_new=vn)
    for length in (500, 1, 130, 0, 257):
        dlens.fill_(length)
        graph.replay()
        torch.cuda.synchronize()
        see = np.tril(np.ones((1, n, n), bool))
        _check(out, _attend(_f64(q), [(ctx[0][0][:length], ctx[0][1][:length])], _f64(kn), _f64(vn), see, None))


def test_cache_and_tree_refusals(lib):
    c = _cache(lib, 4, 16, 2, 32, 256, 8)
    k = torch.zeros((3, 2, D), device="cuda", dtype=torch.bfloat16)
    s = torch.zeros(3, dtype=torch.int32, device="cuda")
    q = torch.zeros((1, 3, 4, D), device="cuda", dtype=torch.bfloat16)
    table, lens = torch.zeros((1, 4), dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    r = lib.Rope(D)
    for bad in (lambda: lib.kv_append(c, k, k.float(), s), lambda: lib.kv_append(c, k[:, :1], k[:, :1], s),
                lambda: lib.kv_append(c, k, k, s.long()), lambda: lib.kv_append(c, k, k, s[:2]),
                lambda: lib.kv_append(c, k, k, s, rope=r), lambda: lib.kv_fetch(c, s.long()),
                lambda: lib.kv_attend_tree(c, q, table, lens, k_new=k[None]), lambda: lib.kv_attend_tree(c, q[0], table, lens),
                lambda: lib.kv_attend_tree(c, q, table, lens.long()), lambda: lib.kv_attend_tree(c, q, table[0], lens),
                lambda: lib.kv_attend_tree(c, q, table, lens, mask=torch.zeros((1, 3), device="cuda", dtype=torch.int32)),
                lambda: lib.kv_attend_tree(c, q, table, lens, k_new=k[None, :2], v_new=k[None, :2]),
                lambda: lib.PagedKVCache.of(lib.KVCache(100, 2, D, 32, c.kcb, c.vcb, c.rot))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: lib.kv_append(c, k.half(), k.half(), s), lambda: lib.kv_append(c, k, k, s, rope=lib.Rope(D, 48), positions=s),
                lambda: lib.kv_append(c, k, k, s, rope=lib.Rope(64), positions=s),
                lambda: lib.kv_attend_tree(c, q.half(), table, lens), lambda: lib.kv_attend_tree(c, q, table, lens, max_len=65),
                lambda: lib.kv_attend_tree(c, q[:, :, :3], table, lens),
                lambda: lib.kv_fetch(_cache(lib, 4, 24, 2, 32, 256, 8), s), lambda: lib.kv_fetch(_cache(lib, 4, 16, 2, 32, 8, 8), s),
                lambda: lib.kv_fetch(_cache(lib, 4, 16, 2, 32, 256, 4), s)):
        with pytest.raises(lib.TQError):
            bad()


def test_serving_step_end_to_end(lib):
    """Three verification steps of two sequences: positions, a tree over the cache, the accepted path appended."""
    g = _rng(16)
    B, n, Hq, H, page = 2, 7, 8, 2, 16
    c = _cache(lib, 40, page, H, 32, 256, 8)
    table = _dev(g.permutation(40)[:32].reshape(B, 16).astype(np.int32))
    lens = _dev([30, 0], torch.int32)
    r = lib.Rope(D)
    start = _dev(_heavy(g, 30, 2 * H), torch.bfloat16)
    i = torch.arange(30, device="cuda")
    lib.kv_append(c, start[:, :H], start[:, H:], (table[0, i // page] * page + i % page).int(), rope=r, positions=i.int())
    for step in range(3):
        see = _tree(g, B, n)
        depth = _dev(see.sum(-1) - 1, torch.int32)
        qkv = _dev(_heavy(g, B * n, Hq + 2 * H), torch.bfloat16).view(B, n, Hq + 2 * H, D)
        pos = lens[:, None] + depth
        q, k = lib.rope(qkv[:, :, :Hq], pos.contiguous(), r, k=qkv[:, :, Hq:Hq + H])
        v = qkv[:, :, Hq + H:]
        got = lib.kv_attend_tree(c, q, table, lens, k_new=k, v_new=v, mask=_dev(_pack_mask(see)))
        ctx = []
        for b in range(B):
            x = np.arange(int(lens[b]))
            ctx.append(_values(c, table[b].cpu().numpy()[x // page] * page + x % page))
        _check(got, _attend(_f64(q), ctx, _f64(k), _f64(v), see, None))
        leaf = see.sum(-1).argmax(-1)
        taken = _dev(np.stack([see[b, leaf[b]] for b in range(B)]))  # the longest path is accepted
        p = pos.long()
        slot = torch.where(taken, table.gather(1, p // page) * page + p % page, -1).int()
        lib.kv_append(c, k, v, slot)
        lens += taken.sum(-1).int()
    assert bool((lens > 3).all())


@pytest.mark.parametrize("n,Hq,H", [(1, 4, 8), (16, 32, 8), (30, 8, 2), (64, 32, 8), (70, 4, 1)])
def test_tree_long_runs_repeat_and_report_nothing(lib, n, Hq, H):
    """Runs of many steps through every kernel form, ten times on fresh queries: no wait runs out, and a repeat is the same."""
    Hq = max(Hq, H)
    g = _rng(17, n)
    context, page = 20011, 64
    pages = -(-context // page)
    c = lib.PagedKVCache(pages, page, H, D, 32, lib.Codebook(256), lib.Codebook(8), lib.Rotation(D, D, seed=77))
    slots = torch.arange(context, dtype=torch.int32, device="cuda")
    lib.kv_append(c, *(torch.randn((context, H, D), device="cuda", dtype=torch.bfloat16) for _ in range(2)), slots)
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    k, v = lib.kv_fetch(c, slots, out_dtype=torch.float32)
    for _ in range(10):
        q, kn, vn = (_dev(g.normal(size=(1, n, h, D)), torch.bfloat16) for h in (Hq, H, H))
        out = [lib.kv_attend_tree(c, q, table, _dev([context], torch.int32), k_new=kn, v_new=vn, err=err) for _ in range(2)]
        assert lib.check_error(err) == 0
        assert torch.equal(*out)
        # rounding of the fp32 sums is far below the tolerance
        kk, vv = (torch.cat([a, b[0].float()]).repeat_interleave(Hq // H, 1).transpose(0, 1) for a, b in ((k, kn), (v, vn)))
        s = q[0].float().transpose(0, 1) @ kk.transpose(1, 2) * D ** -0.5
        s[:, :, context:].masked_fill_(~torch.tril(torch.ones((n, n), dtype=torch.bool, device="cuda")), float("-inf"))
        assert helpers.rel_l2(_f64(out[0][0]), _f64((torch.softmax(s, -1) @ vv).transpose(0, 1))) < ATTEND


@pytest.mark.parametrize("n", [8, 64])
def test_tree_wait_budget(lib, n):
    """With no budget the bounded waits give up, the call reports it, and the next call is as before."""
    g, c, table, dlens, ctx, q, kn, vn = _setup(lib, (18, n), [3000], n, 16, 4, 64)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    before = lib.kv_attend_tree(c, q, table, dlens, k_new=kn, v_new=vn, err=err)
    assert lib.check_error(err) == 0
    lib.set_wait_budget(0)
    try:
        lib.kv_attend_tree(c, q, table, dlens, k_new=kn, v_new=vn, err=err)
        assert lib.check_error(err) == lib.TQ_DEVERR_TIMEOUT
    finally:
        lib.set_wait_budget(-1)
    assert torch.equal(before, lib.kv_attend_tree(c, q, table, dlens, k_new=kn, v_new=vn, err=err))
    assert lib.check_error(err) == 0


def test_example_of_drafted_decoding(lib):
    import importlib.util
    import os

    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "drafted_decode.py")
    spec = importlib.util.spec_from_file_location("drafted_decode", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    worst, bits = example.main()
    assert bits == 0 and worst < ATTEND


# ---------------------------------------------------------------- handles whose tensors are replaced

def test_rope_handle_follows_its_tensors(lib):
    """Frequencies and factor assigned later, or moved under the same tensor, are those of the next call."""
    g = _rng(30)
    x = _dev(g.normal(size=(9, 3, D)), torch.float32)
    pos = _dev(g.integers(0, 5000, 9), torch.int32)
    r, other = lib.Rope(D), lib.Rope(D, base=500000.0, scaling={"kind": "linear", "factor": 4.0})
    r.steps = other.steps
    assert torch.equal(lib.rope(x, pos, r), lib.rope(x, pos, other))
    r.factor = other.factor = 1.5
    assert torch.equal(lib.rope(x, pos, r), lib.rope(x, pos, lib.Rope(D, steps=other.steps, factor=1.5)))
    own = lib.Rope(D)
    r = lib.Rope(D, steps=torch.zeros_like(own.steps))
    r.steps.set_(own.steps.clone())  # the same tensor object, other memory
    assert torch.equal(lib.rope(x, pos, r), lib.rope(x, pos, own))
    r.rotary, r.layout, r.steps = 64, "interleaved", lib.Rope(64).steps
    assert torch.equal(lib.rope(x, pos, r), lib.rope(x, pos, lib.Rope(D, 64, layout="interleaved")))
    r.steps = own.steps  # 64 frequencies for 32 pairs
    with pytest.raises(ValueError):
        lib.rope(x, pos, r)


def _step(lib, c, g):
    """A write, a read and an attention over what was written."""
    k, v = (_dev(g.normal(size=(40, c.heads, D)), torch.bfloat16) for _ in range(2))
    slots = torch.arange(40, dtype=torch.int32, device="cuda")
    lib.kv_append(c, k, v, slots)
    q = _dev(g.normal(size=(1, 2, 2 * c.heads, D)), torch.bfloat16)
    table = torch.arange(c.pages, dtype=torch.int32, device="cuda")[None]
    return (*lib.kv_fetch(c, slots, out_dtype=torch.float32), lib.kv_attend_tree(c, q, table, _dev([40], torch.int32)))


@pytest.mark.parametrize("change", ["arrays", "moved arrays", "books", "tensors of the books", "signs", "pages", "order"])
def test_cache_handle_follows_its_tensors(lib, change):
    c = _cache(lib, 4, 16, 2, 32, 256, 8, poison=False)
    _step(lib, c, _rng(31))
    old = [t.clone() for t in (c.kcodes, c.kscales, c.vcodes, c.vscales)]
    fresh = lambda **kw: lib.PagedKVCache(kw.get("pages", c.pages), 16, 2, D, 32, kw.get("kcb", c.kcb), kw.get("vcb", c.vcb),  # noqa: E731
                                          kw.get("rot", c.rot))
    wide = lambda n: lib.Codebook(n, centroids=lib.codebook(n)[0] * 1.25, thresholds=lib.codebook(n)[1] * 1.25)  # noqa: E731
    want = fresh()
    kept = [c.kcodes, c.kscales, c.vcodes, c.vscales]
    if change == "arrays":
        c.kcodes, c.kscales, c.vcodes, c.vscales = (torch.zeros_like(t) for t in kept)
    elif change == "moved arrays":
        for t in kept:
            t.set_(torch.zeros_like(t))
    elif change == "books":
        c.kcb, c.vcb = wide(256), wide(8)
        want = fresh(kcb=c.kcb, vcb=c.vcb)
    elif change == "tensors of the books":
        a, b = wide(256), wide(8)
        c.kcb.centroids, c.kcb.thresholds, c.vcb.centroids, c.vcb.thresholds = a.centroids, a.thresholds, b.centroids, b.thresholds
        want = fresh(kcb=wide(256), vcb=wide(8))
    elif change == "signs":
        other = lib.Rotation(D, D, seed=78)
        c.rot.signs = other.signs
        want = fresh(rot=other)
    elif change == "pages":
        c.kcodes, c.kscales, c.vcodes, c.vscales = (torch.zeros((7, *t.shape[1:]), dtype=t.dtype, device="cuda") for t in kept)
        c.pages = 7
        want = fresh(pages=7)
    else:  # heads first: one sequence's contiguous rows
        c.kcodes, c.kscales, c.vcodes, c.vscales = (torch.zeros((2, 64, t.shape[-1]), dtype=t.dtype, device="cuda") for t in kept)
        c.page_stride, c.head_stride = 16, 64
    for x, y in zip(_step(lib, c, _rng(32)), _step(lib, want, _rng(32))):
        assert torch.equal(x, y)
    if change == "arrays":  # and what was replaced is left alone
        for x, y in zip(kept, old):
            assert torch.equal(x, y)
    assert c.tree_bytes(1, 40, 4, 64) == want.tree_bytes(1, 40, 4, 64)


def test_cache_handle_refuses_tensors_that_do_not_fit(lib):
    slots = torch.zeros(1, dtype=torch.int32, device="cuda")
    for name, value in (("kcodes", lambda t: t[:2].clone()), ("vscales", lambda t: t.float()), ("kscales", lambda t: t.cpu()),
                        ("vcodes", lambda t: t.transpose(0, 1)), ("pages", lambda n: n + 1), ("head_stride", lambda n: 4 * n),
                        ("kcb", lambda b: lib.Codebook(16)), ("vcb", lambda b: lib.Codebook(8, device="cpu")),
                        ("rot", lambda r: lib.Rotation(D, D, seed=1, device="cpu"))):
        c = _cache(lib, 4, 16, 2, 32, 256, 8)
        lib.kv_fetch(c, slots)
        setattr(c, name, value(getattr(c, name)))
        with pytest.raises(ValueError):
            lib.kv_fetch(c, slots)
    c = _cache(lib, 4, 16, 2, 32, 256, 8)
    for short in (c.kcb.centroids[:200], c.kcb.centroids.double()):
        c.kcb.centroids = short
        with pytest.raises(ValueError):
            lib.kv_fetch(c, slots)
    with pytest.raises(ValueError):  # everything on the host
        lib.kv_fetch(lib.PagedKVCache(4, 16, 2, D, 32, lib.Codebook(256, device="cpu"), lib.Codebook(8, device="cpu"),
                                      lib.Rotation(D, D, seed=1, device="cpu"), device="cpu"), slots.cpu())


def test_cache_handle_is_made_by_two_threads_at_once(lib):
    import sys
    import threading

    kcb, vcb, rot = lib.Codebook(256), lib.Codebook(8), lib.Rotation(D, D, seed=77)
    wrong, interval = [], sys.getswitchinterval()
    sys.setswitchinterval(1e-6)
    try:
        for _ in range(100):
            c = lib.PagedKVCache(4, 16, 2, D, 32, kcb, vcb, rot)

            def use():
                try:
                    if c.tree_bytes(1, 2, 4, 64) <= 0 or c._now()[1].kcodes != c.kcodes.data_ptr():
                        wrong.append("another descriptor")
                except Exception as e:  # noqa: BLE001
                    wrong.append(e)

            threads = [threading.Thread(target=use) for _ in range(4)]
            for t in threads:
                t.start()
            for t in threads:
                t.join()
    finally:
        sys.setswitchinterval(interval)
    assert not wrong


def test_scratch_error_word_and_device_are_checked(lib, monkeypatch):
    """Nothing but memory of the calls' own device goes to a kernel."""
    c = _cache(lib, 4, 16, 2, 32, 256, 8)
    k = torch.zeros((3, 2, D), device="cuda", dtype=torch.bfloat16)
    s, pos = (torch.zeros(3, dtype=torch.int32, device="cuda") for _ in range(2))
    q = torch.zeros((1, 3, 4, D), device="cuda", dtype=torch.bfloat16)
    table, lens = torch.zeros((1, 4), dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    nb = c.tree_bytes(1, 3, 4, 64)
    ws = torch.empty(2 * nb, dtype=torch.uint8, device="cuda")
    calls = [lambda **kw: lib.kv_append(c, k, k, s, **kw), lambda **kw: lib.kv_fetch(c, s, **kw),
             lambda **kw: lib.kv_attend_tree(c, q, table, lens, **kw)]
    for call in calls:
        call(err=torch.zeros(1, dtype=torch.int32, device="cuda"))
        for bad in (torch.zeros(1, dtype=torch.int32), torch.zeros(1, device="cuda"), torch.zeros(1, dtype=torch.int16, device="cuda"),
                    torch.zeros(1, dtype=torch.int64, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda")):
            with pytest.raises(ValueError):
                call(err=bad)
    calls[2](ws=ws)
    for bad in (ws.cpu(), ws[::2]):
        with pytest.raises(ValueError):
            calls[2](ws=bad)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: torch.cuda.device_count())  # as if another device were current
    for call in (*calls, lambda: lib.rope(k, pos, lib.Rope(D))):
        with pytest.raises(ValueError):
            call()


FORMS = [(1, 4), (4, 4), (20, 4), (33, 4)]  # drafts and heads: 4, 16, 80 and 132 rows to a kv head


@pytest.mark.parametrize("n,Hq", FORMS)
def test_tree_large_queries_and_small_scales(lib, n, Hq):
    """Queries of 2^118 under a scale of 2^-118: every score is an ordinary number."""
    g, c, table, dlens, ctx, q, kn, vn = _setup(lib, (40, n), [333, 20], n, Hq, 1, 32)
    see = _tree(g, 2, n)
    q = (q.float() * 2.0 ** 118).bfloat16()
    scale = D ** -0.5 * 2.0 ** -118
    for sign in (1, -1):
        got = lib.kv_attend_tree(c, q, table, dlens, k_new=kn, v_new=vn, mask=_dev(_pack_mask(see)), scale=sign * scale)
        _check(got, _attend(_f64(q), ctx, _f64(kn), _f64(vn), see, None, sign * scale))


@pytest.mark.parametrize("power", [3, 18, 22, 24, 30, 100])
@pytest.mark.parametrize("n,Hq", FORMS)
def test_tree_scores_of_any_size(lib, n, Hq, power):
    """Each row's query points at one token's key: that token's value, up to scores of 2^107."""
    g, c, table, dlens, ctx, q, kn, vn = _setup(lib, (41, n), [500], n, Hq, 1, 32)
    k, v = ctx[0]
    picks = g.integers(0, 500, (n, Hq))
    q = _dev(k[picks, 0], torch.bfloat16)[None]
    got = lib.kv_attend_tree(c, q, table, dlens, scale=2.0 ** power * D ** -0.5)
    ref = _attend(_f64(q), ctx, None, None, None, None, 2.0 ** power * D ** -0.5)
    if power > 3:
        np.testing.assert_array_equal(ref[0], v[picks, 0])
    _check(got, ref)


@pytest.mark.parametrize("size", [1e-5, 1e-6, 1e-7])
@pytest.mark.parametrize("n,Hq", FORMS)
def test_tree_group_scales_of_fp16_subnormals(lib, n, Hq, size):
    """Where group scales are fp16 subnormals a decoded element is off by 2^-25 of the power of two above the book at most
    (4 for 8 value levels), so a row by that times sqrt(128), beside the usual roundings."""
    g, c, table, dlens, ctx, q, kn, vn = _setup(lib, (42, n), [77], n, Hq, 1, 32, spread=size)
    assert float(c.vcb.centroids.abs().max()) < 4
    got = lib.kv_attend_tree(c, q, table, dlens)
    ref = _attend(_f64(q), ctx, None, None, None, None)
    off, norm = (np.linalg.norm(x, axis=-1) for x in (_f64(got) - ref, ref))
    assert np.all(off <= ATTEND_ROW * norm + math.sqrt(D) * 4 * 2.0 ** -25), (off / norm).max()
