"""The latent cache's write and latent attention, absorbed and expanded, against plain 64-bit code.

Tolerances.  Write: rotary angles as of the rotary-position tests (4e-7 of a pair's length) and half a step of the cache's type.
Attention, for each element of a result o = sum p v, with A = sum p |v|:
  u A        each softmax weight is rounded to the type (u = eps / 2: bf16 2^-8, fp16 2^-11);
  u |o|      so is the result;
  2 d A      a score is off by at most d: exact products of 16-bit operands, summed in fp32 over at most 40 steps of 16 elements,
             each step off by 2^-23 of the sum of the products' magnitudes at most, so d = scale 40 2^-23 sum |q k|;
             a relative error e^d - 1 of a weight, above and below the line;
  n 2^-31 max |v|  weights below 2^-31 of the largest vanish or lose bits (fp16's subnormals);
  2^-19 A    fp32 sums of weights and values (a thousand steps of 2^-24 and as many rescalings, each 2^-24), the exponential's 2^-22."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

C, R, W = 512, 64, 576
SCALE = 192 ** -0.5


def _rng(*key):
    return np.random.Generator(np.random.PCG64(list(key)))


def _int(a):
    return torch.tensor(np.ascontiguousarray(a), dtype=torch.int32, device="cuda")


def _gen(*key):
    return torch.Generator(device="cuda").manual_seed(int(_rng(*key).integers(1 << 62)))


def _half_step(dtype):
    return torch.finfo(dtype).eps / 2


# ---------------------------------------------------------------- write

def _turn(x, pos, w, rotary, layout, factor):
    a = pos.double()[:, None] * torch.tensor(w, device="cuda")
    c, s = a.cos() * factor, a.sin() * factor
    y = x.clone()
    if layout == "half":
        p, q = x[:, :rotary // 2], x[:, rotary // 2:rotary]
        y[:, :rotary // 2], y[:, rotary // 2:rotary] = p * c - q * s, p * s + q * c
    else:
        p, q = x[:, 0:rotary:2], x[:, 1:rotary:2]
        y[:, 0:rotary:2], y[:, 1:rotary:2] = p * c - q * s, p * s + q * c
    return y


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("kept", ["bfloat16", "float16"])
@pytest.mark.parametrize("T,page,layout,rotary", [(1, 16, None, 0), (3, 256, "half", 64), (77, 32, "interleaved", 64),
                                                  (500, 64, "interleaved", 24), (4099, 128, "half", 40)])
def test_append_matches_the_definition(lib, dtype, kept, T, page, layout, rotary):
    g, gen = _rng(1, T, page), _gen(2, T, page)
    dt, out = getattr(torch, dtype), getattr(torch, kept)
    pages = -(-T // page) + 2
    cache = lib.LatentCache(pages, page, dtype=out)
    cache.rows.copy_(torch.randn(cache.rows.shape, generator=gen, device="cuda"))
    before = cache.rows.clone()
    x = (torch.randn((T, 1536 + W), generator=gen, device="cuda") * 2).to(dt)  # a fused projection
    slots = g.permutation(pages * page)[:T]
    slots[g.random(T) < 0.2] = -1
    if T > 2:
        slots[1] = pages * page + 5  # past the pool
    pos = g.integers(-5, 1 << 20, T)
    rope = lib.Rope(R, rotary, base=50000.0, layout=layout) if layout else None
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    lib.latent_append(cache, x[:, 1536:1536 + C], x[:, 1536 + C:], _int(slots), rope=rope, positions=_int(pos), err=err)
    want = before.double().flatten(0, 1)
    bound = torch.zeros_like(want)
    k = x[:, 1536 + C:].double()
    slack = torch.zeros_like(k)
    if layout:
        w = 50000.0 ** (-np.arange(0, rotary, 2) / rotary)
        slack[:, :rotary] = 4e-7 * 1.42 * k.abs().amax(1, keepdim=True)
        k = _turn(k, _int(pos), w, rotary, layout, 1.0)
    live = (slots >= 0) & (slots < pages * page)
    at = torch.tensor(slots[live], device="cuda").long()
    live = torch.tensor(live, device="cuda")
    want[at] = torch.cat([x[:, 1536:1536 + C].double(), k], 1)[live]
    bound[at] = torch.cat([torch.zeros((T, C), device="cuda", dtype=torch.float64), slack], 1)[live]
    bound[at] += _half_step(out) * want[at].abs() * 1.001 + (2.0 ** -25 if kept == "float16" else 0.0)
    assert bool(((cache.rows.double().flatten(0, 1) - want).abs() <= bound).all())
    assert lib.check_error(err) == (8 if T > 2 else 0)


@pytest.mark.parametrize("factor", [1.25, 0.5])
@pytest.mark.parametrize("layout,rotary", [("half", 64), ("interleaved", 64), ("interleaved", 24), ("half", 40)])
def test_append_with_a_rotary_factor(lib, layout, rotary, factor):
    """The factor of scaled frequencies: on the rotated part alone."""
    T, page, gen = 300, 32, _gen(23, rotary)
    x = torch.randn((T, W), generator=gen, device="cuda")
    pos = torch.randint(0, 1 << 18, (T,), generator=gen, device="cuda", dtype=torch.int32)
    rope = lib.Rope(R, rotary, base=50000.0, layout=layout)
    rope.factor = factor
    cache = lib.LatentCache(10, page, dtype=torch.float16)
    lib.latent_append(cache, x[:, :C], x[:, C:], _int(np.arange(T)), rope=rope, positions=pos)
    got = cache.rows.view(-1, W)[:T].double()
    k = x[:, C:].double()
    slack = torch.zeros_like(k)
    slack[:, :rotary] = 4e-7 * 1.42 * factor * k.abs().amax(1, keepdim=True)
    want = torch.cat([x[:, :C].double(), _turn(k, pos, 50000.0 ** (-np.arange(0, rotary, 2) / rotary), rotary, layout, factor)], 1)
    bound = _half_step(torch.float16) * want.abs() * 1.001 + 2.0 ** -25
    bound[:, C:] += slack
    assert bool(((got - want).abs() <= bound).all())


@pytest.mark.parametrize("page,stride", [(16, 17), (64, 100), (32, 32 * 3)])
def test_pages_further_apart_than_they_are_long(lib, page, stride):
    """Pages inside larger blocks, as the C call takes them: written and attended like pages that follow one another, what lies between
    them neither read nor written."""
    import ctypes

    g, gen, pages, lens, H, n = _rng(24, page), _gen(25, page), 40, [150, 3], 16, 2
    dt = torch.bfloat16
    close = lib.LatentCache(pages, page, dtype=dt)
    wide = torch.full((pages, stride, W), float("nan"), dtype=dt, device="cuda")
    wide[:, :page] = 0
    apart = lib.tq_latent_pages_t(wide.data_ptr(), lib.TQ_BF16, C, R, page, pages, stride)
    table = g.permutation(pages)[:20].reshape(2, 10)
    slots = np.concatenate([[table[b, t // page] * page + t % page for t in range(lens[b])] for b in range(2)])
    x = torch.randn((len(slots), W), generator=gen, device="cuda").to(dt)
    lib.latent_append(close, x[:, :C], x[:, C:], _int(slots))
    stream, at = torch.cuda.current_stream().cuda_stream, _int(slots)
    assert lib.load().tq_latent_append(ctypes.byref(apart), x.data_ptr(), W, x.data_ptr() + 2 * C, W, lib.TQ_BF16, len(slots),
                                       at.data_ptr(), None, 0, 0, stream) == 0
    assert torch.equal(wide[:, :page], close.rows) and bool(wide[:, page:].isnan().all())
    q, fresh = (torch.randn(s, generator=gen, device="cuda").to(dt) for s in ((2, n, H, W), (2, n, W)))
    want = lib.latent_attend_tree(close, q, _int(table), _int(lens), SCALE, new=fresh)
    nb = lib.load().tq_latent_attend_tree_workspace_bytes(ctypes.byref(apart), 2, n, H, 10 * page)
    ws, o, tab, ln = torch.empty(nb, dtype=torch.uint8, device="cuda"), torch.empty_like(want), _int(table), _int(lens)
    assert lib.load().tq_latent_attend_tree(ctypes.byref(apart), q.data_ptr(), H * W, 2, n, H, tab.data_ptr(), 10, ln.data_ptr(),
                                            10 * page, fresh.data_ptr(), W, 0, 0, SCALE, o.data_ptr(), ws.data_ptr(), nb, 0, stream) == 0
    assert torch.equal(o, want)


# ---------------------------------------------------------------- absorbed

def _bound(o, A, d, n, top, dtype):
    u = _half_step(dtype)
    return u * A * 1.01 + u * o.abs() * 1.02 + 2 * d * A + n * 2.0 ** -31 * top + 2.0 ** -19 * A + (2.0 ** -24 if dtype == torch.float16 else 1e-30)


def _attend(q, rows, values, see, scale):
    """o, sum p |v| and the score's error of queries [r, d] over rows [t, d], values [t, e] through see [r, t], in 64 bits."""
    q, rows, values = q.double(), rows.double(), values.double()
    s = (q @ rows.T * scale).masked_fill(~see, float("-inf"))
    p = torch.softmax(s, 1).masked_fill(~see, 0.0)
    d = (q.abs() @ rows.abs().T * abs(scale)).masked_fill(~see, 0.0).amax(1, keepdim=True) * 40 * 2.0 ** -23
    return p @ values, p @ values.abs(), d


class Scene:
    def __init__(self, lib, B, n, H, context, page, dtype, ragged=True, tree="random", fresh=True, spread=1.0):
        g, gen = _rng(3, B, n, H, context, page), _gen(4, B, n, H, context, page)
        self.dt = getattr(torch, dtype)
        self.B, self.n, self.H, self.most = B, n, H, context
        lens = g.integers(0, context + 1, B) if ragged else np.full(B, context)
        if ragged:
            lens[0] = context
            lens[-1] = 0 if B > 1 else context
        need = -(-lens // page)
        order, at = g.permutation(int(need.sum()) + 2), 0
        self.table = np.full((B, max(1, -(-context // page))), -1)
        for b in range(B):
            self.table[b, :need[b]] = order[at:at + need[b]]
            at += need[b]
        self.cache = lib.LatentCache(len(order), page, dtype=self.dt)
        rand = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
        self.cache.rows.copy_(rand(*self.cache.rows.shape))
        self.cache.rows[torch.tensor(order[at:], device="cuda").long()] = float("nan")
        for b in range(B):
            if lens[b] % page:
                self.cache.rows[int(self.table[b, need[b] - 1]), int(lens[b] % page):] = float("inf")
        self.lens, self.q = lens, (rand(B, n, H, W) * spread).to(self.dt)
        self.fresh = rand(B, n, W).to(self.dt) if fresh else None
        self.see, self.count = np.zeros((B, n, -(-n // 64) * 64), dtype=bool), np.full(B, n)
        for b in range(B):
            if ragged:
                self.count[b] = g.integers(1, n + 1)
            for i in range(n):
                parent = i - 1 if tree == "chain" else int(g.integers(max(-1, i - 6), i)) if i else -1
                if parent >= 0:
                    self.see[b, i] = self.see[b, parent]
                self.see[b, i, i] = True
        if ragged:
            self.see[-1, self.count[-1] - 1] = False  # a row that sees nothing where there is no context
            self.count[B // 2] = 0 if B > 2 else self.count[B // 2]
        self.mask = torch.tensor(np.packbits(self.see, axis=-1, bitorder="little").view(np.int64), device="cuda")
        self.lib = lib

    def run(self, **kw):
        args = dict(new=self.fresh, mask=self.mask, n_tok=_int(self.count), max_len=self.most)
        args.update(kw)
        return self.lib.latent_attend_tree(self.cache, self.q, _int(self.table), _int(self.lens), args.pop("scale", SCALE), **args)

    def check(self, o, scale=SCALE, count=None):
        count = self.count if count is None else count
        assert o.shape == (self.B, self.n, self.H, C) and o.dtype == self.dt
        page = self.cache.page
        for b in range(self.B):
            pages = torch.tensor(self.table[b, :-(-self.lens[b] // page)], device="cuda").long()
            old = self.cache.rows[pages].reshape(-1, W)[:self.lens[b]]
            m = int(count[b])
            assert not o[b, m:].any()
            if m == 0:
                continue
            rows = torch.cat([old, self.fresh[b, :m]]) if self.fresh is not None else old
            see = torch.ones((m, len(rows)), dtype=torch.bool, device="cuda")
            see[:, len(old):] = torch.tensor(self.see[b, :m, :len(rows) - len(old)], device="cuda")
            for h0 in range(0, self.H, 16):
                hh = slice(h0, min(h0 + 16, self.H))
                k = hh.stop - h0
                q = self.q[b, :m, hh].reshape(m * k, W)
                s = see.repeat_interleave(k, 0)
                if len(rows) == 0:
                    assert not o[b, :m, hh].any()
                    continue
                want, A, d = _attend(q, rows, rows[:, :C], s, scale)
                want[~s.any(1)] = 0.0
                A[~s.any(1)] = 0.0
                got = o[b, :m, hh].double().reshape(m * k, C)
                top = float(rows[:, :C].double().abs().max())
                bad = ~((got - want).abs() <= _bound(want, A, d, len(rows), top, self.dt))
                assert not bool(bad.any()), (b, h0, float((got - want).abs().max()), int(bad.sum()))


SHAPES = [
    (1, 1, 1, 1, 16), (1, 1, 64, 63, 64), (1, 1, 64, 64, 64), (1, 1, 64, 65, 16), (2, 1, 128, 300, 32), (3, 5, 24, 300, 16),
    (1, 1, 16, 4097, 256), (5, 3, 8, 129, 128), (2, 17, 12, 1000, 64), (1, 64, 16, 511, 64), (2, 65, 4, 190, 32), (4, 1, 64, 2500, 64),
    (1, 8, 64, 5000, 64), (40, 2, 16, 700, 64), (3, 130, 3, 70, 16), (1, 2, 200, 100, 64), (300, 1, 8, 90, 16),
]


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("B,n,H,context,page", SHAPES)
def test_absorbed_matches_the_definition(lib, dtype, B, n, H, context, page):
    s = Scene(lib, B, n, H, context, page, dtype)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    o = s.run(err=err)
    s.check(o)
    assert lib.check_error(err) == 0
    assert torch.equal(o, s.run())  # no atomics on results


@pytest.mark.parametrize("B,n,H,context", [(1, 1, 64, 20000), (2, 3, 64, 9000), (7, 1, 32, 6000)])
def test_absorbed_long_contexts(lib, B, n, H, context):
    s = Scene(lib, B, n, H, context, 64, "bfloat16", ragged=B > 2)
    s.check(s.run())


def test_absorbed_without_drafts_and_chains(lib):
    s = Scene(lib, 3, 4, 20, 200, 32, "bfloat16", fresh=False)
    s.check(s.run(new=None, mask=None))
    s = Scene(lib, 3, 70, 5, 200, 32, "float16", tree="chain")
    s.see[:] = np.tril(np.ones((70, s.see.shape[2]), dtype=bool))[None]
    s.check(s.run(mask=None))
    s = Scene(lib, 2, 3, 16, 0, 16, "bfloat16")  # nothing cached
    s.check(s.run())
    s = Scene(lib, 2, 3, 16, 100, 16, "bfloat16", ragged=False)
    s.check(s.run(n_tok=None))


@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0, 1e-30, 300.0])
def test_absorbed_scales(lib, scale):
    s = Scene(lib, 2, 2, 16, 500, 64, "bfloat16", ragged=False)
    s.check(s.run(scale=scale), scale=scale)


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_absorbed_peaks_that_rise_late(lib, dtype):
    """Each row's largest score at its end, after many of every size: the running maximum moves again and again."""
    s = Scene(lib, 1, 1, 64, 3000, 64, dtype, ragged=False)
    ramp = torch.linspace(0, 1, 3000, device="cuda")[:, None]
    direction = s.q[0, 0, 0].float() / s.q[0, 0, 0].float().norm()
    flat = s.cache.rows.view(-1, W)
    for j, p in enumerate(s.table[0]):
        part = ramp[j * 64:(j + 1) * 64]
        flat[p * 64:p * 64 + len(part)] = (flat[p * 64:p * 64 + len(part)].float() + 25 * part * direction).to(s.dt)
    s.check(s.run())


def test_absorbed_what_is_not_seen_does_not_matter(lib):
    """NaN and infinities in drafts that a row does not see, past the drafts in use, in pages of other sequences."""
    s = Scene(lib, 3, 9, 16, 150, 16, "bfloat16")
    o = s.run()
    clean = s.fresh.clone()
    for b in range(3):
        m = int(s.count[b])
        s.fresh[b, m:] = float("nan")
    assert torch.equal(s.run(), o)
    b = 0
    m = int(s.count[b])
    for j in range(m):
        s.fresh.copy_(clean)
        s.fresh[b, j, 5] = float("inf") if j % 2 else float("nan")
        got = s.run()
        for i in range(m):
            if s.see[b, i, j]:
                assert bool(got[b, i].isnan().all())
            else:
                assert torch.equal(got[b, i], o[b, i])
        assert torch.equal(got[1:], o[1:])
    # a query that is not finite spoils its own row alone
    s.fresh.copy_(clean)
    s.q[0, 0, 3, 7] = float("nan")
    got = s.run()
    assert bool(got[0, 0, 3].isnan().all())
    got[0, 0, 3] = o[0, 0, 3]
    assert torch.equal(got, o)


def test_absorbed_cached_nan_reaches_the_rows_that_see_it(lib):
    s = Scene(lib, 2, 2, 16, 500, 64, "bfloat16", ragged=False)
    o = s.run()
    s.cache.rows[int(s.table[1, 3]), 10, 100] = float("nan")
    got = s.run()
    assert torch.equal(got[0], o[0]) and bool(got[1].isnan().all())


def test_absorbed_bad_pages_and_lengths(lib):
    """Pages outside the pool are left out, lengths clamped, each reported; the table past a length is not read."""
    s = Scene(lib, 2, 1, 16, 300, 64, "bfloat16", ragged=False)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    s.table[0, 2] = 99999
    s.table[1, 1] = -3
    o = s.run(err=err)
    assert lib.check_error(err) == 8
    for b, out in ((0, 2), (1, 1)):
        pages = [int(p) for j, p in enumerate(s.table[b]) if j != out]
        rows = torch.cat([s.cache.rows[p] for p in pages])[:300 - 64]
        rows = torch.cat([rows, s.fresh[b]])
        want, A, d = _attend(s.q[b, 0], rows, rows[:, :C], torch.ones((16, len(rows)), dtype=torch.bool, device="cuda"), SCALE)
        assert bool(((o[b, 0].double() - want).abs() <= _bound(want, A, d, 300, 6.0, s.dt)).all())
    s = Scene(lib, 2, 1, 16, 300, 64, "bfloat16", ragged=False)
    s.lens = np.array([-4, 300])
    o = s.run(err=err)
    assert lib.check_error(err) == 8
    s.lens = np.array([0, 300])
    s.check(o)
    s.lens = np.array([300, 500])
    o = s.run(err=err, max_len=256)
    assert lib.check_error(err) == 8
    s.lens = np.array([256, 256])
    s.check(o)


def test_absorbed_strided_queries_and_drafts(lib):
    s = Scene(lib, 3, 4, 16, 200, 32, "float16")
    o = s.run()
    big = torch.full((3, 4, 18, W), float("nan"), dtype=s.dt, device="cuda")
    big[:, :, 1:17] = s.q
    wide = torch.full((3, 4, W + 40), float("nan"), dtype=s.dt, device="cuda")
    wide[:, :, 8:8 + W] = s.fresh
    s.q, fresh = big[:, :, 1:17], wide[:, :, 8:8 + W]
    assert torch.equal(s.run(new=fresh), o)


def test_absorbed_slots_past_31_bits_of_elements(lib):
    """A pool of more than 2^31 elements: its last pages."""
    pages = 62000
    rows = torch.empty((pages, 64, W), dtype=torch.bfloat16, device="cuda")
    cache = lib.LatentCache(pages, 64, storage=rows)
    gen = _gen(9)
    c = torch.randn((200, W), generator=gen, device="cuda").bfloat16()
    table = np.array([[pages - 1, pages - 3, 1, pages - 2]])
    slots = (table[0].repeat(64) * 64 + np.tile(np.arange(64), 4))[:200]
    lib.latent_append(cache, c[:, :C], c[:, C:], _int(slots))
    q = torch.randn((1, 1, 16, W), generator=gen, device="cuda").bfloat16()
    o = lib.latent_attend_tree(cache, q, _int(table), _int([200]), SCALE)
    want, A, d = _attend(q[0, 0], c, c[:, :C], torch.ones((16, 200), dtype=torch.bool, device="cuda"), SCALE)
    assert bool(((o[0, 0].double() - want).abs() <= _bound(want, A, d, 200, 6.0, q.dtype)).all())


def test_absorbed_in_a_graph_and_on_another_stream(lib):
    s = Scene(lib, 6, 2, 64, 700, 64, "bfloat16")
    want = s.run()
    table, lens, count = _int(s.table), _int(s.lens), _int(s.count)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            got = lib.latent_attend_tree(s.cache, s.q, table, lens, SCALE, new=s.fresh, mask=s.mask, n_tok=count, max_len=s.most)
        for _ in range(3):
            graph.replay()
        # other lengths in the same graph
        stream.synchronize()
        assert torch.equal(got, want)
        s.lens = s.lens // 2
        lens.copy_(_int(s.lens))
        graph.replay()
    stream.synchronize()
    s.check(got)


def test_absorbed_calls_that_share_a_workspace_in_turn(lib):
    s, t = Scene(lib, 6, 2, 64, 700, 64, "bfloat16"), Scene(lib, 2, 1, 16, 4000, 64, "bfloat16")
    ws = torch.empty(1 << 28, dtype=torch.uint8, device="cuda").fill_(255)
    a, b = s.run(ws=ws), t.run(ws=ws)
    ws.fill_(255)
    assert torch.equal(s.run(), a) and torch.equal(t.run(), b)


# ---------------------------------------------------------------- expanded

def _prompts(ql, kl, H, dtype, *key, spread=1.0):
    gen, dt = _gen(*key), getattr(torch, dtype)
    qs, ks = np.concatenate([[0], np.cumsum(ql)]), np.concatenate([[0], np.cumsum(kl)])
    q = (torch.randn((int(qs[-1]), H, 192), generator=gen, device="cuda") * spread).to(dt)
    kv = torch.randn((int(ks[-1]), H, 256), generator=gen, device="cuda").to(dt)
    return q, kv, torch.randn((int(ks[-1]), R), generator=gen, device="cuda").to(dt), qs, ks


def _check_prompts(o, q, k, v, kr, qs, ks, scale=SCALE, causal=True):
    assert o.shape == (*q.shape[:2], 128) and o.dtype == q.dtype
    for b in range(len(qs) - 1):
        q0, q1, k0, k1 = (int(x) for x in (qs[b], qs[b + 1], ks[b], ks[b + 1]))
        if q1 == q0:
            continue
        if k1 == k0:
            assert not o[q0:q1].any()
            continue
        see = torch.ones((q1 - q0, k1 - k0), dtype=torch.bool, device="cuda")
        if causal:
            see = torch.arange(k1 - k0, device="cuda")[None] <= torch.arange(q1 - q0, device="cuda")[:, None] + (k1 - k0 - q1 + q0)
        for h in range(q.shape[1]):
            rows = torch.cat([k[k0:k1, h], kr[k0:k1]], 1)
            want, A, d = _attend(q[q0:q1, h], rows, v[k0:k1, h], see, scale)
            want[~see.any(1)] = 0.0
            A[~see.any(1)] = 0.0
            top = float(v[k0:k1, h].double().abs().max())
            bad = ~((o[q0:q1, h].double() - want).abs() <= _bound(want, A, d, k1 - k0, top, q.dtype))
            assert not bool(bad.any()), (b, h, float((o[q0:q1, h].double() - want).abs().max()), int(bad.sum()))


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("ql,kl,H", [
    ([1], [1], 1), ([5], [5], 3), ([127], [127], 2), ([128], [128], 1), ([129], [129], 2), ([256], [256], 2), ([257], [300], 2),
    ([1], [1000], 4), ([700], [700], 2), ([3, 0, 130, 64], [3, 40, 500, 64], 3), ([10, 20], [0, 20], 2), ([40], [17], 2),
    ([300, 1, 77], [100, 900, 77], 2), ([1] * 70, list(range(70)), 2), ([1300], [2000], 1), ([64, 65, 63, 1], [64, 65, 127, 128], 5)])
def test_expanded_matches_the_definition(lib, dtype, causal, ql, kl, H):
    q, kv, kr, qs, ks = _prompts(ql, kl, H, dtype, 5, sum(ql), H)
    k, v = kv[..., :128], kv[..., 128:]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    o = lib.latent_attend_prompt(q, k, v, kr, _int(qs), _int(ks), SCALE, causal=causal, err=err)
    _check_prompts(o, q, k, v, kr, qs, ks, causal=causal)
    assert lib.check_error(err) == 0
    assert torch.equal(o, lib.latent_attend_prompt(q, k.contiguous(), v.contiguous(), kr, _int(qs), _int(ks), SCALE, causal=causal))


@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0, 300.0])
def test_expanded_scales(lib, scale):
    q, kv, kr, qs, ks = _prompts([200, 33], [333, 33], 2, "bfloat16", 6)
    k, v = kv[..., :128], kv[..., 128:]
    _check_prompts(lib.latent_attend_prompt(q, k, v, kr, _int(qs), _int(ks), scale), q, k, v, kr, qs, ks, scale=scale)


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("scale", [1e6, -1e9, 1e15, 1e30])
def test_scores_of_any_size(lib, dtype, scale):
    """Scores up to 2^110: all weight lies on the highest (whichever the sums' roundings make that), so a result is a value's row."""
    s = Scene(lib, 2, 1, 16, 300, 64, dtype, ragged=False)
    o = s.run(scale=scale)
    for b in range(2):
        pages = torch.tensor(s.table[b], device="cuda").long()
        rows = torch.cat([s.cache.rows[pages].reshape(-1, W)[:300], s.fresh[b]])[:, :C]
        assert bool((o[b, 0][:, None] == rows[None]).all(-1).any(-1).all())
    q, kv, kr, qs, ks = _prompts([130, 33], [300, 33], 2, dtype, 14)
    o = lib.latent_attend_prompt(q, kv[..., :128], kv[..., 128:], kr, _int(qs), _int(ks), scale)
    for b in range(2):
        for h in range(2):
            rows = kv[ks[b]:ks[b + 1], h, 128:]
            assert bool((o[qs[b]:qs[b + 1], h][:, None] == rows[None]).all(-1).any(-1).all())


def test_expanded_peaks_that_rise_late(lib):
    q, kv, kr, qs, ks = _prompts([700], [700], 2, "bfloat16", 7)
    ramp = torch.linspace(0, 1, 700, device="cuda")[:, None, None]
    d = q[-1:, :, :128].float()
    kv[..., :128] = (kv[..., :128].float() + 20 * ramp * d / d.norm(dim=-1, keepdim=True)).to(kv.dtype)
    k, v = kv[..., :128], kv[..., 128:]
    _check_prompts(lib.latent_attend_prompt(q, k, v, kr, _int(qs), _int(ks), SCALE), q, k, v, kr, qs, ks)


@pytest.mark.parametrize("what", ["k", "v", "kr"])
def test_expanded_what_is_not_seen_does_not_matter(lib, what):
    """A token's key or value that is not finite: the rows before it and the other sequences as they were."""
    q, kv, kr, qs, ks = _prompts([200, 150], [260, 150], 2, "bfloat16", 8)
    o = lib.latent_attend_prompt(q, kv[..., :128], kv[..., 128:], kr, _int(qs), _int(ks), SCALE)
    for at, first in ((259, 199), (130, 70), (260 + 3, 200 + 3), (260 + 149, 349), (260 + 64, 264)):
        for x in (float("nan"), float("inf")):
            kv2, kr2 = kv.clone(), kr.clone()
            if what == "kr":
                kr2[at, 5] = x
            else:
                kv2[at, :, 3 if what == "k" else 131] = x
            got = lib.latent_attend_prompt(q, kv2[..., :128], kv2[..., 128:], kr2, _int(qs), _int(ks), SCALE)
            end = 200 if first < 200 else 350
            assert torch.equal(got[:first], o[:first]) and torch.equal(got[end:], o[end:])
            if what == "v":
                assert not bool(got[first:end, :, 3].isfinite().any())
            elif x != x:
                assert bool(got[first:end].isnan().all())


def test_expanded_rows_behind_the_last_sequence_and_bad_starts(lib):
    q, kv, kr, qs, ks = _prompts([100, 60, 40], [100, 60, 40], 2, "bfloat16", 10)
    k, v = kv[..., :128], kv[..., 128:]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = lib.latent_attend_prompt(q, k, v, kr, _int(qs), _int(ks), SCALE)
    o = lib.latent_attend_prompt(q, k, v, kr, _int(qs[:3]), _int(ks[:3]), SCALE, err=err)
    assert torch.equal(o[:160], want[:160]) and lib.check_error(err) == 0
    o = lib.latent_attend_prompt(q, k, v, kr, _int([0, 100, 160, 300]), _int(ks), SCALE, err=err)
    assert torch.equal(o[:160], want[:160]) and lib.check_error(err) == 8
    o = lib.latent_attend_prompt(q, k, v, kr, _int(qs), _int([0, 100, 90, 200]), SCALE, err=err)
    assert torch.equal(o[:100], want[:100]) and lib.check_error(err) == 8


@pytest.mark.parametrize("H", [2, 64])
@pytest.mark.parametrize("starts,kept", [
    ([0, 500, 100, 600], [0]),  # the third begins within the first
    ([0, 1 << 30, 300, 600], [2]), ([0, -7, 300, 600], [2]),  # one start alone is wrong
    ([0, 600] * 12, [0]),  # far more tiles than there are rows, were they all taken
    ([0] * 40 + [300, 299, 300, 600], [39, 42]),  # the last begins where an earlier one ends
    ([0, 200, 1 << 30, 100, 600], [0]), ([100, 50, 600, 50, 600], [])])
def test_expanded_sequences_that_would_overlap_are_left_out(lib, H, starts, kept):
    """Starts that fall and rise again: the sequences before the fall as they are alone, and nothing written over them."""
    q, kv, kr, _, _ = _prompts([600], [600], H, "bfloat16", 17)
    k, v, B = kv[..., :128], kv[..., 128:], len(starts) - 1
    keys = np.minimum(np.arange(B + 1) * 15, 600)
    if B < 8:
        keys = np.linspace(0, 600, B + 1).astype(int)
    fits = [b for b in range(B) if 0 <= starts[b] <= starts[b + 1] <= 600
            and all(not 0 <= x <= 600 or x <= starts[b] for x in starts[:b])]
    assert [b for b in fits if starts[b + 1] > starts[b]] == kept
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    o = lib.latent_attend_prompt(q, k, v, kr, _int(starts), _int(keys), SCALE, err=err)
    assert lib.check_error(err) == 8
    for b in fits:
        q0, q1, k0, k1 = starts[b], starts[b + 1], keys[b], keys[b + 1]
        if q1 > q0:
            alone = lib.latent_attend_prompt(q[q0:q1], k[k0:k1], v[k0:k1], kr[k0:k1], _int([0, q1 - q0]), _int([0, k1 - k0]), SCALE)
            assert torch.equal(o[q0:q1], alone)


def _soil(shape, dtype):
    """Memory that the next result of this shape is likely to lie in, full of NaN."""
    torch.cuda.synchronize()
    torch.full(shape, float("nan"), dtype=dtype, device="cuda")
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("ql,starts,H,kl", [
    ([200, 100], [0, 200, 250], 2, [200, 50]),  # 50 rows behind the last sequence
    ([200, 100], [70, 200, 300], 3, [130, 100]),  # 70 before the first
    ([600], [0, 500, 100, 600], 64, [200, 0, 300]), ([600], [0, 1 << 30, 300, 600], 2, [100, 100, 300]),  # left out
    ([4000], [0, 40], 16, [40]), ([300], [0, 20, 20, 20], 1, [2000, 0, 0]), ([3000], [3000, 0], 2, [100]),
    ([100], [0], 4, []), ([70], [0] * 71, 2, [1] * 70)])
def test_expanded_rows_of_no_sequence_are_zeros(lib, dtype, ql, starts, H, kl):
    q, kv, kr, _, ks = _prompts(ql, kl or [10], H, dtype, 18, sum(ql))
    ks = ks if kl else np.zeros(1, dtype=int)
    _soil((sum(ql), H, 128), q.dtype)
    o = lib.latent_attend_prompt(q, kv[..., :128], kv[..., 128:], kr, _int(starts), _int(ks), SCALE)
    assert not bool(o.isnan().any())
    rest = torch.ones(sum(ql), dtype=torch.bool, device="cuda")
    for b in range(len(starts) - 1):
        if starts[b] <= starts[b + 1] <= len(q) and max((x for x in starts[:b] if x <= len(q)), default=0) <= starts[b]:
            rest[starts[b]:starts[b + 1]] = False
            if starts[b + 1] > starts[b] and kl[b]:
                one = lib.latent_attend_prompt(q[starts[b]:starts[b + 1]], kv[ks[b]:ks[b + 1], :, :128], kv[ks[b]:ks[b + 1], :, 128:],
                                               kr[ks[b]:ks[b + 1]], _int([0, starts[b + 1] - starts[b]]), _int([0, kl[b]]), SCALE)
                assert torch.equal(o[starts[b]:starts[b + 1]], one)
    assert bool(rest.any()) and not bool(o[rest].any())


def test_a_plan_and_its_prompts_leave_no_old_memory(lib):
    """Prompts planned into more packed places than they fill: the attention gives zeros in the places behind the last token."""
    pool = lib.PagePool(20, 16, 2, 8)
    plan = lib.kv_plan(pool, _int([0, 0]), _int([30, 21]), tokens=64)
    q, kv, kr, _, _ = _prompts([64], [64], 2, "bfloat16", 19)
    _soil((64, 2, 128), q.dtype)
    o = lib.latent_attend_prompt(q, kv[..., :128], kv[..., 128:], kr, plan.starts, plan.starts, SCALE)
    assert not bool(o[51:].any()) and bool(o[:51].isfinite().all()) and bool(o[:51].any(-1).all())


def test_expanded_in_a_graph_and_on_another_stream(lib):
    q, kv, kr, qs, ks = _prompts([100, 160], [100, 300], 2, "bfloat16", 11)
    k, v, dq, dk = kv[..., :128], kv[..., 128:], _int(qs), _int(ks)
    want = lib.latent_attend_prompt(q, k, v, kr, dq, dk, SCALE)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            got = lib.latent_attend_prompt(q, k, v, kr, dq, dk, SCALE)
        for _ in range(3):
            graph.replay()
        stream.synchronize()
        assert torch.equal(got, want)
        dq.copy_(_int([0, 30, 260]))  # other lengths in the same graph
        dk.copy_(_int([0, 50, 400]))
        graph.replay()
    stream.synchronize()
    _check_prompts(got, q, k, v, kr, [0, 30, 260], [0, 50, 400])


def test_expired_waits_are_reported(lib):
    """A wait budget of 0: a status and not a hang, and the next call as before."""
    s = Scene(lib, 3, 2, 64, 700, 64, "bfloat16")
    q, kv, kr, qs, ks = _prompts([300, 50], [700, 50], 2, "bfloat16", 13)
    prompt = lambda err=None: lib.latent_attend_prompt(q, kv[..., :128], kv[..., 128:], kr, _int(qs), _int(ks), SCALE, err=err)  # noqa: E731
    want, want2 = s.run(), prompt()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    lib.set_wait_budget(0)
    try:
        s.run(err=err)
        assert lib.check_error(err) & 2
        prompt(err=err)
        assert lib.check_error(err) & 2
    finally:
        lib.set_wait_budget(-1)
    assert torch.equal(s.run(err=err), want) and torch.equal(prompt(err), want2) and lib.check_error(err) == 0


@pytest.mark.parametrize("B,n,H,context", [(3, 2, 64, 700), (1, 1, 64, 6000), (200, 1, 64, 300)])
@pytest.mark.parametrize("word", [-1, 0, 0x01010101, 0x7fffffff, 151])
def test_expired_waits_over_scratch_that_holds_anything(lib, word, B, n, H, context):
    """A wait budget of 0 over scratch whose words name no CTAs, or others': a status, and the next call as before."""
    s = Scene(lib, B, n, H, context, 64, "bfloat16")
    ws = torch.full((1 << 26,), word, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    lib.set_wait_budget(0)
    try:
        s.run(err=err, ws=ws)
        assert lib.check_error(err) & 2
    finally:
        lib.set_wait_budget(-1)
    ws.fill_(word)
    o = s.run(err=err, ws=ws)
    s.check(o)
    assert lib.check_error(err) == 0


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("ql,kl,H", [([1], [5000], 2), ([16], [9000], 1), ([300], [4200], 3), ([5, 0, 260], [3000, 2000, 1030], 4),
                                     ([700], [1100], 1), ([2, 3, 4], [1024, 0, 7], 5), ([3000], [2500], 1)])
def test_expanded_few_rows_over_many_keys(lib, dtype, causal, ql, kl, H):
    """Jobs cut along the keys and joined: parts that a row sees all, part and nothing of, rows that see nothing, short sequences beside."""
    q, kv, kr, qs, ks = _prompts(ql, kl, H, dtype, 16, sum(ql), H)
    k, v = kv[..., :128], kv[..., 128:]
    ws = torch.full((1 << 26,), 255, dtype=torch.uint8, device="cuda")
    o = lib.latent_attend_prompt(q, k, v, kr, _int(qs), _int(ks), SCALE, causal=causal, ws=ws)
    _check_prompts(o, q, k, v, kr, qs, ks, causal=causal)
    assert torch.equal(o, lib.latent_attend_prompt(q, k, v, kr, _int(qs), _int(ks), SCALE, causal=causal))
    # what the rows do not see: past the sequence's keys, and the last key of all (its last row alone)
    if causal and len(ql) == 1 and 1 < ql[0] < kl[0]:
        kv[-1] = float("nan")
        got = lib.latent_attend_prompt(q, k, v, kr, _int(qs), _int(ks), SCALE)
        assert torch.equal(got[:-1], o[:-1]) and bool(got[-1].isnan().all())


def test_expanded_more_jobs_than_sms_in_a_graph(lib):
    """Jobs that CTAs take as they come free, the counter in a workspace that holds anything; replayed, and another call between."""
    q, kv, kr, qs, ks = _prompts([700, 300, 513, 40], [900, 300, 600, 1000], 40, "bfloat16", 15)
    k, v, dq, dk = kv[..., :128], kv[..., 128:], _int(qs), _int(ks)
    ws = torch.full((64,), 255, dtype=torch.uint8, device="cuda")
    want = lib.latent_attend_prompt(q, k, v, kr, dq, dk, SCALE, ws=ws)
    _check_prompts(want[:, :2], q[:, :2], k[:, :2], v[:, :2], kr, qs, ks)
    _check_prompts(want[:, 39:], q[:, 39:], k[:, 39:], v[:, 39:], kr, qs, ks)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            got = lib.latent_attend_prompt(q, k, v, kr, dq, dk, SCALE, ws=ws)
            twice = lib.latent_attend_prompt(q, k, v, kr, dq, dk, SCALE, ws=ws)
        for _ in range(3):
            got.zero_()
            twice.zero_()
            graph.replay()
            assert torch.equal(lib.latent_attend_prompt(q, k, v, kr, dq, dk, SCALE, ws=ws), want)
            assert torch.equal(got, want) and torch.equal(twice, want)
    torch.cuda.current_stream().wait_stream(stream)


@pytest.mark.parametrize("B,n,H,context", [(200, 1, 64, 300), (60, 9, 64, 100), (1, 64, 128, 900), (170, 2, 24, 64)])
def test_absorbed_more_units_than_sms(lib, B, n, H, context):
    """Runs that cross units: several tiles to a CTA, tiles that two of them share."""
    s = Scene(lib, B, n, H, context, 32, "bfloat16")
    o = s.run()
    s.check(o)
    assert torch.equal(o, s.run())


def test_two_streams_at_once(lib):
    """Calls on two streams with scratch of their own."""
    s, t = Scene(lib, 6, 2, 64, 3000, 64, "bfloat16"), Scene(lib, 9, 1, 32, 2000, 16, "float16")
    want = s.run(), t.run()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(a):
            x = s.run()
        with torch.cuda.stream(b):
            y = t.run()
        a.synchronize()
        b.synchronize()
        assert torch.equal(x, want[0]) and torch.equal(y, want[1])


# ---------------------------------------------------------------- together

def test_both_forms_agree_over_a_served_prompt(lib):
    """A prompt planned, written and attended in the expanded form; its last token once more in the absorbed form over the cache:
    the same up to the roundings of two roads (queries and values through a projection each)."""
    H, T, page = 16, 333, 64
    gen = _gen(12)
    dt = torch.bfloat16
    wk = torch.randn((H, 128, C), generator=gen, device="cuda") * C ** -0.5
    wv = torch.randn((H, 128, C), generator=gen, device="cuda") * C ** -0.5
    c = torch.randn((T, C), generator=gen, device="cuda").to(dt)
    kr = torch.randn((T, R), generator=gen, device="cuda").to(dt)
    q = torch.randn((T, H, 192), generator=gen, device="cuda").to(dt)
    rope = lib.Rope(R, R, base=50000.0, layout="interleaved")
    pool, cache = lib.PagePool(12, page, 1, 8), lib.LatentCache(12, page)
    plan = lib.kv_plan(pool, _int([0]), _int([T]), tokens=T)
    lib.latent_append(cache, c, kr, plan.slots, rope=rope, positions=plan.positions)
    turned = lib.rope(kr[:, None], plan.positions, rope)[:, 0]
    qr = lib.rope(q[..., 128:], plan.positions, rope) if q[..., 128:].stride(-2) == R else lib.rope(q[..., 128:].contiguous(), plan.positions, rope)
    q = torch.cat([q[..., :128], qr], -1)
    k = torch.einsum("tc,hdc->thd", c.float(), wk).to(dt)
    v = torch.einsum("tc,hdc->thd", c.float(), wv).to(dt)
    full = lib.latent_attend_prompt(q, k, v, turned, plan.starts, plan.starts, SCALE)
    last = torch.cat([torch.einsum("hd,hdc->hc", q[-1, :, :128].float(), wk).to(dt), q[-1, :, 128:]], -1)[None, None]
    o = lib.latent_attend_tree(cache, last.contiguous(), pool.table, plan.lens, SCALE)
    got = torch.einsum("hc,hdc->hd", o[0, 0].float(), wv)
    # relative 2-norms: bf16 roundings of keys, values, queries, weights and results, each 2^-8 / sqrt(3) rms at most: eight of them
    assert float((got - full[-1].float()).norm() / full[-1].float().norm()) < math.sqrt(8) * 2.0 ** -8


def test_served_requests_with_drafts(lib):
    """The example of all of them in a row: planned, written, attended in both forms, verified; nothing reported, every accepted token
    counted, and both forms the same up to eight bf16 roundings (as above)."""
    import importlib.util
    import os

    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "latent_decode.py")
    spec = importlib.util.spec_from_file_location("latent_decode", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    worst, bits, lens, accepted = example.main()
    assert bits == 0 and sum(lens) == sum(example.PROMPTS) + accepted
    assert worst < math.sqrt(8) * 2.0 ** -8
