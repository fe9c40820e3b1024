"""Pages planned on the GPU and drafted trees verified there, against plain host code.

All results are whole numbers.  The plan is compared with lists of pages kept on the host; the verification with a walk in exact
rational arithmetic (probabilities are binary fractions), so a token can differ only where the kernel's steps of 2^-50 decide: the
numbers u are drawn until no threshold lies within 2^-30 of a border, which the steps of at most 2^20 entries cannot reach."""
from fractions import Fraction

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def _rng(*key):
    return np.random.Generator(np.random.PCG64(list(key)))


def _int(a):
    return torch.tensor(np.ascontiguousarray(a), dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- pages

class Host:
    """A pool kept in lists."""

    def __init__(self, pages, page, owned, free, width):
        self.pages, self.page, self.owned, self.free, self.width = pages, page, [list(o) for o in owned], list(free), width

    def plan(self, lens, new, n=None, tokens=None, path=None):
        B, page, bits = len(lens), self.page, 0
        rows = n if n is not None else tokens
        need = [-(-(lens[b] + new[b]) // page) for b in range(B)]
        bad = [lens[b] < 0 or new[b] < 0 or new[b] > rows or need[b] > self.width for b in range(B)]
        starts, at = [], 0
        for b in range(B):
            starts.append(min(at, tokens or 0))
            room = new[b] if 0 <= new[b] <= rows else 0
            if n is None and at + room > tokens:
                bad[b] = True
            at += room
        starts.append(min(at, tokens or 0))
        back = []
        for b in range(B):
            if not bad[b]:
                back += self.owned[b][need[b]:]
                del self.owned[b][need[b]:]
        self.free += back[::-1]
        asked, stack = 0, list(self.free)
        served, used = [], 0
        for b in range(B):
            more = 0 if bad[b] else max(0, need[b] - len(self.owned[b]))
            ok = not bad[b] and (more == 0 or asked + more <= len(stack))
            if ok and more:
                self.owned[b] += [stack[len(stack) - 1 - asked - k] for k in range(more)]
                used = asked + more
            asked += more
            served.append(ok)
            bits |= 0 if ok else 8 if bad[b] else 16
        self.free = stack[:len(stack) - used]
        shape = (B, n) if n is not None else (tokens,)
        slots, positions = np.full(shape, -1), np.zeros(shape, dtype=np.int64)
        after = [lens[b] + new[b] if served[b] else lens[b] for b in range(B)]
        for b in range(B):
            for i in range(new[b] if served[b] else 0):
                t = lens[b] + i
                where = starts[b] + i if n is None else (b, i if path is None else path[b][i])
                slots[where], positions[where] = self.owned[b][t // page] * page + t % page, t
        return slots, positions, after, starts, bits


def _pool(lib, host):
    pool = lib.PagePool(host.pages, host.page, len(host.owned), host.width)
    table = np.full((len(host.owned), host.width), -1)
    for b, o in enumerate(host.owned):
        table[b, :len(o)] = o
    if host.width and len(host.owned):
        pool.table.copy_(_int(table))
    pool.held.copy_(_int([len(o) for o in host.owned]))
    pool.free.fill_(-7)
    pool.free[:len(host.free)] = _int(host.free)
    pool.n_free.fill_(len(host.free))
    return pool


def _same(pool, host):
    n = int(pool.n_free)
    assert pool.free[:n].tolist() == host.free
    assert pool.held.tolist() == [len(o) for o in host.owned]
    for b, o in enumerate(host.owned):
        assert pool.table[b].tolist() == o + [-1] * (host.width - len(o))


def _scene(g, B, most, page, spare, pages_extra=3, width_extra=2, new=0):
    lens = g.integers(0, most + 1, B)
    held = -(-lens // page)
    total = int(held.sum()) + spare + pages_extra
    order, at, owned = g.permutation(max(total, 1)).tolist(), 0, []
    for h in held:
        owned.append(order[at:at + h])
        at += h
    return lens.tolist(), Host(max(total, 1), page, owned, order[at:at + spare], int(-(-(most + new) // page)) + width_extra)


@pytest.mark.parametrize("B,most,new,page,spare", [
    (1, 0, 1, 16, 1), (1, 100, 5, 16, 0), (7, 300, 9, 16, 40), (64, 1000, 8, 64, 64), (65, 63, 33, 32, 20), (300, 200, 64, 16, 500),
    (1025, 90, 3, 64, 300), (2500, 70, 2, 16, 100), (3, 5000, 3000, 256, 60), (2, 0, 9000, 16, 1200)])
@pytest.mark.parametrize("form", ["padded", "path", "packed"])
def test_plan_matches_lists(lib, B, most, new, page, spare, form):
    g = _rng(1, B, most, new, page, spare)
    lens, host = _scene(g, B, most, page, spare, new=new)
    fresh = g.integers(0, new + 1, B).tolist()
    pool, err = _pool(lib, host), torch.zeros(1, dtype=torch.int32, device="cuda")
    kw, path = dict(n=new), None
    if form == "path":
        path = [g.permutation(new).tolist() for _ in range(B)]
        kw["path"] = _int(path)
    elif form == "packed":
        kw = dict(tokens=sum(fresh) + 5)
    before = pool.free.clone(), pool.table.clone(), pool.held.clone()
    plan = lib.kv_plan(pool, _int(lens), _int(fresh), err=err, **kw)
    slots, positions, after, starts, bits = host.plan(lens, fresh, n=kw.get("n"), tokens=kw.get("tokens"), path=path)
    assert np.array_equal(plan.slots.cpu().numpy(), slots) and np.array_equal(plan.positions.cpu().numpy(), positions)
    assert plan.lens.tolist() == after and lib.check_error(err) == bits
    if form == "packed":
        assert plan.starts.tolist() == starts
    _same(pool, host)
    # the same step undone: the pool as it was
    undone = lib.kv_plan(pool, _int(lens), _int([0] * B), n=1)
    assert torch.equal(undone.slots, torch.full((B, 1), -1, dtype=torch.int32, device="cuda")) and undone.lens.tolist() == lens
    n = int(pool.n_free)
    assert n == spare and torch.equal(pool.free[:n], before[0][:n])
    assert torch.equal(pool.table, before[1]) and torch.equal(pool.held, before[2])


@pytest.mark.parametrize("B", [5, 1500])
def test_plan_gives_and_takes_in_one_call(lib, B):
    """Requests end and grow in the same step, over several steps."""
    g = _rng(2, B)
    lens, host = _scene(g, B, 400, 16, 40)
    pool = _pool(lib, host)
    for step in range(6):
        ends = g.random(B) < 0.3
        lens = [0 if e else n for e, n in zip(ends, lens)]
        new = [0 if e else int(x) for e, x in zip(ends, g.integers(0, 30, B))]
        host.width = max(host.width, 64)
        if pool.width < host.width:
            pool = _pool(lib, host)
        plan = lib.kv_plan(pool, _int(lens), _int(new), n=30)
        slots, positions, after, _, _ = host.plan(lens, new, n=30)
        assert np.array_equal(plan.slots.cpu().numpy(), slots) and np.array_equal(plan.positions.cpu().numpy(), positions)
        assert plan.lens.tolist() == after
        _same(pool, host)
        lens = after


def test_plan_refuses_by_sequence(lib):
    """Bad lengths, counts above the columns, tables too narrow, a pool that runs out: each refused alone, pages kept."""
    page = 16
    host = Host(40, page, [[3, 4], [5], [6, 7, 8], [], [9], [10]], [20, 21, 22, 23], 4)
    pool, err = _pool(lib, host), torch.zeros(1, dtype=torch.int32, device="cuda")
    lens, new = [20, -1, 40, 10, 16, 60], [3, 2, -5, 9, 4, 6]
    plan = lib.kv_plan(pool, _int(lens), _int(new), n=8, err=err)
    slots, positions, after, _, bits = host.plan(lens, new, n=8)
    assert bits == 8 and after == [23, -1, 40, 10, 20, 60]
    assert np.array_equal(plan.slots.cpu().numpy(), slots) and plan.lens.tolist() == after and lib.check_error(err) == bits
    _same(pool, host)
    # three pages left: the second sequence needs four, the third's one comes after it, the fourth needs none
    host = Host(40, page, [[1], [2], [3], [4]], [11, 12, 13], 8)
    pool = _pool(lib, host)
    lens, new = [16, 16, 16, 10], [1, 64, 1, 6]
    plan = lib.kv_plan(pool, _int(lens), _int(new), n=64, err=err)
    slots, positions, after, _, bits = host.plan(lens, new, n=64)
    assert bits == 16 and after == [17, 16, 16, 16] and host.free == [11, 12]
    assert np.array_equal(plan.slots.cpu().numpy(), slots) and plan.lens.tolist() == after and lib.check_error(err) == bits
    _same(pool, host)


def test_plan_packed_tokens_that_do_not_fit(lib):
    host = Host(64, 16, [[], [1, 2, 3], [4]], list(range(20, 40)), 8)
    pool, err = _pool(lib, host), torch.zeros(1, dtype=torch.int32, device="cuda")
    lens, new = [0, 3, 5], [10, 12, 4]
    plan = lib.kv_plan(pool, _int(lens), _int(new), tokens=20, err=err)
    slots, _, after, starts, bits = host.plan(lens, new, tokens=20)
    assert after == [10, 3, 5] and bits == 8 and len(host.owned[1]) == 3  # (refused: it gives nothing back either)
    assert np.array_equal(plan.slots.cpu().numpy(), slots) and plan.starts.tolist() == starts and plan.lens.tolist() == after
    assert lib.check_error(err) == bits
    _same(pool, host)


def test_plan_bad_path_entries_drop_their_tokens(lib):
    host = Host(8, 16, [[2]], [3], 4)
    pool, err = _pool(lib, host), torch.zeros(1, dtype=torch.int32, device="cuda")
    plan = lib.kv_plan(pool, _int([4]), _int([3]), n=3, path=_int([[2, 7, 0]]), err=err)
    assert plan.slots.tolist() == [[2 * 16 + 6, -1, 2 * 16 + 4]] and plan.positions.tolist() == [[6, 0, 4]]
    assert plan.lens.tolist() == [7] and lib.check_error(err) == 8


def test_plan_no_sequences_and_no_tokens(lib):
    pool = lib.PagePool(4, 16, 0, 4)
    empty = torch.zeros(0, dtype=torch.int32, device="cuda")
    plan = lib.kv_plan(pool, empty, empty, n=3)
    assert plan.slots.shape == (0, 3) and plan.lens.numel() == 0
    plan = lib.kv_plan(pool, empty, empty, tokens=7)
    assert plan.slots.tolist() == [-1] * 7 and plan.starts.tolist() == [0]
    pool = lib.PagePool(4, 16, 2, 4)
    plan = lib.kv_plan(pool, _int([0, 0]), _int([0, 0]), tokens=0)
    assert plan.starts.tolist() == [0, 0, 0] and int(pool.n_free) == 4


@pytest.mark.parametrize("form", ["padded", "packed"])
def test_plan_in_a_graph_and_on_another_stream(lib, form):
    g = _rng(3)
    lens, host = _scene(g, 40, 200, 16, 200)
    pool = _pool(lib, host)
    dl, dn = _int(lens), _int([3] * 40)
    kw = dict(n=4) if form == "padded" else dict(tokens=9000)
    lib.kv_plan(_pool(lib, host), dl, dn, **kw)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            plan = lib.kv_plan(pool, dl, dn, **kw)
            dl.copy_(plan.lens)
        for _ in range(5):
            graph.replay()
            slots, positions, after, _, _ = host.plan(lens, [3] * 40, n=kw.get("n"), tokens=kw.get("tokens"))
            stream.synchronize()
            assert np.array_equal(plan.slots.cpu().numpy(), slots) and np.array_equal(plan.positions.cpu().numpy(), positions)
            lens = after
    _same(pool, host)


# ---------------------------------------------------------------- verification

def _walk(p, q, tokens, parent, u, used):
    """The walk of one tree in exact arithmetic: p, q rows of Fractions.  Also the smallest relative distance to a border."""
    n, V = len(p), len(p[0])
    if used == 0:
        return [], -1, 1.0
    node, path, r, R, near = 0, [0], list(p[0]), Fraction(1), 1.0
    for i in range(1, used):
        if parent[i] != node or not 0 <= parent[i] < i or not 0 <= tokens[i] < V:
            continue
        x = tokens[i]
        left = Fraction(u[i]) * (q[node][x] if q is not None else 1) * R
        if left or r[x]:
            near = min(near, float(abs(left - r[x]) / max(left, r[x])))
        if left < r[x]:
            node, r, R = i, list(p[i]), Fraction(1)
            path.append(i)
        elif q is not None:
            r = [max(a - R * b, Fraction(0)) for a, b in zip(r, q[node])]
            R = sum(r)
        else:
            R -= r[x]
            r[x] = Fraction(0)
    total = sum(r)
    if total == 0:
        r = list(p[node])
        total = sum(r)
    if total == 0:
        return path, -1, near
    want, cum, token = Fraction(u[0]) * total, Fraction(0), None
    for t in range(V):
        cum += r[t]
        near = min(near, float(abs(cum - want) / total))
        if token is None and cum > want:
            token = t
    if token is None:
        token = max(t for t in range(V) if r[t] > 0)
    return path, token, near


def _probabilities(g, shape, dtype, peak=3.0):
    x = np.exp(peak * g.normal(size=shape))
    return torch.tensor(x / x.sum(-1, keepdims=True), dtype=torch.float32).to(dtype)


def _exact_rows(t):
    return [[Fraction(x) for x in row] for row in t.double().tolist()]


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("proposal", [True, False])
@pytest.mark.parametrize("B,n,V,tree", [(3, 1, 7, "chain"), (9, 5, 50, "chain"), (6, 12, 33, "random"), (5, 9, 257, "star"),
                                        (2, 64, 40, "bushy"), (3, 6, 2049, "random")])
def test_verify_matches_the_walk(lib, dtype, proposal, B, n, V, tree):
    g = _rng(4, B, n, V, proposal)
    dt = getattr(torch, dtype)
    q = _probabilities(g, (B, n, V), dt)
    p = ((0.6 * q.float() + 0.4 * _probabilities(g, (B, n, V), torch.float32))).to(dt)
    parent = np.full((B, n), -1)
    for b in range(B):
        for i in range(1, n):
            parent[b, i] = {"chain": i - 1, "random": int(g.integers(max(0, i - 4), i)), "star": 0, "bushy": (i - 1) // 4}[tree]
    tokens = np.zeros((B, n), dtype=np.int64)
    pq = q.double().numpy()
    for b in range(B):
        for i in range(1, n):
            row = pq[b, parent[b, i]]
            tokens[b, i] = g.choice(V, p=row / row.sum()) if proposal else np.argsort(-row)[i % min(V, 4)]
    used = np.where(g.random(B) < 0.4, g.integers(1, n + 1, B), n)
    u = np.zeros((B, n), dtype=np.float32)
    want = []
    for b in range(B):
        P, Q = _exact_rows(p[b]), _exact_rows(q[b]) if proposal else None
        while True:
            u[b] = g.random(n).astype(np.float32)
            path, token, near = _walk(P, Q, tokens[b].tolist(), parent[b].tolist(), u[b].tolist(), used[b])
            if near > 2.0 ** -30:
                break
        want.append((path + [-1] * (n - len(path)), len(path), token))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    path, count, token = lib.verify_tree(p.cuda(), _int(tokens), _int(parent), torch.tensor(u, device="cuda"),
                                         q=q.cuda() if proposal else None, n_tok=_int(used), err=err)
    assert path.tolist() == [w[0] for w in want]
    assert count.tolist() == [w[1] for w in want] and token.tolist() == [w[2] for w in want]
    assert lib.check_error(err) == 0


def _plain_next(r, u0):
    cum = np.cumsum(r.astype(np.float64))
    return int(np.searchsorted(cum, u0 * cum[-1], side="right"))


@pytest.mark.parametrize("V", [256, 8191, 8192, 50001, 131072, 1 << 20])
@pytest.mark.parametrize("B", [1, 3, 200])
def test_verify_large_vocabularies(lib, V, B):
    """One rejected draft, so both rows are read; every way of splitting a tree over CTAs.  u at many places, the ends among them.
    64-bit sums of at most 2^20 entries are off by less than 2^-32 of the sum, steps of 2^-50 by 2^-30: borders nearer than 2^-28
    are taken either way."""
    if B * V > 1 << 25:
        pytest.skip("inputs beyond a few hundred MB")
    gen = torch.Generator(device="cuda").manual_seed(V + B)
    q = torch.softmax(2 * torch.randn((B, 2, V), generator=gen, device="cuda"), -1)
    p = torch.softmax(2 * torch.randn((B, 2, V), generator=gen, device="cuda"), -1)
    tokens = torch.zeros((B, 2), dtype=torch.int32, device="cuda")
    tokens[:, 1] = (q[:, 0] - p[:, 0]).argmax(1).int()  # offered far more often than wanted: rejected at u near 1
    u = torch.rand((B, 2), generator=gen, device="cuda")
    u[:, 1] = 0.999999
    u[0, 0] = 0.0
    if B > 1:
        u[1, 0] = 1.0 - 2.0 ** -24
    parent = _int([[-1, 0]] * B)
    path, count, token = lib.verify_tree(p, tokens, parent, u, q=q)
    assert count.tolist() == [1] * B and path.tolist() == [[0, -1]] * B
    r = torch.clamp(p[:, 0].double() - q[:, 0].double(), min=0)
    cum = r.cumsum(1)
    at, total = u[:, 0].double() * cum[:, -1], cum[:, -1]
    rows = torch.arange(B, device="cuda")
    t = token.long()
    assert bool(((t >= 0) & (t < V)).all()) and bool((r[rows, t] > 0).all())
    slack = 2.0 ** -28 * total
    assert bool((cum[rows, t] > at - slack).all()) and bool((cum[rows, t] - r[rows, t] <= at + slack).all())


def test_verify_edges(lib):
    """Equal probabilities, zeros, a u of 0 and of nearly 1, nothing left of the residual, rows of zeros and of NaN."""
    dev, f = "cuda", torch.float32
    one = lambda *x: torch.tensor([x], dtype=f, device=dev)  # noqa: E731
    # p == q: accepted for every u below 1
    p = torch.tensor([[[0.25, 0.75], [0.5, 0.5]]], device=dev)
    assert lib.verify_tree(p, _int([[0, 1]]), _int([[-1, 0]]), one(0.0, 1 - 2.0 ** -24), q=p)[0].tolist() == [[0, 1]]
    # u q = p exactly: not below it, rejected; the residual is all of the other token
    q = torch.tensor([[[0.5, 0.5], [0.5, 0.5]]], device=dev)
    path, count, token = lib.verify_tree(p, _int([[0, 0]]), _int([[-1, 0]]), one(0.0, 0.5), q=q)
    assert path.tolist() == [[0, -1]] and token.tolist() == [1]
    # a rejected token without a residual (u is not below 1): the target's own distribution
    path, count, token = lib.verify_tree(p, _int([[0, 0]]), _int([[-1, 0]]), one(0.3, 1.0), q=p)
    assert count.tolist() == [1] and token.tolist() == [1]
    # u of 1 (outside its range) and above: the last token that has any probability
    z = torch.tensor([[[0.5, 0.5, 0.0]]], device=dev)
    assert lib.verify_tree(z, _int([[0]]), _int([[-1]]), one(1.0))[2].tolist() == [1]
    assert lib.verify_tree(z, _int([[0]]), _int([[-1]]), one(float("nan")))[2].tolist() == [0]
    # rows that hold nothing
    for bad in (0.0, float("nan"), -1.0):
        assert lib.verify_tree(torch.full((1, 1, 5), bad, device=dev), _int([[0]]), _int([[-1]]), one(0.5))[2].tolist() == [-1]
    # NaN and negative entries count as zeros beside others
    z = torch.tensor([[[float("nan"), 0.25, -3.0, 0.75]]], device=dev)
    assert lib.verify_tree(z, _int([[0]]), _int([[-1]]), one(0.2))[2].tolist() == [1]
    assert lib.verify_tree(z, _int([[0]]), _int([[-1]]), one(0.3))[2].tolist() == [3]
    # without proposals: the same token twice is tested once; the rest follows
    z = torch.tensor([[[0.5, 0.25, 0.25]] * 3], device=dev)
    path, count, token = lib.verify_tree(z, _int([[0, 0, 0]]), _int([[-1, 0, 0]]), one(0.6, 0.5, 0.0))
    assert count.tolist() == [1] and token.tolist() == [2]
    # no nodes in use
    path, count, token = lib.verify_tree(z, _int([[0, 0, 0]]), _int([[-1, 0, 0]]), one(0.6, 0.5, 0.0), n_tok=_int([0]))
    assert path.tolist() == [[-1, -1, -1]] and count.tolist() == [0] and token.tolist() == [-1]


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("case", ["apart", "alike", "chosen"])
def test_verify_residuals_computed_anew(lib, dtype, case):
    """80 trees over 131072 tokens: parts too long for shared memory, so that each pass and the search go over the rows and all the
    node's rejections again.  Sums are exact, so one tree alone (whose residual is kept) gives the same.  "alike": next to nothing is
    left after a rejection, so the residual's steps are made finer, again and again."""
    B, n, V = 80, 7, 131072
    dt = getattr(torch, dtype)
    gen = torch.Generator(device="cuda").manual_seed(21)
    q = torch.softmax(2 * torch.randn((B, n, V), generator=gen, device="cuda"), -1)
    if case == "alike":
        p = q * (1 + 2.0 ** -18 * torch.randn((B, n, V), generator=gen, device="cuda")) if dtype == "float32" else q.clone()
        if dtype != "float32":  # a handful of entries apart, a step of the type each
            p[:, :, ::9973] *= 1 + 2.0 ** -6
            p[:, :, 5::9973] *= 1 - 2.0 ** -6
    else:
        p = torch.softmax(2 * torch.randn((B, n, V), generator=gen, device="cuda"), -1)
    p, q = p.to(dt), q.to(dt)
    tokens = (q[:, 0].float() - p[:, 0].float()).argsort(1, descending=True)[:, :n].int()  # offered too often: rejected at u near 1
    u = torch.rand((B, n), generator=gen, device="cuda")
    u[:, 1:4] = 1 - 2.0 ** -24
    parent = _int([[-1, 0, 0, 0, 0, 4, 4]] * B)
    kw = {} if case == "chosen" else dict(q=q)
    got = lib.verify_tree(p, tokens.contiguous(), parent, u, **kw)
    for b in range(0, B, 7):
        kw = {} if case == "chosen" else dict(q=q[b:b + 1])
        one = lib.verify_tree(p[b:b + 1], tokens[b:b + 1].contiguous(), parent[:1], u[b:b + 1], **kw)
        assert all(torch.equal(x[b:b + 1], y) for x, y in zip(got, one))
    if case != "apart" or dtype != "float32":
        return
    # two rejections and more in 64 bits, for the trees whose other children were rejected as well: steps of 2^-51 over 2^17 entries,
    # three times, and fp64 sums: thresholds nearer than 2^-30 are taken either way
    rows = torch.arange(B, device="cuda")
    out = (got[1] == 1).nonzero().flatten()
    assert len(out) >= 10
    P, Q = p[out, 0].double(), q[out, 0].double()
    r, R = P, torch.ones(len(out), 1, dtype=torch.float64, device="cuda")
    for _ in range(4):
        r = torch.clamp(r - R * Q, min=0)
        R = r.sum(1, keepdim=True)
    cum, t = r.cumsum(1), got[2][out].long()
    rows = torch.arange(len(out), device="cuda")
    at = u[out, 0].double() * cum[:, -1]
    assert bool((cum[rows, t] > at - 2.0 ** -30).all()) and bool((cum[rows, t] - r[rows, t] <= at + 2.0 ** -30).all())


@pytest.mark.parametrize("V", [37, 300])
def test_verify_next_to_nothing_left(lib, V):
    """Targets that differ from the proposal by some 2^-18 of a probability: a rejection leaves less than 2^-16, whose steps are made
    finer before the next test.  Against the walk in rational arithmetic."""
    g = _rng(22, V)
    B, n = 40, 6
    q = _probabilities(g, (B, n, V), torch.float32, peak=0.5)
    p = (q.double() * (1 + 2.0 ** -17 * torch.tensor(g.normal(size=(B, n, V))))).float()
    parent = np.array([[-1] + [0] * (n - 1)] * B)
    tokens = g.integers(0, V, (B, n))
    u, want, deep = np.zeros((B, n), dtype=np.float32), [], 0
    for b in range(B):
        tokens[b, 1] = int((q[b, 0] - p[b, 0]).argmax())
        P, Q = _exact_rows(p[b]), _exact_rows(q[b])
        left = sum(max(x - y, Fraction(0)) for x, y in zip(P[0], Q[0]))
        assert 0 < left < Fraction(1, 1 << 16)
        while True:
            u[b] = g.random(n).astype(np.float32)
            u[b, 1] = 1 - 2.0 ** -24
            path, token, near = _walk(P, Q, tokens[b].tolist(), parent[b].tolist(), u[b].tolist(), n)
            if near > 2.0 ** -30:
                break
        deep += len(path) == 1 or path[1] > 2
        want.append((path + [-1] * (n - len(path)), len(path), token))
    assert deep >= B // 4  # two rejections and more
    path, count, token = lib.verify_tree(p.cuda(), _int(tokens), _int(parent), torch.tensor(u, device="cuda"), q=q.cuda())
    assert path.tolist() == [w[0] for w in want] and count.tolist() == [w[1] for w in want]
    assert token.tolist() == [w[2] for w in want]


def _split(x):
    """The whole number x (steps of 2^-50) as fp32 values that add up to it: 24 bits each."""
    out = []
    while x:
        top = x >> max(x.bit_length() - 24, 0) << max(x.bit_length() - 24, 0)
        out.append(top * 2.0 ** -50)
        x -= top
    return out


@pytest.mark.parametrize("V", [40, 100003])
def test_verify_thresholds_to_the_last_step(lib, V):
    """Prefix sums at u R itself, one step of 2^-50 below and above it: u R has 74 bits, of which none is rounded."""
    g = _rng(20, V)
    rows, us, want = [], [], []
    ends = [1 - 2.0 ** -24, 2.0 ** -24, 0.5, 2.0 ** -50, 2.0 ** -60, 2.0 ** -149, 0.75, 1 - 3 * 2.0 ** -24]
    for i in range(64):
        u = float(np.float32(ends[i] if i < len(ends) else g.random()))
        total = (1 << 50) + (1, 0, -1, int(g.integers(-(1 << 30), 1 << 30)))[i % 4]
        at = Fraction(u) * total
        edge = at.numerator // at.denominator + (0, 1, 2)[i % 3]  # the first tokens' sum: at u R or below it, just above it, beyond
        first = _split(edge)
        rest = _split(total - edge)
        row = np.zeros(V, dtype=np.float32)
        row[:len(first)] = first
        row[V - len(rest):] = rest
        exact = [Fraction(float(x)) for x in np.concatenate([row[:20], row[V - 20:]])]  # (zeros between)
        assert sum(exact) == Fraction(total, 1 << 50) and len(first) < 20 and len(rest) < 20
        exact = [min(x, Fraction(1)) for x in exact]  # (as the definition has it: of a total above 1 the first entry may be)
        cum, token = Fraction(0), None
        for t, x in enumerate(exact):
            cum += x
            if token is None and cum > Fraction(u) * sum(exact):
                token = t if t < 20 else V - 40 + t
        rows.append(row)
        us.append(u)
        want.append(token)
    p = torch.tensor(np.stack(rows)[:, None], device="cuda")
    u = torch.tensor(us, dtype=torch.float32, device="cuda")[:, None]
    zero = _int(np.zeros((64, 1)))
    assert lib.verify_tree(p, zero, zero - 1, u)[2].tolist() == want
    for b in (0, 1, 5):  # alone: other clusters
        assert lib.verify_tree(p[b:b + 1], zero[:1], zero[:1] - 1, u[b:b + 1])[2].tolist() == want[b:b + 1]


def test_verify_rows_that_are_no_distributions(lib):
    """Sums past 64 bits and others: some token of the vocabulary, or -1."""
    for x, V in ((1.0, 1 << 17), (3.0, 20000), (0.01, 50000), (float("inf"), 1000)):
        p = torch.full((2, 3, V), x, device="cuda")
        u = torch.full((2, 3), 0.7, device="cuda")
        path, count, token = lib.verify_tree(p, _int([[0, 1, 2]] * 2), _int([[-1, 0, 1]] * 2), u, q=p)
        assert all(-1 <= t < V for t in token.tolist()) and all(1 <= c <= 3 for c in count.tolist())


def test_verify_bad_nodes_are_never_accepted(lib):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    p = torch.full((1, 5, 4), 0.25, device="cuda")
    u = torch.zeros((1, 5), device="cuda")
    path, count, token = lib.verify_tree(p, _int([[0, 9, -1, 2, 1]]), _int([[-1, 0, 0, 3, 0]]), u, err=err)
    assert path.tolist() == [[0, 4, -1, -1, -1]] and lib.check_error(err) == 1
    # what lies past the nodes in use is not looked at
    path, count, token = lib.verify_tree(p, _int([[0, 1, -1, 2, 1]]), _int([[-1, 0, 7, 3, 0]]), u, n_tok=_int([2]), err=err)
    assert path.tolist() == [[0, 1, -1, -1, -1]] and lib.check_error(err) == 0


def test_verify_strided_rows_and_unused_rows(lib):
    """Rows at a stride, an odd start; rows of q that no test needs may hold anything."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    B, n, V = 4, 3, 1001
    big = torch.softmax(torch.randn((B, n, V + 30), generator=gen, device="cuda"), -1)
    p = big[:, :, 7:7 + V]
    q = torch.softmax(torch.randn((B, n, V), generator=gen, device="cuda"), -1)
    q[:, 2] = float("nan")
    parent, u = _int([[-1, 0, 1]] * B), torch.rand((B, n), generator=gen, device="cuda")
    tokens = torch.randint(0, V, (B, n), generator=gen, device="cuda", dtype=torch.int32)
    a = lib.verify_tree(p, tokens, parent, u, q=q)
    b = lib.verify_tree(p.contiguous(), tokens, parent, u, q=q)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("proposal", [True, False])
def test_verified_tokens_follow_the_target(lib, proposal):
    """The first token that comes out (accepted, or sampled in place of a rejected one) is distributed as the target's first row:
    40000 trees of three children; each frequency within 5 standard deviations."""
    g = _rng(6, proposal)
    B, V = 40000, 6
    p1, q1 = np.array([0.05, 0.3, 0.1, 0.25, 0.1, 0.2]), np.array([0.3, 0.05, 0.3, 0.1, 0.15, 0.1])
    p = torch.tensor(p1, dtype=torch.float32, device="cuda").expand(B, 4, V).contiguous()
    q = torch.tensor(q1, dtype=torch.float32, device="cuda").expand(B, 4, V).contiguous()
    tokens = g.choice(V, size=(B, 4), p=q1) if proposal else np.tile([0, 2, 0, 4], (B, 1))
    u = torch.tensor(g.random((B, 4)), dtype=torch.float32, device="cuda")
    path, count, token = lib.verify_tree(p, _int(tokens), _int([[-1, 0, 0, 0]] * B), u, q=q if proposal else None)
    path, count, token = path.cpu().numpy(), count.cpu().numpy(), token.cpu().numpy()
    first = np.where(count > 1, tokens[np.arange(B), path[:, 1]], token)
    freq = np.bincount(first, minlength=V) / B
    assert np.all(np.abs(freq - p1) < 5 * np.sqrt(p1 * (1 - p1) / B))


def test_verify_in_a_graph_and_on_another_stream(lib):
    gen = torch.Generator(device="cuda").manual_seed(8)
    B, n, V = 5, 4, 20000
    p, q = (torch.softmax(torch.randn((B, n, V), generator=gen, device="cuda"), -1) for _ in range(2))
    tokens = torch.randint(0, V, (B, n), generator=gen, device="cuda", dtype=torch.int32)
    parent, u = _int([[-1, 0, 0, 1]] * B), torch.rand((B, n), generator=gen, device="cuda")
    want = lib.verify_tree(p, tokens, parent, u, q=q)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            got = lib.verify_tree(p, tokens, parent, u, q=q)
        for _ in range(3):
            graph.replay()
    stream.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.parametrize("B,V", [(1, 131072), (3, 131072), (40, 50001)])
def test_verify_beside_other_work(lib, B, V):
    """Clusters whose CTAs find the SMs taken by another stream's kernels and start when these let them: the same results."""
    gen = torch.Generator(device="cuda").manual_seed(V + B)
    n = 4
    p, q = (torch.softmax(2 * torch.randn((B, n, V), generator=gen, device="cuda"), -1) for _ in range(2))
    tokens = torch.multinomial(q.flatten(0, 1)[::n].repeat_interleave(n, 0), 1, generator=gen).view(B, n).int()
    parent, u = _int([[-1, 0, 0, 0]] * B), torch.rand((B, n), generator=gen, device="cuda")
    want = lib.verify_tree(p, tokens, parent, u, q=q)
    x = torch.randn((4096, 4096), generator=gen, device="cuda").bfloat16()
    other, mine = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        with torch.cuda.stream(other):
            for _ in range(4):
                y = x @ x
        with torch.cuda.stream(mine):
            got = [lib.verify_tree(p, tokens, parent, u, q=q) for _ in range(4)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for g in got for a, b in zip(g, want))
    del y


@pytest.mark.parametrize("B,n,V", [(1, 3, 131070), (2, 40, 150001), (4, 3, 131073)])
def test_verify_first_call_of_a_size_in_a_graph(lib, B, n, V):
    """Clusters of 16, whose place on the device is asked for while a graph is captured."""
    gen = torch.Generator(device="cuda").manual_seed(V)
    p, q = (torch.softmax(2 * torch.randn((B, n, V), generator=gen, device="cuda"), -1) for _ in range(2))
    tokens = torch.randint(0, V, (B, n), generator=gen, device="cuda", dtype=torch.int32)
    parent, u = _int([[-1] + [0] * (n - 1)] * B), torch.rand((B, n), generator=gen, device="cuda")
    lib.verify_tree(p[:, :, :64].contiguous(), tokens % 64, parent, u)  # (the library is loaded)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = lib.verify_tree(p, tokens, parent, u, q=q)
    graph.replay()
    torch.cuda.synchronize()
    want = lib.verify_tree(p, tokens, parent, u, q=q)
    assert all(torch.equal(x, y) for x, y in zip(got, want)) and bool((got[1] >= 1).all())


def test_refusals(lib):
    pool = lib.PagePool(4, 16, 2, 4)
    a = _int([0, 0])
    for kw in (dict(), dict(n=2, tokens=3), dict(n=0), dict(tokens=4, path=_int([[0, 0], [0, 0]])), dict(n=2, path=_int([0]))):
        with pytest.raises(ValueError):
            lib.kv_plan(pool, a, a, **kw)
    with pytest.raises(ValueError):
        lib.kv_plan(pool, _int([0]), a, n=1)
    with pytest.raises(ValueError):
        lib.kv_plan(pool, a, a.long(), n=1)
    pool.page = 24
    with pytest.raises(lib.TQError):
        lib.kv_plan(pool, a, a, n=1)
    p, u, t = torch.zeros((1, 2, 8), device="cuda"), torch.zeros((1, 2), device="cuda"), _int([[0, 0]])
    with pytest.raises(ValueError):
        lib.verify_tree(p, t, t, u, q=p.half())
    with pytest.raises(ValueError):
        lib.verify_tree(p, t, t, u.double())
    with pytest.raises(ValueError):
        lib.verify_tree(p.transpose(1, 2), t, t, u)
    for x in (p[:, :1].expand(1, 2, 8), torch.zeros((1, 1, 8), device="cuda").expand(3, 1, 8)):  # rows that lie on one another
        with pytest.raises(ValueError):
            lib.verify_tree(x, _int([[0, 0]] if len(x) == 1 else [[0]] * 3), _int([[0, 0]] if len(x) == 1 else [[0]] * 3),
                            torch.zeros(x.shape[:2], device="cuda"))
    with pytest.raises(lib.TQError):
        big = torch.zeros((1, 1025, 8), device="cuda")
        lib.verify_tree(big, _int(np.zeros((1, 1025))), _int(np.zeros((1, 1025))), torch.zeros((1, 1025), device="cuda"))
