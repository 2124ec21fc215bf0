"""Rows that share pages, forked, freed and compacted, against sequential statements
of the rules; copies of pages in every layout; bad lengths, parents, pages and
counts; a run of steps that keeps every page either free or in a row."""
import numpy as np
import pytest

from bitwise_reproducible_fp32_gb300 import detlib
from gen_util import LAYOUTS, make_cache
from gpu_util import host, need_gpu, torch

pytestmark = pytest.mark.gpu
F, I = np.float32, np.int32


@pytest.fixture(scope="module")
def dev():
    return need_gpu()


def on_gpu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def rows(groups, W, ps, prefix, mine, rng, spare=20):
    """Groups of W rows that share the full pages of a prefix: (lens, table, free list,
    its count, pages)."""
    lens = np.zeros(groups * W, I)
    width = max(1, -(-(prefix + mine) // ps))
    ids = rng.permutation(groups * (prefix // ps) + groups * W * (-(-mine // ps) + 2) + spare)
    table, at = np.full((groups * W, width), -1, I), 0
    for g in range(groups):
        p = int(rng.integers(0, prefix + 1))
        shared = ids[at:at + p // ps]
        at += p // ps
        for w in range(W):
            r = g * W + w
            lens[r] = p + rng.integers(0, mine + 1)
            n = -(-int(lens[r]) // ps) - len(shared)
            table[r, :len(shared)] = shared
            table[r, len(shared):len(shared) + n] = ids[at:at + n]
            at += n
    free = np.full(len(ids), -9, I)
    free[:len(ids) - at] = ids[at:]
    return lens, table, free, len(ids) - at, len(ids)


def fork_plain(lens, parents, table, free, count, ps, pages, table_out):
    B, width = table.shape
    room = min(width * ps, 2 ** 31 - 1)
    status, free, out = 0, free.copy(), table_out.copy()
    if count < 0 or count > len(free):
        count, status = 0, 1
    n = [-(-int(x) // ps) if 0 <= x <= room else 0 for x in lens]
    if any(x < 0 or x > room for x in lens):
        status |= 1
    child = {}
    for r, p in enumerate(parents):
        if 0 <= p < B:
            child.setdefault(int(p), r)
        elif p != -1:
            status |= 1
    held = {k: set() for k in (True, False)}
    for b in range(B):
        for i in table[b, :n[b]]:
            if 0 <= i < pages:
                held[b in child].add(int(i))
            else:
                status |= 4
    back = sorted(held[False] - held[True])
    if count + len(back) > len(free):
        back, status = [], status | 1
    free[count:count + len(back)] = back
    count += len(back)
    new = len(parents)
    l_out, src, dst, tok = np.zeros(new, I), np.full(new, -1, I), np.full(new, -1, I), np.zeros(new, I)
    for r, p in enumerate(parents):
        if not 0 <= p < B or n[p] == 0:
            continue
        row, own = table[p, :n[p]].copy(), None
        if lens[p] % ps and child[int(p)] != r and 0 <= row[-1] < pages:
            if count == 0:
                status |= 2
                continue
            count -= 1
            own = free[count]
            if not 0 <= own < pages:
                status |= 4
                continue
            src[r], dst[r], tok[r] = row[-1], own, lens[p] % ps
            row[-1] = own
        out[r, :n[p]], l_out[r] = row, lens[p]
    return out, l_out, count, src, dst, tok, free, status


def run_fork(lens, parents, table, free, count, ps, pages, ld=0):
    new = len(parents)
    before = np.full((new, table.shape[1]), -5, I)
    want = fork_plain(lens, parents, table, free, count, ps, pages, before)
    wide = torch.full((new, table.shape[1] + ld), -5, dtype=torch.int32, device="cuda")
    td, fd = on_gpu(table), on_gpu(free)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = detlib.detpages_fork(on_gpu(lens), on_gpu(parents), td, fd, on_gpu(np.array([count], I)),
                               ps, pages, table_out=wide[:, :table.shape[1]], dev_status=status)
    for g, w, name in zip((*map(host, got), host(fd), int(status)), want,
                          ("table", "lens", "count", "src", "dst", "tokens", "free", "status")):
        assert np.array_equal(g, w) or (name == "count" and int(g[0]) == w), (name, g, w)
    assert np.array_equal(host(td), table) and (host(wide)[:, table.shape[1]:] == -5).all()
    return want


@pytest.mark.parametrize("groups,W", [(1, 1), (1, 4), (16, 4), (300, 3), (1024, 8)])
@pytest.mark.parametrize("ps,prefix,mine", [(1, 5, 3), (16, 200, 40), (7, 0, 30), (64, 5000, 10),
                                            (16, 64, 0)])
def test_fork(dev, groups, W, ps, prefix, mine):
    rng = np.random.default_rng(groups * 100 + W + ps)
    lens, table, free, count, pages = rows(groups, W, ps, prefix, mine, rng, spare=groups * W)
    B = groups * W
    beams = rng.integers(0, W, B) + np.repeat(np.arange(groups) * W, W)
    beams = np.where(rng.random(B) < 0.1, -1, beams).astype(I)
    for parents in (beams, np.arange(B, dtype=I), np.full(B, -1, I), rng.permutation(B).astype(I),
                    np.zeros(min(2 * B, 8192), I), beams[:B // 2]):
        want = run_fork(lens, parents, table, free, count, ps, pages, ld=3)
    # nothing free but what is given back, then nothing
    run_fork(lens, beams, table, free, 0, ps, pages)
    run_fork(lens, np.zeros(B, I), table, free[:count], count, ps, pages)
    assert want[-1] in (0, 1)


def test_fork_out_of_order(dev):
    rng = np.random.default_rng(2)
    lens, table, free, count, pages = rows(8, 4, 16, 100, 60, rng)
    parents = rng.integers(0, 32, 32).astype(I)
    for bad in (dict(count=-1), dict(count=len(free) + 1), dict(free=free[:count + 1])):
        run_fork(**{**dict(lens=lens, parents=parents, table=table, free=free, count=count, ps=16,
                           pages=pages), **bad})
    lens[3], lens[7], lens[11] = -1, 2 ** 31 - 1, 16 * table.shape[1] + 1
    parents[:5] = [-2, 32, 2 ** 31 - 1, 3, 7]
    run_fork(lens, parents, table, free, count, 16, pages)
    table[12, 0], table[13, -(-int(lens[13]) // 16) - 1] = -1, pages
    parents[20:26] = [12, 12, 13, 13, 13, -2 ** 31]
    run_fork(lens, parents, table, free, count, 16, pages)
    free[:count] = -3                        # a free list that lost its pages
    run_fork(lens, parents, table, free, count, 16, pages)
    run_fork(lens, parents, table, free, count, 16, pages // 3)
    e = np.zeros(0, I)
    run_fork(e, np.array([-1, 0], I), table[:0], free, count, 16, pages)
    run_fork(lens, e, table, free, count, 16, pages)


def test_fork_of_a_large_pool(dev):
    # more pages than one CTA marks, ids up to the limit
    rng = np.random.default_rng(3)
    pages = 1 << 23
    lens = np.array([70_000 * 16, 70_000 * 16 - 5, 33, 0], I)
    table = np.full((4, 70_000), -1, I)
    ids = rng.choice(pages, 140_003, replace=False).astype(I)
    ids[0] = pages - 1
    table[0], table[1], table[2, :3] = ids[:70_000], ids[70_000:140_000], ids[140_000:]
    free = np.full(pages, -9, I)
    for parents in ([1, 1, 2], [0, 0, -1], [3, 3]):
        run_fork(lens, np.array(parents, I), table, free, 0, 16, pages)


def compact_plain(lens, table, ps, pages, table_out, half):
    width = table.shape[1]
    room = min(width * ps, 2 ** 31 - 1)
    status, out = 0, table_out.copy()
    n = [-(-int(x) // ps) if 0 <= x <= room else 0 for x in lens]
    if any(x < 0 or x > room for x in lens):
        status |= 1
    held = np.zeros(pages, bool)
    for b in range(len(lens)):
        row = table[b, :n[b]]
        ok = (row >= 0) & (row < pages)
        status |= 0 if ok.all() else 4
        held[row[ok]] = True
    U = int(held.sum())
    src = np.flatnonzero(held & (np.arange(pages) >= U))
    dst = np.flatnonzero(~held & (np.arange(pages) < U))
    to = np.arange(pages)
    to[src] = dst
    for b in range(len(lens)):
        row = table[b, :n[b]]
        ok = (row >= 0) & (row < pages)
        out[b, :n[b]] = np.where(ok, to[np.where(ok, row, 0)] if pages else row, row)
    free = np.full(pages, -5, I)
    free[:pages - U] = np.arange(pages - 1, U - 1, -1)
    s, d = np.full(half, -5, I), np.full(half, -5, I)
    s[:len(src)], d[:len(src)] = src, dst
    return out, pages - U, len(src), s, d, free, status


def run_compact(lens, table, ps, pages, in_place=False):
    before = table if in_place else np.full(table.shape, -5, I)
    half = pages // 2
    want = compact_plain(lens, table, ps, pages, before, half)
    td = on_gpu(table)
    i = lambda n: torch.full((n,), -5, dtype=torch.int32, device="cuda")     # noqa: E731
    free, status = i(pages), torch.zeros(1, dtype=torch.int32, device="cuda")
    got = detlib.detpages_compact(on_gpu(lens), td, free, ps,
                                  table_out=td if in_place else on_gpu(before), src=i(half),
                                  dst=i(half), dev_status=status)
    out, count, moves, src, dst = got
    for g, w, name in zip((host(out), int(count), int(moves), host(src), host(dst), host(free),
                           int(status)), want,
                          ("table", "count", "moves", "src", "dst", "free", "status")):
        assert np.array_equal(g, w), (name, g, w)
    return want


@pytest.mark.parametrize("groups,W,ps,prefix,mine", [(1, 1, 16, 3, 2), (16, 4, 16, 200, 40),
                                                     (200, 8, 1, 30, 9), (1024, 8, 16, 500, 100),
                                                     (3, 2, 64, 0, 0)])
def test_compact(dev, groups, W, ps, prefix, mine):
    rng = np.random.default_rng(groups + ps)
    lens, table, _, _, pages = rows(groups, W, ps, prefix, mine, rng, spare=40)
    for alive in (1.0, 0.5, 0.02, 0.0):
        some = np.where(rng.random(len(lens)) < alive, lens, 0).astype(I)
        want = run_compact(some, table, ps, pages)
        run_compact(some, table, ps, pages, in_place=True)
        # a compacted pool stays as it is
        again = run_compact(some, want[0], ps, pages)
        assert again[2] == 0 and again[1] == want[1]


def test_compact_out_of_order(dev):
    rng = np.random.default_rng(4)
    lens, table, _, _, pages = rows(8, 4, 16, 100, 60, rng)
    lens[3], lens[7], table[12, 0], table[13, 0] = -1, 2 ** 31 - 1, -1, pages
    run_compact(lens, table, 16, pages)
    run_compact(lens, table, 16, pages // 3)
    run_compact(lens, table, 16, 1)
    run_compact(lens[:0], table[:0], 16, pages)
    run_compact(lens, table, 16, 1 << 23)


def copy_plain(k, v, src, dst, tokens, n):
    pages, ps = k.shape[:2]
    status, ok = 0, []
    for i in range(n):
        s, d, t = int(src[i]), int(dst[i]), ps if tokens is None else int(tokens[i])
        if s < 0 or d < 0:
            continue
        if s >= pages or d >= pages or not 0 <= t <= ps:
            status |= 1
        elif s != d and t:
            ok.append((s, d, t))
    read = {s for s, _, _ in ok}
    k2, v2 = k.copy(), v.copy()
    last = {d: (s, t) for s, d, t in ok}
    for d, (s, t) in last.items():
        if d in read:
            status |= 2
            continue
        k2[d, :t], v2[d, :t] = k[s, :t], v[s, :t]
    return k2, v2, status


def run_copy(kc, vc, src, dst, tokens=None, count=None):
    n = len(src)
    want = copy_plain(host(kc), host(vc), src, dst, tokens,
                      n if count is None else min(max(count, 0), n))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    detlib.detkv_copy_f32(kc, vc, on_gpu(src), on_gpu(dst),
                          None if tokens is None else on_gpu(tokens),
                          None if count is None else on_gpu(np.array([count], I)),
                          dev_status=status)
    for c, w in ((kc, want[0]), (vc, want[1])):
        assert np.array_equal(host(c).view(I), w.view(I))
    bad = count is not None and not 0 <= count <= n
    assert int(status) == want[2] | bad


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("ps,G,d", [(16, 12, 64), (1, 1, 1), (7, 3, 10), (64, 8, 128), (5, 2, 250), (120, 4, 64),
                                    (300, 2, 16)])
def test_copy(dev, layout, ps, G, d):
    rng = np.random.default_rng(ps + d)
    pages = 60
    kc, vc = make_cache(pages, ps, G, d, layout)
    for c in (kc, vc):
        c.copy_(on_gpu(rng.standard_normal((pages, ps, G, d)).astype(F)))
    ids = rng.permutation(pages).astype(I)
    src, dst = ids[rng.integers(0, 20, 25)], ids[30:55]
    run_copy(kc, vc, src, dst)
    run_copy(kc, vc, src, dst, rng.integers(0, ps + 1, 25).astype(I))
    run_copy(kc, vc, src, dst, count=7)
    run_copy(kc, vc, src, dst, rng.integers(0, ps + 1, 25).astype(I), count=0)
    # destinations twice, as sources, pages to themselves, nothing, out of range
    src, dst = rng.integers(-2, pages + 2, 50).astype(I), rng.integers(-2, pages + 2, 50).astype(I)
    run_copy(kc, vc, src, dst, rng.integers(-1, ps + 2, 50).astype(I))
    run_copy(kc, vc, ids[:25], np.full(25, ids[40], I), rng.integers(0, ps + 1, 25).astype(I))
    run_copy(kc, vc, ids[:2], ids[1:3])
    run_copy(kc, vc, ids[:2], ids[3:5], count=-1)
    run_copy(kc, vc, ids[:2], ids[5:7], count=3)


def test_copy_of_many_pages_past_the_filter(dev):
    # 300,000 small pages: several to a bit of the filter
    rng = np.random.default_rng(5)
    pages = 300_000
    kc, vc = (on_gpu(rng.standard_normal((pages, 2, 1, 4)).astype(F)) for _ in range(2))
    ids = rng.permutation(pages).astype(I)
    run_copy(kc, vc, ids[:5000], ids[100_000:105_000])
    dst = ids[100_000:105_000].copy()
    dst[::50], dst[1::70] = dst[7], ids[3]
    run_copy(kc, vc, ids[:5000], dst)


def test_copy_of_more_than_l2_holds(dev):
    rng = np.random.default_rng(6)
    pages = 330
    kc, vc = (on_gpu(rng.standard_normal((pages, 64, 8, 128)).astype(F)) for _ in range(2))
    ids = rng.permutation(pages).astype(I)
    run_copy(kc, vc, ids[:160], ids[160:320])
    dst = ids[160:320].copy()
    dst[::50], dst[1::70] = dst[7], ids[3]
    run_copy(kc, vc, ids[:160], dst, rng.integers(0, 65, 160).astype(I))


def test_copy_past_32_bit_offsets(dev):
    pages, ps, G, d = 35_000, 64, 8, 128          # 2.3e9 floats each
    kc, vc = (torch.full((pages, ps, G, d), float("nan"), device="cuda") for _ in range(2))
    x = torch.randn((ps, G, d), device="cuda")
    kc[34_999], vc[34_999] = x, -x
    detlib.detkv_copy_f32(kc, vc, on_gpu(np.array([34_999, 34_999], I)),
                          on_gpu(np.array([33_000, 2], I)))
    for p in (33_000, 2):
        assert torch.equal(kc[p], x) and torch.equal(vc[p], -x)
    assert bool(kc[32_999].isnan().all()) and bool(kc[33_001].isnan().all())


def test_binding_refusals(dev):
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")          # noqa: E731
    f, c = detlib.detpages_fork, detlib.detpages_compact
    kc, vc = make_cache(4, 2, 1, 4)
    for call in (lambda: f(i(4), i(5), i(3, 2), i(9), i(1), 16, 9),
                 lambda: f(i(4), i(5), i(4, 2), i(9), i(2), 16, 9),
                 lambda: f(i(4), i(5), i(4, 2), i(9), i(1), 16, 9, table_out=i(4, 2)),
                 lambda: f(i(4), i(5), i(4, 2), i(9), i(1), 16, 9, src=i(4)),
                 lambda: c(i(4), i(3, 2), i(9), 16), lambda: c(i(4), i(4, 2), i(9), 16, dst=i(3)),
                 lambda: detlib.detkv_copy_f32(kc, vc, i(3), i(4)),
                 lambda: detlib.detkv_copy_f32(kc, vc, i(3), i(3), tokens=i(2)),
                 lambda: detlib.detkv_copy_f32(kc, vc, i(3), i(3), count=i(2)),
                 lambda: detlib.detkv_copy_f32(kc, vc[:3], i(3), i(3))):
        with pytest.raises(ValueError):
            call()
    t = i(4, 2)
    with pytest.raises(detlib.DetError):
        f(i(4), i(4), t, i(9), i(1), 16, 9, table_out=t)
    with pytest.raises(detlib.DetError):
        c(i(4), t, i(9), 16, src=i(3), dst=i(3))


def test_a_run_of_steps_keeps_every_page_in_a_row_or_free(dev):
    # grow, fork, compact: what the rows read stays what was written for them
    rng = np.random.default_rng(8)
    B, ps, width, pages = 24, 4, 16, 300
    kc, vc = make_cache(pages, ps, 1, 4, fill=0.0)
    lens, table = (torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((B,), (B, width)))
    free = on_gpu(rng.permutation(pages).astype(I))
    count = torch.tensor([pages], dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    story = [[] for _ in range(B)]
    for step in range(40):
        new = rng.integers(0, 4, B).astype(I)
        new = np.minimum(new, width * ps - host(lens))
        lens, count, start, _, slots = detlib.detpages_extend(lens, on_gpu(new), table, free, count,
                                                              ps, 100, dev_status=status)
        at = host(slots)
        for b in range(B):
            for s in at[host(start)[b]:host(start)[b + 1]]:
                x = float(rng.random())
                kc.view(-1, 4)[int(s), 0] = x
                story[b].append(F(x))
        parents = np.where(rng.random(B) < 0.2, -1, rng.integers(0, B, B)).astype(I)
        table, lens, count, src, dst, tokens = detlib.detpages_fork(
            lens, on_gpu(parents), table, free, count, ps, pages, dev_status=status)
        detlib.detkv_copy_f32(kc, vc, src, dst, tokens, dev_status=status)
        story = [list(story[p]) if p >= 0 else [] for p in parents]
        if step % 3 == 2:
            table, count, moves, src, dst = detlib.detpages_compact(lens, table, free, ps,
                                                                    dev_status=status)
            detlib.detkv_copy_f32(kc, vc, src, dst, count=moves, dev_status=status)
        h, t, f, c = host(lens), host(table), host(free), int(count)
        held = [t[b, :-(-int(h[b]) // ps)] for b in range(B)]
        full = [i for b in range(B) for i in held[b][:int(h[b]) // ps]]
        part = [held[b][-1] for b in range(B) if h[b] % ps]
        assert len(set(part)) == len(part) and not set(part) & set(full)
        assert sorted(set(full) | set(part) | set(f[:c].tolist())) == list(range(pages))
        assert len(set(full)) + len(part) + c == pages
        for b in range(B):
            got = host(kc)[held[b]].reshape(-1, 4)[:int(h[b]), 0] if h[b] else []
            assert np.array_equal(got, np.array(story[b], F)), (step, b)
    assert int(status) == 0


def test_captured_and_on_another_stream(dev):
    rng = np.random.default_rng(9)
    lens, table, free, count, pages = rows(16, 4, 16, 100, 60, rng, spare=99)
    parents = rng.integers(0, 64, 64).astype(I)
    want = fork_plain(lens, parents, table, free, count, 16, pages, np.full_like(table, -5))
    ld, pd, td, fd, cd = (on_gpu(a) for a in (lens, np.zeros_like(parents), table, free,
                                              np.array([count], I)))
    out = torch.full_like(td, -5)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    detlib.detpages_fork(ld, pd, td, fd, cd, 16, pages, table_out=out, stream=s)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = detlib.detpages_fork(ld, pd, td, fd, cd, 16, pages, table_out=out)
        comp = detlib.detpages_compact(ld, td, fd.clone(), 16)
    pd.copy_(on_gpu(parents))
    fd.copy_(on_gpu(free))
    out.fill_(-5)
    g.replay()
    for a, w in zip(got, want):
        assert np.array_equal(host(a), w) or int(host(a)[0]) == w
    assert int(comp[2]) == compact_plain(lens, table, 16, pages, table, pages // 2)[2]
