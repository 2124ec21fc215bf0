"""The block tables and slot maps of a paged cache against a sequential
statement of their rules: ragged requests, no room, bad lengths, empty steps,
release, and a run of steps that keeps every page owned once."""
import numpy as np
import pytest

from bitwise_reproducible_fp32_gb300 import detlib
from gpu_util import host, need_gpu, torch

pytestmark = pytest.mark.gpu
I = np.int32


@pytest.fixture(scope="module")
def dev():
    return need_gpu()


def on_gpu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def extend_plain(lens, new, table, free, count, ps, max_rows):
    """The rules one request at a time."""
    table, status, row, taken = table.copy(), 0, 0, 0
    B, width = table.shape
    if count < 0 or count > len(free):
        count, status = 0, 1
    lens_out, starts = lens.copy(), np.zeros(B + 1, I)
    pos, slots = np.full(max_rows, -1, I), np.full(max_rows, -1, np.int64)
    out_of_pages = False
    for b in range(B):
        n0, add = int(lens[b]), int(new[b])
        starts[b] = min(row, max_rows)
        if n0 < 0 or add < 0 or n0 + add > min(width * ps, 2 ** 31 - 1):
            status |= 1
            continue
        first, row = row, row + add
        if row > max_rows:
            status |= 4
            continue
        need = -(-(n0 + add) // ps) - -(-n0 // ps)
        if need and (out_of_pages or taken + need > count):
            out_of_pages = True
            status |= 2
            continue
        for i in range(need):
            table[b, -(-n0 // ps) + i] = free[count - 1 - taken - i]
        taken += need
        lens_out[b] = n0 + add
        for i in range(add):
            pos[first + i] = n0 + i
            page = table[b, (n0 + i) // ps]
            slots[first + i] = int(page) * ps + (n0 + i) % ps if page >= 0 else -1
    starts[B] = min(row, max_rows)
    return lens_out, count - taken, starts, pos, slots, table, status


def release_plain(lens, done, table, free, count, ps):
    free, lens_out, status, full, given = free.copy(), lens.copy(), 0, False, 0
    if count < 0 or count > len(free):
        count, status = 0, 1
    for b in range(len(lens)):
        if not done[b]:
            continue
        if lens[b] < 0 or lens[b] > table.shape[1] * ps:
            status |= 1
            continue
        n = -(-int(lens[b]) // ps)
        if full or count + given + n > len(free):
            full = True
            status |= 2
            continue
        free[count + given:count + given + n] = table[b, :n]
        given += n
        lens_out[b] = 0
    return lens_out, count + given, free, status


def run_extend(lens, new, table, free, count, ps, max_rows):
    want = extend_plain(lens, new, table, free, count, ps, max_rows)
    td, fd = on_gpu(table), on_gpu(free)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lo, co, st, po, sl = detlib.detpages_extend(on_gpu(lens), on_gpu(new), td, fd,
                                                on_gpu(np.array([count], I)), ps, max_rows,
                                                dev_status=status)
    for got, w, name in zip((host(lo), int(co), host(st), host(po), host(sl), host(td),
                             int(status)), want,
                            ("lens", "count", "row_start", "positions", "slots", "table",
                             "status")):
        assert np.array_equal(got, w), (name, got, w)
    assert np.array_equal(host(fd), free)
    return want


def state(B, ps, longest, width, rng, spare=None):
    lens = rng.integers(0, longest + 1, B).astype(I)
    owned = -(-lens // ps)
    total = int(owned.sum()) + (spare if spare is not None else B * width)
    perm = rng.permutation(total).astype(I)
    table = np.full((B, width), -1, I)
    at = 0
    for b in range(B):
        table[b, :owned[b]] = perm[at:at + owned[b]]
        at += owned[b]
    free = np.full(total, -9, I)
    free[:total - at] = perm[at:]
    return lens, table, free, total - at


@pytest.mark.parametrize("B", [1, 2, 31, 256, 1024, 1025, 5000, 8192])
@pytest.mark.parametrize("ps,most", [(1, 1), (16, 1), (16, 40), (7, 9), (64, 300)])
def test_extend(dev, B, ps, most):
    rng = np.random.default_rng(B * ps + most)
    longest = 100
    width = -(-(longest + most) // ps)
    lens, table, free, count = state(B, ps, longest, width, rng)
    new = rng.integers(0, most + 1, B).astype(I)
    want = run_extend(lens, new, table, free, count, ps, int(new.sum()) + 5)
    assert want[-1] == 0
    # no room for some of the pages, then of the rows
    run_extend(lens, new, table, free, count // 9, ps, int(new.sum()))
    run_extend(lens, new, table, free, count, ps, int(new.sum()) * 2 // 3)
    run_extend(lens, new, table, free, 0, ps, int(new.sum()))


def test_extend_refusals_on_the_device(dev):
    rng = np.random.default_rng(3)
    lens, table, free, count = state(40, 8, 50, 10, rng)
    new = rng.integers(0, 20, 40).astype(I)
    lens[3], new[5], new[7], lens[9], new[9] = -1, -2, 2 ** 31 - 1, 2 ** 31 - 1, 1
    run_extend(lens, new, table, free, count, 8, 400)
    run_extend(lens, new, table, free, -1, 8, 400)
    run_extend(lens, new, table, free, len(free) + 1, 8, 400)
    run_extend(lens, np.full(40, 2 ** 31 - 1, I), table, free, count, 8, 0)
    table[11] = -5                              # a table that lost its pages
    run_extend(lens, new, table, free, count, 8, 400)
    # nothing to do: no requests, no rows
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    lo, co, st, po, sl = detlib.detpages_extend(
        e, e, torch.empty((0, 4), dtype=torch.int32, device="cuda"), on_gpu(free),
        on_gpu(np.array([count], I)), 8, 3)
    assert int(co) == count and host(st).tolist() == [0] and host(po).tolist() == [-1] * 3


@pytest.mark.parametrize("B", [1, 33, 2000, 8192])
@pytest.mark.parametrize("ps", [1, 16])
def test_release(dev, B, ps):
    rng = np.random.default_rng(B + ps)
    lens, table, free, count = state(B, ps, 60, -(-60 // ps), rng, spare=7)
    lens[B // 2] = -1 if B > 1 else lens[0]
    for done in (rng.integers(0, 2, B).astype(I), np.ones(B, I), np.zeros(B, I)):
        for cap in (len(free), count + (len(free) - count) // 3):
            want = release_plain(lens, done, table, free[:cap], count, ps)
            fd = on_gpu(free[:cap])
            status = torch.zeros(1, dtype=torch.int32, device="cuda")
            lo, co = detlib.detpages_release(on_gpu(lens), on_gpu(done), on_gpu(table), fd,
                                             on_gpu(np.array([count], I)), ps,
                                             dev_status=status)
            assert np.array_equal(host(lo), want[0]) and int(co) == want[1]
            assert np.array_equal(host(fd), want[2]) and int(status) == want[3]


def test_a_run_of_steps_keeps_every_page_owned_once(dev):
    rng = np.random.default_rng(8)
    B, ps, width = 50, 4, 12
    total = 300
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    free = on_gpu(rng.permutation(total).astype(I))
    count = torch.tensor([total], dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for step in range(60):
        new = on_gpu(rng.integers(0, 4, B).astype(I))
        lens, count, _, _, slots = detlib.detpages_extend(lens, new, table, free, count, ps, 200,
                                                          dev_status=status)
        live = host(slots)
        live = live[live >= 0]
        assert len(set(live.tolist())) == len(live)
        done = on_gpu((rng.random(B) < 0.1).astype(I))
        lens, count = detlib.detpages_release(lens, done, table, free, count, ps,
                                              dev_status=status)
        h, t, f, c = host(lens), host(table), host(free), int(count)
        owned = np.concatenate([t[b, :-(-int(h[b]) // ps)] for b in range(B)] + [f[:c]])
        assert sorted(owned.tolist()) == list(range(total)), step
    assert int(status) & ~3 == 0
