"""GPU parity (0 ULP) of the attention of requests that share a prefix with decode
attention over the same tables (and through it, and directly, with the oracle and 64
bits): groups and rows of every tile's size, prefixes around the chunks, page sizes
that end inside them, layouts, shared heads, requests that share nothing, empty and
bad ones, infinities and NaN, graphs, streams and threads."""
import threading

import numpy as np
import pytest

from bitcmp import assert_bitwise
from bitwise_reproducible_fp32_gb300 import detlib
from exp_cases import exp_tie_arguments
from gen_util import F, LAYOUTS, decode64, decode_oracle, make_cache
from gpu_util import host, need_gpu, to_dev, torch

pytestmark = pytest.mark.gpu


WIDE = 1 << 20                  # tokens


@pytest.fixture(scope="module")
def dev():
    return need_gpu()


def on_gpu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def shared_cache(prefixes, own, ps, G, d, layout, rng, edit=None):
    """Requests in groups: group g's share the full pages of prefixes[g] tokens, request
    b has own[b] more after them. (k, v, table, lens, per-request K, V)."""
    B, W = len(own), -(-len(own) // len(prefixes))
    pages, lists, Ks, Vs, lens = 0, [], [], [], []
    kinds = [rng.standard_normal((2, p, G, d)).astype(F) for p in prefixes]
    fill, at = [], [None] * len(prefixes)
    for b in range(B):
        g = b // W
        p = prefixes[g]
        mine = rng.standard_normal((2, own[b], G, d)).astype(F)
        kv = np.concatenate([kinds[g], mine], axis=1)
        if edit is not None:
            kv = edit(b, kv)
        n = p + own[b]
        full, need = p // ps, -(-n // ps)
        if at[g] is None:
            at[g] = list(range(pages, pages + full))
            pages += full
        row = at[g] + list(range(pages, pages + need - full))
        pages += need - full
        for j, page in enumerate(row):
            fill.append((page, kv[:, j * ps:(j + 1) * ps]))
        lists.append(row)
        Ks.append(kv[0])
        Vs.append(kv[1])
        lens.append(n)
    perm = rng.permutation(pages + 2).astype(np.int32)
    width = max(1, max(map(len, lists)))
    table = np.full((B, width), -7, np.int32)
    for b, row in enumerate(lists):
        table[b, :len(row)] = perm[row]
    kh, vh = (np.full((pages + 2, ps, G, d), np.nan, F) for _ in range(2))
    for page, x in fill:
        kh[perm[page], :x.shape[1]], vh[perm[page], :x.shape[1]] = x
    kc, vc = make_cache(pages + 2, ps, G, d, layout)
    kc.copy_(torch.from_numpy(kh))
    vc.copy_(torch.from_numpy(vh))
    return kc, vc, on_gpu(table), np.array(lens, np.int32), Ks, Vs


def both(q, kc, vc, table, lens, H, group, layout="dense", **kw):
    """The shared attention's output, after its bits and status have been compared with
    decode attention's; also over the same table with room for much longer requests (short
    ones are not worth reading together)."""
    qd, ld = to_dev(q, layout), on_gpu(np.asarray(lens, np.int32))
    s1, s2 = (torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(2))
    want = host(detlib.detdecode_attention_f32(qd, kc, vc, table, ld, H, dev_status=s1, **kw))
    out = torch.full((len(lens), q.shape[1] + 3), 5.0, device="cuda")
    got = host(detlib.detdecode_attention_shared_f32(qd, kc, vc, table, ld, H, group,
                                                     out=out[:, :-3], dev_status=s2, **kw))
    assert_bitwise(got, want, f"group {group}")
    assert int(s1) == int(s2)
    assert bool((out[:, -3:] == 5.0).all())
    cols = WIDE // kc.shape[1]
    if table.shape[1] < cols:
        wide = torch.full((table.shape[0], cols), -7, dtype=torch.int32, device="cuda")
        wide[:, :table.shape[1]] = table
        s2.zero_()
        got = host(detlib.detdecode_attention_shared_f32(qd, kc, vc, wide, ld, H, group,
                                                         out=out[:, :-3], dev_status=s2, **kw))
        assert_bitwise(got, want, f"group {group} of a wide table")
        if not (np.asarray(lens) > table.shape[1] * kc.shape[1]).any():
            assert int(s1) == int(s2)
        assert bool((out[:, -3:] == 5.0).all())
    return got


@pytest.mark.parametrize("H,G,d", [(1, 1, 64), (4, 4, 16), (12, 12, 64), (8, 2, 128), (6, 2, 80),
                                   (16, 1, 64), (24, 2, 32), (3, 3, 7), (2, 1, 1), (10, 5, 36),
                                   (2, 2, 256), (9, 1, 250), (4, 2, 200)])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("ps", [16, 5])
def test_ragged_groups(dev, H, G, d, layout, ps):
    rng = np.random.default_rng(H * 1000 + d + ps)
    prefixes = [700, 513, 300, 20]
    own = rng.integers(0, 300, 15)
    kc, vc, table, lens, Ks, Vs = shared_cache(prefixes, own, ps, G, d, layout, rng)
    q = (2 * rng.standard_normal((15, H * d))).astype(F)
    scale = float(F(1.0 / np.sqrt(d)))
    got = both(q, kc, vc, table, lens, H, 4, "offset" if layout == "offset" else "padded")
    some = [0, 5, 14]
    assert_bitwise(got[some], decode_oracle(q[some], [Ks[b] for b in some], [Vs[b] for b in some],
                                            H, scale))
    for b in some:
        for h in range(H):
            want, bound = decode64(q[b, h * d:(h + 1) * d], Ks[b][:, h // (H // G)],
                                   Vs[b][:, h // (H // G)], scale)
            assert (np.abs(got[b, h * d:(h + 1) * d] - want) <= bound).all(), (b, h)
    # groups that are not the sharing ones
    for group in (2, 3, 15, 1000):
        both(q, kc, vc, table, lens, H, group)


@pytest.mark.parametrize("group,per", [(2, 1), (2, 2), (5, 1), (4, 2), (3, 4), (16, 1), (17, 1),
                                       (4, 8), (33, 1), (64, 1), (9, 7), (65, 1), (20, 8),
                                       (130, 1)])
@pytest.mark.parametrize("d", [16, 64, 128, 256])
def test_rows_of_every_tile(dev, group, per, d):
    rng = np.random.default_rng(group * 10 + per + d)
    own = rng.integers(1, 40, group + 1)            # a last group of one
    kc, vc, table, lens, _, _ = shared_cache([600, 600], own, 16, 2, d, "token", rng)
    # as one cache of two lists of groups: the second prefix is another
    q = (2 * rng.standard_normal((group + 1, 2 * per * d))).astype(F)
    both(q, kc, vc, table, lens, 2 * per, -(-(group + 1) // 2))
    kc, vc, table, lens, _, _ = shared_cache([1030], own, 16, 2, d, "token", rng)
    both(q, kc, vc, table, lens, 2 * per, group + 1)
    both(q, kc, vc, table, lens, 2 * per, group)


@pytest.mark.parametrize("prefix", [0, 1, 255, 256, 257, 511, 512, 513, 767, 1024, 1279, 2048, 2303])
@pytest.mark.parametrize("ps", [1, 8, 32, 64, 100, 192, 256, 300, 4096])
def test_prefixes_around_the_chunks(dev, prefix, ps):
    rng = np.random.default_rng(prefix + ps)
    for own in ([1] * 6, [0, 1, 2, 300, 700, 5], [256] * 6):
        if prefix + min(own) == 0:
            continue
        kc, vc, table, lens, _, _ = shared_cache([prefix, prefix], own, ps, 2, 64, "token", rng)
        q = rng.standard_normal((6, 256)).astype(F)
        both(q, kc, vc, table, lens, 4, 3)


@pytest.mark.parametrize("B,H,G,d,prefix,ps", [(3, 2, 2, 64, 20000, 16), (5, 8, 1, 128, 9001, 64),
                                               (64, 12, 12, 64, 3000, 16), (2, 4, 4, 16, 33000, 100),
                                               (48, 32, 8, 128, 2100, 64), (4, 1, 1, 256, 5000, 1),
                                               (2, 1, 1, 64, 70001, 4096)])
def test_long(dev, B, H, G, d, prefix, ps):
    rng = np.random.default_rng(prefix)
    own = rng.integers(1, 700, B)
    kc, vc, table, lens, Ks, Vs = shared_cache([prefix], own, ps, G, d, "token", rng)
    q = (2 * rng.standard_normal((B, H * d))).astype(F)
    got = both(q, kc, vc, table, lens, H, B)
    assert_bitwise(got[:1], decode_oracle(q[:1], Ks[:1], Vs[:1], H, float(F(1.0 / np.sqrt(d)))))


def test_many_groups(dev):
    rng = np.random.default_rng(3)
    for groups, W in ((400, 2), (70, 5), (1000, 3)):
        prefixes = rng.integers(0, 900, groups)
        own = rng.integers(1, 60, groups * W)
        kc, vc, table, lens, _, _ = shared_cache(list(prefixes), own, 16, 1, 32, "token", rng)
        q = rng.standard_normal((groups * W, 64)).astype(F)
        lens[rng.integers(0, len(lens), 30)] = 0
        both(q, kc, vc, table, lens, 2, W)


def test_empty_and_bad_requests_in_a_group(dev):
    rng = np.random.default_rng(24)
    own = [40, 300, 5, 60, 700, 90]
    kc, vc, table, lens, _, _ = shared_cache([600], own, 16, 2, 64, "token", rng)
    q = rng.standard_normal((6, 128)).astype(F)
    both(q, kc, vc, table, lens, 2, 6)
    for at, n in ((0, 0), (3, -1), (5, 16 * table.shape[1] + 1), (2, 1), (2, 256), (2, 257), (2, 514)):
        other = lens.copy()
        other[at] = n
        both(q, kc, vc, table, other, 2, 6)
    both(q, kc, vc, table, [0] * 6, 2, 6)
    both(q, kc, vc, table, [0, 0, 0, 0, 700, 0], 2, 6)
    # pages out of range: in one request's shared part, in everyone's, in an own part
    pages = kc.shape[0]
    for row, col, id in ((1, 3, pages), (1, 0, -1), (slice(None), 20, pages), (slice(None), 0, -1),
                         (4, 60, 10 ** 6), (0, 39, -5)):
        bad = table.clone()
        bad[row, col] = id
        both(q, kc, vc, bad, lens, 2, 6)
    # entries past the lengths are not used
    wide = torch.full((6, 900), 10 ** 6, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = torch.where(table < 0, 10 ** 6, table)
    both(q, kc, vc, wide, lens, 2, 6)


def test_requests_with_the_same_pages_all_through(dev):
    # the same rows several times: every page is shared, the last token's too
    rng = np.random.default_rng(4)
    for n in (1, 256, 257, 512, 800, 1025):
        kc, vc, table, lens, _, _ = shared_cache([0], [n], 16, 2, 64, "token", rng)
        q = rng.standard_normal((5, 256)).astype(F)
        both(q, kc, vc, table.expand(5, -1).contiguous(), [n] * 5, 4, 5)
        both(q, kc, vc, table.expand(5, -1).contiguous(), [n, n // 2, n, 1, n], 4, 5)


def test_infinities_and_nan(dev):
    rng = np.random.default_rng(23)
    H = G = 3

    def edit(b, kv):
        K, V = kv = kv.copy()
        if kind == 0:
            K[5, 0, 3] = np.nan
        if kind == 1:
            K[6, 1, :] = np.inf
        if kind == 2:
            V[599, 2, 1] = np.inf
        if kind == 3:
            V[300, 0, 7] = np.nan
        if kind == 4:
            K *= F(1e30)
        if kind == 5 and b == 1:
            K[-1, 1, :] = np.inf
        if kind == 6 and b == 2:
            K[-3, 0, 0] = np.nan
        if kind == 7:
            K[:, :, :] = 0.0
            K[-1, :, 0] = -1000.0
        if kind == 8:
            K[:600] = -np.inf
        return kv

    for kind in range(9):
        kc, vc, table, lens, Ks, Vs = shared_cache([600], [40, 90, 300, 7], 16, G, 64, "token", rng,
                                                   edit)
        q = rng.standard_normal((4, H * 64)).astype(F)
        got = both(q, kc, vc, table, lens, H, 4)
        with np.errstate(all="ignore"):
            assert_bitwise(got, decode_oracle(q, Ks, Vs, H, 0.125))


@pytest.mark.parametrize("B,H", [(2, 1), (3, 2), (20, 1)])
def test_exps_at_the_ties_of_their_rounding(dev, B, H):
    ties, w, n = exp_tie_arguments(-127, 0), 128, 600
    rng = np.random.default_rng(H)
    for r in range(0, len(ties), w):
        part = ties[r:r + w]
        K, V = np.zeros((n, 1, w), F), np.zeros((n, 1, w), F)
        K[1:, :, 0] = -F(200.0)
        at = 1 + rng.permutation(n - 1)[:len(part)]
        K[at, :, 0] = part[:, None]
        V[at, :, np.arange(len(part))] = 1.0
        kc, vc, table, lens, Ks, Vs = shared_cache([0], [n], 16, 1, w, "token", rng,
                                                   lambda b, kv: np.stack([K, V]))
        q = np.zeros((B, H * w), F)
        q[:, ::w] = 1.0
        got = both(q, kc, vc, table.expand(B, -1).contiguous(), [n] * B, H, B, scale=1.0)
        assert_bitwise(got, decode_oracle(q, Ks * B, Vs * B, H, 1.0))


def test_cache_past_32_bit_offsets(dev):
    G, d, ps = 8, 128, 64
    pages = 35_000                      # 2.3e9 floats each
    kc, vc = (torch.full((pages, ps, G, d), float("nan"), device="cuda") for _ in range(2))
    ids = torch.tensor([pages - 1, 34_000, 32_768, 1, 16_384, 33_333], device="cuda")
    for c in (kc, vc):
        c[ids] = torch.randn((6, ps, G, d), device="cuda")
    table = ids.int().expand(3, -1).contiguous()
    table[1, 5], table[2, 5] = 34_000, 2
    kc[2], vc[2] = kc[1], vc[1]
    q = np.random.default_rng(25).standard_normal((3, 2 * G * d)).astype(F)
    both(q, kc, vc, table, [330, 384, 321], 2 * G, 3)
    del kc, vc
    torch.cuda.empty_cache()


def test_heads_in_rounds_of_the_workspace(dev):
    # a table so wide that one round of heads does not hold the scores of all
    rng = np.random.default_rng(8)
    kc, vc, table, lens, _, _ = shared_cache([700], [9, 30], 16, 6, 64, "token", rng)
    wide = torch.full((2, 3_000_000), -1, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    q = rng.standard_normal((2, 12 * 64)).astype(F)
    need = detlib.detdecode_attention_shared_workspace_bytes(2, 2, 12, 6, 64, 48_000_000)
    assert need < 6 << 30
    both(q, kc, vc, wide, lens, 12, 2)


def test_captured_replayed_and_on_another_stream(dev):
    rng = np.random.default_rng(26)
    kc, vc, table, lens, Ks, Vs = shared_cache([600], [500, 33, 90], 16, 4, 64, "token", rng)
    q = rng.standard_normal((3, 256)).astype(F)
    want = decode_oracle(q, Ks, Vs, 4, 0.125)
    s = torch.cuda.Stream()
    qd, ld = to_dev(q), on_gpu(lens)
    s.wait_stream(torch.cuda.current_stream())
    outs = [detlib.detdecode_attention_shared_f32(qd, kc, vc, table, ld, 4, 3, stream=s)
            for _ in range(3)]
    s.synchronize()
    for o in outs:
        assert_bitwise(host(o), want)
    out = torch.empty_like(qd)
    n = detlib.detdecode_attention_shared_workspace_bytes(3, 3, 4, 4, 64, table.shape[1] * 16)
    ws = torch.full(((n + 3) // 4,), float("nan"), device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        detlib.detdecode_attention_shared_f32(qd, kc, vc, table, ld, 4, 3, out=out, workspace=ws)
    for n in (lens, [1, 0, 9], [499, 32, 900], lens):
        ld.copy_(on_gpu(np.array(n, np.int32)))
        out.fill_(7.0)
        g.replay()
        n = [min(int(m), len(k)) for m, k in zip(n, Ks)]
        # tokens past a request's own are another's: only those it has
        if all(m <= len(k) for m, k in zip(n, Ks)):
            want = decode_oracle(q, [k[:m] for k, m in zip(Ks, n)], [v[:m] for v, m in zip(Vs, n)],
                                 4, 0.125)
            assert_bitwise(host(out)[:1], want[:1])
    # other sharing under the same graph: the second request leaves the prefix
    table[1] = table[0]
    g.replay()
    ld2 = ld.clone()
    assert_bitwise(host(out), host(detlib.detdecode_attention_f32(qd, kc, vc, table, ld2, 4)))


def test_two_threads_at_once(dev):
    rng = np.random.default_rng(27)
    jobs = []
    for prefix, own, H, d in ((600, [20, 17], 4, 64), (1500, list(range(1, 41)), 8, 128)):
        kc, vc, table, lens, _, _ = shared_cache([prefix], own, 16, 4, d, "token", rng)
        q = rng.standard_normal((len(own), H * d)).astype(F)
        want = both(q, kc, vc, table, lens, H, len(own))
        jobs.append(((to_dev(q), kc, vc, table, on_gpu(lens), H, len(own)), want))
    torch.cuda.synchronize()
    failed = []

    def work(job):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(1000):
                    out = detlib.detdecode_attention_shared_f32(*job[0])
                got = host(out)
            assert_bitwise(got, job[1])
        except Exception as e:      # noqa: BLE001 (an error of the other thread)
            failed.append(e)

    threads = [threading.Thread(target=work, args=(job,)) for job in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed


@pytest.mark.parametrize("B,H,G,group", [(20, 4, 4, 20), (24, 4, 2, 3), (12, 9, 1, 12)])
def test_read_together_captured_and_on_two_streams(dev, B, H, G, group):
    # tables wide enough that requests are read together or in groups; two captured calls
    # replayed on two streams at once, on other queries each time
    rng = np.random.default_rng(B)
    own = rng.integers(1, 600, B)
    kc, vc, table, lens, _, _ = shared_cache([1500], own, 16, G, 64, "token", rng)
    wide = torch.full((B, WIDE // 16), -7, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    ld = on_gpu(lens)
    jobs = []
    for _ in range(2):
        q = torch.zeros((B, H * 64), device="cuda")
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            detlib.detdecode_attention_shared_f32(q, kc, vc, wide, ld, H, group)
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            out = detlib.detdecode_attention_shared_f32(q, kc, vc, wide, ld, H, group)
        jobs.append((q, s, g, out))
    for step in range(5):
        for q, _, _, _ in jobs:
            q.copy_(on_gpu(rng.standard_normal((B, H * 64)).astype(F)))
        torch.cuda.synchronize()
        for q, s, g, out in jobs:
            with torch.cuda.stream(s):
                for _ in range(3):
                    g.replay()
        torch.cuda.synchronize()
        for q, s, g, out in jobs:
            want = detlib.detdecode_attention_f32(q, kc, vc, table, ld, H)
            assert_bitwise(host(out), host(want), f"replay {step}")
