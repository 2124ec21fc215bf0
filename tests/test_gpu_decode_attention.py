"""GPU parity (0 ULP) of decode attention over a paged cache: against the oracle,
against the last row of the training attention, and against 64 bits within a
derived bound; lengths from 0 to long, page sizes that end inside every tile,
layouts, shared heads, infinities and NaN, bad lengths and pages."""
import threading

import numpy as np
import pytest

from bitcmp import assert_bitwise
from bitwise_reproducible_fp32_gb300 import detlib
from exp_cases import exp_tie_arguments
from gen_util import F, LAYOUTS, decode64, decode_oracle, fill_cache
from gpu_util import host, need_gpu, to_dev, torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return need_gpu()


def on_gpu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def run(q, kc, vc, table, lens, H, layout="dense", **kw):
    return detlib.detdecode_attention_f32(to_dev(q, layout), kc, vc, table,
                                          on_gpu(np.asarray(lens, np.int32)), H, **kw)


@pytest.mark.parametrize("H,G,d", [(1, 1, 64), (4, 4, 16), (12, 12, 64), (8, 2, 128), (6, 2, 80),
                                   (16, 1, 64), (24, 2, 32), (3, 3, 7), (2, 1, 1), (10, 5, 36),
                                   (2, 2, 256), (9, 1, 250)])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("ps", [16, 5])
def test_ragged_lengths(dev, H, G, d, layout, ps):
    rng = np.random.default_rng(H * 1000 + d + ps)
    lens = [0, 1, 2, 31, 32, 33, 255, 256, 257, 600, 1023, 1025]
    kc, vc, table, Ks, Vs = fill_cache(lens, ps, G, d, layout, rng)
    q = (2 * rng.standard_normal((len(lens), H * d))).astype(F)
    scale = float(F(1.0 / np.sqrt(d)))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = host(run(q, kc, vc, table, lens, H, "offset" if layout == "offset" else "padded",
                   dev_status=status))
    assert_bitwise(got, decode_oracle(q, Ks, Vs, H, scale), f"{layout} ps={ps}")
    assert int(status) == 0
    for b, n in enumerate(lens):
        for h in range(H) if n else ():
            want, bound = decode64(q[b, h * d:(h + 1) * d], Ks[b][:, h // (H // G)],
                                   Vs[b][:, h // (H // G)], scale)
            assert (np.abs(got[b, h * d:(h + 1) * d] - want) <= bound).all(), (b, h)


@pytest.mark.parametrize("B,H,G,d,longest,ps", [(1, 2, 2, 64, 20000, 16), (1, 8, 1, 128, 9001, 64),
                                                (2, 12, 12, 64, 4097, 16), (3, 4, 4, 16, 33000, 100),
                                                (1, 1, 1, 256, 5000, 1), (40, 12, 12, 64, 700, 16),
                                                (1, 1, 1, 64, 70001, 4096)])
def test_long(dev, B, H, G, d, longest, ps):
    rng = np.random.default_rng(longest)
    lens = rng.integers(longest // 2, longest + 1, B)
    lens[0] = longest
    kc, vc, table, Ks, Vs = fill_cache(lens, ps, G, d, "token", rng)
    q = (2 * rng.standard_normal((B, H * d))).astype(F)
    got = host(run(q, kc, vc, table, lens, H))
    assert_bitwise(got, decode_oracle(q, Ks, Vs, H, float(F(1.0 / np.sqrt(d)))))


def test_last_row_of_the_training_attention(dev):
    # 3 sequences of 700: the attention's last row of each, and its first
    rng = np.random.default_rng(21)
    B, T, H, d = 3, 700, 12, 64
    qkv = rng.standard_normal((B * T, 3 * H * d)).astype(F)
    att = host(detlib.detattention_f32(to_dev(qkv), B, T, H, d))
    X = qkv.reshape(B, T, 3, H, d)
    for n in (T, 1):
        kc, vc, table, _, _ = fill_cache([n] * B, 16, H, d, "head", rng,
                                         K=[X[b, :n, 1] for b in range(B)],
                                         V=[X[b, :n, 2] for b in range(B)])
        q = np.ascontiguousarray(X[:, n - 1, 0].reshape(B, H * d))
        assert_bitwise(host(run(q, kc, vc, table, [n] * B, H)),
                       att.reshape(B, T, H * d)[:, n - 1])


def test_other_requests_and_wider_tables_change_nothing(dev):
    rng = np.random.default_rng(22)
    lens = [300, 40, 2000, 17]
    kc, vc, table, _, _ = fill_cache(lens, 16, 4, 64, "token", rng)
    q = rng.standard_normal((4, 512)).astype(F)
    all_ = host(run(q, kc, vc, table, lens, 8))
    for b in range(4):
        one = host(run(q[b:b + 1], kc, vc, table[b:b + 1], lens[b:b + 1], 8))
        assert_bitwise(one, all_[b:b + 1])
    wide = torch.full((4, 4000), -1, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    assert_bitwise(host(run(q, kc, vc, wide, lens, 8)), all_)


def test_infinities_and_nan(dev):
    rng = np.random.default_rng(23)
    H = G = 3
    d, n = 64, 700
    Ks = [rng.standard_normal((n, G, d)).astype(F) for _ in range(6)]
    Vs = [rng.standard_normal((n, G, d)).astype(F) for _ in range(6)]
    q = rng.standard_normal((6, H * d)).astype(F)
    Ks[0][5, 0, 3] = np.nan             # a NaN score: the head is NaN
    Ks[1][6, 1, :] = np.inf             # inf - inf or inf in the chain
    Vs[2][699, 2, 1] = np.inf           # one component infinite
    Vs[3][300, 0, 7] = np.nan
    Ks[4][:] *= F(1e30)                 # scores far apart: exps underflow to 0
    q[5] *= F(1e-30)                    # all scores alike
    kc, vc, table, _, _ = fill_cache([n] * 6, 16, G, d, "token", rng, K=Ks, V=Vs)
    with np.errstate(all="ignore"):
        want = decode_oracle(q, Ks, Vs, H, 0.125)
    assert_bitwise(host(run(q, kc, vc, table, [n] * 6, H)), want)


def test_bad_lengths_and_pages(dev):
    rng = np.random.default_rng(24)
    lens = [100, 100, 100, 100, 100, 0]
    kc, vc, table, Ks, Vs = fill_cache(lens, 16, 2, 64, "token", rng)
    q = rng.standard_normal((6, 128)).astype(F)
    want = decode_oracle(q, Ks, Vs, 2, 0.125)
    bad = table.clone()
    bad[1, 6] = kc.shape[0]             # the last page the request reads
    bad[2, 0] = -1
    bad[5, 0] = 10 ** 6                 # not read: no tokens
    n = [100, 100, 100, -1, 16 * table.shape[1] + 1, 0]
    want[1:5] = np.nan
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert_bitwise(host(run(q, kc, vc, bad, n, 2, dev_status=status)), want)
    assert int(status) == 3
    # with no status word, and with pages past the length out of range
    assert_bitwise(host(run(q, kc, vc, bad, n, 2)), want)
    ok = table.clone()
    ok[0, 6] = 10 ** 6
    status.zero_()
    got = host(run(q[:1], kc, vc, ok[:1], [96], 2, dev_status=status))
    assert_bitwise(got, decode_oracle(q[:1], [Ks[0][:96]], [Vs[0][:96]], 2, 0.125))
    assert int(status) == 0


def test_cache_past_32_bit_offsets(dev):
    G, d, ps, n = 8, 128, 64, 300
    pages = 35_000                      # 2.3e9 floats each
    kc, vc = (torch.full((pages, ps, G, d), float("nan"), device="cuda") for _ in range(2))
    rng = np.random.default_rng(25)
    ids = np.array([pages - 1, 34_000, 32_768, 1, 16_384], np.int32)
    K, V = (rng.standard_normal((n, G, d)).astype(F) for _ in range(2))
    pad = np.full((len(ids) * ps, G, d), np.nan, F)
    for c, x in ((kc, K), (vc, V)):
        full = pad.copy()
        full[:n] = x
        c[on_gpu(ids).long()] = on_gpu(full.reshape(len(ids), ps, G, d))
    q = rng.standard_normal((1, 2 * G * d)).astype(F)
    got = host(run(q, kc, vc, on_gpu(ids[None]), [n], 2 * G))
    assert_bitwise(got, decode_oracle(q, [K], [V], 2 * G, float(F(1 / np.sqrt(d)))))


def test_captured_replayed_and_on_another_stream(dev):
    rng = np.random.default_rng(26)
    lens = [500, 33]
    kc, vc, table, Ks, Vs = fill_cache(lens, 16, 4, 64, "token", rng)
    q = rng.standard_normal((2, 256)).astype(F)
    want = decode_oracle(q, Ks, Vs, 4, 0.125)
    s = torch.cuda.Stream()
    qd, ld = to_dev(q), on_gpu(np.array(lens, np.int32))
    s.wait_stream(torch.cuda.current_stream())
    outs = [detlib.detdecode_attention_f32(qd, kc, vc, table, ld, 4, stream=s) for _ in range(3)]
    s.synchronize()
    for o in outs:
        assert_bitwise(host(o), want)
    out = torch.empty_like(qd)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        detlib.detdecode_attention_f32(qd, kc, vc, table, ld, 4, out=out)
    for n in (lens, [1, 0], [499, 32]):
        ld.copy_(on_gpu(np.array(n, np.int32)))
        out.fill_(7.0)
        g.replay()
        assert_bitwise(host(out), decode_oracle(q, [k[:m] for k, m in zip(Ks, n)],
                                                [v[:m] for v, m in zip(Vs, n)], 4, 0.125))


@pytest.mark.parametrize("H,G", [(1, 1), (2, 1), (4, 1), (8, 1), (3, 3)])
@pytest.mark.parametrize("n", [256, 3000])
def test_exps_at_the_ties_of_their_rounding(dev, H, G, n):
    # scores 0, then every d at which rounding d log2 e once or twice differs, 128 a
    # request; a value has a one where its token is, so the outputs are the
    # probabilities one by one
    ties, w = exp_tie_arguments(-127, 0), 128
    rng = np.random.default_rng(n + H)
    Ks, Vs = [], []
    for r in range(-(-len(ties) // w)):
        part = ties[r * w:(r + 1) * w]
        K, V = np.zeros((n, G, w), F), np.zeros((n, G, w), F)
        K[1:, :, 0] = -F(200.0)
        at = 1 + rng.permutation(n - 1)[:len(part)]
        K[at, :, 0] = part[:, None]
        V[at, :, np.arange(len(part))] = 1.0
        Ks.append(K)
        Vs.append(V)
    lens = [n] * len(Ks)
    kc, vc, table, _, _ = fill_cache(lens, 16, G, w, "token", rng, K=Ks, V=Vs)
    q = np.zeros((len(Ks), H * w), F)
    q[:, ::w] = 1.0
    got = host(run(q, kc, vc, table, lens, H, scale=1.0))
    assert_bitwise(got, decode_oracle(q, Ks, Vs, H, 1.0))
    assert (got != 0).sum() > 300 * H


def test_two_threads_at_once(dev):
    # short rows, and many of four chunks a CTA, whose launches take different amounts
    # of shared memory, from two host threads on streams of their own
    rng = np.random.default_rng(27)
    jobs = []
    for lens in ([200, 17], [1000] * 40):
        kc, vc, table, Ks, Vs = fill_cache(lens, 16, 4, 64, "token", rng)
        q = rng.standard_normal((len(lens), 256)).astype(F)
        jobs.append((to_dev(q), kc, vc, table, on_gpu(np.array(lens, np.int32)),
                     decode_oracle(q, Ks, Vs, 4, 0.125)))
    torch.cuda.synchronize()
    failed = []

    def work(job):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(4000):
                    out = detlib.detdecode_attention_f32(*job[:5], 4)
                got = host(out)
            assert_bitwise(got, job[5])
        except Exception as e:      # noqa: BLE001 (an error of the other thread)
            failed.append(e)

    threads = [threading.Thread(target=work, args=(job,)) for job in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
