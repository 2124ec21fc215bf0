"""The selection of the next beams against a sequential statement of its rules:
ties, ended and dead beams, masked and NaN scores, weights, histories of odd
sizes and strides, captured and on another stream."""
import threading

import numpy as np
import pytest

from bitwise_reproducible_fp32_gb300 import detlib
from gpu_util import host, need_gpu, torch

pytestmark = pytest.mark.gpu
F, I = np.float32, np.int32


@pytest.fixture(scope="module")
def dev():
    return need_gpu()


def on_gpu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def select_plain(scores, ids, logp, beams, eos=-1, finished=None, lens=None, weights=None,
                 hist=None, hist_out=None):
    R, W = scores.shape
    k = ids.shape[1]
    new = R * beams
    s_out = np.full((R, beams), -np.inf, F)
    tok, par, forks = (np.full(new, -1, I) for _ in range(3))
    fin, l_out = np.ones(new, I), np.zeros(new, I)
    h_out = None if hist is None else hist_out.copy()
    status = 0
    for r in range(R):
        cand = []
        for w in range(W):
            row = r * W + w
            n = int(lens[row]) if lens is not None else 0
            done = finished is not None and finished[row] != 0
            if scores[r, w] == -np.inf:
                continue
            for j in range(1 if done else k):
                with np.errstate(all="ignore"):
                    s = scores[r, w] if done else F(scores[r, w] + logp[row, j])
                    m = n if done else n + 1
                    rank = s if weights is None else F(
                        s * weights[min(max(m, 0), len(weights) - 1)])
                if s == -np.inf:
                    continue
                if np.isnan(rank):
                    status |= 1
                    continue
                cand.append((-float(rank), w, eos if done else int(ids[row, j]), j, s, m, done))
        for c, (_, w, t, j, s, m, done) in enumerate(sorted(cand, key=lambda c: c[:4])[:beams]):
            row, out = r * W + w, r * beams + c
            s_out[r, c], tok[out], par[out], l_out[out] = s, t, row, m
            fin[out] = done or t == eos
            forks[out] = -1 if fin[out] else row
            if hist is not None:
                n, cols = int(lens[row]), hist.shape[1]
                if n < 0 or n + (not done) > cols:
                    status |= 2
                n = max(n, 0)
                h_out[out, :min(n, cols)] = hist[row, :min(n, cols)]
                if not done and 0 <= lens[row] < cols:
                    h_out[out, n] = t
    return s_out, tok, par, forks, fin, l_out if lens is not None else None, h_out, status


def check(scores, ids, logp, beams, layout="dense", **kw):
    hist = kw.get("hist")
    if hist is not None:
        kw["hist_out"] = np.full((scores.shape[0] * beams, hist.shape[1]), -77, I)
    want = select_plain(scores, ids, logp, beams, **kw)
    dk = {n: on_gpu(v) if isinstance(v, np.ndarray) else v for n, v in kw.items()}
    if hist is not None and layout != "dense":
        for n in ("hist", "hist_out"):
            wide = torch.full((dk[n].shape[0], dk[n].shape[1] + 5), -9, dtype=torch.int32,
                              device="cuda")
            wide[:, 1:-4] = dk[n]
            dk[n] = wide[:, 1:-4]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = detlib.detbeam_select_f32(on_gpu(scores), on_gpu(ids), on_gpu(logp), beams,
                                    dev_status=status, **dk)
    for g, w, name in zip(got, want, got._fields):
        if w is None:
            assert g is None
        else:
            assert np.array_equal(host(g), w), (name, host(g), w)
    assert int(status) == want[-1]
    return got


def draw(R, W, k, rng, V=1000):
    logp = -rng.exponential(2.0, (R * W, k)).astype(F)
    ids = np.argsort(rng.random((R * W, V)), axis=1)[:, :k].astype(I)
    return (-rng.exponential(5.0, (R, W))).astype(F), ids, logp


@pytest.mark.parametrize("R", [1, 3, 70])
@pytest.mark.parametrize("W,k,beams", [(1, 1, 1), (1, 32, 32), (4, 8, 4), (2, 3, 32), (5, 7, 6),
                                       (32, 32, 32), (31, 1, 17), (17, 32, 1), (3, 31, 29)])
def test_select(dev, R, W, k, beams):
    rng = np.random.default_rng(R * 1000 + W * 32 + k)
    scores, ids, logp = draw(R, W, k, rng)
    check(scores, ids, logp, beams)
    lens = rng.integers(0, 40, R * W).astype(I)
    done = (rng.random(R * W) < 0.3).astype(I) * 5
    check(scores, ids, logp, beams, eos=int(ids[0, 0]), finished=done, lens=lens)
    weights = (np.arange(1, 30) ** -0.7).astype(F)
    hist = rng.integers(0, 1000, (R * W, 41)).astype(I)
    for layout in ("dense", "offset"):
        check(scores, ids, logp, beams, layout, eos=int(ids[0, 0]), finished=done, lens=lens,
              weights=weights, hist=hist)


def test_ties_go_to_the_lowest_beam_then_id(dev):
    rng = np.random.default_rng(5)
    R, W, k = 40, 6, 16
    scores = rng.integers(-3, 1, (R, W)).astype(F)
    logp = rng.integers(-3, 1, (R * W, k)).astype(F)
    ids = rng.integers(-4, 20, (R * W, k)).astype(I)         # one id more than once, too
    scores[scores == 0] = F(-0.0)
    check(scores, ids, logp, 20, eos=3, lens=np.full(R * W, 2, I),
          hist=rng.integers(0, 9, (R * W, 3)).astype(I))


def test_dead_masked_infinite_and_nan(dev):
    rng = np.random.default_rng(6)
    R, W, k = 12, 4, 8
    scores, ids, logp = draw(R, W, k, rng)
    scores[:, 1:] = -np.inf                     # a first step: one live beam
    logp[::3, 4:] = -np.inf                     # masked alternatives
    scores[2] = -np.inf                         # nothing left
    logp[4 * W, 2] = np.nan
    scores[5, 0] = np.nan
    scores[6, 0] = np.inf
    logp[7 * W] = np.inf
    scores[8, 2], logp[8 * W + 2] = 1e30, -3e38
    lens = np.zeros(R * W, I)
    hist = np.zeros((R * W, 4), I)
    done = np.zeros(R * W, I)
    done[9 * W], scores[10, 3], done[10 * W + 3] = 1, np.nan, 1
    check(scores, ids, logp, 6, eos=int(ids[3 * W, 0]), finished=done, lens=lens, hist=hist)
    # weights that make 0 * inf, and a negative zero
    check(scores, ids, logp, 6, finished=done, lens=lens, weights=np.array([0.0, 0.0], F))
    check(scores, ids, logp, 6, finished=done, lens=lens, weights=np.array([1.0, -1.0], F))


def test_histories(dev):
    rng = np.random.default_rng(7)
    for R, W, beams, cols in ((3, 4, 4, 5000), (2, 2, 5, 1), (1, 1, 3, 1024), (5, 3, 3, 1025),
                              (2, 16, 16, 2047)):
        scores, ids, logp = draw(R, W, 8, rng)
        hist = rng.integers(0, 1000, (R * W, cols)).astype(I)
        lens = rng.integers(0, cols + 1, R * W).astype(I)
        for layout in ("dense", "offset"):
            check(scores, ids, logp, beams, layout, lens=lens, hist=hist)
        # lengths that do not fit, and none
        lens[0], lens[-1] = cols + 3, -2
        check(scores, ids, logp, beams, lens=lens, hist=hist)
        lens[:] = 2 ** 31 - 2
        check(scores, ids, logp, beams, lens=lens, hist=hist, weights=np.array([1.0, 2.0], F))


def test_no_requests(dev):
    e = lambda *s: torch.empty(s, device="cuda")                       # noqa: E731
    got = detlib.detbeam_select_f32(e(0, 4), e(0, 8).int(), e(0, 8), 4, lens=e(0).int())
    assert got.scores.shape == (0, 4) and got.tokens.numel() == 0 and got.lens.numel() == 0


def test_a_negative_ending_ends_nothing(dev):
    # an id of -1 with a score is a token like others where eos says that there is no ending
    s, lp = torch.zeros((1, 1), device="cuda"), torch.tensor([[-1.0, -2.0]], device="cuda")
    ids = torch.tensor([[-1, 5]], dtype=torch.int32, device="cuda")
    got = detlib.detbeam_select_f32(s, ids, lp, 2)
    assert host(got.tokens).tolist() == [-1, 5] and host(got.finished).tolist() == [0, 0]
    assert host(got.forks).tolist() == [0, 0]


def test_histories_without_columns(dev):
    # the C entry takes histories of no columns: nothing is written, and every one is cut
    lib, prof = detlib.load(), detlib.det_profile_default()
    rng = np.random.default_rng(12)
    s, i, lp = (on_gpu(a) for a in draw(3, 2, 4, rng))
    n = torch.zeros(6, dtype=torch.int32, device="cuda")
    h, ho = (torch.full((6,), v, dtype=torch.int32, device="cuda") for v in (3, 4))
    so = torch.empty(6, device="cuda")
    tok, par, st = (torch.zeros(6, dtype=torch.int32, device="cuda") for _ in range(3))
    args = [detlib.BeamsArg(2, s.data_ptr(), None, n.data_ptr(), h.data_ptr(), 1),
            detlib.BeamsArg(2, so.data_ptr(), None, None, ho.data_ptr(), 1)]
    rc = lib.detbeam_select_f32(prof, 3, *args, 4, i.data_ptr(), lp.data_ptr(), -1, None, 0, 0,
                                tok.data_ptr(), par.data_ptr(), None, st.data_ptr(),
                                torch.cuda.current_stream().cuda_stream)
    assert rc == 0 and int(st[0]) == 2 and bool((ho == 4).all())
    want = select_plain(*map(host, (s, i, lp)), 2)
    assert np.array_equal(host(so).reshape(3, 2), want[0]) and np.array_equal(host(tok), want[1])


def test_binding_refusals(dev):
    rng = np.random.default_rng(8)
    s, i, lp = (on_gpu(a) for a in draw(2, 4, 8, rng))
    n = torch.zeros(8, dtype=torch.int32, device="cuda")
    h = torch.zeros((8, 9), dtype=torch.int32, device="cuda")
    f = detlib.detbeam_select_f32
    for call in (lambda: f(s, i[:7], lp[:7], 4), lambda: f(s, i, lp[:, :7], 4),
                 lambda: f(s, i, lp, 0), lambda: f(s, i, lp, 33), lambda: f(s, i, lp, 4, hist=h),
                 lambda: f(s, i, lp, 4, lens=n, hist=h[:, :0]),
                 lambda: f(s, i, lp, 4, weights=lp[0]),
                 lambda: f(s, i, lp, 4, lens=n, hist_out=h),
                 lambda: f(s, i, lp, 4, lens=n, hist=h, hist_out=h[:, :8]),
                 lambda: f(s, i, lp, 4, lens=n[:7]), lambda: f(s, i, lp, 4, lens_out=n),
                 lambda: f(s, i[:, ::2], lp[:, ::2], 4),
                 lambda: f(s, i, lp, 4, scores_out=s[:, :3])):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(detlib.DetError):
        f(s, i, lp, 4, lens=n, hist=h, hist_out=h)
    with pytest.raises(detlib.DetError):
        f(s, i, lp, 4, scores_out=s)
    with pytest.raises(TypeError):
        f(s, i.long(), lp, 4)


def test_captured_and_from_two_threads(dev):
    rng = np.random.default_rng(9)
    jobs = []
    for R, W, k, cols in ((30, 4, 8, 100), (3, 32, 32, 3000)):
        scores, ids, logp = draw(R, W, k, rng)
        lens = rng.integers(0, cols, R * W).astype(I)
        hist = rng.integers(0, 1000, (R * W, cols)).astype(I)
        want = select_plain(scores, ids, logp, W, lens=lens, hist=hist,
                            hist_out=np.zeros_like(hist))
        jobs.append(([on_gpu(a) for a in (scores, ids, logp)], W,
                     dict(lens=on_gpu(lens), hist=on_gpu(hist),
                          hist_out=torch.zeros_like(on_gpu(hist))), want))
    torch.cuda.synchronize()
    # captured, replayed on other scores
    args, W, kw, want = jobs[0]
    g = torch.cuda.CUDAGraph()
    keep = args[0].clone()
    detlib.detbeam_select_f32(*args, W, **kw)
    with torch.cuda.graph(g):
        out = detlib.detbeam_select_f32(*args, W, **kw)
    args[0].neg_()
    g.replay()
    args[0].copy_(keep)
    kw["hist_out"].zero_()          # columns past a length are not touched
    g.replay()
    assert np.array_equal(host(out.scores), want[0]) and np.array_equal(host(out.hist), want[6])
    failed = []

    def work(job):
        args, W, kw, want = job
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(300):
                    out = detlib.detbeam_select_f32(*args, W, **kw)
                for g, w in zip(out, want):
                    assert np.array_equal(host(g), w)
        except Exception as e:      # noqa: BLE001 (an error of the other thread)
            failed.append(e)

    threads = [threading.Thread(target=work, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
