"""GPU parity (0 ULP) of the token log probabilities, entropies, alternatives and
their gradient against the oracle, and against 64 bits within derived bounds."""
import numpy as np
import pytest

import oracle
from bitcmp import assert_bitwise
from bitwise_reproducible_fp32_gb300 import detlib
from exp_cases import exp_tie_arguments
from gen_util import F, U, logprob64
from gpu_util import host, need_gpu, to_dev, torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return need_gpu()


def on_gpu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def check(x, y, k, layout="dense", bwd=True, seed=0):
    with np.errstate(all="ignore"):
        want = oracle.logprob(x, y, k)
    xd, yd = to_dev(x, layout), on_gpu(y.astype(np.int32))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    logp, ent, ids, top, stats = detlib.detlogprob_f32(xd, yd, top_k=k, dev_status=status)
    for got, w, name in ((logp, want[0], "logp"), (ent, want[1], "entropy"),
                         (stats, want[2], "stats"), (top, want[4], "top_logp")):
        assert_bitwise(host(got), w, f"{name} V={x.shape[1]} {layout}")
    assert np.array_equal(host(ids), want[3])
    assert int(status) == int(((y < -1) | (y >= x.shape[1])).any())
    if not bwd:
        return want
    rng = np.random.default_rng(seed)
    g, gH = (rng.standard_normal(len(x)).astype(F) for _ in range(2))
    for h in (None, gH):
        w = oracle.logprob_bwd(x, y, want[2], g, h)
        hd = None if h is None else on_gpu(h)
        assert_bitwise(host(detlib.detlogprob_bwd_f32(xd, yd, stats, on_gpu(g), hd)), w, "grad")
        out = to_dev(np.full(x.shape, 3.0, F), "offset")
        detlib.detlogprob_bwd_f32(xd, yd, stats, on_gpu(g), hd, dlogits=out)
        assert_bitwise(host(out), w, "grad, other alignment")
    detlib.detlogprob_bwd_f32(xd, yd, stats, on_gpu(g), hd, dlogits=xd)
    assert_bitwise(host(xd), w, "grad in place")
    return want


@pytest.mark.parametrize("V", [1, 2, 3, 5, 64, 255, 256, 1000, 1023, 1024, 1025, 4096, 4099, 10001,
                               32000, 50257, 57590, 57601, 70001, 151936])
@pytest.mark.parametrize("layout", ["dense", "padded", "offset"])
def test_sizes(dev, V, layout):
    rng = np.random.default_rng(V)
    rows = 7 if V > 5000 else 400
    x = (2 * rng.standard_normal((rows, V))).astype(F)
    y = rng.integers(0, V, rows)
    y[:3] = [-1, V, -2]
    want = check(x, y, min(V, 20), layout)
    logp, ent, b1, b2 = logprob64(x[3:], y[3:])
    assert (np.abs(want[0][3:] - logp) <= b1).all() and (np.abs(want[1][3:] - ent) <= b2).all()


@pytest.mark.parametrize("k", [0, 1, 2, 31, 32])
@pytest.mark.parametrize("V", [32, 777, 50257, 80000])
def test_alternatives_with_ties(dev, k, V):
    # values of few distinct levels, constant rows, ascending and descending
    # rows, the largest values side by side and far apart
    rng = np.random.default_rng(k + V)
    x = rng.integers(-3, 4, (12, V)).astype(F)
    x[1] = 0.5
    x[2] = np.arange(V) / V
    x[3] = -np.arange(V) / V
    x[4] = (2 * rng.standard_normal(V)).astype(F)
    x[4, V // 2:V // 2 + 16] = 30.0
    x[5] = np.where(np.arange(V) % 2, F(0.0), F(-0.0))
    x[6] = rng.standard_normal(V)
    x[6, [0, V - 1, V // 3]] = 9.0
    x[7] = np.where(rng.random(V) < 0.001, 4.0, -4.0)
    x[8, :] = -np.inf
    x[8, V // 4] = 1.0
    x[9] = np.repeat(rng.standard_normal(V // 8 + 1), 8)[:V]
    check(x, np.full(12, V // 4), k, bwd=False)


def test_infinities_and_nan(dev):
    rng = np.random.default_rng(4)
    for V in (40, 1000, 5003, 50257, 60011):
        x = (2 * rng.standard_normal((9, V))).astype(F)
        x[0, 3] = np.nan
        x[1, [5, V - 1]] = np.nan
        x[2, 7] = np.inf
        x[3, :] = -np.inf
        x[4, ::2] = -np.inf
        x[5, :] = np.finfo(F).min
        x[6, :] = np.finfo(F).min
        x[6, V // 2] = 0.0
        x[7, 1:] = -200.0
        x[7, 0] = 0.0
        x[8, 2] = np.finfo(F).max
        check(x, np.array([3, 0, 7, 0, 1, 2, V // 2, 1, 2]), min(V, 32), "padded")


def test_logp_is_the_cross_entropy(dev):
    rng = np.random.default_rng(6)
    x = (2 * rng.standard_normal((64, 50257))).astype(F)
    y = on_gpu(rng.integers(0, 50257, 64).astype(np.int32))
    xd = to_dev(x)
    loss, _, dl = detlib.detxent_f32(xd, y, want_dlogits=True, dscale=1.0)
    logp = detlib.detlogprob_f32(xd, y)[0]
    assert_bitwise(host(logp), -host(loss))
    # and its gradient with dlogp = -1: -(hot - p), the cross-entropy's p - hot
    st = detlib.detlogprob_f32(xd, y)[4]
    got = detlib.detlogprob_bwd_f32(xd, y, st, torch.full((64,), -1.0, device="cuda"))
    assert_bitwise(host(got), host(dl))


def test_gradient_formula_and_differences(dev):
    rng = np.random.default_rng(9)
    V, rows = 37, 5
    x = rng.standard_normal((rows, V)).astype(F)
    y = np.array([0, 36, 5, -1, 9])
    g, gH = (rng.standard_normal(rows).astype(F) for _ in range(2))
    st = detlib.detlogprob_f32(to_dev(x), on_gpu(y.astype(np.int32)))[4]
    got = host(detlib.detlogprob_bwd_f32(to_dev(x), on_gpu(y.astype(np.int32)), st, on_gpu(g),
                                         on_gpu(gH)))

    def f(z):
        d = z - z.max(1, keepdims=True)
        lp = d - np.log(np.exp(d).sum(1, keepdims=True))
        at = np.where(y < 0, 0.0, lp[np.arange(rows), np.maximum(y, 0)])
        return g * at - gH * (np.exp(lp) * lp).sum(1)

    x64 = x.astype(np.float64)
    d = x64 - x64.max(1, keepdims=True)
    lp = d - np.log(np.exp(d).sum(1, keepdims=True))
    p, ent = np.exp(lp), -(np.exp(lp) * lp).sum(1, keepdims=True)
    hot = (np.arange(V)[None] == y[:, None]).astype(float)
    want = np.where(y[:, None] < 0, 0.0, g[:, None] * (hot - p)) - gH[:, None] * p * (lp + ent)
    # p is off by at most |d| + 2 (exp) + 24 (S) + 3 roundings, w by 40 more
    size = np.abs(g[:, None]) * (hot + p) + np.abs(gH[:, None]) * p * (np.abs(lp) + ent + 1)
    assert (np.abs(got - want) <= size * (np.abs(d) + 70) * U).all()
    h = 1e-5        # central differences: h^2 / 6 of third derivatives below 8, 1e-16 / h
    for j in range(V):
        step = np.zeros_like(x64)
        step[:, j] = h
        quot = (f(x64 + step) - f(x64 - step)) / (2 * h)
        assert (np.abs(want[:, j] - quot) <= 1e-9 * 8).all()


def test_rows_cycle_through_the_grid_on_a_stream_and_captured(dev):
    rng = np.random.default_rng(10)
    V = 2001
    x = (2 * rng.standard_normal((1500, V))).astype(F)
    y = rng.integers(0, V, 1500).astype(np.int32)
    want = oracle.logprob(x, y, 4)
    xd, yd = to_dev(x), on_gpu(y)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = detlib.detlogprob_f32(xd, yd, top_k=4, stream=s)
    s.synchronize()
    assert_bitwise(host(got[0]), want[0])
    assert np.array_equal(host(got[2]), want[3])
    outs = [torch.empty_like(t) for t in got]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        detlib.detlogprob_f32(xd, yd, top_k=4, logp=outs[0], entropy=outs[1], top_ids=outs[2],
                              top_logp=outs[3], stats=outs[4])
    xd.copy_(to_dev(x[::-1].copy()))
    yd.copy_(on_gpu(y[::-1].copy()))
    g.replay()
    assert_bitwise(host(outs[0]), want[0][::-1])
    assert_bitwise(host(outs[1]), want[1][::-1])
    assert np.array_equal(host(outs[2]), want[3][::-1])
    assert detlib.det_watchdog_status() == 0


def test_no_rows(dev):
    e = torch.empty((0, 10), device="cuda")
    t = torch.empty(0, dtype=torch.int32, device="cuda")
    out = detlib.detlogprob_f32(e, t, top_k=3)
    assert [tuple(o.shape) for o in out] == [(0,), (0,), (0, 3), (0, 3), (0, 4)]
    assert detlib.detlogprob_bwd_f32(e, t, out[4], out[0]).shape == (0, 10)


@pytest.mark.parametrize("V", [4097, 4099, 16001, 50257, 70001, 151936, 256003])
@pytest.mark.parametrize("layout", ["dense", "padded", "offset"])
def test_the_number_of_rows_changes_no_bit(dev, V, layout):
    # few rows are split over clusters, many are not: the same rows in calls of
    # 1, 12, 24, 36, 60 and 168, with ties, equal logits, infinities, NaN and
    # masks at the lowest value among them
    rng = np.random.default_rng(V)
    x = (3 * rng.standard_normal((12, V))).astype(F)
    x[1] = rng.integers(-3, 4, V)
    x[2] = 0.25
    x[3, rng.random(V) < 0.9] = -np.inf
    x[4, :] = -np.inf
    x[5, V // 3] = np.inf
    x[6, V - 1] = np.nan
    x[7, rng.random(V) < 0.5] = np.finfo(F).min
    x[8] = np.where(np.arange(V) % 2, F(0.0), F(-0.0))
    x[9] = np.arange(V) / V * 200
    x[10, :] = -np.inf
    x[10, V - 1] = 2.0
    x[11] = x[11] * 40
    y = rng.integers(0, V, 12).astype(np.int32)
    y[:2] = [-1, V - 1]
    want = check(x, y, 32, layout)
    full = np.tile(x, (14, 1)), np.tile(y, 14)
    for rows in (1, 24, 36, 60, 168):
        xd = to_dev(full[0][:rows], layout)
        yd = torch.from_numpy(full[1][:rows]).cuda()
        logp, ent, ids, top, stats = (host(t) for t in detlib.detlogprob_f32(xd, yd, top_k=32))
        for r in range(0, rows, 12):
            n = min(12, rows - r)
            for got, w, name in zip((logp, ent, stats, ids, top), want,
                                    ("logp", "entropy", "stats", "ids", "top")):
                if name == "ids":
                    assert np.array_equal(got[r:r + n], w[:n]), (rows, r)
                else:
                    assert_bitwise(got[r:r + n], w[:n], f"{name}, row {r} of {rows}")


@pytest.mark.parametrize("V", [400001, 444416, 444417, 600000, 1048577])
def test_long_rows(dev, V):
    # the longest share of a cluster, and rows past it
    rng = np.random.default_rng(V)
    check((2 * rng.standard_normal((2, V))).astype(F), np.array([V - 1, 5], np.int32), 7, "offset")


def special_rows(x, rng):
    """Rows that leave the ordinary way, mixed between ordinary ones: a list of
    alternatives that overflows, NaN, infinities, masks that leave a few or none."""
    V = x.shape[1]
    for r in range(0, len(x), 9):
        kind = r // 9 % 7
        if kind == 0:
            x[r] = 0.25
        elif kind == 1:
            x[r, rng.integers(0, V)] = np.nan
        elif kind == 2:
            x[r] = -np.inf
        elif kind == 3:
            x[r, rng.integers(0, V)] = np.inf
        elif kind == 4:
            keep = rng.permutation(V)[:min(V, 10)]
            some = x[r, keep].copy()
            x[r] = -np.inf
            x[r, keep] = some
        elif kind == 5:
            x[r, rng.random(V) < 0.5] = -np.inf
        else:
            x[r] = rng.integers(-2, 3, V)
    return x


@pytest.mark.parametrize("V,k,layout", [(4099, 32, "dense"), (4099, 5, "offset"),
                                        (5003, 20, "padded"), (16001, 20, "dense"),
                                        (16001, 5, "offset"), (50257, 5, "dense")])
def test_a_cta_takes_many_rows(dev, V, k, layout):
    # the persistent kernel: 16 rows a CTA (8 a team) and a few more, so that
    # every slot, barrier phase and list is used again several times; 50257: 5
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    rows = (16 if V < 50000 else 5) * sms + 5
    rng = np.random.default_rng(V + k)
    x = special_rows((2 * rng.standard_normal((rows, V), dtype=F)), rng)
    y = rng.integers(0, V, rows)
    y[::11] = -1
    check(x, y, k, layout)
    assert detlib.det_watchdog_status() == 0


@pytest.mark.parametrize("rows,V", [(12001, 300), (12001, 20), (10007, 1500), (70003, 7)])
def test_a_warp_takes_many_rows(dev, rows, V):
    # more rows than the short rows' kernel has warps; 70003: more than the
    # gradient's grid has rows
    rng = np.random.default_rng(V)
    x = special_rows((2 * rng.standard_normal((rows, V), dtype=F)), rng)
    y = rng.integers(0, V, rows)
    y[::13] = -1
    check(x, y, min(V, 20), "padded")


@pytest.mark.parametrize("rows", [3, 700])
def test_long_rows_captured(dev, rows):
    # over clusters (3 rows) and over persistent CTAs
    rng = np.random.default_rng(rows)
    V = 20011
    x = (2 * rng.standard_normal((rows, V))).astype(F)
    y = rng.integers(0, V, rows).astype(np.int32)
    want = oracle.logprob(x, y, 6)
    xd, yd = to_dev(x), on_gpu(y)
    outs = [torch.empty_like(t) for t in detlib.detlogprob_f32(xd, yd, top_k=6)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        detlib.detlogprob_f32(xd, yd, top_k=6, logp=outs[0], entropy=outs[1], top_ids=outs[2],
                              top_logp=outs[3], stats=outs[4])
    for flip in (True, False, True):
        xd.copy_(to_dev(x[::-1].copy() if flip else x))
        yd.copy_(on_gpu(y[::-1].copy() if flip else y))
        for o in outs:
            o.fill_(7)
        g.replay()
        step = -1 if flip else 1
        for o, w in ((0, 0), (1, 1), (3, 4), (4, 2)):
            assert_bitwise(host(outs[o]), np.ascontiguousarray(want[w][::step]))
        assert np.array_equal(host(outs[2]), want[3][::step])


@pytest.mark.parametrize("V,rows", [(2, None), (30, None), (256, None), (300, None), (1023, None),
                                    (1500, None), (4096, None), (4099, None), (5003, 6),
                                    (50257, 2)])
@pytest.mark.parametrize("layout", ["dense", "offset"])
def test_exps_at_the_ties_of_their_rounding(dev, V, rows, layout):
    # rows [0, d, d, ...]: at these d the exp's integer n is d log2 e rounded to a
    # float and then to an integer; rounded once, it is another one, and e and
    # with it S and T move by a step
    d = exp_tie_arguments(-127, 0)
    x = np.repeat(d[:, None], V, 1)
    x[:, 0] = 0.0
    y = np.ones(len(d), np.int32)
    want = oracle.logprob(x, y, 1)
    for r0 in range(0, len(d), rows or len(d)):
        part = slice(r0, r0 + (rows or len(d)))
        logp, ent, _, _, stats = detlib.detlogprob_f32(to_dev(x[part], layout), on_gpu(y[part]))
        for got, w, name in ((logp, want[0], "logp"), (ent, want[1], "entropy"),
                             (stats, want[2], "stats")):
            assert_bitwise(host(got), w[part], f"{name} of rows from {r0}")


def test_every_float_below_0_in_short_rows(dev):
    # rows [0, d, d, d, -inf ..., d, d, d, d, -inf ...]: one lane forms all seven exps,
    # in its groups 0 and 32, for every d in [-104, -2^-26]; what S and T are then is
    # formed from detexp_f32 and detlog_f32 (themselves tested on every float)
    lo, hi = (int(np.array(v, F).view(np.uint32)) for v in (-2.0 ** -26, -104.0))
    step = 1 << 22
    x = torch.full((step, 256), -np.inf, device="cuda")
    x[:, 0] = 0.0
    y = torch.ones(step, dtype=torch.int32, device="cuda")
    for at in range(lo, hi + 1, step):
        d = torch.arange(at, at + step, device="cuda").int().view(torch.float32)
        x[:, 1:4] = d[:, None]
        x[:, 128:132] = d[:, None]
        logp, ent, _, _, _ = detlib.detlogprob_f32(x, y, want_stats=False)
        e = detlib.detexp_f32(d)
        t = e * d
        S = (((1.0 + e) + e) + e) + (((e + e) + e) + e)
        T = ((t + t) + t) + (((t + t) + t) + t)
        log_s = detlib.detlog_f32(S)
        for got, w, name in ((logp, d - log_s, "logp"), (ent, log_s - T / S, "entropy")):
            diff = got.view(torch.int32) != w.view(torch.int32)
            assert not diff.any(), (name, int(diff.sum()), d[diff][:5].tolist())


def test_gradient_at_the_ties_of_the_exps_rounding(dev):
    # rows [0, every such d, -inf ...]: the probabilities one by one
    d = exp_tie_arguments(-127, 0)
    for V in (len(d) + 1, 5003):
        x = np.full((3, V), -np.inf, F)
        x[:, 0] = 0.0
        for r in range(3):
            x[r, 1:len(d) + 1] = np.roll(d, r)
        check(x, np.array([-1, 0, 7]), 20, "offset")
