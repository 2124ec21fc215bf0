"""GPU parity (0 ULP) of the rotary embedding at given positions and of the
append to a paged cache against the oracle; both against the formula in 64
bits; layouts, strides, padding, shared slots, far positions, streams."""
import numpy as np
import pytest

import oracle
from bitcmp import assert_bitwise
from bitwise_reproducible_fp32_gb300 import detlib
from gen_util import F, LAYOUTS, U, make_cache, rotate64, turns_of
from gpu_util import host, need_gpu, to_dev, torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return need_gpu()


def on_gpu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def dev_turns(t):
    return on_gpu(t.view(np.int64))


@pytest.mark.parametrize("rows,heads,d", [(1, 1, 2), (5, 3, 16), (64, 12, 64), (33, 7, 80),
                                          (300, 24, 64), (7, 2, 10), (2, 70, 128)])
@pytest.mark.parametrize("layout", ["dense", "padded", "offset"])
@pytest.mark.parametrize("half", [False, True])
def test_theta_angles_match_the_oracle(dev, rows, heads, d, layout, half):
    rng = np.random.default_rng(rows * 100 + d)
    x = rng.standard_normal((rows, heads * d)).astype(F)
    pos = rng.integers(-1, 2048, rows).astype(np.int32)
    for rot in {d, max(2, d // 4 * 2)}:
        for inverse in (False, True):
            want = oracle.rope_at(x, pos, heads, d, rot=rot, half=half, inverse=inverse)
            got = detlib.detrope_at_f32(to_dev(x, layout), on_gpu(pos), heads, d, rot_dim=rot,
                                        half=half, inverse=inverse)
            assert_bitwise(host(got), want, f"rot={rot} inverse={inverse}")
            xd = to_dev(x, layout)
            detlib.detrope_at_f32(xd, on_gpu(pos), heads, d, rot_dim=rot, half=half,
                                  inverse=inverse, out=xd)
            assert_bitwise(host(xd), want, "in place")


def test_bits_of_the_training_rotary(dev):
    # 2 sequences of 300: the positions t mod seq_len, forward and backward
    rng = np.random.default_rng(7)
    x = rng.standard_normal((600, 6 * 64)).astype(F)
    pos = on_gpu((np.arange(600) % 300).astype(np.int32))
    a, b = to_dev(x), to_dev(x)
    assert_bitwise(host(detlib.detrope_at_f32(a, pos, 6, 64)),
                   host(detlib.detrope_f32(b, 6, 64, 300)))
    b = to_dev(x)
    assert_bitwise(host(detlib.detrope_at_f32(a, pos, 6, 64, inverse=True)),
                   host(detlib.detrope_bwd_f32(b, 6, 64, 300)))


@pytest.mark.parametrize("d,rot,half", [(64, 64, False), (64, 32, True), (128, 64, True),
                                        (80, 20, False), (24, 12, True), (6, 2, False)])
@pytest.mark.parametrize("longest", [1, 4096, 2 ** 31 - 1])
def test_turns_oracle_and_formula(dev, d, rot, half, longest):
    rng = np.random.default_rng(d + rot)
    heads, rows = 5, 70
    x = rng.standard_normal((rows, heads * d)).astype(F)
    pos = rng.integers(0, longest, rows).astype(np.int32)
    pos[3], pos[-1] = -1, longest - 1
    t = turns_of(rot, factor=4.0 if longest > 4096 else 1.0)
    for inverse in (False, True):
        got = host(detlib.detrope_at_f32(to_dev(x), on_gpu(pos), heads, d, turns=dev_turns(t),
                                         half=half, inverse=inverse))
        assert_bitwise(got, oracle.rope_at(x, pos, heads, d, turns=t, rot=rot, half=half,
                                           inverse=inverse))
        want = rotate64(x, pos, t, heads, d, half, inverse)
        # r is off by at most 3 U pi/4 and the polynomials by a step (2 U): sin
        # and cos by 5 U; two products and a sum: 2 U more of |x0| + |x1|
        pair = np.abs(x.reshape(rows, heads, d)).max(2)[..., None] * 2
        err = np.abs(got - want).reshape(rows, heads, d)
        assert (err <= 7 * U * pair).all(), (err / pair).max() / U


def test_angles_of_every_quadrant_and_border(dev):
    # phases on and next to the quarter-turn borders: position 1, turns = phase
    q = np.arange(8, dtype=np.uint64) << np.uint64(61)
    phases = np.concatenate([q - np.uint64(1), q, q + np.uint64(1)])
    x = np.random.default_rng(1).standard_normal((4, 2 * phases.size)).astype(F)
    pos = np.array([1, 0, 3, 2 ** 31 - 1], np.int32)
    got = detlib.detrope_at_f32(to_dev(x), on_gpu(pos), 1, 2 * phases.size,
                                turns=dev_turns(phases))
    assert_bitwise(host(got), oracle.rope_at(x, pos, 1, 2 * phases.size, turns=phases,
                                             rot=2 * phases.size))
    assert np.abs(host(got) - rotate64(x, pos, phases, 1, 2 * phases.size)).max() <= \
        7 * U * 2 * np.abs(x).max()


def test_columns_past_the_heads_stay(dev):
    rng = np.random.default_rng(3)
    x = rng.standard_normal((9, 200)).astype(F)
    pos = np.arange(9, dtype=np.int32)
    xd = to_dev(x)
    detlib.detrope_at_f32(xd, on_gpu(pos), 2, 64, out=xd)
    assert_bitwise(host(xd)[:, 128:], x[:, 128:])
    assert detlib.detrope_at_f32(xd[:0], on_gpu(pos[:0]), 2, 64).shape == (0, 128)


def test_gradient_against_differences(dev):
    # f(x) = sum(w * y(x)) is linear, so the backward of w is its gradient: the
    # difference quotient with step 1 along each axis, in 64 bits
    rng = np.random.default_rng(5)
    d, t = 16, turns_of(8)
    x, w = (rng.standard_normal((3, d)).astype(F) for _ in range(2))
    pos = np.array([0, 77, 100003], np.int32)
    dx = host(detlib.detrope_at_f32(to_dev(w), on_gpu(pos), 1, d, turns=dev_turns(t), half=True,
                                    inverse=True))
    for i in range(d):
        step = np.zeros_like(x, dtype=np.float64)
        step[:, i] = 1.0
        hi, lo = (rotate64(x + s, pos, t, 1, d, half=True) for s in (step, 0 * step))
        quot = (w * (hi - lo)).sum(1)
        assert (np.abs(dx[:, i] - quot) <= 7 * U * 2 * np.abs(w).max(1) + 1e-14 * 16).all()


# ---------------------------------------------------------------- append
def append_oracle(qkv, slots, pos, H, G, d, nslots, turns, rot, half, k, v, q):
    """numpy statement of the append, rows in order (the last of a slot stays)."""
    n = len(qkv)
    turned = qkv[:, :(H + G) * d]
    if pos is not None:
        turned = oracle.rope_at(turned, pos, H + G, d, turns=turns, rot=rot, half=half)
    X, Y = turned.reshape(n, H + G, d), qkv.reshape(n, H + 2 * G, d)
    for t in range(n):
        if slots[t] < 0 or slots[t] >= nslots or (pos is not None and pos[t] < 0):
            continue
        k[slots[t]], v[slots[t]] = X[t, H:], Y[t, H + G:]
        if q is not None:
            q[t] = X[t, :H].ravel()


@pytest.mark.parametrize("rows,H,G,d,ps", [(1, 1, 1, 64, 16), (16, 4, 4, 16, 16),
                                           (64, 12, 12, 64, 16), (100, 8, 2, 128, 64),
                                           (37, 3, 1, 80, 5), (5, 2, 2, 7, 3), (9, 6, 3, 10, 1),
                                           (600, 4, 2, 256, 100)])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("mode", ["plain", "theta", "turns", "half"])
def test_append(dev, rows, H, G, d, ps, layout, mode):
    if d % 2 and mode != "plain":
        rot = d - 1
    else:
        rot = d
    rng = np.random.default_rng(rows + d)
    pages = -(-rows // ps) + 3
    n = pages * ps
    qkv = rng.standard_normal((rows, (H + 2 * G) * d)).astype(F)
    slots = rng.permutation(n)[:rows].astype(np.int64)
    pos = rng.integers(0, 5000, rows).astype(np.int32)
    if rows > 4:
        slots[1], pos[2] = -1, -1
        slots[4] = slots[rows - 1]                  # shared: the last row stays
        slots[0] = n + 3                            # out of range
    half = mode == "half" and rot % 2 == 0
    t = turns_of(rot) if mode in ("turns", "half") else None
    p = None if mode == "plain" else pos
    k, v = (np.full((n, G, d), np.nan, F) for _ in range(2))
    q = np.full((rows, H * d), 5.0, F)
    append_oracle(qkv, slots, p, H, G, d, n, t, rot, half, k, v, None if p is None else q)
    kc, vc = make_cache(pages, ps, G, d, layout)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    qd = to_dev(np.full((rows, H * d), 5.0, F))
    kw = {} if p is None else dict(positions=on_gpu(p), rot_dim=rot, half=half, q_out=qd,
                                   turns=None if t is None else dev_turns(t))
    src = to_dev(qkv, "offset" if layout == "offset" else "padded")
    out = detlib.detkv_append_f32(src, on_gpu(slots), kc, vc, H, dev_status=status, **kw)
    assert_bitwise(host(kc).reshape(n, G, d), k, "keys")
    assert_bitwise(host(vc).reshape(n, G, d), v, "values")
    assert_bitwise(host(src), qkv, "the rows stay")
    assert (out is None) == (p is None)
    if p is not None:
        assert_bitwise(host(qd), q, "queries")
    assert int(status) == (1 if rows > 4 else 0)


def test_append_turns_q_in_place(dev):
    rng = np.random.default_rng(11)
    H, G, d, rows = 4, 2, 32, 20
    qkv = rng.standard_normal((rows, (H + 2 * G) * d)).astype(F)
    pos = np.arange(rows, dtype=np.int32) * 7
    kc, vc = make_cache(2, 16, G, d)
    src = to_dev(qkv)
    out = detlib.detkv_append_f32(src, on_gpu(np.arange(rows, dtype=np.int64)), kc, vc, H,
                                  positions=on_gpu(pos))
    want = oracle.rope_at(qkv[:, :H * d], pos, H, d)
    assert out.data_ptr() == src.data_ptr() and out.shape == (rows, H * d)
    assert_bitwise(host(out), want)
    assert_bitwise(host(src)[:, H * d:], qkv[:, H * d:])


def test_append_all_rows_to_one_slot(dev):
    # 5000 rows name slot 3: the cache holds the last one, every time
    rng = np.random.default_rng(12)
    G, d, rows = 2, 64, 5000
    qkv = rng.standard_normal((rows, 3 * G * d)).astype(F)
    slots = on_gpu(np.full(rows, 3, np.int64))
    for _ in range(3):
        kc, vc = make_cache(1, 16, G, d)
        detlib.detkv_append_f32(to_dev(qkv), slots, kc, vc, G)
        assert_bitwise(host(kc)[0, 3].ravel(), qkv[-1, G * d:2 * G * d])
        assert_bitwise(host(vc)[0, 3].ravel(), qkv[-1, 2 * G * d:])
        assert np.isnan(np.delete(host(kc)[0], 3, 0)).all()


def test_append_past_32_bit_offsets(dev):
    # a cache of 2.3e9 floats: slots whose offsets pass 2^31 and 2^32 bytes
    G, d, ps = 8, 128, 64
    pages = 35_000
    kc = torch.zeros((pages, ps, G, d), device="cuda")
    vc = torch.zeros((pages, ps, G, d), device="cuda")
    rng = np.random.default_rng(13)
    slots = np.array([pages * ps - 1, 2 ** 31 // (G * d), 2 ** 20 - 1], np.int64)
    qkv = rng.standard_normal((3, 3 * G * d)).astype(F)
    detlib.detkv_append_f32(to_dev(qkv), on_gpu(slots), kc, vc, G)
    for i, s in enumerate(slots):
        assert_bitwise(host(kc[s // ps, s % ps]).ravel(), qkv[i, G * d:2 * G * d])
        assert_bitwise(host(vc[s // ps, s % ps]).ravel(), qkv[i, 2 * G * d:])
    assert int((kc != 0).any(-1).sum()) == 3 * G


def test_on_another_stream_and_captured(dev):
    rng = np.random.default_rng(14)
    x = rng.standard_normal((50, 256)).astype(F)
    pos = np.arange(50, dtype=np.int32)
    want = oracle.rope_at(x, pos, 4, 64)
    s = torch.cuda.Stream()
    xd, pd = to_dev(x), on_gpu(pos)
    s.wait_stream(torch.cuda.current_stream())
    got = detlib.detrope_at_f32(xd, pd, 4, 64, stream=s)
    s.synchronize()
    assert_bitwise(host(got), want)
    out = torch.empty_like(xd)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        detlib.detrope_at_f32(xd, pd, 4, 64, out=out)
    xd.copy_(to_dev(2 * x))
    g.replay()
    assert_bitwise(host(out), oracle.rope_at(2 * x, pos, 4, 64))


@pytest.mark.parametrize("rows", [1, 2])
def test_in_place_on_the_first_columns(dev, rows):
    # out (q_out) is a view of the rows' first columns: one row as well as several
    rng = np.random.default_rng(15)
    H, G, d = 4, 2, 32
    qkv = rng.standard_normal((rows, (H + 2 * G) * d)).astype(F)
    pos = np.arange(rows, dtype=np.int32) * 9 + 3
    want = oracle.rope_at(qkv[:, :H * d], pos, H, d)
    src = to_dev(qkv)
    view = src[:, :H * d]
    assert detlib.detrope_at_f32(src, on_gpu(pos), H, d, out=view) is view
    assert_bitwise(host(view), want)
    assert_bitwise(host(src)[:, H * d:], qkv[:, H * d:], "the other columns stay")
    src = to_dev(qkv)
    view = src[:, :H * d]
    kc, vc = make_cache(1, 16, G, d)
    out = detlib.detkv_append_f32(src, on_gpu(np.arange(rows, dtype=np.int64)), kc, vc, H,
                                  positions=on_gpu(pos), q_out=view)
    assert out is view
    assert_bitwise(host(view), want)
    assert_bitwise(host(src)[:, H * d:], qkv[:, H * d:], "keys and values stay")
    assert_bitwise(host(kc)[0, :rows].reshape(rows, -1),
                   oracle.rope_at(qkv[:, H * d:(H + G) * d], pos, G, d))
    assert_bitwise(host(vc)[0, :rows].reshape(rows, -1), qkv[:, (H + G) * d:])
