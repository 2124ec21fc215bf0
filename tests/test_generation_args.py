"""The generation entry points refuse bad arguments on the host (no GPU), and
the rotary frequencies' helper; the oracle's new functions against 64 bits."""
import ctypes
import math

import numpy as np
import pytest

import oracle
from bitwise_reproducible_fp32_gb300 import build, detlib

F = np.float32
D = ctypes.c_void_p(0x1000)
N = ctypes.c_void_p()


@pytest.fixture(scope="module")
def lib():
    build.build()
    return detlib.load()


def prof(**kw):
    p = detlib.det_profile_default()
    for k, v in kw.items():
        setattr(p, k, v)
    return ctypes.byref(p)


def cache(**kw):
    a = dict(k=0x1000, v=0x2000, num_pages=8, page_size=16, kv_heads=2, head_dim=64,
             page_stride=2048, token_stride=128, head_stride=64)
    a.update(kw)
    return ctypes.byref(detlib.KVCache(**a))


def rotary(rot_dim=64, half=0, theta=1e4):
    return ctypes.byref(detlib.Rotary(rot_dim, half, theta, None))


def test_other_profiles_are_refused(lib):
    p = prof(k_chunk=128)
    assert lib.detrope_at_f32(p, 1, 1, 64, D, 64, D, rotary(), 0, D, 64, N) == 2
    assert lib.detkv_append_f32(p, 1, 2, D, 384, D, D, rotary(), cache(), D, 128, N, N) == 2
    assert lib.detpages_extend(p, 1, 16, D, D, D, 4, 4, D, 8, D, 4, D, D, D, D, D, N, N) == 2
    assert lib.detpages_release(p, 1, 16, D, D, D, 4, 4, D, 8, D, D, D, N, N) == 2
    assert lib.detdecode_attention_f32(p, 1, 2, D, 128, cache(), D, 4, 4, D, 1.0, D, 128, D,
                                       1 << 20, N, N) == 2
    n = ctypes.c_size_t()
    assert lib.detdecode_attention_workspace_bytes(p, 1, 2, 2, 64, 64, ctypes.byref(n)) == 2
    assert lib.detlogprob_f32(p, 1, 8, D, 8, D, 0, D, D, N, N, N, N, N) == 2
    assert lib.detlogprob_bwd_f32(p, 1, 8, D, 8, D, D, D, N, D, 8, N) == 2


def test_rotary_refusals(lib):
    f = lambda rows=4, heads=2, hd=64, x=D, ldx=128, pos=D, ro=rotary(), out=D, ldo=128: \
        lib.detrope_at_f32(prof(), rows, heads, hd, x, ldx, pos, ro, 0, out, ldo, N)  # noqa: E731
    for kw in (dict(rows=-1), dict(heads=0), dict(heads=65537, ldx=1 << 30, ldo=1 << 30),
               dict(hd=0), dict(ldx=127), dict(ldo=127), dict(x=N), dict(pos=N), dict(out=N),
               dict(ro=None), dict(ro=rotary(63)), dict(ro=rotary(66)), dict(ro=rotary(0)),
               dict(ldo=132)):
        assert f(**kw) == 1, kw
    assert f(rows=0, x=N, out=N, pos=N) == 0


def test_append_refusals(lib):
    f = lambda rows=4, heads=2, qkv=D, ld=384, slots=D, pos=D, ro=rotary(), c=cache(), q=D, \
        ldq=384: lib.detkv_append_f32(prof(), rows, heads, qkv, ld, slots, pos, ro, c, q, ldq, N,
                                      N)  # noqa: E731
    for kw in (dict(rows=-1), dict(rows=2 ** 20 + 1), dict(heads=0), dict(qkv=N), dict(ld=383),
               dict(slots=N),
               dict(pos=N), dict(ro=rotary(128)), dict(c=None), dict(ldq=127), dict(ldq=400),
               dict(c=cache(k=None)), dict(c=cache(v=None)), dict(c=cache(num_pages=0)),
               dict(c=cache(page_size=0)), dict(c=cache(kv_heads=0)), dict(c=cache(head_dim=0)),
               dict(c=cache(head_dim=257)), dict(c=cache(page_stride=63)),
               dict(c=cache(token_stride=63)), dict(c=cache(head_stride=0))):
        assert f(**kw) == 1, kw
    assert f(rows=0, qkv=N, slots=N, pos=N) == 0


def test_pages_refusals(lib):
    e = lambda B=2, ps=16, lens=D, new=D, table=D, mp=4, ldt=4, free=D, cap=8, cnt=D, rows=4, \
        lo=ctypes.c_void_p(0x3000), co=ctypes.c_void_p(0x4000), rs=D, pos=D, sl=D: \
        lib.detpages_extend(prof(), B, ps, lens, new, table, mp, ldt, free, cap, cnt, rows, lo,
                            co, rs, pos, sl, N, N)  # noqa: E731
    for kw in (dict(B=-1), dict(B=8193), dict(ps=0), dict(lens=N), dict(new=N), dict(table=N),
               dict(mp=0), dict(ldt=3), dict(free=N), dict(cap=-1), dict(cnt=N), dict(rows=-1),
               dict(lo=N), dict(lo=D), dict(co=N), dict(co=D), dict(rs=N), dict(pos=N),
               dict(sl=N)):
        assert e(**kw) == 1, kw
    r = lambda B=2, ps=16, lens=D, done=D, table=D, mp=4, ldt=4, free=D, cap=8, cnt=D, \
        lo=ctypes.c_void_p(0x3000), co=ctypes.c_void_p(0x4000): \
        lib.detpages_release(prof(), B, ps, lens, done, table, mp, ldt, free, cap, cnt, lo, co, N,
                             N)  # noqa: E731
    for kw in (dict(B=-1), dict(B=8193), dict(ps=0), dict(lens=N), dict(done=N), dict(table=N),
               dict(mp=0), dict(ldt=3), dict(free=N), dict(cap=-1), dict(cnt=N), dict(lo=N),
               dict(lo=D), dict(co=N), dict(co=D)):
        assert r(**kw) == 1, kw


def test_decode_refusals(lib):
    f = lambda B=2, H=4, q=D, ldq=256, c=cache(), t=D, mp=4, ldt=4, lens=D, out=D, ldo=256, ws=D, \
        wsn=1 << 30: lib.detdecode_attention_f32(prof(), B, H, q, ldq, c, t, mp, ldt, lens, 0.125,
                                                 out, ldo, ws, wsn, N, N)  # noqa: E731
    for kw in (dict(B=-1), dict(B=65536), dict(H=0), dict(H=3), dict(q=N), dict(ldq=255),
               dict(c=None), dict(c=cache(head_dim=300)), dict(t=N), dict(mp=0), dict(ldt=3),
               dict(mp=1 << 27, ldt=1 << 27), dict(lens=N), dict(out=N), dict(ldo=255)):
        assert f(**kw) == 1, kw
    assert f(B=0, q=N, t=N, lens=N, out=N, ws=N, wsn=0) == 0
    n = ctypes.c_size_t()
    w = lambda B, H, G, d, m: lib.detdecode_attention_workspace_bytes(  # noqa: E731
        prof(), B, H, G, d, m, ctypes.byref(n))
    assert w(2, 4, 3, 64, 10) == 1 and w(2, 4, 2, 64, 0) == 1 and w(2, 4, 2, 257, 5) == 1
    assert w(2, 4, 2, 64, 1 << 20) == 0
    if n.value:
        big = dict(mp=1 << 16, ldt=1 << 16)
        assert f(ws=N, wsn=0, **big) == 5 and f(wsn=n.value - 1, **big) == 5
        assert f(ws=ctypes.c_void_p(0x1008), **big) == 5


def test_logprob_refusals(lib):
    f = lambda rows=2, V=8, x=D, ld=8, y=D, k=2, lp=D, en=D, st=D, ids=D, top=D: \
        lib.detlogprob_f32(prof(), rows, V, x, ld, y, k, lp, en, st, ids, top, N, N)  # noqa: E731
    for kw in (dict(rows=-1), dict(V=0), dict(V=2 ** 30 + 1, ld=2 ** 31), dict(x=N), dict(ld=7),
               dict(y=N), dict(k=-1), dict(k=9), dict(k=33, V=64, ld=64), dict(lp=N),
               dict(en=N), dict(ids=N), dict(top=N)):
        assert f(**kw) == 1, kw
    assert f(st=ctypes.c_void_p(0x1004)) == 4
    assert f(rows=0, x=N, y=N, lp=N, en=N) == 0
    b = lambda rows=2, V=8, x=D, ld=8, y=D, st=D, g=D, dx=D, ldd=8: \
        lib.detlogprob_bwd_f32(prof(), rows, V, x, ld, y, st, g, N, dx, ldd, N)  # noqa: E731
    for kw in (dict(rows=-1), dict(V=0), dict(x=N), dict(ld=7), dict(y=N), dict(st=N), dict(g=N),
               dict(dx=N), dict(ldd=7), dict(ldd=12)):
        assert b(**kw) == 1, kw
    assert b(st=ctypes.c_void_p(0x1004)) == 4


def test_the_binding_refuses_cpu_tensors(lib):
    import torch
    x, i = torch.zeros(2, 4), torch.zeros(2, dtype=torch.int32)
    c = torch.zeros(2, 2, 2, 2)
    for call in (lambda: detlib.detrope_at_f32(x, i, 1, 4),
                 lambda: detlib.detkv_append_f32(x, i.long(), c, c, 1),
                 lambda: detlib.detpages_extend(i, i, i.view(2, 1), i, i[:1], 4, 4),
                 lambda: detlib.detpages_release(i, i, i.view(2, 1), i, i[:1], 4),
                 lambda: detlib.detdecode_attention_f32(x, c, c, i.view(2, 1), i, 2),
                 lambda: detlib.detlogprob_f32(x, i),
                 lambda: detlib.detlogprob_bwd_f32(x, i, x, x[0])):
        with pytest.raises(TypeError):
            call()


def test_rope_turns(lib):
    t = detlib.rope_turns(64, device="cpu").numpy().view(np.uint64)
    w = 10000.0 ** (-np.arange(0, 64, 2) / 64)
    assert np.allclose(t.astype(np.float64) * 2 * math.pi / 2.0 ** 64, w, rtol=2e-16 * 8)
    s = detlib.rope_turns(64, factor=8.0, device="cpu").numpy().view(np.uint64)
    # each rounded to a whole number: 8 halves and one half apart, plus the
    # doubles' own two roundings
    assert np.allclose(s.astype(np.float64) * 8, t.astype(np.float64), rtol=2 * 2.0 ** -52,
                       atol=4.5)
    # by parts: fast pairs stay, slow ones are stretched, a blend between
    b = detlib.rope_turns(64, factor=8.0, low=1.0, high=4.0, trained=8192,
                          device="cpu").numpy().view(np.uint64)
    r = 8192 * w / (2 * math.pi)
    assert (b[r >= 4] == t[r >= 4]).all() and (b[r <= 1] == s[r <= 1]).all()
    mid = (r > 1) & (r < 4)
    assert mid.any() and (b[mid] < t[mid]).all() and (b[mid] > s[mid]).all()
    for kw in (dict(rot_dim=63), dict(rot_dim=0), dict(factor=0.5), dict(theta=-1.0),
               dict(low=1.0), dict(trained=100), dict(trained=100, low=2.0, high=1.0)):
        with pytest.raises(ValueError):
            detlib.rope_turns(**{"rot_dim": 64, "device": "cpu", **kw})


def test_oracle_log_probabilities_in_64_bits():
    from gen_util import U, logprob64
    rng = np.random.default_rng(2)
    for V in (1, 2, 7, 300, 5000, 50257):
        x = (2 * rng.standard_normal((3, V))).astype(F)
        y = rng.integers(0, V, 3)
        lp, ent, st, ids, top = oracle.logprob(x, y, min(V, 5))
        want, went, b1, b2 = logprob64(x, y)
        assert (np.abs(lp - want) <= b1).all() and (np.abs(ent - went) <= b2).all()
        assert np.array_equal(ids, np.argsort(-x, axis=1, kind="stable")[:, :min(V, 5)])
        loss, _, _ = oracle.xent(x, y.astype(np.int32))
        assert np.array_equal(lp, -loss)
        assert U == 2.0 ** -24


def test_oracle_decode_attention_in_64_bits():
    from gen_util import decode64
    rng = np.random.default_rng(3)
    for n, d in ((1, 1), (5, 16), (257, 64), (2000, 128)):
        q, K, V = (rng.standard_normal(s).astype(F) for s in ((d,), (n, d), (n, d)))
        want, bound = decode64(q, K, V, 1 / math.sqrt(d))
        got = oracle.decode_attention(q, K, V, float(F(1 / math.sqrt(d))))
        assert (np.abs(got - want) <= bound).all()
    assert (oracle.decode_attention(q, K[:0], V[:0], 1.0) == 0).all()


def test_oracle_rotary_in_64_bits():
    from gen_util import U, rotate64, turns_of
    rng = np.random.default_rng(4)
    x = rng.standard_normal((200, 3 * 64)).astype(F)
    pos = rng.integers(-1, 2 ** 31 - 1, 200).astype(np.int32)
    for rot in (64, 32, 2):
        for half in (False, True):
            t = turns_of(rot)
            got = oracle.rope_at(x, pos, 3, 64, turns=t, rot=rot, half=half)
            err = np.abs(got - rotate64(x, pos, t, 3, 64, half)).max(1)
            assert (err <= 7 * U * 2 * np.abs(x).max(1)).all()


def test_a_decoder_refuses_what_its_calls_would(lib):
    from bitwise_reproducible_fp32_gb300.decode import Decoder
    model = dict(heads=4, d=64, dff=172, vocab=20, blocks=[])
    for kw in (dict(max_batch=0), dict(max_batch=8193), dict(max_len=0), dict(max_len=2 ** 20 + 1, pages=9),
               dict(page_size=0),
               dict(top_k=-1), dict(top_k=21), dict(pages=0)):
        with pytest.raises(ValueError):
            Decoder(model, **{"max_batch": 2, "max_len": 16, "device": "cpu", **kw})
    with pytest.raises(ValueError):
        Decoder(dict(model, vocab=256), 2, 16, "cpu", top_k=33)
