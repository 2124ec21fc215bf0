"""The entry points for several answers of a prompt refuse bad arguments on the
host (no GPU)."""
import ctypes

import pytest

from bitwise_reproducible_fp32_gb300 import build, detlib
from test_generation_args import cache, prof

D, E = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x9000)
N = ctypes.c_void_p()


@pytest.fixture(scope="module")
def lib():
    build.build()
    return detlib.load()


def beams(n=4, scores=0x1000, finished=0x2000, lens=0x3000, hist=0x4000, ldh=8):
    return ctypes.byref(detlib.BeamsArg(n, scores, finished, lens, hist, ldh))


def after(**kw):
    return beams(**{**dict(scores=0x11000, finished=0x12000, lens=0x13000, hist=0x14000), **kw})


def test_other_profiles_are_refused(lib):
    p = prof(xent_lanes=128)
    n = ctypes.c_size_t()
    assert lib.detbeam_select_f32(p, 1, beams(), after(), 8, D, D, 0, N, 0, 8, D, D, D, N, N) == 2
    assert lib.detpages_fork(p, 1, 1, 16, 8, D, D, D, 4, 4, E, 4, D, 8, D, E, E, E, E, E, N, N) == 2
    assert lib.detpages_compact(p, 1, 16, 8, D, D, 4, 4, E, 4, D, E, D, D, 4, E, N, N) == 2
    assert lib.detkv_copy_f32(p, 1, D, D, N, N, cache(), N, N) == 2
    for group in (0, 2):
        assert lib.detdecode_attention_shared_f32(p, 2, group, 2, D, 128, cache(), D, 4, 4, D, 1.0,
                                                  D, 128, D, 1 << 20, N, N) == 2
        assert lib.detdecode_attention_shared_workspace_bytes(p, 2, group, 2, 2, 64, 64,
                                                              ctypes.byref(n)) == 2


def test_select_refusals(lib):
    f = lambda R=2, i=beams(), o=after(), k=8, ids=D, lp=D, w=N, wn=0, cols=8, tok=D, par=D: \
        lib.detbeam_select_f32(prof(), R, i, o, k, ids, lp, 5, w, wn, cols, tok, par, D, N,
                               N)  # noqa: E731
    for kw in (dict(R=-1), dict(R=2 ** 29), dict(R=2 ** 62), dict(i=None), dict(o=None),
               dict(i=beams(0)),
               dict(i=beams(33)), dict(o=after(n=0)), dict(o=after(n=33)), dict(k=0), dict(k=33),
               dict(ids=N), dict(lp=N), dict(tok=N), dict(par=N), dict(w=D, wn=0),
               dict(cols=-1), dict(i=beams(ldh=7)), dict(o=after(ldh=7)),
               dict(i=beams(hist=None)), dict(o=after(hist=None)), dict(i=beams(lens=None)),
               dict(i=beams(scores=None)), dict(o=after(scores=None)), dict(o=after(scores=0x1000)),
               dict(o=after(finished=0x2000)), dict(o=after(lens=0x3000)),
               dict(o=after(hist=0x4000)),
               dict(i=beams(lens=None, hist=None), o=after(lens=None, hist=None), w=D, wn=4),
               dict(i=beams(lens=None, hist=None), o=after(hist=None))):
        assert f(**kw) == 1, kw
    assert f(R=0, ids=N, lp=N, tok=N, par=N) == 0


def test_fork_refusals(lib):
    f = lambda B=2, Bo=3, ps=16, P=8, lens=D, par=D, t=D, mp=4, ldt=4, to=E, ldo=4, free=D, cap=8, \
        cnt=D, lo=E, co=E, src=E, dst=E, tok=E: \
        lib.detpages_fork(prof(), B, Bo, ps, P, lens, par, t, mp, ldt, to, ldo, free, cap, cnt, lo,
                          co, src, dst, tok, N, N)  # noqa: E731
    for kw in (dict(B=-1), dict(B=8193), dict(Bo=-1), dict(Bo=8193), dict(ps=0), dict(P=-1),
               dict(P=2 ** 23 + 1), dict(lens=N), dict(par=N), dict(t=N), dict(mp=0), dict(ldt=3),
               dict(to=N), dict(to=D), dict(ldo=3), dict(free=N), dict(cap=-1), dict(cnt=N),
               dict(lo=N), dict(lo=D), dict(co=N), dict(co=D), dict(src=N), dict(dst=N),
               dict(tok=N)):
        assert f(**kw) == 1, kw


def test_compact_refusals(lib):
    f = lambda B=2, ps=16, P=9, lens=D, t=D, mp=4, ldt=4, to=E, ldo=4, free=D, co=E, src=E, dst=E, \
        mm=4, mv=E: lib.detpages_compact(prof(), B, ps, P, lens, t, mp, ldt, to, ldo, free, co, src,
                                         dst, mm, mv, N, N)  # noqa: E731
    for kw in (dict(B=-1), dict(B=8193), dict(ps=0), dict(P=-1), dict(P=2 ** 23 + 1), dict(lens=N),
               dict(t=N), dict(mp=0), dict(ldt=3), dict(to=N), dict(ldo=3), dict(to=D, ldo=5),
               dict(free=N), dict(co=N), dict(src=N), dict(dst=N), dict(mm=3), dict(mv=N)):
        assert f(**kw) == 1, kw


def test_copy_refusals(lib):
    f = lambda n=4, src=D, dst=D, c=cache(): lib.detkv_copy_f32(prof(), n, src, dst, N, N, c, N,
                                                               N)  # noqa: E731
    for kw in (dict(n=-1), dict(n=2 ** 23 + 1), dict(src=N), dict(dst=N), dict(c=None),
               dict(c=cache(k=None)), dict(c=cache(head_dim=257)), dict(c=cache(token_stride=1))):
        assert f(**kw) == 1, kw
    assert f(n=0, src=N, dst=N) == 0


def test_shared_attention_refusals(lib):
    f = lambda B=2, gr=2, H=4, q=D, ldq=256, c=cache(), t=D, mp=4, ldt=4, lens=D, out=D, ldo=256, \
        ws=D, wsn=1 << 40: lib.detdecode_attention_shared_f32(
            prof(), B, gr, H, q, ldq, c, t, mp, ldt, lens, 0.125, out, ldo, ws, wsn, N,
            N)  # noqa: E731
    for kw in (dict(B=-1), dict(B=65536), dict(gr=0), dict(gr=-3), dict(H=0), dict(H=3), dict(q=N),
               dict(ldq=255), dict(c=None), dict(c=cache(head_dim=300)), dict(t=N), dict(mp=0),
               dict(ldt=3), dict(mp=1 << 27, ldt=1 << 27), dict(lens=N), dict(out=N),
               dict(ldo=255)):
        assert f(**kw) == 1, kw
    assert f(B=0, q=N, t=N, lens=N, out=N, ws=N, wsn=0) == 0
    n = ctypes.c_size_t()
    w = lambda B, gr, H, G, d, m: lib.detdecode_attention_shared_workspace_bytes(  # noqa: E731
        prof(), B, gr, H, G, d, m, ctypes.byref(n))
    assert w(2, 0, 4, 2, 64, 9) == 1 and w(2, 2, 4, 3, 64, 9) == 1 and w(2, 2, 4, 2, 64, 0) == 1
    assert lib.detdecode_attention_shared_workspace_bytes(prof(), 2, 2, 4, 2, 64, 9, None) == 1
    assert w(2, 2, 4, 2, 64, 1 << 20) == 0 and n.value > 0
    big = dict(mp=1 << 16, ldt=1 << 16)
    assert f(ws=N, wsn=0, **big) == 5 and f(wsn=n.value - 1, **big) == 5
    assert f(ws=ctypes.c_void_p(0x1008), **big) == 5


def test_the_binding_refuses_cpu_tensors_and_shapes(lib):
    import torch
    x, i = torch.zeros(2, 4), torch.zeros(8, dtype=torch.int32)
    c, t = torch.zeros(2, 2, 2, 2), torch.zeros(8, 1, dtype=torch.int32)
    for call in (lambda: detlib.detbeam_select_f32(x, t, t.float(), 4),
                 lambda: detlib.detpages_fork(i, i, t, i, i[:1], 16, 8),
                 lambda: detlib.detpages_compact(i, t, i, 16),
                 lambda: detlib.detkv_copy_f32(c, c, i, i),
                 lambda: detlib.detdecode_attention_shared_f32(x, c, c, t[:2], i[:2], 2, 2)):
        with pytest.raises(TypeError):
            call()


def decoder(**kw):
    """A decoder's state on the CPU, as far as refusals look at it."""
    import torch

    from bitwise_reproducible_fp32_gb300.decode import Decoder
    dec = Decoder.__new__(Decoder)
    at = dict(B=4, pages=16, page_size=4, top_k=4, device="cpu", forked=False,
              lens=torch.zeros(4, dtype=torch.int32), table=torch.zeros(4, 4, dtype=torch.int32))
    dec.__dict__.update({**at, **kw})
    return dec


@pytest.mark.parametrize("forked", [False, True])
def test_release_refuses_other_flags(lib, forked):
    import torch
    dec = decoder(forked=forked)
    for done in ([1, 0, 0, 0], True, torch.ones(4), torch.ones(4, dtype=torch.bool),
                 torch.ones(4, dtype=torch.int32)):
        with pytest.raises(TypeError, match="done must be a CUDA tensor"):
            dec.release(done)


def test_beam_search_refuses_before_it_takes_pages(lib):
    import torch
    dec = decoder()
    dec.prefill = lambda *a: pytest.fail("pages were taken")
    for error, kw in ((TypeError, dict(weights=torch.ones(4))), (TypeError, dict(weights=[1.0])),
                      (ValueError, dict(eos=1 << 31)), (ValueError, dict(eos=(-1 << 31) - 1)),
                      (TypeError, dict(eos="end"))):
        with pytest.raises(error):
            dec.beam_search([[1, 2]], 3, 2, **kw)
    dec.pages = (1 << 23) + 1
    for call in (lambda: dec.beam_search([[1, 2]], 2, 2), lambda: dec.fork(dec.lens), dec.compact):
        with pytest.raises(ValueError, match="caches of up to 8388608 pages"):
            call()
    assert not dec.forked
