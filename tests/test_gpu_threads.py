"""Calls of the C ABI from two host threads at once, each on a stream of its own, of
sizes whose launches of one kernel take different amounts of shared memory: every
call runs, with the bits of a call alone."""
import ctypes
import threading

import numpy as np
import pytest

from bitcmp import assert_bitwise
from bitwise_reproducible_fp32_gb300 import detlib
from gpu_util import host, need_gpu, to_dev, torch

pytestmark = pytest.mark.gpu
F = np.float32


@pytest.fixture(scope="module")
def dev():
    return need_gpu()


def job(kind, n, rng):
    """(function, arguments but for the stream, output) of a call of 8 rows of n, and
    what has to stay allocated."""
    lib, prof = detlib.load(), ctypes.byref(detlib.det_profile_default())
    draw = lambda *s: to_dev(rng.standard_normal(s).astype(F))  # noqa: E731
    x, b, y, inv, g = draw(8, n), draw(8, n), draw(8, n), draw(8), draw(n)
    p = lambda t: t.data_ptr()                                  # noqa: E731
    eps, one = ctypes.c_float(1e-6), ctypes.c_float(1.0)
    keep = [prof, x, b, y, inv, g]
    if kind == "rmsnorm":
        return lib.detrmsnorm_f32, (prof, 8, n, p(x), n, p(g), eps, p(y), n, p(inv)), y, keep
    if kind == "add_rmsnorm":
        s = draw(8, n)
        keep.append(s)
        return (lib.detadd_rmsnorm_f32, (prof, 8, n, p(x), p(b), p(s), p(g), eps, p(y), n,
                                         p(inv)), y, keep)
    if kind == "rmsnorm_bwd":
        detlib.detrmsnorm_f32(x, g, 1e-6, inv_rms=inv)
        need = detlib.detrmsnorm_bwd_workspace_bytes(8, n)
        dgain, ws = draw(n), draw((need + 3) // 4 + 1)
        keep += [dgain, ws]
        return (lib.detrmsnorm_bwd_f32, (prof, 8, n, p(x), n, p(g), p(inv), p(b), n, p(y), n,
                                         p(dgain), p(ws), ws.numel() * 4), y, keep)
    lab = torch.zeros(8, dtype=torch.int32, device="cuda")
    keep.append(lab)
    return (lib.detxent_f32, (prof, 8, n, p(x), n, p(lab), p(inv), None, p(y), n, one, None), y,
            keep)


@pytest.mark.parametrize("first,second,sizes", [
    ("rmsnorm", "rmsnorm", (64, 768)), ("rmsnorm", "add_rmsnorm", (64, 768)),
    ("rmsnorm_bwd", "rmsnorm_bwd", (768, 1024)), ("xent", "xent", (2048, 24576)),
    ("xent", "xent", (20000, 50257))])
def test_two_threads_at_once(dev, first, second, sizes):
    rng = np.random.default_rng(31)
    jobs = [job(kind, n, rng) for kind, n in zip((first, second), sizes)]
    want = []
    for call, args, out, _ in jobs:
        assert call(*args, None) == 0
        want.append(host(out))
        out.zero_()
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    failed, start = [0, 0], threading.Barrier(2)

    def work(i):
        call, args, _, _ = jobs[i]
        stream = streams[i].cuda_stream
        start.wait()
        failed[i] = sum(call(*args, stream) != 0 for _ in range(20000))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert failed == [0, 0]
    for (_, _, out, _), w in zip(jobs, want):
        assert_bitwise(host(out), w)
