"""The give-up path of the RMSNorm backward's row kernel, run on a GPU without a fault: in
a copy of the library every CTA gives up on its copies, which are healthy and land. The
call comes back, bit 2 of the watchdog is set, no row is written, and the next call of the
shipped library has its bits."""
import ctypes
import os

import numpy as np
import pytest

from bitcmp import assert_bitwise
from bitwise_reproducible_fp32_gb300 import build, detlib
from gpu_util import host, need_gpu, to_dev, torch
from test_gpu_rmsnorm_bwd import case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def giving_up(tmp_path_factory):
    need_gpu()
    path = os.path.join(str(tmp_path_factory.mktemp("wd")), "libdetfp32_variant.so")
    build.build_variant(["DET_TEST_RMSBWD_GIVE_UP"], path, ["rmsbwd.cu"])
    lib = ctypes.CDLL(path)
    for name, res, args in detlib.SIGNATURES:
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


@pytest.mark.parametrize("rows,D", [(1, 64), (300, 768), (2000, 1024)])
def test_copies_that_are_given_up_on_are_reported(giving_up, monkeypatch, rows, D):
    x, g, r, dy = (to_dev(a) for a in case(rows, D, 7))
    dgain = torch.empty(D, device="cuda")
    want = host(detlib.detrmsnorm_bwd_f32(x, g, r, dy, dgain=dgain)[0])
    assert detlib.det_watchdog_status(clear=True) == 0
    dx = torch.full_like(x, float("nan"))
    with monkeypatch.context() as m:
        m.setattr(detlib, "_lib", giving_up)
        detlib.detrmsnorm_bwd_f32(x, g, r, dy, dx=dx, dgain=dgain)
        torch.cuda.synchronize()
        assert detlib.det_watchdog_status(clear=True) == 4
        assert detlib.det_watchdog_status() == 0
    assert np.isnan(host(dx)).all()
    got = host(detlib.detrmsnorm_bwd_f32(x, g, r, dy, dgain=dgain)[0])
    assert_bitwise(got, want, "the shipped library afterwards")
    assert detlib.det_watchdog_status() == 0
