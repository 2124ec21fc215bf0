"""The order of the RMSNorm backward's two kernels, which overlap: dx in place over dy is
written only once the columns have read dy, at sizes where rows and columns run at once; and
the next overlapping kernel finds both complete."""
import numpy as np
import pytest

from bitcmp import assert_bitwise
from bitwise_reproducible_fp32_gb300 import detlib
from gpu_util import host, need_gpu, to_dev, torch
from test_gpu_rmsnorm_bwd import case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return need_gpu()


@pytest.mark.parametrize("rows,D", [(8192, 768), (20000, 256), (256, 2048), (5000, 2560)])
def test_dx_in_place_while_the_columns_read(dev, rows, D):
    x, g, r, dy = (to_dev(a) for a in case(rows, D, 8))
    dx, dgain = detlib.detrmsnorm_bwd_f32(x, g, r, dy)
    want = host(dx), host(dgain)
    for _ in range(20):
        both = dy.clone()
        dx, dgain = detlib.detrmsnorm_bwd_f32(x, g, r, both, dx=both)
        assert_bitwise(host(dgain), want[1], "dgain")
        assert_bitwise(host(dx), want[0], "dx")


@pytest.mark.parametrize("rows", [256, 64, 600])
def test_the_next_kernel_finds_the_columns_complete(dev, rows):
    # what the columns read is written, and dgain read, by kernels that overlap their
    # predecessors' ends
    D = 4096
    x, g, r, dy = (to_dev(a) for a in case(rows, D, 9))
    dx, dgain = detlib.detrmsnorm_bwd_f32(x, g, r, dy)
    want = host(dgain).copy()
    normed = host(detlib.detrmsnorm_f32(dx, dgain, 1e-6)[0])
    for _ in range(50):
        xs, out = x.clone(), torch.full((D,), float("nan"), device="cuda")
        dx, dgain = detlib.detrmsnorm_bwd_f32(xs, g, r, dy, dgain=out)
        y, _ = detlib.detrmsnorm_f32(dx, dgain, 1e-6, y=xs)
        assert_bitwise(host(dgain), want, "dgain")
        assert_bitwise(host(y), normed, "the RMSNorm after it")
