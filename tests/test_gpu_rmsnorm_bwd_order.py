"""The order of the RMSNorm backward's two kernels, which overlap: dx in place over dy is
written only once the columns have read dy, at sizes where rows and columns run at once."""
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
