"""The give-up path of decode attention's waits for pieces of the cache, run on a GPU
without a fault: in a copy of the library warps give up on one of their first pieces, on
copies that are healthy and land. The call comes back, bit 5 of the watchdog is
set, every value is NaN or right, requests without tokens are 0, and the next call of the
shipped library has its bits."""
import numpy as np
import pytest

from bitcmp import assert_bitwise
from bitwise_reproducible_fp32_gb300 import detlib
from decode_variants import ALONE, GROUPS, TOGETHER, reading
from gen_util import F
from gpu_util import host, need_gpu, to_dev, torch
from test_gpu_shared_attention import on_gpu, shared_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return need_gpu()


# groups of 4 rows a head; groups of 12 with few own rows and with 10 a request (tiles of
# their own); slices of 32 dimensions that are whole and not; rings of two and three pieces
@pytest.mark.parametrize("how,H,G,d,group,prefix", [
    (GROUPS, 4, 4, 64, 4, 1500), (GROUPS, 8, 4, 40, 4, 1500), (TOGETHER, 8, 4, 64, 6, 1500),
    (TOGETHER, 6, 1, 128, 2, 1500), (TOGETHER, 20, 2, 72, 4, 1500), (ALONE, 4, 4, 64, 4, 200),
    (ALONE, 16, 4, 64, 4, 1500), (ALONE, 1, 1, 100, 4, 9000)])
def test_a_wait_that_runs_out_is_reported(dev, how, H, G, d, group, prefix):
    rng = np.random.default_rng(H + d)
    B = 12
    own = rng.integers(1, 700, B)
    kc, vc, table, lens, _, _ = shared_cache([prefix] * (B // group), own, 16, G, d, "token", rng)
    lens[5] = 0
    q, ld = to_dev(rng.standard_normal((B, H * d)).astype(F)), on_gpu(lens)
    want = host(detlib.detdecode_attention_f32(q, kc, vc, table, ld, H))
    assert detlib.det_watchdog_status(clear=True) == 0
    for _ in range(3):
        with reading(how, giving_up=True):
            assert detlib.det_watchdog_status(clear=True) == 0
            got = host(detlib.detdecode_attention_shared_f32(q, kc, vc, table, ld, H, group))
            assert detlib.det_watchdog_status(clear=True) == 32
        gone = np.isnan(got)
        assert gone.any() and not gone[5].any()
        assert_bitwise(got[~gone], want[~gone], "values of the call that gave up")
    for call in (lambda: detlib.detdecode_attention_f32(q, kc, vc, table, ld, H),
                 lambda: detlib.detdecode_attention_shared_f32(q, kc, vc, table, ld, H, group)):
        assert_bitwise(host(call()), want, "the shipped library afterwards")
    assert detlib.det_watchdog_status() == 0
