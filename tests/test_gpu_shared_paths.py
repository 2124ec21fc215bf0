"""The tests of attention of requests that share a prefix, and of beam search, with every
group read in groups (one launch of clusters) and with every group read together (plan,
scores, sums, P V, join), whatever the sizes: the library's own choice reads most of these
small calls each request for itself. And the sizes for which it chooses each of the ways."""
import threading

import numpy as np
import pytest

from bitcmp import assert_bitwise
from bitwise_reproducible_fp32_gb300 import detlib
from decode_variants import ALONE, GROUPS, TOGETHER, reading
from gpu_util import host, need_gpu, torch
from test_gpu_beam_search import (  # noqa: F401 (run here as well)
    test_a_captured_fork_compaction_and_step, test_beams_are_those_of_rerunning_the_forward,
    test_forks_and_compaction_keep_every_bit)
from test_gpu_shared_attention import (  # noqa: F401
    both, on_gpu, shared_cache, test_cache_past_32_bit_offsets,
    test_captured_replayed_and_on_another_stream, test_empty_and_bad_requests_in_a_group,
    test_exps_at_the_ties_of_their_rounding, test_heads_in_rounds_of_the_workspace,
    test_infinities_and_nan, test_long, test_many_groups, test_prefixes_around_the_chunks,
    test_ragged_groups, test_read_together_captured_and_on_two_streams,
    test_requests_with_the_same_pages_all_through, test_rows_of_every_tile,
    test_two_threads_at_once)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return need_gpu()


@pytest.fixture(autouse=True, params=[GROUPS, TOGETHER], ids=["groups", "together"])
def way(request, dev):
    with reading(request.param):
        yield request.param


def groups_bytes(B, group, H, G, d, max_len):
    """What reading in groups keeps: scores and partials of every chunk and row."""
    return -(-B // group) * G * -(-max_len // 256) * group * (H // G) * (256 + d) * 4


def together_bytes(B, group, H, G, d, max_len):
    """What reading together keeps of a round of heads (scores and partials, and a list or
    two of the requests): at most about 1 GiB, or one head's."""
    chunks, rows = -(-max_len // 256), -(-B // group) * group * (H // G)
    head = rows * chunks * (256 + d) * 4
    return min(G, max(1, (1 << 30) // head)) * head


def way_of(*sizes):
    n = detlib.detdecode_attention_shared_workspace_bytes(*sizes)
    B, _, H, G, d, max_len = sizes
    alone = detlib.detdecode_attention_workspace_bytes(B, H, G, d, max_len)
    assert not n == alone == groups_bytes(*sizes)     # else the sizes do not tell
    if n == alone:
        return ALONE
    if n == groups_bytes(*sizes):
        return GROUPS
    assert abs(n - together_bytes(*sizes)) < together_bytes(*sizes) // 8 + (1 << 16), sizes
    return TOGETHER


def test_this_way_is_taken(way):
    for sizes in ((6, 3, 4, 2, 64, 2000), (12, 4, 4, 4, 16, 300), (9, 2, 6, 2, 80, 5000)):
        assert way_of(*sizes) == way
    for sizes in ((12, 12, 4, 2, 64, 3000), (8, 2, 36, 2, 64, 1000)):        # more than 8 rows
        assert way_of(*sizes) == TOGETHER


def test_the_librarys_own_choice(way):
    with reading(-1):
        for want, sizes in (
                (ALONE, (64, 1, 12, 12, 64, 2048)), (ALONE, (16, 4, 4, 4, 16, 128)),
                (GROUPS, (64, 4, 12, 12, 64, 2048)), (GROUPS, (64, 8, 12, 12, 64, 2048)),
                (TOGETHER, (64, 64, 12, 12, 64, 9216)), (TOGETHER, (48, 48, 32, 8, 128, 24640))):
            assert way_of(*sizes) == want, sizes


def test_a_status_of_each_request(way):
    # one bad request of a group changes nothing for the others, and its own row alone is NaN
    rng = np.random.default_rng(5)
    kc, vc, table, lens, _, _ = shared_cache([900, 300], [30, 400, 1, 77, 260, 5], 16, 2, 64, "token",
                                             rng)
    q = rng.standard_normal((6, 4 * 64)).astype(np.float32)
    good = both(q, kc, vc, table, lens, 4, 3)
    assert not np.isnan(good).any()
    for row, col in ((1, 70), (4, 25)):
        bad = table.clone()
        bad[row, col] = kc.shape[0]
        got = both(q, kc, vc, bad, lens, 4, 3)
        others = np.arange(6) != row
        assert np.isnan(got[row]).all() and (got[others] == good[others]).all()
    assert detlib.det_watchdog_status() == 0


@pytest.mark.parametrize("H,G", [(20, 2), (12, 1), (40, 4)])
@pytest.mark.parametrize("ps", [16, 64, 5])
def test_more_than_8_rows_of_own_tokens(way, H, G, ps):
    # a request's own tokens have tiles of their own then
    rng = np.random.default_rng(H + ps)
    for prefix, own in ((600, [1, 255, 256, 300, 17]), (0, [40, 1, 700, 513, 256])):
        kc, vc, table, lens, _, _ = shared_cache([prefix], own, ps, G, 64, "token", rng)
        q = (2 * rng.standard_normal((5, H * 64))).astype(np.float32)
        both(q, kc, vc, table, lens, H, 5)
        both(q, kc, vc, table, lens, H, 2)


def test_rounds_of_heads_with_more_than_8_rows(way):
    rng = np.random.default_rng(9)
    own = [9, 30, 1, 500, 44]
    kc, vc, table, lens, _, _ = shared_cache([700], own, 16, 5, 64, "token", rng)
    sizes = (5, 5, 10, 5, 64, 16 * 1_300_000)
    if way == TOGETHER:
        # of the five heads' scores, one round's are kept
        need = detlib.detdecode_attention_shared_workspace_bytes(*sizes)
        assert need < 1.3 * (1 << 30) < groups_bytes(*sizes)
    wide = torch.full((5, 1_300_000), -1, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    q = rng.standard_normal((5, 10 * 64)).astype(np.float32)
    both(q, kc, vc, wide, lens, 10, 5)


def test_two_threads_with_groups_of_4_and_12(way):
    rng = np.random.default_rng(28)
    jobs = []
    for B, H, G, d, group in ((8, 4, 4, 64, 4), (24, 8, 2, 128, 12)):
        kc, vc, table, lens, _, _ = shared_cache([1500], rng.integers(1, 300, B), 16, G, d, "token", rng)
        q = on_gpu(rng.standard_normal((B, H * d)).astype(np.float32))
        want = host(detlib.detdecode_attention_f32(q, kc, vc, table, on_gpu(lens), H))
        jobs.append(((q, kc, vc, table, on_gpu(lens), H, group), want))
    torch.cuda.synchronize()
    failed = []

    def work(job):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(300):
                    out = detlib.detdecode_attention_shared_f32(*job[0])
                got = host(out)
            assert_bitwise(got, job[1])
        except Exception as e:      # noqa: BLE001 (an error of the other thread)
            failed.append(e)

    threads = [threading.Thread(target=work, args=(job,)) for job in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
