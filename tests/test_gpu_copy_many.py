"""Copies of many pairs over a pool of a million pages, many times the filters' bits: a
compaction's (each page one, all destinations below the sources), and lists in which
destinations come again and are sources."""
import numpy as np
import pytest

from gpu_util import need_gpu
from test_gpu_fork import F, I, on_gpu, run_copy

pytestmark = pytest.mark.gpu

PAGES, PAIRS = 1 << 20, 150_000


@pytest.fixture(scope="module")
def caches():
    need_gpu()
    rng = np.random.default_rng(40)
    return [on_gpu(rng.standard_normal((PAGES, 1, 1, 4)).astype(F)) for _ in range(2)]


def test_moves_of_a_compaction(caches):
    rng = np.random.default_rng(41)
    low = np.sort(rng.choice(PAGES // 2, PAIRS, replace=False)).astype(I)
    high = np.sort(PAGES // 2 + rng.choice(PAGES // 2, PAIRS, replace=False)).astype(I)
    run_copy(*caches, high, low)
    # of lists with room for more
    pad = np.full(PAGES // 2 - PAIRS, 7, I)
    run_copy(*caches, np.concatenate([high, pad]), np.concatenate([low, pad + 1]), count=PAIRS)


@pytest.mark.parametrize("again,read", [(0, 0), (1, 0), (0, 1), (3000, 3000), (PAIRS, 0)])
def test_destinations_that_come_again_or_are_read(caches, again, read):
    rng = np.random.default_rng(42 + again + read)
    ids = rng.permutation(PAGES).astype(I)
    src, dst = ids[:PAIRS].copy(), ids[PAIRS:2 * PAIRS].copy()
    at = rng.permutation(PAIRS)
    dst[at[:again]] = dst[rng.integers(0, PAIRS, again)]
    dst[at[again:again + read]] = src[rng.integers(0, PAIRS, read)]
    run_copy(*caches, src, dst)
    tokens = rng.integers(0, 2, PAIRS).astype(I)
    run_copy(*caches, src, dst, tokens)
