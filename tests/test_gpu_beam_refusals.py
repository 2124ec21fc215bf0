"""What a decoder refuses for several answers of a prompt leaves it as it was: no request is
released and no page taken by a call that raises."""
import numpy as np
import pytest

from bitwise_reproducible_fp32_gb300 import detlib, inputs
from bitwise_reproducible_fp32_gb300.decode import Decoder
from gpu_util import host, need_gpu, torch
from test_gpu_beam_search import i32, upload

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return need_gpu()


@pytest.fixture(scope="module")
def model(dev):
    c = inputs.byte_lm_cfg2(batch=2, seq=32)
    return upload(c), c["tokens"].reshape(2, 32)


def state(dec):
    return [host(t).tolist() for t in (dec.lens, dec.count, dec.free, dec.table)]


def test_release_takes_one_int32_flag_a_request(dev, model):
    cd, toks = model
    dec = Decoder(cd, 4, 32, torch.device("cuda"), page_size=4)
    dec.prefill([0], [toks[0, :13]])
    wrong = [i32([1]), i32([1] * 5), i32([1, 0, 0]), i32([[1, 0, 0, 0]]), i32([1, 0] * 4)[::2],
             i32(1), torch.ones(4, device="cuda"), torch.ones(4, dtype=torch.bool, device="cuda"),
             torch.ones(4, dtype=torch.int64, device="cuda"), torch.ones(4, dtype=torch.int32)]
    for forked in (False, True):
        if forked:
            dec.fork(i32([0, 0, 0, -1]))
        before = state(dec)
        for done in wrong:
            with pytest.raises((TypeError, ValueError)):
                dec.release(done)
            with pytest.raises((TypeError, ValueError)):
                with torch.cuda.graph(torch.cuda.CUDAGraph()):
                    dec.release(done)
        assert state(dec) == before
    dec.release(i32([1, 0, 1, 0]))
    assert host(dec.lens).tolist() == [0, 13, 0, 0] and int(dec.count) == dec.pages - 4
    dec.release(i32([0, 1, 0, 0]))
    assert sorted(host(dec.free).tolist()) == list(range(dec.pages)) and int(dec.count) == dec.pages
    dec.check()


def test_beam_search_refuses_before_it_takes_pages(dev, model):
    cd, toks = model
    dec = Decoder(cd, 4, 32, torch.device("cuda"), page_size=4, top_k=4)
    before = state(dec)
    for kw in (dict(weights=torch.ones(6)), dict(weights=torch.ones(6, device="cuda").double()),
               dict(weights=torch.ones((2, 3), device="cuda")),
               dict(weights=torch.ones(6, device="cuda")[::2]),
               dict(weights=torch.ones(0, device="cuda")), dict(weights=[1.0] * 6),
               dict(eos=1 << 32), dict(eos=1.5j)):
        with pytest.raises((TypeError, ValueError)):
            dec.beam_search([toks[0, :9]], 5, 4, **kw)
        assert state(dec) == before
    # a cache that a fork does not know: one token needs none
    dec.pages, pages = (1 << 23) + 1, dec.pages
    for call in (lambda: dec.beam_search([toks[0, :9]], 5, 4), dec.compact,
                 lambda: dec.fork(i32([0] * 4))):
        with pytest.raises(ValueError):
            call()
        assert state(dec) == before
    dec.beam_search([toks[0, :9]], 1, 4)
    dec.pages = pages
    dec.beam_search([toks[0, :9]], 5, 4, eos=np.int32(3))
    assert host(dec.lens).tolist() == [0] * 4 and int(dec.count) == dec.pages
    dec.check()


def test_selection_refuses_an_ending_that_is_no_int32(dev):
    x, ids = torch.zeros((1, 2), device="cuda"), torch.zeros((2, 3), dtype=torch.int32, device="cuda")
    for eos in (1 << 31, (1 << 32) + 5, (-1 << 31) - 1):
        with pytest.raises(ValueError):
            detlib.detbeam_select_f32(x, ids, ids.float(), 2, eos=eos)
