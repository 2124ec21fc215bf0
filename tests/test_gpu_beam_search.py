"""Beam search, forks and compaction of a decoder against the models' whole forward: the
beams, scores and lengths are those of a search that runs the forward again for every
beam and token, and after any forks and moves of pages every step's logits are bit for
bit the forward's; endings, weights, page sizes, attention in groups, captured forks and
refusals."""
import numpy as np
import pytest

from bitcmp import assert_bitwise
from bitwise_reproducible_fp32_gb300 import byte_lm, detlib, inputs
from bitwise_reproducible_fp32_gb300.decode import Decoder
from gpu_util import host, need_gpu, to_dev, torch

pytestmark = pytest.mark.gpu
F = np.float32


@pytest.fixture(scope="module")
def dev():
    return need_gpu()


def upload(c):
    cd = dict(c)
    cd["emb"], cd["head"] = to_dev(c["emb"]), to_dev(c["head"])
    cd["blocks"] = [{k: to_dev(v) for k, v in b.items()} for b in c["blocks"]]
    return cd


def last_logits(cd, seqs):
    """The training forward's logits of the last token of equally long sequences."""
    c = dict(cd, batch=len(seqs), seq=len(seqs[0]))
    c["tokens"] = torch.tensor(np.array(seqs, np.int32).reshape(-1), device="cuda")
    c["labels"] = torch.zeros_like(c["tokens"])
    return byte_lm.forward(c, torch.device("cuda"))["logits"].view(len(seqs), len(seqs[0]), -1)[:, -1]


def i32(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def search(cd, prompt, new_tokens, beams, top_k, eos, weights):
    """The same search with the forward run again for each beam and token; scores and
    ranks in float32."""
    state = [([], F(0), 0, False)]
    for _ in range(new_tokens):
        live = [b for b in state if not b[3]]
        top = {}
        if live:
            logits = last_logits(cd, [list(prompt) + b[0] for b in live]).contiguous()
            none = torch.full((len(live),), -1, dtype=torch.int32, device="cuda")
            _, _, ids, logp, _ = detlib.detlogprob_f32(logits, none, top_k, want_stats=False)
            top = {id(b): (host(ids)[i], host(logp)[i]) for i, b in enumerate(live)}
        cand = []
        for w, b in enumerate(state):
            if b[3]:
                cand.append((b[1], w, eos, b))
                continue
            for t, lp in zip(*top[id(b)]):
                cand.append((F(b[1] + lp), w, int(t), (b[0] + [int(t)], F(b[1] + lp), b[2] + 1,
                                                       int(t) == eos)))
        rank = lambda c: c[0] if weights is None else F(                     # noqa: E731
            c[0] * weights[min(c[3][2], len(weights) - 1)])
        state = [c[3] for c in sorted(cand, key=lambda c: (-rank(c), c[1], c[2]))[:beams]]
    return state


@pytest.mark.parametrize("model,lens,new,beams,top_k,page_size,group,weighted", [
    (dict(batch=3, seq=64), (5, 17, 1), 9, 4, 4, 4, 4, False),
    (dict(batch=3, seq=64), (3, 16, 30), 12, 3, 7, 16, 3, True),
    (dict(batch=2, seq=64), (9, 2), 6, 8, 8, 1, 1, False),
    (dict(batch=1, seq=700), (600,), 5, 5, 5, 64, 5, False),
    (dict(batch=2, seq=24, d=96, dff=100, vocab=301, blocks=3, heads=3), (7, 13), 8, 2, 3, 5, 4, True),
    (dict(batch=2, seq=24), (4, 8), 1, 3, 3, 16, 1, False),
])
def test_beams_are_those_of_rerunning_the_forward(dev, model, lens, new, beams, top_k, page_size,
                                                  group, weighted):
    c = inputs.byte_lm_cfg2(**model)
    cd = upload(c)
    toks = c["tokens"].reshape(c["batch"], c["seq"])
    prompts = [toks[b, :n] for b, n in enumerate(lens)]
    weights = (np.arange(1, new + 2, dtype=np.float64) ** -0.7).astype(F) if weighted else None
    k = len(prompts)
    dec = Decoder(cd, k * beams + 1, max(lens) + new + 3, torch.device("cuda"), page_size=page_size,
                  top_k=top_k, group=group)
    # an ending that the search meets: a token of the best beams without one
    free = search(cd, prompts[0], new, beams, top_k, -1, weights)
    eos = free[0][0][new // 2]
    for end in (-1, eos):
        a = dec.beam_search(prompts, new, beams, eos=end,
                            weights=None if weights is None else torch.from_numpy(weights).cuda())
        assert host(dec.lens).tolist() == [0] * dec.B and int(dec.count) == dec.pages
        assert sorted(host(dec.free).tolist()) == list(range(dec.pages))
        ids, n, score = (host(x) for x in a)
        for p in range(k):
            for w, want in enumerate(search(cd, prompts[p], new, beams, top_k, end, weights)):
                assert ids[p, w, :n[p, w]].tolist() == want[0], (p, w)
                assert (ids[p, w, n[p, w]:] == -1).all() and n[p, w] == want[2]
                assert_bitwise(score[p, w:w + 1], np.array([want[1]], F), f"prompt {p} beam {w}")


@pytest.mark.parametrize("page_size,group", [(4, 1), (16, 3), (7, 100)])
def test_forks_and_compaction_keep_every_bit(dev, page_size, group):
    # random forks, steps, releases and compactions; the sequences that the requests
    # should have are kept on the host
    c = inputs.byte_lm_cfg2(batch=4, seq=64)
    cd = upload(c)
    toks = c["tokens"].reshape(4, 64)
    B = 9
    dec = Decoder(cd, B, 64, torch.device("cuda"), page_size=page_size, group=group)
    rng = np.random.default_rng(page_size)
    dec.prefill([0, 4, 7], [toks[0, :20], toks[1, :3], toks[2, :16]])
    seqs = [[] for _ in range(B)]
    seqs[0], seqs[4], seqs[7] = list(toks[0, :20]), list(toks[1, :3]), list(toks[2, :16])
    for t in range(14):
        parents = rng.integers(-1, B, B)
        parents[rng.integers(0, B)] = max(range(B), key=lambda b: len(seqs[b]))
        dec.fork(i32(parents.tolist()))
        seqs = [list(seqs[p]) if p >= 0 else [] for p in parents]
        if t % 3 == 1:
            dec.compact()
            held = set()
            for b, n in enumerate(host(dec.lens)):
                held |= set(host(dec.table)[b, :-(-int(n) // page_size)].tolist())
            assert held == set(range(len(held))) and int(dec.count) == dec.pages - len(held)
        on = [int(len(s) > 0 and rng.random() < 0.8) for s in seqs]
        new = rng.integers(0, 256, B).tolist()
        nx = dec.step(i32(new), i32(on))
        got = host(nx.logits)
        for b in np.flatnonzero(on):
            seqs[b].append(new[b])
            assert_bitwise(got[b], host(last_logits(cd, [seqs[b]]))[0], f"step {t} request {b}")
        assert host(dec.lens).tolist() == [len(s) for s in seqs]
    # all but the longest are released, and what they shared with it stays
    keep = max(range(B), key=lambda b: len(seqs[b]))
    dec.release(i32([int(b != keep) for b in range(B)]))
    seqs = [s if b == keep else [] for b, s in enumerate(seqs)]
    assert int(dec.count) == dec.pages - -(-len(seqs[keep]) // page_size)
    nx = dec.step(i32([7] * B), i32([int(b == keep) for b in range(B)]))
    assert_bitwise(host(nx.logits)[keep], host(last_logits(cd, [seqs[keep] + [7]]))[0])
    dec.release(i32([1] * B))
    assert sorted(host(dec.free).tolist()) == list(range(dec.pages)) and int(dec.count) == dec.pages
    dec.check()


def test_a_captured_fork_compaction_and_step(dev):
    c = inputs.byte_lm_cfg2(batch=4, seq=64)
    cd = upload(c)
    toks = c["tokens"].reshape(4, 64)
    dec = Decoder(cd, 4, 64, torch.device("cuda"), page_size=8, group=2)
    parents, tok = i32([0, 1, 2, 3]), i32([0] * 4)
    on = i32([0] * 4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        dec.fork(parents)
        dec.compact()
        dec.step(tok, on)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dec.fork(parents)
        dec.compact()
        nx = dec.step(tok, on)
    dec.prefill([1], [toks[1, :13]])
    seqs = [[], list(toks[1, :13]), [], []]
    on.fill_(1)
    rng = np.random.default_rng(3)
    for step, move in enumerate(([1, 1, 1, 1], [3, 2, 1, 0], [0, 0, 3, 3], [2, 2, 2, 2])):
        new = rng.integers(0, 256, 4).tolist()
        parents.copy_(i32(move))
        tok.copy_(i32(new))
        graph.replay()
        seqs = [seqs[p] + [new[b]] for b, p in enumerate(move)]
        got = host(nx.logits)
        want = host(last_logits(cd, seqs))
        for b in range(4):
            assert_bitwise(got[b], want[b], f"replay {step} request {b}")
    dec.check()


def test_a_release_captured_before_the_first_fork(dev):
    c = inputs.byte_lm_cfg2(batch=2, seq=32)
    cd = upload(c)
    toks = c["tokens"].reshape(2, 32)
    dec = Decoder(cd, 3, 32, torch.device("cuda"), page_size=4)
    done = i32([0, 0, 0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dec.release(done)
    dec.prefill([0], [toks[0, :13]])
    dec.fork(i32([0, 0, 0]))
    done.copy_(i32([1, 0, 1]))
    graph.replay()
    assert host(dec.lens).tolist() == [0, 13, 0] and int(dec.count) == dec.pages - 4
    nx = dec.step(i32([9, 9, 9]), i32([0, 1, 0]))
    assert_bitwise(host(nx.logits)[1], host(last_logits(cd, [list(toks[0, :13]) + [9]]))[0])
    done.copy_(i32([0, 1, 0]))
    graph.replay()
    assert sorted(host(dec.free).tolist()) == list(range(dec.pages)) and int(dec.count) == dec.pages
    dec.check()


def test_out_of_pages_and_refusals(dev):
    c = inputs.byte_lm_cfg2(batch=2, seq=32)
    cd = upload(c)
    toks = c["tokens"].reshape(2, 32)
    device = torch.device("cuda")
    dec = Decoder(cd, 4, 32, device, page_size=8, pages=3, top_k=4)
    p = toks[0, :12]
    for args in (([p], 3, 5), ([p], 3, 0), ([], 3, 2), ([p, p, p], 3, 2), ([p], 0, 2), ([p], 22, 2),
                 ([[]], 3, 2)):
        with pytest.raises(ValueError):
            dec.beam_search(*args)
    assert host(dec.lens).tolist() == [0] * 4 and int(dec.count) == 3
    with pytest.raises(ValueError):
        Decoder(cd, 4, 32, device, group=0)
    # a request of the beams' that holds tokens is not overwritten
    dec.prefill([1], [p[:3]])
    with pytest.raises(ValueError):
        dec.beam_search([p], 2, 2)
    assert host(dec.lens).tolist() == [0, 3, 0, 0]
    dec.release(i32([0, 1, 0, 0]))
    # two of three copies of the partly filled page find no page and stay empty
    dec.prefill([0], [p])
    dec.fork(i32([0, 0, 0, 0]))
    with pytest.raises(ValueError, match="status 2"):
        dec.check()
    assert host(dec.lens).tolist() == [12, 12, 0, 0] and int(dec.count) == 0
    nx = dec.step(i32([5, 6, 0, 0]), i32([1, 1, 0, 0]))
    want = host(last_logits(cd, [list(p) + [5], list(p) + [6]]))
    assert_bitwise(host(nx.logits)[:2], want)
    dec.check()
    dec.fork(i32([-1, -1, -1, -1]))
    assert int(dec.count) == 3
    dec.fork(i32([0, 9, -2, 1]))
    with pytest.raises(ValueError, match="status 1"):
        dec.check()
