"""Generation from the paged cache against the models' whole forward: every
step's logits are bit for bit the forward's row of that token, the log
probabilities are its losses, ragged prompts, inactive requests, page sizes, a
captured and replayed step, pages that are given back, and refusals."""
import numpy as np
import pytest

from bitcmp import assert_bitwise
from bitwise_reproducible_fp32_gb300 import byte_lm, detlib, inputs
from bitwise_reproducible_fp32_gb300.decode import Decoder
from gpu_util import host, need_gpu, to_dev, torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return need_gpu()


def upload(c):
    cd = dict(c)
    cd["tokens"] = torch.from_numpy(c["tokens"]).cuda()
    cd["labels"] = torch.from_numpy(c["labels"]).cuda()
    cd["emb"], cd["head"] = to_dev(c["emb"]), to_dev(c["head"])
    cd["blocks"] = [{k: to_dev(v) for k, v in b.items()} for b in c["blocks"]]
    return cd


def whole(cd, toks, labels=None):
    """The training forward of equally long sequences: logits and losses."""
    c = dict(cd, batch=toks.shape[0], seq=toks.shape[1])
    c["tokens"] = torch.from_numpy(np.ascontiguousarray(toks).reshape(-1)).cuda()
    lab = np.zeros_like(toks) if labels is None else labels
    c["labels"] = torch.from_numpy(np.ascontiguousarray(lab).reshape(-1)).cuda()
    st = byte_lm.forward(c, torch.device("cuda"))
    return (host(st["logits"]).reshape(*toks.shape, -1), host(st["loss"]).reshape(toks.shape))


def i32(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("model,lens,steps,page_size", [
    (dict(batch=4, seq=40), (5, 1, 31, 17), 9, 16),
    (dict(batch=3, seq=300), (255, 256, 257), 8, 64),
    (dict(batch=2, seq=24, d=96, dff=100, vocab=301, blocks=3, heads=3), (7, 13), 9, 5),
    ("162m", (70, 129), 5, 64),
])
def test_steps_have_the_forwards_bits(dev, model, lens, steps, page_size):
    if model == "162m":
        c = inputs.decoder_162m(layers=2, batch=2, seq=160)
    else:
        c = inputs.byte_lm_cfg2(**model)
    cd = upload(c)
    B, T = c["batch"], c["seq"]
    toks = c["tokens"].reshape(B, T)
    labels = c["labels"].reshape(B, T)
    logits, loss = whole(cd, toks, labels)
    dec = Decoder(cd, B, T, torch.device("cuda"), page_size=page_size, top_k=3)
    order = list(range(B))[::-1]                        # requests in another order
    nx = dec.prefill(order, [toks[b, :lens[b]] for b in order])
    for r, b in enumerate(order):
        assert_bitwise(host(nx.logits)[r], logits[b, lens[b] - 1], f"prompt {b}")
    for t in range(steps):
        at = [lens[b] + t for b in range(B)]
        nx = dec.step(i32([toks[b, at[b]] for b in range(B)]),
                      targets=i32([labels[b, at[b]] for b in range(B)]))
        got, logp, ids, top = (host(a) for a in (nx.logits, nx.logp, nx.ids, nx.top_logp))
        for b in range(B):
            assert_bitwise(got[b], logits[b, at[b]], f"step {t}, request {b}")
            assert_bitwise(-logp[b:b + 1], loss[b, at[b]:at[b] + 1], f"step {t} logp {b}")
            best = np.argsort(-logits[b, at[b]], kind="stable")[:3]
            assert ids[b].tolist() == best.tolist()
    dec.check()


def test_generation_equals_rerunning_the_forward(dev):
    c = inputs.byte_lm_cfg2(batch=3, seq=40)
    cd = upload(c)
    prompts = [c["tokens"].reshape(3, 40)[b, :n] for b, n in enumerate((3, 20, 11))]
    dec = Decoder(cd, 5, 64, torch.device("cuda"), page_size=8, pages=24)
    for _ in range(2):                                  # the second run on returned pages
        ids, logp = (host(a) for a in dec.generate(prompts, 12))
        assert int(dec.count) == 24 and host(dec.lens).tolist() == [0] * 5
        for b, p in enumerate(prompts):
            seq = list(p)
            for t in range(12):
                logits, loss = whole(cd, np.array([seq], np.int32),
                                     np.array([[0] * (len(seq) - 1) + [ids[b, t]]], np.int32))
                assert int(np.argmax(logits[0, -1])) == ids[b, t]
                assert_bitwise(-logp[b, t:t + 1], loss[0, -1:], f"request {b} token {t}")
                seq.append(int(ids[b, t]))


def test_a_captured_step_and_inactive_requests(dev):
    c = inputs.byte_lm_cfg2(batch=4, seq=64)
    cd = upload(c)
    toks = c["tokens"].reshape(4, 64)
    logits, _ = whole(cd, toks)
    device = torch.device("cuda")
    dec = Decoder(cd, 4, 64, device, page_size=16)
    tok, active = i32([0] * 4), i32([0] * 4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        dec.step(tok, active)                           # nobody active: nothing changes
    torch.cuda.current_stream().wait_stream(side)
    assert host(dec.lens).tolist() == [0] * 4
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nx = dec.step(tok, active)
    lens = [9, 0, 2, 33]
    dec.prefill([3, 0, 2], [toks[3, :33], toks[0, :9], toks[2, :2]])
    rng = np.random.default_rng(5)
    for _ in range(25):
        on = rng.integers(0, 2, 4).astype(np.int32)
        tok.copy_(i32([int(toks[b, lens[b]]) for b in range(4)]))
        active.copy_(i32(on.tolist()))
        graph.replay()
        got = host(nx.logits)
        for b in np.flatnonzero(on):
            assert_bitwise(got[b], logits[b, lens[b]], f"request {b} at {lens[b]}")
            lens[b] += 1
        assert host(dec.lens).tolist() == lens
    dec.check()


def test_refusals(dev):
    c = inputs.byte_lm_cfg2(batch=2, seq=16)
    cd = upload(c)
    device = torch.device("cuda")
    dec = Decoder(cd, 2, 16, device, page_size=4, pages=5)
    p = c["tokens"][:12].tolist()
    for req, pro in (([], []), ([0], []), ([0, 0], [p, p]), ([2], [p]), ([-1], [p]), ([0], [[]]),
                     ([0], [p + p])):
        with pytest.raises(ValueError):
            dec.prefill(req, pro)
    dec.prefill([0, 1], [p, p[:8]])                     # 3 + 2 pages: none left
    dec.check()
    with pytest.raises(ValueError):
        dec.prefill([1], [p])
    dec.step(i32([1, 1]))
    with pytest.raises(ValueError, match="status 2"):
        dec.check()
    assert host(dec.lens).tolist() == [12, 8]
    dec.release(i32([0, 1]))
    for _ in range(4):
        dec.step(i32([1, 1]), i32([1, 0]))
    dec.check()
    dec.step(i32([1, 1]), i32([1, 0]))                  # request 0 is at max_len
    with pytest.raises(ValueError, match="status 1"):
        dec.check()
    dec.check()
    with pytest.raises(ValueError):
        Decoder(cd, 0, 16, device)


def test_two_decoders_on_two_streams(dev):
    # rows long enough for the attention's workspace, two steps under way at once
    c = inputs.byte_lm_cfg2(batch=2, seq=700, heads=4)
    cd = upload(c)
    toks = c["tokens"].reshape(2, 700)
    logits, _ = whole(cd, toks)
    device = torch.device("cuda")
    decs = [Decoder(cd, 2, 4096, device, page_size=16, top_k=k) for k in (0, 32)]
    streams = [torch.cuda.Stream() for _ in decs]
    for dec, s, n in zip(decs, streams, (600, 690)):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            dec.prefill([0, 1], [toks[0, :n], toks[1, :n]])
    feeds = [[i32([toks[0, n + t], toks[1, n + t]]) for t in range(10)] for n in (600, 690)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    seen = [[], []]
    for t in range(10):
        for i, (dec, s) in enumerate(zip(decs, streams)):
            with torch.cuda.stream(s):
                seen[i].append(dec.step(feeds[i][t]).logits.clone())
    torch.cuda.synchronize()
    for i, n in enumerate((600, 690)):
        decs[i].check()
        for t in range(10):
            assert_bitwise(host(seen[i][t]), logits[:, n + t], f"decoder {i} step {t}")
    with pytest.raises(ValueError):
        decs[0].generate([toks[0, :3]], 2)              # no ids without top_k


@pytest.mark.parametrize("full", [0, 1, 2, 3])
@pytest.mark.parametrize("masked", [False, True])
def test_a_full_request_leaves_the_others_alone(dev, full, masked):
    # one request at max_len, refused in every step; one inactive when masked;
    # the others' logits stay the forward's, step after step
    c = inputs.byte_lm_cfg2(batch=4, seq=16)
    cd = upload(c)
    toks = c["tokens"].reshape(4, 16)
    logits, _ = whole(cd, toks)
    dec = Decoder(cd, 4, 16, torch.device("cuda"), page_size=4)
    lens = [5, 9, 2, 7]
    lens[full] = 16
    dec.prefill([0, 1, 2, 3], [toks[b, :n] for b, n in enumerate(lens)])
    on = [1] * 4
    if masked:
        on[(full + 2) % 4] = 0
    active = i32(on) if masked else None
    for t in range(5):
        nx = dec.step(i32([int(toks[b, min(n, 15)]) for b, n in enumerate(lens)]), active)
        got = host(nx.logits)
        for b in range(4):
            if on[b] and b != full:
                assert_bitwise(got[b], logits[b, lens[b]], f"step {t}, request {b}")
                lens[b] += 1
        assert host(dec.lens).tolist() == lens
    with pytest.raises(ValueError, match="status 1"):
        dec.check()


@pytest.mark.parametrize("masked", [False, True])
def test_refusals_for_length_and_for_pages_in_one_step(dev, masked):
    # request 0 is full and 2 finds no page: 1 and 3 go on as the forward does
    c = inputs.byte_lm_cfg2(batch=4, seq=16)
    cd = upload(c)
    toks = c["tokens"].reshape(4, 16)
    logits, _ = whole(cd, toks)
    dec = Decoder(cd, 4, 16, torch.device("cuda"), page_size=4, pages=4 + 2 + 2 + 3)
    lens = [16, 5, 8, 9]
    dec.prefill([0, 1, 2, 3], [toks[b, :n] for b, n in enumerate(lens)])
    dec.check()
    for t in range(3):
        nx = dec.step(i32([int(toks[b, min(n, 15)]) for b, n in enumerate(lens)]),
                      i32([1] * 4) if masked else None)
        for b in (1, 3):
            assert_bitwise(host(nx.logits)[b], logits[b, lens[b]], f"step {t}, request {b}")
            lens[b] += 1
        assert host(dec.lens).tolist() == lens
    with pytest.raises(ValueError, match="status 3"):
        dec.check()


def test_a_prompt_batch_of_more_rows_than_one_append_takes(dev):
    # 8192 prompts, the last of 129 tokens and the others of 1: 1,056,768 padded rows
    c = inputs.byte_lm_cfg2(batch=16, seq=132)
    cd = upload(c)
    toks = c["tokens"].reshape(16, 132)
    logits, _ = whole(cd, toks)
    B = 8192
    dec = Decoder(cd, B, 132, torch.device("cuda"), page_size=16, pages=B + 8)
    lens = [1] * (B - 1) + [129]
    nx = dec.prefill(list(range(B)), [toks[b % 16, :n] for b, n in enumerate(lens)])
    look = list(range(16)) + list(range(B - 17, B))
    got = host(nx.logits)
    for b in look:
        assert_bitwise(got[b], logits[b % 16, lens[b] - 1], f"prompt {b}")
    nx = dec.step(i32([int(toks[b % 16, n]) for b, n in enumerate(lens)]))
    got = host(nx.logits)
    for b in look:
        assert_bitwise(got[b], logits[b % 16, lens[b]], f"step, request {b}")
    dec.check()


def test_a_refused_prompt_changes_nothing(dev):
    # longer than the attention takes: the requests stay empty and usable
    c = inputs.byte_lm_cfg2(batch=2, seq=16)
    cd = upload(c)
    toks = c["tokens"].reshape(2, 16)
    logits, _ = whole(cd, toks)
    dec = Decoder(cd, 2, 70000, torch.device("cuda"), page_size=16, pages=5000)
    with pytest.raises(detlib.DetError):
        dec.prefill([1], [np.zeros(65537, np.int32)])
    assert host(dec.lens).tolist() == [0, 0] and int(dec.count) == 5000
    nx = dec.prefill([1, 0], [toks[1, :5], toks[0, :16]])
    assert_bitwise(host(nx.logits), logits[[1, 0], [4, 15]])
    dec.check()
