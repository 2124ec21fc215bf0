"""The operators of a generation step and of token scores, as they are measured:
rotary positions, the append to a paged key-value cache, its block tables and
slot maps, attention of one new token over it, and the log probabilities of given
tokens with entropy, alternatives and gradient.

`run` computes each in its plain form (elementary torch operations, float32) or,
where `own` is true, by the framework's own calls. Sizes are those of the two
models the framework trains (12 heads of 64 over 50,257 ids; 4 heads of 16 over
bytes) and generic ones with shared key-value heads.
"""
import math

import numpy as np
import torch

own = False

DEVICE = "cuda"


def listed():
    return [
        # Q and K of a training batch of packed documents, the 162M decoder's:
        # 4 x 2048 tokens, 24 heads of 64 inside rows of [Q | K | V]
        dict(name="rope_packed_documents", kind="rope", rows=8192, heads=24, head_dim=64, rot=64,
             half=False, inverse=False, longest=2048, stretch=1.0, extra=768),
        # the backward of long-context training: half layout, half of the head
        # turned, positions up to 128k on frequencies stretched 8 times, odd rows
        dict(name="rope_backward_long", kind="rope", rows=4099, heads=40, head_dim=128, rot=64,
             half=True, inverse=True, longest=131072, stretch=8.0, extra=0),
        # one decode step of 64 requests: a row each
        dict(name="append_decode", kind="append", rows=64, heads=12, kv_heads=12, head_dim=64,
             page=16, rot=64, half=False, longest=2048, padded=0),
        # a prefill of 8192 rows with shared key-value heads, an eighth of them padding
        dict(name="append_prefill", kind="append", rows=8192, heads=32, kv_heads=8, head_dim=128,
             page=64, rot=128, half=True, longest=32768, padded=1024),
        # the block tables of a decode step: every request gets one token
        dict(name="pages_decode", kind="extend", batch=256, page=16, longest=2048, most_new=1,
             short=False),
        # those of a prefill: 700 requests of up to 64 tokens, and too few pages for the last
        dict(name="pages_prefill", kind="extend", batch=700, page=16, longest=512, most_new=64,
             short=True),
        # the byte-level model answers 16 short prompts: where latency counts
        dict(name="decode_bytes", kind="decode", batch=16, heads=4, kv_heads=4, head_dim=16,
             page=16, shortest=1, longest=128),
        # the 162M decoder with 64 requests of ragged lengths in flight
        dict(name="decode_162m", kind="decode", batch=64, heads=12, kv_heads=12, head_dim=64,
             page=16, shortest=700, longest=2048),
        # few requests of long contexts, 4 query heads a key-value head
        dict(name="decode_long_shared", kind="decode", batch=4, heads=32, kv_heads=8, head_dim=128,
             page=64, shortest=20001, longest=32768),
        # what a served step answers with: 64 tokens' scores and 20 alternatives
        dict(name="logprob_decode", kind="logprob", rows=64, vocab=50257, top=20),
        # scoring a training batch, the 162M decoder's: 4 x 2048 tokens
        dict(name="logprob_score", kind="logprob", rows=8192, vocab=50257, top=5),
        # and its gradient with an entropy bonus, as policy-gradient training takes it
        dict(name="logprob_backward", kind="logprob_bwd", rows=8192, vocab=50257, entropy=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["rope", "append", "extend", "release", "decode", "decode", "logprob",
                       "logprob_bwd"])
    if kind == "rope":
        hd = rng.choice([16, 64, 80, 128])
        half = rng.random() < 0.5
        rot = rng.choice([r for r in (16, 32, 64, 80, 128) if r <= hd])
        heads = rng.randint(1, 48)
        return dict(kind=kind, rows=_log(rng, 1, 8192 * 24 * 64 // (heads * hd)), heads=heads,
                    head_dim=hd, rot=rot, half=half, inverse=rng.random() < 0.5,
                    longest=_log(rng, 128, 131072), stretch=rng.choice([1.0, 4.0, 8.0]),
                    extra=rng.choice([0, 4, 64]))
    if kind == "append":
        hd = rng.choice([16, 64, 128])
        kvh = rng.choice([1, 2, 4, 8, 12])
        rows = _log(rng, 1, 4096)
        return dict(kind=kind, rows=rows, heads=kvh * rng.choice([1, 2, 4]), kv_heads=kvh,
                    head_dim=hd, page=rng.choice([8, 16, 64]), rot=rng.choice([hd, hd // 2]),
                    half=rng.random() < 0.5, longest=_log(rng, 128, 131072),
                    padded=rng.randint(0, rows // 4))
    if kind == "extend":
        batch = _log(rng, 1, 2000)
        return dict(kind=kind, batch=batch, page=rng.choice([8, 16, 32, 64]),
                    longest=_log(rng, 64, 4096), most_new=rng.choice([1, 1, 8, 100]),
                    short=rng.random() < 0.3)
    if kind == "release":
        return dict(kind=kind, batch=_log(rng, 1, 2000), page=rng.choice([8, 16, 32, 64]),
                    longest=_log(rng, 64, 4096))
    if kind == "decode":
        hd = rng.choice([16, 64, 128])
        kvh = rng.choice([1, 2, 4, 8, 12])
        longest = _log(rng, 8, 32768)
        most = 4 * 32768 * 8 * 128 // (longest * kvh * hd)
        return dict(kind=kind, batch=_log(rng, 1, max(1, min(256, most))),
                    heads=kvh * rng.choice([1, 2, 4, 8]), kv_heads=kvh, head_dim=hd,
                    page=rng.choice([8, 16, 64, 100]), shortest=rng.choice([0, 1, longest // 2]),
                    longest=longest)
    vocab = _log(rng, 256, 160000)
    rows = _log(rng, 1, max(1, min(8192, 8192 * 50257 // vocab)))
    if kind == "logprob":
        return dict(kind=kind, rows=rows, vocab=vocab, top=rng.choice([0, 1, 5, 20]))
    return dict(kind=kind, rows=rows, vocab=vocab, entropy=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs
def _turns(rot, stretch):
    """Frequencies theta^(-2i/rot) / stretch, theta = 10,000, in 2^-64 turns a
    position (what the rotary calls take)."""
    w = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot) / stretch
    return (w / (2.0 * math.pi) * 2.0 ** 64).round().to(torch.int64).to(DEVICE)


def _page_pool(lens, page, spare, rng):
    """Block table of requests of these lengths over a shuffled pool, and the
    pages left over: (table, free pages)."""
    owned = -(-lens // page)
    total = int(owned.sum()) + spare
    perm = rng.permutation(total).astype(np.int32)
    width = max(1, int(owned.max()) if owned.size else 1)
    start = np.concatenate([[0], np.cumsum(owned)])[:-1]
    j = np.arange(width)[None, :]
    table = np.where(j < owned[:, None], perm[np.minimum(start[:, None] + j, total - 1)], -1)
    return table.astype(np.int32), perm[int(owned.sum()):].copy(), total


def _token_rows(case):
    """Rows that a step's new tokens are given: their mean and four deviations."""
    B, most = case["batch"], case["most_new"]
    return min(B * most, B * (most + 1) // 2 + int(4 * most * math.sqrt(B / 12)) + 1)


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEVICE)


def prepare(case, seed):
    rng = np.random.default_rng([seed, 20])
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(int(rng.integers(1 << 40)))

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=DEVICE, dtype=torch.float32)

    st = {"case": case}
    kind = case["kind"]
    if kind == "rope":
        n, width = case["rows"], case["heads"] * case["head_dim"]
        base = randn(n, width + case["extra"])
        # packed documents: positions run up and start again at 0
        cut = rng.random(n) < 2.0 / case["longest"]
        first = int(rng.integers(0, case["longest"]))
        last = np.maximum.accumulate(np.where(cut, np.arange(n), -1))
        pos = np.where(last >= 0, np.arange(n) - last, first + np.arange(n)) % case["longest"]
        st |= dict(x=base[:, :width], positions=_dev(pos.astype(np.int32)),
                   turns=_turns(case["rot"], case["stretch"]))
    elif kind == "append":
        n, H, G, d, page = (case[k] for k in ("rows", "heads", "kv_heads", "head_dim", "page"))
        pages = -(-n // page) + max(4, n // page // 8)
        slots = rng.permutation(pages * page)[:n].astype(np.int64)
        pos = rng.integers(0, case["longest"], n).astype(np.int32)
        pad = rng.permutation(n)[:case["padded"]]
        slots[pad], pos[pad] = -1, -1
        # one slot more than the cache has: the plain form sends padding there
        k, v = randn(pages * page + 1, G, d), randn(pages * page + 1, G, d)
        st |= dict(qkv=randn(n, (H + 2 * G) * d), slots=_dev(slots), positions=_dev(pos),
                   k_all=k, v_all=v, k_cache=k[:-1].view(pages, page, G, d),
                   v_cache=v[:-1].view(pages, page, G, d), q_out=torch.zeros(n, H * d, device=DEVICE),
                   turns=_turns(case["rot"], 1.0))
    elif kind in ("extend", "release"):
        B, page = case["batch"], case["page"]
        lens = rng.integers(0, case["longest"] + 1, B)
        most = case.get("most_new", 0)
        width = -(-(case["longest"] + most) // page)
        owned = int((-(-lens // page)).sum())
        table, free, total = _page_pool(lens, page, B * width - owned, rng)
        wide = np.full((B, width), -1, np.int32)
        wide[:, :table.shape[1]] = table
        room = np.zeros(total + 1, np.int32)
        room[:free.size] = free
        count = free.size
        if kind == "extend":
            new = rng.integers(1, most + 1, B)
            if case["short"]:
                count = int((-(-(lens + new) // page) - -(-lens // page)).sum()) * 3 // 4
            st |= dict(new=_dev(new.astype(np.int32)), rows=_token_rows(case))
        else:
            st |= dict(done=_dev((rng.random(B) < 0.3).astype(np.int32)))
        room = _dev(room)
        # one entry more than the list has: the plain form sends what it skips there
        st |= dict(lens=_dev(lens.astype(np.int32)), table=_dev(wide), free_all=room,
                   free=room[:-1], count=_dev(np.array([count], np.int32)))
    elif kind == "decode":
        B, H, G, d, page = (case[k] for k in ("batch", "heads", "kv_heads", "head_dim", "page"))
        lens = rng.integers(case["shortest"], case["longest"] + 1, B)
        lens[rng.integers(0, B)] = case["longest"]
        table, _, total = _page_pool(lens, page, 3, rng)
        st |= dict(q=randn(B, H * d), k_cache=randn(total, page, G, d),
                   v_cache=randn(total, page, G, d), table=_dev(table),
                   lens=_dev(lens.astype(np.int32)))
    else:
        n, V = case["rows"], case["vocab"]
        logits = randn(n, V).mul_(2.0)
        st |= dict(logits=logits, tokens=_dev(rng.integers(0, V, n).astype(np.int32)))
        if kind == "logprob_bwd":
            # what the forward saved: m, 1 / S, log S and the entropy of each row
            m = logits.amax(1)
            sums = []
            for part, top in zip(logits.split(512), m.split(512)):
                d = part - top[:, None]
                e = d.exp()
                sums.append(torch.stack([e.sum(1), (e * d).sum(1)]))
            S, T = torch.cat(sums, dim=1)
            st |= dict(stats=torch.stack([m, 1.0 / S, S.log(), S.log() - T / S], dim=1),
                       dlogp=randn(n) / n,
                       dentropy=randn(n) * (0.01 / n) if case["entropy"] else None)
    return st


# ------------------------------------------------------------------ plain forms
def _angles(positions, turns):
    a = (positions.long()[:, None] * turns[None, :]).double() * (2.0 * math.pi / 2.0 ** 64)
    return a.cos().float(), a.sin().float()


def _rotate(x, c, s, rot, half):
    """x: rows x heads x head_dim, c and s: rows x rot / 2."""
    c, s = c[:, None, :], s[:, None, :]
    out = x.clone()
    if half:
        x0, x1 = x[..., :rot // 2], x[..., rot // 2:rot]
        out[..., :rot // 2] = x0 * c - x1 * s
        out[..., rot // 2:rot] = x0 * s + x1 * c
    else:
        x0, x1 = x[..., 0:rot:2], x[..., 1:rot:2]
        out[..., 0:rot:2] = x0 * c - x1 * s
        out[..., 1:rot:2] = x0 * s + x1 * c
    return out


def _plain_rope(st):
    k = st["case"]
    c, s = _angles(st["positions"], st["turns"])
    x = st["x"].unflatten(1, (k["heads"], k["head_dim"]))
    return _rotate(x, c, -s if k["inverse"] else s, k["rot"], k["half"]).flatten(1)


def _plain_append(st):
    k = st["case"]
    n, H, G, d = k["rows"], k["heads"], k["kv_heads"], k["head_dim"]
    c, s = _angles(st["positions"], st["turns"])
    x = st["qkv"].view(n, H + 2 * G, d)
    turned = _rotate(x[:, :H + G], c, s, k["rot"], k["half"])
    pad = st["slots"] < 0
    slots = torch.where(pad, st["k_all"].shape[0] - 1, st["slots"])
    st["k_all"].index_copy_(0, slots, turned[:, H:])
    st["v_all"].index_copy_(0, slots, x[:, H + G:])
    st["q_out"].copy_(torch.where(pad[:, None], st["q_out"], turned[:, :H].flatten(1)))
    return {"q": st["q_out"], "k": st["k_cache"], "v": st["v_cache"]}


def _plain_extend(st):
    page, rows = st["case"]["page"], st["rows"]
    lens, new, table, count = (st[k].long() for k in ("lens", "new", "table", "count"))
    total = lens + new
    ok = (lens >= 0) & (new >= 0) & (total <= table.shape[1] * page)
    n = torch.where(ok, new, 0)
    row_end = n.cumsum(0)
    ok = ok & (row_end <= rows)
    owned = (lens + page - 1) // page
    need = torch.where(ok, (total + page - 1) // page - owned, 0)
    page_end = need.cumsum(0)
    ok = ok & ((need == 0) | (page_end <= count))
    taken = torch.where(ok & (need > 0), page_end, 0).amax().view(1)
    # the new entries of the table, newest free page first
    j = torch.arange(table.shape[1], device=table.device)[None, :]
    fresh = ok[:, None] & (j >= owned[:, None]) & (j < (owned + need)[:, None])
    i = (page_end - need)[:, None] + j - owned[:, None]
    pick = (count - 1 - i).clamp(0, st["free_all"].shape[0] - 1)
    table = torch.where(fresh, st["free_all"].long()[pick], table)
    st["table"].copy_(table)
    # rows: the request of each, its position and slot
    r = torch.arange(rows, device=table.device)
    b = torch.searchsorted(row_end, r, right=True).clamp(max=lens.shape[0] - 1)
    live = (r < row_end[-1]) & ok[b]
    pos = lens[b] + r - (row_end - n)[b]
    at = table[b, (pos // page).clamp(0, table.shape[1] - 1)] * page + pos % page
    starts = torch.cat([torch.zeros_like(row_end[:1]), row_end]).clamp(max=rows)
    return {"lens": torch.where(ok, total, lens).int(), "count": (count - taken).int(),
            "row_start": starts.int(), "positions": torch.where(live, pos, -1).int(),
            "slots": torch.where(live, at, -1), "table": st["table"]}


def _plain_release(st):
    page = st["case"]["page"]
    lens, table, count = st["lens"].long(), st["table"], st["count"].long()
    ok = (st["done"] != 0) & (lens >= 0) & (lens <= table.shape[1] * page)
    pages = torch.where(ok, (lens + page - 1) // page, 0)
    end = pages.cumsum(0)
    ok = ok & (count + end <= st["free"].shape[0])
    j = torch.arange(table.shape[1], device=table.device)[None, :]
    given = ok[:, None] & (j < pages[:, None])
    at = torch.where(given, count + (end - pages)[:, None] + j, st["free"].shape[0])
    st["free_all"].scatter_(0, at.flatten(), table.flatten())
    return {"lens": torch.where(ok, 0, lens).int(),
            "count": (count + torch.where(ok, end, 0).amax()).int(), "free": st["free"]}


def _plain_decode(st):
    k = st["case"]
    B, H, G, d, page = (k[n] for n in ("batch", "heads", "kv_heads", "head_dim", "page"))
    table = st["table"].long().clamp(min=0)
    K, V = (st[n][table].view(B, -1, G, d).transpose(1, 2) for n in ("k_cache", "v_cache"))
    q = st["q"].view(B, G, H // G, d)
    x = torch.matmul(q, K.transpose(2, 3)) * (1.0 / math.sqrt(d))
    dead = torch.arange(x.shape[-1], device=x.device) >= st["lens"][:, None, None, None]
    x = x.masked_fill(dead, -math.inf)
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    S = e.sum(-1, keepdim=True)
    p = e / torch.where(S == 0, 1.0, S)
    V = V.masked_fill(dead.view(B, 1, -1, 1), 0.0)
    return torch.matmul(p, V).reshape(B, H * d)


def _top(x, k):
    """Ids of the k largest of each row, the lowest id first among equals, by
    whole-number keys that order as (value, -id)."""
    bits = (x + 0.0).view(torch.int32).long()
    order = torch.where(bits < 0, -(bits & 0x7fffffff), bits)
    ids = torch.arange(x.shape[1], device=x.device)
    keys = order * (1 << 32) - ids
    return (-(keys.topk(k, dim=1).values)) & 0xffffffff


def _plain_logprob(st):
    x, y, k = st["logits"], st["tokens"].long()[:, None], st["case"]["top"]
    d = x - x.amax(1, keepdim=True)
    e = d.exp()
    S = e.sum(1, keepdim=True)
    logS = S.log()
    out = {"logp": (d.gather(1, y) - logS)[:, 0],
           "entropy": (logS - (e * d).sum(1, keepdim=True) / S)[:, 0]}
    if k:
        ids = _top(x, k)
        out |= {"top_ids": ids.int(), "top_logp": d.gather(1, ids) - logS}
    return out


def _plain_logprob_bwd(st):
    x, y = st["logits"], st["tokens"].long()[:, None]
    m, inv, logS, ent = (c[:, None] for c in st["stats"].unbind(1))
    d = x - m
    p = d.exp() * inv
    out = p * -st["dlogp"][:, None]
    out.scatter_add_(1, y, st["dlogp"][:, None])
    if st["dentropy"] is not None:
        out -= st["dentropy"][:, None] * (p * (d - logS + ent))
    return out


def run(st):
    k = st["case"]
    if not own:
        return {"rope": _plain_rope, "append": _plain_append, "extend": _plain_extend,
                "release": _plain_release, "decode": _plain_decode, "logprob": _plain_logprob,
                "logprob_bwd": _plain_logprob_bwd}[k["kind"]](st)
    from bitwise_reproducible_fp32_gb300 import detlib as L
    if k["kind"] == "rope":
        return L.detrope_at_f32(st["x"], st["positions"], k["heads"], k["head_dim"],
                                turns=st["turns"], half=k["half"], inverse=k["inverse"])
    if k["kind"] == "append":
        q = L.detkv_append_f32(st["qkv"], st["slots"], st["k_cache"], st["v_cache"], k["heads"],
                               positions=st["positions"], turns=st["turns"], half=k["half"],
                               q_out=st["q_out"])
        return {"q": q, "k": st["k_cache"], "v": st["v_cache"]}
    if k["kind"] == "extend":
        lens, count, starts, pos, slots = L.detpages_extend(
            st["lens"], st["new"], st["table"], st["free"], st["count"], k["page"], st["rows"])
        return {"lens": lens, "count": count, "row_start": starts, "positions": pos,
                "slots": slots, "table": st["table"]}
    if k["kind"] == "release":
        lens, count = L.detpages_release(st["lens"], st["done"], st["table"], st["free"],
                                         st["count"], k["page"])
        return {"lens": lens, "count": count, "free": st["free"]}
    if k["kind"] == "decode":
        return L.detdecode_attention_f32(st["q"], st["k_cache"], st["v_cache"], st["table"],
                                         st["lens"], k["heads"])
    if k["kind"] == "logprob":
        logp, entropy, ids, top, _ = L.detlogprob_f32(st["logits"], st["tokens"], top_k=k["top"])
        out = {"logp": logp, "entropy": entropy}
        return out | {"top_ids": ids, "top_logp": top} if k["top"] else out
    return L.detlogprob_bwd_f32(st["logits"], st["tokens"], st["stats"], st["dlogp"],
                                st["dentropy"])


def work(case):
    k = case["kind"]
    if k == "rope":
        n = case["rows"] * case["heads"]
        return {"bytes": 8 * n * case["head_dim"] + 4 * case["rows"], "flops": 3 * n * case["rot"]}
    if k == "append":
        n, width = case["rows"] - case["padded"], case["heads"] + 2 * case["kv_heads"]
        return {"bytes": 8 * n * width * case["head_dim"] + 12 * case["rows"],
                "flops": 3 * n * (case["heads"] + case["kv_heads"]) * case["rot"]}
    if k == "extend":
        rows = _token_rows(case)
        return {"bytes": 20 * case["batch"] + 16 * rows, "flops": 10 * (case["batch"] + rows)}
    if k == "release":
        pages = case["batch"] * case["longest"] // (2 * case["page"]) // 3
        return {"bytes": 12 * case["batch"] + 8 * pages, "flops": 10 * case["batch"]}
    if k == "decode":
        tokens = case["batch"] * (case["shortest"] + case["longest"]) // 2
        return {"bytes": 8 * tokens * case["kv_heads"] * case["head_dim"]
                + 8 * case["batch"] * case["heads"] * case["head_dim"],
                "flops": 4 * tokens * case["heads"] * case["head_dim"]}
    n = case["rows"] * case["vocab"]
    if k == "logprob":
        return {"bytes": 4 * n + 8 * case["rows"] * (2 + case["top"]), "flops": 6 * n}
    return {"bytes": 8 * n + 28 * case["rows"], "flops": (10 if case["entropy"] else 6) * n}


# ------------------------------------------------------------------ in 64 bits
def _exact_rotate(x, pos, turns, rot, half, inverse=False):
    """x: rows x heads x head_dim, float64 numpy."""
    phase = pos.astype(np.uint64)[:, None] * turns.astype(np.uint64)[None, :]
    a = phase.astype(np.int64).astype(np.float64) * (math.pi / 2.0 ** 63)
    z = np.exp(-1j * a if inverse else 1j * a)[:, None, :]
    out = x.copy()
    i0, i1 = (slice(0, rot // 2), slice(rot // 2, rot)) if half else (slice(0, rot, 2),
                                                                     slice(1, rot, 2))
    w = (x[..., i0] + 1j * x[..., i1]) * z
    out[..., i0], out[..., i1] = w.real, w.imag
    return out


def exact(case, seed):
    st = prepare(case, seed)
    k = case["kind"]
    if k in ("extend", "release"):
        return None
    if k == "rope":
        x = st["x"].unflatten(1, (case["heads"], case["head_dim"])).double().cpu().numpy()
        out = _exact_rotate(x, st["positions"].cpu().numpy(), st["turns"].cpu().numpy(),
                            case["rot"], case["half"], case["inverse"])
        return out.reshape(x.shape[0], -1)
    if k == "append":
        n, H, G, d = (case[c] for c in ("rows", "heads", "kv_heads", "head_dim"))
        x = st["qkv"].double().cpu().numpy().reshape(n, H + 2 * G, d)
        slots, pos = st["slots"].cpu().numpy(), st["positions"].cpu().numpy()
        live = slots >= 0
        turned = _exact_rotate(x[live, :H + G], pos[live], st["turns"].cpu().numpy(), case["rot"],
                               case["half"])
        q = st["q_out"].double().cpu().numpy()
        kc, vc = (st[c].double().cpu().numpy() for c in ("k_cache", "v_cache"))
        q[live] = turned[:, :H].reshape(-1, H * d)
        kc.reshape(-1, G, d)[slots[live]] = turned[:, H:]
        vc.reshape(-1, G, d)[slots[live]] = x[live, H + G:]
        return {"q": q, "k": kc, "v": vc}
    if k == "decode":
        B, H, G, d, page = (case[c] for c in ("batch", "heads", "kv_heads", "head_dim", "page"))
        out = torch.zeros(B, G, H // G, d, dtype=torch.float64, device=DEVICE)
        for b, n in enumerate(st["lens"].tolist()):
            if n:
                own_pages = st["table"][b, :-(-n // page)].long()
                K, V = (st[c][own_pages].flatten(0, 1)[:n].double() for c in ("k_cache", "v_cache"))
                s = torch.einsum("ghd,ngd->ghn", st["q"][b].view(G, H // G, d).double(), K)
                p = torch.softmax(s / math.sqrt(d), dim=-1)
                out[b] = torch.einsum("ghn,ngd->ghd", p, V)
        return out.view(B, H * d)
    x, y = st["logits"], st["tokens"].long()
    parts = []
    for i in range(0, x.shape[0], 256):
        lp = torch.log_softmax(x[i:i + 256].double(), dim=1)
        at = lp.gather(1, y[i:i + 256, None])
        ent = -(lp.exp() * lp).sum(1)
        if k == "logprob":
            vals, ids = torch.sort(x[i:i + 256], dim=1, descending=True, stable=True)
            top = ids[:, :case["top"]]
            parts.append((at[:, 0], ent, top.int(), lp.gather(1, top)))
        else:
            g = st["dlogp"][i:i + 256, None].double()
            hot = torch.zeros_like(lp).scatter_(1, y[i:i + 256, None], 1.0)
            dx = g * (hot - lp.exp())
            if st["dentropy"] is not None:
                dx -= st["dentropy"][i:i + 256, None].double() * lp.exp() * (lp + ent[:, None])
            parts.append((dx,))
    out = [torch.cat(c) for c in zip(*parts)]
    if k == "logprob_bwd":
        return out[0]
    res = {"logp": out[0], "entropy": out[1]}
    return res | {"top_ids": out[2], "top_logp": out[3]} if case["top"] else res
