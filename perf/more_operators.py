"""The operators of beam search over a paged key-value cache, as they are measured:
attention of requests that share a prefix, the selection of the next beams with their
token histories, and forking, copying and compacting of the cache's pages.

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
        # the byte-level model answers 4 short prompts with 4 beams each: where latency counts
        dict(name="attend_bytes", kind="attend", groups=4, beams=4, heads=4, kv_heads=4,
             head_dim=16, page=16, least_prefix=60, most_prefix=100, most_own=28),
        # the 162M decoder, 16 prompts of ragged lengths with 4 beams each
        dict(name="attend_beams", kind="attend", groups=16, beams=4, heads=12, kv_heads=12,
             head_dim=64, page=16, least_prefix=700, most_prefix=1900, most_own=148),
        # the 162M decoder's width, 64 conversations on one instruction text of 8k tokens
        dict(name="attend_instructions", kind="attend", groups=1, beams=64, heads=12, kv_heads=12,
             head_dim=64, page=16, least_prefix=8100, most_prefix=8192, most_own=1000),
        # 48 questions about one long document, 4 query heads a key-value head
        dict(name="attend_document", kind="attend", groups=1, beams=48, heads=32, kv_heads=8,
             head_dim=128, page=64, least_prefix=20001, most_prefix=24000, most_own=600),
        # one step of 16 prompts with 4 beams each: a few candidates, short answers
        dict(name="select_step", kind="select", prompts=16, beams=4, top=8, vocab=50257,
             answer=148, scaled=False),
        # many prompts with wide beams, long answers, scores divided by a power of the length
        dict(name="select_wide", kind="select", prompts=512, beams=16, top=32, vocab=50257,
             answer=2048, scaled=True),
        # the pages of such a step: 16 prompts with 4 beams each
        dict(name="fork_step", kind="fork", groups=16, beams=4, page=16, most_prefix=1900,
             most_own=148),
        # and of a large one: 512 prompts with 16 beams
        dict(name="fork_wide", kind="fork", groups=512, beams=16, page=16, most_prefix=4000,
             most_own=2000),
        # the partly filled pages that a step's forked beams get copies of (162M decoder, one layer)
        dict(name="copy_step", kind="copy", pairs=40, pages=4000, page=16, kv_heads=12, head_dim=64,
             whole=False),
        # pages that move when a pool is compacted
        dict(name="copy_moves", kind="copy", pairs=4096, pages=10000, page=16, kv_heads=8,
             head_dim=128, whole=True),
        # a pool of the 162M decoder's requests, compacted
        dict(name="compact_small", kind="compact", groups=16, beams=4, page=16, most_prefix=1900,
             most_own=148, alive=0.6),
        # a pool of half a million pages
        dict(name="compact_large", kind="compact", groups=256, beams=8, page=16, most_prefix=8000,
             most_own=3000, alive=0.5),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["attend", "attend", "attend", "select", "fork", "copy", "compact"])
    if kind == "attend":
        hd = rng.choice([16, 64, 64, 80, 128])
        kvh = rng.choice([1, 2, 4, 8, 12])
        per = rng.choice([1, 1, 2, 4, 8])
        groups = _log(rng, 1, 24)
        beams = _log(rng, 2, 64)
        # tokens read and products formed stay within the largest listed case
        most = min(24000, 24000 * 8 * 128 // (groups * kvh * hd),
                   24000 * 48 * 32 * 128 // (groups * beams * kvh * per * hd))
        prefix = _log(rng, 33, max(34, most))
        return dict(kind=kind, groups=groups, beams=beams, heads=kvh * per, kv_heads=kvh,
                    head_dim=hd, page=rng.choice([8, 16, 64, 100]),
                    least_prefix=rng.choice([1, prefix // 2, prefix]), most_prefix=prefix,
                    most_own=max(1, min(rng.choice([1, 40, 300, 1000]),
                                        8_000_000 // (groups * beams * kvh * hd))))
    if kind == "select":
        beams = _log(rng, 1, 32)
        prompts = _log(rng, 1, max(1, 512 * 16 // beams))
        return dict(kind=kind, prompts=prompts, beams=beams, top=rng.choice([beams, 32]),
                    vocab=_log(rng, 64, 160000), answer=_log(rng, 8, 2048),
                    scaled=rng.random() < 0.5)
    sizes = dict(kind=kind, groups=_log(rng, 1, 256), beams=rng.choice([1, 2, 4, 5, 8]),
                 page=rng.choice([8, 16, 32, 64]), most_prefix=_log(rng, 16, 4000),
                 most_own=_log(rng, 8, 2000))
    if kind == "fork":
        return sizes
    if kind == "compact":
        return dict(sizes, alive=rng.choice([0.2, 0.6, 1.0]))
    kvh, hd = rng.choice([1, 4, 8, 12]), rng.choice([16, 64, 80, 128])
    page = rng.choice([8, 16, 64])
    most = 4096 * 16 * 8 * 128 // (page * kvh * hd)
    pairs = _log(rng, 1, min(4096, most))
    return dict(kind=kind, pairs=pairs, pages=2 * pairs + rng.randint(1, 300), page=page,
                kv_heads=kvh, head_dim=hd, whole=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs
def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEVICE)


def _pool(case):
    """Pages with room for every request of a case at its longest, and a few."""
    rows, page = case["groups"] * case["beams"], case["page"]
    return (case["groups"] * (case["most_prefix"] // page)
            + rows * (case["most_own"] // page + 3) + 3)


def _tables(case, rng, alive=1.0):
    """Block tables of groups of rows that share the whole pages of a prefix, over a
    shuffled pool: (lens, table, shared pages a group, pages left over, pool)."""
    n, W, page = case["groups"], case["beams"], case["page"]
    prefix = rng.integers(case.get("least_prefix", 1), case["most_prefix"] + 1, n)
    lens = np.repeat(prefix, W) + rng.integers(1, case["most_own"] + 1, n * W)
    shared = prefix // page
    live = rng.random(n * W) < alive
    live[rng.integers(0, n * W)] = True
    lens = np.where(live, lens, 0)
    owned = -(-lens // page)
    some = live.reshape(n, W).any(1)
    first = np.concatenate([[0], np.cumsum(np.where(some, shared, 0))])
    own_pages = np.maximum(owned - np.repeat(shared, W), 0)
    start = first[-1] + np.concatenate([[0], np.cumsum(own_pages)])
    used = int(start[-1])
    total = _pool(case)
    perm = rng.permutation(total).astype(np.int32)
    width = -(-(case["most_prefix"] + case["most_own"]) // page)
    j = np.arange(width)[None, :]
    sh = np.repeat(shared, W)[:, None]
    at = np.where(j < sh, np.repeat(first[:-1], W)[:, None] + j, start[:-1, None] + j - sh)
    table = np.where(j < owned[:, None], perm[np.clip(at, 0, total - 1)], -1)
    return lens.astype(np.int32), table.astype(np.int32), shared, perm[used:].copy(), total


def prepare(case, seed):
    rng = np.random.default_rng([seed, 33])
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(int(rng.integers(1 << 40)))

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=DEVICE, dtype=torch.float32)

    st = {"case": case}
    kind = case["kind"]
    if kind == "attend":
        H, G, d, page = (case[k] for k in ("heads", "kv_heads", "head_dim", "page"))
        lens, table, shared, _, total = _tables(case, rng)
        st |= dict(q=randn(len(lens), H * d), k_cache=randn(total, page, G, d),
                   v_cache=randn(total, page, G, d), table=_dev(table), lens=_dev(lens),
                   # what the plain form goes by: each group's shared pages
                   shared=_dev(shared), most_shared=int(shared.max()),
                   most_own=int((-(-lens // page) - np.repeat(shared, case["beams"])).max()))
    elif kind == "select":
        R, W, k, V = (case[c] for c in ("prompts", "beams", "top", "vocab"))
        k = min(k, V)
        logp = -np.sort(rng.exponential(2.0, (R * W, k)), axis=1).astype(np.float32)
        ids = rng.integers(0, V, (R * W, 1)) + np.cumsum(
            rng.integers(1, max(2, V // k), (R * W, k)), axis=1)
        ids = (ids % V).astype(np.int32)
        eos = int(ids[0, 0])
        lens = rng.integers(1, case["answer"], R * W).astype(np.int32)
        done = (rng.random(R * W) < 0.1).astype(np.int32)
        lens[done == 0] = case["answer"] - 1
        score = -np.sort(rng.gamma(0.5 * lens.reshape(R, W) + 1.0, 1.0)).astype(np.float32)
        hist = rng.integers(0, V, (R * W, case["answer"])).astype(np.int32)
        power = np.arange(1, case["answer"] + 2, dtype=np.float64) ** -0.6
        st |= dict(scores=_dev(score), ids=_dev(ids), logp=_dev(logp), done=_dev(done),
                   lens=_dev(lens), hist=_dev(hist), hist_out=torch.zeros_like(_dev(hist)),
                   eos=eos,
                   weights=_dev(power.astype(np.float32)) if case["scaled"] else None)
    elif kind == "fork":
        lens, table, _, free, total = _tables(case, rng)
        n, W = case["groups"], case["beams"]
        # most beams go on from a few of the old ones, some have ended
        old = np.minimum(rng.integers(0, W, (n, W)), rng.integers(0, W, (n, W)))
        old = np.sort(old, axis=1) + np.arange(n)[:, None] * W
        old = np.where(rng.random((n, W)) < 0.05, -1, old).reshape(-1)
        pool = np.zeros(total + 1, np.int32)
        pool[:free.size] = free
        pool = _dev(pool)
        i32 = dict(dtype=torch.int32, device=DEVICE)
        st |= dict(lens=_dev(lens), parents=_dev(old.astype(np.int32)), table=_dev(table),
                   total=total, free_all=pool, free=pool[:-1],
                   count=_dev(np.array([free.size], np.int32)),
                   table_out=torch.full(table.shape, -1, **i32))
    elif kind == "compact":
        lens, table, _, _, total = _tables(case, rng, case["alive"])
        i32 = dict(dtype=torch.int32, device=DEVICE)
        st |= dict(lens=_dev(lens), table=_dev(table), total=total,
                   free=torch.full((total,), -1, **i32),
                   table_out=torch.full(table.shape, -1, **i32),
                   src=torch.full((total // 2,), -1, **i32),
                   dst=torch.full((total // 2,), -1, **i32))
    else:
        n, pages, page, G, d = (case[c] for c in ("pairs", "pages", "page", "kv_heads", "head_dim"))
        perm = rng.permutation(pages).astype(np.int32)
        # several copies may have one source
        src = perm[rng.integers(0, pages - n, n)]
        tokens = rng.integers(1, page + 1, n).astype(np.int32)
        st |= dict(k_cache=randn(pages, page, G, d), v_cache=randn(pages, page, G, d),
                   src=_dev(src), dst=_dev(perm[pages - n:]),
                   tokens=None if case["whole"] else _dev(tokens))
    return st


# ------------------------------------------------------------------ plain forms
def _plain_attend(st):
    """Scores and sums of each group's shared pages for all its rows at once, of the
    other pages request by request."""
    k = st["case"]
    n, W, H, G, d, page = (k[c] for c in ("groups", "beams", "heads", "kv_heads", "head_dim",
                                          "page"))
    B, per, S = n * W, H // G, st["most_shared"] * page
    table, lens = st["table"].long(), st["lens"]
    q = st["q"].view(n, W, G, per, d).transpose(1, 2)                  # n, G, W, per, d
    scale = 1.0 / math.sqrt(d)
    # the shared pages of each group's first row
    j = torch.arange(st["most_shared"], device=table.device)
    ids = table[::W, :st["most_shared"]].clamp(min=0)
    Ks, Vs = (st[c][ids].view(n, S, G, d).transpose(1, 2) for c in ("k_cache", "v_cache"))
    xs = torch.matmul(q.reshape(n, G, W * per, d), Ks.transpose(2, 3)) * scale
    dead = (j[None, :] >= st["shared"][:, None]).repeat_interleave(page, dim=1)
    xs = xs.masked_fill(dead[:, None, None, :], -math.inf).view(n, G, W, per, S).transpose(1, 2)
    # each row's own pages
    m = torch.arange(st["most_own"], device=table.device)
    at = st["shared"].repeat_interleave(W)[:, None] + m[None, :]
    ids = table.gather(1, at.clamp(max=table.shape[1] - 1)).clamp(min=0)
    Ko, Vo = (st[c][ids].view(B, -1, G, d).transpose(1, 2) for c in ("k_cache", "v_cache"))
    xo = torch.matmul(q.transpose(1, 2).reshape(B, G, per, d), Ko.transpose(2, 3)) * scale
    pos = (at * page)[:, :, None] + torch.arange(page, device=table.device)
    gone = pos.flatten(1) >= lens[:, None]
    xo = xo.masked_fill(gone[:, None, None, :], -math.inf)
    Vo = Vo.masked_fill(gone[:, None, :, None], 0.0)
    x = torch.cat([xs.reshape(B, G, per, S), xo], dim=3)
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - top)
    p = e / e.sum(-1, keepdim=True)
    ps = p[..., :S].view(n, W, G, per, S).transpose(1, 2).reshape(n, G, W * per, S)
    out = torch.matmul(ps, Vs).view(n, G, W, per, d).transpose(1, 2).reshape(B, H * d)
    return out + torch.matmul(p[..., S:], Vo).reshape(B, H * d)


def _plain_select(st):
    W = st["case"]["beams"]
    R, k = st["scores"].shape[0], st["ids"].shape[1]
    done = (st["done"] != 0).view(R, W, 1)
    slot = torch.arange(k, device=done.device)
    s = st["scores"][:, :, None] + st["logp"].view(R, W, k)
    # a beam that has ended goes on as it is, once
    s = torch.where(done, torch.where(slot == 0, st["scores"][:, :, None], -math.inf), s)
    token = torch.where(done, st["eos"], st["ids"].view(R, W, k))
    length = (st["lens"].view(R, W, 1) + torch.where(done, 0, 1)).expand(R, W, k)
    rank = s
    if st["weights"] is not None:
        rank = s * st["weights"][length.clamp(max=st["weights"].shape[0] - 1).long()]
    beam = torch.arange(W, device=done.device).view(1, W, 1).expand(R, W, k)
    # by rank, the lowest (beam, id) first among equals
    order = (beam.long() * (1 << 32) + token.long()).view(R, -1).sort(dim=1, stable=True)[1]
    order = order.gather(1, rank.reshape(R, -1).gather(1, order).sort(
        dim=1, descending=True, stable=True)[1])[:, :W]
    pick = lambda a: a.reshape(R, -1).gather(1, order)                 # noqa: E731
    score, token, length, beam = pick(s), pick(token), pick(length), pick(beam)
    ended = pick(done.expand(R, W, k)) | (token == st["eos"])
    parent = beam + W * torch.arange(R, device=done.device)[:, None]
    was = pick(done.expand(R, W, k)).view(-1, 1)
    col = torch.arange(st["hist"].shape[1], device=done.device)[None, :]
    hist = st["hist"][parent.view(-1).long()]
    last = length.reshape(-1, 1)
    hist = torch.where((col == last - 1) & ~was, token.reshape(-1, 1), hist)
    st["hist_out"].copy_(torch.where(col < last, hist, st["hist_out"]))
    return {"scores": score, "tokens": token.int().view(-1), "parents": parent.int().view(-1),
            "forks": torch.where(ended, -1, parent).int().view(-1),
            "finished": ended.int().view(-1), "lens": length.int().reshape(-1),
            "hist": st["hist_out"]}


def _plain_fork(st):
    page, total = st["case"]["page"], st["total"]
    lens, parents, table, count = (st[c].long() for c in ("lens", "parents", "table", "count"))
    B, width = table.shape
    owned = (lens + page - 1) // page
    row = torch.arange(B, device=table.device)
    there = parents >= 0
    p = parents.clamp(min=0)
    # the first child of each row
    first = torch.full_like(lens, B).scatter_reduce(0, p, torch.where(there, row, B), "amin")
    kept = first < B
    j = torch.arange(width, device=table.device)[None, :]
    holds = j < owned[:, None]

    def mask(rows):
        m = torch.zeros(total + 1, dtype=torch.bool, device=table.device)
        m[torch.where(holds & rows[:, None], table, total).view(-1)] = True
        return m[:total]

    freed = mask(~kept) & ~mask(kept)
    rank = freed.long().cumsum(0)
    st["free_all"].scatter_(0, torch.where(freed, count + rank - 1, total),
                            torch.arange(total, device=table.device).int())
    count = count + rank[-1]
    # children after the first get a page of their own in the place of a partly filled one
    new_lens = torch.where(there, lens[p], 0)
    need = there & (first[p] != row) & (new_lens % page != 0)
    at = (count - need.long().cumsum(0)).clamp(min=0)
    fresh = st["free_all"][at]
    out = torch.where(holds[p] & there[:, None], st["table"][p], st["table_out"])
    last = (new_lens // page).clamp(max=width - 1)[:, None]
    src = torch.where(need, st["table"][p].gather(1, last)[:, 0], -1)
    dst = torch.where(need, fresh, -1)
    out = torch.where(need[:, None] & (j == last), fresh[:, None], out)
    st["table_out"].copy_(out)
    return {"table": st["table_out"], "lens": new_lens.int(),
            "count": (count - need.sum()).int(), "src": src.int(), "dst": dst.int(),
            "tokens": torch.where(need, new_lens % page, 0).int(), "free": st["free"]}


def _plain_compact(st):
    page, total = st["case"]["page"], st["total"]
    table = st["table"].long()
    owned = (st["lens"].long() + page - 1) // page
    j = torch.arange(table.shape[1], device=table.device)[None, :]
    holds = j < owned[:, None]
    used = torch.zeros(total + 1, dtype=torch.bool, device=table.device)
    used[torch.where(holds, table, total).view(-1)] = True
    used = used[:total]
    n = used.sum().view(1)
    ids = torch.arange(total, device=table.device)
    moving, hole = used & (ids >= n), ~used & (ids < n)
    # the i-th moving page goes to the i-th hole
    spare = torch.zeros(total + 1, dtype=torch.long, device=table.device)
    spare.scatter_(0, torch.where(hole, hole.long().cumsum(0) - 1, total), ids)
    nth = moving.long().cumsum(0) - 1
    to = torch.where(moving, spare[nth.clamp(min=0)], ids)
    moves = moving.sum().view(1)
    half = st["src"].shape[0]
    pad = torch.full((total + 1,), -1, dtype=torch.long, device=table.device)
    at = torch.where(moving, nth, total)
    keep = torch.arange(half, device=table.device) < moves
    st["src"].copy_(torch.where(keep, pad.scatter(0, at, ids)[:half].int(), st["src"]))
    st["dst"].copy_(torch.where(keep, pad.scatter(0, at, to)[:half].int(), st["dst"]))
    st["table_out"].copy_(torch.where(holds, to[table.clamp(min=0)].int(), st["table_out"]))
    st["free"].copy_(torch.where(ids < total - n, (total - 1 - ids).int(), st["free"]))
    return {"table": st["table_out"], "count": (total - n).int(), "src": st["src"],
            "dst": st["dst"], "moves": moves.int(), "free": st["free"]}


def _plain_copy(st):
    src, dst = st["src"].long(), st["dst"].long()
    for c in (st["k_cache"], st["v_cache"]):
        rows = c[src]
        if st["tokens"] is not None:
            t = torch.arange(c.shape[1], device=c.device)[None, :, None, None]
            rows = torch.where(t < st["tokens"][:, None, None, None], rows, c[dst])
        c.index_copy_(0, dst, rows)
    return {"k": st["k_cache"], "v": st["v_cache"]}


def run(st):
    k = st["case"]
    kind = k["kind"]
    if not own:
        return {"attend": _plain_attend, "select": _plain_select, "fork": _plain_fork,
                "compact": _plain_compact, "copy": _plain_copy}[kind](st)
    from bitwise_reproducible_fp32_gb300 import detlib as L
    if kind == "attend":
        return L.detdecode_attention_shared_f32(st["q"], st["k_cache"], st["v_cache"], st["table"],
                                                st["lens"], k["heads"], k["beams"])
    if kind == "select":
        b = L.detbeam_select_f32(st["scores"], st["ids"], st["logp"], k["beams"], eos=st["eos"],
                                 finished=st["done"], lens=st["lens"], weights=st["weights"],
                                 hist=st["hist"], hist_out=st["hist_out"])
        return b._asdict()
    if kind == "fork":
        table, lens, count, src, dst, tokens = L.detpages_fork(
            st["lens"], st["parents"], st["table"], st["free"], st["count"], k["page"],
            st["total"], table_out=st["table_out"])
        return {"table": table, "lens": lens, "count": count, "src": src, "dst": dst,
                "tokens": tokens, "free": st["free"]}
    if kind == "compact":
        table, count, moves, src, dst = L.detpages_compact(
            st["lens"], st["table"], st["free"], k["page"], table_out=st["table_out"],
            src=st["src"], dst=st["dst"])
        return {"table": table, "count": count, "src": src, "dst": dst, "moves": moves,
                "free": st["free"]}
    L.detkv_copy_f32(st["k_cache"], st["v_cache"], st["src"], st["dst"], tokens=st["tokens"])
    return {"k": st["k_cache"], "v": st["v_cache"]}


def work(case):
    kind = case["kind"]
    if kind == "copy":
        tokens = case["pairs"] * (case["page"] if case["whole"] else (case["page"] + 1) / 2)
        return {"bytes": int(16 * tokens * case["kv_heads"] * case["head_dim"]
                             + 12 * case["pairs"]), "flops": 0}
    if kind == "select":
        rows, k = case["prompts"] * case["beams"], min(case["top"], case["vocab"])
        # nine beams of ten have answers of full length, the others half
        return {"bytes": int(rows * (8 * k + 36 + 8 * 0.95 * case["answer"])),
                "flops": rows * k}
    rows = case["groups"] * case["beams"]
    prefix = (case.get("least_prefix", 1) + case["most_prefix"]) / 2
    mine = (1 + case["most_own"]) / 2
    if kind == "attend":
        kept = case["groups"] * prefix + rows * mine
        width = case["heads"] * case["head_dim"]
        return {"bytes": int(8 * kept * case["kv_heads"] * case["head_dim"] + 8 * rows * width),
                "flops": int(4 * rows * (prefix + mine) * width)}
    entries = rows * (prefix + mine) / case["page"]
    if kind == "fork":
        return {"bytes": int(8 * entries + 28 * rows), "flops": int(2 * entries)}
    used = case["alive"] * (case["groups"] * prefix + rows * mine) / case["page"]
    return {"bytes": int(case["alive"] * 8 * entries + 4 * (_pool(case) - used) + 4 * rows),
            "flops": int(2 * entries)}


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    kind = case["kind"]
    if kind not in ("attend", "select"):
        return None                       # whole numbers and copies
    st = prepare(case, seed)
    if kind == "attend":
        H, G, d, page = (case[c] for c in ("heads", "kv_heads", "head_dim", "page"))
        out = torch.zeros(len(st["lens"]), G, H // G, d, dtype=torch.float64, device=DEVICE)
        for b, n in enumerate(st["lens"].tolist()):
            mine = st["table"][b, :-(-n // page)].long()
            K, V = (st[c][mine].flatten(0, 1)[:n].double() for c in ("k_cache", "v_cache"))
            s = torch.einsum("ghd,ngd->ghn", st["q"][b].view(G, H // G, d).double(), K)
            out[b] = torch.einsum("ghn,ngd->ghd", torch.softmax(s / math.sqrt(d), dim=-1), V)
        return out.view(len(st["lens"]), H * d)
    # the order goes by scores in float32, as the operator defines them; the scores
    # themselves in 64 bits
    f32 = lambda c: st[c].cpu().numpy()                                # noqa: E731
    score, ids, logp, done, lens, hist = (f32(c) for c in ("scores", "ids", "logp", "done", "lens",
                                                           "hist"))
    weights = None if st["weights"] is None else f32("weights")
    R, W = score.shape
    k = ids.shape[1]
    res = {c: [] for c in ("scores", "tokens", "parents", "forks", "finished", "lens")}
    rows = np.zeros_like(hist)
    for r in range(R):
        cand = []
        for w in range(W):
            i = r * W + w
            if done[i]:
                cand.append((score[r, w], float(score[r, w]), w, st["eos"], int(lens[i]), True))
            else:
                for a in range(k):
                    cand.append((score[r, w] + logp[i, a], float(score[r, w]) + float(logp[i, a]),
                                 w, int(ids[i, a]), int(lens[i]) + 1, False))
        if weights is None:
            key = lambda c: (-c[0], c[2], c[3])                        # noqa: E731
        else:
            key = lambda c: (-(c[0] * weights[min(c[4], len(weights) - 1)]), c[2], c[3])  # noqa: E731
        for c, (_, s, w, token, n, was) in enumerate(sorted(cand, key=key)[:W]):
            i = r * W + w
            end = was or token == st["eos"]
            for name, v in zip(res, (s, token, i, -1 if end else i, int(end), n)):
                res[name].append(v)
            out = rows[r * W + c]
            out[:n] = hist[i, :n]
            if not was:
                out[n - 1] = token
    out = {c: np.array(v, np.float64 if c == "scores" else np.int32) for c, v in res.items()}
    out["scores"] = out["scores"].reshape(R, W)
    return out | {"hist": rows}
