"""Generation with the models of byte_lm.py (pre-norm blocks, no final norm, an
untied head), from a paged key-value cache: prompts go through the blocks'
training forward once, then every step sends one token a request through the
same operations on one row a request, with the attention reading the cache.

No operation's bits depend on how many rows it gets, and decode attention has
the bits of the last row of the causal attention. So a step's logits are bit for
bit those that byte_lm.forward gives for the last token of the same sequence,
whatever the batch, the page size and the order in which pages were taken.

A step is library calls and copies on device buffers made once; nothing in it
waits for the host, so it can be captured in a CUDA graph and replayed. Each
layer is one page-table-sharing [pages, page_size, heads, head_dim] pair.

Requests can go on from one another's tokens (fork) and then share the pages that
are full; a step reads what neighbours share once. beam_search is made of that and
the selection of the next beams.
"""
from __future__ import annotations

from typing import NamedTuple

APPEND_ROWS = 1 << 20           # detkv_append_f32 takes so many rows in a call
FORK_PAGES = 1 << 23            # detpages_fork and detpages_compact know so many pages


class Next(NamedTuple):
    """What a step (or a prompt) says about each request's next token: its logits,
    the top_k most probable ids with their log probabilities, the entropy of the
    distribution, and the log probability of the target given for it (0 for a
    target of -1)."""
    logits: object
    ids: object
    top_logp: object
    entropy: object
    logp: object


class Answers(NamedTuple):
    """The answers that beam search found: of each prompt `beams` rows, the best first,
    with their tokens (-1 past their length), lengths and scores (the sum of the tokens'
    log probabilities; -inf, and length 0, where there are fewer)."""
    ids: object
    lens: object
    scores: object


class Decoder:
    """The cache, its page tables and a step's buffers for up to max_batch requests
    of up to max_len tokens (prompt and answer; whole pages, so up to the next
    multiple of page_size). model: the tensors of
    inputs.byte_lm_cfg2 or decoder_162m on the device. pages: the pages of
    page_size tokens that all requests share (default: enough for every request
    to reach max_len). group: a step's attention reads what `group` consecutive requests
    share once (1: each request for itself); the bits do not depend on it."""

    def __init__(self, model, max_batch, max_len, device, page_size=64, pages=None, top_k=1,
                 eps=1e-6, theta=10000.0, group=1):
        import torch

        from bitwise_reproducible_fp32_gb300 import detlib as L
        # what a step's calls would refuse, before anything depends on it
        if not 1 <= max_batch <= 8192:
            raise ValueError("max_batch must be in 1..8192")
        # past 2^20 the rotary's angles are NaN
        if not 1 <= max_len <= 1 << 20:
            raise ValueError("max_len must be in 1..2^20")
        if page_size < 1 or (pages is not None and pages < 1):
            raise ValueError("page_size and pages must be at least 1")
        if group < 1:
            raise ValueError("group must be at least 1")
        if not 0 <= top_k <= min(32, model["vocab"]):
            raise ValueError(f"top_k must be in 0..{min(32, model['vocab'])}")
        self.model, self.B, self.max_len, self.device = model, max_batch, max_len, device
        self.page_size, self.top_k, self.eps, self.theta = page_size, top_k, eps, theta
        self.group = min(group, max_batch)
        self.H, D, Fd, V = model["heads"], model["d"], model["dff"], model["vocab"]
        self.hd, B = D // model["heads"], max_batch
        width = -(-max_len // page_size)
        self.pages = pages = max_batch * width if pages is None else pages
        f = lambda *s: torch.empty(s, dtype=torch.float32, device=device)  # noqa: E731
        i = lambda *s: torch.zeros(s, dtype=torch.int32, device=device)    # noqa: E731
        self.cache = [(f(pages, page_size, self.H, self.hd), f(pages, page_size, self.H, self.hd))
                      for _ in model["blocks"]]
        self.table = i(max_batch, width)
        self.free = torch.arange(pages - 1, -1, -1, dtype=torch.int32, device=device)
        # lengths and the count of free pages in one buffer, as is what a step
        # makes of them: one copy takes the new state over
        self.state, self.after = i(B + 1), i(B + 1)
        self.state[B] = pages
        self.lens, self.count = self.state[:B], self.state[B:]
        self.status = i(1)
        self.ones, self.none = i(B) + 1, torch.full((B,), -1, dtype=torch.int32, device=device)
        # one row more than requests: a request that takes no row in a step reads
        # that one, which has no position and no slot
        self.row_start, self.positions = i(B + 1), i(B + 1)
        self.slots = torch.zeros(B + 1, dtype=torch.int64, device=device)
        self.first, self.end, self.past = self.row_start[:B], self.row_start[1:], i(B) + B
        self.took = torch.zeros(B, dtype=torch.bool, device=device)
        self.row, self.pos = i(B), i(B)
        self.slot = torch.zeros(B, dtype=torch.int64, device=device)
        self.buf = dict(x=f(B, D), h=f(B, D), qkv=f(B, 3 * D), att=f(B, D), o=f(B, D), x1=f(B, D),
                        h2=f(B, D), gate=f(B, Fd), up=f(B, Fd), s=f(B, Fd), dn=f(B, D), y=f(B, D))
        self.inv = f(B)
        self.next = Next(f(B, V), i(B, top_k), f(B, top_k), f(B), f(B))
        ws = lambda N, K, t=False: L.gemm_workspace(B, N, K, False, t, device=device)  # noqa: E731
        self.ws = dict(qkv=ws(3 * D, D), o=ws(D, D), down=ws(D, Fd), head=ws(V, D, True))
        wg = model["blocks"][0]
        self.ws["gate_up"] = L.gemm_group_workspace(
            [dict(A=self.buf["h2"], B=wg["W_gate"], C=self.buf["gate"]),
             dict(A=self.buf["h2"], B=wg["W_up"], C=self.buf["up"])])
        sizes = self.H, self.H, self.hd, width * page_size
        n = (L.detdecode_attention_workspace_bytes(B, *sizes) if self.group == 1 else
             L.detdecode_attention_shared_workspace_bytes(B, self.group, *sizes))
        self.ws["att"] = f((n + 3) // 4) if n else None
        # what fork and compact write: the next table, and the pages to copy
        self.next_table = i(max_batch, width)
        self.src, self.dst, self.tokens = i(B), i(B), i(B)
        self.itself = torch.arange(B, dtype=torch.int32, device=device)
        self.forked = False             # whether requests may share pages
        self.moved, self.moves = i(2, pages // 2), i(1)

    def _extend(self, new_tokens, rows, row_start, positions, slots):
        from bitwise_reproducible_fp32_gb300 import detlib as L
        B = self.B
        L.detpages_extend(self.lens, new_tokens, self.table, self.free, self.count,
                          self.page_size, rows, lens_out=self.after[:B],
                          free_count_out=self.after[B:], row_start=row_start,
                          positions=positions, slots=slots, dev_status=self.status)
        self.state.copy_(self.after)

    def prefill(self, requests, prompts):
        """Takes one prompt (a sequence of token ids) for each of the given empty
        requests, fills their cache, and returns what comes next after each (rows
        in the order of requests; no targets). The prompts run as one padded
        batch of the blocks' forward (at most 65,536 tokens each, what its attention
        takes). A request that finds too few free pages stays empty, and check()
        raises."""
        import torch

        from bitwise_reproducible_fp32_gb300 import block, detlib as L
        c, n = self.model, [len(p) for p in prompts]
        if len(requests) != len(prompts) or len(set(requests)) != len(requests) or not requests:
            raise ValueError("one prompt for each of one or more different requests")
        if min(n) < 1 or max(n) > self.max_len:
            raise ValueError(f"prompts must have 1..{self.max_len} tokens")
        if not all(0 <= r < self.B for r in requests):
            raise ValueError(f"requests must be in 0..{self.B - 1}")
        if any(self.lens[torch.tensor(requests)].tolist()):
            raise ValueError("a request still holds tokens; release it first")
        T, k = max(n), len(requests)
        # first what may refuse the sizes or find no memory: nothing is taken then
        blk = block.Block(k, T, c["d"], c["dff"], c["heads"], self.device, self.eps, self.theta)
        order = sorted(range(k), key=lambda a: requests[a])
        new = torch.zeros(self.B, dtype=torch.int32)
        tok = torch.zeros((k, T), dtype=torch.int32)
        # rows of the step are numbered through the requests in ascending order;
        # the padded batch's rows follow `requests`
        at = torch.full((k, T), sum(n), dtype=torch.int64)
        row = 0
        for a in order:
            new[requests[a]] = n[a]
            tok[a, :n[a]] = torch.as_tensor(prompts[a], dtype=torch.int32)
            at[a, :n[a]] = torch.arange(row, row + n[a])
            row += n[a]
        last = torch.tensor([a * T + n[a] - 1 for a in range(k)])
        i32 = lambda m: torch.empty(m, dtype=torch.int32, device=self.device)  # noqa: E731
        rows = sum(n) + 1
        slots = torch.empty(rows, dtype=torch.int64, device=self.device)
        self._extend(new.to(self.device), rows, i32(self.B + 1), i32(rows), slots)
        slots = slots.index_select(0, at.view(-1).to(self.device))
        x = L.detembedding_f32(c["emb"], tok.view(-1).to(self.device), dev_status=self.status)
        for w, (kc, vc) in zip(c["blocks"], self.cache):
            x = blk.forward(x, w)
            # the block's K is turned already
            for qkv, at in zip(blk.qkv.split(APPEND_ROWS), slots.split(APPEND_ROWS)):
                L.detkv_append_f32(qkv, at, kc, vc, self.H, dev_status=self.status)
        x = x.index_select(0, last.to(self.device))
        logits = L.detgemm_f32(x, c["head"], transB=True)
        none = torch.full((k,), -1, dtype=torch.int32, device=self.device)
        logp, entropy, ids, top_logp, _ = L.detlogprob_f32(logits, none, self.top_k,
                                                           want_stats=False,
                                                           dev_status=self.status)
        return Next(logits, ids, top_logp, entropy, logp)

    def step(self, tokens, active=None, targets=None):
        """One token more for every active request. tokens: max_batch int32 ids on
        the device; active: max_batch int32 values, 0 or 1 (default: all 1); the
        rows of the others hold nothing of use (their tokens must be ids all the
        same). targets: max_batch int32 ids whose log probabilities as the next
        tokens are wanted (default: none). Returns this object's Next buffers,
        which the next step overwrites. A request that is at max_len or finds no
        free page keeps its length and its cache, its rows hold nothing of use, and
        check() raises; the others go on as if it were inactive."""
        import torch

        from bitwise_reproducible_fp32_gb300 import detlib as L
        c, b, B = self.model, self.buf, self.B
        new = self.ones if active is None else active
        self._extend(new, B + 1, self.row_start, self.positions, self.slots)
        # an inactive request and one refused for its length take no row, so the
        # rows of those after them move up
        torch.gt(self.end, self.first, out=self.took)
        torch.where(self.took, self.first, self.past, out=self.row)
        pos = torch.index_select(self.positions, 0, self.row, out=self.pos)
        slots = torch.index_select(self.slots, 0, self.row, out=self.slot)
        x = L.detembedding_f32(c["emb"], tokens, out=b["x"], dev_status=self.status)
        for j, (w, (kc, vc)) in enumerate(zip(c["blocks"], self.cache)):
            if j:
                x = b["x"]
                L.detadd_rmsnorm_f32(b["x1"], b["dn"], w["g1"], self.eps, x=x, y=b["h"],
                                     inv_rms=self.inv)
            else:
                L.detrmsnorm_f32(x, w["g1"], self.eps, y=b["h"], inv_rms=self.inv)
            L.detgemm_f32(b["h"], w["W_qkv"], b["qkv"], workspace=self.ws["qkv"])
            q = L.detkv_append_f32(b["qkv"], slots, kc, vc, self.H, positions=pos,
                                   theta=self.theta, dev_status=self.status)
            kw = dict(out=b["att"], workspace=self.ws["att"], dev_status=self.status)
            if self.group == 1:
                L.detdecode_attention_f32(q, kc, vc, self.table, self.lens, self.H, **kw)
            else:
                L.detdecode_attention_shared_f32(q, kc, vc, self.table, self.lens, self.H,
                                                 self.group, **kw)
            L.detgemm_f32(b["att"], w["W_o"], b["o"], workspace=self.ws["o"])
            L.detadd_rmsnorm_f32(x, b["o"], w["g2"], self.eps, x=b["x1"], y=b["h2"],
                                 inv_rms=self.inv)
            L.detgemm_group_f32([dict(A=b["h2"], B=w["W_gate"], C=b["gate"]),
                                 dict(A=b["h2"], B=w["W_up"], C=b["up"])],
                                workspace=self.ws["gate_up"])
            L.detswiglu_f32(b["gate"], b["up"], out=b["s"])
            L.detgemm_f32(b["s"], w["W_down"], b["dn"], workspace=self.ws["down"])
        y = L.detadd_f32(b["x1"], b["dn"], out=b["y"])
        nx = self.next
        L.detgemm_f32(y, c["head"], nx.logits, transB=True, workspace=self.ws["head"])
        L.detlogprob_f32(nx.logits, self.none if targets is None else targets, self.top_k,
                         want_stats=False, logp=nx.logp, entropy=nx.entropy, top_ids=nx.ids,
                         top_logp=nx.top_logp, dev_status=self.status)
        return nx

    def release(self, done):
        """Gives back the pages of the requests with done[b] != 0 (max_batch int32 on
        the device); they are empty then."""
        import torch

        from bitwise_reproducible_fp32_gb300 import detlib as L
        B = self.B
        L.check_values(done, "done", torch.int32, B)
        # pages may be shared (a captured call may be replayed after a later fork):
        # everybody else goes on from itself, and a page that one of them holds stays
        if self.forked or (torch.cuda.is_current_stream_capturing() and self.pages <= FORK_PAGES):
            self._fork(torch.where(done != 0, self.none, self.itself))
            return
        L.detpages_release(self.lens, done, self.table, self.free, self.count, self.page_size,
                           lens_out=self.after[:B], free_count_out=self.after[B:],
                           dev_status=self.status)
        self.state.copy_(self.after)

    def _fork(self, parents):
        from bitwise_reproducible_fp32_gb300 import detlib as L
        B = self.B
        L.detpages_fork(self.lens, parents, self.table, self.free, self.count, self.page_size,
                        self.pages, table_out=self.next_table, lens_out=self.after[:B],
                        free_count_out=self.after[B:], src=self.src, dst=self.dst,
                        tokens=self.tokens, dev_status=self.status)
        self.state.copy_(self.after)

    def _knows_pages(self, what):
        if self.pages > FORK_PAGES:
            raise ValueError(f"{what} takes caches of up to {FORK_PAGES} pages")

    def fork(self, parents):
        """Every request goes on from request parents[b] (max_batch int32 on the device),
        with its tokens; -1 leaves it empty. Requests of one parent share its full
        pages and get copies of a partly filled one; the pages of requests that are
        nobody's parent are given back. Can be captured, as a step can. A request that
        finds no free page is left empty, and check() raises. For caches of up to 2^23
        pages."""
        from bitwise_reproducible_fp32_gb300 import detlib as L
        self._knows_pages("fork")
        self.forked = True
        self._fork(parents)
        self.table.copy_(self.next_table)
        for kc, vc in self.cache:
            L.detkv_copy_f32(kc, vc, self.src, self.dst, tokens=self.tokens,
                             dev_status=self.status)

    def compact(self):
        """Moves the pages that requests hold to the lowest ids, so that the rest of the
        cache is one run of free pages. Can be captured, as a step can. For caches of up to
        2^23 pages."""
        from bitwise_reproducible_fp32_gb300 import detlib as L
        self._knows_pages("compact")
        src, dst = self.moved
        L.detpages_compact(self.lens, self.table, self.free, self.page_size, table_out=self.table,
                           free_count_out=self.count, src=src, dst=dst, moves=self.moves,
                           dev_status=self.status)
        if self.pages > 1:
            for kc, vc in self.cache:
                L.detkv_copy_f32(kc, vc, src, dst, count=self.moves, dev_status=self.status)

    def check(self):
        """Raises if a call since the last check met a token outside the vocabulary,
        a request out of pages of its own or an empty free list. Waits for the device."""
        bits = int(self.status.item())
        self.status.zero_()
        if bits:
            raise ValueError(f"a token, target or length out of range, or no free page "
                             f"(status {bits})")

    def generate(self, prompts, new_tokens):
        """The new_tokens most probable tokens, one after the other, for up to
        max_batch prompts from an empty decoder. Returns (ids, logp): prompts x
        new_tokens. The requests are released after."""
        import torch
        k = len(prompts)
        if self.top_k < 1:
            raise ValueError("generate needs top_k of at least 1")
        ids = torch.empty((self.B, new_tokens), dtype=torch.int32, device=self.device)
        logp = torch.empty((self.B, new_tokens), dtype=torch.float32, device=self.device)
        active = torch.zeros(self.B, dtype=torch.int32, device=self.device)
        active[:k] = 1
        tok = torch.zeros(self.B, dtype=torch.int32, device=self.device)
        nx = self.prefill(list(range(k)), prompts)
        for t in range(new_tokens):
            if t:
                nx = self.step(tok, None if k == self.B else active)
            tok[:k] = nx.ids[:k, 0]
            ids[:k, t], logp[:k, t] = nx.ids[:k, 0], nx.top_logp[:k, 0]
        self.release(active)
        self.check()
        return ids[:k], logp[:k]

    def beam_search(self, prompts, new_tokens, beams, eos=-1, weights=None):
        """The `beams` (up to top_k) most probable answers of up to new_tokens tokens to each
        of up to max_batch // beams prompts, from an empty decoder, by beam search: each
        step keeps the best of all beams' top_k continuations (detbeam_select_f32). eos:
        the id that ends an answer. weights: floats on the device; answers are then
        ranked by score * weights[length]. For caches of up to 2^23 pages. Nothing waits for the host until the end. The
        requests are released after. Decoder(group=beams) reads what a prompt's beams share
        once. Returns Answers (prompts x beams)."""
        import torch

        from bitwise_reproducible_fp32_gb300 import detlib as L
        k, B = len(prompts), self.B
        n = k * beams
        if not 1 <= beams <= self.top_k:
            raise ValueError(f"beams must be in 1..{self.top_k}, the decoder's top_k")
        if not 1 <= n <= B or new_tokens < 1:
            raise ValueError(f"1..{B // beams} prompts and at least one new token")
        if max(map(len, prompts)) + new_tokens - 1 > self.table.size(1) * self.page_size:
            raise ValueError("the prompts leave no room for so many tokens")
        # what a later call would refuse, while no pages are taken
        if new_tokens > 1:
            self._knows_pages("beam search")
        if not -1 << 31 <= eos < 1 << 31:
            raise ValueError("eos must be an int32")
        if weights is not None:
            L.check_values(weights, "weights", torch.float32)
            if not weights.numel():
                raise ValueError("weights must hold at least one value")
        if self.lens[:n].any():
            raise ValueError("a request that the beams need still holds tokens; release it first")
        i32 = dict(dtype=torch.int32, device=self.device)
        hist = [torch.full((n, new_tokens), -1, **i32) for _ in range(2)]
        parents, tok = torch.arange(B, **i32), torch.zeros(B, **i32)
        active = torch.zeros(B, **i32)
        nx = self.prefill([r * beams for r in range(k)], prompts)
        # first each prompt is one beam
        b = L.detbeam_select_f32(torch.zeros((k, 1), dtype=torch.float32, device=self.device),
                                 nx.ids, nx.top_logp, beams, eos=eos, lens=torch.zeros(k, **i32),
                                 weights=weights, hist=hist[1][:k], hist_out=hist[0],
                                 dev_status=self.status)
        for t in range(1, new_tokens):
            # the prompts' requests are beams apart
            parents[:n] = b.forks if t > 1 else torch.where(b.forks < 0, -1, b.forks * beams)
            self.fork(parents)
            torch.clamp(b.tokens, min=0, out=tok[:n])
            active[:n] = 1 - b.finished
            nx = self.step(tok, active)
            b = L.detbeam_select_f32(b.scores, nx.ids[:n], nx.top_logp[:n], beams, eos=eos,
                                     finished=b.finished, lens=b.lens, weights=weights,
                                     hist=hist[(t - 1) % 2], hist_out=hist[t % 2],
                                     dev_status=self.status)
        active[:n] = 1
        self.release(active)
        self.check()
        col = torch.arange(new_tokens, **i32)
        ids = torch.where(col < b.lens[:, None], b.hist, -1)
        return Answers(ids.view(k, beams, new_tokens), b.lens.view(k, beams), b.scores)
