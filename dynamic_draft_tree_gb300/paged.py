"""A paged KV cache and the target rows' token state around a draft-tree round (call sequences, no arithmetic).

``PagedCache`` holds the pages of every layer, the block pool, and the temporary KV of the tree that is being verified,
and strings dt_kv_reserve, dt_commit_kv_paged, dt_tree_attention and dt_kv_release together; around the rounds it has the
prompts' attention (dt_prompt_attention) and requests that continue others (dt_kv_fork, dt_kv_release_shared).
``TokenState`` holds what dt_logits_process needs of a batch of requests, ``TokenLogprobs`` the log probabilities of what a
round answers (dt_token_logprobs). They are handed to ``RoundRunner.run`` (``kv=``, ``tokens=``, ``logprobs=``), or used
by themselves. Every call is asynchronous on the current stream, so a round with them can be captured in a CUDA graph.
"""
import torch

from . import (BlockPool, dt_commit_kv_paged, dt_count_tokens, dt_kv_fork, dt_kv_release, dt_kv_release_shared, dt_kv_reserve,
               dt_logits_process, dt_prompt_attention, dt_prompt_attention_workspace, dt_token_logprobs,
               dt_token_logprobs_workspace, dt_tree_attention, dt_tree_attention_workspace)


class PagedCache:
    """Pages of ``layers`` layers for B requests, and the temporary KV rows of their trees.

    pages [2 * layers][n_blocks][page][H_kv][D]: plane 2 l holds layer l's keys, plane 2 l + 1 its values.
    tmp: the verify forward's keys and values, [2 * layers][B][P][H_kv][D], or [2 * layers][B * P][H_kv][D] with
    ``packed`` (row meta.row_off[b] + i), written by the forward before it attends.
    shared_len: tokens, a multiple of the page, of a prefix that all requests share (``prefix`` fills it once). Its pages
    are in the pool once, stand first in every request's table, and stay there when requests end.
    forks: requests may continue others (``fork``); the pool then counts the owners of its blocks.
    """

    refs = None              # owners of every block beyond its first, with ``forks``
    prompt_workspace = None  # of ``attend_prompts``, made by its first call

    def __init__(self, h, B, P, layers, H_q, H_kv, D, n_blocks, max_blocks, page=16, D_path=64, dtype=torch.bfloat16,
                 packed=False, shared_len=0, device="cuda", forks=False):
        if shared_len < 0 or shared_len % page or shared_len > max_blocks * page:
            raise ValueError("shared_len must be a multiple of page within max_blocks")
        self.h, self.B, self.P, self.H_q, self.H_kv, self.D = h, B, P, H_q, H_kv, D
        self.packed, self.shared_len, self.filled = packed, shared_len, False
        self.pages = torch.zeros((2 * layers, n_blocks, page, H_kv, D), dtype=dtype, device=device)
        rows = (B * P,) if packed else (B, P)
        self.tmp = torch.zeros((2 * layers, *rows, H_kv, D), dtype=dtype, device=device)
        self.pool = BlockPool.empty(B, max_blocks, n_blocks, page, device)
        self.seq_len = torch.zeros((B,), dtype=torch.int32, device=device)
        self.slots = torch.empty((B, D_path), dtype=torch.int64, device=device)
        self.committed = torch.zeros((B,), dtype=torch.int32, device=device)  # tokens that the last commit appended
        self.workspace = dt_tree_attention_workspace(h, B, P, H_q, H_kv, D, shared=shared_len > 0)
        if forks:
            self.refs = torch.zeros((n_blocks,), dtype=torch.int32, device=device)

    def prefix(self, tmp, stream=None):
        """Fills the shared prefix, before any other call: tmp [2 * layers][shared_len][H_kv][D]. Every request owns its
        pages from then on and has the length shared_len. Without pages for it (DT_DEV_KV_FULL) nothing changes."""
        n, blocks = self.shared_len, self.shared_len // self.pool.page
        if n == 0 or tmp.shape[1] != n or self.filled:
            raise ValueError("tmp must hold the shared_len rows of the prefix, which is filled once")
        self.filled = True
        with torch.cuda.stream(stream):
            n_new = torch.full((1,), n, dtype=torch.int32, device=tmp.device)
            slots = torch.empty((1, n), dtype=torch.int64, device=tmp.device)
            table, owned, length = self.pool.block_table, self.pool.n_owned, self.seq_len
            dt_kv_reserve(self.h, self.pool, length[:1], n_new, slots)  # request 0's, then everybody's
            dt_commit_kv_paged(self.h, tmp.unsqueeze(1), self.pages, slots, n_new, length[:1], length[:1])
            table[1:, :blocks] = table[:1, :blocks]
            owned[1:] = owned[:1]
            length[1:] = length[:1]

    def prefill(self, tmp, n_new, row_off, stream=None):
        """Appends the prompts' KV rows: tmp [2 * layers][rows][H_kv][D], request b's n_new[b] rows at row_off[b]."""
        # memory of the stream that the calls run on: nothing queued elsewhere still uses it, nor will before they have run
        with torch.cuda.stream(stream):
            slots = torch.empty((tmp.shape[1],), dtype=torch.int64, device=tmp.device)
        dt_kv_reserve(self.h, self.pool, self.seq_len, n_new, slots, slot_off=row_off, stream=stream)
        dt_commit_kv_paged(self.h, tmp, self.pages, slots, n_new, self.seq_len, self.seq_len, row_off=row_off,
                           slot_off=row_off, stream=stream)

    def attend_prompts(self, layer, q, k, v, row_off, out, scale=None, stream=None):
        """A layer's prompts, or chunks of them, before ``prefill`` appends their rows: q and out [rows][H_q][D], k and v
        [rows][H_kv][D], request b's rows at row_off[b], causal and behind the tokens that are in the pages. Calls of one
        cache share a workspace: one stream at a time. The first one makes it, so that a capture of it is refused."""
        if self.prompt_workspace is None:
            with torch.cuda.stream(stream):  # memory of the stream that the calls run on
                if torch.cuda.is_current_stream_capturing():
                    raise RuntimeError("a cache's first attend_prompts makes its workspace: run one before the capture")
                self.prompt_workspace = dt_prompt_attention_workspace(self.h, self.B, self.H_q, self.H_kv, self.D)
        dt_prompt_attention(self.h, q, k, v, row_off, out, self.prompt_workspace, k_pages=self.pages[2 * layer],
                            v_pages=self.pages[2 * layer + 1], block_table=self.pool.block_table, seq_len=self.seq_len,
                            scale=scale, stream=stream)

    def fork(self, src, dst, length=None, stream=None):
        """Places dst, which own nothing (but the shared prefix), continue requests src behind their first ``length`` tokens
        (default: all of them): int32 tensors, one entry a fork. Token histories go along by ``TokenState.fork``. One that finds
        no page (DT_DEV_KV_FULL) owns nothing still, and its length stays what the place's last request left."""
        if self.refs is None:
            raise ValueError("the cache was made without forks")
        dt_kv_fork(self.h, self.pool, self.refs, self.pages, src, dst, self.seq_len, length=length, shared_len=self.shared_len,
                   stream=stream)

    def attend(self, layer, q, out, meta, scale=None, stream=None):
        """The tree's query rows of a layer (rows as tmp) against the cache and the layer's tmp rows."""
        dt_tree_attention(self.h, q, self.tmp[2 * layer], self.tmp[2 * layer + 1], self.pages[2 * layer],
                          self.pages[2 * layer + 1], self.pool.block_table, self.seq_len, meta.n_pos, out,
                          self.workspace, mask=meta.mask, row_off=meta.row_off if self.packed else None, P=self.P,
                          shared_len=self.shared_len, scale=scale, stream=stream)

    def commit(self, accept_len, accept_path, meta=None, stream=None):
        """Appends the root's and the accepted positions' rows of tmp (after dt_verify); meta with ``packed``. A request
        that finds no pages keeps its length, and its entry of ``committed`` is 0."""
        dt_kv_reserve(self.h, self.pool, self.seq_len, accept_len, self.slots, n_extra=1, stream=stream)
        dt_commit_kv_paged(self.h, self.tmp, self.pages, self.slots, accept_len, self.seq_len, self.seq_len,
                           path=accept_path, n_extra=1, row_off=meta.row_off if self.packed else None,
                           P=self.P if self.packed else None, committed=self.committed, stream=stream)

    def release(self, keep_len, stream=None):
        """Gives back every request's pages past keep_len tokens (0 ends a request); the lengths are the caller's. Pages of
        the shared prefix stay in every table, and a new request's length is shared_len. With ``forks``, pages that other
        requests own stay theirs."""
        if self.shared_len:
            with torch.cuda.stream(stream):
                keep_len = keep_len.clamp(min=self.shared_len)
        if self.refs is not None:
            dt_kv_release_shared(self.h, self.pool, self.refs, keep_len, stream=stream)
        else:
            dt_kv_release(self.h, self.pool, keep_len, stream=stream)


class TokenState:
    """Token history, penalties, biases and grammar words of a batch (the arguments of dt_logits_process)."""

    def __init__(self, h, B, repetition=None, frequency=None, presence=None, bias_ids=None, bias_vals=None, allow=None,
                 device="cuda"):
        self.h = h
        self.counts = torch.zeros((B, h.cfg.V), dtype=torch.int32, device=device)
        self.repetition, self.frequency, self.presence = repetition, frequency, presence
        self.bias_ids, self.bias_vals, self.allow = bias_ids, bias_vals, allow

    def prompt(self, tokens, n_new, row_off=None, stream=None):
        """Marks prompt tokens ([B][P], or packed by row_off)."""
        dt_count_tokens(self.h, self.counts, tokens, n_new, row_off=row_off, prompt=True, stream=stream)

    def fork(self, src, dst, stream=None):
        """Places dst get the histories of requests src (int32 tensors, as for ``PagedCache.fork``, which takes pages and lengths along):
        a fork behind all of its source's tokens. (One behind fewer has a history of its own: a cleared row and ``prompt``.)
        Pairs that ``PagedCache.fork`` refuses for their places (outside the batch, a destination named before, a source
        that is a destination) leave the histories as they are."""
        with torch.cuda.stream(stream):
            B = self.counts.shape[0]
            ok = (src >= 0) & (src < B) & (dst >= 0) & (dst < B) & ~(src[:, None] == dst).any(1)
            ok &= ~(dst[:, None] == dst).tril(-1).any(1)
            s, d = (torch.where(ok, x, 0) for x in (src, dst))
            # differences are added, zero for pairs that are left out: no place is written twice, nor one outside
            self.counts.index_add_(0, d, (self.counts[s] - self.counts[d]) * ok[:, None])

    def process(self, logits, meta, packed=False, out=None, stream=None):
        """Target rows prepared for the verify, in place or into ``out``."""
        out = logits if out is None else out
        dt_logits_process(self.h, logits, out, meta.n_pos, tokens=meta.tokens, mask=meta.mask,
                          row_off=meta.row_off if packed else None, counts=self.counts, repetition=self.repetition,
                          frequency=self.frequency, presence=self.presence, bias_ids=self.bias_ids,
                          bias_vals=self.bias_vals, allow=self.allow, P=meta.P, stream=stream)
        return out

    def commit(self, accept_len, accept_path, meta, stream=None, committed=None):
        """Counts the root's and the accepted positions' tokens; with ``committed`` (PagedCache.committed after its
        commit) only those whose KV is in the pages, so that a refused request keeps its history as it keeps its length."""
        n_new, n_extra = (accept_len, 1) if committed is None else (committed[:accept_len.numel()], 0)
        dt_count_tokens(self.h, self.counts, meta.tokens, n_new, path=accept_path, n_extra=n_extra, stream=stream)


class TokenLogprobs:
    """Log probabilities of the tokens that a round answers, under the target rows that it verified, with the rows' entropies,
    the tokens' ranks and K alternatives: entry j of request b, j <= accept_len[b], is the token behind the j-th position of its
    accepted path (the last one the bonus token), in logp, entropy and rank [B][D_path], top_ids and top_logp [B][D_path][K].
    Rows that ``TokenState`` processed in place are the processed ones."""

    def __init__(self, h, B, D_path, K=0, device="cuda"):
        self.h, self.K = h, K
        self.logp = torch.zeros((B, D_path), dtype=torch.float32, device=device)
        self.entropy = torch.zeros((B, D_path), dtype=torch.float32, device=device)
        self.rank = torch.zeros((B, D_path), dtype=torch.int32, device=device)
        self.top_ids = torch.zeros((B, D_path, K), dtype=torch.int32, device=device) if K else None
        self.top_logp = torch.zeros((B, D_path, K), dtype=torch.float32, device=device) if K else None
        self.workspace = dt_token_logprobs_workspace(h, B * D_path, K)

    def round(self, logits, accept_len, accept_path, bonus, meta, packed=False, stream=None):
        """The round's entries (after dt_verify, on the rows that it verified)."""
        if accept_path.shape != self.logp.shape:
            raise ValueError("accept_path must have the shape of the outputs")
        dt_token_logprobs(self.h, logits, accept_len, self.logp, self.workspace, tokens=meta.tokens, last=bonus, n_extra=1,
                          path=accept_path, row_off=meta.row_off if packed else None, entropy=self.entropy, rank=self.rank,
                          top_ids=self.top_ids, top_logp=self.top_logp, P=meta.P, stream=stream)
