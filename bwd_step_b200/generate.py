"""Generation over the paged KV cache: the state of a set of requests
(PagedCache) and beam search on it.

Every step plans its pages on the GPU (Model.page_plan), runs the model over
the packed new tokens (Model.paged_forward), and for beam search selects the
next candidates (Model.beam_select) and moves the cache after them
(Model.beam_reorder_paged).  Lengths and back-pointers stay on the GPU.
"""
from __future__ import annotations

from . import _lib


class PagedCache:
    """The paged cache of `n_req` requests of at most `max_len` positions on the
    model's GPU: kv [n_layer, 2, pages, page_size, n_kv_head, head_dim], the block
    table, the free pages, and the arrays of the step planned last (cu_rows,
    kv_len, positions, slots)."""

    def __init__(self, model, n_pages, page_size, n_req, max_len, rows):
        import torch
        c = model.cfg
        ws_bytes = model.paged_workspace_bytes(n_req, rows)
        if ws_bytes == 0 or model.paged_kv_bytes(n_pages, page_size) == 0:
            raise ValueError(f"no paged cache of {n_pages} pages of {page_size} positions for {n_req} requests, {rows} rows")
        self.model, self.page_size, self.n_req = model, page_size, n_req
        dev = torch.device("cuda", model.device)
        i32 = dict(dtype=torch.int32, device=dev)
        self.kv = torch.empty(c.n_layer, 2, n_pages, page_size, c.n_kv_head, c.head_dim, dtype=model.weight_dtype,
                              device=dev)
        self.block_table = torch.full((n_req, -(-max_len // page_size)), -1, **i32)
        self.free_pages = torch.arange(n_pages, **i32)
        self.free_count = torch.tensor([n_pages], **i32)
        self.cu_rows = torch.zeros(n_req + 1, **i32)
        self.kv_len = torch.zeros(n_req, **i32)  # positions cached after the step planned last
        self._positions, self._slots = torch.empty(rows, **i32), torch.empty(rows, **i32)
        self.workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)

    def plan(self, new_len, rows, release=None, stream=None):
        """Plans a step of new_len [n_req] (device int32) new positions on top of
        kv_len, in `rows` packed rows, after giving back the requests of release."""
        if not 1 <= rows <= self._positions.numel():
            raise ValueError(f"rows must be 1 to {self._positions.numel()}, the rows that the cache was made for, got {rows}")
        self.positions, self.slots = self._positions[:rows], self._slots[:rows]
        self.model.page_plan(self.page_size, self.kv_len, new_len, self.block_table, self.free_pages, self.free_count,
                             self.cu_rows, self.kv_len, self.positions, self.slots, release=release, stream=stream)

    def forward(self, tokens, weights, logits, max_new=0, stream=None):
        """The planned step over its packed tokens [rows]: logits [n_req, V] of every
        request's last new token."""
        self.model.paged_forward(tokens, self.positions, self.cu_rows, self.kv_len, self.slots, self.block_table, weights,
                                 self.kv, logits, self.workspace, max_new=max_new, stream=stream)


def beam_search(model, weights, prompts, beams, max_new_tokens, eos=-1, page_size=64):
    """The `beams` best continuations of every prompt (lists of token ids) by
    cumulative log-probability, max_new_tokens long (ended ones repeat eos):
    tokens [prompts, beams, max_new_tokens] (int64) and scores [prompts, beams],
    best first, on the model's GPU.

    A prompt is computed once; its full pages are then shared by its beams, and
    what follows is each beam's own.
    """
    import torch
    if not prompts or any(len(p) == 0 for p in prompts):
        raise ValueError("every prompt needs a token")
    if max_new_tokens < 1:
        raise ValueError("max_new_tokens must be positive")
    if not 1 <= beams <= _lib.NC_MAX_BEAMS:
        raise ValueError(f"beams must be 1 to {_lib.NC_MAX_BEAMS}")
    b, k, v = len(prompts), beams, model.cfg.vocab
    lens = [len(p) for p in prompts]
    blocks = [-(-(n + max_new_tokens) // page_size) for n in lens]
    cache = PagedCache(model, k * sum(blocks), page_size, b * k, max(lens) + max_new_tokens, max(sum(lens), b * k))
    dev = cache.kv.device
    i32 = dict(dtype=torch.int32, device=dev)
    first = torch.tensor([n for n in lens for _ in range(k)], **i32)  # prompt lengths of the rows
    lead = torch.tensor([1] + [0] * (k - 1), **i32).repeat(b)
    # the prompts, in the first beam of each row
    cache.plan(first * lead, sum(lens))
    logits = torch.empty(b * k, v, dtype=model.weight_dtype, device=dev)
    tokens = torch.tensor([t for p in prompts for t in p], **i32)
    cache.forward(tokens, weights, logits, max_new=max(lens))
    # its full pages to the other beams' tables; the part of a page after them is copied by the first reorder
    shared = (first // page_size)[:, None]
    lead_table = cache.block_table.view(b, k, -1)[:, :1].expand(b, k, cache.block_table.shape[1]).reshape(b * k, -1)
    in_shared = torch.arange(cache.block_table.shape[1], device=dev)[None, :] < shared
    cache.block_table.copy_(torch.where(in_shared, lead_table, cache.block_table))
    starts = (first // page_size) * page_size
    cache.kv_len.copy_(first)
    scores = torch.full((b, k), float("-inf"), dtype=torch.float32, device=dev)
    scores[:, 0] = 0.0  # one beam so far
    ends = eos >= 0
    finished = torch.zeros(b, k, **i32) if ends else None
    got, back = [], []
    one = torch.ones(b * k, **i32)
    for step in range(max_new_tokens):
        nxt, parents = torch.empty(b, k, **i32), torch.empty(b, k, **i32)
        model.beam_select(logits, scores, scores, nxt, parents, eos=eos, finished=finished, finished_out=finished)
        got.append(nxt)
        back.append(parents)
        if step + 1 == max_new_tokens:
            break
        cached = cache.kv_len.clone()
        cache.plan(one, b * k)
        model.beam_reorder_paged(cache.kv, parents, cache.block_table, starts, cached)
        cache.forward(nxt.view(-1), weights, logits, max_new=1)
    # the tokens along the back-pointers
    at = torch.arange(k, device=dev).expand(b, k)
    out = []
    for nxt, parents in zip(reversed(got), reversed(back)):
        out.append(nxt.gather(1, at))
        at = parents.gather(1, at).long()
    code = model.check()
    if code != 0:
        from .api import NcError
        raise NcError(code, "beam_search")
    return torch.stack(out[::-1], dim=2).long(), scores
