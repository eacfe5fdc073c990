"""The serving operators over a paged KV cache and of beam search, as cases with their plain forms.

  plan       block tables, slot maps and positions of a step, built on the GPU from the requests' lengths
  attention  a chunk of new tokens of every request (one token for a decoding request): its K and V written
             to their pages, and its queries attending over the paged cache
  select     beam search's selection: the best candidates over beams and vocabulary, with back-pointers
  reorder    the generated part of the KV cache moved to follow those back-pointers, dense or paged

`run` computes the plain form in elementary torch operations, or, where `own` is true, makes the calls that a
program makes of the framework.  The lengths of a case are part of the case (drawn from its number "lens"),
its contents come from the seed.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
VOCAB = 65536  # the workloads' vocabulary


def listed():
    return [
        # The smallest step: four requests, each decoding one token, of which some step onto a new page.
        dict(name="plan 4 decoding", op="plan", requests=4, page=16, max_blocks=64, cached_lo=1, cached_hi=900,
             chunked=0, new_lo=1, new_hi=1, released=0, idle=0, pad_rows=0, lens=1),
        # A large step of continuous batching: most requests decode, finished ones give their pages back and
        # prompts take their place in chunks.
        dict(name="plan 512 with turnover", op="plan", requests=512, page=16, max_blocks=256, cached_lo=1,
             cached_hi=3000, chunked=48, new_lo=65, new_hi=1024, released=32, idle=9, pad_rows=37, lens=2),
        # Four requests decoding with the depth-20 model's heads: latency counts.
        dict(name="attention 4 decoding", op="attention", dtype="bf16", heads=10, kv_heads=1, head_dim=128, page=16,
             requests=4, cached_lo=100, cached_hi=700, chunked=0, new_lo=1, new_hi=1, idle=0, pad_rows=0, lens=3),
        # A full batch decoding at ragged lengths up to the long workload's 8192 positions.
        dict(name="attention 128 decoding", op="attention", dtype="bf16", heads=10, kv_heads=1, head_dim=128, page=64,
             requests=128, cached_lo=900, cached_hi=8191, chunked=0, new_lo=1, new_hi=1, idle=2, pad_rows=6, lens=4),
        # Prompts of the 12-head model entering in chunks on what is cached of them already.
        dict(name="attention chunks 64 wide", op="attention", dtype="bf16", heads=12, kv_heads=1, head_dim=64,
             page=32, requests=8, cached_lo=0, cached_hi=700, chunked=8, new_lo=150, new_hi=300, idle=0, pad_rows=0,
             lens=5),
        # Decoding requests and prompt chunks in one step, the depth-30 model's 15 heads.
        dict(name="attention mixed", op="attention", dtype="bf16", heads=15, kv_heads=1, head_dim=128, page=16,
             requests=40, cached_lo=33, cached_hi=1900, chunked=6, new_lo=64, new_hi=256, idle=1, pad_rows=3, lens=6),
        # Long prompts: the largest chunks over the longest caches.
        dict(name="attention long chunks", op="attention", dtype="bf16", heads=10, kv_heads=1, head_dim=128, page=128,
             requests=2, cached_lo=5000, cached_hi=6100, chunked=2, new_lo=1900, new_hi=2048, idle=0, pad_rows=0,
             lens=7),
        # The fp32 path with the tiny workload's 16-wide heads.
        dict(name="attention fp32 16 wide", op="attention", dtype="fp32", heads=4, kv_heads=1, head_dim=16, page=16,
             requests=5, cached_lo=0, cached_hi=90, chunked=2, new_lo=3, new_hi=21, idle=1, pad_rows=2, lens=8),
        # One prompt with four beams: latency counts.
        dict(name="select 1x4", op="select", dtype="bf16", batch=1, beams=4, vocab=VOCAB, finished=0),
        # A batch of prompts with eight beams each, some of them at their end.
        dict(name="select 64x8", op="select", dtype="bf16", batch=64, beams=8, vocab=VOCAB, finished=40),
        # The dense cache of the depth-20 model after 250 generated positions.
        dict(name="reorder dense 16x4", op="reorder", dtype="bf16", batch=16, beams=4, layers=20, kv_heads=1,
             head_dim=128, page=0, start=130, end=380, t_max=512, lens=9),
        # The paged cache of the 12-layer model, ragged: every request has its own prompt and generated lengths.
        dict(name="reorder paged 3x3", op="reorder", dtype="bf16", batch=3, beams=3, layers=12, kv_heads=1,
             head_dim=64, page=16, start=20, end=120, t_max=160, lens=10),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


HEADS = [(10, 1, 128), (12, 1, 64), (15, 1, 128), (4, 1, 16), (4, 2, 32), (8, 2, 64), (6, 3, 128), (16, 1, 128),
         (5, 5, 64), (2, 1, 128)]


def _draw(rng):
    op = rng.choice(["plan", "attention", "attention", "attention", "select", "reorder"])
    lens = rng.randrange(1 << 30)
    if op == "plan":
        requests, page = _log(rng, 1, 512), rng.choice([16, 32, 64, 128])
        chunked = rng.randrange(requests // 4 + 1)
        new_lo = _log(rng, 2, 500)
        new_hi = new_lo + _log(rng, 1, 500)
        cached_hi = _log(rng, 1, 4000)
        return dict(op=op, requests=requests, page=page, max_blocks=(cached_hi + new_hi + 1) // page + 2, cached_lo=0,
                    cached_hi=cached_hi, chunked=chunked, new_lo=new_lo, new_hi=new_hi,
                    released=rng.randrange(requests // 3 + 1), idle=rng.randrange(requests // 5 + 1),
                    pad_rows=rng.randrange(40), lens=lens)
    if op == "attention":
        h, nkv, hd = rng.choice(HEADS)
        dtype = "fp32" if rng.random() < 0.15 else "bf16"
        small = dtype == "fp32" or hd < 64  # these heads' models are small
        requests = _log(rng, 1, 6 if small else 128)
        chunked = rng.choice([0, 0, requests, rng.randrange(requests + 1)])
        new_lo = _log(rng, 1, 40 if small else 1000)
        new_hi = new_lo + _log(rng, 1, 20 if small else 800)
        cached_lo = rng.choice([0, _log(rng, 1, 100)])
        return dict(op=op, dtype=dtype, heads=h, kv_heads=nkv, head_dim=hd, page=rng.choice([16, 32, 64, 128, 256]),
                    requests=requests, cached_lo=cached_lo, cached_hi=cached_lo + _log(rng, 1, 300 if small else 8000),
                    chunked=chunked, new_lo=new_lo if chunked else 1, new_hi=new_hi if chunked else 1,
                    idle=rng.randrange(requests // 6 + 1), pad_rows=rng.randrange(6), lens=lens)
    if op == "select":
        batch, beams = _log(rng, 1, 64), rng.randrange(1, 17)
        return dict(op=op, dtype="fp32" if rng.random() < 0.2 else "bf16", batch=batch, beams=beams,
                    vocab=64 * _log(rng, 2, VOCAB // 64), finished=rng.randrange(batch * beams // 4 + 1))
    _, nkv, hd = rng.choice(HEADS)
    start = _log(rng, 1, 200)
    end = start + _log(rng, 1, 250)
    return dict(op=op, dtype="fp32" if rng.random() < 0.2 else "bf16", batch=_log(rng, 1, 16), beams=rng.randrange(2, 17),
                layers=rng.randrange(1, 21), kv_heads=nkv, head_dim=hd, page=rng.choice([0, 0, 16, 32, 64]), start=start,
                end=end, t_max=end + rng.randrange(100), lens=lens)


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


# The most values that the plain attention may hold at once: its scores, and the gathered keys, in 32 bits.
MOST_VALUES = 600e6


def _plain_values(c):
    if c["op"] == "reorder":
        return c["batch"] * c["beams"] * c["t_max"] * c["layers"] * 2 * c["kv_heads"] * c["head_dim"]
    if c["op"] != "attention":
        return 0
    cached, new = _lengths(c)
    keys = (max(k + n for k, n in zip(cached, new)) + c["page"]) * c["requests"]
    return max(keys * c["kv_heads"] * c["head_dim"], keys * max(new) * c["heads"])


def draw(rng):
    most = max(_cost(c) for c in listed())
    while True:
        case = _draw(rng)
        if _cost(case) <= most and _plain_values(case) <= MOST_VALUES:
            return case


# ---------------------------------------------------------------------------------------------- inputs

def _lengths(c):
    """Cached and new positions of every request (released requests start anew: their `cached` is the old length)."""
    rng = random.Random(c["lens"])
    n = c["requests"]
    cached = [rng.randint(c["cached_lo"], c["cached_hi"]) for _ in range(n)]
    new = [1] * n
    order = list(range(n))
    rng.shuffle(order)
    for r in order[:c["chunked"]]:
        new[r] = rng.randint(c["new_lo"], c["new_hi"])
    for r in order[n - c["idle"]:] if c["idle"] else []:
        new[r] = 0
    if sum(new) == 0:
        new[0] = 1
    return cached, new


def _released(c):
    rng = random.Random(c["lens"] + 1)
    rel = [0] * c["requests"]
    for r in rng.sample(range(c["requests"]), c["released"]):
        rel[r] = 1
    return rel


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _blocks(n, page):
    return -(-n // page)


def _tables(lens, page, max_blocks, n_pages, g):
    """Block tables in which every request's blocks have pages of their own, in no order; the rest is -1.
    Returns the table and the pages that are left, as a stack."""
    perm = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    count = torch.tensor([_blocks(n, page) for n in lens], device=DEV)
    first = torch.cumsum(count, 0) - count
    j = torch.arange(max_blocks, device=DEV)
    at = (first[:, None] + j[None, :]).clamp(max=n_pages - 1)
    table = torch.where(j[None, :] < count[:, None], perm[at], torch.full_like(perm[at], -1))
    return table.contiguous(), perm[int(count.sum()):].contiguous()


def _rms(x):
    return x / x.square().mean(-1, keepdim=True).sqrt()


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return {"plan": _prepare_plan, "attention": _prepare_attention, "select": _prepare_select,
            "reorder": _prepare_reorder}[case["op"]](case, g)


def _prepare_plan(c, g):
    cached, new = _lengths(c)
    rel = _released(c)
    used = sum(_blocks(n, c["page"]) for n in cached)
    more = sum(_blocks((0 if x else k) + n, c["page"]) for k, n, x in zip(cached, new, rel))
    n_pages = max(used, 1) + more + 7
    table, free = _tables(cached, c["page"], c["max_blocks"], n_pages, g)
    stack = torch.full((n_pages,), -1, dtype=torch.int32, device=DEV)
    stack[:free.numel()] = free
    rows = sum(new) + c["pad_rows"]
    e = lambda n: torch.empty(n, dtype=torch.int32, device=DEV)  # noqa: E731
    return dict(case=c, cached=_ints(cached), new=_ints(new), release=_ints(rel), table=table, free=stack,
                free_count=_ints([free.numel()]), cu=e(c["requests"] + 1), kv_len=e(c["requests"]), positions=e(rows),
                slots=e(rows))


def _prepare_attention(c, g):
    t, (h, nkv, hd, page) = TYPES[c["dtype"]], (c["heads"], c["kv_heads"], c["head_dim"], c["page"])
    cached, new = _lengths(c)
    total = [k + n for k, n in zip(cached, new)]
    rows, n_pages = sum(new) + c["pad_rows"], sum(_blocks(n, page) for n in total) + 3
    max_blocks = _blocks(c["cached_hi"] + max(c["new_hi"], 1), page)
    table, _ = _tables(total, page, max_blocks, n_pages, g)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV)
    # q and k as QK-norm and RoPE leave them, of unit mean square, with a part that heads and positions share
    qkv = normal(rows, h + 2 * nkv, hd)
    qkv[:, :h + nkv] = _rms(qkv[:, :h + nkv] + 0.7 * normal(1, 1, hd))
    k = torch.empty(n_pages, page, nkv, hd, dtype=t, device=DEV)
    step = max(1, (1 << 26) // (page * nkv * hd))
    for i in range(0, n_pages, step):
        k[i:i + step] = _rms(normal(min(step, n_pages - i), page, nkv, hd) + 0.7 * normal(1, 1, 1, hd)).to(t)
    v = torch.empty_like(k)
    for i in range(0, n_pages, step):
        v[i:i + step] = normal(min(step, n_pages - i), page, nkv, hd).to(t)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    cu = _ints(cu)
    i = torch.arange(cu[-1].item(), device=DEV)
    r = torch.searchsorted(cu[1:].long(), i, right=True)
    pos = _ints(cached).long()[r] + i - cu.long()[r]
    slots = torch.full((rows,), -1, dtype=torch.int32, device=DEV)
    slots[:i.numel()] = (table.long()[r, pos // page] * page + pos % page).to(torch.int32)
    return dict(case=c, qkv=qkv.reshape(rows, -1).to(t), k=k, v=v, table=table, cu=cu, kv_len=_ints(total), slots=slots,
                o=torch.zeros(rows, h * hd, dtype=t, device=DEV), total=sum(new), max_new=max(new))


def _prepare_select(c, g):
    b, k, v = c["batch"], c["beams"], c["vocab"]
    # softcapped logits: a broad normal with a few likely ids, of the model's range (-15, 15)
    z = torch.randn(b, k, v, generator=g, device=DEV) * 2.0
    likely = torch.randint(0, v, (b, k, 12), generator=g, device=DEV)
    z.scatter_add_(2, likely, 6.0 + 4.0 * torch.rand(b, k, 12, generator=g, device=DEV))
    logits = (15.0 * torch.tanh(z / 15.0)).to(TYPES[c["dtype"]])
    scores = -5.0 - 10.0 * torch.rand(b, k, generator=g, device=DEV)
    scores = torch.sort(scores, dim=1, descending=True).values.contiguous()
    at = torch.randperm(b * k, generator=g, device=DEV)[:c["finished"]]
    fin = torch.zeros(b * k, dtype=torch.int32, device=DEV)
    fin[at] = 1
    e = lambda: torch.empty(b, k, dtype=torch.int32, device=DEV)  # noqa: E731
    return dict(case=c, logits=logits, scores=scores, finished=fin.view(b, k), eos=v // 3, scores_out=torch.empty_like(scores),
                tokens=e(), parents=e(), finished_out=e())


def _spans(c):
    """First and last positions that the beams of each row differ in: one span for a dense cache, ragged for a paged one."""
    rng = random.Random(c["lens"])
    if not c["page"]:
        return [(c["start"], c["end"])] * c["batch"]
    got = []
    for _ in range(c["batch"]):
        a = rng.randint(0, c["start"])
        got.append((a, rng.randint(a, c["end"])))
    got[0] = (c["start"], c["end"])
    return got


def _parents(c):
    """Back-pointers as the selection gives them: the better beams have more children."""
    rng = random.Random(c["lens"] + 2)
    k = c["beams"]
    return [[min(k - 1, int(k * rng.random() ** 1.7)) for _ in range(k)] for _ in range(c["batch"])]


def _prepare_reorder(c, g):
    t, rows, w = TYPES[c["dtype"]], c["batch"] * c["beams"], (c["kv_heads"], c["head_dim"])
    spans = _spans(c)
    s = dict(case=c, parents=_ints(_parents(c)))
    if c["page"]:
        ends = [e for _, e in spans for _ in range(c["beams"])]
        max_blocks = _blocks(c["t_max"], c["page"])
        n_pages = sum(_blocks(e, c["page"]) for e in ends) + 2
        s["table"], _ = _tables(ends, c["page"], max_blocks, n_pages, g)
        s["start"] = _ints([a for a, _ in spans for _ in range(c["beams"])])
        s["end"] = _ints(ends)
        shape = (c["layers"], 2, n_pages, c["page"]) + w
    else:
        shape = (c["layers"], 2, rows, c["t_max"]) + w
    cache = torch.empty(shape, dtype=t, device=DEV)
    for layer in range(c["layers"]):
        cache[layer] = torch.randn(shape[1:], generator=g, device=DEV).to(t)
    s["cache"] = cache
    return s


# ---------------------------------------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return {"plan": _own_plan, "attention": _own_attention, "select": _own_select, "reorder": _own_reorder}[op](state)
    return {"plan": _plan, "attention": _attention, "select": _select, "reorder": _reorder}[op](state)


_models = {}


def _model(c):
    """The handle that a program makes once for its model."""
    key = (c.get("vocab", VOCAB), c.get("layers", 1), c.get("heads", c.get("kv_heads", 1)), c.get("kv_heads", 1),
           c.get("head_dim", 128), c.get("dtype", "bf16"))
    if key not in _models:
        from bwd_step_b200 import Model
        v, layers, h, nkv, hd, t = key
        _models[key] = Model(dict(vocab=v, d_model=64, n_layer=layers, n_head=h, n_kv_head=nkv, head_dim=hd, mlp_mult=4,
                                  softcap=15.0, rope_base=10000.0), t)
    return _models[key]


def _own_plan(s):
    _model(s["case"]).page_plan(s["case"]["page"], s["cached"], s["new"], s["table"], s["free"], s["free_count"], s["cu"],
                                s["kv_len"], s["positions"], s["slots"], release=s["release"])
    return [s[k] for k in ("table", "free", "free_count", "cu", "kv_len", "positions", "slots")]


def _own_attention(s):
    m = _model(s["case"])
    if "ws" not in s:
        s["ws"] = torch.empty(m.paged_attention_workspace_bytes(s["kv_len"].numel(), s["qkv"].shape[0]),
                              dtype=torch.uint8, device=DEV)
    m.paged_attention(s["qkv"], s["cu"], s["kv_len"], s["slots"], s["table"], s["k"], s["v"], s["o"], s["ws"],
                      max_new=s["max_new"])
    return [s["o"], s["k"], s["v"]]


def _own_select(s):
    _model(s["case"]).beam_select(s["logits"], s["scores"], s["scores_out"], s["tokens"], s["parents"], eos=s["eos"],
                                  finished=s["finished"], finished_out=s["finished_out"])
    return [s["scores_out"], s["tokens"], s["parents"], s["finished_out"]]


def _own_reorder(s):
    c, m = s["case"], _model(s["case"])
    if c["page"]:
        m.beam_reorder_paged(s["cache"], s["parents"], s["table"], s["start"], s["end"])
    else:
        m.beam_reorder(s["cache"], c["t_max"], s["parents"], c["start"], c["end"])
    return s["cache"]


def _plan(s):
    """Pages go back in the order of requests and blocks onto the stack, and are taken from its top in that order."""
    c = s["case"]
    page, table, free, n_pages = c["page"], s["table"], s["free"], s["free"].numel()
    rel = s["release"] != 0
    cached = torch.where(rel, 0, s["cached"]).long()
    new = s["new"].long()
    total = cached + new
    cu = torch.cat([new.new_zeros(1), torch.cumsum(new, 0)])
    held = (table >= 0) & (table < n_pages)
    back = held & rel[:, None]
    back_rank = torch.cumsum(back.reshape(-1).long(), 0).view_as(table) - 1
    count = s["free_count"].long()
    grown = count + back.sum()
    pool = torch.cat([free, free.new_zeros(1)])
    pool.scatter_(0, torch.where(back, count + back_rank, n_pages).reshape(-1), table.reshape(-1))
    j = torch.arange(table.shape[1], device=table.device)
    need = (j[None, :] >= (cached // page)[:, None]) & (j[None, :] < ((total + page - 1) // page)[:, None]) & ~(held & ~rel[:, None])
    rank = torch.cumsum(need.reshape(-1).long(), 0).view_as(table) - 1
    taken = pool[(grown - 1 - rank).clamp(0, n_pages)]
    after = torch.where(need, taken, torch.where(back, -1, table))
    ok = (need.sum() <= grown) & (cu[-1] <= s["slots"].numel()) & (total <= table.shape[1] * page).all() & (new >= 0).all() & (s["cached"] >= 0).all()
    table.copy_(torch.where(ok, after, table))
    free.copy_(torch.where(ok, pool[:n_pages], free))
    s["free_count"].copy_(torch.where(ok, grown - need.sum(), count))
    s["cu"].copy_(torch.where(ok, cu, 0))
    s["kv_len"].copy_(torch.where(ok, total, s["cached"]))
    i = torch.arange(s["slots"].numel(), device=table.device)
    live = ok & (i < cu[-1])
    r = torch.searchsorted(cu[1:], i, right=True).clamp(max=new.numel() - 1)
    pos = torch.where(live, cached[r] + i - cu[r], 0)
    s["positions"].copy_(pos)
    s["slots"].copy_(torch.where(live, table[r, (pos // page).clamp(max=table.shape[1] - 1)].long() * page + pos % page, -1))
    return [s[k] for k in ("table", "free", "free_count", "cu", "kv_len", "positions", "slots")]


def _attention(s):
    c = s["case"]
    h, nkv, hd, total, n = c["heads"], c["kv_heads"], c["head_dim"], s["total"], s["max_new"]
    rows = s["qkv"].view(-1, h + 2 * nkv, hd)[:total]
    at = s["slots"][:total].long()
    s["k"].view(-1, nkv, hd)[at] = rows[:, h:h + nkv]
    s["v"].view(-1, nkv, hd)[at] = rows[:, h + nkv:]
    cu, kv_len = s["cu"].long(), s["kv_len"].long()
    pages = s["table"].long().clamp(min=0)
    size = pages.shape[0], -1, nkv, hd
    k = s["k"][pages].view(size).permute(0, 2, 3, 1).float()  # [request, kv head, hd, key]
    v = s["v"][pages].view(size).permute(0, 2, 1, 3).float()
    i = torch.arange(n, device=DEV)
    q = rows[:, :h][(cu[:-1, None] + i).clamp(max=total - 1)].float()  # [request, new, head, hd]
    q = q.view(-1, n, nkv, h // nkv, hd).permute(0, 2, 3, 1, 4).reshape(q.shape[0], nkv, -1, hd)
    score = torch.matmul(q, k).view(q.shape[0], nkv, h // nkv, n, -1) / math.sqrt(hd)
    first = kv_len - (cu[1:] - cu[:-1])  # the position of a request's first new token
    key = torch.arange(score.shape[-1], device=DEV)
    hidden = key[None, None, :] > (first[:, None] + i)[:, :, None]
    score.masked_fill_(hidden[:, None, None], -math.inf)
    p = torch.exp(score - score.amax(-1, keepdim=True))
    p /= p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(p.shape[0], nkv, -1, p.shape[-1]), v).view(-1, h, n, hd).transpose(1, 2)
    row = torch.arange(total, device=DEV)
    r = torch.searchsorted(cu[1:], row, right=True)
    out = s["o"].clone()
    out[:total] = o[r, row - cu[r]].reshape(total, h * hd).to(out.dtype)
    return [out, s["k"], s["v"]]


def _select(s):
    """Each beam's candidates by logit, then id; over the beams by score, then beam.  A finished beam has one: its
    end again at the same score.  In 64 bits: candidates of two beams may be as near as 32 bits tell."""
    b, k, v = s["logits"].shape
    z = s["logits"].double()
    top, ids = torch.sort(z, dim=2, descending=True, stable=True)
    n = min(k, v)
    top, ids = top[..., :n], ids[..., :n]
    most = top[..., :1]
    lse = most + torch.log(torch.exp(z - most).sum(-1, keepdim=True))
    score = s["scores"].double()[..., None] + (top - lse)
    fin = (s["finished"] != 0)[..., None]
    first = torch.arange(n, device=DEV) == 0
    score = torch.where(fin, torch.where(first, s["scores"].double()[..., None], -math.inf), score)
    ids = torch.where(fin, s["eos"], ids)
    score, at = torch.sort(score.reshape(b, k * n), dim=1, descending=True, stable=True)
    at = at[:, :k]
    tokens = ids.reshape(b, k * n).gather(1, at)
    parents = at // n
    done = (s["finished"].gather(1, parents) != 0) | (tokens == s["eos"])
    return [score[:, :k].float(), tokens.to(torch.int32), parents.to(torch.int32), done.to(torch.int32)]


def _reorder(s):
    c, cache = s["case"], s["cache"]
    b, k = s["parents"].shape
    source = (torch.arange(b, device=DEV)[:, None] * k + s["parents"].long()).reshape(-1)
    if not c["page"]:
        cache[:, :, :, c["start"]:c["end"]] = cache[:, :, source, c["start"]:c["end"]]
        return cache
    flat = cache.view(c["layers"], 2, -1, c["kv_heads"], c["head_dim"])
    pos = torch.arange(s["table"].shape[1] * c["page"], device=DEV)
    slot = s["table"].long()[:, pos // c["page"]] * c["page"] + pos % c["page"]
    moved = (pos >= s["start"][:, None]) & (pos < s["end"][:, None])
    to = slot[moved]
    flat[:, :, to] = flat[:, :, slot[source][moved]]
    return cache


# ---------------------------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attention":
        return _exact_attention(s)
    if case["op"] == "select":
        return _exact_select(s)
    if case["op"] == "reorder":
        return _exact_reorder(s)
    return None  # a plan is whole numbers


def _exact_attention(s):
    """Request by request, head by head, from the definition."""
    c = s["case"]
    h, nkv, hd, page = c["heads"], c["kv_heads"], c["head_dim"], c["page"]
    x = s["qkv"].view(-1, h + 2 * nkv, hd)
    out, k_pages, v_pages = s["o"].double(), s["k"], s["v"]
    cu, lens, table = s["cu"].tolist(), s["kv_len"].tolist(), s["table"].tolist()
    for r, length in enumerate(lens):
        lo, hi = cu[r], cu[r + 1]
        if lo == hi:
            continue
        pages = torch.tensor(table[r][:_blocks(length, page)], device=DEV)
        first = length - (hi - lo)
        k = k_pages[pages].reshape(-1, nkv, hd)[:length]
        v = v_pages[pages].reshape(-1, nkv, hd)[:length]
        k[first:], v[first:] = x[lo:hi, h:h + nkv], x[lo:hi, h + nkv:]
        late = torch.arange(length, device=DEV)[None, :] > torch.arange(first, length, device=DEV)[:, None]
        for head in range(h):
            g = head // (h // nkv)
            w = (x[lo:hi, head].double() @ k[:, g].double().T) * hd ** -0.5
            w = torch.softmax(w.masked_fill(late, -math.inf), dim=1)
            out[lo:hi, head * hd:(head + 1) * hd] = w @ v[:, g].double()
    return [out, None, None]


def _exact_select(s):
    scores = []
    for z, before, fin in zip(s["logits"], s["scores"].tolist(), s["finished"].tolist()):
        every = []
        for beam in range(len(before)):
            if fin[beam]:
                every.append(torch.tensor([before[beam]], dtype=torch.float64, device=DEV))
            else:
                every.append(before[beam] + torch.log_softmax(z[beam].double(), 0))
        scores.append(torch.topk(torch.cat(every), len(before)).values)
    return [torch.stack(scores), None, None, None]


def _exact_reorder(s):
    c, cache = s["case"], s["cache"]
    before, k = cache.clone(), c["beams"]
    parents, spans = s["parents"].tolist(), _spans(c)
    for b in range(c["batch"]):
        a, e = spans[b]
        for i in range(k):
            to, source = b * k + i, b * k + parents[b][i]
            if not c["page"]:
                cache[:, :, to, a:e] = before[:, :, source, a:e]
                continue
            for p in range(a, e):
                at = [s["table"][row, p // c["page"]] for row in (to, source)]
                cache[:, :, at[0], p % c["page"]] = before[:, :, at[1], p % c["page"]]
    return cache.double()


# ---------------------------------------------------------------------------------------------- what a pass needs

def work(case):
    c = case
    if c["op"] == "plan":
        cached, new = _lengths(c)
        rel = _released(c)
        back = sum(_blocks(n, c["page"]) for n, x in zip(cached, rel) if x)
        taken = sum(_blocks((0 if x else k) + n, c["page"]) - (0 if x else _blocks(k, c["page"])) for k, n, x in zip(cached, new, rel))
        rows = sum(new) + c["pad_rows"]
        # lengths read and written, pages moved between table and stack, a position and a slot for every row
        return {"bytes": 4 * (6 * c["requests"] + 2 * (back + taken) + 2 * rows + 4), "flops": 0}
    es = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "attention":
        cached, new = _lengths(c)
        h, nkv, hd = c["heads"], c["kv_heads"], c["head_dim"]
        rows = sum(new)
        keys = sum(k for k, n in zip(cached, new) if n)
        seen = sum(n * k + n * (n + 1) // 2 for k, n in zip(cached, new))
        # the cached keys and values once, the new rows' q, k, v in, their k, v to the pages, o out
        return {"bytes": es * hd * (2 * nkv * keys + rows * (h + 2 * nkv) + 2 * nkv * rows + rows * h), "flops": 4 * h * hd * seen}
    if c["op"] == "select":
        n = c["batch"] * c["beams"]
        return {"bytes": es * (n - c["finished"]) * c["vocab"] + 24 * n, "flops": 0}
    moved = 0
    for (a, e), p in zip(_spans(c), _parents(c)):
        changed = [i for i, x in enumerate(p) if x != i]
        moved += (e - a) * (len(changed) + len({p[i] for i in changed}))
    return {"bytes": es * c["layers"] * 2 * c["kv_heads"] * c["head_dim"] * moved, "flops": 0}
