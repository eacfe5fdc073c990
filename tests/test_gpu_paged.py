"""The paged KV cache through the public calls: planning against a plain
allocator, attention against 64 bits, the beams' reordering against copies."""
import math
import random
import threading
import time

import numpy as np
import pytest

import synth

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from bwd_step_b200 import Model, NcError, _lib  # noqa: E402

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _model(h=10, nkv=1, hd=128, dtype="bf16", layers=1, vocab=512):
    d = synth.WORKLOADS["tiny"].model.as_dict()
    d.update(n_head=h, n_kv_head=nkv, head_dim=hd, n_layer=layers, vocab=vocab)
    return Model(d, dtype)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- plan

def _plain_plan(page, cached, new, release, table, free, count, rows):
    """The step in plain Python: (table, free, count, cu, kv_len, positions, slots) or None when refused."""
    table, free = [list(t) for t in table], list(free)
    n_pages = len(free)
    held = lambda e: 0 <= e < n_pages  # noqa: E731
    kept = [0 if x else k for k, x in zip(cached, release)]
    total = [k + n for k, n in zip(kept, new)]
    if min(cached) < 0 or min(new) < 0 or max(total) > len(table[0]) * page or sum(new) > rows:
        return None
    for r, row in enumerate(table):
        if release[r]:
            for j, e in enumerate(row):
                if held(e):
                    free[count] = e
                    count += 1
                    row[j] = -1
    for r, row in enumerate(table):
        for j in range(kept[r] // page, -(-total[r] // page)):
            if not held(row[j]):
                if count == 0:
                    return None
                count -= 1
                row[j] = free[count]
    cu, pos, slots = [0], [], []
    for r, n in enumerate(new):
        cu.append(cu[-1] + n)
        for p in range(kept[r], total[r]):
            pos.append(p)
            slots.append(table[r][p // page] * page + p % page)
    pad = rows - len(pos)
    return table, free, count, cu, total, pos + [0] * pad, slots + [-1] * pad


def _plan_case(rng, n_req, page, max_blocks, spare, rows_pad, chunk, rel_share, prefilled=False):
    cached = [rng.randint(0, (max_blocks - 1) * page - chunk) for _ in range(n_req)]
    new = [rng.choice([0, 1, 1, rng.randint(min(1, chunk), chunk)]) for _ in range(n_req)]
    release = [int(rng.random() < rel_share) for _ in range(n_req)]
    used = sum(-(-c // page) for c in cached)
    n_pages = used + sum(-(-n // page) + 1 for n in new) + spare + n_req
    perm = list(range(n_pages))
    rng.shuffle(perm)
    table = []
    for r, c in enumerate(cached):
        row = [perm.pop() for _ in range(-(-c // page))]
        if prefilled and len(row) < max_blocks:
            row.append(perm.pop())  # a block that has its page before it is needed
        table.append(row + [rng.choice([-1, -1, n_pages, -7])] * (max_blocks - len(row)))
    free = perm + [-1] * (n_pages - len(perm))
    return cached, new, release, table, free, len(perm), sum(new) + rows_pad


def _run_plan(m, page, cached, new, release, table, free, count, rows, kv_alias=False):
    t = dict(cached=_ints(cached), new=_ints(new), table=_ints(table), free=_ints(free), count=_ints([count]))
    e = lambda n: torch.full((n,), -99, dtype=torch.int32, device="cuda")  # noqa: E731
    cu, pos, slots = e(len(new) + 1), e(rows), e(rows)
    kv = t["cached"] if kv_alias else e(len(new))
    m.page_plan(page, t["cached"], t["new"], t["table"], t["free"], t["count"], cu, kv, pos, slots,
                release=None if release is None else _ints(release))
    return t, [t["table"].tolist(), t["free"].tolist(), t["count"].item(), cu.tolist(), kv.tolist(), pos.tolist(),
               slots.tolist()]


@pytest.mark.parametrize("n_req,page,max_blocks,chunk,pad", [
    (1, 16, 1, 1, 0), (1, 256, 3, 300, 1), (3, 16, 9, 40, 5), (31, 32, 40, 200, 0), (33, 64, 12, 65, 7),
    (200, 16, 70, 1, 0), (300, 16, 33, 100, 11), (1500, 128, 5, 30, 3), (4096, 16, 4, 2, 0),
    (5, 16, 700, 6000, 3), (150, 16, 530, 5000, 0), (128, 32, 9, 3, 1)])
@pytest.mark.parametrize("rel_share", [0.0, 0.3, 1.0])
def test_plan_matches_a_plain_allocator(n_req, page, max_blocks, chunk, pad, rel_share):
    rng = random.Random(n_req * 7 + page)
    m = _model()
    c = _plan_case(rng, n_req, page, max_blocks, 3, pad, min(chunk, (max_blocks - 1) * page) or 0, rel_share, n_req % 2 == 1)
    cached, new, release, table, free, count, rows = c
    rows = max(rows, 1)
    want = _plain_plan(page, cached, new, release, table, free, count, rows)
    _, got = _run_plan(m, page, cached, new, release, table, free, count, rows, kv_alias=n_req % 3 == 0)
    assert m.check() == 0
    for name, g, w in zip(("table", "free", "count", "cu", "kv_len", "positions", "slots"), got, want):
        assert g == list(w) if isinstance(w, list) else g == w, name


def test_planning_a_step_again_changes_nothing():
    m = _model()
    cached, new, _, table, free, count, rows = _plan_case(random.Random(5), 40, 16, 20, 2, 3, 60, 0.0)
    t, got = _run_plan(m, 16, cached, new, None, table, free, count, rows)
    _, again = _run_plan(m, 16, cached, new, None, got[0], got[1], got[2], rows)
    assert again == got and m.check() == 0


@pytest.mark.parametrize("what", ["pages", "rows", "long", "negative", "new"])
def test_a_refused_step_changes_nothing(what):
    m = _model()
    cached, new, release, table, free, count, rows = _plan_case(random.Random(9), 20, 16, 20, 2, 0, 60, 0.2)
    if what == "pages":
        count = 1
        release = [0] * 20
    elif what == "rows":
        rows = sum(new) - 1
    elif what == "long":
        cached[3] = 20 * 16
        new[3] = 1
        release[3] = 0
    elif what == "negative":
        cached[4] = -1
    else:
        new[5] = -2
    before = [list(t) for t in table]
    _, got = _run_plan(m, 16, cached, new, release, table, free, count, rows)
    assert got == [before, free, count, [0] * 21, cached, [0] * rows, [-1] * rows]
    assert m.check() == (_lib.NC_ERR_OUT_OF_PAGES if what == "pages" else _lib.NC_ERR_BAD_LENGTH)
    assert m.check() == 0


def test_a_free_page_outside_the_cache_is_reported():
    """What the stack holds goes to the table, but to no slot."""
    m = _model()
    _, got = _run_plan(m, 16, [0, 0], [3, 20], None, [[-1, -1], [-1, -1]], [1 << 28, 2, -5, 1], 4, 23)
    assert m.check() == _lib.NC_ERR_BAD_PAGE
    assert got[0][0][0] == 1 and got[6][:3] == [16, 17, 18]
    assert got[6][3:] == [-1] * 16 + [32, 33, 34, 35]


def test_a_full_launch_queue_leaves_other_threads_running():
    """Launches wait for room in the stream's queue; the program's other threads go on meanwhile."""
    m, stream = _model(), torch.cuda.Stream()
    i = lambda *n: torch.zeros(*n, dtype=torch.int32, device="cuda")  # noqa: E731
    args = (16, i(2), _ints([1, 1]), _ints([[0], [1]]), i(4), i(1), i(3), i(2), i(4), i(4))
    m.page_plan(*args)
    torch.cuda.synchronize()
    gaps, stop = [], threading.Event()

    def beat():
        last = time.monotonic()
        while not stop.is_set():
            time.sleep(0.002)
            now = time.monotonic()
            gaps.append(now - last)
            last = now
    other = threading.Thread(target=beat)
    other.start()
    with torch.cuda.stream(stream):
        torch.cuda._sleep(2_000_000_000)  # about a second of the GPU's clock
    began = time.monotonic()
    for _ in range(6000):
        m.page_plan(*args, stream=stream)
    took = time.monotonic() - began
    stop.set()
    other.join()
    torch.cuda.synchronize()
    assert m.check() == 0
    assert took > 0.5, "the queue was not full"
    assert max(gaps) < 0.25 * took


# ---------------------------------------------------------------- attention

class Step:
    """A planned step with NaN wherever the cache holds no position of a request."""

    def __init__(self, h, nkv, hd, page, lens, dtype="bf16", pad=0, seed=0, extra_blocks=1, hot=0.0):
        t = TYPES[dtype]
        g = torch.Generator(device="cuda").manual_seed(seed)
        rng = random.Random(seed)
        self.h, self.nkv, self.hd, self.page, self.lens = h, nkv, hd, page, lens
        self.total = [c + n for c, n in lens]
        self.rows = max(sum(n for _, n in lens) + pad, 1)
        blocks = [-(-x // page) for x in self.total]
        n_pages = sum(blocks) + 2
        perm = list(range(n_pages))
        rng.shuffle(perm)
        width = max(max(blocks), 1) + extra_blocks
        self.tables = [[perm.pop() for _ in range(b)] for b in blocks]
        self.table = _ints([row + [-1] * (width - len(row)) for row in self.tables])
        self.k = torch.full((n_pages, page, nkv, hd), float("nan"), dtype=t, device="cuda")
        self.v = torch.full_like(self.k, float("nan"))

        def unit(*shape):  # rows of unit mean square, as QK-norm leaves them
            x = torch.randn(*shape, generator=g, device="cuda") + hot
            return x / x.square().mean(-1, keepdim=True).sqrt()
        qkv = torch.randn(self.rows, h + 2 * nkv, hd, generator=g, device="cuda")
        qkv[:, :h + nkv] = unit(self.rows, h + nkv, hd)
        self.qkv = qkv.view(self.rows, -1).to(t)
        cu, slots = [0], []
        for (c, n), row in zip(lens, self.tables):
            cu.append(cu[-1] + n)
            slot = [row[p // page] * page + p % page for p in range(c + n)]
            if c:
                at = torch.tensor(slot[:c], device="cuda")
                self.k.view(-1, nkv, hd)[at] = unit(c, nkv, hd).to(t)
                self.v.view(-1, nkv, hd)[at] = torch.randn(c, nkv, hd, generator=g, device="cuda").to(t)
            slots += slot[c:]
        self.cu, self.kv_len = _ints(cu), _ints(self.total)
        self.slots = _ints(slots + [-1] * (self.rows - len(slots)))
        self.o = torch.full((self.rows, h * hd), 7.0, dtype=t, device="cuda")

    def run(self, m, max_new=None, stream=None):
        ws = torch.full((m.paged_attention_workspace_bytes(len(self.lens), self.rows),), 0xFF, dtype=torch.uint8, device="cuda")
        top = max(n for _, n in self.lens) if max_new is None else max_new
        m.paged_attention(self.qkv, self.cu, self.kv_len, self.slots, self.table, self.k, self.v, self.o, ws, max_new=top,
                          stream=stream)
        return self.o

    def want(self):
        """o in 64 bits and, beside it, sum p |v|, which the error bounds scale with."""
        h, nkv, hd, g = self.h, self.nkv, self.hd, self.h // self.nkv
        o, mass = self.o.double().clone(), torch.zeros(self.rows, h * hd, dtype=torch.float64, device="cuda")
        x = self.qkv.double().view(self.rows, h + 2 * nkv, hd)
        lo = 0
        for (c, n), row in zip(self.lens, self.tables):
            if n:
                pages = torch.tensor(row, device="cuda")
                k = self.k[pages].reshape(-1, nkv, hd)[:c].double()
                v = self.v[pages].reshape(-1, nkv, hd)[:c].double()
                new = x[lo:lo + n]
                k, v = torch.cat([k, new[:, h:h + nkv]]), torch.cat([v, new[:, h + nkv:]])
                late = torch.arange(c + n, device="cuda")[None, :] > torch.arange(c, c + n, device="cuda")[:, None]
                for i in range(h):
                    s = (new[:, i] @ k[:, i // g].T / math.sqrt(hd)).masked_fill(late, -math.inf)
                    p = torch.softmax(s, 1)
                    o[lo:lo + n, i * hd:(i + 1) * hd] = p @ v[:, i // g]
                    mass[lo:lo + n, i * hd:(i + 1) * hd] = p @ v[:, i // g].abs()
            lo += n
        return o, mass


def _bound(dtype, hd, o, mass):
    """How far an output may be.  Scores: products of |q||k| <= hd in all, summed in fp32 in hd steps, give a relative
    error of P of at most 2 hd sqrt(hd) 2^-24 (a score's, and through the sum the normaliser's), and the scaled
    exponentials 2^-20.  bf16 besides: P rounded (half a step, 2^-8), the fitted exponential (7.5e-5 < 2^-13), the
    normaliser summed before that rounding, and the output rounded once (2^-8 of its size)."""
    rel = 2 * hd * math.sqrt(hd) * 2.0 ** -24 + 2.0 ** -20
    if dtype == "bf16":
        return (rel + 2.0 ** -8 + 2.0 ** -12) * mass + 2.0 ** -8 * o.abs() * 1.01 + 1e-30
    return (rel + 2.0 ** -22) * mass


def _check(s, m, dtype, **kw):
    want, mass = s.want()
    live = sum(n for _, n in s.lens)
    k0, v0 = s.k.clone(), s.v.clone()
    s.run(m, **kw)
    assert m.check() == 0
    got = s.o.double()
    err = (got - want).abs()
    assert torch.isfinite(got[:live]).all()
    over = err[:live] > _bound(dtype, s.hd, want[:live], mass[:live])
    assert not over.any(), (int(over.sum()), over.nonzero()[:4].tolist(), float(err[:live].max()))
    assert torch.equal(s.o[live:], torch.full_like(s.o[live:], 7.0))  # rows behind the last request
    # the rows' k, v in their slots, every other slot as it was
    at = s.slots[:live].long()
    x = s.qkv.view(s.rows, -1, s.hd)
    k0.view(-1, s.nkv, s.hd)[at] = x[:live, s.h:s.h + s.nkv]
    v0.view(-1, s.nkv, s.hd)[at] = x[:live, s.h + s.nkv:]
    for a, b in ((s.k, k0), (s.v, v0)):
        assert torch.equal(torch.nan_to_num(a, nan=123.0), torch.nan_to_num(b, nan=123.0))


DECODE = [(0, 1), (1, 1), (15, 1), (16, 1), (63, 1), (64, 1), (127, 1), (128, 1), (129, 1), (300, 1), (40, 0), (1023, 1)]
CHUNKS = [(0, 1), (0, 130), (5, 12), (127, 1), (128, 25), (250, 6), (33, 0), (100, 257), (0, 24), (511, 2)]
HEADS = [(10, 1, 128), (12, 1, 64), (15, 1, 128), (4, 1, 16), (4, 2, 32), (8, 2, 64), (6, 3, 128), (5, 5, 64), (1, 1, 128),
         (16, 1, 64), (17, 1, 128), (33, 1, 64), (130, 1, 64)]


@pytest.mark.parametrize("h,nkv,hd", HEADS)
@pytest.mark.parametrize("lens,page", [(DECODE, 16), (DECODE, 128), (CHUNKS, 32), (CHUNKS, 64), (CHUNKS, 256)])
def test_attention_bf16(h, nkv, hd, lens, page):
    _check(Step(h, nkv, hd, page, lens, pad=3, seed=h + hd), _model(h, nkv, hd), "bf16")


@pytest.mark.parametrize("h,nkv,hd", [(10, 1, 128), (12, 1, 64), (4, 1, 16), (4, 2, 32)])
@pytest.mark.parametrize("lens,page", [(DECODE[:10], 16), (CHUNKS, 64)])
def test_attention_fp32(h, nkv, hd, lens, page):
    _check(Step(h, nkv, hd, page, lens, "fp32", pad=2, seed=h + hd), _model(h, nkv, hd, "fp32"), "fp32")


@pytest.mark.parametrize("lens", [[(0, 1)], [(4000, 1)], [(9000, 3)], [(2000, 40)], [(0, 700)], [(5000, 300), (10, 1)],
                                  [(0, 0), (0, 1)], [(700, 1)] * 150, [(60, 2)] * 97, [(260, 30)] * 40,
                                  [(30, 1), (200, 1), (64, 1), (1, 1)] * 60, [(3000, 9)] * 20 + [(1, 1)] * 3, [(0, 0)] * 5 + [(77, 5)] + [(0, 0)] * 4])
@pytest.mark.parametrize("h,hd", [(10, 128), (12, 64)])
def test_attention_batches(lens, h, hd):
    """Few long requests, many short ones, and both kinds of step at once."""
    _check(Step(h, 1, hd, 16, lens, pad=1, seed=len(lens)), _model(h, 1, hd), "bf16")


@pytest.mark.parametrize("max_new", [0, 1000])
def test_attention_without_a_tight_bound(max_new):
    _check(Step(10, 1, 128, 32, DECODE, seed=4), _model(), "bf16", max_new=max_new)


def test_attention_sharp_scores():
    """Shared directions in q and k: scores up to sqrt(hd), nearly one-hot rows."""
    _check(Step(10, 1, 128, 32, CHUNKS, seed=8, hot=3.0), _model(), "bf16")
    _check(Step(10, 1, 128, 32, DECODE, seed=9, hot=3.0), _model(), "bf16")


def test_attention_is_reproducible():
    m = _model()
    for lens in (DECODE, CHUNKS):
        a = Step(10, 1, 128, 16, lens, seed=3).run(m).clone()
        b = Step(10, 1, 128, 16, lens, seed=3).run(m)
        assert torch.equal(a, b)


def test_attention_on_another_stream():
    m = _model()
    s, t = Step(10, 1, 128, 16, CHUNKS, seed=6), Step(10, 1, 128, 16, CHUNKS, seed=6)
    want = s.run(m).clone()
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    t.run(m, stream=other)
    other.synchronize()
    assert torch.equal(t.o, want)


@pytest.mark.parametrize("lens,longer", [(DECODE, [(c + 37 if n else c, n) for c, n in DECODE]),
                                         (CHUNKS, [(c, max(n - 1, 0)) for c, n in CHUNKS])])
def test_a_captured_step_follows_new_lengths(lens, longer):
    """A graph of the call, replayed after the lengths, tables and rows changed in place."""
    m = _model()
    a, b = Step(10, 1, 128, 16, lens, pad=40, seed=1, extra_blocks=8), Step(10, 1, 128, 16, longer, seed=2, extra_blocks=0)
    ws = torch.empty(m.paged_attention_workspace_bytes(len(lens), a.rows), dtype=torch.uint8, device="cuda")
    n_pages = max(a.k.shape[0], b.k.shape[0])
    width = max(a.table.shape[1], b.table.shape[1])
    k, v = (torch.zeros(n_pages, 16, 1, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")

    def load(s):
        k[:s.k.shape[0]], v[:s.v.shape[0]] = s.k, s.v
        table.fill_(-1)
        table[:, :s.table.shape[1]] = s.table
        n = min(s.rows, a.rows)
        a.qkv[:n] = s.qkv[:n]
        a.slots.fill_(-1)
        a.slots[:n] = s.slots[:n]
        a.cu.copy_(s.cu)
        a.kv_len.copy_(s.kv_len)

    def call():
        m.paged_attention(a.qkv, a.cu, a.kv_len, a.slots, table, k, v, a.o, ws, max_new=max(n for _, n in lens))
    first = a.run(m).clone()
    load(a)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for s, want in ((a, first), (b, b.run(m).clone()), (a, first)):
        load(Step(10, 1, 128, 16, lens, pad=40, seed=1, extra_blocks=8) if s is a else s)
        g.replay()
        live = sum(n for _, n in s.lens)
        assert torch.equal(a.o[:live], want[:live])
    assert m.check() == 0


def test_attention_over_many_requests():
    """As many requests as one call takes, one new token or a few, short and empty ones among them."""
    rng = random.Random(3)
    lens = [(rng.choice([0, 1, 15, 40]), rng.choice([0, 1, 1, 1, 3])) for _ in range(4095)] + [(300, 9)]
    _check(Step(1, 1, 64, 16, lens, seed=5), _model(1, 1, 64), "bf16")


@pytest.mark.parametrize("lens", [[(500, 1), (70, 1)], [(500, 30), (70, 2)]])
def test_attention_at_slots_far_into_a_large_cache(lens):
    """Pages behind the 4 GiB that 32-bit byte offsets reach."""
    m, s = _model(), Step(10, 1, 128, 256, lens, seed=12)
    want = s.run(m).clone()
    t = Step(10, 1, 128, 256, lens, seed=12)
    far = 70000
    k, v = (torch.empty(far + x.shape[0], 256, 1, 128, dtype=torch.bfloat16, device="cuda") for x in (t.k, t.v))
    k[far:], v[far:] = t.k, t.v
    t.k, t.v = k, v
    t.table[t.table >= 0] += far
    t.slots[t.slots >= 0] += far * 256
    assert torch.equal(t.run(m), want) and m.check() == 0
    at = s.slots.long()
    assert torch.equal(k.view(-1, 128)[at + far * 256], s.k.view(-1, 128)[at])


def test_requests_may_share_the_pages_of_a_common_prefix():
    m = _model()
    s = Step(10, 1, 128, 16, [(64, 1), (64, 20), (80, 1)], seed=15)
    for r in (1, 2):  # the first four pages are the first request's
        s.tables[r][:4] = s.tables[0][:4]
    s.table[:, :4] = s.table[0, :4]
    _check(s, m, "bf16")


def test_calls_at_once_on_two_streams():
    """Two steps of one model on two streams, each with its own arrays and workspace."""
    m = _model()
    steps = [Step(10, 1, 128, 16, lens, seed=7) for lens in (CHUNKS, DECODE) for _ in range(4)]
    want = [Step(10, 1, 128, 16, s.lens, seed=7).run(m).clone() for s in steps]
    ws = [torch.empty(m.paged_attention_workspace_bytes(len(s.lens), s.rows), dtype=torch.uint8, device="cuda") for s in steps]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for i, s in enumerate(steps):
        m.paged_attention(s.qkv, s.cu, s.kv_len, s.slots, s.table, s.k, s.v, s.o, ws[i], max_new=max(n for _, n in s.lens),
                          stream=streams[i % 2])
    torch.cuda.synchronize()
    assert m.check() == 0
    for s, w in zip(steps, want):
        assert torch.equal(s.o, w)


@pytest.mark.parametrize("h,hd", [(10, 128), (12, 64), (4, 16)])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_row_that_is_not_finite_stays_in_its_request(h, hd, value):
    """A new v that is not finite: every later row of its request sees it; no other request's row, no decoding
    request's, and no row 256 or more before it changes by a bit."""
    lens = [(20, 300), (33, 50), (70, 1), (5, 1)]
    m = _model(h, 1, hd)
    s, t = (Step(h, 1, hd, 16, lens, seed=11) for _ in range(2))
    want = t.run(m).clone()
    bad = 290
    s.qkv.view(s.rows, h + 2, hd)[bad, h + 1] = value
    s.run(m)
    assert m.check() == 0
    assert not torch.isfinite(s.o[bad:300]).any()
    assert torch.equal(s.o[300:], want[300:])
    assert torch.equal(s.o[:bad - 255], want[:bad - 255])


@pytest.mark.parametrize("h,hd", [(10, 128), (4, 16)])
def test_a_request_with_more_rows_than_max_new_is_reported(h, hd):
    m = _model(h, 1, hd)
    s = Step(h, 1, hd, 16, [(100, 1), (50, 3)], seed=1)
    s.run(m, max_new=1)
    # the plain kernel computes it all the same
    assert m.check() == (_lib.NC_ERR_BAD_LENGTH if hd == 128 else 0)


def test_attention_reports_missing_pages_and_lengths():
    m = _model()
    s = Step(10, 1, 128, 16, [(100, 1), (50, 1)], seed=1)
    s.table[0, 2] = -1
    s.run(m)
    assert m.check() == _lib.NC_ERR_BAD_PAGE
    s = Step(10, 1, 128, 16, [(100, 1), (50, 1)], seed=1)
    s.kv_len[1] = 1 << 20  # longer than the table
    s.table[s.table < 0] = 0
    s.run(m)
    assert m.check() == _lib.NC_ERR_BAD_LENGTH
    s = Step(10, 1, 128, 16, [(100, 1), (50, 1)], seed=1)
    s.slots[0] = 1 << 20
    s.run(m)
    assert m.check() == _lib.NC_ERR_BAD_PAGE
    assert m.check() == 0


@pytest.mark.parametrize("h,hd,dtype", [(10, 128, "bf16"), (12, 64, "bf16"), (4, 16, "bf16"), (10, 128, "fp32")])
@pytest.mark.parametrize("length", [1 << 20, -1])
def test_requests_without_new_rows_have_their_lengths_checked(h, hd, dtype, length):
    """On every path, and the other requests' rows come out all the same."""
    m = _model(h, 1, hd, dtype)
    lens = [(100, 1), (50, 0), (20, 1), (0, 0)]
    s, t = (Step(h, 1, hd, 16, lens, dtype, seed=1) for _ in range(2))
    want = t.run(m).clone()
    assert m.check() == 0
    s.kv_len[1] = length
    s.run(m)
    assert m.check() == _lib.NC_ERR_BAD_LENGTH
    assert torch.equal(s.o, want)


def test_refusals():
    m = _model()
    s = Step(10, 1, 128, 16, [(100, 1), (50, 1)], seed=1)
    ws = torch.empty(m.paged_attention_workspace_bytes(2, s.rows), dtype=torch.uint8, device="cuda")

    def call(qkv=s.qkv, cu=s.cu, kv_len=s.kv_len, slots=s.slots, table=s.table, k=s.k, v=s.v, o=s.o, ws=ws, max_new=1):
        m.paged_attention(qkv, cu, kv_len, slots, table, k, v, o, ws, max_new=max_new)
    call()
    for bad, kind in ((dict(ws=ws[:-256]), NcError), (dict(ws=ws[1:]), NcError), (dict(max_new=-1), NcError),
                      (dict(k=s.k.view(-1, 8, 1, 128), v=s.v.view(-1, 8, 1, 128)), NcError),
                      (dict(k=s.k[:0], v=s.v[:0]), NcError),
                      (dict(qkv=s.qkv.float()), TypeError), (dict(cu=s.cu.long()), TypeError), (dict(cu=s.cu[1:]), ValueError),
                      (dict(slots=s.slots[1:]), ValueError), (dict(table=s.table[:1]), ValueError),
                      (dict(v=s.v[1:]), ValueError), (dict(o=s.o[:, :-1]), ValueError),
                      (dict(table=s.table.t().contiguous().t()), ValueError), (dict(qkv=s.qkv.cpu()), ValueError)):
        with pytest.raises(kind):
            call(**bad)
    i = lambda *n: torch.zeros(*n, dtype=torch.int32, device="cuda")  # noqa: E731
    with pytest.raises(NcError):  # more requests than one plan takes
        m.page_plan(16, i(4097), i(4097), i(4097, 1), i(8), i(1), i(4098), i(4097), i(4), i(4))
    with pytest.raises(NcError):  # not a power of two
        m.page_plan(24, i(2), i(2), i(2, 1), i(8), i(1), i(3), i(2), i(4), i(4))
    with pytest.raises(ValueError):
        m.page_plan(16, i(2), i(2), i(2, 1), i(8), i(1), i(2), i(2), i(4), i(4))
    assert m.check() == 0


# ---------------------------------------------------------------- reorder

@pytest.mark.parametrize("beams", [1, 2, 3, 4, 5, 8, 11, 16, 32])
@pytest.mark.parametrize("dtype,nkv,hd", [("bf16", 1, 128), ("bf16", 1, 16), ("fp32", 2, 32)])
def test_dense_reorder(beams, dtype, nkv, hd):
    m = _model(2 * nkv, nkv, hd, dtype, layers=3)
    batch, t_max = 3, 37
    g = torch.Generator(device="cuda").manual_seed(beams)
    cache = torch.randn(3, 2, batch * beams, t_max, nkv, hd, generator=g, device="cuda").to(TYPES[dtype])
    parents = torch.randint(0, beams, (batch, beams), generator=g, device="cuda").to(torch.int32)
    source = (torch.arange(batch, device="cuda")[:, None] * beams + parents).view(-1)
    for start, end in ((5, 31), (0, t_max), (7, 7), (36, 37)):
        want = cache.clone()
        want[:, :, :, start:end] = cache[:, :, source, start:end]
        m.beam_reorder(cache, t_max, parents, start, end)
        assert torch.equal(cache, want)
    assert m.check() == 0


@pytest.mark.parametrize("beams,page", [(1, 16), (2, 16), (4, 32), (7, 16), (12, 64), (32, 16)])
def test_paged_reorder(beams, page):
    m = _model(2, 1, 64, "bf16", layers=2)
    batch, rng = 4, random.Random(beams)
    g = torch.Generator(device="cuda").manual_seed(beams)
    starts = [rng.randint(0, 60) for _ in range(batch)]
    ends = [s + rng.choice([0, 1, rng.randint(0, 90)]) for s in starts]
    blocks = [-(-e // page) for e in ends]
    n_pages = sum(blocks) * beams + 1
    perm = list(range(n_pages))
    rng.shuffle(perm)
    table = []
    for b in range(batch):
        for i in range(beams):
            row = [perm.pop() for _ in range(blocks[b])]
            if i:  # full pages of the common part are shared
                row[:starts[b] // page] = table[b * beams][:starts[b] // page]
            table.append(row)
    width = max(blocks) + 1
    dev_table = _ints([r + [-1] * (width - len(r)) for r in table])
    kv = torch.randn(2, 2, n_pages, page, 1, 64, generator=g, device="cuda").to(torch.bfloat16)
    parents = [[rng.randrange(beams) for _ in range(beams)] for _ in range(batch)]
    want = kv.clone()
    for b in range(batch):
        for i, par in enumerate(parents[b]):
            for p in range(starts[b], ends[b]):
                to, at = table[b * beams + i][p // page], table[b * beams + par][p // page]
                want[:, :, to, p % page] = kv[:, :, at, p % page]
    m.beam_reorder_paged(kv, _ints(parents), dev_table, _ints([s for s in starts for _ in range(beams)]),
                         _ints([e for e in ends for _ in range(beams)]))
    assert torch.equal(kv, want) and m.check() == 0


@pytest.mark.parametrize("beams,page", [(2, 16), (3, 32), (5, 16), (8, 64), (9, 16), (20, 32), (32, 16)])
@pytest.mark.parametrize("dtype,nkv,hd", [("bf16", 1, 64), ("fp32", 2, 32), ("fp32", 1, 128)])
def test_paged_reorder_with_a_span_for_every_beam(beams, page, dtype, nkv, hd):
    """The spans of a row's beams differ, empty ones among them; a parent gives what it held before the call."""
    m = _model(2 * nkv, nkv, hd, dtype, layers=2)
    batch, rng = 3, random.Random(beams * 5 + page)
    g = torch.Generator(device="cuda").manual_seed(beams)
    starts = [rng.randint(0, 70) for _ in range(batch * beams)]
    ends = [max(0, a + rng.choice([0, -3, 1, rng.randint(0, 80), rng.randint(0, 80)])) for a in starts]
    width = -(-max(max(starts), max(ends)) // page) + 1
    n_pages = batch * beams * width + 1
    perm = list(range(n_pages))
    rng.shuffle(perm)
    table = [[perm.pop() for _ in range(width)] for _ in range(batch * beams)]
    kv = torch.randn(2, 2, n_pages, page, nkv, hd, generator=g, device="cuda").to(TYPES[dtype])
    parents = [[rng.randrange(beams) for _ in range(beams)] for _ in range(batch)]
    want = kv.clone()
    for b in range(batch):
        for i, par in enumerate(parents[b]):
            row, source = table[b * beams + i], table[b * beams + par]
            for p in range(starts[b * beams + i], ends[b * beams + i]):
                want[:, :, row[p // page], p % page] = kv[:, :, source[p // page], p % page]
    m.beam_reorder_paged(kv, _ints(parents), _ints(table), _ints(starts), _ints(ends))
    assert torch.equal(kv, want) and m.check() == 0


def test_reorder_refusals_and_reports():
    m = _model(2, 1, 64, "bf16", layers=2)
    cache = torch.zeros(2, 2, 4, 8, 1, 64, dtype=torch.bfloat16, device="cuda")
    par = _ints([[0, 1], [1, 0]])
    for args in ((cache, 8, par, -1, 4), (cache, 8, par, 5, 4), (cache, 8, par, 0, 9)):
        with pytest.raises(NcError):
            m.beam_reorder(*args)
    with pytest.raises(ValueError):
        m.beam_reorder(cache[:1], 8, par, 0, 4)
    with pytest.raises(TypeError):
        m.beam_reorder(cache, 8, par.long(), 0, 4)
    with pytest.raises(NcError):
        m.beam_reorder(torch.zeros(2, 2, 33, 8, 1, 64, dtype=torch.bfloat16, device="cuda"), 8, _ints([list(range(33))]), 0, 4)
    assert m.check() == 0
    cache.normal_()
    want = cache.clone()
    want[:, :, 3] = cache[:, :, 2]
    m.beam_reorder(cache, 8, _ints([[0, 2], [-1, 0]]), 0, 8)  # two back-pointers out of range
    assert torch.equal(cache, want) and m.check() == _lib.NC_ERR_BAD_LENGTH
