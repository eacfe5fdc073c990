"""Beam search: the selection against 64 bits, and whole searches over the dense
and the paged cache against one that runs the oracle's full forward."""
import numpy as np
import pytest

import oracle
import synth
from harness import to_device_weights

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from bwd_step_b200 import Model, NcError  # noqa: E402
from bwd_step_b200.generate import beam_search  # noqa: E402

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _model(vocab, dtype="bf16"):
    d = synth.WORKLOADS["tiny"].model.as_dict()
    d.update(vocab=vocab)
    return Model(d, dtype)


def _plain(logits, scores, finished, eos):
    """The best candidates of one batch row, from the definition: (scores, tokens, parents, finished)."""
    z = logits.astype(np.float64).copy()
    z[np.isnan(z)] = -np.inf
    every = []
    for k in range(z.shape[0]):
        s = -np.inf if np.isnan(scores[k]) else float(scores[k])
        if finished is not None and finished[k]:
            every.append([(s, 0, eos)])
            continue
        top = z[k].max()
        if not np.isfinite(top):
            lse = np.inf
        else:
            lse = top + np.log(np.exp(z[k] - top).sum())
        order = np.lexsort((np.arange(z.shape[1]), -z[k]))[:z.shape[0]]
        row = []
        for rank, v in enumerate(order):
            c = s + (z[k, v] - lse) if z[k, v] != np.inf else -np.inf
            row.append((-np.inf if np.isnan(c) else c, rank, int(v)))
        every.append(row)
    out = []
    at = [0] * len(every)
    for _ in range(len(every)):
        k = max((k for k in range(len(every)) if at[k] < len(every[k])), key=lambda k: (every[k][at[k]][0], -k))
        s, _, v = every[k][at[k]]
        at[k] += 1
        out.append((s, v, k, int((finished is not None and finished[k]) or v == eos)))
    return [list(x) for x in zip(*out)]


def _check(logits, scores, dtype, finished=None, eos=-1, alias=False):
    b, k, v = logits.shape
    m = _model(v, dtype)
    z = logits.to(TYPES[dtype]).cuda().contiguous()
    s = scores.cuda()
    e = lambda: torch.full((b, k), -77, dtype=torch.int32, device="cuda")  # noqa: E731
    fin = None if finished is None else finished.to(torch.int32).cuda()
    want = [_plain(z[i].float().cpu().numpy(), scores[i].numpy(), None if finished is None else finished[i].tolist(), eos)
            for i in range(b)]
    tok, par = e(), e()
    s_out, f_out = (s, fin) if alias else (torch.full_like(s, 9.0), None if fin is None else e())
    m.beam_select(z, s, s_out, tok, par, eos=eos, finished=fin, finished_out=f_out)
    assert m.check() == 0
    for i in range(b):
        ws, wt, wp, wf = want[i]
        assert tok[i].tolist() == wt and par[i].tolist() == wp, i
        if fin is not None:
            assert f_out[i].tolist() == wf
        got = s_out[i].double().cpu().numpy()
        ws = np.array(ws)
        same = np.isneginf(ws)
        assert np.array_equal(np.isneginf(got), same)
        # one rounding to fp32, and the log-sum-exp: exponentials of relative error 2^-20 at most, however many
        assert np.all(np.abs(got[~same] - ws[~same]) <= 2.0 ** -24 * np.abs(ws[~same]) + 2.0 ** -20)
    # what no beam search reads or writes
    return tok, par


def _random(b, k, v, seed, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(b, k, v, generator=g) * spread, -10.0 * torch.rand(b, k, generator=g)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("b,k,v", [(1, 1, 64), (1, 4, 65536), (3, 5, 512), (2, 32, 64), (2, 32, 8256), (5, 8, 50304), (7, 3, 1088),
                                   (1, 17, 16384), (40, 2, 8128), (2, 9, 9024)])
def test_select(b, k, v, dtype):
    z, s = _random(b, k, v, b * 31 + k)
    _check(z, s, dtype)


@pytest.mark.parametrize("alias", [False, True])
def test_select_with_ended_beams(alias):
    for share, seed in ((0.3, 1), (0.8, 2), (1.0, 3)):
        z, s = _random(6, 6, 1024, seed)
        g = torch.Generator().manual_seed(seed)
        fin = torch.rand(6, 6, generator=g) < share
        z[fin] = float("nan")  # not read
        _check(z, s, "bf16", finished=fin, eos=1023, alias=alias)
    z, s = _random(4, 3, 512, 4)
    z[:, :, 100] = 30.0  # every beam ends now
    _check(z, s, "bf16", finished=torch.zeros(4, 3, dtype=torch.bool), eos=100, alias=alias)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_select_ties_go_to_the_lower_beam_and_id(dtype):
    z = torch.zeros(3, 4, 8192)  # every candidate alike
    _check(z, torch.zeros(3, 4), dtype)
    z[1, 2, 7000] = 1.0
    z[1, 2, 100:8000:700] = 1.0
    z[2, :, 4095] = -0.0
    _check(z, torch.zeros(3, 4), dtype)
    z = torch.randint(-2, 3, (4, 8, 20480)).float()  # few values, many ties
    z[:, 4:] = z[:, :4]  # the same logits in two beams
    s = torch.tensor([[-1.0] * 4 + [-1.0] * 4] * 4)
    _check(z, s, dtype)


def test_select_orders_that_defeat_a_running_threshold():
    up = torch.linspace(-20, 20, 8192).repeat(2, 3, 1)  # every value better than all before it
    _check(up, torch.zeros(2, 3), "fp32")
    _check(up.flip(-1), torch.zeros(2, 3), "fp32")


def test_select_infinities_and_nan():
    inf = float("inf")
    z, s = _random(6, 4, 2048, 11)
    z[0, 1] = -inf  # a beam without a candidate of weight
    z[1, :, 5:] = -inf  # five ids left
    z[2] = -inf  # nothing at all
    z[3, 2, ::3] = float("nan")
    z[4, 0, 17] = inf
    s[5] = torch.tensor([0.0, -inf, -inf, -inf])  # the first step of a search
    s[3, 0] = float("nan")
    _check(z, s, "bf16")
    _check(z, s, "fp32")


@pytest.mark.parametrize("k,v", [(8, 65536), (32, 65536), (32, 512), (5, 2112)])
def test_select_with_few_ids_allowed(k, v):
    """All ids but a few masked: fewer candidates of finite score than lanes, than beams, one, none."""
    z, s = _random(4, k, v, k)
    for b, allowed in enumerate((40, 3, 1, 0)):
        mask = torch.ones(v, dtype=torch.bool)
        mask[torch.randperm(v, generator=torch.Generator().manual_seed(b))[:allowed]] = False
        z[b, :, mask] = -float("inf")
    _check(z, s, "bf16")
    s[:, 1:] = -float("inf")  # and a search's first step
    _check(z, s, "bf16")


@pytest.mark.parametrize("k,v", [(1, 65536), (32, 65536), (16, 320)])
def test_select_of_equal_logits(k, v):
    _check(torch.full((2, k, v), 1.5), torch.linspace(0, -2, 2 * k).view(2, k), "bf16")


def test_select_of_a_large_vocabulary():
    """Several chunks of logits in a block."""
    z, s = _random(2, 3, 64 * 4100, 17)
    _check(z, s, "bf16")
    _check(z, s, "fp32")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("size", [30.0, 1e3, 3e4, 1e10, 3e38])
def test_select_of_large_logits(size, dtype):
    """The log-sum-exp is exact to the same bound whatever the size of the logits: a shift that is rounded on the way does
    not show in it."""
    z, s = _random(3, 4, 4160, 21, spread=1.0)
    z *= size / z.abs().max()
    near = torch.linspace(0.0, -6.0, 64)  # candidates of weight beside the largest, where the type tells them apart
    z[1, :, 100:164] = size + near
    z[2] = -size + torch.randn(4, 4160, generator=torch.Generator().manual_seed(5))  # and far below zero
    _check(z, s, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("top", [15.0, 14.8125, 1003.0, 30000.0])
def test_select_of_beams_with_one_likely_token(top, dtype):
    """All weight on one id: its score is its beam's, and never above it."""
    z = torch.full((2, 3, 65536), -100.0)
    for k in range(3):
        z[:, k, 501 * k + 77] = top
    s = torch.tensor([[-1.25, -2.5, -0.75], [0.0, -3.0, -7.0]])
    _check(z, s, dtype)
    m = _model(65536, dtype)
    i = lambda: torch.empty(2, 3, dtype=torch.int32, device="cuda")  # noqa: E731
    out = torch.empty(2, 3, device="cuda")
    m.beam_select(z.to(TYPES[dtype]).cuda(), s.cuda(), out, i(), i())
    assert torch.equal(out.cpu(), s.sort(dim=1, descending=True).values)


@pytest.mark.parametrize("size", [1.0, 40.0, 5000.0])
def test_select_of_beams_with_the_same_logits_in_another_order(size):
    """Equal beams whose ids are permuted: their candidates tie, and which of them come first is open within the
    log-sum-exp's bound of 2^-18, but the scores are the K best ones."""
    g = torch.Generator().manual_seed(3)
    row = (torch.randn(65536, generator=g) * size).to(torch.bfloat16).float()
    z = torch.stack([row[torch.randperm(65536, generator=g)] for _ in range(6)])[None].contiguous()
    s = torch.full((1, 6), -2.0)
    m = _model(65536)
    i = lambda: torch.empty(1, 6, dtype=torch.int32, device="cuda")  # noqa: E731
    out, tok, par = torch.empty(1, 6, device="cuda"), i(), i()
    m.beam_select(z.bfloat16().cuda(), s.cuda(), out, tok, par)
    assert m.check() == 0
    want = _plain(z[0].numpy(), s[0].numpy(), None, -1)[0]
    assert np.all(np.abs(out[0].cpu().double().numpy() - want) <= 2.0 ** -24 * np.abs(want) + 2.0 ** -18)
    assert len(set(zip(par[0].tolist(), tok[0].tolist()))) == 6
    every = -2.0 + torch.log_softmax(z[0].double(), 1)
    picked = np.array([float(every[p, t]) for p, t in zip(par[0].tolist(), tok[0].tolist())])
    assert np.all(np.abs(picked - want) <= 2.0 ** -17)  # two beams' errors


def test_select_refusals():
    m = _model(512)
    z = torch.zeros(2, 3, 512, dtype=torch.bfloat16, device="cuda")
    s = torch.zeros(2, 3, device="cuda")
    i = lambda *n: torch.zeros(*n, dtype=torch.int32, device="cuda")  # noqa: E731

    def call(z=z, s=s, so=s, t=i(2, 3), p=i(2, 3), **kw):
        m.beam_select(z, s, so, t, p, **kw)
    call()
    f = i(2, 3)
    flat = torch.zeros(2 * 3 * 512 + 1, dtype=torch.bfloat16, device="cuda")
    for bad, kind in ((dict(eos=3), NcError), (dict(finished=f, finished_out=f), NcError),
                      (dict(finished=f, finished_out=f, eos=512), NcError), (dict(finished=f, eos=2), ValueError),
                      (dict(z=flat[1:].view(2, 3, 512)), NcError), (dict(z=z[:, :, :511]), ValueError),
                      (dict(z=z.float()), TypeError), (dict(t=i(2, 4)), ValueError), (dict(s=s[:1]), ValueError),
                      (dict(s=s.double(), so=s), TypeError), (dict(p=i(2, 3).cpu()), ValueError)):
        with pytest.raises(kind):
            call(**bad)
    big = torch.zeros(1, 33, 512, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(NcError):
        m.beam_select(big, torch.zeros(1, 33, device="cuda"), torch.zeros(1, 33, device="cuda"), i(1, 33), i(1, 33))
    assert m.check() == 0


# ---------------------------------------------------------------- whole searches

def _cfg(**kw):
    d = synth.WORKLOADS["tiny"].model.as_dict()
    d.update(kw)
    return synth.ModelConfig(**d)


def _oracle_search(cfg, w, prompt, beams, steps, eos):
    """Beam search by the oracle's full forward at every step."""
    seqs, scores, fin = [list(prompt)] + [list(prompt)] * (beams - 1), [0.0] + [-np.inf] * (beams - 1), [False] * beams
    for _ in range(steps):
        z = np.stack([oracle.forward_logits(cfg, w, np.array([q], dtype=np.int32))[0, -1] for q in seqs])
        s, t, p, f = _plain(z, np.array(scores), fin if eos >= 0 else None, eos)
        seqs, scores, fin = [seqs[k] + [v] for k, v in zip(p, t)], s, [bool(x) for x in f]
    return [q[len(prompt):] for q in seqs], scores


@pytest.mark.parametrize("hd,h,nkv,page,eos", [(16, 4, 1, 16, -1), (64, 4, 1, 16, 3), (32, 4, 2, 32, -1)])
def test_search_matches_the_oracle(hd, h, nkv, page, eos):
    """fp32: the searches follow the same beams, their scores to 1e-3 (five steps of logits within the fp32 path's 1e-4
    relative error of at most softcap 15)."""
    cfg = _cfg(head_dim=hd, n_head=h, n_kv_head=nkv)
    bits, w = synth.make_weights(cfg, seed=hd, dtype="fp32", std=0.3)
    rng = np.random.default_rng(hd)
    prompts = [rng.integers(0, cfg.vocab, n).tolist() for n in (1, 16, 21, 37)]
    m = Model(cfg.as_dict(), "fp32")
    if eos >= 0:  # a token that some beam picks, so that beams do end
        first, _ = _oracle_search(cfg, w, prompts[2], 3, 2, -1)
        eos = first[1][0]
    tokens, scores = beam_search(m, to_device_weights(bits, w, "fp32"), prompts, beams=3, max_new_tokens=5, eos=eos,
                                 page_size=page)
    for i, p in enumerate(prompts):
        want, ws = _oracle_search(cfg, w, p, 3, 5, eos)
        assert tokens[i].tolist() == want, i
        assert np.allclose(scores[i].cpu().numpy(), ws, atol=1e-3)


def test_search_over_the_dense_cache():
    """nc_prefill and nc_decode_step with the same selection and the dense reorder."""
    cfg = _cfg()
    bits, w = synth.make_weights(cfg, seed=5, dtype="fp32", std=0.3)
    W = to_device_weights(bits, w, "fp32")
    m = Model(cfg.as_dict(), "fp32")
    b, k, n, steps, t_max = 2, 4, 11, 5, 24
    rng = np.random.default_rng(3)
    prompts = rng.integers(0, cfg.vocab, (b, n)).astype(np.int32)
    cache = torch.empty(m.kv_cache_bytes(b * k, t_max) // 4, dtype=torch.float32, device="cuda")
    ws = torch.empty(m.inference_workspace_bytes(b * k, t_max), dtype=torch.uint8, device="cuda")
    logits = torch.empty(b * k, cfg.vocab, device="cuda")
    m.prefill(torch.from_numpy(np.repeat(prompts, k, 0)).cuda(), W, cache, t_max, logits, ws)
    scores = torch.tensor([[0.0] + [-float("inf")] * (k - 1)] * b, device="cuda")
    seqs = [[[] for _ in range(k)] for _ in range(b)]
    tok, par = (torch.empty(b, k, dtype=torch.int32, device="cuda") for _ in range(2))
    for step in range(steps):
        m.beam_select(logits, scores, scores, tok, par)
        seqs = [[seqs[i][p] + [t] for p, t in zip(par[i].tolist(), tok[i].tolist())] for i in range(b)]
        m.beam_reorder(cache, t_max, par, n, n + step)
        m.decode_step(tok.view(-1), n + step, W, cache, t_max, logits, ws)
    assert m.check() == 0
    for i in range(b):
        want, ws_ = _oracle_search(cfg, w, prompts[i].tolist(), k, steps, -1)
        assert seqs[i] == want
        assert np.allclose(scores[i].cpu().numpy(), ws_, atol=1e-3)


def test_a_captured_step_of_a_search():
    """Selection, planning, reordering and the model's forward in one graph, replayed, against the same calls made singly."""
    from bwd_step_b200.generate import PagedCache
    cfg = _cfg(head_dim=64)
    bits, w = synth.make_weights(cfg, seed=2, dtype="bf16", std=0.3)
    W = to_device_weights(bits, w, "bf16")
    m = Model(cfg.as_dict(), "bf16")
    b, k, n = 2, 3, 19
    prompts = torch.from_numpy(np.random.default_rng(0).integers(0, cfg.vocab, (b, 1, n)).astype(np.int32)).cuda()

    def begin():
        c = PagedCache(m, 40, 16, b * k, 64, b * k * n)
        c.plan(torch.full((b * k,), n, dtype=torch.int32, device="cuda"), b * k * n)
        s = dict(cache=c, logits=torch.empty(b * k, cfg.vocab, dtype=torch.bfloat16, device="cuda"),
                 scores=torch.tensor([[0.0, -1.0, -2.0]] * b, device="cuda"),
                 tok=torch.empty(b, k, dtype=torch.int32, device="cuda"), par=torch.empty(b, k, dtype=torch.int32, device="cuda"),
                 start=torch.full((b * k,), n, dtype=torch.int32, device="cuda"), end=torch.zeros(b * k, dtype=torch.int32, device="cuda"),
                 one=torch.ones(b * k, dtype=torch.int32, device="cuda"))
        c.forward(prompts.expand(b, k, n).reshape(-1).contiguous(), W, s["logits"], max_new=n)
        return s

    def step(s):
        c = s["cache"]
        m.beam_select(s["logits"], s["scores"], s["scores"], s["tok"], s["par"])
        s["end"].copy_(c.kv_len)
        c.plan(s["one"], b * k)
        m.beam_reorder_paged(c.kv, s["par"], c.block_table, s["start"], s["end"])
        c.forward(s["tok"].view(-1), W, s["logits"], max_new=1)
    one, two = begin(), begin()
    seen = []
    for _ in range(6):
        step(one)
        seen.append((one["tok"].clone(), one["par"].clone(), one["scores"].clone(), one["logits"].clone()))
    step(two)  # the first step outside, as a warm-up
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(two)
    for tok, par, scores, logits in seen[1:]:
        g.replay()
        assert torch.equal(two["tok"], tok) and torch.equal(two["par"], par)
        assert torch.equal(two["scores"], scores) and torch.equal(two["logits"], logits)
    assert m.check() == 0


@pytest.mark.parametrize("precision,hd,h,nkv", [("bf16", 128, 2, 1), ("bf16", 64, 4, 1), ("bf16", 16, 4, 1), ("fp32", 32, 4, 2)])
def test_paged_forward_matches_the_oracle(precision, hd, h, nkv):
    """Requests of different lengths, their prompts in chunks and then token by token, with one that joins late in a
    released request's place: the last logits of every step against the oracle's full forward."""
    from bwd_step_b200.generate import PagedCache
    cfg = _cfg(head_dim=hd, n_head=h, n_kv_head=nkv, d_model=128)
    bits, w = synth.make_weights(cfg, seed=hd, dtype=precision, std=0.1)
    W = to_device_weights(bits, w, precision)
    m = Model(cfg.as_dict(), precision)
    rng = np.random.default_rng(1)
    seqs = [rng.integers(0, cfg.vocab, n).astype(np.int32) for n in (150, 37, 16, 90)]
    full = [oracle.forward_logits(cfg, w, s[None])[0] for s in seqs]
    late = rng.integers(0, cfg.vocab, 40).astype(np.int32)
    late_full = oracle.forward_logits(cfg, w, late[None])[0]
    # (new tokens per request, released requests) of every step
    plan = [((100, 20, 0, 1), ()), ((30, 1, 15, 60), ()), ((1, 1, 1, 1), ()), ((7, 0, 0, 28), ()), ((1, 33, 0, 0), (1,)),
            ((1, 1, 0, 0), ())]
    tol = {"bf16": 2e-2, "fp32": 1e-4}[precision]
    cache = PagedCache(m, 30, 16, 4, 160, 200)
    cache.kv.fill_(float("nan"))
    logits = torch.empty(4, cfg.vocab, dtype=m.weight_dtype, device="cuda")
    at = [0] * 4
    for news, gone in plan:
        for r in gone:
            seqs[r], full[r], at[r] = late, late_full, 0
        toks = np.concatenate([seqs[r][at[r]:at[r] + n] for r, n in enumerate(news)])
        rows = len(toks) + 2
        dev = torch.zeros(rows, dtype=torch.int32, device="cuda")
        dev[:len(toks)] = torch.from_numpy(toks).cuda()
        release = torch.tensor([int(r in gone) for r in range(4)], dtype=torch.int32, device="cuda")
        cache.plan(torch.tensor(news, dtype=torch.int32, device="cuda"), rows, release=release if gone else None)
        cache.forward(dev, W, logits, max_new=max(news))
        assert m.check() == 0
        at = [a + n for a, n in zip(at, news)]
        assert cache.kv_len.tolist() == at
        for r, n in enumerate(news):
            got = logits[r].float().cpu().numpy().astype(np.float64)
            if n == 0:
                assert not got.any()
                continue
            ref = full[r][at[r] - 1]
            assert np.linalg.norm(got - ref) / np.linalg.norm(ref) <= tol, (r, at[r])
