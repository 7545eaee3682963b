"""Decode with attention weights against softmax in 64 bits, eviction against its definition, value for value,
and both together with the allocator."""
import math

import pytest
import torch

import fp64lib as ref
import paged_kv_cache_428_b200 as pa

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def _pool(lens, nb_extra, h_kv, bs, d, g, dtype=torch.bfloat16):
    """(k, v, tables, free blocks): random rows where the sequences' tokens are, NaN (or -128) elsewhere."""
    need = [-(-n // bs) for n in lens]
    nb = sum(need) + nb_extra
    order = torch.randperm(nb, generator=g).tolist()
    tab = torch.full((len(lens), max(need + [1])), -1, dtype=torch.int32)
    used = torch.zeros(nb, bs, dtype=torch.bool)
    at = 0
    for s, n in enumerate(need):
        tab[s, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
        for b in range(n):
            used[tab[s, b], :min(bs, lens[s] - b * bs)] = True
    out = []
    for _ in "kv":
        if dtype == torch.bfloat16:
            x = torch.randn((nb, h_kv, bs, d), generator=g).to(dtype)
            x[~used[:, None, :].expand(nb, h_kv, bs)] = math.nan
        else:
            x = torch.randint(0, 127, (nb, h_kv, bs, d), generator=g, dtype=torch.int16).to(torch.int8)
            x[~used[:, None, :].expand(nb, h_kv, bs)] = -128
            x = x.view(dtype)
        out.append(x)
    return out[0], out[1], tab, order[at:]


# ---------------------------------------------------------------------------------- decode weights
def _decode(q, k, v, tab, ctx, weights, max_len=None, workspace=None):
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device=DEV)
    pa.pa_decode_weights(out, weights, q.to(DEV), k.to(DEV), v.to(DEV), tab.to(DEV), ctx.to(DEV),
                         int(ctx.max()) if max_len is None else max_len, workspace=workspace)
    torch.cuda.synchronize()
    return out


def _check_decode(q, k, v, tab, lens, out, got, before, counted=None):
    g = q.shape[1] // k.shape[1]
    d = q.shape[2]
    for s, n in enumerate(lens):
        if n == 0:
            assert not out[s].any() and torch.equal(got[s].cpu(), before[s])
            continue
        rk, rv = ref.rows_of(k, tab[s], n), ref.rows_of(v, tab[s], n)
        o, mag, w = ref.attend(q[s:s + 1], rk, rv, torch.tensor([n - 1]), 1 / math.sqrt(d))
        ref.check_rows(out[s:s + 1], o, mag, 8, "sequence %d of %d tokens" % (s, n))
        # a logit: D / 16 matrix steps whose sums are cut at 2^-22 of what has been added up, then two roundings;
        # the same for the normaliser; the sums themselves in fp32
        size = (q[s].double().abs().view(k.shape[1], g, d) @ rk.abs().transpose(1, 2)).reshape(-1, n) / math.sqrt(d)
        err = 2.0 ** -22 * ((d // 16 + 2) * size + 2 * size.amax() + 8)
        p = w[0].view(-1, g, n)
        want = before[s].double()
        bound = 2.0 ** -22 * (want.abs() + 1e-30)
        m = n if counted is None else min(n, counted)
        want[:, :m] += p.sum(1)[:, :m]
        bound[:, :m] += (p * (err + err.amax(1, keepdim=True)).view(-1, g, n)).sum(1)[:, :m] + 2.0 ** -22 * p.sum(1)[:, :m]
        far = (got[s].cpu().double() - want).abs()
        assert (far <= bound).all(), (s, n, float((far / bound).max()))
        assert torch.equal(got[s, :, m:].cpu(), before[s, :, m:])                  # nothing behind the last token


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bs", [16, 32, 64])
@pytest.mark.parametrize("g", [1, 2, 4, 8])
def test_decode_weights_every_variant(d, bs, g):
    gen, lens = _gen(d + bs + g), [1, 0, bs, bs + 1, 513, 3 * bs - 1, 100]
    k, v, tab, _ = _pool(lens, 3, 2, bs, d, gen)
    q = (torch.randn((len(lens), 2 * g, d), generator=gen) * 2).to(torch.bfloat16)
    before = torch.rand((len(lens), 2, 520), generator=gen) * 0.01
    w = before.to(DEV)
    out = _decode(q, k, v, tab, torch.tensor(lens, dtype=torch.int32), w)
    _check_decode(q, k, v, tab, lens, out, w, before)
    assert pa.pa_device_errors() == 0


@pytest.mark.parametrize("lens,h_kv,g", [([40000], 1, 4), ([9000, 3], 2, 1), ([(7 * i) % 60 for i in range(200)], 1, 8)])
def test_decode_weights_long_and_many(lens, h_kv, g):
    gen = _gen(3)
    k, v, tab, _ = _pool(lens, 1, h_kv, 16, 64, gen)
    q = torch.randn((len(lens), h_kv * g, 64), generator=gen).to(torch.bfloat16)
    before = torch.zeros((len(lens), h_kv, max(lens) + 1))
    w = before.to(DEV)
    ctx = torch.tensor(lens, dtype=torch.int32)
    out = _decode(q, k, v, tab, ctx, w)
    _check_decode(q, k, v, tab, lens, out, w, before)
    again = before.to(DEV)
    assert torch.equal(_decode(q, k, v, tab, ctx, again), out) and torch.equal(again, w)      # the same bits


def test_decode_weights_add_up_and_bounds():
    gen, lens = _gen(4), [100, 37]
    k, v, tab, _ = _pool(lens, 1, 2, 16, 64, gen)
    q = torch.randn((2, 4, 64), generator=gen).to(torch.bfloat16)
    ctx = torch.tensor(lens, dtype=torch.int32)
    w = torch.zeros((2, 2, 101), device=DEV)
    for _ in range(3):
        _decode(q, k, v, tab, ctx, w)
    assert torch.allclose(w.sum(-1), torch.full((2, 2), 6.0, device=DEV), rtol=1e-5)     # 3 steps x 2 heads
    # a bound below a context: attended as a whole, weights up to the bound, reported
    before = torch.zeros((2, 2, 50))
    w = before.to(DEV)
    pa.pa_device_errors(clear=True)
    out = _decode(q, k, v, tab, ctx, w, max_len=50)
    assert pa.pa_device_errors() == pa.PA_DEVERR_BAD_LENGTH
    _check_decode(q, k, v, tab, lens, out, w, before, counted=50)
    # no tokens counted at all
    w = torch.ones((2, 2, 3), device=DEV)
    out = _decode(q, k, v, tab, ctx, w, max_len=0)
    assert pa.pa_device_errors() == pa.PA_DEVERR_BAD_LENGTH and bool((w == 1).all()) and torch.isfinite(out).all()
    # a block outside the pool: the row is NaN and its weights stay
    bad = tab.clone()
    bad[0, 2] = -1
    w = before.to(DEV).expand(2, 2, 50).contiguous()
    out = _decode(q, k, v, bad, torch.tensor([50, 37], dtype=torch.int32), w)
    assert pa.pa_device_errors() == pa.PA_DEVERR_BAD_BLOCK
    assert torch.isnan(out[0]).all() and not w[0].any() and w[1].any()


def test_decode_weights_workspace_and_graph():
    gen = _gen(5)
    ws = torch.zeros(32 << 20, dtype=torch.uint8, device=DEV)
    cases = []
    for lens, h_kv, g, bs, d in (([300, 20], 2, 4, 16, 128), ([3000], 1, 8, 32, 64), ([64] * 30, 2, 1, 64, 64)):
        k, v, tab, _ = _pool(lens, 1, h_kv, bs, d, gen)
        q = torch.randn((len(lens), h_kv * g, d), generator=gen).to(torch.bfloat16)
        cases.append([t.to(DEV) for t in (q, k, v, tab, torch.tensor(lens, dtype=torch.int32))] + [max(lens)])
    def step(c, out, w):
        return pa.pa_decode_weights(out, w, *c[:5], c[5], workspace=ws)
    alone = []
    for c in cases:
        w = torch.zeros((c[0].shape[0], c[1].shape[1], c[5]), device=DEV)
        out = torch.zeros_like(c[0])
        step(c, out, w)
        alone.append((out, w))
    outs = [(torch.zeros_like(o), torch.zeros_like(w)) for o, w in alone]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        for c, (o, w) in zip(cases, outs):
            step(c, o, w)
    for _ in range(2):
        for o, w in outs:
            w.zero_()
        graph.replay()
    torch.cuda.synchronize()
    for (o, w), (o2, w2) in zip(alone, outs):
        assert torch.equal(o, o2) and torch.equal(w, w2)
    assert int(ws[:65536 * 4].count_nonzero()) == 0


# --------------------------------------------------------------------------------------- eviction
def _choose(w, n, budget, recent):
    """Positions kept of n tokens with weights w (a list)."""
    m = min(n, budget)
    last = min(m, recent)
    key = [x if x > 0 else 0.0 for x in w[:n - last]]
    heavy = sorted(sorted(range(n - last), key=lambda i: (-key[i], i))[:m - last])
    return heavy + list(range(n - last, n))


def _evict_case(lens, h_kv, bs, d, budget, recent, seed, dtype=torch.bfloat16, weights=None, stride=None, max_len=None, extra=0):
    g = _gen(seed)
    fresh = [-(-min(n, budget) // bs) for n in lens]
    k, v, tab, free = _pool(lens, sum(fresh) + 2, h_kv, bs, d, g, dtype)
    stride = max(max(lens), 1) + 3 if stride is None else stride
    if weights is None:
        weights = torch.exp(2 * torch.randn((len(lens), h_kv, stride), generator=g))
        weights = torch.where(torch.rand(weights.shape, generator=g) < 0.4, weights.round(), weights)
    new_tab = torch.full((len(lens), max(fresh + [1])), -1, dtype=torch.int32)
    at = 0
    for s, m in enumerate(fresh):
        new_tab[s, :m] = torch.tensor(free[at:at + m], dtype=torch.int32)
        at += m
    kc, vc = k.to(DEV), v.to(DEV)
    kept = torch.full((len(lens), h_kv, budget), 99, dtype=torch.int32, device=DEV)
    new_w = torch.full((len(lens), h_kv, budget + extra), 99.0, device=DEV)
    new_len = torch.full((len(lens),), 99, dtype=torch.int32, device=DEV)
    pa.pa_evict(kc, vc, weights.to(DEV), tab.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV), new_tab.to(DEV),
                max(lens) if max_len is None else max_len, budget, recent, kept, new_w, new_len)
    torch.cuda.synchronize()
    raw = lambda t: t.cpu().view(torch.uint8 if dtype != torch.bfloat16 else torch.int16)  # noqa: E731
    want_k, want_v = raw(k).clone(), raw(v).clone()
    want_kept = torch.full(kept.shape, -1, dtype=torch.int32)
    want_w = torch.zeros(new_w.shape)
    for s, n in enumerate(lens):
        for h in range(h_kv):
            keep = torch.tensor(_choose(weights[s, h].tolist(), n, budget, recent), dtype=torch.long)
            m = keep.numel()
            want_kept[s, h, :m] = keep.int()
            want_w[s, h, :m] = weights[s, h, keep]
            j = torch.arange(m)
            src, dst = tab[s].long()[keep // bs], new_tab[s].long()[j // bs]
            for want in (want_k, want_v):
                want[dst, h, j % bs] = want[src, h, keep % bs]
    assert torch.equal(new_len.cpu(), torch.tensor([min(n, budget) for n in lens], dtype=torch.int32))
    assert torch.equal(kept.cpu(), want_kept)
    assert torch.equal(new_w.cpu().nan_to_num(nan=-5.0), want_w.nan_to_num(nan=-5.0))
    assert torch.equal(raw(kc), want_k) and torch.equal(raw(vc), want_v)
    assert pa.pa_device_errors() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bs", [16, 32, 64])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.int8, torch.float8_e4m3fn])
def test_evict_every_variant(d, bs, dtype):
    _evict_case([1, 0, 200, 50, 51, 333, 7], 3, bs, d, 50, 13, d + bs, dtype, extra=9)


@pytest.mark.parametrize("budget,recent", [(1, 0), (1, 1), (64, 0), (64, 64), (63, 62), (700, 3), (5, 2)])
def test_evict_budgets(budget, recent):
    _evict_case([700, 64, 63, 65, 2, 1], 2, 16, 64, budget, recent, budget)


@pytest.mark.parametrize("n", [8192, 8193, 20000, 66000, 140000])
def test_evict_long(n):
    """One CTA, clusters of 2, 4 and 8, and rows that do not fit their shared memory."""
    _evict_case([n, n // 3, 100], 2, 64, 64, 600, 100, n)


def test_evict_a_bound_below_the_contexts():
    _evict_case([20000, 9000], 1, 64, 64, 600, 100, 1, max_len=700)


@pytest.mark.parametrize("max_len", [0, 1, 200, 599])
def test_evict_a_bound_below_the_budget(max_len):
    """The bound sizes the launch only: contexts that pass it, and the budget above it, keep all their rows."""
    _evict_case([20000, 9000, 50, 0, 601], 2, 64, 64, 600, 100, 1, max_len=max_len)


@pytest.mark.parametrize("what", ["zero", "one", "nan", "negative", "inf", "tiny", "two"])
@pytest.mark.parametrize("n", [600, 30000])
def test_evict_weights_that_are_alike(what, n):
    w = torch.zeros((1, 2, n))
    g = _gen(2)
    if what == "one":
        w += 1
    elif what == "nan":
        w = torch.where(torch.rand(w.shape, generator=g) < 0.5, torch.tensor(math.nan), torch.rand(w.shape, generator=g))
    elif what == "negative":
        w = -torch.rand(w.shape, generator=g)
        w[..., ::7] = -0.0
    elif what == "inf":
        w = torch.where(torch.rand(w.shape, generator=g) < 0.3, torch.tensor(math.inf), torch.rand(w.shape, generator=g))
    elif what == "tiny":
        w = torch.randint(0, 40, w.shape, generator=g).float() * 2.0 ** -149
    elif what == "two":
        w = torch.where(torch.rand(w.shape, generator=g) < 0.5, 1.0, 1.0 + 2.0 ** -23)
    _evict_case([n], 2, 16, 64, 250, 20, 3, weights=w, stride=n)


def test_evict_captured_and_on_another_stream():
    g = _gen(9)
    lens = [700, 90, 3]
    k, v, tab, free = _pool(lens, 20, 2, 16, 64, g)
    new_tab = torch.tensor(free[:15], dtype=torch.int32, device=DEV).view(3, 5)
    w = torch.rand((3, 2, 700), generator=g).to(DEV)
    tab, ctx = tab.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)

    def buffers():
        return (k.to(DEV), v.to(DEV), torch.zeros((3, 2, 70), dtype=torch.int32, device=DEV),
                torch.zeros((3, 2, 80), device=DEV), torch.zeros(3, dtype=torch.int32, device=DEV))

    def call(b, **kw):
        pa.pa_evict(b[0], b[1], w, tab, ctx, new_tab, 700, 70, 9, b[2], b[3], b[4], **kw)

    first, second, third = buffers(), buffers(), buffers()
    call(first)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    call(second, stream=side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(third)
    for _ in range(2):
        for t in third[2:]:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
    for other in (second, third):
        for a, b in zip(first, other):
            assert torch.equal(a.nan_to_num(nan=5.0), b.nan_to_num(nan=5.0))


def test_evict_bad_blocks_and_lengths():
    g = _gen(6)
    k, v, tab, free = _pool([100, 100, 100], 12, 2, 16, 64, g)
    tab[0, 1] = -1
    new_tab = torch.tensor(free[:12], dtype=torch.int32).view(3, 4)
    new_tab[1, 2] = 10 ** 6
    kc, vc = k.to(DEV), v.to(DEV)
    kept = torch.zeros((3, 2, 50), dtype=torch.int32, device=DEV)
    new_w, new_len = torch.zeros((3, 2, 50), device=DEV), torch.zeros(3, dtype=torch.int32, device=DEV)
    pa.pa_device_errors(clear=True)
    pa.pa_evict(kc, vc, torch.rand((3, 2, 100), device=DEV), tab.to(DEV), torch.tensor([100, 100, 101], dtype=torch.int32, device=DEV),
                new_tab.to(DEV), 100, 50, 5, kept, new_w, new_len)
    assert pa.pa_device_errors() == pa.PA_DEVERR_BAD_BLOCK | pa.PA_DEVERR_BAD_LENGTH
    assert new_len.tolist() == [50, 50, 0] and bool((kept[2] == -1).all()) and not new_w[2].any()
    for b in free[8:]:
        assert torch.isnan(kc[b]).all()                              # the third sequence's new blocks: untouched
    with pytest.raises(pa.PagedKVError):
        pa.pa_evict(kc, vc, new_w, tab.to(DEV), new_len, new_tab.to(DEV), 50, 50, 5, kept, new_w, new_len.clone())


def test_evict_a_context_past_the_countable():
    """A length near the end of 32 bits over a row of weights that has room for it keeps nothing and is reported."""
    g = _gen(8)
    k, v, tab, free = _pool([100], 4, 1, 16, 64, g)
    w = torch.empty((1, 1, 2 ** 31), device=DEV)
    kept = torch.zeros((1, 1, 20), dtype=torch.int32, device=DEV)
    new_w, new_len = torch.ones((1, 1, 20), device=DEV), torch.ones(1, dtype=torch.int32, device=DEV)
    pa.pa_device_errors(clear=True)
    for n in (2 ** 30 + 1, 2 ** 31 - 1):
        pa.pa_evict(k.to(DEV), v.to(DEV), w, tab.to(DEV), torch.tensor([n], dtype=torch.int32, device=DEV),
                    torch.tensor([free[:2]], dtype=torch.int32, device=DEV), 100, 20, 5, kept, new_w, new_len)
        assert pa.pa_device_errors() == pa.PA_DEVERR_BAD_LENGTH
        assert new_len.tolist() == [0] and bool((kept == -1).all()) and not new_w.any()


def test_a_chat_that_outgrows_its_budget():
    """Append, decode with weights, evict when the budget is exceeded, go on: the attention is over the kept
    rows, and two sequences that share blocks do not disturb each other."""
    g, h, grp, d, bs, nb, budget, recent = _gen(7), 2, 4, 64, 16, 64, 48, 8
    alloc = pa.BlockAllocator(nb, bs, seed=1)
    kc = torch.full((nb, h, bs, d), math.nan, dtype=torch.bfloat16, device=DEV)
    vc = kc.clone()
    rows = []                                            # per sequence: [h][t] -> (k, v) rows of the model
    first = alloc.new_seq()
    slots, _ = alloc.append_n(first, 40)
    k, v = (torch.randn((40, h, d), generator=g).to(torch.bfloat16) for _ in "kv")
    pa.pa_reshape_and_cache(k.to(DEV), v.to(DEV), kc, vc, torch.tensor(slots, device=DEV))
    seqs = [first, alloc.fork(first)]
    rows = [[[(k[t, i], v[t, i]) for t in range(40)] for i in range(h)] for _ in seqs]
    weights = torch.zeros((2, h, 64), device=DEV)
    evictions = 0
    for step in range(40):
        slots, cow = alloc.append_batch(seqs)
        if cow:
            pa.pa_copy_blocks([kc], [vc], torch.tensor(cow, dtype=torch.int64, device=DEV))
        k, v = (torch.randn((2, h, d), generator=g).to(torch.bfloat16) for _ in "kv")
        pa.pa_reshape_and_cache(k.to(DEV), v.to(DEV), kc, vc, torch.tensor(slots, device=DEV))
        for s in range(2):
            for i in range(h):
                rows[s][i].append((k[s, i], v[s, i]))
        tab, ctx = alloc.block_table(seqs, 8)
        q = torch.randn((2, h * grp, d), generator=g).to(torch.bfloat16)
        out = torch.empty_like(q, device=DEV)
        pa.pa_decode_weights(out, weights, q.to(DEV), kc, vc, tab.to(DEV), ctx.to(DEV), 64)
        for s in range(2):
            n = int(ctx[s])
            rk, rv = (torch.stack([torch.stack([r[j] for r in rows[s][i]]) for i in range(h)]).double() for j in (0, 1))
            o, mag, _ = ref.attend(q[s:s + 1], rk, rv, torch.tensor([n - 1]), 1 / math.sqrt(d))
            ref.check_rows(out[s:s + 1], o, mag, 8, "step %d" % step)
        if int(ctx.max()) > budget + 8:
            evictions += 1
            fresh = [alloc.new_seq() for _ in seqs]
            for s, n in zip(fresh, ctx.tolist()):
                alloc.append_n(s, min(n, budget))
            new_tab, _ = alloc.block_table(fresh, 8)
            kept = torch.empty((2, h, budget), dtype=torch.int32, device=DEV)
            new_w, new_len = torch.empty_like(weights), torch.empty(2, dtype=torch.int32, device=DEV)
            pa.pa_evict(kc, vc, weights, tab.to(DEV), ctx.to(DEV), new_tab.to(DEV), 64, budget, recent, kept, new_w, new_len)
            before = weights.cpu()
            for s in range(2):
                alloc.free_seq(seqs[s])
                assert int(new_len[s]) == alloc.seq_len(fresh[s])
                for i in range(h):
                    keep = _choose(before[s, i].tolist(), int(ctx[s]), budget, recent)
                    assert kept[s, i].tolist() == keep
                    rows[s][i] = [rows[s][i][t] for t in keep]
            seqs, weights = fresh, new_w
    assert evictions >= 2 and pa.pa_device_errors() == 0
