"""Attention with modified scores (cap, distance bias, window, prefix) against its definition in 64 bits, for
single tokens and for chunks."""
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


def _pool(lens, h_kv, bs, d, g, window=0, new=None):
    """(k, v, tables): NaN in every slot without a token.  With a window, what lies before it for every query of
    the call is gone: rows are NaN, and the table entries of whole blocks before it are -1."""
    need = [-(-n // bs) for n in lens]
    nb = sum(need) + 3
    order = torch.randperm(nb, generator=g).tolist()
    tab = torch.full((len(lens), max(need + [1]) + 1), -1, dtype=torch.int32)
    used = torch.zeros(nb, bs, dtype=torch.bool)
    gone = []
    at = 0
    for s, (n, blocks) in enumerate(zip(lens, need)):
        tab[s, :blocks] = torch.tensor(order[at:at + blocks], dtype=torch.int32)
        at += blocks
        lo = max(0, n - (new[s] if new else 1) - window + 1) if window and n else 0
        for b in range(blocks):
            used[tab[s, b], :min(bs, n - b * bs)] = True
            used[tab[s, b], :max(0, min(bs, lo - b * bs))] = False
        gone.append(lo // bs)
    k, v = (torch.randn((nb, h_kv, bs, d), generator=g).to(torch.bfloat16) for _ in "kv")
    for x in (k, v):
        x[~used[:, None, :].expand(nb, h_kv, bs)] = math.nan
    full = tab.clone()
    for s, n in enumerate(gone):
        tab[s, :n] = -1
    return k, v, tab, full


def _slopes(h_q):
    return torch.exp2(-8.0 * torch.arange(1, h_q + 1) / h_q)


def _logit_error(q, k, scale, cap, slopes, d):
    """Of one logit: D / 16 matrix steps whose sums are cut at 2^-22 of what has been added up, two more
    roundings, tanh to 2^-22 of the cap (and its result rounded), the distance bias rounded at its own size."""
    far = float(slopes.max()) * k.shape[1] if slopes is not None else 0.0
    size = float(q.double().abs().amax() * k.abs().sum(-1).amax()) * scale
    return 2.0 ** -22 * ((d // 16 + 2) * size + 2 * cap + far + 1)


MODS = [dict(softcap=30.0), dict(alibi=True), dict(window=40), dict(softcap=4.0, alibi=True, window=100)]


# ----------------------------------------------------------------------------------------- decode
def _decode(lens, h_kv, g, bs, d, seed, softcap=0.0, alibi=False, window=0, max_len=None, workspace=None, q_factor=2.0):
    gen = _gen(seed)
    k, v, tab, full = _pool(lens, h_kv, bs, d, gen, window)
    q = (torch.randn((len(lens), h_kv * g, d), generator=gen) * q_factor).to(torch.bfloat16)
    slopes = _slopes(h_kv * g) if alibi else None
    ctx = torch.tensor(lens, dtype=torch.int32)
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device=DEV)
    pa.pa_decode_scoremod(out, q.to(DEV), k.to(DEV), v.to(DEV), tab.to(DEV), ctx.to(DEV), max(lens) if max_len is None else max_len,
                          softcap=softcap, alibi_slopes=None if slopes is None else slopes.to(DEV), window=window,
                          workspace=workspace)
    torch.cuda.synchronize()
    assert pa.pa_device_errors() == 0
    for s, n in enumerate(lens):
        if n == 0:
            assert not out[s].any()
            continue
        rk, rv = (ref.rows_of(x, full[s], n).nan_to_num(0.0) for x in (k, v))
        o, mag, _ = ref.attend(q[s:s + 1], rk, rv, torch.tensor([n - 1]), 1 / math.sqrt(d), softcap, slopes, window)
        ref.check_rows(out[s:s + 1], o, mag, 8, "sequence %d of %d tokens" % (s, n),
                       _logit_error(q[s], rk, 1 / math.sqrt(d), softcap, slopes, d))
    return out


@pytest.mark.parametrize("mod", MODS, ids=lambda m: "-".join(m))
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bs", [16, 32, 64])
@pytest.mark.parametrize("g", [1, 2, 4, 8])
def test_decode_every_variant(d, bs, g, mod):
    _decode([1, 0, bs, bs + 1, 3 * bs - 1, 333, 40, 41], 2, g, bs, d, d + bs + g, **mod)


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 63, 64, 65, 200, 299, 300, 301, 10 ** 6])
def test_decode_window_edges(window):
    _decode([300, 16, 17, 1, 64], 2, 4, 32, 64, window, window=window, softcap=20.0, alibi=True)


@pytest.mark.parametrize("lens,h_kv,g,window", [([50000], 1, 4, 0), ([50000, 100], 2, 8, 20000), ([(11 * i) % 70 for i in range(300)], 1, 2, 33)])
def test_decode_long_and_many(lens, h_kv, g, window):
    out = _decode(lens, h_kv, g, 16, 64, 3, softcap=50.0, alibi=True, window=window)
    assert torch.equal(out, _decode(lens, h_kv, g, 16, 64, 3, softcap=50.0, alibi=True, window=window))
    # a bound that is too low costs speed only (and splits the work elsewhere, so bits may differ)
    _decode(lens, h_kv, g, 16, 64, 3, softcap=50.0, alibi=True, window=window, max_len=1)


def test_decode_large_scores():
    """Scores far beyond the cap, where tanh is +-1 to the last bit."""
    _decode([200, 33], 2, 4, 16, 128, 4, softcap=3.0, q_factor=300.0)


def test_a_cache_past_32_bits():
    """Blocks whose elements lie past 2^32 bytes and 2^31 elements, in a pool that is mostly untouched memory."""
    nb, h, bs, d, n = 1 << 19, 4, 16, 128, 150
    assert nb * h * bs * d > 2 ** 31
    gen = _gen(17)
    kc, vc = (torch.empty((nb, h, bs, d), dtype=torch.bfloat16, device=DEV) for _ in "kv")
    k, v = (torch.randn((n, h, d), generator=gen).to(torch.bfloat16) for _ in "kv")
    blocks = torch.tensor([nb - 1 - 3 * i for i in range(10)])
    t = torch.arange(n)
    pa.pa_reshape_and_cache(k.to(DEV), v.to(DEV), kc, vc, (blocks[t // bs] * bs + t % bs).to(DEV))
    tab = blocks.int().view(1, 10).to(DEV)
    ctx = torch.tensor([n], dtype=torch.int32, device=DEV)
    q = torch.randn((n, h * 2, d), generator=gen).to(torch.bfloat16)
    rk, rv = k.double().transpose(0, 1), v.double().transpose(0, 1)
    o, mag, _ = ref.attend(q, rk, rv, t, 1 / math.sqrt(d), 10.0, None, 60)
    err = _logit_error(q, rk, 1 / math.sqrt(d), 10.0, None, d)
    out, one = torch.empty_like(q, device=DEV), torch.empty_like(q[:1], device=DEV)
    pa.pa_prefill_scoremod(out, q.to(DEV), kc, vc, tab, torch.tensor([0, n], dtype=torch.int32, device=DEV), ctx, n,
                           pa.make_prefill_workspace(), softcap=10.0, window=60)
    pa.pa_decode_scoremod(one, q[-1:].to(DEV), kc, vc, tab, ctx, n, softcap=10.0, window=60)
    ref.check_rows(out, o, mag, 8, "prefill", err)
    ref.check_rows(one, o[-1:], mag[-1:], 8, "decode", err)
    # eviction from there to there
    w = torch.rand((1, h, n), generator=gen).to(DEV)
    fresh = torch.tensor([[nb - 2, nb - 50]], dtype=torch.int32, device=DEV)
    kept, nw = torch.empty((1, h, 30), dtype=torch.int32, device=DEV), torch.empty((1, h, 30), device=DEV)
    pa.pa_evict(kc, vc, w, tab, ctx, fresh, n, 30, 4, kept, nw, ctx.clone())
    for i in range(h):
        rows = k[kept[0, i].cpu().long(), i]
        assert torch.equal(torch.cat([kc[nb - 2, i], kc[nb - 50, i, :14]]).cpu(), rows)
    # and a block-scaled write and decode past 2^31 bytes of codes
    del kc, vc
    kq, vq = (torch.empty((nb, h, bs, d), dtype=torch.int8, device=DEV) for _ in "kv")
    ks, vs = pa.make_block_scales(nb, h)
    pa.pa_reshape_and_cache_block_scales(k.to(DEV), v.to(DEV), kq, vq, ks, vs, (blocks[t // bs] * bs + t % bs).to(DEV))
    pa.pa_decode_block_scales(one, q[-1:].to(DEV), kq, vq, ks, vs, tab, ctx, n)
    b = blocks.to(DEV)
    rk, rv = ((c[b].double() * s[b].double()[:, :, None, None]).permute(1, 0, 2, 3).reshape(h, -1, d)[:, :n].cpu()
              for c, s in ((kq, ks), (vq, vs)))
    o, mag, _ = ref.attend(q[-1:], rk, rv, t[-1:], 1 / math.sqrt(d))
    ref.check_rows(one, o, mag, 11, "codes", extra=2.0 ** -40 * 127 * float(vs.max()) * n)
    assert pa.pa_device_errors() == 0


@pytest.mark.parametrize("softcap", [2.0 ** -64, 1e3, 1e6, 1e20])
def test_caps_far_from_the_scores(softcap):
    """A cap far above the scores leaves them as they are; one far below leaves their signs."""
    _decode([200, 33], 2, 4, 16, 64, 14, softcap=softcap)
    _prefill([60, 0], [80, 30], 2, 4, 16, 64, 14, softcap=softcap)


@pytest.mark.parametrize("softcap", [2.0 ** -64, 1e-15, 1e-11, 1e-6, 50.0, 1e25, 2e38])
def test_scores_that_are_all_zero(softcap):
    """Zero queries (as in padded rows) under caps of any size: plain means of V."""
    _decode([200, 33], 2, 4, 16, 64, 24, softcap=softcap, q_factor=0.0)
    _prefill([60, 0], [80, 30], 2, 4, 16, 64, 24, softcap=softcap, q_factor=0.0)


def test_prefill_scores_whose_squares_leave_fp32():
    """Scores of 1e19 and more under a cap far above them."""
    _prefill([60, 0], [80, 30], 2, 4, 16, 64, 25, softcap=1e25, q_factor=1e19)
    _decode([200, 33], 2, 4, 16, 64, 25, softcap=1e25, q_factor=1e19)


def test_decode_without_any_is_decode():
    gen = _gen(5)
    k, v, tab, _ = _pool([400, 77], 2, 16, 128, gen)
    q = torch.randn((2, 8, 128), generator=gen).to(torch.bfloat16)
    args = [t.to(DEV) for t in (q, k, v, tab, torch.tensor([400, 77], dtype=torch.int32))]
    a, b = torch.empty_like(args[0]), torch.empty_like(args[0])
    pa.pa_decode_scoremod(a, *args, 400)
    pa.pa_decode(b, *args, 400)
    assert (a.float() - b.float()).abs().max() <= 2.0 ** -7 * b.float().abs().max()


def test_decode_bad_block_inside_the_window():
    gen = _gen(6)
    k, v, tab, _ = _pool([100, 100], 2, 16, 64, gen)
    q = torch.randn((2, 4, 64), generator=gen).to(torch.bfloat16).to(DEV)
    tab[0, 5], tab[1, 1] = 999, 999
    out = torch.empty_like(q)
    pa.pa_device_errors(clear=True)
    pa.pa_decode_scoremod(out, q, k.to(DEV), v.to(DEV), tab.to(DEV), torch.tensor([100, 100], dtype=torch.int32, device=DEV), 100,
                          window=40)
    assert pa.pa_device_errors() == pa.PA_DEVERR_BAD_BLOCK
    assert torch.isnan(out[0]).all() and torch.isfinite(out[1]).all()


# ---------------------------------------------------------------------------------------- prefill
def _prefill(cached, chunk, h_kv, g, bs, d, seed, softcap=0.0, alibi=False, window=0, prefix=None, rows=None, q_factor=2.0,
             max_query=None, workspace=None):
    gen = _gen(seed)
    lens = [a + b for a, b in zip(cached, chunk)]
    k, v, tab, full = _pool(lens, h_kv, bs, d, gen, window, chunk)
    start = torch.zeros(len(lens) + 1, dtype=torch.int32)
    start[1:] = torch.cumsum(torch.tensor(chunk), 0)
    q = (torch.randn((int(start[-1]) + 2, h_kv * g, d), generator=gen) * q_factor).to(torch.bfloat16)
    slopes = _slopes(h_kv * g) if alibi else None
    ctx = torch.tensor(lens, dtype=torch.int32)
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device=DEV)
    ws = pa.make_prefill_workspace() if workspace is None else workspace
    pa.pa_prefill_scoremod(out, q.to(DEV), k.to(DEV), v.to(DEV), tab.to(DEV), start.to(DEV), ctx.to(DEV),
                           max(chunk) if max_query is None else max_query, ws, softcap=softcap,
                           alibi_slopes=None if slopes is None else slopes.to(DEV), window=window,
                           prefix_lens=None if prefix is None else torch.tensor(prefix, dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    assert pa.pa_device_errors() == 0 and int(ws.count_nonzero()) == 0
    assert bool((out[int(start[-1]):] == 7.0).all())                 # rows behind the last sequence
    for s, n in enumerate(lens):
        a, m = int(start[s]), chunk[s]
        pick = torch.arange(m) if rows is None else torch.unique(torch.tensor([0, m - 1] + [(i * 7919) % m for i in range(rows)]))
        if not m:
            continue
        rk, rv = (ref.rows_of(x, full[s], n).nan_to_num(0.0) for x in (k, v))
        o, mag, _ = ref.attend(q[a + pick], rk, rv, n - m + pick, 1 / math.sqrt(d), softcap, slopes, window,
                               min(n, prefix[s]) if prefix else 0)
        ref.check_rows(out[a + pick.to(DEV)], o, mag, 8, "sequence %d: %d rows of %d tokens" % (s, m, n),
                       _logit_error(q[a + pick], rk, 1 / math.sqrt(d), softcap, slopes, d))
    return out


@pytest.mark.parametrize("mod", MODS + [dict(prefix=[9, 300, 0, 70, 1, 40])], ids=lambda m: "-".join(m))
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bs", [16, 32, 64])
@pytest.mark.parametrize("g", [1, 2, 4, 8])
def test_prefill_every_variant(d, bs, g, mod):
    _prefill([0, 37, 100, 63, 5, 130], [70, 1, 150, 65, 0, 40], 2, g, bs, d, d + bs + g, **mod)


@pytest.mark.parametrize("window", [1, 2, 16, 63, 64, 65, 130, 400])
@pytest.mark.parametrize("g,bs", [(1, 16), (4, 64), (8, 32)])
def test_prefill_window_edges(window, g, bs):
    """Windows from one token to more than the context, chunks of several query tiles: rows of one tile whose
    first tokens lie in different KV tiles, tiles that the first or last rows do not see at all."""
    _prefill([0, 200, 129], [300, 257, 64], 1, g, bs, 64, window, window=window, alibi=True)


@pytest.mark.parametrize("prefix", [[1, 1], [128, 64], [300, 299], [10 ** 6, 257], [-4, 0]])
@pytest.mark.parametrize("window", [0, 50, 200])
def test_prefill_prefix_edges(prefix, window):
    _prefill([0, 100], [300, 200], 2, 2, 16, 64, 7, prefix=prefix, window=window, softcap=15.0, alibi=True)


@pytest.mark.parametrize("softcap,q_factor", [(0.5, 2.0), (5.0, 2.0), (50.0, 0.1), (50.0, 60.0)])
def test_prefill_cap_of_any_size(softcap, q_factor):
    """Both ways of computing tanh, and tiles that differ in it."""
    _prefill([100, 0], [130, 70], 2, 4, 32, 128, 8, softcap=softcap, q_factor=q_factor)


@pytest.mark.parametrize("kw", [dict(softcap=50.0, window=1024), dict(alibi=True, prefix=[200, 900]), dict(window=300, alibi=True)])
def test_prefill_large(kw):
    _prefill([3584, 700], [512, 2048], 2, 4, 16, 128, 9, rows=12, **kw)


def test_prefill_does_not_depend_on_what_lies_in_masked_places():
    """The same call before and after calls that leave very large K and V in shared memory, and with other
    garbage in the slots that hold no token: the same bits, whichever way tanh is computed."""
    kw = dict(softcap=8.0, window=50, q_factor=0.7, rows=4)
    lens = ([130, 77, 300], [70, 130, 20])
    first = _prefill(*lens, 2, 4, 16, 128, 15, **kw)
    gen = _gen(16)
    big = (torch.randn((64, 2, 16, 128), generator=gen) * 1e4).to(torch.bfloat16).to(DEV)
    q = (torch.randn((2000, 8, 128), generator=gen) * 1e4).to(torch.bfloat16).to(DEV)
    tab = torch.arange(64, dtype=torch.int32, device=DEV).view(1, 64).repeat(16, 1)
    start = torch.arange(0, 2001, 125, dtype=torch.int32, device=DEV)
    for _ in range(3):
        pa.pa_prefill_scoremod(torch.empty_like(q), q, big, big, tab, start, torch.full((16,), 1000, dtype=torch.int32, device=DEV),
                               125, pa.make_prefill_workspace(), softcap=8.0)
        assert torch.equal(first, _prefill(*lens, 2, 4, 16, 128, 15, **kw))


@pytest.mark.parametrize("bs", [16, 32, 64])
@pytest.mark.parametrize("kw", [dict(window=50), dict(), dict(alibi=True, prefix=True, window=90)], ids=str)
def test_prefill_bits_do_not_depend_on_free_slots(bs, kw):
    """Whatever an earlier owner left in slots without a token, behind the contexts and before the window: NaN, small
    or large numbers, the output's bits are the same."""
    gen, d, h, g = _gen(26), 128, 2, 4
    cached, chunk = [130, 77, 300, 0], [70, 130, 20, 33]
    lens = [a + b for a, b in zip(cached, chunk)]
    k, v, tab, full = _pool(lens, h, bs, d, gen, kw.get("window", 0), chunk)
    start = torch.zeros(5, dtype=torch.int32)
    start[1:] = torch.cumsum(torch.tensor(chunk), 0)
    q = torch.randn((sum(chunk), h * g, d), generator=gen).to(torch.bfloat16)
    slopes = _slopes(h * g).to(DEV) if "alibi" in kw else None
    prefix = torch.tensor([140, 0, 310, 9], dtype=torch.int32, device=DEV) if "prefix" in kw else None
    ctx = torch.tensor(lens, dtype=torch.int32)
    outs = []
    for fill in (None, 0.0, 1.0, 1e4, 1e30):
        kf, vf = (x if fill is None else torch.where(torch.isnan(x), (fill * torch.randn(x.shape, generator=gen)).to(x.dtype), x)
                  for x in (k, v))
        out = torch.empty_like(q, device=DEV)
        pa.pa_prefill_scoremod(out, q.to(DEV), kf.to(DEV), vf.to(DEV), tab.to(DEV), start.to(DEV), ctx.to(DEV), max(chunk),
                               pa.make_prefill_workspace(), softcap=30.0, alibi_slopes=slopes, window=kw.get("window", 0),
                               prefix_lens=prefix)
        outs.append(out)
    assert torch.isfinite(outs[0]).all() and pa.pa_device_errors() == 0
    for out in outs[1:]:
        assert torch.equal(outs[0], out)


def test_prefill_more_sequences_than_the_claim_order_keeps():
    n = 1100
    _prefill([(i * 5) % 40 for i in range(n)], [(i * 3) % 4 for i in range(n)], 1, 1, 16, 64, 10, window=20, softcap=10.0)


def test_prefill_without_any_is_prefill():
    gen = _gen(11)
    k, v, tab, _ = _pool([400, 77], 2, 16, 128, gen)
    q = torch.randn((150, 8, 128), generator=gen).to(torch.bfloat16)
    start = torch.tensor([0, 100, 150], dtype=torch.int32)
    args = [t.to(DEV) for t in (q, k, v, tab, start, torch.tensor([400, 77], dtype=torch.int32))]
    a, b = torch.empty_like(args[0]), torch.empty_like(args[0])
    ws = pa.make_prefill_workspace()
    pa.pa_prefill_scoremod(a, *args, 100, ws)
    pa.pa_prefill_ws(b, *args, 100, ws)
    assert (a.float() - b.float()).abs().max() <= 2.0 ** -7 * b.float().abs().max()


def test_prefill_errors_and_graph():
    gen = _gen(12)
    k, v, tab, _ = _pool([400, 77], 2, 16, 128, gen)
    q = torch.randn((150, 8, 128), generator=gen).to(torch.bfloat16)
    start = torch.tensor([0, 100, 150], dtype=torch.int32)
    args = [t.to(DEV) for t in (q, k, v, tab, start, torch.tensor([400, 77], dtype=torch.int32))]
    ws = pa.make_prefill_workspace()
    good, out = torch.empty_like(args[0]), torch.empty_like(args[0])
    kw = dict(softcap=20.0, window=64, prefix_lens=torch.tensor([5, 70], dtype=torch.int32, device=DEV))
    pa.pa_prefill_scoremod(good, *args, 100, ws, **kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_prefill_scoremod(out, *args, 100, ws, **kw)
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, good)
    bad = args[3].clone()
    bad[0, 24] = 10 ** 6                                              # the last block of sequence 0
    pa.pa_device_errors(clear=True)
    pa.pa_prefill_scoremod(out, args[0], args[1], args[2], bad, *args[4:], 100, ws, **kw)
    assert pa.pa_device_errors() == pa.PA_DEVERR_BAD_BLOCK and bool(torch.isnan(out[99]).all())
    assert int(ws.count_nonzero()) == 0
    with pytest.raises(ValueError):
        pa.pa_prefill_scoremod(out, *args, 100, ws, prefix_lens=torch.zeros(3, dtype=torch.int32, device=DEV))


def test_a_prompt_in_chunks_then_tokens():
    """A prompt in three chunks and a few decode steps of a windowed, capped layer, blocks given back to the
    allocator's pool once they lie before the window; the same rows as in one piece."""
    gen, d, bs, h, g, window = _gen(13), 64, 16, 2, 4, 48
    alloc = pa.BlockAllocator(16, bs, seed=2)
    seq = alloc.new_seq()
    kc = torch.full((16, h, bs, d), math.nan, dtype=torch.bfloat16, device=DEV)
    vc = kc.clone()
    ws, rows = pa.make_prefill_workspace(), []
    q_all = []
    for n in (70, 33, 50, 1, 1, 1):
        slots, _ = alloc.append_n(seq, n)
        k, v = (torch.randn((n, h, d), generator=gen).to(torch.bfloat16) for _ in "kv")
        rows += list(zip(k, v))
        pa.pa_reshape_and_cache(k.to(DEV), v.to(DEV), kc, vc, torch.tensor(slots, device=DEV))
        tab, ctx = alloc.block_table([seq], 16)
        total = int(ctx[0])
        first = max(0, total - n - window + 1)
        dead = tab[0, :first // bs].long()
        kc[dead.to(DEV)], vc[dead.to(DEV)] = math.nan, math.nan          # whatever their next owner writes
        tab[0, :first // bs] = -1
        q = torch.randn((n, h * g, d), generator=gen).to(torch.bfloat16)
        out = torch.empty_like(q, device=DEV)
        if n > 1:
            pa.pa_prefill_scoremod(out, q.to(DEV), kc, vc, tab.to(DEV), torch.tensor([0, n], dtype=torch.int32, device=DEV),
                                   ctx.to(DEV), n, ws, softcap=25.0, window=window)
        else:
            pa.pa_decode_scoremod(out, q.to(DEV), kc, vc, tab.to(DEV), ctx.to(DEV), total, softcap=25.0, window=window)
        rk, rv = (torch.stack([r[j] for r in rows]).double().transpose(0, 1) for j in (0, 1))
        o, mag, _ = ref.attend(q, rk, rv, torch.arange(total - n, total), 1 / math.sqrt(d), 25.0, None, window)
        ref.check_rows(out, o, mag, 8, "%d tokens" % total, _logit_error(q, rk, 1 / math.sqrt(d), 25.0, None, d))
    assert pa.pa_device_errors() == 0
