"""The 8-bit cache with a scale for each (block, KV head): the write is bit for bit what its definition in 64
bits says, the decode agrees with attention over code * scale, and the two run together."""
import math

import pytest
import torch

import fp64lib as ref
import paged_kv_cache_428_b200 as pa

pytestmark = pytest.mark.gpu
DEV = "cuda"
KINDS = ["e4m3", "int8"]
UNUSED = {"e4m3": 0x7F, "int8": 0x80}          # codes that no write produces


def _gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def _rows(n, h, d, g, spread=0.7):
    return (torch.randn((n, h, d), generator=g) * torch.exp(spread * torch.randn((n, h, 1), generator=g))).to(torch.bfloat16)


class Cache:
    """A pair of pools on the GPU beside their 64-bit counterparts."""

    def __init__(self, nb, h, bs, d, kind):
        self.kind, self.bs = kind, bs
        make = lambda: torch.full((nb, h, bs, d), UNUSED[kind], dtype=torch.uint8, device=DEV).view(ref.DTYPE[kind])  # noqa: E731
        self.k, self.v = make(), make()
        self.ks, self.vs = pa.make_block_scales(nb, h)
        self.ks.fill_(9.0)                      # leftovers of earlier owners
        self.vs.fill_(0.001)
        self.rk, self.rv, self.rks, self.rvs = (t.cpu().double() for t in (self.k, self.v, self.ks, self.vs))

    def write(self, key, value, slots, **kw):
        sl = torch.tensor(slots, dtype=torch.int64)
        pa.pa_reshape_and_cache_block_scales(key.to(DEV) if not key.is_cuda else key, value.to(DEV) if not value.is_cuda else value,
                                             self.k, self.v, self.ks, self.vs, sl.to(DEV), **kw)
        ref.write_block_scales(key.cpu().double(), self.rk, self.rks, slots, self.kind)
        ref.write_block_scales(value.cpu().double(), self.rv, self.rvs, slots, self.kind)

    def check(self):
        torch.cuda.synchronize()
        for got, want in ((self.k, self.rk), (self.v, self.rv), (self.ks, self.rks), (self.vs, self.rvs)):
            assert torch.equal(got.cpu().double().nan_to_num(nan=777.0), want.nan_to_num(nan=777.0))


def _slots(table, start, n, bs):
    return [table[t // bs] * bs + t % bs for t in range(start, start + n)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bs", [16, 32, 64])
def test_write_every_variant(kind, d, bs):
    """Ragged prompts, then appends whose scale grows, shrinks or stays, then a second chunk."""
    g, h, nb = _gen(d + bs), 3, 24
    c = Cache(nb, h, bs, d, kind)
    order = torch.randperm(nb, generator=g).tolist()
    tables = [order[0:8], order[8:16], order[16:24]]
    lens = [2 * bs + 5, 1, bs]
    slots = [s for tab, n in zip(tables, lens) for s in _slots(tab, 0, n, bs)]
    c.write(_rows(len(slots), h, d, g), _rows(len(slots), h, d, g), slots)
    c.check()
    for step in range(5):
        slots = [_slots(tab, n, 1, bs)[0] for tab, n in zip(tables, lens)]
        lens = [n + 1 for n in lens]
        f = 4.0 ** (step - 2)
        c.write(_rows(3, h, d, g) * f, _rows(3, h, d, g) / f, slots)
    c.check()
    more = [3, 2 * bs + 1, bs - 1]
    slots = [s for tab, n, m in zip(tables, lens, more) for s in _slots(tab, n, m, bs)]
    c.write(_rows(len(slots), h, d, g), _rows(len(slots), h, d, g), slots)
    c.check()
    assert pa.pa_device_errors() == 0


@pytest.mark.parametrize("kind", KINDS)
def test_write_many_tokens(kind):
    """Enough tokens for the launch shape of prompts: runs that cross the CTAs' borders, 5 heads."""
    g, h, d, bs, nb = _gen(9), 5, 64, 32, 40
    c = Cache(nb, h, bs, d, kind)
    order = torch.randperm(nb, generator=g).tolist()
    first = [s for i, n in enumerate((7, 0, 31)) for s in _slots(order[13 * i:13 * i + 13], 0, n, bs)]
    c.write(_rows(len(first), h, d, g), _rows(len(first), h, d, g), first)
    slots = [s for i, (a, n) in enumerate(((7, 300), (0, 333), (31, 290))) for s in _slots(order[13 * i:13 * i + 13], a, n, bs)]
    assert len(slots) > 512
    c.write(_rows(len(slots), h, d, g, 1.5), _rows(len(slots), h, d, g, 1.5), slots)
    c.check()


def _write_all_heads(rows, cache, scales, slots, kind):
    """ref.write_block_scales with all heads of a block at once (each slot once, finite values)."""
    bs = cache.shape[2]
    blocks = {}
    for t, s in enumerate(slots):
        blocks.setdefault(s // bs, []).append((s % bs, t))
    for b, pairs in blocks.items():
        off, t = (torch.tensor(x) for x in zip(*pairs))
        first = int(off.min())
        want = rows[t].abs().amax((0, 2)) / ref.QMAX[kind]
        unit = 2.0 ** (torch.floor(torch.log2(want)) - 7)
        old = scales[b] if first else torch.zeros_like(want)
        now = torch.maximum(old, torch.ceil(want / unit) * unit)
        grew = (now > old)[:, None, None]
        again = ref.encode(cache[b, :, :first] * (old / now)[:, None, None], 1.0, kind)
        cache[b, :, :first] = torch.where(grew, again, cache[b, :, :first])
        cache[b][:, off] = ref.encode(rows[t] / now[:, None], 1.0, kind).transpose(0, 1)
        scales[b] = now


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("seqs,h,bs,d", [(600, 1, 16, 64), (600, 3, 64, 128), (600, 16, 16, 64),
                                           (900, 12, 32, 128), (1100, 16, 64, 64), (4096, 19, 16, 64)])
def test_write_many_short_runs(kind, seqs, h, bs, d):
    """The append of a large batch, one token for most sequences and prompts of up to five blocks for some, in
    between: every number of tokens that a CTA looks after, CTAs with long runs, with short ones and with both."""
    g, nb = _gen(seqs), seqs + 300
    c = Cache(nb, h, bs, d, kind)
    order = torch.randperm(nb, generator=g).tolist()
    fill = torch.randint(0, 100, (nb, h, bs, d), generator=g).to(torch.int8)
    fill = fill if kind == "int8" else fill.float().to(torch.float8_e4m3fn)
    for got, want in ((c.k, c.rk), (c.v, c.rv)):
        got.copy_(fill)
        want.copy_(fill.double())
    scale = 2.0 ** torch.randint(-12, -4, (nb, h), generator=g).float()
    for t in (c.ks, c.vs, c.rks, c.rvs):
        t.copy_(scale)
    slots, at = [], 0
    for s in range(seqs):
        n = int(torch.randint(2, 5 * bs, (1,), generator=g)) if s % 31 == 7 and s < 900 else 1
        blocks = 1 if n == 1 else -(-n // bs)
        tab, at = order[at:at + blocks], at + blocks
        slots += _slots(tab, 0, n, bs) if n > 1 else [tab[0] * bs + int(torch.randint(0, bs, (1,), generator=g))]
    key, value = _rows(len(slots), h, d, g), _rows(len(slots), h, d, g)
    pa.pa_reshape_and_cache_block_scales(key.to(DEV), value.to(DEV), c.k, c.v, c.ks, c.vs, torch.tensor(slots, device=DEV))
    _write_all_heads(key.double(), c.rk, c.rks, slots, kind)
    _write_all_heads(value.double(), c.rv, c.rvs, slots, kind)
    c.check()
    assert pa.pa_device_errors() == 0


@pytest.mark.parametrize("kind", KINDS)
def test_write_values_where_it_can_go_wrong(kind):
    g, h, d, bs = _gen(3), 2, 64, 16
    c = Cache(6, h, bs, d, kind)
    k = _rows(20, h, d, g)
    k[0] = 0.0                                   # a block whose first row is all zero
    k[3, 0, 5], k[3, 1, 7], k[4, 0, 0] = math.inf, -math.inf, math.nan
    k[6] = 2.0 ** -130                           # subnormal in fp32
    k[7, 0] = 3.3e38
    k[8] = k[9] / 2                              # exact halves: ties
    v = torch.zeros_like(k)                      # a cache of zeros: scale 0
    v[18] = torch.tensor([1.0, -1.0]).repeat(d // 2)
    slots = [0] + list(range(17, 30)) + [-1, 33, 32, 5 * bs + 2, 48, -7]
    c.write(k, v, slots)
    c.check()
    c.write(k[:1] * 0 + 1e-20, k[:1] * 0, [1])   # a tiny row after a zero block
    c.write(k[:1] * 0 + 5, k[10:11], [2])
    c.write(k[11:12] * 100, k[12:13], [30])
    c.check()


@pytest.mark.parametrize("kind", KINDS)
def test_tiny_values_beside_ordinary_ones(kind):
    """Blocks of values near and below the floor of the scales, alone and beside blocks of ordinary ones: written as
    defined, and the attention over both is that over code * scale."""
    g, h, d, bs = _gen(13), 2, 64, 16
    c = Cache(12, h, bs, d, kind)
    order = [3, 7, 1, 9, 0, 5]
    k, v = _rows(96, h, d, g), _rows(96, h, d, g)
    for b, f in ((1, 2.0 ** -90), (3, 2.0 ** -120), (4, 2.0 ** -70)):
        v[16 * b:16 * b + 16] *= f
    k[32:48] *= 2.0 ** -100
    c.write(k, v, _slots(order, 0, 96, bs))
    c.check()
    q = (torch.randn((3, 4 * h, d), generator=g) * 0.5).to(torch.bfloat16)
    tab = torch.full((3, 6), -1, dtype=torch.int32)
    tab[0] = torch.tensor(order, dtype=torch.int32)
    tab[1, :2] = torch.tensor([order[1], order[3]], dtype=torch.int32)       # tiny ones only
    tab[2, :1] = order[4]
    case = (q, (c.k.cpu(), c.v.cpu()), (c.ks.cpu(), c.vs.cpu()), tab, torch.tensor([96, 32, 10], dtype=torch.int32))
    _check(case, _run(case))


@pytest.mark.parametrize("kind", KINDS)
def test_write_ratios_that_are_ties(kind):
    """Scales that grow by simple ratios: requantised codes fall on ties of the rounding."""
    h, d, bs = 1, 128, 16
    c = Cache(8, h, bs, d, kind)
    base = torch.arange(-64, 64).to(torch.bfloat16).view(1, 1, d)
    for b, f in enumerate((1.0, 4.0 / 3.0, 1.5, 2.0, 3.0, 4.0, 127.0, 1.0078125)):
        x = base.clone()
        x[..., 0] = -127.0
        c.write(x, x, [b * bs])
        y = torch.full((1, 1, d), 127.0 * f).to(torch.bfloat16)
        c.write(y, -y, [b * bs + 1])
    c.check()


@pytest.mark.parametrize("n", [40, 700])
def test_write_slots_given_twice_and_bad_slots(n):
    """Of tokens with one slot the last counts (also where the run is longer than a block); slots outside the
    pool are reported and skipped, rows that are not written stay."""
    g, h, d, bs = _gen(4), 2, 64, 16
    c = Cache(64, h, bs, d, "int8")
    slots = [16 * (i // 25 % 60) + (7 * i) % 13 for i in range(n)]
    pa.pa_device_errors(clear=True)
    c.write(_rows(n, h, d, g), _rows(n, h, d, g), slots)
    c.check()
    assert pa.pa_device_errors() == 0
    c.write(_rows(3, h, d, g), _rows(3, h, d, g), [64 * bs, 61 * bs, 1 << 40])
    c.check()
    assert pa.pa_device_errors() == pa.PA_DEVERR_BAD_SLOT


def test_write_strided_rows_and_no_rows():
    g, h, d, bs = _gen(5), 2, 64, 16
    c = Cache(4, h, bs, d, "e4m3")
    qkv = torch.randn((20, 4 * h, d), generator=g).to(torch.bfloat16).to(DEV)
    c.write(qkv[:, h:2 * h], qkv[:, 3 * h:], list(range(20)))
    c.write(qkv[:0, :h], qkv[:0, :h], [])
    c.write(qkv[3:4, :h].as_strided((1, h, d), (1, d, 1), qkv.storage_offset()), qkv[4:5, h:2 * h], [33])   # one row: any stride
    c.check()
    with pytest.raises(ValueError):              # rows on top of each other: a stride of 0 would mean packed rows
        c.write(qkv[:1, :h].expand(3, h, d), qkv[:3, :h].contiguous(), [0, 1, 2])


def test_copy_scales_with_the_blocks():
    c = [Cache(6, 3, 16, 64, "int8") for _ in range(3)]
    for i, x in enumerate(c):
        x.ks.copy_(torch.arange(18.0, device=DEV).view(6, 3) + 100 * i)
        x.vs.copy_(-x.ks)
    want = [(x.ks.clone(), x.vs.clone()) for x in c]
    pairs = torch.tensor([[0, 4], [2, 5], [9, 1], [1, -1]], device=DEV)
    pa.pa_device_errors(clear=True)
    pa.pa_copy_block_scales([x.ks for x in c], [x.vs for x in c], pairs)
    assert pa.pa_device_errors() == pa.PA_DEVERR_BAD_PAIR
    for x, (k, v) in zip(c, want):
        for t, w in ((x.ks, k), (x.vs, v)):
            w[4], w[5] = w[0].clone(), w[2].clone()
            assert torch.equal(t, w)


# ------------------------------------------------------------------------------------------ decode
def _decode_case(kind, d, bs, g, lens, seed=0, h_kv=2, spread=1.0, q_factor=2.0):
    gen = _gen(seed)
    need = [-(-n // bs) for n in lens]
    nb = sum(need) + 3
    order = torch.randperm(nb, generator=gen).tolist()
    tab = torch.full((len(lens), max(need + [1]) + 1), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(need):
        tab[s, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    if kind == "int8":
        codes = [torch.randint(-127, 128, (nb, h_kv, bs, d), generator=gen, dtype=torch.int16).to(torch.int8) for _ in "kv"]
    else:
        codes = [(torch.randn((nb, h_kv, bs, d), generator=gen) * 60).clamp(-448, 448).to(torch.float8_e4m3fn) for _ in "kv"]
    # rows past each context, and blocks of nobody: codes that no write produces
    for s, n in enumerate(lens):
        if n % bs:
            for c in codes:
                c[tab[s, n // bs], :, n % bs:].view(torch.uint8).fill_(UNUSED[kind])
    for b in order[at:]:
        for c in codes:
            c[b].view(torch.uint8).fill_(UNUSED[kind])
    scales = [torch.exp(spread * torch.randn((nb, h_kv), generator=gen)) * 0.01 for _ in "kv"]
    q = (torch.randn((len(lens), h_kv * g, d), generator=gen) * q_factor).to(torch.bfloat16)
    return q, codes, scales, tab, torch.tensor(lens, dtype=torch.int32)


def _run(case, max_len=None, workspace=None, out=None, stream=None):
    q, (k, v), (ks, vs), tab, ctx = case
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device=DEV) if out is None else out
    pa.pa_decode_block_scales(out, q.to(DEV), k.to(DEV), v.to(DEV), ks.to(DEV), vs.to(DEV), tab.to(DEV), ctx.to(DEV),
                              int(ctx.max()) if max_len is None else max_len, workspace=workspace, stream=stream)
    torch.cuda.synchronize()
    return out


def _check(case, out, skip=(), what=""):
    q, (k, v), (ks, vs), tab, ctx = case
    for s in range(q.shape[0]):
        n = int(ctx[s])
        if s in skip:
            continue
        if n == 0:
            assert not out[s].any()
            continue
        rk, rv = ref.rows_of(k, tab[s], n, ks), ref.rows_of(v, tab[s], n, vs)
        o, mag, w = ref.attend(q[s:s + 1], rk, rv, torch.tensor([n - 1]), 1 / math.sqrt(q.shape[2]))
        # fp16 steps of the probabilities: half a step relative to each down to 2^-14 where the largest
        # p * scale stands at 2^15, below that an absolute 2^-25, which is 2^-40 of the largest
        g = q.shape[1] // rk.shape[0]
        each = ref.rows_of(torch.ones_like(v, dtype=torch.float32), tab[s], n, vs)[:, :, 0].repeat_interleave(g, 0)
        code = ref.rows_of(v, tab[s], n).abs().sum(1).repeat_interleave(g, 0)
        extra = 2.0 ** -40 * (w[0] * each).amax(1)[:, None] * code
        ref.check_rows(out[s:s + 1], o, mag, 11, "%s sequence %d of %d tokens" % (what, s, n), extra=extra)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bs", [16, 32, 64])
@pytest.mark.parametrize("g", [1, 2, 4, 8])
def test_decode_every_variant(kind, d, bs, g):
    case = _decode_case(kind, d, bs, g, [1, 0, bs, bs + 1, 3 * bs - 1, 333, 17], seed=d + bs + g)
    _check(case, _run(case))
    assert pa.pa_device_errors() == 0


@pytest.mark.parametrize("kind", KINDS)
def test_decode_scales_far_apart(kind):
    """Block scales over 2^40, some of them 0 (their codes are then 0): no block drowns another's share."""
    case = _decode_case(kind, 128, 16, 4, [400, 90], seed=11, spread=0.0)
    q, codes, scales, tab, ctx = case
    g = _gen(12)
    scales[1].copy_(0.01 * 2.0 ** torch.randint(-20, 21, scales[1].shape, generator=g))
    scales[0].copy_(0.002 * 2.0 ** torch.randint(-3, 2, scales[0].shape, generator=g))
    for i in (0, 1):
        zero = torch.rand(scales[i].shape, generator=g) < 0.1
        scales[i][zero] = 0.0
        codes[i].view(torch.uint8)[zero] = 0
    # where one block outweighs all by 2^20 the others' outputs are below its rounding: also look at each alone
    _check(case, _run(case))
    small = 2.0 ** -30
    scales[1].fill_(small)
    _check(case, _run(case))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("power", [-20, -34, -44, -60, -80])
def test_decode_zero_blocks_beside_small_scales(kind, power):
    """Blocks with V scale 0 (all their rows were 0) beside blocks whose V scales are as small as the write leaves
    them: the others' share of the output keeps its digits, a sequence of nothing else gives 0."""
    q, codes, scales, tab, ctx = _decode_case(kind, 128, 16, 4, [400, 90, 40], seed=31, spread=0.0)
    scales[0].fill_(0.002)
    scales[1].fill_(2.0 ** power)
    zero = torch.cat([tab[0, 1:25:3], tab[1, 2:4], tab[2, :3]]).long()
    scales[1][zero] = 0.0
    codes[1].view(torch.uint8)[zero] = 0
    case = (q, codes, scales, tab, ctx)
    out = _run(case)
    _check(case, out)
    assert not out[2].any()


@pytest.mark.parametrize("kind", KINDS)
def test_zero_rows_written_beside_tiny_ones(kind):
    """The same through the write: a block of zero V rows, then blocks of tiny ones."""
    g, h, d, bs = _gen(32), 2, 64, 16
    c = Cache(9, h, bs, d, kind)
    order = [3, 1, 5, 0, 8, 2, 7]
    k, v = _rows(112, h, d, g), _rows(112, h, d, g) * 2.0 ** -45
    v[:16] = 0
    c.write(k, v, _slots(order, 0, 112, bs))
    c.check()
    q = (torch.randn((1, 4 * h, d), generator=g) * 0.5).to(torch.bfloat16)
    case = (q, (c.k.cpu(), c.v.cpu()), (c.ks.cpu(), c.vs.cpu()), torch.tensor([order], dtype=torch.int32),
            torch.tensor([105], dtype=torch.int32))
    _check(case, _run(case))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("power", [-60, -20, 40])
def test_decode_queries_of_any_size(kind, power):
    """Tiny queries over large keys and the other way round: the logits are ordinary."""
    q, codes, scales, tab, ctx = _decode_case(kind, 64, 16, 4, [90, 17], seed=21, spread=0.3)
    q = (q.float() * 2.0 ** power).to(torch.bfloat16)
    q[:, 1] = 0.0
    scales[0] *= 2.0 ** -power
    _check((q, codes, scales, tab, ctx), _run((q, codes, scales, tab, ctx)))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("lens,h_kv,g,d,bs", [
    ([70001], 1, 4, 64, 16),                    # one group, as many pieces as there can be
    ([33000, 5], 2, 1, 128, 64),
    ([(i * 37) % 90 for i in range(300)], 1, 2, 64, 16),    # many short ones, several groups a CTA
    ([4096] * 3 + [1] * 20, 4, 1, 128, 32)])
def test_decode_long_and_many(kind, lens, h_kv, g, d, bs):
    case = _decode_case(kind, d, bs, g, lens, seed=5, h_kv=h_kv, q_factor=1.0)
    out = _run(case)
    _check(case, out)
    # a bound that is too low costs speed only
    assert torch.equal(_run(case, max_len=1), _run(case, max_len=1))
    _check(case, _run(case, max_len=1))


def test_decode_bad_blocks_and_short_tables():
    case = _decode_case("int8", 64, 16, 2, [100, 100, 100, 100], seed=6)
    q, codes, scales, tab, ctx = case
    good = _run(case)
    _check(case, good)
    bad = tab.clone()
    bad[1, 3], bad[2, 0] = codes[0].shape[0], -5
    pa.pa_device_errors(clear=True)
    out = _run((q, codes, scales, bad, ctx))
    assert pa.pa_device_errors() == pa.PA_DEVERR_BAD_BLOCK
    assert torch.isnan(out[1]).all() and torch.isnan(out[2]).all()
    assert torch.equal(out[0], good[0]) and torch.equal(out[3], good[3])
    # a context longer than its table's row
    long = ctx.clone()
    long[3] = 10 ** 6
    out = _run((q, codes, scales, tab[:, :7].contiguous(), long), max_len=100)
    assert pa.pa_device_errors() == pa.PA_DEVERR_BAD_BLOCK
    assert torch.isnan(out[3]).all() and torch.equal(out[0], good[0])
    neg = ctx.clone()
    neg[0] = -3
    assert not _run((q, codes, scales, tab, neg))[0].any()
    assert pa.pa_device_errors() == 0


def test_decode_workspace_of_many_shapes_streams_and_graphs():
    """One workspace for calls of different shapes, on another stream, captured and replayed; it ends as it
    began.  Sequences are in no fixed number of pieces: every call leaves its counters at zero."""
    ws = torch.zeros(16 << 20, dtype=torch.uint8, device=DEV)
    cases = [_decode_case("e4m3", 64, 16, 2, [900, 3, 77], 1), _decode_case("int8", 128, 32, 8, [5000], 2, h_kv=1),
             _decode_case("e4m3", 128, 16, 1, [300] * 40, 3), _decode_case("int8", 64, 64, 4, [64, 65], 4)]
    first = [_run(c, workspace=ws) for c in cases]
    for c, o in zip(cases, first):
        _check(c, o)
        assert torch.equal(o, _run(c, workspace=ws)) and torch.equal(o, _run(c))
    assert int(ws[:65536 * 4].count_nonzero()) == 0
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        assert torch.equal(first[0], _run(cases[0], workspace=ws))
    assert torch.equal(first[1], _run(cases[1], workspace=ws, stream=side))
    args = [[t.to(DEV) if isinstance(t, torch.Tensor) else [x.to(DEV) for x in t] for t in c] for c in cases[:2]]
    outs = [torch.zeros_like(a[0]) for a in args]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for a, o in zip(args, outs):
            pa.pa_decode_block_scales(o, a[0], a[1][0], a[1][1], a[2][0], a[2][1], a[3], a[4], 5000, workspace=ws)
    for _ in range(3):
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, f) for o, f in zip(outs, first))


def test_a_chat_from_prompt_to_fork():
    """Prompt write, decode steps, a fork whose first append copies a block and its scales, all through the
    allocator: after every step the attention is that over code * scale of the 64-bit model."""
    g, h, grp, d, bs, nb = _gen(8), 2, 4, 64, 16, 32
    alloc = pa.BlockAllocator(nb, bs, seed=3)
    c = Cache(nb, h, bs, d, "int8")
    seq = alloc.new_seq()
    slots, _ = alloc.append_n(seq, 41)
    assert pa.pa_validate_block_runs(torch.tensor(slots), bs, nb) == 0
    c.write(_rows(41, h, d, g), _rows(41, h, d, g), slots)
    seqs = [seq, alloc.fork(seq)]
    ws = torch.zeros(pa.pa_decode_block_scales_workspace_size(2, h * grp, h, d, 64), dtype=torch.uint8, device=DEV)
    for step in range(12):
        slots, cow = alloc.append_batch(seqs)
        if cow:
            pairs = torch.tensor(cow, dtype=torch.int64, device=DEV)
            pa.pa_copy_blocks([c.k], [c.v], pairs)
            pa.pa_copy_block_scales([c.ks], [c.vs], pairs)
            for a, b in cow:
                for t in (c.rk, c.rv, c.rks, c.rvs):
                    t[b] = t[a]
        c.write(_rows(2, h, d, g), _rows(2, h, d, g), slots)
        tab, ctx = alloc.block_table(seqs, 4)
        q = torch.randn((2, h * grp, d), generator=g).to(torch.bfloat16)
        out = torch.empty_like(q, device=DEV)
        pa.pa_decode_block_scales(out, q.to(DEV), c.k, c.v, c.ks, c.vs, tab.to(DEV), ctx.to(DEV), 64, workspace=ws)
        c.check()
        _check((q, (c.rk, c.rv), (c.rks, c.rvs), tab, ctx), out, what="step %d" % step)
    assert pa.pa_device_errors() == 0


def test_tensors_of_another_place_are_refused():
    case = _decode_case("int8", 64, 16, 2, [10], seed=6)
    q, codes, scales, tab, ctx = case
    with pytest.raises(ValueError):
        pa.pa_decode_block_scales(torch.empty_like(q, device=DEV), q, codes[0].to(DEV), codes[1].to(DEV), scales[0].to(DEV),
                                  scales[1].to(DEV), tab.to(DEV), ctx.to(DEV), 10)
    with pytest.raises(ValueError):
        pa.pa_decode_block_scales(torch.empty_like(q, device=DEV), q.to(DEV), codes[0].to(DEV), codes[1].to(DEV),
                                  scales[0].to(DEV)[:-1], scales[1].to(DEV)[:-1], tab.to(DEV), ctx.to(DEV), 10)
