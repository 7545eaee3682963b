"""The operators measured on a B200: attention with modified scores, a cache in 8 bits with a scale for
each block and head, and eviction by accumulated attention weight.

All of them work on the library's paged cache: K and V are [num_blocks, h_kv, block_size, head_dim], a
block table maps a sequence's logical blocks to physical ones, and the slots that no sequence owns hold
NaN, so that any read of them shows up.  ``run`` is the plain form in elementary torch operations, or,
where ``own`` is true, the calls that a user of the library makes.
"""
import math

import torch

own = False

DEV = "cuda"
QMAX = {"e4m3": 448.0, "int8": 127.0}          # largest magnitude of a code


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of two short chats on a small model: the call's latency is what counts
        dict(name="decode_scoremod_tiny", op="decode_scoremod", B=2, lo=37, hi=81, h_q=4, h_kv=2, d=64, bs=16,
             softcap=30.0, alibi=False, window=64),
        # the 64-sequence serving step with capped scores and a bias that falls with the distance
        dict(name="decode_scoremod_b64", op="decode_scoremod", B=64, lo=512, hi=4096, h_q=32, h_kv=8, d=128, bs=16,
             softcap=50.0, alibi=True, window=0),
        # chunked prefill after cached prefixes in a layer with capped scores and a sliding window
        dict(name="prefill_scoremod_chunk512", op="prefill_scoremod", B=8, lo=0, hi=3584, qlo=512, qhi=512, h_q=32,
             h_kv=8, d=128, bs=16, softcap=50.0, alibi=False, window=1024, prefix=0),
        # whole prompts of ragged lengths whose first part is attended in both directions, distance bias
        dict(name="prefill_scoremod_prompt", op="prefill_scoremod", B=8, lo=0, hi=0, qlo=256, qhi=2048, h_q=32,
             h_kv=8, d=128, bs=16, softcap=0.0, alibi=True, window=0, prefix=200),
        # the append of a decode step: one token for each of 32 sequences, somewhere inside its last block
        dict(name="write_block_scales_step", op="write_block_scales", cache="e4m3", B=32, lo=40, hi=4096, qlo=1, qhi=1,
             h_kv=32, d=128, bs=16),
        # the prompts of a batch written at once, ragged, starting inside partly filled blocks
        dict(name="write_block_scales_prompt", op="write_block_scales", cache="int8", B=32, lo=0, hi=100, qlo=256,
             qhi=2048, h_kv=8, d=128, bs=64),
        # the 32-head decode step over an 8-bit cache of 4096 tokens a sequence
        dict(name="decode_block_scales_mha_b32", op="decode_block_scales", cache="e4m3", B=32, lo=4096, hi=4096,
             h_q=32, h_kv=32, d=128, bs=16),
        # three short ragged sequences, grouped heads of 64 dims
        dict(name="decode_block_scales_small", op="decode_block_scales", cache="int8", B=3, lo=1, hi=301, h_q=16,
             h_kv=2, d=64, bs=32),
        # one sequence of a chat whose cache is about to outgrow its budget
        dict(name="decode_weights_one", op="decode_weights", B=1, lo=1001, hi=1001, h_q=32, h_kv=8, d=128, bs=16),
        # the 64-sequence serving step that also keeps count of what every cached token is worth
        dict(name="decode_weights_b64", op="decode_weights", B=64, lo=512, hi=4096, h_q=32, h_kv=8, d=128, bs=16),
        # the batch brought down to 512 tokens a sequence, the last 64 of them kept in any case
        dict(name="evict_b64", op="evict", B=64, lo=512, hi=4096, h_kv=8, d=128, bs=16, budget=512, recent=64),
        # two long documents brought down to 8192 tokens
        dict(name="evict_long", op="evict", B=2, lo=32768, hi=131072, h_kv=8, d=128, bs=64, budget=8192, recent=256),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    """One more case of the listed ranges: any operator, heads, block size and head dim that the library takes."""
    most = {}
    for c in listed():
        w = work(c)
        most[c["op"]] = max(most.get(c["op"], 0.0), max(w["bytes"], w["flops"] / 50))
    op = rng.choice(sorted(most))
    d, bs = rng.choice([64, 128]), rng.choice([16, 32, 64])
    h_kv, g = rng.choice([1, 2, 4, 5, 8, 16]), rng.choice([1, 2, 4, 8])
    c = dict(op=op, B=_log_int(rng, 1, 64), h_kv=h_kv, d=d, bs=bs)
    if op in ("decode_scoremod", "prefill_scoremod"):
        c.update(h_q=h_kv * g, softcap=rng.choice([0.0, rng.uniform(5.0, 60.0)]), alibi=rng.random() < 0.5,
                 window=rng.choice([0, _log_int(rng, 1, 4096)]))
    if op == "decode_scoremod":
        c["hi"] = _log_int(rng, 2, 8192)
        c["lo"] = _log_int(rng, 1, c["hi"])
    elif op == "prefill_scoremod":
        c["hi"] = _log_int(rng, 1, 4096) - 1
        c["lo"] = rng.randint(0, c["hi"])
        c["qhi"] = _log_int(rng, 1, 2048)
        c["qlo"] = _log_int(rng, 1, c["qhi"])
        c["prefix"] = rng.choice([0, _log_int(rng, 1, 1024)])
        c["B"] = min(c["B"], 8)
    elif op == "write_block_scales":
        c.update(cache=rng.choice(["e4m3", "int8"]), lo=0, hi=_log_int(rng, 1, 4096), qhi=_log_int(rng, 1, 2048))
        c["qlo"] = _log_int(rng, 1, c["qhi"])
    elif op == "decode_block_scales":
        c.update(cache=rng.choice(["e4m3", "int8"]), h_q=h_kv * g, hi=_log_int(rng, 2, 8192))
        c["lo"] = _log_int(rng, 1, c["hi"])
    elif op == "decode_weights":
        c.update(h_q=h_kv * g, hi=_log_int(rng, 2, 8192))
        c["lo"] = _log_int(rng, 1, c["hi"])
    else:
        c["hi"] = _log_int(rng, 64, 32768)
        c["lo"] = _log_int(rng, 1, c["hi"])
        c["budget"] = _log_int(rng, 16, c["hi"])
        c["recent"] = rng.randint(0, c["budget"])

    def over():
        """More than the operator's largest listed case: work, size of the cache, or scores of the plain form."""
        w, n = work(c), c["hi"] + c.get("qhi", 0)
        scores = c["B"] * c["qhi"] * n * c["h_q"] if op == "prefill_scoremod" else 0
        return (max(w["bytes"], w["flops"] / 50) > most[op] or c["B"] * n * c["h_kv"] * d > 32 * 4096 * 32 * 128
                or scores > 8 * 2048 * 2048 * 32)

    while over() and c["B"] > 1:
        c["B"] = (c["B"] + 1) // 2
    while over() and c["h_kv"] > 1:
        c["h_kv"] //= 2
        if "h_q" in c:
            c["h_q"] = c["h_kv"] * g
    return c


def _spread(n, lo, hi, shift):
    """n lengths between lo and hi, spread evenly and out of order; the last one is hi."""
    got = [lo + int((hi - lo + 1) * ((0.5 + shift + i * 0.6180339887498949) % 1.0)) for i in range(n)]
    return [min(x, hi) for x in got[:-1]] + [hi]


def _lengths(case):
    """(tokens that the cache holds before the call, tokens that the call brings) of each sequence."""
    held = _spread(case["B"], case["lo"], case["hi"], 0.0)
    new = _spread(case["B"], case["qlo"], case["qhi"], 0.3) if "qlo" in case else [0] * case["B"]
    return held, new


def _prefixes(case):
    """Length of the part that is attended in both directions, for each sequence of a prefill."""
    return _spread(case["B"], case["prefix"] // 2, case["prefix"], 0.1)


def _allowed_pairs(case):
    """(query, key) pairs that the mask leaves, over the sequences of a prefill chunk."""
    held, new = _lengths(case)
    window, total = case["window"], 0
    for h, n, prefix in zip(held, new, _prefixes(case)):
        ctx = h + n
        for p in range(h, ctx):
            first = max(0, p - window + 1) if window else 0
            last = max(p, min(prefix, ctx) - 1)
            total += last - first + 1
    return total


def work(case):
    op, B, h_kv, d = case["op"], case["B"], case["h_kv"], case["d"]
    held, new = _lengths(case)
    blocks = lambda n: -(-n // case["bs"])  # noqa: E731
    if op in ("decode_scoremod", "decode_block_scales", "decode_weights"):
        window = case.get("window", 0)
        seen = [min(n, window) if window else n for n in held]
        elem = 2 if op != "decode_block_scales" else 1
        tokens = sum(seen)
        nbytes = 2 * tokens * h_kv * d * elem + 2 * B * case["h_q"] * d * 2 + 4 * sum(map(blocks, seen))
        if op == "decode_block_scales":
            nbytes += 2 * 4 * h_kv * sum(map(blocks, seen))
        if op == "decode_weights":
            nbytes += 2 * 4 * h_kv * tokens
        return {"bytes": nbytes, "flops": 4 * tokens * case["h_q"] * d}
    if op == "prefill_scoremod":
        window = case["window"]
        seen = [n + (min(h, window - 1) if window else h) for h, n in zip(held, new)]
        nbytes = 2 * sum(seen) * h_kv * d * 2 + 2 * sum(new) * case["h_q"] * d * 2 + 4 * sum(map(blocks, seen))
        return {"bytes": nbytes, "flops": 4 * _allowed_pairs(case) * case["h_q"] * d}
    if op == "write_block_scales":
        touched = sum(blocks(h + n) - h // case["bs"] for h, n in zip(held, new))
        return {"bytes": sum(new) * (h_kv * d * 2 * (2 + 1) + 8) + 2 * 2 * 4 * touched * h_kv,
                "flops": 4 * sum(new) * h_kv * d}
    kept = sum(min(n, case["budget"]) for n in held)
    return {"bytes": 4 * h_kv * sum(held) + 2 * 2 * kept * h_kv * d * 2 + 2 * 4 * h_kv * kept, "flops": h_kv * sum(held)}


# ----------------------------------------------------------------------------------------- inputs
def _tables(blocks, pool, gen):
    """Block tables [B, max] that hand shuffled physical blocks to the sequences; -1 past each row's end."""
    n = torch.tensor(blocks, device=DEV)
    order = torch.randperm(pool, generator=gen, device=DEV)
    width = max(1, max(blocks))
    col = torch.arange(width, device=DEV)
    start = torch.cumsum(n, 0) - n
    tab = order[(start[:, None] + col).clamp(max=pool - 1)]
    return torch.where(col < n[:, None], tab, -1).to(torch.int32).contiguous(), order[int(n.sum()):]


def _slots(tab, pos, row, bs):
    """Slot of token pos[i] of sequence row[i]."""
    return tab[row, pos // bs].long() * bs + pos % bs


def _ramp(lengths):
    """(sequence, place within it) of every token of sequences of these lengths."""
    n = torch.tensor(lengths, device=DEV)
    row = torch.repeat_interleave(torch.arange(len(lengths), device=DEV), n)
    return row, torch.arange(row.numel(), device=DEV) - (torch.cumsum(n, 0) - n)[row]


def _rand(shape, gen, factor=1.0):
    return (torch.randn(shape, generator=gen, device=DEV) * factor).to(torch.bfloat16)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op, B, h_kv, d, bs = case["op"], case["B"], case["h_kv"], case["d"], case["bs"]
    held, new = _lengths(case)
    ctx = [h + n for h, n in zip(held, new)]
    need = [-(-n // bs) for n in ctx]
    kept = [min(n, case["budget"]) for n in ctx] if op == "evict" else [0] * B
    after = [-(-n // bs) for n in kept]
    pool = int(1.05 * sum(need)) + sum(after) + 2
    tab, rest = _tables(need, pool, gen)
    st = dict(case=case, block_tables=tab, context_lens=torch.tensor(ctx, dtype=torch.int32, device=DEV),
              max_len=max(ctx), scale=1.0 / math.sqrt(d))

    def cache(held_lengths, factor=None):
        """A pool of bf16 rows, and the slots that hold no token: those are NaN."""
        rows = torch.empty((pool, h_kv, bs, d), dtype=torch.bfloat16, device=DEV)
        for i in range(0, pool, 4096):
            rows[i:i + 4096] = _rand((min(4096, pool - i), h_kv, bs, d), gen)
        free = torch.ones(pool * bs, dtype=torch.bool, device=DEV)
        row, pos = _ramp(held_lengths)
        free[_slots(tab, pos, row, bs)] = False
        free = free.view(pool, 1, bs, 1)
        return (rows if factor is None else rows.mul_(factor)).masked_fill_(free, float("nan")), free

    # a few channels of K are larger than the others, as in trained models; V rows vary in size
    channel = torch.where(torch.rand((h_kv, 1, d), generator=gen, device=DEV) < 0.03, 4.0, 1.0).to(torch.bfloat16)
    size = lambda n, m: torch.exp(0.5 * torch.randn((n, 1, m, 1), generator=gen, device=DEV)).to(torch.bfloat16)  # noqa: E731
    if op in ("decode_scoremod", "prefill_scoremod", "decode_weights"):
        rows = B if op != "prefill_scoremod" else sum(new)
        st.update(q=_rand((rows, case["h_q"], d), gen, 2.0), k_cache=cache(ctx)[0], v_cache=cache(ctx)[0])
        st["out"] = torch.zeros_like(st["q"])
        if case.get("alibi"):
            st["slopes"] = torch.exp2(-8.0 * torch.arange(1, case["h_q"] + 1, device=DEV) / case["h_q"]).float()
        if op == "prefill_scoremod":
            start = torch.zeros(B + 1, dtype=torch.int32, device=DEV)
            start[1:] = torch.cumsum(torch.tensor(new, device=DEV), 0)
            st.update(query_start=start, max_query=max(new))
            if case["prefix"]:
                st["prefix_lens"] = torch.tensor(_prefixes(case), dtype=torch.int32, device=DEV)
        if op == "decode_weights":
            st["weights"] = 0.1 * torch.rand((B, h_kv, max(ctx) + bs), generator=gen, device=DEV)
    elif op in ("write_block_scales", "decode_block_scales"):
        # the held rows are in the cache already, with the scales that their values called for; slots that
        # hold no token have a code that no write produces (NaN, -128)
        for name, factor in (("k", channel), ("v", size(pool, bs))):
            rows, free = cache(held, factor)
            rows = rows.float().nan_to_num_(0.0)
            scales = _scale_of(rows.abs().amax(dim=(2, 3)), case["cache"])
            code = _encode(rows, scales[:, :, None, None], case["cache"])
            code.view(torch.uint8).masked_fill_(free, 0x80 if case["cache"] == "int8" else 0x7F)
            st[name + "_cache"], st[name + "_scales"] = code, scales
        if op == "write_block_scales":
            row, pos = _ramp(new)
            pos = pos + torch.tensor(held, device=DEV)[row]
            st["slot_mapping"] = _slots(tab, pos, row, bs)
            st["key"] = _rand((row.numel(), h_kv, d), gen) * channel[:, 0]
            st["value"] = _rand((row.numel(), h_kv, d), gen) * size(row.numel(), 1)[:, 0]
        else:
            st["q"] = _rand((B, case["h_q"], d), gen, 2.0)
            st["out"] = torch.zeros_like(st["q"])
    else:
        st.update(k_cache=cache(ctx)[0], v_cache=cache(ctx)[0])
        # a few heavy tokens and a long tail, some of them equal: weights that attention has left behind
        w = torch.exp(2.0 * torch.randn((B, h_kv, max(ctx)), generator=gen, device=DEV))
        st["weights"] = torch.where(torch.rand(w.shape, generator=gen, device=DEV) < 0.2, w.round(), w)
        n = torch.tensor(after, device=DEV)
        col = torch.arange(max(1, max(after)), device=DEV)
        start = torch.cumsum(n, 0) - n
        st["new_tables"] = torch.where(col < n[:, None], rest[(start[:, None] + col).clamp(max=rest.numel() - 1)],
                                       -1).to(torch.int32).contiguous()
        st["kept"] = torch.zeros((B, h_kv, case["budget"]), dtype=torch.int32, device=DEV)
        st["new_weights"] = torch.zeros((B, h_kv, case["budget"] + bs), device=DEV)
        st["new_context_lens"] = torch.zeros(B, dtype=torch.int32, device=DEV)
    # scratch memory that a serving program keeps from step to step
    if op == "prefill_scoremod":
        st["workspace"] = torch.zeros(4096, dtype=torch.uint8, device=DEV)
    elif "h_q" in case:
        logits = case["h_q"] * B * (max(ctx) + 64) * 4 if op == "decode_weights" else 0
        st["workspace"] = torch.zeros(logits + (16 << 20), dtype=torch.uint8, device=DEV)
    return st


# ------------------------------------------------------------------------------------- plain forms
def _scale_of(amax, kind):
    """The smallest number of 8 significant bits (a bf16) that is not below amax / QMAX."""
    # divided by a tensor: by a plain number it would be a product with the rounded reciprocal
    bits = (amax.float() / torch.full_like(amax, QMAX[kind], dtype=torch.float32)).view(torch.int32)
    return torch.bitwise_and(bits + 0xFFFF, -65536).view(torch.float32)


def _encode(x, scale, kind):
    """Codes of x / scale, to nearest (ties to even); 0 where the scale is 0."""
    y = torch.where(scale > 0, x / scale, 0.0)
    y = y.clamp(-QMAX[kind], QMAX[kind])
    return y.round().to(torch.int8) if kind == "int8" else y.to(torch.float8_e4m3fn)


def _gather(cache, tab, length):
    """Rows of the first `length` places of every sequence, in 32 bits: [B, h_kv, length, d]."""
    B, h_kv, bs, d = tab.shape[0], cache.shape[1], cache.shape[2], cache.shape[3]
    rows = cache[tab.clamp(min=0).long()].float()
    return rows.permute(0, 2, 1, 3, 4).reshape(B, h_kv, -1, d)[:, :, :length]


def _weights_of(x, allowed):
    """Softmax over the last axis where `allowed`, 0 elsewhere (a row with nothing allowed is 0)."""
    x = torch.where(allowed, x, -math.inf)
    m = x.amax(-1, keepdim=True)
    e = torch.where(allowed, torch.exp(x - torch.where(m == -math.inf, 0.0, m)), 0.0)
    s = e.sum(-1, keepdim=True)
    return torch.where(s > 0, e / s, 0.0)


def _modify(x, case, slopes, distance):
    """Scores capped by a tanh, then a bias that falls with the distance.  slopes: [h_kv, G, 1, 1]."""
    if case.get("softcap"):
        x = case["softcap"] * torch.tanh(x / case["softcap"])
    return x if slopes is None else x - slopes * distance


def _plain_decode(st):
    case = st["case"]
    h_kv, n = case["h_kv"], st["max_len"]
    q = st["q"].float().view(case["B"], h_kv, -1, case["d"])
    pos = torch.arange(n, device=DEV)
    ctx = st["context_lens"].long()[:, None]
    allowed = pos < ctx
    if case.get("window"):
        allowed = allowed & (pos >= ctx - case["window"])
    k, v = _gather(st["k_cache"], st["block_tables"], n), _gather(st["v_cache"], st["block_tables"], n)
    if "k_scales" in st:
        at = st["block_tables"].clamp(min=0).long()
        each = lambda s: s[at].permute(0, 2, 1).repeat_interleave(case["bs"], 2)[:, :, :n, None]  # noqa: E731
        k, v = k * each(st["k_scales"]), v * each(st["v_scales"])
    k, v = (torch.where(allowed[:, None, :, None], t, 0.0) for t in (k, v))
    x = torch.matmul(q, k.transpose(2, 3)) * st["scale"]
    slopes = st["slopes"].view(h_kv, -1, 1) if "slopes" in st else None
    p = _weights_of(_modify(x, case, slopes, (ctx - 1 - pos)[:, None, None].float()), allowed[:, None, None])
    out = torch.matmul(p, v).reshape(st["q"].shape).to(torch.bfloat16)
    if case["op"] != "decode_weights":
        return out
    st["weights"][:, :, :n] += p.sum(2)
    return out, st["weights"]


def _plain_prefill(st):
    case = st["case"]
    h_kv, n, m = case["h_kv"], st["max_len"], st["max_query"]
    start, ctx = st["query_start"].long(), st["context_lens"].long()
    count = start[1:] - start[:-1]
    i = torch.arange(m, device=DEV)
    real = i < count[:, None]
    at = start[:-1, None] + torch.minimum(i, count[:, None] - 1)
    q = st["q"][at].float().view(case["B"], m, h_kv, -1, case["d"]).permute(0, 2, 3, 1, 4)
    p = (ctx - count)[:, None] + i
    t = torch.arange(n, device=DEV)
    allowed = t <= p[:, :, None]
    if "prefix_lens" in st:
        allowed = allowed | (t < st["prefix_lens"].long()[:, None, None])
    allowed = allowed & (t < ctx[:, None, None])
    if case["window"]:
        allowed = allowed & (t > p[:, :, None] - case["window"])
    held = (t < ctx[:, None])[:, None, :, None]
    k, v = (torch.where(held, _gather(st[c], st["block_tables"], n), 0.0) for c in ("k_cache", "v_cache"))
    x = torch.matmul(q, k[:, :, None].transpose(3, 4)) * st["scale"]
    slopes = st["slopes"].view(h_kv, -1, 1, 1) if "slopes" in st else None
    far = (p[:, :, None] - t).abs().float()[:, None, None]
    o = torch.matmul(_weights_of(_modify(x, case, slopes, far), allowed[:, None, None]), v[:, :, None])
    o = o.permute(0, 3, 1, 2, 4).reshape(case["B"], m, -1, case["d"])
    st["out"][at[real]] = o[real].to(torch.bfloat16)
    return st["out"]


def _plain_write(st):
    case = st["case"]
    kind, bs = case["cache"], case["bs"]
    slots = st["slot_mapping"]
    blk, group = torch.unique(slots // bs, return_inverse=True)
    first = torch.full((blk.numel(),), bs, device=DEV).scatter_reduce(0, group, slots % bs, "amin")
    row = torch.arange(bs, device=DEV)
    for new, cache, scales in ((st["key"], st["k_cache"], st["k_scales"]), (st["value"], st["v_cache"], st["v_scales"])):
        top = new.float().abs().amax(2)
        amax = torch.zeros((blk.numel(), top.shape[1]), device=DEV).scatter_reduce(0, group[:, None].expand_as(top), top,
                                                                                   "amax")
        old = torch.where(first[:, None] > 0, scales[blk], 0.0)
        now = torch.maximum(old, _scale_of(amax, kind))
        again = _encode(cache[blk].float() * old[:, :, None, None], now[:, :, None, None], kind)
        live = (row < first[:, None])[:, None, :, None] & (now > old)[:, :, None, None]
        cache.view(torch.uint8)[blk] = torch.where(live, again.view(torch.uint8), cache.view(torch.uint8)[blk])
        cache.view(torch.uint8)[slots // bs, :, slots % bs] = _encode(new.float(), now[group][:, :, None],
                                                                      kind).view(torch.uint8)
        scales[blk] = now
    return _written(st)


def _written(st):
    """The cache after a write: E4M3 and whole-number codes as the values they are, and what one unit is worth."""
    return {k: st[k] for k in ("k_cache", "v_cache", "k_scales", "v_scales")}


def _plain_evict(st):
    case = st["case"]
    h_kv, bs, budget, n = case["h_kv"], case["bs"], case["budget"], st["max_len"]
    ctx = st["context_lens"].long()
    size = ctx.clamp(max=budget)
    pos = torch.arange(n, device=DEV)
    last = size.clamp(max=case["recent"])
    w = torch.where(st["weights"] > 0, st["weights"], 0.0)
    # heaviest first, the earlier of equals first; behind them what is kept in any case, or not there at all
    older = (pos < (ctx - last)[:, None])[:, None]
    rank = torch.sort(torch.where(older, w, -1.0), dim=-1, descending=True, stable=True)[1][..., :budget]
    rank = torch.where(torch.arange(rank.shape[-1], device=DEV) < (size - last)[:, None, None], rank, n)
    j = torch.arange(case["recent"], device=DEV)
    tail = torch.where(j < last[:, None], (ctx - last)[:, None] + j, n)[:, None].expand(-1, h_kv, -1)
    chosen = torch.cat([rank, tail], -1).sort(-1)[0][..., :budget]
    real = chosen < n
    at = chosen.clamp(max=n - 1)
    st["kept"].fill_(-1)
    st["kept"][..., :chosen.shape[-1]] = torch.where(real, at, -1).to(torch.int32)
    st["new_weights"].zero_()
    st["new_weights"][..., :chosen.shape[-1]] = torch.where(real, st["weights"].gather(-1, at), 0.0)
    st["new_context_lens"].copy_(size)
    b, h, j = real.nonzero(as_tuple=True)
    src, dst = st["block_tables"].long()[b, at[b, h, j] // bs], st["new_tables"].long()[b, j // bs]
    for cache in (st["k_cache"], st["v_cache"]):
        cache[dst, h, j % bs] = cache[src, h, at[b, h, j] % bs]
    return _evicted(st)


def _evicted(st):
    return {k: st[k] for k in ("kept", "new_weights", "new_context_lens", "k_cache", "v_cache")}


def run(st):
    case = st["case"]
    op = case["op"]
    if not own:
        if op == "prefill_scoremod":
            return _plain_prefill(st)
        if op == "write_block_scales":
            return _plain_write(st)
        return _plain_evict(st) if op == "evict" else _plain_decode(st)

    import paged_kv_cache_428_b200 as pa
    if op == "decode_scoremod":
        return pa.pa_decode_scoremod(st["out"], st["q"], st["k_cache"], st["v_cache"], st["block_tables"],
                                     st["context_lens"], st["max_len"], softcap=case["softcap"],
                                     alibi_slopes=st.get("slopes"), window=case["window"], scale=st["scale"],
                                     workspace=st["workspace"])
    if op == "prefill_scoremod":
        return pa.pa_prefill_scoremod(st["out"], st["q"], st["k_cache"], st["v_cache"], st["block_tables"],
                                      st["query_start"], st["context_lens"], st["max_query"], st["workspace"],
                                      softcap=case["softcap"], alibi_slopes=st.get("slopes"), window=case["window"],
                                      prefix_lens=st.get("prefix_lens"), scale=st["scale"])
    if op == "write_block_scales":
        pa.pa_reshape_and_cache_block_scales(st["key"], st["value"], st["k_cache"], st["v_cache"], st["k_scales"],
                                             st["v_scales"], st["slot_mapping"])
        return _written(st)
    if op == "decode_block_scales":
        return pa.pa_decode_block_scales(st["out"], st["q"], st["k_cache"], st["v_cache"], st["k_scales"],
                                         st["v_scales"], st["block_tables"], st["context_lens"], st["max_len"],
                                         scale=st["scale"], workspace=st["workspace"])
    if op == "decode_weights":
        return pa.pa_decode_weights(st["out"], st["weights"], st["q"], st["k_cache"], st["v_cache"],
                                    st["block_tables"], st["context_lens"], st["max_len"], scale=st["scale"],
                                    workspace=st["workspace"]), st["weights"]
    pa.pa_evict(st["k_cache"], st["v_cache"], st["weights"], st["block_tables"], st["context_lens"], st["new_tables"],
                st["max_len"], case["budget"], case["recent"], st["kept"], st["new_weights"], st["new_context_lens"])
    return _evicted(st)


# --------------------------------------------------------------------------------- 64-bit definition
def _rows64(cache, scales, tab, s, count):
    """The first `count` rows of sequence s in 64 bits: [h_kv, count, d]."""
    blocks = tab[s, :-(-count // cache.shape[2])].long()
    rows = cache[blocks].double()
    if scales is not None:
        rows = rows * scales[blocks].double()[:, :, None, None]
    return rows.permute(1, 0, 2, 3).reshape(cache.shape[1], -1, cache.shape[3])[:, :count]


def _attend64(q, k, v, case, scale, slopes, p, prefix):
    """Rows q [r, h_q, d] at positions p [r] over k, v [h_kv, n, d]: (outputs, weights [h_q, r, n])."""
    n, g = k.shape[1], q.shape[1] // k.shape[0]
    t = torch.arange(n, device=DEV)
    gap = p[:, None] - t
    see = (gap >= 0) | (t < prefix)
    if case.get("window"):
        see &= gap < case["window"]
    out = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    weights = torch.zeros((q.shape[1], q.shape[0], n), dtype=torch.float64, device=DEV)
    for h in range(q.shape[1]):
        x = q[:, h].double() @ k[h // g].T * scale
        if case.get("softcap"):
            x = torch.tanh(x / case["softcap"]) * case["softcap"]
        if slopes is not None:
            x = x - slopes[h].double() * gap.abs()
        weights[h] = torch.softmax(x.masked_fill(~see, -math.inf), -1)
        out[:, h] = weights[h] @ v[h // g]
    return out, weights


def exact(case, seed):
    st = prepare(case, seed)
    op, tab = case["op"], st["block_tables"]
    held, new = _lengths(case)
    if op in ("decode_scoremod", "decode_block_scales", "decode_weights", "prefill_scoremod"):
        out = torch.zeros(st["out"].shape, dtype=torch.float64, device=DEV)
        total = st["weights"].double() if op == "decode_weights" else None
        row = 0
        for s in range(case["B"]):
            n, r = held[s] + new[s], new[s] if op == "prefill_scoremod" else 1
            prefix = int(st["prefix_lens"][s]) if "prefix_lens" in st else 0
            k, v = (_rows64(st[a], st.get(b), tab, s, n) for a, b in (("k_cache", "k_scales"), ("v_cache", "v_scales")))
            for i in range(0, r, 512):
                m = min(512, r - i)
                at = torch.arange(n - r + i, n - r + i + m, device=DEV)
                o, w = _attend64(st["q"][row + i:row + i + m], k, v, case, st["scale"], st.get("slopes"), at, prefix)
                out[row + i:row + i + m] = o
                if total is not None:
                    total[s, :, :n] += w[:, 0].view(case["h_kv"], -1, n).sum(1)
            row += r
        return out if total is None else (out, total)
    if op == "write_block_scales":
        return _exact_write(st, case)
    return _exact_evict(st, case)


def _nearest(x, kind):
    """x to the nearest code in 64 bits, ties to the even one."""
    if kind == "int8":
        return torch.round(x).clamp(-127, 127)
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def _exact_write(st, case):
    kind, bs = case["cache"], case["bs"]
    got = {}
    slots = st["slot_mapping"].cpu()
    order = torch.argsort(slots)
    cut = torch.unique_consecutive(slots[order] // bs, return_counts=True)
    for name, rows in (("k", st["key"]), ("v", st["value"])):
        value, scale = st[name + "_cache"].double(), st[name + "_scales"].double()
        rows64 = rows.double()
        at = 0
        for b, count in zip(cut[0].tolist(), cut[1].tolist()):
            mine = order[at:at + count].to(DEV)
            off = st["slot_mapping"][mine] % bs
            at += count
            first = int(off.min())
            want = rows64[mine].abs().amax(dim=(0, 2)) / QMAX[kind]
            exponent = torch.floor(torch.log2(want.clamp(min=1e-300)))
            unit = torch.exp2(exponent - 7)
            want = torch.ceil(want / unit) * unit
            old = scale[b].clone()
            now = torch.maximum(old, want) if first else want
            if first:
                fresh = _nearest(value[b, :, :first] * (old / now)[:, None, None], kind)
                value[b, :, :first] = torch.where((now > old)[:, None, None], fresh, value[b, :, :first])
            value[b, :, off] = _nearest(rows64[mine] / now[None, :, None], kind).transpose(0, 1)
            scale[b] = now
        got[name + "_cache"] = value.to(torch.int8) if kind == "int8" else value
        got[name + "_scales"] = scale
    return got


def _exact_evict(st, case):
    """Moves and choices only: nothing is rounded, so the values are those of the inputs."""
    bs, budget = case["bs"], case["budget"]
    for s in range(case["B"]):
        n = int(st["context_lens"][s])
        size = min(n, budget)
        last = min(size, case["recent"])
        st["new_context_lens"][s] = size
        blocks, fresh = st["block_tables"][s].long(), st["new_tables"][s].long()
        for h in range(case["h_kv"]):
            w = st["weights"][s, h, :n - last].clamp(min=0)
            heavy = torch.argsort(-w, stable=True)[:size - last]
            keep = torch.cat([heavy.sort()[0], torch.arange(n - last, n, device=DEV)])
            j = torch.arange(size, device=DEV)
            st["kept"][s, h] = -1
            st["kept"][s, h, :size] = keep.int()
            st["new_weights"][s, h, :size] = st["weights"][s, h, keep]
            for cache in (st["k_cache"], st["v_cache"]):
                cache[fresh[j // bs], h, j % bs] = cache[blocks[keep // bs], h, keep % bs]
    return {k: st[k] for k in ("kept", "new_weights", "new_context_lens", "k_cache", "v_cache")}
