"""Definitions in 64 bits of the calls with modified scores, block scales and attention weights, and the bounds
that their outputs are held to.  (Test infrastructure, numpy / torch on the CPU only.)"""
from __future__ import annotations

import math

import torch

QMAX = {"e4m3": 448.0, "int8": 127.0}
DTYPE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}


def block_scale(amax: float, kind: str) -> float:
    """The smallest bf16 number s with QMAX s >= amax, at least 2^-80 unless amax is 0."""
    if amax == 0:
        return 0.0
    want = amax / QMAX[kind]
    unit = 2.0 ** (max(math.floor(math.log2(want)), -126) - 7)
    return max(math.ceil(want / unit) * unit, 2.0 ** -80)


def encode(x: torch.Tensor, s: float, kind: str) -> torch.Tensor:
    """Values (64 bits) of the codes of x at scale s."""
    if s == 0:
        return torch.zeros_like(x)
    y = x / s
    if kind == "int8":
        return torch.where(torch.isnan(y), torch.zeros_like(y), torch.round(y).clamp(-127, 127))
    mag = y.abs().clamp(max=1e30)
    step = 2.0 ** (torch.floor(torch.log2(mag.clamp(min=2.0 ** -6))) - 3)
    return torch.where(torch.isnan(y), y, (torch.round(y / step) * step).clamp(-448, 448))


def write_block_scales(rows, cache, scales, slots, kind):
    """The write, in place: rows [T, h, d] f64, cache [NB, h, bs, d] f64 code values, scales [NB, h] f64."""
    bs, n = cache.shape[2], cache.shape[0]
    groups = {}
    for t, s in enumerate(slots):
        if 0 <= s < n * bs:
            groups.setdefault(s // bs, {})[s % bs] = t          # the last of equal slots
    for b, owner in groups.items():
        first = min(owner)
        for h in range(cache.shape[1]):
            new = torch.stack([rows[t, h] for t in owner.values()])
            new = new[torch.isfinite(new)]
            s = block_scale(float(new.abs().max()) if new.numel() else 0.0, kind)
            old = float(scales[b, h]) if first else 0.0
            now = max(old, s)
            if first and now > old:
                cache[b, h, :first] = encode(cache[b, h, :first] * old, now, kind)
            for off, t in owner.items():
                cache[b, h, off] = encode(rows[t, h], now, kind)
            scales[b, h] = now


def rows_of(cache, table_row, count, scales=None):
    """The first `count` rows of a sequence: [h_kv, count, d] in 64 bits."""
    bs = cache.shape[2]
    blocks = table_row[:-(-count // bs)].long() if count else table_row[:0].long()
    rows = cache[blocks].double()
    if scales is not None:
        rows = rows * scales[blocks].double()[:, :, None, None]
    return rows.permute(1, 0, 2, 3).reshape(cache.shape[1], -1, cache.shape[3])[:, :count]


def attend(q, k, v, positions, scale, softcap=0.0, slopes=None, window=0, prefix=0):
    """q [r, h_q, d] at `positions` over k, v [h_kv, n, d]: outputs [r, h_q, d], sum of p |v| likewise, and
    the weights [r, h_q, n]."""
    r, h_q, d = q.shape
    h_kv, n, _ = k.shape
    g = h_q // h_kv
    t = torch.arange(n)
    gap = positions[:, None] - t
    see = (gap >= 0) | (t < prefix)
    if window:
        see &= gap < window
    out = torch.zeros((r, h_q, d), dtype=torch.float64)
    mag = torch.zeros_like(out)
    weights = torch.zeros((r, h_q, n), dtype=torch.float64)
    for h in range(h_q):
        x = (q[:, h].double() @ k[h // g].T) * scale
        if softcap:
            x = softcap * torch.tanh(x / softcap)
        if slopes is not None:
            x = x - float(slopes[h]) * gap.abs()
        x = x.masked_fill(~see, -math.inf)
        p = torch.softmax(x, -1)
        use = see.any(0)
        p = torch.where(see, p, torch.zeros_like(p))
        weights[:, h] = p
        kv = torch.where(use[:, None], v[h // g], torch.zeros_like(v[h // g]))
        out[:, h] = p @ kv
        mag[:, h] = p @ kv.abs()
    return out, mag, weights


def check_rows(got, ref, mag, p_bits, what="", logit_err=2e-5, extra=0.0):
    """Every value of `got` (bf16) within: half a step of bf16 for the output; p_bits for the rounding of the
    probabilities (half a step relative to each, so relative to sum p |v|); and for fp32 arithmetic an
    error `logit_err` of the logits, which moves each probability by that factor and the normaliser by as much.
    `extra`: a further absolute term that the caller derives."""
    g = got.detach().double().cpu()
    bound = 2.0 ** -8 * ref.abs() + (2.0 ** -p_bits + 2 * logit_err) * (1 + 2.0 ** -8) * mag + extra + 1e-30
    over = (g - ref).abs() > bound
    assert torch.isfinite(g).all(), what + ": non-finite output"
    assert not over.any(), "%s: %d of %d values off, worst %.3g times the bound" % (
        what, int(over.sum()), g.numel(), float(((g - ref).abs() / bound).max()))
