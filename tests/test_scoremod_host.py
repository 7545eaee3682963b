"""Attention with modified scores, as far as the CPU goes: argument checks (nothing is launched), sizes, and the
polynomial that stands in for tanh."""
import math
import re
from pathlib import Path

import pytest
import torch

import paged_kv_cache_428_b200 as pa

L = pa.lib()
FAKE = 1 << 20            # aligned, non-null, never dereferenced on these paths
NAN, INF = float("nan"), float("inf")


def _decode(**kw):
    a = dict(out=FAKE, q=FAKE, k=FAKE, v=FAKE, bt=FAKE, mb=8, ctx=FAKE, B=2, mc=100, hq=4, hkv=2, d=64, bs=16, nb=16, scale=0.125,
             cap=0.0, sl=0, win=0, dt=0, ws=FAKE, wsb=1 << 40)
    a.update(kw)
    return L.pa_decode_scoremod(a["out"], a["q"], a["k"], a["v"], a["bt"], a["mb"], a["ctx"], a["B"], a["mc"], a["hq"], a["hkv"],
                                a["d"], a["bs"], a["nb"], a["scale"], a["cap"], a["sl"], a["win"], a["dt"], a["ws"], a["wsb"],
                                None)


@pytest.mark.parametrize("kw,status", [
    (dict(cap=-1.0), -1), (dict(cap=NAN), -1), (dict(cap=INF), -1), (dict(cap=2.0 ** -65), -1), (dict(win=-1), -1), (dict(dt=1), -2), (dict(dt=9), -1),
    (dict(scale=NAN), -1), (dict(hq=5), -1), (dict(hq=32), -2), (dict(d=256), -2), (dict(bs=1), -2), (dict(B=5000), -2),
    (dict(out=0), -1), (dict(ctx=0), -1), (dict(ws=0), -3), (dict(wsb=100), -3), (dict(B=0), 0), (dict(B=0, cap=-1.0), -1)])
def test_decode_refusals(kw, status):
    assert _decode(**kw) == status


def _prefill(**kw):
    a = dict(out=FAKE, q=FAKE, k=FAKE, v=FAKE, bt=FAKE, mb=8, qs=FAKE, ctx=FAKE, B=2, mq=50, hq=4, hkv=2, d=64, bs=16, nb=16,
             scale=0.125, cap=0.0, sl=0, win=0, pl=0, dt=0, ws=FAKE, wsb=256)
    a.update(kw)
    return L.pa_prefill_scoremod(a["out"], a["q"], a["k"], a["v"], a["bt"], a["mb"], a["qs"], a["ctx"], a["B"], a["mq"], a["hq"],
                                 a["hkv"], a["d"], a["bs"], a["nb"], a["scale"], a["cap"], a["sl"], a["win"], a["pl"], a["dt"],
                                 a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(cap=-0.5), -1), (dict(cap=NAN), -1), (dict(win=-3), -1), (dict(dt=2), -2), (dict(dt=-1), -1), (dict(scale=INF), -1),
    (dict(scale=0.0), -1), (dict(scale=-0.1), -1), (dict(mq=-1), -1), (dict(hq=6, hkv=4), -1), (dict(hq=48), -2), (dict(nb=2 ** 28), -2), (dict(qs=0), -1), (dict(q=FAKE + 8), -1),
    (dict(ws=0), -3), (dict(wsb=255), -3), (dict(ws=FAKE + 1), -3), (dict(B=0), 0), (dict(mq=0), 0)])
def test_prefill_refusals(kw, status):
    assert _prefill(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(cap=2.3e38), 0), (dict(cap=2.4e38), -1), (dict(cap=2.0 ** -64), 0), (dict(cap=2.0 ** -64, scale=1e19), -1),
    (dict(cap=1.0, scale=1e19), 0), (dict(scale=2.4e38), -1), (dict(cap=0.5, scale=1e38), -1)])
def test_scales_and_caps_that_leave_fp32(kw, status):
    """What scores are multiplied by is finite: infinity times a score of 0 would be NaN."""
    assert _decode(B=0, **kw) == status
    assert _prefill(B=0, **kw) == status


def test_workspace_goes_by_the_window():
    size = pa.pa_decode_scoremod_workspace_size
    assert size(1, 8, 2, 64, 100000, 100) < size(1, 8, 2, 64, 100000, 0)
    assert _decode(wsb=size(2, 4, 2, 64, 100) - 1) == -3
    assert size(2, 4, 2, 64, 100, -1) == 0 and size(2, 4, 3, 64, 100) == 0


@pytest.mark.parametrize("name,rng,terms,error", [("PA_TANH_C", "PA_TANH_RANGE", 3, 4e-7)])
def test_polynomial_of_tanh(name, rng, terms, error):
    """tanh(y) = y q(y^2) on the range in which the kernel uses it."""
    text = (Path(__file__).resolve().parents[1] / "paged_kv_cache_428_b200" / "csrc" / "tanh_poly.cuh").read_text()
    get = lambda what: float(re.search(r"#define %s (-?[0-9.]+)f" % what, text).group(1))  # noqa: E731
    c, top = [get("%s%d" % (name, i)) for i in range(terms)], get(rng)
    worst = relative = 0.0
    for i in range(20001):
        y = top * i / 20000
        q = 0.0
        for a in reversed(c):
            q = q * y * y + a
        worst = max(worst, abs(y * q - math.tanh(y)))
        if y:
            relative = max(relative, abs(y * q / math.tanh(y) - 1))
    assert worst < error and relative < 1.2e-6


def test_binding_refuses():
    q = torch.zeros((1, 4, 64), dtype=torch.bfloat16)
    c = torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError):                                   # CPU tensors
        pa.pa_decode_scoremod(q, q, c, c, i32(1, 2), i32(1), 32)
    assert pa._window(2 ** 40) == 2 ** 31 - 1 and pa._window(0) == 0
    with pytest.raises(ValueError):
        pa._window(-1)
    with pytest.raises(TypeError):
        pa.pa_decode_scoremod(q.float(), q, c, c, i32(1, 2), i32(1), 32)
