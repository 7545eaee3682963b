"""Attention weights and eviction, as far as the CPU goes: argument checks (nothing is launched) and sizes."""
import pytest
import torch

import paged_kv_cache_428_b200 as pa

L = pa.lib()
FAKE = 1 << 20            # aligned, non-null, never dereferenced on these paths
FAR = 1 << 34


def _decode(**kw):
    a = dict(out=FAKE, w=FAKE, st=100, q=FAKE, k=FAKE, v=FAKE, bt=FAKE, mb=8, ctx=FAKE, B=2, mc=100, hq=4, hkv=2, d=64, bs=16,
             nb=16, scale=0.125, dt=0, ws=FAKE, wsb=1 << 40)
    a.update(kw)
    return L.pa_decode_weights(a["out"], a["w"], a["st"], a["q"], a["k"], a["v"], a["bt"], a["mb"], a["ctx"], a["B"], a["mc"],
                               a["hq"], a["hkv"], a["d"], a["bs"], a["nb"], a["scale"], a["dt"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(dt=1), -2), (dict(dt=2), -2), (dict(dt=3), -1), (dict(st=99), -1), (dict(B=-1), -1), (dict(mc=-1), -1), (dict(hq=3), -1),
    (dict(hq=0), -1), (dict(d=80), -2), (dict(bs=24), -2), (dict(hq=32), -2), (dict(w=0), -1), (dict(out=FAKE + 1), -1),
    (dict(ws=0), -3), (dict(wsb=1 << 18), -3), (dict(scale=float("nan")), -1), (dict(B=0), 0)])
def test_decode_weights_refusals(kw, status):
    assert _decode(**kw) == status


def test_decode_weights_workspace():
    n = pa.pa_decode_weights_workspace_size(2, 4, 2, 64, 100)
    assert _decode(wsb=n - 1) == -3
    # the logits are the part that grows with the context
    big = pa.pa_decode_weights_workspace_size(64, 32, 8, 128, 4096)
    assert big >= 64 * 32 * 4096 * 4 + pa.pa_decode_block_scales_workspace_size(64, 32, 8, 128, 4096)
    assert pa.pa_decode_weights_workspace_size(0, 4, 2, 64, 100) == 0


def _evict(**kw):
    a = dict(k=FAKE, v=FAKE, w=FAKE, st=200, bt=FAKE, mb=16, ctx=FAKE, nt=FAKE, nm=4, B=2, mc=200, budget=50, recent=10, h=2, d=64,
             bs=16, nb=64, dt=0, kept=FAR, nw=FAR, ns=64, nl=FAR)
    a.update(kw)
    return L.pa_evict(a["k"], a["v"], a["w"], a["st"], a["bt"], a["mb"], a["ctx"], a["nt"], a["nm"], a["B"], a["mc"], a["budget"],
                      a["recent"], a["h"], a["d"], a["bs"], a["nb"], a["dt"], a["kept"], a["nw"], a["ns"], a["nl"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(budget=0), -1), (dict(recent=-1), -1), (dict(recent=51), -1), (dict(mc=-1), -1), (dict(mc=201), -1), (dict(ns=49), -1),
    (dict(nm=3), -1), (dict(dt=5), -1), (dict(d=100), -2), (dict(bs=4), -2), (dict(h=0), -1), (dict(h=70000), -2),
    (dict(kept=0), -1), (dict(nl=0), -1), (dict(nw=0), -1), (dict(w=0), -1), (dict(k=FAKE + 8), -1),
    (dict(nw=FAKE + 4 * 799), -1), (dict(nw=FAKE - 4 * 255), -1), (dict(nl=FAKE + 4), -1), (dict(B=0), 0), (dict(B=0, kept=0), 0)])
def test_evict_refusals(kw, status):
    assert _evict(**kw) == status


def test_sizes_near_the_end_of_32_bits():
    """Places are counted in 32 bits, in steps: bounds above 2^30 are refused before anything is computed from them."""
    big, more = 2 ** 31 - 1, 2 ** 30 + 1
    assert pa.pa_decode_weights_workspace_size(1, 1, 1, 64, 2 ** 30) > 2 ** 32
    assert pa.pa_decode_weights_workspace_size(1, 1, 1, 64, more) == 0
    for n in (more, big - 3, big):
        assert _decode(B=1, hq=1, hkv=1, mc=n, st=1 << 31, wsb=1 << 62) == -2
        assert _evict(B=0, mc=n, st=1 << 31) == -2
        assert _evict(B=0, budget=n, ns=1 << 31, nm=1 << 28) == -2


def test_binding_refuses():
    c = torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError):                                   # CPU tensors
        pa.pa_evict(c, c, torch.zeros(1, 2, 32), i32(1, 2), i32(1), i32(1, 2), 32, 8, 2, i32(1, 2, 8), torch.zeros(1, 2, 8),
                    i32(1))
    with pytest.raises(ValueError):
        pa.pa_decode_weights(c[:1, :, 0], torch.zeros(1, 2, 32), c[:1, :, 0], c, c, i32(1, 2), i32(1), 32)
