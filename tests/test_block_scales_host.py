"""The 8-bit cache with a scale per block and KV head, as far as the CPU goes: argument checks (nothing is
launched), workspace sizes, the host check of slots, and the binding's refusals."""
import pytest
import torch

import paged_kv_cache_428_b200 as pa

L = pa.lib()
FAKE = 1 << 20            # aligned, non-null, never dereferenced on these paths


def _write(**kw):
    a = dict(k=FAKE, v=FAKE, ks=0, vs=0, kc=FAKE, vc=FAKE, sk=FAKE, sv=FAKE, slots=FAKE, T=4, h=2, d=64, bs=16, nb=8, dt=1)
    a.update(kw)
    return L.pa_reshape_and_cache_block_scales(a["k"], a["v"], a["ks"], a["vs"], a["kc"], a["vc"], a["sk"], a["sv"],
                                               a["slots"], a["T"], a["h"], a["d"], a["bs"], a["nb"], a["dt"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(dt=0), -1), (dict(dt=3), -1), (dict(T=-1), -1), (dict(h=0), -1), (dict(nb=0), -1), (dict(d=96), -2), (dict(bs=8), -2),
    (dict(ks=64), -1), (dict(vs=132), -1), (dict(k=0), -1), (dict(sk=0), -1), (dict(sv=0), -1), (dict(slots=0), -1),
    (dict(v=FAKE + 8), -1), (dict(kc=FAKE + 4), -1), (dict(T=0), 0), (dict(T=0, k=0, slots=0), 0), (dict(h=70000), -2)])
def test_write_refusals(kw, status):
    assert _write(**kw) == status


def _decode(**kw):
    a = dict(out=FAKE, q=FAKE, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, bt=FAKE, mb=8, ctx=FAKE, B=2, mc=100, hq=4, hkv=2, d=64, bs=16,
             nb=16, scale=0.125, dt=1, ws=FAKE, wsb=1 << 40)
    a.update(kw)
    return L.pa_decode_block_scales(a["out"], a["q"], a["k"], a["v"], a["ks"], a["vs"], a["bt"], a["mb"], a["ctx"], a["B"],
                                    a["mc"], a["hq"], a["hkv"], a["d"], a["bs"], a["nb"], a["scale"], a["dt"], a["ws"],
                                    a["wsb"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(dt=0), -1), (dict(B=-1), -1), (dict(mc=-1), -1), (dict(hq=0), -1), (dict(hkv=0), -1), (dict(nb=0), -1), (dict(mb=0), -1),
    (dict(hq=5), -1), (dict(scale=float("inf")), -1), (dict(scale=float("nan")), -1), (dict(d=32), -2), (dict(bs=128), -2),
    (dict(hq=32), -2), (dict(B=4097), -2), (dict(B=4096, hkv=32, hq=32), -2), (dict(mb=2 ** 30, B=4), -2),
    (dict(nb=2 ** 27), -2), (dict(out=0), -1), (dict(q=FAKE + 2), -1), (dict(ks=0), -1), (dict(vs=0), -1),
    (dict(ws=0), -3), (dict(ws=FAKE + 8), -3), (dict(wsb=1000), -3), (dict(B=0), 0)])
def test_decode_refusals(kw, status):
    assert _decode(**kw) == status


def test_workspace_size_is_what_the_call_asks_for():
    n = pa.pa_decode_block_scales_workspace_size(2, 4, 2, 64, 100)
    assert _decode(wsb=n - 1) == -3
    assert pa.pa_decode_block_scales_workspace_size(0, 4, 2, 64, 100) == 0
    assert pa.pa_decode_block_scales_workspace_size(2, 5, 2, 64, 100) == 0
    # bounded by the GPU, not by the context
    assert pa.pa_decode_block_scales_workspace_size(1, 8, 1, 128, 10 ** 8) < 16 << 20


def test_copy_refusals():
    import ctypes
    one = ctypes.cast((ctypes.c_void_p * 1)(FAKE), ctypes.c_void_p)
    none = ctypes.cast((ctypes.c_void_p * 1)(None), ctypes.c_void_p)
    f = L.pa_copy_block_scales
    assert f(one, one, 1, FAKE, 1, 0, 8, None) == -1
    assert f(one, one, 1, FAKE, -1, 2, 8, None) == -1
    assert f(one, none, 1, FAKE, 1, 2, 8, None) == -1
    assert f(None, one, 1, FAKE, 1, 2, 8, None) == -1
    assert f(one, one, 1, FAKE, 1, 2, 0, None) == -1
    assert f(one, one, 1, None, 0, 2, 8, None) == 0


@pytest.mark.parametrize("slots,status", [
    ([], 0), ([0, 1, 2, 15, 16], 0), ([5, 4, 3], 0), ([-1, 5, -1, 20], 0), ([5, 20, 6], -1), ([5, -1, 6], -1), ([127], 0),
    ([128], -1), ([7, 7], 0)])
def test_validate_block_runs(slots, status):
    assert pa.pa_validate_block_runs(torch.tensor(slots, dtype=torch.int64), 16, 8) == status


def test_binding_refuses():
    k = torch.zeros((2, 2, 64), dtype=torch.bfloat16)
    c = torch.zeros((4, 2, 16, 64), dtype=torch.int8)
    s, _ = pa.make_block_scales(4, 2, device="cpu")
    slots = torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError):                                   # CPU tensors
        pa.pa_reshape_and_cache_block_scales(k, k, c, c, s, s, slots)
    with pytest.raises(TypeError):                                    # a bf16 cache has no scales
        pa.pa_reshape_and_cache_block_scales(k, k, k.view(1, 2, 2, 64), k.view(1, 2, 2, 64), s, s, slots)
    with pytest.raises(ValueError):
        pa.pa_copy_block_scales([s], [], slots.view(1, 2))
