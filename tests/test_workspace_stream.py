"""Calls without a workspace allocate one that belongs to the stream they run on."""
import contextlib
import math

import pytest
import torch

import paged_kv_cache_428_b200 as pa


def test_owner_of_a_workspace(monkeypatch):
    """None: the current stream.  A raw handle: that stream for torch's allocator too (0 and 1 are the default one)."""
    seen = []

    @contextlib.contextmanager
    def entered(stream):
        seen.append(stream)
        yield

    monkeypatch.setattr(torch.cuda, "stream", entered)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h: "external %d" % h)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda: "default")
    q = torch.zeros(2)
    for stream in (None, 0, 1, 4096):
        ws = pa._new_workspace(100, q, stream)
        assert ws.numel() == 100 and not ws.any()
    assert seen == ["default", "default", "external 4096"]
    with pytest.raises(ValueError):
        pa._new_workspace(100, q, 2)


def _inputs(codes):
    g = torch.Generator().manual_seed(5)
    h_kv, grp, bs, d, lens = 2, 4, 16, 64, [3000, 40]
    nb = sum(-(-n // bs) for n in lens)
    tab = torch.full((2, -(-max(lens) // bs)), -1, dtype=torch.int32)
    order = torch.randperm(nb, generator=g).int()
    tab[0], tab[1, :3] = order[:188], order[188:]
    kv = [torch.randn((nb, h_kv, bs, d), generator=g) for _ in "kv"]
    kv = [(x * 30).clamp(-127, 127).to(torch.int8) if codes else x.to(torch.bfloat16) for x in kv]
    q = torch.randn((2, h_kv * grp, d), generator=g).to(torch.bfloat16)
    return [t.cuda() for t in (q, kv[0], kv[1], tab, torch.tensor(lens, dtype=torch.int32))]


# Each call with what it needs besides q, caches, tables and lengths (made before the stream is kept busy).
def _decode_scoremod(a, more, out, **kw):
    pa.pa_decode_scoremod(out, *a, 3000, softcap=20.0, **kw)


def _decode_block_scales(a, more, out, **kw):
    pa.pa_decode_block_scales(out, a[0], a[1], a[2], more["scales"], more["scales"], a[3], a[4], 3000, **kw)


def _decode_weights(a, more, out, **kw):
    pa.pa_decode_weights(out, more["weights"], *a, 3000, **kw)


def _decode(a, more, out, **kw):
    pa.pa_decode(out, *a, 3000, partition_size=256, **kw)


def _decode_auto(a, more, out, **kw):
    pa.pa_decode(out, *a, 3000, partition_size=pa.PA_PARTITION_AUTO, **kw)


def _decode_step(a, more, out, **kw):
    pa.pa_decode_step(more["rows"], more["rows"], more["slots"], out, *a, 3000, partition_size=256, **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("call", [_decode_scoremod, _decode_block_scales, _decode_weights, _decode, _decode_auto, _decode_step],
                         ids=lambda f: f.__name__)
def test_call_on_another_stream_while_the_current_one_is_busy(call):
    """The workspace is zero when the kernel starts, though the current stream is busy, and what the current stream
    allocates next does not get its memory."""
    a = _inputs(call is _decode_block_scales)
    more = dict(scales=torch.full((a[1].shape[0], 2), 1 / 30, device="cuda"), weights=torch.zeros((2, 2, 3000), device="cuda"),
                rows=torch.zeros((2, 2, 64), dtype=torch.bfloat16, device="cuda"),
                slots=torch.full((2,), -1, dtype=torch.int64, device="cuda"))
    want = torch.empty_like(a[0])
    call(a, more, want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    sizes = [1 << 20, 2 << 20, 4 << 20, 16 << 20]
    for stream in (side, side.cuda_stream, 0, None):
        dirt = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in sizes]      # what freed memory holds
        del dirt
        out = torch.zeros_like(want)
        more["weights"].zero_()
        torch.cuda.synchronize()
        torch.cuda._sleep(40_000_000)                                                        # the current stream is busy
        call(a, more, out, stream=stream)
        after = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in sizes]
        torch.cuda.synchronize()
        assert torch.equal(out, want), stream
        assert all(bool((t == 255).all()) for t in after)
        if call is _decode_weights:
            assert math.isclose(float(more["weights"].sum()), 16.0, rel_tol=1e-4)
    assert pa.pa_device_errors() == 0
