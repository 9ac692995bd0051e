"""The binding's own checks of the cache's calls: what a C entry cannot see in an address.  No GPU: every call below is
refused before the library is reached, which a stub would tell."""
from types import SimpleNamespace

import pytest
import torch


@pytest.fixture()
def kq(monkeypatch):
    from kronecker_factored_transforms_b200 import build
    build.build()
    from kronecker_factored_transforms_b200 import _lib
    _lib._device_calls()
    monkeypatch.setattr(_lib, "_current_device", lambda: -1)  # CPU tensors are on device -1
    monkeypatch.setattr(_lib, "_raw_stream", lambda device: 0)
    reached = []
    entry = lambda *a: reached.append(a) or 0
    monkeypatch.setattr(_lib, "lib", SimpleNamespace(kq_kv_append=entry, kq_kv_gather=entry, kq_kv_attention=entry,
                                                     kq_kv_attention_shared=entry))
    _lib.reached = reached
    return _lib


def handle(**kw):
    return SimpleNamespace(**dict(dict(device=-1, head_dim=64, ptr=1), **kw))


B16, I32, I64, F32 = torch.bfloat16, torch.int32, torch.int64, torch.float32
T, H, HK, D = 4, 4, 2, 64


def append(kq, cache=None, tf=None, **kw):
    qkv = torch.zeros(T, H + 2 * HK, D, dtype=B16)
    a = dict(q=qkv[:, :H], k=qkv[:, H:H + HK], v=qkv[:, H + HK:], pos=torch.zeros(T, dtype=I32),
             slot=torch.zeros(T, dtype=I64), out=torch.zeros(T, H, D, dtype=B16))
    a.update(kw)
    s = qkv.stride(0)
    kq.kq_kv_append(cache or handle(), tf or handle(), a["q"], s, a["k"], s, a["v"], s, a["pos"], a["slot"], a["out"], T, H)


def gather(kq, **kw):
    a = dict(slot=torch.zeros(T, dtype=I64), k=torch.zeros(T, HK, D, dtype=B16), v=torch.zeros(T, HK, D, dtype=B16))
    a.update(kw)
    kq.kq_kv_gather(handle(), a["slot"], a["k"], a["v"], T)


def attend(kq, shared=False, **kw):
    a = dict(q=torch.zeros(T, H, D, dtype=B16), start=torch.zeros(3, dtype=I32), pre=torch.zeros(2, dtype=I32),
             table=torch.zeros(2, 5, dtype=I32), len=torch.zeros(2, dtype=I32), out=torch.zeros(T, H, D, dtype=B16),
             lse=torch.zeros(T, H), ws=torch.zeros(1000, dtype=torch.uint8))
    a.update(kw)
    tail = (a["table"], 5, a["len"], 0.1, 0.0, 0, a["out"], a["lse"], a["ws"], 1000, T, 2, H, 3)
    if shared:
        kq.kq_kv_attention_shared(handle(), a["q"], a["start"], a["pre"], 20, *tail)
    else:
        kq.kq_kv_attention(handle(), a["q"], a["start"], *tail)


def refused(kq, call, **kw):
    with pytest.raises(ValueError):
        call(kq, **kw)
    assert not kq.reached


def test_the_calls_as_they_are_meant(kq):
    append(kq)
    append(kq, q=torch.zeros(T, H, D, dtype=torch.int16), pos=None, out=torch.zeros(T, H, D, dtype=torch.uint16))
    append(kq, q=1 << 40, k=1 << 41, v=1 << 42, pos=None, slot=1 << 43, out=1 << 44)  # addresses
    gather(kq)
    attend(kq)
    attend(kq, shared=True, start=None, lse=None, ws=torch.zeros(250))
    assert len(kq.reached) == 6


def test_a_transform_of_another_device_or_size(kq):
    """Its addresses would be followed on this device, past its factors' ends."""
    refused(kq, append, tf=handle(device=1))
    refused(kq, append, tf=handle(head_dim=32))
    refused(kq, append, cache=handle(head_dim=128))


def test_handles_know_their_head_dim(kq):
    codes, scale = torch.zeros(3, 2, 16, 64, dtype=torch.uint8), torch.zeros(3, 2, 16)
    P = torch.zeros(64, 64, dtype=B16)
    kept = []

    class Handle(kq._Handle):
        def __init__(self, struct, tensors, head_dim):
            kept.append(head_dim)

    kq._Handle, base = Handle, kq._Handle
    try:
        kq.kv_cache(codes, scale, codes, scale)
        kq.kv_transform(P, P, P, 0.9, 0.9)
    finally:
        kq._Handle = base
    assert kept == [128, 64]


def test_fp16_factors(kq):
    """Two bytes an element, but other numbers."""
    P = torch.zeros(64, 64, dtype=B16)
    for bad in ((P.half(), P, P), (P, P.half(), P), (P, P, P.half())):
        with pytest.raises(ValueError, match="bf16"):
            kq.kv_transform(*bad, 0.9, 0.9)


@pytest.mark.parametrize("kw", [
    dict(pos=torch.zeros(T, dtype=I64)), dict(pos=torch.zeros(T)), dict(slot=torch.zeros(T, dtype=I32)),
    dict(pos=torch.zeros(2 * T, dtype=I32)[::2]), dict(slot=torch.zeros(2 * T, dtype=I64)[::2]),
    dict(q=torch.zeros(T, H, D)), dict(k=torch.zeros(T, HK, D, dtype=torch.float16)),
    dict(v=torch.zeros(T, D, HK, dtype=B16).transpose(1, 2)), dict(out=torch.zeros(T, H, D)),
    dict(out=torch.zeros(T, 2 * H, D, dtype=B16)[:, :H])])
def test_append_types_and_strides(kq, kw):
    refused(kq, append, **kw)


@pytest.mark.parametrize("kw", [dict(slot=torch.zeros(T, dtype=I32)), dict(k=torch.zeros(T, HK, D)),
                                dict(v=torch.zeros(T, 2 * HK, D, dtype=B16)[:, :HK])])
def test_gather_types_and_strides(kq, kw):
    refused(kq, gather, **kw)


@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("kw", [
    dict(table=torch.zeros(2, 5, dtype=I64)), dict(table=torch.zeros(2, 10, dtype=I32)[:, :5]), dict(len=torch.zeros(2, dtype=I64)),
    dict(len=torch.zeros(4, dtype=I32)[::2]), dict(start=torch.zeros(3, dtype=I64)), dict(start=torch.zeros(6, dtype=I32)[::2]),
    dict(q=torch.zeros(T, 2 * H, D, dtype=B16)[:, :H]), dict(q=torch.zeros(T, H, D, dtype=torch.float16)),
    dict(out=torch.zeros(T, H, D, dtype=torch.float16)), dict(out=torch.zeros(H, T, D, dtype=B16).transpose(0, 1)),
    dict(lse=torch.zeros(T, H, dtype=torch.float64)), dict(lse=torch.zeros(H, T).T), dict(ws=torch.zeros(2000, dtype=torch.uint8)[::2])])
def test_attention_types_and_strides(kq, kw, shared):
    refused(kq, lambda kq, **a: attend(kq, shared, **a), **kw)


def test_prefix_types_and_strides(kq):
    for pre in (torch.zeros(2, dtype=I64), torch.zeros(4, dtype=I32)[::2]):
        refused(kq, lambda kq, **a: attend(kq, True, **a), pre=pre)
