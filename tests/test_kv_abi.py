"""The cache's entry points reject bad arguments on the host before anything is launched
(no GPU needed: every call below fails validation or is empty)."""
import ctypes
import math

import numpy as np
import pytest


@pytest.fixture(scope="module")
def kq():
    from kronecker_factored_transforms_b200 import build
    build.build()
    from kronecker_factored_transforms_b200 import _lib
    return _lib


# Fake, never-dereferenced device addresses, far apart.
KC, KS, VC, VS = 0x100000000, 0x200000000, 0x300000000, 0x400000000
Q, K, V, POS, SLOT, QO, PQ, PK, PV, ROPE = [0x500000000 + 0x10000000 * i for i in range(10)]
QS, TAB, LEN, OUT, LSE, WS, PRE = [0x700000000 + 0x10000000 * i for i in range(7)]


def cache(kq, **kw):
    a = dict(k_codes=KC, k_scale=KS, v_codes=VC, v_scale=VS, num_pages=10, page_size=16, kv_heads=2, head_dim=128)
    a.update(kw)
    return kq._KVCacheStruct(*a.values())


def transform(kq, **kw):
    a = dict(Pq=PQ, Pk=PK, Pv=PV, alpha_k=0.9, alpha_v=0.9, rope=ROPE, rope_positions=100, rope_dim=128,
             rope_interleaved=0)
    a.update(kw)
    return kq._KVTransformStruct(*a.values())


def ref(x):
    return None if x is None else ctypes.addressof(x)


def append(kq, c=None, t=None, no=(), **kw):
    a = dict(q=Q, qs=1024, k=K, ks=256, v=V, vs=256, pos=POS, slot=SLOT, qo=QO, T=8, H=8)
    a.update(kw)
    c, t = c or cache(kq), t or transform(kq)
    return kq.lib.kq_kv_append(None if "cache" in no else ref(c), None if "tf" in no else ref(t), a["q"], a["qs"], a["k"],
                               a["ks"], a["v"], a["vs"], a["pos"], a["slot"], a["qo"], a["T"], a["H"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(num_pages=0), "SHAPE"), (dict(num_pages=2 ** 31), "SHAPE"), (dict(kv_heads=0), "SHAPE"),
    (dict(kv_heads=1025), "SHAPE"), (dict(head_dim=0), "SHAPE"), (dict(head_dim=96), "UNSUPPORTED"),
    (dict(head_dim=256), "UNSUPPORTED"), (dict(page_size=0), "SHAPE"), (dict(page_size=8), "UNSUPPORTED"),
    (dict(page_size=48), "UNSUPPORTED"), (dict(page_size=512), "UNSUPPORTED"), (dict(k_codes=None), "NULL"),
    (dict(v_scale=None), "NULL"), (dict(k_scale=KS + 8), "ALIGN"), (dict(v_codes=VC + 4), "ALIGN")])
def test_cache_descriptions_that_are_refused(kq, kw, status):
    want = getattr(kq, "KQ_ERR_" + status)
    c = cache(kq, **kw)
    assert append(kq, c, ks=4096 * 256, vs=4096 * 256) == want
    assert kq.lib.kq_kv_gather(ref(c), SLOT, K, V, 4, None) == want
    assert attend(kq, c) == want


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), "SHAPE"), (dict(H=-1), "SHAPE"), (dict(H=1025), "SHAPE"), (dict(T=2 ** 31 // 10), "SHAPE"),
    (dict(q=None), "NULL"), (dict(k=None), "NULL"), (dict(v=None), "NULL"), (dict(pos=None), "NULL"),
    (dict(slot=None), "NULL"), (dict(qo=None), "NULL"), (dict(qs=1016), "ARG"), (dict(ks=248), "ARG"),
    (dict(vs=0), "ARG"), (dict(vs=2 ** 40), "ARG"), (dict(qs=1028), "ALIGN"), (dict(ks=260), "ALIGN"),
    (dict(q=Q + 2), "ALIGN"), (dict(k=K + 8), "ALIGN"), (dict(qo=QO + 8), "ALIGN"), (dict(slot=SLOT + 4), "ALIGN"),
    (dict(pos=POS + 2), "ALIGN"), (dict(qo=Q + 64), "ARG"), (dict(qo=PK), "ARG"), (dict(qo=KC + 64), "ARG"),
    (dict(k=VS), "ARG"), (dict(slot=KS), "ARG")])
def test_append_refusals(kq, kw, status):
    assert append(kq, **kw) == getattr(kq, "KQ_ERR_" + status)


@pytest.mark.parametrize("kw,status", [
    (dict(alpha_k=0.0), "ARG"), (dict(alpha_v=1.01), "ARG"), (dict(alpha_k=math.nan), "ARG"),
    (dict(alpha_v=1e-7), "UNSUPPORTED"), (dict(rope_dim=0), "SHAPE"), (dict(rope_dim=144), "SHAPE"),
    (dict(rope_dim=24), "UNSUPPORTED"), (dict(rope_positions=0), "SHAPE"), (dict(Pk=None), "NULL"),
    (dict(Pq=None), "NULL"), (dict(Pv=PV + 8), "ALIGN"), (dict(rope=ROPE + 4), "ALIGN"), (dict(Pv=KC), "ARG")])
def test_append_transform_refusals(kq, kw, status):
    assert append(kq, t=transform(kq, **kw)) == getattr(kq, "KQ_ERR_" + status)


def test_append_empty_and_null(kq):
    assert append(kq, T=0, no=("cache", "tf"), q=None, k=None, v=None, pos=None, slot=None, qo=None) == kq.KQ_OK
    assert append(kq, no=("cache",)) == kq.KQ_ERR_NULL and append(kq, no=("tf",)) == kq.KQ_ERR_NULL
    # one part of the cache over another
    assert append(kq, cache(kq, v_codes=KC + 4096)) == kq.KQ_ERR_ARG


def test_gather_refusals(kq):
    f, c = kq.lib.kq_kv_gather, cache(kq)
    assert f(ref(c), SLOT, K, V, -1, None) == kq.KQ_ERR_SHAPE
    assert f(ref(c), SLOT, K, V, 2 ** 30, None) == kq.KQ_ERR_SHAPE
    assert f(None, None, None, None, 0, None) == kq.KQ_OK
    assert f(None, SLOT, K, V, 3, None) == kq.KQ_ERR_NULL
    for bad in ((None, K, V), (SLOT, None, V), (SLOT, K, None)):
        assert f(ref(c), *bad, 3, None) == kq.KQ_ERR_NULL
    for bad in ((SLOT + 4, K, V), (SLOT, K + 8, V), (SLOT, K, V + 2)):
        assert f(ref(c), *bad, 3, None) == kq.KQ_ERR_ALIGN
    for bad in ((SLOT, K, K + 512), (SLOT, KC, V), (SLOT, K, SLOT - 16)):
        assert f(ref(c), *bad, 3, None) == kq.KQ_ERR_ARG


def attend(kq, c=None, shared=False, no_cache=False, **kw):
    a = dict(q=Q, qs=QS, pre=PRE, plen=40, tab=TAB, pages=5, len=LEN, scale=0.1, cap=0.0, window=0, out=OUT, lse=LSE,
             ws=WS, bytes=1 << 40, T=6, B=3, H=8, max_q=3)
    a.update(kw)
    c = c or cache(kq)
    head = (None if no_cache else ref(c), a["q"], a["qs"])
    tail = (a["tab"], a["pages"], a["len"], a["scale"], a["cap"], a["window"], a["out"], a["lse"], a["ws"], a["bytes"],
            a["T"], a["B"], a["H"], a["max_q"], None)
    if shared:
        return kq.lib.kq_kv_attention_shared(*head, a["pre"], a["plen"], *tail)
    return kq.lib.kq_kv_attention(*head, *tail)


@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), "SHAPE"), (dict(B=-1), "SHAPE"), (dict(H=0), "SHAPE"), (dict(H=7), "SHAPE"), (dict(H=1026), "SHAPE"),
    (dict(B=65536), "SHAPE"), (dict(qs=None), "SHAPE"), (dict(pages=0), "SHAPE"), (dict(pages=2 ** 27), "SHAPE"),
    (dict(T=2 ** 29, B=1), "SHAPE"), (dict(scale=math.inf), "ARG"), (dict(scale=math.nan), "ARG"), (dict(scale=3e38), "ARG"), (dict(cap=3e38), "ARG"),
    (dict(scale=1.0, cap=1e-39), "ARG"),
    (dict(cap=-1.0), "ARG"), (dict(cap=math.inf), "ARG"), (dict(window=-1), "ARG"), (dict(max_q=0), "ARG"),
    (dict(q=None), "NULL"), (dict(tab=None), "NULL"), (dict(len=None), "NULL"), (dict(out=None), "NULL"),
    (dict(ws=None), "NULL"), (dict(q=Q + 8), "ALIGN"), (dict(out=OUT + 2), "ALIGN"), (dict(ws=WS + 8), "ALIGN"),
    (dict(tab=TAB + 2), "ALIGN"), (dict(len=LEN + 1), "ALIGN"), (dict(qs=QS + 2), "ALIGN"), (dict(lse=LSE + 2), "ALIGN"),
    (dict(bytes=0), "ARG"), (dict(out=Q), "ARG"), (dict(lse=OUT + 256), "ARG"), (dict(ws=TAB), "ARG"),
    (dict(ws=OUT + 1024), "ARG"), (dict(out=KC), "ARG"), (dict(lse=VS), "ARG"), (dict(ws=LEN), "ARG")])
def test_attention_refusals(kq, kw, status, shared):
    assert attend(kq, shared=shared, **kw) == getattr(kq, "KQ_ERR_" + status)


def test_attention_empty_null_and_prefix(kq):
    assert attend(kq, T=0, B=0, q=None, out=None, ws=None, no_cache=True) == kq.KQ_OK
    assert attend(kq, no_cache=True) == kq.KQ_ERR_NULL
    assert attend(kq, shared=True, plen=-1) == kq.KQ_ERR_SHAPE
    assert attend(kq, shared=True, plen=2 ** 30) == kq.KQ_ERR_SHAPE
    assert attend(kq, shared=True, pre=None) == kq.KQ_ERR_NULL
    assert attend(kq, shared=True, pre=PRE + 2) == kq.KQ_ERR_ALIGN
    assert attend(kq, shared=True, out=PRE) == kq.KQ_ERR_ARG


def test_workspace_bytes(kq):
    f = kq.kq_kv_attention_workspace_bytes
    assert f(6, 3, 8, 2, 128, 3) > 0
    assert f(0, 3, 8, 2, 128, 3) == 0 and f(6, 0, 8, 2, 128, 3) == 0
    for bad in ((6, 3, 7, 2, 128, 3), (6, 3, 8, 2, 96, 3), (6, 3, 8, 2, 128, 0), (2 ** 30, 3, 8, 2, 128, 1)):
        assert f(*bad) == 0
    n = f(6, 3, 8, 2, 128, 3)
    assert attend(kq, bytes=n - 1) == kq.KQ_ERR_ARG and attend(kq, shared=True, bytes=n - 1) == kq.KQ_ERR_ARG


def test_handles_check_their_tensors(kq):
    import torch
    codes, scale = torch.zeros(3, 2, 16, 64, dtype=torch.uint8), torch.zeros(3, 2, 16)
    with pytest.raises(ValueError):
        kq.kv_cache(codes, scale, codes, scale)          # not on a CUDA device
    with pytest.raises(ValueError):
        kq.kv_cache(codes, scale.double(), codes, scale)
    with pytest.raises(ValueError):
        kq.kv_cache(codes, scale[:, :, :8], codes, scale)
    with pytest.raises(ValueError):
        kq.kv_cache(codes.int(), scale, codes, scale)
    P = torch.zeros(64, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        kq.kv_transform(P, P, P, 0.9, 0.9)               # not on a CUDA device
    with pytest.raises(ValueError):
        kq.kv_transform(P, P, P[:32], 0.9, 0.9)
    with pytest.raises(ValueError):
        kq.kv_transform(P, P, P, 0.9, 0.9, rope=torch.zeros(4, 64, dtype=torch.float64))


def test_weight_helpers_refuse(kq):
    from kronecker_factored_transforms_b200 import weights
    with pytest.raises(ValueError):
        weights.fold_value_factor(np.zeros((4, 100)), np.zeros((64, 64), np.uint16))
    with pytest.raises(ValueError):
        weights.query_factor_bf16(np.zeros((64, 64), np.uint16))
