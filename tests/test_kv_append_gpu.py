"""kq_kv_append and kq_kv_gather against their 64-bit forms: rotated and transformed
queries, INT4 rows of keys and values at their slots, and nothing else written."""
import numpy as np
import pytest
import torch

from kv_testutil import quantise, rotate, unpack

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kq():
    from kronecker_factored_transforms_b200 import _lib
    return _lib


def make(T, H, Hk, D, page, rope, seed, packed=True, extra_pages=2, positions=4096):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")
    P = [torch.linalg.qr(rn(D, D).double())[0] for _ in range(2)]
    d = torch.exp(0.1 * rn(D).double())
    s = dict(T=T, H=H, Hk=Hk, D=D, page=page, rope=rope)
    s["Pk"], s["Pq"], s["Pv"] = [x.to(torch.bfloat16).contiguous() for x in (P[0] * d, P[0] / d, P[1])]
    if packed:
        qkv = rn(T, H + 2 * Hk, D)
        qkv[:, H:H + Hk, 5] *= 20.0  # a large channel of the keys
        qkv = qkv.to(torch.bfloat16)
        s["q"], s["k"], s["v"] = qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:]
    else:
        s["q"], s["k"], s["v"] = [rn(T, h, D).to(torch.bfloat16) for h in (H, Hk, Hk)]
    pages = (T + page - 1) // page + extra_pages
    s["slots"] = torch.randperm(pages * page, generator=g, device="cuda")[:T]
    s["positions"] = torch.randint(0, positions, (T,), generator=g, device="cuda").to(torch.int32)
    s["table"] = None
    if rope:
        ang = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * \
            10000.0 ** (-torch.arange(rope // 2, device="cuda", dtype=torch.float64) / (rope // 2))
        s["table"] = torch.cat([ang.cos(), ang.sin()], 1).float()
    s["pool"] = [torch.full((pages, Hk, page, D // 2), 0x5A, dtype=torch.uint8, device="cuda"),
                 torch.full((pages, Hk, page), -7.0, device="cuda"),
                 torch.full((pages, Hk, page, D // 2), 0xA5, dtype=torch.uint8, device="cuda"),
                 torch.full((pages, Hk, page), -9.0, device="cuda")]
    s["q_out"] = torch.full((T + 1, H, D), 3.0, dtype=torch.bfloat16, device="cuda")
    return s


def append(kq, s, alpha_k=0.9, alpha_v=0.8, inter=False, stream=None):
    s["cache"] = kq.kv_cache(*s["pool"])
    tf = kq.kv_transform(s["Pq"], s["Pk"], s["Pv"], alpha_k, alpha_v, rope=s["table"], interleaved=inter)
    s["tf"] = tf
    kq.kq_kv_append(s["cache"], tf, s["q"], s["q"].stride(0), s["k"], s["k"].stride(0), s["v"], s["v"].stride(0),
                    s["positions"] if s["rope"] else None, s["slots"], s["q_out"], s["T"], s["H"], stream=stream)


def check(s, alpha_k=0.9, alpha_v=0.8, inter=False, skip=()):
    """skip: tokens whose keys and values are not stored."""
    torch.cuda.synchronize()
    T, H, Hk, D, page = s["T"], s["H"], s["Hk"], s["D"], s["page"]
    ang = s["table"][s["positions"].long()].double() if s["rope"] else None
    xq = rotate(s["q"].double(), ang, s["rope"], inter)
    ref = xq @ s["Pq"].double()
    # q_out: rounded once to bf16 (half a step 2^-8); a rotated element carried in 16 bits or more
    # (2^-16 of each product) and fp32 sums of D products
    bound = 2.0 ** -8 * ref.abs() + (2.0 ** -16 + D * 2.0 ** -24) * (xq.abs() @ s["Pq"].double().abs())
    assert ((s["q_out"][:T].double() - ref).abs() <= bound).all()
    assert (s["q_out"][T:] == 3.0).all(), "rows past T"
    written = torch.zeros(s["pool"][1].shape, dtype=torch.bool, device="cuda")
    keep = [t for t in range(T) if t not in set(skip)]
    slots = s["slots"][keep]
    pg, off = slots // page, slots % page
    for name, P, alpha, codes, scale, canary in (("k", s["Pk"], alpha_k, s["pool"][0], s["pool"][1], 0x5A),
                                                 ("v", s["Pv"], alpha_v, s["pool"][2], s["pool"][3], 0xA5)):
        x = s[name].double()
        if name == "k":
            x = rotate(x, ang, s["rope"], inter)
        c_ref, s_ref, dist = quantise((x @ P.double())[keep], alpha)
        c = unpack(codes[pg, :, off])
        sure = dist > 1e-9  # fp64's own rounding decides nearer to a border
        assert torch.equal(c[sure], c_ref[sure]), "%s codes: %d differ" % (name, int((c != c_ref)[sure].sum()))
        assert ((c - c_ref).abs() <= 1).all()
        sc = scale[pg, :, off].double()
        # alpha / 7 of the largest of D sums of D products in fp32: each of D + 8 additions may lose a whole step
        # (2^-23, where the tensor core truncates) of the products' absolute sum; and the scale's own roundings
        size = (x.abs() @ P.double().abs()).amax(-1)[keep]
        bound = alpha / 7 * (D + 8) * 2.0 ** -23 * size + 2.0 ** -22 * s_ref
        assert ((sc - s_ref).abs() <= bound).all(), name
        mask = torch.zeros_like(written)
        mask[pg, :, off] = True
        assert (codes[~mask] == canary).all(), "%s codes outside the slots" % name
        assert (scale[~mask] == (-7.0 if name == "k" else -9.0)).all(), "%s scales outside the slots" % name


@pytest.mark.parametrize("T,H,Hk,D,page,rope,inter", [
    (1, 32, 8, 128, 16, 128, False), (1, 1, 1, 64, 16, 64, True), (3, 5, 5, 128, 32, 0, False),
    (17, 14, 2, 128, 16, 64, True), (67, 28, 4, 128, 64, 128, True), (130, 12, 12, 64, 16, 32, False),
    (257, 8, 1, 128, 256, 16, False), (1000, 6, 3, 64, 128, 48, True), (2051, 16, 8, 128, 16, 128, False),
    (40011, 2, 1, 128, 16, 112, False), (9000, 4, 2, 64, 16, 48, False), (30000, 1, 1, 128, 16, 128, True)])
def test_append(kq, T, H, Hk, D, page, rope, inter):
    s = make(T, H, Hk, D, page, rope, T * 7 + H)
    append(kq, s, inter=inter)
    check(s, inter=inter)
    assert kq.kq_device_error() == 0


@pytest.mark.parametrize("alpha_k,alpha_v", [(1.0, 0.5), (0.97, 2.0 ** -19), (0.013, 1.0)])
def test_append_clip_ratios(kq, alpha_k, alpha_v):
    s = make(200, 8, 4, 128, 16, 128, 5)
    append(kq, s, alpha_k, alpha_v)
    check(s, alpha_k, alpha_v)


def test_append_dense_rows(kq):
    s = make(90, 8, 4, 64, 16, 64, 6, packed=False)
    append(kq, s)
    check(s)


def test_append_without_queries(kq):
    s = make(33, 4, 4, 128, 16, 128, 7)
    cache = kq.kv_cache(*s["pool"])
    tf = kq.kv_transform(None, s["Pk"], s["Pv"], 0.9, 0.8, rope=s["table"])
    kq.kq_kv_append(cache, tf, None, 0, s["k"], s["k"].stride(0), s["v"], s["v"].stride(0), s["positions"],
                    s["slots"], None, s["T"], 0)
    s["H"], s["q"], s["q_out"] = 0, s["q"][:, :0], s["q_out"][:, :0]
    check(s)


def test_append_zero_and_extreme_rows(kq):
    """Zero rows have scale 0 and codes 0; very large and very small rows keep their codes."""
    s = make(40, 4, 2, 128, 16, 0, 8)
    s["k"][3] = 0
    s["v"][5, 1] = 0
    s["k"][7] = (s["k"][7].float() * 1e30).to(torch.bfloat16)
    s["v"][9] = (s["v"][9].float() * 1e-30).to(torch.bfloat16)
    append(kq, s)
    check(s)
    pg, off = s["slots"] // s["page"], s["slots"] % s["page"]
    assert (s["pool"][1][pg[3], :, off[3]] == 0).all() and (s["pool"][0][pg[3], :, off[3]] == 0).all()
    assert s["pool"][3][pg[5], 1, off[5]] == 0


def test_append_values_on_borders(kq):
    """Rows whose values meet rounding borders exactly (halves go to the even code) or miss them by
    less than fp32 tells: an identity factor, alpha = 1, the largest value 7 steps."""
    s = make(6, 2, 1, 128, 16, 0, 9)
    s["Pk"] = s["Pv"] = s["Pq"] = torch.eye(128, device="cuda").to(torch.bfloat16)
    v = torch.zeros(128)
    v[0] = 7.0
    v[1:14] = torch.arange(13) - 6.5
    s["v"][:, 0] = v.cuda().to(torch.bfloat16)
    s["k"][:, 0] = (2.0 ** -40 * v).cuda().to(torch.bfloat16)
    append(kq, s, 1.0, 1.0)
    torch.cuda.synchronize()
    want = torch.round(v)  # halves to even
    pg, off = s["slots"] // s["page"], s["slots"] % s["page"]
    assert torch.equal(unpack(s["pool"][2][pg, 0, off]).cpu(), want.double().expand(6, 128))
    assert torch.equal(unpack(s["pool"][0][pg, 0, off]).cpu(), want.double().expand(6, 128))


def test_append_near_borders(kq):
    """Values a few 2^-26 of the maximum beside a border: the codes are still those of exact arithmetic.
    Element 1 of each row sums two products that place it there (a factor with two entries in column 1)."""
    T = 64
    s = make(T, 2, 1, 128, 16, 0, 10)
    P = torch.eye(128, dtype=torch.float64)
    P[2, 1] = 2.0 ** -26  # y_1 = x_1 + 2^-26 x_2
    s["Pk"] = s["Pv"] = s["Pq"] = P.cuda().to(torch.bfloat16)
    x = torch.zeros(T, 128)
    x[:, 0] = 7.0
    x[:, 1] = 2.5
    x[:, 2] = torch.where(torch.arange(T) % 2 == 0, 1.0, -1.0)
    s["v"][:, 0] = x.cuda().to(torch.bfloat16)
    s["k"][:, 0] = -s["v"][:, 0]
    append(kq, s, 1.0, 1.0)
    torch.cuda.synchronize()
    pg, off = s["slots"] // s["page"], s["slots"] % s["page"]
    want = torch.where(torch.arange(T) % 2 == 0, 3.0, 2.0).double()  # 2.5 + 2^-26 and 2.5 - 2^-26
    assert torch.equal(unpack(s["pool"][2][pg, 0, off])[:, 1].cpu(), want)
    assert torch.equal(unpack(s["pool"][0][pg, 0, off])[:, 1].cpu(), -want)


def test_append_padding_and_refused_indexes(kq):
    s = make(50, 4, 2, 128, 16, 128, 11)
    assert kq.kq_device_error() == 0
    s["slots"][[4, 9, 49]] = torch.tensor([-1, -5, -2 ** 62], device="cuda")
    append(kq, s)
    check(s, skip=(4, 9, 49))
    assert kq.kq_device_error() == 0  # padding is no error
    s = make(50, 4, 2, 128, 16, 128, 12)
    n = s["pool"][0].shape[0] * 16
    s["slots"][[3, 40]] = torch.tensor([n, 2 ** 40], device="cuda")
    append(kq, s)
    check(s, skip=(3, 40))
    assert kq.kq_device_error() == 65536 and kq.kq_device_error() == 0
    s = make(50, 4, 2, 128, 16, 128, 13)
    good = s["positions"].clone()
    s["positions"][[0, 20]] = torch.tensor([-1, 4096], dtype=torch.int32, device="cuda")
    append(kq, s)
    torch.cuda.synchronize()
    assert (s["q_out"][[0, 20]] == 0).all()
    s["positions"] = good
    s["q"], s["q_out"] = s["q"].clone(), s["q_out"].clone()
    s["q"][[0, 20]] = 0
    check(s, skip=(0, 20))
    assert kq.kq_device_error() == 65536


def test_append_nan_stays_in_its_row(kq):
    s = make(20, 4, 2, 128, 16, 128, 14)
    s["k"][6, 1, 17] = float("nan")
    s["v"][8, 0, 3] = float("inf")
    append(kq, s)
    t = make(20, 4, 2, 128, 16, 128, 14)
    append(kq, t)
    torch.cuda.synchronize()
    pg, off = s["slots"] // 16, s["slots"] % 16
    same = torch.ones_like(s["pool"][1], dtype=torch.bool)
    same[pg[6], 1, off[6]] = False
    assert torch.equal(s["pool"][0][same], t["pool"][0][same]) and torch.equal(s["pool"][1][same], t["pool"][1][same])
    same = torch.ones_like(same)
    same[pg[8], 0, off[8]] = False
    assert torch.equal(s["pool"][2][same], t["pool"][2][same]) and torch.equal(s["pool"][3][same], t["pool"][3][same])


@pytest.mark.parametrize("T,Hk,D,page", [(1, 8, 128, 16), (37, 3, 64, 32), (1000, 8, 128, 64)])
def test_gather(kq, T, Hk, D, page):
    s = make(T, Hk, Hk, D, page, 0, 15 + T)
    append(kq, s)
    slots = s["slots"][torch.randint(0, T, (2 * T + 3,), device="cuda")]  # repeated slots
    slots[1::5] = -3
    n = slots.numel()
    k = torch.full((n + 1, Hk, D), 2.0, dtype=torch.bfloat16, device="cuda")
    v = torch.full_like(k, 4.0)
    kq.kq_kv_gather(s["cache"], slots, k, v, n)
    torch.cuda.synchronize()
    ok = (slots >= 0)[:, None, None]
    at = slots.clamp(min=0)
    for got, codes, scale, tail in ((k, s["pool"][0], s["pool"][1], 2.0), (v, s["pool"][2], s["pool"][3], 4.0)):
        ref = unpack(codes[at // page, :, at % page]) * scale[at // page, :, at % page].double()[..., None]
        # fp32 holds code * s to 2^-24; bf16 to half a step
        assert ((got[:n].double() - torch.where(ok, ref, 0.0)).abs() <= (2.0 ** -8 + 2.0 ** -23) * ref.abs()).all()
        assert (got[:n][~ok.expand_as(ref)] == 0).all() and (got[n:] == tail).all()
    assert kq.kq_device_error() == 0
    slots[0] = s["pool"][0].shape[0] * page
    kq.kq_kv_gather(s["cache"], slots, k, v, n)
    torch.cuda.synchronize()
    assert (k[0] == 0).all() and kq.kq_device_error() == 65536


def test_append_past_32_bits(kq):
    """Rows whose byte offset in the codes is past 2^32."""
    Hk, D, page = 8, 128, 256
    pages = 2 ** 32 // (Hk * page * 64) + 40
    codes = [torch.empty(pages, Hk, page, D // 2, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.empty(pages, Hk, page, device="cuda") for _ in range(2)]
    s = make(100, 8, Hk, D, page, 128, 16)
    small = [x.clone() for x in s["pool"]]
    append(kq, s)
    s2 = dict(s, pool=[codes[0], scales[0], codes[1], scales[1]])
    shift = (pages - s["pool"][0].shape[0]) * page
    s2["slots"] = s["slots"] + shift
    append(kq, s2)
    torch.cuda.synchronize()
    a, b = s["slots"], s2["slots"]
    for x, y in zip(s["pool"], s2["pool"]):
        assert torch.equal(x[a // page, :, a % page], y[b // page, :, b % page])
    k, v = [torch.empty(2, 100, Hk, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    kq.kq_kv_gather(s["cache"], a, k[0], v[0], 100)
    kq.kq_kv_gather(s2["cache"], b, k[1], v[1], 100)
    torch.cuda.synchronize()
    assert torch.equal(k[0], k[1]) and torch.equal(v[0], v[1])
    del small


def test_append_on_a_side_stream_and_in_a_graph(kq):
    s, ref = make(300, 8, 4, 128, 16, 128, 17), make(300, 8, 4, 128, 16, 128, 17)
    append(kq, ref)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    append(kq, s, stream=side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(s["pool"], ref["pool"])) and torch.equal(s["q_out"], ref["q_out"])
    g = make(300, 8, 4, 128, 16, 128, 17)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        append(kq, g)
    for _ in range(2):
        for x in g["pool"]:
            x.zero_()
        graph.replay()
    torch.cuda.synchronize()
    at, page = g["slots"], 16
    for x, y in zip(g["pool"], ref["pool"]):
        assert torch.equal(x[at // page, :, at % page], y[at // page, :, at % page])
    assert torch.equal(g["q_out"], ref["q_out"])


def test_weight_helpers_match_the_factors(kq):
    """(q Pk^-T).(k Pk) = q.k and Wo' (o Pv) = Wo o, to the factors' bf16 rounding."""
    from kronecker_factored_transforms_b200 import weights, workloads
    rng = np.random.default_rng(3)
    D = 64
    Pk = workloads.f32_to_bf16_bits((np.linalg.qr(rng.standard_normal((D, D)))[0] * 1.1).astype(np.float32))
    F = workloads.bf16_bits_to_f32(weights.query_factor_bf16(Pk)).astype(np.float64)
    K = workloads.bf16_bits_to_f32(Pk).astype(np.float64)
    assert np.abs(F @ K.T - np.eye(D)).max() < 2.0 ** -8 * np.sqrt(D)
    Wo, o = rng.standard_normal((10, 3 * D)), rng.standard_normal(3 * D)
    Wf = weights.fold_value_factor(Wo, Pk)
    assert np.allclose(Wf @ (o.reshape(3, D) @ K).ravel(), Wo @ o, rtol=0, atol=1e-9)
