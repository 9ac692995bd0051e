"""kq_kv_attention and kq_kv_attention_shared against their 64-bit forms."""
import math

import pytest
import torch

from kv_testutil import attention, check_attention

pytestmark = pytest.mark.gpu
CODES = torch.tensor([-8, -7, -5, -4, -3, -2, -1, -1, 0, 0, 1, 2, 3, 4, 5, 7])


@pytest.fixture(scope="module")
def kq():
    from kronecker_factored_transforms_b200 import _lib
    return _lib


def make(keys, nqs, G, Hk, D, page, seed, prefix=0, q_std=1.5, spare=2, scale_mid=0.3, scale_spread=0.25, mean=0.0):
    """Pools with NaN scales everywhere that no key lies, page tables in any order with
    out-of-range numbers behind the used entries, padded rows behind the last sequence."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, T = len(keys), sum(nqs)
    need = [(n + page - 1) // page for n in keys]
    pre = (prefix + page - 1) // page
    total = sum(need) + pre + spare
    perm = torch.randperm(total, generator=g, device="cuda").cpu()
    lut = (CODES & 15).to(torch.uint8).cuda()
    pool = []
    used = torch.zeros(total, page, dtype=torch.bool)
    tables, at = [], 0
    for n, k in zip(keys, need):
        tables.append(perm[at:at + k].tolist())
        for j, p in enumerate(tables[-1]):
            used[p, :min(page, n - j * page)] = True
        at += k
    prefix_pages = perm[at:at + pre].tolist()
    for j, p in enumerate(prefix_pages):
        used[p, :min(page, prefix - j * page)] = True
    hide = ~used.cuda()[:, None, :].expand(total, Hk, page)
    for _ in range(2):
        idx = torch.randint(0, 256, (total, Hk, page, D // 2), generator=g, device="cuda", dtype=torch.int32)
        pool.append(lut[idx >> 4] << 4 | lut[idx & 15])
        sc = scale_mid * torch.exp(scale_spread * torch.randn(total, Hk, page, generator=g, device="cuda"))
        sc[hide] = float("nan")
        pool.append(sc)
    width = max(1, max(need)) + 1
    table = torch.full((B, width), 0x7FFFFFF0, dtype=torch.int32)
    for b, t in enumerate(tables):
        table[b, :len(t)] = torch.tensor(t, dtype=torch.int32)
    q = (mean + q_std * torch.randn(T + 3, G * Hk, D, generator=g, device="cuda")).to(torch.bfloat16)
    q[T:] = float("nan")
    return dict(keys=list(keys), nqs=list(nqs), G=G, Hk=Hk, D=D, page=page, B=B, T=T, pool=pool, tables=tables,
                table=table.cuda(), width=width, q=q, prefix=prefix,
                prefix_pages=torch.tensor(prefix_pages + [-9], dtype=torch.int32).cuda(), prefix_list=prefix_pages,
                kv_len=torch.tensor(keys, dtype=torch.int32).cuda(),
                q_start=torch.tensor([0] + list(nqs)).cumsum(0).to(torch.int32).cuda(),
                scale=1.0 / math.sqrt(D))


def launch(kq, s, softcap=0.0, window=0, lse=True, q_start=True, max_q=None, out=None, workspace=None, T=None,
           shared=None, stream=None):
    H, T = s["G"] * s["Hk"], s["T"] + 3 if T is None else T
    max_q = max(max_q or 0, max(s["nqs"]))
    s["cache"] = kq.kv_cache(*s["pool"])
    if out is None:
        out = torch.full((s["T"] + 3, H, s["D"]), 5.0, dtype=torch.bfloat16, device="cuda")
    l = torch.full((s["T"] + 3, H), 6.0, device="cuda") if lse else None
    n = kq.kq_kv_attention_workspace_bytes(T, s["B"], H, s["Hk"], s["D"], max_q)
    if workspace is None:  # no initial contents are needed: every byte set, as NaN and huge integers
        workspace = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    qs = s["q_start"] if q_start else None
    if shared is None:
        shared = s["prefix"] > 0
    if shared:
        kq.kq_kv_attention_shared(s["cache"], s["q"], qs, s["prefix_pages"], s["prefix"], s["table"], s["width"],
                                  s["kv_len"], s["scale"], softcap, window, out, l, workspace, n, T, s["B"], H, max_q,
                                  stream=stream)
    else:
        kq.kq_kv_attention(s["cache"], s["q"], qs, s["table"], s["width"], s["kv_len"], s["scale"], softcap, window,
                           out, l, workspace, n, T, s["B"], H, max_q, stream=stream)
    return out, l


def verify(kq, s, softcap=0.0, window=0, **kw):
    out, lse = launch(kq, s, softcap, window, **kw)
    torch.cuda.synchronize()
    T = s["T"]
    assert (out[T:] == 5.0).all() and (lse is None or (lse[T:] == 6.0).all()), "rows behind the last sequence"
    ref = attention(s["q"][:T], s["pool"], s["tables"], s["keys"], s["nqs"], s["scale"], softcap, window,
                    (s["prefix_list"], s["prefix"]) if s["prefix"] else None)
    check_attention(out[:T], None if lse is None else lse[:T], ref)
    assert kq.kq_device_error() == 0
    return out, lse


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 3, 5, 8, 12, 16, 24])
def test_single_tokens_of_every_group_size(kq, D, G):
    keys = [1, 2, 15, 16, 17, 0, 63, 64, 65, 127, 128, 129, 300, 1000]
    verify(kq, make(keys, [1] * len(keys), G, 2, D, 16, 100 * G + D))


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_page_sizes(kq, page):
    verify(kq, make([5, 255, 256, 257, 700], [1] * 5, 4, 3, 128, page, page))


@pytest.mark.parametrize("keys", [[1], [16], [1531], [4096], [33333], [0], [0, 0, 0], [9000, 1, 1, 1, 1, 1, 0, 40]])
def test_lengths(kq, keys):
    verify(kq, make(keys, [1] * len(keys), 4, 8, 128, 16, sum(keys)))


def test_long_context(kq):
    verify(kq, make([131072 + 5, 70001], [1, 1], 4, 2, 128, 64, 3, q_std=0.7))


def test_many_sequences(kq):
    keys = [(i * 37) % 211 for i in range(700)]
    verify(kq, make(keys, [1] * 700, 2, 1, 64, 16, 4))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G,nqs,keys", [
    (1, [2, 3, 1, 5, 4], [2, 100, 1, 5, 333]), (4, [5, 1, 2, 4], [700, 64, 2, 4]), (8, [2, 2, 1], [50, 2, 129]),
    (3, [8, 7, 1, 2], [9, 500, 0, 2]), (2, [16, 9, 0, 1], [77, 12, 30, 5]), (16, [1, 4, 2], [10, 400, 3])])
def test_a_few_queries(kq, D, G, nqs, keys):
    verify(kq, make(keys, nqs, G, 2, D, 32, 10 * G + D))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G,nqs,keys", [
    (1, [200], [200]), (4, [129, 64], [129, 1000]), (8, [33, 100, 1], [4000, 100, 7]), (3, [170], [555]),
    (16, [40, 41], [41, 41]), (7, [300], [1700]), (2, [1, 400, 0, 30], [900, 401, 10, 31])])
def test_chunks_of_prompts(kq, D, G, nqs, keys):
    verify(kq, make(keys, nqs, G, 2, D, 16, 10 * G + D + 1))


@pytest.mark.parametrize("page", [32, 64, 128, 256])
def test_chunks_on_pages_of_any_size(kq, page):
    verify(kq, make([700, 90, 257], [70, 90, 1], 4, 2, 128, page, page))
    verify(kq, make([700, 90, 257], [70, 90, 100], 2, 3, 64, page, page + 1, prefix=301), window=200)


@pytest.mark.parametrize("G,nqs,keys", [(1024, [1, 1], [300, 17]), (128, [1, 3, 1], [129, 300, 1]), (49, [1], [700])])
def test_one_key_head_of_many_query_heads(kq, G, nqs, keys):
    verify(kq, make(keys, nqs, G, 1, 128, 16, G))
    verify(kq, make(keys, nqs, G, 1, 64, 16, G, prefix=200), softcap=9.0)


@pytest.mark.parametrize("G,D,nqs,keys,kw", [
    (4, 128, [8192], [8192], {}), (8, 64, [5000, 1, 3000, 1, 1], [5100, 7000, 3000, 1, 9000], dict(window=700)),
    (2, 128, [40, 64], [131072, 100001], {}), (1, 128, [20000], [21003], dict(softcap=20.0)),
    (4, 64, [1] * 300 + [2000], [500] * 300 + [2000], {})])
def test_long_prompts(kq, G, D, nqs, keys, kw):
    """Many row tiles, and many keys for a few; sampled queries as sequences of their own against the 64-bit form."""
    s = make(keys, nqs, G, 2, D, 64, len(nqs) + D)
    out, lse = launch(kq, s, **kw)
    torch.cuda.synchronize()
    assert kq.kq_device_error() == 0 and (out[s["T"]:] == 5.0).all()
    g = torch.Generator().manual_seed(sum(nqs))
    b = [0, len(nqs) - 1] + torch.randint(len(nqs), (22,), generator=g).tolist()
    i = [0, nqs[-1] - 1] + [int(torch.randint(nqs[x], (1,), generator=g)) for x in b[2:]]
    at = [sum(nqs[:x]) + y for x, y in zip(b, i)]
    ref = attention(s["q"][at], s["pool"], [s["tables"][x] for x in b], [keys[x] - nqs[x] + y + 1 for x, y in zip(b, i)],
                    [1] * len(at), s["scale"], kw.get("softcap", 0.0), kw.get("window", 0))
    check_attention(out[at], lse[at], ref)


def spread(keys, nqs):
    """As many keys as queries at least, and more for some."""
    return [max(m, (keys * (i % 5)) // 4 + i) for i, m in enumerate(nqs)]


@pytest.mark.parametrize("D,G,nqs,keys,kw", [
    (128, 4, [1, 1, 200, 1, 2], 400, {}), (64, 4, [12, 13, 1, 0, 1, 100, 1, 1], 300, {}),
    (128, 4, [1] * 40 + [90] + [1] * 10, 700, {}), (64, 8, [3, 0, 7, 6, 1] * 9 + [300], 500, dict(window=60)),
    (128, 2, [1, 600, 1, 1], 9000, dict(softcap=8.0)), (128, 4, [1] * 30 + [150, 20] + [1] * 30, 500, dict(prefix=333)),
    (64, 50, [1] * 20 + [8] + [1] * 20, 200, {}), (128, 4, [100] + [61] * 35, 150, {}),
    (64, 1, [49] + [48, 1, 1, 1] * 12, 100, dict(prefix=50, window=90))])
def test_prompts_and_single_tokens_at_once(kq, D, G, nqs, keys, kw):
    """Sequences with few rows and with many, each for its own kernel."""
    kw = dict(kw)
    s = make(spread(keys, nqs), nqs, G, 2, D, 16, len(nqs) + G, prefix=kw.pop("prefix", 0))
    verify(kq, s, **kw)
    verify(kq, s, max_q=max(nqs) + 37, **kw)


def test_single_tokens_under_a_high_bound(kq):
    nqs = [1] * 70
    verify(kq, make(spread(600, nqs), nqs, 4, 2, 128, 16, 31), max_q=4096)


@pytest.mark.parametrize("nqs,keys", [([4, 3], [2, 0]), ([1, 20], [0, 5]), ([200], [150]), ([64, 64], [0, 1])])
def test_more_queries_than_keys(kq, nqs, keys):
    """The first queries see nothing: zeros and -infinity."""
    verify(kq, make(keys, nqs, 4, 2, 128, 16, 8))


@pytest.mark.parametrize("window", [1, 7, 16, 64, 100, 1000, 100000])
def test_windows(kq, window):
    verify(kq, make([1, 17, 100, 700, 1500], [1] * 5, 4, 2, 128, 16, window), window=window)
    verify(kq, make([50, 17, 100, 700], [3, 5, 1, 4], 2, 2, 64, 32, window), window=window)
    verify(kq, make([150, 900], [150, 200], 4, 2, 128, 16, window), window=window)


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 100])
@pytest.mark.parametrize("prefix", [0, 300])
def test_the_largest_windows(kq, window, prefix):
    """More queries than keys: a query's place less the window passes 32 bits."""
    verify(kq, make([2, 0, 40], [5, 3, 1], 4, 2, 64, 16, 21, prefix=prefix), window=window)
    verify(kq, make([100, 5], [150, 70], 4, 2, 64, 16, 22, prefix=prefix), window=window)


@pytest.mark.parametrize("prefix", [0, 300])
def test_more_sequences_than_tokens(kq, prefix):
    """Idle slots of a batch that bring no query."""
    verify(kq, make([40, 7, 0, 300, 5, 9], [0, 1, 0, 0, 1, 0], 4, 2, 128, 16, 23, prefix=prefix))
    verify(kq, make([40] * 90, [0] * 70 + [60] + [0] * 19, 4, 2, 128, 16, 24, prefix=prefix))


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("m,softcap", [(4, 0.0), (80, 0.0), (80, 20.0)])
def test_scales_of_rows_that_a_query_does_not_see(kq, bad, m, softcap):
    """A key that only the last query sees, and one before every window, do not reach the others."""
    keys, window = 300, 100
    s = make([keys], [m], 4, 2, 128, 16, 25)
    for t in (keys - 1, keys - m - window):
        for pool in (s["pool"][1], s["pool"][3]):
            pool[s["tables"][0][t // 16], :, t % 16] = bad
    out, lse = launch(kq, s, softcap, window)
    ref = attention(s["q"][:m], s["pool"], s["tables"], [keys], [m], s["scale"], softcap, window)
    check_attention(out[:m - 1], lse[:m - 1], [r[:m - 1] for r in ref])
    assert kq.kq_device_error() == 0


@pytest.mark.parametrize("nqs", [[1, 1, 3], [70, 90, 33]])
def test_pages_below_the_window_are_not_looked_at(kq, nqs):
    """A sliding-window cache gives such pages back: their entries may hold anything."""
    keys, window = [700, 300, 1500], 100
    s = make(keys, nqs, 4, 2, 128, 16, 77)
    for b, (n, m) in enumerate(zip(keys, nqs)):
        s["table"][b, :max(0, n - m - window + 1) // 16] = -7
    verify(kq, s, window=window)


@pytest.mark.parametrize("softcap", [0.5, 5.0, 30.0])
def test_capped_scores(kq, softcap):
    verify(kq, make([1, 17, 100, 700], [1] * 4, 4, 2, 128, 16, 5, q_std=6.0), softcap=softcap)
    verify(kq, make([150, 900], [150, 200], 4, 2, 64, 16, 6, q_std=6.0), softcap=softcap, window=90)


def test_scores_far_apart(kq):
    """Scores of hundreds: one key takes all the weight; and the largest score last or first."""
    for seed, keys, nqs in ((1, [400, 37], [1, 1]), (2, [300, 64], [130, 64])):
        s = make(keys, nqs, 4, 2, 128, 16, seed, q_std=40.0, scale_spread=1.0)
        verify(kq, s)


@pytest.mark.parametrize("softcap", [0.0, 150.0])
@pytest.mark.parametrize("nqs", [[1, 3], [70, 150], [2, 150]])
def test_scores_that_jump_on_the_way(kq, nqs, softcap):
    """Key scales that rise, or fall, by magnitudes inside a chunk of 128 keys and between chunks: the largest score so
    far is passed by hundreds, late in a long row."""
    steps = [(0, 1e-3), (300, 0.05), (555, 3.0), (640, 0.2), (1000, 12.0), (1663, 40.0)]
    for turn in (steps, [(t, f) for (t, _), (_, f) in zip(steps, steps[::-1])]):
        s = make([2100, 1700], nqs, 4, 2, 128, 16, 18)
        for b, n in enumerate(s["keys"]):
            for t in range(n):
                s["pool"][1][s["tables"][b][t // 16], :, t % 16] *= [f for at, f in turn if at <= t][-1]
        verify(kq, s, softcap=softcap)


@pytest.mark.parametrize("mid", [1e-12, 1e-4, 1e3, 1e8])
def test_value_scales_of_any_size(kq, mid):
    s = make([300, 20, 1], [1, 1, 1], 4, 2, 128, 16, 9)
    s["pool"][3] *= mid
    verify(kq, s)
    s = make([300, 90], [70, 90], 4, 2, 128, 16, 9)
    s["pool"][3] *= mid
    verify(kq, s)


def test_scales_that_differ_by_magnitudes_and_zero_rows(kq):
    for nqs in ([1, 1, 1], [80, 64, 33]):
        s = make([300, 64, 33], nqs, 4, 2, 128, 16, 10, scale_spread=3.0, q_std=0.05)
        s["pool"][3][:, :, 3::7] = 0  # rows that were all zero when they were stored
        s["pool"][1][:, :, 2::5] = 0
        s["pool"][2][:, :, 3::7] = 0
        verify(kq, s)
    s = make([40], [1], 4, 2, 128, 16, 11)
    s["pool"][3].zero_()
    s["pool"][2].zero_()
    verify(kq, s)


def test_queries_with_a_mean(kq):
    """All elements of a query of one sign: sums over the codes that do not cancel."""
    verify(kq, make([700, 64], [1, 1], 8, 2, 128, 16, 12, mean=3.0, q_std=0.1))
    verify(kq, make([700], [100], 8, 2, 128, 16, 13, mean=3.0, q_std=0.1))


@pytest.mark.parametrize("scale", [1e-30, 1e20])
def test_queries_of_any_size(kq, scale):
    """The softmax scale undoes the size of the queries."""
    for nqs in ([1, 1], [70, 90]):
        s = make([300, 90], nqs, 4, 2, 128, 16, 14)
        s["q"] = (s["q"].double() * scale).to(torch.bfloat16)
        s["scale"] = s["scale"] / scale
        verify(kq, s)


def test_zero_scale_and_negative_scale(kq):
    for nqs in ([1, 1], [70, 90]):
        for f in (0.0, -1.0):
            s = make([300, 90], nqs, 4, 2, 128, 16, 15)
            s["scale"] *= f
            verify(kq, s)


def test_optional_arguments(kq):
    s = make([50, 0, 17, 300], [1] * 4, 4, 2, 128, 16, 16)
    a, _ = verify(kq, s, lse=False)
    b, _ = verify(kq, s, max_q=7)  # a loose bound
    out, lse = launch(kq, s, q_start=False, T=4)
    torch.cuda.synchronize()
    check_attention(out[:4], lse[:4], attention(s["q"][:4], s["pool"], s["tables"], s["keys"], s["nqs"], s["scale"]))
    s = make([150, 90], [150, 20], 4, 2, 128, 16, 17)
    verify(kq, s, lse=False, max_q=153)


def test_negative_lengths_count_as_zero(kq):
    s = make([50, 0], [1, 1], 4, 2, 128, 16, 18)
    s["kv_len"][1] = -5
    verify(kq, s)


@pytest.mark.parametrize("nqs", [[1, 1, 1], [66, 70, 5]])
def test_refused_indexes_are_masked(kq, nqs):
    """Page numbers outside the cache, lengths past the table: those keys do not count, and the status says so."""
    s = make([200, 100, 300], nqs, 4, 2, 128, 16, 19)
    s["table"][0, 3] = s["pool"][0].shape[0]
    s["table"][2, 0] = -1
    s["table"][2, 18] = 0x7FFFFFFF
    out, lse = launch(kq, s)
    torch.cuda.synchronize()
    assert kq.kq_device_error() == 131072
    assert torch.isfinite(out[:s["T"]].float()).all()
    ok = s["q_start"][1:3].tolist()
    t = make([200, 100, 300], nqs, 4, 2, 128, 16, 19)
    ref = attention(t["q"][:t["T"]], t["pool"], t["tables"], t["keys"], t["nqs"], t["scale"])
    check_attention(out[ok[0]:ok[1]], lse[ok[0]:ok[1]], tuple(r[ok[0]:ok[1]] for r in ref))
    s = make([20], [nqs[0]], 4, 2, 128, 16, 20)
    s["kv_len"][0] = 10 ** 6
    s["table"][:] = s["tables"][0][0]
    s["pool"][1][torch.isnan(s["pool"][1])] = 1.0
    s["pool"][3][torch.isnan(s["pool"][3])] = 1.0
    out, _ = launch(kq, s)
    torch.cuda.synchronize()
    assert kq.kq_device_error() == 131072 and torch.isfinite(out[:s["T"]].float()).all()


def test_queries_past_the_bound_stay_beside_single_tokens(kq):
    nqs = [1, 300, 1, 1, 1, 90]
    s = make(spread(400, nqs), nqs, 4, 2, 128, 16, 32)
    T, H = s["T"] + 3, 8
    out = torch.full((T, H, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, H), 6.0, device="cuda")
    n = kq.kq_kv_attention_workspace_bytes(T, 6, H, 2, 128, 120)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    kq.kq_kv_attention(kq.kv_cache(*s["pool"]), s["q"], s["q_start"], s["table"], s["width"], s["kv_len"], s["scale"],
                       0.0, 0, out, lse, ws, n, T, 6, H, 120)
    torch.cuda.synchronize()
    assert kq.kq_device_error() == 131072
    ref = attention(s["q"][:s["T"]], s["pool"], s["tables"], s["keys"], nqs, s["scale"])
    done = torch.ones(T, dtype=torch.bool)
    done[1 + 120:1 + 300] = done[s["T"]:] = False
    assert (out[~done] == 5.0).all() and (lse[~done] == 6.0).all()
    check_attention(out[done], lse[done], [r[done[:s["T"]]] for r in ref])


def test_queries_past_the_bound_stay(kq):
    s = make([200, 100], [3, 1], 4, 2, 128, 16, 21)
    H = 8
    cache = kq.kv_cache(*s["pool"])
    n = kq.kq_kv_attention_workspace_bytes(4, 2, H, 2, 128, 2)
    out = torch.full((4, H, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    kq.kq_kv_attention(cache, s["q"], s["q_start"], s["table"], s["width"], s["kv_len"], s["scale"], 0.0, 0, out, None,
                       torch.empty(n, dtype=torch.uint8, device="cuda"), n, 4, 2, H, 2)
    torch.cuda.synchronize()
    assert kq.kq_device_error() == 131072
    ref = attention(s["q"][:4], s["pool"], s["tables"], s["keys"], s["nqs"], s["scale"])
    keep = [0, 1, 3]
    check_attention(out[keep], None, tuple(r[keep] for r in ref))
    assert (out[2] == 5.0).all()


# ---- a shared prefix ------------------------------------------------------------------

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G,Hk,B,prefix", [(1, 3, 2, 1), (4, 2, 8, 100), (8, 1, 3, 1000), (8, 2, 40, 515), (1, 4, 150, 300),
                                           (16, 1, 9, 64), (5, 2, 31, 129)])
def test_shared_prefix(kq, D, G, Hk, B, prefix):
    keys = [(i * 53) % 190 for i in range(B)]  # the first has no key of its own
    verify(kq, make(keys, [1] * B, G, Hk, D, 16, B + D + G, prefix=prefix))


@pytest.mark.parametrize("G,nqs,keys,prefix", [(4, [2, 1, 3], [5, 1, 300], 77), (2, [40, 1, 0, 9], [40, 0, 3, 200], 400),
                                               (8, [100, 30], [100, 500], 1500), (1, [3, 2], [1, 0], 33)])
def test_shared_prefix_with_several_queries(kq, G, nqs, keys, prefix):
    verify(kq, make(keys, nqs, G, 2, 128, 32, prefix, prefix=prefix))


@pytest.mark.parametrize("window", [1, 60, 200, 700])
def test_shared_prefix_windows_and_caps(kq, window):
    verify(kq, make([5, 0, 130, 500], [1, 1, 1, 1], 4, 2, 128, 16, window, prefix=450), window=window, softcap=20.0)
    verify(kq, make([5, 0, 130, 500] * 12, [1, 2, 1, 1] * 12, 4, 2, 64, 16, window, prefix=450), window=window)


def test_prefix_of_length_zero_and_equal_results(kq):
    s = make([50, 0, 17, 300], [1] * 4, 4, 2, 128, 16, 22)
    a, la = verify(kq, s)
    b, lb = verify(kq, s, shared=True)
    assert torch.equal(a, b) and torch.equal(la, lb)


@pytest.mark.parametrize("G,B,prefix", [(4, 5, 100), (2, 90, 700), (64, 3, 50)])
def test_shared_prefix_of_single_tokens_without_starts(kq, G, B, prefix):
    keys = [(7 * i) % 150 for i in range(B)]
    s = make(keys, [1] * B, G, 2, 128, 16, G + B, prefix=prefix)
    with_starts = launch(kq, s, T=B)
    without = launch(kq, s, T=B, q_start=False)
    torch.cuda.synchronize()
    assert torch.equal(with_starts[0], without[0]) and torch.equal(with_starts[1], without[1])
    ref = attention(s["q"][:B], s["pool"], s["tables"], keys, [1] * B, s["scale"], 0.0, 0, (s["prefix_list"], prefix))
    check_attention(without[0][:B], without[1][:B], ref)


def test_shared_prefix_long(kq):
    verify(kq, make([20, 300, 77, 0], [1, 1, 1, 1], 8, 2, 128, 16, 23, prefix=20000))
    verify(kq, make([20 + i for i in range(64)], [1] * 64, 8, 1, 128, 64, 24, prefix=9001))


def test_refused_prefix_pages(kq):
    s = make([5, 30], [1, 1], 4, 2, 128, 16, 25, prefix=200)
    s["prefix_pages"][4] = -1
    out, _ = launch(kq, s)
    torch.cuda.synchronize()
    assert kq.kq_device_error() == 131072 and torch.isfinite(out[:2].float()).all()


# ---- streams, graphs, order -----------------------------------------------------------

CASES = [dict(keys=[900, 33, 0, 410], nqs=[1] * 4, prefix=0), dict(keys=[700, 300], nqs=[90, 150], prefix=0),
         dict(keys=[20, 33, 0, 300] * 10, nqs=[1] * 40, prefix=600),
         dict(keys=[20, 700, 33, 300, 64], nqs=[1, 90, 1, 7, 2], prefix=0),
         dict(keys=[20, 700, 33, 300, 64], nqs=[1, 90, 1, 7, 2], prefix=200)]


@pytest.mark.parametrize("case", CASES)
def test_same_inputs_same_bits(kq, case):
    s = make(G=8, Hk=2, D=128, page=16, seed=30, **case)
    first = launch(kq, s)
    for _ in range(20):
        again = launch(kq, s)
        assert torch.equal(first[0][:s["T"]], again[0][:s["T"]]) and torch.equal(first[1], again[1])


def test_calls_in_a_row_on_one_workspace(kq):
    """Different batches one behind another, nothing between them: no call meets what another left."""
    sets = [make(G=8, Hk=2, D=128, page=16, seed=40 + i, **case) for i, case in enumerate(CASES)]
    alone = [[t.clone() for t in launch(kq, s)] for s in sets]
    torch.cuda.synchronize()
    most = max(kq.kq_kv_attention_workspace_bytes(s["T"] + 3, s["B"], 16, 2, 128, max(s["nqs"])) for s in sets)
    ws = torch.full((most,), 0xFF, dtype=torch.uint8, device="cuda")
    order = [(i * 7 + i // 5) % len(sets) for i in range(60)]
    outs = [torch.full_like(alone[i][0], 5.0) for i in order]
    for s in sets:
        launch(kq, s)  # handles made, kernels loaded
    torch.cuda.synchronize()
    for i, o in zip(order, outs):
        launch(kq, sets[i], lse=False, out=o, workspace=ws)
    torch.cuda.synchronize()
    for i, o in zip(order, outs):
        assert torch.equal(o, alone[i][0]), i
    assert kq.kq_device_error() == 0


@pytest.mark.parametrize("case", CASES)
def test_two_streams_at_once(kq, case):
    sets = [make(G=8, Hk=2, D=128, page=16, seed=31 + i, **case) for i in range(2)]
    want = [launch(kq, s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    n = kq.kq_kv_attention_workspace_bytes(sets[0]["T"] + 3, sets[0]["B"], 16, 2, 128, max(case["nqs"]))
    ws = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in sets]
    outs = [torch.zeros_like(want[0][0]) for _ in sets]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, st, w, o in zip(sets, streams, ws, outs):
            launch(kq, s, lse=False, out=o, workspace=w, stream=st)
    torch.cuda.synchronize()
    for o, w, s in zip(outs, want, sets):
        assert torch.equal(o[:s["T"]], w[0][:s["T"]])


@pytest.mark.parametrize("case", CASES)
def test_captured_call_follows_growing_sequences(kq, case):
    """A captured call replayed with other lengths, pages and queries, and a second graph on the same workspace."""
    s = make(G=8, Hk=2, D=128, page=16, seed=40, **case)
    t = make([max(0, k - 15 - i % 3) if m == 1 else k for i, (k, m) in enumerate(zip(s["keys"], s["nqs"]))], s["nqs"],
             8, 2, 128, 16, 41, prefix=case["prefix"])
    n = kq.kq_kv_attention_workspace_bytes(s["T"] + 3, s["B"], 16, 2, 128, max(case["nqs"]))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    want = [launch(kq, x)[0] for x in (s, t)]
    out = torch.zeros_like(want[0])
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            launch(kq, s, lse=False, out=out, workspace=ws)
        graphs.append(graph)
    for k, x in enumerate((s, t, s)):
        if x is t:
            s["keep"] = [y.clone() for y in (s["q"], s["kv_len"], s["table"], s["prefix_pages"], *s["pool"])]
            w = min(s["width"], t["width"])
            s["q"].copy_(t["q"])
            s["kv_len"].copy_(t["kv_len"])
            s["table"][:, :w] = t["table"][:, :w]
            s["prefix_pages"].copy_(t["prefix_pages"])
            for a, b in zip(s["pool"], t["pool"]):
                a[:b.shape[0]] = b
        elif k == 2:
            for y, z in zip((s["q"], s["kv_len"], s["table"], s["prefix_pages"], *s["pool"]), s["keep"]):
                y.copy_(z)
        out.zero_()
        graphs[k % 2].replay()
        torch.cuda.synchronize()
        assert torch.equal(out[:s["T"]], want[1 if x is t else 0][:s["T"]]), k


def test_pages_past_32_bits(kq):
    D, Hk, page, G = 128, 8, 256, 4
    s = make([700, 33], [1, 1], G, Hk, D, page, 50)
    want = launch(kq, s)
    s3 = make([700], [90], G, Hk, D, page, 51)
    want3 = launch(kq, s3)
    pages = 2 ** 32 // (Hk * page * 64) + 40
    big = [torch.empty(pages, Hk, page, D // 2, dtype=torch.uint8, device="cuda"), torch.empty(pages, Hk, page, device="cuda"),
           torch.empty(pages, Hk, page, D // 2, dtype=torch.uint8, device="cuda"), torch.empty(pages, Hk, page, device="cuda")]
    for x, w in ((s, want), (s3, want3)):
        k = x["pool"][0].shape[0]
        for a, b in zip(big, x["pool"]):
            a[pages - k:] = b
        y = dict(x, pool=big, table=x["table"] + (pages - k))
        y["table"][x["table"] > 10 ** 6] = -1
        got = launch(kq, y)
        torch.cuda.synchronize()
        assert torch.equal(got[0][:x["T"]], w[0][:x["T"]]) and torch.equal(got[1], w[1])


def test_append_then_attend(kq):
    """The calls in the order of use, with no synchronisation between them: prompt, then single tokens, each
    appended and attended to, then a batch behind the prompt as a shared prefix; against the 64-bit form over the
    rows that the cache holds, and against attention over the unquantised tokens to INT4's accuracy."""
    from test_kv_append_gpu import append, make as make_tokens
    H, Hk, D, page, T = 16, 4, 128, 16, 333
    p = make_tokens(T, H, Hk, D, page, 128, 60, extra_pages=30)
    order = torch.randperm(p["pool"][0].shape[0])
    table = order[:28].to(torch.int32).cuda()[None].contiguous()
    place = lambda a, b: (table[0, torch.arange(a, b, device="cuda") // page].long() * page
                          + torch.arange(a, b, device="cuda") % page)
    p["positions"] = torch.arange(T, device="cuda", dtype=torch.int32)
    p["slots"] = place(0, T)
    scale = 1.0 / math.sqrt(D)
    calls = []

    def attend(tok, n, m):
        ws = torch.empty(kq.kq_kv_attention_workspace_bytes(m, 1, H, Hk, D, m), dtype=torch.uint8, device="cuda")
        out = torch.empty(m, H, D, dtype=torch.bfloat16, device="cuda")
        kq.kq_kv_attention(tok["cache"], tok["q_out"], torch.tensor([0, m], dtype=torch.int32, device="cuda"), table, 28,
                           torch.tensor([n], dtype=torch.int32, device="cuda"), scale, 0.0, 0, out, None, ws, ws.numel(),
                           m, 1, H, m)
        calls.append((out, tok, n, m))

    append(kq, p)
    attend(p, T, T)
    for j in range(3):
        d = make_tokens(1, H, Hk, D, page, 128, 61 + j)
        d.update(pool=p["pool"], slots=place(T + j, T + j + 1), Pq=p["Pq"], Pk=p["Pk"], Pv=p["Pv"], table=p["table"],
                 positions=torch.tensor([T + j], dtype=torch.int32, device="cuda"))
        append(kq, d)
        attend(d, T + j + 1, 1)
    torch.cuda.synchronize()
    pages = table[0].tolist()
    for out, tok, n, m in calls:
        # rows appended later lie past n, so the final cache serves every call's reference
        check_attention(out, None, attention(tok["q_out"][:m], p["pool"], [pages], [n], [m], scale))
    # the prompt alone, unquantised: R q.R k over the tokens themselves
    from kv_testutil import rotate
    ang = p["table"][p["positions"].long()].double()
    q, k = rotate(p["q"].double(), ang, 128, False), rotate(p["k"].double(), ang, 128, False)
    v = p["v"].double() @ p["Pv"].double()
    x = torch.einsum("qhd,khd->hqk", q, k.repeat_interleave(H // Hk, 1)) * scale
    x = x.masked_fill(torch.ones(T, T, device="cuda").triu(1).bool(), -math.inf)
    full = torch.einsum("hqk,khd->qhd", torch.softmax(x, -1), v.repeat_interleave(H // Hk, 1))
    err = float((calls[0][0].double() - full).norm() / full.norm())
    assert err < 0.5, err  # INT4 keys with one large channel and INT4 values: a tenth to a quarter; nonsense is above 1
