"""The cache's attention by the size of its error over a row, on long contexts.

An output of n keys with values of both signs is about sum p |v| / sqrt(n): a bound that adds up all keys' roundings
allows an error as large as that.  Roundings of different keys are independent, though, and so are those of a row's
elements.  With r the largest relative rounding of a weight and a half step 2^-8 of the bf16 result, both at most
evenly spread (a factor 1 / sqrt 3), and scores off by `off` (see kv_testutil.check_attention), a row's error is

    rms <= (r / sqrt 3 + off) rms(sqrt(sum_t p_t^2 v_t^2)) + (2^-8 / sqrt 3 + 2^-18) rms(out)

of its head_dim elements in the mean.  Four times that is asked: the rms of 64 elements passes its mean by half at
most, and the rest covers weights whose mantissas lie at the lower end and what the scores' roundings have in common.
One wrong page of 64 keys among 131072 moves a row by sqrt(2 64) / 131072 |v|, more than that."""
import math

import pytest
import torch

from kv_testutil import unpack
from test_kv_attention_gpu import kq, launch, spread  # noqa: F401  (the fixture)
from test_kv_attention_gpu import make as make_any

pytestmark = pytest.mark.gpu
ROWS, TILES = 2.0 ** -11, 2.0 ** -8  # a weight's rounding in the row kernel (fp16) and in the tile kernel (bf16)


def make(*args, **kw):
    """The same with values of mean zero: a mean, which all keys share, would be all of an output."""
    s = make_any(*args, **kw)
    codes = torch.tensor([-7, -5, -4, -3, -2, -1, -1, 0, 0, 1, 1, 2, 3, 4, 5, 7])
    lut = (codes & 15).to(torch.uint8).cuda()
    g = torch.Generator(device="cuda").manual_seed(sum(s["keys"]))
    two = torch.randint(0, 256, s["pool"][2].shape, generator=g, device="cuda", dtype=torch.int32)
    s["pool"][2] = lut[two >> 4] << 4 | lut[two & 15]
    return s


def check_rms(s, out, sample, r, softcap=0.0, window=0):
    """sample: (sequence, query) pairs that are looked at, all heads of them."""
    kc, ks, vc, vs = s["pool"]
    page, G, D, pre = s["page"], s["G"], s["D"], s["prefix"]
    starts = [sum(s["nqs"][:b]) for b in range(s["B"])]

    def rows(codes, scale, pages, n, h):
        at = torch.tensor(pages[:(n + page - 1) // page], dtype=torch.long, device="cuda")
        return (unpack(codes[at, h]) * scale[at, h].double()[..., None]).reshape(-1, D)[:n]

    worst = 0.0
    for h in range(s["Hk"]):
        Kp, Vp = [rows(c, x, s["prefix_list"], pre, h) for c, x in ((kc, ks), (vc, vs))]
        for b in sorted({b for b, _ in sample}):
            n, m = s["keys"][b], s["nqs"][b]
            K, V = [torch.cat([p, rows(c, x, s["tables"][b], n, h)]) for p, c, x in ((Kp, kc, ks), (Vp, vc, vs))]
            pos = torch.arange(pre + n, device="cuda")
            for i in [i for c, i in sample if c == b]:
                see = pos <= max(pre - 1, pre + n - m + i)
                if window:
                    see &= pos > pre + n - m + i - window
                at = starts[b] + i
                q = s["q"][at, h * G:(h + 1) * G].double()
                x = q @ K[see].T * s["scale"]
                size = (q.abs() @ K[see].abs().T).amax(-1) * s["scale"]
                if softcap:
                    x = softcap * torch.tanh(x / softcap)
                w = torch.softmax(x, -1)
                ref, square = w @ V[see], w.square() @ V[see].square()
                rms = lambda t: t.square().mean(-1).sqrt()
                off = (D + 8) * 2.0 ** -24 * size + 2.0 ** -18
                # weights in fp16 have a smallest step, half of it 2^-31 of the largest p s'; times a code of 8
                floor = 8 * 2.0 ** -31 * (w * (V[see].abs().amax(-1) / 7)).amax(-1) * math.sqrt(w.shape[-1]) if r == ROWS else 0.0
                bound = (r / math.sqrt(3) + off) * square.mean(-1).sqrt() + (2.0 ** -8 / math.sqrt(3) + 2.0 ** -18) * rms(ref) \
                    + floor + 1e-30
                err = rms(out[at, h * G:(h + 1) * G].double() - ref)
                worst = max(worst, float((err / (4 * bound)).max()))
    assert worst <= 1.0, "rms off by %.3g of its bound" % worst


@pytest.mark.parametrize("D,G,keys,kw", [
    (128, 4, [131072 + 5, 70001], {}), (64, 4, [131072, 100003, 17], {}), (128, 8, [40000] * 3, dict(window=30000)),
    (64, 1, [65537], dict(softcap=20.0)), (128, 16, [30011, 9000], {}), (128, 4, [20000 + 500 * i for i in range(24)], {})])
def test_single_tokens_on_long_contexts(kq, D, G, keys, kw):
    s = make(keys, [1] * len(keys), G, 2, D, 64, len(keys) + D, q_std=0.5)
    out, _ = launch(kq, s, **kw)
    torch.cuda.synchronize()
    check_rms(s, out, [(b, 0) for b in range(len(keys))], ROWS, **kw)


@pytest.mark.parametrize("page", [16, 128])
def test_a_few_tokens_on_long_contexts(kq, page):
    s = make([50021, 33333, 80000], [5, 1, 3], 4, 2, 128, page, page, q_std=0.5)
    out, _ = launch(kq, s)
    torch.cuda.synchronize()
    check_rms(s, out, [(0, i) for i in range(5)] + [(1, 0), (2, 0), (2, 2)], ROWS)


@pytest.mark.parametrize("D,G,nqs,keys,kw", [
    (128, 4, [1024], [60000], {}), (64, 8, [300, 90], [100003, 40000], {}), (128, 2, [40, 64], [131072, 100001], {}),
    (128, 4, [8192], [8192], {}), (64, 4, [2000], [50000], dict(window=9000)), (128, 8, [200], [40001], dict(softcap=20.0))])
def test_prompts_on_long_contexts(kq, D, G, nqs, keys, kw):
    s = make(keys, nqs, G, 2, D, 64, len(nqs) + D, q_std=0.5)
    out, _ = launch(kq, s, **kw)
    torch.cuda.synchronize()
    check_rms(s, out, [(b, i) for b, m in enumerate(nqs) for i in sorted({0, m // 3, m // 2, m - 1})], TILES, **kw)


def test_prompts_and_single_tokens_on_long_contexts(kq):
    nqs = [1, 600, 1, 1, 90] + [1] * 20
    s = make(spread(40000, nqs), nqs, 4, 2, 128, 64, 3, q_std=0.5)
    out, _ = launch(kq, s)
    torch.cuda.synchronize()
    single = [(b, 0) for b, m in enumerate(nqs) if m == 1 and s["keys"][b] > 1]
    check_rms(s, out, single, ROWS)
    check_rms(s, out, [(1, 0), (1, 599), (4, 0), (4, 89)], TILES)


@pytest.mark.parametrize("D,G,B,prefix", [(128, 4, 5, 60000), (64, 1, 20, 30001)])
def test_a_long_prefix_of_few_rows(kq, D, G, B, prefix):
    keys = [(7 * i) % 150 for i in range(B)]
    s = make(keys, [1] * B, G, 2, D, 64, B, prefix=prefix, q_std=0.5)
    out, _ = launch(kq, s)
    torch.cuda.synchronize()
    check_rms(s, out, [(b, 0) for b in range(B)], ROWS)


@pytest.mark.parametrize("D,G,B,prefix,kw", [(128, 8, 40, 60000, {}), (64, 4, 100, 30001, dict(softcap=30.0))])
def test_a_long_prefix_of_many_rows(kq, D, G, B, prefix, kw):
    keys = [(7 * i) % 150 for i in range(B)]
    s = make(keys, [1] * B, G, 2, D, 64, B, prefix=prefix, q_std=0.5)
    out, _ = launch(kq, s, **kw)
    torch.cuda.synchronize()
    check_rms(s, out, [(b, 0) for b in range(0, B, 3)], TILES, **kw)


@pytest.mark.parametrize("wrong", ["page", "scale"])
def test_the_bound_sees_one_page(kq, wrong):
    """A page of 64 keys among 131072 with another's values, in the reference alone."""
    s = make([131072], [1], 4, 2, 128, 64, 5, q_std=0.5)
    out, _ = launch(kq, s)
    torch.cuda.synchronize()
    check_rms(s, out, [(0, 0)], ROWS)
    p, other = s["tables"][0][1000], s["tables"][0][7]
    k = 2 if wrong == "page" else 3
    s["pool"][k][p] = s["pool"][k][other] if wrong == "page" else 2 * s["pool"][k][p]
    with pytest.raises(AssertionError, match="rms"):
        check_rms(s, out, [(0, 0)], ROWS)
