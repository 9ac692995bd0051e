"""Capped scores of the cache's attention over the whole range of caps: a large cap leaves ordinary scores as they
are, a tiny one makes all weights alike; against the 64-bit form."""
import pytest
import torch

from kv_testutil import attention, check_attention
from test_kv_attention_gpu import kq, launch, make, verify  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("softcap", [1e3, 1e4, 1e6, 1e9, 1e30])
def test_large_caps(kq, softcap, D):
    """Scores far below the cap are those without one, in chunks with a mask and without."""
    verify(kq, make([1, 17, 100, 700, 129, 0], [1] * 6, 4, 2, D, 16, 1), softcap=softcap)
    verify(kq, make([300, 40, 700], [3, 5, 1], 2, 2, D, 32, 2), softcap=softcap, window=150)
    verify(kq, make([150, 900, 700], [150, 200, 128], 4, 2, D, 16, 3), softcap=softcap)
    verify(kq, make([400, 900], [150, 200], 4, 2, D, 16, 4), softcap=softcap, window=190)
    verify(kq, make([5, 0, 130, 60] * 5, [1] * 20, 4, 2, D, 16, 5, prefix=450), softcap=softcap)


@pytest.mark.parametrize("softcap", [40.0, 1e4, 1e7])
@pytest.mark.parametrize("nqs", [[1, 2, 4], [70, 128, 150]])
def test_queries_near_the_cap_beside_ordinary_ones(kq, nqs, softcap):
    """Every third query's scores are of the cap's size; its neighbours', in the same tiles, are not."""
    s = make([700, 300, 400], nqs, 4, 2, 128, 16, 6)
    q = s["q"].double()
    q[0:s["T"]:3] *= softcap / 3
    s["q"] = q.to(torch.bfloat16)
    verify(kq, s, softcap=softcap)


@pytest.mark.parametrize("nqs", [[1, 2, 4], [70, 128, 150]])
def test_keys_near_the_cap_beside_ordinary_ones(kq, nqs):
    """One key in fifty, of negative products, lies at the cap's far side: the others keep their differences."""
    s = make([700, 300, 400], nqs, 4, 2, 128, 16, 7, mean=1.0, q_std=0.2)
    softcap, T = 1e6, s["T"]
    form = lambda: attention(s["q"][:T], s["pool"], s["tables"], s["keys"], s["nqs"], s["scale"], softcap)
    size = form()[3]  # of the ordinary keys: the others' weights are e^-1e6, so that their rounding does not count
    for pages in s["tables"]:
        for p in pages[::3]:
            s["pool"][0][p, :, 5] = 0xCC  # codes of -4, against queries that are mostly positive
            s["pool"][1][p, :, 5] *= 1e6
    out, lse = launch(kq, s, softcap=softcap)
    torch.cuda.synchronize()
    ref = form()
    assert float(ref[3].max()) > 10 * softcap
    check_attention(out[:T], lse[:T], (*ref[:3], size, ref[4]))
