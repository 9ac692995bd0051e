"""Factors of the scores at the ends of fp32: products of the scales that pass it do not make a zero score a NaN."""
import pytest
import torch

from test_kv_attention_gpu import kq, make, verify  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("nqs", [[1, 2, 3], [70, 80, 128]])
@pytest.mark.parametrize("softcap", [4e-39, 1e-37, 1e-30])
def test_tiny_caps(kq, nqs, softcap):
    """All scores are within the cap of 0, a key of zeros at 0 exactly: the weights are all alike."""
    s = make([300, 90, 140], nqs, 4, 2, 128, 16, 1)
    for pages in s["tables"]:
        for p in pages:
            s["pool"][0][p, :, 3::4] = 0
    s["pool"][1] *= 50.0
    verify(kq, s, softcap=softcap)


@pytest.mark.parametrize("nqs", [[1, 2, 3], [70, 80, 128]])
@pytest.mark.parametrize("scale", [1e33, -1e33])
def test_zero_queries_under_a_large_scale(kq, nqs, scale):
    """The softmax scale undoes the size of the queries, some of which are zero."""
    s = make([300, 90, 140], nqs, 4, 2, 128, 16, 2)
    s["q"] = (s["q"].double() * 0.1e-33).to(torch.bfloat16)
    s["q"][0:s["T"]:2] = 0
    s["scale"] = scale
    verify(kq, s)
