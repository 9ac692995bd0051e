"""Value scales at the ends of their range, 0 and 2^-100 to 2^96, in both kernels of the cache's attention."""
import pytest
import torch

from kv_testutil import attention
from test_kv_attention_gpu import kq, launch, make, verify  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


def jumps(s):
    """Key scales that rise inside a chunk: scores of a few hundredths, then of tens."""
    for b, n in enumerate(s["keys"]):
        for t in range(n):
            s["pool"][1][s["tables"][b][t // 16], :, t % 16] *= 0.01 if t % 400 < 330 else 11.0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("mid", [1e12, 1e20, 1e25, 1e28])
@pytest.mark.parametrize("nqs", [[1, 3], [150, 200]])
def test_large_value_scales_under_scores_that_jump(kq, nqs, mid, D):
    s = make([1500, 1100], nqs, 4, 2, D, 16, 1)
    s["pool"][3] *= mid
    jumps(s)
    verify(kq, s)
    s = make([600, 500], nqs, 4, 2, D, 16, 2, prefix=800)
    s["pool"][3] *= mid
    verify(kq, s, softcap=20.0)


@pytest.mark.parametrize("nqs", [[1, 3], [150, 200]])
def test_value_scales_of_all_sizes_in_one_row(kq, nqs):
    """Scales from 2^-100 to 2^90 side by side: the large ones decide, whatever their neighbours."""
    s = make([1500, 1100], nqs, 4, 2, 128, 16, 3)
    g = torch.Generator(device="cuda").manual_seed(3)
    e = torch.randint(-95, 90, s["pool"][3].shape, generator=g, device="cuda").float()
    s["pool"][3] *= torch.exp2(e)
    verify(kq, s)


@pytest.mark.parametrize("nqs", [[1, 3], [150, 200]])
def test_the_smallest_value_scales(kq, nqs):
    """Under 2^-100 the row kernel's weights lose bits, but not their size: within 2^-6 of the terms."""
    for mid, bits in ((1e-29, 7.5), (1e-33, 6), (1e-35, 3)):
        s = make([300, 140], nqs, 4, 2, 128, 16, 4)
        s["pool"][3] *= mid
        out, _ = launch(kq, s)
        torch.cuda.synchronize()
        T = s["T"]
        ref, _, mean, _, _ = attention(s["q"][:T], s["pool"], s["tables"], s["keys"], s["nqs"], s["scale"])
        # bf16's half steps of the result and of a weight, 2^-8 each, or what is left of the weight's bits
        assert ((out[:T].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -bits * mean + 1e-40).all(), mid


@pytest.mark.parametrize("prefix", [0, 200])
@pytest.mark.parametrize("nqs", [[1, 3], [150, 200]])
def test_codes_under_a_scale_of_zero_count_nothing(kq, nqs, prefix):
    s = make([300, 140], nqs, 4, 2, 128, 16, 5, prefix=prefix)
    s["pool"][3][~torch.isnan(s["pool"][3])] = 0.0
    out, _ = launch(kq, s)
    torch.cuda.synchronize()
    assert (out[:s["T"]] == 0).all()
