"""kq_kv_append's codes are those of exact arithmetic whatever the factor does to a row: rows along the directions
that it shrinks, where the products cancel and fp32's error is far above the result's own rounding."""
import pytest
import torch

from test_kv_append_gpu import append, check, kq, make  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


def factor(D, condition, seed):
    """A bf16 factor with singular values from 1 to 1 / condition, and its left singular vectors, smallest last."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    u, v = [torch.linalg.qr(torch.randn(D, D, generator=g, device="cuda", dtype=torch.float64))[0] for _ in range(2)]
    s = condition ** -torch.linspace(0, 1, D, device="cuda", dtype=torch.float64)
    P = (u * s @ v.T).to(torch.bfloat16).contiguous()
    return P, torch.linalg.svd(P.double())[0]


@pytest.mark.parametrize("alpha", [1.0, 0.7])
@pytest.mark.parametrize("D,rope,inter", [(128, 0, False), (128, 128, False), (64, 64, True), (64, 0, False)])
@pytest.mark.parametrize("condition", [10, 100, 1000, 10000])
def test_ill_conditioned_factors(kq, condition, D, rope, inter, alpha):
    """Rows in the eight directions that the factor shrinks most (before a rotation turns them)."""
    s = make(1500, 2, 2, D, 16, rope, condition + D)
    P, u = factor(D, condition, condition + D)
    s["Pk"] = s["Pv"] = P
    g = torch.Generator(device="cuda").manual_seed(condition)
    for name in ("k", "v"):
        c = torch.randn(1500, 2, 8, generator=g, device="cuda", dtype=torch.float64)
        s[name][:] = (c @ u[:, -8:].T * 5).to(torch.bfloat16)
    append(kq, s, alpha, alpha, inter=inter)
    check(s, alpha, alpha, inter=inter)
    assert kq.kq_device_error() == 0


@pytest.mark.parametrize("D", [64, 128])
def test_products_that_cancel(kq, D):
    """Two elements of up to 2^24 times the others whose products cancel exactly, in one step of 16 products
    and in two steps."""
    T = 1500
    s = make(T, 2, 2, D, 16, 0, D)
    g = torch.Generator(device="cuda").manual_seed(D)
    P = torch.randn(D, D, generator=g, device="cuda").to(torch.bfloat16)
    P[1], P[D - 3] = -P[0], -P[2]
    s["Pk"] = s["Pv"] = P
    big = torch.exp2((torch.arange(T, device="cuda") % 25).float())[:, None].to(torch.bfloat16)
    for name in ("k", "v"):
        s[name][..., 0] = s[name][..., 1] = big
        s[name][..., 2] = s[name][..., D - 3] = 0
        s[name][::2, :, 2] = s[name][::2, :, D - 3] = big[::2]
    append(kq, s, 0.9, 0.8)
    check(s)
    assert kq.kq_device_error() == 0


def test_products_that_cancel_to_nothing_in_fp32(kq):
    """What is left lies 2^-40 below the products: fp32 has lost all of it."""
    T, D = 200, 128
    s = make(T, 2, 2, D, 16, 0, 3)
    P = torch.zeros(D, D, dtype=torch.bfloat16, device="cuda")
    P[0], P[1] = 1.0, -1.0
    P[2] = torch.linspace(-1, 1, D, device="cuda").to(torch.bfloat16)
    s["Pk"] = s["Pv"] = P
    for name in ("k", "v"):
        s[name][:] = 0
        s[name][..., 0] = s[name][..., 1] = 1.5
        s[name][..., 2] = 2.0 ** -40
    append(kq, s)
    check(s)


def test_rows_of_any_size_in_exact_codes(kq):
    """Rows from 2^-98 to 2^110: the codes do not depend on a power of two."""
    s, t = make(400, 2, 2, 128, 16, 128, 4), make(400, 2, 2, 128, 16, 128, 4)
    e = (torch.arange(400, device="cuda") * 0.52 - 98).round().double()
    for name in ("k", "v"):
        s[name][:] = (s[name].double() * torch.exp2(e)[:, None, None]).to(torch.bfloat16)
    append(kq, s)
    append(kq, t)
    torch.cuda.synchronize()
    check(s)
    for i in (0, 2):
        assert torch.equal(s["pool"][i], t["pool"][i])
