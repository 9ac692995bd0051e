"""Plain 64-bit forms of the key / value cache calls (torch float64, loops over
sequences and heads), shared by the cache's tests.  Nothing here calls the library."""
from __future__ import annotations

import math

import torch


def unpack(codes: torch.Tensor) -> torch.Tensor:
    """Packed INT4 bytes [..., n] -> signed values [..., 2 n], element 2k from the low nibble."""
    lo, hi = (codes & 15).to(torch.int32), (codes >> 4).to(torch.int32)
    v = torch.stack([lo, hi], -1).flatten(-2)
    return torch.where(v > 7, v - 16, v).double()


def rotate(x, angles, rope_dim, interleaved):
    """x [T, heads, D] fp64, angles [T, rope_dim] fp64 (cosines, then sines)."""
    if not rope_dim:
        return x
    x = x.clone()
    half = rope_dim // 2
    c, s = angles[:, None, :half], angles[:, None, half:]
    first = slice(0, rope_dim, 2) if interleaved else slice(0, half)
    second = slice(1, rope_dim, 2) if interleaved else slice(half, rope_dim)
    a, b = x[..., first].clone(), x[..., second].clone()
    x[..., first], x[..., second] = a * c - b * s, a * s + b * c
    return x


def quantise(y, alpha):
    """Codes, scales and each value's distance to the nearest rounding border (in steps), per row, fp64."""
    s = float(torch.tensor(alpha, dtype=torch.float32)) * y.abs().amax(-1, keepdim=True) / 7
    r = torch.where(s > 0, y / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(y))
    dist = ((r - torch.floor(r)) - 0.5).abs()
    return torch.clamp(torch.round(r), -8, 7), s[..., 0], dist


def attention(q, cache, tables, keys, nqs, scale, softcap=0.0, window=0, prefix=None):
    """out, lse in fp64, with the sums that bound an implementation's rounding:
    mean = sum_t p_t |v_t| / sum_t p_t per output element, size = max_t scale sum_d |q_d k_td| per row,
    floor = n max_t p_t s'_t / sum_t p_t per row of n keys (s' the value scales).

    cache = (k_codes, k_scale, v_codes, v_scale); tables[b]: page numbers of sequence b (a list);
    prefix = (pages, length) or None."""
    kc, ks, vc, vs = cache
    Hk, page = kc.shape[1], kc.shape[2]
    T, H, D = q.shape
    G = H // Hk
    out = torch.zeros(T, H, D, dtype=torch.float64, device=q.device)
    mean, lse = torch.zeros_like(out), torch.full((T, H), -math.inf, dtype=torch.float64, device=q.device)
    size, floor = torch.zeros_like(lse), torch.zeros_like(out[..., :1])

    def rows(codes, sc, pages, n, h):
        """[n, D + 1]: the values of n rows, and their scales."""
        if n == 0:
            return torch.zeros(0, D + 1, dtype=torch.float64, device=q.device)
        at = torch.as_tensor(list(pages)[:(n + page - 1) // page], device=q.device, dtype=torch.long)
        s = sc[at, h].double()[..., None]
        return torch.cat([unpack(codes[at, h]) * s, s], -1).reshape(-1, D + 1)[:n]

    pre = prefix[1] if prefix else 0
    first = 0
    for b, (n, m) in enumerate(zip(keys, nqs)):
        for h in range(Hk):
            K, V = rows(kc, ks, tables[b], n, h), rows(vc, vs, tables[b], n, h)
            if pre:
                K = torch.cat([rows(kc, ks, prefix[0], pre, h), K])
                V = torch.cat([rows(vc, vs, prefix[0], pre, h), V])
            K, V, S = K[:, :D], V[:, :D], V[:, D]
            pos = torch.arange(pre + n, device=q.device)
            for i in range(m):
                p = pre + n - m + i
                see = (pos <= p) | (pos < pre)
                if window:
                    see &= pos > p - window
                if not bool(see.any()):
                    continue
                qi = q[first + i, h * G:(h + 1) * G].double()
                x = qi @ K[see].T * scale
                size[first + i, h * G:(h + 1) * G] = (qi.abs() @ K[see].abs().T).amax(-1) * abs(scale)
                if softcap:
                    x = softcap * torch.tanh(x / softcap)
                z = torch.logsumexp(x, -1)
                w = torch.exp(x - z[:, None])
                out[first + i, h * G:(h + 1) * G] = w @ V[see]
                mean[first + i, h * G:(h + 1) * G] = w @ V[see].abs()
                lse[first + i, h * G:(h + 1) * G] = z
                floor[first + i, h * G:(h + 1) * G, 0] = (w * S[see]).amax(-1) * w.shape[-1]
        first += m
    return out, lse, mean, size, floor


def check_attention(out, lse, ref):
    """The rounding an implementation may have: a score is a sum of D products of 24-bit values (off by at most
    (D + 8) 2^-24 of the products' absolute sum), its exponential and the sums of them are fp32 (2^-18 covers
    thousands of terms with their maxima moved along), every weight is rounded once to no fewer than bf16's bits
    before it meets the values (half a step: 2^-8 of each term), and the result once to bf16 (2^-8 of it).
    Weights kept in fp16 with their largest at 2^6 or more have a smallest step besides: 2^-24, half of it
    2^-25 = 2^-31 2^6, so each of n weights p s' may be off by 2^-31 of the largest, times a code of at most 8:
    8 2^-31 floor in all (an element that is 0 in every key but those of the smallest weights shows it)."""
    r_out, r_lse, mean, size, floor = ref
    D = r_out.shape[-1]
    off = (D + 8) * 2.0 ** -24 * size + 2.0 ** -18
    if lse is not None:
        fin = torch.isfinite(r_lse)
        assert torch.equal(fin, torch.isfinite(lse)), "rows without keys"
        assert (lse[~fin] == -math.inf).all()
        d = (lse.double() - r_lse).abs()[fin]
        assert (d <= (off + 2.0 ** -23 * r_lse.abs())[fin]).all(), "lse off by %.3g" % float(d.max())
    bound = 2.0 ** -8 * r_out.abs() + (2.0 ** -8 + 2 * off[..., None]) * mean + 8 * 2.0 ** -31 * floor + 1e-30
    d = (out.double() - r_out).abs()
    worst = float((d / bound).max()) if d.numel() else 0.0
    assert worst <= 1.0, "out off by %.3g of its bound" % worst
