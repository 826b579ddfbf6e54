"""The 4-bit KV cache's definition in 64 bits: the reference of test_gpu_kv4*.py."""
import math

import torch


def minifloat(bits, ebits, mbits, bias):
    bits = bits.to(torch.int64)
    e, m = bits >> mbits & (1 << ebits) - 1, (bits & (1 << mbits) - 1).double() / (1 << mbits)
    mag = torch.where(e == 0, m * 2.0 ** (1 - bias), (1 + m) * torch.exp2((e - bias).double()))
    return torch.where(bits >> (ebits + mbits) & 1 == 1, -mag, mag)


def e2m1(bits):
    return minifloat(bits, 2, 1, 1)


def e4m3(bits):
    return minifloat(bits, 4, 3, 7)


def values(codes, scales):
    """codes [.., hd/2], scales [.., hd/16] (uint8) -> FP64 [.., hd]."""
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    return e2m1(c) * e4m3(scales).repeat_interleave(16, -1)


def nearest_even(x, grid):
    """Index of the entry of the ascending grid nearest to x, halves to the even index, the ends for what lies outside."""
    mid = (grid[:-1] + grid[1:]) / 2
    i = torch.searchsorted(mid, x.contiguous())          # mid[i-1] < x <= mid[i]
    tie = (i < len(mid)) & (mid[i.clamp(max=len(mid) - 1)] == x) & (i % 2 == 1)
    return i + tie.long()


def quantise(x):
    """FP [.., hd] -> (codes, scales), uint8: infinities as the largest finite value, NaN as 0."""
    top = torch.finfo(torch.float32).max
    b = torch.nan_to_num(x.double(), nan=0.0, posinf=top, neginf=-top).unflatten(-1, (-1, 16))
    sg, mg = e4m3(torch.arange(127, device=x.device)), e2m1(torch.arange(8, device=x.device))
    s8 = nearest_even(b.abs().amax(-1) / 6, sg)
    s = sg[s8].unsqueeze(-1)
    c = nearest_even(torch.where(s > 0, b.abs() / s, torch.zeros_like(b)), mg)
    c = c | ((b < 0) & (s > 0)).long() << 3
    c = c.flatten(-2)
    return (c[..., 0::2] | c[..., 1::2] << 4).to(torch.uint8), s8.to(torch.uint8)


def seen(n, pos, length, window, device):
    at = torch.arange(pos, pos + n, device=device)[:, None]
    j = torch.arange(length, device=device)[None]
    m = j <= at
    return m & (j > at - window) if window else m


def attention(q, k, v, pos, length, window, scale):
    """q [n, Hq, hd]; k, v [Hkv, >= length, hd] in FP64.  Returns (out, bound): per element how far a kernel may be
    off that keeps scores and sums in FP32 and rounds the probabilities as q's type has it.

    With S = sum_j p_j |v_j| (p normalised), in units of S:
      - the probabilities' rounding: 2^-11 (FP16), or 2^-21 for FP32 q (head and remainder, 2^-11 * 2^-11, and the
        same of q and of exp2);
      - a score off by d shifts p by d: d = (hd + 8) 2^-23 * scale sum_i |q_i k_i|, from FP32 sums over hd products
        and the conversions of q (BF16: exact or 2^-25 of the row's largest); twice, as the sum is off as well;
      - FP32 sums over the positions, rounded or cut off at every 16 of them: (length / 16 + 16) 2^-23;
    and besides S:
      - FP16 runs out of exponents: the kernels scale the row's largest probability to 2^7 at least, so that a
        head or remainder that is subnormal is off by up to 2^-25, 2^-25 / 2^7 = 2^-32 of the largest; each position
        may be (the sum is at least the largest): length * 2^-32 max|v|;
      - the output's own rounding, half a step of its type."""
    n, Hq, hd = q.shape
    G = Hq // k.shape[0]
    vis = seen(n, pos, length, window, q.device)
    out = torch.zeros(n, Hq, hd, dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(out)
    scale = scale or 1 / math.sqrt(hd)
    wide = q.dtype == torch.float32
    for h in range(Hq):
        kk, vv, qq = k[h // G, :length], v[h // G, :length], q[:, h].double()
        if length == 0:
            continue
        s = (qq @ kk.T * scale).masked_fill(~vis, -math.inf)
        some = vis.any(-1, keepdim=True)
        e = torch.exp(s - torch.where(some, s.amax(-1, keepdim=True), torch.zeros_like(s[:, :1])))
        p = e / e.sum(-1, keepdim=True).clamp(min=1e-300)
        out[:, h] = p @ vv
        mag = p @ vv.abs()
        d = (hd + 8) * 2.0 ** -23 * abs(scale) * ((qq.abs() @ kk.abs().T) * vis).amax(-1, keepdim=True)
        d = d + 2.0 ** -25 * abs(scale) * qq.abs().amax(-1, keepdim=True) * (kk.abs().sum(-1) * vis).amax(-1, keepdim=True)
        rel = (2.0 ** -20 if wide else 2.0 ** -11 + 2.0 ** -20) + 2 * d + (length / 16 + 16) * 2.0 ** -23
        bound[:, h] = mag * rel + length * 2.0 ** -32 * vv.abs().amax()
    half = torch.finfo(q.dtype).eps / 2
    return out, bound + (out.abs() + bound) * half + torch.finfo(q.dtype).tiny
