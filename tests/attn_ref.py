"""Plain 64-bit forms of the operators of include/strata_attn.h, and the
error bounds that the GPU tests hold the kernels to."""
import math

import numpy as np
import torch

import oracle


def rope_frequencies(rd, theta, scaling="none", factor=1.0, original=0, fast=32.0, slow=1.0, attn=0.0):
    """f_i as fp64 (numpy, with the header's formulas) and m."""
    if scaling == "ntk":
        theta = theta * factor ** (rd / (rd - 2.0))
    f = np.array([theta ** (-2.0 * i / rd) for i in range(rd // 2)])
    if scaling == "linear":
        f = f / factor
    m = 1.0
    if scaling == "yarn":
        def pair_of(t):
            return rd * math.log(original / (t * 2 * math.pi)) / (2 * math.log(theta))
        lo, hi = max(math.floor(pair_of(fast)), 0), min(math.ceil(pair_of(slow)), rd - 1)
        r = np.clip((np.arange(rd // 2) - lo) / ((hi - lo) or 0.001), 0.0, 1.0)
        f = f / factor * r + f * (1 - r)
        m = 0.1 * math.log(factor) + 1.0
    return f, attn or m


def rope_cs(positions, f, m):
    """cos and sin as fp32 [tokens, rd/2]; the angle in extended precision."""
    turn = f.astype(np.longdouble) / (2 * np.longdouble("3.14159265358979323846264338327950288"))
    a = positions.astype(np.longdouble)[:, None] * turn
    a = (a - np.rint(a)) * (2 * np.longdouble("3.14159265358979323846264338327950288"))
    return (np.cos(a) * m).astype(np.float32), (np.sin(a) * m).astype(np.float32)


def bf16_round(x):
    """fp32 -> the nearest bf16 as fp32, ties to even (finite values)."""
    b = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32)
    return ((b + (0x7FFF + ((b >> 16) & 1))) & np.uint32(0xFFFF0000)).view(np.float32)


def rope_rows(x, cs, rd, layout):
    """The header's rotary step on fp32 rows [tokens, heads, D], every product and sum rounded to fp32; not yet to bf16."""
    c, s = cs[0][:, None, :], cs[1][:, None, :]
    y = x.copy()
    iu = np.arange(rd // 2) if layout == "half" else np.arange(0, rd, 2)
    iv = iu + rd // 2 if layout == "half" else iu + 1
    u, v = x[..., iu], x[..., iv]
    y[..., iu] = u * c - v * s
    y[..., iv] = v * c + u * s
    return y


def sylvester(D, device):
    h = torch.ones((1, 1), dtype=torch.float64, device=device)
    while h.shape[0] < D:
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
    return h / math.sqrt(D)


def encode_rows(bits):
    """Oracle codes and scales of bf16 rows (uint16 [rows, D])."""
    return oracle.kv4_encode(np.ascontiguousarray(bits))


def dequant(codes, scales):
    """(c - 8) s in fp64 for codes [..., D/2] and scales [..., D/32]: the rotated rows."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).double() - 8
    return c * scales.double().repeat_interleave(32, -1)


def attention(q, q_offsets, kv_lens, table, cache, window, scale, out):
    """Attention in 64 bits. q: fp64 [tokens, heads, D] (rotary applied); cache: the four tensors. Writes `out`
    (fp64) for the rows inside sequences; returns the bound of each such row's error as a 2-norm [tokens, heads],
    and which rows they are.

    The bound, in the rotated basis (the transform keeps the 2-norm). fp16 rounding is off by at most 2^-11 of the
    value (the power-of-two scale of a query row keeps every value within 2^-13 of its largest a normal number; the
    smaller ones are off by 2^-25 of the largest at most, which the second term covers), so logit j moves by at most
      e_j = scale * (2^-11 sum_i |q_i| |y_ji| + 1032 * 2^-21 sum_i |q_i| s_ji) + 2^-20 |logit|.
    The middle term is the fp32 accumulation in the tensor core: codes enter as offset values of at most 1032 before
    the offset is taken out again, and a block's sum takes four adds (two products of 16, each with its running
    sum), each off by at most 2^-23 of the largest partial sum, 1032 sum |q_i|, times the block's scale s. The last
    term is the fp32 rest: four block sums, the scale, the exponent's argument. A probability moves by a factor of
    exp(e_j + max e) at most; it and the value are rounded to fp16 once each (2^-11 each), the sums in fp32 and the
    exponential add 2^-18. The result is rounded to bf16 once: 2^-8 of the value."""
    n, heads, D = q.shape
    kc, ks, vc, vs = cache
    page = kc.shape[2]
    G = heads // kc.shape[1]
    H = sylvester(D, q.device)
    bound = torch.zeros((n, heads), dtype=torch.float64, device=q.device)
    inside = torch.zeros(n, dtype=torch.bool, device=q.device)
    lens, offs = kv_lens.tolist(), q_offsets.tolist()
    for b, L in enumerate(lens):
        t0, t1 = offs[b], offs[b + 1]
        L = min(max(L, 0), table.shape[1] * page)
        if t1 <= t0:
            continue
        inside[t0:t1] = True
        pages = table[b, : -(-L // page)].long()
        ok_page = (pages >= 0) & (pages < kc.shape[0])
        ok = ok_page.repeat_interleave(page)[:L]
        safe = torch.where(ok_page, pages, torch.zeros_like(pages))
        j = torch.arange(L, device=q.device)[None]
        for lo in range(t0, t1, 512):
            hi = min(t1, lo + 512)
            p = torch.arange(L - t1 + lo, L - t1 + hi, device=q.device)[:, None]
            seen = (j <= p) & ok[None]
            if window:
                seen &= j > p - window
            for hk in range(kc.shape[1]):
                y = [dequant(c[safe, hk].flatten(0, 1)[:L], s[safe, hk].flatten(0, 1)[:L])
                     for c, s in ((kc, ks), (vc, vs))]
                for t in y:
                    t[~ok] = 0  # whatever an evicted page holds
                z = q[lo:hi, hk * G : (hk + 1) * G].transpose(0, 1) @ H  # [G, rows, D]
                x = (z @ y[0].T) * scale
                s = torch.where(ok[:, None], ks[safe, hk].flatten(0, 1)[:L].double(), 0.0).abs().repeat_interleave(32, -1)
                e = abs(scale) * (2.0**-11 * (z.abs() @ y[0].abs().T) + 1032 * 2.0**-21 * (z.abs() @ s.T)) + \
                    2.0**-20 * x.abs()
                x = x.masked_fill(~seen, -math.inf)
                top = x.amax(-1, keepdim=True) if L else x.sum(-1, keepdim=True)
                w = torch.exp(x - top.masked_fill(top == -math.inf, 0.0)) if L else x
                l = w.sum(-1, keepdim=True)
                w = w / l.masked_fill(l == 0, 1.0)
                o = w @ y[1]
                e = e.masked_fill(~seen, 0.0)
                rel = torch.expm1(e + (e.amax(-1, keepdim=True) if L else 0.0)) + 2 * 2.0**-11 + 2.0**-18
                err = (w * rel) @ y[1].abs()
                out[lo:hi, hk * G : (hk + 1) * G] = (o @ H).transpose(0, 1)
                bound[lo:hi, hk * G : (hk + 1) * G] = (err.norm(dim=-1) + 2.0**-8 * o.norm(dim=-1)).transpose(0, 1)
    return bound, inside
