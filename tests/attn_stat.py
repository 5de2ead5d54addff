"""What the error of an attention row is, as a second moment: sharp where the
worst case of attn_ref.attention is not (it adds every key's error in absolute
value, while the row itself shrinks with the number of keys, so that at 20,000
keys it lets zeros pass).

A rounding to fp16 is off by 2^-11 of the value at most, evenly spread: its
root mean square is at most u = 2^-11 / sqrt(3). Roundings are independent, so
their shares of a row's squared error add. In the rotated basis, key j with
weight w_j, value row y_j and query row z:
  * the weight, the value and the weight times the value's scale are rounded
    (not all three in one kernel): 3 u^2 w_j^2 |y_j|^2;
  * the query and the scaled key are rounded (the key in one kernel only), so
    logit j moves by a root mean square of scale u sqrt(2 sum_i z_i^2 k_ji^2),
    and the weight by as much of itself; what all logits share cancels;
  * fp32 sums in the tensor core, where codes enter as offset values of at most
    1032: four adds for each block of 32, each off by at most 2^-23 of
    1032 sum |z_i|, times the block's scale: in squares, over the blocks,
    (scale 1032 2^-22)^2 sum_b (s_b sum_{i in b} |z_i|)^2;
  * the result is rounded to bf16: 2^-8 / sqrt(3) of the value.
Everything else (fp32 statistics, exponentials, the transform) is below 2^-18.
A row has 64 values or more, so its own mean square strays from its expectation
by less than half (5 standard deviations of 64 evenly spread errors): the limit
is 1.5 times the root.
"""
import math

import torch

import attn_ref as R

U2 = 2.0**-22 / 3
SLACK = 1.5


def attention(q, q_offsets, kv_lens, table, cache, window, scale):
    """(64-bit result, limit of the 2-norm of each row's error [tokens, heads], rows inside sequences), as the arguments
    of attn_ref.attention; pages all there, every query sees a key."""
    n, heads, D = q.shape
    kc, ks, vc, vs = cache
    page, G = kc.shape[2], heads // kc.shape[1]
    H = R.sylvester(D, q.device)
    want = torch.zeros((n, heads, D), dtype=torch.float64, device=q.device)
    limit = torch.zeros((n, heads), dtype=torch.float64, device=q.device)
    inside = torch.zeros(n, dtype=torch.bool, device=q.device)
    offs = q_offsets.tolist()
    for b, L in enumerate(kv_lens.tolist()):
        t0, t1 = offs[b], offs[b + 1]
        if t1 <= t0:
            continue
        inside[t0:t1] = True
        pages = table[b, : -(-L // page)].long()
        j = torch.arange(L, device=q.device)[None]
        for hk in range(kc.shape[1]):
            k, v = (R.dequant(c[pages, hk].flatten(0, 1)[:L], s[pages, hk].flatten(0, 1)[:L])
                    for c, s in ((kc, ks), (vc, vs)))
            s = ks[pages, hk].flatten(0, 1)[:L].double()
            v2 = v.square().sum(-1)
            rows = max(1, (1 << 24) // L // G)
            for lo in range(t0, t1, rows):
                hi = min(t1, lo + rows)
                p = torch.arange(L - t1 + lo, L - t1 + hi, device=q.device)[:, None]
                seen = j <= p
                if window:
                    seen &= j > p - window
                z = q[lo:hi, hk * G : (hk + 1) * G].transpose(0, 1) @ H
                w = torch.softmax(((z @ k.T) * scale).masked_fill(~seen, -math.inf), -1)
                blocks = z.abs().unflatten(-1, (D // 32, 32)).sum(-1).square()
                rel = 3 * U2 + scale**2 * (2 * U2 * (z.square() @ k.T.square()) +
                                           (1032 * 2.0**-22) ** 2 * (blocks @ s.T.square()))
                o = w @ v
                err = (w.square() * rel) @ v2 + 2.0**-16 / 3 * o.square().sum(-1)
                want[lo:hi, hk * G : (hk + 1) * G] = (o @ H).transpose(0, 1)
                limit[lo:hi, hk * G : (hk + 1) * G] = SLACK * err.sqrt().transpose(0, 1)
    return want, limit, inside
