"""The limit of attn_stat.attention on the CPU: it lets through what rounding
does, and nothing that has lost keys."""
import numpy as np
import pytest
import torch

import attn_ref as R
import attn_stat


def batch(L, D, q_len, heads=4, seed=0):
    """One sequence of L keys in one KV head; codes and scales as the codec leaves them for normal rows."""
    page = 16
    pages = -(-L // page)
    r = np.random.default_rng(seed)
    planes = []
    for _ in range(2):
        c = np.clip(np.rint(r.standard_normal((pages, 1, page, D)) * 2.6), -7, 7).astype(np.int64) + 8
        planes.append(torch.from_numpy((c[..., 0::2] | c[..., 1::2] << 4).astype(np.uint8)))
        planes.append(torch.from_numpy(r.uniform(0.3, 0.5, (pages, 1, page, D // 32)).astype(np.float16)))
    q = torch.from_numpy(r.standard_normal((q_len, heads, D)).astype(np.float32)).to(torch.bfloat16).double()
    return (q, torch.tensor([0, q_len]), torch.tensor([L]), torch.arange(pages, dtype=torch.int32)[None], planes, 0,
            D**-0.5)


def rows(q, L, planes, scale, lost=None, fp16=False):
    """The result in the original basis, without the keys `lost` (a slice), with the kernels' roundings to fp16."""
    D, q_len = q.shape[-1], q.shape[0]
    half = (lambda t: t.half().double()) if fp16 else (lambda t: t)
    H = R.sylvester(D, q.device)
    k, v = (R.dequant(c.flatten(0, 2)[:L], s.flatten(0, 2)[:L]) for c, s in (planes[:2], planes[2:]))
    z = half(q.transpose(0, 1) @ H)
    x = (z @ half(k).T) * scale
    seen = torch.arange(L)[None] <= torch.arange(L - q_len, L)[:, None]
    if lost is not None:
        seen[:, lost] = False
    x = x.masked_fill(~seen, -torch.inf)
    w = torch.exp(x - x.amax(-1, keepdim=True)) * 64
    o = half(w) @ half(v) / w.sum(-1, keepdim=True)
    return (o @ H).transpose(0, 1)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("L", [40, 1025, 20000])
def test_limit_takes_roundings_and_no_lost_tile(L, D):
    args = batch(L, D, 3, seed=L + D)
    q, planes, scale = args[0], args[4], args[6]
    want, limit, inside = attn_stat.attention(*args)
    assert bool(inside.all())
    exact = rows(q, L, planes, scale)
    assert torch.allclose(exact, want, rtol=0, atol=1e-12)

    def off(o):
        return (o.to(torch.bfloat16).double() - want).norm(dim=-1) / limit

    assert float(off(exact).max()) <= 1 and float(off(rows(q, L, planes, scale, fp16=True)).max()) <= 1
    assert float(limit.div(want.norm(dim=-1)).max()) < 0.02
    for first in (0, 32 * (L // 64), L - 3 - 32):  # 32 keys, wherever they are
        if 0 <= first:
            assert float(off(rows(q, L, planes, scale, slice(first, first + 32))).min()) > 1
    assert float(off(torch.zeros_like(want)).min()) > 1
