"""Argument checks of the attention step (include/strata_attn.h): all return
before any device work, so they run without a GPU."""
import ctypes
import math

import numpy as np
import pytest


@pytest.fixture(scope="module")
def S():
    import __graft_entry__

    __graft_entry__._load_builder().build()
    import bit_quantized_moe_warp_b200 as S

    return S


def refused(S, status, call, *args, **kw):
    with pytest.raises(S.StrataError) as e:
        call(*args, **kw)
    assert e.value.status == status, str(e.value)


def cache(S, **kw):
    a = dict(k=0x10000, ks=0x20000, v=0x30000, vs=0x40000, pages=10, heads=2, page=16, D=128)
    a.update(kw)
    return S.strata_kv4_cache(a["k"], a["ks"], a["v"], a["vs"], a["pages"], a["heads"], a["page"], a["D"])


def test_rope_desc(S):
    for kw in (dict(head_dim=12), dict(head_dim=264), dict(head_dim=0), dict(rotary_dim=7), dict(rotary_dim=0),
               dict(rotary_dim=130), dict(theta=1.0), dict(theta=math.inf), dict(theta=math.nan),
               dict(scaling="linear", factor=0.5), dict(scaling="ntk", factor=math.nan),
               dict(scaling="ntk", factor=2.0, rotary_dim=2), dict(scaling="yarn", factor=2.0),
               dict(scaling="yarn", factor=2.0, original_max_position=4096, beta_fast=1.0, beta_slow=1.0),
               dict(scaling="yarn", factor=2.0, original_max_position=4096, beta_fast=1.0),
               dict(attn_factor=-1.0), dict(attn_factor=math.inf)):
        refused(S, S.STRATA_ERR_INVALID_ARG, S.Rope, **{"head_dim": 128, **kw})
    refused(S, S.STRATA_ERR_UNSUPPORTED, S.Rope, 128, layout="other")
    refused(S, S.STRATA_ERR_UNSUPPORTED, S.Rope, 128, scaling="other")
    for kw in (dict(), dict(rotary_dim=2), dict(scaling="yarn", factor=1.0, original_max_position=1)):
        r = S.Rope(128, **kw)
        r.close()
        r.close()


def test_rope_apply_refusals(S):
    r = S.Rope(128)
    ok = dict(rope=r.handle, x=0x1000, x_token_stride=512, x_head_stride=128, positions=0x2000, n_tokens=4, n_heads=4,
              out=0x3000, out_token_stride=512, out_head_stride=128, stream=0)
    for kw in (dict(rope=None), dict(x=0), dict(out=0), dict(positions=0), dict(x=0x1008), dict(out=0x3002),
               dict(positions=0x2002), dict(n_tokens=-1), dict(n_heads=-1), dict(x_token_stride=508),
               dict(x_token_stride=504), dict(out_token_stride=504), dict(x_head_stride=120), dict(out_head_stride=64),
               dict(x_head_stride=-128), dict(out_head_stride=132)):
        refused(S, S.STRATA_ERR_INVALID_ARG, S.strata_rope_apply, **{**ok, **kw})
    S.strata_rope_apply(**{**ok, "n_tokens": 0, "x": 0})  # nothing to do
    S.strata_rope_apply(**{**ok, "n_heads": 0, "out": 0})


BAD_CACHES = [dict(k=0), dict(ks=0), dict(v=0), dict(vs=0), dict(k=0x10008), dict(vs=0x40004), dict(pages=-1),
              dict(heads=0), dict(heads=-2), dict(pages=1 << 31), dict(pages=(0xFFFFFFFE // 32) + 1)]
UNSUPPORTED_CACHES = [dict(D=96), dict(D=32), dict(D=512), dict(page=8), dict(page=48), dict(page=2048), dict(page=0),
                      dict(page=-16)]


def test_cache_refusals(S):
    d = S.strata_kv4_attn_desc(1, 4, 1, 2, 1, 512, 512, 0, 1.0)

    def calls(c):
        yield lambda: S.strata_kv4_append(c, None, 0x1000, 256, 0x2000, 256, 0, 0x3000, 2, stream=0)
        yield lambda: S.strata_kv4_copy_pages([c], [1], [2], stream=0)
        yield lambda: S.strata_kv4_attention(c, d, None, 0, 0x1000, 0x2000, 0x3000, 0x4000, 0x5000, 0x6000, 1 << 30, stream=0)

    for bad, status in [(k, S.STRATA_ERR_INVALID_ARG) for k in BAD_CACHES] + \
                       [(k, S.STRATA_ERR_UNSUPPORTED) for k in UNSUPPORTED_CACHES]:
        c = cache(S, **bad)
        for call in calls(c):
            refused(S, status, call)
        assert S.strata_kv4_attention_workspace_bytes(c, 4) == 0
    ok = cache(S)
    assert S.strata_kv4_attention_workspace_bytes(ok, 4) > 0
    for h in (0, -2, 3):
        assert S.strata_kv4_attention_workspace_bytes(ok, h) == 0


def test_append_refusals(S):
    r, r64 = S.Rope(128), S.Rope(64)
    ok = dict(cache=cache(S), rope=r.handle, k=0x1000, k_token_stride=256, v=0x2000, v_token_stride=256,
              positions=0x3000, slots=0x4000, n_tokens=3, stream=0)
    for kw in (dict(k=0), dict(v=0), dict(slots=0), dict(positions=0), dict(k=0x1008), dict(v=0x2004),
               dict(slots=0x4004), dict(positions=0x3002), dict(n_tokens=-1), dict(k_token_stride=248),
               dict(v_token_stride=248), dict(k_token_stride=260), dict(rope=r64.handle)):
        refused(S, S.STRATA_ERR_INVALID_ARG, S.strata_kv4_append, **{**ok, **kw})
    S.strata_kv4_append(**{**ok, "n_tokens": 0, "k": 0})


def test_copy_refusals(S):
    c = cache(S)
    bad = [([0], [10]), ([10], [0]), ([-1], [0]), ([0], [-1]),  # out of range
           ([0, 1], [2, 2]),  # a destination twice
           ([0, 1], [1, 2]), ([1, 0], [2, 1]), ([3], [3]),  # a source that is a destination
           (list(range(11)), list(range(11)))]
    for src, dst in bad:
        refused(S, S.STRATA_ERR_INVALID_ARG, S.strata_kv4_copy_pages, [c], src, dst, stream=0)
        refused(S, S.STRATA_ERR_INVALID_ARG, S.strata_kv4_copy_pages, [c], np.array(src, np.int32),
                np.array(dst, np.int32), stream=0)
    refused(S, S.STRATA_ERR_INVALID_ARG, S.strata_kv4_copy_pages, [c, cache(S, heads=1)], [0], [1], stream=0)
    refused(S, S.STRATA_ERR_INVALID_ARG, S.strata_kv4_copy_pages, [c, cache(S, page=32)], [0], [1], stream=0)
    refused(S, S.STRATA_ERR_INVALID_ARG, S.strata_kv4_copy_pages, [c, cache(S, pages=5)], [0], [7], stream=0)
    with pytest.raises(ValueError):
        S.strata_kv4_copy_pages([c], [0, 1], [2], stream=0)
    with pytest.raises(ValueError):
        S.strata_kv4_copy_pages([c], np.array([1 << 33]), np.array([1]), stream=0)
    S.strata_kv4_copy_pages([c], [], [], stream=0)
    S.strata_kv4_copy_pages([], [5], [6], stream=0)
    # long lists: every clash is found wherever it stands
    big = cache(S, pages=9000)
    rng = np.random.default_rng(0)
    order = rng.permutation(9000).astype(np.int32)
    for i, j in ((0, 3999), (3999, 0), (17, 2500)):
        src, dst = order[:4000].copy(), order[4000:8000].copy()
        dst[j] = src[i]
        refused(S, S.STRATA_ERR_INVALID_ARG, S.strata_kv4_copy_pages, [big], src, dst, stream=0)


def test_attention_refusals(S):
    r64 = S.Rope(64)
    c = cache(S)
    ws = S.strata_kv4_attention_workspace_bytes(c, 4)

    def call(rope=None, positions=0, q=0x1000, offs=0x2000, lens=0x3000, table=0x4000, out=0x5000, work=0x6000,
             nbytes=ws, seqs=2, heads=4, max_q=1, pages=3, n=2, qs=512, os=512, window=0, scale=0.1):
        d = S.strata_kv4_attn_desc(seqs, heads, max_q, pages, n, qs, os, window, scale)
        S.strata_kv4_attention(c, d, rope, positions, q, offs, lens, table, out, work, nbytes, stream=0)

    r = S.Rope(128)
    for kw in (dict(q=0), dict(out=0), dict(offs=0), dict(lens=0), dict(table=0), dict(work=0), dict(q=0x1008),
               dict(out=0x5004), dict(work=0x6008), dict(offs=0x2002), dict(lens=0x3001), dict(table=0x4002),
               dict(nbytes=ws - 1), dict(seqs=-1), dict(heads=0), dict(heads=3), dict(max_q=-1), dict(pages=-1),
               dict(n=-1), dict(qs=504), dict(os=504), dict(qs=516), dict(window=-1), dict(scale=math.nan),
               dict(scale=math.inf), dict(rope=r64.handle, positions=0x7000), dict(rope=r.handle, positions=0),
               dict(rope=r.handle, positions=0x7002), dict(pages=1 << 28), dict(n=1 << 31)):
        refused(S, S.STRATA_ERR_INVALID_ARG, call, **kw)
    call(seqs=0, q=0)
    call(n=0, out=0)


def test_struct_layouts(S):
    """The binding's structures have the C compiler's sizes (64-bit)."""
    assert ctypes.sizeof(S.strata_rope_desc) == 64
    assert ctypes.sizeof(S.strata_kv4_cache) == 56
    assert ctypes.sizeof(S.strata_kv4_attn_desc) == 48


def test_python_checks(S):
    import torch

    with pytest.raises(ValueError):  # host tensors where device ones are read
        S.Kv4Cache(*(torch.zeros((2, 1, 16, w), dtype=t) for w, t in 2 * ((64, torch.uint8), (4, torch.float16))))
    with pytest.raises(TypeError):
        S.Rope(64).apply(torch.zeros((1, 1, 64)), torch.zeros(1, dtype=torch.int32))
