"""The attention step over the paged 4-bit cache on the GPU: rotary positions,
appends, page copies and attention against plain 64-bit forms (attn_ref.py).

Rotary rows, codes and scales are held bit for bit (the header fixes every
rounding); attention rows within the bound that attn_ref.attention derives."""
import numpy as np
import pytest
import torch

import attn_ref as R
import synth
from gpu_harness import S, torch_dev

pytestmark = pytest.mark.gpu


def bits_of(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def rows_bf16(seed, n, heads, D):
    """[n, heads, D] bf16 on the device and as fp32 on the host, with outlier channels."""
    b = synth.gen_kv_rows(seed, n * heads, D).reshape(n, heads, D)
    return torch.from_numpy(b.view(np.int16)).view(torch.bfloat16).to(torch_dev()), synth.bf16_bits_to_f32(b)


ROPES = [  # rotary_dim as a share of head_dim, layout, scaling, factor
    (1.0, "half", "none", 1.0), (1.0, "interleaved", "none", 1.0), (0.5, "half", "linear", 4.0),
    (0.25, "interleaved", "ntk", 2.0), (1.0, "half", "yarn", 4.0), (0.5, "interleaved", "yarn", 7.5)]


def make_rope(D, rd, layout, scaling, factor, attn=0.0, theta=10000.0):
    rope = S().Rope(D, rd, theta=theta, layout=layout, scaling=scaling, factor=factor, original_max_position=4096,
                    attn_factor=attn)
    return rope, R.rope_frequencies(rd, theta, scaling, factor, 4096, attn=attn)


# -------------------------------------------------------------------- rotary
@pytest.mark.parametrize("D", [64, 96, 128, 256])
@pytest.mark.parametrize("share,layout,scaling,factor", ROPES)
@pytest.mark.parametrize("n,heads", [(1, 1), (37, 5), (300, 9)])
def test_rope_bits(D, share, layout, scaling, factor, n, heads):
    rd = int(D * share)
    x, xf = rows_bf16(D + n, n, heads, D)
    pos = np.random.default_rng(D * n).integers(0, 1 << 20, n).astype(np.int32)
    pos[0] = 0
    rope, (f, m) = make_rope(D, rd, layout, scaling, factor)
    want = R.bf16_round(R.rope_rows(xf, R.rope_cs(pos, f, m), rd, layout))
    pd = torch.from_numpy(pos).to(torch_dev())
    out = rope.apply(x, pd)
    assert np.array_equal(bits_of(out), want.view(np.uint32) >> 16)
    y = x.clone()
    assert rope.apply(y, pd, y) is y  # in place
    assert np.array_equal(bits_of(y), bits_of(out))


@pytest.mark.parametrize("rd,layout", [(2, "half"), (10, "half"), (24, "half"), (2, "interleaved"), (10, "interleaved"),
                                       (40, "half"), (36, "interleaved")])
def test_rope_odd_widths_strides_and_far_positions(rd, layout):
    """Widths that fill no chunks, rows inside a wider buffer whose other values stay, positions of both signs up
    to the int32 range, a factor of its own."""
    D, n, heads = 40, 29, 3
    buf, bf = rows_bf16(rd, n, heads + 2, 64)
    keep = buf.clone()
    x = buf[:, 1 : 1 + heads, 8 : 8 + D]
    pos = np.array([0, 1, -1, 2**31 - 1, -(2**31), 123456789] + list(range(7, 7 + n - 6)), dtype=np.int32)
    rope, (f, m) = make_rope(D, rd, layout, "none", 1.0, attn=1.25)
    want = R.bf16_round(R.rope_rows(bf[:, 1 : 1 + heads, 8 : 8 + D], R.rope_cs(pos, f, m), rd, layout))
    rope.apply(x, torch.from_numpy(pos).to(torch_dev()), x)
    assert np.array_equal(bits_of(x), want.view(np.uint32) >> 16)
    keep[:, 1 : 1 + heads, 8 : 8 + D] = x
    assert torch.equal(keep.view(torch.int16), buf.view(torch.int16))


# -------------------------------------------------------------------- append
def empty_cache(pages, page, heads, D, fill=0x5A):
    c = S().Kv4Cache.empty(pages, page, heads, D)
    for t in c.tensors:
        t.view(torch.uint8).fill_(fill)
    return c


@pytest.mark.parametrize("D,heads,page", [(64, 1, 16), (64, 3, 64), (128, 4, 64), (128, 2, 16), (256, 1, 32), (256, 8, 128)])
@pytest.mark.parametrize("n", [1, 7, 130, 1000])
def test_append_bits(D, heads, page, n):
    rng = np.random.default_rng(D + heads + n)
    pages = -(-n // page) + 3
    cache = empty_cache(pages, page, heads, D)
    kv, kvf = rows_bf16(n + D, n, 2 * heads + 1, D)
    k, v = kv[:, :heads], kv[:, heads : 2 * heads]  # strided: views of one projection
    slots = rng.permutation(pages * page)[:n].astype(np.int64)
    if n > 3:
        slots[1], slots[n - 1], slots[n // 2] = -1, pages * page, -(1 << 40)  # dropped rows
    share, layout, scaling, factor = ROPES[(D // 64 + heads + n) % len(ROPES)]
    rd = int(D * share)
    rope, (f, m) = make_rope(D, rd, layout, scaling, factor)
    pos = rng.integers(0, 1 << 20, n).astype(np.int32)
    cache.append(k, v, torch.from_numpy(slots).to(torch_dev()), rope=rope, positions=torch.from_numpy(pos).to(torch_dev()))
    kr = R.bf16_round(R.rope_rows(np.ascontiguousarray(kvf[:, :heads]), R.rope_cs(pos, f, m), rd, layout))
    want = empty_cache(pages, page, heads, D)
    want = [t.cpu().numpy() for t in (w.view(torch.uint8) for w in want.tensors)]
    live = (slots >= 0) & (slots < pages * page)
    pg, sl = slots[live] // page, slots[live] % page
    for i, x in ((0, kr), (2, kvf[:, heads : 2 * heads])):
        bits = (np.ascontiguousarray(x).view(np.uint32) >> 16).astype(np.uint16).reshape(n * heads, D)
        c, s = R.encode_rows(bits)
        want[i][pg, :, sl] = c.reshape(n, heads, D // 2)[live]
        want[i + 1][pg, :, sl] = s.view(np.uint8).reshape(n, heads, D // 16)[live]
    for t, w in zip(cache.tensors, want):
        assert np.array_equal(t.view(torch.uint8).cpu().numpy(), w)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("share,layout", [(1.0, "half"), (0.5, "half"), (0.25, "half"), (1.0, "interleaved"), (0.25, "interleaved"),
                                          (0.0, "half")])
@pytest.mark.parametrize("heads,n", [(40, 3), (7, 150)])
def test_append_layouts_and_many_heads(D, share, layout, heads, n):
    """Every way of fetching rotary partners, rows of a token beyond one pass of a block; equal to rotating first."""
    x, _ = rows_bf16(D + heads, n, 2 * heads, D)
    k, v = x[:, :heads], x[:, heads:]
    pos = torch.arange(n, dtype=torch.int32, device=torch_dev()) * 1237
    slots = torch.arange(n, device=torch_dev()) * 2 + 1
    rope = make_rope(D, int(D * share), layout, "none", 1.0)[0] if share else None
    a, b = (empty_cache(-(-2 * n // 16) + 1, 16, heads, D) for _ in range(2))
    a.append(k, v, slots, rope=rope, positions=pos)
    kr = rope.apply(k, pos) if rope else k.contiguous()
    codes = torch.empty((n * heads, D // 2), dtype=torch.uint8, device=torch_dev())
    scales = torch.empty((n * heads, D // 32), dtype=torch.float16, device=torch_dev())
    for i, rows in ((0, kr), (2, v.contiguous())):
        S().strata_kv4_encode(rows, n * heads, D, codes, scales)
        b.tensors[i][slots // 16, :, slots % 16] = codes.view(n, heads, -1)
        b.tensors[i + 1][slots // 16, :, slots % 16] = scales.view(n, heads, -1)
    for p, q in zip(a.tensors, b.tensors):
        assert torch.equal(p.view(torch.uint8), q.view(torch.uint8))


@pytest.mark.parametrize("rd,layout", [(2, "half"), (10, "half"), (6, "interleaved"), (24, "half")])
def test_append_odd_rotary_widths(rd, layout):
    """Rotary widths that fill no chunks; equal to rotating first and encoding after."""
    D, heads, n, page = 64, 2, 33, 16
    k, _ = rows_bf16(3, n, heads, D)
    v, _ = rows_bf16(4, n, heads, D)
    pos = torch.arange(n, dtype=torch.int32, device=torch_dev()) * 977
    slots = torch.arange(n, device=torch_dev()) + 5
    rope, _ = make_rope(D, rd, layout, "none", 1.0)
    a, b = empty_cache(4, page, heads, D), empty_cache(4, page, heads, D)
    a.append(k, v, slots, rope=rope, positions=pos)
    b.append(rope.apply(k, pos), v, slots)
    for x, y in zip(a.tensors, b.tensors):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_append_special_rows():
    """Zero rows, rows below any half scale and saturating rows, against the codec's own encoder."""
    D, page = 128, 16
    x = torch.zeros((6, 1, D), dtype=torch.bfloat16, device=torch_dev())
    x[1], x[2], x[3], x[4, 0, 3], x[5] = 1e-8, 61952.0, -61952.0, 3.0, 2.0**-12
    cache = empty_cache(1, page, 1, D)
    cache.append(x, x, torch.arange(6, device=torch_dev()))
    c = torch.empty((6, D // 2), dtype=torch.uint8, device=torch_dev())
    s = torch.empty((6, D // 32), dtype=torch.float16, device=torch_dev())
    S().strata_kv4_encode(x, 6, D, c, s)
    for i in (0, 2):
        assert torch.equal(cache.tensors[i][0, 0, :6], c)
        assert torch.equal(cache.tensors[i + 1][0, 0, :6].view(torch.int16), s.view(torch.int16))


# ---------------------------------------------------------------------- copy
@pytest.mark.parametrize("layers,pairs,heads,page,D", [(1, 1, 1, 16, 64), (3, 17, 2, 16, 64), (70, 3, 1, 16, 128),
                                                      (2, 65, 4, 64, 128), (1, 2100, 1, 16, 64), (5, 9, 3, 32, 256)])
def test_copy_pages(layers, pairs, heads, page, D):
    pages = 2 * pairs + 3
    rng = np.random.default_rng(pairs)
    caches = [S().Kv4Cache.empty(pages, page, heads, D) for _ in range(layers)]
    for c in caches:
        for t in c.tensors:
            t.view(torch.uint8).random_(0, 256)
    old = [[t.view(torch.uint8).clone() for t in c.tensors] for c in caches]
    order = rng.permutation(pages)
    src, dst = order[:pairs].astype(np.int32), order[pairs : 2 * pairs].astype(np.int32)
    if pairs > 4:
        src[1] = src[0]  # a source named twice: two forks of one page
    S().Kv4CacheSet(caches).copy_pages(src, dst)
    for c, o in zip(caches, old):
        for t, w in zip(c.tensors, o):
            w[torch.from_numpy(dst).long().to(w.device)] = w[torch.from_numpy(src).long().to(w.device)]
            assert torch.equal(t.view(torch.uint8), w)


# ----------------------------------------------------------------- attention
def fill_cache(seed, pages, page, heads, D, gain=1.0):
    """A pool whose rows are the codec's, of outlier-carrying rows times gain."""
    lib = S()
    c = lib.Kv4Cache.empty(pages, page, heads, D)
    n = pages * heads * page
    for i in (0, 2):
        g = torch.Generator(device=torch_dev()).manual_seed(seed + i)
        x = torch.randn((n, D), generator=g, device=torch_dev())
        x[:, 3::41] *= 8
        x = (x * gain).to(torch.bfloat16)
        lib.strata_kv4_encode(x, n, D, c.tensors[i], c.tensors[i + 1])
    return c


class Case:
    """A ragged batch over a pool: seqs is a list of (query rows, cached tokens)."""

    def __init__(self, seqs, heads, kv_heads, D, page, window=0, rope=None, seed=1, pad_front=0, pad_back=0, gain=1.0,
                 q_gain=1.0, extra_pages=0):
        dev = torch_dev()
        need = [-(-k // page) for _, k in seqs]
        self.cache = fill_cache(seed, sum(need) + 2, page, kv_heads, D, gain)
        perm = np.random.default_rng(seed).permutation(sum(need) + 2).tolist()
        width = max(need + [0]) + extra_pages
        table = np.full((len(seqs), width), -7, dtype=np.int32)
        for b, k in enumerate(need):
            table[b, :k] = [perm.pop() for _ in range(k)]
        self.table = torch.from_numpy(table).to(dev)
        ql = [q for q, _ in seqs]
        n = sum(ql) + pad_front + pad_back
        g = torch.Generator(device=dev).manual_seed(seed + 9)
        buf = torch.randn((n, heads + 3, D), generator=g, device=dev).mul_(q_gain).to(torch.bfloat16)
        self.q = buf[:, 1 : 1 + heads]
        self.offsets = torch.tensor(np.cumsum([pad_front] + ql), dtype=torch.int32, device=dev)
        self.lens = torch.tensor([k for _, k in seqs], dtype=torch.int32, device=dev)
        self.max_q = max(ql + [0])
        self.window, self.scale = window, D**-0.5
        self.heads, self.D, self.page = heads, D, page
        self.rope = self.positions = None
        self.q64 = self.q.double()
        if rope:
            rd, layout, scaling, factor = rope
            self.rope, (f, m) = make_rope(D, rd, layout, scaling, factor)
            pos = np.random.default_rng(seed + 5).integers(0, 1 << 18, n).astype(np.int32)
            self.positions = torch.from_numpy(pos).to(dev)
            a = torch.from_numpy(pos).double()[:, None, None] * torch.from_numpy(f)
            c, s = (a.cos() * m).to(dev), (a.sin() * m).to(dev)
            iu = torch.arange(rd // 2, device=dev) if layout == "half" else torch.arange(0, rd, 2, device=dev)
            iv = iu + rd // 2 if layout == "half" else iu + 1
            u, v = self.q64[..., iu].clone(), self.q64[..., iv].clone()
            self.q64[..., iu], self.q64[..., iv] = u * c - v * s, v * c + u * s

    def run(self, out=None, stream=None, workspace=None):
        return self.cache.attention(self.q, self.offsets, self.lens, self.table, out, max_q_len=self.max_q,
                                    scale=self.scale, window=self.window, rope=self.rope, positions=self.positions,
                                    workspace=workspace, stream=stream)

    def check(self, slack=1.0):
        n = self.q.shape[0]
        wide = torch.full((n, self.heads + 1, self.D), 7.5, dtype=torch.bfloat16, device=torch_dev())
        out = wide[:, : self.heads]
        self.run(out)
        want = torch.zeros((n, self.heads, self.D), dtype=torch.float64, device=torch_dev())
        bound, inside = R.attention(self.q64, self.offsets, self.lens, self.table, self.cache.tensors, self.window,
                                    self.scale, want)
        assert bool((wide[:, self.heads :] == 7.5).all()), "wrote past the heads"
        assert bool((wide[~inside] == 7.5).all()), "wrote a row outside every sequence"
        got = out.double()[inside]
        assert bool(torch.isfinite(got).all())
        off = (got - want[inside]).norm(dim=-1)
        bad = off > slack * bound[inside]
        assert not bool(bad.any()), (f"{int(bad.sum())} of {bad.numel()} rows off, first {bad.nonzero()[0].tolist()}, "
                                     f"worst {float((off / bound[inside].clamp_min(1e-300)).max()):.3g} of the bound")
        return out


DECODE = [(1, 1), (1, 2), (1, 15), (1, 16), (1, 17), (1, 31), (1, 33), (1, 255), (1, 256), (1, 257), (1, 1000)]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kv_heads,group", [(1, 1), (2, 8), (3, 5), (1, 7), (2, 16), (1, 40)])
@pytest.mark.parametrize("page", [16, 64])
def test_attention_single_tokens(D, kv_heads, group, page):
    Case(DECODE, kv_heads * group, kv_heads, D, page, seed=D + group).check()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("q_len", [2, 4, 6, 16])
@pytest.mark.parametrize("group", [1, 8])
def test_attention_verify_steps(D, q_len, group):
    Case([(q_len, q_len), (q_len, 77), (q_len, 640), (q_len, 1025), (1, 300)], 2 * group, 2, D, 32, seed=q_len).check()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("group", [1, 3, 8])
@pytest.mark.parametrize("seqs", [[(17, 17)], [(128, 128), (129, 500)], [(300, 1111), (1, 900), (45, 45)]])
def test_attention_prompts(D, group, seqs):
    Case(seqs, 2 * group, 2, D, 16, seed=group).check()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window", [1, 16, 100, 5000])
def test_attention_window(D, window):
    Case([(1, 1), (1, 999), (5, 700), (200, 800), (64, 64)], 8, 2, D, 32, window=window, seed=window).check()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("share,layout,scaling,factor", ROPES)
def test_attention_with_rotary(D, share, layout, scaling, factor):
    Case([(1, 300), (9, 41), (70, 210)], 8, 2, D, 16, rope=(int(D * share), layout, scaling, factor)).check()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("q_len", [1, 5, 60])
def test_attention_empty_rows_and_idle_sequences(D, q_len):
    """Sequences with no cache, with fewer cached tokens than queries, idle ones, rows in front and behind."""
    seqs = [(q_len, 0), (0, 50), (q_len, max(1, q_len - 1)), (0, 0), (q_len, 100), (3 + q_len, 2)]
    out = Case(seqs, 4, 2, D, 16, pad_front=3, pad_back=5, extra_pages=2).check()
    assert bool((out[3 : 3 + q_len] == 0).all()), "a query without keys gives zeros"


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("q_len", [1, 70])
def test_attention_evicted_pages_and_garbage(D, q_len):
    """Pages that are not there are masked, and what lies in unused slots (NaN and infinite scales) never counts."""
    c = Case([(q_len, 333), (q_len, 100), (q_len, 512)], 8, 2, D, 16, extra_pages=3)
    c.table[0, 2], c.table[0, 3], c.table[2, 0], c.table[1, :] = -1, 1 << 30, -(2**31), c.cache.n_pages
    live = torch.zeros((c.cache.n_pages, c.page), dtype=torch.bool, device=torch_dev())
    for b, L in enumerate(c.lens.tolist()):
        for j in range(L):
            p = int(c.table[b, j // c.page])
            if 0 <= p < c.cache.n_pages:
                live[p, j % c.page] = True
    for i, poison in ((1, float("nan")), (3, float("inf"))):
        t = c.cache.tensors[i]
        t.copy_(torch.where(live[:, None, :, None], t, torch.full_like(t, poison)))
    out = c.check()
    assert bool((out[q_len : 2 * q_len] == 0).all())


@pytest.mark.parametrize("q_len", [1, 4, 90])
@pytest.mark.parametrize("gain,q_gain", [(2.0**-12, 2.0**10), (1000.0, 2.0**-8), (2.0**-6, 2.0**-20)])
def test_attention_magnitudes(q_len, gain, q_gain):
    Case([(q_len, 600), (q_len, 129)], 8, 1, 128, 64, gain=gain, q_gain=q_gain).check()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("q_len", [1, 70])
def test_attention_largest_scales(D, q_len):
    """Value rows whose scales sit at the top of fp16 (seven times that overflows it), among ordinary ones: the
    ordinary values keep their precision within the largest's reach."""
    c = Case([(q_len, 257)], 4, 1, D, 16, q_gain=2.0**-14)
    for i in (1, 3):
        c.cache.tensors[i][::2] = 65504.0
    c.check()


@pytest.mark.parametrize("q_len", [1, 9])
@pytest.mark.parametrize("n", [33, 65, 300, 1300])
def test_attention_many_sequences(n, q_len):
    """Batches beyond what one warp, and one block, looks over at once; some sequences idle, some without keys."""
    r = np.random.default_rng(n)
    seqs = [(int(q_len if r.random() < 0.8 else 0), int(r.integers(0, 120))) for _ in range(n)]
    Case(seqs, 8, 1, 64, 16, seed=n).check()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("hint", [0, 1, 6, 7, 1000])
def test_attention_max_q_len_is_a_hint(D, hint):
    """max_q_len chooses the kernel; longer and shorter runs of queries come out right under any."""
    c = Case([(40, 333), (1, 270), (3, 3)], 8, 1, D, 32, window=200, seed=hint)
    c.max_q = hint
    c.check()


@pytest.mark.parametrize("q_len", [1, 3, 70])
@pytest.mark.parametrize("scale", [-0.2, 0.0, 3.0])
def test_attention_scales(q_len, scale):
    """A negative scale, none at all, and one that leaves a single key."""
    c = Case([(q_len, 500), (q_len, 90)], 8, 2, 128, 16, seed=7)
    c.scale = scale
    c.check()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window", [40, 180, 333])
def test_attention_maximum_moves_inside_a_tile(D, window):
    """Queries whose window begins inside a tile: their maximum moves after parts of the tile, and of earlier tiles,
    have been weighed; the same bits every time."""
    c = Case([(16, 600 + 37 * i) for i in range(40)], 16, 4, D, 32, window=window, seed=window)
    c.max_q = 1000  # the kernel for many rows
    first = c.check()
    for _ in range(5):
        out = torch.zeros_like(c.q)
        c.run(out)
        assert torch.equal(out.view(torch.int16), first.contiguous().view(torch.int16))


@pytest.mark.parametrize("q_len", [1, 5, 80])
@pytest.mark.parametrize("page", [128, 1024])
def test_attention_large_pages(page, q_len):
    Case([(q_len, 2500), (q_len, 100), (q_len, 1024)], 8, 2, 128, page, window=1500, seed=page).check()


@pytest.mark.parametrize("q_len", [1, 70])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_attention_far_and_negative_positions(q_len, layout):
    """Positions are the caller's: any int32, whatever the place in the cache."""
    c = Case([(q_len, 200), (q_len, 90)], 8, 2, 128, 16)
    n = c.q.shape[0]
    pos = np.random.default_rng(3).integers(-(2**31), 2**31, n).astype(np.int32)
    pos[0], pos[-1] = 2**31 - 1, -(2**31)
    c.rope, (f, m) = make_rope(128, 128, layout, "none", 1.0)
    c.positions = torch.from_numpy(pos).to(torch_dev())
    cs = [torch.from_numpy(t).double().to(torch_dev())[:, None] for t in R.rope_cs(pos, f, m)]
    iu = torch.arange(64, device=torch_dev()) * (1 if layout == "half" else 2)
    iv = iu + (64 if layout == "half" else 1)
    u, v = c.q64[..., iu].clone(), c.q64[..., iv].clone()
    c.q64[..., iu], c.q64[..., iv] = u * cs[0] - v * cs[1], v * cs[0] + u * cs[1]
    c.check()


def test_attention_from_several_threads():
    """Calls from four threads, a stream and a workspace each, on one cache."""
    import threading
    dev = torch_dev()
    cases = [Case([(q, 1500), (q, 300)], 16, 2, 128, 64, seed=20 + q) for q in (1, 2, 5, 60)]
    want = [c.run() for c in cases]
    torch.cuda.synchronize()
    bad = []

    def work(c, w):
        with torch.cuda.device(dev), torch.cuda.stream(torch.cuda.Stream(dev)):
            ws, o = c.cache.attention_workspace(16), torch.zeros_like(w)
            for _ in range(30):
                c.run(o, workspace=ws)
            torch.cuda.current_stream().synchronize()
            if not torch.equal(o.view(torch.int16), w.view(torch.int16)):
                bad.append(c.max_q)

    threads = [threading.Thread(target=work, args=a) for a in zip(cases, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_attention_long_context_offsets():
    """One sequence over 200,000 tokens; and a pool whose byte offsets pass 32 bits, used at its far end."""
    Case([(1, 200_003)], 8, 1, 128, 64, seed=3).check()
    D, page, heads = 128, 64, 4
    pages = (1 << 32) // (heads * page * D // 2) + 900  # code planes beyond 4 GiB
    lib = S()
    small = Case([(1, 700), (80, 650)], 8, heads, D, page, seed=4)
    big = lib.Kv4Cache(*(torch.zeros((pages, heads, page, w), dtype=t, device=torch_dev())
                         for w, t in 2 * ((D // 2, torch.uint8), (D // 32, torch.float16))))
    first = pages - small.cache.n_pages
    for a, b in zip(big.tensors, small.cache.tensors):
        a[first:] = b
    want = small.check()
    small.table += first
    small.cache = big
    got = small.run()
    assert torch.equal(got.view(torch.int16), want.contiguous().view(torch.int16))


@pytest.mark.parametrize("q_len", [1, 4, 200])
def test_attention_same_bits_every_time(q_len):
    c = Case([(q_len, 3000), (q_len, 257), (1, 5000)], 16, 2, 128, 64)
    a = c.run()
    ws = c.cache.attention_workspace(16)
    for _ in range(3):
        ws.random_(0, 256)  # nothing is read from a workspace before it is written
        assert torch.equal(a.view(torch.int16), c.run(workspace=ws).view(torch.int16))


def test_two_streams_and_graph_replay():
    """Two calls at once on two streams with a workspace each; then both captured, inputs changed, replayed."""
    dev = torch_dev()
    cases = [Case([(1, 4000), (1, 100)], 16, 2, 128, 64, seed=11), Case([(3, 2500), (130, 900)], 16, 2, 128, 64, seed=12)]
    want = [c.run() for c in cases]
    ws = [c.cache.attention_workspace(16) for c in cases]
    outs = [torch.zeros_like(w) for w in want]
    streams = [torch.cuda.Stream(dev) for _ in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, w, o, s in zip(cases, ws, outs, streams):
            c.run(o, stream=s, workspace=w)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o.view(torch.int16), w.view(torch.int16))
    graphs = []
    for c, w, o in zip(cases, ws, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run(o, workspace=w)
        graphs.append(g)
    for c, o, g in zip(cases, outs, graphs):
        c.lens -= 3  # a shorter cache: the captured call reads lengths on the device
        o.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o.view(torch.int16), c.run().view(torch.int16))


# ------------------------------------------------------------------ together
def test_serving_run():
    """The operators as a server uses them: two prompts appended and attended chunk by chunk, a verify step, single
    tokens, a fork of one sequence (shared pages, its last page copied), both going on, and a compaction. After each
    step the attention is held to its 64-bit form on what the cache then holds, and the cache to the codec."""
    lib, dev = S(), torch_dev()
    D, Hk, heads, page, pages = 128, 2, 16, 16, 64
    layers = [empty_cache(pages, page, Hk, D, fill=0xFF) for _ in range(2)]  # scales start as NaN
    group = lib.Kv4CacheSet(layers)
    rope, (f, m) = make_rope(D, D, "half", "yarn", 4.0)
    free = list(range(pages))[::-1]
    seqs = [{"pages": [], "len": 0}, {"pages": [], "len": 0}]
    gen = torch.Generator(device=dev).manual_seed(3)

    def step(which, counts):
        n = sum(counts)
        slots, pos = [], []
        for i, c in zip(which, counts):
            s = seqs[i]
            while len(s["pages"]) * page < s["len"] + c:
                s["pages"].append(free.pop())
            for p in range(s["len"], s["len"] + c):
                slots.append(s["pages"][p // page] * page + p % page)
                pos.append(p)
            s["len"] += c
        width = max(len(seqs[i]["pages"]) for i in which)
        table = torch.tensor([seqs[i]["pages"] + [-1] * (width - len(seqs[i]["pages"])) for i in which],
                             dtype=torch.int32, device=dev)
        lens = torch.tensor([seqs[i]["len"] for i in which], dtype=torch.int32, device=dev)
        offs = torch.tensor(np.cumsum([0] + list(counts)), dtype=torch.int32, device=dev)
        slots = torch.tensor(slots, device=dev)
        pos = torch.tensor(pos, dtype=torch.int32, device=dev)
        for cache in layers:
            qkv = torch.randn((n, heads + 2 * Hk, D), generator=gen, device=dev).to(torch.bfloat16)
            q, k, v = qkv[:, :heads], qkv[:, heads : heads + Hk], qkv[:, heads + Hk :]
            cache.append(k, v, slots, rope=rope, positions=pos)
            kc = torch.empty((n * Hk, D // 2), dtype=torch.uint8, device=dev)
            ks = torch.empty((n * Hk, D // 32), dtype=torch.float16, device=dev)
            lib.strata_kv4_encode(rope.apply(k, pos), n * Hk, D, kc, ks)
            assert torch.equal(cache.tensors[0][slots // page, :, slots % page], kc.view(n, Hk, -1))
            out = cache.attention(q, offs, lens, table, max_q_len=max(counts), rope=rope, positions=pos)
            q64 = q.double()
            c, s = (torch.from_numpy(t).double().to(dev)[:, None] for t in R.rope_cs(pos.cpu().numpy(), f, m))
            u, w = q64[..., : D // 2], q64[..., D // 2 :]
            q64 = torch.cat([u * c - w * s, w * c + u * s], -1)
            want = torch.zeros_like(q64)
            bound, inside = R.attention(q64, offs, lens, table, cache.tensors, 0, D**-0.5, want)
            assert bool(inside.all())
            assert bool(((out.double() - want).norm(dim=-1) <= bound).all())

    step([0, 1], [50, 33])
    step([0, 1], [50, 7])  # second chunks
    step([0, 1], [4, 4])  # verify 1 + 3
    for s in seqs:
        s["len"] -= 2  # two drafts rejected
    step([0, 1], [1, 1])
    full = seqs[0]["len"] // page  # fork: full pages shared, the open one copied
    last = free.pop()
    seqs.append({"pages": seqs[0]["pages"][:full] + [last], "len": seqs[0]["len"]})
    group.copy_pages([seqs[0]["pages"][full]], [last])
    for _ in range(3):
        step([0, 1, 2], [1, 1, 1])
    used = sorted({p for s in seqs for p in s["pages"]})
    holes = [p for p in range(pages) if p not in used][::-1]
    moves = [(p, holes.pop(0)) for p in used[: len(used) // 2]]  # to the other end of the pool
    group.copy_pages([a for a, _ in moves], [b for _, b in moves])
    new = dict(moves)
    for s in seqs:
        s["pages"] = [new.get(p, p) for p in s["pages"]]
    free[:] = [p for p in range(pages) if p not in {q for s in seqs for q in s["pages"]}]
    step([0, 2, 1], [1, 2, 20])
