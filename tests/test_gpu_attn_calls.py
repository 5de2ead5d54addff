"""Calls of the attention step on the GPU that its documentation allows and
that test_gpu_attn.py does not make; its cases and bounds are used here."""
import pytest
import torch

import attn_ref as R
import attn_stat
from gpu_harness import S, torch_dev
from test_gpu_attn import Case

pytestmark = pytest.mark.gpu


def same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("q_len", [1, 90])
def test_stream_without_buffers(q_len, raw):
    """A call on a stream of the caller's that makes its own result and workspace, while the current stream is busy and
    goes on to allocate and overwrite blocks of the same sizes."""
    dev = torch_dev()
    c = Case([(q_len, 3000), (q_len, 257), (1, 5000)], 16, 2, 128, 64, rope=(128, "half", "none", 1.0), seed=31)
    want = c.run()
    turned = c.rope.apply(c.q, c.positions)
    size = c.cache.attention_workspace(16).numel()
    side = torch.cuda.Stream(dev)
    busy = torch.randn((4096, 4096), device=dev)
    torch.cuda.synchronize()
    for _ in range(10):
        for _ in range(4):
            busy @ busy  # the current stream is behind the calls on the other one
        with torch.cuda.stream(side):
            busy @ busy  # and that one behind the host
        stream = side.cuda_stream if raw else side
        got = c.run(stream=stream)
        rows = c.rope.apply(c.q, c.positions, stream=stream)
        for _ in range(3):  # blocks that were free, or have just been given back
            torch.empty(size, dtype=torch.uint8, device=dev).fill_(0xFF)
            torch.empty_like(want).fill_(float("nan"))
        side.synchronize()
        assert same_bits(got, want)
        assert same_bits(rows, turned)
        torch.cuda.synchronize()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("q_len", [1, 5, 70])
@pytest.mark.parametrize("window", [1, 21, 150])
def test_garbage_in_front_of_the_window(D, q_len, window):
    """Positions in front of the first query's window may hold anything: not-a-number and infinite scales on the page
    and in the tile where the window begins never count."""
    c = Case([(q_len, 333), (q_len, 100 + q_len), (q_len, 512)], 8, 2, D, 16, window=window, seed=D + window)
    live = torch.zeros((c.cache.n_pages, c.page), dtype=torch.bool, device=torch_dev())
    for b, L in enumerate(c.lens.tolist()):
        for j in range(max(L - q_len - window + 1, 0), L):
            live[int(c.table[b, j // c.page]), j % c.page] = True
    assert not bool(live.all())
    for i, poison in ((1, float("nan")), (3, float("inf"))):
        t = c.cache.tensors[i]
        t.copy_(torch.where(live[:, None, :, None], t, torch.full_like(t, poison)))
    c.cache.tensors[3][..., 0].masked_fill_(~live[:, None], float("nan"))
    c.check()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("q_len", [1, 6, 70])
@pytest.mark.parametrize("gain", [2.0**6, 2.0**12, 2.0**20, 2.0**30, 1.7e9, 7.3e7, -(2.0**12), -(2.0**30), -3.3e8])
@pytest.mark.parametrize("place", [3, 150])
def test_logits_of_a_great_size(D, q_len, gain, place):
    """Logits so large that fp32 numbers of their size lie 8 and more apart, with one key far above the others: the
    result is that key's value.

    Every key is a multiple s of one row, and the queries are `gain` times that row, so the logits are gain * s times a
    positive number. The winner's logit is ahead by at least half its size or by its size, thousands at least, so all
    other weights are 0. Its own weight and value are rounded to fp16 (2^-11 each, the weight times the value's scale
    once more), the sums add 2^-18, the result is rounded to bf16 (2^-8)."""
    dev = torch_dev()
    c = Case([(q_len, 333), (q_len, 160 + q_len)], 8, 2, D, 16, seed=D + q_len)
    kc, ks = c.cache.tensors[:2]
    g = torch.Generator(device=dev).manual_seed(D)
    row = torch.randint(1, 16, (D,), generator=g, device=dev)  # codes; the row they stand for is row - 8
    kc.copy_((row[0::2] | row[1::2] << 4).to(torch.uint8).expand_as(kc))
    ks.fill_(2.0**12 if gain > 0 else 0.5)
    for b in range(2):
        page = int(c.table[b, place // c.page])
        ks[page, :, place % c.page] = 2.0**13 if gain > 0 else 0.125
    c.q.copy_((gain * (row.double() - 8) @ R.sylvester(D, dev)).to(torch.bfloat16).expand_as(c.q))
    c.q64 = c.q.double()
    out = c.run().double()
    want = torch.zeros_like(c.q64)
    R.attention(c.q64, c.offsets, c.lens, c.table, c.cache.tensors, 0, c.scale, want)
    assert bool(torch.isfinite(out).all())
    off, size = (out - want).norm(dim=-1), want.norm(dim=-1)
    assert bool((size > 0).all())
    assert float((off / size).max()) <= 2.0**-8 + 3 * 2.0**-11 + 2.0**-18


@pytest.mark.parametrize("layout,rd", [("half", 128), ("interleaved", 64), ("half", 20)])
@pytest.mark.parametrize("n,heads", [(1, 5), (37, 5), (300, 3), (9, 1)])
def test_rotary_of_rows_head_by_head(layout, rd, n, heads):
    """Rows of a head together, as a transposed view has them, on either side and in place."""
    dev = torch_dev()
    rope = S().Rope(128, rd, layout=layout)
    g = torch.Generator(device=dev).manual_seed(n)
    x = torch.randn((n, heads, 128), generator=g, device=dev).to(torch.bfloat16)
    pos = torch.arange(n, dtype=torch.int32, device=dev) * 91
    want = rope.apply(x, pos)
    by_head = x.transpose(0, 1).contiguous().transpose(0, 1)
    assert n == 1 or heads == 1 or by_head.stride()[:2] == (128, n * 128)
    assert same_bits(rope.apply(by_head, pos), want)
    out = torch.zeros((heads, n, 128), dtype=torch.bfloat16, device=dev).transpose(0, 1)
    assert same_bits(rope.apply(x, pos, out), want)
    assert same_bits(rope.apply(by_head, pos, by_head), want)
    if n > 1 and heads > 1:
        with pytest.raises(S().StrataError):  # every token in one place
            rope.apply(x, pos, x[:1].expand(n, -1, -1))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("role", [0, 1, 2, 3])
@pytest.mark.parametrize("piece", [0, 1])
def test_waits_that_run_out_leave_no_row_that_passes_for_a_result(D, role, piece):
    """Four of the tensor-core kernel's 148 blocks stop signalling (5 ms limit): every row is NaN or what the undisturbed
    call gives, though result and workspace hold an earlier call's values; and the next call is right again."""
    lib, dev = S(), torch_dev()
    # two or three pieces for each block
    c = Case([(90, 700), (33, 2000)] * 30 + [(60, 60), (7, 3000), (60, 0)], 16, 2, D, 16, seed=D + 8, pad_back=4)
    ws = c.cache.attention_workspace(16)
    want = torch.full_like(c.q, 7.5, memory_format=torch.contiguous_format)
    c.run(want, workspace=ws)
    n = c.q.shape[0]
    desc = lib.strata_kv4_attn_desc(len(c.lens), 16, c.max_q, c.table.shape[1], n, c.q.stride(0), 16 * D, 0, c.scale)
    for fill in (7.5, None):
        out = want.clone() if fill is None else torch.full_like(want, fill)
        ws.view(torch.float32).fill_(1.0)  # partial results that look like some
        lib.strata_selftest_attention_timeout(c.cache.desc, desc, c.q, c.offsets, c.lens, c.table, out, ws, ws.numel(),
                                              role, 37, piece)
        torch.cuda.synchronize()
        lost = out.isnan().all(-1)
        same = (out.view(torch.int16) == want.view(torch.int16)).all(-1)
        assert bool((lost | same).all()), f"{int((~(lost | same)).sum())} rows are neither lost nor right"
        assert bool((out[-4:] == 7.5).all())
        assert bool(same[:-4].any()) and bool(lost.any())
    out = torch.full_like(want, 7.5)
    c.run(out, workspace=ws)
    assert same_bits(out, want)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("seqs,heads,kv_heads,window", [
    ([(1, 200_003)], 8, 1, 0), ([(1, 20_000), (1, 77_777), (1, 1025)], 16, 2, 0), ([(2, 131_072)], 8, 1, 0),
    ([(6, 60_000), (6, 33_333), (6, 1025)], 8, 1, 0), ([(70, 60_001)], 4, 1, 0),
    ([(300, 20_000), (1, 30_000), (5, 700)], 8, 2, 0), ([(1, 40_000), (200, 30_000)], 8, 2, 9_000)])
def test_rows_over_long_contexts(D, seqs, heads, kv_heads, window):
    """Every row within what rounding does in the mean (attn_stat): a lost tile, part or page of any length would show."""
    c = Case(seqs, heads, kv_heads, D, 64, window=window, rope=(D, "half", "none", 1.0), seed=D + len(seqs))
    want, limit, inside = attn_stat.attention(c.q64, c.offsets, c.lens, c.table, c.cache.tensors, c.window, c.scale)
    off = (c.run().double() - want).norm(dim=-1)
    assert bool(inside.all())
    assert bool((off <= limit).all()), f"worst {float((off / limit).max()):.3g} of the limit"


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("q_len", [1, 6, 120])
def test_result_in_the_queries_place(D, q_len):
    """out may be q: every query row is read before its result is written, by whichever block."""
    c = Case([(q_len, 900), (q_len, 9000), (2, 40)], 16, 2, D, 32, rope=(D, "half", "none", 1.0), seed=q_len + D)
    want = c.run()
    wide = torch.full((c.q.shape[0], 19, D), 7.5, dtype=torch.bfloat16, device=torch_dev())
    for _ in range(5):
        x = wide[:, 1:17]
        x.copy_(c.q)
        c.cache.attention(x, c.offsets, c.lens, c.table, x, max_q_len=c.max_q, scale=c.scale, rope=c.rope,
                          positions=c.positions)
        assert same_bits(x, want)
        assert bool((wide[:, 0] == 7.5).all()) and bool((wide[:, 17:] == 7.5).all())


@pytest.mark.parametrize("q_len", [1, 70])
def test_captured_step(q_len):
    """A layer's whole step in one graph (a fork's page copy, rotary rows, append, attention, with buffers of the
    graph's own), replayed on new inputs: the same bits as the calls one by one."""
    lib, dev = S(), torch_dev()
    D, heads, hk, page, pages = 128, 16, 2, 16, 80
    rope = lib.Rope(D, D, layout="half")
    g = torch.Generator(device=dev).manual_seed(q_len)
    start = [torch.randint(0, 256, t.shape, generator=g, device=dev, dtype=torch.uint8) if t.dtype == torch.uint8 else
             torch.rand(t.shape, generator=g, device=dev).half() for t in lib.Kv4Cache.empty(pages, page, hk, D).tensors]
    lens = torch.tensor([200, 333], dtype=torch.int32, device=dev) + q_len
    table = torch.arange(2 * 36, dtype=torch.int32, device=dev).view(2, 36)
    offs = torch.tensor([0, q_len, 2 * q_len], dtype=torch.int32, device=dev)

    def inputs(seed):
        r = torch.Generator(device=dev).manual_seed(seed)
        qkv = torch.randn((2 * q_len, heads + 2 * hk, D), generator=r, device=dev).to(torch.bfloat16)
        pos = torch.cat([torch.arange(int(n) - q_len, int(n), device=dev) for n in lens])
        slots = torch.cat([table[b].long()[pos[b * q_len : (b + 1) * q_len] // page] * page +
                           pos[b * q_len : (b + 1) * q_len] % page for b in range(2)])
        return qkv, pos.to(torch.int32) + seed, slots

    def step(cache, qkv, pos, slots):
        q, k, v = qkv[:, :heads], qkv[:, heads : heads + hk], qkv[:, heads + hk :]
        lib.Kv4CacheSet([cache]).copy_pages([3, 5], [75, 76])
        cache.append(k, v, slots, rope=rope, positions=pos)
        return rope.apply(k, pos), cache.attention(q, offs, lens, table, max_q_len=q_len, rope=rope, positions=pos)

    def fresh():
        return lib.Kv4Cache(*(t.clone() for t in start))

    static = [t.clone() for t in inputs(1)]
    cache = fresh()
    graph = torch.cuda.CUDAGraph()
    step(fresh(), *static)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = step(cache, *static)
    for seed in (2, 3, 2):
        other = fresh()
        for a, b in zip(cache.tensors, start):
            a.copy_(b)
        for a, b in zip(static, inputs(seed)):
            a.copy_(b)
        graph.replay()
        want = step(other, *inputs(seed))
        torch.cuda.synchronize()
        assert same_bits(got[0], want[0]) and same_bits(got[1], want[1])
        for a, b in zip(cache.tensors, other.tensors):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("q_len", [1, 70])
def test_a_page_in_many_tables_and_twice_in_one(q_len):
    """Sequences that share their prefix's pages, the same page several times in a table, and two views of a cache."""
    c = Case([(q_len, 500), (q_len, 500), (q_len, 130)], 8, 2, 128, 16, seed=5)
    c.table[1, :20] = c.table[0, :20]
    c.table[2] = c.table[0, 1]
    c.check()
    c.cache = S().Kv4Cache(*(t.view(t.shape) for t in c.cache.tensors))
    c.check()


@pytest.mark.parametrize("q_len", [1, 70])
def test_table_without_pages_and_batch_without_sequences(q_len):
    """A block table of no columns leaves every query without keys; no sequences leave every row as it was."""
    dev = torch_dev()
    c = Case([(q_len, 40), (q_len, 20)], 8, 2, 128, 16)
    c.table = c.table[:, :0].contiguous()
    out = torch.full_like(c.q, 7.5, memory_format=torch.contiguous_format)
    assert bool((c.run(out) == 0).all())
    c.offsets, c.lens, c.table = c.offsets[:1], c.lens[:0], c.table[:0]
    out.fill_(7.5)
    assert bool((c.run(out) == 7.5).all())


@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("q_len", [1, 3])
def test_many_query_heads_of_one_kv_head(D, q_len):
    """300 query heads: a token's rows fill more than one item."""
    Case([(q_len, 700), (q_len, 33)], 300, 1, D, 16, rope=(D, "half", "none", 1.0), seed=D).check()
