"""What is measured of the attention-side operators of the 4-bit rotated KV cache.

Operators: rotary positions on head rows, appending rows to the paged 4-bit
cache (rotary of the keys and the codec's encoder in one call), attention over
that cache, and copying of its pages. Every case says what it stands for; the
plain forms below use elementary torch operations in 32 bits (64 for angles
and for the exact product that a code is rounded from).

Cache: pages of `page` token slots; codes [pages, kv_heads, page, D/2] uint8
(value 2j in the low nibble of byte j) and fp16 scales [pages, kv_heads, page,
D/32], for keys and for values. A row x of D values is held as
y = H x / sqrt(D) (H the Sylvester matrix) in blocks of 32: s = fp16(absmax / 7),
code = clamp(rint(y / s), -7, 7) + 8. The format fixes every bit of codes and
scales (the rounding of each step, ties to even), so an appended or copied pool
is returned as the bytes that it holds, and they have to be equal.
"""
import math
import random

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of a 64-sequence batch: a few hundred rows, all launch latency
        dict(name="rope_decode_64", op="rope", tokens=64, heads=36, head_dim=128, rotary=128, layout="half",
             scaling="none", factor=1.0, far=131072, fused=False),
        # q and k of an 8,192-token prompt chunk inside the fused projection's output, context stretched
        dict(name="rope_prompt_8192", op="rope", tokens=8192, heads=36, head_dim=128, rotary=128, layout="half",
             scaling="yarn", factor=4.0, far=131072, fused=True),
        # a verify step: 16 sequences of 1 + 3 drafted tokens join the cache
        dict(name="append_verify_64", op="append", tokens=64, kv_heads=4, head_dim=128, page=64, rotary=128,
             layout="half", scaling="none", factor=1.0, far=131072, padded=0),
        # a whole prompt chunk joins the cache, some rows padding
        dict(name="append_prompt_8192", op="append", tokens=8192, kv_heads=4, head_dim=128, page=64, rotary=128,
             layout="half", scaling="yarn", factor=4.0, far=131072, padded=57),
        # one chat at a short context, one token
        dict(name="decode_short", op="attention", seqs=1, q_len=1, context=777, ragged=False, heads=32, kv_heads=4,
             head_dim=128, page=16, window=0, rotary=128, layout="half"),
        # one chat at the longest context, one token: a whole layer's cache is read
        dict(name="decode_128k", op="attention", seqs=1, q_len=1, context=131072, ragged=False, heads=32, kv_heads=4,
             head_dim=128, page=64, window=0, rotary=128, layout="half"),
        # a serving batch, one token each, contexts of all lengths
        dict(name="decode_batch_64", op="attention", seqs=64, q_len=1, context=16384, ragged=True, heads=32, kv_heads=4,
             head_dim=128, page=64, window=0, rotary=128, layout="half"),
        # 1 + 5 drafted tokens of 8 sequences verified in one pass
        dict(name="verify6_batch_8", op="attention", seqs=8, q_len=6, context=32768, ragged=True, heads=32, kv_heads=4,
             head_dim=128, page=32, window=0, rotary=128, layout="half"),
        # the last 8,192-token chunk of a 32,768-token prompt
        dict(name="prompt_8192_of_32k", op="attention", seqs=1, q_len=8192, context=32768, ragged=False, heads=32,
             kv_heads=4, head_dim=128, page=64, window=0, rotary=128, layout="half"),
        # short prompts and decode steps mixed in one batch, narrow heads, a sliding window, odd sizes
        dict(name="mixed_window_d64", op="attention", seqs=11, q_len=517, context=5003, ragged=True, heads=14,
             kv_heads=2, head_dim=64, page=16, window=1021, rotary=32, layout="interleaved"),
        # 8 sampled continuations fork: the last page of each, in every one of 48 layers
        dict(name="fork_8_pages", op="copy", layers=48, pages=64, pairs=8, kv_heads=4, head_dim=128, page=64),
        # a fragmented pool is compacted: many pages, in every layer
        dict(name="compact_400_pages", op="copy", layers=48, pages=1024, pairs=400, kv_heads=4, head_dim=128, page=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "attention", "attention", "attention", "copy"])
    head_dim = rng.choice([64, 128, 128, 256])
    page = rng.choice([16, 32, 64, 128])
    layout = rng.choice(["half", "interleaved"])
    rotary = rng.choice([head_dim, head_dim, head_dim // 2, head_dim // 4])
    scaling = rng.choice(["none", "linear", "ntk", "yarn"])
    factor = 1.0 if scaling == "none" else rng.choice([2.0, 4.0, 7.5])
    if op == "rope":
        heads = rng.randint(1, 40)
        tokens = min(_log(rng, 1, 8192), 8192 * 36 * 128 // (heads * head_dim))
        return dict(op=op, tokens=tokens, heads=heads, head_dim=head_dim, rotary=rotary, layout=layout, scaling=scaling,
                    factor=factor, far=_log(rng, 4096, 1 << 20), fused=rng.random() < 0.5)
    if op == "append":
        kv_heads = rng.choice([1, 2, 3, 4, 8])
        tokens = min(_log(rng, 1, 8192), 8192 * 4 * 128 // (kv_heads * head_dim))
        return dict(op=op, tokens=tokens, kv_heads=kv_heads, head_dim=head_dim, page=page,
                    rotary=rng.choice([0, rotary]), layout=layout, scaling=scaling, factor=factor,
                    far=_log(rng, 4096, 1 << 20), padded=rng.randint(0, tokens // 4))
    if op == "copy":
        layers = _log(rng, 1, 48)
        kv_heads = rng.choice([1, 2, 4, 8])
        pairs = max(1, min(_log(rng, 1, 400), 48 * 400 * 4 * 128 * 64 // (layers * kv_heads * head_dim * page)))
        return dict(op=op, layers=layers, pages=2 * pairs + rng.randint(1, 9), pairs=pairs, kv_heads=kv_heads,
                    head_dim=head_dim, page=page)
    kv_heads = rng.choice([1, 2, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 4, 5, 7, 8])
    kind = rng.choice(["decode", "decode", "verify", "prompt"])
    if kind == "prompt":
        seqs, q_len = _log(rng, 1, 8), _log(rng, 17, 8192)
        q_len = max(17, q_len // seqs)
        context = _log(rng, q_len, 32768)
        while seqs * q_len * context * heads * head_dim > 8192 * 32768 * 32 * 128 // 8:
            context = max(q_len, context // 2)
            q_len = min(q_len, max(17, context // 2))
    else:
        seqs, q_len = _log(rng, 1, 64), 1 if kind == "decode" else rng.randint(2, 16)
        context = min(_log(rng, 16, 131072), 131072 * 4 * 128 // (kv_heads * head_dim * max(1, seqs // 4)))
        context = max(context, 16)
    return dict(op="attention", seqs=seqs, q_len=q_len, context=context, ragged=rng.random() < 0.7, heads=heads,
                kv_heads=kv_heads, head_dim=head_dim, page=page, window=rng.choice([0, 0, _log(rng, 16, context)]),
                rotary=rng.choice([0, rotary]), layout=layout)


def lengths(case):
    """Query and cache lengths of the sequences, by the case alone: a ragged batch has contexts of all sizes and,
    from four sequences on, one that is idle in this step."""
    n, q, ctx = case["seqs"], case["q_len"], case["context"]
    q = min(q, ctx)
    if not case["ragged"]:
        return [q] * n, [ctx] * n
    r = random.Random("%d %d %d" % (n, q, ctx))
    kv = [_log(r, max(q, ctx // 16, 1), ctx) for _ in range(n)]
    kv[r.randrange(n)] = ctx
    ql = [q if q <= 16 else _log(r, 1, q) for _ in range(n)]
    ql[r.randrange(n)] = q
    if n >= 4:
        ql[r.randrange(n)] = 0
    return ql, kv


def frequencies(case):
    """Angle per position of each rotated pair, and the factor of cos and sin."""
    d, base, f, kind = case["rotary"], 1000000.0, case.get("factor", 1.0), case.get("scaling", "none")
    if kind == "ntk":
        base *= f ** (d / (d - 2.0))
    inv = [base ** (-2.0 * i / d) for i in range(d // 2)]
    if kind == "linear":
        inv = [v / f for v in inv]
    if kind == "yarn":
        def pair_of(turns):
            return d * math.log(32768 / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(math.floor(pair_of(32.0)), 0), min(math.ceil(pair_of(1.0)), d - 1)
        ramp = [min(max((i - lo) / ((hi - lo) or 0.001), 0.0), 1.0) for i in range(d // 2)]
        inv = [v / f * r + v * (1 - r) for v, r in zip(inv, ramp)]
        return inv, 0.1 * math.log(f) + 1.0
    return inv, 1.0


# ------------------------------------------------------------------ inputs
def _rows(g, n, heads, D):
    """Head rows as they come: normal, with four channels 16 times as large."""
    x = torch.randn((n, heads, D), generator=g, device=DEV, dtype=torch.float32)
    ch = torch.randint(0, D, (4,), generator=g, device=DEV)
    gain = torch.ones(D, device=DEV)
    gain[ch] = 16.0
    return (x * gain).to(torch.bfloat16)


def _pool(g, shape_pages, kv_heads, page, D):
    """Keys' and values' codes and scales of a pool of pages, as the codec leaves them for rows like _rows()."""
    out = {}
    for n in ("k", "v"):
        z = torch.randn((shape_pages, kv_heads, page, D // 2, 2), generator=g, device=DEV, dtype=torch.float16)
        c = (z * 2.6).round_().clamp_(-7, 7).add_(8).to(torch.uint8)
        out[n + "_codes"] = c[..., 0] | (c[..., 1] << 4)
        s = torch.rand((shape_pages, kv_heads, page, D // 32), generator=g, device=DEV)
        out[n + "_scales"] = (0.35 + 0.4 * s).to(torch.float16)
    return out


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    host = random.Random(seed)
    st = {"case": dict(case)}
    op = case["op"]
    if op in ("rope", "append"):
        n, D = case["tokens"], case["head_dim"]
        st["positions"] = torch.randint(0, case["far"], (n,), generator=g, device=DEV, dtype=torch.int32)
    if op == "rope":
        extra = 4 if case["fused"] else 0  # the value heads of the fused projection, left alone
        st["x"] = _rows(g, n, case["heads"] + extra, D)[:, : case["heads"]]
        st["out"] = torch.zeros((n, case["heads"], D), dtype=torch.bfloat16, device=DEV)
    elif op == "append":
        heads, page = case["kv_heads"], case["page"]
        n_pages = n // page + 9
        kv = _rows(g, n, 2 * heads, D)
        st["k"], st["v"] = kv[:, :heads], kv[:, heads:]
        st.update(_pool(g, n_pages, heads, page, D))
        slots = torch.randperm(n_pages, generator=g, device=DEV)[:, None] * page + torch.arange(page, device=DEV)
        slots = slots.reshape(-1)[3 : 3 + n].clone()
        slots[n - case["padded"] :] = -1  # padding rows of the batch go nowhere
        st["slots"] = slots
    elif op == "copy":
        layers, pages = case["layers"], case["pages"]
        one = _pool(g, pages, case["kv_heads"], case["page"], case["head_dim"])
        for k, t in one.items():  # layers differ by a rotation of their pages
            st[k] = torch.stack([t.roll(l * 7 + 1, 0) for l in range(layers)])
        order = host.sample(range(pages), 2 * case["pairs"])
        # the page allocator works on the host: its lists are host arrays
        order = torch.tensor(order, dtype=torch.int32)
        st["src"], st["dst"] = order[: case["pairs"]].clone(), order[case["pairs"] :].clone()
    else:
        D, page, Hq, Hk = case["head_dim"], case["page"], case["heads"], case["kv_heads"]
        ql, kl = lengths(case)
        need = [-(-k // page) for k in kl]
        st.update(_pool(g, sum(need) + 3, Hk, page, D))
        perm = torch.randperm(sum(need) + 3, generator=g, device=DEV).tolist()
        table = torch.full((len(kl), max(need)), -1, dtype=torch.int32)
        for b, n in enumerate(need):
            table[b, :n] = torch.tensor([perm.pop() for _ in range(n)], dtype=torch.int32)
        st["block_table"] = table.to(DEV)
        n = sum(ql)
        st["q"] = torch.randn((n, Hq + 2 * Hk, D), generator=g, device=DEV).to(torch.bfloat16)[:, :Hq]
        st["q_offsets"] = torch.tensor([0] + ql).cumsum(0).to(torch.int32).to(DEV)
        st["kv_lens"] = torch.tensor(kl, dtype=torch.int32).to(DEV)
        st["positions"] = torch.cat([torch.arange(k - q, k, dtype=torch.int32) for q, k in zip(ql, kl)]).to(DEV)
        st["out"] = torch.zeros((n, Hq, D), dtype=torch.bfloat16, device=DEV)
        st["max_q_len"], st["scale"] = max(ql), D ** -0.5
    if own:
        _handles(st)
    return st


def _handles(st):
    """The handles that a program keeps: the rotary table, the cache's description, the attention's workspace."""
    import bit_quantized_moe_warp_b200 as S

    case = st["case"]
    if case.get("rotary"):
        st["rope"] = S.Rope(case["head_dim"], case["rotary"], theta=1000000.0, layout=case["layout"],
                            scaling=case.get("scaling", "none"), factor=case.get("factor", 1.0),
                            original_max_position=32768)
    if case["op"] == "copy":
        st["caches"] = S.Kv4CacheSet([S.Kv4Cache(*(st[k][l] for k in ("k_codes", "k_scales", "v_codes", "v_scales")))
                                      for l in range(case["layers"])])
    elif case["op"] != "rope":
        st["cache"] = S.Kv4Cache(st["k_codes"], st["k_scales"], st["v_codes"], st["v_scales"])
        if case["op"] == "attention":
            st["workspace"] = st["cache"].attention_workspace(case["heads"])


# ------------------------------------------------------------------ plain forms
def _rotate(x, case, positions):
    """Rotary positions of fp32 rows [tokens, heads, D], every product and sum rounded to 32 bits."""
    d = case["rotary"]
    inv, m = frequencies(case)
    turn = torch.tensor(inv, dtype=torch.float64, device=x.device) / (2 * math.pi)
    head = (turn * 2.0**26).round() / 2.0**26  # so that position * head is exact
    p = positions.to(torch.float64)[:, None]
    a = (torch.remainder(p * head, 1.0) + p * (turn - head)) * (2 * math.pi)
    c, s = (a.cos() * m).float()[:, None], (a.sin() * m).float()[:, None]
    r = x[..., :d]
    u, v = (r[..., : d // 2], r[..., d // 2 :]) if case["layout"] == "half" else (r[..., 0::2], r[..., 1::2])
    pu, pv = u * c - v * s, v * c + u * s
    rot = torch.cat([pu, pv], -1) if case["layout"] == "half" else torch.stack([pu, pv], -1).flatten(-2)
    return torch.cat([rot, x[..., d:]], -1)


def _encode(x):
    """Codes and scales of fp32 rows [..., D]: butterflies in stride order, the block rule, each step rounded to 32 bits."""
    D = x.shape[-1]
    for k in range(D.bit_length() - 1):
        w = x.unflatten(-1, (D >> (k + 1), 2, 1 << k))
        x = torch.stack([w[..., 0, :] + w[..., 1, :], w[..., 0, :] - w[..., 1, :]], -2).flatten(-3)
    y = (x * torch.tensor(1 / math.sqrt(D), dtype=torch.float32, device=x.device)).unflatten(-1, (D // 32, 32))
    a = y.abs().amax(-1)
    s = torch.minimum(a / torch.full_like(a, 7.0), torch.full_like(a, 65504.0)).half()
    f = s.float()
    inv = torch.where(f > 0, torch.ones_like(f) / f, torch.zeros_like(f))
    q = (y.double() * inv.double()[..., None]).round().clamp(-7, 7).to(torch.int32).flatten(-2) + 8
    return (q[..., 0::2] | (q[..., 1::2] << 4)).to(torch.uint8), s


def _hadamard(D, dtype):
    i = torch.arange(D, device=DEV)
    bits = i[:, None] & i[None, :]
    bits = bits ^ (bits >> 4)
    bits = bits ^ (bits >> 2)
    bits = bits ^ (bits >> 1)
    return 1 - 2 * (bits & 1).to(dtype)


def _attend(st):
    case = st["case"]
    D, page, Hq, Hk = case["head_dim"], case["page"], case["heads"], case["kv_heads"]
    G, w = Hq // Hk, case["window"]
    q = st["q"].float()
    if case["rotary"]:
        q = _rotate(q, case, st["positions"])
    lens, off = st["kv_lens"].long(), st["q_offsets"].long()
    n_q = off[1:] - off[:-1]
    B, Q = lens.numel(), st["max_q_len"]
    i = torch.arange(Q, device=q.device)
    at = (off[:-1, None] + i).clamp_max(q.shape[0] - 1)
    table = st["block_table"].long()
    L = table.shape[1] * page
    key = torch.arange(L, device=q.device)
    pos = (lens - n_q)[:, None] + i
    seen = (key <= pos[..., None]) & (key < lens[:, None, None]) & (i < n_q[:, None])[..., None]
    if w:
        seen &= key > pos[..., None] - w
    H = _hadamard(D, torch.float32) / math.sqrt(D)
    out = torch.zeros((q.shape[0], Hq, D), dtype=torch.float32, device=q.device)

    def rows(name, h):
        c = st[name + "_codes"][:, h][table.clamp_min(0)].flatten(1, 2)
        s = st[name + "_scales"][:, h][table.clamp_min(0)].flatten(1, 2).float()
        y = torch.stack([c & 15, c >> 4], -1).flatten(-2).float() - 8
        return (y.unflatten(-1, (D // 32, 32)) * s[..., None]).flatten(-2) @ H

    live = i < n_q[:, None]
    for h in range(Hk):
        qh = q[at][:, :, h * G : (h + 1) * G].transpose(1, 2)  # [B, G, Q, D]
        sc = (qh.flatten(1, 2) @ rows("k", h).transpose(1, 2)).unflatten(1, (G, Q)).mul_(st["scale"])
        sc.masked_fill_(~seen[:, None], -math.inf)
        m = sc.amax(-1, keepdim=True)
        sc.sub_(m.masked_fill(m == -math.inf, 0.0)).exp_()
        l = sc.sum(-1, keepdim=True)
        o = (sc.flatten(1, 2) @ rows("v", h)).unflatten(1, (G, Q)) / l.masked_fill(l == 0, 1.0)
        out[:, h * G : (h + 1) * G][at[live]] = o.transpose(1, 2)[live]
    return out.to(torch.bfloat16)


def _append(st):
    case = st["case"]
    page = case["page"]
    k = st["k"].float()
    if case["rotary"]:
        k = _rotate(k, case, st["positions"]).to(torch.bfloat16).float()
    keep = st["slots"] >= 0
    where = st["slots"][keep]
    at, slot = where // page, where % page
    for name, x in (("k", k), ("v", st["v"].float())):
        c, s = _encode(x[keep])
        st[name + "_codes"][at, :, slot] = c
        st[name + "_scales"][at, :, slot] = s
    return {n: st[n] for n in ("k_codes", "k_scales", "v_codes", "v_scales")}


def _copy(st):
    src, dst = st["src"].to(DEV).long(), st["dst"].to(DEV).long()
    for n in ("k_codes", "k_scales", "v_codes", "v_scales"):
        st[n][:, dst] = st[n][:, src]
    return {n: st[n] for n in ("k_codes", "k_scales", "v_codes", "v_scales")}


# ------------------------------------------------------------------ one pass
def run(st):
    op = st["case"]["op"]
    if own:
        if op == "rope":
            return st["rope"].apply(st["x"], st["positions"], st["out"])
        if op == "append":
            st["cache"].append(st["k"], st["v"], st["slots"], rope=st.get("rope"), positions=st["positions"])
            return {n: st[n] for n in ("k_codes", "k_scales", "v_codes", "v_scales")}
        if op == "copy":
            st["caches"].copy_pages(st["src"], st["dst"])
            return {n: st[n] for n in ("k_codes", "k_scales", "v_codes", "v_scales")}
        return st["cache"].attention(st["q"], st["q_offsets"], st["kv_lens"], st["block_table"], st["out"],
                                     max_q_len=st["max_q_len"], scale=st["scale"], window=st["case"]["window"],
                                     rope=st.get("rope"), positions=st["positions"], workspace=st["workspace"])
    if op == "rope":
        return _rotate(st["x"].float(), st["case"], st["positions"]).to(torch.bfloat16)
    return {"append": _append, "copy": _copy, "attention": _attend}[op](st)


def work(case):
    op, D = case["op"], case["head_dim"]
    if op == "rope":
        v = case["tokens"] * case["heads"] * D
        return {"bytes": 4 * v + 4 * case["tokens"], "flops": 3 * case["tokens"] * case["heads"] * case["rotary"]}
    if op == "append":
        n = case["tokens"] - case["padded"]
        v = 2 * n * case["kv_heads"] * D
        return {"bytes": 2 * v + v * 9 // 16 + 8 * case["tokens"] + 4 * n, "flops": v * (D.bit_length() + 3)}
    if op == "copy":
        one = case["kv_heads"] * case["page"] * 2 * (D // 2 + D // 16)
        return {"bytes": 2 * one * case["pairs"] * case["layers"], "flops": 0}
    ql, kl = lengths(case)
    keys = pairs = 0
    for q, k in zip(ql, kl):
        w = case["window"] or k
        pairs += sum(min(k - q + i + 1, w) for i in range(q))
        keys += min(k, w + q - 1) if q else 0
    n = sum(ql)
    return {"bytes": keys * case["kv_heads"] * 2 * (D // 2 + D // 16) + 4 * n * case["heads"] * D
            + 4 * sum(-(-k // case["page"]) for k in kl) + 4 * n,
            "flops": 4 * D * case["heads"] * pairs}


# ------------------------------------------------------------------ 64 bits
def _sylvester(D):
    h = torch.ones((1, 1), dtype=torch.float64, device=DEV)
    while h.shape[0] < D:
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
    return h / math.sqrt(D)


def _turned(x, case, positions):
    """Rotary positions in 64 bits, pairs as complex numbers."""
    d = case["rotary"]
    if not d:
        return x
    inv, m = frequencies(case)
    angle = positions.double()[:, None] * torch.tensor(inv, dtype=torch.float64, device=x.device)
    z = torch.polar(torch.full_like(angle, m), angle)[:, None]
    r = x.clone()
    if case["layout"] == "half":
        y = torch.complex(x[..., : d // 2].contiguous(), x[..., d // 2 : d].contiguous()) * z
        r[..., : d // 2], r[..., d // 2 : d] = y.real, y.imag
    else:
        y = torch.complex(x[..., 0:d:2].contiguous(), x[..., 1:d:2].contiguous()) * z
        r[..., 0:d:2], r[..., 1:d:2] = y.real, y.imag
    return r


def exact(case, seed):
    st = prepare(case, seed)
    op, D = case["op"], case["head_dim"]
    if op == "rope":
        return _turned(st["x"].double(), case, st["positions"])
    none = {n: None for n in ("k_codes", "v_codes")}
    if op == "copy":
        for n in ("k_scales", "v_scales"):
            old = st[n].double()
            for a, b in zip(st["src"].tolist(), st["dst"].tolist()):
                st[n][:, b] = old[:, a].half()
        return {**none, "k_scales": st["k_scales"].double(), "v_scales": st["v_scales"].double()}
    H = _sylvester(D)
    if op == "append":
        got = {}
        for n in ("k", "v"):
            x = st[n].double()
            if n == "k":
                x = _turned(x, case, st["positions"]).to(torch.bfloat16).double()
            s = (x @ H).unflatten(-1, (D // 32, 32)).abs().amax(-1) / 7
            pool = st[n + "_scales"].double().transpose(1, 2).flatten(0, 1)  # [slots, heads, blocks]
            live = st["slots"] >= 0
            pool[st["slots"][live]] = s[live]
            got[n + "_scales"] = pool.unflatten(0, (-1, case["page"])).transpose(1, 2).contiguous()
        return {**none, **got}
    q = _turned(st["q"].double(), case, st["positions"])
    ql, kl = lengths(case)
    G, page, w = case["heads"] // case["kv_heads"], case["page"], case["window"]
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device=DEV)
    first = 0
    for b, (nq, nk) in enumerate(zip(ql, kl)):
        pages = st["block_table"][b, : -(-nk // page)].long()
        for h in range(case["kv_heads"] if nq else 0):
            kv = []
            for n in ("k", "v"):
                c = st[n + "_codes"][pages, h].flatten(0, 1)[:nk]
                y = torch.empty((nk, D), dtype=torch.float64, device=DEV)
                y[:, 0::2], y[:, 1::2] = (c & 15).double() - 8, (c >> 4).double() - 8
                s = st[n + "_scales"][pages, h].flatten(0, 1)[:nk].double()
                kv.append((y * s.repeat_interleave(32, 1)) @ H)
            for g in range(h * G, (h + 1) * G):
                for lo in range(0, nq, 2048):
                    hi = min(nq, lo + 2048)
                    x = q[first + lo : first + hi, g] @ kv[0].T * st["scale"]
                    p = torch.arange(nk - nq + lo, nk - nq + hi, device=DEV)[:, None]
                    j = torch.arange(nk, device=DEV)[None]
                    x[(j > p) | ((j <= p - w) if w else False)] = -math.inf
                    out[first + lo : first + hi, g] = torch.softmax(x, -1) @ kv[1]
        first += nq
    return out
