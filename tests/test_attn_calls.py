"""What the Python classes of the attention step (Rope, Kv4Cache) hand to the
library, with the device and the library replaced by recorders: no GPU."""
import ctypes

import pytest
import torch


class Stream:
    """Stands for a torch.cuda.Stream."""

    def __init__(self, handle):
        self.cuda_stream = handle


class Tensor:
    """Stands for a contiguous CUDA tensor; `stream` is the stream it was made on."""

    def __init__(self, shape, dtype, stream=None):
        self.shape, self.dtype, self.stream = tuple(shape), dtype, stream
        self.device = torch.device("cuda", 0)

    def get_device(self):
        return 0

    def dim(self):
        return len(self.shape)

    def stride(self):
        s = [1]
        for n in self.shape[:0:-1]:
            s.append(s[-1] * n)
        return tuple(s[::-1])

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x10000 + (id(self) << 8)

    def numel(self):
        n = 1
        for k in self.shape:
            n *= k
        return n

    def element_size(self):
        return torch.empty((), dtype=self.dtype).element_size()


CURRENT = 0x11  # the stream that torch has as the current one


@pytest.fixture
def rig(monkeypatch):
    """The package with a recording library and a recording allocator: .made, .calls (name, arguments)."""
    import __graft_entry__

    __graft_entry__._load_builder().build()
    import bit_quantized_moe_warp_b200 as S

    class Rig:
        pass

    rig = Rig()
    rig.S, rig.made, rig.calls, rig.current = S, [], [], [CURRENT]
    real = S._lib
    host_empty, host_zeros = torch.empty, torch.zeros

    class Library:
        def __getattr__(self, name):
            fn = getattr(real, name)
            if name not in ("strata_rope_apply", "strata_kv4_append", "strata_kv4_attention"):
                return fn

            def call(*args):
                rig.calls.append((name, args))
                return S.STRATA_OK

            return call

    class Using:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            rig.current.append(self.stream.cuda_stream)

        def __exit__(self, *exc):
            rig.current.pop()

    def maker(host):
        def make(*shape, dtype=None, device=None):
            if device is None:
                return host(*shape, dtype=dtype)
            shape = shape[0] if not isinstance(shape[0], int) else shape
            t = Tensor(shape, dtype, rig.current[-1])
            rig.made.append(t)
            return t

        return make

    monkeypatch.setattr(S, "_lib", Library())
    monkeypatch.setattr(torch, "empty", maker(host_empty))
    monkeypatch.setattr(torch, "zeros", maker(host_zeros))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "stream", Using)
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: Stream(handle))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: Stream(0))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: rig.current[-1], raising=False)

    def cache(pages=4, heads=2, page=16, D=128):
        return S.Kv4Cache(*(Tensor((pages, heads, page, w), t)
                            for w, t in 2 * ((D // 2, torch.uint8), (D // 32, torch.float16))))

    rig.cache = cache
    rig.i32 = lambda *shape: Tensor(shape, torch.int32)
    rig.bf16 = lambda *shape: Tensor(shape, torch.bfloat16)
    return rig


STREAMS = [(None, CURRENT), (0, 0), (0x77, 0x77), (Stream(0x99), 0x99)]


@pytest.mark.parametrize("stream,handle", STREAMS)
def test_buffers_are_made_on_the_stream_of_the_call(rig, stream, handle):
    """What a call allocates itself belongs to the stream that its kernels run on: a fill on another stream could come
    after them, and memory given back to another stream's pool could be somebody else's before they are done."""
    n, B = 3, 2
    out = rig.cache().attention(rig.bf16(n, 8, 128), rig.i32(B + 1), rig.i32(B), rig.i32(B, 2), max_q_len=2,
                                stream=stream)
    (name, args), = rig.calls
    assert name == "strata_kv4_attention" and args[-1] == handle
    assert len(rig.made) == 2 and out in rig.made  # the result and the workspace
    assert {t.data_ptr() for t in rig.made} == {args[8], args[9]}
    assert [t.stream for t in rig.made] == [handle, handle]

    rig.made.clear()
    rig.calls.clear()
    rope = rig.S.Rope(128)
    out = rope.apply(rig.bf16(n, 8, 128), rig.i32(n), stream=stream)
    (name, args), = rig.calls
    assert name == "strata_rope_apply" and args[-1] == handle and args[7] == out.data_ptr()
    assert rig.made == [out] and out.stream == handle
    assert rig.current == [CURRENT]


def test_closed_rope_is_refused(rig):
    """The library reads a missing rotary handle as no rotation: a closed one must not pass for that."""
    rope, cache = rig.S.Rope(128), rig.cache()
    rope.close()
    with pytest.raises(ValueError, match="closed"):
        cache.append(rig.bf16(3, 2, 128), rig.bf16(3, 2, 128), Tensor((3,), torch.int64), rope=rope, positions=rig.i32(3))
    with pytest.raises(ValueError, match="closed"):
        cache.attention(rig.bf16(3, 8, 128), rig.i32(3), rig.i32(2), rig.i32(2, 2), max_q_len=2, rope=rope,
                        positions=rig.i32(3))
    with pytest.raises(ValueError, match="closed"):
        rope.apply(rig.bf16(3, 8, 128), rig.i32(3))
    assert not rig.calls


@pytest.mark.parametrize("wide", [1 << 32, (1 << 32) + 5, (1 << 31), -(1 << 32) + 3])
def test_numbers_wider_than_the_fields_are_refused(rig, wide):
    """The library's structures hold 32-bit numbers; ctypes keeps the low bits of a wider one, and a window of 2^32
    would be no window."""
    cache = rig.cache()
    ok = dict(max_q_len=2, window=0)
    for kw in (dict(window=wide), dict(max_q_len=wide)):
        with pytest.raises(ValueError):
            cache.attention(rig.bf16(3, 8, 128), rig.i32(3), rig.i32(2), rig.i32(2, 2), **{**ok, **kw})
    with pytest.raises(ValueError):
        cache.attention_workspace(wide + 8)
    for kw in (dict(head_dim=wide + 128, rotary_dim=64), dict(rotary_dim=wide + 64),
               dict(scaling="yarn", factor=2.0, original_max_position=wide + 4096)):
        with pytest.raises((ValueError, rig.S.StrataError)):
            rig.S.Rope(**{"head_dim": 128, **kw})
    assert not rig.calls


def test_scale_beyond_fp32_is_refused(rig):
    """The kernels work with scale * log2(e) in fp32: a scale that overflows there would make every row NaN."""
    S = rig.S
    c = S.strata_kv4_cache(0x10000, 0x20000, 0x30000, 0x40000, 10, 2, 16, 128)
    real = ctypes.CDLL(S.LIB_PATH).strata_kv4_attention
    real.restype, real.argtypes = S._SIGS["strata_kv4_attention"]

    def status(scale):  # of a call without tokens, which has nothing to do
        d = S.strata_kv4_attn_desc(0, 4, 1, 3, 0, 512, 512, 0, scale)
        return real(ctypes.addressof(c), ctypes.addressof(d), *[None] * 8, 0, None)

    assert status(2.3e38) == status(-2.3e38) == S.STRATA_OK
    for scale in (2.4e38, 3.4e38, -2.4e38):
        assert status(scale) == S.STRATA_ERR_INVALID_ARG


def test_timeout_selftest_refusals(rig):
    S = rig.S
    c = S.strata_kv4_cache(0x10000, 0x20000, 0x30000, 0x40000, 10, 2, 16, 128)
    d = S.strata_kv4_attn_desc(0, 4, 1, 3, 0, 512, 512, 0, 1.0)
    args = (c, d, 0, 0, 0, 0, 0, 0, 0)
    for bad in ((-1, 1, 0), (4, 1, 0), (0, 0, 0), (0, 1, -1)):
        with pytest.raises(S.StrataError) as e:
            S.strata_selftest_attention_timeout(*args, *bad, stream=0)
        assert e.value.status == S.STRATA_ERR_INVALID_ARG
    S.strata_selftest_attention_timeout(*args, 0, 1, 0, stream=0)  # no tokens: nothing to do
