"""Outputs that a call allocates come from the stream that the call writes them on: memory freed on the caller's
current stream may still be read there."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fx():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import top_fp4_lightning_amd

    return top_fp4_lightning_amd


def stream_of(t):
    """the handle of the stream whose allocations the tensor's memory belongs to"""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not in the allocator's memory")


def calls(fx):
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(300, 4, 128, device="cuda", generator=g).bfloat16()
    kv = torch.randn(300, 512, device="cuda", generator=g).bfloat16()
    pos = torch.arange(300, device="cuda")
    freq, _ = fx.rope_freqs(64)
    signs = torch.ones(128, dtype=torch.int8, device="cuda")
    codes, scales = fx.idx_quantize_kv(kv)
    base = torch.zeros(2, dtype=torch.int64, device="cuda")
    nv = torch.full((2,), 300, dtype=torch.int32, device="cuda")
    idx = torch.randint(0, 300, (2, 200), device="cuda", generator=g).int()
    return {
        "idx_rope": lambda s: (fx.idx_rope(x, pos, freq, stream=s),),
        "idx_quantize_q": lambda s: fx.idx_quantize_q(x, signs, stream=s),
        "idx_quantize_kv": lambda s: fx.idx_quantize_kv(kv, stream=s),
        "idx_gather_kv": lambda s: (fx.idx_gather_kv(codes, scales, base, nv, idx, stream=s),),
    }


@pytest.mark.parametrize("name", ["idx_rope", "idx_quantize_q", "idx_quantize_kv", "idx_gather_kv"])
def test_allocated_outputs_belong_to_the_stream(fx, name):
    call = calls(fx)[name]
    here = torch.cuda.current_stream().cuda_stream
    want = call(None)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert all(stream_of(t) == here for t in want)
    # a Stream, its handle, an object that only has one, and the default stream by either name
    class Handle:
        cuda_stream = side.cuda_stream

    for s, handle in ((side, side.cuda_stream), (side.cuda_stream, side.cuda_stream), (Handle(), side.cuda_stream),
                      (torch.cuda.default_stream(), 0), (0, 0)):
        got = call(s)
        torch.cuda.synchronize()
        assert all(stream_of(t) == handle for t in got), (name, s)
        assert all(torch.equal(a, b) and a.dtype is b.dtype and a.is_contiguous() for a, b in zip(got, want)), (name, s)
        assert torch.cuda.current_stream().cuda_stream == here


def test_strided_rows_give_a_contiguous_output(fx):
    x = torch.randn(4, 300, 128, device="cuda").bfloat16().transpose(0, 1)
    pos, (freq, _) = torch.arange(300, device="cuda"), fx.rope_freqs(64)
    y = fx.idx_rope(x, pos, freq, stream=torch.cuda.current_stream())
    assert y.is_contiguous() and torch.equal(y, fx.idx_rope(x.contiguous(), pos, freq))


def test_an_output_read_on_the_current_stream_outlives_its_name(fx):
    """freed while work that reads it is queued on the current stream: the next output of the side stream lies elsewhere
    until that work is done"""
    side = torch.cuda.Stream()
    freq, _ = fx.rope_freqs(64)
    pos = torch.arange(300, device="cuda")
    x = torch.randn(300, 4, 128, device="cuda").bfloat16()
    big, other = torch.randn(4096, 4096, device="cuda"), -x
    want = fx.idx_rope(x, pos, freq)
    torch.mm(big, big)
    torch.cuda.synchronize()
    for rep in range(3):
        y = fx.idx_rope(x, pos, freq, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        for _ in range(20):
            torch.mm(big, big)  # the current stream is busy; the read of y stands behind
        got, place = y.clone(), y.data_ptr()
        read = torch.cuda.Event()
        read.record()
        del y
        z = fx.idx_rope(other, pos, freq, stream=side)
        assert z.data_ptr() != place or read.query(), rep
        torch.cuda.synchronize()
        assert torch.equal(got, want), rep
        del z
