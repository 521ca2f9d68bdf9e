"""What the few-token layer and the MXFP4 calls allocate for work on a `stream` of the caller's comes from
that stream's memory pool: a block of the current stream's pool may still be in use by kernels queued there."""
import contextlib
import math
from types import SimpleNamespace

import pytest
import torch

import moe_prefill_ffn_amd as mp
from test_decode import Layer, inputs
from test_mxfp4 import random_mx

gpu = pytest.mark.gpu


# --------------------------------------------- which stream allocates (CPU) ---

class FakeTensor:
    """As much of a device tensor as the binding looks at."""
    is_cuda = True

    def __init__(self, shape, dtype):
        self.shape, self.dtype, self.recorded = torch.Size(shape if isinstance(shape, (tuple, list)) else (shape,)), dtype, []

    def get_device(self):
        return 0

    def dim(self):
        return len(self.shape)

    def numel(self):
        return math.prod(self.shape)

    def stride(self):
        return self.shape[1], 1

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 4096

    def record_stream(self, s):
        self.recorded.append(s)


@pytest.fixture
def fake(monkeypatch):
    """The binding over a library that takes every call, with the stream of each allocation noted."""
    real, current = mp.lib(), SimpleNamespace(device_index=0, cuda_stream=11)
    state = SimpleNamespace(stack=[current], made=[], calls=[], current=current)

    @contextlib.contextmanager
    def on(stream):
        state.stack.append(stream)
        yield
        state.stack.pop()

    def empty(shape, dtype, device):
        t = FakeTensor(shape, dtype)
        state.made.append((t, state.stack[-1]))
        return t

    def call(name):
        def f(*a):
            state.calls.append((name, a[-1]))
            return mp.MOE_OK
        return f

    names = ["moe_decode_run_layer", "moe_mxfp4_quantize", "moe_mxfp4_dequantize", "moe_mxfp4_gemm"]
    lib = SimpleNamespace(moe_decode_workspace_size=real.moe_decode_workspace_size, **{n: call(n) for n in names})
    monkeypatch.setattr(mp, "lib", lambda: lib)
    monkeypatch.setattr(mp, "_raw_stream", lambda index: current.cuda_stream)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: state.stack[-1])
    return state


def calls():
    u8 = lambda *s: FakeTensor(s, torch.uint8)  # noqa: E731
    f32 = lambda *s: FakeTensor(s, torch.float32)  # noqa: E731
    handle = SimpleNamespace(params=dict(d_model=64, d_ff=96, n_experts=4, top_k=2, device=0), layer_bytes=10, ptr=None)
    return {
        "moe_decode_run_layer": lambda s: mp.moe_decode_run_layer(handle, f32(3, 64), f32(3, 4), f32(3, 64), weights=u8(10), stream=s),
        "moe_mxfp4_quantize": lambda s: mp.moe_mxfp4_quantize(f32(3, 64), stream=s),
        "moe_mxfp4_dequantize": lambda s: mp.moe_mxfp4_dequantize(u8(3, 32), u8(3, 2), stream=s),
        "moe_mxfp4_gemm": lambda s: mp.moe_mxfp4_gemm(u8(3, 32), u8(3, 2), u8(5, 32), u8(5, 2), stream=s),
    }


@pytest.mark.parametrize("name", list(calls()))
def test_memory_comes_from_the_stream_that_uses_it(fake, name):
    side = SimpleNamespace(device_index=0, cuda_stream=22)
    r = calls()[name](side)
    assert fake.calls == [(name, 22)]
    assert fake.made and all(s is side for _, s in fake.made)
    for t in (r if isinstance(r, tuple) else () if r is None else (r,)):
        assert t.recorded == [fake.current]               # the caller goes on with it there
    fake.made.clear()
    calls()[name](None)
    assert fake.calls[1:] == [(name, 11)]
    assert fake.made and all(s is fake.current for _, s in fake.made)


@pytest.mark.parametrize("name", list(calls()))
def test_a_stream_of_another_device_is_refused(fake, name):
    with pytest.raises(ValueError):
        calls()[name](SimpleNamespace(device_index=1, cuda_stream=33))
    assert not fake.calls and not fake.made


# ---------------------------------------- a block that is still being read ---

def after_a_freed_block(nbytes, side, call):
    """`call(side)` while the current stream has yet to read a block of nbytes that the allocator would
    hand out next: what was read must be what the block held."""
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    block = torch.full((nbytes,), 7, dtype=torch.uint8, device="cuda")
    copy = torch.zeros_like(block)
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)                         # some 10 ms
    copy.copy_(block)
    del block
    r = call(side)
    torch.cuda.synchronize()
    assert (copy == 7).all()
    return r


@gpu
@pytest.mark.parametrize("T", [1, 5, 40])
def test_a_layer_next_to_a_freed_block(T):
    L = Layer(1024, 512, 8, 4)
    h, blob = mp.moe_prefill_create(L.d, L.f, L.E, L.k, 4), L.host.cuda()
    x, lg = (t.cuda() for t in inputs(T, L, torch.float32))
    want = torch.empty_like(x)
    mp.moe_decode_run_layer(h, x, lg, want, weights=blob)
    nbytes = mp.moe_decode_workspace_size(L.d, L.f, L.E, L.k, T)
    for _ in range(3):
        y = torch.full_like(x, 77.0)
        after_a_freed_block(nbytes, torch.cuda.Stream(),
                            lambda s: mp.moe_decode_run_layer(h, x, lg, y, weights=blob, stream=s))
        assert torch.equal(y, want)
    h.close()


@gpu
def test_mxfp4_results_next_to_a_freed_block():
    g = torch.Generator().manual_seed(3)
    x = torch.randn(300, 2048, generator=g).cuda()
    b = [t.cuda() for t in random_mx(g, 500, 2048, hi=120)]
    codes, scales = mp.moe_mxfp4_quantize(x)
    values, out = mp.moe_mxfp4_dequantize(codes, scales), mp.moe_mxfp4_gemm(codes, scales, *b)
    for want, call in ((codes, lambda s: mp.moe_mxfp4_quantize(x, stream=s)[0]),
                       (scales, lambda s: mp.moe_mxfp4_quantize(x, stream=s)[1]),
                       (values, lambda s: mp.moe_mxfp4_dequantize(codes, scales, stream=s)),
                       (out, lambda s: mp.moe_mxfp4_gemm(codes, scales, *b, stream=s))):
        assert torch.equal(after_a_freed_block(want.numel() * want.element_size(), torch.cuda.Stream(), call), want)


@gpu
def test_results_belong_to_the_stream_that_wrote_them():
    """The allocator's own record of the segments that the results lie in."""
    side = torch.cuda.Stream()
    x = torch.randn(300, 2048, device="cuda")
    torch.cuda.synchronize()
    codes, scales = mp.moe_mxfp4_quantize(x, stream=side)
    owner = {}
    for seg in torch.cuda.memory_snapshot():
        for t in (codes, scales):
            if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
                owner[t.data_ptr()] = seg["stream"]
    side.synchronize()
    assert owner == {codes.data_ptr(): side.cuda_stream, scales.data_ptr(): side.cuda_stream}
