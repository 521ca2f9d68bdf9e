"""What the calls of 16-bit experts and adapters allocate for work on a `stream` of the caller's comes from that stream's
memory pool, and a stream of another device is refused."""
from types import SimpleNamespace

import pytest
import torch

import moe_prefill_ffn_amd as mp
from test_operator_streams import FakeTensor, after_a_freed_block, fake as operator_fake  # noqa: F401

gpu = pytest.mark.gpu


@pytest.fixture
def fake(operator_fake):  # noqa: F811
    real, lib = mp.__dict__["_lib"], mp.lib()
    for name in ("moe_group_rows", "moe_grouped_gemm", "moe_combine_rows", "moe_lora_add"):
        setattr(lib, name, lambda *a, name=name: operator_fake.calls.append((name, a[-1])) or mp.MOE_OK)
    lib.moe_group_workspace_size, lib.moe_lora_workspace_size = real.moe_group_workspace_size, real.moe_lora_workspace_size
    return operator_fake


class Tensor(FakeTensor):
    def stride(self, dim=None):
        s = [1]
        for n in reversed(self.shape[1:]):
            s.insert(0, s[0] * n)
        return tuple(s) if dim is None else s[dim]


def calls():
    bf = lambda *s: Tensor(s, torch.bfloat16)  # noqa: E731
    i32 = lambda *s: Tensor(s, torch.int32)  # noqa: E731
    f32 = lambda *s: Tensor(s, torch.float32)  # noqa: E731
    return {
        "moe_group_rows": lambda s: mp.moe_group_rows(i32(3000, 2), 5, stream=s),
        "moe_grouped_gemm": lambda s: mp.moe_grouped_gemm(bf(3, 64), bf(5, 64), stream=s),
        "moe_combine_rows": lambda s: mp.moe_combine_rows(bf(6, 64), f32(3, 2), i32(3, 2), stream=s),
        "moe_lora_add": lambda s: mp.moe_lora_add(bf(3, 64), bf(2, 8, 64), bf(2, 40, 8), i32(3), stream=s),
    }


@pytest.mark.parametrize("name", list(calls()))
def test_memory_comes_from_the_stream_that_uses_it(fake, name):
    side = SimpleNamespace(device_index=0, cuda_stream=22)
    r = calls()[name](side)
    assert fake.calls == [(name, 22)]
    assert fake.made and all(s is side for _, s in fake.made)
    for t in (r if isinstance(r, tuple) else (r,)):
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


@gpu
def test_results_next_to_a_freed_block():
    g = torch.Generator().manual_seed(3)
    eidx = torch.randint(-1, 40, (3000, 4), generator=g).int().cuda()
    x, w = torch.randn(1500, 512, generator=g).bfloat16().cuda(), torch.randn(700, 512, generator=g).bfloat16().cuda()
    a, b = torch.randn(3, 16, 512, generator=g).bfloat16().cuda(), torch.randn(3, 700, 16, generator=g).bfloat16().cuda()
    ids = torch.randint(-1, 3, (1500,), generator=g).int().cuda()
    pos, wts = torch.randint(-1, 1500, (900, 4), generator=g).int().cuda(), torch.randn(900, 4, generator=g).cuda()
    n_lora, n_group = mp.moe_lora_workspace_size(1500, 512, 16), mp.moe_group_workspace_size(12000, 40)
    for nbytes, call in ((n_group, lambda s: mp.moe_group_rows(eidx, 40, stream=s)[2]), (1500 * 700 * 2, lambda s: mp.moe_grouped_gemm(x, w, stream=s)),
                         (900 * 512 * 2, lambda s: mp.moe_combine_rows(x, wts, pos, stream=s)), (n_lora, lambda s: mp.moe_lora_add(x, a, b, ids, stream=s)),
                         (1500 * 700 * 2, lambda s: mp.moe_lora_add(x, a, b, ids, stream=s))):
        want = call(None)
        assert torch.equal(after_a_freed_block(nbytes, torch.cuda.Stream(), call), want)
