"""A base at the output's address: of the same type and row stride it is the call in place, of another one refused."""
import pytest
import torch

import moe_prefill_ffn_amd as mp
from test_experts16 import combine_args
from test_lora import lora_args

gpu = pytest.mark.gpu


@pytest.mark.parametrize("bad", [
    dict(base=65536, y=65536, base_dtype=mp.MOE_F32, y_dtype=mp.MOE_BF16), dict(base=65536, y=65536, base_dtype=mp.MOE_F16, y_dtype=mp.MOE_BF16),
    dict(base=65536, y=65536, base_stride=128), dict(base=65536, y=65536, n_tokens=1, y_dtype=mp.MOE_F16)])
def test_combine_refusals(bad):
    assert mp.lib().moe_combine_rows(combine_args(**bad), None) == mp.MOE_EINVAL
    assert "base is y" in mp.moe_prefill_last_error()


@pytest.mark.parametrize("bad", [
    dict(base=262144, base_dtype=mp.MOE_F32, out_dtype=mp.MOE_BF16), dict(base=262144, base_dtype=mp.MOE_BF16, out_dtype=mp.MOE_F16),
    dict(base=262144, base_stride=48), dict(base=262144, out_stride=41), dict(base=262144, M=1, base_dtype=mp.MOE_F16)])
def test_lora_refusals(bad):
    assert mp.lib().moe_lora_add(lora_args(**bad), None) == mp.MOE_EINVAL
    assert "base is out" in mp.moe_prefill_last_error()


@gpu
@pytest.mark.parametrize("T", [1, 40])
def test_views_of_one_buffer(T):
    """The same tensor, a view of it with another type or stride, and a base beside the output in its rows."""
    g = torch.Generator().manual_seed(T)
    buf = torch.randn(T, 128, generator=g).cuda()
    d, w, pos = torch.randn(6, 64, generator=g).cuda(), torch.rand(T, 2, generator=g).cuda(), torch.randint(-1, 6, (T, 2), generator=g).int().cuda()
    x, a, b = [torch.randn(*s, generator=g).bfloat16().cuda() for s in ((T, 64), (3, 8, 64), (3, 64, 8))]
    ids = torch.randint(-1, 3, (T,), generator=g).int().cuda()
    for call in (lambda base, out: mp.moe_combine_rows(d, w, pos, out, base=base), lambda base, out: mp.moe_lora_add(x, a, b, ids, base, out)):
        want = call(buf[:, :64].clone(), torch.empty(T, 64, device="cuda"))
        beside = buf.clone()
        assert torch.equal(call(beside[:, :64], beside[:, 64:]), want) and torch.equal(beside[:, :64], buf[:, :64])
        inner = buf.clone()
        assert torch.equal(call(inner[:, :64], inner[:, :64]), want) and torch.equal(inner[:, 64:], buf[:, 64:])
        with pytest.raises(mp.MoePrefillError):
            call(inner[:, :64], inner.view(torch.bfloat16)[:, :64])
        if T > 1:
            with pytest.raises(mp.MoePrefillError):
                call(inner[:, :64], inner.view(-1)[: T * 64].view(T, 64))
