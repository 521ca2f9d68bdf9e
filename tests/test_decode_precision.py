"""The few-token layer holds bf16 and fp16 activations, and h, to as many bits as fp32 ones: the bound of
24 bits a block for every type, blocks with an outlier, and the same bits as a call in fp32."""
import numpy as np
import pytest
import torch

import moe_prefill_ffn_amd as mp
import mx_reference as ref
from test_decode import DTYPES, Layer, inputs, layers, run  # noqa: F401  (layers: a fixture)

gpu = pytest.mark.gpu


def check24(y, L, x, lg, more=0.0):
    """As test_decode's check, with the bound of 24-bit blocks whatever x's type; more: of the norm."""
    want, bound, _, _ = L.reference(x.float(), lg)
    assert ((y.double() - want).abs() <= bound + ref.half_step(x.dtype) * (want.abs() + bound) + ref.least_step(x.dtype)).all()
    limit = (2e-6 + more + 1.2 * ref.half_step(x.dtype)) * float(want.norm()) + ref.least_step(x.dtype) * y.numel() ** 0.5
    assert float((y.double() - want).norm()) <= limit, (float((y.double() - want).norm()), limit)


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", [(96, 64, 5, 2), (1184, 352, 12, 4), (2048, 768, 9, 8)])
@pytest.mark.parametrize("T", [1, 5, 40])
def test_24_bits_of_every_type(layers, shape, T, dtype):
    L, h, blob = layers(*shape)
    x, lg = inputs(T, L, dtype, seed=T)
    check24(run(L, h, x, lg, blob)[0], L, x, lg)


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("shape", [(96, 64, 5, 2), (1184, 352, 12, 4), (2048, 768, 9, 8)])
@pytest.mark.parametrize("T", [1, 2, 7, 40])
def test_a_16_bit_call_is_the_fp32_call_rounded(layers, shape, T, dtype):
    L, h, blob = layers(*shape)
    x, lg = inputs(T, L, dtype, seed=T)
    assert torch.equal(run(L, h, x, lg, blob)[0], run(L, h, x.float(), lg, blob)[0].to(dtype))


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("ratio", [30, 300, 3000])
@pytest.mark.parametrize("T", [1, 5, 40])
def test_an_outlier_that_the_weights_ignore(T, ratio, dtype):
    """One channel of every block is `ratio` times the others and its weights are 0, so that y holds
    nothing of it.  A unit of the block is ratio 2^-23 (1 + 1/64), its rounding's rms 0.29 of that for each
    of x's other values (of size 1), for gate and up each: 0.9 ratio 2^-24 of y, and 5 here."""
    L = Layer(1024, 256, 6, 2)
    L.gu_q[:, :, 7::32] = 0

    class W:
        pass

    def expert(e):
        w = W()
        bits = lambda t: t[e].contiguous().numpy().view(np.uint16)  # noqa: E731
        w.wgu_q, w.wgu_s, w.wd_q, w.wd_s = L.gu_q[e].numpy(), bits(L.gu_s), L.d_q[e].numpy(), bits(L.d_s)
        return w

    mp.pack_layer(L.d, L.f, L.E, expert, L.host)
    h = mp.moe_prefill_create(L.d, L.f, L.E, L.k, 4)
    x, lg = inputs(T, L, dtype, seed=T)
    x[:, 7::32] = ratio
    y, _ = run(L, h, x, lg, L.host.cuda())
    h.close()
    check24(y, L, x, lg, more=5 * ratio * 2.0 ** -24)
