"""Edges of the expert layers and of the products' epilogues: infinities, values
that cancel or vanish, rows that nobody names, tails of the activations, the
default stream by its number; against definitions in 64 bits. Tolerances stand
beside each test, in units of u = 2^-24, half a step of f32."""

import math

import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def bq():
    import dequantize_absmax_reduce_b200 as m
    assert torch.cuda.is_available()
    return m


def gen(seed):
    return torch.Generator().manual_seed(seed)


# ---------------------------------------------------------------- the default stream by its number
def test_stream_zero_is_the_default_stream(bq):
    """stream=0, the default stream's handle: calls stay in the order of that stream's work."""
    g = gen(91)
    e, h = 8, 256
    w1, s1 = bq.api.fp8_block_quantize((0.05 * torch.randn((e * 512, h), generator=g)).bfloat16().cuda(), 128)
    w2, s2 = bq.api.fp8_block_quantize((0.05 * torch.randn((e * h, 256), generator=g)).bfloat16().cuda(), 128)
    weights = (w1.view(e, 512, h), s1.view(e, 4, 2), w2.view(e, h, 256), s2.view(e, 2, 2))
    new = torch.randn((300, h), generator=g).bfloat16().cuda()
    logits = torch.randn((300, e), generator=g).cuda()
    want = bq.api.fp8_moe(new, logits, *weights, 4)
    x = torch.zeros_like(new)
    bq.api.fp8_moe(x, logits, *weights, 4, stream=0)
    torch.cuda.synchronize()
    assert torch.cuda.current_stream().cuda_stream == 0
    torch.cuda._sleep(100_000_000)                    # some 50 ms, behind which x gets its values
    x.copy_(new)
    out = bq.api.fp8_moe(x, logits, *weights, 4, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
