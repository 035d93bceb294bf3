"""Rows of the paged 4-bit cache at the edges of the format, and calls on another stream than the current one."""
import numpy as np
import pytest
import torch

import _history_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ikbo():
    import attention_ikbo_b200 as m

    m.load_library()
    return m


@pytest.mark.parametrize("dh", [64, 128])
def test_steps_midway_between_two_bf16_values(ikbo, dh):
    """Ranges that are 15 times a number of nine bits: a fifteenth lies midway between two bf16 values.  The format takes it as
    the fp32 product with 1/15, which may fall to either side of the middle (292 or 294 for a range of 4395): the step is
    that product's rounding, bit for bit, and as near to the exact fifteenth as any bf16 value, up to fp32."""
    ranges = torch.arange(257, 512, 2).float()[:, None] * 15.0 * 2.0 ** torch.arange(-8, 9, 4)[None]
    ranges = torch.cat((torch.tensor([4395.0]), ranges.flatten()))
    n = len(ranges)
    x = torch.rand(n, 1, dh, generator=torch.Generator().manual_seed(dh)) * ranges[:, None, None]
    x[:, 0, 3], x[:, 0, dh - 2] = 0.0, ranges
    cache = ikbo.CacheQ4.empty(-(-n // 16), 16, 1, dh)
    table = torch.arange(-(-n // 16), dtype=torch.int32, device="cuda")[None]
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    ikbo.rocs_cache_append(cache, x.cuda(), (-x).cuda(), [0, n], zero, table)
    step = torch.from_numpy(ranges.numpy() * np.float32(1 / 15)).bfloat16()
    assert step[0] == 294.0
    exact = ranges.double() / 15
    half = 2.0 ** (torch.floor(torch.log2(exact)) - 8)  # half a step of bf16, which has 8 bits
    assert torch.all((step.double() - exact).abs() <= half + 2.0 ** -23 * exact)
    for codes, scale, y in ((cache.k_codes, cache.k_scale, x), (cache.v_codes, cache.v_scale, -x)):
        got = scale.cpu().transpose(1, 2).reshape(-1, 2)[:n]
        assert torch.equal(got[:, 0], step) and torch.equal(got[:, 1], y[:, 0].amin(-1).bfloat16())
        want = ((y[:, 0] - got[:, 1:].float()) / step.float()[:, None]).round().clamp(0, 15).long()
        assert torch.equal(ref.codes_of(codes.transpose(1, 2).reshape(-1, dh // 2)[:n]), want)
    # bf16 input: 4800 and -15 have a range of 15 * 321
    b = torch.zeros(1, 1, dh)
    b[0, 0, 1], b[0, 0, 2] = 4800.0, -15.0
    ikbo.rocs_cache_append(cache, b.bfloat16().cuda(), b.bfloat16().cuda(), [0, 1], zero, table)
    assert cache.k_scale[0, 0, 0].tolist() == [322.0, -15.0] and cache.v_scale[0, 0, 0].tolist() == [322.0, -15.0]
