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


@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("n", [3, 200])
def test_large_finite_values(ikbo, n, dh):
    """A row of V from about -1.2e38 to 1.2e38, which the cache holds as finite values, is no row of NaN: with one key the
    output is that row.  Each value is off by the roundings of P and V (one each) and of the output: 3 * 2^-8 of the row's
    largest."""
    x = torch.linspace(-1.2e38, 1.2e38, dh)[torch.randperm(dh, generator=torch.Generator().manual_seed(1))].view(1, 1, dh)
    cache = ikbo.CacheQ4.empty(1, 16, 1, dh)
    for t in cache:
        t.view(torch.uint8).fill_(255)
    table, zero = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    ikbo.rocs_cache_append(cache, torch.ones(1, 1, dh, device="cuda"), x.cuda(), [0, 1], zero, table)
    held = ref.values(cache.v_codes.cpu()[0, 0, :1], cache.v_scale.cpu()[0, 0, :1])
    assert torch.isfinite(held).all()
    q = torch.randn(n, 1, dh, device="cuda").bfloat16()
    o, _ = ikbo.rocs_dca_cache_forward(q, cache, table, zero + 1, [0, n], 1, dh ** -0.5)
    assert torch.isfinite(o).all()
    assert torch.all((o.cpu().double()[:, 0] - held).abs() <= 3 * 2.0 ** -8 * held.abs().max())


def late_write(shape, dtype):
    """A tensor's memory given back while a write to it still waits on the current stream."""
    t = torch.empty(shape, dtype=dtype, device="cuda")
    torch.cuda._sleep(30_000_000)
    t.view(torch.uint8).fill_(255)


@pytest.mark.parametrize("op", ["norm_rope", "read", "attend", "attend_workspace", "table"])
def test_memory_of_another_stream(ikbo, op):
    """A call on a stream of its own while the current one still writes to memory that it has given back: outputs and
    workspaces must not come from there."""
    g = torch.Generator(device="cuda").manual_seed(2)
    T, H, dh = 4096, 4, 128
    x = torch.randn(T, H, dh, generator=g, device="cuda").bfloat16()
    cache = ikbo.CacheQ4.empty(T // 64, 64, H, dh)
    table, zero = torch.arange(T // 64, dtype=torch.int32, device="cuda")[None], torch.zeros(1, dtype=torch.int32, device="cuda")
    off, coff = ikbo.offsets([0, T]), ikbo.offsets([0, T])
    ikbo.rocs_cache_append(cache, x, x, off, zero, table)
    lens = zero + 700
    o, lse = torch.empty_like(x), torch.empty(T, H, device="cuda")
    side = torch.cuda.Stream()

    def call(stream):
        if op == "norm_rope":
            return ikbo.rocs_qk_norm_rope_forward(x, stream=stream)[:1]
        if op == "read":
            return ikbo.rocs_cache_read(cache, off, zero, table, stream=stream)
        if op == "attend":
            return ikbo.rocs_dca_cache_forward(x, cache, table, lens, coff, 1, 0.1, stream=stream)
        if op == "table":
            return (ikbo.rocs_rope_table(8192, 128, stream=stream),)
        return ikbo.rocs_dca_cache_forward(x, cache, table, lens, coff, 1, 0.1, o=o, lse=lse, stream=stream)

    want = [t.clone() for t in call(None)]
    nbytes = ikbo.rocs_dca_cache_forward.last_workspace.numel() if op == "attend_workspace" else None
    ikbo.rocs_dca_cache_forward.last_workspace = None
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    if op == "attend_workspace":
        late_write(nbytes, torch.uint8)
    else:
        late_write(want[0].shape, want[0].dtype)
    got = call(side)
    if op == "attend_workspace":
        got = [t.clone() for t in got] if side.synchronize() is None else None
        assert ikbo.rocs_read_status(ikbo.rocs_dca_cache_forward.last_workspace) == (0, 0)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("op", ["norm_rope", "read", "attend"])
def test_outputs_of_another_stream_read_later(ikbo, op):
    """Outputs of a call on a stream of its own, read on the current one behind other work and then given back: a second
    call must not be handed their memory before that."""
    g = torch.Generator(device="cuda").manual_seed(3)
    T, H, dh = 4096, 4, 128
    x, y = (torch.randn(T, H, dh, generator=g, device="cuda").bfloat16() for _ in range(2))
    caches = [ikbo.CacheQ4.empty(T // 64, 64, H, dh) for _ in range(2)]
    table, zero = torch.arange(T // 64, dtype=torch.int32, device="cuda")[None], torch.zeros(1, dtype=torch.int32, device="cuda")
    off, lens = ikbo.offsets([0, T]), zero + 300
    for c, t in zip(caches, (x, y)):
        ikbo.rocs_cache_append(c, t, t, off, zero, table)
    side = torch.cuda.Stream()

    def call(i, stream):
        if op == "norm_rope":
            return ikbo.rocs_qk_norm_rope_forward((x, y)[i], stream=stream)[0]
        if op == "read":
            return ikbo.rocs_cache_read(caches[i], off, zero, table, stream=stream)[0]
        return ikbo.rocs_dca_cache_forward(x, caches[i], table, lens, off, 1, 0.1, stream=stream)[0]

    want = [call(i, None).clone() for i in range(2)]
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    first = call(0, side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(30_000_000)
    copy = torch.empty_like(first).copy_(first)
    del first
    second = call(1, side)
    torch.cuda.synchronize()
    assert torch.equal(copy, want[0]) and torch.equal(second, want[1])
