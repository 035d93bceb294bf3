"""Calls on a stream of their own while the current stream still writes to memory that it has given back: neither outputs nor
workspaces may come from there.  And their outputs, read later on the current stream and given back."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ikbo():
    import attention_ikbo_b200 as m

    m.load_library()
    return m


def make(ikbo, op, seed):
    """call(stream) -> outputs, the largest first"""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def r(*s):
        return torch.randn(*s, generator=g, device="cuda").bfloat16()

    R, C, n, d = 4, 256, 64, 128
    off = ikbo.offsets([0, 60, 100, 100, C])
    if op == "lcb":
        x, y, w = r(R, d, d), r(C, d, d), [r(d, d) / 8 for _ in range(3)]
        return lambda stream: ikbo.rocs_lcb_forward(x, y, *w, off, stream=stream)[::-1]
    if op == "fm":
        x, y = r(R, n, d), r(C, n, d)
        return lambda stream: ikbo.rocs_fm_forward(x, y, off, stream=stream)[::-1]
    if op == "dca":
        q, k, v, seq = r(4096, 4, d), r(1200, 4, d), r(1200, 4, d), ikbo.offsets([0, 300, 500, 900, 1200])
        cand = ikbo.offsets([0, 1000, 2000, 2000, 4096])
        return lambda stream: ikbo.rocs_dca_forward(q, k, v, cand, seq, 1, 0.1, stream=stream)
    if op == "proj":
        x, w = r(4096, 512), r(512, 512) / 16
        return lambda stream: (ikbo.rocs_proj_forward(x, w, stream=stream),)
    if op == "cache":
        k, v, q, tok = r(1200, 4, d), r(1200, 4, d), r(4096, 4, d), ikbo.offsets([0, 300, 500, 900, 1200])
        cache, cand = ikbo.CacheQ4.empty(28, 64, 4, d), ikbo.offsets([0, 1000, 2000, 2000, 4096])
        table = torch.arange(28, dtype=torch.int32, device="cuda").view(4, 7)
        zero, lens = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.tensor([300, 200, 400, 300], dtype=torch.int32, device="cuda")

        def call(stream):
            ikbo.rocs_cache_append(cache, k, v, tok, zero, table, stream=stream)
            x, _ = ikbo.rocs_qk_norm_rope_forward(q, stream=stream)
            return ikbo.rocs_dca_cache_forward(x, cache, table, lens, cand, 1, 0.1, stream=stream)

        return call
    x = r(4096, 500)
    return lambda stream: (ikbo.rocs_pad_cols(x, 512, stream=stream),)


OPS = ["lcb", "fm", "dca", "proj", "cache", "pad_cols"]


@pytest.mark.parametrize("op", OPS)
def test_memory_given_back_with_a_write_pending(ikbo, op):
    call, side = make(ikbo, op, 1), torch.cuda.Stream()
    want = [t.clone() for t in call(None)]
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    late = torch.empty_like(want[0])
    torch.cuda._sleep(30_000_000)
    late.view(torch.uint8).fill_(255)
    del late
    got = call(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("op", OPS)
def test_outputs_read_later_and_given_back(ikbo, op):
    calls, side = [make(ikbo, op, s) for s in (1, 2)], torch.cuda.Stream()
    want = [c(None)[0].clone() for c in calls]
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    first = calls[0](side)[0]
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(30_000_000)
    copy = torch.empty_like(first).copy_(first)
    del first
    second = calls[1](side)[0]
    torch.cuda.synchronize()
    assert torch.equal(copy, want[0]) and torch.equal(second, want[1])


@pytest.mark.parametrize("op", OPS)
def test_captured_on_a_forked_stream(ikbo, op):
    """A capture whose call is given the capturing stream, and one that forks a stream of its own for it."""
    call = make(ikbo, op, 1)
    want = [t.clone() for t in call(None)]
    for fork in (False, True):
        graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            here = torch.cuda.current_stream()
            if fork:
                side.wait_stream(here)
                got = call(side)
                here.wait_stream(side)
            else:
                got = call(here)
        for _ in range(2):
            for t in got:
                t.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))
