"""Calls of the cache attention at the edges of what its contract allows; every row within its own bounds (those of
test_gpu_cache_units)."""
import math

import pytest
import torch

import _history_ref as ref
from test_gpu_cache_attend import Setup
from test_gpu_cache_units import check_rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ikbo():
    import attention_ikbo_b200 as m

    m.load_library()
    return m


def check(ikbo, s, out):
    assert ikbo.rocs_read_status(ikbo.rocs_dca_cache_forward.last_workspace) == (0, 0)
    check_rows(*out, s.q.cuda(), tuple(s.cache), s.table, s.lens, s.off, s.q_tokens, s.scale, None if s.limit is None else s.limit.cuda())


@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("G", [31, 43, 63, 64, 65, 128])
def test_many_heads_share_keys(ikbo, G, dh):
    """Tiles of 128 rows filled by 4, 2 and 1 query tokens, with rows left over and without."""
    s = Setup(ikbo, [9, 0, 1, 5], 1, [300, 20, 129, 128], 2 * G, 2, dh, 32, G + dh, limits=True)
    check(ikbo, s, s.call(ikbo))


@pytest.mark.parametrize("n", [2, 150])
def test_extreme_limits_and_no_scale(ikbo, n):
    s = Setup(ikbo, [n, n], 2, [400, 129], 2, 1, 128, 64, 41)
    s.limit = torch.tensor([(2 ** 31 - 1, -2 ** 31, 1, 0, -1, 128, 129, 2 ** 30)[i % 8] for i in range(2 * n)], dtype=torch.int32)
    check(ikbo, s, s.call(ikbo))
    s.scale = 0.0  # the mean of the visible values
    check(ikbo, s, s.call(ikbo))
    s.limit = torch.zeros(2 * n, dtype=torch.int32)
    o, lse = s.call(ikbo)
    assert torch.all(o == 0) and torch.all(lse == -math.inf)


@pytest.mark.parametrize("count", [1, 120])
def test_requests_far_apart(ikbo, count):
    """A hundred thousand requests of which a few have candidates, the first and the last among them."""
    R, g = 100_000, torch.Generator().manual_seed(5)
    counts = torch.zeros(R, dtype=torch.long)
    counts[torch.randint(0, R, (60,), generator=g)] = count
    counts[0] = counts[R - 1] = count
    k, v, ks, vs = ref.make_cache(30, 16, 2, 64, g)
    lens = torch.randint(0, 5 * 16, (R,), generator=g)
    table = torch.randint(0, 30, (R, 5), generator=g, dtype=torch.int32)
    off = torch.cat((torch.zeros(1, dtype=torch.long), counts.cumsum(0))).tolist()
    q = torch.randn(off[-1], 4, 64, generator=g).bfloat16().cuda()
    cache = tuple(t.cuda() for t in (k, v, ks, vs))
    o, lse = ikbo.rocs_dca_cache_forward(q, ikbo.CacheQ4(*cache), table.cuda(), lens.to(torch.int32).cuda(), off, 1, 0.125)
    assert ikbo.rocs_read_status(ikbo.rocs_dca_cache_forward.last_workspace) == (0, 0)
    check_rows(o, lse, q, cache, table, lens.tolist(), off, 1, 0.125)


def test_graphs_that_share_a_workspace(ikbo):
    """Two captured calls of different kernels in one workspace, replayed in turn with eager calls in between."""
    a, b = Setup(ikbo, [200, 3], 1, [900, 90], 2, 2, 128, 64, 51), Setup(ikbo, [2, 5, 1], 2, [700, 20, 3000], 4, 2, 64, 16, 52)
    ws, graphs, outs = torch.empty(1 << 27, dtype=torch.uint8, device="cuda"), [], []
    for s in (a, b):
        q, table, lens, off = s.q.cuda(), s.table.cuda(), torch.tensor(s.lens, dtype=torch.int32).cuda(), ikbo.offsets(s.off)
        o, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")

        def call(s=s, q=q, table=table, lens=lens, off=off, o=o, lse=lse):
            return ikbo.rocs_dca_cache_forward(q, s.cache, table, lens, off, s.q_tokens, s.scale, o=o, lse=lse, workspace=ws)

        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        graphs.append((graph, call))
        outs.append((o, lse))
    for turn in range(3):
        for s, (graph, call), out in zip((a, b), graphs, outs):
            for t in out:
                t.fill_(math.nan)
            graph.replay() if turn != 1 else call()
            b.call(ikbo)
            torch.cuda.synchronize()
            assert ikbo.rocs_read_status(ws) == (0, 0)
            check(ikbo, s, out)


@pytest.mark.parametrize("n", [1, 3, 140])
@pytest.mark.parametrize("dh", [64, 128])
def test_lengths_around_every_border(ikbo, n, dh):
    """Histories that end at, before and behind the borders of pages, granules and blocks."""
    lens = [x + d for x in (16, 32, 64, 128, 256, 384) for d in (-1, 0, 1)] + [1, 2, 0]
    for page in (16, 128):
        s = Setup(ikbo, [n] * len(lens), 1, lens, 2, 1, dh, page, 60 + n + page)
        check(ikbo, s, s.call(ikbo))
