"""Attention over the paged 4-bit cache: calls of thousands of short units, so that each block of the grid takes many of
them, with empty histories and rows that are not finite among them; every row against its own bounds.

Bounds for a row, with its own sums over the keys j that it sees (probabilities p_j): scores are off by at most
    d = 2^-22 (dh + 8) scale sum_d |q_d| max_j (47 step_j + |minimum_j|) + 2^-21 |score|
(fp32 sums of dh exact products, codes held as 16 + c), the LSE by d and 2^-22 of itself.  P and V are rounded to bf16 once
each, at most 2^-8 relative, and the output once: |o - exact| <= 2^-8 |o| + (2 * 2^-8 + 2 d) sum_j p_j (|v_j| + |minimum_j|)
always.  These roundings are independent of each other with mean zero, so that a sum of them beyond 8 times
2^-8 sqrt(2 sum_j (p_j v_j)^2) has a probability below 2 exp(-32) for each value: 1e-6 for 10^8 of them.
"""
import math

import pytest
import torch

import _history_ref as ref
from test_gpu_cache_attend import CASES, Setup

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ikbo():
    import attention_ikbo_b200 as m

    m.load_library()
    return m


def check_rows(o, lse, q, cache, table, lens, off, q_tokens, scale, limit=None):
    """Every value of o and lse within its row's bounds; NaN exactly where a visible row is held as NaN."""
    ro, rl, mag, spread = ref.attend_rows(q, cache, table, lens, off, q_tokens, scale, limit)
    top = (cache[2][..., 0].double() * 47 + cache[2][..., 1].double().abs()).nan_to_num(0.0).max()
    fin = rl > -math.inf
    assert torch.equal(lse > -math.inf, fin) and torch.equal(torch.isnan(lse), torch.isnan(rl))
    assert torch.equal(torch.isnan(o), torch.isnan(ro))
    assert torch.all(o[~fin & ~torch.isnan(rl)] == 0)
    d = 2.0 ** -22 * (q.shape[2] + 8) * scale * q.double().abs().sum(-1) * top
    d = d + 2.0 ** -21 * rl.where(fin, torch.zeros_like(rl)).abs() + 2.0 ** -20
    assert torch.all(((lse - rl).abs() <= d)[fin])
    o = o.double()
    bound = torch.minimum(2 * mag, 8 * 2 ** 0.5 * spread) * 2.0 ** -8 + 2.0 ** -8 * ro.abs() + 2 * d[..., None] * mag
    far = ((o - ro).abs() > bound) & ~torch.isnan(ro)
    assert not far.any(), (far.nonzero()[:5].tolist(), float((o - ro).abs()[far].max()))


def histories(R, hk, dh, page, longest, seed):
    """R histories of 0 ... longest tokens (one in five empty, alone and in rows) over a small pool whose pages they share.
    Every seventh one ends with a page whose last row of V is held as NaN."""
    g = torch.Generator().manual_seed(seed)
    pool = 24
    k, v, ks, vs = ref.make_cache(pool + 1, page, hk, dh, g)
    vs[pool, :, page - 1] = math.nan
    lens = torch.randint(1, longest + 1, (R,), generator=g)
    lens[torch.rand(R, generator=g) < 0.1] = 0
    for at in torch.randint(0, R, (R // 30,), generator=g).tolist():
        lens[at:at + 1 + at % 7] = 0
    cols = -(-longest // page)
    table = torch.randint(0, pool, (R, cols), generator=g, dtype=torch.int32)
    for r in range(0, R, 7):
        if lens[r] > 0:
            n = max(1, min(cols, -(-int(lens[r]) // page)))
            lens[r] = n * page
            table[r, n - 1] = pool
    assert (lens == 0).sum() > R // 10
    return tuple(t.cuda() for t in (k, v, ks, vs)), table, lens


MANY = [  # requests, fewest and most candidates, query tokens, key heads, heads to each, dh, page, longest, limits
    (1500, 70, 300, 1, 1, 1, 128, 64, 400, False),
    (1000, 40, 150, 1, 3, 2, 64, 16, 400, False),
    (400, 70, 300, 1, 8, 1, 128, 128, 384, False),
    (700, 20, 100, 1, 2, 5, 64, 32, 300, True),
    (2000, 70, 128, 1, 1, 1, 64, 16, 128, False),
    (900, 30, 130, 2, 2, 1, 128, 32, 250, True),
]


@pytest.mark.parametrize("R,lo,hi,q,hk,G,dh,page,longest,limits", MANY)
def test_thousands_of_short_units(ikbo, R, lo, hi, q, hk, G, dh, page, longest, limits):
    cache, table, lens = histories(R, hk, dh, page, longest, 7 * R + dh)
    g = torch.Generator().manual_seed(R)
    counts = torch.randint(lo, hi + 1, (R,), generator=g)
    off = [0] + counts.cumsum(0).tolist()
    qt = (1.5 * torch.randn(off[-1] * q, hk * G, dh, generator=g)).bfloat16().cuda()
    limit = None
    if limits:
        limit = ((torch.rand(off[-1], generator=g) * 1.4 - 0.2) * lens.repeat_interleave(counts)).floor().to(torch.int32).cuda()
    c, tb, ln, scale = ikbo.CacheQ4(*cache), table.cuda(), lens.to(torch.int32).cuda(), dh ** -0.5
    o, lse = ikbo.rocs_dca_cache_forward(qt, c, tb, ln, off, q, scale, key_limit=limit)
    assert ikbo.rocs_read_status(ikbo.rocs_dca_cache_forward.last_workspace) == (0, 0)
    assert ikbo.last_launch_count() == 1
    check_rows(o, lse, qt, cache, table, lens, off, q, scale, limit)
    assert torch.isnan(o).any()
    again = ikbo.rocs_dca_cache_forward(qt, c, tb, ln, off, q, scale, key_limit=limit)
    assert torch.equal(o.view(torch.int16), again[0].view(torch.int16)) and torch.equal(lse, again[1])
    # the first candidates of each request by the kernel for few rows
    rows = torch.tensor(off[:-1])[:, None] * q + torch.arange(q)
    few = ikbo.rocs_dca_cache_forward(qt[rows.flatten().cuda()], c, tb, ln, list(range(R + 1)), q, scale,
                                      key_limit=None if limit is None else limit[torch.tensor(off[:-1]).cuda()])
    assert ikbo.rocs_read_status(ikbo.rocs_dca_cache_forward.last_workspace) == (0, 0)
    check_rows(*few, qt[rows.flatten().cuda()], cache, table, lens, list(range(R + 1)), q, scale,
               None if limit is None else limit[torch.tensor(off[:-1]).cuda()])


@pytest.mark.parametrize("counts,q,lens,H,hk,dh,page,limits", CASES)
def test_every_row_within_its_own_bounds(ikbo, counts, q, lens, H, hk, dh, page, limits):
    s = Setup(ikbo, counts, q, lens, H, hk, dh, page, 31 + sum(counts) + dh, limits)
    o, lse = s.call(ikbo)
    check_rows(o, lse, s.q.cuda(), tuple(s.cache), s.table, s.lens, s.off, q, s.scale, None if s.limit is None else s.limit.cuda())
