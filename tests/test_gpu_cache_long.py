"""Attention over long cached histories: the error must not grow with the number of keys.

The output's rounding to bf16 is at most 2^-8 of each value, so at most 2^-8 of a row's norm, and 2^-8 / sqrt(3) of the
norm over many rows (half a step is uniform, and a step is at most 2^-7 of the value).  Few rows: codes are exact, P' has 16
bits (2^-17 of it is left, independent from key to key), and fp32 sums that are joined every so many keys are off by far
less: 2^-12 of the norm is left for all of it, scores' fp32 sums among them (a score's error that all keys share cancels in
the softmax).  Many rows: P and V carry one rounding to bf16 each, independent from key to key, at most 2^-8 of each
product's size and 2^-8 / sqrt(3) in the mean square: with the products' own norm sqrt(sum_j (p_j v_j)^2) per value that is
sqrt(2 / 3) 2^-8 of it.
"""
import math

import pytest
import torch

import _history_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ikbo():
    import attention_ikbo_b200 as m

    m.load_library()
    return m


def shared_history(n, hk, dh, page, offset, seed):
    """One history of n keys (values around `offset`) that all requests of a call share."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    pages = -(-n // page)

    def side(mean):
        x = torch.randn(pages, hk, page, dh, generator=g, device="cuda") + mean
        lo, hi = x.amin(-1), x.amax(-1)
        step, mn = ((hi - lo) / 15).bfloat16(), lo.bfloat16()
        c = ((x - mn.float()[..., None]) / step.float()[..., None]).round().clamp(0, 15).long()
        w = (c << ref.channel_shift(dh).cuda()).unflatten(-1, (dh // 8, 8)).sum(-1)
        return torch.stack([w >> 8 * k & 255 for k in range(4)], -1).flatten(-2).to(torch.uint8), torch.stack((step, mn), -1)

    (kc, ks), (vc, vs) = side(0.0), side(offset)
    return (kc, vc, ks, vs), torch.arange(pages, dtype=torch.int32)[None]


CASES = [  # keys, requests, candidates, key heads, heads to each, dh, offset of V
    (65536, 64, 4, 8, 1, 128, 0.0),
    (131072, 64, 4, 8, 1, 128, 0.0),
    (131072, 60, 12, 4, 1, 128, 0.0),
    (131072, 64, 2, 4, 4, 64, 0.0),
    (300007, 40, 1, 8, 1, 64, 0.0),
    (131072, 64, 4, 8, 1, 128, 3.0),
    (131072, 8, 300, 8, 1, 128, 0.0),
    (262144, 6, 300, 8, 1, 64, 3.0),
    (600000, 40, 300, 2, 1, 64, 3.0),
]


@pytest.mark.parametrize("n,R,cand,hk,G,dh,offset", CASES)
def test_error_does_not_grow_with_the_history(ikbo, n, R, cand, hk, G, dh, offset):
    page, rows = 128, R * cand
    cache, one = shared_history(n, hk, dh, page, offset, n + dh)
    g = torch.Generator(device="cuda").manual_seed(5)
    q = torch.randn(rows, hk * G, dh, generator=g, device="cuda").bfloat16()
    lens = torch.full((R,), n, dtype=torch.int32, device="cuda")
    o, lse = ikbo.rocs_dca_cache_forward(q, ikbo.CacheQ4(*cache), one.cuda().repeat(R, 1), lens, [cand * r for r in range(R + 1)], 1,
                                         dh ** -0.5)
    assert ikbo.rocs_read_status(ikbo.rocs_dca_cache_forward.last_workspace) == (0, 0)
    # the requests share one history: the exact form takes a sample of rows as one request's
    take = torch.arange(0, rows, max(1, rows // 60), device="cuda")
    ro, rl, _, spread = ref.attend_rows(q[take], cache, one, [n], [0, len(take)], 1, dh ** -0.5)
    assert torch.all((lse[take] - rl).abs() <= 2.0 ** -16 * rl.abs())
    err, many = (o[take].double() - ro), cand * G > 48
    extra = (2 / 3) ** 0.5 * 2.0 ** -8 * spread.pow(2).sum().sqrt() / ro.norm() if many else 0.0
    print(f"error {err.norm() / ro.norm():.6f} of the norm, worst row {(err.norm(dim=-1) / ro.norm(dim=-1)).max():.6f}, extra {extra:.6f}")
    assert err.norm() <= math.hypot(2.0 ** -8 / 3 ** 0.5 + 2.0 ** -12, float(extra)) * ro.norm()
    if not many:
        assert torch.all(err.norm(dim=-1) <= (2.0 ** -8 + 2.0 ** -12) * ro.norm(dim=-1))


@pytest.mark.parametrize("n,R,cand,G,dh", [(20000, 300, 2, 1, 128), (20000, 300, 3, 4, 64), (100000, 110, 70, 1, 128),
                                           (70001, 150, 150, 2, 64)])
def test_maxima_and_limits_over_a_long_run(ikbo, n, R, cand, G, dh):
    """Runs long enough that sums are joined several times on the way: scores that grow along the history, limits that end
    anywhere (rows that see nothing, or nothing of what comes later), a NaN row behind most limits."""
    from test_gpu_cache_units import check_rows

    page, bad = 64, n * 3 // 5
    cache, one = shared_history(n, 1, dh, page, 0.5, 9)
    j = torch.arange(n, device="cuda")
    cache[2][j // page, 0, j % page] *= (2.0 ** (j // (n // 8)))[:, None].bfloat16()
    cache[3][bad // page, 0, bad % page] = math.nan
    g = torch.Generator().manual_seed(6)
    q = (0.05 * torch.randn(R * cand, G, dh, generator=g)).bfloat16().cuda()
    limit = torch.randint(0, n + 1, (R * cand,), generator=g, dtype=torch.int32)
    limit[::7] = torch.randint(0, 70, (len(limit[::7]),), generator=g, dtype=torch.int32)
    limit[3], limit[4], limit[5], limit[9] = 0, n, bad, bad + 1
    off, lens = [cand * r for r in range(R + 1)], [n - 17 * r for r in range(R)]
    table = one.repeat(R, 1)
    o, lse = ikbo.rocs_dca_cache_forward(q, ikbo.CacheQ4(*cache), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), off, 1,
                                         dh ** -0.5, key_limit=limit.cuda())
    assert ikbo.rocs_read_status(ikbo.rocs_dca_cache_forward.last_workspace) == (0, 0)
    check_rows(o, lse, q, cache, table, lens, off, 1, dh ** -0.5, limit.cuda())
    assert torch.isnan(o[4]).all() and not torch.isnan(o[5]).any() and torch.isnan(o[9]).all() and torch.all(o[3] == 0)
