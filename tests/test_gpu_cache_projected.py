"""From a request's sequence to attention over its cached history with the framework's own entry points: the stacked K/V
projection (rocs_proj_forward), its two halves appended as they lie, the queries normed and rotated, IKBO-DCA."""
import pytest
import torch

from test_gpu_cache_units import check_rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ikbo():
    import attention_ikbo_b200 as m

    m.load_library()
    return m


@pytest.mark.parametrize("H,dh,d_s", [(2, 128, 64), (4, 64, 256)])
@pytest.mark.parametrize("n", [2, 90])
def test_sequence_to_attention(ikbo, H, dh, d_s, n):
    """The cache's rows: half a step of the code, what the rounded step (15 of it) and minimum lose, one rounding when read.
    The attention: each row within its own bounds."""
    g = torch.Generator(device="cuda").manual_seed(H + n)
    R, page = 3, 32
    w_kv = (torch.randn(2 * H * dh, d_s, generator=g, device="cuda") * d_s ** -0.5).bfloat16()
    cache = ikbo.CacheQ4.empty(60, page, H, dh)
    table = torch.randperm(60, generator=g, device="cuda").to(torch.int32).view(R, 20)
    lens = torch.zeros(R, dtype=torch.int32, device="cuda")
    for counts in ([130, 7, 0], [5, 200, 1]):
        off = [0, counts[0], sum(counts[:2]), sum(counts)]
        s_seq = torch.randn(off[-1], d_s, generator=g, device="cuda").bfloat16()
        kv = ikbo.rocs_proj_forward(s_seq, w_kv).view(-1, 2, H, dh)
        k, v = kv[:, 0], kv[:, 1]
        ikbo.rocs_cache_append(cache, k, v, off, lens, table)
        kr, vr = ikbo.rocs_cache_read(cache, off, lens, table)
        assert ikbo.rocs_read_status(ikbo.rocs_cache_append.last_workspace) == (0, 0)
        for got, x in ((kr, k.double()), (vr, v.double())):
            lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
            step = (hi - lo) / 15
            tol = 0.5 * step + 15 * 2.0 ** -8 * step + 2.0 ** -8 * lo.abs() + 2.0 ** -8 * (x.abs() + step)
            assert torch.all((got.double() - x).abs() <= tol)
        lens += torch.tensor(counts, dtype=torch.int32, device="cuda")
    off = [0, n, n, 2 * n]
    q, _ = ikbo.rocs_qk_norm_rope_forward(torch.randn(2 * n, H, dh, generator=g, device="cuda").bfloat16())
    o, lse = ikbo.rocs_dca_cache_forward(q, cache, table, lens, off, 1, dh ** -0.5)
    assert ikbo.rocs_read_status(ikbo.rocs_dca_cache_forward.last_workspace) == (0, 0)
    clean = ikbo.CacheQ4(cache.k_codes, cache.v_codes, cache.k_scale.nan_to_num(0.0, 0.0, 0.0), cache.v_scale.nan_to_num(0.0, 0.0, 0.0))
    used = torch.zeros(60, page, dtype=torch.bool, device="cuda")
    for r in range(R):
        j = torch.arange(int(lens[r]), device="cuda")
        used[table[r].long()[j // page], j % page] = True
    for t in (clean.k_scale, clean.v_scale):  # places that no token has been put to hold anything
        t[~used[:, None].expand(-1, H, -1)] = 0.0
    check_rows(o, lse, q, tuple(clean), table, lens.tolist(), off, 1, dh ** -0.5)
