"""Paged 4-bit cache: append and read on the GPU against 64-bit plain forms.

Without rotation the codes, steps and minima must be exact: the kernel's fp32 quotient (x - minimum) / step is correctly
rounded from a correctly rounded difference, and a code can differ from the 64-bit one only where the exact quotient is
within 16 * 2^-23 of a half; such a code may be the neighbour.  With rotation the keys carry two products and a sum in
fp32 (relative 2^-23 of the pair's magnitudes): a minimum or a step may then round to its bf16 neighbour, and a code
to its neighbour where the quotient is that near to a half.
"""
import pytest
import torch

import _history_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ikbo():
    import attention_ikbo_b200 as m

    m.load_library()
    return m


def gen(seed):
    return torch.Generator().manual_seed(seed)


def status(ikbo, fn):
    return ikbo.rocs_read_status(fn.last_workspace)


def setup(ikbo, counts, base, page, heads, dh, seed, dt=torch.bfloat16, spare=3):
    g = gen(seed)
    T = sum(counts)
    k, v = (torch.randn(T, heads, dh, generator=g) * 2 + 0.3).to(dt), torch.randn(T, heads, dh, generator=g).to(dt)
    need = [-(-(b + c) // page) for b, c in zip(base, counts)]
    cols, total = max(need + [1]), sum(need)
    order = torch.randperm(total + spare, generator=g).to(torch.int32)
    table = torch.full((len(counts), cols), -1, dtype=torch.int32)
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = order[at:at + n]
        at += n
    cache = ikbo.CacheQ4.empty(total + spare, page, heads, dh)
    for t in cache:
        t.view(torch.uint8).random_(0, 256)
    off = [0]
    for c in counts:
        off.append(off[-1] + c)
    return k, v, off, torch.tensor(base, dtype=torch.int32), table, cache


def places(off, base, table, page):
    """(page, slot in page) of each token."""
    pg, sl = [], []
    for r in range(len(off) - 1):
        for i in range(off[r + 1] - off[r]):
            j = int(base[r]) + i
            pg.append(int(table[r, j // page]))
            sl.append(j % page)
    return torch.tensor(pg, dtype=torch.long), torch.tensor(sl, dtype=torch.long)


def check_rows(codes, scale, x, slack):
    """Rows [T, heads, ...] of the cache against the 64-bit format of x; `slack`: relative error of x's values."""
    c, step, mn = ref.quantise(x)
    got_s, got_c = scale.cpu().double(), ref.codes_of(codes)
    if slack == 0:
        assert torch.equal(got_s[..., 0], step) and torch.equal(got_s[..., 1], mn)
    else:  # the bf16 neighbour where the exact value is that near to the middle between two
        big = x.abs().amax(-1)
        assert torch.all((got_s[..., 1] - x.amin(-1)).abs() <= 2.0 ** -8 * x.amin(-1).abs() + slack * big)
        exact = (x.amax(-1) - x.amin(-1)) / 15
        assert torch.all((got_s[..., 0] - exact).abs() <= 2.0 ** -8 * exact + slack * big)
    st, m = got_s[..., :1], got_s[..., 1:]
    quotient = torch.where(st > 0, (x - m) / torch.where(st > 0, st, 1.0), 0.0)
    near = 16 * 2.0 ** -23 + torch.where(st > 0, slack * x.abs().amax(-1, keepdim=True) / torch.where(st > 0, st, 1.0), 0.0)
    assert torch.all((got_c - quotient.clamp(0, 15)).abs() <= 0.5 + near)


CASES = [  # counts, base, page, heads, dh, dtype, rot, interleaved
    ([1], [0], 16, 1, 64, torch.bfloat16, 0, False),
    ([3, 0, 40, 1], [15, 7, 0, 128], 16, 3, 128, torch.bfloat16, 128, False),
    ([100, 1, 300], [0, 63, 1000], 64, 8, 128, torch.bfloat16, 64, True),
    ([7, 129, 0, 2], [125, 0, 3, 31], 128, 5, 64, torch.bfloat16, 64, False),
    ([50, 33], [31, 32], 32, 2, 64, torch.float32, 32, True),
    ([64] * 40, list(range(40)), 32, 4, 128, torch.float32, 128, False),
    ([2] * 1100, [5] * 1100, 16, 1, 64, torch.bfloat16, 16, False),
]


@pytest.mark.parametrize("counts,base,page,heads,dh,dt,rot,inter", CASES)
def test_append_and_read(ikbo, counts, base, page, heads, dh, dt, rot, inter):
    k, v, off, b, table, cache = setup(ikbo, counts, base, page, heads, dh, 3 + dh + page, dt)
    before = [t.clone() for t in cache]
    rope = ikbo.rocs_rope_table(2000, rot) if rot else None
    args = (off, b.cuda(), table.cuda())
    ikbo.rocs_cache_append(cache, k.cuda(), v.cuda(), *args, rope=rope, interleaved=inter)
    assert status(ikbo, ikbo.rocs_cache_append) == (0, 0)
    pg, sl = places(off, b, table, page)
    x = k.double()
    if rot:
        pos = torch.cat([torch.arange(int(b[r]), int(b[r]) + c) for r, c in enumerate(counts)])
        x = ref.rotate(x, rope.cpu().double()[pos], rot, inter)
    check_rows(cache.k_codes[pg.cuda(), :, sl.cuda()], cache.k_scale[pg.cuda(), :, sl.cuda()], x, 3 * 2.0 ** -23 if rot else 0)
    check_rows(cache.v_codes[pg.cuda(), :, sl.cuda()], cache.v_scale[pg.cuda(), :, sl.cuda()], v.double(), 0)
    # every other row of the cache as it was
    for now, was in zip(cache, before):
        was[pg.cuda(), :, sl.cuda()] = now[pg.cuda(), :, sl.cuda()]
        assert torch.equal(now.view(torch.uint8), was.view(torch.uint8))
    # and back: exactly the values that the rows stand for, rounded once
    kr, vr = ikbo.rocs_cache_read(cache, *args)
    assert status(ikbo, ikbo.rocs_cache_read) == (0, 0)
    for got, codes, scale in ((kr, cache.k_codes, cache.k_scale), (vr, cache.v_codes, cache.v_scale)):
        want = ref.values(codes.cpu()[pg, :, sl], scale.cpu()[pg, :, sl])
        assert torch.all((got.cpu().double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -24 * want.abs().amax(-1, keepdim=True))
        assert torch.equal(got.cpu(), want.float().bfloat16())


def test_positions_given(ikbo):
    k, v, off, b, table, cache = setup(ikbo, [5, 9], [3, 0], 16, 2, 64, 1)
    pos = torch.tensor([9, 1, 0, 49, 7, 3, 3, 3, 2, 1, 0, 11, 12, 13], dtype=torch.int32)
    rope = ikbo.rocs_rope_table(50, 64)
    ikbo.rocs_cache_append(cache, k.cuda(), v.cuda(), off, b.cuda(), table.cuda(), rope=rope, pos=pos.cuda())
    assert status(ikbo, ikbo.rocs_cache_append) == (0, 0)
    pg, sl = places(off, b, table, 16)
    x = ref.rotate(k.double(), rope.cpu().double()[pos.long()], 64, False)
    check_rows(cache.k_codes[pg.cuda(), :, sl.cuda()], cache.k_scale[pg.cuda(), :, sl.cuda()], x, 3 * 2.0 ** -23)


def test_strided_rows(ikbo):
    k, v, off, b, table, cache = setup(ikbo, [30, 4], [0, 9], 16, 3, 128, 2)
    wide = torch.randn(34, 1600, device="cuda").bfloat16()
    kw, vw = wide[:, 8:8 + 384].unflatten(1, (3, 128)), wide[:, 800:800 + 384].unflatten(1, (3, 128))
    kw.copy_(k), vw.copy_(v)
    other = ikbo.CacheQ4(*[t.clone() for t in cache])
    ikbo.rocs_cache_append(cache, k.cuda(), v.cuda(), off, b.cuda(), table.cuda())
    ikbo.rocs_cache_append(other, kw, vw, off, b.cuda(), table.cuda())
    for x, y in zip(cache, other):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    out = torch.zeros_like(wide)
    ko, vo = out[:, 8:8 + 384].unflatten(1, (3, 128)), out[:, 800:800 + 384].unflatten(1, (3, 128))
    ikbo.rocs_cache_read(cache, off, b.cuda(), table.cuda(), k=ko, v=vo)
    kr, vr = ikbo.rocs_cache_read(cache, off, b.cuda(), table.cuda())
    assert torch.equal(ko, kr) and torch.equal(vo, vr)
    assert torch.all(out[:, :8] == 0) and torch.all(out[:, 392:800] == 0) and torch.all(out[:, 1184:] == 0)


def test_special_rows(ikbo):
    """Constant rows (step 0), rows with infinities and NaN, tiny, denormal and huge ranges."""
    rows = torch.zeros(10, 1, 64)
    rows[0] = 3.25
    rows[1, 0, 5] = float("nan")
    rows[2, 0, 63] = float("inf")
    rows[3, 0, 0] = -float("inf")
    rows[4] = torch.linspace(-1, 1, 64) * 3e38
    rows[5] = torch.linspace(-1, 1, 64) * 1e-39
    rows[6] = torch.linspace(0, 1, 64) * 2.0 ** -133
    rows[7] = 1000 + torch.linspace(0, 1, 64)
    rows[8] = torch.linspace(-1, 1, 64) * 1.5e38
    cache = ikbo.CacheQ4.empty(1, 16, 1, 64)
    args = ([0, 10], torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(1, 1, dtype=torch.int32, device="cuda"))
    ikbo.rocs_cache_append(cache, rows.cuda(), rows.cuda(), *args)
    k, v = ikbo.rocs_cache_read(cache, *args)
    assert torch.equal(k.view(torch.int16), v.view(torch.int16))
    k = k.cpu().float()
    assert torch.all(k[0] == 3.25) and torch.all(k[9] == 0)
    assert torch.isnan(k[1:5]).all()  # the range of row 4, 6e38, is past fp32
    check_rows(cache.k_codes[0, :, [5, 6, 7, 8]].transpose(0, 1), cache.k_scale[0, :, [5, 6, 7, 8]].transpose(0, 1),
               rows[[5, 6, 7, 8]].double(), 0)
    assert torch.isfinite(k[5:]).all()


def test_bad_places_are_reported(ikbo):
    k, v, off, b, table, cache = setup(ikbo, [4, 4, 4], [0, 14, 0], 16, 2, 64, 5)
    before = [t.clone() for t in cache]
    pool = cache.k_codes.shape[0]
    bad = table.clone()
    bad[0, 0] = pool  # past the pool
    bad[1, 1] = -1    # request 1's last two tokens have no page
    base = torch.tensor([0, 14, 30], dtype=torch.int32)  # request 2: two tokens on no page, two past the table
    ikbo.rocs_cache_append(cache, k.cuda(), v.cuda(), off, base.cuda(), bad.cuda())
    code, detail = status(ikbo, ikbo.rocs_cache_append)
    assert (code, detail) == (7, 911)
    pg, sl = int(table[1, 0]), [14, 15]
    for now, was in zip(cache, before):
        was[pg, :, sl] = now[pg, :, sl]
        assert torch.equal(now.view(torch.uint8), was.view(torch.uint8))
    kr, _ = ikbo.rocs_cache_read(cache, off, base.cuda(), bad.cuda())
    assert status(ikbo, ikbo.rocs_cache_read) == (7, 921)
    assert torch.all(kr[[0, 1, 2, 3, 6, 7, 8, 9, 10, 11]] == 0)
    neg = torch.tensor([-3, -2147483648, 2147483647], dtype=torch.int32)
    ikbo.rocs_cache_append(cache, k.cuda(), v.cuda(), off, neg.cuda(), table.cuda())
    assert status(ikbo, ikbo.rocs_cache_append) == (7, 911)
    rope = ikbo.rocs_rope_table(2, 64)
    ikbo.rocs_cache_append(cache, k.cuda(), v.cuda(), off, b.cuda(), table.cuda(), rope=rope)
    assert status(ikbo, ikbo.rocs_cache_append) == (7, 912)
    ikbo.rocs_cache_append(cache, k.cuda(), v.cuda(), off, b.cuda(), table.cuda())
    assert status(ikbo, ikbo.rocs_cache_append) == (0, 0)


def test_graph_replay_grows_histories(ikbo):
    """A captured step (append one token a request, then count it) replayed: each replay goes one slot further."""
    R, page, heads, dh, n = 3, 16, 2, 64, 40
    k, v, off, b, table, cache = setup(ikbo, [n] * R, [0] * R, page, heads, dh, 6)
    whole = ikbo.CacheQ4(*[t.clone() for t in cache])
    rope = ikbo.rocs_rope_table(n, dh)
    ikbo.rocs_cache_append(whole, k.cuda(), v.cuda(), off, b.cuda(), table.cuda(), rope=rope)
    ks, vs = k.cuda().view(R, n, heads, dh), v.cuda().view(R, n, heads, dh)
    k1, v1 = ks[:, 0].contiguous(), vs[:, 0].contiguous()
    lens, tb, one = torch.zeros(R, dtype=torch.int32, device="cuda"), table.cuda(), ikbo.offsets(list(range(R + 1)))
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ikbo.rocs_cache_append(cache, k1, v1, one, lens, tb, rope=rope, workspace=ws)
        lens.add_(1)
    for i in range(n):
        k1.copy_(ks[:, i])
        v1.copy_(vs[:, i])
        g.replay()
    torch.cuda.synchronize()
    assert lens.tolist() == [n] * R
    for x, y in zip(cache, whole):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_dense_path_reads_the_cache(ikbo):
    """rocs_cache_read gives what rocs_dca_forward takes: attention over the read-back K/V runs."""
    k, v, off, b, table, cache = setup(ikbo, [100, 40], [0, 0], 32, 2, 64, 7)
    args = (off, b.cuda(), table.cuda())
    ikbo.rocs_cache_append(cache, k.cuda(), v.cuda(), *args)
    kr, vr = ikbo.rocs_cache_read(cache, *args)
    q = torch.randn(5, 2, 64, generator=gen(8)).bfloat16().cuda()
    o, lse = ikbo.rocs_dca_forward(q, kr, vr, [0, 3, 5], off, 1, 0.125)
    oo, ll = ref.attend(q, [t.cpu() for t in cache], table, [100, 40], [0, 3, 5], 1, 0.125)
    assert (o.cpu().double() - oo).abs().max() <= 1e-2 * oo.abs().max() + 1e-3


def test_tokens_behind_many_empty_requests(ikbo):
    """Tokens of one warp that belong to requests far apart."""
    counts = [0] * 5000 + [2] + [0] * 4000 + [3, 0, 1] + [0] * 3000
    base = [7 * (i % 3) for i in range(len(counts))]
    k, v, off, b, table, cache = setup(ikbo, counts, base, 16, 2, 64, 5)
    ikbo.rocs_cache_append(cache, k.cuda(), v.cuda(), off, b.cuda(), table.cuda())
    assert status(ikbo, ikbo.rocs_cache_append) == (0, 0)
    pg, sl = places(off, b, table, 16)
    check_rows(cache.k_codes[pg.cuda(), :, sl.cuda()], cache.k_scale[pg.cuda(), :, sl.cuda()], k.double(), 0)
    kr, vr = ikbo.rocs_cache_read(cache, off, b.cuda(), table.cuda())
    assert torch.equal(kr.cpu(), ref.values(cache.k_codes.cpu()[pg, :, sl], cache.k_scale.cpu()[pg, :, sl]).float().bfloat16())
    assert vr.shape == v.shape


def test_quotients_of_exactly_a_half(ikbo):
    """Values on a grid whose quotients are n + 1/2: half to even, and every code is used."""
    dh = 128
    x = torch.empty(40, 2, dh)
    x[..., 0::2] = torch.arange(dh // 2) % 16           # whole codes 0 ... 15: step 1, minimum 0
    x[..., 1::2] = (torch.arange(dh // 2) % 15) + 0.5   # halves
    x = x * torch.tensor([2.0 ** (i - 20) for i in range(40)])[:, None, None]
    cache = ikbo.CacheQ4.empty(3, 16, 2, dh)
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32).cuda()
    zero = torch.zeros(1, dtype=torch.int32).cuda()
    for dt in (torch.bfloat16, torch.float32):
        ikbo.rocs_cache_append(cache, x.to(dt).cuda(), (-x).to(dt).cuda(), [0, 40], zero, table)
        j = torch.arange(40)
        pg, sl = table.cpu()[0].long()[j // 16], j % 16
        c, step, mn = ref.quantise(x.double())
        assert torch.equal(ref.codes_of(cache.k_codes[pg.cuda(), :, sl.cuda()]), c)
        assert torch.equal(cache.k_scale[pg.cuda(), :, sl.cuda()].cpu().double(), torch.stack((step, mn), -1))
        assert torch.equal(ref.codes_of(cache.v_codes[pg.cuda(), :, sl.cuda()]), ref.quantise(-x.double())[0])


def test_refused_workspaces(ikbo):
    x = torch.randn(4, 2, 64, device="cuda").bfloat16()
    for ws in (torch.empty(256, dtype=torch.uint8), torch.empty(512, dtype=torch.uint8, device="cuda")[::2],
               torch.empty(100, dtype=torch.uint8, device="cuda"), torch.empty(512, dtype=torch.uint8, device="cuda")[16:]):
        with pytest.raises(ikbo.RocsError):
            ikbo.rocs_qk_norm_rope_forward(x, workspace=ws)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_codes_of_rotated_keys_are_the_definitions(ikbo, dt, inter):
    """Codes, steps and minima of rotated keys, bit for bit: rotation in fp32 with every operation rounded, then the format
    by fp32 division."""
    dh, heads, T = 128, 4, 4000
    g = torch.Generator(device="cuda").manual_seed(9)
    k = (torch.randn(T, heads, dh, generator=g, device="cuda") * 1.7).to(dt)
    rope = ikbo.rocs_rope_table(T, dh)
    cache = ikbo.CacheQ4.empty(T // 16, 16, heads, dh)
    table = torch.arange(T // 16, dtype=torch.int32, device="cuda")[None]
    ikbo.rocs_cache_append(cache, k, k, [0, T], torch.zeros(1, dtype=torch.int32, device="cuda"), table, rope=rope, interleaved=inter)
    c, s = rope[:, None, :dh // 2], rope[:, None, dh // 2:]
    x = k.float()
    a, b = (x[..., 0::2], x[..., 1::2]) if inter else (x[..., :dh // 2], x[..., dh // 2:])
    u, v = a * c - b * s, b * c + a * s
    rotated = torch.stack((u, v), -1).flatten(-2) if inter else torch.cat((u, v), -1)
    for codes, scale, y in ((cache.k_codes, cache.k_scale, rotated), (cache.v_codes, cache.v_scale, x)):
        lo, hi = y.amin(-1), y.amax(-1)
        step, mn = ((hi - lo) / 15).bfloat16(), lo.bfloat16()
        want = ((y - mn.float()[..., None]) / step.float()[..., None]).round().clamp(0, 15)
        got = codes.transpose(1, 2).reshape(T, heads, dh // 2)
        sc = scale.transpose(1, 2).reshape(T, heads, 2)
        assert torch.equal(sc[..., 0], step) and torch.equal(sc[..., 1], mn)
        assert torch.equal(ref.codes_of(got), want.cpu().long())
