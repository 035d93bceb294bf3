"""Attention over the paged 4-bit cache on the GPU against the 64-bit plain form.

Bounds, derived from the arithmetic: scores are sums of dh exact products in fp32, each addition off by at most 2^-22 of
the sum of magnitudes (a tensor core may truncate), so a score is off by at most
    d_i = 2^-22 (dh + 8) scale sum_d |q_id| max_j (47 step_j + |minimum_j|)
(codes are held as 16 + c <= 31, and 16 steps are taken off again), plus 2^-21 |score| for the exponent's argument.  An
LSE is off by the largest d and 2^-22 of itself.  Probabilities (or their products with a step) and values are rounded to
bf16 once each, the output once: |o - exact| <= 2^-8 |o| + (2 * 2^-8 + 2 d) sum_j p_j (|v_j| + |minimum_j|).
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


class Setup:
    """Histories in a shuffled page pool whose every place past a history holds NaN rows."""

    def __init__(self, ikbo, counts, q, lens, H, hk, dh, page, seed, limits=False, spare=2, std=1.0):
        g = self.g = torch.Generator().manual_seed(seed)
        self.counts, self.q_tokens, self.lens, self.page = counts, q, lens, page
        need = [-(-n // page) for n in lens]
        cols, total = max(need + [1]), sum(need)
        k, v, ks, vs = ref.make_cache(total + spare, page, hk, dh, g, std)
        order = torch.randperm(total + spare, generator=g).to(torch.int32)
        table = torch.full((len(lens), cols), -1, dtype=torch.int32)
        used = torch.zeros(total + spare, page, dtype=torch.bool)
        at = 0
        for r, n in enumerate(need):
            table[r, :n] = order[at:at + n]
            at += n
            j = torch.arange(lens[r])
            used[table[r].long()[j // page], j % page] = True
        for t in (ks, vs):  # [pages, heads, page, 2]
            t[~used[:, None, :].expand(-1, hk, -1)] = math.nan
        self.host = (k, v, ks, vs)
        self.cache = ikbo.CacheQ4(*(t.cuda() for t in self.host))
        self.table = table
        self.off = [0]
        for c in counts:
            self.off.append(self.off[-1] + c)
        C = self.off[-1]
        self.q = (1.5 * torch.randn(C * q, H, dh, generator=g)).bfloat16()
        self.limit = None
        if limits:
            of = torch.tensor([n for n, c in zip(lens, counts) for _ in range(c)], dtype=torch.float64)
            self.limit = ((torch.rand(C, generator=g).double() * 1.4 - 0.2) * of).floor().to(torch.int32)
        self.scale = 1.0 / math.sqrt(dh)

    def call(self, ikbo, **kw):
        lens = torch.tensor(self.lens, dtype=torch.int32).cuda()
        return ikbo.rocs_dca_cache_forward(kw.pop("q", None) if "q" in kw else self.q.cuda(), self.cache, self.table.cuda(), lens,
                                           self.off, self.q_tokens, self.scale,
                                           key_limit=None if self.limit is None else self.limit.cuda(), **kw)

    def check(self, o, lse):
        if o.numel() == 0:
            assert self.off[-1] == 0
            return
        ro, rl = ref.attend(self.q, self.host, self.table, self.lens, self.off, self.q_tokens, self.scale, self.limit)
        # magnitudes: the same sums with |v| + |minimum|
        mag_v = (ref.values(self.host[1], self.host[3]).abs() + self.host[3][..., 1:].double().abs()).nan_to_num(0.0)
        scales = torch.stack([self.host[2][..., 0].double() * 47 + self.host[2][..., 1].double().abs()]).nan_to_num(0.0)
        dh = self.q.shape[2]
        d = 2.0 ** -22 * (dh + 8) * self.scale * self.q.double().abs().sum(-1) * scales.max()
        fin = rl > -math.inf
        o, lse = o.cpu().double(), lse.cpu().double()
        assert torch.equal(lse > -math.inf, fin) and torch.equal(o[~fin], torch.zeros_like(o[~fin]))
        d = d + 2.0 ** -21 * rl.where(fin, torch.zeros(())).abs() + 2.0 ** -20
        assert torch.all((lse - rl)[fin].abs() <= d[fin])
        bound = mag_v.max()  # of every row's weighted mean of |v| + |minimum|
        assert torch.all((o - ro).abs() <= 2.0 ** -8 * ro.abs() + (2 * 2.0 ** -8 + 2 * d[..., None]) * bound)
        # and, far tighter than the bound of the worst case, on average
        assert (o - ro).abs().mean() <= 2.0 ** -8 * (ro.abs().mean() + 0.1 * bound)


CASES = [  # counts, q, lens, H, key heads, dh, page, limits
    ([1], 1, [1], 1, 1, 64, 16, False),
    ([1], 1, [1000], 8, 8, 128, 64, False),
    ([1, 0, 2, 3], 4, [17, 40, 0, 129], 3, 3, 128, 16, False),
    ([2, 1, 5, 1], 1, [2049, 63, 700, 1], 8, 2, 64, 32, False),
    ([4, 7, 1], 2, [300, 15, 128], 6, 2, 128, 128, True),
    ([16], 1, [4000], 2, 2, 64, 64, True),
    ([17, 16, 1], 1, [500, 500, 500], 4, 4, 128, 64, False),
    ([20, 3], 1, [200, 257], 5, 1, 64, 16, True),
    ([129, 0, 40, 300], 1, [129, 50, 0, 260], 2, 2, 128, 64, False),
    ([33, 200], 4, [1000, 127], 1, 1, 64, 32, True),
    ([90, 11], 1, [385, 1], 6, 2, 128, 128, True),
    ([257], 1, [1100], 3, 3, 64, 16, False),
    ([1] * 300, 1, [(7 * i) % 90 for i in range(300)], 2, 1, 64, 16, True),
    ([3] * 40, 2, [1 + 31 * i for i in range(40)], 4, 1, 128, 64, False),
    ([60] * 9, 1, [13 * i for i in range(9)], 7, 1, 128, 32, True),
    ([1] * 40 + [300, 0, 200], 1, [(11 * i) % 200 for i in range(43)], 2, 2, 128, 64, True),
    ([3] * 30 + [260] + [2] * 10, 1, [(17 * i) % 150 for i in range(41)], 4, 2, 64, 16, False),
    ([9, 30, 2], 1, [600, 70, 33], 1, 1, 128, 16, False),
    ([2, 1], 1, [300, 129], 130, 2, 64, 32, True),
]


@pytest.mark.parametrize("counts,q,lens,H,hk,dh,page,limits", CASES)
def test_against_plain(ikbo, counts, q, lens, H, hk, dh, page, limits):
    s = Setup(ikbo, counts, q, lens, H, hk, dh, page, 11 + sum(counts) + dh, limits)
    o, lse = s.call(ikbo)
    assert ikbo.rocs_read_status(ikbo.rocs_dca_cache_forward.last_workspace) == (0, 0)
    s.check(o, lse)
    again = s.call(ikbo)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


def test_seeded_shapes(ikbo):
    import random

    rng = random.Random(5)
    for i in range(40):
        R = rng.randint(1, 6)
        hk, G = rng.choice((1, 2, 3)), rng.choice((1, 2, 3, 5, 8))
        counts = [rng.choice((0, 1, 2, rng.randint(1, 40), rng.randint(1, 150))) for _ in range(R)]
        lens = [rng.choice((0, 1, 16, 127, 128, 129, rng.randint(1, 900))) for _ in range(R)]
        s = Setup(ikbo, counts, rng.choice((1, 2, 4)), lens, hk * G, hk, rng.choice((64, 128)), rng.choice((16, 32, 64, 128)),
                  100 + i, rng.random() < 0.5)
        o, lse = s.call(ikbo)
        assert ikbo.rocs_read_status(ikbo.rocs_dca_cache_forward.last_workspace) == (0, 0)
        s.check(o, lse)


@pytest.mark.parametrize("n", [2, 150])
def test_masked_and_visible_nan_rows(ikbo, n):
    s = Setup(ikbo, [n, n], 1, [300, 200], 2, 1, 128, 64, 3, limits=True)
    s.limit = torch.tensor([100 + i % 40 for i in range(n)] + [200] * n, dtype=torch.int32)
    k, v, ks, vs = s.host
    for t in (ks, vs):  # a NaN row that only limits above 120 see, one that the second request sees
        t[int(s.table[0, 1]), :, 120 - 64] = math.nan
    o, lse = Setup.call(_moved(ikbo, s), ikbo)
    seen = (s.limit[:n] > 120).tolist() + [False] * n
    for i, bad in enumerate(seen):
        assert bool(torch.isnan(o[i]).all()) == bad and bool(torch.isnan(lse[i]).any()) == bad, i
    # only the values' row is NaN: O is NaN where it is seen, the LSE is not
    ks[int(s.table[0, 1]), :, 120 - 64] = 0.25
    o, lse = Setup.call(_moved(ikbo, s), ikbo)
    for i, bad in enumerate(seen):
        assert bool(torch.isnan(o[i]).all()) == bad and not torch.isnan(lse[i]).any(), i
    # a constant key row (step 0), a row of large finite values behind every limit
    ks[int(s.table[0, 1]), :, 120 - 64] = torch.tensor([0.0, 0.5]).bfloat16()
    vs[int(s.table[0, 1]), :, 120 - 64] = torch.tensor([0.0, -0.5]).bfloat16()
    for t in (ks, vs):
        t[int(s.table[0, 3]), :, 7] = torch.tensor([1e37, -3e38]).bfloat16()
    o, lse = Setup.call(_moved(ikbo, s), ikbo)
    for t in (ks, vs):
        t[int(s.table[0, 3]), :, 7] = 0.5
    s.check(o, lse)


def _moved(ikbo, s):
    s.cache = ikbo.CacheQ4(*(t.cuda() for t in s.host))
    return s


@pytest.mark.parametrize("n", [3, 140])
def test_strided_queries_streams_and_no_lse(ikbo, n):
    s = Setup(ikbo, [n, 1], 2, [333, 20], 4, 2, 64, 32, 8)
    o, lse = s.call(ikbo)
    wide = torch.full(((n + 1) * 2, 4 * 64 + 72), math.nan, dtype=torch.bfloat16, device="cuda")
    view = wide[:, 8:8 + 256].view(-1, 4, 64)
    view.copy_(s.q.cuda())
    o2, none = s.call(ikbo, q=view, lse=False)
    assert none is None and torch.equal(o, o2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o3, lse3 = s.call(ikbo, stream=side)
    side.synchronize()
    assert torch.equal(o, o3) and torch.equal(lse, lse3)
    s.check(o, lse)


@pytest.mark.parametrize("n", [2, 200])
def test_captured_call_follows_lengths(ikbo, n):
    s = Setup(ikbo, [n, n], 1, [400, 300], 2, 2, 128, 64, 9)
    lens = torch.tensor(s.lens, dtype=torch.int32).cuda()
    off = ikbo.offsets(s.off)
    q, table = s.q.cuda(), s.table.cuda()
    ws = torch.empty(1 << 27, dtype=torch.uint8, device="cuda")
    o, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")

    def call():
        ikbo.rocs_dca_cache_forward(q, s.cache, table, lens, off, 1, s.scale, o=o, lse=lse, workspace=ws)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for new in ([400, 300], [1, 300], [257, 0], [0, 0], [399, 128]):
        lens.copy_(torch.tensor(new, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        s.lens = new
        s.check(o, lse)
        assert ikbo.rocs_read_status(ws) == (0, 0)


@pytest.mark.parametrize("n", [2, 150])
def test_bad_pages_and_lengths_are_reported(ikbo, n):
    s = Setup(ikbo, [n, n], 1, [200, 100], 2, 2, 64, 64, 10)
    good = s.call(ikbo)[0]
    table = s.table.clone()
    table[0, 1] = 10 ** 6
    s.table = table
    o, _ = s.call(ikbo)
    assert ikbo.rocs_read_status(ikbo.rocs_dca_cache_forward.last_workspace)[0] == 7
    assert torch.equal(o[n:], good[n:])  # the other request is as it was
    s = Setup(ikbo, [n, n], 1, [200, 100], 2, 2, 64, 64, 10)
    s.lens = [10 ** 6, 100]
    o, _ = s.call(ikbo)
    assert ikbo.rocs_read_status(ikbo.rocs_dca_cache_forward.last_workspace)[0] == 7
    assert torch.equal(o[n:], good[n:])


def test_no_candidates(ikbo):
    s = Setup(ikbo, [0, 0], 1, [20, 100], 2, 2, 64, 64, 10)
    o, lse = s.call(ikbo)
    assert o.shape == (0, 2, 64) and lse.shape == (0, 2)
    e = ikbo.CacheQ4.empty(0, 16, 2, 64)  # no pages at all: every history is empty
    o, lse = ikbo.rocs_dca_cache_forward(torch.ones(3, 2, 64, dtype=torch.bfloat16, device="cuda"), e,
                                         torch.zeros(1, 0, dtype=torch.int32, device="cuda"),
                                         torch.zeros(1, dtype=torch.int32, device="cuda"), [0, 3], 1, 1.0)
    assert torch.all(o == 0) and torch.all(lse == -math.inf)


@pytest.mark.parametrize("n", [1, 70])
def test_norm_append_attend_together(ikbo, n):
    """A request's history grown in two additions, queries normed and rotated, all as a user runs them; the dense path
    (read back as bf16, rocs_dca_forward) agrees to bf16."""
    g = torch.Generator().manual_seed(4)
    H, dh, page = 4, 128, 16
    cache = ikbo.CacheQ4.empty(40, page, H, dh)
    for t in cache:
        t.view(torch.uint8).fill_(255)
    table = torch.randperm(40, generator=g).to(torch.int32).view(2, 20).cuda()
    rope = ikbo.rocs_rope_table(600, dh)
    gam = torch.rand(dh, generator=g).cuda() + 0.5
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    for counts in ([130, 7], [3, 64], [0, 1]):
        T = sum(counts)
        k = torch.randn(T, H, dh, generator=g).bfloat16().cuda()
        v = torch.randn(T, H, dh, generator=g).bfloat16().cuda()
        _, k = ikbo.rocs_qk_norm_rope_forward(None, k, gamma_k=gam)
        ikbo.rocs_cache_append(cache, k, v, [0, counts[0], T], lens, table, rope=rope)
        lens += torch.tensor(counts, dtype=torch.int32, device="cuda")
    off = [0, n, 2 * n]
    pos = torch.cat([torch.full((n,), int(x), dtype=torch.int32) for x in lens.tolist()]).cuda()
    q, _ = ikbo.rocs_qk_norm_rope_forward(torch.randn(2 * n, H, dh, generator=g).bfloat16().cuda(), pos_q=pos, rope=rope, gamma_q=gam)
    o, lse = ikbo.rocs_dca_cache_forward(q, cache, table, lens, off, 1, dh ** -0.5)
    host = tuple(t.cpu() for t in cache)
    ro, rl = ref.attend(q.cpu(), host, table.cpu(), lens.tolist(), off, 1, dh ** -0.5)
    vmax = 4 * float(ro.abs().max())
    assert torch.all((o.cpu().double() - ro).abs() <= 2.0 ** -8 * ro.abs() + 2.0 ** -6 * vmax)
    assert torch.all((lse.cpu().double() - rl).abs() <= 1e-3)
    seq = [0, int(lens[0]), int(lens.sum())]
    kd, vd = ikbo.rocs_cache_read(cache, seq, torch.zeros_like(lens), table)
    od, _ = ikbo.rocs_dca_forward(q, kd, vd, off, seq, 1, dh ** -0.5)
    assert torch.all((od.cpu().double() - ro).abs() <= 2.0 ** -8 * ro.abs() + 2.0 ** -5 * vmax)


def test_outputs_over_queries_are_refused(ikbo):
    s = Setup(ikbo, [3], 1, [40], 2, 2, 64, 16, 21)
    q = s.q.cuda()
    with pytest.raises(ikbo.RocsError):
        s.call(ikbo, q=q, o=q)


@pytest.mark.parametrize("n", [4, 300])
def test_infinite_and_nan_queries_stay_in_their_rows(ikbo, n):
    s = Setup(ikbo, [n, 2], 1, [260, 40], 2, 1, 64, 32, 22)
    good = s.call(ikbo)
    s.q[1, 0, 5] = math.nan
    s.q[2, 1, 9] = math.inf
    s.limit = torch.tensor([260] * (n + 2), dtype=torch.int32)
    s.limit[3] = 0
    s.q[3] = math.nan  # sees nothing: O = 0, LSE = -inf all the same
    o, lse = s.call(ikbo)
    assert torch.isnan(o[1, 0]).all() and torch.isnan(lse[1, 0]) and torch.isnan(o[2, 1]).any()
    assert torch.all(o[3] == 0) and torch.all(lse[3] == -math.inf)
    keep = torch.ones(n + 2, 2, dtype=torch.bool)
    keep[1, 0] = keep[2, 1] = False
    keep[3] = False
    # Not the same bits: which maximum a row's sums are taken against depends on its neighbours in the warp (votes, limits).
    # Each side's LSE is off by at most 260 additions of 2^-24 and 2^-24 of scores below 2^6 (in base 2), each P by one
    # rounding to bf16, each output by another.
    assert torch.all((lse.cpu() - good[1].cpu())[keep].abs() <= 2 * (260 + 64 + 16) * 2.0 ** -24)
    vmax = float(ref.values(s.host[1], s.host[3]).nan_to_num(0.0).abs().max())
    assert torch.all((o.cpu().float() - good[0].cpu().float())[keep].abs() <= 2 * 2.0 ** -8 * 2 * vmax)


def test_two_streams_at_once(ikbo):
    """Calls on two streams at the same time, each with its own workspace."""
    a, b = Setup(ikbo, [300, 3], 1, [500, 90], 2, 2, 128, 64, 23), Setup(ikbo, [2, 5], 2, [700, 20], 4, 2, 64, 16, 24)
    want = a.call(ikbo), b.call(ikbo)
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(5):
        with torch.cuda.stream(sa):
            x = a.call(ikbo)
        with torch.cuda.stream(sb):
            y = b.call(ikbo)
        got.append((x, y))
    torch.cuda.synchronize()
    for x, y in got:
        assert all(torch.equal(u, w) for u, w in zip(x + y, want[0] + want[1]))


def test_scores_that_grow_along_the_history(ikbo):
    """Every block of keys raises the rows' maxima by far: what was summed before moves to the new maximum each time."""
    for n in (3, 20, 200):
        s = Setup(ikbo, [n], 1, [700], 1, 1, 128, 64, 25)
        k, v, ks, vs = s.host
        j = torch.arange(700)
        pg, sl = s.table[0].long()[j // 64], j % 64
        ks[pg, 0, sl] = ks[pg, 0, sl] * (2.0 ** (j // 70).float())[:, None].bfloat16()
        o, lse = Setup.call(_moved(ikbo, s), ikbo)
        s.check(o, lse)


def test_long_cache_rows_past_32_bits(ikbo):
    """A pool whose rows lie past 2^31 codes and 2^32 bytes from its start."""
    page, heads, dh = 128, 16, 128
    pages = (1 << 32) // (page * heads * dh // 2) + 40  # 4.3 GB of codes each
    c = ikbo.CacheQ4(*(torch.zeros(pages, heads, page, dh // 2, dtype=torch.uint8, device="cuda") for _ in range(2)),
                     *(torch.zeros(pages, heads, page, 2, dtype=torch.bfloat16, device="cuda") for _ in range(2)))
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn(200, heads, dh, generator=g).bfloat16() for _ in range(2))
    table = torch.tensor([[pages - 1, pages - 30]], dtype=torch.int32).cuda()
    zero = torch.zeros(1, dtype=torch.int32).cuda()
    ikbo.rocs_cache_append(c, k.cuda(), v.cuda(), [0, 200], zero, table)
    kr, vr = ikbo.rocs_cache_read(c, [0, 200], zero, table)
    small = ikbo.CacheQ4(*(t[[pages - 1, pages - 30]].contiguous() for t in c))
    t2 = torch.tensor([[0, 1]], dtype=torch.int32).cuda()
    lens = torch.tensor([200], dtype=torch.int32).cuda()
    k2, v2 = ikbo.rocs_cache_read(small, [0, 200], zero, t2)
    assert torch.equal(kr, k2) and torch.equal(vr, v2)
    for n in (2, 150):
        q = torch.randn(n, heads, dh, generator=g).bfloat16().cuda()
        far = ikbo.rocs_dca_cache_forward(q, c, table, lens, [0, n], 1, 0.1)
        near = ikbo.rocs_dca_cache_forward(q, small, t2, lens, [0, n], 1, 0.1)
        assert torch.equal(far[0], near[0]) and torch.equal(far[1], near[1])
