"""Per-head norm with the position rotation on the GPU against 64-bit plain forms.

Tolerance: one rounding to the output's type (half a step: eps/2 relative) and the fp32 arithmetic before it.  In fp32 a
row's sum of dh squares (or its mean) is off by at most dh + 8 roundings of 2^-24, the square root, quotient, products
with gamma and the two products and the sum of the rotation by some 12 more, of values no larger than the sum of the
pair's magnitudes: (dh + 20) * 2^-24 * 2 max|y| of the row covers them.
"""
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


def ok_status(ikbo):
    code, detail = ikbo.rocs_read_status(ikbo.rocs_qk_norm_rope_forward.last_workspace)
    assert code == 0, (code, detail)


def check(got, x, kind, gamma, beta, eps, table, pos, rot, interleaved):
    y = ref.norm(x.cpu().double(), kind, None if gamma is None else gamma.cpu(), None if beta is None else beta.cpu(), eps)
    big = y.abs().amax(-1, keepdim=True) if y.numel() else y
    if table is not None:
        y = ref.rotate(y, table.cpu().double()[pos.cpu().long()], rot, interleaved)
    dh = x.shape[-1]
    tol = torch.finfo(x.dtype).eps / 2 * y.abs() + (dh + 20) * 2.0 ** -24 * 2 * (big + (0 if beta is None else 1))
    assert got.dtype == x.dtype and got.shape == x.shape
    err = (got.cpu().double() - y).abs()
    assert torch.all(err <= tol), float((err - tol).max())


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


CASES = [  # nq, nk, hq, hk, dh, rot, norm, interleaved, dtype
    (4, 1, 8, 8, 128, 128, "rmsnorm", False, torch.bfloat16),
    (33, 70, 3, 1, 64, 64, "layernorm", False, torch.bfloat16),
    (17, 5, 5, 2, 128, 64, "rmsnorm", True, torch.bfloat16),
    (1, 130, 16, 4, 64, 16, "none", False, torch.bfloat16),
    (200, 31, 9, 7, 128, 128, "layernorm", True, torch.float32),
    (64, 64, 1, 1, 64, 32, "rmsnorm", False, torch.float32),
    (3, 0, 7, 2, 128, 48, "rmsnorm", False, torch.float32),
    (0, 9, 2, 12, 64, 48, "none", True, torch.bfloat16),
    (1000, 2001, 4, 4, 128, 96, "rmsnorm", False, torch.bfloat16),
]


@pytest.mark.parametrize("nq,nk,hq,hk,dh,rot,kind,inter,dt", CASES)
@pytest.mark.parametrize("params", [True, False])
def test_norm_rope(ikbo, nq, nk, hq, hk, dh, rot, kind, inter, dt, params):
    g = gen(nq + nk + dh)
    q = (torch.randn(nq, hq, dh, generator=g, device="cuda") * 3).to(dt)
    k = (torch.randn(nk, hk, dh, generator=g, device="cuda") + 0.7).to(dt)
    table = ikbo.rocs_rope_table(777, rot)
    pq = torch.randint(0, 777, (nq,), generator=g, device="cuda", dtype=torch.int32)
    pk = torch.randint(0, 777, (nk,), generator=g, device="cuda", dtype=torch.int32)
    w = [torch.randn(dh, generator=g, device="cuda") if params else None for _ in range(4)]
    qo, ko = ikbo.rocs_qk_norm_rope_forward(q, k, pq, pk, table, norm=kind, gamma_q=w[0], gamma_k=w[1], beta_q=w[2],
                                            beta_k=w[3], eps=1e-5, interleaved=inter)
    ok_status(ikbo)
    assert ikbo.last_launch_count() == 1
    check(qo, q, kind, w[0], w[2], 1e-5, table, pq, rot, inter)
    check(ko, k, kind, w[1], w[3], 1e-5, table, pk, rot, inter)


@pytest.mark.parametrize("kind", ["none", "layernorm", "rmsnorm"])
def test_no_rotation(ikbo, kind):
    q = torch.randn(50, 6, 64, generator=gen(1), device="cuda").bfloat16()
    qo, ko = ikbo.rocs_qk_norm_rope_forward(q, norm=kind)
    assert ko is None
    check(qo, q, kind, None, None, 1e-6, None, None, 0, False)
    if kind == "none":
        assert torch.equal(qo, q)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("inter", [True, False])
def test_in_place_inside_a_wider_projection(ikbo, dt, inter):
    """q, k and v side by side in one projection output; q and k turned in place, v and the rest untouched."""
    hq, hk, dh, n = 6, 2, 128, 77
    wide = torch.randn(n, (hq + 2 * hk) * dh + 8, generator=gen(2), device="cuda").to(dt)
    was = wide.clone()
    q = wide[:, : hq * dh].unflatten(1, (hq, dh))
    k = wide[:, hq * dh: (hq + hk) * dh].unflatten(1, (hk, dh))
    pos = torch.arange(n, device="cuda", dtype=torch.int32)
    table = ikbo.rocs_rope_table(n, dh)
    q2, k2 = ikbo.rocs_qk_norm_rope_forward(q, k, pos, pos, table, interleaved=inter, q_out=q, k_out=k)
    ok_status(ikbo)
    assert q2.data_ptr() == q.data_ptr()
    w = was[:, : (hq + hk) * dh].unflatten(1, (hq + hk, dh))
    check(q2, w[:, :hq], "rmsnorm", None, None, 1e-6, table, pos, dh, inter)
    check(k2, w[:, hq:], "rmsnorm", None, None, 1e-6, table, pos, dh, inter)
    assert torch.equal(wide[:, (hq + hk) * dh:], was[:, (hq + hk) * dh:])
    dense = ikbo.rocs_qk_norm_rope_forward(w[:, :hq].contiguous(), None, pos, None, table, interleaved=inter)[0]
    assert torch.equal(dense, q2)


def test_rope_table(ikbo):
    """Table entries are the rounded cosines and sines of the 64-bit angles, far positions among them.  The device's and
    the host's 64-bit angles differ by some 2^-50 of the angle (power and product), far below half a step of fp32."""
    n, rot = 100001, 64
    t = ikbo.rocs_rope_table(n, rot, base=500000.0).cpu().double()
    sel = np.array([0, 1, 2, 100, 4095, 65535, 99999, 100000])
    a = torch.from_numpy(ref.rope_angles(n, rot, 500000.0)[sel])
    want = torch.cat((a.cos(), a.sin()), 1)
    assert torch.all((t[sel] - want).abs() <= 2.0 ** -24 * want.abs() + 100001 * 2.0 ** -48)


def test_zero_rows_and_infinities(ikbo):
    x = torch.randn(5, 2, 64, generator=gen(3), device="cuda").bfloat16()
    x[1] = 0
    x[3, 1, 7] = float("inf")
    y, _ = ikbo.rocs_qk_norm_rope_forward(x, norm="rmsnorm", eps=1e-6)
    assert torch.all(y[1] == 0)
    assert not torch.isfinite(y[3, 1, 7])
    sel = [0, 2, 4]
    check(y[sel], x[sel], "rmsnorm", None, None, 1e-6, None, None, 0, False)
    check(y[3:4, :1], x[3:4, :1], "rmsnorm", None, None, 1e-6, None, None, 0, False)


def test_bad_position_is_reported(ikbo):
    x = torch.randn(4, 2, 64, generator=gen(4), device="cuda").bfloat16()
    table = ikbo.rocs_rope_table(10, 64)
    for bad in (10, -1, 2 ** 31 - 1):
        pos = torch.tensor([1, bad, 2, 9], dtype=torch.int32, device="cuda")
        y, _ = ikbo.rocs_qk_norm_rope_forward(x, None, pos, None, table)
        assert ikbo.rocs_read_status(ikbo.rocs_qk_norm_rope_forward.last_workspace) == (7, 901)
        sel = [0, 2, 3]
        check(y[sel], x[sel], "rmsnorm", None, None, 1e-6, table, pos[sel], 64, False)
    ikbo.rocs_qk_norm_rope_forward(x, None, pos.clamp(0, 9), None, table)
    ok_status(ikbo)


def test_graph_and_other_stream(ikbo):
    x = torch.randn(40, 8, 128, generator=gen(5), device="cuda").bfloat16()
    pos = torch.arange(40, device="cuda", dtype=torch.int32)
    table = ikbo.rocs_rope_table(64, 128)
    want, _ = ikbo.rocs_qk_norm_rope_forward(x, None, pos, None, table)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, _ = ikbo.rocs_qk_norm_rope_forward(x, None, pos, None, table, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    out, ws = torch.empty_like(x), torch.empty(256, dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ikbo.rocs_qk_norm_rope_forward(x, None, pos, None, table, q_out=out, workspace=ws)
    x.mul_(0.5)
    g.replay()
    want, _ = ikbo.rocs_qk_norm_rope_forward(x, None, pos, None, table)
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dh,rot", [(128, 128), (128, 64), (64, 64), (64, 32)])
def test_rotation_rounds_products_and_sums_one_by_one(ikbo, dh, rot, inter):
    """The bits of a * c - b * s and b * c + a * s with every operation rounded: what 4-bit codes are taken from must not
    depend on how the expression was compiled."""
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(3000, 3, dh, generator=g, device="cuda")
    pos = torch.randint(0, 4000, (3000,), generator=g, device="cuda", dtype=torch.int32)
    rope = ikbo.rocs_rope_table(4000, rot)
    y, _ = ikbo.rocs_qk_norm_rope_forward(x, pos_q=pos, rope=rope, norm="none", interleaved=inter)
    cs = rope[pos.long()][:, None]
    c, s = cs[..., :rot // 2], cs[..., rot // 2:]
    pick = (lambda t: (t[..., 0:rot:2], t[..., 1:rot:2])) if inter else (lambda t: (t[..., :rot // 2], t[..., rot // 2:rot]))
    a, b = pick(x)
    u, v = pick(y)
    assert torch.equal(u, a * c - b * s) and torch.equal(v, b * c + a * s) and torch.equal(y[..., rot:], x[..., rot:])
