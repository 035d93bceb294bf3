"""The history-cache entry points without a GPU: refusals of malformed arguments on the host, and the 64-bit plain forms
that the GPU tests compare with."""
import ctypes

import numpy as np
import pytest
import torch

import _history_ref as ref

FAKE = 0x100000  # aligned non-null placeholder: validation fails before any dereference
P = ctypes.byref


@pytest.fixture(scope="module")
def lib():
    from attention_ikbo_b200.build import build

    build()
    import attention_ikbo_b200 as m

    return m._history._lib()


def _norm_args(m, side=None, **kw):
    s = dict(x=FAKE, out=FAKE + (1 << 20), pos=FAKE, n=4, heads=2)
    s.update(side or {})
    a = dict(q=m.NormRopeSide(**s), dh=128, dtype=1, norm=2, eps=1e-6, rope=FAKE, max_pos=100, rot=128, workspace=FAKE,
             workspace_bytes=256)
    a.update(kw)
    return m.NormRopeArgs(**a)


def test_norm_rope_refusals(lib):
    import attention_ikbo_b200._history as m

    f = lib.rocs_qk_norm_rope_forward
    for kw, code in [({"dh": 96}, 3), ({"dh": 0}, 1), ({"dtype": 2}, 1), ({"norm": 3}, 1), ({"eps": -1.0}, 1),
                     ({"eps": float("nan")}, 1), ({"eps": float("inf")}, 1), ({"rot": 24}, 3), ({"rot": 144}, 3),
                     ({"rot": 0}, 3), ({"max_pos": 0}, 1), ({"rope": FAKE + 4}, 1), ({"workspace": None}, 6),
                     ({"workspace_bytes": 255}, 6), ({"workspace": FAKE + 16}, 6)]:
        assert f(P(_norm_args(m, **kw)), None) == code, kw
    for side, code in [({"n": -1}, 1), ({"heads": 0}, 1), ({"x": None}, 1), ({"out": None}, 1), ({"x": FAKE + 2}, 1),
                       ({"pos": None}, 1), ({"gamma": FAKE + 4}, 1), ({"beta": FAKE + 8}, 1), ({"ld_x": 128}, 1),
                       ({"ld_out": 100}, 1), ({"ld_x": 260}, 3), ({"n": 1 << 31}, 3), ({"out": FAKE + 16}, 1),
                       ({"out": FAKE, "ld_out": 264}, 1)]:
        assert f(P(_norm_args(m, side)), None) == code, side
    assert f(None, None) == 1
    # an output on the other side's input, and the two outputs on each other
    both = dict(x=FAKE + (4 << 20), out=FAKE + (5 << 20), pos=FAKE, n=4, heads=2)
    a = _norm_args(m, {"out": FAKE + (4 << 20)}, k=m.NormRopeSide(**both))
    assert f(P(a), None) == 1
    a = _norm_args(m, {"out": FAKE + (5 << 20) + 512}, k=m.NormRopeSide(**both))
    assert f(P(a), None) == 1
    # side by side in one wide buffer is fine: the check passes on to the workspace
    wide = m.NormRopeSide(x=FAKE + 512, out=FAKE + 512, pos=FAKE, n=4, heads=2, ld_x=1024, ld_out=1024)
    a = _norm_args(m, {"out": FAKE, "ld_x": 1024, "ld_out": 1024}, k=wide, workspace=None)
    assert f(P(a), None) == 6
    a = _norm_args(m, {"out": FAKE, "ld_x": 1024, "ld_out": 1024, "heads": 3}, k=wide, workspace=None)
    assert f(P(a), None) == 1
    assert lib.rocs_qk_norm_rope_workspace_size(P(_norm_args(m))) == 256
    assert lib.rocs_qk_norm_rope_workspace_size(P(_norm_args(m, dh=32))) == 0


def test_rope_table_refusals(lib):
    f = lib.rocs_rope_table
    for args, code in [((FAKE, 10, 24, 1e4), 3), ((FAKE, 10, 144, 1e4), 3), ((FAKE, -1, 64, 1e4), 1), ((FAKE, 10, 64, 1.0), 1),
                       ((FAKE, 10, 64, float("nan")), 1), ((FAKE, 10, 64, float("inf")), 1), ((None, 10, 64, 1e4), 1),
                       ((FAKE + 4, 10, 64, 1e4), 1), ((FAKE, 1 << 31, 64, 1e4), 3), ((None, 0, 64, 1e4), 0)]:
        assert f(*args, None) == code, args


def _cache_args(m, **kw):
    c = dict(k_codes=FAKE, v_codes=FAKE, k_scale=FAKE, v_scale=FAKE, pages=10, page=16, heads=2, dh=64)
    c.update(kw)
    return m.CacheQ4Args(**c)


BAD_CACHES = [({"dh": 32}, 3), ({"dh": 0}, 1), ({"page": 8}, 3), ({"page": 48}, 3), ({"page": 0}, 1), ({"heads": 0}, 1),
              ({"heads": 1 << 16}, 3), ({"pages": -1}, 1), ({"pages": 1 << 31}, 3), ({"pages": 1 << 30, "heads": 1000}, 3),
              ({"k_codes": None}, 1), ({"v_scale": None}, 1), ({"v_codes": FAKE + 8}, 1), ({"k_scale": FAKE + 4}, 1)]


def test_cache_refusals(lib):
    import attention_ikbo_b200._history as m

    def args(off=(0, 3, 5), cache=None, **kw):
        off = np.asarray(off, np.int32)
        a = dict(cache=cache or _cache_args(m), R=len(off) - 1, max_pages=4, tok_off_dev=FAKE, tok_off_host=off.ctypes.data,
                 base=FAKE, page_table=FAKE, k=FAKE, v=FAKE, dtype=1, workspace=FAKE, workspace_bytes=256)
        a.update(kw)
        x = m.CacheMoveArgs(**a)
        x.keep = off
        return x

    for f in (lib.rocs_cache_append, lib.rocs_cache_read):
        for kw, code in BAD_CACHES:
            assert f(P(args(cache=_cache_args(m, **kw))), None) == code, kw
        for kw, code in [({"off": (0, 3, 2)}, 2), ({"off": (1, 3, 5)}, 2), ({"tok_off_host": None}, 1), ({"tok_off_dev": None}, 1),
                         ({"base": None}, 1), ({"page_table": None}, 1), ({"k": None}, 1), ({"v": None}, 1),
                         ({"k": FAKE + 8}, 1), ({"base": FAKE + 2}, 1), ({"k_ld": 64}, 1), ({"v_ld": 132}, 3),
                         ({"dtype": 5}, 1), ({"R": -1}, 1), ({"max_pages": -1}, 1), ({"max_pages": 1 << 27}, 3),
                         ({"workspace": None}, 6), ({"workspace_bytes": 100}, 6)]:
            assert f(P(args(**kw)), None) == code, kw
        assert f(None, None) == 1
    assert lib.rocs_cache_read(P(args(dtype=0)), None) == 3
    for kw, code in [({"rot": 24}, 3), ({"rot": 80}, 3), ({"max_pos": 0}, 1), ({"rope": FAKE + 4}, 1)]:
        full = dict(rope=FAKE, max_pos=10, rot=64)
        full.update(kw)
        assert lib.rocs_cache_append(P(args(**full)), None) == code, kw
    assert lib.rocs_cache_workspace_size(P(args())) == 256
    assert lib.rocs_cache_workspace_size(P(args(off=(0, 3, 2)))) == 0


def test_cache_attention_refusals(lib):
    import attention_ikbo_b200._history as m

    def args(off=(0, 3, 5), cache=None, **kw):
        off = np.asarray(off, np.int32)
        a = dict(cache=cache or _cache_args(m), R=len(off) - 1, q=1, H=4, max_pages=4, scale=0.1, cand_off_dev=FAKE,
                 cand_off_host=off.ctypes.data, seq_len=FAKE, page_table=FAKE, q_ptr=FAKE, o_ptr=FAKE + (1 << 20), workspace=FAKE,
                 workspace_bytes=1 << 40)
        a.update(kw)
        x = m.DcaCacheArgs(**a)
        x.keep = off
        return x

    f, size = lib.rocs_dca_cache_forward, lib.rocs_dca_cache_workspace_size
    for kw, code in BAD_CACHES:
        a = args(cache=_cache_args(m, **kw), H=max(4, 2 * kw.get("heads", 2)))
        assert f(P(a), None) == code and size(P(a)) == 0, kw
    for kw, code in [({"off": (0, 3, 2)}, 2), ({"off": (1, 3, 5)}, 2), ({"cand_off_host": None}, 1), ({"cand_off_dev": None}, 1),
                     ({"seq_len": None}, 1), ({"page_table": None}, 1), ({"q_ptr": None}, 1), ({"o_ptr": None}, 1),
                     ({"q_ptr": FAKE + 8}, 1), ({"o_ptr": FAKE + 2}, 1), ({"lse_ptr": FAKE + 2}, 1), ({"key_limit": FAKE + 1}, 1),
                     ({"seq_len": FAKE + 2}, 1), ({"H": 5}, 1), ({"H": 0}, 1), ({"q": 0}, 1), ({"R": -1}, 1), ({"max_pages": -1}, 1),
                     ({"max_pages": 1 << 26}, 3), ({"q": 1 << 20}, 3), ({"H": 1 << 16}, 3), ({"q": 1 << 19, "H": 1 << 15}, 3),
                     ({"scale": -1.0}, 1), ({"scale": float("nan")}, 1), ({"scale": float("inf")}, 1), ({"q_ld": 64}, 1),
                     ({"q_ld": 260}, 3), ({"q_ld": 1 << 31}, 3), ({"o_ptr": FAKE}, 1), ({"o_ptr": FAKE + 2032}, 1),
                     ({"lse_ptr": FAKE + 64}, 1), ({"lse_ptr": FAKE + (1 << 20) + 2044}, 1),
                     ({"q_ld": 1 << 18, "o_ptr": FAKE + 1024}, 1)]:
        assert f(P(args(**kw)), None) == code, kw
        assert size(P(args(**kw))) == 0, kw
    need = size(P(args()))
    assert need > 256 and need % 256 == 0
    for kw in ({"workspace": None}, {"workspace_bytes": need - 1}, {"workspace": FAKE + 16}):
        assert f(P(args(**kw)), None) == 6, kw
    assert f(None, None) == 1
    # nothing to compute: pointers are not needed
    assert size(P(args(off=(0, 0), q_ptr=None, o_ptr=None, seq_len=None, page_table=None))) == 256


def test_packed_arguments_match_the_structures():
    import attention_ikbo_b200._history as m

    for pack, args in ((m._PACK_NORM, m.NormRopeArgs), (m._PACK_MOVE, m.CacheMoveArgs), (m._PACK_DCA, m.DcaCacheArgs)):
        assert pack.size == ctypes.sizeof(args)
        # every field at its place: distinct numbers through both forms
        flat = []

        def walk(t, at):
            for name, kind in t._fields_:
                off = at + getattr(t, name).offset
                if issubclass(kind, ctypes.Structure):
                    walk(kind, off)
                else:
                    flat.append((off, kind))
        walk(args, 0)
        data = bytearray(pack.pack(*range(1, len(flat) + 1)))
        assert [kind.from_buffer(data, off).value for off, kind in flat] == list(range(1, len(flat) + 1))


def test_binding_refuses_host_tensors():
    import attention_ikbo_b200 as m

    x = torch.zeros(2, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(m.RocsError):
        m.rocs_qk_norm_rope_forward(x)
    with pytest.raises(m.RocsError):
        m.rocs_qk_norm_rope_forward(None, None)
    with pytest.raises(m.RocsError):
        m.rocs_qk_norm_rope_forward(x.half())


def test_reference_format_round_trip():
    g = torch.Generator().manual_seed(0)
    c = torch.randint(0, 16, (5, 3, 128), generator=g)
    assert torch.equal(ref.codes_of(ref.pack(c)), c)
    # channel 1 of a word is nibble 0 of its high half, channel 2 nibble 1 of its low half
    one = torch.zeros(8, dtype=torch.long)
    one[1], one[2] = 5, 9
    assert ref.pack(one).tolist() == [0x90, 0, 5, 0]
    x = torch.randn(40, 64, generator=g).double()
    codes, step, mn = ref.quantise(x)
    err = (mn[:, None] + step[:, None] * codes - x).abs()
    # half a step, and what the rounded step (15 codes of it) and minimum lose
    assert torch.all(err <= step[:, None] / 2 + 15 * 2.0 ** -8 * step[:, None] + 2.0 ** -8 * mn.abs()[:, None])
    assert codes.min() == 0 and codes.max() == 15


def test_reference_rotation_keeps_angles():
    """Scores of rotated pairs depend on the distance of their positions only."""
    g = torch.Generator().manual_seed(1)
    q, k = torch.randn(1, 1, 64, generator=g).double(), torch.randn(1, 1, 64, generator=g).double()
    a = torch.from_numpy(ref.rope_angles(60, 64))
    cs = torch.cat((a.cos(), a.sin()), 1)
    for inter in (False, True):
        def score(i, j):
            return float((ref.rotate(q, cs[i:i + 1], 64, inter) * ref.rotate(k, cs[j:j + 1], 64, inter)).sum())
        assert abs(score(7, 3) - score(47, 43)) < 1e-9
        assert abs(score(7, 3) - score(8, 3)) > 1e-6
