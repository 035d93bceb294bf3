"""Calls of the history cache whose outputs overlap what they read or write elsewhere are refused on the host (no GPU)."""
import ctypes

import numpy as np
import pytest

FAKE = 0x10000000  # aligned placeholders far apart: every call here is refused before anything is launched
MB = 1 << 20
P = ctypes.byref


@pytest.fixture(scope="module")
def hist():
    from attention_ikbo_b200.build import build

    build()
    import attention_ikbo_b200 as m

    m._history._lib()
    return m._history


def _cache(m, **kw):
    c = dict(k_codes=FAKE, v_codes=FAKE + MB, k_scale=FAKE + 2 * MB, v_scale=FAKE + 3 * MB, pages=10, page=16, heads=2, dh=64)
    c.update(kw)
    return m.CacheQ4Args(**c)


def _move(m, cache=None, **kw):
    off = np.array([0, 3, 5], np.int32)
    a = dict(cache=cache or _cache(m), R=2, max_pages=4, tok_off_dev=FAKE + 8 * MB, tok_off_host=off.ctypes.data, base=FAKE + 9 * MB,
             page_table=FAKE + 10 * MB, k=FAKE + 4 * MB, v=FAKE + 5 * MB, dtype=1, workspace=FAKE + 11 * MB, workspace_bytes=256)
    a.update(kw)
    x = m.CacheMoveArgs(**a)
    x.keep = off
    return x


CODES, SCALE = 10 * 2 * 16 * 32, 10 * 2 * 16 * 4  # bytes of one buffer of the cache
ROWS = 5 * 2 * 64 * 2                             # bytes of k or v

INTO_CACHE = [{"k": FAKE}, {"v": FAKE + CODES - 16}, {"k": FAKE + MB - ROWS + 16}, {"v": FAKE + 2 * MB + 16},
              {"k": FAKE + 3 * MB + SCALE - 16}, {"v": FAKE + 4096, "v_ld": 1024}]


def test_read_and_append_refuse_rows_in_the_cache(hist):
    lib = hist._lib()
    for f in (lib.rocs_cache_read, lib.rocs_cache_append):
        for kw in INTO_CACHE:
            assert f(P(_move(hist, **kw)), None) == 1, kw


def test_read_refuses_outputs_over_each_other(hist):
    f, k = hist._lib().rocs_cache_read, FAKE + 4 * MB
    for kw in ({"v": k}, {"v": k + 16}, {"v": k + ROWS - 16}, {"v": k - ROWS + 16}, {"v": k + 128, "k_ld": 256, "v_ld": 256},
               {"v": k + 256, "k_ld": 256, "v_ld": 264}, {"v": k + 384, "k_ld": 192, "v_ld": 192}):
        assert f(P(_move(hist, **kw)), None) == 1, kw


def test_append_refuses_buffers_over_each_other(hist):
    f = hist._lib().rocs_cache_append
    for kw in ({"v_codes": FAKE}, {"v_codes": FAKE + CODES - 16}, {"v_scale": FAKE + 2 * MB}, {"k_scale": FAKE + MB + 32},
               {"v_scale": FAKE + 2 * MB + SCALE - 16}):
        assert f(P(_move(hist, cache=_cache(hist, **kw))), None) == 1, kw


def test_attention_refuses_outputs_in_the_cache(hist):
    lib, off = hist._lib(), np.array([0, 3, 5], np.int32)
    for kw in ({"o_ptr": FAKE}, {"o_ptr": FAKE + MB + CODES - 16}, {"lse_ptr": FAKE + 2 * MB + 4}, {"lse_ptr": FAKE + 3 * MB + SCALE - 4},
               {"o_ptr": FAKE + 2 * MB - 16}):
        a = dict(cache=_cache(hist), R=2, q=1, H=4, max_pages=4, scale=0.1, cand_off_dev=FAKE + 8 * MB, cand_off_host=off.ctypes.data,
                 seq_len=FAKE + 9 * MB, page_table=FAKE + 10 * MB, q_ptr=FAKE + 4 * MB, o_ptr=FAKE + 5 * MB, workspace=FAKE + 32 * MB,
                 workspace_bytes=1 << 40)
        a.update(kw)
        x = hist.DcaCacheArgs(**a)
        assert lib.rocs_dca_cache_workspace_size(P(x)) == 0 and lib.rocs_dca_cache_forward(P(x), None) == 1, kw
