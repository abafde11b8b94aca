"""The paged cache's entry points on the host: refusals before any launch, scratch sizes, and the
oracle's own bookkeeping against small cases worked by hand. No GPU needed."""

import ctypes
import os

import numpy as np
import pytest
import torch

from oracle import paged as op

FAKE = 0x7f0000000000  # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    from block_sparse_long_bigbird_gb300 import _build, _lib

    if not os.path.exists(_lib.LIB_PATH):
        _build.build()
    return _lib.lib()


def _attend(lib, **kw):
    a = dict(Q=FAKE, K=FAKE + 0x100000, V=FAKE + 0x200000, O=FAKE + 0x300000, B=1, Hq=4, Hkv=2, m=1, d=64, page=64,
             num_pages=8, max_pages=4, table=FAKE + 0x400000, lens=FAKE + 0x500000, q=None, window=64, dil=None,
             gidx=FAKE + 0x600000, ng=2, ws=FAKE + 0x700000, wsb=1 << 30, dtype=0)
    a.update(kw)
    return lib.longformer_attn_paged_fwd(a["Q"], a["K"], a["V"], a["O"], a["B"], a["Hq"], a["Hkv"], a["m"], a["d"],
                                         a["page"], a["num_pages"], a["max_pages"], a["table"], a["lens"], a["q"],
                                         a["window"], a["dil"], a["gidx"], a["ng"], a["ws"], a["wsb"], a["dtype"], None)


@pytest.mark.parametrize("bad", [
    dict(Q=None), dict(K=None), dict(V=FAKE + 8), dict(O=None), dict(O=FAKE), dict(O=FAKE + 0x100000), dict(B=0),
    dict(Hq=0), dict(Hkv=0), dict(Hq=3), dict(m=0), dict(d=96), dict(page=8), dict(page=48), dict(num_pages=0),
    dict(max_pages=0), dict(table=None), dict(lens=None), dict(table=FAKE + 0x400002), dict(window=-2),
    dict(window=63), dict(ng=-1), dict(gidx=None), dict(dtype=5), dict(q=FAKE + 1),
])
def test_attention_refuses_invalid_arguments(lib, bad):
    assert _attend(lib, **bad) == 1


@pytest.mark.parametrize("bad", [dict(B=1025), dict(Hq=130), dict(ng=513), dict(max_pages=(1 << 24) + 1),
                                 dict(num_pages=1 << 30)])
def test_attention_names_its_limits(lib, bad):
    assert _attend(lib, **bad) == 2


def _append(lib, **kw):
    a = dict(Kn=FAKE, Vn=FAKE + 0x100000, K=FAKE + 0x200000, V=FAKE + 0x300000, B=1, Hkv=2, m=1, d=64, page=64,
             num_pages=8, max_pages=4, table=FAKE + 0x400000, lens=FAKE + 0x500000, q=None, dtype=0)
    a.update(kw)
    return lib.sa_cache_append(a["Kn"], a["Vn"], a["K"], a["V"], a["B"], a["Hkv"], a["m"], a["d"], a["page"],
                               a["num_pages"], a["max_pages"], a["table"], a["lens"], a["q"], a["dtype"], None)


@pytest.mark.parametrize("bad", [
    dict(Kn=None), dict(Vn=FAKE + 4), dict(K=FAKE + 0x300000), dict(K=FAKE), dict(V=FAKE + 0x100000), dict(B=0),
    dict(Hkv=-1), dict(m=0), dict(d=32), dict(page=0), dict(page=256), dict(num_pages=-1), dict(lens=None),
    dict(dtype=9),
])
def test_append_refuses_invalid_arguments(lib, bad):
    assert _append(lib, **bad) == 1


def test_page_calls_refuse_invalid_arguments(lib):
    K, V, I, W = FAKE, FAKE + 0x1000000, FAKE + 0x2000000, FAKE + 0x3000000
    need = lib.sa_cache_workspace_bytes(64, 4)
    assert need > 0 and lib.sa_cache_workspace_bytes(0, 4) == 0 and lib.sa_cache_workspace_bytes(64, 1025) == 0
    copy = lib.sa_cache_copy_pages
    assert copy(None, V, 1, 64, 2048, I, I, 1, None) == 1
    assert copy(K, K, 1, 64, 2048, I, I, 1, None) == 1
    assert copy(K, V, 0, 64, 2048, I, I, 1, None) == 1
    assert copy(K, V, 1, 64, 2040, I, I, 1, None) == 1
    assert copy(K, V, 1, 64, 2048, None, I, 1, None) == 1
    assert copy(K, V, 1, 64, 2048, I, I, -1, None) == 1
    fork = lib.sa_cache_fork
    assert fork(K, V, 1, 64, 2048, 24, 4, 4, I, I, 1, I, I, I, I, I, I, W, need, None) == 1   # page
    assert fork(K, V, 1, 64, 2048, 16, 4, 4, I, I, 1, I, None, I, I, I, I, W, need, None) == 1
    assert fork(K, V, 1, 64, 2048, 16, 4, 4, I, I, 1, I, I, I, I, I, I, W, need - 1, None) == 1
    assert fork(K, V, 1, 64, 2048, 16, 4, 4, I, I, 1, I, I, I, I, I, I, None, need, None) == 1
    assert fork(K, V, 1, 64, 2048, 16, 1025, 4, I, I, 1, I, I, I, I, I, I, W, 1 << 30, None) == 2
    assert lib.sa_cache_free(64, 4, 4, None, 1, I, I, I, I, I, I, None) == 1
    assert lib.sa_cache_free(64, 4, 0, I, 1, I, I, I, I, I, I, None) == 1
    assert lib.sa_cache_trim(64, 16, 4, 4, -1, None, 0, I, I, I, I, I, None) == 1
    assert lib.sa_cache_trim(64, 16, 4, 4, 8, None, 3, I, I, I, I, I, None) == 1
    assert lib.sa_cache_reserve(64, 16, 4, 4, I, None, I, I, I, I, W, need, None) == 1
    assert lib.sa_cache_compact(K, V, 1, 64, 2048, 4, 4, I, I, None, I, W, need, None) == 1
    assert lib.sa_cache_compact(K, V, 1, 64, 2048, 4, 4, I, I, I, I, W, need - 4, None) == 1
    assert lib.sa_status_string(6) == b"SA_ERR_NO_PAGES"


def test_binding_refuses_before_any_device_work():
    import block_sparse_long_bigbird_gb300 as sa

    K, V = torch.zeros(4, 2, 16, 64), torch.zeros(4, 2, 16, 64)
    table, lens = torch.zeros(1, 2, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        sa.longformer_attn_paged_fwd(torch.zeros(1, 2, 1, 64), K, V, table, lens, 16)
    with pytest.raises(TypeError):
        sa.longformer_attn_paged_fwd(torch.zeros(1, 2, 1, 64).half(), K.half(), V.half(), table, lens, 16)
    with pytest.raises(ValueError):
        sa.cache_append(torch.zeros(1, 2, 1, 64), torch.zeros(1, 2, 1, 64), K, V, table, lens)
    with pytest.raises(ValueError):
        sa.cache_copy_pages(K, V, lens, lens)
    with pytest.raises(ValueError):
        sa.cache_compact(K, V, table, lens)
    with pytest.raises(ValueError):
        sa.cache_free(table, lens, torch.zeros(4, dtype=torch.int32), lens)


def test_oracle_bookkeeping_by_hand():
    table = [[0, 3, 5], [-1, -1, -1], [4, -1, -1]]
    lens, refs = [20, 0, 8], [1, 0, 0, 1, 1, 1]
    t, l, r, mv = op.fork(table, lens, refs, 8, [0], [1])
    assert t == [[0, 3, 5], [0, 3, 1], [4, -1, -1]] and l == [20, 20, 8] and r == [2, 1, 0, 2, 1, 1] and mv == [(5, 1)]
    t2, l2, r2 = op.free_rows(t, l, r, [0, 0])
    assert t2[0] == [-1] * 3 and l2 == [0, 20, 8] and r2 == [1, 1, 0, 1, 1, 0]
    t3, r3, mv3 = op.compact(t2, r2)
    assert mv3 == [(4, 2)] and t3 == [[-1] * 3, [0, 3, 1], [2, -1, -1]] and r3 == [1, 1, 1, 1, 0, 0]
    t4, r4 = op.reserve(t3, [4, 24, 9], [4, 4, 1], r3, 8)
    assert t4 == [[4, -1, -1], [0, 3, 1], [2, 5, -1]] and r4 == [1] * 6
    t5, r5 = op.trim(t4, [4, 24, 9], r4, 8, 8, (0, 1))
    assert t5 == [[4, -1, -1], [0, -1, 1], [2, 5, -1]] and r5 == [1, 1, 1, 0, 1, 1]
    assert op.trim(t4, [4, 24, 9], r4, 8, 8, (0, 24))[0] == t4  # a global token still to come sees everything


def test_oracle_attention_of_one_chunk_is_the_causal_longformer():
    from oracle import oracle_longformer

    rng = np.random.default_rng(3)
    n, d, page = 40, 64, 16
    q, k, v = (rng.standard_normal((1, 2, n, d)) for _ in range(3))
    K, V = np.zeros((3, 2, page, d)), np.zeros((3, 2, page, d))
    K, V = op.append(k, v, K, V, [[2, 0, 1]], [n], None)
    got = op.oracle_paged(q, K, V, [[2, 0, 1]], [n], None, 8, (0, 17), (0, 2))[0]
    for h, dil in enumerate((0, 2)):
        ref = oracle_longformer(torch.from_numpy(q[:, h:h + 1]), torch.from_numpy(k[:, h:h + 1]),
                                torch.from_numpy(v[:, h:h + 1]), 8, np.array([0, 17]), dilation=[dil], causal=True)
        assert np.allclose(got[:, h:h + 1], ref, atol=1e-12)
