"""The paged cache on the GPU where it could go wrong: calls that need no plan, lists and lengths that break
the contract, rows computed again by the definition, long walks that few tiles hold."""

import numpy as np
import pytest
import torch

import block_sparse_long_bigbird_gb300 as sa
from block_sparse_long_bigbird_gb300 import _lib
from block_sparse_long_bigbird_gb300.inputs import make_grad_out, make_qkv
from oracle import paged as op
from paged_util import attend_and_check, dev, f64, ints, make_cache

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ chunks that need no plan
def _dense_calls():
    """Dense forward and backward kernels, whose shared memory and TMEM the next kernel finds as they left it."""
    q, k, v = (t.cuda() for t in make_qkv(1, 2, 512, 64, "bf16", cfg_id=90))
    do = make_grad_out(1, 2, 512, 64, "bf16", cfg_id=90).cuda()
    table = sa.build_bigbird_pattern(0, 2, 512, 64, 2, 3, 3).cuda()
    for _ in range(3):
        sa.bigbird_attn_fwd(q, k, v, 64, 2, 3, 3, table)
        sa.longformer_attn_fwd(q, k, v, 128, None, causal=True)
        sa.bigbird_attn_bwd(q, k, v, do, 64, 2, 3, 3, table)


@pytest.mark.parametrize("d", [64, 128])
# of one tile and of two; several to a CTA, and fewer than there are CTAs
@pytest.mark.parametrize("B,Hq,Hkv,m", [(8, 20, 20, 48), (8, 20, 20, 150), (3, 8, 2, 40), (1, 4, 4, 260)])
def test_chunks_with_a_plain_window_right_after_dense_calls(B, Hq, Hkv, m, d):
    lens = [m + (23 * i) % 60 for i in range(B)]
    Q, K, V, table = make_cache(81 + m, B, Hq, Hkv, m, d, 64, lens)
    _dense_calls()
    first = attend_and_check(Q, K, V, table, lens, None, 64)
    assert _lib.lib().sa_last_launch_count() == 1  # no plan, nothing to join
    args = dev(Q, K, V, table, ints(lens))
    for _ in range(4):
        _dense_calls()
        assert torch.equal(sa.longformer_attn_paged_fwd(*args, 64), first)
    assert sa.get_last_device_status() == 0


# ------------------------------------------------------------------ lists that break the contract
def _counted(g):
    """The entries of a list that count: in range and above every one that counts before them."""
    kept = []
    for v in g:
        if 0 <= v < 2 ** 30 and (not kept or v > kept[-1]):
            kept.append(v)
    return kept


LISTS = [[1000, 1100, 5, 6, 64, 128], [200, 264, 10, 20, 70], [7, 7], [5, -3, 4, 300], [2 ** 30, 7, 8],
         [-1], list(range(60, 0, -1)) + list(range(100, 170)), [65 * i % 400 for i in range(100)]]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("m,Hq", [(1, 2), (3, 8), (40, 2), (40, 4), (150, 4)])
def test_global_lists_out_of_order_or_range(m, Hq, dtype):
    lens = [400, 300]
    Q, K, V, table = make_cache(91, 2, Hq, 2, m, 64, 16, lens, dtype)
    args = dev(Q, K, V, table, ints(lens))
    for g in LISTS:
        want = attend_and_check(Q, K, V, table, lens, None, 64, _counted(g), None, dtype)
        got = sa.longformer_attn_paged_fwd(*args, 64, ints(g).cuda())
        assert sa.get_last_device_status() == _lib.SA_ERR_BAD_INDEX
        torch.testing.assert_close(got, want, rtol=2.0 ** -6 if dtype == "bf16" else 2e-5, atol=2.0 ** -7 if dtype == "bf16" else 2e-6)


@pytest.mark.parametrize("m,Hq", [(1, 2), (3, 8), (40, 2), (150, 4)])
def test_dilations_out_of_range_count_as_none(m, Hq):
    lens = [400, 300]
    Q, K, V, table = make_cache(92, 2, Hq, 2, m, 64, 32, lens)
    for bad in (64, -1, 2 ** 31 - 1):
        dil = [2] * Hq
        want = attend_and_check(Q, K, V, table, lens, None, 64, [3], dil[:-1] + [0])
        got = sa.longformer_attn_paged_fwd(*dev(Q, K, V, table, ints(lens)), 64, ints([3]).cuda(),
                                           dilation=ints(dil[:-1] + [bad]).cuda())
        assert sa.get_last_device_status() == _lib.SA_ERR_BAD_INDEX
        assert torch.equal(got, want)


# ------------------------------------------------------------------ bookkeeping of values that break the contract
def _book():
    """A table [4, 6] of pages of 16 tokens over 30 pages; the third row is empty."""
    table = np.full((4, 6), -1, np.int32)
    table[0], table[1, :4], table[3, :2] = [7, 3, 20, 1, 9, 28], [5, 6, 29, 0], [11, 12]
    refs = np.zeros(30, np.int32)
    np.add.at(refs, table[table >= 0], 1)
    return table, [96, 50, 0, 30], refs


@pytest.mark.parametrize("in_place", [False, True])
def test_trim_keeps_the_pages_of_rows_and_lists_that_break_the_contract(in_place):
    table, lens, refs = _book()
    for row, n in ((0, 97), (1, -5), (1, 10 ** 6), (3, 2 ** 31 - 1)):
        T, R = dev(*map(torch.from_numpy, (table, refs)))
        bad = lens[:row] + [n] + lens[row + 1:]
        got = sa.cache_trim(T, ints(bad).cuda(), R, 16, 8, ints([1]).cuda(), out=(T, R) if in_place else None)
        assert sa.get_last_device_status() == _lib.SA_ERR_BAD_INDEX
        held = lens[:row] + [0] + lens[row + 1:]  # a sequence without tokens gives up nothing
        assert [x.tolist() for x in got] == list(op.trim(table, held, refs, 16, 8, [1]))
    for g in ([3, 2], [40, 40], [-1, 5], [1, 70, 20]):
        T, R = dev(*map(torch.from_numpy, (table, refs)))
        got = sa.cache_trim(T, ints(lens).cuda(), R, 16, 8, ints(g).cuda(), out=(T, R) if in_place else None)
        assert sa.get_last_device_status() == _lib.SA_ERR_BAD_INDEX
        assert got[0].tolist() == table.tolist() and got[1].tolist() == refs.tolist()


@pytest.mark.parametrize("in_place", [False, True])
def test_table_entries_that_name_no_page_are_latched(in_place):
    """Entries outside [-1, 30) count as none in every call that uses them."""
    table, lens, refs = _book()

    def call(f, bad, *more):
        T, R = dev(*map(torch.from_numpy, (bad, refs)))
        L = ints(lens).cuda()
        out = {"out": (T, L, R) if f in (sa.cache_fork, sa.cache_free) else (T, R)} if in_place else {}
        if f is sa.cache_fork or f is sa.cache_compact:
            K, V = (torch.arange(30, dtype=torch.float32, device="cuda").view(30, 1, 1, 1).expand(30, 1, 16, 64).contiguous()
                    for _ in range(2))
            got = f(K, V, T, L, R, *more, **out) if f is sa.cache_fork else f(K, V, T, R, **out)
        elif f is sa.cache_free:
            got = f(T, L, R, *more, **out)
        elif f is sa.cache_trim:
            got = f(T, L, R, *more, **out)
        else:
            got = f(T, L, more[0], R, *more[1:], **out)
        return [x.tolist() for x in got], sa.get_last_device_status()

    src, dst, row1 = ints([1]).cuda(), ints([2]).cuda(), ints([1]).cuda()
    for v in (-2, 30, -2 ** 31, 2 ** 31 - 1):
        # a page of the middle, the partial last one, and one past the length
        for col, calls in ((1, ((sa.cache_fork, (src, dst)), (sa.cache_free, (row1,)), (sa.cache_trim, (16, 8)), (sa.cache_compact, ()))),
                           (3, ((sa.cache_fork, (src, dst)), (sa.cache_free, (row1,)), (sa.cache_compact, ()))),
                           (2, ((sa.cache_reserve, (ints([0, 20, 0, 0]).cuda(), 16)),))):
            bad, none = table.copy(), table.copy()
            bad[1, col], none[1, col] = v, -1
            for f, more in calls:
                want, ok = call(f, none, *more)
                assert ok == 0
                got, status = call(f, bad, *more)
                assert status == _lib.SA_ERR_BAD_INDEX, (f.__name__, v, col)
                if got[0][1][col] == v:  # a call that leaves the row as it is leaves the entry too
                    got[0][1][col] = -1
                assert got == want, (f.__name__, v, col)


@pytest.mark.parametrize("in_place", [False, True])
def test_compact_does_not_follow_entries_of_free_pages(in_place):
    """An entry whose page has the count 0 would name another sequence's page after the move: it becomes -1."""
    table, lens, refs = _book()
    table[1, 0], table[3, 1] = 2, 25  # free: below and past the pages in use
    refs = np.zeros(30, np.int32)
    np.add.at(refs, table[table >= 0], 1)
    refs[2] = refs[25] = 0
    want = table.copy()
    want[1, 0] = want[3, 1] = -1
    wt, wr, moves = op.compact(want, refs)
    K = torch.arange(30, dtype=torch.float32, device="cuda").view(30, 1, 1, 1).expand(30, 1, 16, 64).contiguous()
    V = K + 100
    T, R = dev(*map(torch.from_numpy, (table, refs)))
    t, r = sa.cache_compact(K, V, T, R, out=(T, R) if in_place else None)
    assert sa.get_last_device_status() == _lib.SA_ERR_BAD_INDEX
    assert t.tolist() == wt and r.tolist() == wr
    for a, b in moves:
        assert float(K[b].min()) == float(K[b].max()) == a and float(V[b].min()) == 100 + a
    negative = refs.copy()
    negative[2] = -1  # a count below 0 is no count: the page is free
    T, R = dev(*map(torch.from_numpy, (want, negative)))
    t, r = sa.cache_compact(K, V, T, R)
    assert sa.get_last_device_status() == _lib.SA_ERR_BAD_INDEX and t.tolist() == wt and r.tolist() == wr


# ------------------------------------------------------------------ rows computed again by the definition
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("m,H,G", [(300, 110, 1), (60, 160, 1), (64, 40, 4)])
def test_an_infinity_that_every_row_sees_of_a_long_history(m, H, G, d):
    """Every row of every unit is computed again, several units to a CTA, and no wait runs out over it."""
    n = 16000
    gen = torch.Generator(device="cuda").manual_seed(5)
    K, V = (torch.randn(n // 128, H, 128, d, generator=gen, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    Q = torch.randn(1, H * G, m, d, generator=gen, device="cuda", dtype=torch.bfloat16)
    T, L = torch.arange(n // 128, dtype=torch.int32, device="cuda")[None].contiguous(), ints([n]).cuda()
    clean = sa.longformer_attn_paged_fwd(Q, K, V, T, L, 2 * n)
    V[0, :, 0, 7] = float("inf")
    torch.cuda.synchronize()
    sa.set_option(sa.SA_OPT_WAIT_LIMIT, 10_000)  # a unit's rows take longer than these 10 ms, its waits microseconds
    try:
        got = sa.longformer_attn_paged_fwd(Q, K, V, T, L, 2 * n)
        torch.cuda.synchronize()
    finally:
        sa.set_option(sa.SA_OPT_WAIT_LIMIT, 0)
    assert sa.get_last_device_status() == 0
    assert bool(torch.isposinf(got[..., 7]).all())
    got[..., 7] = clean[..., 7]
    # the weights' rounding of one (2^-8 of a mean of |v| < 2 over 16000 keys), the results' of both
    torch.testing.assert_close(got.float(), clean.float(), rtol=2.0 ** -7, atol=2.0 ** -7)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("m,Hq,Hkv,dtype", [(40, 2, 2, "bf16"), (150, 2, 2, "bf16"), (50, 16, 2, "bf16"), (20, 2, 2, "fp32"), (5, 16, 2, "fp32"),
                                            (150, 2, 2, "simt")])
def test_rows_taken_again_in_split_tiles(m, Hq, Hkv, dtype, d):
    """Infinities and NaN in the last token, which only its own rows see, in tiles cut into many pieces; and
    an infinite key that some rows' windows hold."""
    lens, simt, dtype = [4000, 77 + m], dtype == "simt", dtype.replace("simt", "bf16")
    sa.set_option(sa.SA_OPT_FORCE_SIMT, int(simt))
    try:
        Q, K, V, table = make_cache(96, 2, Hq, Hkv, m, d, 16, lens, dtype)
        clean = f64(attend_and_check(Q, K, V, table, lens, None, 9000, None, None, dtype))
        Vc = V.clone()
        for b, n in enumerate(lens):
            Vc[int(table[b, (n - 1) // 16]), :, (n - 1) % 16, 0] = float("inf")
            Vc[int(table[b, (n - 1) // 16]), :, (n - 1) % 16, 1] = float("nan")
        got = f64(sa.longformer_attn_paged_fwd(*dev(Q, K, Vc, table, ints(lens)), 9000))
        assert np.isposinf(got[:, :, -1, 0]).all() and np.isnan(got[:, :, -1, 1]).all()
        got[:, :, -1, :2] = clean[:, :, -1, :2]
        # bf16: the weights' rounding of one (2^-8 of a mean of |v| < 4), the results' of both; fp32: sums in another order
        assert np.allclose(got, clean, rtol=2.0 ** -7 if dtype == "bf16" else 2e-5, atol=2.0 ** -6 if dtype == "bf16" else 2e-6)
        Kc = K.clone()  # one row's q k is infinite or NaN where the window holds the key: all of that row is NaN
        at = lens[0] - m // 2 - 20
        Kc[int(table[0, at // 16]), :, at % 16, 3] = float("inf")
        want = f64(attend_and_check(Q, K, V, table, lens, None, 40, None, None, dtype))
        got = f64(sa.longformer_attn_paged_fwd(*dev(Q, Kc, V, table, ints(lens)), 40))
        seen = np.array([at <= lens[0] - m + t <= at + 20 for t in range(m)])
        q3 = f64(Q)[0, :, :, 3]
        nan = seen[None] & (q3 >= 0)  # +inf or NaN; a score of -inf is a weight of 0
        assert np.isnan(got[0][nan]).all() and np.isfinite(got[0][~nan]).all() and np.isfinite(got[1]).all()
        same = ~seen
        assert np.allclose(got[0][:, same], want[0][:, same], rtol=2.0 ** -7 if dtype == "bf16" else 2e-5,
                           atol=2.0 ** -6 if dtype == "bf16" else 2e-6)
    finally:
        sa.set_option(sa.SA_OPT_FORCE_SIMT, 0)
    assert sa.get_last_device_status() == 0


# ------------------------------------------------------------------ long walks that few tiles hold
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("m,Hq", [(1, 2), (3, 2), (40, 2), (150, 2)])
def test_a_global_token_of_a_long_sequence_is_shared_out(m, Hq, dtype):
    """One token among the new ones is global: its tile walks all keys, which no single CTA should do alone."""
    lens, g = [30000, 200], [0, 29999 - m // 2]
    Q, K, V, table = make_cache(95, 2, Hq, 2, m, 64, 64, lens, dtype)
    attend_and_check(Q, K, V, table, lens, None, 256, g, None, dtype)
    assert _lib.lib().sa_last_launch_count() == 2  # the sweeps, and the join of their pieces
    attend_and_check(Q, K, V, table, lens, None, 256, list(range(0, 29000, 64))[:400], None, dtype)  # a block each
