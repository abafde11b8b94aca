"""The paged cache on the GPU: attention of new tokens against the float64 oracle, appending, and the
pages' bookkeeping against plain Python, alone and together as a serving loop uses them."""

import numpy as np
import pytest
import torch

import block_sparse_long_bigbird_gb300 as sa
from block_sparse_long_bigbird_gb300 import _lib
from oracle import paged as op
from paged_util import attend_and_check, dev, f64, ints, make_cache

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ attention against the oracle
# B, Hq, Hkv, m, d, page, lens, q_lens, window, globals, dilation
CASES = {
    "one key": (1, 1, 1, 1, 64, 16, [1], None, 0, None, None),
    "one token, window": (2, 3, 3, 1, 64, 64, [700, 65], None, 512, None, None),
    "one token, full, pages of 16": (2, 2, 2, 1, 128, 16, [333, 16], None, 2000, None, None),
    "one token, globals": (2, 2, 2, 1, 64, 32, [600, 129], None, 64, [0, 1, 63, 64, 300, 599], None),
    "one token, global itself": (1, 2, 2, 1, 64, 64, [301], None, 16, [300], None),
    "one token, dilated": (2, 4, 4, 1, 64, 16, [500, 77], None, 128, None, [0, 1, 3, 63]),
    "one token, dilated group and globals": (1, 4, 2, 1, 128, 32, [450], None, 64, [5, 200], [0, 3, 2, 0]),
    "one token, group of 3": (2, 6, 2, 1, 128, 64, [200, 321], None, 1000, None, None),
    "one token, group of 8": (2, 16, 2, 1, 128, 128, [300, 1], None, 1000, None, None),
    "no tokens and none new": (3, 2, 2, 3, 64, 16, [40, 0, 9], [3, 0, 0], 20, None, None),
    "drafted, ragged": (4, 8, 2, 5, 128, 32, [100, 64, 5, 333], [5, 1, 5, 0], 2000, None, None),
    "drafted, window 0": (2, 4, 4, 3, 64, 16, [50, 3], [3, 3], 0, None, None),
    "chunk, whole sequence": (1, 2, 2, 200, 64, 64, [200], None, 64, None, None),
    "chunk, window and globals": (2, 4, 2, 130, 64, 16, [400, 131], [130, 77], 100, [0, 3, 64, 290, 350], None),
    "chunk, dilated": (1, 4, 4, 150, 64, 64, [420], None, 32, None, [0, 1, 2, 7]),
    "chunk, dilated group": (1, 4, 2, 90, 128, 32, [300], None, 48, [7], [0, 5, 1, 1]),
    "chunk, full, d 128": (2, 4, 1, 100, 128, 128, [260, 100], [100, 33], 4000, None, None),
    "chunk, group of 5": (1, 10, 2, 60, 64, 64, [222], None, 80, [1], None),
    "chunk, group of 64": (1, 64, 1, 3, 64, 64, [70], None, 80, None, None),
    "chunk over 257 rows": (1, 1, 1, 300, 64, 64, [300], [257], 1000, None, None),
}


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("name", CASES)
def test_attention_matches_the_oracle(name, dtype):
    B, Hq, Hkv, m, d, page, lens, q, window, g, dil = CASES[name]
    Q, K, V, table = make_cache(len(name), B, Hq, Hkv, m, d, page, lens, dtype)
    attend_and_check(Q, K, V, table, lens, q, window, g, dil, dtype)


@pytest.mark.parametrize("name", ["drafted, ragged", "chunk, window and globals", "chunk, dilated group",
                                  "chunk, full, d 128", "chunk, group of 64"])
def test_attention_on_the_ordinary_units(name):
    B, Hq, Hkv, m, d, page, lens, q, window, g, dil = CASES[name]
    Q, K, V, table = make_cache(5, B, Hq, Hkv, m, d, page, lens)
    sa.set_option(sa.SA_OPT_FORCE_SIMT, 1)
    try:
        attend_and_check(Q, K, V, table, lens, q, window, g, dil)
    finally:
        sa.set_option(sa.SA_OPT_FORCE_SIMT, 0)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("m,Hq,Hkv", [(1, 2, 2), (1, 4, 2), (1, 8, 2), (4, 2, 2), (40, 4, 2), (1, 32, 2)])
def test_long_sweeps_are_split_and_joined(m, Hq, Hkv, dtype):
    lens = [3001, 1700, m]
    Q, K, V, table = make_cache(9, 3, Hq, Hkv, m, 64, 64, lens, dtype, sigma=2.0)
    attend_and_check(Q, K, V, table, lens, None, 8000, None, None, dtype)


# B, Hkv: few tiles (large CTAs) and many (small ones)
@pytest.mark.parametrize("B,Hkv", [(2, 1), (110, 3)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("m,group", [(1, 2), (7, 1), (2, 4), (1, 9), (4, 4), (1, 17), (23, 1), (3, 8), (5, 5)])
def test_few_rows_per_key_head(m, group, d, B, Hkv):
    """2 to 8 rows: weights as the sum of two bf16 numbers; 9 to 24: bf16 weights; one more goes to the 128-row tiles."""
    lens = [max(m, (37 * i + 5) % 190) for i in range(B)]
    lens[0], lens[1] = 190, m
    q = None if m == 1 else [m] + [i % (m + 1) for i in range(1, B)]
    Q, K, V, table = make_cache(m + group + d, B, Hkv * group, Hkv, m, d, 32, lens, sigma=1.5)
    attend_and_check(Q, K, V, table, lens, q, 128, [0, 1, 70], None, weights=2.0 ** -8 if m * group > 8 else 2.0 ** -16)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("m,Hq,Hkv", [(1, 2, 2), (5, 4, 2), (3, 16, 2), (70, 4, 2)])
def test_tables_wider_than_the_sequences(m, Hq, Hkv, dtype):
    """Room for long sequences, but short ones (whole tiles in turn), then one long among short and empty ones."""
    for lens, q in (([100, m, 77], None), ([5000, 0, m, 333, 40], [m, 0, m, 0, m // 2])):
        lens = [max(n, 0 if q is None else k) for n, k in zip(lens, q or lens)]
        Q, K, V, table = make_cache(15, len(lens), Hq, Hkv, m, 64, 64, lens, dtype, width=700)
        attend_and_check(Q, K, V, table, lens, q, 20000, None, None, dtype)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group", [1, 4, 12])
def test_values_beyond_the_largest_number_in_a_split_sweep(group, d):
    """A row that sees an infinity or NaN has it; rows of the same tile that do not see it are as without it."""
    lens, m = [4000], 2
    Q, K, V, table = make_cache(51, 1, group, 1, m, d, 16, lens)
    clean = attend_and_check(Q, K, V, table, lens, None, 9000)
    Vc = V.clone()
    last = lens[0] - 1
    Vc[int(table[0, last // 16]), 0, last % 16, 0] = float("inf")
    Vc[int(table[0, last // 16]), 0, last % 16, 1] = float("nan")
    got = sa.longformer_attn_paged_fwd(*dev(Q, K, Vc, table, ints(lens)), 9000)
    a, b = f64(got), f64(clean)
    assert np.isposinf(a[:, :, 1, 0]).all() and np.isnan(a[:, :, 1, 1]).all()
    # summed again by the definition: the weights' rounding of one (2^-8 of a mean of |v| < 2), the results' of both
    assert np.allclose(a[:, :, 0], b[:, :, 0], rtol=2.0 ** -7, atol=2.0 ** -7)
    assert np.allclose(a[:, :, 1, 2:], b[:, :, 1, 2:], rtol=2.0 ** -7, atol=2.0 ** -7)
    assert sa.get_last_device_status() == 0


@pytest.mark.parametrize("m,group,d", [(2, 1, 64), (2, 2, 128), (2, 10, 64), (40, 1, 64)])
def test_infinities_in_some_of_many_tiles(m, group, d):
    """CTAs that compute rows again between units that need none of that."""
    B, Hkv = 120, 3
    lens = [m + (29 * i) % 90 for i in range(B)]
    Q, K, V, table = make_cache(52, B, Hkv * group, Hkv, m, d, 16, lens)
    clean = attend_and_check(Q, K, V, table, lens, None, 300)
    Vc = V.clone()
    for b in range(0, B, 2):
        last = lens[b] - 1
        Vc[int(table[b, last // 16]), :, last % 16, 5] = float("-inf")
    got = sa.longformer_attn_paged_fwd(*dev(Q, K, Vc, table, ints(lens)), 300)
    assert torch.equal(got[1::2], clean[1::2])
    a, b = f64(got[::2]), f64(clean[::2])
    assert np.isneginf(a[:, :, -1, 5]).all()
    a[:, :, -1, 5] = b[:, :, -1, 5]
    # the weights' rounding of one (2^-8 of a mean of |v| < 4), the results' of both
    assert np.allclose(a, b, rtol=2.0 ** -7, atol=2.0 ** -6)
    assert sa.get_last_device_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("m", [1, 3, 70])
def test_missing_pages_and_empty_rows(m, dtype):
    # whole stretches without pages: rows that see nothing are zeros
    lens = [200, 130]
    Q, K, V, table = make_cache(21, 2, 4, 2, m, 64, 16, lens, dtype)
    table[0, 0:10] = -1
    table[1, :] = -1
    O = attend_and_check(Q, K, V, table, lens, None, 40, [2, 50], None, dtype)
    assert (O[1] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("m,Hq", [(1, 2), (2, 2), (60, 2), (60, 8), (1, 16)])
def test_what_a_row_does_not_see_does_not_reach_it(m, Hq, dtype):
    # NaN and infinities at keys outside the rows' windows, and in later tokens of the same chunk
    lens = [260]
    Q, K, V, table = make_cache(33, 1, Hq, 2, m, 64, 32, lens, dtype)
    Kc, Vc = K.clone(), V.clone()

    def put(pos, k, v):
        Kc[int(table[0, pos // 32]), :, pos % 32] = k
        Vc[int(table[0, pos // 32]), :, pos % 32] = v

    first = 260 - m
    put(first - 45, float("nan"), float("inf"))      # before every window (half 40)
    put(first - 60, float("-inf"), float("nan"))
    put(259, float("inf"), float("nan"))             # only the last token sees it
    args = dev(table, ints(lens))
    run = lambda k, v: sa.longformer_attn_paged_fwd(Q.cuda(), k.cuda(), v.cuda(), *args, 80)  # noqa: E731
    want, got = run(K, V), run(Kc, Vc)
    # rows are summed again by the definition, in another order: equal up to the rounding of the result
    a, b = f64(got[:, :, :m - 1]), f64(want[:, :, :m - 1])
    assert np.isfinite(a).all() and np.allclose(a, b, rtol=2.0 ** -6 if dtype == "bf16" else 2e-5,
                                                atol=2.0 ** -7 if dtype == "bf16" else 2e-6)
    assert np.isnan(f64(got[:, :, m - 1])).all()
    assert sa.get_last_device_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("m,Hq,dil", [(1, 2, None), (70, 2, None), (70, 4, [0, 3, 1, 0])])
def test_many_far_globals(m, Hq, dil, dtype):
    """More global keys before the window than one step takes, some without a page, some later than the sequence."""
    lens = [2000, 700]
    g = sorted(set(range(0, 40)) | set(range(50, 1900, 13)) | {1975, 2600})
    Q, K, V, table = make_cache(71, 2, Hq, 2, m, 64, 16, lens, dtype)
    table[0, 20:30] = -1
    attend_and_check(Q, K, V, table, lens, None, 64, g, dil, dtype)
    # an infinite value at a far global key: every row has it, computed by the definition
    Vc = V.clone()
    Vc[int(table[1, 0]), :, 3, 0] = float("inf")
    got = f64(sa.longformer_attn_paged_fwd(*dev(Q, K, Vc, table, ints(lens)), 64, ints(g).cuda(), dilation=dev(ints(dil))[0]))
    assert np.isposinf(got[1, :, :, 0]).all() and np.isfinite(got[1, :, :, 1:]).all() and np.isfinite(got[0]).all()
    assert sa.get_last_device_status() == 0


def test_bad_lengths_and_pages_are_zeroed_and_latched():
    lens = [64, 100, 30]
    Q, K, V, table = make_cache(2, 3, 4, 2, 2, 64, 16, lens, width=7)
    Qd, Kd, Vd, T = dev(Q, K, V, table)
    ref = sa.longformer_attn_paged_fwd(Qd, Kd, Vd, T, ints(lens).cuda(), 40)
    assert sa.get_last_device_status() == 0
    for bad in ([64, 1000, 30], [64, -5, 30], [64, 1, 30]):  # past its table row, negative, fewer than the new ones
        O = sa.longformer_attn_paged_fwd(Qd, Kd, Vd, T, ints(bad).cuda(), 40)
        assert sa.get_last_device_status() == _lib.SA_ERR_BAD_INDEX
        assert (O[1] == 0).all() and torch.equal(O[0], ref[0]) and torch.equal(O[2], ref[2])
    T2 = T.clone()
    T2[0, 3] = 10 ** 6  # a page that does not exist counts as missing
    O = sa.longformer_attn_paged_fwd(Qd, Kd, Vd, T2, ints(lens).cuda(), 40)
    assert sa.get_last_device_status() == _lib.SA_ERR_BAD_INDEX
    T3 = table.clone()
    T3[0, 3] = -1
    assert torch.equal(O, sa.longformer_attn_paged_fwd(Qd, Kd, Vd, T3.cuda(), ints(lens).cuda(), 40))
    assert sa.get_last_device_status() == 0


@pytest.mark.parametrize("m,Hq", [(1, 2), (1, 16), (130, 4)])
def test_deterministic_and_independent_of_the_stream(m, Hq):
    lens = [900, 2500]
    Q, K, V, table = make_cache(4, 2, Hq, 2, m, 128, 64, lens)
    Qd, Kd, Vd, T, L = dev(Q, K, V, table, ints(lens))
    first = sa.longformer_attn_paged_fwd(Qd, Kd, Vd, T, L, 6000)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for _ in range(4):  # two streams at once, without order between them
        for s in (s1, s2):
            with torch.cuda.stream(s):
                outs.append(sa.longformer_attn_paged_fwd(Qd, Kd, Vd, T, L, 6000))
            outs.append(sa.longformer_attn_paged_fwd(Qd, Kd, Vd, T, L, 6000, stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(o, first) for o in outs)
    assert sa.get_last_device_status() == 0


def test_results_on_another_stream_are_not_in_memory_that_this_one_still_writes():
    lens, m = [3000, 2100], 2100  # outputs of over a megabyte, which torch keeps apart from small ones
    Q, K, V, table = make_cache(4, 2, 4, 2, m, 64, 64, lens)
    Qd, Kd, Vd, T, L = dev(Q, K, V, table, ints(lens))
    want = sa.longformer_attn_paged_fwd(Qd, Kd, Vd, T, L, 6000)
    wide = torch.full((2, 600_000), -1, dtype=torch.int32, device="cuda")
    wide[0, :2] = torch.tensor([3, 5], dtype=torch.int32)
    refs = torch.ones(600_000, dtype=torch.int32, device="cuda")
    rows, lens2 = ints([0]).cuda(), ints([100, 0]).cuda()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    s = torch.cuda.Stream()
    scratch = sa.paged_workspace_bytes(2, 4, 2, m, 64, 64, T.shape[1], Qd.dtype)
    old = [torch.empty_like(x) for x in (Qd, wide, refs) for _ in range(3)]
    old += [torch.empty(scratch, dtype=torch.uint8, device="cuda") for _ in range(3)]
    for x in old:
        x.fill_(7)  # (a kernel's first launch would wait for the sleep)
    torch.cuda._sleep(1000)
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)  # some 10 ms
    for x in old:
        x.fill_(77)
    del old, x  # free again for this stream, while its fills are still to come
    got = sa.longformer_attn_paged_fwd(Qd, Kd, Vd, T, L, 6000, stream=s)
    new_table, new_lens, new_refs = sa.cache_free(wide, lens2, refs, rows, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    assert bool((new_table == -1).all()) and new_lens.tolist() == [0, 0]
    assert int(new_refs.sum()) == 600_000 - 2 and sa.get_last_device_status() == 0


def test_the_widest_windows():
    lens = [300]
    Q, K, V, table = make_cache(4, 1, 2, 2, 3, 64, 64, lens)
    args = dev(Q, K, V, table, ints(lens))
    want = sa.longformer_attn_paged_fwd(*args, 600)
    for window in (2 ** 31 - 2, 2 ** 31, 2 ** 40):  # what C takes at most, and more
        assert torch.equal(sa.longformer_attn_paged_fwd(*args, window), want)
    refs = torch.ones(K.shape[0], dtype=torch.int32, device="cuda")
    for reach in (2 ** 31 - 1, 2 ** 32 + 1):
        t, r = sa.cache_trim(args[3], args[4], refs, 64, reach)
        assert torch.equal(t, args[3]) and torch.equal(r, refs)


@pytest.mark.parametrize("m,Hq", [(1, 2), (3, 8), (130, 4)])
def test_captured_graphs_follow_the_lengths(m, Hq):
    # one graph, replayed while lengths, table and pools move on; two graphs replayed together
    lens = [400, 300]
    Q, K, V, table = make_cache(6, 2, Hq, 2, m, 64, 64, lens)
    Qd, Kd, Vd, T, L = dev(Q, K, V, table, ints(lens))
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(sa.longformer_attn_paged_fwd(Qd, Kd, Vd, T, L, 300, dilation=torch.zeros(Hq, dtype=torch.int32, device="cuda")))
        graphs.append(g)
    for new in ([400, 300], [399, 131], [m, m]):
        L.copy_(ints(new))
        torch.cuda.synchronize()
        s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
        with torch.cuda.stream(s1):
            graphs[0].replay()
        with torch.cuda.stream(s2):
            graphs[1].replay()
        torch.cuda.synchronize()
        want = sa.longformer_attn_paged_fwd(Qd, Kd, Vd, T, L, 300)
        assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
    assert sa.get_last_device_status() == 0


@pytest.mark.parametrize("m,Hq", [(1, 1), (1, 8), (20, 8)])
def test_offsets_past_32_bits(m, Hq):
    # a pool of over 2^32 bytes and 2^31 elements; the tokens lie at its end
    P, page, d, n = 262200, 128, 64, 300
    K = torch.zeros(P, 1, page, d, dtype=torch.bfloat16, device="cuda")
    V = torch.zeros_like(K)
    assert K.numel() > 2 ** 31
    Q, Ks, Vs, table = make_cache(8, 1, Hq, 1, m, d, page, [n], spare=0)
    K[-3:], V[-3:] = Ks.cuda(), Vs.cuda()
    Qd, T, L = dev(Q, table, ints([n]))
    got = sa.longformer_attn_paged_fwd(Qd, K, V, T + (P - 3), L, 1000)
    want = sa.longformer_attn_paged_fwd(Qd, Ks.cuda(), Vs.cuda(), T, L, 1000)
    assert torch.equal(got, want)
    # appending and copying there
    kn, vn = (torch.randn(1, 1, 5, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    sa.cache_append(kn, vn, K, V, T + (P - 3), L)
    assert torch.equal(K[int(table[0, 2]) + P - 3, 0, n - 5 - 256:n - 256], kn[0, 0])
    sa.cache_copy_pages(K, V, ints([P - 1]).cuda(), ints([P - 9]).cuda())
    assert torch.equal(V[P - 9].nan_to_num(7.0), V[P - 1].nan_to_num(7.0))
    assert sa.get_last_device_status() == 0


@pytest.mark.parametrize("m,Hq", [(40, 2), (300, 4)])
def test_a_wait_that_runs_out_ends_the_call_and_the_next_one_is_exact(m, Hq):
    lens = [3000, 700]
    Q, K, V, table = make_cache(61, 2, Hq, 2, m, 64, 64, lens)
    Qd, Kd, Vd, T, L = dev(Q, K, V, table, ints(lens))
    want = sa.longformer_attn_paged_fwd(Qd, Kd, Vd, T, L, 8000)
    torch.cuda.synchronize()
    assert sa.get_last_device_status() == 0
    sa.set_option(sa.SA_OPT_WAIT_LIMIT, 1)  # 1 microsecond: waits on copies and MMAs run out
    try:
        for _ in range(3):
            sa.longformer_attn_paged_fwd(Qd, Kd, Vd, T, L, 8000)
        torch.cuda.synchronize()  # every wait and every drain is bounded
    finally:
        sa.set_option(sa.SA_OPT_WAIT_LIMIT, 0)
    got = sa.longformer_attn_paged_fwd(Qd, Kd, Vd, T, L, 8000)
    torch.cuda.synchronize()
    assert sa.get_last_device_status() in (_lib.SA_OK, _lib.SA_ERR_TIMEOUT)
    assert sa.get_last_device_status() == 0 and torch.equal(got, want)


def test_many_sequences_and_many_globals():
    # the largest batch and the longest global list
    B, g = 1024, list(range(0, 1024, 2))
    lens = [1 + (i * 7) % 90 for i in range(B)]
    Q, K, V, table = make_cache(12, B, 1, 1, 1, 64, 16, lens)
    attend_and_check(Q, K, V, table, lens, None, 8, g[:512])


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d,page,m", [(64, 16, 1), (64, 64, 37), (128, 32, 200), (128, 128, 5)])
def test_append_writes_the_new_tokens_and_nothing_else(d, page, m, dtype):
    lens, q = [m + 3, 300, m], [m, min(m, 2), 0]
    Q, K, V, table = make_cache(13, 3, 2, 2, m, d, page, lens, dtype)
    kn, vn = (torch.randn(3, 2, m, d).to(K.dtype) for _ in range(2))
    for ql in (q, None):
        Kd, Vd = dev(K.clone(), V.clone())
        a, b = sa.cache_append(kn.cuda(), vn.cuda(), Kd, Vd, table.cuda(), ints(lens).cuda(),
                               q_lens=None if ql is None else ints(ql).cuda())
        assert a is Kd and b is Vd and sa.get_last_device_status() == 0
        wk, wv = op.append(f64(kn), f64(vn), f64(K), f64(V), table.numpy(), lens, ql)
        assert np.array_equal(f64(Kd), wk, equal_nan=True) and np.array_equal(f64(Vd), wv, equal_nan=True)


def test_append_drops_tokens_without_a_page():
    Q, K, V, table = make_cache(14, 2, 1, 1, 4, 64, 16, [20, 20])
    table[0, 1], table[1, 1] = -1, 99
    kn = torch.randn(2, 1, 8, 64).to(K.dtype)
    Kd, Vd = dev(K.clone(), V.clone())
    sa.cache_append(kn.cuda(), kn.cuda(), Kd, Vd, table.cuda(), ints([20, 20]).cuda())
    assert sa.get_last_device_status() == _lib.SA_ERR_BAD_INDEX
    wk, _ = op.append(f64(kn), f64(kn), f64(K), f64(V), table.numpy(), [20, 20], None)
    assert np.array_equal(f64(Kd), wk, equal_nan=True)
    sa.cache_append(kn.cuda(), kn.cuda(), Kd, Vd, table.cuda(), ints([5, 1000]).cuda())  # lengths out of contract
    assert sa.get_last_device_status() == _lib.SA_ERR_BAD_INDEX
    assert np.array_equal(f64(Kd), wk, equal_nan=True)


# ------------------------------------------------------------------ pages
def _pool(seed, layers=2, P=40, Hkv=2, page=16, d=64, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    K, V = (torch.randn(layers, P, Hkv, page, d, generator=g).to(dtype) for _ in range(2))
    return K, V


def _moved(pool, moves):
    out = pool.clone()
    for a, b in moves:
        out[:, b] = pool[:, a]
    return out


def _book(seed, B=9, slots=6, P=40, page=16, empty=(1, 4, 8)):
    r = np.random.RandomState(seed)
    order = r.permutation(P)
    table, lens, refs, at = np.full((B, slots), -1, np.int32), np.zeros(B, np.int32), np.zeros(P, np.int32), 0
    for b in range(B):
        if b in empty:
            continue
        n = int(r.randint(1, slots * page + 1)) if b else slots * page
        k = min(-(-n // page), 4)
        n = min(n, k * page)
        table[b, :k], lens[b] = order[at:at + k], n
        at += k
    table[3, 0] = table[0, 0]  # a shared page
    np.add.at(refs, table[table >= 0], 1)
    return table, lens, refs


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layers", [0, 3])
def test_copy_pages(layers, dtype):
    K, V = _pool(1, max(1, layers), 12, 3, 16, 64, dtype)
    if not layers:
        K, V = K[0], V[0]
    src, dst = [3, 7, 7, 0, 99], [1, 2, 11, 4, 5]
    Kd, Vd = dev(K.clone(), V.clone())
    sa.cache_copy_pages(Kd, Vd, ints(src).cuda(), ints(dst).cuda())
    assert sa.get_last_device_status() == _lib.SA_ERR_BAD_INDEX  # the pair out of range; the others are copied
    idx = (slice(None),) if layers else ()
    for pool, got in ((K, Kd), (V, Vd)):
        want = pool.clone()
        for a, b in list(zip(src, dst))[:-1]:
            want[idx + (b,)] = pool[idx + (a,)]
        assert torch.equal(got.cpu(), want)
    empty = torch.zeros(0, dtype=torch.int32, device="cuda")
    sa.cache_copy_pages(Kd, Vd, empty, empty)
    assert sa.get_last_device_status() == 0


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("src,dst,ok", [
    ([0], [1], True), ([2, 2, 0], [1, 4, 8], True), ([], [], True),
    ([0, 2], [1, 1], False),       # one destination twice: the first counts
    ([0, 1, 5], [1, 4, 8], False),  # a destination as a source
    ([0, 2], [3, 4], False),       # a destination in use
    ([0, -1, 2], [1, 4, 9], False),
])
def test_fork(src, dst, ok, in_place):
    table, lens, refs = _book(5)
    K, V = _pool(2)
    wt, wl, wr, moves = op.fork(table, lens, refs, 16, src, dst)
    Kd, Vd, T, L, R = dev(K, V, *map(torch.from_numpy, (table, lens, refs)))
    ins = (T.clone(), L.clone(), R.clone())
    t, n, r = sa.cache_fork(Kd, Vd, T, L, R, ints(src).cuda(), ints(dst).cuda(), out=(T, L, R) if in_place else None)
    assert sa.get_last_device_status() == (0 if ok else _lib.SA_ERR_BAD_INDEX)
    assert t.tolist() == wt and n.tolist() == wl and r.tolist() == wr
    assert torch.equal(Kd.cpu(), _moved(K, moves)) and torch.equal(Vd.cpu(), _moved(V, moves))
    if not in_place:
        assert all(torch.equal(a, b) for a, b in zip(ins, (T, L, R)))


def test_fork_without_free_pages_leaves_the_row_empty():
    table, lens, refs = _book(5)
    refs[refs == 0] = 7  # held by someone else
    last = int(np.flatnonzero(refs == 7)[0])
    refs[last] = 0       # one page left
    lens[lens == 96] = 95
    table, lens = table.copy(), lens.copy()
    src = [b for b in (2, 5, 6) if lens[b] % 16][:2]
    wt, wl, wr, moves = op.fork(table, lens, refs, 16, src, [1, 4])
    K, V = _pool(3)
    Kd, Vd, T, L, R = dev(K, V, *map(torch.from_numpy, (table, lens, refs)))
    t, n, r = sa.cache_fork(Kd, Vd, T, L, R, ints(src).cuda(), ints([1, 4]).cuda())
    assert len(moves) == 1 and sa.get_last_device_status() == _lib.SA_ERR_NO_PAGES
    assert t.tolist() == wt and n.tolist() == wl and r.tolist() == wr
    assert torch.equal(Kd.cpu(), _moved(K, moves))


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("rows,ok", [([0, 3], True), ([3, 3, 0, 3], True), ([], True), (list(range(9)), True), ([9, 2], False)])
def test_free(rows, ok, in_place):
    table, lens, refs = _book(7)
    T, L, R = dev(*map(torch.from_numpy, (table, lens, refs)))
    got = sa.cache_free(T, L, R, ints(rows).cuda(), out=(T, L, R) if in_place else None)
    assert [x.tolist() for x in got] == list(op.free_rows(table, lens, refs, rows))
    assert sa.get_last_device_status() == (0 if ok else _lib.SA_ERR_BAD_INDEX)


def test_free_never_makes_a_count_negative():
    table, lens, refs = _book(7)
    refs[table[0, 0]] = 1  # two rows name it
    T, L, R = dev(*map(torch.from_numpy, (table, lens, refs)))
    _, _, r = sa.cache_free(T, L, R, ints([0, 3]).cuda())
    assert int(r.min()) == 0 and sa.get_last_device_status() == _lib.SA_ERR_BAD_INDEX


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("reach,g", [(0, []), (20, []), (20, [0, 17, 40]), (33, [31, 32]), (20, [0, 95]), (1 << 30, [])])
def test_trim(reach, g, in_place):
    table, lens, refs = _book(11)
    T, L, R = dev(*map(torch.from_numpy, (table, lens, refs)))
    got = sa.cache_trim(T, L, R, 16, reach, ints(g).cuda(), out=(T, R) if in_place else None)
    assert [x.tolist() for x in got] == list(op.trim(table, lens, refs, 16, reach, g))
    assert sa.get_last_device_status() == 0


@pytest.mark.parametrize("in_place", [False, True])
def test_reserve(in_place):
    table, lens, refs = _book(13)
    q = np.array([0, 5, 16, 33, 0, 1, 17, 2, 40], np.int32)
    new = np.minimum(lens + q, 96).astype(np.int32)
    q = (new - lens).astype(np.int32)
    T, L, N, R = dev(*map(torch.from_numpy, (table, new, q, refs)))
    got = sa.cache_reserve(T, L, N, R, 16, out=(T, R) if in_place else None)
    want = op.reserve(table, new, q, refs, 16)
    assert [x.tolist() for x in got] == list(want) and sa.get_last_device_status() == 0
    again = sa.cache_reserve(*got[:1], L, N, got[1], 16)  # what is there is kept
    assert [x.tolist() for x in again] == list(want)
    refs[refs == 0] = 3
    refs[[8, 30]] = 0 if refs[8] == 3 and refs[30] == 3 else refs[[8, 30]]
    T, R = dev(*map(torch.from_numpy, (table, refs)))
    got = sa.cache_reserve(T, L, N, R, 16)
    assert [x.tolist() for x in got] == list(op.reserve(table, new, q, refs, 16))
    assert sa.get_last_device_status() == _lib.SA_ERR_NO_PAGES


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("P,B,slots", [(40, 9, 6), (5000, 700, 6), (64, 9, 6)])
def test_compact(P, B, slots, in_place):
    table, lens, refs = _book(17, B=B, slots=slots, P=P) if P < 5000 else _book(17, B=B, slots=slots, P=P, empty=())
    K, V = _pool(4, layers=2, P=P, Hkv=1)
    wt, wr, moves = op.compact(table, refs)
    Kd, Vd, T, R = dev(K, V, *map(torch.from_numpy, (table, refs)))
    t, r = sa.cache_compact(Kd, Vd, T, R, out=(T, R) if in_place else None)
    assert sa.get_last_device_status() == 0 and t.tolist() == wt and r.tolist() == wr
    live = sum(c > 0 for c in refs)
    assert torch.equal(Kd.cpu()[:, :live], _moved(K, moves)[:, :live])
    assert torch.equal(Vd.cpu(), _moved(V, moves))
    t2, r2 = sa.cache_compact(Kd, Vd, t, r)  # nothing left to move
    assert torch.equal(t2, t) and torch.equal(r2, r)


def test_compact_of_an_empty_and_a_full_pool():
    K, V = _pool(4, P=33)
    for fill in (0, 1):
        Kd, Vd, R = dev(K, V, torch.full((33,), fill, dtype=torch.int32))
        T = torch.full((2, 3), -1 if fill == 0 else 32, dtype=torch.int32, device="cuda")
        t, r = sa.cache_compact(Kd, Vd, T, R)
        assert torch.equal(t, T) and torch.equal(r, R) and torch.equal(Kd.cpu(), K)


# ------------------------------------------------------------------ together, as a serving loop uses them
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("window,g,dil", [(64, [0, 1, 2], None), (32, None, [0, 0, 1, 3]), (4000, None, None)])
def test_chunks_and_steps_give_the_whole_sequence(window, g, dil, dtype):
    """Reserve, append, attend (chunks, drafts, single tokens), trim and compact between them, and fork:
    every row must be the row of longformer_attn_fwd(causal) over the whole sequence."""
    n, H, d, page, P = 420, 4, 64, 16, 96
    gen = torch.Generator().manual_seed(77)
    q, k, v = (torch.randn(2, H, n, d, generator=gen).to(dtype).cuda() for _ in range(3))
    gd, dd = dev(ints(g), ints(dil))
    whole = sa.longformer_attn_fwd(q, k, v, window, gd, dilation=dd, causal=True)
    K = torch.full((P, H, page, d), float("nan"), dtype=dtype, device="cuda")
    V = K.clone()
    table = torch.full((4, 40), -1, dtype=torch.int32, device="cuda")
    refs = torch.zeros(P, dtype=torch.int32, device="cuda")
    lens = torch.zeros(4, dtype=torch.int32, device="cuda")
    reach = window // 2 * (max(dil or [0]) + 1)
    rows = [0, 1, None, None]  # which sequence each row of the table holds
    done = 0
    tol = dict(rtol=2.0 ** -6, atol=2.0 ** -6) if dtype is torch.bfloat16 else dict(rtol=1e-4, atol=2e-5)
    for i, m in enumerate([150, 1, 5, 64, 1, 1, 90, 3, 100, 1]):
        new = torch.tensor([m if r is not None else 0 for r in rows], dtype=torch.int32, device="cuda")
        lens = lens + new
        sa.cache_reserve(table, lens, new, refs, page, out=(table, refs))
        take = lambda x: torch.stack([x[0 if r is None else r, :, done:done + m] for r in rows]).contiguous()  # noqa: E731
        sa.cache_append(take(k), take(v), K, V, table, lens, q_lens=new)
        O = sa.longformer_attn_paged_fwd(take(q), K, V, table, lens, window, gd, dilation=dd, q_lens=new)
        for b, r in enumerate(rows):
            if r is None:
                assert (O[b] == 0).all()
            else:
                torch.testing.assert_close(O[b].float(), whole[r, :, done:done + m].float(), **tol)
        done += m
        if window < 1000:
            sa.cache_trim(table, lens, refs, page, reach, gd, out=(table, refs))
        if i % 3 == 2:
            sa.cache_compact(K, V, table, refs, out=(table, refs))
        if i == 3:  # both go on twice
            sa.cache_fork(K, V, table, lens, refs, ints([0, 1]).cuda(), ints([2, 3]).cuda(), out=(table, lens, refs))
            rows = [0, 1, 0, 1]
        if i == 7:
            sa.cache_free(table, lens, refs, ints([0]).cuda(), out=(table, lens, refs))
            rows[0] = None
            lens[0] = 0
    used = torch.zeros_like(refs).index_add_(0, table[table >= 0].long(), torch.ones_like(table[table >= 0]))
    assert torch.equal(used, refs) and sa.get_last_device_status() == 0
