"""Pages held in 4 bits and the rotation of positions where they could go wrong: weights far below the largest, results of
split tiles that are taken again."""

import math

import numpy as np
import pytest
import torch

import block_sparse_long_bigbird_gb300 as sa
from oracle import paged4 as o4
from oracle.paged import oracle_paged
from paged4_util import attend4_and_check, bound4, make_cache4
from paged_util import DT, dev, f64, ints
from test_paged4_gpu import CASES

pytestmark = pytest.mark.gpu


def _converts_first(Q, K, V, table, lens, q, window, g=None, dil=None):
    """Whether a bf16 call turns its pages into bf16 ones first: a launch more than over bf16 pages. (No call of up to three
    tiles, four at d = 64, of 24 rows per key head does.)"""
    m, group, d = Q.shape[2], Q.shape[1] // K.shape[1], Q.shape[3]
    if group <= 24 and -(-m // (24 // group)) <= (4 if d == 64 else 3):
        return False
    counts = []
    shape = K.shape[:3] + (d,)
    for pools in ((K, V), [torch.zeros(shape, dtype=torch.bfloat16) for _ in "KV"]):
        sa.longformer_attn_paged_fwd(*dev(Q, *pools, table, ints(lens)), window, *dev(ints(g)), dilation=dev(ints(dil))[0],
                                     q_lens=dev(ints(q))[0])
        counts.append(sa._lib.lib().sa_last_launch_count())
    return counts[0] > counts[1]


def _weights(Q, K, V, table, lens, q, window, g=None, dil=None):
    """How far off weights are: bf16 numbers (2^-8) only where the pages become bf16 ones first, else as the inputs' type says."""
    first = Q.dtype is torch.bfloat16 and _converts_first(Q, K, V, table, lens, q, window, g, dil)
    return 2.0 ** -8 if first else None


# ------------------------------------------------------------------ weights far below the largest
def _one_above_many(m, group, d, n, top, dtype):
    """Every key is zero but the one at position `top`, which is 14 to 30 powers of two above the others, another power for
    every row; its value is zero, so the others, however small their weights, are all there is of the result."""
    rng = np.random.default_rng(m + d + n)
    page = 64
    pages = -(-n // page)
    table = torch.from_numpy(rng.permutation(pages).astype(np.int32))[None].contiguous()
    codes = [np.zeros((pages, 1, page, d // 2), dtype=np.uint8), rng.integers(0, 8, (pages, 1, page, d // 2), dtype=np.uint8)]
    codes[1] |= rng.integers(0, 8, codes[1].shape, dtype=np.uint8) << 4
    scales = [np.full((pages, 1, page, d // 16), 120, dtype=np.uint8) for _ in "KV"]  # 1
    at = (int(table[0, top // page]), 0, top % page)
    codes[0][at][0] = 7  # 6
    codes[1][at] = 0
    rows = np.linspace(14.0, 30.0, m * group).reshape(1, group, m)
    Q = rng.standard_normal((1, group, m, d))
    Q[..., 0] = rows * math.log(2.0) * math.sqrt(d) / 6
    pools = [torch.from_numpy(o4.joined(c, s)) for c, s in zip(codes, scales)]
    values = [o4.decode(c, s) for c, s in zip(codes, scales)]
    return torch.from_numpy(Q).to(torch.bfloat16 if dtype == "bf16" else torch.float32), pools[0], pools[1], values, table


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d", [64, 128])
# few rows; chunks whose pages are converted on the way, of one tile and of two, whole and split
@pytest.mark.parametrize("m,group,n,late", [(1, 1, 700, False), (1, 8, 5000, True), (24, 1, 3000, True), (100, 1, 1500, False),
                                            (100, 1, 1500, True), (100, 1, 9000, False), (50, 2, 9000, True),
                                            (200, 1, 500, False), (200, 1, 6000, True), (100, 2, 6000, False)])
def test_weights_far_below_the_largest(m, group, n, late, d, dtype):
    """2^-14 to 2^-30 of the largest: no coarser than 2^-32 of it, in whichever kernel."""
    Q, K, V, values, table = _one_above_many(m, group, d, n, n - m if late else 0, dtype)
    attend4_and_check(Q, K, V, values, table, [n], None, 4 * n, dtype=dtype, weights=_weights(Q, K, V, table, [n], None, 4 * n))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("m,group,n,late", [(1, 1, 700, False), (1, 8, 5000, True), (16, 1, 3000, True), (100, 1, 1500, False),
                                            (2, 12, 9000, True)])
def test_weights_far_below_the_largest_in_fp32(m, group, n, late, d):
    """As above, no coarser than 2^-39 of the largest."""
    Q, K, V, values, table = _one_above_many(m, group, d, n, n - m if late else 0, "fp32")
    O = f64(sa.longformer_attn_paged_fwd(*dev(Q, K, V, table, ints([n])), 4 * n))
    ref, A, S = oracle_paged(f64(Q), *values, table.numpy(), [n], None, 4 * n)
    lim = bound4(ref, A, S, "fp32", n, d, 2.0 ** -7 * np.nanmax(np.abs(values[1])))  # that much finer than 2^-32
    assert (np.abs(O - ref) <= lim).all()


@pytest.mark.parametrize("m,group,d,n", [(100, 1, 64, 9000), (50, 2, 128, 9000), (200, 1, 64, 6000), (200, 1, 128, 6000),
                                         (20, 1, 64, 9000), (4, 4, 128, 9000)])
def test_parts_that_are_taken_again_join_those_that_are_not(m, group, d, n):
    """Rows that a NaN at a masked key spoils are taken again in one part of a split tile only; the other parts stay."""
    Q, K, V, values, table = make_cache4(91, 1, group, 1, m, d, 16, [n])
    codes, scales = (x.copy() for x in o4.parts(V.numpy(), d))
    last = n - 1
    scales[int(table[0, last // 16]), 0, last % 16, 1] = 255
    bad = torch.from_numpy(o4.joined(codes, scales))
    args = dev(Q, K, bad, table, ints([n]))
    got = f64(sa.longformer_attn_paged_fwd(*args, 4 * n))
    assert sa._lib.lib().sa_last_launch_count() == 2  # split, not converted first
    ref, A, S = oracle_paged(f64(Q), *values, table.numpy(), [n], None, 4 * n)
    lim = bound4(ref, A, S, "bf16", n, d, np.nanmax(np.abs(values[1])))
    assert (np.abs(got - ref)[:, :, :-1] <= lim[:, :, :-1]).all()
    assert np.isnan(got[:, :, -1, 16:32]).all()
    assert sa.get_last_device_status() == 0


# ------------------------------------------------------------------ waits that run out while the last copies are on their way
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("m,Hq,Hkv,d", [(100, 2, 2, 64), (100, 1, 1, 128), (60, 4, 2, 128), (200, 2, 2, 64), (256, 1, 1, 128)])
def test_waits_that_run_out_after_the_last_unit_was_seen(m, Hq, Hkv, d, packed):
    """A unit or less to a CTA: its loader has nothing left to do while its copies, out of cold memory, are still in flight and
    the other roles give up. No copy may outlive its CTA; the calls that follow are exact."""
    lens = [m + 100]
    Q, K, V, values, table = make_cache4(95, 1, Hq, Hkv, m, d, 64, lens)
    if not packed:
        K, V = (torch.from_numpy(np.nan_to_num(v)).to(torch.bfloat16) for v in values)
    args = dev(Q, K, V, table, ints(lens))
    want = sa.longformer_attn_paged_fwd(*args, 4000)
    cold = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")  # larger than the L2
    torch.cuda.synchronize()
    assert sa.get_last_device_status() == 0 and torch.isfinite(want).all()
    for _ in range(4):
        sa.set_option(sa.SA_OPT_WAIT_LIMIT, 1)  # 1 microsecond
        try:
            cold.zero_()
            sa.longformer_attn_paged_fwd(*args, 4000)
            torch.cuda.synchronize()
        finally:
            sa.set_option(sa.SA_OPT_WAIT_LIMIT, 0)
        got = sa.longformer_attn_paged_fwd(*args, 4000)
        torch.cuda.synchronize()
        assert sa.get_last_device_status() in (sa._lib.SA_OK, sa._lib.SA_ERR_TIMEOUT)
        assert torch.equal(got, want)
    assert sa.get_last_device_status() == 0


# ------------------------------------------------------------------ scratch sizes
@pytest.mark.parametrize("pool", [0, 1])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("B,Hq,Hkv,m,d,page,width", [(1, 12, 12, 1, 64, 64, 1024), (1, 4, 2, 7, 128, 16, 2000),
                                                     (2, 8, 2, 100, 64, 32, 700), (1, 16, 4, 600, 128, 128, 70),
                                                     (1, 64, 1, 20, 64, 64, 300)])
def test_exactly_the_scratch_that_is_asked_for_will_do(B, Hq, Hkv, m, d, page, width, dtype, pool):
    """Through the C entry points, for small and large windows, with and without dilations and global positions: the call takes
    the scratch that the size function names for the same arguments, and touches nothing behind it."""
    lib = sa._lib.lib()
    lens = [width * page, width * page // 2 + m][:B]
    Q, K, V, values, table = make_cache4(97, B, Hq, Hkv, m, d, page, lens, dtype)
    if pool == 0:
        K, V = (torch.from_numpy(np.nan_to_num(v)).to(DT[dtype]) for v in values)
    Q, K, V, table, L = dev(Q, K, V, table, ints(lens))
    g, dil = dev(ints([0, 3, 70, 900]), ints([h % 3 for h in range(Hq)]))
    for window in (0, 64, 512, 4000, 0x7ffffffe):
        for dilated in (0, 1):
            for ng in (0, 4):
                n = lib.sa_longformer_paged_workspace_bytes_ex(B, Hq, Hkv, m, d, page, width, window, dilated, ng, dtype == "fp32", pool)
                ws = torch.full((n + 64,), 171, dtype=torch.uint8, device="cuda")
                O = torch.full_like(Q, float("nan"))
                status = lib.longformer_attn_paged_fwd_ex(
                    Q.data_ptr(), K.data_ptr(), V.data_ptr(), O.data_ptr(), B, Hq, Hkv, m, d, page, K.shape[0], width,
                    table.data_ptr(), L.data_ptr(), None, window, dil.data_ptr() if dilated else None, g.data_ptr() if ng else None, ng,
                    ws.data_ptr() if n else None, n, dtype == "fp32", pool, torch.cuda.current_stream().cuda_stream)
                assert status == 0, (window, dilated, ng, n)
                assert torch.isfinite(O).all() and (ws[n:] == 171).all(), (window, dilated, ng, n)
    assert sa.get_last_device_status() == 0


# ------------------------------------------------------------------ rows that are only moved
def _any_bits(shape, dtype, seed):
    """Every pattern of bits as likely: infinities and NaNs of all kinds among them."""
    g = torch.Generator().manual_seed(seed)
    of = torch.int16 if dtype == "bf16" else torch.int32
    return torch.randint(torch.iinfo(of).min, torch.iinfo(of).max + 1, shape, generator=g, dtype=torch.int64).to(of)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d,rot,interleaved", [(64, 32, False), (64, 16, True), (128, 48, False), (128, 128, True), (64, 64, False)])
def test_what_is_not_rotated_keeps_its_bits(d, rot, interleaved, dtype):
    """Values, elements from rot on, and rows read from plain pages: a NaN's bits too, as sa_cache_append moves them."""
    B, Hkv, Hq, m, page, lens, q = 3, 2, 4, 9, 16, [40, 9, 23], [9, 9, 4]
    bits = [_any_bits((B, h, m, d), dtype, i) for i, h in enumerate((Hkv, Hkv, Hq))]
    assert all(torch.isnan(x.view(DT[dtype])).any() for x in bits)
    kn, vn, qn = (x.view(DT[dtype]).cuda() for x in bits)
    table = torch.arange(9, dtype=torch.int32).reshape(3, 3)
    T, L, n = dev(table, ints(lens), ints(q))
    K, V = (torch.zeros(9, Hkv, page, d, dtype=DT[dtype], device="cuda") for _ in "KV")
    Kp, Vp = torch.zeros_like(K), torch.zeros_like(V)
    sa.cache_append(kn, vn, Kp, Vp, T, L, q_lens=n)
    _, _, Q = sa.cache_append(kn, vn, K, V, T, L, q_lens=n, rope=sa.rope_table(64, rot), interleaved=interleaved, Q_new=qn)
    of = bits[0].dtype
    assert torch.equal(V.view(of), Vp.view(of)) and torch.equal(K.view(of)[..., rot:], Kp.view(of)[..., rot:])
    rows = [t.view(of).cpu() for t in sa.cache_read(Kp, Vp, T, L, m, q_lens=n)]
    for b in range(B):
        assert torch.equal(Q.view(of).cpu()[b, :, :q[b], rot:], bits[2][b, :, :q[b], rot:])
        for got, want in zip(rows, bits):
            assert torch.equal(got[b, :, :q[b]], want[b, :, :q[b]]) and (got[b, :, q[b]:] == 0).all()
    assert sa.get_last_device_status() == 0


@pytest.mark.parametrize("packed", [False, True])
def test_windows_past_32_bits(packed):
    """A window whose lower 32 bits are those of a small or a negative one: all that is seen, and its scratch; or a refusal."""
    lens, m = [9000], 1100
    Q, K, V, values, table = make_cache4(98, 1, 2, 2, m, 64, 64, lens)
    if not packed:
        K, V = (torch.from_numpy(np.nan_to_num(v)).to(torch.bfloat16) for v in values)
    args = dev(Q, K, V, table, ints(lens))
    want = sa.longformer_attn_paged_fwd(*args, 20000)
    sizes = (1, 2, 2, m, 64, 64, table.shape[1], torch.bfloat16)
    all_of_it = sa.paged_workspace_bytes(*sizes, packed=packed)
    for window in (2 ** 31, 2 ** 32, 2 ** 32 + 64, 2 ** 40, 2 ** 63 + 2):
        n = sa.paged_workspace_bytes(*sizes, packed=packed, window=window)
        assert n == all_of_it
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        assert torch.equal(sa.longformer_attn_paged_fwd(*args, window, workspace=ws), want)
    for window in (-2, -2 ** 32, 64 - 2 ** 32, -2 ** 40):
        with pytest.raises(sa.SparseAttnError):
            sa.longformer_attn_paged_fwd(*args, window)
        assert not packed or sa.paged_workspace_bytes(*sizes, packed=True, window=window) == 0
    assert sa.get_last_device_status() == 0


# ------------------------------------------------------------------ weights as fine as each path holds them
@pytest.mark.parametrize("name", [k for k, c in CASES.items() if c[3] * (c[1] // c[2]) > 24])
def test_weights_of_more_than_24_rows(name):
    """Halves (2^-11) wherever the pages are not converted first, in further tiles of few rows and in chunks alike."""
    B, Hq, Hkv, m, d, page, lens, q, window, g, dil = CASES[name]
    Q, K, V, values, table = make_cache4(len(name), B, Hq, Hkv, m, d, page, lens)
    w = _weights(Q, K, V, table, lens, q, window, g, dil)
    attend4_and_check(Q, K, V, values, table, lens, q, window, g, dil, weights=w)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("m,group,n", [(30, 1, 2500), (72, 1, 2500), (40, 2, 3100), (100, 1, 2500), (3, 40, 2500), (120, 2, 1900)])
def test_weights_of_more_than_24_rows_in_long_sweeps(m, group, n, d):
    Q, K, V, values, table = make_cache4(m + n, 1, group, 1, m, d, 32, [n], sigma=1.0)
    attend4_and_check(Q, K, V, values, table, [n], None, 2 * n, weights=_weights(Q, K, V, table, [n], None, 2 * n))


# ------------------------------------------------------------------ queries
# few rows; chunks of one tile and of two, which turn their queries into halves in place
_ROWS = [(2, 2), (20, 1), (100, 1), (50, 2), (200, 1)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("m,group", _ROWS)
@pytest.mark.parametrize("above", [12, 24, 30])
def test_queries_with_elements_far_above_the_others(above, m, group, d, dtype):
    """In places where every key is zero, so that the ordinary elements, 2^-above of the largest, make the scores: no coarser
    than 2^-38 of the largest (half of a half's smallest number, the largest being at least 2^13)."""
    n = 300
    Q, K, V, values, table = make_cache4(m + d + above, 1, group, 1, m, d, 16, [n], dtype)
    codes, scales = (x.copy() for x in o4.parts(K.numpy(), d))
    codes[..., :8] = 0
    K, values[0] = torch.from_numpy(o4.joined(codes, scales)), o4.decode(codes, scales)
    Q[..., :16] *= 2.0 ** above
    O = sa.longformer_attn_paged_fwd(*dev(Q, K, V, table, ints([n])), 4 * n)
    ref, A, S = oracle_paged(f64(Q), *values, table.numpy(), [n], None, 4 * n)
    # the scores' error joins the others': of weight and sum alike
    k = np.nansum(np.abs(values[0]), -1).max()
    off = 2 * np.expm1(2.0 ** -38 * np.abs(f64(Q)).max(-1) * k / math.sqrt(d))
    lim = bound4(ref, A, S, dtype, n, d, np.nanmax(np.abs(values[1])))
    lim += (1 + 2.0 ** -8) * off[..., None] * A
    assert (np.abs(f64(O) - ref) <= lim).all()
    assert sa.get_last_device_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("m,group", _ROWS)
@pytest.mark.parametrize("e", [-133, -120, -20, 60, 110, 127])
def test_queries_of_every_exponent(e, m, group, dtype):
    """Elements of 2^e: a third of the keys are opposite to them, the others zero where the queries are not. Those of large
    queries get no weight, and all the others the same; of tiny ones every key does."""
    n, d = 300, 64
    Q, K, V, values, table = make_cache4(m + 200 + e, 1, group, 1, m, d, 16, [n], dtype)
    codes, scales = (x.copy() for x in o4.parts(K.numpy(), d))
    codes[..., :16] = 0
    drop = np.arange(n) % 3 == 1
    for j in np.flatnonzero(drop):
        codes[int(table[0, j // 16]), 0, j % 16, :16] = 0xff  # -6, twice
    scales[..., :2] = np.where(scales[..., :2] == 255, 255, 120)  # 1
    K = torch.from_numpy(o4.joined(codes, scales))
    g = torch.Generator().manual_seed(e + 200)
    Q = torch.zeros(Q.shape, dtype=torch.float64)
    Q[..., :32] = torch.ldexp(1 + torch.rand(1, group, m, 32, generator=g).double(), torch.tensor(e)) * (127 / 128)
    Q = Q.to(DT[dtype])
    O = f64(sa.longformer_attn_paged_fwd(*dev(Q, K, V, table, ints([n])), 4 * n))
    assert torch.isfinite(Q).all() and (Q[..., :32] > 0).all()
    v = np.stack([values[1][int(table[0, j // 16]), 0, j % 16] for j in range(n)])
    # a mean of |v| <= 6 * 2^2 by equal weights, which are exact; tiny queries' scores of less than 2^-9 move them by 2^-8
    tiny = e < 0
    for t in range(m):
        take = np.arange(n) <= n - m + t
        take &= True if tiny else ~drop
        want, size = v[take].mean(0), np.abs(v[take]).mean(0)
        off = np.abs(O[0, :, t] - want)
        assert (off <= 2.0 ** -8 * np.abs(want) * (1 + 2.0 ** -7) + ((2.0 ** -7 if e == -20 else 0) + 2.0 ** -12) * size).all()
    assert sa.get_last_device_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("m,group", _ROWS)
def test_queries_that_are_infinite_or_nan_reach_their_own_rows_only(m, group, dtype):
    n, d = 300, 64
    Q, K, V, values, table = make_cache4(m + 300, 1, group, 1, m, d, 16, [n], dtype)
    ref, A, S = oracle_paged(f64(Q), *values, table.numpy(), [n], None, 4 * n)
    lim = bound4(ref, A, S, dtype, n, d, np.nanmax(np.abs(values[1])))
    bad = Q.clone()
    bad[0, 0, 0, 5], bad[0, group - 1, m // 2, 40], bad[0, 0, m - 1, 63] = float("inf"), float("nan"), -float("inf")
    got = sa.longformer_attn_paged_fwd(*dev(bad, K, V, table, ints([n])), 4 * n)
    spoiled = ~torch.isfinite(bad).all(-1).numpy()
    assert np.isnan(f64(got)[spoiled]).all() and (np.abs(f64(got) - ref) <= lim)[~spoiled].all()
    assert sa.get_last_device_status() == 0


# ------------------------------------------------------------------ pools of more than 2^32 bytes
@pytest.mark.parametrize("d", [64, 128])
def test_offsets_past_32_bits_everywhere(d):
    """Tokens behind the first 2^32 bytes of both pools: every kernel of the attention, rows taken again, writing, reading."""
    page = 128
    P = (2 ** 32 + 2 ** 29) // (page * 9 * d // 16)
    K = torch.zeros(sa.pool_shape_4bit(P, 1, page, d), dtype=torch.uint8, device="cuda")
    V = torch.zeros_like(K)
    # one row; several; tiles of few rows; chunks of one tile and of two; converted first; on the ordinary units
    for m, Hq, n, dtype, simt in ((1, 1, 300, "bf16", 0), (1, 16, 300, "bf16", 0), (40, 1, 700, "bf16", 0), (9, 3, 300, "fp32", 0),
                                  (100, 1, 300, "bf16", 0), (200, 1, 9000, "bf16", 0), (1100, 4, 9000, "bf16", 0),
                                  (40, 1, 300, "fp32", 1)):
        Q, Ks, Vs, _, table = make_cache4(8 + m, 1, Hq, 1, m, d, page, [n], dtype, spare=0)
        codes, scales = (x.copy() for x in o4.parts(Vs.numpy(), d))
        scales[int(table[0, (n - 1) // page]), 0, (n - 1) % page, 0] = 255  # the last token's: for its own row only
        Vn = torch.from_numpy(o4.joined(codes, scales))
        need = Ks.shape[0]
        Qd, T, L = dev(Q, table, ints([n]))
        far = T + (P - need)
        assert (P - need) * Ks[0].numel() > 2 ** 32
        assert dtype == "fp32" or _converts_first(Q, Ks, Vs, table, [n], None, 2 * n) == (m == 1100)
        sa.set_option(sa.SA_OPT_FORCE_SIMT, simt)
        try:
            for v in (Vs, Vn):
                K[-need:], V[-need:] = Ks.cuda(), v.cuda()
                got = sa.longformer_attn_paged_fwd(Qd, K, V, far, L, 2 * n)
                want = sa.longformer_attn_paged_fwd(Qd, Ks.cuda(), v.cuda(), T, L, 2 * n)
                assert torch.equal(got.nan_to_num(77.0), want.nan_to_num(77.0))
                assert torch.isnan(want).any() == (v is Vn) and (want[:, :, 0] != 0).any()
        finally:
            sa.set_option(sa.SA_OPT_FORCE_SIMT, 0)
    for dtype, inter in ((torch.bfloat16, False), (torch.float32, True)):
        kn, vn, qn = (torch.randn(1, 1, 50, d, device="cuda").to(dtype) for _ in "kvq")
        rope = sa.rope_table(n, d)
        small = sa.cache_append(kn, vn, Ks.cuda(), Vs.cuda(), T, L, rope=rope, interleaved=inter, Q_new=qn)
        K[-need:], V[-need:] = Ks.cuda(), Vs.cuda()
        large = sa.cache_append(kn, vn, K, V, far, L, rope=rope, interleaved=inter, Q_new=qn)
        assert torch.equal(K[-need:], small[0]) and torch.equal(V[-need:], small[1]) and torch.equal(large[2], small[2])
        assert not torch.equal(small[0].cpu(), Ks)
        a, b = (sa.cache_read(x, y, t, L, n, dtype=dtype) for x, y, t in ((K, V, far), (*small[:2], T)))
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and (a[0] != 0).any()
    sa.cache_copy_pages(K, V, ints([P - 1]).cuda(), ints([P - 9]).cuda())
    assert torch.equal(V[P - 9], V[P - 1]) and torch.equal(K[P - 9], K[P - 1])
    assert sa.get_last_device_status() == 0


# ------------------------------------------------------------------ long sums in fp32
@pytest.mark.parametrize("d,group", [(64, 1), (64, 20), (128, 1), (128, 12)])
def test_long_sums_in_fp32(d, group):
    """Relative error of the results' root mean square, over sequences so many and long that a warp sums n / 8 keys.

    u = 2^-24; a rounding to the nearest is off by u / sqrt(3) of its result in the mean square. Values of either sign, so
    that sums grow as the root of their terms. A result: 256 additions of 16 keys' sums, u sqrt(256 / 6) = 6.5 u. The weights'
    sum: 512 additions of a lane, growing evenly, u sqrt(512) / 3 = 7.5 u. Scores, of mean square 1.3: each of d = 128 products
    off by 2 u at most (two halves, the sum's last place) at random, 15 u. The exponential 4 u, weights as two halves 1 u.
    Together 19 u; as much again, and some for what leans: 45 u. (Sums of all keys in the matrix instructions' own
    accumulators, which cut off: 74 to 81 u.)
    """
    B, Hkv, n, page = 16, 8, 32768, 128
    g = torch.Generator(device="cuda").manual_seed(d + group)
    P, codes = B * n // page, page * d // 2
    K, V = (torch.randint(0, 256, sa.pool_shape_4bit(P, Hkv, page, d), generator=g, dtype=torch.uint8, device="cuda")
            for _ in "KV")
    for x in (K, V):  # one scale: the numbers themselves, of mean square 8.6
        x.view(P, Hkv, -1)[..., codes:] = 120
    table = torch.randperm(P, generator=g, device="cuda").to(torch.int32).reshape(B, -1).contiguous()
    Q = torch.randn(B, Hkv * group, 1, d, generator=g, device="cuda") / 6.7 ** 0.5
    O = sa.longformer_attn_paged_fwd(Q, K, V, table, torch.full((B,), n, dtype=torch.int32, device="cuda"), 2 * n)
    one = torch.tensor(o4.MAGNITUDES, device="cuda")
    value = torch.cat([one, -one])
    off = size = 0.0
    for b, h in ((0, 0), (7, 3), (B - 1, Hkv - 1)):
        k, v = (x.view(P, Hkv, -1)[table[b].long(), h, :codes].reshape(-1, d // 2).int() for x in (K, V))
        k, v = (torch.stack([value[x & 15], value[x >> 4]], -1).reshape(n, d) for x in (k, v))
        q = Q[b, h * group:(h + 1) * group, 0].double()
        want = torch.softmax(q @ k.T / math.sqrt(d), -1) @ v
        off += float(((O[b, h * group:(h + 1) * group, 0] - want) ** 2).sum())
        size += float((want ** 2).sum())
    assert math.sqrt(off / size) <= 45 * 2.0 ** -24
    assert sa.get_last_device_status() == 0
