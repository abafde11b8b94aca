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

pytestmark = pytest.mark.gpu


def _converts_first(B, Hq, Hkv, m, d, page, width, window, dilated=False, n_global=0):
    """Whether a bf16 call turns its pages into scratch of bf16 ones first: only then is its scratch as large as they are."""
    n = sa.paged_workspace_bytes(B, Hq, Hkv, m, d, page, width, torch.bfloat16, packed=True, window=window, dilated=dilated,
                                 n_global=n_global)
    return n >= 2 * B * width * Hkv * page * d * 2


def _weights(Q, table, page, Hkv, window, dtype, **kw):
    """How far off weights are: bf16 numbers (2^-8) only where the pages become bf16 ones first, halves (2^-11) else."""
    B, Hq, m, d = Q.shape
    first = dtype == "bf16" and _converts_first(B, Hq, Hkv, m, d, page, table.shape[1], window, **kw)
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
    attend4_and_check(Q, K, V, values, table, [n], None, 4 * n, dtype=dtype, weights=_weights(Q, table, 64, 1, 4 * n, dtype))


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
