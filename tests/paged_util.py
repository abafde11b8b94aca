"""A random paged cache and the error bounds of the paged attention, for its GPU tests."""

import numpy as np
import torch

import block_sparse_long_bigbird_gb300 as sa
from oracle.paged import oracle_paged

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def make_cache(seed, B, Hq, Hkv, m, d, page, lens, dtype="bf16", sigma=1.0, spare=3, width=None):
    """CPU tensors Q, K, V and a table whose pages lie in random order; NaN wherever no token was written."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in lens]
    P = sum(need) + spare
    order = torch.randperm(P, generator=g).tolist()
    table = torch.full((B, width or max(max(need), 1)), -1, dtype=torch.int32)
    K = torch.full((P, Hkv, page, d), float("nan"), dtype=DT[dtype])
    V = K.clone()
    at = 0
    for b, n in enumerate(lens):
        for c in range(need[b]):
            pg = order[at]
            at += 1
            table[b, c] = pg
            w = min(page, n - c * page)
            K[pg, :, :w] = (torch.randn(Hkv, w, d, generator=g) * sigma).to(DT[dtype])
            V[pg, :, :w] = torch.randn(Hkv, w, d, generator=g).to(DT[dtype])
    Q = (torch.randn(B, Hq, m, d, generator=g) * sigma).to(DT[dtype])
    return Q, K, V, table


def f64(t):
    return t.detach().cpu().double().numpy()


def bound(O, A, S, dtype, n, d, weights=2.0 ** -8):
    """Largest allowed |error| per element.

    u = 2^-24. A score's fp32 sum of d products is off by (d + 3) u S; the exponential by 2^-22
    relative; weights and their sum each carry that error, so their ratio twice it; sums over n keys add n u
    each. bf16 kernels round the weights by `weights` (to a bf16 number: half a step, 2^-8; to the sum of
    two: 2^-16) before the product with V, and every output is rounded once (2^-8 or 2^-24 of its value).
    """
    u = 2.0 ** -24
    eps = 2 * (np.expm1((d + 3) * u * S) + 2.0 ** -22) + 2 * n * u + 8 * u
    half = 2.0 ** -8 if dtype == "bf16" else u
    w = weights if dtype == "bf16" else 0.0
    return (eps[..., None] + w) * A + half * (np.abs(O) + (eps[..., None] + w) * A)


def dev(*ts):
    return [None if t is None else t.cuda() for t in ts]


def ints(x):
    return None if x is None else torch.as_tensor(list(x), dtype=torch.int32)


def attend_and_check(Q, K, V, table, lens, q_lens, window, gidx=None, dil=None, dtype="bf16", status=0, weights=2.0 ** -8):
    """Run on the GPU, compare every row with the oracle; returns O on the GPU."""
    Qd, Kd, Vd, Td, Ld, ql, gd, dd = dev(Q, K, V, table, ints(lens), ints(q_lens), ints(gidx), ints(dil))
    O = torch.full_like(Qd, float("nan"))
    sa.longformer_attn_paged_fwd(Qd, Kd, Vd, Td, Ld, window, gd, dilation=dd, q_lens=ql, out=O)
    torch.cuda.synchronize()
    assert sa.get_last_device_status() == status
    ref, A, S = oracle_paged(f64(Q), f64(K), f64(V), table.numpy(), lens, q_lens, window, gidx or (), dil)
    err = np.abs(f64(O) - ref)
    lim = bound(ref, A, S, dtype, max(lens), Q.shape[-1], weights)
    assert np.isfinite(f64(O)).all(), "output not finite"
    worst = np.unravel_index(np.argmax(err - lim), err.shape)
    assert (err <= lim).all(), f"at {worst}: {f64(O)[worst]} for {ref[worst]}, off {err[worst]:.3e}, allowed {lim[worst]:.3e}"
    return O
