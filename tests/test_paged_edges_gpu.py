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
