"""Limits and refusals of the paged cache's entry points, before any launch. No GPU needed."""

import os

import pytest
import torch

FAKE = 0x7f0000000000  # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    from block_sparse_long_bigbird_gb300 import _build, _lib

    if not os.path.exists(_lib.LIB_PATH):
        _build.build()
    return _lib.lib()


def test_reserve_refuses_tables_whose_pages_it_cannot_count(lib):
    """Every entry may ask for a page; with 2^31 of them a 32-bit count would be negative and index before the list."""
    I, W = FAKE, FAKE + 0x1000000
    need = lib.sa_cache_workspace_bytes(64, 1024)

    def reserve(B, max_pages):
        return lib.sa_cache_reserve(64, 16, B, max_pages, I, I, I, I, I, I, W, need, None)

    assert reserve(1024, 1 << 21) == 2 and reserve(32, 1 << 26) == 2 and reserve(1023, (1 << 31) // 1023 + 1) == 2


def test_scratch_of_an_unsupported_dtype_is_a_type_error():
    import block_sparse_long_bigbird_gb300 as sa

    with pytest.raises(TypeError):
        sa.paged_workspace_bytes(1, 2, 2, 1, 64, 16, 4, torch.float16, device="cuda:0")
