"""Paged key/value cache of an autoregressive Longformer: attention of new tokens over it, and its pages.

Thin wrappers of the ``longformer_attn_paged_fwd`` and ``sa_cache_*`` entry
points (include/sparse_attn.h says what each computes). A pool of one layer is
a ``[num_pages, Hkv, page, d]`` tensor; the calls that move pages take either
one layer or all of them, ``[layers, num_pages, Hkv, page, d]``. A pool held in
4 bits is a uint8 tensor whose last size is 9 * d / 16 (``pool_shape_4bit``); what the
bytes of a page mean is in include/sparse_attn.h. Every call takes either kind.

The bookkeeping calls return new tables, lengths and counts; with ``out`` they
write into the tensors given there, which may be the inputs themselves. Pools
are always changed in place. Nothing here waits for the device: what a kernel
finds wrong in a table or a list is reported by ``get_last_device_status``.
"""

import functools

import torch

from . import _lib

# torch's allocation without its dispatcher, which costs 4 us of a call of 16; on the current device only
_new_cuda = getattr(getattr(getattr(torch._C, "_dynamo", None), "guards", None), "_empty_strided_cuda", None)

_DTYPE = {torch.bfloat16: _lib.SA_BF16, torch.float32: _lib.SA_FP32}
_INT = torch.int32
_HEAD_4BIT = {36: 64, 72: 128}  # a token's bytes in a 4-bit page: head size
_WIDEST = 0x7ffffffe  # a window: half of it is more than any position


def _call(name, device, stream, *args):
    """Run a C entry point on `device` and `stream` (default: its current one)."""
    fn = getattr(_lib.lib(), name)
    index = device.index
    handle = torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream
    if torch._C._cuda_getDevice() == index:
        st = fn(*args, handle)
    else:
        with torch.cuda.device(device):
            st = fn(*args, handle)
    if st != _lib.SA_OK:
        raise _lib.SparseAttnError(st, name)


def _new(shape, strides, dtype, device, stream):
    """An uninitialised tensor for a call on `stream`.

    Memory of that stream, so that nothing that the current one still has to do may touch it; the current one, where
    the caller goes on, keeps it from reuse too.
    """
    if stream is not None:
        caller = torch.cuda.current_stream(device)
        with torch.cuda.stream(stream):
            t = torch.empty_strided(shape, strides, dtype=dtype, device=device)
        t.record_stream(caller)
        return t
    if _new_cuda is not None and torch._C._cuda_getDevice() == device.index:
        return _new_cuda(shape, strides, dtype)
    return torch.empty_strided(shape, strides, dtype=dtype, device=device)


def _scratch(n_bytes, device, stream):
    """Workspace of one call."""
    return None if n_bytes == 0 else _new((n_bytes,), (1,), torch.uint8, device, stream)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _ints(name, t, device, *shape):
    """`t` must be a contiguous int32 tensor on `device` of `shape` (-1: any size there)."""
    got = t.shape
    if t.dtype is _INT and t.device == device and t.is_contiguous() and len(got) == len(shape):
        if got == shape or (got[0] == shape[0] or shape[0] < 0) and (len(got) == 1 or got[1] == shape[1] or shape[1] < 0):
            return
    raise ValueError(f"{name} must be a contiguous int32 tensor {list(shape)} on {device} (-1: any size)")


def _pools(K_pages, V_pages, dims):
    """The pools' head size, and whether they are held in 4 bits."""
    packed = K_pages.dtype is torch.uint8
    if K_pages.dtype not in _DTYPE and not packed:
        raise TypeError(f"unsupported dtype {K_pages.dtype}; use bfloat16 or float32, or uint8 pages held in 4 bits")
    if not K_pages.is_cuda or K_pages.dim() not in dims or V_pages.shape != K_pages.shape \
            or V_pages.dtype is not K_pages.dtype or V_pages.device != K_pages.device \
            or not K_pages.is_contiguous() or not V_pages.is_contiguous():
        raise ValueError("K_pages and V_pages must be contiguous CUDA tensors [num_pages, Hkv, page, d]"
                         + (" or [layers, num_pages, Hkv, page, d]" if 5 in dims else "")
                         + " of one shape, dtype and device")
    if packed and K_pages.shape[-1] not in _HEAD_4BIT:
        raise ValueError("pages held in 4 bits must have 9 * d / 16 bytes per token and head: 36 or 72")
    return (_HEAD_4BIT[K_pages.shape[-1]] if packed else K_pages.shape[-1]), packed


def pool_shape_4bit(num_pages, Hkv, page, d, layers=None):
    """Shape of a uint8 pool whose pages are held in 4 bits."""
    if d not in _HEAD_4BIT.values() or page not in (16, 32, 64, 128):
        raise ValueError("d must be 64 or 128, page 16, 32, 64 or 128")
    return (() if layers is None else (layers,)) + (num_pages, Hkv, page, 9 * d // 16)


def rope_table(n, rot, base=10000.0, device="cuda"):
    """(cos, sin) of the angles p * base ** (-2 i / rot) as fp32 [n, rot / 2]; worked out in 64 bits."""
    if n < 1 or rot < 16 or rot % 16:
        raise ValueError("n must be positive and rot a positive multiple of 16")
    turn = base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot)
    angle = torch.arange(n, dtype=torch.float64, device=device)[:, None] * turn
    return angle.cos().float(), angle.sin().float()


def _new_rows(name, t, dtype, device, d, heads):
    if t.dtype is not dtype or t.device != device or t.dim() != 4 or not t.is_contiguous() \
            or t.shape[3] != d or (heads is not None and t.shape[1] != heads):
        raise ValueError(f"{name} must be a contiguous [B, heads, m, d] tensor matching the pools in dtype, device "
                         "and head size")


def longformer_attn_paged_fwd(Q, K_pages, V_pages, block_table, seq_lens, window, global_idx=None, dilation=None,
                              q_lens=None, out=None, stream=None, workspace=None):
    """Autoregressive Longformer attention of new tokens over a paged cache; returns O shaped like Q.

    Q: [B, Hq, m, d], the new tokens' queries (Hq a multiple of the pools' heads; m = 1 for a single-token step).
    block_table: int32 [B, max_pages], page of each stretch of tokens or -1; seq_lens: int32 [B], tokens in the
    cache with the new ones (already appended); q_lens: int32 [B], new tokens of each sequence, or None (m each).
    window, global_idx, dilation: as for longformer_attn_fwd (causal); 2 * (longest sequence) sees every token.
    workspace: uint8 CUDA tensor of paged_workspace_bytes(...), or None to allocate it here.
    With uint8 pools, held in 4 bits, Q may be bf16 or fp32.
    Rows past q_lens and rows that see no key are zeros.
    """
    dtype, dev, shape, strides = Q.dtype, Q.device, Q.shape, Q.stride()
    pool, table = K_pages.shape, block_table.shape
    # every test below in one expression; where it fails, the tests one by one say which
    kind = K_pages.dtype
    packed = kind is torch.uint8
    if not (len(shape) == len(pool) == 4 and V_pages.shape == pool and dtype in _DTYPE and V_pages.dtype is kind
            and (shape[3] == pool[3] and kind is dtype if not packed else _HEAD_4BIT.get(pool[3]) == shape[3])
            and block_table.dtype is _INT and seq_lens.dtype is _INT and K_pages.device == dev and V_pages.device == dev
            and block_table.device == dev and seq_lens.device == dev
            and Q.is_cuda and Q.is_contiguous() and K_pages.is_contiguous() and V_pages.is_contiguous()
            and block_table.is_contiguous() and seq_lens.is_contiguous()
            and len(table) == 2 and table[0] == shape[0] and seq_lens.shape == shape[:1]):
        d, packed = _pools(K_pages, V_pages, (4,))
        if dtype not in _DTYPE:
            raise TypeError(f"unsupported dtype {dtype}; use bfloat16 or float32")
        _new_rows("Q", Q, dtype if packed else kind, K_pages.device, d, None)
        _ints("block_table", block_table, dev, shape[0], -1)
        _ints("seq_lens", seq_lens, dev, shape[0])
    num_pages, Hkv, page, _ = pool
    B, Hq, m, d = shape
    if q_lens is not None:
        _ints("q_lens", q_lens, dev, B)
    if dilation is not None:
        _ints("dilation", dilation, dev, Hq)
    if global_idx is not None:
        _ints("global_idx", global_idx, dev, -1)
    n_global = 0 if global_idx is None else global_idx.numel()
    if not 0 <= window <= _WIDEST:
        window = _in_32_bits(window)
    max_pages = table[1]
    dt = _DTYPE[dtype]
    if workspace is None:
        n = (_workspace_bytes(dev.index, B, Hq, Hkv, m, d, page, max_pages, dt, True, window, dilation is not None, n_global)
             if packed else _workspace_bytes(dev.index, B, Hq, Hkv, m, d, page, max_pages, dt))
        workspace = _scratch(n, dev, stream)
    elif not workspace.is_cuda or workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor on Q's device")
    if out is None:
        out = _new(tuple(shape), strides, dtype, dev, stream)
    elif out.shape != Q.shape or out.dtype is not Q.dtype or out.device != dev or not out.is_contiguous():
        raise ValueError("out must be a contiguous CUDA tensor shaped and typed like Q")
    _call("longformer_attn_paged_fwd_ex", dev, stream, Q.data_ptr(), K_pages.data_ptr(), V_pages.data_ptr(),
          out.data_ptr(), B, Hq, Hkv, m, d, page, num_pages, max_pages, block_table.data_ptr(), seq_lens.data_ptr(),
          _ptr(q_lens), window, _ptr(dilation), global_idx.data_ptr() if n_global else None, n_global,
          _ptr(workspace), 0 if workspace is None else workspace.numel() * workspace.element_size(), dt, packed)
    return out


def _in_32_bits(window):
    """A window as the C calls take it, which see 32 bits of any number: the widest, or one that they refuse."""
    return _WIDEST if window > 0 else -2


@functools.lru_cache(maxsize=1024)  # the sizes and the device's number of SMs are all it depends on
def _workspace_bytes(index, B, Hq, Hkv, m, d, page, max_pages, dtype, packed=False, window=_WIDEST, dilated=False,
                     n_global=0):
    sizes = (B, Hq, Hkv, m, d, page, max_pages)
    with torch.cuda.device(index):
        if not packed:  # whatever the window
            return _lib.lib().sa_longformer_paged_workspace_bytes(*sizes, dtype)
        return _lib.lib().sa_longformer_paged_workspace_bytes_ex(*sizes, window, dilated, n_global, dtype, packed)


def paged_workspace_bytes(B, Hq, Hkv, m, d, page, max_pages, dtype, device=None, packed=False, window=_WIDEST,
                          dilated=False, n_global=0):
    """Scratch bytes of a longformer_attn_paged_fwd call of these sizes on `device` (default: the current one).

    dtype: Q's; packed: whether the pages are held in 4 bits, and then the window, whether there are dilations, and how
    many global positions (of other pages the scratch is the same for all).
    """
    if dtype not in _DTYPE:
        raise TypeError(f"unsupported dtype {dtype}; use bfloat16 or float32")
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    if dev.index is None:
        dev = torch.device("cuda", torch.cuda.current_device())
    if not 0 <= window <= _WIDEST:
        window = _in_32_bits(window)
    return _workspace_bytes(dev.index, B, Hq, Hkv, m, d, page, max_pages, _DTYPE[dtype], bool(packed), window, bool(dilated),
                            n_global)


def cache_append(K_new, V_new, K_pages, V_pages, block_table, seq_lens, q_lens=None, stream=None, rope=None,
                 interleaved=False, Q_new=None, Q_out=None):
    """Write the new tokens' keys and values [B, Hkv, m, d] into their pages; returns (K_pages, V_pages).

    rope: (cos, sin), fp32 [positions, rot / 2] each (rope_table): the keys are rotated to their positions on the way,
    pairs of elements (i, i + rot / 2), or (2 i, 2 i + 1) if interleaved. With it Q_new [B, Hq, m, d] may be given too:
    rotated into Q_out (None: allocated here; Q_new itself: in place), rows past q_lens zeros, and returned third.
    uint8 pages: written in 4 bits.
    """
    dtype, dev, shape = K_new.dtype, K_new.device, K_new.shape
    pool, table, kind = K_pages.shape, block_table.shape, K_pages.dtype
    packed = kind is torch.uint8
    if not (len(shape) == len(pool) == 4 and V_pages.shape == pool and V_new.shape == shape and shape[1] == pool[1]
            and dtype in _DTYPE and V_new.dtype is dtype and V_pages.dtype is kind
            and (shape[3] == pool[3] and kind is dtype if not packed else _HEAD_4BIT.get(pool[3]) == shape[3])
            and block_table.dtype is _INT and seq_lens.dtype is _INT
            and V_new.device == dev and K_pages.device == dev and V_pages.device == dev and block_table.device == dev
            and seq_lens.device == dev and K_new.is_cuda and K_new.is_contiguous() and V_new.is_contiguous()
            and K_pages.is_contiguous() and V_pages.is_contiguous() and block_table.is_contiguous()
            and seq_lens.is_contiguous() and len(table) == 2 and table[0] == shape[0] and seq_lens.shape == shape[:1]):
        d, packed = _pools(K_pages, V_pages, (4,))
        if dtype not in _DTYPE:
            raise TypeError(f"unsupported dtype {dtype}; use bfloat16 or float32")
        _new_rows("K_new", K_new, dtype if packed else kind, K_pages.device, d, pool[1])
        _new_rows("V_new", V_new, dtype if packed else kind, K_pages.device, d, pool[1])
        if V_new.shape != shape:
            raise ValueError("K_new and V_new must share shape")
        _ints("block_table", block_table, dev, shape[0], -1)
        _ints("seq_lens", seq_lens, dev, shape[0])
    num_pages, Hkv, page, _ = pool
    B, _, m, d = shape
    if q_lens is not None:
        _ints("q_lens", q_lens, dev, B)
    if rope is None and not packed:
        if Q_new is not None or Q_out is not None:
            raise ValueError("Q_new and Q_out go with rope")
        _call("sa_cache_append", dev, stream, K_new.data_ptr(), V_new.data_ptr(), K_pages.data_ptr(), V_pages.data_ptr(),
              B, Hkv, m, d, page, num_pages, table[1], block_table.data_ptr(), seq_lens.data_ptr(), _ptr(q_lens), _DTYPE[dtype])
        return K_pages, V_pages
    cos_at = sin_at = None
    length = rot = Hq = 0
    if rope is not None:
        cos, sin = rope
        angles = cos.shape
        if not (len(angles) == 2 and sin.shape == angles and cos.dtype is torch.float32 and sin.dtype is torch.float32
                and cos.device == dev and sin.device == dev and cos.is_contiguous() and sin.is_contiguous()
                and angles[0] > 0 and angles[1] > 0 and angles[1] % 8 == 0 and 2 * angles[1] <= d):
            raise ValueError("rope must be two contiguous float32 tensors [positions, rot / 2] on the pools' device, rot a "
                             "multiple of 16 up to d")
        length, rot = min(angles[0], 0x7fffffff), 2 * angles[1]
        cos_at, sin_at = cos.data_ptr(), sin.data_ptr()
    if Q_new is not None:
        rows = Q_new.shape
        if rope is None:
            raise ValueError("Q_new and Q_out go with rope")
        if not (len(rows) == 4 and rows[0] == B and rows[2] == m and rows[3] == d and Q_new.dtype is dtype
                and Q_new.device == dev and Q_new.is_contiguous()):
            _new_rows("Q_new", Q_new, dtype, dev, d, None)
            raise ValueError("Q_new and K_new must have the same B and m")
        Hq = rows[1]
        if Q_out is None:
            Q_out = _new(tuple(rows), Q_new.stride(), dtype, dev, stream)
        elif Q_out.shape != rows or Q_out.dtype is not dtype or Q_out.device != dev or not Q_out.is_contiguous():
            raise ValueError("Q_out must be a contiguous CUDA tensor shaped and typed like Q_new")
    elif Q_out is not None:
        raise ValueError("Q_out goes with Q_new")
    _call("sa_cache_append_ex", dev, stream, K_new.data_ptr(), V_new.data_ptr(), _ptr(Q_new), _ptr(Q_out),
          K_pages.data_ptr(), V_pages.data_ptr(), B, Hq, Hkv, m, d, page, num_pages, table[1], block_table.data_ptr(),
          seq_lens.data_ptr(), _ptr(q_lens), cos_at, sin_at, length, rot, 1 if interleaved else 0, _DTYPE[dtype], packed)
    return (K_pages, V_pages) if Q_new is None else (K_pages, V_pages, Q_out)


def cache_read(K_pages, V_pages, block_table, seq_lens, m, q_lens=None, dtype=None, out=None, stream=None):
    """Keys and values of each sequence's last q_lens (None: m) tokens as rows [B, Hkv, m, d]; returns (K, V).

    Rows past q_lens and tokens whose page is missing are zeros. dtype: of the rows (the pages' own; bf16 or fp32, by
    default bf16, of uint8 pages held in 4 bits, exact in either). out: two tensors to write into.
    """
    pool, table, kind, dev = K_pages.shape, block_table.shape, K_pages.dtype, K_pages.device
    packed = kind is torch.uint8
    if not (len(pool) == 4 and V_pages.shape == pool and V_pages.dtype is kind
            and (kind in _DTYPE or packed and pool[3] in _HEAD_4BIT)
            and V_pages.device == dev and block_table.device == dev and seq_lens.device == dev and block_table.dtype is _INT
            and seq_lens.dtype is _INT and K_pages.is_cuda and K_pages.is_contiguous() and V_pages.is_contiguous()
            and block_table.is_contiguous() and seq_lens.is_contiguous() and len(table) == 2 and seq_lens.shape == table[:1]):
        _pools(K_pages, V_pages, (4,))
        _ints("block_table", block_table, dev, -1, -1)
        _ints("seq_lens", seq_lens, dev, table[0])
    num_pages, Hkv, page, d = pool
    if packed:
        d = _HEAD_4BIT[d]
    B = table[0]
    if dtype is None:
        dtype = torch.bfloat16 if packed else kind
    if dtype not in _DTYPE:
        raise TypeError(f"unsupported dtype {dtype}; use bfloat16 or float32")
    if not packed and dtype is not kind:
        raise ValueError("rows read from plain pages have the pages' dtype")
    if q_lens is not None:
        _ints("q_lens", q_lens, dev, B)
    if m < 1:
        raise ValueError("m must be positive")
    shape = (B, Hkv, m, d)
    if out is None:
        strides = (Hkv * m * d, m * d, d, 1)
        K, V = _new(shape, strides, dtype, dev, stream), _new(shape, strides, dtype, dev, stream)
    else:
        K, V = out
        for t in (K, V):
            if tuple(t.shape) != shape or t.dtype is not dtype or t.device != dev or not t.is_contiguous():
                raise ValueError("out must be two contiguous CUDA tensors [B, Hkv, m, d] of the rows' dtype")
    _call("sa_cache_read", dev, stream, K_pages.data_ptr(), V_pages.data_ptr(), K.data_ptr(), V.data_ptr(), B, Hkv, m, d,
          page, num_pages, table[1], block_table.data_ptr(), seq_lens.data_ptr(), _ptr(q_lens), _DTYPE[dtype], packed)
    return K, V


def _pool_args(K_pages, V_pages):
    """(layers, num_pages, bytes of a page of one layer, page) of pools of one layer or several."""
    _pools(K_pages, V_pages, (4, 5))
    num_pages, Hkv, page, row = K_pages.shape[-4:]
    layers = K_pages.shape[0] if K_pages.dim() == 5 else 1
    return layers, num_pages, Hkv * page * row * K_pages.element_size(), page


def _outputs(out, ins, stream):
    if out is None:
        if stream is None and _new_cuda is not None and torch._C._cuda_getDevice() == ins[0].get_device():
            return [_new_cuda(tuple(t.shape), t.stride(), _INT) for t in ins]
        return [_new(tuple(t.shape), t.stride(), _INT, t.device, stream) for t in ins]
    if len(out) != len(ins):
        raise ValueError(f"out must hold {len(ins)} tensors")
    for o, t in zip(out, ins):
        if o.dtype is not t.dtype or o.shape != t.shape or o.device != t.device or not o.is_contiguous():
            raise ValueError("out tensors must be contiguous and match the inputs in shape, dtype and device")
    return list(out)


def _book(block_table, ref_count, num_pages=None, device=None):
    dev = block_table.device
    if not block_table.is_cuda or (device is not None and dev != device):
        raise ValueError("block_table must be a CUDA tensor on the pools' device")
    _ints("block_table", block_table, dev, -1, -1)
    _ints("ref_count", ref_count, dev, -1 if num_pages is None else num_pages)
    return dev, block_table.shape[0], block_table.shape[1], ref_count.numel()


def cache_workspace_bytes(num_pages, B):
    """Scratch bytes of cache_fork, cache_reserve and cache_compact."""
    return _lib.lib().sa_cache_workspace_bytes(num_pages, B)


def cache_copy_pages(K_pages, V_pages, src, dst, stream=None):
    """Copy page src[i] to page dst[i] in every layer; returns (K_pages, V_pages). No page twice in dst, or in both."""
    layers, num_pages, page_bytes, _ = _pool_args(K_pages, V_pages)
    dev = K_pages.device
    _ints("src", src, dev, -1)
    _ints("dst", dst, dev, src.numel())
    _call("sa_cache_copy_pages", dev, stream, K_pages.data_ptr(), V_pages.data_ptr(), layers, num_pages, page_bytes,
          src.data_ptr(), dst.data_ptr(), src.numel())
    return K_pages, V_pages


def cache_fork(K_pages, V_pages, block_table, seq_lens, ref_count, src, dst, out=None, stream=None):
    """Rows dst[i] become copies of rows src[i]: whole pages shared, a partial last page copied.

    Returns (block_table, seq_lens, ref_count).
    """
    layers, num_pages, page_bytes, page = _pool_args(K_pages, V_pages)
    dev, B, max_pages, _ = _book(block_table, ref_count, num_pages, K_pages.device)
    _ints("seq_lens", seq_lens, dev, B)
    _ints("src", src, dev, -1)
    _ints("dst", dst, dev, src.numel())
    table, lens, refs = _outputs(out, (block_table, seq_lens, ref_count), stream)
    n_bytes = cache_workspace_bytes(num_pages, B)
    ws = _scratch(n_bytes, dev, stream)
    _call("sa_cache_fork", dev, stream, K_pages.data_ptr(), V_pages.data_ptr(), layers, num_pages, page_bytes, page, B,
          max_pages, src.data_ptr(), dst.data_ptr(), src.numel(), block_table.data_ptr(), seq_lens.data_ptr(),
          ref_count.data_ptr(), table.data_ptr(), lens.data_ptr(), refs.data_ptr(), _ptr(ws), n_bytes)
    return table, lens, refs


def cache_free(block_table, seq_lens, ref_count, rows, out=None, stream=None):
    """The rows give up their pages; returns (block_table, seq_lens, ref_count)."""
    dev, B, max_pages, num_pages = _book(block_table, ref_count)
    _ints("seq_lens", seq_lens, dev, B)
    _ints("rows", rows, dev, -1)
    table, lens, refs = _outputs(out, (block_table, seq_lens, ref_count), stream)
    _call("sa_cache_free", dev, stream, num_pages, B, max_pages, rows.data_ptr(), rows.numel(), block_table.data_ptr(),
          seq_lens.data_ptr(), ref_count.data_ptr(), table.data_ptr(), lens.data_ptr(), refs.data_ptr())
    return table, lens, refs


def cache_trim(block_table, seq_lens, ref_count, page, reach, global_idx=None, out=None, stream=None):
    """Rows give up the pages that the window (reach tokens back) has left; returns (block_table, ref_count)."""
    dev, B, max_pages, num_pages = _book(block_table, ref_count)
    _ints("seq_lens", seq_lens, dev, B)
    if global_idx is not None:
        _ints("global_idx", global_idx, dev, -1)
    n_global = 0 if global_idx is None else global_idx.numel()
    table, refs = _outputs(out, (block_table, ref_count), stream)
    _call("sa_cache_trim", dev, stream, num_pages, page, B, max_pages, min(reach, 0x7fffffff),
          global_idx.data_ptr() if n_global else None, n_global, block_table.data_ptr(), seq_lens.data_ptr(),
          ref_count.data_ptr(), table.data_ptr(), refs.data_ptr())
    return table, refs


def cache_reserve(block_table, seq_lens, q_lens, ref_count, page, out=None, stream=None):
    """Pages for the new tokens [seq_lens - q_lens, seq_lens) of every row; returns (block_table, ref_count)."""
    dev, B, max_pages, num_pages = _book(block_table, ref_count)
    _ints("seq_lens", seq_lens, dev, B)
    _ints("q_lens", q_lens, dev, B)
    table, refs = _outputs(out, (block_table, ref_count), stream)
    n_bytes = cache_workspace_bytes(num_pages, B)
    ws = _scratch(n_bytes, dev, stream)
    _call("sa_cache_reserve", dev, stream, num_pages, page, B, max_pages, seq_lens.data_ptr(), q_lens.data_ptr(),
          block_table.data_ptr(), ref_count.data_ptr(), table.data_ptr(), refs.data_ptr(), _ptr(ws), n_bytes)
    return table, refs


def cache_compact(K_pages, V_pages, block_table, ref_count, out=None, stream=None):
    """Leave the L pages in use at [0, L), in every layer; returns (block_table, ref_count)."""
    layers, num_pages, page_bytes, _ = _pool_args(K_pages, V_pages)
    dev, B, max_pages, _ = _book(block_table, ref_count, num_pages, K_pages.device)
    table, refs = _outputs(out, (block_table, ref_count), stream)
    n_bytes = cache_workspace_bytes(num_pages, B)
    ws = _scratch(n_bytes, dev, stream)
    _call("sa_cache_compact", dev, stream, K_pages.data_ptr(), V_pages.data_ptr(), layers, num_pages, page_bytes, B,
          max_pages, block_table.data_ptr(), ref_count.data_ptr(), table.data_ptr(), refs.data_ptr(), _ptr(ws),
          n_bytes)
    return table, refs
