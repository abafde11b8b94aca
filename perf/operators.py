"""Cases of the paged key/value cache: the attention of new tokens over it, writing new tokens into it, and moving its pages.

With ``own`` false ``run`` computes each operator in its plain form with
elementary torch operations; with ``own`` true it makes the calls a user makes
of the package. Both take what ``prepare`` gives.
"""

import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases
def _attend(name, **kw):
    c = dict(op="attend", B=1, Hq=12, Hkv=12, d=64, page=64, m=1, len=1024, ragged=False, window=0, n_global=0,
             dilated=False, dtype="bf16")
    c.update(kw)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one user, one token: Longformer's window and 16 global tokens; latency is all there is
        _attend("step, one sequence", len=1000, window=512, n_global=16),
        # one token for each of a batch of sequences of many lengths, every earlier token seen
        _attend("step, a batch", B=64, len=4096, ragged=True),
        # one token for each of a few long sequences, eight query heads to a key head
        _attend("step, long, grouped", B=16, Hq=32, Hkv=4, d=128, page=128, len=65536, ragged=True),
        # a step of a 32-bit model whose upper heads are dilated, in small pages
        _attend("step, 32 bits, dilated", B=8, len=2048, page=16, window=512, dilated=True, dtype="fp32"),
        # a few drafted tokens per sequence to be verified at once, some sequences with none
        _attend("drafted tokens", B=32, Hq=16, Hkv=4, d=128, page=32, m=5, len=8191, ragged=True),
        # a chunk of the character model's long sequences: 8 heads of 64, window 512, dilated heads
        _attend("chunk, window, dilated", B=4, Hq=8, Hkv=8, m=2048, len=23040, window=512, dilated=True),
        # a large chunk at the end of a long prompt, every earlier token seen
        _attend("chunk, long, grouped", Hq=16, Hkv=4, d=128, page=128, m=4096, len=32768),
        # a ragged chunk of a 32-bit model, window and global tokens
        _attend("chunk, 32 bits", B=2, m=300, len=1500, ragged=True, page=16, window=512, n_global=16, dtype="fp32"),
        # the new token's keys and values of one layer
        dict(name="append a step", op="append", B=64, Hkv=12, d=64, page=64, m=1, len=4096, ragged=True, dtype="bf16"),
        # a prompt's keys and values of one layer
        dict(name="append a chunk", op="append", B=4, Hkv=8, d=128, page=64, m=4096, len=8191, ragged=True, dtype="bf16"),
        # half of a batch forked for sampling: shared pages, an own last page in all 12 layers
        dict(name="fork", op="pages", do="fork", layers=12, pages=1024, Hkv=12, d=64, page=64, B=64, slots=64, n=32, dtype="bf16"),
        # a pool with holes after many sequences ended
        dict(name="compact", op="pages", do="compact", layers=4, pages=4096, Hkv=8, d=128, page=16, B=96, slots=64, n=0,
             dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(["attend", "attend", "attend", "append", "pages", "pages"])
        dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
        d, page = rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
        if op == "attend":
            hkv, group = rng.choice([1, 2, 4, 8, 12]), rng.choice([1, 1, 2, 3, 4, 8])
            m = rng.choice([1, 1, rng.randint(2, 9), _log(rng, 10, 4096)])
            ln = max(m, _log(rng, 40, 65536 if m < 10 else 32768))
            window = rng.choice([0, 2 * _log(rng, 16, 1024)])
            c = _attend("", B=_log(rng, 1, 64), Hq=hkv * group, Hkv=hkv, d=d, page=page, m=m, len=ln,
                        ragged=rng.random() < 0.7, window=window, n_global=rng.choice([0, 1, 16, 61]) if window else 0,
                        dilated=bool(window) and rng.random() < 0.3, dtype=dtype)
            # what the plain form holds: scores, and keys and values in 32 bits
            if c["B"] * c["Hq"] * m * ln > 2.2e9 or c["B"] * hkv * ln * d > 4.3e9:
                continue
            # 32-bit products run on the ordinary units: a smaller share of the largest case
            if work(c)["flops"] > (1.1e12 if dtype == "bf16" else 6e10) or work(c)["bytes"] > 2.5e9:
                continue
        elif op == "append":
            m = rng.choice([1, rng.randint(2, 9), _log(rng, 10, 8192)])
            c = dict(op="append", B=_log(rng, 1, 64), Hkv=rng.choice([1, 2, 4, 8, 12]), d=d, page=page, m=m,
                     len=max(m, _log(rng, 40, 16384)), ragged=rng.random() < 0.7, dtype=dtype)
            if c["B"] * c["Hkv"] * c["len"] * d > 5e8:
                continue
        else:
            B, slots = _log(rng, 4, 128), _log(rng, 8, 512)
            c = dict(op="pages", do=rng.choice(["copy", "fork", "free", "compact"]), layers=rng.randint(1, 12),
                     pages=_log(rng, 64, 8192), Hkv=rng.choice([1, 2, 4, 8, 12]), d=d, page=page, B=B, slots=slots,
                     n=_log(rng, 1, max(1, B // 2)), dtype=dtype)
            if c["do"] == "compact":
                c["n"] = 0
            if c["layers"] * c["pages"] * c["Hkv"] * page * d > 6.5e8:
                continue
        return c


# ------------------------------------------------------------------ what a case fixes: lengths, pattern, table
def _rng(case, salt):
    key = ",".join("%s=%s" % (k, case[k]) for k in sorted(case) if k not in ("name", "dtype"))
    return random.Random(key + salt)


def _lengths(case):
    """Tokens in the cache (new ones included) and new tokens of every sequence: fixed by the case."""
    r, B, m, ln = _rng(case, "lengths"), case["B"], case["m"], case["len"]
    if not case["ragged"]:
        return [ln] * B, [m] * B
    q = [m if m == 1 or i == 0 else r.randint(0, m) for i in range(B)]
    s = [ln if i == 0 else r.randint(max(q[i], ln // 8), ln) for i in range(B)]
    return s, q


def _pattern(case):
    """Half window, the heads' strides and the global positions (spread over the first sequence's length)."""
    half = case["window"] // 2 if case["window"] else case["len"]
    stride = [4 if case["dilated"] and h >= case["Hq"] - max(1, case["Hq"] // 4) else 1 for h in range(case["Hq"])]
    g, k = [], case["n_global"]
    if k:  # most at the front, as a prompt's first tokens; some further in
        front = max(1, 3 * k // 4)
        g = list(range(min(front, case["len"])))
        r = _rng(case, "global")
        rest = [j for j in range(len(g), case["len"])]
        g += r.sample(rest, min(len(rest), k - front))
    return half, stride, sorted(g)


def _rows_of(case):
    """Every new token's position, sequence by sequence."""
    s, q = _lengths(case)
    return [np.arange(a - b, a, dtype=np.int64) for a, b in zip(s, q)]


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "append":
        new = sum(_lengths(case)[1])
        return {"bytes": 4 * new * case["Hkv"] * case["d"] * e + 8 * case["B"], "flops": 0}
    if case["op"] == "pages":
        page = case["layers"] * case["Hkv"] * case["page"] * case["d"] * e
        table, refs, _, moved, _ = _pool(case)
        meta = 8 * (table.size + refs.size)
        if case["do"] == "copy":
            meta = 0
        return {"bytes": 4 * page * len(moved) + meta + 8 * case["n"], "flops": 0}
    half, stride, g = _pattern(case)
    g, d, group = np.asarray(g, dtype=np.int64), case["d"], case["Hq"] // case["Hkv"]
    pairs, keys, new = 0, 0, 0
    for p in _rows_of(case):
        new += len(p)
        if not len(p):
            continue
        glob = np.isin(p, g)
        for hk in range(case["Hkv"]):
            seen = 0
            for st in sorted(set(stride[hk * group:(hk + 1) * group])):
                n_h = sum(1 for x in stride[hk * group:(hk + 1) * group] if x == st)
                n = np.minimum(p // st, half) + 1
                for j in g.tolist():
                    gap = p - j
                    n += (gap >= 0) & ((gap % st != 0) | (gap // st > half))
                n[glob] = p[glob] + 1
                pairs += n_h * int(n.sum())
                lo = max(0, int(p[0]) - half * st)
                band = min(int(p[-1]) + 1 - lo, len(p) * (half + 1))
                if glob.any():
                    band = max(band, int(p[glob].max()) + 1)
                seen = max(seen, band + int((g < lo).sum()))
            keys += seen
    rows = new * case["Hq"]
    return {"bytes": 2 * keys * d * e + 2 * rows * d * e + 4 * sum(-(-s // case["page"]) for s in _lengths(case)[0]),
            "flops": 4 * d * pairs}


def _pool(case):
    """A pool in use, as numpy arrays: table, reference counts, lengths, the pages that move, and the rows or pages named."""
    r = np.random.RandomState(_rng(case, "pool").randrange(1 << 31))
    B, slots, P, page, do = case["B"], case["slots"], case["pages"], case["page"], case["do"]
    idle = case["n"] if do == "fork" else 0          # rows that a fork fills
    share = 0.4 if do == "compact" else 0.6          # of the pool in use
    want = r.randint(1, slots * page + 1, size=B)
    want[B - idle:] = 0
    need = -(-want // page)
    budget = max(B, int(share * P))
    if need.sum() > budget:                          # shorter sequences, so that they fit
        want = np.where(want > 0, np.maximum(1, (want * (budget / need.sum())).astype(np.int64)), 0)
        need = -(-want // page)
    order = r.permutation(P)
    table = np.full((B, slots), -1, dtype=np.int32)
    refs = np.zeros(P, dtype=np.int32)
    lens = np.zeros(B, dtype=np.int32)
    at = 0
    for b in range(B):
        k = int(need[b])
        if at + k > P:
            break
        table[b, :k] = order[at:at + k]
        lens[b] = want[b]
        at += k
        if b and k and lens[b - 1] and r.rand() < 0.3:  # a shared beginning
            c = min(k, int(lens[b - 1]) // page) // 2
            table[b, :c] = table[b - 1, :c]
    np.add.at(refs, table[table >= 0], 1)
    busy = np.nonzero(lens)[0]
    if do == "copy":
        live, free = np.nonzero(refs)[0], np.nonzero(refs == 0)[0]
        n = min(len(live), len(free), 8 * case["n"])
        src, dst = r.permutation(live)[:n].astype(np.int32), r.permutation(free)[:n].astype(np.int32)
        return table, refs, lens, src, (src, dst)
    if do == "fork":
        src = busy[r.randint(0, len(busy), size=idle)].astype(np.int32)
        dst = np.arange(B - idle, B, dtype=np.int32)
        return table, refs, lens, np.nonzero(lens[src] % page)[0][:int((refs == 0).sum())], (src, dst)
    if do == "free":
        return table, refs, lens, [], (r.permutation(B)[:case["n"]].astype(np.int32),)
    n_live = int((refs > 0).sum())
    return table, refs, lens, np.nonzero(refs[n_live:])[0], ()


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=dev, dtype=dt)

    st = {"case": dict(case)}
    if case["op"] == "pages":
        table, refs, lens, _, named = _pool(case)
        shape = (case["layers"], case["pages"], case["Hkv"], case["page"], case["d"])
        st.update(K=randn(*shape), V=randn(*shape), table=torch.from_numpy(table).to(dev),
                  refs=torch.from_numpy(refs).to(dev), lens=torch.from_numpy(lens).to(dev),
                  named=[torch.from_numpy(x).to(dev) for x in named])
        return st
    s, q = _lengths(case)
    B, Hkv, d, page, m = case["B"], case["Hkv"], case["d"], case["page"], case["m"]
    need = [-(-x // page) for x in s]
    P, width = sum(need) + 3, max(need)
    order = torch.randperm(P, generator=gen, device=dev).to(torch.int32)
    table = torch.full((B, width), -1, dtype=torch.int32, device=dev)
    lens = torch.tensor(s, device=dev)
    cols = torch.arange(width, device=dev)
    used = cols[None] < torch.tensor(need, device=dev)[:, None]
    table[used] = order[:sum(need)]
    K, V = randn(P, Hkv, page, d), randn(P, Hkv, page, d)
    if case["op"] == "attend":
        # what no token was written to holds anything at all
        last = table[torch.arange(B, device=dev), torch.tensor(need, device=dev) - 1].long()
        tail = torch.arange(page, device=dev)[None] >= (lens - (torch.tensor(need, device=dev) - 1) * page)[:, None]
        fill = tail[:, None, :, None]
        K[last] = torch.where(fill, torch.full((), float("nan"), dtype=dt, device=dev), K[last])
        V[last] = torch.where(fill, torch.full((), float("nan"), dtype=dt, device=dev), V[last])
        K[order[sum(need):].long()], V[order[sum(need):].long()] = float("nan"), float("nan")
        half, stride, g = _pattern(case)
        st.update(Q=randn(B, case["Hq"], m, d), window=2 * half,
                  gidx=torch.tensor(g, dtype=torch.int32, device=dev) if g else None,
                  dil=torch.tensor([x - 1 for x in stride], dtype=torch.int32, device=dev) if case["dilated"] else None)
    else:
        st.update(Kn=randn(B, Hkv, m, d), Vn=randn(B, Hkv, m, d))
    st.update(K=K, V=V, table=table, lens=lens.to(torch.int32), q=torch.tensor(q, dtype=torch.int32, device=dev))
    return st


# ------------------------------------------------------------------ plain forms
def _plain_attend(st):
    Q, K, V, table, dev = st["Q"], st["K"], st["V"], st["table"].long(), st["Q"].device
    B, Hq, m, d = Q.shape
    Hkv, page, half = K.shape[1], K.shape[2], st["window"] // 2
    L = table.shape[1] * page
    j = torch.arange(L, device=dev, dtype=torch.int32)
    lens, q = st["lens"], st["q"]
    there = (j[None] < lens[:, None]) & (table >= 0).repeat_interleave(page, 1)                    # [B, L]
    k, v = (x[table.clamp(min=0)].transpose(1, 2).reshape(B, Hkv, L, d).float() for x in (K, V))
    v = torch.where(there[:, None, :, None], v, 0.0)
    t = torch.arange(m, device=dev, dtype=torch.int32)
    p = (lens - q)[:, None] + t[None]                                                              # [B, m]
    gap = (p[:, :, None] - j[None, None])[:, None]                                                 # [B, 1, m, L]
    if st["dil"] is None:
        see = gap <= half
    else:
        s = (st["dil"] + 1)[None, :, None, None]
        see = (gap % s == 0) & (gap <= half * s)
    if st["gidx"] is not None:
        glob = torch.zeros(L + m, dtype=torch.bool, device=dev)
        glob[st["gidx"].long()] = True
        see = see | glob[:L][None, None, None] | glob[p.long()][:, None, :, None]
    see = see & (gap >= 0) & there[:, None, None] & (t[None] < q[:, None])[:, None, :, None]
    s = torch.matmul((Q.float() * (1.0 / math.sqrt(d))).reshape(B, Hkv, -1, d), k.transpose(2, 3)).reshape(B, Hq, m, L)
    s = s.masked_fill(~see, float("-inf"))
    top = s.amax(-1, keepdim=True)
    s = s.sub_(torch.where(top == float("-inf"), 0.0, top)).exp_()
    total = s.sum(-1, keepdim=True)
    o = torch.matmul(s.reshape(B, Hkv, -1, L), v).reshape(B, Hq, m, d)
    return (o / torch.where(total == 0, 1.0, total)).to(Q.dtype)


def _plain_append(st):
    Kn, K, V, table = st["Kn"], st["K"], st["V"], st["table"].long()
    B, Hkv, m, d = Kn.shape
    page = K.shape[2]
    t = torch.arange(m, device=Kn.device)
    p = (st["lens"] - st["q"])[:, None] + t[None]
    b, i = (t[None] < st["q"][:, None]).nonzero(as_tuple=True)
    at = p[b, i]
    pg = table[b, at // page]
    K[pg, :, at % page] = Kn[b, :, i]
    V[pg, :, at % page] = st["Vn"][b, :, i]
    return K, V


def _plain_pages(st):
    do, K, V, table, refs, lens = st["case"]["do"], st["K"], st["V"], st["table"], st["refs"], st["lens"]
    P, page = K.shape[1], K.shape[3]
    slots = torch.arange(table.shape[1], device=table.device)
    if do == "copy":
        src, dst = (x.long() for x in st["named"])
        K[:, dst], V[:, dst] = K[:, src], V[:, src]
        return K, V
    if do == "fork":
        src, dst = (x.long() for x in st["named"])
        n = lens[src]
        full, part = n // page, n % page > 0
        free = (refs == 0).nonzero()[:, 0]
        part_at = part.long().cumsum(0) - 1
        fits = ~part | (part_at < free.numel())
        own_page = free[part_at.clamp(min=0, max=max(0, free.numel() - 1))].to(torch.int32)
        rows = table[src]
        rows = torch.where(slots[None] < full[:, None], rows, -1)
        old = table[src, full.clamp(max=table.shape[1] - 1).long()].long()
        rows = torch.where(part[:, None] & (slots[None] == full[:, None]), own_page[:, None], rows)
        rows = torch.where(fits[:, None], rows, -1)
        table, refs, lens = table.clone(), refs.clone(), lens.clone()
        table[dst], lens[dst] = rows, torch.where(fits, n, 0)
        refs.index_add_(0, rows[rows >= 0].long(), torch.ones_like(rows[rows >= 0]))
        use = part & fits
        K[:, own_page[use].long()], V[:, own_page[use].long()] = K[:, old[use]], V[:, old[use]]
        return K, V, table, lens, refs
    if do == "free":
        rows = st["named"][0].long()
        gone = table[rows]
        table, refs, lens = table.clone(), refs.clone(), lens.clone()
        refs.index_add_(0, gone[gone >= 0].long(), -torch.ones_like(gone[gone >= 0]))
        table[rows], lens[rows] = -1, 0
        return table, lens, refs
    live = refs > 0
    n = live.sum()
    at = torch.arange(P, device=refs.device)
    movers, holes = (live & (at >= n)).nonzero()[:, 0], (~live & (at < n)).nonzero()[:, 0]
    K[:, holes], V[:, holes] = K[:, movers], V[:, movers]
    to = at.to(torch.int32)
    to[movers] = holes.to(torch.int32)
    out = torch.zeros_like(refs)
    out[to[live].long()] = refs[live]
    return K, V, torch.where(table >= 0, to[table.clamp(min=0).long()], table), out


def run(state):
    op = state["case"]["op"]
    if not own:
        return {"attend": _plain_attend, "append": _plain_append, "pages": _plain_pages}[op](state)
    import block_sparse_long_bigbird_gb300 as sa
    st = state
    if op == "attend":
        return sa.longformer_attn_paged_fwd(st["Q"], st["K"], st["V"], st["table"], st["lens"], st["window"],
                                            st["gidx"], dilation=st["dil"], q_lens=st["q"])
    if op == "append":
        return sa.cache_append(st["Kn"], st["Vn"], st["K"], st["V"], st["table"], st["lens"], q_lens=st["q"])
    do = st["case"]["do"]
    if do == "copy":
        return sa.cache_copy_pages(st["K"], st["V"], *st["named"])
    if do == "fork":
        return (st["K"], st["V"]) + tuple(sa.cache_fork(st["K"], st["V"], st["table"], st["lens"], st["refs"], *st["named"]))
    if do == "free":
        return sa.cache_free(st["table"], st["lens"], st["refs"], *st["named"])
    return (st["K"], st["V"]) + tuple(sa.cache_compact(st["K"], st["V"], st["table"], st["refs"]))


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    """Row by row from the definition: each new token's keys, their softmax and the weighted values, in float64.

    Moved and copied pages are not computed: their values have no 64-bit form.
    """
    if case["op"] != "attend":
        return None
    st = prepare(case, seed)
    s, q = _lengths(case)
    half, stride, g = _pattern(case)
    dev, d, page, group = st["Q"].device, case["d"], case["page"], case["Hq"] // case["Hkv"]
    out = torch.zeros(st["Q"].shape, dtype=torch.float64, device=dev)
    gset = torch.zeros(case["len"] + 1, dtype=torch.bool, device=dev)
    gset[torch.tensor(g, dtype=torch.long, device=dev)] = True
    for b, (n, new) in enumerate(zip(s, q)):
        if not new:
            continue
        ids = st["table"][b, : -(-n // page)].long()
        pos = torch.arange(n, device=dev)
        first = n - new
        for hk in range(case["Hkv"]):
            k, v = (x[ids, hk].reshape(-1, d)[:n].double() for x in (st["K"], st["V"]))
            for h in range(hk * group, (hk + 1) * group):
                for a in range(0, new, 1024):
                    z = min(new, a + 1024)
                    p = torch.arange(first + a, first + z, device=dev)
                    back = p[:, None] - pos[None, :]
                    ok = (torch.remainder(back, stride[h]) == 0) & (torch.div(back, stride[h], rounding_mode="floor") <= half)
                    ok = (ok | gset[pos][None, :] | gset[p][:, None]) & (back >= 0)
                    sc = (st["Q"][b, h, a:z].double() @ k.T) / math.sqrt(d)
                    out[b, h, a:z] = torch.softmax(torch.where(ok, sc, -math.inf), -1) @ v
    return out
