"""Float64 oracle of the paged cache: attention row by row from the definition,
and the bookkeeping of pages as plain Python over lists."""

import numpy as np


def visible_keys(p, n_keys, half, stride, global_set, have):
    """Positions that the token at position p sees: earlier ones in its (dilated) window, global ones, all if p is global."""
    keys = []
    for j in range(min(p, n_keys - 1) + 1):
        if not have[j]:
            continue
        if j in global_set or p in global_set or ((p - j) % stride == 0 and (p - j) // stride <= half):
            keys.append(j)
    return keys


def oracle_paged(Q, K, V, table, lens, q_lens, window, global_idx=(), dilation=None):
    """O, and per element the sum of weight x |value| and per row the largest sum |q k| / sqrt(d) (for error bounds).

    Q [B, Hq, m, d], K and V [P, Hkv, page, d], numpy; table [B, max_pages]."""
    Q, K, V = (np.asarray(x, dtype=np.float64) for x in (Q, K, V))
    B, Hq, m, d = Q.shape
    P, Hkv, page, _ = K.shape
    group = Hq // Hkv
    gset = set(int(g) for g in global_idx)
    O, A, S = np.zeros_like(Q), np.zeros_like(Q), np.zeros(Q.shape[:3])
    for b in range(B):
        n = int(lens[b])
        nq = m if q_lens is None else int(q_lens[b])
        have = [table[b][j // page] >= 0 for j in range(n)]
        for hk in range(Hkv):
            k, v = np.zeros((n, d)), np.zeros((n, d))
            for j in range(n):
                if have[j]:
                    k[j], v[j] = K[table[b][j // page], hk, j % page], V[table[b][j // page], hk, j % page]
            for h in range(hk * group, (hk + 1) * group):
                stride = 1 if dilation is None else int(dilation[h]) + 1
                for t in range(nq):
                    keys = visible_keys(n - nq + t, n, window // 2, stride, gset, have)
                    if not keys:
                        continue
                    s = k[keys] @ Q[b, h, t] / np.sqrt(d)
                    w = np.exp(s - s.max())
                    w /= w.sum()
                    O[b, h, t] = w @ v[keys]
                    A[b, h, t] = w @ np.abs(v[keys])
                    S[b, h, t] = (np.abs(k[keys]) @ np.abs(Q[b, h, t])).max() / np.sqrt(d)
    return O, A, S


def append(K_new, V_new, K, V, table, lens, q_lens):
    """K, V (copies) with the new tokens written."""
    K, V = K.copy(), V.copy()
    page = K.shape[2]
    for b in range(K_new.shape[0]):
        nq = K_new.shape[2] if q_lens is None else int(q_lens[b])
        for t in range(nq):
            pos = int(lens[b]) - nq + t
            pg = int(table[b][pos // page])
            if 0 <= pg < K.shape[0]:
                K[pg, :, pos % page] = K_new[b, :, t]
                V[pg, :, pos % page] = V_new[b, :, t]
    return K, V


def fork(table, lens, refs, page, src, dst):
    """(table, lens, refs, moves): moves are (from, to) pages whose data is copied."""
    t0, l0 = [list(map(int, r)) for r in table], list(map(int, lens))
    table, lens, refs = [list(r) for r in t0], list(l0), list(map(int, refs))
    B, width = len(t0), len(t0[0])
    free = [i for i, c in enumerate(refs) if c == 0]
    moves, taken = [], set()
    dsts = set(d for d in dst if 0 <= d < B)
    for s, d in zip(src, dst):
        if not (0 <= s < B and 0 <= d < B) or s in dsts or l0[d] != 0 or d in taken:
            taken.add(d)
            continue
        taken.add(d)
        full, part = divmod(l0[s], page)
        row = t0[s][:full] + [-1] * (width - full)
        if part and t0[s][full] >= 0:
            if not free:
                continue
            row[full] = free.pop(0)
            moves.append((t0[s][full], row[full]))
        for old in t0[d]:
            if old >= 0:
                refs[old] -= 1
        for pg in row:
            if pg >= 0:
                refs[pg] += 1
        table[d], lens[d] = row, l0[s]
    return table, lens, refs, moves


def free_rows(table, lens, refs, rows):
    table, lens, refs = [list(map(int, r)) for r in table], list(map(int, lens)), list(map(int, refs))
    for b in set(r for r in rows if 0 <= r < len(table)):
        for pg in table[b]:
            if pg >= 0:
                refs[pg] = max(0, refs[pg] - 1)
        table[b], lens[b] = [-1] * len(table[b]), 0
    return table, lens, refs


def trim(table, lens, refs, page, reach, global_idx=()):
    table, refs = [list(map(int, r)) for r in table], list(map(int, refs))
    for b, n in enumerate(lens):
        n = int(n)
        if any(g >= n for g in global_idx):
            continue
        for c, pg in enumerate(table[b]):
            tokens = range(c * page, (c + 1) * page)
            if pg >= 0 and tokens[-1] < n - reach and not any(g in tokens for g in global_idx):
                refs[pg] -= 1
                table[b][c] = -1
    return table, refs


def reserve(table, lens, q_lens, refs, page):
    table, refs = [list(map(int, r)) for r in table], list(map(int, refs))
    free = [i for i, c in enumerate(refs) if c == 0]
    for b, (n, nq) in enumerate(zip(lens, q_lens)):
        for c in range(-(-(int(n) - int(nq)) // page), -(-int(n) // page)):
            if table[b][c] < 0 and free:
                table[b][c] = free.pop(0)
                refs[table[b][c]] = 1
    return table, refs


def compact(table, refs):
    """(table, refs, moves)."""
    refs = list(map(int, refs))
    live = [i for i, c in enumerate(refs) if c > 0]
    L = len(live)
    moves = list(zip([i for i in live if i >= L], [i for i in range(L) if refs[i] == 0]))
    to = dict(moves)
    new = list(refs)
    for a, b in moves:
        new[b], new[a] = refs[a], 0
    return [[to.get(int(v), int(v)) for v in r] for r in table], new, moves
