"""Plain 64-bit forms of the cache operators, one request and one token at a time, for the tests."""
import math

import numpy as np

TWO64 = 1 << 64


def tables(seq_len, new_len, table, free, count, bs, T, num_blocks, parent=None, words=0, max_tree=2049):
    R, mb = table.shape
    table = table.copy()
    cu, kv = [0], []
    slot, pos = np.full(T, -1, np.int64), np.full(T, -1, np.int32)
    mask = np.zeros((T, words), np.uint32)
    status = np.zeros(R, np.int32)
    count = min(max(count, 0), num_blocks)
    tokens, asked, taken = 0, 0, 0
    for r in range(R):
        L, n = int(seq_len[r]), int(new_len[r])
        bad = L < 0 or n < 0 or L + n > mb * bs or (parent is not None and (n > max_tree or n > 32 * words))
        held = 0 if bad else -(-L // bs)
        need = 0 if bad else -(-(L + n) // bs) - held
        t0, n = min(tokens, T), max(n, 0)
        tokens += n
        full = not bad and ((need > 0 and asked + need > count) or (n > 0 and tokens > T))
        first, asked = asked, asked + need
        cu.append(min(tokens, T))
        if bad or full:
            status[r] = 1024 if bad else 256
            kv.append(0)
            continue
        taken += need
        for i in range(need):
            table[r, held + i] = free[count - 1 - first - i]
        kv.append(L + n)
        depth = []
        for j in range(n):
            at = L + j
            b = int(table[r, at // bs])
            if 0 <= b < num_blocks:
                slot[t0 + j] = b * bs + at % bs
            else:
                status[r] |= 2048
            if parent is None:
                depth.append(j)
            else:
                p = int(parent[t0 + j])
                if p >= j or p < -1:
                    status[r] |= 512
                    p = -1
                depth.append(0 if p < 0 else depth[p] + 1)
                if p >= 0:
                    mask[t0 + j] = mask[t0 + p]
                mask[t0 + j, j // 32] |= np.uint32(1 << (j % 32))
            pos[t0 + j] = L + depth[j]
    return dict(cu_tokens=np.array(cu, np.int32), kv_len=np.array(kv, np.int32), slot=slot, position=pos,
                mask=mask.view(np.int32), block_table=table, free_count=np.array([count - taken], np.int32),
                status=status)


def turns(freqs, position):
    """Angles [T, pairs] in radians, the 64-bit product taken in whole numbers."""
    out = np.zeros((len(position), len(freqs)))
    for t, p in enumerate(position):
        for i, f in enumerate(freqs):
            out[t, i] = (int(p) * (int(f) % TWO64) % TWO64) / TWO64
    return out * (2 * math.pi)


def rotate(x, ang, interleaved, mscale):
    """x [T, heads, D] in fp64."""
    half = ang.shape[1]
    y = x.copy()
    first = np.arange(half) * (2 if interleaved else 1)
    second = first + (1 if interleaved else half)
    c, s = mscale * np.cos(ang)[:, None, :], mscale * np.sin(ang)[:, None, :]
    y[..., first] = x[..., first] * c - x[..., second] * s
    y[..., second] = x[..., first] * s + x[..., second] * c
    return y


def visible(i, n, ctx, kv, mask_row):
    """Positions that the request's token i sees: those before its n step tokens, and of those the chosen ones."""
    x = np.arange(kv)
    j = x - ctx
    if mask_row is None:
        new = j <= i
    else:
        words = mask_row.view(np.uint32)
        inside = (j >= 0) & (j < 32 * len(words))
        jj = np.where(inside, j, 0)
        new = inside & ((words[jj // 32] >> (jj % 32).astype(np.uint32)) & 1).astype(bool)
    return (j < 0) | ((j < n) & new)


def attention(q, K, V, ctx, n, scale, mask):
    """One request: q [n, Hq, D], K and V [kv, Hk, D], mask [n, words] int32 or None.  Returns out, lse and for the
    error bounds sum p |v| [n, Hq, D] and max over visible x of scale sum |q| |k_x| [n, Hq]."""
    Hq, Hk, kv = q.shape[1], K.shape[1], K.shape[0]
    out = np.zeros(q.shape)
    spread = np.zeros(q.shape)
    lse = np.full(q.shape[:2], -np.inf)
    reach = np.zeros(q.shape[:2])
    for i in range(q.shape[0]):
        see = visible(i, n, ctx, kv, None if mask is None else mask[i])
        if not see.any():
            continue
        for h in range(Hq):
            k, v = K[see, h * Hk // Hq], V[see, h * Hk // Hq]
            s = scale * (k @ q[i, h])
            top = s.max()
            e = np.exp(s - top)
            tot = e.sum()
            out[i, h] = (e / tot) @ v
            spread[i, h] = (e / tot) @ np.abs(v)
            lse[i, h] = top + np.log(tot)
            reach[i, h] = abs(scale) * (np.abs(k) @ np.abs(q[i, h])).max()
    return out, lse, spread, reach


def commit(kc, vc, table, seq_len, kv_len, cu, accept, k, free, count, branch=None, path=None):
    """kc, vc [layers, blocks, bs, heads, D]; changed copies come back."""
    kc, vc, free = kc.copy(), vc.copy(), free.copy()
    bs, R = kc.shape[2], len(seq_len)
    seq, status = np.array(seq_len, np.int32).copy(), np.zeros(R, np.int32)
    top = int(count)
    old = kc.copy(), vc.copy()
    for r in range(R):
        L, n = int(seq_len[r]), int(cu[r + 1] - cu[r])
        if L < 0 or n <= 0 or L + n != int(kv_len[r]):
            continue
        a, last = min(max(int(accept[r]), 0), k), 0
        for i in range(a):
            x = int(path[r, i]) if path is not None else 1 + (int(branch[r]) if branch is not None else 0) * k + i
            if x <= last or x >= n:
                status[r] = 512
                a = i
                break
            for c, o in zip((kc, vc), old):
                c[:, table[r, (L + 1 + i) // bs], (L + 1 + i) % bs] = o[:, table[r, (L + x) // bs], (L + x) % bs]
            last = x
        seq[r] = L + 1 + a
        for b in range(-(-int(seq[r]) // bs), -(-int(kv_len[r]) // bs)):
            free[top] = table[r, b]
            top += 1
    return dict(k=kc, v=vc, seq_len=seq, free=free, free_count=np.array([top], np.int32), status=status)
