"""Plain 64-bit forms of the operators at the two ends of a verify step, one row and one token at a time, for the tests."""
import numpy as np

from tests import cache_plain as plain

ST_RANGE, ST_NO_BLOCKS, ST_LENGTH, ST_BLOCK, ST_PENALTY, ST_MASK, ST_SOURCE = 1, 256, 1024, 2048, 4096, 8192, 16384


def _overflow(z):
    """Values whose rounding to fp32 is infinite."""
    return np.where(np.abs(z) >= 2.0 ** 128 - 2.0 ** 103, np.copysign(np.inf, z), z)


def adjust(z, R, k, branches, draft, history=None, history_len=None, prompt_len=None, repetition=None, presence=None,
           frequency=None, bias=None, mask=None, mask_row=None):
    """z [rows, V] in fp64: the adjusted rows, the bound of fp32's roundings on the way there and the status."""
    n, V = 1 + branches * k, z.shape[1]
    z, err, status = z.copy(), np.zeros(z.shape), np.zeros(R, np.int32)
    for r in range(R):
        said, seen = np.zeros(V, np.int64), np.zeros(V, bool)

        def inside(tokens):
            tokens = np.asarray(tokens, np.int64)
            ok = (tokens >= 0) & (tokens < V)
            if not ok.all():
                status[r] |= ST_RANGE
            return tokens[ok]

        if history is not None:
            width, given = history.shape[1], int(history_len[r])
            L = min(max(given, 0), width)
            p = 0 if prompt_len is None else int(prompt_len[r])
            P = min(max(p, 0), L)
            if L != given or P != p:
                status[r] |= ST_LENGTH
            seen[inside(history[r, :P])] = True
            np.add.at(said, inside(history[r, P:L]), 1)
        rep, pres, freq = (1.0 if x is None and i == 0 else 0.0 if x is None else float(x[r])
                           for i, x in enumerate((repetition, presence, frequency)))
        if not (0 < rep < np.inf):
            rep, status[r] = 1.0, status[r] | ST_PENALTY
        if not np.isfinite(pres):
            pres, status[r] = 0.0, status[r] | ST_PENALTY
        if not np.isfinite(freq):
            freq, status[r] = 0.0, status[r] | ST_PENALTY
        add, has = np.zeros(V), np.zeros(V, bool)
        if bias is not None:
            start, ids, values = bias
            m = len(ids)
            if m:
                b0 = min(max(int(start[r]), 0), m)
                b1 = min(max(int(start[r + 1]), b0), m)
                if b0 != start[r] or b1 != start[r + 1]:
                    status[r] |= ST_LENGTH
                inside(ids[b0:b1])
                for x, v in zip(ids[b0:b1], values[b0:b1]):
                    if 0 <= x < V:
                        add[x], has[x] = v, True
        way = [np.asarray(draft[r, b], np.int64) for b in range(branches)] if k else []
        for w in way:
            inside(w)
        for j in range(n):
            b, i = divmod(j - 1, k) if j else (0, -1)
            count = said.copy()
            if j:
                w = way[b][: i + 1]
                np.add.at(count, w[(w >= 0) & (w < V)], 1)
            row = z[r * n + j]
            met = seen | (count > 0)
            z1 = _overflow(np.where(met, np.where(row > 0, row / rep, row * rep), row))
            pen = np.where(count > 0, pres + freq * count, 0.0)
            size = np.where(count > 0, abs(pres) + abs(freq) * count, 0.0)
            z2 = _overflow(np.where(count > 0, z1 - pen, z1))
            z3 = _overflow(np.where(has, z2 + add, z2))
            # a rounding of each step, of the product and of the sum in the penalty
            with np.errstate(invalid="ignore"):
                e = 2.0 ** -24 * (np.where(met, np.abs(z1), 0) + 2 * size + np.where(count > 0, np.abs(z2), 0)
                                  + np.where(has, np.abs(z3), 0))
            if mask is not None:
                m = r * n + j if mask_row is None else int(mask_row[r * n + j])
                if m >= len(mask):
                    status[r] |= ST_MASK
                elif m >= 0:
                    words = mask[m].view(np.uint32)
                    x = np.arange(V)
                    ok = ((words[x // 32] >> (x % 32).astype(np.uint32)) & 1).astype(bool)
                    z3 = np.where(ok, z3, -np.inf)
            z[r * n + j], err[r * n + j] = z3, np.where(np.isfinite(z3), e, 0)
    return z, err, status


def norm_rope(x, weight, eps, ang, interleaved, mscale):
    """x [T, heads, D] in fp64: the normed heads, and the normed and rotated ones."""
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    if weight is not None:
        y = y * weight
    return y, plain.rotate(y, ang, interleaved, mscale)


def held(table, seq_len, bs):
    """The entries that each row holds, and its status: a length above the table holds all of it."""
    rows, status = [], np.zeros(len(seq_len), np.int32)
    for r, L in enumerate(int(x) for x in seq_len):
        room = table.shape[1] * bs
        if not 0 <= L <= room:
            status[r] = ST_LENGTH
        rows.append([int(x) for x in table[r, : -(-min(max(L, 0), room) // bs)]])
    return rows, status


def fork(kc, vc, table, seq_len, source, free, count):
    """kc, vc [layers, blocks, bs, heads, D]; changed copies come back."""
    kc, vc, table = kc.copy(), vc.copy(), table.copy()
    N, bs, R = kc.shape[1], kc.shape[2], len(seq_len)
    room = table.shape[1] * bs
    old, seq, status = table.copy(), np.array(seq_len, np.int32).copy(), np.zeros(R, np.int32)
    count = min(max(int(count), 0), N)
    asked = 0
    for r in range(R):
        s, own = int(source[r]), int(seq_len[r])
        if not 0 <= own <= room:
            status[r] |= ST_LENGTH
        if s < 0:
            continue
        if s >= R or own != 0:
            status[r] |= ST_SOURCE
            continue
        L = int(seq_len[s])
        if not 0 <= L <= room:
            status[r] |= ST_LENGTH
            continue
        full, tail = divmod(L, bs)
        if tail:
            asked += 1
            if asked > count:
                status[r] |= ST_NO_BLOCKS
                continue
        table[r, :full] = old[s, :full]
        bad = ((old[s, :full] < 0) | (old[s, :full] >= N)).any()
        if tail:
            a, b = int(old[s, full]), int(free[count - asked])
            table[r, full] = b
            if 0 <= a < N and 0 <= b < N:
                for c in (kc, vc):
                    c[:, b, :tail] = c[:, a, :tail]
            else:
                bad = True
        status[r] |= ST_BLOCK if bad else 0
        seq[r] = L
    return dict(k=kc, v=vc, block_table=table, seq_len=seq, free_count=np.array([max(count - asked, 0)], np.int32),
                status=status)


def free_rows(table, seq_len, leave, free, count, bs, N):
    rows, status = held(table, seq_len, bs)
    count = min(max(int(count), 0), N)
    stay = {int(x) for x in free[:count]}
    gone, seq, free = set(), np.array(seq_len, np.int32).copy(), free.copy()
    for r, ids in enumerate(rows):
        leaves, bad = leave[r] != 0, status[r] != 0
        if bad and leaves:
            continue
        status[r] |= ST_BLOCK if any(not 0 <= x < N for x in ids) else 0
        (gone if leaves else stay).update(x for x in ids if 0 <= x < N)
        if leaves:
            seq[r] = 0
    new = sorted(gone - stay)[: N - count]
    free[count:count + len(new)] = new
    return dict(free_blocks=free, free_count=np.array([count + len(new)], np.int32), seq_len=seq, status=status)


def compact(kc, vc, table, seq_len):
    kc, vc = kc.copy(), vc.copy()
    N, bs = kc.shape[1], kc.shape[2]
    rows, status = held(table, seq_len, bs)
    used = sorted({x for ids in rows for x in ids if 0 <= x < N})
    U = len(used)
    move = dict(zip([x for x in used if x >= U], sorted(set(range(U)) - set(used))))
    for c in (kc, vc):
        o = c.copy()
        for a, b in move.items():
            c[:, b] = o[:, a]
    out = np.full(table.shape, -1, np.int32)
    for r, ids in enumerate(rows):
        status[r] |= ST_BLOCK if any(not 0 <= x < N for x in ids) else 0
        out[r, : len(ids)] = [move.get(x, x) for x in ids]
    free = np.full(N, -1, np.int32)
    free[: N - U] = np.arange(N - 1, U - 1, -1)
    return dict(k=kc, v=vc, block_table=out, free_blocks=free, free_count=np.array([N - U], np.int32), status=status)
