"""Plain 64-bit references of the serving operators, written from their
formulas in include/sq.h (numpy, one token or one request at a time)."""
import numpy as np


def prefill(q, k, v, alpha, beta, cu, S0, delta):
    """torch tensors q, k [N][Hk][dk], v [N][H][dv], alpha, beta [N][H], S0 [n][H][dk][dv] or None."""
    q, k, v, alpha, beta = (x.numpy().astype(np.float64) for x in (q, k, v, alpha, beta))
    n, H, dk, dv = len(cu) - 1, v.shape[1], q.shape[2], v.shape[2]
    rep = H // q.shape[1]
    q, k = np.repeat(q, rep, axis=1), np.repeat(k, rep, axis=1)
    S = np.zeros((n, H, dk, dv)) if S0 is None else S0.numpy().astype(np.float64)
    o = np.zeros(v.shape)
    for s in range(n):
        R = S[s]
        for t in range(cu[s], cu[s + 1]):
            a, b = alpha[t][:, None], beta[t][:, None]
            w = b * v[t]
            if delta:
                w = b * (v[t] - a * np.einsum("hi,hij->hj", k[t], R))
            R = a[..., None] * R + k[t][:, :, None] * w[:, None, :]
            o[t] = np.einsum("hi,hij->hj", q[t], R)
        S[s] = R
    return o, S


def attention(q, kc, vc, table, lens, scale, window):
    """kc [pages][Hkv][P][d], vc [pages][Hkv][d][P]; returns o, lse and
    sum_x p_x |v_x| (the size that rounding errors go by)."""
    q, kc, vc = (np.asarray(x, np.float64) for x in (q, kc, vc))
    n, H, d = q.shape
    pages, hkv, P = kc.shape[:3]
    o, mag, lse = np.zeros((n, H, d)), np.zeros((n, H, d)), np.full((n, H), -np.inf)
    for r in range(n):
        first = max(0, lens[r] - window) if window else 0
        pos = [x for x in range(first, lens[r]) if 0 <= table[r][x // P] < pages]
        if not pos:
            continue
        ids = np.array([table[r][x // P] for x in pos])
        off = np.array([x % P for x in pos])
        for h in range(H):
            kv = h // (H // hkv)
            x = scale * (kc[ids, kv, off] @ q[r, h])
            top = x.max()
            p = np.exp(x - top)
            lse[r, h] = top + np.log(p.sum())
            p /= p.sum()
            o[r, h] = p @ vc[ids, kv, :, off]
            mag[r, h] = p @ np.abs(vc[ids, kv, :, off])
    return o, lse, mag


def block_tables(ctx, new, P, free, table, capacity):
    """Returns table, seq, cu_new, cu_pages, slots, result."""
    table, n_free, stride = np.array(table), len(free), np.shape(table)[1]
    seq, cu_new, cu_pages, slots, flag = [], [0], [0], [], 0
    for i, (c, m) in enumerate(zip(ctx, new)):
        if c < 0 or m < 0 or c + m > 2 ** 31 - 1:
            c = m = 0
            flag |= 1
        held, total = -(-c // P), -(-(c + m) // P)
        for p in range(held, total):
            j = cu_pages[-1] + p - held
            if p < stride:
                table[i][p] = free[j] if j < n_free else -1
        if total > stride:
            flag |= 4
        for x in range(c, c + m):
            page = table[i][x // P] if x // P < stride else -1
            slots.append(page * P + x % P if page >= 0 else -1)
        seq.append(c + m)
        cu_new.append(cu_new[-1] + m)
        cu_pages.append(cu_pages[-1] + total - held)
    if cu_pages[-1] > n_free:
        flag |= 2
    if len(slots) > capacity:
        flag |= 8
    slots = (slots + [-1] * capacity)[:capacity]
    return table, np.array(seq, int), np.array(cu_new), np.array(cu_pages), np.array(slots, np.int64), flag
