"""Plain 64-bit forms of the 8-bit paged KV cache's operators (numpy), written
from their definitions in include/idx.h."""

import numpy as np

QMAX = {"e4m3": 448.0, "int8": 127.0}
MIN_SCALE = 2.0 ** -100


def _e4m3_table():
    out = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = (m / 8.0) * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7)
        if (c & 127) == 127:
            x = np.nan
        out[c] = -x if c & 128 else x
    return out


E4M3 = _e4m3_table()
_POS = E4M3[:127]  # the finite magnitudes, rising with their code


def decode(codes, fmt):
    """Codes (uint8) as the numbers they are, in units of the scale."""
    return E4M3[codes] if fmt == "e4m3" else codes.view(np.int8).astype(np.float64)


def encode(x, fmt):
    """Numbers in units of the scale as codes: nearest, ties to even, saturated."""
    x = np.asarray(x, np.float64)
    if fmt == "int8":
        r = np.rint(np.clip(np.nan_to_num(x, nan=0.0, posinf=127.0, neginf=-127.0), -127, 127))
        return r.astype(np.int8).view(np.uint8)
    a = np.minimum(np.abs(np.nan_to_num(x, nan=0.0, posinf=448.0, neginf=-448.0)), 448.0)
    hi = np.searchsorted(_POS, a)  # first magnitude >= a
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _POS[lo], _POS[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi).astype(np.uint8)
    code = code | np.where(np.signbit(x), 128, 0)
    return np.where(np.isnan(x), 127, code).astype(np.uint8)  # one NaN code, without a sign


def scale_for(amax, fmt):
    s = MIN_SCALE
    while QMAX[fmt] * s < amax:
        s *= 2
    return s


def block_tables(cached, fresh, T, P, N, table, n_blocks, free, head):
    """(table, slots, key_counts, page_counts, head_out) in order of requests."""
    B = len(cached)
    table = table.copy()
    slots = np.full((B, T), -1, np.int32)
    keys = np.zeros((B, T), np.int32)
    at = head
    for b in range(B):
        have, want = -(-int(cached[b]) // P), -(-(int(cached[b]) + int(fresh[b])) // P)
        for j in range(have, want):
            ok = at < len(free) and 0 <= free[at] < n_blocks
            table[b, j] = free[at] if ok else -1
            at += 1
        for t in range(int(fresh[b])):
            pos = int(cached[b]) + t
            block = table[b, pos // P]
            if 0 <= block < n_blocks:
                slots[b, t] = block * P + pos % P
                keys[b, t] = pos + 1
    return table, slots, keys, -(-keys // P), min(at, len(free))


def append(x, slots, codes, scales, fmt):
    """(codes, scales) after rows x [R][H][D] (float64) went to their slots."""
    codes, scales = codes.copy(), scales.copy()
    n, H, P, D = codes.shape
    t, R = 0, len(slots)
    while t < R:
        if not 0 <= slots[t] < n * P:
            t += 1
            continue
        page, row = divmod(int(slots[t]), P)
        rows = 1
        while row + rows < P and t + rows < R and slots[t + rows] == slots[t] + rows:
            rows += 1
        for h in range(H):
            part = x[t:t + rows, h]
            fin = part[np.isfinite(part)]
            s = scale_for(np.abs(fin).max() if fin.size else 0.0, fmt)
            old = float(scales[page, h])
            if row and old >= s:
                s = old
            elif row:
                codes[page, h, :row] = encode(decode(codes[page, h, :row], fmt) * np.float64(
                    np.float32(old) / np.float32(s)), fmt)
            codes[page, h, row:row + rows] = encode(part / s, fmt)
            scales[page, h] = s
        t += rows
    return codes, scales


def attention(q, kcodes, vcodes, ks, vs, table, counts, page_idx, scale, fmt):
    """(out, lse, A, ds, top): A = sum_i p_i |v_i|; ds bounds how far fp32 scores are off, see
    tolerance(); top = n * max_i p_i * vscale_i * QMAX, what fp16 weights next to zero lose by."""
    B, T, Q, D = q.shape
    n, H, P, _ = kcodes.shape
    G = Q // H
    out = np.zeros((B, T, Q, D))
    A = np.zeros((B, T, Q, D))
    lse = np.full((B, T, Q), -np.inf)
    ds = np.zeros((B, T, Q, 1))
    top = np.zeros((B, T, Q, 1))
    N = table.shape[1]
    for b in range(B):
        for t in range(T):
            c = int(min(max(counts[b, t], 0), N * P))
            pages = range(-(-c // P)) if page_idx is None else page_idx[b * T + t]
            cells = [(table[b, p], p, min(P, c - p * P)) for p in pages
                     if 0 <= p < N and p * P < c and 0 <= table[b, p] < n]
            if not cells:
                continue
            for h in range(H):
                k = np.concatenate([decode(kcodes[i, h, :m], fmt) * float(ks[i, h]) for i, _, m in cells])
                v = np.concatenate([decode(vcodes[i, h, :m], fmt) * float(vs[i, h]) for i, _, m in cells])
                w = np.concatenate([np.full(m, float(vs[i, h])) for i, _, m in cells])
                for g in range(h * G, (h + 1) * G):
                    s = (k @ q[b, t, g]) * scale
                    sabs = (np.abs(k) @ np.abs(q[b, t, g])) * abs(scale)
                    m = s.max()
                    p = np.exp(s - m)
                    l = p.sum()
                    p /= l
                    out[b, t, g] = p @ v
                    A[b, t, g] = p @ np.abs(v)
                    lse[b, t, g] = m + np.log(l)
                    # products exact, D/1 fp32 additions, then the scales and the exponent's
                    # argument: a few roundings of |s| and of the largest |s - m|
                    ds[b, t, g] = 2.0 ** -24 * ((D + 8) * sabs.max() + 8 * np.abs(s).max() + 8)
                    top[b, t, g] = len(p) * (p * w).max() * QMAX[fmt]
    return out, lse, A, ds, top


def tolerance(out, A, ds, top, keys):
    """bf16's half step of the result; the weights' fp16 half step (2^-11, 2^-25 below its
    normal range), twice the scores' error (weights and their sum), fp32 sums over the keys."""
    return 2.0 ** -8 * np.abs(out) + A * (2.0 ** -11 + 2 * ds + 2.0 ** -23 * (keys + 64)) \
        + 2.0 ** -25 * top + 1e-37
