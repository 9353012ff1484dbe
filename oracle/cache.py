"""Paged 4-bit cache: tables, rounding and storage, attention over it.

Plain loops over requests, tokens and groups; numbers in float64 except where
the definition names float32 (y = x * (1 / g)).  The byte layout is built from
its definition with explicit offsets."""

import numpy as np

from .attention import softmax_attention

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def e4m3_value(byte):
    """Value of an E4M3 byte: sign, 4 exponent bits (bias 7), 3 mantissa bits; 0x7f / 0xff are NaN."""
    s, e, m = byte >> 7, (byte >> 3) & 15, byte & 7
    if e == 15 and m == 7:
        return float("nan")
    x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
    return -x if s else x


def _nearest(x, values):
    """Index of the value nearest to x >= 0 in an ascending list, ties to the even index, the last for larger x."""
    if x >= values[-1]:
        return len(values) - 1
    i = int(np.searchsorted(values, x, side="right")) - 1
    lo, hi = x - values[i], values[i + 1] - x
    if lo == hi:
        return i if i % 2 == 0 else i + 1
    return i if lo < hi else i + 1


_E4M3_POS = [e4m3_value(b) for b in range(127)]


def quantise_group(x, g=1.0):
    """16 channels x, head scale g -> (codes [16], scale byte)."""
    with np.errstate(all="ignore"):
        y = (np.float32(x) * (np.float32(1.0) / np.float32(g))).astype(np.float32).astype(np.float64)
    signs = np.signbit(y)
    if not np.all(np.isfinite(y)):
        return None, 0x7F
    byte = _nearest(float(np.max(np.abs(y))) / 6.0, _E4M3_POS)
    s = _E4M3_POS[byte]
    codes = np.array([_nearest(abs(v) / s, E2M1) if s > 0 else 0 for v in y], dtype=np.int64)
    return codes | (signs.astype(np.int64) << 3), byte


def code_value(code):
    x = E2M1[code & 7]
    return -x if code & 8 else x


def empty_cache(n_pages, H, P, D):
    return np.zeros((n_pages, H, P // 16, 18 * D), dtype=np.uint8)


def _offsets(D, j, c):
    """Offsets in a strip of token j's channel c: K byte, V byte, K scale, V scale."""
    return (j * (D // 2) + c // 2, 8 * D + ((c // 16) * 16 + j) * 8 + (c % 16) // 2,
            16 * D + j * (D // 16) + c // 16, 17 * D + (c // 16) * 16 + j)


def store(cache, slot, k, v, k_scale=None, v_scale=None):
    """Rounds one token's K and V rows [H, D] into its slot."""
    n_pages, H, strips, width = cache.shape
    D, P = width // 18, strips * 16
    page, j = slot // P, slot % 16
    for h in range(H):
        strip = cache[page, h, slot % P // 16]
        for which, x, g in ((0, k, k_scale), (1, v, v_scale)):
            for grp in range(D // 16):
                codes, byte = quantise_group(x[h, grp * 16:grp * 16 + 16], 1.0 if g is None else g[h])
                strip[_offsets(D, j, grp * 16)[2 + which]] = byte
                if codes is None:
                    continue
                for c in range(16):
                    at = _offsets(D, j, grp * 16 + c)[which]
                    shift = 4 * (c % 2)
                    strip[at] = (int(strip[at]) & (0xF0 >> shift)) | (int(codes[c]) << shift)


def load(cache, slot, k_scale=None, v_scale=None):
    """The K and V rows [H, D] that a slot holds."""
    n_pages, H, strips, width = cache.shape
    D, P = width // 18, strips * 16
    ch = np.arange(D)
    out = np.zeros((2, H, D))
    codes = np.array([code_value(c) for c in range(16)])
    scales = np.array([e4m3_value(b) for b in range(256)])
    for h in range(H):
        strip = cache[slot // P, h, slot % P // 16].astype(np.int64)
        offs = _offsets(D, slot % 16, ch)
        for which, g in ((0, k_scale), (1, v_scale)):
            b = strip[offs[which]] >> (4 * (ch % 2)) & 15
            out[which, h] = codes[b] * scales[strip[offs[2 + which]]] * (1.0 if g is None else float(g[h]))
    return out[0], out[1]


def cache_tables(old, new, P, table, pool, count, max_tokens, n_pages=None):
    """One step of the tables with the pool as a Python list used as a stack.
    Returns (ok, table, pool, count, query_start, req, pos, slots)."""
    R, max_pages = table.shape
    n_pages = len(pool) if n_pages is None else n_pages
    table, pool = table.copy(), np.array(pool).copy()
    fail = (False, table.copy(), pool.copy(), count, np.zeros(R + 1, np.int64), np.full(max_tokens, -1),
            np.full(max_tokens, -1), np.full(max_tokens, -1))
    if any(x < 0 or x > max_pages * P for x in list(old) + list(new)) or not 0 <= count <= n_pages:
        return fail
    stack = [int(x) for x in pool[:count]]
    pages = lambda n: -(-int(n) // P)  # noqa: E731
    for r in reversed(range(R)):
        for j in reversed(range(pages(new[r]), pages(old[r]))):
            stack.append(int(table[r, j]))
    for r in range(R):
        for j in range(pages(old[r]), pages(new[r])):
            if not stack:
                return fail
            table[r, j] = stack.pop()
    if len(stack) > n_pages:
        return fail
    start, req, pos, slots = [0], [], [], []
    for r in range(R):
        for p in range(int(old[r]), int(new[r])):
            req.append(r)
            pos.append(p)
            slots.append(int(table[r, p // P]) * P + p % P)
        start.append(len(req))
    if len(req) > max_tokens:
        return fail
    pool[count:len(stack)] = stack[count:]
    pad = [-1] * (max_tokens - len(req))
    return (True, table, pool, len(stack), np.array(start), np.array(req + pad, np.int64),
            np.array(pos + pad, np.int64), np.array(slots + pad, np.int64))


def cache_attention(q, cache, table, req, pos, k_scale=None, v_scale=None, block_indices=None, block_counts=None,
                    block_size=0, scale=None):
    """q [T, HQ, D] over the cache; rows of tokens with req < 0 come back as NaN (they are not part of the result)."""
    q = np.asarray(q, dtype=np.float64)
    T, HQ, D = q.shape
    n_pages, H, strips, _ = cache.shape
    P, G = strips * 16, HQ // H
    scale = D ** -0.5 if scale is None else scale
    o, lse = np.full((T, HQ, D), np.nan), np.full((T, HQ), np.nan)
    memo = {}

    def row(slot):
        if slot not in memo:
            memo[slot] = load(cache, slot, k_scale, v_scale)
        return memo[slot]

    for t in range(T):
        if req[t] < 0:
            continue
        for h in range(H):
            if block_indices is None:
                keys = list(range(int(pos[t]) + 1))
            else:
                keys = [int(b) * block_size + u for b in block_indices[t, h, :max(0, block_counts[t, h])]
                        for u in range(block_size)]
                keys = [x for x in keys if x <= pos[t]]
            kv = [row(int(table[req[t], x // P]) * P + x % P) for x in keys]
            K = np.array([a[h] for a, _ in kv]).reshape(len(keys), D)
            V = np.array([b[h] for _, b in kv]).reshape(len(keys), D)
            o[t, h * G:(h + 1) * G], lse[t, h * G:(h + 1) * G] = softmax_attention(
                q[t, h * G:(h + 1) * G], K, V, scale)
    return o, lse
