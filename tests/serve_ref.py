"""Plain 64-bit forms of the drafted-token verification operators (test
infrastructure, numpy only; nothing here is shared with the library)."""
import numpy as np


def unpack_codes(codes: np.ndarray, K: int) -> np.ndarray:
    """[N, K] codes of uint8 [N, ceil(K/2)] (k = 2j in byte j's low nibble)."""
    return np.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[0], -1)[:, :K]


def q4_group_matmul(X, codes, scales, zeros, K, group):
    """(Y, bound): the product in 64 bits, and sum_k |s| (32 + q + z) |x|, the
    size of the terms that a kernel working on 16 + q and 16 + z adds up."""
    q = unpack_codes(codes, K).astype(np.float64)
    of = np.arange(K) // group
    z = np.full(q.shape, 8.0) if zeros is None else zeros.astype(np.float64)[:, of]
    s = scales.astype(np.float64)[:, of]
    X = X.astype(np.float64)
    return X @ ((q - z) * s).T, np.abs(X) @ ((32 + q + z) * np.abs(s)).T


def kv_plan(ctx, new, table, free, page, max_tokens, begin=0):
    """One request after the other, one token after the other."""
    table = table.copy()
    R, width = table.shape
    flags, taken, total, longest = 0, begin, 0, 0
    cu, slots, positions = [0], np.full(max_tokens, -1, np.int64), np.zeros(max_tokens, np.int32)
    for r in range(R):
        if ctx[r] < 0 or new[r] < 0:
            flags |= 1
        c, n = max(int(ctx[r]), 0), max(int(new[r]), 0)
        longest = max(longest, c + n)
        if -(-(c + n) // page) > width:
            flags |= 2
        if n > 0 and c % page and c // page < width and table[r, c // page] < 0:
            flags |= 16
        for pos in range(c, c + n):
            j = pos // page
            t = total + pos - c
            fresh = None
            if j < width and pos % page == 0:
                fresh = int(free[taken]) if taken < len(free) else -1
                if fresh < 0 and taken >= len(free):
                    flags |= 4
                taken += 1
                if t < max_tokens:
                    table[r, j] = fresh
            if t < max_tokens:
                positions[t] = min(pos, 2 ** 31 - 1)
                if j < width and table[r, j] >= 0:
                    slots[t] = int(table[r, j]) * page + pos % page
        total += n
        cu.append(total)
    if total > max_tokens:
        flags |= 8
    info = np.array([min(taken, max(len(free), begin)), total, flags, min(longest, 2 ** 31 - 1)], np.int32)
    return table, np.array(cu, np.int32), slots, positions, info


def quantize_rows(x):
    """amax/127 by row: fp32 scale and quotient, ties to even."""
    x = x.astype(np.float32)
    s = (np.abs(x).max(-1) / np.float32(127)).astype(np.float32)
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.where(s[..., None] > 0, x / s[..., None], np.float32(0))
    return np.clip(np.rint(q), -127, 127).astype(np.int8), s


def tree_attention(q, k_rows, v_rows, sees, scale):
    """One (query row, head) against key rows: (o, sum of w |v|, largest sum of
    |q k| scale) over the keys that `sees` names; zeros where it names none."""
    k, v = k_rows[sees].astype(np.float64), v_rows[sees].astype(np.float64)
    q = q.astype(np.float64)
    if len(k) == 0:
        return np.zeros(v_rows.shape[1]), np.zeros(v_rows.shape[1]), 0.0
    with np.errstate(invalid="ignore", over="ignore"):
        s = (k @ q) * scale
        if s.max() == -np.inf:
            return np.zeros(v.shape[1]), np.zeros(v.shape[1]), 0.0
        w = np.exp(s - s.max())
        w /= w.sum()
        return w @ v, w @ np.abs(v), float((np.abs(k) @ np.abs(q)).max() * abs(scale))


def chain_mask(new):
    return np.tril(np.ones((new, new), bool))


def random_tree(g, new):
    """mask[t, i] of a random tree: ancestors and the token itself."""
    m = np.zeros((new, new), bool)
    for i in range(new):
        if i:
            p = int(g.integers(max(-1, i - 4), i))
            if p >= 0:
                m[i] = m[p]
        m[i, i] = True
    return m
