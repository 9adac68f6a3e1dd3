"""Plain 64-bit forms of the long-context serving operators (test infrastructure;
nothing here is shared with the library)."""
import numpy as np
import torch

NIBBLE = [0, 2, 4, 6, 1, 3, 5, 7]  # the element of each 8 that nibble i of a word holds


def bf16(x):
    """fp32 values rounded to bf16, as fp32."""
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).bfloat16().float().numpy()


def quantize_q4(x):
    """Rows [..., D] in 4 bits: codes, step and minimum (bf16 values, as fp32); all of it in fp32 steps."""
    x = x.astype(np.float32)
    with np.errstate(all="ignore"):
        lo, hi = x.min(-1), x.max(-1)
        m = bf16(lo)
        step = bf16(np.maximum((hi - m) / np.float32(15), np.float32(0)))
        bad = ~np.isfinite(x).all(-1) | ~np.isfinite(m) | ~np.isfinite(step)
        step = np.where(bad, np.float32(0), step)
        m = np.where(bad, np.float32(np.nan), m)
        q = np.where(step[..., None] > 0, (x - m[..., None]) / step[..., None], np.float32(0))
    return np.clip(np.rint(q), 0, 15).astype(np.uint8), step, m


def pack_q4(codes):
    """Codes [..., D] -> bytes [..., D / 2]."""
    w = codes.reshape(codes.shape[:-1] + (-1, 8))[..., NIBBLE]
    return (w[..., 0::2] | (w[..., 1::2] << 4)).reshape(codes.shape[:-1] + (-1,)).astype(np.uint8)


def unpack_q4(b):
    """Bytes [..., D / 2] -> codes [..., D], element by element."""
    out = np.zeros(b.shape[:-1] + (2 * b.shape[-1],), np.uint8)
    for d in range(out.shape[-1]):
        nibble = NIBBLE.index(d % 8)
        out[..., d] = b[..., d // 8 * 4 + nibble // 2] >> (4 * (nibble % 2)) & 15
    return out


def window_sees(ctx, n, length, window, sinks):
    """[n, length]: new token i of a request sees position j."""
    pos, j = ctx + np.arange(n)[:, None], np.arange(length)[None]
    return (j <= pos) & ((j > pos - window) | (j < sinks))


def attention(q, k, v, sees, scale):
    """q [n, Hq, D], k and v [L, Hkv, D], sees [n, L], all fp64: (o, the size of what is added up for it); zeros
    where a row sees nothing, or only scores of -inf."""
    n, Hq, D = q.shape
    G = Hq // k.shape[1]
    o, size = np.zeros(q.shape), np.zeros(q.shape)
    for h in range(Hq):
        with np.errstate(all="ignore"):
            s = np.where(sees, q[:, h] @ k[:, h // G].T * scale, -np.inf)
            top = s.max(-1, keepdims=True) if s.shape[1] else np.full((n, 1), -np.inf)
            w = np.exp(s - np.where(top == -np.inf, 0, top))
            w = w / np.maximum(w.sum(-1, keepdims=True), 1e-300)
            vh = np.where(sees.any(0)[:, None], v[:, h // G], 0)
            o[:, h], size[:, h] = w @ vh, w @ np.abs(vh)
    return o, size


def lora(X, A, B, ids, base, scales):
    """(out, the size of its terms): fp64."""
    out = np.zeros((X.shape[0], B.shape[1])) if base is None else base.astype(np.float64).copy()
    size = np.zeros_like(out)
    for t, a in enumerate(ids):
        if 0 <= a < A.shape[0]:
            s = 1.0 if scales is None else float(scales[a])
            out[t] += s * (B[a] @ (A[a] @ X[t]))
            size[t] = abs(s) * (np.abs(B[a]) @ (np.abs(A[a]) @ np.abs(X[t])))
    return out, size


def logprobs(x, tokens, top, scale=1.0):
    """(logprobs, entropy, top ids, their logprobs) of logits [T, V] in fp64, tokens [T, n]."""
    T, V = x.shape
    with np.errstate(all="ignore"):
        z = x * scale
        m = z.max(-1, keepdims=True)
        y = z - np.where(m == -np.inf, 0, m)
        e = np.exp(y)
        S = e.sum(-1, keepdims=True)
        lp = y - np.log(S)
        empty = (x == -np.inf).all(-1)
        bad = np.isnan(x).any(-1) | (x == np.inf).any(-1)
        ent = np.log(S[:, 0]) - np.where(e > 0, e * y, 0).sum(-1) / S[:, 0]
    lp[empty], ent[empty] = -np.inf, 0
    lp[bad], ent[bad] = np.nan, np.nan
    inside = (tokens >= 0) & (tokens < V)
    given = np.where(inside, np.take_along_axis(lp, np.where(inside, tokens, 0), 1), -np.inf)
    order = np.argsort(np.where(np.isnan(x), np.inf, -x), axis=-1, kind="stable")[:, :top]
    ids = np.full((T, top), -1, np.int64)
    ids[:, :order.shape[1]] = order
    values = np.where(ids >= 0, np.take_along_axis(lp, np.maximum(ids, 0), 1), -np.inf)
    return given, ent, ids, values
