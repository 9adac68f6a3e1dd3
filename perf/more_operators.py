"""Cases of the operators that serve many requests with long contexts: the cache
held in 4 bits (append, and the tree attention over it), attention with a sliding
window and first tokens that stay visible, low-rank adapters beside a shared
projection, and log probabilities of given tokens.

`run` computes a case in plain torch (``own`` false) or with the library's
kernels (``own`` true); `exact` gives the same outputs from the definitions in
64 bits.  The shapes are those of the workloads module (the Qwen3-0.6B
projections, its 16 query over 8 key/value heads of 128 and its vocabulary of
151936, the 8B-class 4096 x 14336 projections) and odd ones beside them.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "s8": torch.int8}
BYTES = {"f32": 4, "f16": 2, "bf16": 2, "s8": 1, "q4": 0.5}
NIBBLE = [0, 2, 4, 6, 1, 3, 5, 7]  # the element of each 8 that nibble i of a 4-bit row's word holds


# ------------------------------------------------------------------ cases ---

def listed():
    return [
        # the new rows of one verification step of 16 requests into a 4-bit cache
        dict(name="append4_256_bf16", op="append", T=256, heads=8, dim=128, page=16, x="bf16"),
        # a prompt's rows, straight from fp32 projections, into a 4-bit cache
        dict(name="append4_8190_f32", op="append", T=8190, heads=8, dim=128, page=64, x="f32"),
        # a small batch of trees over a 4-bit cache
        dict(name="tree4_r4_ctx2000_new9", op="tree", R=4, ctx=2000, new=9, hq=16, hkv=8, dim=128, page=16, lens=1),
        # a long ragged batch of trees over a 4-bit cache
        dict(name="tree4_r32_ctx32768_new16", op="tree", R=32, ctx=32768, new=16, hq=16, hkv=8, dim=128, page=32, lens=2),
        # one decoded token of one request behind a window
        dict(name="window_r1_ctx5000_w1024_bf16", op="window", R=1, ctx=5000, new=1, window=1024, sinks=4, hq=16, hkv=8,
             dim=128, page=16, c="bf16", lens=3),
        # a batch of decoded tokens, a long window over a 4-bit cache
        dict(name="window_r61_ctx60000_w16384_q4", op="window", R=61, ctx=60000, new=1, window=16384, sinks=64, hq=32,
             hkv=8, dim=128, page=64, c="q4", lens=4),
        # ragged prompts in fp16, 8B-class heads
        dict(name="window_r3_new5000_w1000_f16", op="window", R=3, ctx=0, new=5000, window=1000, sinks=5, hq=32, hkv=8,
             dim=128, page=24, c="f16", lens=5),
        # one decoded token beside the smallest projection: latency counts
        dict(name="lora_m1_1024x2048_r16_bf16", op="lora", T=1, K=1024, N=2048, rank=16, adapters=4, runs=False, x="bf16"),
        # a decode batch in fp32 (the type of the library's other products), an adapter per request, odd sizes
        dict(name="lora_m61_4100x4099_r12_f32", op="lora", T=61, K=4100, N=4099, rank=12, adapters=24, runs=False, x="f32"),
        # prompts of several requests beside an 8B-class projection
        dict(name="lora_m4001_4096x14336_r64_bf16", op="lora", T=4001, K=4096, N=14336, rank=64, adapters=6, runs=True, x="bf16"),
        # one token's logits with its five best alternatives
        dict(name="logprobs_1x151936_f32_top5", op="logprobs", T=1, V=151936, given=0, top=5, x="f32"),
        # a prompt's logits
        dict(name="logprobs_1000x151936_bf16_top20", op="logprobs", T=1000, V=151936, given=0, top=20, x="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "tree", "window", "window", "lora", "lora", "logprobs"])
    if op == "append":
        return dict(op=op, T=_log(rng, 1, 8190), heads=rng.choice([1, 2, 4, 8]), dim=rng.choice([64, 80, 96, 128]),
                    page=rng.choice([1, 16, 24, 64]), x=rng.choice(["f32", "f16", "bf16"]))
    if op == "lora":
        x = rng.choice(["f32", "f16", "bf16"])
        return dict(op=op, T=_log(rng, 1, 4000), K=_log(rng, 64, 4096), N=_log(rng, 16, 14336),
                    rank=rng.choice([3, 4, 8, 12, 16, 16, 32, 64]), adapters=_log(rng, 1, 32), runs=rng.random() < 0.5, x=x)
    if op == "logprobs":
        x = rng.choice(["f32", "f16", "bf16"])
        V = rng.choice([151936, _log(rng, 100, 151936)])
        return dict(op=op, T=_log(rng, 1, min(4000, 1000 * 151936 // V // (2 if x == "f32" else 1))), V=V,
                    given=rng.choice([0, 0, rng.randint(1, 8)]), top=rng.choice([0, 1, 5, rng.randint(1, 20), 20]), x=x)
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 8])
    c = "q4" if op == "tree" else rng.choice(["f16", "bf16", "s8", "q4"])
    case = dict(op=op, hq=hq, hkv=hkv, dim=rng.choice([64, 80, 96, 128]), page=rng.choice([1, 16, 24, 32, 64, 128]),
                lens=rng.randrange(1 << 30))
    if op == "tree":
        ctx, new = rng.choice([0, _log(rng, 1, 32768), _log(rng, 64, 8192)]), _log(rng, 1, 64)
        return dict(case, R=_log(rng, 1, max(1, min(64, 32 * 32768 // (ctx + new), 2048 // new))), ctx=ctx, new=new)
    window, sinks = _log(rng, 16, 16384), rng.choice([0, 1, 4, 5, 64, 100])
    if rng.random() < 0.35:  # prompts, or pieces of them
        new, ctx = _log(rng, 64, 4096), rng.choice([0, 0, _log(rng, 1, 4096)])
        case["hkv"] = hkv = min(hkv, 4)
        case["hq"] = hkv * rng.choice([1, 2, 3, 4])
        R = _log(rng, 1, max(1, min(16, 8192 // new)))
    else:
        new, ctx = rng.choice([1, 1, _log(rng, 1, 16)]), _log(rng, 1, 65536)
        R = _log(rng, 1, max(1, min(64, 32 * 32768 // (ctx + new))))
    return dict(case, R=R, ctx=ctx, new=new, window=window, sinks=sinks, c=c)


def _lengths(case):
    """Ragged context and new lengths that a case stands for (the same for every seed)."""
    rng = random.Random(case["lens"])
    R, ctx, new = case["R"], case["ctx"], case["new"]
    c = [rng.randint(ctx // 4, ctx) for _ in range(R)]
    n = [rng.randint((new + 1) // 2, new) for _ in range(R)]
    c[rng.randrange(R)] = ctx
    n[rng.randrange(R)] = new
    if R > 8:  # a new request and one that sits this step out
        a, b = rng.sample(range(R), 2)
        c[a], n[b] = 0, 0
    return c, n


def _masks(case, n):
    """mask[t, i]: drafted token t of a request sees drafted token i of it (its ancestors and itself)."""
    rng = random.Random(case["lens"] + 1)
    mask = np.zeros((sum(n), max(max(n), 1)), dtype=bool)
    t = 0
    for k in n:
        first = t
        for i in range(k):
            p = -1 if i == 0 else rng.randint(max(-1, i - 6), i - 1)
            if p >= 0:
                mask[t] = mask[first + p]
            mask[t, i] = True
            t += 1
    return mask


def _ids(case):
    """The adapter of each row, -1 for none: by request where rows come in runs, else row by row."""
    rng = random.Random(case["T"] * 31 + case["N"])
    T, n = case["T"], case["adapters"]
    out = []
    while len(out) < T:
        a = rng.randrange(-1, n) if T > 1 else 0
        out += [a] * (rng.randint(1, max(1, T // 4)) if case["runs"] else 1)
    return out[:T]


def _row_bytes(case, c):
    """A cached row of K and of V, of one head."""
    return 2 * (case["dim"] * BYTES[c] + (4 if c in ("s8", "q4") else 0))


def work(case):
    op = case["op"]
    if op == "append":
        rows = case["T"] * case["heads"]
        slots = -(-case["T"] // case["page"]) * case["page"] * case["heads"]
        # the rows in, codes and scales out; then the values that the whole cache stands for, which the pass returns
        by = 2.0 * rows * case["dim"] * BYTES[case["x"]] + rows * _row_bytes(case, "q4") + 8 * case["T"]
        return dict(bytes=by + slots * (_row_bytes(case, "q4") + 8.0 * case["dim"]), flops=0)
    if op == "lora":
        T, K, N, r, b = case["T"], case["K"], case["N"], case["rank"], BYTES[case["x"]]
        ids = _ids(case)
        rows, used = sum(i >= 0 for i in ids), len(set(ids) - {-1})
        by = b * (rows * K + 2.0 * T * N) + used * r * (K + N) * (2 if b == 4 else b) + 4 * T
        return dict(bytes=by, flops=2.0 * rows * r * (K + N))
    if op == "logprobs":
        T, n, k = case["T"], max(case["given"], 1), case["top"]
        return dict(bytes=T * (float(case["V"]) * BYTES[case["x"]] + 12 * n + 4 + 12 * k), flops=4.0 * T * case["V"])
    c, n = _lengths(case)
    if op == "tree":
        keys = sum(a + b for a, b in zip(c, n) if b)
        pairs = sum(a * b for a, b in zip(c, n)) + float(_masks(case, n).sum())
    else:
        W, S = case["window"], case["sinks"]
        keys = sum(min(a + b, S + W - 1 + b) for a, b in zip(c, n) if b)
        pairs = float(sum(min(i + 1, W) + min(S, max(0, i + 1 - W)) for a, b in zip(c, n) for i in range(a, a + b)))
    x = BYTES["f16" if op == "window" and case["c"] == "f16" else "bf16"]
    by = float(keys * case["hkv"]) * _row_bytes(case, "q4" if op == "tree" else case["c"])
    by += 2.0 * sum(n) * case["hq"] * case["dim"] * x + (sum(n) * max(n) if op == "tree" else 0)
    return dict(bytes=by, flops=4.0 * pairs * case["hq"] * case["dim"])


# ----------------------------------------------------------------- inputs ---

def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _randn(g, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device=DEV) * std).to(dtype)


def _int32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _rows_s8(x):
    """Rows quantised with amax / 127: codes and scales."""
    s = x.abs().amax(-1)
    s = s / s.new_full((), 127.0)
    return torch.where(s[..., None] > 0, (x / s[..., None]).round(), 0.0).clamp(-127, 127).to(torch.int8), s


def _rows_q4(x):
    """Rows in 4 bits: codes 0..15 (one a byte) and (step, minimum) in bf16, in the definition's own fp32 steps."""
    m = x.amin(-1).bfloat16()
    d = ((x.amax(-1) - m.float()) / x.new_full((), 15.0)).clamp(min=0).bfloat16()
    df = d.float()[..., None]
    q = torch.where(df > 0, ((x - m.float()[..., None]) / df).round(), 0.0).clamp(0, 15)
    return q.to(torch.uint8), torch.stack([d, m], -1)


def _pack(q):
    """Codes [..., D] -> bytes [..., D / 2]: nibble i of each 8 elements' word holds element NIBBLE[i]."""
    w = q.unflatten(-1, (-1, 8))[..., NIBBLE]
    return (w[..., 0::2] | (w[..., 1::2] << 4)).flatten(-2)


def _unpack(b):
    """Bytes [..., D / 2] -> codes [..., D]."""
    w = torch.stack([b & 15, b >> 4], -1).flatten(-2).unflatten(-1, (-1, 8))
    order = [NIBBLE.index(e) for e in range(8)]
    return w[..., order].flatten(-2)


def prepare(case, seed):
    """What a program has in hand before the call.  Caches are filled with normal rows at pages in random order, and the
    queries are scaled so that the softmax is as peaked as a trained model's; adapters are as large as a trained one's
    beside the projection; logits are normal with a few likely tokens on top, among them most of the given ones."""
    g = _generator(seed)
    op = case["op"]
    st = dict(case=case)
    if op == "append":
        T, H, D, P = case["T"], case["heads"], case["dim"], case["page"]
        pages = -(-T // P)
        st["K"] = _randn(g, T, H, D, dtype=TYPES[case["x"]])
        st["V"] = _randn(g, T, H, D, dtype=TYPES[case["x"]])
        st["slots"] = torch.randperm(pages * P, generator=g, device=DEV)[:T]
        st["all"] = torch.arange(pages * P, device=DEV)
        st["k_cache"], st["v_cache"] = (torch.zeros(pages, P, H, D // 2, dtype=torch.uint8, device=DEV) for _ in range(2))
        st["k_scale"], st["v_scale"] = (torch.zeros(pages, P, H, 2, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        return st
    if op == "lora":
        T, K, N, r, n = case["T"], case["K"], case["N"], case["rank"], case["adapters"]
        x = TYPES[case["x"]]
        w = torch.bfloat16 if case["x"] == "f32" else x
        st["X"], st["base"] = _randn(g, T, K, dtype=x), _randn(g, T, N, dtype=x)
        st["A"], st["B"] = _randn(g, n, r, K, std=K ** -0.5, dtype=w), _randn(g, n, N, r, std=r ** -0.5, dtype=w)
        st["scales"] = torch.rand(n, generator=g, device=DEV) + 0.5
        st["ids"] = _int32(_ids(case))
        return st
    if op == "logprobs":
        T, V, n = case["T"], case["V"], max(case["given"], 1)
        z = _randn(g, T, V, std=2.0)
        likely = torch.randint(0, V, (T, 8), generator=g, device=DEV)
        z.scatter_(1, likely, _randn(g, T, 8, std=2.0) + 12)
        ids = likely[:, torch.arange(n, device=DEV) % 8]
        stray = torch.rand(T, n, generator=g, device=DEV) < 0.25
        st["ids"] = torch.where(stray, torch.randint(0, V, (T, n), generator=g, device=DEV), ids)
        if case["given"] == 0:
            st["ids"] = st["ids"][:, 0].contiguous()
        st["logits"] = z.to(TYPES[case["x"]])
        return st
    c, n = _lengths(case)
    R, P = case["R"], case["page"]
    need = [-(-(a + b) // P) for a, b in zip(c, n)]
    width, pages = max(need), sum(need) + 7
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    j = torch.arange(width, device=DEV)[None]
    counts = torch.tensor(need, device=DEV)
    at = (counts.cumsum(0) - counts)[:, None] + j
    st["table"] = torch.where(j < counts[:, None], order[at.clamp(max=pages - 1)], -1).to(torch.int32).contiguous()
    st["ctx"], st["cu"] = _int32(c), _int32([0] + np.cumsum(n).tolist())
    T, Hq, Hkv, D = sum(n), case["hq"], case["hkv"], case["dim"]
    kind = "q4" if op == "tree" else case["c"]
    x = TYPES["f16" if kind == "f16" else "bf16"]
    st["q"] = _randn(g, T, Hq, D, std=2.5, dtype=x)
    st["k_scale"] = st["v_scale"] = None
    for name in ("k", "v"):
        if kind in ("s8", "q4"):  # by pages, so that the fp32 rows need not all be there at once
            codes, scales = [], []
            for p0 in range(0, pages, max(1, (1 << 27) // (P * Hkv * D))):
                p1 = min(pages, p0 + max(1, (1 << 27) // (P * Hkv * D)))
                q, s = (_rows_s8 if kind == "s8" else _rows_q4)(_randn(g, p1 - p0, P, Hkv, D))
                codes.append(q if kind == "s8" else _pack(q))
                scales.append(s)
            st[name + "_cache"], st[name + "_scale"] = torch.cat(codes), torch.cat(scales)
        else:
            st[name + "_cache"] = _randn(g, pages, P, Hkv, D, dtype=x)
    st["mask"] = torch.from_numpy(_masks(case, n)).to(DEV) if op == "tree" else None
    st["longest"], st["most"] = max(a + b for a, b in zip(c, n)), max(n)
    return st


# -------------------------------------------------------------------- run ---

def run(st):
    op = st["case"]["op"]
    if own:
        return {"append": _own_append, "tree": _own_tree, "window": _own_window, "lora": _own_lora,
                "logprobs": _own_logprobs}[op](st)
    return {"append": _plain_append, "tree": _plain_attention, "window": _plain_attention, "lora": _plain_lora,
            "logprobs": _plain_logprobs}[op](st)


def _own_append(st):
    import int8_bit_weight_amd as qmm
    cache = (st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"])
    qmm.kv_append(st["K"], st["V"], st["slots"], *cache)
    k, v = qmm.kv_gather(st["all"], *cache, dtype=torch.float32)
    return [k, v, st["k_scale"], st["v_scale"]]


def _own_tree(st):
    import int8_bit_weight_amd as qmm
    return qmm.tree_attention(st["q"], st["k_cache"], st["v_cache"], st["table"], st["ctx"], st["cu"], st["mask"],
                              k_scale=st["k_scale"], v_scale=st["v_scale"])


def _own_window(st):
    import int8_bit_weight_amd as qmm
    return qmm.window_attention(st["q"], st["k_cache"], st["v_cache"], st["table"], st["ctx"], st["cu"],
                                st["case"]["window"], st["case"]["sinks"], k_scale=st["k_scale"], v_scale=st["v_scale"])


def _own_lora(st):
    import int8_bit_weight_amd as qmm
    return qmm.lora_matmul(st["X"], st["A"], st["B"], st["ids"], st["base"], st["scales"])


def _own_logprobs(st):
    import int8_bit_weight_amd as qmm
    r = qmm.token_logprobs(st["logits"], st["ids"], st["case"]["top"])
    return [r.logprobs, r.entropy, r.top_ids, r.top_logprobs]


def _plain_append(st):
    kc, vc, P, at = st["k_cache"], st["v_cache"], st["k_cache"].shape[1], st["slots"]
    out = []
    for x, cache, scale in ((st["K"], kc, st["k_scale"]), (st["V"], vc, st["v_scale"])):
        q, s = _rows_q4(x.float())
        cache[at // P, at % P], scale[at // P, at % P] = _pack(q), s
        rows, dm = cache[st["all"] // P, st["all"] % P], scale[st["all"] // P, st["all"] % P].float()
        out.append(_unpack(rows).float() * dm[..., :1] + dm[..., 1:])
    return out + [st["k_scale"], st["v_scale"]]


def _gather(cache, scale, slot, P):
    """Cached rows [R, H, L, D] of the slots [R, L] in 32 bits."""
    x = cache[slot // P, slot % P]
    if scale is None:
        x = x.float()
    elif x.dtype == torch.int8:
        x = x.float() * scale[slot // P, slot % P][..., None]
    else:
        dm = scale[slot // P, slot % P].float()
        x = _unpack(x).float() * dm[..., :1] + dm[..., 1:]
    return x.transpose(1, 2)


def _plain_attention(st):
    case = st["case"]
    R, P, Hq, Hkv, D = case["R"], case["page"], case["hq"], case["hkv"], case["dim"]
    W, S = case.get("window", 1 << 40), case.get("sinks", 0)
    most, q = st["most"], st["q"]
    G, T = Hq // Hkv, q.shape[0]
    ctx, cu = st["ctx"].long(), st["cu"].long()
    new = cu[1:] - cu[:-1]
    # query rows of each request, padded to the most new tokens of any
    i = torch.arange(most, device=DEV)[None]
    row = (cu[:-1, None] + i).clamp(max=T - 1)
    real = i < new[:, None]
    x = q.float()[row].view(R, most, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(R, Hkv, most * G, D)
    # cached rows that a request's new tokens can see: the first S, and from the first token's window on
    L = min(st["longest"], S + W - 1 + most)
    j = torch.arange(L, device=DEV)[None]
    begin = (ctx + 1 - W).clamp(min=S)[:, None]
    pos = torch.where(j < S, j, begin + j - S)
    page = torch.gather(st["table"].long(), 1, (pos // P).clamp(max=st["table"].shape[1] - 1)).clamp(min=0)
    slot = page * P + pos % P
    k, v = _gather(st["k_cache"], st["k_scale"], slot, P), _gather(st["v_cache"], st["v_scale"], slot, P)
    # what each new token sees
    d = (pos - ctx[:, None])[:, None]
    if st["mask"] is None:
        at = pos[:, None]
        sees = (d <= i[..., None]) & ((d > i[..., None] - W) | (at < S)) & (d < new[:, None, None])
    else:
        m = st["mask"][row]
        sees = (d < 0) | ((d < new[:, None, None]) & torch.gather(m, 2, d.clamp(0, m.shape[2] - 1).expand(R, most, L)))
    sees = sees.repeat_interleave(G, 1)[:, None]
    s = torch.where(sees, x @ k.transpose(-1, -2).contiguous() * (1.0 / math.sqrt(D)), -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top == -math.inf, 0.0, top))
    o = p @ v.contiguous() / p.sum(-1, keepdim=True).clamp(min=1e-30)
    o = o.view(R, Hkv, most, G, D).permute(0, 2, 1, 3, 4).reshape(R, most, Hq, D)
    out = q.new_zeros(T + 1, Hq, D)
    out[torch.where(real, row, T)] = o.to(q.dtype)
    return out[:T]


def _plain_lora(st):
    A, B, ids = st["A"], st["B"], st["ids"].long()
    n, r, K = A.shape
    T, at = ids.shape[0], ids.clamp(min=0)
    z = (st["X"].float() @ A.reshape(n * r, K).float().t()).view(T, n, r)[torch.arange(T, device=DEV), at]
    z = torch.where(ids[:, None] >= 0, z * st["scales"][at][:, None], 0.0)
    wide = z.new_zeros(T, n, r)
    wide[torch.arange(T, device=DEV), at] = z
    y = wide.view(T, n * r) @ B.float().transpose(1, 2).reshape(n * r, -1)
    return (st["base"].float() + y).to(st["base"].dtype)


def _plain_logprobs(st):
    x, ids, k = st["logits"].float(), st["ids"], min(st["case"]["top"], st["logits"].shape[1])
    V = x.shape[1]
    y = x - x.amax(-1, keepdim=True)
    e = torch.exp(y)
    s = e.sum(-1)
    log_s = torch.log(s)
    entropy = log_s - (e * y).sum(-1) / s
    given = y.gather(1, ids.view(x.shape[0], -1)).view(ids.shape) - log_s.view([-1] + [1] * (ids.dim() - 1))
    # the order of (value, lowest index): a whole number of 64 bits that grows with it
    bits = (x + 0.0).view(torch.int32).long()
    bits = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits)
    order = (bits << 32) + (V - 1 - torch.arange(V, device=DEV))
    top = V - 1 - (torch.topk(order, k, -1).values & 0xFFFFFFFF)
    return [given, entropy, top, y.gather(1, top) - log_s[:, None]]


# ------------------------------------------------------------------ exact ---

def exact(case, seed):
    st = prepare(case, seed)
    return {"append": _exact_append, "tree": _exact_attention, "window": _exact_attention, "lora": _exact_lora,
            "logprobs": _exact_logprobs}[case["op"]](case, st)


def _exact_append(case, st):
    out, scales = [], []
    slots, n = st["slots"], st["all"].numel()
    for x in (st["K"], st["V"]):
        x = x.double()
        m = x.min(-1).values.float().bfloat16().double()
        # the step and the quotient are fp32 by definition, the step then bf16
        d = torch.clamp(((x.max(-1).values - m).float().double() / 15).float(), min=0).bfloat16().double()
        q = ((x - m[..., None]).float().double() / d[..., None]).float().double()
        q = torch.where(d[..., None] > 0, torch.round(q), 0.0).clamp(0, 15)
        values = torch.zeros(n, case["heads"], case["dim"], dtype=torch.float64, device=DEV)
        scale = torch.zeros(n, case["heads"], 2, dtype=torch.float64, device=DEV)
        values[slots] = q * d[..., None] + m[..., None]
        scale[slots, :, 0], scale[slots, :, 1] = d, m
        out.append(values)
        scales.append(scale.view(st["k_scale"].shape))
    return out + scales


def _exact_rows(st, name, kind, pages, h, length, D):
    """Rows 0 .. length-1 of one head of a request, as the values they stand for."""
    x = st[name + "_cache"][pages, :, h]
    x = x.reshape(-1, x.shape[-1])[:length]
    if kind == "s8":
        return x.double() * st[name + "_scale"][pages, :, h].reshape(-1, 1)[:length].double()
    if kind == "q4":
        d, m = st[name + "_scale"][pages, :, h].reshape(-1, 2)[:length].double().unbind(-1)
        out = torch.empty(length, D, dtype=torch.float64, device=DEV)
        for e in range(8):  # element e of each eight: nibble e / 2 of the low half of its word, or of the high one
            byte = x[:, (e // 4) + 2 * (e % 2)::4].long()
            out[:, e::8] = ((byte >> (4 * (e // 2 % 2))) & 15).double()
        return out * d[:, None] + m[:, None]
    return x.double()


def _exact_attention(case, st):
    P, Hq, Hkv, D = case["page"], case["hq"], case["hkv"], case["dim"]
    kind = "q4" if case["op"] == "tree" else case["c"]
    G = Hq // Hkv
    cu, ctx = st["cu"].tolist(), st["ctx"].tolist()
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV)
    for r in range(case["R"]):
        n, length = cu[r + 1] - cu[r], ctx[r] + cu[r + 1] - cu[r]
        if n == 0:
            continue
        pages = st["table"][r, :-(-length // P)].long()
        if st["mask"] is not None:
            sees = torch.ones(n, length, dtype=torch.bool, device=DEV)
            sees[:, ctx[r]:] = st["mask"][cu[r]:cu[r + 1], :n]
        else:
            i, j = torch.arange(ctx[r], length, device=DEV)[:, None], torch.arange(length, device=DEV)[None]
            sees = (j <= i) & ((i - j < case["window"]) | (j < case["sinks"]))
        for h in range(Hkv):
            k, v = (_exact_rows(st, name, kind, pages, h, length, D) for name in "kv")
            for a in range(G):
                s = st["q"][cu[r]:cu[r + 1], h * G + a].double() @ k.t() / math.sqrt(D)
                out[cu[r]:cu[r + 1], h * G + a] = torch.softmax(s.masked_fill(~sees, -math.inf), -1) @ v
    return out


def _exact_lora(case, st):
    out = st["base"].double()
    for a in range(case["adapters"]):
        rows = (st["ids"] == a).nonzero().flatten()
        if len(rows):
            z = st["X"][rows].double() @ st["A"][a].double().t()
            out[rows] += st["scales"][a].double() * (z @ st["B"][a].double().t())
    return out


def _exact_logprobs(case, st):
    given, entropy, tops, values = [], [], [], []
    k = min(case["top"], case["V"])
    for t0 in range(0, case["T"], 256):
        x, ids = st["logits"][t0:t0 + 256].double(), st["ids"][t0:t0 + 256]
        lp = torch.log_softmax(x, -1)
        given.append(lp.gather(1, ids.view(x.shape[0], -1)).view(ids.shape))
        entropy.append(-(lp.exp() * lp).sum(-1))
        if k:  # a stable sort leaves equal values in the order of their indexes
            top = torch.sort(x, dim=-1, descending=True, stable=True).indices[:, :k]
        else:
            top = ids.new_zeros(x.shape[0], 0)
        tops.append(top)
        values.append(lp.gather(1, top))
    return [torch.cat(given), torch.cat(entropy), torch.cat(tops), torch.cat(values)]
