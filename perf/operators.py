"""Cases of the drafted-token verification operators: the 4-bit group-scaled
product, the cache plan (block tables and slot maps), the cache append and the
tree attention over a paged cache.

`run` computes a case in plain torch (``own`` false) or with the library's
kernels (``own`` true); `exact` gives the same outputs from the definitions in
64 bits.  The shapes are those of the workloads module (the Qwen3-0.6B
projections and its 16 query over 8 key/value heads of 128, the 8B-class
4096 x 14336 projections) and odd ones beside them.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "s8": torch.int8}
BYTES = {"f32": 4, "f16": 2, "bf16": 2, "s8": 1}


# ------------------------------------------------------------------ cases ---

def listed():
    return [
        # one decoded token through the smallest projection: latency counts
        dict(name="q4g_m1_2048x1024_bf16", op="q4g", M=1, K=2048, N=1024, group=128, zeros=False, x="bf16", s="bf16"),
        # one decoded token through an 8B-class up projection: weight bytes count
        dict(name="q4g_m1_4096x14336_f16", op="q4g", M=1, K=4096, N=14336, group=128, zeros=True, x="f16", s="f16"),
        # a short draft in fp32 (the type of the library's other products), sizes that fill no tile
        dict(name="q4g_m5_4100x11003_f32", op="q4g", M=5, K=4100, N=11003, group=32, zeros=True, x="f32", s="f16"),
        # a whole tree of drafted tokens through an 8B-class down projection
        dict(name="q4g_m64_14336x4096_bf16", op="q4g", M=64, K=14336, N=4096, group=64, zeros=True, x="bf16", s="bf16"),
        # the plan of one decode step of a small batch, trees of up to 16 drafted tokens
        dict(name="plan_r64_new16", op="plan", R=64, ctx=4096, new=16, page=16, lens=1),
        # the plan of a prefill batch: ragged prompts on an empty cache
        dict(name="plan_r509_new2048", op="plan", R=509, ctx=0, new=2048, page=16, lens=2),
        # the new rows of one verification step into a bf16 cache
        dict(name="append_256_bf16", op="append", T=256, heads=8, dim=128, page=16, x="bf16", c="bf16"),
        # a prompt's rows, straight from fp32 projections, into an int8 cache
        dict(name="append_8190_f32_s8", op="append", T=8190, heads=8, dim=128, page=64, x="f32", c="s8"),
        # one decoded token of one request
        dict(name="tree_r1_ctx1000_one_bf16", op="tree", R=1, ctx=1000, new=1, hq=16, hkv=8, dim=128, page=16, tree=False,
             x="bf16", c="bf16", lens=3),
        # a small ragged batch of trees in fp16, 8B-class heads
        dict(name="tree_r16_ctx4096_new16_f16", op="tree", R=16, ctx=4096, new=16, hq=32, hkv=8, dim=128, page=16, tree=True,
             x="f16", c="f16", lens=4),
        # one long document with a large tree
        dict(name="tree_r1_ctx131000_new64_bf16", op="tree", R=1, ctx=131000, new=64, hq=16, hkv=8, dim=128, page=64,
             tree=True, x="bf16", c="bf16", lens=5),
        # a long ragged batch over the int8 cache
        dict(name="tree_r32_ctx32768_new32_s8", op="tree", R=32, ctx=32768, new=32, hq=16, hkv=8, dim=128, page=32,
             tree=True, x="bf16", c="s8", lens=6),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["q4g", "q4g", "plan", "append", "tree", "tree"])
    if op == "q4g":
        M, K = _log(rng, 1, 64), _log(rng, 64, 14336)
        N = _log(rng, 16, min(16384, 14336 * 4096 // K))
        if rng.random() < 0.5:
            K = max(64, K // 64 * 64)
        return dict(op=op, M=M, K=K, N=N, group=rng.choice([32, 64, 128, 256]), zeros=rng.random() < 0.5,
                    x=rng.choice(["f32", "f16", "bf16"]), s=rng.choice(["f16", "bf16"]))
    if op == "plan":
        R = _log(rng, 1, 500)
        return dict(op=op, R=R, ctx=rng.choice([0, _log(rng, 1, 8192)]), new=_log(rng, 1, 2048),
                    page=rng.choice([1, 16, 24, 32, 64, 128]), lens=rng.randrange(1 << 30))
    if op == "append":
        return dict(op=op, T=_log(rng, 1, 4096), heads=rng.choice([1, 2, 4, 8, 12]), dim=rng.choice([64, 80, 128]),
                    page=rng.choice([1, 16, 24, 64]), x=rng.choice(["f32", "f16", "bf16"]),
                    c=rng.choice(["f16", "bf16", "s8"]))
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 8])
    c = rng.choice(["f16", "bf16", "s8"])
    ctx = rng.choice([0, _log(rng, 1, 32768), _log(rng, 64, 8192)])
    new = _log(rng, 1, 64)
    R = _log(rng, 1, max(1, min(64, 32 * 32768 // (ctx + new), 4096 // new)))
    return dict(op=op, R=R, ctx=ctx, new=new, hq=hq, hkv=hkv, dim=rng.choice([64, 80, 128]),
                page=rng.choice([1, 16, 24, 32, 64, 128]), tree=rng.random() < 0.7, x="bf16" if c == "s8" else c, c=c,
                lens=rng.randrange(1 << 30))


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


def _parents(case, n):
    """Each request's tree: the parent of each drafted token among those before it, -1 for a child of the context."""
    rng = random.Random(case["lens"] + 1)
    return [[-1 if i == 0 else rng.randint(max(-1, i - 6), i - 1) for i in range(k)] for k in n]


def _masks(case, n):
    """mask[t, i]: drafted token t of a request sees drafted token i of it (its ancestors and itself)."""
    T, most = sum(n), max(max(n), 1)
    mask = np.zeros((T, most), dtype=bool)
    t = 0
    for par in _parents(case, n):
        first = t
        for i, p in enumerate(par):
            if p >= 0:
                mask[t] = mask[first + p]
            mask[t, i] = True
            t += 1
    return mask


def work(case):
    op = case["op"]
    if op == "q4g":
        M, K, N, G = case["M"], case["K"], case["N"], case["group"]
        groups = -(-K // G)
        by = N * K / 2 + N * groups * (2.5 if case["zeros"] else 2) + M * (K + N) * BYTES[case["x"]]
        return dict(bytes=by, flops=2.0 * M * N * K)
    if op == "plan":
        c, n = _lengths(case)
        P = case["page"]
        pages = sum(-(-(a + b) // P) - -(-a // P) for a, b in zip(c, n))
        return dict(bytes=12.0 * case["R"] + 12.0 * sum(n) + 8.0 * pages, flops=0)
    if op == "append":
        values = 2.0 * case["T"] * case["heads"] * case["dim"]
        by = values * (BYTES[case["x"]] + BYTES[case["c"]]) + 8 * case["T"]
        if case["c"] == "s8":
            # the scales, and the values that the whole cache stands for, which the pass returns
            slots = -(-case["T"] // case["page"]) * case["page"]
            by += 8.0 * case["T"] * case["heads"] + 2.0 * slots * case["heads"] * (5 * case["dim"] + 4)
        return dict(bytes=by, flops=0)
    c, n = _lengths(case)
    per = 2 * (case["dim"] * BYTES[case["c"]] + (4 if case["c"] == "s8" else 0))
    by = float(sum(a + b for a, b in zip(c, n) if b) * case["hkv"] * per)
    by += 2.0 * sum(n) * case["hq"] * case["dim"] * BYTES[case["x"]]
    if case["tree"]:
        seen = float(_masks(case, n).sum())
        by += sum(n) * max(n)
    else:
        seen = float(sum(b * (b + 1) // 2 for b in n))
    keys = sum(a * b for a, b in zip(c, n)) + seen
    return dict(bytes=by, flops=4.0 * keys * case["hq"] * case["dim"])


# ----------------------------------------------------------------- inputs ---

def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _randn(g, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device=DEV) * std).to(dtype)


def _rows_s8(x):
    """Rows quantised with amax / 127: codes and scales (a tensor for 127: a number would multiply by its reciprocal)."""
    s = x.abs().amax(-1)
    s = s / s.new_full((), 127.0)
    return torch.where(s[..., None] > 0, (x / s[..., None]).round(), 0.0).clamp(-127, 127).to(torch.int8), s


def _int32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    """What a program has in hand before the call.  Weights are 4-bit codes of a normal weight (a minimum and a
    step per group where there are zeros); caches are filled with normal rows at pages in random order, and the
    queries are scaled so that the softmax is as peaked as a trained model's."""
    g = _generator(seed)
    op = case["op"]
    st = dict(case=case)
    if op == "q4g":
        M, K, N, G = case["M"], case["K"], case["N"], case["group"]
        groups = -(-K // G)
        q = (_randn(g, N, K, std=2.9) + 7.5).round().clamp(0, 15).to(torch.uint8)
        if K % 2:
            q = torch.nn.functional.pad(q, (0, 1))
        st["codes"] = q[:, 0::2] | (q[:, 1::2] << 4)  # byte j: k = 2j in the low nibble, 2j + 1 in the high one
        st["scales"] = ((torch.rand(N, groups, generator=g, device=DEV) + 0.5) * 0.007).to(TYPES[case["s"]])
        st["zeros"] = None
        if case["zeros"]:
            st["zeros"] = torch.randint(5, 11, (N, groups), generator=g, device=DEV, dtype=torch.uint8)
        st["X"] = _randn(g, M, K, dtype=TYPES[case["x"]])
        if own:
            import int8_bit_weight_amd as qmm
            st["W"] = qmm.q4_group_repack(st["codes"], st["scales"], st["zeros"], K=K, group=G)
        return st
    if op == "append":
        T, H, D, P = case["T"], case["heads"], case["dim"], case["page"]
        pages = -(-T // P)
        st["K"] = _randn(g, T, H, D, dtype=TYPES[case["x"]])
        st["V"] = _randn(g, T, H, D, dtype=TYPES[case["x"]])
        st["slots"] = torch.randperm(pages * P, generator=g, device=DEV)[:T]
        st["k_cache"], st["v_cache"] = (torch.zeros(pages, P, H, D, dtype=TYPES[case["c"]], device=DEV) for _ in range(2))
        st["k_scale"] = st["v_scale"] = None
        if case["c"] == "s8":
            st["k_scale"], st["v_scale"] = (torch.zeros(pages, P, H, device=DEV) for _ in range(2))
        return st
    c, n = _lengths(case)
    R, P = case["R"], case["page"]
    width = max(-(-(a + b) // P) for a, b in zip(c, n))
    have = [-(-a // P) for a in c]
    need = [-(-(a + b) // P) for a, b in zip(c, n)]
    pages = sum(need) + 7
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    j = torch.arange(width, device=DEV)[None]
    counts = torch.tensor(have if op == "plan" else need, device=DEV)
    at = (counts.cumsum(0) - counts)[:, None] + j
    st["table"] = torch.where(j < counts[:, None], order[at.clamp(max=pages - 1)], -1).to(torch.int32).contiguous()
    st["ctx"] = _int32(c)
    if op == "plan":
        st["new"], st["free"], st["tokens"] = _int32(n), order[sum(have):].contiguous(), sum(n)
        return st
    T, Hq, Hkv, D = sum(n), case["hq"], case["hkv"], case["dim"]
    x = TYPES[case["x"]]
    st["cu"] = _int32([0] + np.cumsum(n).tolist())
    st["q"] = _randn(g, T, Hq, D, std=2.5, dtype=x)
    if case["c"] == "s8":
        st["k_cache"], st["k_scale"] = _rows_s8(_randn(g, pages, P, Hkv, D))
        st["v_cache"], st["v_scale"] = _rows_s8(_randn(g, pages, P, Hkv, D))
    else:
        st["k_cache"], st["v_cache"] = _randn(g, pages, P, Hkv, D, dtype=x), _randn(g, pages, P, Hkv, D, dtype=x)
        st["k_scale"] = st["v_scale"] = None
    st["mask"] = torch.from_numpy(_masks(case, n)).to(DEV) if case["tree"] else None
    st["longest"], st["most"] = max(a + b for a, b in zip(c, n)), max(n)
    return st


# -------------------------------------------------------------------- run ---

def run(st):
    op = st["case"]["op"]
    if own:
        return {"q4g": _own_q4g, "plan": _own_plan, "append": _own_append, "tree": _own_tree}[op](st)
    return {"q4g": _plain_q4g, "plan": _plain_plan, "append": _plain_append, "tree": _plain_tree}[op](st)


def _own_q4g(st):
    import int8_bit_weight_amd as qmm
    return qmm.q4_group_matmul(st["X"], st["W"])


def _own_plan(st):
    import int8_bit_weight_amd as qmm
    plan = qmm.kv_plan(st["ctx"], st["new"], st["table"], st["free"], st["case"]["page"], st["tokens"])
    return [st["table"], plan.cu_new, plan.slots, plan.positions, plan.info]


def _own_append(st):
    import int8_bit_weight_amd as qmm
    qmm.kv_append(st["K"], st["V"], st["slots"], st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"])
    return _cache_values(st)


def _own_tree(st):
    import int8_bit_weight_amd as qmm
    return qmm.tree_attention(st["q"], st["k_cache"], st["v_cache"], st["table"], st["ctx"], st["cu"], st["mask"],
                              k_scale=st["k_scale"], v_scale=st["v_scale"])


def _cache_values(st):
    """What the caches hold: 16-bit caches as they are, int8 ones as the values they stand for."""
    if st["k_scale"] is None:
        return [st["k_cache"], st["v_cache"]]
    return [torch.mul(st["k_cache"], st["k_scale"][..., None]), torch.mul(st["v_cache"], st["v_scale"][..., None]),
            st["k_scale"], st["v_scale"]]


def _plain_q4g(st):
    K, G = st["case"]["K"], st["case"]["group"]
    codes = st["codes"]
    q = torch.stack([codes & 15, codes >> 4], -1).flatten(1)[:, :K].float()
    of = torch.arange(K, device=DEV) // G
    zero = 8.0 if st["zeros"] is None else st["zeros"].float()[:, of]
    W = (q - zero) * st["scales"].float()[:, of]
    return (st["X"].float() @ W.t()).to(st["X"].dtype)


def _plain_plan(st):
    P, T, table, free = st["case"]["page"], st["tokens"], st["table"], st["free"]
    ctx, new = st["ctx"].long(), st["new"].long()
    W, F = table.shape[1], free.numel()
    total = ctx + new
    have, need = (ctx + P - 1) // P, (total + P - 1) // P
    take = need - have
    first = take.cumsum(0) - take
    j = torch.arange(W, device=DEV)[None]
    at = first[:, None] + j - have[:, None]
    fresh = (j >= have[:, None]) & (j < need[:, None])
    table.copy_(torch.where(fresh, free[at.clamp(0, F - 1)], table))
    ends = new.cumsum(0)
    cu = torch.cat([ends.new_zeros(1), ends])
    t = torch.arange(T, device=DEV)
    r = torch.searchsorted(ends, t, right=True)
    pos = ctx[r] + t - cu[r]
    slots = table[r, pos // P].long() * P + pos % P
    info = torch.stack([take.sum(), ends[-1], torch.zeros_like(ends[-1]), total.max()])
    return [table, cu.int(), slots, pos.int(), info.int()]


def _plain_append(st):
    D = st["case"]["dim"]
    kc, vc = st["k_cache"], st["v_cache"]
    P, at = kc.shape[1], st["slots"]
    k, v = st["K"].float(), st["V"].float()
    if st["k_scale"] is not None:
        (k, ks), (v, vs) = _rows_s8(k), _rows_s8(v)
        st["k_scale"][at // P, at % P], st["v_scale"][at // P, at % P] = ks, vs
    kc[at // P, at % P], vc[at // P, at % P] = k.to(kc.dtype), v.to(vc.dtype)
    return _cache_values(st)


def _gather(cache, scale, slot, P):
    """Cached rows [R, H, L, D] of the slots [R, L] in 32 bits."""
    x = cache[slot // P, slot % P].float()
    if scale is not None:
        x = x * scale[slot // P, slot % P][..., None]
    return x.transpose(1, 2)


def _plain_tree(st):
    case = st["case"]
    R, P, Hq, Hkv, D = case["R"], case["page"], case["hq"], case["hkv"], case["dim"]
    L, most, q = st["longest"], st["most"], st["q"]
    G, T = Hq // Hkv, q.shape[0]
    ctx, cu = st["ctx"].long(), st["cu"].long()
    new = cu[1:] - cu[:-1]
    # query rows of each request, padded to the most drafted tokens of any
    i = torch.arange(most, device=DEV)[None]
    row = (cu[:-1, None] + i).clamp(max=T - 1)
    real = i < new[:, None]
    x = q.float()[row].view(R, most, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(R, Hkv, most * G, D)
    # cached rows of each request, padded to the longest
    j = torch.arange(L, device=DEV)
    page = st["table"].long()[:, j // P].clamp(min=0)
    slot = page * P + j % P
    k, v = _gather(st["k_cache"], st["k_scale"], slot, P), _gather(st["v_cache"], st["v_scale"], slot, P)
    # what each drafted token sees: the context, and drafted tokens by the mask (or all up to itself)
    d = j[None, None] - ctx[:, None, None]
    drafted = (d >= 0) & (d < new[:, None, None])
    if st["mask"] is None:
        sees = drafted & (d <= i[..., None])
    else:
        m = st["mask"][row]
        sees = drafted & torch.gather(m, 2, d.clamp(0, m.shape[2] - 1).expand(R, most, L))
    sees = ((d < 0) | sees).repeat_interleave(G, 1)[:, None]
    s = torch.where(sees, x @ k.transpose(-1, -2) * (1.0 / math.sqrt(D)), -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top == -math.inf, 0.0, top))
    o = p @ v / p.sum(-1, keepdim=True).clamp(min=1e-30)
    o = o.view(R, Hkv, most, G, D).permute(0, 2, 1, 3, 4).reshape(R, most, Hq, D)
    out = q.new_zeros(T + 1, Hq, D)
    out[torch.where(real, row, T)] = o.to(q.dtype)
    return out[:T]


# ------------------------------------------------------------------ exact ---

def exact(case, seed):
    st = prepare(case, seed)
    return {"q4g": _exact_q4g, "plan": _exact_plan, "append": _exact_append, "tree": _exact_tree}[case["op"]](case, st)


def _exact_q4g(case, st):
    # group by group: s (sum q x - z sum x)
    M, K, N, G = case["M"], case["K"], case["N"], case["group"]
    x = st["X"].double()
    y = torch.zeros(M, N, dtype=torch.float64, device=DEV)
    even, odd = (st["codes"] & 15).double(), (st["codes"] >> 4).double()
    for g in range(-(-K // G)):
        lo, hi = g * G, min(K, g * G + G)
        a, b = x[:, lo:hi:2], x[:, lo + 1:hi:2]
        dot = a @ even[:, lo // 2:lo // 2 + a.shape[1]].t() + b @ odd[:, lo // 2:lo // 2 + b.shape[1]].t()
        z = 8.0 if st["zeros"] is None else st["zeros"][:, g].double()
        y += st["scales"][:, g].double() * (dot - z * x[:, lo:hi].sum(1, keepdim=True))
    return y


def _exact_plan(case, st):
    P = case["page"]
    ctx, new = st["ctx"].tolist(), st["new"].tolist()
    table, free = st["table"].cpu().numpy().copy(), st["free"].tolist()
    taken, cu, slots, positions = 0, [0], [], []
    for r, (c, n) in enumerate(zip(ctx, new)):
        for pos in range(c, c + n):
            if pos % P == 0:
                table[r, pos // P] = free[taken]
                taken += 1
            slots.append(int(table[r, pos // P]) * P + pos % P)
            positions.append(pos)
        cu.append(cu[-1] + n)
    info = [taken, cu[-1], 0, max(c + n for c, n in zip(ctx, new))]
    return [torch.from_numpy(table), torch.tensor(cu, dtype=torch.int32), torch.tensor(slots, dtype=torch.int64),
            torch.tensor(positions, dtype=torch.int32), torch.tensor(info, dtype=torch.int32)]


def _exact_append(case, st):
    out, scales = [], []
    slots = st["slots"]
    for x in (st["K"], st["V"]):
        x = x.double()
        pages = st["k_cache"].shape[0]
        values = torch.zeros(pages * case["page"], case["heads"], case["dim"], dtype=torch.float64, device=DEV)
        scale = torch.zeros(pages * case["page"], case["heads"], dtype=torch.float64, device=DEV)
        if case["c"] == "s8":
            s = (x.abs().amax(-1) / 127).float().double()  # the scale and the quotient are fp32 by definition
            scale[slots] = s
            x = torch.clamp(torch.round((x / s[..., None]).float()), -127, 127).double() * s[..., None]
        values[slots] = x
        out.append(values.view(pages, case["page"], case["heads"], case["dim"]))
        scales.append(scale.view(pages, case["page"], case["heads"]))
    return out + scales if case["c"] == "s8" else out


def _exact_tree(case, st):
    P, Hq, Hkv, D = case["page"], case["hq"], case["hkv"], case["dim"]
    G = Hq // Hkv
    cu, ctx = st["cu"].tolist(), st["ctx"].tolist()
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV)
    for r in range(case["R"]):
        n, length = cu[r + 1] - cu[r], ctx[r] + cu[r + 1] - cu[r]
        if n == 0:
            continue
        pages = st["table"][r, :-(-length // P)].long()
        sees = torch.ones(n, length, dtype=torch.bool, device=DEV)
        sees[:, ctx[r]:] = torch.ones(n, n, device=DEV).tril().bool() if st["mask"] is None else st["mask"][cu[r]:cu[r + 1], :n]
        for h in range(Hkv):
            k = st["k_cache"][pages, :, h].reshape(-1, D)[:length].double()
            v = st["v_cache"][pages, :, h].reshape(-1, D)[:length].double()
            if case["c"] == "s8":
                k = k * st["k_scale"][pages, :, h].reshape(-1, 1)[:length].double()
                v = v * st["v_scale"][pages, :, h].reshape(-1, 1)[:length].double()
            for i in range(G):
                s = st["q"][cu[r]:cu[r + 1], h * G + i].double() @ k.t() / math.sqrt(D)
                w = torch.softmax(s.masked_fill(~sees, -math.inf), -1)
                out[cu[r]:cu[r + 1], h * G + i] = w @ v
    return out
