"""One attention layer through a prompt and steps that verify drafted tokens.

    python examples/verify_step.py [--requests 4] [--prompt 300] [--drafts 7] [--steps 3] [--cache bf16|int8|q4]

The layer has the Qwen3-0.6B shapes (hidden 1024, 16 query over 8 key/value
heads of 128; norms and rotary embeddings are left out, so the layer is
x + o(attention(q(x), k(x), v(x)))).  Its four projections are 4-bit weights with
group scales.  Every call is one of int8_bit_weight_amd's:

    kv_plan          pages and slots of the new tokens, from lengths on the GPU
    q4_group_matmul  q, k, v
    kv_append        the new rows of K and V into the paged cache
    tree_attention   the new tokens over the cache: causal for the prompt, by the
                     tree's mask for drafted tokens
    q4_group_matmul  o

After a step the accepted tokens of each request are the ones on one path of its
tree; their rows are moved together by appending them again at the accepted
positions, and the lengths grow by their number.  The result of every step is
compared with a plain fp32 computation of the same layer: the largest error
relative to the layer's output, and the attention branch's, y - x, relative to that
branch's own size, which shows what the residual would hide.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import int8_bit_weight_amd as qmm  # noqa: E402

HIDDEN, Q_HEADS, KV_HEADS, DIM, GROUP, PAGE = 1024, 16, 8, 128, 128, 16


class Projection:
    """A random 4-bit weight [K, N] and its plain fp32 form."""

    def __init__(self, g, K, N):
        codes = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
        scales = ((torch.rand(N, K // GROUP, generator=g, device="cuda") + 0.5) / (4.6 * K ** 0.5)).bfloat16()
        zeros = torch.randint(6, 10, (N, K // GROUP), generator=g, device="cuda", dtype=torch.uint8)
        self.W = qmm.q4_group_repack(codes, scales, zeros, K=K, group=GROUP)
        q = torch.stack([codes & 15, codes >> 4], -1).flatten(1).float()
        self.plain = ((q - zeros.float().repeat_interleave(GROUP, 1)) * scales.float().repeat_interleave(GROUP, 1)).t()

    def __call__(self, x):
        return qmm.q4_group_matmul(x, self.W)


def tree(g, n):
    """Parents of n drafted tokens, and mask[i, j]: j is i or an ancestor of it."""
    parents, mask = [], torch.zeros(n, n, dtype=torch.bool)
    for i in range(n):
        p = -1 if i == 0 else int(torch.randint(max(-1, i - 3), i, (1,), generator=g))
        parents.append(p)
        if p >= 0:
            mask[i] = mask[p]
        mask[i, i] = True
    return parents, mask


def plain_layer(w, x, seen):
    """The layer on one request's rows x (context and new): seen[i, j], new row i sees row j."""
    q = (x[-seen.shape[0]:] @ w["q"].plain).view(-1, KV_HEADS, Q_HEADS // KV_HEADS, DIM)
    k, v = ((x @ w[n].plain).view(-1, KV_HEADS, DIM) for n in "kv")
    s = torch.einsum("thgd,jhd->hgtj", q, k) / DIM ** 0.5
    p = torch.softmax(s.masked_fill(~seen, -float("inf")), -1)
    return x[-seen.shape[0]:] + torch.einsum("hgtj,jhd->thgd", p, v).reshape(-1, Q_HEADS * DIM) @ w["o"].plain


def run(requests=4, prompt=300, drafts=7, steps=3, cache="bf16", seed=1, verbose=False, record=None):
    """Returns the largest error of any step, relative to the layer's largest output.  record: a list that gets, for
    each step and request, its accepted rows, new rows, what they see, the output, which new rows it keeps and the
    plain weights."""
    g, cpu = torch.Generator("cuda").manual_seed(seed), torch.Generator().manual_seed(seed)
    w = dict(q=Projection(g, HIDDEN, Q_HEADS * DIM), k=Projection(g, HIDDEN, KV_HEADS * DIM),
             v=Projection(g, HIDDEN, KV_HEADS * DIM), o=Projection(g, Q_HEADS * DIM, HIDDEN))
    longest = prompt + (steps + 1) * drafts
    width = -(-longest // PAGE)
    pages = requests * width
    ct, width_of_row = {"bf16": (torch.bfloat16, DIM), "int8": (torch.int8, DIM), "q4": (torch.uint8, DIM // 2)}[cache]
    kc, vc = (torch.zeros(pages, PAGE, KV_HEADS, width_of_row, dtype=ct, device="cuda") for _ in range(2))
    ks = vs = None
    if cache == "int8":
        ks, vs = (torch.zeros(pages, PAGE, KV_HEADS, device="cuda") for _ in range(2))
    elif cache == "q4":
        ks, vs = (torch.zeros(pages, PAGE, KV_HEADS, 2, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = torch.full((requests, width), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(pages, generator=g, device="cuda").int()
    taken = torch.zeros(1, dtype=torch.int32, device="cuda")
    ctx = torch.zeros(requests, dtype=torch.int32, device="cuda")
    rows = [torch.zeros(0, HIDDEN, dtype=torch.bfloat16, device="cuda") for _ in range(requests)]  # accepted inputs
    worst = 0.0

    def layer(x, new, mask):
        nonlocal taken
        plan = qmm.kv_plan(ctx, new, table, free, PAGE, x.shape[0], free_begin=taken)
        taken = plan.info[0:1]
        q, k, v = (w[n](x) for n in "qkv")
        qmm.kv_append(k.view(-1, KV_HEADS, DIM), v.view(-1, KV_HEADS, DIM), plan.slots, kc, vc, ks, vs)
        a = qmm.tree_attention(q.view(-1, Q_HEADS, DIM), kc, vc, table, ctx, plan.cu_new, mask, k_scale=ks, v_scale=vs)
        return x + w["o"](a.view(-1, Q_HEADS * DIM)), k, v

    for step in range(steps + 1):
        n = prompt if step == 0 else drafts
        x = torch.randn(requests * n, HIDDEN, generator=g, device="cuda").bfloat16()
        new = torch.full((requests,), n, dtype=torch.int32, device="cuda")
        trees = None if step == 0 else [tree(cpu, n) for _ in range(requests)]
        mask = None if step == 0 else torch.cat([m for _, m in trees]).cuda()
        torch.cuda.synchronize()
        t = time.perf_counter()
        y, k, v = layer(x, new, mask)
        torch.cuda.synchronize()
        t = time.perf_counter() - t
        # plain check, then what each request keeps: the prompt, or one path of its tree
        keep, off, size = [], 0.0, 0.0
        for r in range(requests):
            xr = torch.cat([rows[r], x[r * n:(r + 1) * n]])
            seen = torch.ones(n, xr.shape[0], dtype=torch.bool, device="cuda")
            seen[:, -n:] = torch.ones(n, n, device="cuda").tril().bool() if step == 0 else trees[r][1].cuda()
            want = plain_layer(w, xr.float(), seen)
            error, mine = y[r * n:(r + 1) * n].float() - want, x[r * n:(r + 1) * n]
            worst = max(worst, float(error.abs().max() / want.abs().max()))
            off, size = off + float(error.square().sum()), size + float((want - mine.float()).square().sum())
            path = list(range(n)) if step == 0 else trees[r][1][int(torch.randint(0, n, (1,), generator=cpu))].nonzero().flatten().tolist()
            keep.append([r * n + i for i in path])
            if record is not None:
                record.append(dict(step=step, request=r, accepted=rows[r], new=mine, seen=seen, y=y[r * n:(r + 1) * n],
                                   path=path, plain={k: p.plain for k, p in w.items()}))
            rows[r] = torch.cat([rows[r], x[keep[-1]]])
        if step > 0:  # accepted rows of K and V to the accepted positions, on pages that the step has taken
            at = torch.tensor([i for p in keep for i in p], device="cuda")
            slots = torch.cat([table[r, pos // PAGE].long() * PAGE + pos % PAGE for r, p in enumerate(keep)
                               for pos in [int(ctx[r]) + torch.arange(len(p), device="cuda")]])
            qmm.kv_append(k[at].view(-1, KV_HEADS, DIM), v[at].view(-1, KV_HEADS, DIM), slots, kc, vc, ks, vs)
            # pages that hold no accepted token go back to the free list
            used = -(-(ctx + torch.tensor([len(p) for p in keep], device="cuda").int()) // PAGE)
            have = -(-(ctx + new) // PAGE)
            for r in range(requests):
                spare = table[r, int(used[r]):int(have[r])]
                free = torch.cat([free, spare])
        ctx += torch.tensor([len(p) for p in keep], dtype=torch.int32, device="cuda")
        if verbose:
            print("step %d: %d tokens, %.0f us, lengths %s, error so far %.2e, of the attention branch %.2e"
                  % (step, x.shape[0], t * 1e6, ctx.tolist(), worst, (off / size) ** 0.5))
    return worst


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    for name, default in (("requests", 4), ("prompt", 300), ("drafts", 7), ("steps", 3)):
        ap.add_argument("--" + name, type=int, default=default)
    ap.add_argument("--cache", choices=("bf16", "int8", "q4"), default="bf16")
    a = ap.parse_args()
    print("largest error relative to the largest output: %.2e" % run(a.requests, a.prompt, a.drafts, a.steps, a.cache, verbose=True))
