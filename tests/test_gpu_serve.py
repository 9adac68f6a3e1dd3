"""GPU parity of the drafted-token verification operators against their plain
64-bit forms (tests/serve_ref.py).

Bounds.  A rounding to a type is off by at most eps/2 of the value.
  * group product: each output is rounded once to its type; before that, at
    most 48 + K/128 fp32 additions (32 products and 4 steps of one matrix
    accumulation, the groups of a wavefront, 8 to 16 wavefronts) over terms
    whose sizes add up to `bound`.  Over many outputs these roundings are
    independent: a group's partial sums of sqrt(128) * 24 * |x| against a
    result of sqrt(K) * 4.6 * |x| give a relative 2-norm error of about
    8.4 * 2^-24; four times that is asserted for fp32.
  * attention: one rounding of the output; weights held to 2^-16 (two 8-bit
    terms, or fp32); a score's fp32 sum of D products, which moves a weight by
    the same relative amount.
  * int8 rows, 16-bit rows, plans: equal.
"""
import numpy as np
import pytest
import torch

import serve_ref as ref
from gpu_util import to_dev, to_np, torch_dev

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
U = 2.0 ** -24


@pytest.fixture(scope="module")
def q():
    import int8_bit_weight_amd as q
    return q


def f64(t):
    torch.cuda.synchronize()
    return t.detach().double().cpu().numpy()


# ----------------------------------------------------------- group product ---

def _weight(g, K, N, group, zeros, st):
    codes = torch.from_numpy(g.integers(0, 256, (N, (K + 1) // 2)).astype(np.uint8))
    groups = -(-K // group)
    s = torch.from_numpy((g.random((N, groups)) + 0.5) * 0.01 * g.choice([-1.0, 1.0], (N, groups))).to(st)
    z = torch.from_numpy(g.integers(0, 16, (N, groups)).astype(np.uint8)) if zeros else None
    return codes, s, z


def _check_product(Y, X, codes, s, z, K, group):
    want, size = ref.q4_group_matmul(f64(X), codes.numpy(), s.double().numpy(), None if z is None else z.numpy(), K, group)
    got = f64(Y)
    tol = torch.finfo(Y.dtype).eps / 2 * np.abs(want) + (48 + K / 128) * U * size
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= tol).all(), float((np.abs(got - want) / tol).max())
    if Y.dtype == F32 and K >= 256 and want.size >= 64:
        assert np.linalg.norm(got - want) <= 4 * 8.4 * U * np.linalg.norm(want)


PRODUCTS = [(1, 128, 16, 128), (1, 1, 1, 32), (1, 7, 3, 32), (2, 33, 17, 64), (1, 1000, 300, 128), (3, 4100, 70, 32),
            (5, 515, 129, 128), (1, 2048, 1024, 128), (16, 2048, 100, 64), (17, 640, 48, 256), (33, 1032, 257, 32),
            (64, 1024, 272, 128), (7, 14336, 33, 128), (1, 14336, 530, 64), (70, 520, 40, 128), (130, 256, 64, 64),
            (1, 384, 20000, 128), (4, 900, 5, 4096), (9, 2056, 4099, 32)]


@pytest.mark.parametrize("xt", [F32, F16, BF16], ids=["f32", "f16", "bf16"])
@pytest.mark.parametrize("M,K,N,group", PRODUCTS)
def test_group_product(q, M, K, N, group, xt):
    g = np.random.default_rng(M * 7 + K + N)
    for zeros, st in ((True, F16), (False, BF16)):
        codes, s, z = _weight(g, K, N, group, zeros, st)
        W = q.q4_group_repack(to_dev(codes.numpy()), s.to(torch_dev()), None if z is None else to_dev(z.numpy()), K=K, group=group)
        X = torch.from_numpy(g.standard_normal((M, K))).to(xt).to(torch_dev())
        _check_product(q.q4_group_matmul(X, W), X, codes, s, z, K, group)


@pytest.mark.parametrize("xt", [F32, F16, BF16], ids=["f32", "f16", "bf16"])
@pytest.mark.parametrize("M,K,N,group", [(64, 14336, 100, 64), (33, 5000, 2100, 32), (40, 4104, 1000, 256), (128, 1920, 130, 64),
                                         (17, 10000, 40, 10112), (2, 1028, 4200, 64), (16, 8200, 31, 32)])
def test_group_product_split(q, M, K, N, group, xt):
    """Sizes whose records are split over workgroups, odd numbers of records in a range, one group per column."""
    g = np.random.default_rng(M + K)
    codes, s, z = _weight(g, K, N, group, True, F16)
    W = q.q4_group_repack(to_dev(codes.numpy()), s.to(torch_dev()), to_dev(z.numpy()), K=K, group=group)
    X = torch.from_numpy(g.standard_normal((M, K))).to(xt).to(torch_dev())
    _check_product(q.q4_group_matmul(X, W), X, codes, s, z, K, group)
    # a workspace of the caller's with any contents, and the same bits again
    ws = torch.full((max(1, q.lib.qmm_q4_group_matmul_workspace_bytes(M, K, N, group, q._DTYPES[xt])),), 255, dtype=torch.uint8,
                    device=torch_dev())
    assert torch.equal(q.q4_group_matmul(X, W, ws=ws), q.q4_group_matmul(X, W))


@pytest.mark.parametrize("xt", [F32, F16, BF16], ids=["f32", "f16", "bf16"])
def test_group_product_strides_and_neighbours(q, xt):
    """Misaligned rows and outputs, padded leading dimensions; what lies beside the output stays, and NaN
    beside the activations does not get in."""
    g = np.random.default_rng(5)
    for M, K, N, off in ((3, 264, 40, 1), (16, 1024, 130, 8), (20, 1001, 64, 3), (1, 136, 16, 5)):
        codes, s, z = _weight(g, K, N, 128, True, F16)
        W = q.q4_group_repack(to_dev(codes.numpy()), s.to(torch_dev()), to_dev(z.numpy()), K=K, group=128)
        big = torch.full((M + 2, K + 24), float("nan"), dtype=xt, device=torch_dev())
        X = big[1:M + 1, off:off + K]
        X.copy_(torch.from_numpy(g.standard_normal((M, K))).to(xt))
        room = torch.full((M + 2, N + 9), 7.0, dtype=xt, device=torch_dev())
        out = room[1:M + 1, 3:3 + N]
        assert q.q4_group_matmul(X, W, out=out) is out
        _check_product(out, X, codes, s, z, K, 128)
        room[1:M + 1, 3:3 + N] = 7.0
        assert (room == 7.0).all()


def test_group_product_extremes(q):
    """Every code against every zero; rows of zeros; fp16's subnormals and largest values; a NaN row stays its own."""
    N, K = 16, 32
    codes = np.tile(np.arange(16, dtype=np.uint8) | (np.arange(16, dtype=np.uint8) << 4), (N, 1))
    z = np.arange(16, dtype=np.uint8)[:, None]
    W = q.q4_group_repack(to_dev(codes), torch.ones(N, 1, dtype=F16, device=torch_dev()), to_dev(z), K=K, group=32)
    eye = torch.eye(K, device=torch_dev())
    for xt in (F32, F16, BF16):
        Y = q.q4_group_matmul(eye.to(xt), W)
        want = np.repeat(np.arange(16.0), 2)[:, None] - np.arange(16.0)[None]
        assert np.array_equal(f64(Y), want)
    X = torch.zeros(4, K, dtype=F16, device=torch_dev())
    X[1, 5], X[2, 0], X[3] = 2.0 ** -24, 60000.0, float("nan")
    Y = f64(q.q4_group_matmul(X, W))
    assert not Y[0].any() and np.isnan(Y[3]).all()
    assert np.array_equal(Y[1], 2.0 ** -24 * (2 - np.arange(16.0)))
    want = (60000.0 * (0 - np.arange(16.0))).astype(np.float16).astype(np.float64)
    assert np.array_equal(Y[2], want)


# -------------------------------------------------------------------- plan ---

def _check_plan(q, ctx, new, table, free, page, T, begin=None):
    want = ref.kv_plan(ctx, new, table, free, page, T, begin or 0)
    tab = to_dev(table)
    b = None if begin is None else torch.tensor([begin], dtype=torch.int32, device=torch_dev())
    plan = q.kv_plan(to_dev(ctx), to_dev(new), tab, to_dev(free), page, T, free_begin=b)
    for name, got, w in zip(("table", "cu_new", "slots", "positions", "info"),
                            (tab, plan.cu_new, plan.slots, plan.positions, plan.info), want):
        assert np.array_equal(to_np(got), w), name


def _plan_case(g, R, max_ctx, max_new, page):
    ctx = g.integers(0, max_ctx + 1, R).astype(np.int32)
    new = g.integers(0, max_new + 1, R).astype(np.int32)
    width = max(1, int(max(-(-(int(c) + int(n)) // page) for c, n in zip(ctx, new))))
    have = [-(-int(c) // page) for c in ctx]
    free = g.permutation(sum(have) + R * (max_new // page + 2)).astype(np.int32)
    table = np.full((R, width), -1, np.int32)
    at = 0
    for r in range(R):
        table[r, :have[r]] = free[at:at + have[r]]
        at += have[r]
    return ctx, new, table, free[at:].copy()


@pytest.mark.parametrize("R,max_ctx,max_new,page", [(1, 0, 1, 16), (1, 100, 1, 16), (3, 50, 20, 1), (64, 500, 16, 16),
                                                    (255, 90, 9, 24), (257, 0, 40, 16), (1000, 64, 3, 7),
                                                    (8192, 20, 2, 16), (5, 3000, 4000, 128)])
def test_plan(q, R, max_ctx, max_new, page):
    g = np.random.default_rng(R + page)
    ctx, new, table, free = _plan_case(g, R, max_ctx, max_new, page)
    T = int(new.astype(np.int64).sum())
    _check_plan(q, ctx, new, table, free, page, T)
    _check_plan(q, ctx, new, table, free, page, T + 1500)          # room for more tokens: slots of -1
    _check_plan(q, ctx, new, table, free, page, T // 2)            # and for fewer
    _check_plan(q, ctx, new, table, free, page, T, begin=2)
    _check_plan(q, ctx, new, table, free[:R // 2], page, T)        # too few pages
    _check_plan(q, ctx, new, table, free, page, T, begin=len(free) + 5)
    if table.shape[1] > 1:
        _check_plan(q, ctx, new, np.ascontiguousarray(table[:, :-1]), free, page, T)  # too narrow a table


def test_plan_many_tokens(q):
    """More tokens than one thread each: the form of four tokens a thread, with and without tokens to fill it."""
    g = np.random.default_rng(77)
    ctx, new, table, free = _plan_case(g, 300, 500, 2200, 16)
    T = int(new.astype(np.int64).sum())
    assert T > 256 * 1024
    _check_plan(q, ctx, new, table, free, 16, T)
    ctx, new, table, free = _plan_case(g, 40, 90, 30, 24)
    _check_plan(q, ctx, new, table, free, 24, 300000)


def test_plan_odd_input(q):
    i = lambda *v: np.array(v, np.int32)  # noqa: E731
    free = np.arange(50, dtype=np.int32)
    _check_plan(q, i(-3, 5, 2), i(4, -7, 3), np.full((3, 4), -1, np.int32), free, 4, 10)
    _check_plan(q, i(), i(), np.zeros((0, 4), np.int32), free, 4, 3)
    _check_plan(q, i(0, 0), i(0, 0), np.full((2, 4), -1, np.int32), free, 4, 0)
    _check_plan(q, i(3), i(9), np.zeros((1, 0), np.int32), free, 4, 9)
    _check_plan(q, i(2 ** 31 - 1, 7), i(6, 2), np.full((2, 4), 3, np.int32), free, 4, 40)
    # a wider row than the table is used, in place
    big = torch.full((3, 9), 77, dtype=torch.int32, device=torch_dev())
    plan = q.kv_plan(to_dev(i(0, 4, 8)), to_dev(i(5, 1, 1)), big[:, 2:6], to_dev(free), 4, 7)
    assert (to_np(big)[:, [0, 1, 6, 7, 8]] == 77).all()
    assert to_np(big)[:, 2:6].tolist() == [[0, 1, 77, 77], [77, 2, 77, 77], [77, 77, 3, 77]]
    assert to_np(plan.slots).tolist() == [0, 1, 2, 3, 4, 8, 12]


# ------------------------------------------------------------------ append ---

@pytest.mark.parametrize("ct", [F16, BF16, torch.int8], ids=["c_f16", "c_bf16", "c_s8"])
@pytest.mark.parametrize("xt", [F32, F16, BF16], ids=["x_f32", "x_f16", "x_bf16"])
@pytest.mark.parametrize("T,H,D,page", [(1, 1, 8, 1), (5, 3, 80, 7), (33, 8, 128, 16), (2, 2, 256, 64), (300, 1, 64, 16)])
def test_append(q, T, H, D, page, xt, ct):
    g = np.random.default_rng(T + D)
    pages = -(-T // page) + 2
    for order in ("nhd", "hnd"):
        caches, scales = [], []
        for _ in range(2):
            shape = (pages, page, H, D) if order == "nhd" else (pages, H, page, D)
            c = torch.full(shape, 3, dtype=ct, device=torch_dev())
            s = torch.full(shape[:3], 9.0, device=torch_dev())
            caches.append(c if order == "nhd" else c.transpose(1, 2))
            scales.append(s if order == "nhd" else s.transpose(1, 2))
        x = [torch.from_numpy(g.standard_normal((T, 2 * H, D + 8))).to(xt).to(torch_dev()) for _ in range(2)]
        if T > 4:
            x[0][1] = 0
            x[1][2, 0, 3] = float("inf")
            x[1][3, 0, 3] = float("nan")
        off = 0 if order == "nhd" else 3                            # a misaligned source too
        K, V = (t[:, H:, off:off + D] for t in x)
        slots = g.permutation(pages * page)[:T].astype(np.int64)
        if T > 4:
            slots[4], slots[0] = -1, pages * page                   # rows to skip
        sc = scales if ct == torch.int8 else [None, None]
        q.kv_append(K, V, to_dev(slots), caches[0], caches[1], *sc)
        for src, c, s in zip((K, V), caches, scales):
            want = torch.full((pages * page, H, D), 3, dtype=ct)
            wants = torch.full((pages * page, H), 9.0)
            for t in range(T):
                if 0 <= slots[t] < pages * page:
                    if ct == torch.int8:
                        row = src[t].float().cpu().numpy()
                        codes, scale = ref.quantize_rows(row)
                        codes[~np.isfinite(scale)] = 0
                        want[slots[t]], wants[slots[t]] = torch.from_numpy(codes), torch.from_numpy(scale)
                    else:
                        want[slots[t]] = src[t].float().cpu().to(ct)
            got = c.reshape(pages * page, H, D).cpu()
            assert torch.equal(torch.nan_to_num(got.float(), 1e30), torch.nan_to_num(want.float(), 1e30))
            if ct == torch.int8:
                assert np.array_equal(s.reshape(pages * page, H).cpu().numpy(), wants.numpy(), equal_nan=True)


# --------------------------------------------------------------- attention ---

class Batch:
    """Requests, their tables and filled caches, with a plain copy of each request's keys and values."""

    def __init__(self, g, ctx, new, Hq, Hkv, D, page, ct, masks="tree", order="nhd", cols=None, spare_rows=0, std=2.0):
        self.ctx, self.new, self.Hq, self.Hkv, self.D, self.page, self.ct = ctx, new, Hq, Hkv, D, page, ct
        R = len(ctx)
        need = [-(-(c + n) // page) for c, n in zip(ctx, new)]
        self.width = max(max(need), 1)
        pages = sum(need) + 3
        ids = g.permutation(pages).astype(np.int32)
        self.table = np.full((R, self.width), -1, np.int32)
        at = 0
        for r in range(R):
            self.table[r, :need[r]] = ids[at:at + need[r]]
            at += need[r]
        shape = (pages, page, Hkv, D)
        self.kv, self.scales = [], []
        for _ in range(2):
            x = torch.from_numpy(g.standard_normal(shape).astype(np.float32))
            s = None
            if ct == torch.int8:
                c, s = ref.quantize_rows(x.numpy())
                x, s = torch.from_numpy(c), torch.from_numpy(s)
            else:
                x = x.to(ct)
            self.kv.append(x)
            self.scales.append(s)
        self.T = sum(new) + spare_rows
        self.xt = BF16 if ct == torch.int8 else ct
        self.q = torch.from_numpy(g.standard_normal((self.T, Hq, D)) * std).to(self.xt)
        self.cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.mask = None
        if masks is not None:
            cols = max(max(new), 1) if cols is None else cols
            self.mask = g.random((self.T, cols)) < 0.5           # what lies outside the trees is noise
            for r in range(R):
                m = ref.random_tree(g, new[r]) if masks == "tree" else g.random((new[r], new[r])) < 0.4
                if masks == "none":
                    m[:] = False
                n = min(cols, new[r])
                self.mask[self.cu[r]:self.cu[r + 1], :n] = m[:, :n]
        self.order = order

    def dev(self, x):
        if x is None:
            return None
        if self.order == "hnd":
            return x.transpose(1, 2).contiguous().to(torch_dev()).transpose(1, 2)
        if self.order == "wide":                                  # heads of a wider tensor, padded rows
            wide = torch.zeros(x.shape[0], x.shape[1] + 1, x.shape[2] + 2, *[d + 8 for d in x.shape[3:]], dtype=x.dtype, device=torch_dev())
            view = wide[:, :x.shape[1], 1:-1]
            view = view[..., 8:] if x.dim() == 4 else view
            view.copy_(x.to(torch_dev()))
            return view
        return x.to(torch_dev())

    def run(self, q, scale=None, **kw):
        (k, v), (ks, vs) = [self.dev(x) for x in self.kv], [self.dev(x) for x in self.scales]
        mask = None if self.mask is None else to_dev(self.mask)
        return q.tree_attention(self.q.to(torch_dev()), k, v, to_dev(self.table), to_dev(np.array(self.ctx, np.int32)),
                                to_dev(self.cu), mask, scale, k_scale=ks, v_scale=vs, **kw)

    def check(self, out, scale=None):
        scale = self.D ** -0.5 if scale is None else scale
        got = f64(out)
        G, pages = self.Hq // self.Hkv, self.kv[0].shape[0]
        worst = 0.0
        for r, (c, n) in enumerate(zip(self.ctx, self.new)):
            L = min(c + n, self.width * self.page)
            pos = np.arange(L)
            page = self.table[r, pos // self.page]
            ok = (page >= 0) & (page < pages)
            rows = []
            for x, s in zip(self.kv, self.scales):
                y = x.double().numpy()[np.where(ok, page, 0), pos % self.page]
                if s is not None:
                    y = y * s.double().numpy()[np.where(ok, page, 0), pos % self.page][..., None]
                rows.append(y)
            for i in range(n):
                t = self.cu[r] + i
                sees = ok & (pos < c)
                for j in range(max(0, L - c)):
                    seen = j <= i if self.mask is None else j < self.mask.shape[1] and self.mask[t, j]
                    sees[c + j] = ok[c + j] and seen
                for h in range(self.Hq):
                    o, size, dot = ref.tree_attention(self.q[t, h].double().numpy(), rows[0][:, h // G], rows[1][:, h // G], sees, scale)
                    delta = (self.D + 8) * U * dot
                    tol = torch.finfo(self.xt).eps / 2 * np.abs(o) + (2.0 ** -16 + 2 * delta + 64 * U) * size
                    tol = tol + torch.finfo(self.xt).smallest_normal * torch.finfo(self.xt).eps
                    err = np.abs(got[t, h] - o)
                    same = (err <= tol) | (np.isnan(o) & np.isnan(got[t, h]))
                    assert same.all(), (r, i, h, float(np.nanmax(err / tol)), got[t, h][:4], o[:4])
                    worst = max(worst, float(np.nanmax(err / tol)) if len(tol) else 0.0)
        return worst


TYPES = pytest.mark.parametrize("ct", [F16, BF16, torch.int8], ids=["f16", "bf16", "s8"])


@TYPES
@pytest.mark.parametrize("ctx,new,Hq,Hkv,D,page,masks", [
    ([0], [1], 1, 1, 64, 16, None),                      # one token that sees itself
    ([1], [1], 2, 1, 128, 16, None),
    ([37], [1], 16, 8, 128, 16, None),                   # one decoded token
    ([100, 0, 63, 64, 65], [1, 3, 0, 1, 2], 4, 2, 128, 16, None),
    ([5, 130, 33], [7, 16, 1], 4, 4, 64, 7, "tree"),     # pages that end inside every tile
    ([300, 17], [20, 33], 8, 2, 128, 24, "tree"),
    ([90], [70], 6, 2, 80, 1, "tree"),
    ([31, 200], [9, 5], 8, 1, 256, 32, "tree"),
    ([10, 0, 40], [6, 9, 3], 2, 2, 8, 16, "any"),        # rows with nothing drafted to see
    ([0, 0], [5, 1], 4, 2, 64, 16, "none"),              # rows that see nothing at all
    ([257], [130], 2, 1, 64, 64, None),                  # a chunk of a prompt
])
def test_attention(q, ctx, new, Hq, Hkv, D, page, masks, ct):
    b = Batch(np.random.default_rng(len(ctx) + D), ctx, new, Hq, Hkv, D, page, ct, masks)
    out = b.run(q)
    b.check(out)
    if masks == "none":
        assert not out.any()


@TYPES
def test_attention_many_requests(q, ct):
    """More requests than threads of a workgroup: ragged, new ones and ones that sit out among them."""
    g = np.random.default_rng(30)
    ctx = g.integers(0, 70, 600).tolist()
    new = g.integers(0, 3, 600).tolist()
    ctx[5] = ctx[6] = 0
    ctx[300] = 1500
    new[300], new[599] = 2, 2
    b = Batch(g, ctx, new, 2, 1, 64, 16, ct, "tree")
    b.check(b.run(q))


@TYPES
@pytest.mark.parametrize("D,page", [(64, 16), (80, 24), (128, 32), (256, 16)])
def test_attention_tiles_and_parts(q, ct, D, page):
    """Several row tiles to a cache head, and items that many workgroups share, in each head dimension."""
    g = np.random.default_rng(D)
    b = Batch(g, [700, 90, 0], [40, 3, 21], 8, 1, D, page, ct, "tree")
    b.check(b.run(q))
    b = Batch(g, [9001], [2], 2, 2, D, page, ct, "tree")
    out = b.run(q)
    b.check(out)
    ws = torch.full((q.lib.qmm_tree_attention_workspace_bytes(2, 2, 1, 2, D),), 255, dtype=torch.uint8, device=torch_dev())
    assert torch.equal(b.run(q, ws=ws), out)
    b = Batch(g, [3000], [33], 2, 1, D, page, ct, None)
    b.check(b.run(q))


@TYPES
def test_attention_hidden_nan_in_shared_items(q, ct):
    """NaN behind a mask where several workgroups share an item, beside requests that are whole and finite."""
    g = np.random.default_rng(31)
    b = Batch(g, [5000, 40, 2100], [6, 3, 20], 4, 2, 64, 16, ct, "tree")
    hidden = []
    for r, i in ((0, 3), (2, 11)):
        p = b.ctx[r] + i
        page, at = b.table[r, p // 16], p % 16
        if ct == torch.int8:
            b.scales[0][page, at] = b.scales[1][page, at] = float("nan")
        else:
            b.kv[0][page, at] = b.kv[1][page, at] = float("nan")
        rows = np.arange(b.cu[r], b.cu[r + 1])
        b.mask[rows, i] = rows % 2 == 0
        hidden += [t for t in rows if not b.mask[t, i]]
    out = b.run(q)
    assert hidden and torch.isfinite(out[hidden]).all() and torch.isfinite(out[b.cu[1]:b.cu[2]]).all()
    b.check(out)


@TYPES
@pytest.mark.parametrize("order", ["hnd", "wide"])
def test_attention_cache_orders(q, ct, order):
    b = Batch(np.random.default_rng(9), [70, 3], [5, 11], 6, 3, 64, 16, ct, "tree", order)
    b.check(b.run(q))


@TYPES
def test_attention_long_context(q, ct):
    """Lengths over which the work is split, ragged, with large and with equal scores."""
    g = np.random.default_rng(10)
    b = Batch(g, [5003, 0, 2048, 1], [4, 9, 1, 3], 4, 2, 128, 16, ct, "tree", std=6.0)
    b.check(b.run(q))
    b = Batch(g, [3001], [2], 2, 1, 64, 64, ct, "tree")
    b.q[:] = 0
    b.check(b.run(q))


@TYPES
def test_attention_scale_and_outputs(q, ct):
    """Another scale, a negative and a zero one; strided queries and outputs; rows past the last request stay."""
    g = np.random.default_rng(11)
    b = Batch(g, [50, 9], [6, 3], 4, 2, 64, 16, ct, "tree", spare_rows=2)
    for scale in (0.02, -0.1, 0.0):
        room = torch.full((b.T, 6, 72), 5.0, dtype=b.xt, device=torch_dev())
        out = room[:, 1:5, 3:67]
        assert b.run(q, scale, out=out) is out
        b.check(out, scale)
        assert (room[-2:] == 5.0).all()
        out.fill_(5.0)
        assert (room == 5.0).all()
    wide = torch.full((b.T, 5, 70), float("nan"), dtype=b.xt)
    wide[:, 1:, 1:65] = b.q
    b.q = wide[:, 1:, 1:65]
    keep = b.q
    qd = wide.to(torch_dev())[:, 1:, 1:65]
    (k, v), (ks, vs) = [b.dev(x) for x in b.kv], [b.dev(x) for x in b.scales]
    out = q.tree_attention(qd, k, v, to_dev(b.table), to_dev(np.array(b.ctx, np.int32)), to_dev(b.cu), to_dev(b.mask),
                           k_scale=ks, v_scale=vs)
    b.q = keep
    b.check(out)


@TYPES
def test_attention_masked_places_may_hold_anything(q, ct):
    """NaN and infinities in page tails, in unused pages and in drafted tokens that a row does not see stay
    out of it; a row that sees them has them."""
    g = np.random.default_rng(12)
    b = Batch(g, [20, 45], [6, 9], 4, 2, 64, 16, ct, "tree")
    bad = [float("nan"), float("inf"), float("-inf")]
    used = np.zeros(b.kv[0].shape[:2], bool)
    for r in range(2):
        for p in range(b.ctx[r] + b.new[r]):
            used[b.table[r, p // 16], p % 16] = True
    poison = [(i, j) for i, j in zip(*np.nonzero(~used))]
    # drafted token 4 of request 0 and token 7 of request 1 are hidden from half the rows
    for r, i in ((0, 4), (1, 7)):
        p = b.ctx[r] + i
        poison.append((b.table[r, p // 16], p % 16))
        rows = np.arange(b.cu[r], b.cu[r + 1])
        b.mask[rows, i] = rows % 2 == 0
    hidden = [t for r, i in ((0, 4), (1, 7)) for t in range(b.cu[r], b.cu[r + 1]) if not b.mask[t, i]]
    for n, (i, j) in enumerate(poison):
        if ct == torch.int8:
            b.scales[0][i, j], b.scales[1][i, j] = bad[n % 3], bad[(n + 1) % 3]
        else:
            b.kv[0][i, j], b.kv[1][i, j, :, ::3] = bad[n % 3], bad[(n + 1) % 3]
    out = b.run(q)
    assert hidden and torch.isfinite(out[hidden]).all()
    b.check(out)
    # finite keys, infinite values of one visible drafted token: only where they are seen, only where they are
    if ct != torch.int8:
        b = Batch(g, [20], [6], 4, 2, 64, 16, ct, "tree")
        b.mask[:, 2] = [True, False, True, False, True, False]
        p = b.ctx[0] + 2
        b.kv[1][b.table[0, p // 16], p % 16, 0, 5:9] = float("inf")
        out = b.run(q)
        assert torch.isfinite(out[1::2]).all() and torch.isfinite(out[:, 2:]).all()
        assert torch.isinf(out[0::2, :2, 5:9]).all() and torch.isfinite(out[:, :, 9:]).all()


@TYPES
def test_attention_bad_pages(q, ct):
    """Pages outside the cache, tables that are too narrow and mask columns that are missing hide keys."""
    g = np.random.default_rng(13)
    b = Batch(g, [60, 30, 5], [5, 4, 2], 4, 2, 64, 16, ct, "tree", cols=3)
    b.table[0, 1], b.table[0, 2] = -1, b.kv[0].shape[0]
    b.table[1, 0] = 2 ** 30
    b.check(b.run(q))
    b.table = np.ascontiguousarray(b.table[:, :2])
    b.width = 2
    b.check(b.run(q))
    b.table[:] = -5
    assert not b.run(q).any()
    b.mask = np.zeros((b.T, 0), bool)                                # no columns: a mask all the same
    b.table[:] = [[0, 1], [2, 3], [4, 5]]
    b.check(b.run(q))


def test_attention_scores_at_the_edges(q):
    """Scores of -inf weigh nothing; a row of nothing else is zeros; scores far apart."""
    g = np.random.default_rng(14)
    b = Batch(g, [40], [3], 2, 1, 64, 16, BF16, "tree")
    b.q[0, 0] = 0
    b.q[0, 0, 0] = 1.0
    b.kv[0][..., 0] = -float("inf")
    b.kv[0][b.table[0, 0], 3, 0] = 0.5
    b.q[1:] = 0
    b.q[1, :, 1] = 3e30
    b.q[1, 1] = -b.q[1, 1]
    b.kv[0][..., 1] = b.kv[0][..., 1].sign()
    b.q[1, :, 0] = 1.0
    b.q[2, :, 0] = 1.0
    out = b.run(q)
    assert torch.isfinite(out).all()
    b.check(out)
    b.kv[0][..., 0] = -float("inf")
    assert not b.run(q)[0, 0].any()


# ------------------------------------------------- as a program uses them ---

def _step(q, dev, g):
    """One verification step: plan, append, attention, projection; returns (call, outputs)."""
    R, Hq, Hkv, D, page, width = 5, 4, 2, 64, 16, 12
    ctx = torch.tensor([0, 17, 64, 100, 31], dtype=torch.int32, device=dev)
    new = torch.tensor([3, 4, 1, 0, 5], dtype=torch.int32, device=dev)
    T = 13
    table = torch.arange(R * width, dtype=torch.int32, device=dev).view(R, width)
    free = torch.arange(R * width, R * width + 20, dtype=torch.int32, device=dev)
    gen = torch.Generator(device=dev).manual_seed(7)
    kc, vc = (torch.randn(R * width + 20, page, Hkv, D, device=dev, generator=gen).to(BF16) for _ in range(2))
    x = torch.randn(T, Hq + 2 * Hkv, D, device=dev, generator=gen).to(BF16)
    mask = torch.ones(T, 5, dtype=torch.bool, device=dev)
    codes, s, z = _weight(g, Hq * D, 200, 128, True, BF16)
    W = q.q4_group_repack(codes.to(dev), s.to(dev), z.to(dev), K=Hq * D, group=128)
    plan = q.KvPlan(torch.empty(R + 1, dtype=torch.int32, device=dev), torch.empty(T, dtype=torch.int64, device=dev),
                    torch.empty(T, dtype=torch.int32, device=dev), torch.empty(4, dtype=torch.int32, device=dev))
    o = torch.zeros(T, Hq, D, dtype=BF16, device=dev)
    y = torch.zeros(T, 200, dtype=BF16, device=dev)

    def call(stream=None):
        q.kv_plan(ctx, new, table, free, page, T, out=plan, stream=stream)
        q.kv_append(x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], plan.slots, kc, vc, stream=stream)
        q.tree_attention(x[:, :Hq], kc, vc, table, ctx, plan.cu_new, mask, out=o, stream=stream)
        q.q4_group_matmul(o.view(T, -1), W, out=y, stream=stream)
    return call, [table, plan.slots, kc, vc, o, y]


def test_step_in_a_graph_and_on_another_stream(q):
    dev = torch_dev()
    call, outs = _step(q, dev, np.random.default_rng(20))
    call()
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    side = torch.cuda.Stream()
    for t in outs[4:]:
        t.zero_()
    side.wait_stream(torch.cuda.current_stream())
    call(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        for t in outs[4:]:
            t.fill_(-1.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
        call()                                                      # eager work between the replays
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_calls_repeat_bit_for_bit(q):
    g = np.random.default_rng(21)
    b = Batch(g, [2000, 500], [6, 9], 8, 2, 128, 16, BF16, "tree")
    first = b.run(q)
    assert all(torch.equal(b.run(q), first) for _ in range(3))


def test_outputs_of_other_streams_are_their_own(q):
    """Allocated results of a call on a side stream, used there, equal the main stream's."""
    b = Batch(np.random.default_rng(22), [900], [4], 4, 2, 64, 16, BF16, "tree")
    want = b.run(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = b.run(q, stream=side)
    side.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("cache,bound", [("bf16", 2 ** -5), ("int8", 2 ** -4)])
def test_example(cache, bound):
    """The example's layer against its plain fp32 form.  Along the layer q, k, v and a are rounded to bf16 (2^-9 each)
    and the sum once; an int8 row adds half a step of 127 (2^-8) to K and V.  Scores of size up to about 5 turn 2^-8 of
    theirs into 2 % of a weight, of which the output keeps the part that does not cancel; with the rounding of outputs
    up to the largest (2^-9) the bf16 layer stays within 2^-5 of it, twice that over an int8 cache."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "verify_step.py")
    spec = importlib.util.spec_from_file_location("verify_step", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    assert m.run(requests=3, prompt=130, drafts=6, steps=3, cache=cache) <= bound


# The plain sum of (q - z) s x, K products and additions in fp32 in the order of k, that takes the place of an output whose
# group sums leave fp32: each step is off by at most U of the sum of sizes so far.
def _check_product_extremes(Y, X, codes, s, z, K, group):
    z = None if z is None else z.numpy()
    with np.errstate(invalid="ignore"):
        x, scales = f64(X), s.double().numpy()
        want, size = ref.q4_group_matmul(x, codes.numpy(), scales, z, K, group)
        plain = ref.q4_group_matmul(np.where(np.isfinite(x), np.abs(x), 0.0), codes.numpy(), np.abs(scales), np.zeros(scales.shape), K, group)[1]
    got, top = f64(Y), float(torch.finfo(Y.dtype).max)
    with np.errstate(over="ignore"):
        rounded = np.where(np.abs(want) > top * (1 + 2.0 ** -12), np.sign(want) * np.inf, want)
    tol = torch.finfo(Y.dtype).eps / 2 * np.abs(want) + (48 + K / 128 + K) * U * np.where(np.isfinite(size), size, plain)
    finite = np.isfinite(rounded)
    assert np.array_equal(np.isnan(got), np.isnan(rounded))
    assert np.array_equal(got[~finite & ~np.isnan(rounded)], rounded[~finite & ~np.isnan(rounded)])
    assert (np.abs(got[finite] - want[finite]) <= tol[finite]).all(), float(np.max(np.abs(got[finite] - want[finite]) / tol[finite]))
    return rounded


@pytest.mark.parametrize("xt", [F32, F16, BF16], ids=["f32", "f16", "bf16"])
@pytest.mark.parametrize("M,K,N,group,variant", [(1, 1000, 40, 128, "q4g_mm16"), (9, 8200, 24, 32, "q4g_mm16"),
                                                 (5, 264, 33, 64, "q4g_mm16"), (20, 300, 50, 64, "q4g_mm"),
                                                 (70, 2056, 40, 128, "q4g_mm_split"), (33, 1536, 20, 256, "q4g_mm_split")])
def test_group_product_of_infinite_and_large_activations(q, M, K, N, group, variant, xt):
    """An infinite activation makes an output infinite where its code is not the zero, and NaN where it is; activations
    whose sums of (16 + q) x pass fp32 give the scaled sum all the same.  In every launch form."""
    g = np.random.default_rng(M + K)
    for zeros, st in ((True, F16), (False, BF16)):
        codes, s, z = _weight(g, K, N, group, zeros, st)
        W = q.q4_group_repack(to_dev(codes.numpy()), s.to(torch_dev()), None if z is None else to_dev(z.numpy()), K=K, group=group)
        x = torch.from_numpy(g.standard_normal((M, K))).to(xt)
        x[0, K // 3] = float("inf")
        if M > 3:
            x[1, K - 1], x[1, 2] = -float("inf"), float("-inf")
            x[2, 0], x[2, K // 2] = float("inf"), float("nan")
        Y = q.q4_group_matmul(x.to(torch_dev()), W)
        assert q.last_variant() == (variant if xt != F32 or variant != "q4g_mm16" else q.last_variant())
        rounded = _check_product_extremes(Y, x, codes, s, z, K, group)
        assert np.isinf(rounded[0]).any() and (M <= 3 or np.isfinite(rounded[3:]).all())
        if xt == F16:
            continue                                            # 65504 * 31 * K stays far inside fp32
        x = torch.from_numpy(g.standard_normal((M, K))).to(xt)
        big = torch.finfo(xt).max
        x[0, ::7] *= 2.0 ** 122
        if M > 3:
            x[1] = 1e37
            x[2, 5], x[2, 6], x[2, K // 2] = big, -big, big
            x[3, 1::2] = 2.0 ** 124
        Y = q.q4_group_matmul(x.to(torch_dev()), W)
        rounded = _check_product_extremes(Y, x, codes, s, z, K, group)
        assert np.isfinite(rounded[0]).all() and (M <= 3 or np.isfinite(rounded[2]).all())


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M", [1, 5, 40])
def test_group_product_fp32_keeps_its_bits(q, M, group):
    """fp32 rows lose nothing to the codes' offset.  If every product of the three terms were added with a rounding of its
    own to the partial sum, which grows as sqrt(k), the 3 K roundings of U / sqrt(3) would leave a relative 2-norm error
    of U sqrt(K / 2); offsets of 16 and more on every code leave more (8e-7 to 1.6e-6 at K = 128)."""
    g = np.random.default_rng(M + group)
    K, N = 128, 800
    for zeros in (True, False):
        codes, s, z = _weight(g, K, N, group, zeros, F16)
        W = q.q4_group_repack(to_dev(codes.numpy()), s.to(torch_dev()), None if z is None else to_dev(z.numpy()), K=K, group=group)
        X = torch.from_numpy(g.standard_normal((M, K))).to(F32).to(torch_dev())
        want = ref.q4_group_matmul(f64(X), codes.numpy(), s.double().numpy(), None if z is None else z.numpy(), K, group)[0]
        got = f64(q.q4_group_matmul(X, W))
        assert np.linalg.norm(got - want) <= U * (K / 2) ** 0.5 * np.linalg.norm(want)


def test_group_repack_of_one_column(q):
    """A weight of one column, as a transposed vector gives it: the row stride of a single row is no size."""
    g = np.random.default_rng(40)
    K, group = 200, 64
    codes, s, z = _weight(g, K, 1, group, True, F16)
    dev = [t.to(torch_dev()).flatten().view(-1, 1).t() for t in (codes, s, z)]
    assert [t.stride(0) for t in dev] == [1, 1, 1]
    X = torch.from_numpy(g.standard_normal((3, K))).to(F32).to(torch_dev())
    _check_product(q.q4_group_matmul(X, q.q4_group_repack(*dev, K=K, group=group)), X, codes, s, z, K, group)


@pytest.mark.parametrize("xt", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("M,K", [(1, 9), (1, 15), (1, 515), (1, 1001), (1, 14851), (1, 16007), (2, 1001), (2, 7445), (3, 9),
                                 (7, 139), (16, 1006), (16, 129)])
def test_group_product_octet_that_k_ends_in(q, M, K, xt):
    """The form of few rows where K is no multiple of eight: rows in LDS (up to 29 KiB of whole records) and read in the
    loop, with NaN right behind each row."""
    g = np.random.default_rng(M * K)
    N, group = 50, 64
    codes, s, z = _weight(g, K, N, group, True, F16)
    W = q.q4_group_repack(to_dev(codes.numpy()), s.to(torch_dev()), to_dev(z.numpy()), K=K, group=group)
    room = torch.full((M, (K + 15) // 8 * 8), float("nan"), dtype=xt, device=torch_dev())
    X = room[:, :K]
    X.copy_(torch.from_numpy(g.standard_normal((M, K))).to(xt))
    Y = q.q4_group_matmul(X, W)
    assert q.last_variant() == "q4g_mm16"
    _check_product(Y, X, codes, s, z, K, group)


@pytest.mark.parametrize("xt", [F32, F16, BF16], ids=["f32", "f16", "bf16"])
def test_which_form_of_the_product_runs(q, xt):
    """The rules that choose a form, at sizes on both sides of each."""
    g = np.random.default_rng(41)
    forms = set()
    for M, K, N, off, want in ((1, 256, 40, 0, "q4g_mm16"), (16, 256, 40, 0, "q4g_mm16"), (17, 256, 40, 0, "q4g_mm"),
                               (16, 256, 40, 1, "q4g_mm"), (1, 7, 40, 0, "q4g_mm"), (64, 1024, 40, 0, "q4g_mm_split"),
                               (64, 896, 40, 0, "q4g_mm"), (16, 1024, 40, 1, "q4g_mm_split")):
        codes, s, z = _weight(g, K, N, 128, True, F16)
        W = q.q4_group_repack(to_dev(codes.numpy()), s.to(torch_dev()), to_dev(z.numpy()), K=K, group=128)
        room = torch.from_numpy(g.standard_normal((M, K + 8))).to(xt).to(torch_dev())
        X = room[:, off:off + K]
        Y = q.q4_group_matmul(X, W)
        _check_product(Y, X, codes, s, z, K, 128)
        if xt == F32 and want == "q4g_mm16":                     # fp32 rows are always laid out
            want = "q4g_mm"
        assert q.last_variant() == want, (M, K, off)
        forms.add(want)
    assert len(forms) == (2 if xt == F32 else 3)


@TYPES
@pytest.mark.parametrize("D", [40, 72, 88, 96, 136, 192, 248])
def test_attention_head_dimensions(q, ct, D):
    """Head dimensions that fill no kernel's own (64, 96, 128, 256), with one and with two tiles of rows a wavefront."""
    g = np.random.default_rng(D)
    for new, want in ((9, "tree_rows64"), (50, "tree_rows128" if D <= 128 else "tree_rows64")):
        b = Batch(g, [210, 33], [new, 5], 6, 2, D, 16, ct, "tree")
        out = b.run(q)
        assert q.last_variant() == want
        b.check(out)


@TYPES
def test_attention_of_a_chain_is_the_causal_one(q, ct):
    """Without a mask a token sees those up to itself: the bits are those of the mask that says so."""
    g = np.random.default_rng(42)
    b = Batch(g, [70, 0, 900], [5, 70, 33], 4, 2, 64, 16, ct, None)
    causal = b.run(q)
    b.check(causal)
    b.mask = np.zeros((b.T, 70), bool)
    for r, n in enumerate(b.new):
        b.mask[b.cu[r]:b.cu[r + 1], :n] = ref.chain_mask(n)
    assert torch.equal(b.run(q), causal)


def test_attention_beside_its_queries(q):
    """Queries and output as slices of one tensor, which the call tells from an output over its queries."""
    b = Batch(np.random.default_rng(43), [50, 9], [6, 3], 4, 2, 64, 16, BF16, "tree")
    want = b.run(q)
    (k, v), (ks, vs) = [b.dev(x) for x in b.kv], [b.dev(x) for x in b.scales]
    room = torch.full((b.T, 11, 64), 5.0, dtype=BF16, device=torch_dev())
    room[:, 1:5] = b.q.to(torch_dev())
    args = (room[:, 1:5], k, v, to_dev(b.table), to_dev(np.array(b.ctx, np.int32)), to_dev(b.cu), to_dev(b.mask))
    q.tree_attention(*args, out=room[:, 6:10])
    assert torch.equal(room[:, 6:10], want) and torch.equal(room[:, 1:5], b.q.to(torch_dev()))
    assert (room[:, [0, 5, 10]] == 5.0).all()
    for out in (room[:, 1:5], room[:, 4:8]):
        with pytest.raises(q.QmmError) as e:
            q.tree_attention(*args, out=out)
        assert e.value.status == q.QMM_ERR_INVALID


class _Steps:
    """Plan, append, attention and projection over tensors that keep their places while lengths change.  T and the table
    have room to spare; `reset` puts everything that a call writes out of the way."""
    R, Hq, Hkv, D, page, width, T, N = 5, 4, 2, 64, 16, 45, 64, 200
    LENGTHS = [([0, 17, 64, 100, 31], [3, 4, 1, 0, 5]), ([0, 17, 64, 100, 31], [0, 0, 0, 0, 0]),
               ([400, 0, 5, 600, 17], [20, 9, 1, 30, 4]), ([0, 0, 300, 0, 0], [0, 0, 7, 0, 0]), ([650, 15, 16, 0, 1], [1, 1, 1, 1, 1])]

    def __init__(self, q, dev, ct):
        self.q, g = q, np.random.default_rng(50)
        R, Hq, Hkv, D, page, width, T = self.R, self.Hq, self.Hkv, self.D, self.page, self.width, self.T
        gen = torch.Generator(device=dev).manual_seed(51)
        ids = torch.from_numpy(g.permutation(R * width + 40).astype(np.int32)).to(dev)
        self.table0, self.free = ids[:R * width].view(R, width).clone(), ids[R * width:].clone()
        shape = (R * width + 40, page, Hkv, D)
        if ct == torch.int8:
            self.cache0 = [torch.randint(-127, 128, shape, generator=gen, device=dev, dtype=torch.int8) for _ in range(2)]
            self.cache0 += [torch.rand(shape[:3], generator=gen, device=dev) * 0.02 for _ in range(2)]
        else:
            self.cache0 = [torch.randn(shape, generator=gen, device=dev).to(ct) for _ in range(2)]
        self.cache = [c.clone() for c in self.cache0]
        self.ctx, self.new = (torch.zeros(R, dtype=torch.int32, device=dev) for _ in range(2))
        self.table = self.table0.clone()
        self.x = torch.randn(T, Hq + 2 * Hkv, D, device=dev, generator=gen).to(BF16 if ct == torch.int8 else ct)
        self.mask = torch.rand(T, 30, device=dev, generator=gen) < 0.6
        self.weight = _weight(g, Hq * D, self.N, 128, True, BF16)
        codes, s, z = (t.to(dev) for t in self.weight)
        self.W = q.q4_group_repack(codes, s, z, K=Hq * D, group=128)
        i32, i64 = (lambda n, t=t: torch.empty(n, dtype=t, device=dev) for t in (torch.int32, torch.int64))
        self.plan = q.KvPlan(i32(R + 1), i64(T), i32(T), i32(4))
        self.o, self.y = (torch.empty(T, n, dtype=self.x.dtype, device=dev) for n in (Hq * D, self.N))
        self.outs = [self.table, self.plan.cu_new, self.plan.slots, self.plan.positions, self.plan.info, *self.cache, self.o, self.y]

    def reset(self, lengths):
        for t, v in zip((self.ctx, self.new), lengths):
            t.copy_(torch.tensor(v, dtype=torch.int32))
        self.table.copy_(self.table0)
        for c, c0 in zip(self.cache, self.cache0):
            c.copy_(c0)
        for t in (self.plan.cu_new, self.plan.slots, self.plan.positions, self.plan.info, self.o, self.y):
            t.fill_(-7)

    def __call__(self, stream=None):
        q, Hq, Hkv = self.q, self.Hq, self.Hkv
        kc, vc, *scales = self.cache
        ks, vs = scales or (None, None)
        q.kv_plan(self.ctx, self.new, self.table, self.free, self.page, self.T, out=self.plan, stream=stream)
        q.kv_append(self.x[:, Hq:Hq + Hkv], self.x[:, Hq + Hkv:], self.plan.slots, kc, vc, ks, vs, stream=stream)
        q.tree_attention(self.x[:, :Hq], kc, vc, self.table, self.ctx, self.plan.cu_new, self.mask, k_scale=ks, v_scale=vs,
                         out=self.o.view(self.T, Hq, self.D), stream=stream)
        q.q4_group_matmul(self.o, self.W, out=self.y, stream=stream)

    def check(self, lengths):
        """Everything that a call wrote, from the definitions."""
        ctx, new = (np.array(v, np.int32) for v in lengths)
        want = ref.kv_plan(ctx, new, to_np(self.table0), to_np(self.free), self.page, self.T)
        for got, w in zip((self.table, self.plan.cu_new, self.plan.slots, self.plan.positions, self.plan.info), want):
            assert np.array_equal(to_np(got), w)
        table, cu, slots, _, _ = want
        G, s8 = self.Hq // self.Hkv, len(self.cache) == 4
        x, used = f64(self.x), slots[slots >= 0]
        values = []
        for i in range(2):
            src = self.x[:len(used), self.Hq + i * self.Hkv:self.Hq + (i + 1) * self.Hkv].cpu()
            rows = self.cache0[i].cpu().view(-1, self.Hkv, self.D).clone()
            if s8:
                scale = self.cache0[2 + i].cpu().view(-1, self.Hkv).clone()
                codes, sc = ref.quantize_rows(src.float().numpy())
                rows[used], scale[used] = torch.from_numpy(codes), torch.from_numpy(sc)
                assert torch.equal(self.cache[2 + i].cpu().view(-1, self.Hkv), scale)
                values.append(rows.double().numpy() * scale.double().numpy()[..., None])
            else:
                rows[used] = src
                values.append(rows.double().numpy())
            assert torch.equal(self.cache[i].cpu().view(-1, self.Hkv, self.D), rows)
        o, mask = f64(self.o).reshape(self.T, self.Hq, self.D), to_np(self.mask)
        eps = torch.finfo(self.o.dtype).eps
        for r in range(self.R):
            pos = np.arange(ctx[r] + new[r])
            at = table[r, pos // self.page] * self.page + pos % self.page
            for t in range(cu[r], cu[r + 1]):
                sees = np.concatenate([np.ones(ctx[r], bool), mask[t, :new[r]]])
                for h in range(self.Hq):
                    w, size, dot = ref.tree_attention(x[t, h], values[0][at, h // G], values[1][at, h // G], sees, self.D ** -0.5)
                    tol = eps / 2 * np.abs(w) + (2.0 ** -16 + 2 * (self.D + 8) * U * dot + 64 * U) * size + 1e-30
                    assert (np.abs(o[t, h] - w) <= tol).all(), (r, t, h)
        assert (o[cu[-1]:] == -7).all()
        _check_product(self.y, self.o, *self.weight, self.Hq * self.D, 128)


@TYPES
def test_steps_of_any_lengths_on_another_stream(q, ct):
    """Each output of each call is put out of the way before the call, so what a side stream leaves out shows."""
    s = _Steps(q, torch_dev(), ct)
    side = torch.cuda.Stream()
    for lengths in s.LENGTHS:
        s.reset(lengths)
        s()
        s.check(lengths)
        want = [t.clone() for t in s.outs]
        s.reset(lengths)
        side.wait_stream(torch.cuda.current_stream())
        s(side)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(s.outs, want)), lengths


@TYPES
def test_one_graph_serves_any_lengths(q, ct):
    """One captured step, replayed over other lengths in the same tensors: none, longer ones that fill T, one request."""
    s = _Steps(q, torch_dev(), ct)
    s.reset(s.LENGTHS[0])
    s()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s()
    for lengths in s.LENGTHS + s.LENGTHS[2::-1]:
        s.reset(lengths)
        s()                                                         # eager work between the replays
        want = [t.clone() for t in s.outs]
        for _ in range(2):
            s.reset(lengths)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(s.outs, want)), lengths
        s.check(lengths)


@TYPES
def test_cache_of_more_than_2_31_elements(q, ct):
    """Pages on both sides of element 2^31 of a cache: the same bits as over a small one, and nothing beside them."""
    dev, page, H, D = torch_dev(), 16, 8, 128
    first = 2 ** 31 // (page * H * D)                               # the page that begins at element 2^31
    pages = first + 40
    small = _random_pages(ct, 40, page, H, D)
    big = [torch.zeros(pages, *t.shape[1:], dtype=t.dtype, device=dev) for t in small]
    ids = torch.arange(40, device=dev) + first - 20                 # page i of the small cache lies at first - 20 + i
    for b, t in zip(big, small):
        assert t.dim() == 3 or b.numel() > 2 ** 31
        b[ids] = t
    g = np.random.default_rng(52)
    xt = BF16 if ct == torch.int8 else ct
    order = torch.from_numpy(g.permutation(40).astype(np.int32)).to(dev)
    table = order[:36].view(2, 18)
    ctx, cu = (torch.tensor(v, dtype=torch.int32, device=dev) for v in ([270, 33], [0, 9, 14]))
    Q = torch.from_numpy(g.standard_normal((14, 16, D))).to(xt).to(dev)
    K, V = (torch.from_numpy(g.standard_normal((14, H, D))).to(xt).to(dev) for _ in range(2))
    slots = torch.cat([table[r, p // page].long() * page + p % page for r, p in
                       ((0, torch.arange(270, 279, device=dev)), (1, torch.arange(33, 38, device=dev)))])
    outs = []
    for cache, shift in ((small, 0), (big, first - 20)):
        kc, vc, *scales = cache
        ks, vs = scales or (None, None)
        q.kv_append(K, V, slots + shift * page, kc, vc, ks, vs)
        outs.append(q.tree_attention(Q, kc, vc, table + shift, ctx, cu, k_scale=ks, v_scale=vs))
    assert torch.equal(*outs) and torch.isfinite(outs[0]).all() and outs[0].any()
    for b, t in zip(big, small):
        assert torch.equal(b[ids], t)
        b[ids] = 0
        assert not any(bool(c.any()) for c in b.split(1 << 14))
        del b


def _random_pages(ct, pages, page, H, D):
    """K and V (and scales) of a cache."""
    gen = torch.Generator(device=torch_dev()).manual_seed(53)
    if ct == torch.int8:
        kv = [torch.randint(-127, 128, (pages, page, H, D), generator=gen, device=torch_dev(), dtype=torch.int8) for _ in range(2)]
        return kv + [torch.rand(pages, page, H, generator=gen, device=torch_dev()) * 0.02 for _ in range(2)]
    return [torch.randn(pages, page, H, D, generator=gen, device=torch_dev()).to(ct) for _ in range(2)]


def _example():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "verify_step.py")
    spec = importlib.util.spec_from_file_location("verify_step", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _branch(m, accepted, e, seen):
    """The attention branch of the example's layer for one request's new rows, in 64 bits on the CPU."""
    plain = {k: v.double().cpu().numpy() for k, v in e["plain"].items()}
    new = e["new"].double().cpu().numpy()
    x = np.concatenate([accepted, new])
    G = m.Q_HEADS // m.KV_HEADS
    q, k, v = new @ plain["q"], x @ plain["k"], x @ plain["v"]
    out = np.zeros_like(q)
    for h in range(m.Q_HEADS):
        cols, kv = slice(h * m.DIM, (h + 1) * m.DIM), slice(h // G * m.DIM, (h // G + 1) * m.DIM)
        s = np.where(seen, q[:, cols] @ k[:, kv].T * m.DIM ** -0.5, -np.inf)
        w = np.exp(s - s.max(1, keepdims=True))
        out[:, cols] = w @ v[:, kv] / w.sum(1, keepdims=True)
    return out @ plain["o"]


@pytest.mark.parametrize("cache,bound", [("bf16", 2 ** -6), ("int8", 2 ** -5)])
def test_example_attention_branch(cache, bound):
    """The example's y - x against the branch's own size, over short prompts, where drafted and moved rows weigh.

    Unit-size q, k, v and scores, and some 15 keys: the branch has a size of about 0.4, y one of about 1.1.  A bf16
    rounding's rms is 2^-9 x 0.42 = 0.0008 of the value: of y 0.0023 of the branch; of q and k together 0.0012 of a
    score and so of a; of v and of a 0.0008 each: 0.003 together.  An int8 row's step of amax / 127 = 0.021 adds an rms of
    0.006 to k (a score) and to v each: 0.009 together.  The bounds are four to five times that.  Plain layers that leave
    something out have to miss them by as much again: a causal mask for the tree's, no drafted tokens but the row's own,
    accepted rows that were not moved to their places."""
    m, record = _example(), []
    m.run(requests=5, prompt=9, drafts=7, steps=3, cache=cache, record=record)
    assert len(record) == 20
    unmoved = {r: np.zeros((0, m.HIDDEN)) for r in range(5)}
    off = {k: np.zeros(4) for k in ("right", "causal", "alone", "unmoved")}
    size = np.zeros(4)
    for e in record:
        n, step, r = e["new"].shape[0], e["step"], e["request"]
        got = e["y"].double().cpu().numpy() - e["new"].double().cpu().numpy()
        accepted, seen = e["accepted"].double().cpu().numpy(), e["seen"].cpu().numpy()
        c = len(accepted)
        causal, alone = seen.copy(), seen.copy()
        causal[:, c:], alone[:, c:] = np.tril(np.ones((n, n), bool)), np.eye(n, dtype=bool)
        want = _branch(m, accepted, e, seen)
        size[step] += (want ** 2).sum()
        for name, w in (("right", want), ("causal", _branch(m, accepted, e, causal)), ("alone", _branch(m, accepted, e, alone)),
                        ("unmoved", _branch(m, unmoved[r], e, seen))):
            off[name][step] += ((got - w) ** 2).sum()
        # without the move a request's next rows stay the first ones of its tree
        keep = list(range(n)) if step == 0 else list(range(len(e["path"])))
        unmoved[r] = np.concatenate([unmoved[r], e["new"].double().cpu().numpy()[keep]])
    error = {k: np.sqrt(v / size) for k, v in off.items()}
    assert (error["right"] <= bound).all(), error
    assert (error["causal"][1:] >= 2 * bound).all() and (error["alone"][1:] >= 2 * bound).all(), error
    assert (error["unmoved"][2:] >= 2 * bound).all(), error
