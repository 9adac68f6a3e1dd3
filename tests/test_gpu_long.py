"""GPU parity of the long-context serving operators against their plain 64-bit
forms (tests/long_ref.py).

Bounds.  A rounding to a type is off by at most eps/2 of the value; U = 2^-24.
  * 4-bit rows: codes, steps and minima equal; their values one fp32 rounding of
    code * step + minimum (two roundings where the test computes it in fp64 and
    rounds: equal, since both are the nearest fp32).
  * attention: one rounding of the output; weights held to 2^-16; a score's sum of D
    products in fp32 moves a weight by twice its error.  A 4-bit row's products are of
    16 + code, so its score adds up terms of at most 31 step |x| and (|m| + 16 step)
    |x|, and its output terms of at most 31 step + |m| + 16 step.  With few rows a request
    weight x step is one fp16 number, off by 2^-12 of it, which moves step (code - 8) of
    the value, at most 8 step; below 2^-14 of the largest step's weight it is off by 2^-25
    instead, in units of at most 2^-5 of that step: by 2^-30, times 8, a key.
  * adapters: one rounding of the output; the inner sum of K products and the outer
    one of rank in fp32, each at most (n + 8) U of the sum of its terms' sizes (n
    additions in any order); the inner sum enters the outer one as 16 bits (2^-16)
    for 16-bit rows, 24 for fp32 ones.  Over many outputs the roundings are
    independent: the relative 2-norm error of fp32 outputs stays below 8 sqrt(K / 32 +
    rank / 32 + 8) U of the terms' size.
  * log probabilities: a lane adds up to 64 weights and a tree 20 sums more, each off
    by 2 U and, by its exponent's rounding, by |y| U: below 128 U on the logarithm (the
    mean |y| of the weights is at most log2 V); the difference and its logarithm
    are rounded at most four times.  Entropy: the same error on sum e |y| / S <=
    log2 V + 1.
"""
import numpy as np
import pytest
import torch

import long_ref as ref
import serve_ref
from gpu_util import to_dev, torch_dev

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


X3 = pytest.mark.parametrize("xt", [F32, F16, BF16], ids=["f32", "f16", "bf16"])


# ------------------------------------------------------------- cache rows ---

def _q4_cache(pages, page, H, D, fill=0):
    dev = torch_dev()
    codes = [torch.full((pages, page, H, D // 2), fill, dtype=torch.uint8, device=dev) for _ in range(2)]
    return codes, [torch.full((pages, page, H, 2), float(fill), dtype=BF16, device=dev) for _ in range(2)]


@X3
@pytest.mark.parametrize("T,H,D,page", [(1, 1, 16, 1), (5, 3, 64, 4), (33, 2, 80, 7), (64, 8, 128, 16), (9, 1, 256, 32), (300, 2, 96, 64)])
def test_append_q4(q, T, H, D, page, xt):
    """Codes, steps and minima by the definition; other rows stay; slots outside the cache are skipped."""
    g = np.random.default_rng(T + D)
    pages = -(-T // page) + 2
    codes, scales = _q4_cache(pages, page, H, D, 0x5a)
    slots = g.permutation(pages * page)[:T].astype(np.int64)
    if T > 4:
        slots[1], slots[3] = -1, pages * page
    rows = [torch.from_numpy(g.standard_normal((T, H, D)) * 3 + off).to(xt) for off in (0, 5)]
    q.kv_append(*[r.to(torch_dev()) for r in rows], to_dev(slots), *codes, *scales)
    for r, c, s in zip(rows, codes, scales):
        want = np.full((pages * page, H, D // 2), 0x5a, np.uint8)
        pair = np.full((pages * page, H, 2), float(0x5a), np.float32)
        ok = (slots >= 0) & (slots < pages * page)
        k, step, m = ref.quantize_q4(r.float().numpy())
        want[slots[ok]], pair[slots[ok]] = ref.pack_q4(k)[ok], np.stack([step, m], -1)[ok]
        assert np.array_equal(f64(c).reshape(want.shape), want)
        assert np.array_equal(f64(s).reshape(pair.shape), pair)


def test_append_q4_extremes(q):
    """Constant rows, zeros of both signs, one value apart, subnormals, the ends of fp32, NaN and infinities."""
    D, T = 32, 14
    x = np.random.default_rng(1).standard_normal((T, 1, D)).astype(np.float32)
    x[0], x[1], x[2] = 0, -0.0, -7.125
    x[3] = 0
    x[3, 0, 5] = 1e-3
    x[4] *= np.float32(1e-41)
    x[5] *= np.float32(1e37)
    x[6, 0, 0], x[6, 0, 1] = 3e38, -3e38            # the range leaves fp32
    x[7, 0, 3] = np.inf
    x[8, 0, 31] = np.nan
    x[9, 0, 8] = -np.inf
    x[10] = 3.4028e38                               # rounds to infinity in bf16
    x[11] = 1 + np.arange(D) * np.float32(2.0 ** -12)   # the minimum's rounding is larger than the step
    x[12] = np.arange(D)
    x[13] = -0.0
    x[13, 0, 4] = 0.0
    codes, scales = _q4_cache(1, T, 1, D)
    q.kv_append(to_dev(x), to_dev(-x), to_dev(np.arange(T)), *codes, *scales)
    for r, c, s in zip((x, -x), codes, scales):
        k, step, m = ref.quantize_q4(r)
        assert np.array_equal(f64(c)[0], ref.pack_q4(k))
        assert np.array_equal(f64(s)[0], np.stack([step, m], -1), equal_nan=True)
    v = f64(q.kv_gather(to_dev(np.arange(T)), *codes, *scales)[0])[:, 0]
    assert np.isnan(v[6:11]).all() and np.isfinite(np.delete(v, range(6, 11), 0)).all() and not np.signbit(v[1]).any()


@X3
def test_append_q4_strides(q, xt):
    """Rows inside wider tensors, unaligned ones among them, caches whose heads come first or lie in a wider tensor."""
    g = np.random.default_rng(3)
    T, H, D, page, pages = 21, 3, 48, 8, 4
    for off in (0, 1, 8):
        wide = torch.full((T, H + 1, D + 24), float("nan"), dtype=xt, device=torch_dev())
        rows = wide[:, 1:, off:off + D]
        rows.copy_(torch.from_numpy(g.standard_normal((T, H, D))))
        slots = to_dev(g.permutation(pages * page)[:T].astype(np.int64))
        codes, scales = _q4_cache(pages, page, H, D)
        q.kv_append(rows, rows, slots, *codes, *scales)
        wide_c = torch.zeros(pages, H + 1, page, D // 2 + 8, dtype=torch.uint8, device=torch_dev())
        wide_s = torch.zeros(pages, H + 1, page, 4, dtype=BF16, device=torch_dev())
        c2, s2 = wide_c[:, 1:, :, 8:].transpose(1, 2), wide_s[:, 1:, :, 2:].transpose(1, 2)
        v2, t2 = torch.zeros_like(wide_c)[:, 1:, :, 8:].transpose(1, 2), torch.zeros_like(wide_s)[:, 1:, :, 2:].transpose(1, 2)
        q.kv_append(rows, rows, slots, c2, v2, s2, t2)
        assert torch.equal(c2, codes[0]) and torch.equal(s2, scales[0]) and torch.equal(v2, codes[1]) and torch.equal(t2, scales[1])
        assert not wide_c[:, 0].any() and not wide_c[..., :8].any() and not wide_s[..., :2].any()
        for dtype in (F32, F16, BF16):
            room = torch.full((T, H + 1, D + 24), 7.0, dtype=dtype, device=torch_dev())
            out = (room[:, 1:, off:off + D], torch.empty(T, H, D, dtype=dtype, device=torch_dev()))
            assert q.kv_gather(slots, c2, v2, s2, t2, dtype=dtype, out=out)[0] is not None
            k, step, m = ref.quantize_q4(rows.float().cpu().numpy())
            want = torch.from_numpy(k * step[..., None].astype(np.float64) + m[..., None]).float().to(dtype)
            assert torch.equal(out[0].cpu(), want) and torch.equal(out[1].cpu(), want)
            out[0].fill_(7.0)
            assert (room == 7.0).all()


@pytest.mark.parametrize("ct", [F16, BF16, torch.int8, torch.uint8], ids=["f16", "bf16", "s8", "q4"])
@pytest.mark.parametrize("D,H,page", [(16, 1, 1), (80, 3, 7), (128, 8, 16), (256, 2, 64)])
def test_gather(q, ct, D, H, page):
    """Rows of every kind of cache, twice the same ones and slots outside it, in every type."""
    g = np.random.default_rng(D)
    pages, T = 5, 37
    slots = g.integers(-3, pages * page + 3, T)
    slots[-1] = slots[0]
    slots[5], slots[6] = 1 << 40, -(1 << 40)
    x = [g.standard_normal((pages, page, H, D)).astype(np.float32) for _ in range(2)]
    scales = [None, None]
    if ct == torch.uint8:
        parts = [ref.quantize_q4(y) for y in x]
        cache = [to_dev(ref.pack_q4(k)) for k, _, _ in parts]
        scales = [to_dev(np.stack([s, m], -1)).to(BF16) for _, s, m in parts]
        values = [k * s[..., None].astype(np.float64) + m[..., None] for k, s, m in parts]
    elif ct == torch.int8:
        parts = [serve_ref.quantize_rows(y) for y in x]
        cache, scales = [to_dev(k) for k, _ in parts], [to_dev(s) for _, s in parts]
        values = [k * s[..., None].astype(np.float64) for k, s in parts]
    else:
        cache = [to_dev(y).to(ct) for y in x]
        values = [f64(c) for c in cache]
    ok = (slots >= 0) & (slots < pages * page)
    for dtype in (F32, F16, BF16):
        got = q.kv_gather(to_dev(slots), *cache, *scales, dtype=dtype)
        for y, v in zip(got, values):
            rows = v.reshape(-1, H, D)[np.where(ok, slots, 0)]
            rows[~ok] = 0
            assert torch.equal(y.cpu(), torch.from_numpy(rows).float().to(dtype))
    assert [t.shape for t in q.kv_gather(to_dev(slots[:0]), *cache, *scales)] == [(0, H, D)] * 2


# --------------------------------------------------------------- attention ---

KINDS = pytest.mark.parametrize("kind", ["f16", "bf16", "s8", "q4"])


class Batch:
    """Requests with their tables and filled caches of one kind, and the values that the caches stand for."""

    def __init__(self, g, kind, ctx, new, Hq, Hkv, D, page, order="nhd", std=2.0, spare_rows=0):
        self.kind, self.ctx, self.new, self.Hq, self.Hkv, self.D, self.page = kind, ctx, new, Hq, Hkv, D, page
        R = len(ctx)
        need = [-(-(c + n) // page) for c, n in zip(ctx, new)]
        self.width = max(max(need), 1)
        self.pages = sum(need) + 3
        ids = g.permutation(self.pages).astype(np.int32)
        self.table = np.full((R, self.width), -1, np.int32)
        at = 0
        for r in range(R):
            self.table[r, :need[r]] = ids[at:at + need[r]]
            at += need[r]
        self.order, self.xt = order, F16 if kind == "f16" else BF16
        self.kv, self.scales, self.size, self.values = [], [None, None], [], []
        for i in range(2):
            x = g.standard_normal((self.pages, page, Hkv, D)).astype(np.float32)
            if kind == "q4":
                k, s, m = ref.quantize_q4(x)
                self.kv.append(torch.from_numpy(ref.pack_q4(k)))
                self.scales[i] = torch.from_numpy(np.stack([s, m], -1)).to(BF16)
                self.values.append(k * s[..., None].astype(np.float64) + m[..., None])
                self.size.append(np.broadcast_to((47 * s + np.abs(m))[..., None].astype(np.float64), x.shape))
                self.step = np.broadcast_to(s[..., None].astype(np.float64), x.shape)  # of V, the last
            elif kind == "s8":
                k, s = serve_ref.quantize_rows(x)
                self.kv.append(torch.from_numpy(k))
                self.scales[i] = torch.from_numpy(s)
                self.values.append(k * s[..., None].astype(np.float64))
                self.size.append(np.abs(self.values[i]))
            else:
                self.kv.append(torch.from_numpy(x).to(self.xt))
                self.values.append(self.kv[i].double().numpy())
                self.size.append(np.abs(self.values[i]))
        self.T = sum(new) + spare_rows
        self.q = torch.from_numpy(g.standard_normal((self.T, Hq, D)) * std).to(self.xt)
        self.cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)

    def dev(self, x):
        if x is None:
            return None
        if self.order == "hnd":
            return x.transpose(1, 2).contiguous().to(torch_dev()).transpose(1, 2)
        if self.order == "wide":  # heads of a wider tensor, padded rows
            pad = {0: 8, 1: 2}[int(x.dim() == 4 and x.shape[3] == 2 and self.kind == "q4")]
            wide = torch.zeros(x.shape[0], x.shape[1] + 1, x.shape[2] + 2, *[d + pad for d in x.shape[3:]], dtype=x.dtype, device=torch_dev())
            view = wide[:, :x.shape[1], 1:-1]
            view = view[..., pad:] if x.dim() == 4 else view
            view.copy_(x.to(torch_dev()))
            return view
        return x.to(torch_dev())

    def args(self):
        (k, v), (ks, vs) = [self.dev(x) for x in self.kv], [self.dev(x) for x in self.scales]
        return [self.q.to(torch_dev()), k, v, to_dev(self.table), to_dev(np.array(self.ctx, np.int32)), to_dev(self.cu)], dict(k_scale=ks, v_scale=vs)

    def window(self, q, window, sinks, scale=None, **kw):
        args, scales = self.args()
        return q.window_attention(*args, window, sinks, scale, **scales, **kw)

    def check(self, out, sees_of, scale=None):
        """sees_of(r): [n, length] bool, what request r's new tokens see where there is a page."""
        scale = self.D ** -0.5 if scale is None else scale
        got = f64(out)
        for r, (c, n) in enumerate(zip(self.ctx, self.new)):
            if n == 0:
                continue
            pos = np.arange(min(c + n, self.width * self.page))
            page = self.table[r, pos // self.page]
            ok = (page >= 0) & (page < self.pages)
            k, v, ks, vs = [x[np.where(ok, page, 0), pos % self.page] for x in self.values + self.size]
            sees = sees_of(r)[:, :len(pos)] & ok
            x = f64(self.q[self.cu[r]:self.cu[r + 1]])
            o, _ = ref.attention(x, k, v, sees, scale)
            _, size = ref.attention(x, k, vs, sees, scale)
            G = self.Hq // self.Hkv
            # the largest sum of a visible key's terms
            dot = np.zeros((n, self.Hq))
            for h in range(self.Hq):
                with np.errstate(invalid="ignore"):
                    dot[:, h] = np.where(sees, np.abs(x[:, h]) @ ks[:, h // G].T, 0).max(-1) if len(pos) else 0
            delta = (self.D + 8) * U * dot * abs(scale)
            eps = torch.finfo(self.xt).eps / 2
            tol = eps * np.abs(o) + (2.0 ** -16 + 2 * delta + 64 * U)[..., None] * size
            tol = tol + torch.finfo(self.xt).smallest_normal * torch.finfo(self.xt).eps
            if self.kind == "q4":
                step = self.step[np.where(ok, page, 0), pos % self.page]
                tol = tol + 2.0 ** -12 * 8 * ref.attention(x, k, step, sees, scale)[0]
                tol = tol + len(pos) * 2.0 ** -27 * (float(np.nanmax(step)) if len(pos) else 0.0)
            err = np.abs(got[self.cu[r]:self.cu[r + 1]] - o)
            same = (err <= tol) | (np.isnan(o) & np.isnan(got[self.cu[r]:self.cu[r + 1]]))
            assert same.all(), (r, np.argwhere(~same)[:4].tolist(), float(np.nanmax(err / tol)))

    def behind(self, window, sinks):
        return lambda r: ref.window_sees(self.ctx[r], self.new[r], self.ctx[r] + self.new[r], window, sinks)


CASES = [
    ([0], [1], 1, 1, 64, 16, 1, 0),                         # one token that sees itself
    ([300], [1], 16, 8, 128, 16, 100, 4),                   # one decoded token
    ([64, 0, 63, 65, 128], [1, 3, 0, 1, 2], 4, 2, 128, 16, 64, 1),
    ([500, 130, 33], [7, 16, 1], 4, 4, 64, 7, 50, 5),       # pages that end inside every tile
    ([300, 17], [20, 33], 8, 2, 128, 24, 30, 70),           # first keys past one block, longer than a request
    ([90], [70], 6, 2, 80, 1, 3, 2),
    ([310, 200], [9, 5], 8, 1, 256, 32, 33, 40),
    ([0, 10], [300, 129], 4, 2, 64, 64, 65, 3),             # pieces of prompts
    ([0], [150], 9, 3, 96, 16, 1000, 4),                    # a window past the first key
    ([777], [5], 130, 1, 16, 16, 200, 0),                   # more heads of a group than a tile's rows
    ([1, 700, 64], [1, 1, 1], 5, 5, 112, 16, 2147483647, 9),
    ([1000], [3], 2, 1, 64, 16, 10, 2000),                  # every key is a first one
]


@KINDS
@pytest.mark.parametrize("ctx,new,Hq,Hkv,D,page,window,sinks", CASES)
def test_window(q, kind, ctx, new, Hq, Hkv, D, page, window, sinks):
    b = Batch(np.random.default_rng(len(ctx) + D), kind, ctx, new, Hq, Hkv, D, page)
    b.check(b.window(q, window, sinks), b.behind(window, sinks))


@KINDS
def test_window_longer_than_int32(q, kind):
    """The largest window and more are plain causal attention."""
    b = Batch(np.random.default_rng(5), kind, [70], [9], 2, 1, 64, 16)
    out = b.window(q, 2 ** 31 - 1, 0)
    b.check(out, b.behind(1 << 40, 0))
    assert torch.equal(b.window(q, 1 << 40, 1 << 40), out)


@KINDS
def test_window_many_requests(q, kind):
    """More requests than threads of a workgroup: ragged, new ones and ones that sit out among them."""
    g = np.random.default_rng(30)
    ctx, new = g.integers(0, 200, 600).tolist(), g.integers(0, 3, 600).tolist()
    ctx[300], new[300], new[599] = 3000, 90, 2
    b = Batch(g, kind, ctx, new, 2, 1, 64, 16)
    b.check(b.window(q, 77, 3), b.behind(77, 3))


@KINDS
@pytest.mark.parametrize("D,page", [(64, 16), (80, 24), (128, 32), (256, 16)])
def test_window_tiles_and_parts(q, kind, D, page):
    """Several row tiles to a cache head, and items that many workgroups share, in each head dimension."""
    g = np.random.default_rng(D)
    b = Batch(g, kind, [700, 90, 0], [40, 3, 210], 8, 1, D, page)
    b.check(b.window(q, 150, 70), b.behind(150, 70))
    b = Batch(g, kind, [9001], [2], 2, 2, D, page)
    for window, sinks in ((4000, 5), (1 << 20, 0), (20, 4097)):
        out = b.window(q, window, sinks)
        b.check(out, b.behind(window, sinks))
        ws = torch.full((q.lib.qmm_window_attention_workspace_bytes(2, 2, 1, 2, D),), 255, dtype=torch.uint8, device=torch_dev())
        assert torch.equal(b.window(q, window, sinks, ws=ws), out)


@KINDS
def test_window_pages_behind_it_are_free(q, kind):
    """Blocks that no token sees are not read: their entries may be anything.  Entries of blocks that are read may be
    missing or name no page: their tokens are not visible."""
    g = np.random.default_rng(7)
    b = Batch(g, kind, [1000, 2000], [2, 100], 4, 2, 64, 16)
    out = b.window(q, 100, 10)
    table = b.table.copy()
    for r in range(2):
        low = b.ctx[r] - 99
        b.table[r, 1:low // 16] = g.choice([-1, -(1 << 31), (1 << 31) - 1, b.pages], low // 16 - 1)
    assert torch.equal(b.window(q, 100, 10), out)
    b.table = table
    b.table[0, 62], b.table[1, -3], b.table[1, 0] = -1, b.pages, -7
    b.check(b.window(q, 100, 10), b.behind(100, 10))
    b.table[:] = -1                                         # rows that see nothing
    assert not b.window(q, 100, 10).any()


@KINDS
def test_window_past_the_table(q, kind):
    """A context longer than its table row: what is left of the window is seen, or nothing but the first keys."""
    g = np.random.default_rng(8)
    for window, sinks in ((40, 3), (500, 0), (5, 0)):
        b = Batch(g, kind, [160, 90], [4, 6], 4, 2, 64, 16)
        b.table, b.width = b.table[:, :9].copy(), 9
        b.check(b.window(q, window, sinks), b.behind(window, sinks))


@KINDS
def test_window_hidden_places_may_hold_anything(q, kind):
    """NaN and infinities behind the window, in page tails and in later tokens stay out; a row that sees them has them."""
    g = np.random.default_rng(12)
    b = Batch(g, kind, [200, 3000], [6, 40], 4, 2, 64, 16)
    rows = [(0, 150), (0, 203), (1, 2900), (1, 3020)]       # out of sight of some tokens, or of all
    for r, pos in rows:
        page, at = b.table[r, pos // 16], pos % 16
        for i in range(2):
            if kind in ("s8", "q4"):
                b.scales[i][page, at] = float("nan")
            else:
                b.kv[i][page, at] = float("nan") if pos % 2 else float("inf")
            b.values[i][page, at] = np.nan
    window, sinks = 45, 2
    out = b.window(q, window, sinks)
    sees = b.behind(window, sinks)
    for r in range(2):
        hit = np.zeros(b.new[r], bool)
        for rr, pos in rows:
            if rr == r:
                hit |= sees(r)[:, pos]
        got = f64(out)[b.cu[r]:b.cu[r + 1]]
        assert np.isfinite(got[~hit]).all() and (~np.isfinite(got[hit])).any(-1).all() and hit.any() and not hit.all()
    for i in range(2):                                      # the rows that see none of it, by value
        for r, pos in rows:
            b.values[i][b.table[r, pos // 16], pos % 16] = 0
            b.size[i] = np.array(b.size[i])
    clean = out.clone()
    for r in range(2):
        for t in range(b.new[r]):
            if any(rr == r and sees(r)[t, pos] for rr, pos in rows):
                clean[b.cu[r] + t] = 0

    def only(r):
        s = sees(r)
        for rr, pos in rows:
            if rr == r:
                s[s[:, pos]] = False
        return s
    b.check(clean, only)


@KINDS
@pytest.mark.parametrize("order", ["hnd", "wide"])
def test_window_cache_orders(q, kind, order):
    b = Batch(np.random.default_rng(9), kind, [170, 3], [5, 11], 6, 3, 64, 16, order)
    b.check(b.window(q, 60, 4), b.behind(60, 4))


@KINDS
def test_window_scale_and_outputs(q, kind):
    """Other scales; strided queries and outputs; rows past the last request stay."""
    b = Batch(np.random.default_rng(11), kind, [50, 90], [6, 3], 4, 2, 64, 16, spare_rows=2)
    for scale in (0.02, -0.1, 0.0):
        room = torch.full((b.T, 6, 72), 5.0, dtype=b.xt, device=torch_dev())
        out = room[:, 1:5, 3:67]
        assert b.window(q, 30, 3, scale, out=out) is out
        b.check(out, b.behind(30, 3), scale)
        assert (room[-2:] == 5.0).all()
        out.fill_(5.0)
        assert (room == 5.0).all()
    wide = torch.full((b.T, 5, 70), float("nan"), dtype=b.xt, device=torch_dev())
    wide[:, 1:, 1:65] = b.q.to(torch_dev())
    args, scales = b.args()
    out = q.window_attention(wide[:, 1:, 1:65], *args[1:], 30, 3, **scales)
    b.check(out, b.behind(30, 3))


@KINDS
def test_window_large_and_equal_scores(q, kind):
    g = np.random.default_rng(10)
    b = Batch(g, kind, [5003, 0, 2048, 1], [4, 90, 1, 3], 4, 2, 128, 16, std=6.0)
    b.check(b.window(q, 1000, 100), b.behind(1000, 100))
    b.q[:] = 0
    b.check(b.window(q, 1000, 100), b.behind(1000, 100))


def test_window_agrees_with_the_tree(q):
    """A chain of drafted tokens without a window: both calls within a rounding of each other."""
    for kind in ("f16", "bf16", "s8", "q4"):
        b = Batch(np.random.default_rng(13), kind, [400, 30], [17, 80], 8, 2, 128, 16)
        args, scales = b.args()
        out = q.tree_attention(*args, **scales)
        b.check(out, b.behind(1 << 40, 0))
        b.check(b.window(q, 1 << 31, 0), b.behind(1 << 40, 0))


@pytest.mark.parametrize("ctx,new,Hq,Hkv,D,page", [
    ([0], [1], 1, 1, 16, 16), ([37], [1], 16, 8, 128, 16), ([5, 130, 33], [7, 16, 1], 4, 4, 64, 7),
    ([300, 17], [20, 33], 8, 2, 128, 24), ([90], [70], 6, 2, 80, 1), ([310, 200], [9, 5], 8, 1, 256, 32),
    ([9001, 0, 2100], [2, 30, 1], 2, 2, 96, 16), ([3000], [66], 4, 1, 48, 64)])
def test_tree_over_4_bits(q, ctx, new, Hq, Hkv, D, page):
    g = np.random.default_rng(len(ctx) + D)
    b = Batch(g, "q4", ctx, new, Hq, Hkv, D, page)
    mask = np.zeros((b.T, max(new)), bool)
    for r in range(len(ctx)):
        mask[b.cu[r]:b.cu[r + 1], :new[r]] = serve_ref.random_tree(g, new[r])
    if len(ctx) == 3:
        mask[b.cu[1]] = False                               # a row with nothing drafted to see
    args, scales = b.args()

    def sees(r):
        n, L = new[r], ctx[r] + new[r]
        s = np.ones((n, L), bool)
        s[:, ctx[r]:] = mask[b.cu[r]:b.cu[r + 1], :n]
        return s
    out = q.tree_attention(*args, to_dev(mask), **scales)
    b.check(out, sees)
    ws = torch.full((q.lib.qmm_tree_attention_workspace_bytes(b.T, Hq, len(ctx), Hkv, D),), 255, dtype=torch.uint8, device=torch_dev())
    assert torch.equal(q.tree_attention(*args, to_dev(mask), **scales, ws=ws), out)


@pytest.mark.parametrize("ctx,new,Hq,Hkv,D,page", [
    ([5000, 4100, 300, 9000], [1, 2, 1, 1], 16, 8, 128, 16),   # eight heads a workgroup
    ([9000, 0, 4100, 7], [9, 3, 11, 8], 16, 8, 80, 24),        # two tiles of 16 rows
    ([4500, 6000], [6, 1], 24, 8, 256, 64), ([7000, 9000, 8000], [1, 1, 2], 32, 8, 64, 7),
    ([12000, 100, 9000, 8000, 12345, 6000], [1, 1, 2, 1, 1, 1], 8, 4, 96, 32),  # four heads
    ([9000, 8000, 12000], [8, 7, 9], 8, 4, 128, 16), ([40000], [1], 4, 4, 256, 64)])
def test_few_rows_over_4_bits_by_heads(q, ctx, new, Hq, Hkv, D, page):
    """Long enough contexts that a wavefront takes a cache head, with the whole context and behind windows; NaN in a row
    that a later token alone sees; steps that grow and fall by orders of magnitude along the keys."""
    g = np.random.default_rng(sum(ctx))
    b = Batch(g, "q4", ctx, new, Hq, Hkv, D, page)
    args, scales = b.args()
    out = q.tree_attention(*args, **scales)
    b.check(out, b.behind(1 << 40, 0))
    assert torch.equal(q.tree_attention(*args, **scales), out)
    for window, sinks in ((3500, 70), (40, 9000)):
        b.check(b.window(q, window, sinks), b.behind(window, sinks))
    b.size[1], b.step = np.array(b.size[1]), np.array(b.step)
    for sign in (1, -1):
        for r in range(len(ctx)):
            for j in range(0, ctx[r] + new[r], page):
                f = 2.0 ** (sign * (12 * j // (ctx[r] + new[r]) - 6))
                where = b.table[r, j // page]
                b.scales[1][where] *= f
                b.values[1][where] *= f
                b.size[1][where] *= f
                b.step[where] *= f
        b.check(b.window(q, 1 << 31, 0), b.behind(1 << 40, 0))


@pytest.mark.parametrize("ctx,new,Hq,Hkv,D,page", [
    ([5000, 4100, 300, 9000], [16, 12, 9, 14], 16, 8, 128, 16),   # eight heads a workgroup
    ([5000, 4100, 300, 9000], [16, 12, 9, 14], 16, 8, 64, 16), ([6000, 31, 4100], [9, 5, 7], 32, 8, 80, 7),
    ([9000, 8000, 12000], [16, 12, 9], 8, 4, 128, 16),            # four
    ([9000, 8000, 12000], [16, 12, 9], 8, 4, 96, 24), ([5000, 9000], [5, 6], 16, 4, 256, 32),
    ([300, 200], [16, 12], 4, 2, 128, 16), ([0, 1700], [12, 17], 6, 3, 80, 5),  # keys side by side
    ([333, 64, 0], [5, 8, 6], 4, 1, 256, 64), ([29], [30], 2, 2, 16, 1)])
def test_two_row_tiles_over_4_bits(q, ctx, new, Hq, Hkv, D, page):
    """More than 16 and at most 32 rows a request: causal, behind trees, behind masks narrower than the drafted tokens
    and behind windows."""
    rows = sum(new) * (Hq // Hkv) / len(ctx)
    assert 16 < rows <= 32
    g = np.random.default_rng(sum(ctx) + D)
    b = Batch(g, "q4", ctx, new, Hq, Hkv, D, page)
    args, scales = b.args()
    out = q.tree_attention(*args, **scales)
    b.check(out, b.behind(1 << 40, 0))
    assert torch.equal(q.tree_attention(*args, **scales), out)
    most = max(new)
    for cols in (most + 3, most, most - 2, 1):
        mask = np.zeros((b.T, cols), bool)
        for r in range(len(ctx)):
            n = min(new[r], cols)
            mask[b.cu[r]:b.cu[r + 1], :n] = serve_ref.random_tree(g, new[r])[:, :n]
        mask[b.cu[1] if len(ctx) > 1 else 3] = False
        wide = torch.ones(b.T, cols + 5, dtype=torch.bool, device=torch_dev())
        wide[:, 2:2 + cols] = to_dev(mask)

        def sees(r):
            s = np.ones((new[r], ctx[r] + new[r]), bool)
            n = min(new[r], cols)
            s[:, ctx[r]:] = False
            s[:, ctx[r]:ctx[r] + n] = mask[b.cu[r]:b.cu[r + 1], :n]
            return s
        b.check(q.tree_attention(*args, wide[:, 2:2 + cols], **scales), sees)
    for window, sinks in ((1 << 31, 0), (3500, 70), (40, 9000), (7, 3)):
        b.check(b.window(q, window, sinks), b.behind(window, sinks))


def test_few_rows_over_4_bits_nan(q):
    """NaN behind a tree's mask, by heads and by keys: the rows that see it have it, the others are finite and right."""
    for ctx, Hkv in (([5000, 4100, 300, 9000], 8), ([900, 70], 2)):
        g = np.random.default_rng(Hkv)
        new = [3] * len(ctx)
        b = Batch(g, "q4", ctx, new, 2 * Hkv, Hkv, 64, 16)
        mask = np.zeros((b.T, 3), bool)
        mask[0::3, 0] = mask[1::3, 1] = mask[2::3, 2] = mask[2::3, 1] = True
        for r in range(len(ctx)):
            p = ctx[r] + 1                                  # the second drafted token, which the third sees
            for i in range(2):
                b.scales[i][b.table[r, p // 16], p % 16] = float("nan")
                b.values[i][b.table[r, p // 16], p % 16] = 0
        args, scales = b.args()
        out = q.tree_attention(*args, to_dev(mask), **scales)
        got = f64(out)
        assert np.isnan(got[1::3]).all() and np.isnan(got[2::3]).all() and np.isfinite(got[0::3]).all()
        out[1::3] = out[2::3] = 0

        def sees(r):
            s = np.zeros((3, ctx[r] + 3), bool)
            s[0, :ctx[r] + 1] = True
            return s
        b.check(out, sees)


def test_cache_past_31_bits(q):
    """A cache of more than 2^31 bytes, and of more than 2^32 elements: rows at its end."""
    pages, page, H, D = 2100, 128, 128, 128                 # 2.2e9 bytes of codes in K alone
    dev = torch_dev()
    kc, vc = (torch.zeros(pages, page, H, D // 2, dtype=torch.uint8, device=dev) for _ in range(2))
    ks, vs = (torch.zeros(pages, page, H, 2, dtype=BF16, device=dev) for _ in range(2))
    g = np.random.default_rng(2)
    T = 200
    slots = torch.arange(pages * page - T, pages * page, device=dev)
    x = [to_dev(g.standard_normal((T, H, D)).astype(np.float32)) for _ in range(2)]
    q.kv_append(*x, slots, kc, vc, ks, vs)
    values = []
    for y, got in zip(x, q.kv_gather(slots, kc, vc, ks, vs)):
        k, s, m = ref.quantize_q4(y.cpu().numpy())
        values.append(k * s[..., None].astype(np.float64) + m[..., None])
        assert np.array_equal(f64(got), values[-1].astype(np.float32).astype(np.float64))
    table = torch.tensor([[pages - 2, pages - 1]], dtype=torch.int32, device=dev)
    Q = to_dev(g.standard_normal((1, H, D))).to(BF16)
    first = 2 * page - T
    ctx, cu = torch.tensor([2 * page - 1], dtype=torch.int32, device=dev), torch.tensor([0, 1], dtype=torch.int32, device=dev)
    out = f64(q.window_attention(Q, kc, vc, table, ctx, cu, T, 0, k_scale=ks, v_scale=vs))
    want, size = ref.attention(f64(Q), values[0], values[1], np.ones((1, T), bool), D ** -0.5)
    assert first > 0 and np.abs(out - want).max() <= (2.0 ** -8 + 2.0 ** -9) * np.abs(want).max() + 2.0 ** -10 * size.max()


# ---------------------------------------------------------------- adapters ---

def _lora_case(g, T, K, N, rank, n, xt, ids=None, base=True, scales=True):
    wt = BF16 if xt == F32 else xt
    X = torch.from_numpy(g.standard_normal((T, K))).to(xt)
    A = torch.from_numpy(g.standard_normal((n, rank, K)) * K ** -0.5).to(wt)
    B = torch.from_numpy(g.standard_normal((n, N, rank)) * max(rank, 1) ** -0.5).to(wt)
    Y = torch.from_numpy(g.standard_normal((T, N))).to(xt) if base else None
    s = torch.from_numpy((g.random(n) + 0.5).astype(np.float32)) if scales else None
    if ids is None:
        ids = g.integers(-1, n + 1, T)                     # rows without an adapter on both sides
    return X, A, B, torch.from_numpy(np.asarray(ids, np.int32)), Y, s


def _dev(*ts):
    return [None if t is None else t.to(torch_dev()) for t in ts]


def _check_lora(out, X, A, B, ids, Y, s):
    K, rank = X.shape[1], A.shape[1]
    args = [None if t is None else t.double().numpy() for t in (X, A, B)]
    want, size = ref.lora(*args, ids.numpy(), None if Y is None else Y.double().numpy(), None if s is None else s.numpy())
    got, xt = f64(out), X.dtype
    z = 2.0 ** -16 if xt != F32 else 4 * U
    tol = torch.finfo(xt).eps / 2 * np.abs(want) + ((K + rank + 32) * U + z) * size + 2 * U * np.abs(want)
    tol = tol + torch.finfo(xt).smallest_normal * torch.finfo(xt).eps
    assert np.isfinite(got).all() and (np.abs(got - want) <= tol).all(), float((np.abs(got - want) / tol).max())
    if xt == F32 and want.size >= 64:
        assert np.linalg.norm(got - want) <= 8 * np.sqrt(K / 32 + rank / 32 + 8) * U * np.linalg.norm(np.abs(want) + size)


@X3
@pytest.mark.parametrize("T,K,N,rank,n", [
    (1, 1, 1, 1, 1), (1, 64, 16, 8, 3), (2, 33, 17, 3, 2), (15, 100, 70, 16, 4), (16, 128, 64, 17, 20), (17, 520, 65, 33, 5),
    (61, 1025, 300, 12, 24), (64, 2048, 256, 64, 2), (100, 40, 1000, 100, 7), (33, 4100, 130, 128, 3), (513, 260, 90, 16, 6),
    (600, 96, 520, 64, 40), (1030, 64, 33, 5, 1), (300, 200, 150, 128, 3), (129, 1000, 700, 40, 9), (260, 5000, 130, 100, 2),
    (700, 130, 2000, 16, 3)])
def test_lora(q, T, K, N, rank, n, xt):
    c = _lora_case(np.random.default_rng(T + K + N), T, K, N, rank, n, xt)
    out = q.lora_matmul(*_dev(*c))
    _check_lora(out, *c)
    ws = torch.full((q.lib.qmm_lora_matmul_workspace_bytes(T, K, rank),), 255, dtype=torch.uint8, device=torch_dev())
    assert torch.equal(q.lora_matmul(*_dev(*c), ws=ws), out)
    base = c[4].to(torch_dev())
    X, A, B, ids, _, s = _dev(*c)
    assert q.lora_matmul(X, A, B, ids, base, s, out=base) is base and torch.equal(base, out)


@X3
def test_lora_rows_in_runs(q, xt):
    """Rows of one adapter together, as in prompts, and one adapter for all; without base and scales."""
    g = np.random.default_rng(4)
    for T in (40, 700):
        ids = np.sort(g.integers(-1, 5, T))
        for i in (ids, np.zeros(T, int), np.full(T, -1)):
            c = _lora_case(g, T, 300, 200, 16, 5, xt, i, base=False, scales=False)
            X, A, B, dev_ids, _, _ = _dev(*c)
            _check_lora(q.lora_matmul(X, A, B, dev_ids), *c)


@X3
def test_lora_strides_and_neighbours(q, xt):
    """Misaligned and padded rows of everything; what lies beside the output stays, and NaN beside the inputs stays out."""
    g = np.random.default_rng(6)
    wt = BF16 if xt == F32 else xt

    def inside(t, off, pad):
        if t is None:
            return None
        wide = torch.full([d + 1 for d in t.shape[:-1]] + [t.shape[-1] + pad], float("nan"), dtype=t.dtype, device=torch_dev())
        view = wide[tuple(slice(0, d) for d in t.shape[:-1]) + (slice(off, off + t.shape[-1]),)]
        view.copy_(t.to(torch_dev()))
        return view
    for T, off, pad in ((7, 1, 5), (30, 8, 16), (600, 3, 4)):
        X, A, B, ids, Y, s = _lora_case(g, T, 136, 72, 24, 6, xt)
        room = torch.full((T + 2, 72 + 9), 7.0, dtype=xt, device=torch_dev())
        out = room[1:T + 1, 3:75]
        got = q.lora_matmul(inside(X, off, pad), inside(A, off, pad), inside(B, off, pad), ids.to(torch_dev()), inside(Y, off, pad),
                            s.to(torch_dev()), out=out)
        assert got is out and A.dtype == wt
        _check_lora(out, X, A, B, ids, Y, s)
        out.fill_(7.0)
        assert (room == 7.0).all()


@X3
def test_lora_nan_and_infinity_stay_where_they_are(q, xt):
    g = np.random.default_rng(7)
    for T in (20, 600):
        X, A, B, ids, Y, s = _lora_case(g, T, 70, 90, 16, 4, xt, g.integers(0, 4, T))
        A[2] = float("nan")
        B[3] = float("inf")
        X[5], ids[5] = float("nan"), 0
        X[6, 3], ids[6] = float("inf"), 1
        X[7], ids[7], Y[7] = float("inf"), -1, 3.0
        out = f64(q.lora_matmul(*_dev(X, A, B, ids, Y, s)))
        i = ids.numpy()
        bad = (i == 2) | (i == 3)
        bad[[5, 6]] = True
        assert not np.isfinite(out[bad]).any() and np.isfinite(out[~bad]).all() and (out[7] == 3.0).all()
        keep = torch.from_numpy(~bad)
        A[2] = B[3] = 0
        X[7] = 0
        _check_lora(torch.from_numpy(out[~bad]).to(xt), X[keep], A, B, ids[keep], Y[keep], s)


def test_lora_large_and_small_values(q):
    """Inner sums past the range of fp16, and far below it, beside rows of ordinary ones."""
    g = np.random.default_rng(8)
    for T in (12, 520):
        X, A, B, ids, Y, s = _lora_case(g, T, 256, 64, 16, 3, F16, g.integers(0, 3, T), base=False)
        X[1] *= 20000.0
        A[1] *= 200.0
        X[2] *= 2.0 ** -12
        A[2] *= 2.0 ** -10
        B[1] *= 2.0 ** -12
        B[2] *= 2.0 ** 10
        X = X.clamp(-60000, 60000)
        _check_lora(q.lora_matmul(*_dev(X, A, B, ids, None, s)), X, A, B, ids, None, s)


def test_lora_nothing_to_do(q):
    X, A, B, ids, Y, s = _dev(*_lora_case(np.random.default_rng(9), 5, 32, 24, 8, 2, BF16))
    assert q.lora_matmul(X[:0], A, B, ids[:0], Y[:0], s).shape == (0, 24)
    assert q.lora_matmul(X, A, B[:, :0], ids, Y[:, :0], s).shape == (5, 0)
    assert torch.equal(q.lora_matmul(X, A[:0], B[:0], ids, Y, s[:0]), Y)


# ------------------------------------------------------- log probabilities ---

def _check_logprobs(r, x, tokens, top, scale=1.0):
    V = x.shape[1]
    lp, ent, ids, values = ref.logprobs(x, tokens.reshape(x.shape[0], -1), top, float(np.float32(scale)))
    assert np.array_equal(r.top_ids.cpu().numpy(), ids)
    for got, want in ((r.logprobs, lp.reshape(tokens.shape)), (r.top_logprobs, values)):
        got = f64(got)
        assert got.shape == want.shape
        same = (np.isnan(got) & np.isnan(want)) | (got == want)
        with np.errstate(invalid="ignore"):
            same |= np.abs(got - want) <= 128 * U + 4 * U * np.abs(want)
        assert same.all(), (np.argwhere(~same)[:4], got[~same][:4], want[~same][:4])
    got = f64(r.entropy)
    with np.errstate(invalid="ignore"):
        same = (np.isnan(got) & np.isnan(ent)) | (np.abs(got - ent) <= 128 * U * (np.log2(V) + 3))
    assert same.all(), (got[~same][:4], ent[~same][:4])


@X3
@pytest.mark.parametrize("T,V,top,n", [(1, 1, 1, 1), (1, 2, 32, 3), (3, 7, 0, 1), (2, 31, 5, 2), (5, 33, 32, 1), (4, 100, 20, 8),
                                       (3, 4097, 1, 0), (2, 50021, 20, 1), (1, 151936, 5, 1), (70, 1001, 3, 1), (3000, 50, 4, 1),
                                       (600, 9000, 20, 2)])
def test_logprobs(q, T, V, top, n, xt):
    g = np.random.default_rng(T + V)
    x = torch.from_numpy(g.standard_normal((T, V)) * 3).to(xt)
    tokens = g.integers(0, V, (T, n))
    if n == 1:
        tokens = tokens[:, 0]
    for scale in (1.0, 0.6):
        r = q.token_logprobs(x.to(torch_dev()), to_dev(tokens), top, scale)
        _check_logprobs(r, x.double().numpy(), tokens, top, scale)
    none = q.token_logprobs(x.to(torch_dev()), None, top, 0.6)
    assert none.logprobs.shape == (T, 0) and torch.equal(none.entropy, r.entropy) and torch.equal(none.top_ids, r.top_ids)


@X3
def test_logprobs_rows_of_wider_tensors(q, xt):
    """Every alignment of a row; NaN beside it stays out; tokens in strided rows, outside the vocabulary and twice the same."""
    g = np.random.default_rng(2)
    for T, V, off in [(9, 1000, 1), (3, 5003, 3), (130, 2500, 5), (2, 17, 2)]:
        wide = torch.full((T + 1, V + 9), float("nan"), dtype=xt, device=torch_dev())
        x = wide[:T, off:off + V]
        x.copy_(torch.from_numpy(g.standard_normal((T, V)) * 4))
        tokens = g.integers(-2, V + 2, (T, 5))
        tokens[0] = [V - 1, V, -1, 1 << 40, V - 1]
        for view in (to_dev(np.pad(tokens, ((0, 0), (2, 1))))[:, 2:7], to_dev(tokens)[:, :1], to_dev(tokens)[:, 1]):
            r = q.token_logprobs(x, view, 7)
            _check_logprobs(r, f64(x), view.cpu().numpy(), 7)


@X3
def test_logprobs_ties_and_orders(q, xt):
    """Equal logits stand by their tokens, of few values and of one; ascending and descending rows; rows whose largest
    logits lie where the kernel's first bound says least."""
    V = 40000
    v = np.arange(V)
    rows = [np.zeros(V), np.where(v % 2, 0.0, -0.0), v % 7, -(v // 5000), v * 0.01, -v * 0.01, np.where(v == V - 1, 9.0, 0.0),
            np.where(v // 32 % 256 < 128, 1.0 + (v % 3), 0.0), np.random.default_rng(3).integers(-3, 4, V)]
    x = torch.from_numpy(np.stack([np.asarray(r, np.float64) for r in rows])).to(xt)
    tokens = np.zeros(len(rows), np.int64)
    for top in (1, 20, 32):
        _check_logprobs(q.token_logprobs(x.to(torch_dev()), to_dev(tokens), top), x.double().numpy(), tokens, top)


def test_logprobs_more_groups_than_are_listed(q):
    """The largest logits in the groups of few threads, more of them than the first list holds."""
    V = 500000
    v = np.arange(V)
    x = np.where(v // 32 % 256 < 80, (v // 32 // 256 * 7 % 61) * 0.25, -1.0)[None].astype(np.float32)
    tokens = np.array([5])
    for top in (20, 32):
        _check_logprobs(q.token_logprobs(to_dev(x), to_dev(tokens), top), x.astype(np.float64), tokens, top)


@X3
def test_logprobs_masked_rows(q, xt):
    """-inf for tokens that a grammar rules out, in all of a row, in all but one and in whole pieces of it; NaN and +inf
    make a row NaN and no other; the type's lowest and largest values."""
    g = np.random.default_rng(4)
    T, V = 12, 9000
    x = torch.from_numpy(g.standard_normal((T, V))).to(xt)
    low = torch.finfo(xt).min if xt != F32 else -1e38
    x[0] = -float("inf")
    x[1] = -float("inf")
    x[1, 8999] = -4.0
    x[2, 100:] = -float("inf")
    x[3, :8900] = -float("inf")
    x[4, 77] = float("nan")
    x[5, 4500] = float("inf")
    x[6] = low
    x[7] = low
    x[7, 13] = 2.0
    x[8] = float("nan")
    x[9, ::2] = -float("inf")
    x[10, 3] = x[10, 5] = 60000.0
    tokens = np.stack([np.full(T, 13), np.full(T, 8999), np.full(T, -1)], 1)
    r = q.token_logprobs(x.to(torch_dev()), to_dev(tokens), 6)
    _check_logprobs(r, x.double().numpy(), tokens, 6)
    assert float(r.logprobs[1, 1]) == 0.0 and float(r.entropy[0]) == 0.0


def test_logprobs_refuses_an_output_of_another_shape(q):
    x = torch.zeros(3, 40, device=torch_dev())
    t = torch.zeros(3, dtype=torch.int64, device=torch_dev())
    r = q.token_logprobs(x, t, 2)
    assert q.token_logprobs(x, t, 2, out=r) is r
    for field, bad in (("logprobs", r.logprobs[:2]), ("entropy", r.entropy.double()), ("top_ids", r.top_ids.int()),
                       ("top_logprobs", r.top_logprobs[:, :1])):
        import dataclasses
        with pytest.raises(ValueError):
            q.token_logprobs(x, t, 2, out=dataclasses.replace(r, **{field: bad}))


# ------------------------------------------------- streams, graphs, together ---

def test_side_stream_and_graph(q):
    """Every call on another stream than the tensors' and in one captured graph, over changing inputs: each replay gives
    the eager call's bits."""
    g = np.random.default_rng(20)
    dev = torch_dev()
    b = Batch(g, "q4", [300, 40, 129], [3, 1, 5], 8, 2, 64, 16)
    args, scales = b.args()
    lora = _dev(*_lora_case(g, 9, 200, 512, 16, 3, BF16))
    x, tokens = to_dev(g.standard_normal((9, 3001)).astype(np.float32)), to_dev(g.integers(0, 3001, 9))
    rows = [to_dev(g.standard_normal((9, 2, 64)).astype(np.float32)) for _ in range(2)]
    slots = to_dev(g.permutation(b.pages * 16)[:9].astype(np.int64))
    cache = (args[1], args[2], scales["k_scale"], scales["v_scale"])
    outs = dict(k=torch.empty(9, 2, 64, device=dev), v=torch.empty(9, 2, 64, device=dev), w=torch.empty_like(args[0]),
                t=torch.empty_like(args[0]), y=torch.empty(9, 512, dtype=BF16, device=dev))
    lp = q.token_logprobs(x, tokens, 5)
    wss = [torch.empty(n, dtype=torch.uint8, device=dev) for n in (
        q.lib.qmm_window_attention_workspace_bytes(9, 8, 3, 2, 64), q.lib.qmm_lora_matmul_workspace_bytes(9, 200, 16),
        q.lib.qmm_token_logprobs_workspace_bytes(9, 3001))]

    def run(stream=None):
        q.kv_append(*rows, slots, *cache, stream=stream)
        q.kv_gather(slots, *cache, out=(outs["k"], outs["v"]), stream=stream)
        q.window_attention(*args, 70, 3, **scales, out=outs["w"], ws=wss[0], stream=stream)
        q.tree_attention(*args, **scales, out=outs["t"], ws=wss[0], stream=stream)
        q.lora_matmul(*lora[:4], lora[4], lora[5], out=outs["y"], ws=wss[1], stream=stream)
        q.token_logprobs(x, tokens, 5, out=lp, ws=wss[2], stream=stream)

    def take():
        torch.cuda.synchronize()
        return [t.clone() for t in list(outs.values()) + [lp.logprobs, lp.entropy, lp.top_ids, lp.top_logprobs, *cache]]

    def spoil():
        for t in list(outs.values()) + [lp.logprobs, lp.entropy, lp.top_ids, lp.top_logprobs, *wss]:
            t.fill_(99)

    def change():
        for t in (*rows, x, lora[0], args[0]):
            t.copy_(torch.from_numpy(g.standard_normal(t.shape)))
        args[4].copy_(torch.from_numpy(g.integers(0, 40, 3)))
        lora[3].copy_(torch.from_numpy(g.integers(-1, 3, 9)))
        tokens.copy_(torch.from_numpy(g.integers(0, 3001, 9)))
    side = torch.cuda.Stream()
    run()
    want = take()
    spoil()
    torch.cuda.synchronize()
    run(side)
    assert all(torch.equal(a, c) for a, c in zip(take(), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(4):
        change()
        spoil()
        torch.cuda.synchronize()
        graph.replay()
        got = take()
        spoil()
        run()
        assert all(torch.equal(a, c) for a, c in zip(got, take()))


def test_a_layer_over_a_4_bit_cache(q):
    """Projections with adapters, the plan, the append into 4 bits, attention behind a window, logits and their log
    probabilities: prompts and then single tokens, with the pages behind the window given back."""
    g = np.random.default_rng(21)
    dev = torch_dev()
    R, hidden, Hq, Hkv, D, page, V, window, sinks, rank = 3, 256, 4, 2, 64, 16, 700, 40, 2, 8

    def weight(K, N):
        codes = to_dev(g.integers(0, 256, (N, K // 2)).astype(np.uint8))
        s = (to_dev(g.random((N, K // 64)).astype(np.float32)) + 0.5) * (0.2 / K ** 0.5)
        W = q.q4_group_repack(codes, s.half(), K=K, group=64)
        k = np.stack([f64(codes) % 16, f64(codes) // 16], -1).reshape(N, K)
        return W, ((k - 8) * np.repeat(f64(s.half()), 64, 1)).T
    wq, wk, wv, wo = weight(hidden, Hq * D), weight(hidden, Hkv * D), weight(hidden, Hkv * D), weight(hidden, V)
    A = torch.from_numpy(g.standard_normal((2, rank, hidden)) / 16).to(BF16).to(dev)
    B = torch.from_numpy(g.standard_normal((2, Hq * D, rank)) / 3).to(BF16).to(dev)
    scales = torch.tensor([0.5, 2.0], device=dev)
    of_request = np.array([1, -1, 0])
    prompt = [70, 33, 9]
    width, pages = 8, 24
    (kc, vc), (ks, vs) = _q4_cache(pages, page, Hkv, D)
    table = torch.full((R, width), -1, dtype=torch.int32, device=dev)
    free = to_dev(g.permutation(pages).astype(np.int32))
    taken = torch.zeros(1, dtype=torch.int32, device=dev)
    ctx = torch.zeros(R, dtype=torch.int32, device=dev)
    held = [[[], []] for _ in range(R)]                     # the rows that the cache stands for
    for step in range(5):
        new = prompt if step == 0 else [1] * R
        T = sum(new)
        X = torch.from_numpy(g.standard_normal((T, hidden))).to(BF16).to(dev)
        ids = to_dev(np.repeat(of_request, new).astype(np.int32))
        plan = q.kv_plan(ctx, to_dev(np.array(new, np.int32)), table, free, page, T, free_begin=taken)
        taken = plan.info[0:1]
        Q = q.lora_matmul(X, A, B, ids, q.q4_group_matmul(X, wq[0]), scales)
        K, Vv = q.q4_group_matmul(X, wk[0]), q.q4_group_matmul(X, wv[0])
        q.kv_append(K.view(T, Hkv, D), Vv.view(T, Hkv, D), plan.slots, kc, vc, ks, vs)
        o = q.window_attention(Q.view(T, Hq, D), kc, vc, table, ctx, plan.cu_new, window, sinks, k_scale=ks, v_scale=vs)
        logits = q.q4_group_matmul(o.view(T, Hq * D), wo[0])
        tokens = to_dev(g.integers(0, V, T))
        r = q.token_logprobs(logits, tokens, 3)
        assert int(plan.info[2]) == 0
        # each step from what the one before it gave
        want, size = ref.lora(f64(X), f64(A), f64(B), ids.cpu().numpy(), f64(X) @ wq[1], f64(scales))
        assert np.abs(f64(Q) - want).max() <= 3 * 2.0 ** -8 * np.abs(want).max() + 2.0 ** -14 * size.max()
        rows = [ref.quantize_q4(t.float().cpu().numpy().reshape(T, Hkv, D)) for t in (K, Vv)]
        rows = [k * s[..., None].astype(np.float64) + m[..., None] for k, s, m in rows]
        cu = plan.cu_new.cpu().numpy()
        for i in range(R):
            for h, x in zip(held[i], rows):
                h.append(x[cu[i]:cu[i + 1]])
            k, v = (np.concatenate(h) for h in held[i])
            c = int(ctx[i])
            assert len(k) == c + new[i]
            want, size = ref.attention(f64(Q)[cu[i]:cu[i + 1]].reshape(-1, Hq, D), k, v, ref.window_sees(c, new[i], len(k), window, sinks), D ** -0.5)
            assert np.abs(f64(o)[cu[i]:cu[i + 1]] - want).max() <= 2.0 ** -8 * np.abs(want).max() + 2.0 ** -11 * size.max()
        _check_logprobs(r, f64(logits), tokens.cpu().numpy(), 3)
        ctx = ctx + to_dev(np.array(new, np.int32))
        for i in range(R):                                  # pages behind the window, but the first, leave the table
            table[i, 1:max(1, (int(ctx[i]) + 1 - window) // page)] = -1


def test_example_over_4_bits(q):
    """The example's layer over a 4-bit cache.  A row of 128 unit normals spans about 5.4, a step 0.36, so k and v are off
    by an rms of 0.1 each: 0.1 of a score and of a value, about a sixth of the attention branch, which is 0.4 of the
    output's unit size.  Five times that 0.07, over the largest output of about 4, stays below 2^-3."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "verify_step.py")
    spec = importlib.util.spec_from_file_location("verify_step", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    assert 0 < m.run(requests=3, prompt=130, drafts=6, steps=3, cache="q4") <= 2.0 ** -3
