"""CPU checks of the long-context serving operators: the plain forms against
independent statements of the same thing, and every refusal of the C ABI and the
binding (each fails before any HIP call)."""
import ctypes

import numpy as np
import pytest
import torch

import long_ref as ref

FAKE = 4096  # never dereferenced: each call below fails validation first


@pytest.fixture(scope="module")
def q():
    import int8_bit_weight_amd as q
    return q


# ------------------------------------------------------------ plain forms ---

def test_plain_q4_rows():
    g = np.random.default_rng(1)
    codes = g.integers(0, 16, (3, 5, 48)).astype(np.uint8)
    b = ref.pack_q4(codes)
    assert b.shape == (3, 5, 24) and np.array_equal(ref.unpack_q4(b), codes)
    word = ref.pack_q4(np.arange(8, dtype=np.uint8)[None]).view(np.uint32)[0, 0]
    assert word == 0x75316420                               # nibbles from the low end: 0 2 4 6 1 3 5 7
    x = g.standard_normal((40, 64)).astype(np.float32)
    x[3], x[4] = 0, 2.5
    q, step, m = ref.quantize_q4(x)
    y = q * step[:, None].astype(np.float64) + m[:, None]
    # half a step for the code, and what the bf16 roundings of step (over 15 of them) and minimum move
    tol = step / 2 + (15 * step + np.abs(m)) * 2.0 ** -8
    assert (np.abs(y - x) <= tol[:, None]).all() and step[3] == 0 and (y[4] == 2.5).all()


def test_plain_window_is_the_set():
    for ctx, n, window, sinks in ((5, 4, 3, 2), (0, 7, 1, 0), (3, 3, 100, 1), (20, 2, 4, 30)):
        sees = ref.window_sees(ctx, n, ctx + n, window, sinks)
        for i in range(n):
            want = {j for j in range(ctx + i + 1) if ctx + i - j < window or j < sinks}
            assert set(np.flatnonzero(sees[i])) == want


def test_plain_attention_is_the_softmax():
    g = np.random.default_rng(2)
    q, k, v = g.standard_normal((3, 4, 8)), g.standard_normal((9, 2, 8)), g.standard_normal((9, 2, 8))
    sees = g.random((3, 9)) < 0.6
    sees[1] = False
    o, _ = ref.attention(q, k, v, sees, 0.3)
    for i in (0, 2):
        for h in range(4):
            s = torch.from_numpy(k[:, h // 2] @ q[i, h] * 0.3).masked_fill(~torch.from_numpy(sees[i]), -np.inf)
            assert np.abs(torch.softmax(s, 0).numpy() @ v[:, h // 2] - o[i, h]).max() < 1e-14
    assert not o[1].any()


def test_plain_logprobs_are_the_log_softmax():
    g = np.random.default_rng(3)
    x = g.standard_normal((4, 50))
    x[1, ::2] = -np.inf
    x[2, 7] = x[2, 30] = x[2].max() + 1
    ids = g.integers(0, 50, (4, 3))
    given, ent, top, values = ref.logprobs(x, ids, 5, 0.7)
    lp = torch.log_softmax(torch.from_numpy(x * 0.7), -1).numpy()
    assert np.allclose(given, np.take_along_axis(lp, ids, 1)) and list(top[2, :2]) == [7, 30]
    p = np.exp(lp)
    assert np.allclose(ent, -(p * np.where(p > 0, lp, 0)).sum(-1))
    assert np.allclose(values, -np.sort(-lp, -1)[:, :5])
    given, ent, top, _ = ref.logprobs(np.array([[-np.inf] * 3, [1, np.nan, 2], [0, np.inf, 1]]), np.array([[0], [2], [5]]), 4)
    assert given[0, 0] == -np.inf and ent[0] == 0 and np.isnan(given[1, 0]) and given[2, 0] == -np.inf and np.isnan(ent[2])
    assert top.tolist() == [[0, 1, 2, -1], [2, 0, 1, -1], [1, 2, 0, -1]]


# --------------------------------------------------------------- refusals ---

def _cache(q, **kw):
    d = dict(k=FAKE, v=FAKE, type=4, num_pages=4, page_size=16, n_heads=2, head_dim=64, page_stride=1024,
             token_stride=64, head_stride=32, k_scale=FAKE, v_scale=FAKE, scale_page_stride=32, scale_token_stride=2,
             scale_head_stride=1)
    d.update(kw)
    return q.qmm_kv_cache(**d)


BAD_CACHES = [(dict(k=None), 1), (dict(v=None), 1), (dict(type=0), 1), (dict(type=5), 1), (dict(num_pages=0), 1),
              (dict(k_scale=None), 1), (dict(v_scale=None), 1), (dict(v_scale=FAKE + 2), 1), (dict(scale_page_stride=-1), 1),
              (dict(page_stride=-8), 1), (dict(head_dim=72), 2), (dict(head_dim=264), 2), (dict(head_dim=272), 2),
              (dict(token_stride=36), 2), (dict(k=FAKE + 4), 2), (dict(page_size=1 << 20), 2)]


def test_cache_refusals(q):
    def append(T=3, slots=FAKE, **kw):
        return q.lib.kv_append(FAKE, 128, 64, FAKE, 128, 64, 2, T, slots, _cache(q, **kw), None)

    def gather(T=3, slots=FAKE, K=FAKE, V=1 << 20, xt=0, ks=128, **kw):
        return q.lib.kv_gather(slots, T, _cache(q, **kw), K, ks, 64, V, 128, 64, xt, None)

    def tree(**kw):
        return q.lib.tree_attention(FAKE, 256, 64, 2, 3, 4, _cache(q, **kw), FAKE, 8, 8, FAKE, FAKE, 2, None, 0, 0, 1.0, FAKE,
                                    256, 64, None, 0, None)
    for kw, want in BAD_CACHES:
        assert append(**kw) == want and gather(**kw) == want and tree(**kw) == want, kw
    assert append(T=0) == 0 and gather(T=0) == 0 and tree() == q.QMM_ERR_WORKSPACE
    for name in ("slots", "K", "V"):
        assert gather(**{name: None}) == 1, name
    assert gather(xt=3) == 1 and gather(xt=4) == 1 and gather(T=-1) == 1 and gather(ks=-1) == 1 and gather(K=FAKE + 2) == 1
    assert gather(V=FAKE) == 1 and gather(V=FAKE + 4 * 64) == 1   # K and V share memory
    assert gather(T=1 << 31) == 2
    for xt in (0, 1):                                             # 4-bit rows are attended to in bf16
        assert q.lib.tree_attention(FAKE, 256, 64, xt, 3, 4, _cache(q), FAKE, 8, 8, FAKE, FAKE, 2, None, 0, 0, 1.0, FAKE,
                                    256, 64, None, 0, None) == 2


def test_window_refusals(q):
    INV, UNS = q.QMM_ERR_INVALID, q.QMM_ERR_UNSUPPORTED

    def f(Q=FAKE, qs=256, xt=2, T=3, Hq=4, table=FAKE, ld=8, width=8, ctx=FAKE, cu=FAKE, R=2, window=100, sinks=4, scale=1.0,
          O=FAKE, ws=None, nbytes=0, **kw):
        return q.lib.window_attention(Q, qs, 64, xt, T, Hq, _cache(q, **kw), table, ld, width, ctx, cu, R, window, sinks,
                                      scale, O, 256, 64, ws, nbytes, None)
    for name in ("Q", "table", "ctx", "cu", "O"):
        assert f(**{name: None}) == INV, name
    assert f(window=0) == INV and f(window=-5) == INV and f(sinks=-1) == INV
    assert f(T=-1) == INV and f(Hq=0) == INV and f(Hq=3) == INV and f(R=-1) == INV and f(ld=7) == INV
    assert f(scale=float("nan")) == INV and f(Q=FAKE + 1) == INV and f(xt=3) == INV
    for kw, want in BAD_CACHES:
        assert f(**kw) == want, kw
    assert f(xt=0) == UNS and f(xt=1) == UNS and f(width=1 << 30, ld=1 << 30) == UNS
    assert f() == q.QMM_ERR_WORKSPACE and f(ws=FAKE + 8, nbytes=1 << 40) == q.QMM_ERR_WORKSPACE
    assert f(ws=FAKE, nbytes=1 << 40) == INV                      # the output is the queries
    far = 1 << 30
    need = q.lib.qmm_window_attention_workspace_bytes(3, 4, 2, 2, 64)
    assert f(O=far, ws=FAKE, nbytes=1000) == q.QMM_ERR_WORKSPACE and need > 1000
    assert f(T=0) == q.QMM_OK and f(R=0) == q.QMM_OK
    assert q.lib.qmm_window_attention_workspace_bytes(0, 4, 2, 2, 64) == 0


def test_lora_refusals(q):
    INV, UNS, WS = q.QMM_ERR_INVALID, q.QMM_ERR_UNSUPPORTED, q.QMM_ERR_WORKSPACE
    far = 1 << 30

    def f(X=FAKE, xt=2, T=3, K=64, ldx=64, A=FAKE, sa=512, lda=64, B=FAKE, sb=256, ldb=8, wt=2, n=2, rank=8, N=32, ids=FAKE,
          scales=None, base=None, ld_base=0, out=far, ld_out=32, ws=2 * far, nbytes=1 << 30):
        return q.lib.lora_matmul(X, xt, T, K, ldx, A, sa, lda, B, sb, ldb, wt, n, rank, N, ids, scales, base, ld_base, out,
                                 ld_out, ws, nbytes, None)
    for name in ("X", "A", "B", "ids", "out"):
        assert f(**{name: None}) == INV, name
    assert f(T=-1) == INV and f(K=0) == INV and f(N=-1) == INV and f(rank=0) == INV and f(n=-1) == INV
    assert f(ldx=63) == INV and f(lda=63) == INV and f(ldb=7) == INV and f(ld_out=31) == INV and f(base=FAKE, ld_base=31) == INV
    assert f(xt=3) == INV and f(wt=4) == INV and f(sa=-1) == INV
    assert f(X=FAKE + 1) == INV and f(A=FAKE + 1) == INV and f(ids=FAKE + 2) == INV and f(scales=FAKE + 2) == INV
    assert f(wt=1) == UNS and f(wt=0) == UNS and f(xt=0, wt=1) == UNS and f(xt=0, wt=0) == UNS
    assert f(rank=129, ldb=129) == UNS and f(T=1 << 24, N=64, ld_out=64) == UNS and f(T=1 << 31) == UNS
    assert f(ws=None) == WS and f(ws=2 * far + 8) == WS and f(nbytes=3 * 16 * 4 - 1) == WS
    assert f(base=far, ld_base=33) == INV and f(base=far + 2, ld_base=32) == INV   # base over out, but not out itself
    assert f(out=FAKE) == INV                                                     # out over X
    assert f(T=0) == q.QMM_OK and f(N=0) == q.QMM_OK
    size = q.lib.qmm_lora_matmul_workspace_bytes
    assert size(3, 64, 8) == 3 * 16 * 4 and size(0, 64, 8) == 0 and size(3, 0, 8) == 0 and size(3, 64, 129) == 0


def test_logprobs_refusals(q):
    INV, UNS, WS = q.QMM_ERR_INVALID, q.QMM_ERR_UNSUPPORTED, q.QMM_ERR_WORKSPACE

    def f(x=FAKE, xt=0, T=3, V=100, ld=100, tokens=FAKE, ldt=1, n=1, top=5, scale=1.0, lp=FAKE, ent=FAKE, ids=FAKE, tl=FAKE,
          ws=FAKE, nbytes=1 << 30):
        return q.lib.token_logprobs(x, xt, T, V, ld, tokens, ldt, n, top, scale, lp, ent, ids, tl, ws, nbytes, None)
    for name in ("x", "tokens", "lp", "ids", "tl"):
        assert f(**{name: None}) == INV, name
    assert f(T=-1) == INV and f(V=0) == INV and f(ld=99) == INV and f(n=-1) == INV and f(top=-1) == INV and f(n=2) == INV
    for scale in (0.0, -1.0, float("nan"), float("inf"), 3e38):
        assert f(scale=scale) == INV
    assert f(xt=3) == INV and f(x=FAKE + 2) == INV and f(tokens=FAKE + 4) == INV and f(ids=FAKE + 4) == INV and f(lp=FAKE + 2) == INV
    assert f(top=33) == UNS and f(V=1 << 29, ld=1 << 29) == UNS and f(T=1 << 24, V=4096, ld=4096) == UNS
    assert f(ws=None) == WS and f(ws=FAKE + 8) == WS and f(nbytes=100) == WS
    assert f(T=0) == q.QMM_OK
    size = q.lib.qmm_token_logprobs_workspace_bytes
    assert size(0, 5) == 0 and size(5, 0) == 0 and size(1, 1 << 29) == 0 and size(1, 100) > 0


def test_binding_refusals(q):
    """What the binding refuses before it looks for a GPU."""
    u8, i32, bf = torch.uint8, torch.int32, torch.bfloat16
    kc, ks = torch.zeros(2, 4, 2, 32, dtype=u8), torch.zeros(2, 4, 2, 2, dtype=bf)
    x, slots = torch.zeros(3, 2, 64), torch.zeros(3, dtype=torch.int64)
    odd = torch.zeros(2, 4, 2, 3, dtype=bf)[..., :2]
    for args in [(kc, kc), (kc, kc, ks, ks.float()), (kc, kc, ks[..., :1], ks[..., :1]), (kc, kc, ks[:1], ks[:1]),
                 (kc, kc, odd, odd), (kc, kc, ks, None), (kc.to(bf), kc.to(bf), ks, ks), (kc, kc, ks, ks)]:
        with pytest.raises(ValueError):
            q.kv_append(x, x, slots, *args)                # the last: CPU tensors
        with pytest.raises(ValueError):
            q.kv_gather(slots, *args)
    with pytest.raises(ValueError):
        q.kv_append(x[..., :32], x[..., :32], slots, kc, kc, ks, ks)
    with pytest.raises(ValueError, match="dtype"):
        q.kv_gather(slots, kc, kc, ks, ks, dtype=torch.int8)
    with pytest.raises(ValueError):
        q.kv_gather(slots.int(), kc, kc, ks, ks)
    Q, table, n, cu = torch.zeros(3, 4, 64, dtype=bf), torch.zeros(2, 3, dtype=i32), torch.zeros(2, dtype=i32), torch.zeros(3, dtype=i32)
    ok = [Q, kc, kc, table, n, cu]
    for i, bad in [(0, Q[..., :32]), (0, Q.to(torch.int8)), (3, table[:1]), (4, n.long()), (5, cu[:2])]:
        args = list(ok)
        args[i] = bad
        with pytest.raises(ValueError):
            q.window_attention(*args, 8, 1, k_scale=ks, v_scale=ks)
    for kw in (dict(window=8), dict(window=8, sinks=1)):
        with pytest.raises(ValueError, match="device"):
            q.window_attention(*ok, **kw, k_scale=ks, v_scale=ks)
    with pytest.raises((ValueError, TypeError)):
        q.window_attention(*ok, 8.5, k_scale=ks, v_scale=ks)
    A, B, X, ids = torch.zeros(2, 8, 64, dtype=bf), torch.zeros(2, 32, 8, dtype=bf), torch.zeros(3, 64, dtype=bf), torch.zeros(3, dtype=i32)
    base = torch.zeros(3, 32, dtype=bf)
    for args in [(X[:, :32], A, B, ids), (X.int(), A, B, ids), (X, A[:1], B, ids), (X, A, B.half(), ids), (X, A, B[..., :4], ids),
                 (X, A, B, ids.long()), (X, A, B, ids[:2]), (X, A, B, ids, base[:2]), (X, A, B, ids, base.float()),
                 (X, A, B, ids, base, torch.zeros(3)), (X, A, B, ids, base, torch.zeros(2, dtype=bf)), (X, A.int(), B.int(), ids),
                 (X, A.transpose(1, 2).contiguous().transpose(1, 2), B, ids), (X, A, B, ids, base)]:
        with pytest.raises(ValueError):
            q.lora_matmul(*args)
    z, t = torch.zeros(3, 50), torch.zeros(3, dtype=torch.int64)
    for args in [(z.int(), t), (z[0], t), (z.t().contiguous().t(), t), (z, t.int()), (z, t[:2]), (z, t[None]), (z, t, -1), (z, t, 2)]:
        with pytest.raises(ValueError):
            q.token_logprobs(*args)
    for call in (lambda ws: q.lora_matmul(X, A, B, ids, ws=ws), lambda ws: q.token_logprobs(z, t, ws=ws),
                 lambda ws: q.window_attention(*ok, 8, k_scale=ks, v_scale=ks, ws=ws)):
        with pytest.raises(ValueError, match="ws must be contiguous"):
            call(torch.zeros(1 << 12, dtype=u8)[::2])
