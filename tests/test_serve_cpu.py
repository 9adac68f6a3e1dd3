"""CPU checks of the drafted-token verification operators: the plain 64-bit
forms against independent statements of the same thing, and every refusal of
the C ABI and the binding (each fails before any HIP call)."""
import ctypes

import numpy as np
import pytest
import torch

import serve_ref as ref

FAKE = 4096  # never dereferenced: each call below fails validation first


@pytest.fixture(scope="module")
def q():
    import int8_bit_weight_amd as q
    return q


# ------------------------------------------------------------ plain forms ---

def test_plain_group_product_is_the_dequantised_product():
    g = np.random.default_rng(1)
    K, N, group = 70, 5, 32
    q = g.integers(0, 16, (N, K))
    pad = np.concatenate([q, np.zeros((N, 0), int)], 1)
    codes = (pad[:, 0::2] | (pad[:, 1::2] << 4)).astype(np.uint8)
    s, z = g.random((N, 3)), g.integers(0, 16, (N, 3)).astype(np.uint8)
    X = g.standard_normal((3, K))
    want = np.zeros((3, N))
    for m in range(3):
        for n in range(N):
            want[m, n] = sum(X[m, k] * (int(q[n, k]) - int(z[n, k // group])) * s[n, k // group] for k in range(K))
    got, bound = ref.q4_group_matmul(X, codes, s, z, K, group)
    assert np.abs(got - want).max() < 1e-12 and (np.abs(want) <= bound).all()


def test_plain_plan_gives_every_token_a_row_of_its_own():
    g = np.random.default_rng(2)
    for page in (1, 4, 16):
        ctx, new = g.integers(0, 40, 9), g.integers(0, 30, 9)
        width = int(max(-(-(c + n) // page) for c, n in zip(ctx, new)))
        have = [-(-int(c) // page) for c in ctx]
        order = g.permutation(1000)
        table = np.full((9, width), -1, np.int32)
        at = 0
        for r in range(9):
            table[r, :have[r]] = order[at:at + have[r]]
            at += have[r]
        T = int(new.sum())
        out, cu, slots, pos, info = ref.kv_plan(ctx, new, table, order[at:], page, T)
        assert info[2] == 0 and info[1] == T and len(set(slots.tolist())) == T
        for r in range(9):
            row = [int(out[r, p // page]) * page + p % page for p in range(int(ctx[r] + new[r]))]
            assert len(set(row)) == len(row)
            assert row[int(ctx[r]):] == slots[cu[r]:cu[r + 1]].tolist()
        assert info[0] == sum(-(-int(c + n) // page) - h for c, n, h in zip(ctx, new, have))


def test_plain_attention_is_the_softmax():
    g = np.random.default_rng(3)
    qv, k, v = g.standard_normal(16), g.standard_normal((20, 16)), g.standard_normal((20, 16))
    sees = g.random(20) < 0.5
    s = torch.from_numpy(k @ qv * 0.25).masked_fill(~torch.from_numpy(sees), -float("inf"))
    want = torch.softmax(s, 0).numpy() @ v
    k[~sees], v[~sees] = np.nan, np.inf
    assert np.abs(ref.tree_attention(qv, k, v, sees, 0.25)[0] - want).max() < 1e-14
    assert not ref.tree_attention(qv, k, v, np.zeros(20, bool), 0.25)[0].any()


def test_plain_row_quantiser_is_the_library_rule(orc):
    x = np.random.default_rng(4).standard_normal((7, 64)).astype(np.float32)
    x[3] = 0
    c, s = ref.quantize_rows(x)
    oc, os_ = orc.quantize_rows_int8(x)
    assert np.array_equal(c, oc) and np.array_equal(s, os_)


# --------------------------------------------------------------- refusals ---

def test_group_sizes(q):
    f = q.lib.qmm_q4_group_packed_bytes
    assert f(128, 16, 128) == 1024 + 64
    assert f(128, 16, 32) == 1024 + 256
    assert f(129, 17, 128) == 4 * (1024 + 64)
    assert f(300, 16, 4096) == 3 * 1024 + 64
    assert f(0, 16, 128) == 0 and f(128, 0, 128) == 0
    for group in (0, -1, 16, 48, 96, 160):
        assert f(128, 16, group) == 0


def test_group_repack_refusals(q):
    INV, UNS, WS = q.QMM_ERR_INVALID, q.QMM_ERR_UNSUPPORTED, q.QMM_ERR_WORKSPACE

    def f(codes=FAKE, ldc=64, scales=FAKE, st=1, lds=1, zeros=None, ldz=0, K=128, N=16, group=128, packed=FAKE,
          nbytes=1 << 20):
        return q.lib.q4_group_repack(codes, ldc, scales, st, lds, zeros, ldz, K, N, group, packed, nbytes, None)
    assert f(codes=None) == INV and f(scales=None) == INV and f(packed=None) == INV
    assert f(K=0) == INV and f(N=0) == INV and f(group=0) == INV
    assert f(ldc=63) == INV and f(lds=0) == INV and f(zeros=FAKE, ldz=0) == INV
    assert f(st=0) == INV and f(st=3) == INV          # scales are fp16 or bf16
    assert f(packed=FAKE + 64) == INV and f(scales=FAKE + 1) == INV
    assert f(group=96, lds=2) == UNS
    assert f(nbytes=1000) == WS


def test_group_matmul_refusals(q):
    INV, UNS = q.QMM_ERR_INVALID, q.QMM_ERR_UNSUPPORTED

    def f(X=FAKE, xt=2, M=1, K=128, ldx=128, W=FAKE, N=16, group=128, Y=FAKE, ldy=16):
        return q.lib.q4_group_matmul(X, xt, M, K, ldx, W, N, group, Y, ldy, None, 0, None)
    assert f(X=None) == INV and f(W=None) == INV and f(Y=None) == INV
    assert f(xt=3) == INV and f(M=-1) == INV and f(K=0) == INV and f(N=-1) == INV
    assert f(ldx=127) == INV and f(ldy=15) == INV
    assert f(W=FAKE + 16) == INV and f(X=FAKE + 1) == INV and f(xt=0, Y=FAKE + 2) == INV
    assert f(group=48) == UNS and f(M=1 << 21) == UNS and f(M=16 * 65520 + 1) == UNS
    assert f(M=17) == q.QMM_ERR_WORKSPACE and f(xt=0) == q.QMM_ERR_WORKSPACE and f(ldx=131, M=2) == q.QMM_ERR_WORKSPACE
    assert f(M=0) == q.QMM_OK and f(N=0) == q.QMM_OK


def test_plan_refusals(q):
    INV, UNS = q.QMM_ERR_INVALID, q.QMM_ERR_UNSUPPORTED

    def f(ctx=FAKE, new=FAKE, R=4, table=FAKE, ld=8, width=8, page=16, free=FAKE, nf=9, begin=None, T=10, cu=FAKE,
          slots=FAKE, pos=FAKE, info=2 * FAKE):
        return q.lib.kv_plan(ctx, new, R, table, ld, width, page, free, nf, begin, T, cu, slots, pos, info, None)
    for name in ("ctx", "new", "table", "free", "cu", "slots", "pos", "info"):
        assert f(**{name: None}) == INV, name
    assert f(R=-1) == INV and f(ld=7) == INV and f(page=0) == INV and f(nf=-1) == INV and f(T=-1) == INV
    assert f(ctx=FAKE + 2) == INV and f(slots=FAKE + 4) == INV
    assert f(begin=2 * FAKE + 8) == INV                # this call's own info
    assert f(R=8193) == UNS
    assert f(width=1 << 20, ld=1 << 20, page=1 << 12) == UNS


def _cache(q, **kw):
    d = dict(k=FAKE, v=FAKE, type=2, num_pages=4, page_size=16, n_heads=2, head_dim=64, page_stride=2048,
             token_stride=128, head_stride=64, k_scale=None, v_scale=None, scale_page_stride=0, scale_token_stride=0,
             scale_head_stride=0)
    d.update(kw)
    return q.qmm_kv_cache(**d)


BAD_CACHES = [(dict(k=None), 1), (dict(v=None), 1), (dict(type=0), 1), (dict(type=4), 1), (dict(num_pages=0), 1),
              (dict(page_size=0), 1), (dict(n_heads=0), 1), (dict(head_dim=0), 1), (dict(page_stride=-8), 1),
              (dict(page_stride=1 << 62), 1), (dict(type=3), 1), (dict(head_dim=264), 2), (dict(head_dim=60), 2),
              (dict(page_size=1 << 20), 2), (dict(token_stride=132), 2), (dict(k=FAKE + 8), 2)]


def test_append_refusals(q):
    INV, UNS = q.QMM_ERR_INVALID, q.QMM_ERR_UNSUPPORTED

    def f(K=FAKE, V=FAKE, xt=2, T=3, slots=FAKE, c=None, ks=128, **kw):
        c = _cache(q, **kw) if c is None else c
        return q.lib.kv_append(K, ks, 64, V, 128, 64, xt, T, slots, c, None)
    assert f(K=None) == INV and f(V=None) == INV and f(slots=None) == INV and f(slots=FAKE + 4) == INV
    assert f(xt=3) == INV and f(T=-1) == INV and f(ks=-1) == INV and f(K=FAKE + 1) == INV
    assert q.lib.kv_append(FAKE, 128, 64, FAKE, 128, 64, 2, 3, FAKE, None, None) == INV
    for kw, want in BAD_CACHES:
        assert f(**kw) == want, kw
    assert f(T=1 << 31) == UNS
    assert f(T=0) == q.QMM_OK


def test_attention_refusals(q):
    INV, UNS = q.QMM_ERR_INVALID, q.QMM_ERR_UNSUPPORTED

    def f(Q=FAKE, qs=256, xt=2, T=3, Hq=4, table=FAKE, ld=8, width=8, ctx=FAKE, cu=FAKE, R=2, mask=None, ldm=0, cols=0,
          scale=1.0, O=FAKE, **kw):
        return q.lib.tree_attention(Q, qs, 64, xt, T, Hq, _cache(q, **kw), table, ld, width, ctx, cu, R, mask, ldm,
                                    cols, scale, O, 256, 64, None, 0, None)
    for name in ("Q", "table", "ctx", "cu", "O"):
        assert f(**{name: None}) == INV, name
    assert f(T=-1) == INV and f(Hq=0) == INV and f(R=-1) == INV and f(ld=7) == INV and f(qs=-1) == INV
    assert f(Hq=3) == INV                              # not a multiple of the cache's heads
    assert f(mask=FAKE, ldm=3, cols=4) == INV and f(mask=FAKE, cols=-1) == INV
    assert f(scale=float("nan")) == INV and f(scale=float("inf")) == INV
    assert f(xt=3) == INV and f(Q=FAKE + 1) == INV
    for kw, want in BAD_CACHES:
        assert f(**kw) == want, kw
    assert f(xt=0) == UNS and f(xt=1) == UNS           # fp32 rows; fp16 rows over a bf16 cache
    s8 = dict(type=3, k_scale=FAKE, v_scale=FAKE)
    assert f(xt=1, **s8) == UNS
    assert f(width=1 << 30, ld=1 << 30) == UNS
    assert f(T=1 << 29, qs=0) == UNS                   # rows of a cache head: T * (Hq / n_heads)
    assert f() == q.QMM_ERR_WORKSPACE
    assert f(T=0) == q.QMM_OK and f(R=0) == q.QMM_OK


def test_attention_workspace(q):
    f = q.lib.qmm_tree_attention_workspace_bytes
    assert f(0, 4, 2, 2, 64) == 0 and f(3, 4, 0, 2, 64) == 0 and f(3, 3, 1, 2, 64) == 0 and f(3, 4, 1, 2, 264) == 0
    # 512 headers of 56 bytes, two slots a workgroup of (m, l, sums) per row, up to 64 or 128 rows
    assert f(1, 2, 1, 1, 128) == 512 * 56 + 512 * 2 * 2 * 130 * 4
    assert f(1000, 8, 1, 1, 128) == 512 * 56 + 512 * 2 * 128 * 130 * 4
    assert f(1000, 8, 1, 1, 256) == 512 * 56 + 512 * 2 * 64 * 258 * 4


def test_binding_refusals(q):
    """What the binding refuses before it looks for a GPU."""
    u8, i32 = torch.uint8, torch.int32
    codes, scales = torch.zeros(4, 16, dtype=u8), torch.zeros(4, 1, dtype=torch.float16)
    good = dict(K=32, group=32)
    for args, kw in [((codes.int(), scales), good), ((codes, scales.float()), good), ((codes, scales), dict(K=34, group=32)),
                     ((codes, scales, torch.zeros(4, 2, dtype=u8)), good), ((codes, scales), dict(K=32, group=0)),
                     ((codes, scales), good)]:  # the last: CPU tensors
        with pytest.raises(ValueError):
            q.q4_group_repack(*args, **kw)
    with pytest.raises(q.QmmError) as e:               # a group the library does not have, wherever the tensors are
        q.q4_group_repack(codes, scales, K=32, group=48)
    assert e.value.status == q.QMM_ERR_UNSUPPORTED
    W = q.PackedQ4Group(torch.zeros(64, dtype=u8), 32, 4, 32)
    for X in (torch.zeros(1, 31), torch.zeros(32), torch.zeros(1, 32, dtype=torch.float64), torch.zeros(1, 64)[:, ::2],
              torch.zeros(1, 32)):
        with pytest.raises(ValueError):
            q.q4_group_matmul(X, W)
    n, t, f = torch.zeros(2, dtype=i32), torch.zeros(2, 3, dtype=i32), torch.zeros(4, dtype=i32)
    for args in [(n.long(), n, t, f), (n, n[:1], t, f), (n, n, t[:1], f), (n, n, t.long(), f), (n, n, t, f.long()),
                 (n, n, t.t().contiguous().t(), f), (n, n, t, f)]:
        with pytest.raises(ValueError):
            q.kv_plan(*args, 16, 4)
    kc = torch.zeros(2, 4, 2, 64, dtype=torch.bfloat16)
    x, slots = torch.zeros(3, 2, 64), torch.zeros(3, dtype=torch.int64)
    for args in [(x, x, slots, kc.float(), kc.float()), (x, x, slots, kc, kc[:1]), (x, x, slots.int(), kc, kc),
                 (x[:, :1], x[:, :1], slots, kc, kc), (x, x.half(), slots, kc, kc), (x, x, slots, kc.to(torch.int8), kc.to(torch.int8)),
                 (x, x, slots, kc, kc.transpose(1, 2).contiguous().transpose(1, 2)), (x, x, slots, kc, kc)]:
        with pytest.raises(ValueError):
            q.kv_append(*args)
    Q, cu = torch.zeros(3, 4, 64, dtype=torch.bfloat16), torch.zeros(3, dtype=i32)
    ok = [Q, kc, kc, t, n, cu]
    for i, bad in [(0, Q[..., :32]), (0, Q.to(torch.int8)), (3, t[:1]), (4, n.long()), (5, cu[:2]), (1, kc[..., :32])]:
        args = list(ok)
        args[i] = bad
        with pytest.raises(ValueError):
            q.tree_attention(*args)
    for mask in (torch.zeros(2, 4, dtype=torch.bool), torch.zeros(3, 4), torch.zeros(4, 3, dtype=u8).t()):
        with pytest.raises(ValueError):
            q.tree_attention(*ok, mask)
    with pytest.raises(ValueError):
        q.tree_attention(*ok)                          # CPU tensors


def test_binding_refuses_a_weight_that_is_too_small(q):
    """The C call takes K, N and group on trust: a packed buffer that cannot hold them would be read past its end."""
    nbytes = q.lib.qmm_q4_group_packed_bytes(300, 40, 64)
    X = torch.zeros(2, 300)
    for data in (torch.zeros(nbytes - 1, dtype=torch.uint8), torch.zeros(nbytes // 4, dtype=torch.int32),
                 torch.zeros(2 * nbytes, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="packed weight"):
            q.q4_group_matmul(X, q.PackedQ4Group(data, 300, 40, 64))
    whole = torch.zeros(nbytes, dtype=torch.uint8)
    for W in (q.PackedQ4Group(whole, 300, 57, 64), q.PackedQ4Group(whole, 300, 40, 32)):
        with pytest.raises(ValueError, match="packed weight"):
            q.q4_group_matmul(X, W)
    with pytest.raises(ValueError, match="device"):    # a whole one is refused for lying on the CPU only
        q.q4_group_matmul(X, q.PackedQ4Group(whole, 300, 40, 64))


def test_binding_refuses_a_workspace_with_gaps(q):
    """Its size is taken as bytes that follow one another."""
    gaps = torch.zeros(1 << 12, dtype=torch.uint8)[::2]
    W = q.PackedQ4Group(torch.zeros(q.lib.qmm_q4_group_packed_bytes(32, 4, 32), dtype=torch.uint8), 32, 4, 32)
    with pytest.raises(ValueError, match="ws must be contiguous"):
        q.q4_group_matmul(torch.zeros(1, 32), W, ws=gaps)
    kc = torch.zeros(2, 4, 2, 64, dtype=torch.bfloat16)
    n = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="ws must be contiguous"):
        q.tree_attention(torch.zeros(3, 4, 64, dtype=torch.bfloat16), kc, kc, torch.zeros(2, 3, dtype=torch.int32), n,
                         torch.zeros(3, dtype=torch.int32), ws=gaps)


def test_attention_refuses_lengths_whose_last_step_wraps(q):
    """Keys are counted in 32 bits, 64 at a time: tables of more than 2^31 - 64 of them would make a loop that never
    ends.  Pages of 899658 tokens (a little below 2^20): 2387 of them are 2^31 - 2."""
    def f(width, page):
        return q.lib.tree_attention(FAKE, 256, 64, 2, 3, 4, _cache(q, page_size=page), FAKE, width, width, FAKE, FAKE, 2, None,
                                    0, 0, 1.0, FAKE, 256, 64, None, 0, None)
    assert 899658 * 2387 == 2 ** 31 - 2
    assert f(2387, 899658) == q.QMM_ERR_UNSUPPORTED
    assert f((1 << 31) - 63, 1) == q.QMM_ERR_UNSUPPORTED
    assert f((1 << 31) - 64, 1) == q.QMM_ERR_WORKSPACE
    assert f(2386, 899658) == q.QMM_ERR_WORKSPACE


def test_other_calls_do_without_the_native_binding(tmp_path):
    """A package with the library alone imports and checks arguments as before; the calls that go through the binding
    say what is missing."""
    import os
    import shutil
    import subprocess
    import sys
    import int8_bit_weight_amd as q
    here = os.path.dirname(os.path.abspath(q.__file__))
    package = tmp_path / "int8_bit_weight_amd"
    package.mkdir()
    shutil.copy(os.path.join(here, "__init__.py"), package)
    os.symlink(os.path.join(here, "libqmm.so"), package / "libqmm.so")
    code = """
import torch, int8_bit_weight_amd as q
assert q.__file__.startswith(%r), q.__file__
assert q.lib.qmm_pack_b_int8_bytes(1024, 1024) == 64 + 1024 * 1024 + 8 * 1024
assert q.lib.q4_1_matmul(None, 1, 32, 32, None, 16, None, 16, None, 0, None) == q.QMM_ERR_INVALID
try:
    q.q4_group_repack(torch.zeros(4, 16, dtype=torch.uint8), torch.zeros(4, 1).half(), K=32, group=48)
except q.QmmError as e:
    assert e.status == q.QMM_ERR_UNSUPPORTED
n = torch.zeros(2, dtype=torch.int32)
for call in (lambda: q.q4_group_matmul(torch.zeros(1, 32), q.PackedQ4Group(n, 32, 4, 32)),
             lambda: q.kv_plan(n, n, n.view(2, 1), n, 16, 4), lambda: q.kv_append(n, n, n, n, n),
             lambda: q.tree_attention(n, n, n, n, n, n)):
    try:
        call()
    except ImportError as e:
        assert "build.py" in str(e)
    else:
        raise AssertionError("no binding was missed")
""" % str(tmp_path)
    r = subprocess.run([sys.executable, "-c", code], cwd=tmp_path, capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, PYTHONPATH=str(tmp_path)))
    assert r.returncode == 0, r.stderr


def test_attention_refuses_an_output_over_its_queries(q):
    """Rows whose sums are not finite are computed again from Q after O has been written, so O must lie beside Q.
    Slices of one tensor do.  Sizes in elements of two bytes: 3 tokens of 4 heads of 64."""
    def f(o, qs=256, qh=64, os=256, oh=64, T=3, Hq=4):
        return q.lib.tree_attention(FAKE, qs, qh, 2, T, Hq, _cache(q), FAKE, 8, 8, FAKE, FAKE, 2, None, 0, 0, 1.0,
                                    FAKE + 2 * o, os, oh, FAKE, 0, None)
    inside, beside = q.QMM_ERR_INVALID, q.QMM_ERR_WORKSPACE
    assert f(0) == inside and f(64) == inside and f(3 * 256 - 1) == inside and f(-3 * 256 + 1) == inside
    assert f(3 * 256) == beside and f(-3 * 256) == beside
    # heads 0..3 and 8..11, or 4..7, of tokens of 12 heads; heads 3..6 overlap
    assert f(8 * 64, qs=768, os=768) == beside and f(4 * 64, qs=768, os=768) == beside
    assert f(3 * 64, qs=768, os=768) == inside and f(-4 * 64, qs=768, os=768) == beside
    # the last heads of a token and the first of the next one
    assert f(9 * 64, qs=768, os=768) == inside
    # every second head; head-major rows of one tensor
    assert f(64, qs=1024, qh=128, os=1024, oh=128) == beside and f(63, qs=1024, qh=128, os=1024, oh=128) == inside
    assert f(3 * 64, qs=64, qh=6 * 64, os=64, oh=6 * 64) == beside and f(64, qs=64, qh=6 * 64, os=64, oh=6 * 64) == inside
    # one token or one head: its stride means nothing
    assert f(256, qs=0, os=0, T=1) == beside and f(128, qs=0, os=0, T=1) == inside
    # an output of other strides in between is not told apart
    assert f(4 * 64, qs=768, os=512) == inside


def test_group_matmul_refuses_an_output_over_its_activations(q):
    """Workgroups read all rows of X while others write their columns of Y.  Columns of one matrix are told apart."""
    def f(y, xt=0, M=2, ldx=300, ldy=300, ws=FAKE):
        return q.lib.q4_group_matmul(FAKE, xt, M, 100, ldx, FAKE, 80, 128, FAKE + 4 * y, ldy, ws, 0, None)
    inside, beside = q.QMM_ERR_INVALID, q.QMM_ERR_WORKSPACE
    assert f(0) == inside and f(99) == inside and f(100) == beside and f(220) == beside and f(221) == inside
    assert f(-80) == beside and f(-79) == inside and f(-380) == beside and f(400) == beside and f(399) == inside
    assert f(100, M=1, ldx=100, ldy=80) == beside and f(99, M=1, ldx=100, ldy=80) == inside
    # 16-bit rows of the call that needs no workspace
    assert f(0, xt=2, M=1, ws=None) == inside


def test_sizes_past_one_grid_are_refused(q):
    """A grid has fewer than 2^32 threads: 64 of the repack to a record of 128 k x 16 columns, 512 of the product of few
    rows to 16 columns, head_dim / 8 of the append to a row."""
    UNS, WS, INV = q.QMM_ERR_UNSUPPORTED, q.QMM_ERR_WORKSPACE, q.QMM_ERR_INVALID

    def repack(K, N):
        return q.lib.q4_group_repack(FAKE, K, FAKE, 1, K, None, 0, K, N, 128, FAKE, 0, None)

    def product(K, N):
        return q.lib.q4_group_matmul(FAKE, 0, 1, K, K, FAKE, N, 128, 1 << 40, N, None, 0, None)
    for K, N, fits in ((1 << 17, 1 << 20, False), (1 << 17, (1 << 20) - 16, True), (128, 1 << 27, False),
                       (128, (1 << 27) - 16, True)):
        assert repack(K, N) == (WS if fits else UNS), (K, N)
        assert product(K, N) == (WS if fits else UNS), (K, N)
        assert (q.lib.qmm_q4_group_packed_bytes(K, N, 128) > 0) == fits
        assert (q.lib.qmm_q4_group_matmul_workspace_bytes(1, K, N, 128, q.QMM_T_F32) > 0) == fits

    def append(T, H, D):                               # without K and V: INVALID where the sizes are taken
        c = _cache(q, n_heads=H, head_dim=D)
        return q.lib.kv_append(None, 128, 64, None, 128, 64, 2, T, FAKE, c, None)
    assert append(1 << 26, 2, 256) == UNS and append((1 << 26) - 16, 2, 256) == INV
    assert append(1 << 29, 1, 64) == UNS and append((1 << 29) - 64, 1, 64) == INV
    assert append(1 << 30, 1 << 30, 8) == UNS
