"""The cache operators on the GPU against plain 64-bit references: batch plan,
query/key norm with rotation, append, read and attention over the 4-bit cache,
each at the sizes and masks where it can go wrong, and a run of them together
between two 4-bit layers.  Integers and cache bytes are exact; the tolerances of
the others are derived in kv_ref.py."""
import numpy as np
import pytest
import torch

import kv_ref as R
from gpu_common import require_gpu, svdq

pytestmark = pytest.mark.gpu

FMTS = ["nvfp4", "fp4g32", "int4"]


@pytest.fixture(scope="module")
def S():
    require_gpu()
    mod = svdq()
    mod.svdq_get_error()
    return mod


def dev(a, dtype=None):
    return torch.as_tensor(np.ascontiguousarray(a), device="cuda") if dtype is None else \
        torch.as_tensor(np.ascontiguousarray(a), device="cuda").to(dtype)


def within(got, want, tol):
    got = got.double().cpu().numpy()
    same = np.isfinite(want)
    assert np.array_equal(np.isfinite(got), same)
    err = np.abs(np.where(same, got, 0) - np.where(same, want, 0)) / np.where(same, tol, 1)
    assert err.size == 0 or err.max() <= 1, f"error / tolerance = {err.max():.3g} at {np.unravel_index(err.argmax(), err.shape)}"


def cache_of(S, b):
    return S.KVCache(b.fmt, b.hk, b.D, b.page, dev(b.pool))


def attend(S, b, scale=None, causal=True, window=0, **more):
    scale = b.D ** -0.5 if scale is None else scale
    out, lse = S.svdq_kv_attention(cache_of(S, b), more.pop("q", b.q.cuda()), dev(b.cu), dev([kv for _, kv in b.lens], torch.int32),
                                   dev(b.table), scale=scale, causal=causal, window=window, return_lse=True, **more)
    torch.cuda.synchronize()
    assert S.svdq_get_error() == 0
    live = b.cu[-1]
    o, l, to, tl = b.expected(scale, causal, window)
    within(out[:live], o, to)
    within(lse[:live], l, tl)
    return out, lse


# --------------------------------------------------------------------- plan ---
@pytest.mark.parametrize("seed,batch,q,kv,page,pad", [
    (0, 1, 1, 0, 16, 0), (1, 1, 1, 63, 64, 0), (2, 7, 3, 40, 16, 5), (3, 64, 1, 4000, 64, 0), (4, 33, 200, 100, 32, 1),
    (5, 513, 5, 300, 128, 77), (6, 2000, 2, 30, 16, 0), (9, 16384, 3, 40, 32, 300), (7, 3, 3000, 5000, 256, 2000), (8, 4, 0, 90, 16, 9)])
def test_plan(S, seed, batch, q, kv, page, pad):
    rng = np.random.default_rng(seed)
    ql, kl = rng.integers(0, q + 1, batch), rng.integers(0, kv + 1, batch)
    if q == 1:
        ql[:] = 1
    held, need = -(-kl // page), -(-(kl + ql) // page)
    ids = rng.permutation(need.sum() + 4).astype(np.int32)
    table = np.full((batch, need.max() + 2), -7, np.int32)
    at = 0
    for b in range(batch):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    free, rows = ids[at:], int(ql.sum()) + pad
    want = R.plan(ql, kl, table, free, rows, page)
    assert not want[6]
    wide = torch.full((batch, table.shape[1] + 3), 99, dtype=torch.int32, device="cuda")   # a view of a wider table
    t = wide[:, :table.shape[1]]
    t.copy_(dev(table))
    for _ in range(2):                  # the same inputs again: the same results
        got = S.svdq_kv_plan(dev(ql, torch.int32), dev(kl, torch.int32), t, dev(free), rows, page)
        for g, w in zip(got, want[:5]):
            assert np.array_equal(g.cpu().numpy().reshape(-1), np.asarray(w).reshape(-1))
        assert np.array_equal(t.cpu().numpy(), want[5])
        assert (wide[:, table.shape[1]:] == 99).all()
    assert S.svdq_get_error() == 0


@pytest.mark.parametrize("what", ["few_rows", "few_pages", "narrow", "negative", "long", "no_requests", "no_free"])
def test_plan_out_of_range(S, what):
    ql, kl, page, rows, width, nfree = [5, 20, 0, 30], [3, 16, 9, 0], 16, 55, 4, 8
    if what == "few_rows":
        rows = 17
    elif what == "few_pages":
        nfree = 2
    elif what == "narrow":
        width = 1
    elif what == "negative":
        ql[1], kl[2] = -3, -1
    elif what == "long":
        kl[1] = 2 ** 31 - 5
    elif what == "no_free":
        nfree = 0
    table = np.full((4, width), -1, np.int32)
    table[0, 0], table[1, 0], table[2, 0] = 40, 41, 42
    free = np.arange(nfree, dtype=np.int32) + 7
    if what == "no_requests":
        ql, kl, table = [], [], np.zeros((0, width), np.int32)
    want = R.plan(ql, kl, table, free, rows, page)
    t = dev(table)
    got = S.svdq_kv_plan(dev(ql, torch.int32), dev(kl, torch.int32), t, dev(free), rows, page)
    for g, w in zip(got, want[:5]):
        assert np.array_equal(g.cpu().numpy().reshape(-1), np.asarray(w).reshape(-1)), what
    assert np.array_equal(t.cpu().numpy(), want[5])
    assert S.svdq_get_error() == (8 if want[6] else 0)
    assert bool(want[6]) == (what not in ("no_requests",))


# ---------------------------------------------------------------- norm, rope ---
@pytest.mark.parametrize("rows,hq,hk,D,rot,inter,norm,weights", [
    (1, 8, 2, 128, 128, False, True, True), (37, 6, 6, 128, 128, True, True, True), (130, 5, 1, 64, 32, False, True, True),
    (9, 3, 3, 96, 96, False, True, True), (11, 2, 1, 256, 256, True, True, False), (300, 32, 8, 128, 64, False, True, True),
    (17, 1, 1, 16, 16, False, True, True), (5, 4, 0, 80, 16, True, False, False), (6, 0, 4, 64, 64, False, False, False),
    (1000, 24, 24, 128, 128, True, True, True), (33, 7, 7, 192, 112, False, True, True), (4, 2, 2, 64, 0, False, True, True)])
def test_norm_rope(S, rows, hq, hk, D, rot, inter, norm, weights):
    g = torch.Generator().manual_seed(rows * 7 + D)
    qkv = torch.randn(rows, (hq + 2 * hk) * D + 8, generator=g).to(torch.bfloat16)
    table = R.rotation(4096, rot) if rot else None
    pos = torch.randint(0, 4096, (rows,), generator=g, dtype=torch.int32)
    w = [(1 + 0.3 * torch.randn(D, generator=g)).to(torch.bfloat16) if weights else None for _ in range(2)]
    d = qkv.cuda()
    q, k = d[:, :hq * D].unflatten(-1, (hq, D)), d[:, hq * D:(hq + hk) * D].unflatten(-1, (hk, D))
    up = lambda x: None if x is None else (dev(x) if isinstance(x, np.ndarray) else x.cuda())  # noqa: E731
    args = (up(table), pos.cuda() if rot else None, up(w[0]), up(w[1]))
    got = S.svdq_qk_norm_rope(q, k, *args, eps=1e-5, norm=norm, interleaved=inter)
    src = qkv.double().numpy()
    for y, lo, h, wt in ((got[0], 0, hq, w[0]), (got[1], hq * D, hk, w[1])):
        x = src[:, lo:lo + h * D].reshape(rows, h, D)
        want, tol = R.norm_rope(x, None if wt is None else wt.double().numpy(), table, pos.numpy(), 1e-5, norm, inter)
        within(y, want, tol)
    S.svdq_qk_norm_rope(q, k, *args, eps=1e-5, norm=norm, interleaved=inter, q_out=q, k_out=k)     # in place
    assert torch.equal(q, got[0]) and torch.equal(k, got[1])
    assert torch.equal(d[:, (hq + hk) * D:].cpu(), qkv[:, (hq + hk) * D:])                         # the rest stays
    assert S.svdq_get_error() == 0


def test_norm_rope_rows_left_alone_and_far_positions(S):
    D, rows = 128, 6
    x = torch.randn(rows, 2, D, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    x[2] = 0                                          # a row of zeros: the norm's eps
    x[3] *= 1e-20
    table = dev(R.rotation(64, D))
    pos = torch.tensor([5, -1, 63, 0, 64, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    out = torch.full_like(x, 7.0)
    S.svdq_qk_norm_rope(x, x[:, :1], table, pos, q_out=out, k_out=torch.empty_like(x[:, :1].contiguous()))
    assert (out[[1, 4, 5]] == 7).all() and (out[2] == 0).all() and torch.isfinite(out.float()).all()
    assert (out[[0, 3]] != 7).any()
    assert S.svdq_get_error() == 8
    S.svdq_qk_norm_rope(x, x[:, :1], table, pos.clamp(max=63), q_out=out)
    assert S.svdq_get_error() == 0


# -------------------------------------------------------------- append, read ---
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D,page,heads,rows", [(128, 16, 8, 1), (128, 64, 1, 33), (64, 32, 5, 130), (64, 256, 3, 7), (128, 128, 2, 600)])
def test_append_and_read(S, fmt, D, page, heads, rows):
    rng = np.random.default_rng(rows)
    g = torch.Generator().manual_seed(rows)
    pages = rows // page + 3
    pool = rng.integers(0, 256, (pages, heads, R.pieces(fmt, D, page)[3]), dtype=np.uint8)
    slots = rng.permutation(pages * page)[:rows].astype(np.int64)
    if rows > 5:
        slots[3], slots[5] = -1, -5
    qkv = torch.randn(rows, 3 * heads, D, generator=g)
    qkv[:, :, 5] *= 50
    qkv[rows // 2] = 0                                # a group of zeros: scale 0, codes 0
    qkv[-1] *= 2.0 ** -14                             # scales below the formats' smallest
    qkv[0, :, -1] = 3e4                               # scales above E4M3's largest
    qkv = qkv.to(torch.bfloat16)
    k, v = qkv[:, heads:2 * heads], qkv[:, 2 * heads:]
    want = pool.copy()
    kq, vq = R.store(want, fmt, D, page, slots, k, v)
    d = qkv.cuda()
    c = S.KVCache(fmt, heads, D, page, dev(pool))
    S.svdq_kv_append(c, d[:, heads:2 * heads], d[:, 2 * heads:], dev(slots))
    got = c.pool.cpu().numpy()
    if fmt != "int4":      # a code of magnitude 0 may carry a sign: compare those bytes as values
        assert np.array_equal(strip(got, fmt, D, page), strip(want, fmt, D, page))
    else:
        assert np.array_equal(got, want)
    for dtype in (torch.float32, torch.bfloat16):
        for y, w in zip(S.svdq_kv_read(c, dev(slots), dtype), (kq, vq)):
            w = np.where((slots >= 0)[:, None, None], w, 0)
            exact = torch.from_numpy(w).to(dtype) if fmt == "int4" else torch.from_numpy(w)
            assert torch.equal(y.double().cpu(), exact.double())
    assert S.svdq_get_error() == 0


def strip(pool, fmt, D, page):
    ks, vc, vs, _ = R.pieces(fmt, D, page)
    out = pool.copy()
    for a, b in ((0, ks), (vc, vs)):
        c = out[:, :, a:b]
        lo, hi = c & 15, c >> 4
        out[:, :, a:b] = np.where(lo == 8, 0, lo) | (np.where(hi == 8, 0, hi) << 4)
    return out


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("lens", [(3, 100), (100, 100)])
def test_append_of_what_is_not_finite(S, fmt, lens):
    """A token with infinities and NaN is held by finite values, and rows that mask it do not see it."""
    b = R.Batch(fmt, 128, 16, 4, 2, [lens], seed=14)
    c, n, kv = cache_of(S, b), *lens
    bad = torch.randn(1, 4, 128, generator=torch.Generator().manual_seed(1))
    bad[0, :, 7], bad[0, :, 40], bad[0, :, 90] = float("inf"), float("-inf"), float("nan")
    bad[0, 1] = float("nan")
    bad[0, 3] = float("inf")
    bad = bad.to(torch.bfloat16).cuda()
    slot = int(b.table[0, (kv - 1) // 16]) * 16 + (kv - 1) % 16
    S.svdq_kv_append(c, bad[:, :2], bad[:, 2:], dev([slot], torch.int64))
    k, v = S.svdq_kv_read(c, dev([slot], torch.int64), torch.float32)
    assert torch.isfinite(k).all() and torch.isfinite(v).all()
    most = 7 * 65504 if fmt == "int4" else 6 * 448
    assert (v[0, 1] == most).all() and (k[0, 1] == 0).all()
    assert (k[0, 0, 7], k[0, 0, 40], v[0, 0, 7], v[0, 0, 40]) == (most, -most, most, -most)
    b.keys[0][-1], b.values[0][-1] = k[0].double().cpu(), v[0].double().cpu()
    out, lse = S.svdq_kv_attention(c, b.q.cuda(), dev(b.cu), dev([kv], torch.int32), dev(b.table), return_lse=True)
    o, l, to, tl = b.expected(128 ** -0.5, True, 0)
    within(out[:n - 1], o[:n - 1], to[:n - 1])
    within(lse[:n - 1], l[:n - 1], tl[:n - 1])


def test_append_and_read_past_the_pool(S):
    c = S.KVCache("nvfp4", 2, 64, 16, torch.zeros(3, 2, 2 * 16 * 36, dtype=torch.uint8, device="cuda"))
    k = torch.ones(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    slots = torch.tensor([48, 5, 2 ** 40], device="cuda")
    S.svdq_kv_append(c, k, k, slots)
    assert S.svdq_get_error() == 8
    for y in S.svdq_kv_read(c, slots):      # ones: the scale 1 / 6 rounds to 11 / 64 in E4M3, so they read 6 * 11 / 64
        assert (y[1] == 66 / 64).all() and (y[[0, 2]] == 0).all()
    assert S.svdq_get_error() == 8
    S.svdq_kv_append(c, k[:0], k[:0], slots[:0])
    assert S.svdq_kv_read(c, slots[:0])[0].shape == (0, 2, 64)


# ---------------------------------------------------------------- attention ---
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D,page,hq,hk,lens", [
    (128, 16, 8, 1, [(1, 1)]), (128, 64, 4, 4, [(1, 63), (1, 64), (1, 65), (1, 0)]), (64, 32, 6, 2, [(1, 200), (3, 129), (0, 50), (2, 2)]),
    (128, 128, 32, 8, [(1, 700)]), (64, 16, 5, 5, [(17, 17), (1, 31), (40, 300)]), (128, 256, 16, 1, [(1, 257), (4, 511)]),
    (128, 32, 3, 1, [(130, 130)]), (64, 64, 24, 2, [(1, 1000)]), (128, 16, 20, 1, [(2, 90), (1, 17)])])
def test_attention(S, fmt, D, page, hq, hk, lens):
    attend(S, R.Batch(fmt, D, page, hq, hk, lens, seed=len(lens) + D))


@pytest.mark.parametrize("causal,window", [(False, 0), (True, 1), (True, 5), (True, 64), (False, 100), (True, 10 ** 6)])
@pytest.mark.parametrize("D,hq,hk,lens", [(128, 8, 2, [(1, 150), (9, 75)]), (64, 4, 2, [(300, 333), (129, 129)])])
def test_attention_masks(S, causal, window, D, hq, hk, lens):
    attend(S, R.Batch("nvfp4", D, 16, hq, hk, lens, seed=3), causal=causal, window=window)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D,page,causal,window,lens", [
    (128, 16, True, 70, [(1, 900), (2, 333)]), (64, 64, True, 1, [(1, 700), (1, 65)]), (128, 128, False, 33, [(4, 1000)]),
    (64, 32, True, 200, [(1, 3000)]), (128, 16, True, 40, [(150, 900), (100, 333)]), (64, 64, True, 1, [(300, 700)]),
    (128, 256, False, 33, [(70, 1000)])])
def test_attention_in_front_of_the_window(S, fmt, D, page, causal, window, lens):
    """Pages that lie in front of every query's window may be gone (-1) or hold anything, and so may the tokens
    in front of it in its first page: infinite and NaN scales there reach nothing, and no bit is set."""
    b = R.Batch(fmt, D, page, 8, 2, lens, seed=60)
    ks, vc, vs, end = R.pieces(fmt, D, page)
    gone = b.table.copy()
    spare = (set(range(b.pool.shape[0])) - set(b.table.reshape(-1).tolist())).pop()
    other = b.table.copy()
    for r, (n, kv) in enumerate(lens):
        low = max(0, kv - n - window + 1)             # the first query's first key
        gone[r, :low // page] = -1
        other[r, :low // page] = spare
        p, o = b.table[r, low // page], low % page
        for c0, s0, s1 in ((0, ks, vc), (vc, vs, end)):
            w = (s1 - s0) // page
            b.pool[p, :, c0:c0 + o * D // 2] = 0x5A
            b.pool[p, :, s0:s0 + o * w] = 0x7F if fmt != "int4" else np.tile(np.array([0x00, 0x7C], np.uint8), o * w // 2)
    for byte in (0x7F, 0x7C, 0xFF):                   # NaN; fp16 NaN and E4M3 384; NaN
        b.pool[spare] = byte
        for t in (gone, other):
            b.table = t
            attend(S, b, causal=causal, window=window)


@pytest.mark.parametrize("lens", [[(5, 3)], [(200, 70), (1, 0), (3, 0)], [(1, 0)], [(0, 0), (0, 9)]])
@pytest.mark.parametrize("causal", [True, False])
def test_attention_rows_without_keys(S, lens, causal):
    """More queries than keys: the first rows of a causal request see nothing."""
    b = R.Batch("int4", 64, 16, 4, 2, lens, seed=8)
    attend(S, b, causal=causal)
    attend(S, b, causal=causal, window=2)


@pytest.mark.parametrize("fmt", FMTS)
def test_attention_scores_far_apart(S, fmt):
    """Keys 30 times larger: weights from 1 down to nothing, and a maximum that keeps moving."""
    attend(S, R.Batch(fmt, 128, 32, 8, 2, [(1, 400), (70, 400)], seed=5, k_scale=30.0))
    attend(S, R.Batch(fmt, 64, 32, 8, 2, [(1, 400), (70, 400)], seed=6, k_scale=0.001), scale=-2.5)
    attend(S, R.Batch(fmt, 64, 32, 8, 2, [(2, 300)], seed=7), scale=0.0)


@pytest.mark.parametrize("D,lens", [(128, (200, 200)), (64, (130, 400)), (128, (2, 200))])
def test_attention_int4_small_keys_beside_large_ones(S, D, lens):
    """From key 100 on 2^17 times larger: a causal row before it sees only the small ones, in the same tiles."""
    size = torch.ones(lens[1], 1, 1) * 2.0 ** -6
    size[100:] = 2.0 ** 11
    attend(S, R.Batch("int4", D, 16, 4, 2, [lens], seed=13, k_scale=size), scale=D ** -0.5 * 2.0 ** 6)


def test_attention_large_queries(S):
    """Queries across the range of bf16: 2^-60 to 2^60 with scales that bring the scores back."""
    for e in (-60, -20, 20, 60):
        b = R.Batch("nvfp4", 128, 16, 4, 2, [(1, 100), (40, 100)], seed=9)
        b.q = (b.q.float() * 2.0 ** e).to(torch.bfloat16)
        attend(S, b, scale=128 ** -0.5 * 2.0 ** -e)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("lens", [[(1, 300), (2, 90)], [(1, 9000)], [(150, 300)], [(500, 2500)]])
def test_attention_queries_that_are_not_finite(S, fmt, lens):
    """A query with a NaN or an infinity gives NaN in its output and in its lse (-inf says that a query sees no
    key), whole or joined from parts, and the other rows and heads of its tile do not see it."""
    b = R.Batch(fmt, 64, 64, 6, 2, lens, seed=70)
    q = b.q.clone()
    bad = torch.zeros(b.rows, 6, dtype=torch.bool)
    for row, head, at, x in ((0, 0, 5, "nan"), (0, 4, slice(None), "nan"), (-1, 1, 7, "inf"), (-1, 5, slice(None), "-inf")):
        q[row, head, at] = float(x)
        bad[row, head] = True
    out, lse = S.svdq_kv_attention(cache_of(S, b), q.cuda(), dev(b.cu), dev([kv for _, kv in lens], torch.int32), dev(b.table),
                                   return_lse=True)
    assert out.cpu()[bad].isnan().all() and lse.cpu()[bad].isnan().all()
    o, l, to, tl = b.expected(64 ** -0.5, True, 0)
    fine = ~bad.numpy()
    within(out[~bad.cuda()], o[fine], to[fine])
    within(lse[~bad.cuda()], l[fine], tl[fine])
    assert S.svdq_get_error() == 0


@pytest.mark.parametrize("lens", [[(1, 300), (1, 40)], [(150, 300), (20, 40)]])
def test_attention_strided_padded_and_repeated(S, lens):
    """Queries as a view of wider rows, an output of its own stride with padded rows and
    columns, which stay; two calls give the same bits."""
    b = R.Batch("fp4g32", 64, 16, 6, 2, lens, seed=4, spare_rows=5)
    wide = torch.full((b.rows, 3 * 6, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 6:12] = b.q.cuda()
    room = torch.full((b.rows, 8, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    out, lse = attend(S, b, q=wide[:, 6:12], out=room[:, 1:7])
    assert (room[:, 0] == 3).all() and (room[:, 7] == 3).all() and (room[b.cu[-1]:] == 3).all()
    first = room.clone()
    attend(S, b, q=wide[:, 6:12], out=room[:, 1:7])
    assert torch.equal(first, room)


@pytest.mark.parametrize("lens", [[(1, 100), (1, 60)], [(80, 100), (60, 60)]])
def test_attention_bad_indices_are_masked(S, lens):
    """A page outside the pool masks its keys, a length past the table row is cut; bit 3 says so."""
    b = R.Batch("nvfp4", 64, 16, 4, 2, lens, seed=12)
    c, q, cu = cache_of(S, b), b.q.cuda(), dev(b.cu)
    for bad in (-1, b.pool.shape[0], 2 ** 31 - 1):
        table = b.table.copy()
        table[0, 1] = bad                         # keys 16 .. 31 of request 0
        out, lse = S.svdq_kv_attention(c, q, cu, dev([kv for _, kv in b.lens], torch.int32), dev(table), return_lse=True)
        assert S.svdq_get_error() == 8
        keep = np.r_[0:16, 32:100]
        n, kv = b.lens[0]
        pos = kv - n + np.arange(n)
        for i in {0, n // 2, n - 1}:              # one query: its visible keys among the kept ones
            sel = keep[keep <= pos[i]]
            o, l, to, tl = R.attention(b.q[i:i + 1].double().numpy(), b.keys[0][sel], b.values[0][sel], 64 ** -0.5, False, 0)
            within(out[i:i + 1], o, to)
            within(lse[i:i + 1], l, tl)
        o, l, to, tl = b.expected(64 ** -0.5, True, 0)
        within(out[n:], o[n:], to[n:])
    width = b.table.shape[1] * 16
    out = S.svdq_kv_attention(c, q, cu, dev([width + 1, -4], torch.int32), dev(np.maximum(b.table, 0)), causal=False)
    # request 0 now counts tokens that nobody wrote (random bytes, NaN scales among them) as keys: only request 1 is known
    assert S.svdq_get_error() == 8 and (out[b.cu[1]:] == 0).all()


def test_attention_past_32_bit_offsets(S):
    """A pool of 5 GB whose used pages lie past 2^32 bytes."""
    fmt, D, page, hk = "int4", 128, 256, 8
    block = R.pieces(fmt, D, page)[3]
    pages = 5 * 2 ** 30 // (block * hk)
    pool = torch.zeros(pages, hk, block, dtype=torch.uint8, device="cuda")
    c = S.KVCache(fmt, hk, D, page, pool)
    b = R.Batch(fmt, D, page, 8, hk, [(1, 600), (30, 300)], seed=2)
    high = pages - b.pool.shape[0]
    pool[high:] = dev(b.pool)
    table = np.where(b.table >= 0, b.table + high, -1).astype(np.int32)
    out, lse = S.svdq_kv_attention(c, b.q.cuda(), dev(b.cu), dev([600, 300], torch.int32), dev(table), return_lse=True)
    assert S.svdq_get_error() == 0
    o, l, to, tl = b.expected(D ** -0.5, True, 0)
    within(out, o, to)
    within(lse, l, tl)
    slots = torch.tensor([pages * page - 1, high * page], device="cuda")
    x = torch.randn(2, hk, D, device="cuda").to(torch.bfloat16)
    S.svdq_kv_append(c, x, x, slots)
    kq = torch.from_numpy(R.quantize(fmt, x.cpu())[2])
    assert torch.equal(S.svdq_kv_read(c, slots, torch.float32)[0].double().cpu(), kq)


@pytest.mark.parametrize("lens", [[(1, 500), (1, 900), (1, 3)], [(100, 500), (33, 333)]])
def test_attention_on_a_stream_and_in_a_graph(S, lens):
    """Another stream than the current one, then a captured call replayed on new queries and lengths."""
    b = R.Batch("nvfp4", 128, 64, 8, 2, lens, seed=21)
    c, table, cu = cache_of(S, b), dev(b.table), dev(b.cu)
    kl = dev([kv for _, kv in lens], torch.int32)
    q = b.q.cuda()
    want, _ = attend(S, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = S.svdq_kv_attention(c, q, cu, kl, table, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    ws = torch.empty(max(1, S.svdq_kv_attention_workspace_bytes(c, 8, b.rows, len(lens))), dtype=torch.uint8, device="cuda")
    got, graph = torch.zeros_like(want), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        S.svdq_kv_attention(c, q, cu, kl, table, out=got, workspace=ws)
        again = torch.cuda.CUDAGraph()
    other = torch.zeros_like(want)
    with torch.cuda.graph(again):                      # a second graph on the same workspace, run in turn
        S.svdq_kv_attention(c, q, cu, kl, table, out=other, workspace=ws)
    ws.random_(0, 256)
    graph.replay(), again.replay(), graph.replay()
    assert torch.equal(got, want) and torch.equal(other, want)
    shorter = [(n, max(n, kv - 65)) if kv else (n, kv) for n, kv in lens]
    kl.copy_(torch.tensor([kv for _, kv in shorter], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    b.lens = shorter
    b.keys, b.values = [k[:kv] for k, (_, kv) in zip(b.keys, shorter)], [v[:kv] for v, (_, kv) in zip(b.values, shorter)]
    o, _, to, _ = b.expected(128 ** -0.5, True, 0)
    within(got, o, to)
    assert S.svdq_get_error() == 0


# ------------------------------------------------------------------ together ---
@pytest.mark.parametrize("fmt", FMTS)
def test_serving_steps(S, fmt):
    """A ragged prompt step and two decode steps of a block's attention: 4-bit QKV layer, plan,
    norm and rotation, append, attention, 4-bit output layer; the attention of each step is checked
    against the 64-bit reference on the same normed rows, over all that was appended before."""
    K, hq, hk, D, page = 512, 8, 2, 64, 16
    g = torch.Generator().manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    wqkv = S.svdq_prepare_weights((rnd(K, (hq + 2 * hk) * D) * 0.05).to(torch.bfloat16).cuda(), rank=16)
    wout = S.svdq_prepare_weights((rnd(hq * D, K) * 0.05).to(torch.bfloat16).cuda(), rank=16)
    weight = [(1 + 0.1 * rnd(D)).to(torch.bfloat16).cuda() for _ in range(2)]
    rope = dev(R.rotation(256, D))
    cache = S.KVCache(fmt, hk, D, page, num_pages=32)
    table = torch.full((3, 8), -1, dtype=torch.int32, device="cuda")
    free = torch.arange(31, -1, -1, dtype=torch.int32, device="cuda")
    lens, taken = torch.zeros(3, dtype=torch.int32, device="cuda"), 0
    held = [[np.zeros((0, hk, D))] * 2 for _ in range(3)]
    for step, new in enumerate([[37, 1, 16], [1, 1, 1], [1, 1, 1]]):
        rows = sum(new) + 3                               # a padded batch
        x = rnd(rows, K).to(torch.bfloat16).cuda()
        qkv = S.svdq_forward(wqkv, x).view(rows, hq + 2 * hk, D)
        cu, lens, pos, slots, used = S.svdq_kv_plan(torch.tensor(new, dtype=torch.int32, device="cuda"), lens, table,
                                                    free[taken:].contiguous(), rows, page)
        taken += int(used)
        q, k = S.svdq_qk_norm_rope(qkv[:, :hq], qkv[:, hq:hq + hk], rope, pos, *weight,
                                   q_out=qkv[:, :hq], k_out=qkv[:, hq:hq + hk])
        v = qkv[:, hq + hk:]
        S.svdq_kv_append(cache, k, v, slots)
        out = torch.zeros(rows, hq, D, dtype=torch.bfloat16, device="cuda")
        S.svdq_kv_attention(cache, q, cu, lens, table, out=out)
        y = S.svdq_forward(wout, out.view(rows, hq * D))
        torch.cuda.synchronize()
        assert S.svdq_get_error() == 0 and torch.isfinite(y.float()).all()
        at = 0
        for b, n in enumerate(new):
            for side, t in enumerate((k, v)):
                held[b][side] = np.concatenate((held[b][side], R.quantize(fmt, t[at:at + n].cpu())[2]))
            o, _, to, _ = R.attention(q[at:at + n].double().cpu().numpy(), *held[b], D ** -0.5, True, 0, fmt == "int4")
            within(out[at:at + n], o, to)
            at += n
        assert (out[at:] == 0).all()
    wqkv.close(), wout.close()


@pytest.mark.parametrize("fmt", FMTS)
def test_serving_steps_with_a_window(S, fmt):
    """A prompt and decode steps under a sliding window in a pool that holds a fraction of the tokens: pages that the
    window has left go back to the free list, their entries become -1, and other tokens are written into them."""
    hq, hk, D, page, window, batch = 4, 2, 64, 16, 20, 2
    g = torch.Generator().manual_seed(17)
    cache = S.KVCache(fmt, hk, D, page, num_pages=14)
    table = torch.full((batch, 12), -1, dtype=torch.int32, device="cuda")
    free, lens = list(range(14)), torch.zeros(batch, dtype=torch.int32, device="cuda")
    held = [[np.zeros((0, hk, D))] * 2 for _ in range(batch)]
    reused = set()
    for step, new in enumerate([[60, 70]] + [[1, 2]] * 45):
        q, k, v = (torch.randn(sum(new), h, D, generator=g).to(torch.bfloat16) for h in (hq, hk, hk))
        cu, lens, pos, slots, used = S.svdq_kv_plan(torch.tensor(new, dtype=torch.int32, device="cuda"), lens, table,
                                                    dev(free, torch.int32), sum(new), page)
        reused |= {p for p in free[:int(used)] if step}
        free = free[int(used):]
        S.svdq_kv_append(cache, k.cuda(), v.cuda(), slots)
        out = S.svdq_kv_attention(cache, q.cuda(), cu, lens, table, window=window)
        at = 0
        for b, n in enumerate(new):
            for side, t in enumerate((k, v)):
                held[b][side] = np.concatenate((held[b][side], R.quantize(fmt, t[at:at + n])[2]))
            o, _, to, _ = R.attention(q[at:at + n].double().numpy(), *held[b], D ** -0.5, True, window, fmt == "int4")
            within(out[at:at + n], o, to)
            at += n
        for b, kv in enumerate(lens.tolist()):
            for col in range(max(0, kv + 1 - window) // page):      # the next query's first key
                if int(table[b, col]) >= 0:
                    free.append(int(table[b, col]))
                    table[b, col] = -1
    assert S.svdq_get_error() == 0 and lens.tolist() == [105, 160] and len(reused) > 5


# ------------------------------------------------------ longer, split, together ---
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D,hq,hk,lens", [
    (128, 4, 2, [(700, 2500), (1, 3000), (333, 900)]), (64, 6, 2, [(500, 1700), (64, 64)]), (128, 1, 1, [(1200, 1200)]),
    (128, 8, 1, [(1, 20000)]), (64, 4, 1, [(1, 9000), (1, 1)]), (128, 9, 3, [(3, 5000), (2, 700)])])
def test_attention_split_items(S, fmt, D, hq, hk, lens):
    """Items cut between many CTAs, by both kernels, causal and with a window that skips whole tiles."""
    b = R.Batch(fmt, D, 64, hq, hk, lens, seed=31)
    attend(S, b)
    attend(S, b, window=300)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128])
def test_attention_ends_of_items(S, fmt, D):
    """Full tiles of 256 rows followed by tiles of 1 to 32, several of each per CTA: the warps of a half that have
    no row of the next item start on it at once, while the others still write the last one's rows.  Every
    row is right, and every call gives the same bits."""
    b = R.Batch(fmt, D, 16, 8, 8, [(257 + i % 32, 257 + i % 32 + 37 * (i % 7)) for i in range(40)], seed=50)
    out, lse = attend(S, b)
    args = (cache_of(S, b), b.q.cuda(), dev(b.cu), dev([kv for _, kv in b.lens], torch.int32), dev(b.table))
    for _ in range(30):
        again = S.svdq_kv_attention(*args, return_lse=True)
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)


@pytest.mark.parametrize("hk,lens", [(46, [(700, 700)]), (18, [(1000, 1000), (1000, 1020)]), (40, [(1000, 250), (1000, 200)]),
                                     (24, [(1000, 1000), (1000, 1200)])])
def test_attention_items_of_one_length(S, hk, lens):
    """Fewer equal items than CTAs, as many and more; equal keys from unequal lengths; and items that are not equal."""
    b = R.Batch("fp4g32", 64, 32, hk, hk, lens, seed=80)
    attend(S, b, causal=False)
    attend(S, b, causal=False, window=400)


def test_attention_many_requests(S):
    """More requests than a scan's first level, most of them without new tokens."""
    rng = np.random.default_rng(5)
    lens = [(int(n), int(n) + int(kv)) for n, kv in zip(rng.integers(0, 3, 1500) * (rng.random(1500) < 0.3), rng.integers(0, 60, 1500))]
    attend(S, R.Batch("nvfp4", 64, 16, 4, 2, lens, seed=6))


@pytest.mark.parametrize("lens", [[(1, 700), (1, 900)], [(90, 700), (200, 900)]])
def test_attention_on_two_streams_at_once(S, lens):
    """Two calls in flight together, each with its own workspace, give what each gives alone."""
    batches = [R.Batch("nvfp4", 128, 64, 8, 2, lens, seed=s) for s in (40, 41)]
    want = [attend(S, b)[0] for b in batches]
    args = [(cache_of(S, b), b.q.cuda(), dev(b.cu), dev([kv for _, kv in b.lens], torch.int32), dev(b.table)) for b in batches]
    streams = [torch.cuda.Stream() for _ in batches]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i in (0, 1):
            got[i].append(S.svdq_kv_attention(*args[i], stream=streams[i]))
    torch.cuda.synchronize()
    for i in (0, 1):
        assert all(torch.equal(g, want[i]) for g in got[i])
    assert S.svdq_get_error() == 0


def test_step_in_a_graph(S):
    """Plan, norm, append and attention of a decode step captured once and replayed as the requests grow."""
    hq, hk, D, page, batch = 8, 2, 64, 16, 3
    g = torch.Generator().manual_seed(9)
    cache = S.KVCache("nvfp4", hk, D, page, num_pages=24)
    table = torch.full((batch, 8), -1, dtype=torch.int32, device="cuda")
    free = torch.arange(24, dtype=torch.int32, device="cuda")
    ones, lens = torch.ones(batch, dtype=torch.int32, device="cuda"), torch.zeros(batch, dtype=torch.int32, device="cuda")
    taken = torch.zeros(1, dtype=torch.int64, device="cuda")
    qkv = torch.zeros(batch, hq + 2 * hk, D, dtype=torch.bfloat16, device="cuda")
    rope = dev(R.rotation(128, D))
    out = torch.zeros(batch, hq, D, dtype=torch.bfloat16, device="cuda")
    q_out, k_out = torch.zeros_like(out), torch.zeros(batch, hk, D, dtype=torch.bfloat16, device="cuda")

    def step():
        cu, total, pos, slots, used = S.svdq_kv_plan(ones, lens, table, torch.roll(free, 0)[:24], batch, page)
        S.svdq_qk_norm_rope(qkv[:, :hq], qkv[:, hq:hq + hk], rope, pos, q_out=q_out, k_out=k_out)
        S.svdq_kv_append(cache, k_out, qkv[:, hq + hk:], slots)
        S.svdq_kv_attention(cache, q_out, cu, total, table, out=out)
        lens.copy_(total)
        taken.add_(used)
        free.copy_(free[(torch.arange(24, device="cuda") + used) % 24])      # the taken pages go to the end

    step()                                            # sets kernel attributes; then start over
    torch.cuda.synchronize()
    table.fill_(-1), lens.zero_(), taken.zero_(), free.copy_(torch.arange(24, dtype=torch.int32))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    held = [[np.zeros((0, hk, D))] * 2 for _ in range(batch)]
    for i in range(40):
        x = torch.randn(batch, hq + 2 * hk, D, generator=g).to(torch.bfloat16)
        qkv.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        for b in range(batch):
            for side, t in enumerate((k_out, x[:, hq + hk:])):
                held[b][side] = np.concatenate((held[b][side], R.quantize("nvfp4", t[b:b + 1].cpu())[2]))
            o, _, to, _ = R.attention(q_out[b:b + 1].double().cpu().numpy(), *held[b], D ** -0.5, True, 0)
            within(out[b:b + 1], o, to)
    assert S.svdq_get_error() == 0 and lens.tolist() == [40] * 3 and int(taken) == 9


@pytest.mark.parametrize("lens", [[(1, 3000), (1, 500)], [(300, 900)]])
def test_attention_wait_expiry_is_reported_and_recovered(S, lens):
    """Budget of one cycle: waits that outlast their first poll (the hardware holds one for a while) run out,
    the error word says so (bit 4 alone), and with the budget restored the same call gives the same bits again."""
    b = R.Batch("nvfp4", 128, 64, 8, 2, lens, seed=14)
    want, _ = attend(S, b)
    args = (cache_of(S, b), b.q.cuda(), dev(b.cu), dev([kv for _, kv in b.lens], torch.int32), dev(b.table))
    try:
        S.svdq_set_wait_budget(1)
        for _ in range(10):
            S.svdq_kv_attention(*args)
            err = S.svdq_get_error()
            assert err >= 0 and (err & ~16) == 0, err
    finally:
        S.svdq_set_wait_budget(1 << 31)
    again = S.svdq_kv_attention(*args)
    torch.cuda.synchronize()
    assert S.svdq_get_error() == 0 and torch.equal(again, want)


@pytest.mark.parametrize("fmt", ["nvfp4", "int4"])
def test_attention_wait_expiry_of_long_items(S, fmt):
    """Items of many tiles, whose roles wait for each other longer than the hardware holds a poll: with a budget of one
    cycle a wait of the many-row kernel does run out (bit 4 is seen, and no other), the launch ends by itself, and
    with the budget restored the same call gives the same bits again.  (The few-row kernel waits for nothing but its own
    copies, which land within a poll.)"""
    lens = [(1500, 3000)] * 3
    b = R.Batch(fmt, 128, 64, 8, 2, lens, seed=14)
    args = (cache_of(S, b), b.q.cuda(), dev(b.cu), dev([kv for _, kv in lens], torch.int32), dev(b.table))
    want = S.svdq_kv_attention(*args)
    torch.cuda.synchronize()
    assert S.svdq_get_error() == 0
    seen = []
    try:
        S.svdq_set_wait_budget(1)
        for _ in range(20):
            S.svdq_kv_attention(*args)
            seen.append(S.svdq_get_error())
    finally:
        S.svdq_set_wait_budget(1 << 31)
    assert set(seen) <= {0, 16} and 16 in seen, seen
    again = S.svdq_kv_attention(*args)
    torch.cuda.synchronize()
    assert S.svdq_get_error() == 0 and torch.equal(again, want)


def test_refused_tensors(S):
    """What the Python calls refuse before anything is launched."""
    c = S.KVCache("nvfp4", 2, 64, 16, num_pages=4)
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    slots = torch.zeros(3, dtype=torch.int64, device="cuda")
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    table = torch.zeros(1, 4, dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        S.svdq_kv_append(c, x.half(), x, slots)
    with pytest.raises(TypeError):
        S.svdq_kv_append(c, x.cpu(), x, slots)
    with pytest.raises(TypeError):
        S.svdq_kv_append(c, x, x, slots.int())
    with pytest.raises(ValueError):
        S.svdq_kv_append(c, x, x, slots[:2])
    with pytest.raises(ValueError):
        S.svdq_kv_append(c, x.transpose(1, 2).contiguous().transpose(1, 2), x, slots)      # heads not contiguous
    with pytest.raises(ValueError):
        S.svdq_kv_append(c, torch.zeros(400, dtype=torch.bfloat16, device="cuda")[1:385].view(3, 2, 64), x, slots)   # 2-byte start
    with pytest.raises(TypeError):
        S.svdq_kv_read(c, slots, torch.float16)
    with pytest.raises(ValueError):
        S.svdq_kv_attention(c, x, i32(0, 3), i32(3, 3), table)
    with pytest.raises(ValueError):
        S.svdq_kv_attention(c, x, i32(0, 3), i32(3), table, out=x[:1].expand(3, 2, 64))     # rows of the output overlap
    with pytest.raises(ValueError):
        S.svdq_kv_attention(c, x, i32(0, 3), i32(3), table, workspace=torch.zeros(8, dtype=torch.uint8, device="cuda"))
    with pytest.raises(S.SvdqError):
        S.svdq_kv_attention(c, torch.zeros(3, 3, 64, dtype=torch.bfloat16, device="cuda"), i32(0, 3), i32(3), table)
    with pytest.raises(S.SvdqError):
        S.svdq_kv_attention(c, x, i32(0, 3), i32(3), table, window=-1)
    with pytest.raises(S.SvdqError):
        S.svdq_kv_attention(c, x, i32(0, 3), i32(3), table, scale=float("nan"))
    with pytest.raises(ValueError):
        S.svdq_kv_plan(i32(1), i32(1, 2), table, i32(1), 1, 16)
    with pytest.raises(S.SvdqError):
        S.svdq_kv_plan(i32(1), i32(1), table, i32(1), 1, 24)
    with pytest.raises(ValueError):
        S.svdq_qk_norm_rope(x, x, torch.zeros(4, 64, device="cuda"), i32(0))
    with pytest.raises(S.SvdqError):
        S.svdq_qk_norm_rope(x, x, torch.zeros(2, 64, device="cuda"))        # fewer table rows than rows
    with pytest.raises(ValueError):
        S.KVCache("nvfp4", 2, 64, 16, torch.zeros(4, 2, 100, dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    assert S.svdq_get_error() == 0


@pytest.mark.parametrize("flag", ["norm", "interleaved", "causal", "return_lse"])
def test_refused_truth_values(S, flag):
    """A flag that has no truth value is a TypeError, and nothing is written."""
    x = torch.ones(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    out, two = torch.full_like(x, 7), torch.zeros(2)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    with pytest.raises(TypeError):
        if flag in ("norm", "interleaved"):
            S.svdq_qk_norm_rope(x, x, q_out=out, k_out=out.clone(), **{flag: two})
        else:
            c = S.KVCache("nvfp4", 2, 64, 16, torch.zeros(4, 2, 1152, dtype=torch.uint8, device="cuda"))
            S.svdq_kv_attention(c, x, i32(0, 3), i32(3), torch.zeros(1, 4, dtype=torch.int32, device="cuda"), out=out, **{flag: two})
    torch.cuda.synchronize()
    assert (out == 7).all()
