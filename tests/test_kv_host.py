"""What the cache operators refuse, on the CPU: the C entries before they touch the device,
and the references of the GPU tests against hand-worked values."""
import ctypes

import numpy as np
import pytest
import torch

import kv_ref as R


@pytest.fixture(scope="module")
def S():
    from w4a4_gemm_b200 import build as B
    B.build()
    import w4a4_gemm_b200 as S
    S.lib()
    return S


FAKE = 0x1000


def cache(S, fmt=0, heads=2, dim=64, page=16, pages=4, pool=FAKE):
    return S._KvCache(fmt, heads, dim, page, pages, pool)


def test_page_bytes_and_refused_caches(S):
    n = ctypes.c_size_t()
    call = lambda c: S.lib().svdq_kv_page_bytes(ctypes.byref(c), ctypes.byref(n))  # noqa: E731
    for fmt, dim, token in ((0, 128, 72), (2, 128, 68), (1, 128, 68), (0, 64, 36), (2, 64, 34), (1, 64, 34)):
        assert call(cache(S, fmt=fmt, dim=dim, heads=3, page=32)) == 0 and n.value == 3 * 32 * 2 * token
    assert call(cache(S, fmt=3)) == 1                  # W8A8 is no cache format
    for bad in (dict(dim=96), dict(dim=256), dict(heads=0), dict(page=8), dict(page=24), dict(page=512), dict(pages=-1),
                dict(pages=2 ** 31), dict(heads=1025)):
        assert call(cache(S, **bad)) == 2, bad
    assert S.lib().svdq_kv_page_bytes(None, ctypes.byref(n)) == 1
    assert S.lib().svdq_kv_page_bytes(ctypes.byref(cache(S)), None) == 1


def test_refused_appends_and_reads(S):
    L, c = S.lib(), cache(S)
    ok = [ctypes.byref(c), FAKE, FAKE, 128, 128, FAKE, 4, None]
    for at, bad in ((1, None), (1, 0x1008), (2, 0x1002), (3, 129), (4, -8), (5, None), (6, -1)):
        args = list(ok)
        args[at] = bad
        assert L.svdq_kv_append(*args) == 1, (at, bad)
    for args in ([FAKE, 4, 0, None, FAKE], [FAKE, 4, 0, FAKE, 0x1004], [None, 4, 0, FAKE, FAKE], [FAKE, -1, 0, FAKE, FAKE]):
        assert L.svdq_kv_read(ctypes.byref(c), *args, None) == 1
    assert L.svdq_kv_append(ctypes.byref(cache(S, pool=None)), FAKE, FAKE, 128, 128, FAKE, 4, None) == 1
    assert L.svdq_kv_append(ctypes.byref(cache(S, pool=0x1008)), FAKE, FAKE, 128, 128, FAKE, 4, None) == 1
    assert L.svdq_kv_append(ctypes.byref(c), None, None, 0, 0, None, 0, None) == 0        # no rows: nothing to do
    assert L.svdq_kv_read(ctypes.byref(c), None, 0, 0, None, None, None) == 0


def test_refused_plans(S):
    names = [f[0] for f in S._KvPlanDesc._fields_]
    good = dict(q_lens=FAKE, kv_lens=FAKE, block_table=FAKE, table_stride=4, table_width=4, free_pages=FAKE, free_count=3, batch=2,
                rows=5, page_size=16, cu_q=FAKE, total_lens=FAKE, positions=FAKE, slots=FAKE, used=FAKE)
    call = lambda **kw: S.lib().svdq_kv_plan(ctypes.byref(S._KvPlanDesc(*[{**good, **kw}[n] for n in names])), None)  # noqa: E731
    for bad in (dict(q_lens=None), dict(kv_lens=None), dict(block_table=None), dict(table_stride=3), dict(table_width=-1),
                dict(free_pages=None), dict(free_count=-1), dict(batch=-1), dict(rows=-1), dict(cu_q=None), dict(total_lens=None),
                dict(positions=None), dict(slots=None), dict(used=None)):
        assert call(**bad) == 1, bad
    for bad in (dict(page_size=8), dict(page_size=48), dict(page_size=512), dict(batch=16385)):
        assert call(**bad) == 2, bad
    assert S.lib().svdq_kv_plan(None, None) == 1


def test_refused_norms(S):
    names = [f[0] for f in S._QkNormRopeDesc._fields_]
    good = dict(q=FAKE, k=FAKE, q_out=FAKE, k_out=FAKE, q_stride=256, k_stride=128, q_out_stride=256, k_out_stride=128, q_weight=FAKE,
                k_weight=None, table=FAKE, positions=FAKE, table_rows=9, rows=3, q_heads=2, k_heads=1, head_dim=128, rot_dim=64,
                norm=1, interleaved=0, eps=1e-6)
    call = lambda **kw: S.lib().svdq_qk_norm_rope(ctypes.byref(S._QkNormRopeDesc(*[{**good, **kw}[n] for n in names])), None)  # noqa: E731
    for bad in (dict(q=None), dict(k=0x1004), dict(q_out=None), dict(k_out=0x1008), dict(q_stride=250), dict(q_out_stride=128),
                dict(k_out_stride=120), dict(q_weight=0x1002), dict(table=None), dict(rows=-1), dict(q_heads=-1), dict(eps=-1.0),
                dict(eps=float("nan")), dict(positions=None, table_rows=2), dict(table_rows=-1)):
        assert call(**bad) == 1, bad
    for bad in (dict(head_dim=120, rot_dim=0), dict(head_dim=272), dict(rot_dim=144), dict(rot_dim=24), dict(head_dim=0, rot_dim=0)):
        assert call(**bad) == 2, bad
    assert call(rows=0) == 0 and call(q_heads=0, k_heads=0) == 0
    assert S.lib().svdq_qk_norm_rope(None, None) == 1


def test_refused_attentions(S):
    names = [f[0] for f in S._KvAttentionDesc._fields_]
    good = dict(cache=cache(S), q=FAKE, q_stride=256, out=2 * FAKE, out_stride=256, lse=FAKE, cu_q=FAKE, kv_lens=FAKE, block_table=FAKE,
                table_stride=4, table_width=4, batch=2, rows=5, q_heads=4, causal=1, window=0, scale=0.1, workspace=FAKE)
    call = lambda **kw: S.lib().svdq_kv_attention(ctypes.byref(S._KvAttentionDesc(*[{**good, **kw}[n] for n in names])), None)  # noqa: E731
    for bad in (dict(q=None), dict(q=0x1008), dict(q_stride=252), dict(out=None), dict(out_stride=248), dict(cu_q=None), dict(kv_lens=None),
                dict(block_table=None), dict(table_stride=3), dict(batch=-1), dict(rows=-1), dict(window=-1), dict(scale=float("nan")),
                dict(scale=float("inf")), dict(cache=cache(S, pool=None)), dict(workspace=None), dict(workspace=0x1080), dict(out=FAKE), dict(cache=cache(S, fmt=3)), dict(table_width=-1)):
        assert call(**bad) == 1, bad
    for bad in (dict(q_heads=3), dict(q_heads=0), dict(batch=65537), dict(cache=cache(S, dim=32)), dict(cache=cache(S, page=20))):
        assert call(**bad) == 2, bad
    assert call(rows=0) == 0 and call(batch=0) == 0
    assert S.lib().svdq_kv_attention(None, None) == 1
    n = ctypes.c_size_t()
    assert S.lib().svdq_kv_attention_workspace_bytes(None, ctypes.byref(n)) == 1


def test_refused_row_counts(S):
    """Rows past 2^30 would pass 32 bits where the kernels count rows and CTAs."""
    L, c, many = S.lib(), ctypes.byref(cache(S)), 2 ** 30 + 1
    assert L.svdq_kv_append(c, FAKE, FAKE, 0, 0, FAKE, many, None) == 2
    assert L.svdq_kv_read(c, FAKE, many, 0, FAKE, FAKE, None) == 2
    names = [f[0] for f in S._KvPlanDesc._fields_]
    plan = dict.fromkeys(names, FAKE) | dict(table_stride=4, table_width=4, free_count=3, batch=2, page_size=16)
    assert L.svdq_kv_plan(ctypes.byref(S._KvPlanDesc(*[{**plan, "rows": many}[n] for n in names])), None) == 2


def test_a_cache_keeps_its_pool(S):
    """The calls hold the pool's address: a pool put in its place would be freed under it."""
    with pytest.raises(AttributeError):
        S.KVCache.__new__(S.KVCache).pool = torch.zeros(1, dtype=torch.uint8)


def test_python_refusals_without_a_gpu(S):
    """CPU tensors and wrong formats never reach the library."""
    with pytest.raises(TypeError):
        S.KVCache("nvfp4", 2, 64, 16, torch.zeros(1, 2, 1152, dtype=torch.uint8))
    with pytest.raises(S.SvdqError):
        S.KVCache("nvfp4", 2, 80, 16, num_pages=1)
    with pytest.raises(S.SvdqError):
        S.KVCache("w8a8", 2, 64, 16, num_pages=1)
    with pytest.raises(KeyError):
        S.KVCache("fp8", 2, 64, 16)
    with pytest.raises(TypeError):
        S.KVCache("nvfp4", 2.5, 64, 16, num_pages=1)
    with pytest.raises(TypeError):
        S._ext().kv_append(b"not a cache", None, None, None)          # too few arguments


def test_reference_plan_by_hand():
    """Pages of 16: request 0 has 15 tokens in page 9 and brings 2 (slot 9 * 16 + 15, then the free
    page 5); request 1 has none and brings 17 (pages 3 and 8); one padded row."""
    table = np.array([[9, -1], [-1, -1]], np.int32)
    cu, total, pos, slots, used, t, bad = R.plan([2, 17], [15, 0], table, np.array([5, 3, 8, 1], np.int32), 20, 16)
    assert cu.tolist() == [0, 2, 19] and total.tolist() == [17, 17] and used == 3 and not bad
    assert pos.tolist() == [15, 16] + list(range(17)) + [-1]
    assert slots.tolist() == [159, 80] + [48 + i for i in range(16)] + [128, -1]
    assert t.tolist() == [[9, 5], [3, 8]]


def test_reference_attention_by_hand():
    """Two keys with scores 0 and log 3: weights 1/4 and 3/4; a causal first row sees the first key alone."""
    q = np.array([[[1.0, 0.0]], [[1.0, 0.0]]])
    k = np.array([[[0.0, 1.0]], [[np.log(3.0), 0.0]]])
    v = np.array([[[4.0, 0.0]], [[0.0, 8.0]]])
    o, l, _, _ = R.attention(q, k, v, 1.0, False, 0)
    assert np.allclose(o[0, 0], [1, 6]) and np.allclose(l, np.log(4.0))
    o, l, _, _ = R.attention(q, k, v, 1.0, True, 0)
    assert np.allclose(o[0, 0], [4, 0]) and np.allclose(l[0], 0) and np.allclose(o[1, 0], [1, 6])
    o, l, _, _ = R.attention(q, k[:1], v[:1], 1.0, True, 0)       # more queries than keys
    assert np.all(o[0] == 0) and l[0, 0] == -np.inf and np.allclose(o[1, 0], [4, 0])


def test_reference_rotation_by_hand():
    x = np.array([[[3.0, 4.0, 1.0, 2.0]]])
    table = np.array([[0.0, 1.0, 1.0, 0.0]], np.float32)          # pair 0 turns by 90 degrees, pair 1 by none
    y, _ = R.norm_rope(x, None, table, np.array([0]), 0.0, False, False)
    assert np.allclose(y, [[[-1, 4, 3, 2]]])
    y, _ = R.norm_rope(x, None, table, np.array([0]), 0.0, False, True)
    assert np.allclose(y, [[[-4, 3, 1, 2]]])
    y, _ = R.norm_rope(x, np.array([2.0, 2, 2, 2]), None, np.array([0]), 0.0, True, False)
    assert np.allclose(y, x / np.sqrt(7.5) * 2)
