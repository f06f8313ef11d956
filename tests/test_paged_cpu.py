"""The paged-cache operators without a GPU: pins of their oracle, and the
refusals that come before any CUDA call."""

import ctypes

import numpy as np
import pytest
import torch

import oracle
from oracle import paged


def _data(L, H, Hkv, d, seed):
    g = np.random.default_rng(seed)
    return (g.standard_normal((L, H, d)), g.standard_normal((L, Hkv, d)),
            g.standard_normal((L, Hkv, d)))


# ---------------------------------------------------------------------------
# oracle pins
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("L,T,m,n", [(9, 9, 0, 100), (12, 5, 4, 3), (12, 1, 4, 3), (7, 7, 3, 1),
                                     (8, 3, 0, 2), (8, 6, 5, 2)])
def test_attend_is_the_prefill_oracle(L, T, m, n):
    Q, K, V = _data(L, 4, 2, 8, 1)
    o, lse, mass, size = paged.attend(Q[L - T:], K, V, m, n)
    ro, rl = oracle.prefill_attention(Q, K, V, m, n, range(L - T, L))
    np.testing.assert_allclose(o, ro, atol=1e-12)
    np.testing.assert_allclose(lse, rl, atol=1e-12)
    assert (mass >= np.abs(o) - 1e-12).all() and (size > 0).all()


@pytest.mark.parametrize("L,m,n", [(6, 0, 3), (10, 3, 4), (10, 20, 1), (5, 0, 1 << 30)])
def test_mask(L, m, n):
    for a in range(L):
        want = [j for j in range(L) if j <= a and (j < m or a - j < n)]
        assert paged.sees(a, m, n) == want and a in want


def test_weights_of_a_row_sum_to_one_and_give_its_output():
    Q, K, V = _data(11, 6, 2, 8, 2)
    o, lse, _, _ = paged.attend(Q[8:], K, V, 3, 4)
    w = paged.weigh(Q[8:], K, lse, 3, 4)
    np.testing.assert_allclose(w.sum(-1), 3 * 3)           # 3 rows of 3 heads
    one = paged.weigh(Q[8:9, :3], K[:9, :1], lse[:1, :3], 3, 4)
    np.testing.assert_allclose(one @ V[:9, 0], o[0, :3].sum(0)[None], atol=1e-12)


def test_evict_keeps_ends_and_the_heaviest():
    assert paged.evict([5, 1, 9, 1, 9, 2, 0, 7], 5, 1, 1) == [0, 2, 4, 5, 7]
    assert paged.evict([1, 1, 1, 1, 1], 3, 0, 0) == [0, 1, 2]      # ties: the lower
    assert paged.evict([1, 3, 3, 3, 1], 3, 1, 1) == [0, 1, 4]
    assert paged.evict([1, 2], 2, 0, 0) == [0, 1]
    assert paged.evict([np.nan, -np.inf, 0.0, -1.0], 2, 0, 0) == [2, 3]
    assert paged.evict([np.nan, -np.inf, np.nan], 2, 0, 0) == [0, 1]
    assert paged.evict([0.0, -0.0, 0.0], 2, 0, 0) == [0, 1]


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------

@pytest.fixture(scope="module")
def rswa():
    from sliding_window_attention_02_gb300 import _build
    _build.build()
    import sliding_window_attention_02_gb300 as m
    m.load()
    return m


def _footprint(rswa, **kw):
    a = dict(pages=10, page_size=16, heads=10, kv_heads=10, head_dim=128, dtype=1)
    a.update(kw)
    out = ctypes.c_size_t(0)
    return rswa.load().rswa_pages_footprint(*a.values(), ctypes.byref(out)), out.value


def test_footprint(rswa):
    st, size = _footprint(rswa)
    assert st == 0 and 2 * 10 * 16 * 10 * 128 * 2 <= size <= 2 * 10 * 16 * 10 * 128 * 2 + 1024
    st, big = _footprint(rswa, dtype=0)
    assert st == 0 and big > 1.9 * size
    assert _footprint(rswa, pages=1 << 23, kv_heads=8, heads=32)[0] == 0     # 2^30 rows
    assert rswa.load().rswa_pages_footprint(10, 16, 10, 10, 128, 1, None) == 1


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), 3), (dict(head_dim=96), 3), (dict(pages=0), 1), (dict(pages=-1), 1),
    (dict(page_size=8), 1), (dict(page_size=48), 1), (dict(page_size=512), 1), (dict(page_size=0), 1),
    (dict(heads=0), 1), (dict(kv_heads=0), 1), (dict(kv_heads=3), 1), (dict(heads=4100, kv_heads=1), 1),
    (dict(pages=(1 << 23) + 1, kv_heads=8, heads=32), 1), (dict(pages=1 << 62), 1),
])
def test_footprint_refuses(rswa, kw, status):
    assert _footprint(rswa, **kw)[0] == status


def test_create_refuses_before_cuda(rswa):
    lib, h = rswa.load(), ctypes.c_void_p()
    need = _footprint(rswa)[1]

    def create(buf=0x100000, size=need, page_size=16, out=ctypes.byref(h)):
        return lib.rswa_pages_create(10, page_size, 10, 10, 128, 1, buf, size, out)

    assert create(buf=None) == 1 and create(buf=0x100080) == 1 and create(out=None) == 1
    assert create(size=need - 1) == 2 and create(page_size=24) == 1
    lib.rswa_debug_fail_next_cuda(1)
    assert create() == 5
    assert h.value is None


def test_bad_handles(rswa):
    lib, size = rswa.load(), ctypes.c_size_t(0)
    bt = rswa._BatchStruct(16, 16, None, None, 1, 1, 1)
    ref = ctypes.byref(bt)
    for handle in (None, ctypes.c_void_p(0x1234)):
        assert lib.rswa_pages_destroy(handle) == 4
        assert lib.rswa_pages_append(handle, ref, 1, 16, 0, 16, 0, None) == 4
        assert lib.rswa_pages_attend_workspace(handle, 1, ctypes.byref(size)) == 4
        assert lib.rswa_pages_attend(handle, ref, 1, 16, 0, 16, None, 256, 1 << 20, None) == 4
        assert lib.rswa_pages_weigh(handle, ref, 1, 16, 0, 16, 16, 1.0, None) == 4
        assert lib.rswa_pages_evict_workspace(handle, 1, 1, ctypes.byref(size)) == 4
        assert lib.rswa_pages_evict(handle, ref, 16, 1, 0, 0, None, 16, None, 256, 1 << 20,
                                    None) == 4
        assert lib.rswa_pages_kv_offsets(handle, ctypes.byref(size), ctypes.byref(size)) == 4
        assert lib.rswa_pages_sync_status(handle) == 4


def test_binding_refuses_cpu_tensors(rswa):
    with pytest.raises(ValueError):
        rswa.RswaBatch(torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        rswa.RswaBatch(torch.zeros(2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32))
