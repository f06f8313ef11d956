"""The draft-and-verify operators without a GPU: pins of their oracle, and the
refusals that come before any CUDA call."""

import ctypes

import numpy as np
import pytest
import torch

import oracle
from oracle import drafts


# ---------------------------------------------------------------------------
# oracle pins
# ---------------------------------------------------------------------------

def _data(rows, H, Hkv, d, seed):
    g = np.random.default_rng(seed)
    return (g.standard_normal((rows, H, d)), g.standard_normal((rows, Hkv, d)),
            g.standard_normal((rows, Hkv, d)))


@pytest.mark.parametrize("m,n,t,N", [(5, 4, 7, 6), (0, 3, 0, 5), (3, 100, 9, 8), (2, 1, 4, 3)])
def test_a_chain_is_a_block_of_outputs(m, n, t, N):
    H, Hkv, d = 4, 2, 8
    Q, K, V = _data(m + t + N, H, Hkv, d, 1)
    state = oracle.prefill_cache(K[:m + t], V[:m + t], m, n, t)
    sl = slice(m + t, m + t + N)
    o, lse, _ = drafts.tree_attention(state, Q[sl], K[sl], V[sl], list(range(-1, N - 1)), n)
    ro, rl = oracle.prefill_attention(Q, K, V, m, n, range(m + t, m + t + N))
    np.testing.assert_allclose(o, ro, atol=1e-12)
    np.testing.assert_allclose(lse, rl, atol=1e-12)


def test_a_tree_is_masked_attention():
    """Every node sees what the end of its own chain of outputs sees."""
    m, n, t = 4, 5, 8
    parents = [-1, 0, 0, 1, -1, 3, 5, 6, 2]
    Q, K, V = _data(m + t + len(parents), 2, 1, 8, 2)
    state = oracle.prefill_cache(K[:m + t], V[:m + t], m, n, t)
    q, k, v = (x[m + t:] for x in (Q, K, V))
    o, lse, _ = drafts.tree_attention(state, q, k, v, parents, n)
    for i in range(len(parents)):
        up = drafts.chain(parents, i)[::-1]
        rows = list(range(m + t)) + [m + t + a for a in up]
        ro, rl = oracle.prefill_attention(Q[rows], K[rows], V[rows], m, n, [len(rows) - 1])
        np.testing.assert_allclose(o[i], ro[0], atol=1e-12)
        np.testing.assert_allclose(lse[i], rl[0], atol=1e-12)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_lengths_and_relative_positions(interleaved):
    d, f = 16, 10000.0 ** (-np.arange(6) / 6)
    q, k, _ = _data(1, 1, 1, d, 3)

    def dot(pq, pk):
        a = drafts.norm_rope(q, None, [pq], f, 0.0, interleaved)
        b = drafts.norm_rope(k, None, [pk], f, 0.0, interleaved)
        np.testing.assert_allclose((a * a).sum(), (q * q).sum(), rtol=1e-12)
        np.testing.assert_array_equal(a[..., 12:], q[..., 12:])
        return (a * b).sum()

    np.testing.assert_allclose(dot(7, 4), dot(1003, 1000), rtol=1e-9)
    assert abs(dot(7, 4) - dot(7, 5)) > 1e-6


def test_norm_has_unit_mean_square():
    x, _, _ = _data(3, 2, 1, 64, 4)
    y = drafts.norm_rope(x, np.ones(64), [0, 0, 0], [], 0.0, False)
    np.testing.assert_allclose((y * y).mean(-1), 1.0, rtol=1e-12)


def test_commit_is_repeated_append():
    m, n, t = 2, 3, 2
    _, K, V = _data(m + t, 1, 1, 4, 5)
    _, k, v = _data(8, 1, 1, 4, 6)
    state = oracle.prefill_cache(K, V, m, n, t)
    new = drafts.commit_tree(state, k, v, [0, 2, 5, 6, 7], n)
    assert new["t"] == 7
    for slot, node in ((4 % n, 5), (5 % n, 6), (6 % n, 7)):
        np.testing.assert_array_equal(new["Kr"][slot], k[node])
        np.testing.assert_array_equal(new["Vr"][slot], v[node])
    assert state["t"] == 2


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


def _rope(rswa, **kw):
    f = dict(q_weight=0x1000, k_weight=0x1000, inv_freq=0x1000, eps=1e-6, rotary_dim=64,
             interleaved=0)
    f.update(kw)
    return rswa._RopeStruct(**f)


def _norm_rope(rswa, rope, **kw):
    a = dict(q=0x10000, q_stride=1280, k=0x20000, k_stride=1280, positions=0x30000, rows=4,
             heads=10, kv_heads=10, head_dim=128, dtype=1, q_out=0x40000, k_out=0x50000)
    a.update(kw)
    rswa.rswa_debug_fail_next_cuda(1)      # a call that is not refused ends here, with 5
    try:
        return rswa.load().rswa_qk_norm_rope(
            None if rope is None else ctypes.byref(rope), *a.values(), None)
    finally:
        rswa.rswa_debug_fail_next_cuda(0)


def test_norm_rope_takes_what_it_should(rswa):
    ok = _rope(rswa)
    assert _norm_rope(rswa, ok) == 5
    assert _norm_rope(rswa, ok, q_stride=1288, k_stride=3840) == 5
    assert _norm_rope(rswa, ok, rows=1, q_stride=0, k_stride=7) == 5   # one row: no stride
    assert _norm_rope(rswa, ok, rows=0, q=None, k=None, positions=None) == 0
    assert _norm_rope(rswa, ok, dtype=0, head_dim=64, q_stride=640, k_stride=644) == 5
    assert _norm_rope(rswa, _rope(rswa, q_weight=None, k_weight=None)) == 5
    assert _norm_rope(rswa, _rope(rswa, rotary_dim=0, inv_freq=None)) == 5
    assert _norm_rope(rswa, _rope(rswa, eps=0.0, interleaved=1)) == 5


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), 3), (dict(head_dim=96), 3), (dict(rows=-1), 1), (dict(heads=0), 1),
    (dict(kv_heads=0), 1), (dict(heads=5000), 1), (dict(q=None), 1), (dict(k=None), 1),
    (dict(positions=None), 1), (dict(q_out=None), 1), (dict(k_out=None), 1),
    (dict(q=0x10008), 1), (dict(k=0x10002), 1), (dict(q_out=0x10008), 1),
    (dict(k_out=0x10008), 1), (dict(positions=0x10004), 1), (dict(q_stride=1279), 1),
    (dict(q_stride=1284), 1), (dict(k_stride=1272), 1), (dict(k_stride=-1280), 1),
    (dict(q_stride=1 << 41), 1), (dict(rows=1 << 31), 1),
])
def test_norm_rope_refuses_arguments(rswa, kw, status):
    assert _norm_rope(rswa, _rope(rswa), **kw) == status


# Rows of 1280 bf16 elements: 2560 bytes, 4 of them dense 10240 (0x2800).
@pytest.mark.parametrize("kw,status", [
    # in place, rows side by side or only one row
    (dict(q_out=0x10000), 5), (dict(k_out=0x20000), 5),
    (dict(rows=1, q_stride=3840, q_out=0x10000), 5), (dict(rows=1, q_stride=0, q_out=0x10000), 5),
    # in place, rows part of longer ones: a row of the result is another's input
    (dict(q_stride=3840, q_out=0x10000), 1), (dict(k_stride=1288, k_out=0x20000), 1),
    (dict(rows=2, q_stride=3840, q_out=0x10000), 1),
    # shifted
    (dict(q_out=0x10010), 1), (dict(q_out=0x10000 - 16), 1), (dict(q_out=0x10000 + 0x2800 - 16), 1),
    (dict(q_out=0x10000 + 0x2800), 5), (dict(q_out=0x10000 - 0x2800), 5),
    (dict(k_out=0x20000 - 0x2800 + 16), 1), (dict(rows=1, q_out=0x10010), 1),
    # over the other's input, and over each other
    (dict(q_out=0x20000), 1), (dict(k_out=0x10000), 1), (dict(k_out=0x40000), 1),
    (dict(k_out=0x40000 + 0x2800), 5), (dict(q_out=0x50000 - 16), 1),
    # in and beside the gaps of packed rows (queries, keys, values: 7680 bytes apart)
    (dict(k=0x10000 + 2560, q_stride=3840, k_stride=3840, rows=1, q_out=0x10000 + 5120), 5),
    (dict(k=0x10000 + 2560, q_stride=3840, k_stride=3840, rows=2, q_out=0x10000 + 5120), 1),
    (dict(q_stride=1 << 20, q_out=0x10000 + 2560), 5), (dict(q_stride=1 << 20, q_out=0x10000 + 2544), 1),
    (dict(q_stride=1 << 20, k=0x2000000, q_out=0x10000 + 3 * (2 << 20) - 0x2800), 5),
    (dict(q_stride=1 << 20, k=0x2000000, q_out=0x10000 + 3 * (2 << 20) - 0x2800 + 16), 1),
    (dict(q_stride=1 << 20, k=0x2000000, q_out=0x10000 + 3 * (2 << 20) + 2560), 5),
    (dict(q_stride=1 << 20, k=0x2000000, q_out=0x10000 + 3 * (2 << 20) + 2544), 1),
])
def test_norm_rope_refuses_results_over_inputs(rswa, kw, status):
    assert _norm_rope(rswa, _rope(rswa), **kw) == status


@pytest.mark.parametrize("kw", [
    dict(rotary_dim=-16), dict(rotary_dim=144), dict(rotary_dim=24), dict(rotary_dim=2),
    dict(inv_freq=None), dict(inv_freq=0x1004), dict(q_weight=0x1008), dict(k_weight=0x1002),
    dict(eps=-1e-6), dict(eps=float("nan")), dict(eps=float("inf")),
])
def test_norm_rope_refuses_ropes(rswa, kw):
    assert _norm_rope(rswa, _rope(rswa, **kw)) == 1


def test_norm_rope_refuses_no_rope(rswa):
    assert _norm_rope(rswa, None) == 1


def test_bad_handles(rswa):
    lib, rope, size = rswa.load(), _rope(rswa), ctypes.c_size_t(0)
    for handle in (None, ctypes.c_void_p(0x1234)):
        assert lib.rswa_qk_norm_rope_cached(handle, ctypes.byref(rope), 16, 0, 16, 0, None, 1,
                                            16, 16, None) == 4
        assert lib.rswa_append_kv_rope(handle, ctypes.byref(rope), 16, 0, 16, 0, 16, 0, 16,
                                       None) == 4
        assert lib.rswa_decode_tree_workspace(handle, 4, ctypes.byref(size)) == 4
        assert lib.rswa_decode_tree(handle, 16, 16, 16, 16, None, 4, 16, None, 256, 256,
                                    None) == 4
        assert lib.rswa_commit_tree(handle, 16, 16, 4, 16, 16, 4, None) == 4


def test_binding_refuses_cpu_tensors_and_types(rswa):
    f = torch.ones(8, dtype=torch.float64)
    with pytest.raises(ValueError):
        rswa.RswaRope(f)                               # not on a GPU
    with pytest.raises(ValueError):
        rswa.RswaRope(f.float())
    rope = rswa.RswaRope(None)
    x = torch.zeros(2, 3, 64)
    with pytest.raises(ValueError):
        rswa.rswa_qk_norm_rope(rope, x, x, torch.zeros(2, dtype=torch.int64), x, x)
