"""GPU parity of the draft-and-verify operators (norm and rotation of query and
key heads, rotated append, tree attention, commit of the accepted path) against
their float64 oracle.

Tolerances come from the arithmetic of each operator; a rounding to a type is
off by at most half a step, eps / 2 (bf16 2^-8, float32 2^-24) relative to the
value.

norm_rope.  In float32, relative to the length |a| + |b| of a rotated pair: the
sum of squares (at most 16 products in sequence and 4 shuffle sums, halved by the
square root: 10 half steps), the reciprocal root (4), the products with it and the
weight (2), sine and cosine (4) of an angle off by half a step of at most pi (4),
the rotation's products and sum (3): 27, taken as 32.  Then one rounding to the
type.

tree.  A logit is a dot product of d terms, off by at most (d + 8) half steps of
sum |q k| / sqrt(d) (twice that on the tensor cores, which truncate); weights and
sums over S keys by S half steps more, and 2^-21 for the exponential.  That bounds
the log-sum-exp directly, and o relative to sum p |v|, twice (numerator and
denominator).  In bf16 the weights are rounded to bf16 (2^-8 of sum p |v|) and o is
(2^-8 of |o|).
"""

import numpy as np
import pytest
import torch

import oracle
import workloads
from oracle import drafts

pytestmark = pytest.mark.gpu

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
RSWA_EDEVICE = 6


def f64(t):
    return t.detach().double().cpu().numpy()


def inv_freq(rot):
    if rot == 0:
        return None
    i = torch.arange(rot // 2, dtype=torch.float64)
    return (10000.0 ** (-2.0 * i / rot)).cuda()


def normal(shape, seed, dtype=torch.bfloat16, std=1.0):
    return workloads.normal(shape, seed, std, dtype, "cuda")


def weight(d, seed, dtype):
    return (1 + 0.2 * normal((d,), seed, torch.float32)).to(dtype)


def same(got, want):
    np.testing.assert_array_equal(f64(got), want)


# ---------------------------------------------------------------------------
# norm and rotation
# ---------------------------------------------------------------------------

def check_rope(got, x, w, pos, rope, what):
    rot = rope.rotary_dim
    f = [] if rot == 0 else f64(rope.inv_freq)
    il = bool(rope._struct.interleaved)
    eps = rope._struct.eps
    ref = drafts.norm_rope(f64(x), None if w is None else f64(w), pos, f, eps, il)
    size = np.abs(ref)
    if rot:                                    # |a| + |b| of each pair, before the turn
        y = np.abs(drafts.norm_rope(f64(x), None if w is None else f64(w),
                                    [0] * len(pos), f, eps, il))
        a, b = (slice(0, rot, 2), slice(1, rot, 2)) if il else (slice(0, rot // 2),
                                                                slice(rot // 2, rot))
        size[..., a] = size[..., b] = y[..., a] + y[..., b]
    tol = 32 * 2.0 ** -24 * size
    if got.dtype == torch.bfloat16:
        tol = tol + HALF[torch.bfloat16] * (np.abs(ref) + tol)
    err = np.abs(f64(got) - ref)
    assert np.isfinite(err).all() and (err <= tol).all(), \
        f"{what}: worst {np.max(err / np.maximum(tol, 1e-300)):.3g} of the bound"


ROPE_CASES = [
    # rows, H, Hkv, d, rot, interleaved, norm, dtype
    (1, 1, 1, 64, 64, False, True, torch.float32),
    (1, 10, 10, 128, 128, False, True, torch.bfloat16),
    (3, 5, 1, 128, 128, True, True, torch.bfloat16),
    (7, 32, 8, 128, 64, False, True, torch.bfloat16),
    (5, 9, 3, 128, 16, False, True, torch.bfloat16),
    (6, 4, 2, 128, 112, True, True, torch.bfloat16),
    (6, 7, 7, 64, 48, False, True, torch.bfloat16),
    (9, 6, 2, 64, 32, True, True, torch.float32),
    (4, 3, 3, 128, 80, False, True, torch.float32),
    (4, 3, 1, 128, 128, True, False, torch.float32),
    (11, 10, 10, 128, 0, False, True, torch.bfloat16),
    (2, 2, 2, 64, 0, True, False, torch.bfloat16),
    (700, 10, 10, 128, 128, False, True, torch.bfloat16),
    (333, 33, 11, 64, 64, False, True, torch.bfloat16),
]


@pytest.mark.parametrize("rows,H,Hkv,d,rot,il,norm,dtype", ROPE_CASES)
@pytest.mark.parametrize("packed", [False, True])
def test_norm_rope(cuda_lib, rows, H, Hkv, d, rot, il, norm, dtype, packed):
    rswa = cuda_lib
    if packed:
        qkv = normal((rows, H + 2 * Hkv, d), 1, dtype)
        q, k = qkv[:, :H], qkv[:, H:H + Hkv]
    else:
        q, k = normal((rows, H, d), 1, dtype), normal((rows, Hkv, d), 2, dtype)
    qw, kw = (weight(d, 3, dtype), weight(d, 4, dtype)) if norm else (None, None)
    rope = rswa.RswaRope(inv_freq(rot), qw, kw, eps=1e-5, interleaved=il)
    pos = (torch.arange(rows, dtype=torch.int64) * 37 + 5) % 1500
    qo, ko = (torch.full((rows, h, d), float("nan"), dtype=dtype, device="cuda")
              for h in (H, Hkv))
    rswa.rswa_qk_norm_rope(rope, q, k, pos.cuda(), qo, ko)
    check_rope(qo, q, qw, pos.tolist(), rope, "q")
    check_rope(ko, k, kw, pos.tolist(), rope, "k")


def test_norm_rope_far_and_negative_positions(cuda_lib):
    """Far positions keep the accuracy of near ones; a negative one turns back."""
    rswa = cuda_lib
    pos = [0, 1, -1, -77777, 999_983, 2 ** 24 + 1, 2 ** 31 - 1, 2 ** 31 + 5]
    q, k = normal((len(pos), 2, 128), 5, torch.float32), normal((len(pos), 1, 128), 6, torch.float32)
    qw = weight(128, 7, torch.float32)
    rope = rswa.RswaRope(inv_freq(128), qw, None)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    rswa.rswa_qk_norm_rope(rope, q, k, torch.tensor(pos).cuda(), qo, ko)
    check_rope(qo, q, qw, pos, rope, "q")
    check_rope(ko, k, None, pos, rope, "k")
    same(qo[:0], f64(q[:0]))


def test_rotation_angles_are_as_exact_as_stated(cuda_lib):
    """Cosine and sine of angles at near and far positions and of small and huge
    frequencies, against exact integer arithmetic (2^200 / (2 pi) as an integer).
    The angle: 2^-26 + 2^-32 + |pos| max(1, |f|) 2^-63 turns.  Sine and cosine of
    it: 4 half steps of 1; the rotation's products with 1 and 0 and the norm are
    exact or left out."""
    from fractions import Fraction
    rswa = cuda_lib
    two_pi = Fraction(628318530717958647692528676655900576839433879875021164194988918461563281257,
                      10 ** 74)
    freqs = [1.0, -1.0, 0.75, 2 ** -20 / 3, 1e-9, 1e-30, 5e-324, 0.0, 10000 ** -0.3, 3.0, -1e3, 1e6,
             123456.789, 2.0 ** 52 + 1, 2.0 ** 100, -1e300, 2 * np.pi, np.pi / 2, 1e-3, 7.0]
    freqs += [10000.0 ** (-i / 20) for i in range(32 - len(freqs))]
    pos = [0, 1, -1, 2, 77, 1000, -77777, 999_983, 2 ** 31 + 5, -2 ** 40 - 3]
    q = torch.zeros(len(pos), 1, 64, device="cuda")
    q[..., :32] = 1.0                            # pairs (1, 0): cosine, sine
    rope = rswa.RswaRope(torch.tensor(freqs, dtype=torch.float64).cuda())
    qo, ko = torch.empty_like(q), torch.empty_like(q)
    rswa.rswa_qk_norm_rope(rope, q, q, torch.tensor(pos).cuda(), qo, ko)
    got = f64(qo)[:, 0]
    assert np.array_equal(got, f64(ko)[:, 0])
    for r, p in enumerate(pos):
        for i, f in enumerate(freqs):
            bound = 2.0 ** -26 + 2.0 ** -32 + abs(p) * max(1.0, abs(f)) * 2.0 ** -63
            if bound > 2.0 ** -10:
                continue                         # the statement says little there
            turn = Fraction(f) * p / two_pi
            turn -= int(turn)
            tol = 2 * np.pi * bound + 4 * 2.0 ** -24
            assert abs(got[r, i] - np.cos(2 * np.pi * float(turn))) <= tol, (p, f)
            assert abs(got[r, 32 + i] - np.sin(2 * np.pi * float(turn))) <= tol, (p, f)
    assert np.abs(got).max() <= 1 + 4 * 2.0 ** -24


def test_norm_rope_in_place_and_only_one_norm(cuda_lib):
    rswa = cuda_lib
    q, k = normal((50, 4, 64), 8), normal((50, 2, 64), 9)
    kw = weight(64, 10, torch.bfloat16)
    rope = rswa.RswaRope(inv_freq(64), None, kw)
    q0, k0 = q.clone(), k.clone()
    pos = torch.arange(50)
    rswa.rswa_qk_norm_rope(rope, q, k, pos.cuda(), q, k)
    check_rope(q, q0, None, pos.tolist(), rope, "q")
    check_rope(k, k0, kw, pos.tolist(), rope, "k")


def test_norm_rope_extreme_rows(cuda_lib):
    """A zero row stays zero (eps), a NaN or an infinity stays in its own head,
    elements that are not rotated are not mixed."""
    rswa = cuda_lib
    q = normal((4, 3, 64), 11, torch.float32)
    k = torch.zeros(4, 1, 64, device="cuda")
    q[1, 1, 40] = float("inf")
    q[2, 2, 3] = float("nan")
    rope = rswa.RswaRope(inv_freq(32), None, weight(64, 12, torch.float32))
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    rswa.rswa_qk_norm_rope(rope, q, k, torch.arange(4).cuda(), qo, ko)
    assert (ko == 0).all()
    bad = ~torch.isfinite(qo)
    where = bad.nonzero().tolist()
    assert where == [[1, 1, 40], [2, 2, 3], [2, 2, 19]]


def test_norm_rope_refusals(cuda_lib):
    rswa = cuda_lib
    q, k = normal((4, 2, 64), 13), normal((4, 1, 64), 14)
    pos = torch.arange(4).cuda()
    rope = rswa.RswaRope(inv_freq(64), weight(64, 15, torch.bfloat16))
    out = torch.empty_like(q), torch.empty_like(k)
    rswa.rswa_qk_norm_rope(rope, q, k, pos, *out)
    rswa.rswa_qk_norm_rope(rope, q[:0], k[:0], pos[:0], out[0][:0], out[1][:0])
    for bad in [
        (rope, q, k, pos.int(), *out), (rope, q, k, pos[:3], *out),
        (rope, q, k[:3], pos, *out), (rope, q, k.float(), pos, *out),
        (rope, q, k, pos, out[0].float(), out[1]), (rope, q, k, pos, out[0][:3], out[1]),
        (rope, q.half(), k.half(), pos, *out), (rope, q.float(), k.float(), pos, *out),
        (rope, q.transpose(0, 1), k, pos, *out), (rope, q, k, pos, *(x.cpu() for x in out)),
        (rswa.RswaRope(inv_freq(128)[:20].contiguous()), q, k, pos, *out),    # 40: no multiple of 16
        (rswa.RswaRope(inv_freq(128)), q, k, pos, *out),                      # more than the head
    ]:
        with pytest.raises((ValueError, rswa.RswaError)):
            rswa.rswa_qk_norm_rope(*bad)


def test_results_over_inputs_are_refused(cuda_lib):
    """A result over rows that other CTAs have yet to read: refused by all three
    calls, with nothing written; in place is taken where rows lie side by side."""
    rswa = cuda_lib
    B, H, Hkv, d, n = 4, 4, 2, 64, 8
    cache, states = make_cache(rswa, [9] * B, [3] * B, n, H, Hkv, d, BF, 16)
    rope = rswa.RswaRope(inv_freq(d), weight(d, 17, BF), weight(d, 18, BF))
    flat = normal((B * (H + 2 * Hkv) * d,), 19)
    before = flat.clone()
    qkv = flat.view(B, H + 2 * Hkv, d)
    q, k, v = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
    over_q, over_k = flat[:B * H * d].view(B, H, d), flat[H * d:][:B * Hkv * d].view(B, Hkv, d)
    qo, ko = torch.empty_like(over_q), torch.empty_like(over_k)
    pos = torch.arange(B).cuda()
    both = torch.empty(B * (H + Hkv) * d - 8, dtype=BF, device="cuda")
    for a, b in ((over_q, ko), (qo, over_k),
                 (both[:B * H * d].view(B, H, d), both[-B * Hkv * d:].view(B, Hkv, d))):
        for call in (lambda: rswa.rswa_qk_norm_rope(rope, q, k, pos, a, b),
                     lambda: cache.qk_norm_rope(rope, q, k, a, b)):
            with pytest.raises(rswa.RswaError) as e:
                call()
            assert e.value.status == 1
    for a in (over_q, flat[-B * H * d:].view(B, H, d), flat[H * d:][:B * H * d].view(B, H, d)):
        with pytest.raises(rswa.RswaError) as e:
            cache.append_kv_rope(rope, q, k, v, a)
        assert e.value.status == 1
    torch.cuda.synchronize()
    assert torch.equal(flat, before)
    check_ring(cache, states, n)
    # in place
    q1, k1 = q.contiguous(), k.contiguous()
    cache.qk_norm_rope(rope, q1, k1, q1, k1)
    check_rope(q1, q, rope.q_weight, [12] * B, rope, "q")
    check_rope(k1, k, rope.k_weight, [12] * B, rope, "k")
    q1 = q.contiguous()
    cache.append_kv_rope(rope, q1, k, v, q1)
    check_rope(q1, q, rope.q_weight, [12] * B, rope, "q")
    one = flat[:(H + 2 * Hkv) * d].view(1, H + 2 * Hkv, d)      # one row: beside its own key
    want = torch.empty(1, H, d, dtype=BF, device="cuda"), torch.empty(1, Hkv, d, dtype=BF, device="cuda")
    rswa.rswa_qk_norm_rope(rope, one[:, :H], one[:, H:H + Hkv], pos[:1], *want)
    rswa.rswa_qk_norm_rope(rope, one[:, :H], one[:, H:H + Hkv], pos[:1],
                           flat[:H * d].view(1, H, d), flat[H * d:(H + Hkv) * d].view(1, Hkv, d))
    assert torch.equal(one[:, :H], want[0]) and torch.equal(one[:, H:H + Hkv], want[1])
    assert cache.sync_status() == 0


# ---------------------------------------------------------------------------
# caches
# ---------------------------------------------------------------------------

def make_cache(rswa, m, t, n, H, Hkv, d, dtype, seed, cap=None):
    """A cache of sequences with prefixes m[b] and t[b] outputs, and their
    oracle states."""
    code = rswa.RSWA_F32 if dtype == torch.float32 else rswa.RSWA_BF16
    rows = sum(m) + sum(t)
    K, V = normal((rows, Hkv, d), seed, dtype), normal((rows, Hkv, d), seed + 1, dtype)
    cache = rswa.RswaCache(max(m) if cap is None else cap, n, H, d, len(m), code, kv_heads=Hkv)
    cache.prefill_varlen(None, K if rows else None, V if rows else None, None, m, t)
    states, at = [], 0
    for mb, tb in zip(m, t):
        sl = slice(at, at + mb + tb)
        states.append(oracle.prefill_cache(f64(K[sl]), f64(V[sl]), mb, n, tb))
        at += mb + tb
    return cache, states


def check_ring(cache, states, n):
    Ks, Vs = cache.slabs()
    for b, st in enumerate(states):
        assert cache.get_t(b) == st["t"]
        filled = sorted(oracle.ring_outputs(st["t"], n))
        for slab, name in ((Ks, "Kr"), (Vs, "Vr")):
            got = f64(slab[b, :, cache.m:]).transpose(1, 0, 2)
            np.testing.assert_array_equal(got[filled], st[name][filled])


@pytest.mark.parametrize("dtype,H,Hkv,d,rot,il", [
    (torch.bfloat16, 10, 10, 128, 128, False), (torch.bfloat16, 32, 8, 128, 64, True),
    (torch.bfloat16, 7, 1, 64, 64, False), (torch.float32, 6, 2, 64, 32, False),
    (torch.float32, 40, 1, 128, 128, True)])
@pytest.mark.parametrize("strided", [False, True])
def test_append_kv_rope(cuda_lib, dtype, H, Hkv, d, rot, il, strided):
    """Several steps over a wrapping ring: the queries, the stored keys and
    values and t_b of every step, and the decode step that follows."""
    rswa = cuda_lib
    m, t, n = [3, 0, 290], [0, 5, 9], 4
    cache, states = make_cache(rswa, m, t, n, H, Hkv, d, dtype, 20)
    qw, kw = weight(d, 21, dtype), weight(d, 22, dtype)
    rope = rswa.RswaRope(inv_freq(rot), qw, kw, interleaved=il)
    Ks, Vs = cache.slabs()
    for step in range(6):
        qkv = normal((3, H + 2 * Hkv, d), 30 + step, dtype)
        q, k, v = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
        if not strided:
            q, k, v = (x.contiguous() for x in (q, k, v))
        qo = torch.full((3, H, d), float("nan"), dtype=dtype, device="cuda")
        before = Ks.clone(), Vs.clone()
        cache.append_kv_rope(rope, q, k, v, qo)
        pos = [a + b for a, b in zip(m, t)]
        check_rope(qo, q, qw, pos, rope, "q")
        stored = torch.stack([Ks[b, :, cache.m + t[b] % n] for b in range(3)])
        check_rope(stored, k, kw, pos, rope, "k")
        for b in range(3):
            slot = cache.m + t[b] % n
            same(Vs[b, :, slot], f64(v[b]))
            for old, new in zip(before, (Ks, Vs)):         # nothing else was written
                old[b, :, slot] = new[b, :, slot]
            states[b] = oracle.append_kv(states[b], f64(stored[b]), f64(v[b]), n)
        assert torch.equal(before[0], Ks) and torch.equal(before[1], Vs)
        t = [x + 1 for x in t]
        o = torch.empty(3, H, d, dtype=dtype, device="cuda")
        cache.decode_step(qo, o)
        for b in range(3):
            ref, _ = oracle.decode_step(states[b], f64(qo[b]), n)
            err = np.abs(f64(o[b]) - ref)
            assert err.max() <= (1e-4 if dtype == torch.float32 else 2e-2)
    check_ring(cache, states, n)
    assert cache.sync_status() == 0


def test_qk_norm_rope_of_a_cache(cuda_lib):
    """Positions m_b + t_b + offsets; without offsets m_b + t_b + i; the same
    rows as with those positions given."""
    rswa = cuda_lib
    m, t, n, H, Hkv, d, N = [17, 0, 5], [3, 200, 0], 6, 4, 2, 128, 5
    cache, states = make_cache(rswa, m, t, n, H, Hkv, d, torch.bfloat16, 40)
    rope = rswa.RswaRope(inv_freq(d), weight(d, 41, torch.bfloat16), weight(d, 42, torch.bfloat16))
    qkv = normal((3 * N, H + 2 * Hkv, d), 43)
    q, k = qkv[:, :H], qkv[:, H:H + Hkv]
    off = torch.tensor([[0, 1, 1, 2, 7], [0, 0, 1, 2, 3], [4, 0, 0, 0, -2]], dtype=torch.int32).cuda()
    for offsets in (None, off):
        rel = torch.arange(N).expand(3, N) if offsets is None else off.cpu().long()
        pos = (torch.tensor(m)[:, None] + torch.tensor(t)[:, None] + rel).reshape(-1)
        a = torch.empty(3 * N, H, d, dtype=torch.bfloat16, device="cuda"), \
            torch.empty(3 * N, Hkv, d, dtype=torch.bfloat16, device="cuda")
        b = torch.empty_like(a[0]), torch.empty_like(a[1])
        cache.qk_norm_rope(rope, q, k, *a, offsets=offsets)
        rswa.rswa_qk_norm_rope(rope, q, k, pos.cuda(), *b)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        check_rope(a[0], q, rope.q_weight, pos.tolist(), rope, "q")
    check_ring(cache, states, n)


# ---------------------------------------------------------------------------
# tree attention
# ---------------------------------------------------------------------------

def random_tree(N, seed):
    g = np.random.default_rng(seed)
    return [-1 if i == 0 or g.random() < 0.1 else
            (i - 1 if g.random() < 0.4 else int(g.integers(max(0, i - 20), i)))
            for i in range(N)]


def check_tree(o, lse, q, k, v, state, parents, n, what, rows=None):
    """o, lse, q, k, v: one sequence's live rows."""
    dtype, d = q.dtype, q.shape[-1]
    H, Hkv = q.shape[1], k.shape[1]
    G = H // Hkv
    half = 2.0 ** -24 * (1 if dtype == torch.float32 else 2)
    qd = f64(q)
    ro, rl, seen = drafts.tree_attention(state, qd, f64(k), f64(v), parents, n)
    go, gl = f64(o), f64(lse)
    for i in range(len(parents)):
        K, V = seen[i]
        S = len(K)
        Kh, Vh = np.repeat(K, G, 1), np.repeat(V, G, 1)           # [S][H][d]
        logit = np.einsum("shd,hd->sh", Kh, qd[i]) / np.sqrt(d)
        p = np.exp(logit - rl[i])
        big = np.einsum("shd,hd->sh", np.abs(Kh), np.abs(qd[i])).max(0) / np.sqrt(d)
        rel = (d + 8) * half * big + 2 * S * half + 2.0 ** -21    # [H]
        assert np.isfinite(gl[i]).all() and np.isfinite(go[i]).all(), f"{what} node {i}"
        assert (np.abs(gl[i] - rl[i]) <= rel + 2 * half * (1 + np.abs(rl[i]))).all(), \
            f"{what} node {i}: lse {np.abs(gl[i] - rl[i]).max():.3g}, bound {rel.min():.3g}"
        mass = np.einsum("sh,shd->hd", p, np.abs(Vh))
        tol = (2 * rel[:, None] + half) * mass
        if dtype == torch.bfloat16:
            tol = tol + HALF[dtype] * (mass + np.abs(ro[i]))
        err = np.abs(go[i] - ro[i])
        assert (err <= tol).all(), f"{what} node {i}: {np.max(err / tol):.3g} of the bound"


def run_tree(rswa, m, t, n, H, Hkv, d, N, dtype, seed, counts=None, cap=None, std=1.0,
             parents=None):
    B = len(m)
    cache, states = make_cache(rswa, m, t, n, H, Hkv, d, dtype, seed, cap)
    q = normal((B, N, H, d), seed + 2, dtype, std)
    k, v = (normal((B, N, Hkv, d), seed + 3 + i, dtype) for i in range(2))
    par = parents or [random_tree(N, seed + b) for b in range(B)]
    o = torch.full((B, N, H, d), 7.0, dtype=dtype, device="cuda")
    lse = torch.full((B, N, H), 7.0, device="cuda")
    cnt = None if counts is None else torch.tensor(counts, dtype=torch.int32).cuda()
    live = [N] * B if counts is None else counts
    if counts is not None:                       # padding may hold anything
        for b in range(B):
            for x in (q, k, v):
                x[b, live[b]:] = float("nan")
    Ks, Vs = cache.slabs()
    before = Ks.clone(), Vs.clone()
    cache.decode_tree(q, k, v, torch.tensor(par, dtype=torch.int32).cuda(), o, lse, counts=cnt)
    assert cache.sync_status() == 0
    for b in range(B):
        c = live[b]
        check_tree(o[b, :c], lse[b, :c], q[b, :c], k[b, :c], v[b, :c], states[b], par[b][:c], n,
                   f"sequence {b}")
        assert (o[b, c:] == 7).all() and (lse[b, c:] == 7).all()
    assert torch.equal(before[0], Ks) and torch.equal(before[1], Vs)
    check_ring(cache, states, n)
    return cache, states, (q, k, v, par, o, lse)


BF, F32 = torch.bfloat16, torch.float32
TREE_CASES = [
    # m, t, n, H, Hkv, d, nodes, dtype
    ([0], [0], 8, 1, 1, 128, 1, BF),                      # only itself
    ([0], [0], 1, 2, 2, 128, 7, BF),                      # a window of one
    ([1], [0], 4, 2, 1, 128, 9, BF),
    ([288], [200], 128, 10, 10, 128, 16, BF),             # a page
    ([288], [1], 128, 10, 10, 128, 33, BF),
    ([127], [127], 127, 3, 3, 128, 31, BF),
    ([128], [128], 128, 3, 3, 128, 32, BF),
    ([129], [129], 129, 3, 3, 128, 64, BF),
    ([1000], [700], 300, 2, 2, 128, 65, BF),
    ([130], [40], 20, 2, 2, 128, 127, BF),
    ([130], [40], 20, 2, 2, 128, 128, BF),
    ([130], [40], 20, 2, 2, 128, 129, BF),
    ([260], [333], 77, 2, 1, 128, 200, BF),
    ([260], [333], 5, 1, 1, 128, 400, BF),
    ([100], [10], 128, 32, 8, 128, 16, BF),               # 64 rows a key head
    ([100], [300], 128, 32, 8, 128, 33, BF),              # 132 rows
    ([700], [300], 128, 32, 8, 128, 64, BF),              # 256 rows
    ([64], [300], 128, 12, 4, 128, 50, BF),               # groups of 3: 42 nodes a tile
    ([64], [300], 16, 20, 2, 128, 30, BF),                # groups of 10
    ([200], [20], 16, 130, 1, 128, 3, BF),                # more heads than a tile has rows
    ([200], [20], 16, 128, 1, 128, 3, BF),
    ([300], [20], 16, 100, 1, 128, 3, BF),
    ([288], [200], 128, 10, 10, 64, 16, BF),              # head_dim 64
    ([500], [60], 40, 8, 2, 64, 70, BF),
    ([260], [333], 77, 2, 1, 64, 200, BF),
    ([3000], [100], 64, 2, 2, 128, 20, BF),               # split over many CTAs
    ([5, 0, 300, 129], [0, 3, 500, 128], 128, 5, 5, 128, 12, BF),
    ([9] * 70, [12] * 70, 8, 2, 2, 128, 5, BF),
    ([300 + 11 * i for i in range(20)], [30 * i for i in range(20)], 128, 8, 2, 128, 24, BF),
    ([16], [20], 8, 1, 1, 64, 64, F32),
    ([288], [200], 128, 4, 2, 128, 16, F32),
    ([310, 0, 77], [30, 90, 0], 77, 4, 2, 64, 33, F32),
    ([260], [333], 77, 2, 1, 64, 150, F32),
]


@pytest.mark.parametrize("m,t,n,H,Hkv,d,N,dtype", TREE_CASES)
def test_decode_tree(cuda_lib, m, t, n, H, Hkv, d, N, dtype):
    run_tree(cuda_lib, m, t, n, H, Hkv, d, N, dtype, 50)


# A prefix capacity above 1200 keys takes small work to the tensor cores too.
WIDE = 1300


@pytest.mark.parametrize("m,t,n,H,Hkv,d,N,dtype", [c for c in TREE_CASES if c[7] is BF])
def test_decode_tree_with_room_in_the_cache(cuda_lib, m, t, n, H, Hkv, d, N, dtype):
    run_tree(cuda_lib, m, t, n, H, Hkv, d, N, dtype, 55, cap=max(m) + WIDE)


@pytest.mark.parametrize("dtype,cap", [(BF, None), (BF, 300 + WIDE), (F32, None)])
@pytest.mark.parametrize("H,Hkv,d,N", [(4, 4, 128, 40), (8, 2, 128, 70), (8, 2, 64, 70)])
def test_decode_tree_ragged_counts(cuda_lib, H, Hkv, d, N, dtype, cap):
    """Padded trees: rows past the count are left, whatever the padding holds;
    an empty sequence and a whole one among them, and all of them empty."""
    counts = [N, 0, 1, 17, N - 1, 33]
    m, t = [200, 10, 0, 129, 300, 5], [0, 4, 50, 140, 9, 64]
    run_tree(cuda_lib, m, t, 64, H, Hkv, d, N, dtype, 60, counts, cap)
    run_tree(cuda_lib, m[:2], t[:2], 64, H, Hkv, d, N, dtype, 61, [0, 0], cap)


@pytest.mark.parametrize("cap", [40, 40 + WIDE])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_tree_deep_chain_and_star(cuda_lib, d, cap):
    """Depth beyond the window (ancestors and the ring fall out of it), and all
    nodes at depth 0."""
    N = 150
    run_tree(cuda_lib, [40], [60], 48, 2, 2, d, N, BF, 70, cap=cap, parents=[list(range(-1, N - 1))])
    run_tree(cuda_lib, [40], [60], 48, 2, 2, d, N, BF, 71, cap=cap, parents=[[-1] * N])
    run_tree(cuda_lib, [40], [60], 48, 2, 2, d, N, BF, 72, cap=cap, parents=[[-1] + [0] * (N - 1)])


def test_decode_tree_1024_nodes(cuda_lib):
    run_tree(cuda_lib, [150], [100], 64, 1, 1, 128, 1024, BF, 73)


def test_decode_tree_a_prefix_capacity_with_room(cuda_lib):
    """Prefixes far below the capacity: tiles behind them hold zeros."""
    run_tree(cuda_lib, [10, 700, 0], [5, 0, 300], 100, 4, 2, 128, 20, BF, 74, cap=2000)


def test_decode_tree_large_logits(cuda_lib):
    """Logits of several hundred: the running maximum moves, nothing overflows."""
    run_tree(cuda_lib, [700], [200], 128, 4, 2, 128, 40, BF, 75, std=40.0)
    run_tree(cuda_lib, [300], [20], 16, 2, 2, 64, 20, F32, 76, std=40.0)


@pytest.mark.parametrize("d,dtype,cap", [(128, BF, None), (128, BF, 200 + WIDE), (64, BF, None),
                                         (64, BF, 200 + WIDE), (64, F32, None)])
def test_decode_tree_counts_its_keys(cuda_lib, d, dtype, cap):
    """q = 0 weighs every visible key alike, and with it exactly: lse is the
    logarithm of their number, and with values 1 for the tree's nodes and 0 in
    the cache o is the share of ancestors."""
    rswa = cuda_lib
    m, t, n, H, N = 200, 90, 50, 2, 140
    cache, states = make_cache(rswa, [m], [t], n, H, H, d, dtype, 80, cap)
    Ks, Vs = cache.slabs()
    Vs.zero_()
    cache.set_t([t])
    par = random_tree(N, 81)
    q = torch.zeros(1, N, H, d, dtype=dtype, device="cuda")
    k = normal((1, N, H, d), 82, dtype)
    v = torch.ones(1, N, H, d, dtype=dtype, device="cuda")
    o, lse = torch.empty_like(q), torch.empty(1, N, H, device="cuda")
    cache.decode_tree(q, k, v, torch.tensor([par], dtype=torch.int32).cuda(), o, lse)
    for i in range(N):
        up = drafts.chain(par, i)
        here = t + len(up) - 1
        keys = m + (t - max(0, here - n + 1) if here - n + 1 < t else 0) + len(up[:n])
        assert abs(lse[0, i, 0].item() - np.log(keys)) <= 2.0 ** -20
        share = len(up[:n]) / keys
        assert (o[0, i].double() - share).abs().max().item() <= share * (HALF[dtype] + 2.0 ** -20)


def test_decode_tree_bad_parents_and_counts(cuda_lib):
    """Parents that do not come before their child and counts out of range set
    the flag; the parent counts as -1, the count as the nearest in range."""
    rswa = cuda_lib
    m, t, n, H, d, N = [50, 60], [5, 6], 16, 2, 128, 12
    for dtype, cap in ((BF, None), (BF, 60 + WIDE), (F32, None)):
        cache, states = make_cache(rswa, m, t, n, H, H, d, dtype, 85, cap)
        q, k, v = (normal((2, N, H, d), 86 + i, dtype) for i in range(3))
        good = [random_tree(N, 88), random_tree(N, 89)]
        good[0][3], good[0][4], good[1][5], good[1][11] = -1, -1, -1, -1
        bad = [list(x) for x in good]
        bad[0][3], bad[0][4], bad[1][5], bad[1][11] = 3, 2 ** 31 - 1, -2, 7000
        for par, counts, status in ((bad, None, RSWA_EDEVICE), (good, [N + 1, -3], RSWA_EDEVICE),
                                    (good, None, 0)):
            o = torch.full_like(q, 7)
            lse = torch.full((2, N, H), 7.0, device="cuda")
            cnt = None if counts is None else torch.tensor(counts, dtype=torch.int32).cuda()
            cache.decode_tree(q, k, v, torch.tensor(par, dtype=torch.int32).cuda(), o, lse, counts=cnt)
            assert cache.sync_status() == status
            assert cache.sync_status() == 0
            for b in range(2):
                if counts is not None and counts[b] < 0:
                    assert (o[b] == 7).all() and (lse[b] == 7).all()
                    continue
                check_tree(o[b], lse[b], q[b], k[b], v[b], states[b], good[b], n, f"{dtype} {b}")


def test_decode_tree_equals_block_on_a_chain(cuda_lib):
    """A chain of drafts is a block of outputs."""
    rswa = cuda_lib
    m, t, n, H, Hkv, d, N = [290], [40], 128, 8, 2, 128, 20
    cache, states = make_cache(rswa, m, t, n, H, Hkv, d, BF, 90)
    q, k, v = normal((1, N, H, d), 91), normal((1, N, Hkv, d), 92), normal((1, N, Hkv, d), 93)
    par = torch.arange(-1, N - 1, dtype=torch.int32)[None].cuda()
    o, ob = torch.empty_like(q), torch.empty_like(q)
    lse, lb = torch.empty(1, N, H, device="cuda"), torch.empty(1, N, H, device="cuda")
    cache.decode_tree(q, k, v, par, o, lse)
    cache.decode_block(q, k, v, ob, lb)
    assert (lse - lb).abs().max().item() <= 1e-4
    assert (o - ob).abs().max().item() <= 2e-2
    assert cache.get_t(0) == t[0] + N


@pytest.mark.parametrize("H,Hkv,d,dtype", [(2, 2, 128, BF), (8, 2, 64, BF), (96, 1, 128, BF), (2, 1, 64, F32)])
def test_decode_tree_deepest_chain(cuda_lib, H, Hkv, d, dtype):
    """1024 nodes in one chain inside the window (every node walks to the root):
    a block of 1024 outputs.  Both are off by the bounds above, with sum |q k| at
    most the product of the lengths and |o| at most the largest value."""
    rswa = cuda_lib
    m, t, n, N = [150], [900], 2000, 1024
    cache, _ = make_cache(rswa, m, t, n, H, Hkv, d, dtype, 500)
    q, k, v = normal((1, N, H, d), 501, dtype), normal((1, N, Hkv, d), 502, dtype), normal((1, N, Hkv, d), 503, dtype)
    par = torch.arange(-1, N - 1, dtype=torch.int32)[None].cuda()
    o, ob = torch.empty_like(q), torch.empty_like(q)
    lse, lb = torch.empty(1, N, H, device="cuda"), torch.empty(1, N, H, device="cuda")
    cache.decode_tree(q, k, v, par, o, lse)
    cache.decode_block(q, k, v, ob, lb)
    assert cache.sync_status() == 0
    logit = (q.float().norm(dim=-1).max() * k.float().norm(dim=-1).max()).item() / d ** 0.5
    half = 2.0 ** -24 * (1 if dtype is F32 else 2)
    rel = (d + 8) * half * logit + 2 * (m[0] + n) * half + 2.0 ** -21
    assert (lse - lb).abs().max().item() <= 2 * rel + 4 * half * (1 + lb.abs().max().item())
    big = v.float().abs().max().item()
    tol = 2 * (2 * rel + half + (2 * HALF[dtype] if dtype is BF else 0)) * big
    assert (o.float() - ob.float()).abs().max().item() <= tol
    assert cache.get_t(0) == t[0] + N


def test_decode_tree_refusals(cuda_lib):
    rswa = cuda_lib
    H, Hkv, d, N = 4, 2, 128, 6
    cache, _ = make_cache(rswa, [9], [0], 8, H, Hkv, d, BF, 95)
    q, k, v = normal((1, N, H, d), 96), normal((1, N, Hkv, d), 97), normal((1, N, Hkv, d), 98)
    par = torch.full((1, N), -1, dtype=torch.int32, device="cuda")
    o, lse = torch.empty_like(q), torch.empty(1, N, H, device="cuda")
    cnt = torch.ones(1, dtype=torch.int32, device="cuda")
    ws = cache.tree_workspace(N)
    ok = dict(q=q, k=k, v=v, parents=par, o=o, lse=lse, counts=cnt, workspace=ws)
    cache.decode_tree(**ok)
    cache.decode_tree(**dict(ok, lse=None, counts=None, workspace=None))
    for bad in [dict(q=q.float()), dict(k=k[:, :5].contiguous()), dict(v=v.transpose(1, 2)),
                dict(parents=par.long()), dict(parents=par[:, :5].contiguous()),
                dict(o=o[:, :, :2].contiguous()), dict(lse=lse.double()), dict(counts=cnt.long()),
                dict(counts=cnt.cpu()), dict(workspace=ws[:0]), dict(workspace=ws[16:])]:
        with pytest.raises((ValueError, rswa.RswaError)):
            cache.decode_tree(**dict(ok, **bad))
    big = torch.zeros(1, 1025, H, d, dtype=BF, device="cuda")
    bk = torch.zeros(1, 1025, Hkv, d, dtype=BF, device="cuda")
    with pytest.raises(rswa.RswaError):
        cache.decode_tree(big, bk, bk, torch.full((1, 1025), -1, dtype=torch.int32).cuda(),
                          torch.empty_like(big), workspace=ws)
    lib, h = rswa.load(), cache.handle
    p = lambda x: x.data_ptr()                                         # noqa: E731
    good = [p(q), p(k), p(v), p(par), None, N, p(o), None, p(ws), ws.numel(), None]
    for at, value, status in ((0, None, 1), (0, p(q) + 2, 1), (1, None, 1), (2, p(v) + 8, 1),
                              (3, None, 1), (3, p(par) + 2, 1), (4, p(cnt) + 1, 1), (5, 0, 1),
                              (5, 1025, 1), (6, None, 1), (6, p(o) + 4, 1), (7, p(lse) + 2, 1),
                              (8, None, 1), (8, p(ws) + 16, 1), (9, ws.numel() - 1, 2)):
        args = list(good)
        args[at] = value
        assert lib.rswa_decode_tree(h, *args) == status, at
    rswa.rswa_debug_fail_next_cuda(1)
    assert lib.rswa_decode_tree(h, *good) == 5
    assert lib.rswa_decode_tree(h, *good) == 0
    assert cache.sync_status() == 0


def test_decode_tree_refuses_results_over_inputs(cuda_lib):
    """o, lse or the workspace over what other CTAs still read: refused, with
    nothing written."""
    rswa = cuda_lib
    B, H, Hkv, d, N = 2, 4, 2, 64, 6
    cache, _ = make_cache(rswa, [9] * B, [2] * B, 8, H, Hkv, d, BF, 440)
    need = rswa.rswa_decode_tree_workspace(cache.handle, N)
    mem = normal((1 << 20,), 441)
    base, before = mem.data_ptr(), mem.clone()
    assert base % 256 == 0 and need <= 4096
    qb, kb = B * N * H * d * 2, B * N * Hkv * d * 2
    at = dict(q=0, k=0x10000, v=0x20000, par=0x30000, cnt=0x40000, o=0x50000, lse=0x60000, ws=0x70000)
    for name, x in (("par", [-1] * (B * N)), ("cnt", [N, N])):
        x = torch.tensor(x, dtype=torch.int32).cuda().view(BF)
        mem[at[name] // 2:][:x.numel()] = x
    before = mem.clone()

    def call(**kw):
        p = {x: base + y for x, y in dict(at, **kw).items()}
        return rswa.load().rswa_decode_tree(cache.handle, p["q"], p["k"], p["v"], p["par"], p["cnt"], N,
                                            p["o"], p["lse"], p["ws"], need, None)

    for bad in (dict(o=16), dict(o=qb - 16), dict(q=16, o=0), dict(o=at["k"]), dict(o=at["k"] - qb + 16),
                dict(o=at["v"] + kb - 16), dict(o=at["par"]), dict(o=at["cnt"]), dict(lse=0),
                dict(lse=at["k"] + kb - 4), dict(lse=at["o"] + qb - 4), dict(lse=at["par"]),
                dict(ws=0), dict(ws=at["v"]), dict(ws=at["par"]), dict(ws=at["cnt"]), dict(ws=at["o"]),
                dict(ws=at["lse"]), dict(o=at["ws"]), dict(lse=at["ws"] + need - 4)):
        assert call(**bad) == 1, bad
    torch.cuda.synchronize()
    assert torch.equal(mem.view(torch.int16), before.view(torch.int16))
    assert call(k=at["q"], v=at["q"]) == 0                 # inputs may be one tensor
    assert call(o=at["k"] + kb, lse=at["o"] + qb) == 0     # side by side
    assert cache.sync_status() == 0


@pytest.mark.parametrize("m,H,Hkv,d,N,dtype", [(200, 4, 2, 64, 9, F32), (200, 4, 4, 128, 5, BF),
                                               (3000, 2, 2, 128, 20, BF), (1500, 32, 8, 128, 60, BF),
                                               (400, 4, 2, 64, 300, BF)])
def test_decode_tree_in_place(cuda_lib, m, H, Hkv, d, N, dtype):
    """o may be q, with NaN in dead nodes: the same bits (CUDA cores; one query
    tile and pairs, cut and whole)."""
    rswa = cuda_lib
    B, n = 40, 48
    ms, ts = [max(0, m - 31 * b) for b in range(B)], [5 * b for b in range(B)]
    cache, _ = make_cache(rswa, ms, ts, n, H, Hkv, d, dtype, 445)
    for B_live in (B, 1):
        counts = torch.tensor([(N - b % 3 if b < B_live else 0) for b in range(B)], dtype=torch.int32).cuda()
        q, k, v = normal((B, N, H, d), 446, dtype), normal((B, N, Hkv, d), 447, dtype), normal((B, N, Hkv, d), 448, dtype)
        dead = torch.arange(N, device="cuda") >= counts[:, None]
        q[dead] = float("nan")
        par = torch.tensor([random_tree(N, 449 + b) for b in range(B)], dtype=torch.int32).cuda()
        o, lse, l2 = torch.full_like(q, float("nan")), torch.zeros(B, N, H, device="cuda"), torch.zeros(B, N, H, device="cuda")
        cache.decode_tree(q, k, v, par, o, lse, counts=counts)
        for _ in range(3):
            x = q.clone()
            cache.decode_tree(x, k, v, par, x, l2, counts=counts)
            assert torch.equal(x[~dead], o[~dead]) and torch.equal(l2, lse)
            assert torch.isnan(x[dead]).all()
    assert cache.sync_status() == 0


def test_decode_tree_ignores_what_is_no_key(cuda_lib):
    """NaN in prefix rows past m_b and in ring slots that hold no output yet (a
    caller's own writes into the slabs) does not reach any row."""
    rswa = cuda_lib
    m, t, n, H, d, N = [200, 5], [3, 0], 40, 2, 128, 20
    for dtype, cap in ((BF, None), (BF, 200 + WIDE), (F32, None)):
        cache, states = make_cache(rswa, m, t, n, H, H, d, dtype, 240, cap)
        for slab in cache.slabs():
            for b in range(2):
                slab[b, :, m[b]:cache.m] = float("nan")
                slab[b, :, cache.m + t[b]:] = float("nan")
        cache.set_t(t)
        q, k, v = (normal((2, N, H, d), 241 + i, dtype) for i in range(3))
        par = [random_tree(N, 244), random_tree(N, 245)]
        o, lse = torch.empty_like(q), torch.empty(2, N, H, device="cuda")
        cache.decode_tree(q, k, v, torch.tensor(par, dtype=torch.int32).cuda(), o, lse)
        for b in range(2):
            check_tree(o[b], lse[b], q[b], k[b], v[b], states[b], par[b], n, f"{dtype} {b}")


def test_decode_tree_wait_runs_out_then_recovers(cuda_lib):
    """The tensor-core kernel with its waits bounded to 1 ns gives up, reports
    RSWA_EDEVICE and leaves the cache usable: after rswa_cache_set_t the next
    call is right (few units cut into many parts, a pair of query tiles, a CTA
    for every unit)."""
    rswa = cuda_lib
    for m, H, Hkv, N, cap in ((3000, 2, 2, 20, None), (1500, 8, 2, 64, None), (100, 8, 2, 200, 500)):
        cache, states = make_cache(rswa, [m], [70], 64, H, Hkv, 128, BF, 250, cap)
        q, k, v = normal((1, N, H, 128), 251), normal((1, N, Hkv, 128), 252), normal((1, N, Hkv, 128), 253)
        par = [random_tree(N, 254)]
        dev = torch.tensor(par, dtype=torch.int32).cuda()
        o, lse = torch.empty_like(q), torch.empty(1, N, H, device="cuda")
        rswa.rswa_debug_set_wait_limit_ns(1)
        try:
            cache.decode_tree(q, k, v, dev, o, lse)
        finally:
            rswa.rswa_debug_set_wait_limit_ns(0)
        assert cache.sync_status() == RSWA_EDEVICE
        assert cache.sync_status() == 0
        cache.set_t([70])                           # the documented way back
        cache.decode_tree(q, k, v, dev, o, lse)
        assert cache.sync_status() == 0
        check_tree(o[0], lse[0], q[0], k[0], v[0], states[0], par[0], 64, "after the timeout")


def test_decode_tree_workspaces(cuda_lib):
    """A workspace for more nodes serves fewer; what it holds does not matter."""
    rswa = cuda_lib
    m, t, n, H, Hkv, d = [1400], [30], 64, 8, 2, 128
    cache, states = make_cache(rswa, m, t, n, H, Hkv, d, BF, 260)
    ws = cache.tree_workspace(300)
    sizes = [rswa.rswa_decode_tree_workspace(cache.handle, x) for x in (1, 5, 32, 33, 64, 65, 300, 1024)]
    assert sizes == sorted(sizes) and sizes[0] >= 256
    for N in (300, 40, 3, 32):
        ws.fill_(0xff)
        q, k, v = normal((1, N, H, d), 261), normal((1, N, Hkv, d), 262), normal((1, N, Hkv, d), 263)
        par = [random_tree(N, 264)]
        o, lse = torch.empty_like(q), torch.empty(1, N, H, device="cuda")
        cache.decode_tree(q, k, v, torch.tensor(par, dtype=torch.int32).cuda(), o, lse, workspace=ws)
        check_tree(o[0], lse[0], q[0], k[0], v[0], states[0], par[0], n, f"{N} nodes")


@pytest.mark.parametrize("m,n,B,H,Hkv,d,most,fewer", [
    (704, 128, 1, 10, 10, 128, 257, (256, 40)), (800, 128, 2, 10, 10, 128, 300, (256, 129)),
    (1000, 128, 3, 64, 8, 64, 40, (32, 33)), (900, 100, 1, 32, 8, 128, 193, (192, 65)),
    (250, 200, 1, 10, 10, 128, 800, (768, 257)), (100, 8, 1, 2, 2, 64, 1024, (300, 1))])
def test_decode_tree_workspace_serves_fewer_nodes(cuda_lib, m, n, B, H, Hkv, d, most, fewer):
    """Shapes where more nodes take the launch form that cuts no unit, and uses no
    workspace, and fewer nodes, of fewer units, the one that does."""
    rswa = cuda_lib
    cache, states = make_cache(rswa, [m] * B, [30] * B, n, H, Hkv, d, BF, 420)
    sizes = [rswa.rswa_decode_tree_workspace(cache.handle, x) for x in range(1, 1025)]
    assert sizes == sorted(sizes) and sizes[0] >= 256
    ws = cache.tree_workspace(most)
    ws.fill_(0xff)
    for N in (most,) + fewer:
        q, k, v = normal((B, N, H, d), 421), normal((B, N, Hkv, d), 422), normal((B, N, Hkv, d), 423)
        par = [random_tree(N, 424 + b) for b in range(B)]
        dev = torch.tensor(par, dtype=torch.int32).cuda()
        o, lse = torch.zeros_like(q), torch.zeros(B, N, H, device="cuda")
        cache.decode_tree(q, k, v, dev, o, lse, workspace=ws)
        assert cache.sync_status() == 0
        c = min(N, 40)                           # nodes come before their children
        check_tree(o[-1, :c], lse[-1, :c], q[-1, :c], k[-1, :c], v[-1, :c], states[-1], par[-1][:c],
                   n, f"{N} nodes")
        o2, l2 = torch.zeros_like(o), torch.zeros_like(lse)
        cache.decode_tree(q, k, v, dev, o2, l2)
        assert torch.equal(o, o2) and torch.equal(lse, l2)


def test_decode_tree_back_to_back_and_after_other_calls(cuda_lib):
    """Calls queued without a wait, each on inputs of its own, between appends
    and decode steps (programmatic dependents that start early)."""
    rswa = cuda_lib
    m, n, H, Hkv, d, N = [1300, 40], 32, 8, 2, 128, 33
    cache, states = make_cache(rswa, m, [10, 0], n, H, Hkv, d, BF, 270)
    par = [random_tree(N, 271), random_tree(N, 272)]
    dev = torch.tensor(par, dtype=torch.int32).cuda()
    rounds = []
    torch.cuda.synchronize()
    for r in range(4):
        q, k, v = normal((2, N, H, d), 280 + r), normal((2, N, Hkv, d), 290 + r), normal((2, N, Hkv, d), 300 + r)
        q1, k1, v1 = normal((2, H, d), 310 + r), normal((2, Hkv, d), 320 + r), normal((2, Hkv, d), 330 + r)
        o, lse, o1 = torch.empty_like(q), torch.empty(2, N, H, device="cuda"), torch.empty_like(q1)
        rounds.append((q, k, v, q1, k1, v1, o, lse, o1))
    torch.cuda.synchronize()
    for q, k, v, q1, k1, v1, o, lse, o1 in rounds:
        cache.decode_tree(q, k, v, dev, o, lse)
        cache.decode_step_fused(q1, k1, v1, o1)
    for r, (q, k, v, q1, k1, v1, o, lse, o1) in enumerate(rounds):
        for b in range(2):
            check_tree(o[b], lse[b], q[b], k[b], v[b], states[b], par[b], n, f"round {r}")
            states[b], ref, _ = oracle.decode_step_fused(states[b], f64(q1[b]), f64(k1[b]), f64(v1[b]), n)
            assert np.abs(f64(o1[b]) - ref).max() <= 2e-2
    check_ring(cache, states, n)
    assert cache.sync_status() == 0


@pytest.mark.parametrize("H,Hkv,N", [(2, 2, 12), (8, 2, 60)])
def test_decode_tree_after_commits_that_move_the_plan(cuda_lib, H, Hkv, N):
    """Commits and trees queued without a wait while t_b crosses tile boundaries
    of the ring: what a tree call reads before its dependency wait is stale."""
    rswa = cuda_lib
    m, t, n, d, P, rounds = [1300, 700, 20], [100, 120, 0], 300, 128, 6, 50
    cache, states = make_cache(rswa, m, t, n, H, Hkv, d, BF, 340)
    par = [random_tree(N, 341 + b) for b in range(3)]
    dev = torch.tensor(par, dtype=torch.int32).cuda()
    path = torch.tensor([[0, 1, 3, 5, 7, 9]] * 3, dtype=torch.int32).cuda()
    accs = [[6, 5, 6 if r % 2 else 0] for r in range(rounds)]
    accd = [torch.tensor(x, dtype=torch.int32).cuda() for x in accs]
    k, v = normal((3, N, Hkv, d), 344), normal((3, N, Hkv, d), 345)
    q = normal((3, N, H, d), 346)
    out = [(torch.empty_like(q), torch.empty(3, N, H, device="cuda")) for _ in range(rounds)]
    cache.decode_tree(q, k, v, dev, *out[0])
    torch.cuda.synchronize()
    for r in range(rounds):
        cache.commit_tree(k, v, path, accd[r])
        cache.decode_tree(q, k, v, dev, *out[r])
    assert cache.sync_status() == 0
    for r in range(rounds):
        for b in range(3):
            states[b] = drafts.commit_tree(states[b], f64(k[b]), f64(v[b]), path[b, :accs[r][b]].tolist(), n)
            if r % 7 == 0 or any(states[b]["t"] - x <= 6 for x in (128, 256)):
                check_tree(out[r][0][b], out[r][1][b], q[b], k[b], v[b], states[b], par[b], n, f"round {r}")
    check_ring(cache, states, n)


@pytest.mark.parametrize("B,H,Hkv,N,d", [(40, 6, 6, 20, 128), (40, 12, 3, 60, 128), (60, 4, 4, 9, 64)])
def test_decode_tree_many_units(cuda_lib, B, H, Hkv, N, d):
    """More units than SMs: units cut between two CTAs and joined by the last of
    them, call after call on the same counters, and the same bits every time;
    then a wait that runs out, and the way back."""
    rswa = cuda_lib
    g = np.random.default_rng(350)
    m, t = [int(x) for x in g.integers(0, 700, B)], [int(x) for x in g.integers(0, 150, B)]
    counts = [int(x) for x in g.integers(0, N + 1, B)]
    cache, states = make_cache(rswa, m, t, 100, H, Hkv, d, BF, 351, 1400)
    q, k, v = normal((B, N, H, d), 352), normal((B, N, Hkv, d), 353), normal((B, N, Hkv, d), 354)
    par = [random_tree(N, 355 + b) for b in range(B)]
    dev = torch.tensor(par, dtype=torch.int32).cuda()
    cnt = torch.tensor(counts, dtype=torch.int32).cuda()
    outs = []
    for _ in range(6):
        outs.append((torch.zeros_like(q), torch.zeros(B, N, H, device="cuda")))
        cache.decode_tree(q, k, v, dev, *outs[-1], counts=cnt)
    assert cache.sync_status() == 0
    o, lse = outs[0]
    for o2, l2 in outs[1:]:
        assert torch.equal(o, o2) and torch.equal(lse, l2)
    for b in list(range(0, B, 7)) + [B - 1]:
        c = counts[b]
        check_tree(o[b, :c], lse[b, :c], q[b, :c], k[b, :c], v[b, :c], states[b], par[b][:c], 100, f"{b}")
    rswa.rswa_debug_set_wait_limit_ns(1)
    try:
        cache.decode_tree(q, k, v, dev, torch.zeros_like(q), torch.zeros_like(lse), counts=cnt)
    finally:
        rswa.rswa_debug_set_wait_limit_ns(0)
    assert cache.sync_status() == RSWA_EDEVICE
    cache.set_t(t)
    o2, l2 = torch.zeros_like(q), torch.zeros_like(lse)
    cache.decode_tree(q, k, v, dev, o2, l2, counts=cnt)
    assert cache.sync_status() == 0
    assert torch.equal(o, o2) and torch.equal(lse, l2)


@pytest.mark.parametrize("B,H,Hkv,N,d", [(60, 12, 3, 60, 128), (40, 8, 2, 100, 128), (40, 4, 4, 200, 64),
                                         (40, 4, 4, 300, 128), (20, 64, 8, 17, 64)])
def test_decode_tree_many_pairs(cuda_lib, B, H, Hkv, N, d):
    """As many units of two query tiles as SMs or more (one unit or two a key
    head, some of them with one tile's rows only): the same bits call after call
    and in a graph, and a decode step after them as on a cache that saw none."""
    rswa = cuda_lib
    g = np.random.default_rng(360)
    m, t = [int(x) for x in g.integers(0, 500, B)], [int(x) for x in g.integers(0, 150, B)]
    counts = [int(x) for x in g.integers(0, N + 1, B)]
    counts[0], counts[1], m[2], t[2] = N, 0, 0, 0
    cache, states = make_cache(rswa, m, t, 100, H, Hkv, d, BF, 361, 600)
    other, _ = make_cache(rswa, m, t, 100, H, Hkv, d, BF, 361, 600)
    q, k, v = normal((B, N, H, d), 362), normal((B, N, Hkv, d), 363), normal((B, N, Hkv, d), 364)
    par = [random_tree(N, 365 + b) for b in range(B)]
    dev = torch.tensor(par, dtype=torch.int32).cuda()
    cnt = torch.tensor(counts, dtype=torch.int32).cuda()
    o, lse = torch.zeros_like(q), torch.zeros(B, N, H, device="cuda")
    o2, l2 = torch.zeros_like(o), torch.zeros_like(lse)
    cache.decode_tree(q, k, v, dev, o, lse, counts=cnt)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(4):
            cache.decode_tree(q, k, v, dev, o2, l2, counts=cnt)
    for _ in range(3):
        o2.zero_()
        l2.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, o2) and torch.equal(lse, l2)
    assert cache.sync_status() == 0
    for b in [0, 1, 2] + list(range(3, B, 9)):
        c = counts[b]
        check_tree(o[b, :c], lse[b, :c], q[b, :c], k[b, :c], v[b, :c], states[b], par[b][:c], 100, f"{b}")
        assert not o[b, c:].any()
    q1, k1, v1 = normal((B, H, d), 370), normal((B, Hkv, d), 371), normal((B, Hkv, d), 372)
    steps = torch.empty_like(q1), torch.empty_like(q1)
    for c, out in zip((cache, other), steps):
        c.decode_step_fused(q1, k1, v1, out)
        assert c.sync_status() == 0
    assert torch.equal(*steps)


@pytest.mark.parametrize("H,Hkv,N,d,n", [(2, 2, 21, 128, 40), (4, 2, 50, 64, 40), (8, 2, 70, 128, 33)])
def test_decode_tree_sources_meet_inside_a_tile(cuda_lib, H, Hkv, N, d, n):
    """Prefix, ring and nodes that end before, at and past multiples of 16 and of
    128; NaN in every row of the slabs that is no key, and in dead nodes."""
    rswa = cuda_lib
    g = np.random.default_rng(400)
    m = [x for x in (0, 1, 15, 16, 17, 95, 96, 111, 112, 113, 127, 128, 129, 144) for _ in range(4)]
    t = [x for _ in range(14) for x in (0, 16, 31, 3 * n + 5)]
    B = len(m)
    cache, states = make_cache(rswa, m, t, n, H, Hkv, d, BF, 401, 147)
    Ks, Vs = cache.slabs()
    rows = torch.arange(147 + n, device="cuda")
    for b in range(B):
        dead = (rows >= m[b]) & (rows < 147) | (rows >= 147 + min(n, t[b]))
        Ks[b, :, dead] = float("nan")
        Vs[b, :, dead] = float("nan")
    counts = [int(x) for x in g.choice([1, 15, 16, 17, N - 1, N], B)]
    q, k, v = normal((B, N, H, d), 402), normal((B, N, Hkv, d), 403), normal((B, N, Hkv, d), 404)
    for b in range(B):
        for x in (q, k, v):
            x[b, counts[b]:] = float("nan")
    par = [random_tree(N, 405 + b) for b in range(B)]
    o, lse = torch.zeros_like(q), torch.zeros(B, N, H, device="cuda")
    cache.decode_tree(q, k, v, torch.tensor(par, dtype=torch.int32).cuda(), o, lse,
                      counts=torch.tensor(counts, dtype=torch.int32).cuda())
    assert cache.sync_status() == 0
    for b in range(B):
        c = counts[b]
        check_tree(o[b, :c], lse[b, :c], q[b, :c], k[b, :c], v[b, :c], states[b], par[b][:c], n, f"{b}")
        assert not o[b, c:].any() and not lse[b, c:].any()


def test_decode_tree_many_pairs_wait_runs_out_then_recovers(cuda_lib):
    """Units whose CTAs meet on the cache's counters: cleared by set_t."""
    rswa = cuda_lib
    B, H, Hkv, N, d = 60, 12, 3, 60, 128
    m, t = [100 + 9 * b for b in range(B)], [3 * b for b in range(B)]
    cache, _ = make_cache(rswa, m, t, 100, H, Hkv, d, BF, 390, 700)
    q, k, v = normal((B, N, H, d), 391), normal((B, N, Hkv, d), 392), normal((B, N, Hkv, d), 393)
    dev = torch.tensor([random_tree(N, 394 + b) for b in range(B)], dtype=torch.int32).cuda()
    want = torch.zeros_like(q), torch.zeros(B, N, H, device="cuda")
    cache.decode_tree(q, k, v, dev, *want)
    assert cache.sync_status() == 0
    for _ in range(3):
        rswa.rswa_debug_set_wait_limit_ns(1)
        try:
            cache.decode_tree(q, k, v, dev, torch.zeros_like(q))
        finally:
            rswa.rswa_debug_set_wait_limit_ns(0)
        assert cache.sync_status() == RSWA_EDEVICE
        cache.set_t(t)
        got = torch.zeros_like(q), torch.zeros(B, N, H, device="cuda")
        cache.decode_tree(q, k, v, dev, *got)
        assert cache.sync_status() == 0
        assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def arrivals(cache, B, H):
    """The cache's arrival counters, [B][H]: the last words before the keys."""
    keys = cache.slabs()[0].data_ptr() - cache.buf.data_ptr()
    return cache.buf[keys - -(-4 * B * H // 256) * 256:][:4 * B * H].view(torch.int32)


@pytest.mark.parametrize("B,H,Hkv,N,d,m", [(60, 12, 3, 60, 128, 300), (160, 8, 1, 20, 64, 200)])
def test_set_t_clears_the_counters_that_joins_meet_on(cuda_lib, B, H, Hkv, N, d, m):
    """The counters are zero after a call whose CTAs join cut units; words that a
    call which gave up may have left there are cleared by set_t, and the next
    call has the same bits."""
    rswa = cuda_lib
    ms, ts = [m + 9 * b for b in range(B)], [3 * b % 110 for b in range(B)]
    cache, states = make_cache(rswa, ms, ts, 100, H, Hkv, d, BF, 460, m + 9 * B)
    q, k, v = normal((B, N, H, d), 461), normal((B, N, Hkv, d), 462), normal((B, N, Hkv, d), 463)
    par = [random_tree(N, 464 + b) for b in range(B)]
    dev = torch.tensor(par, dtype=torch.int32).cuda()
    want = torch.zeros_like(q), torch.zeros(B, N, H, device="cuda")
    cache.decode_tree(q, k, v, dev, *want)
    assert cache.sync_status() == 0
    cnt = arrivals(cache, B, H)
    assert not cnt.any()
    for left in (1, 2, 7):
        cnt.fill_(left)
        cache.set_t(ts)
        assert not cnt.any()
        got = torch.zeros_like(q), torch.zeros(B, N, H, device="cuda")
        cache.decode_tree(q, k, v, dev, *got)
        assert cache.sync_status() == 0 and not cnt.any()
        assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    for b in (0, B // 2, B - 1):
        check_tree(want[0][b], want[1][b], q[b], k[b], v[b], states[b], par[b], 100, f"{b}")


@pytest.mark.parametrize("live", [{7: 20}, {0: 20, 159: 17}, {3: 20, 80: 1, 81: 19}, {158: 33}, {}])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_tree_few_live_sequences_of_many(cuda_lib, live, d):
    """A launch of pairs planned for 160 units of which a few are live: each is
    cut into many parts, which the CTA that arrives last joins alone."""
    rswa = cuda_lib
    B, H, N, n = 160, 8, 33, 100
    m, t = [6000 - 500 * (b % 3) if b in live else 0 for b in range(B)], [70 + b if b in live else 0 for b in range(B)]
    cache, states = make_cache(rswa, m, t, n, H, 1, d, BF, 470, 6000)
    counts = [live.get(b, 0) for b in range(B)]
    q, k, v = normal((B, N, H, d), 471), normal((B, N, 1, d), 472), normal((B, N, 1, d), 473)
    for b in range(B):
        for x in (q, k, v):
            x[b, counts[b]:] = float("nan")
    par = [random_tree(N, 474 + b) for b in range(B)]
    dev = torch.tensor(par, dtype=torch.int32).cuda()
    cnt = torch.tensor(counts, dtype=torch.int32).cuda()
    outs = [(torch.full_like(q, 7.0), torch.full((B, N, H), 7.0, device="cuda")) for _ in range(5)]
    o, lse = outs[0]
    for o2, l2 in outs:
        cache.decode_tree(q, k, v, dev, o2, l2, counts=cnt)
        assert cache.sync_status() == 0 and not arrivals(cache, B, H).any()
        assert torch.equal(o, o2) and torch.equal(lse, l2)
    for b, c in live.items():
        check_tree(o[b, :c], lse[b, :c], q[b, :c], k[b, :c], v[b, :c], states[b], par[b][:c], n, f"{b}")
    for b in range(B):
        assert (o[b, counts[b]:] == 7).all() and (lse[b, counts[b]:] == 7).all()


@pytest.mark.parametrize("B,H,Hkv,N,d", [(2, 10, 10, 40, 128), (2, 8, 2, 60, 64), (40, 16, 4, 60, 128)])
def test_decode_tree_output_at_16_bytes(cuda_lib, B, H, Hkv, N, d):
    """o 16 and not 32 bytes aligned, lse 4: the same bits."""
    rswa = cuda_lib
    cache, _ = make_cache(rswa, [300 + 7 * b for b in range(B)], [90 + b for b in range(B)], 64, H, Hkv, d, BF, 380,
                          700)
    q, k, v = normal((B, N, H, d), 381), normal((B, N, Hkv, d), 382), normal((B, N, Hkv, d), 383)
    dev = torch.tensor([random_tree(N, 384 + b) for b in range(B)], dtype=torch.int32).cuda()
    o, lse = torch.zeros_like(q), torch.zeros(B, N, H, device="cuda")
    cache.decode_tree(q, k, v, dev, o, lse)
    buf, lbuf = torch.zeros(q.numel() + 24, dtype=BF, device="cuda"), torch.zeros(lse.numel() + 2, device="cuda")
    o2, l2 = buf[8:8 + q.numel()].view(q.shape), lbuf[1:1 + lse.numel()].view(lse.shape)
    assert o2.data_ptr() % 32 == 16
    cache.decode_tree(q, k, v, dev, o2, l2)
    assert cache.sync_status() == 0
    assert torch.equal(o, o2) and torch.equal(lse, l2)
    assert not buf[:8].any() and not buf[-16:].any() and lbuf[0] == 0 and lbuf[-1] == 0


# ---------------------------------------------------------------------------
# commit
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,H,Hkv,d", [(BF, 10, 10, 128), (BF, 32, 8, 64), (F32, 6, 1, 128)])
@pytest.mark.parametrize("n", [1, 3, 40])
def test_commit_tree(cuda_lib, dtype, H, Hkv, d, n):
    """Accepted counts from none to all, more than the window, the same node
    twice; nodes past the count may be anything; a bad path changes nothing in
    its sequence alone."""
    rswa = cuda_lib
    N, P = 30, 8
    m, t = [5, 0, 12, 3, 7, 9], [0, 2, 100, 41, 6, 1]
    cache, states = make_cache(rswa, m, t, n, H, Hkv, d, dtype, 100)
    k, v = normal((6, N, Hkv, d), 101, dtype), normal((6, N, Hkv, d), 102, dtype)
    path = torch.tensor([[0, 2, 5, 9, 29, -7, 99, 1], [3] * 8, [0, 1, 2, 3, 4, 5, 6, 7],
                         [-1] * 8, [4, 4, 4, 9, 9, 1, 1, 0], [28, 29, -9, 0, 0, 0, 0, 0]],
                        dtype=torch.int32)
    acc = [5, 1, 8, 0, 7, 2]
    Ks, Vs = cache.slabs()
    for _ in range(2):
        before = Ks.clone(), Vs.clone()
        cache.commit_tree(k, v, path.cuda(), torch.tensor(acc, dtype=torch.int32).cuda())
        assert cache.sync_status() == 0
        for b in range(6):
            nodes = path[b, :acc[b]].tolist()
            for j in range(acc[b]):
                slot = cache.m + (states[b]["t"] + j) % n
                before[0][b, :, slot], before[1][b, :, slot] = Ks[b, :, slot], Vs[b, :, slot]
            states[b] = drafts.commit_tree(states[b], f64(k[b]), f64(v[b]), nodes, n)
        check_ring(cache, states, n)
        assert torch.equal(before[0], Ks) and torch.equal(before[1], Vs)
    for b, value, where in ((0, N, 4), (2, -1, 0), (4, 2 ** 31 - 1, 6)):
        p2 = path.clone()
        p2[b, where] = value
        cache.commit_tree(k, v, p2.cuda(), torch.tensor(acc, dtype=torch.int32).cuda())
        assert cache.sync_status() == RSWA_EDEVICE
        for x in range(6):
            if x != b:
                states[x] = drafts.commit_tree(states[x], f64(k[x]), f64(v[x]),
                                               path[x, :acc[x]].tolist(), n)
        check_ring(cache, states, n)
    for bad in (-1, P + 1):
        cache.commit_tree(k, v, path.cuda(), torch.tensor([bad, 0, 0, 0, 0, 0], dtype=torch.int32).cuda())
        assert cache.sync_status() == RSWA_EDEVICE
        check_ring(cache, states, n)


def test_commit_and_append_refusals(cuda_lib):
    rswa = cuda_lib
    H, Hkv, d = 4, 2, 128
    cache, states = make_cache(rswa, [9, 3], [0, 2], 8, H, Hkv, d, BF, 110)
    k, v = normal((2, 5, Hkv, d), 111), normal((2, 5, Hkv, d), 112)
    path = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    acc = torch.zeros(2, dtype=torch.int32, device="cuda")
    for bad in ((k.float(), v, path, acc), (k, v[:, :4].contiguous(), path, acc),
                (k, v, path.long(), acc), (k, v, path, acc.long()), (k, v, path[:1], acc),
                (k, v, path, acc[:1]), (k[:1], v, path, acc),
                (k, v, torch.zeros(2, 1025, dtype=torch.int32).cuda(), acc)):
        with pytest.raises((ValueError, rswa.RswaError)):
            cache.commit_tree(*bad)
    rope = rswa.RswaRope(inv_freq(d))
    q1, k1 = normal((2, H, d), 113), normal((2, Hkv, d), 114)
    out = torch.empty_like(q1)
    for bad in ((q1[:1], k1, k1, out), (q1, k1, k1.float(), out), (q1, k1[:, :1], k1, out),
                (q1, k1, k1, out[:1]), (q1, k1, k1, out.float()), (q1.transpose(1, 2), k1, k1, out)):
        with pytest.raises(ValueError):
            cache.append_kv_rope(rope, *bad)
    lib, h, p = rswa.load(), cache.handle, torch.Tensor.data_ptr
    good = [rope.ref, p(q1), H * d, p(k1), Hkv * d, p(k1), Hkv * d, p(out), None]
    for at, value in ((0, None), (1, None), (2, H * d - 8), (2, H * d + 4), (3, p(k1) + 2),
                      (5, None), (6, 1), (7, None), (7, p(out) + 8)):
        args = list(good)
        args[at] = value
        assert lib.rswa_append_kv_rope(h, *args) == 1, at
    check_ring(cache, states, 8)
    assert cache.sync_status() == 0


# ---------------------------------------------------------------------------
# the operators together, streams and graphs
# ---------------------------------------------------------------------------

def draft_round(rswa, cache, states, rope, m, n, H, Hkv, d, N, seed, ws=None):
    """One round of draft and verify through the entry points, checked."""
    B = len(m)
    qkv = normal((B * N, H + 2 * Hkv, d), seed)
    q, k = qkv[:, :H], qkv[:, H:H + Hkv]
    v = qkv[:, H + Hkv:].contiguous().view(B, N, Hkv, d)
    par = [random_tree(N, seed + b) for b in range(B)]
    depth = torch.tensor([[len(drafts.chain(p, i)) - 1 for i in range(N)] for p in par],
                         dtype=torch.int32)
    qr = torch.empty(B * N, H, d, dtype=BF, device="cuda")
    kr = torch.empty(B * N, Hkv, d, dtype=BF, device="cuda")
    cache.qk_norm_rope(rope, q, k, qr, kr, offsets=depth.cuda())
    pos = (torch.tensor([mb + st["t"] for mb, st in zip(m, states)])[:, None] + depth).reshape(-1)
    check_rope(qr, q, rope.q_weight, pos.tolist(), rope, "q")
    check_rope(kr, k, rope.k_weight, pos.tolist(), rope, "k")
    qt, kt = qr.view(B, N, H, d), kr.view(B, N, Hkv, d)
    o, lse = torch.empty_like(qt), torch.empty(B, N, H, device="cuda")
    cache.decode_tree(qt, kt, v, torch.tensor(par, dtype=torch.int32).cuda(), o, lse, workspace=ws)
    g = np.random.default_rng(seed)
    paths, acc = [], []
    for b in range(B):
        check_tree(o[b], lse[b], qt[b], kt[b], v[b], states[b], par[b], n, f"sequence {b}")
        best = drafts.chain(par[b], int(g.integers(N)))[::-1]
        acc.append(int(g.integers(len(best) + 1)))
        paths.append((best + [0] * N)[:N])
    cache.commit_tree(kt, v, torch.tensor(paths, dtype=torch.int32).cuda(),
                      torch.tensor(acc, dtype=torch.int32).cuda())
    for b in range(B):
        states[b] = drafts.commit_tree(states[b], f64(kt[b]), f64(v[b]), paths[b][:acc[b]], n)
    check_ring(cache, states, n)


def test_prefill_draft_verify_and_decode_together(cuda_lib):
    """Prompt normed, rotated and prefilled; rounds of drafts; then single
    steps through the rotated append and through the fused step."""
    rswa = cuda_lib
    m, n, H, Hkv, d, N = [150, 40], 32, 8, 2, 128, 13
    rope = rswa.RswaRope(inv_freq(d), weight(d, 120, BF), weight(d, 121, BF))
    rows = sum(m)
    qkv = normal((rows, H + 2 * Hkv, d), 122)
    pos = torch.cat([torch.arange(x) for x in m])
    q, k = torch.empty(rows, H, d, dtype=BF, device="cuda"), torch.empty(rows, Hkv, d, dtype=BF, device="cuda")
    rswa.rswa_qk_norm_rope(rope, qkv[:, :H], qkv[:, H:H + Hkv], pos.cuda(), q, k)
    v = qkv[:, H + Hkv:].contiguous()
    cache = rswa.RswaCache(max(m), n, H, d, 2, rswa.RSWA_BF16, kv_heads=Hkv)
    O = torch.empty_like(q)
    cache.prefill(q, k, v, O, m, 0)
    states, at = [], 0
    for mb in m:
        sl = slice(at, at + mb)
        states.append(oracle.prefill_cache(f64(k[sl]), f64(v[sl]), mb, n, 0))
        ref, _ = oracle.prefill_attention(f64(q[sl]), f64(k[sl]), f64(v[sl]), mb, n)
        assert np.abs(f64(O[sl]) - ref).max() <= 2e-2
        at += mb
    for r in range(5):
        draft_round(rswa, cache, states, rope, m, n, H, Hkv, d, N, 130 + r)
        qkv = normal((2, H + 2 * Hkv, d), 140 + r)
        q1, k1, v1 = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:].contiguous()
        qo, ko = torch.empty(2, H, d, dtype=BF, device="cuda"), torch.empty(2, Hkv, d, dtype=BF, device="cuda")
        o = torch.empty_like(qo)
        if r % 2:
            cache.append_kv_rope(rope, q1, k1, v1, qo)
            cache.decode_step(qo, o)
            Ks, _ = cache.slabs()
            ko = torch.stack([Ks[b, :, cache.m + states[b]["t"] % n] for b in range(2)])
        else:
            cache.qk_norm_rope(rope, q1, k1, qo, ko)
            cache.decode_step_fused(qo, ko, v1, o)
        for b in range(2):
            states[b], ref, _ = oracle.decode_step_fused(states[b], f64(qo[b]), f64(ko[b]), f64(v1[b]), n)
            assert np.abs(f64(o[b]) - ref).max() <= 2e-2
    check_ring(cache, states, n)
    assert cache.sync_status() == 0


@pytest.mark.parametrize("H,Hkv,d,dtype", [(10, 10, 128, BF), (8, 2, 64, BF), (4, 2, 64, F32)])
def test_captured_round_replays_on_new_inputs(cuda_lib, H, Hkv, d, dtype):
    """Norm and rotation, tree, commit and a rotated append captured in one
    graph: each replay works on the state that the last one left, and gives
    what the same calls give one by one."""
    rswa = cuda_lib
    m, t, n, N, P = [260, 30], [7, 90], 48, 21, 6
    caches = [make_cache(rswa, m, t, n, H, Hkv, d, dtype, 150)[0] for _ in range(2)]
    rope = rswa.RswaRope(inv_freq(d), weight(d, 151, dtype), weight(d, 152, dtype))
    q, k = normal((2 * N, H, d), 153, dtype), normal((2 * N, Hkv, d), 154, dtype)
    v = normal((2, N, Hkv, d), 155, dtype)
    par = torch.tensor([random_tree(N, 1), random_tree(N, 2)], dtype=torch.int32).cuda()
    off = torch.tensor([[len(drafts.chain(p, i)) - 1 for i in range(N)] for p in par.tolist()],
                       dtype=torch.int32).cuda()
    path = torch.tensor([[0, 3, 4, 6, 9, 20], [0, 1, 2, 3, 4, 5]], dtype=torch.int32).cuda()
    acc = torch.tensor([4, 2], dtype=torch.int32).cuda()
    q1, k1, v1 = normal((2, H, d), 156, dtype), normal((2, Hkv, d), 157, dtype), normal((2, Hkv, d), 158, dtype)

    def buffers():
        return dict(qr=torch.zeros_like(q), kr=torch.zeros_like(k),
                    o=torch.zeros(2, N, H, d, dtype=dtype, device="cuda"),
                    lse=torch.zeros(2, N, H, device="cuda"), qo=torch.zeros_like(q1), o1=torch.zeros_like(q1))

    def calls(c, x, ws):
        c.qk_norm_rope(rope, q, k, x["qr"], x["kr"], offsets=off)
        kt = x["kr"].view(2, N, Hkv, d)
        c.decode_tree(x["qr"].view(2, N, H, d), kt, v, par, x["o"], x["lse"], workspace=ws)
        c.commit_tree(kt, v, path, acc)
        c.append_kv_rope(rope, q1, k1, v1, x["qo"])
        c.decode_step(x["qo"], x["o1"])

    x, y = buffers(), buffers()
    ws = caches[0].tree_workspace(N)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls(caches[0], x, ws)                    # once outside the capture, on another stream
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls(caches[0], x, ws)
    calls(caches[1], y, None)
    for r in range(3):
        for a in (q, k, v, q1, k1, v1):
            a.copy_(normal(a.shape, 160 + r, dtype))
        acc.copy_(torch.tensor([[0, 6], [5, 1], [6, 0]][r], dtype=torch.int32))
        graph.replay()
        calls(caches[1], y, None)
        torch.cuda.synchronize()
        for name in x:
            assert torch.equal(x[name], y[name]), name
        for b in range(2):
            assert caches[0].get_t(b) == caches[1].get_t(b)
        assert all(torch.equal(a, b) for a, b in zip(caches[0].slabs(), caches[1].slabs()))
    assert caches[0].sync_status() == 0 and caches[1].sync_status() == 0


def test_capture_needs_a_workspace(cuda_lib):
    rswa = cuda_lib
    cache, _ = make_cache(rswa, [9], [0], 8, 2, 2, 128, BF, 170)
    q = normal((1, 4, 2, 128), 171)
    par = torch.full((1, 4), -1, dtype=torch.int32, device="cuda")
    o = torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(ValueError):
            cache.decode_tree(q, q, q, par, o)
    cache.decode_tree(q, q, q, par, o)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.decode_tree(q, q, q, par, o)
    graph.replay()
    torch.cuda.synchronize()
    assert cache.sync_status() == 0


def test_calls_by_handle_refuse_cpu_tensors(cuda_lib):
    rswa = cuda_lib
    H, Hkv, d = 4, 2, 128
    cache, _ = make_cache(rswa, [9], [0], 8, H, Hkv, d, BF, 190)
    rope = rswa.RswaRope(inv_freq(d))
    q, k, v = normal((1, H, d), 191), normal((1, Hkv, d), 192), normal((1, Hkv, d), 193)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    for bad in ((q.cpu(), k, v), (q, k.cpu(), v)):
        with pytest.raises(ValueError):
            rswa.rswa_qk_norm_rope_cached(cache.handle, rope, bad[0], H * d, bad[1], Hkv * d,
                                          None, 1, qo, ko)
    for bad in ((q.cpu(), k, v), (q, k.cpu(), v), (q, k, v.cpu())):
        with pytest.raises(ValueError):
            rswa.rswa_append_kv_rope(cache.handle, rope, bad[0], H * d, bad[1], Hkv * d,
                                     bad[2], Hkv * d, qo)
    o = torch.empty(1, 1, H, d, dtype=BF, device="cuda")
    par = torch.full((1, 1), -1, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        cache.decode_tree(q[None], k[None], v[None], par, o,
                          workspace=cache.tree_workspace(1).cpu())
    assert cache.sync_status() == 0 and cache.get_t(0) == 0


def test_two_caches_on_two_streams(cuda_lib):
    """Calls on different caches overlap; each has its own workspace."""
    rswa = cuda_lib
    made = [make_cache(rswa, [900], [100], 64, 10, 10, 128, BF, 180 + i) for i in range(2)]
    x = [[normal((1, 24, 10, 128), 190 + 10 * i + j) for j in range(3)] for i in range(2)]
    par = [random_tree(24, i) for i in range(2)]
    dev = [torch.tensor([p], dtype=torch.int32).cuda() for p in par]
    out = [(torch.empty_like(x[i][0]), torch.empty(1, 24, 10, device="cuda")) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            made[i][0].decode_tree(*x[i], dev[i], *out[i], stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        check_tree(out[i][0][0], out[i][1][0], *(a[0] for a in x[i]), made[i][1][0], par[i], 64, f"cache {i}")


def test_own_workspaces_belong_to_their_streams(cuda_lib):
    """The workspace that a cache makes for itself comes from the pool of the
    stream that the call runs on (named, or torch's current one), whose queued
    work orders its use and its release."""
    rswa = cuda_lib
    cache, states = make_cache(rswa, [1500], [40], 64, 8, 2, 128, BF, 410)
    q, k, v = normal((1, 60, 8, 128), 411), normal((1, 60, 2, 128), 412), normal((1, 60, 2, 128), 413)
    par = [random_tree(60, 414)]
    dev = torch.tensor(par, dtype=torch.int32).cuda()
    default, named, current = torch.cuda.current_stream(), torch.cuda.Stream(), torch.cuda.Stream()
    outs = [(torch.empty_like(q), torch.empty(1, 60, 8, device="cuda")) for _ in range(4)]

    def pool(w):
        at, size = w.data_ptr(), w.numel()
        assert size > 1 << 20                    # of the tensor-core kernel
        return [s["stream"] for s in torch.cuda.memory_snapshot()
                if s["address"] <= at and at + size <= s["address"] + s["total_size"]]

    torch.cuda.synchronize()
    cache.decode_tree(q, k, v, dev, *outs[0], stream=named)
    current.wait_stream(named)
    with torch.cuda.stream(current):
        cache.decode_tree(q, k, v, dev, *outs[1])
    default.wait_stream(current)
    cache.decode_tree(q, k, v, dev, *outs[2])
    cache.decode_tree(q[:, :9].contiguous(), k[:, :9].contiguous(), v[:, :9].contiguous(),
                      dev[:, :9].contiguous(), outs[3][0][:, :9].contiguous())   # fewer: the same one
    torch.cuda.synchronize()
    used = sorted({w.data_ptr(): pool(w) for w in cache._tree_ws.values()}.values())
    assert used == sorted([s.cuda_stream] for s in (named, current, default))
    for o, lse in outs[:3]:
        check_tree(o[0], lse[0], q[0], k[0], v[0], states[0], par[0], 64, "on three streams")
        assert torch.equal(o, outs[0][0])
    assert cache.sync_status() == 0


def test_own_workspace_and_a_capture_on_a_named_stream(cuda_lib):
    """Whether a call is part of a capture goes by the stream that it names."""
    rswa = cuda_lib
    cache, states = make_cache(rswa, [1500], [40], 64, 2, 2, 128, BF, 415)
    q, k, v = (normal((1, 20, 2, 128), 416 + i) for i in range(3))
    par = [random_tree(20, 419)]
    dev = torch.tensor(par, dtype=torch.int32).cuda()
    o, lse = torch.empty_like(q), torch.empty(1, 20, 2, device="cuda")
    side, away = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        other = torch.cuda.current_stream()
        side.wait_stream(other)
        with torch.cuda.stream(away):
            with pytest.raises(ValueError):      # side is part of the capture, the current one not
                cache.decode_tree(q, k, v, dev, o, lse, stream=side)
        other.wait_stream(side)
    assert not cache._tree_ws
    cache.decode_tree(q, k, v, dev, o, lse)
    o.zero_(), lse.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.decode_tree(q, k, v, dev, o, lse)
    graph.replay()
    torch.cuda.synchronize()
    assert len({w.data_ptr() for w in cache._tree_ws.values()}) == 1
    check_tree(o[0], lse[0], q[0], k[0], v[0], states[0], par[0], 64, "replayed")
    assert cache.sync_status() == 0


@pytest.mark.parametrize("dtype,N", [(BF, 2), (BF, 33), (F32, 2)])
def test_more_sequences_than_a_grid_dimension(cuda_lib, dtype, N):
    """66000 sequences: trees, the accepted nodes and the rotated append of all
    of them."""
    rswa = cuda_lib
    B, m, n, d = 66000, 2, 2, 64
    code = rswa.RSWA_BF16 if dtype is BF else rswa.RSWA_F32
    K, V = normal((B * (m + 1), 1, d), 430, dtype), normal((B * (m + 1), 1, d), 431, dtype)
    cache = rswa.RswaCache(m, n, 1, d, B, code)
    cache.prefill(None, K, V, None, [m] * B, 1)
    q, k, v = (normal((B, N, 1, d), 432 + i, dtype) for i in range(3))
    par = random_tree(N, 435)
    dev = torch.tensor([par], dtype=torch.int32).expand(B, N).contiguous().cuda()
    counts = (torch.arange(B, dtype=torch.int32) % (N + 1)).cuda()
    counts[65534:65538] = N
    o, lse = torch.full_like(q, 7.0), torch.full((B, N, 1), 7.0, device="cuda")
    cache.decode_tree(q, k, v, dev, o, lse, counts=counts)
    assert cache.sync_status() == 0
    at = [0, N, 65534, 65535, 65536, 65537, B - 1]
    for b in at:
        sl, c = slice(b * (m + 1), (b + 1) * (m + 1)), int(counts[b])
        state = oracle.prefill_cache(f64(K[sl]), f64(V[sl]), m, n, 1)
        check_tree(o[b, :c], lse[b, :c], q[b, :c], k[b, :c], v[b, :c], state, par[:c], n, f"{b}")
    live = torch.arange(N, device="cuda") < counts[:, None]
    assert torch.equal((o == 7).all(-1)[..., 0], ~live) and torch.equal(lse[..., 0] == 7, ~live)
    path = torch.zeros(B, 1, dtype=torch.int32, device="cuda")
    acc = (counts > 0).int()
    cache.commit_tree(k, v, path, acc)
    rope = rswa.RswaRope(inv_freq(d), None, weight(d, 436, dtype))
    qkv = normal((B, 3, d), 437, dtype)
    qo = torch.empty(B, 1, d, dtype=dtype, device="cuda")
    cache.append_kv_rope(rope, qkv[:, :1], qkv[:, 1:2], qkv[:, 2:], qo)
    assert cache.sync_status() == 0
    Ks, Vs = cache.slabs()
    for b in at:
        a = int(acc[b])
        slot = m + (1 + a) % n                   # of the appended token
        assert cache.get_t(b) == 2 + a
        check_rope(qo[b:b + 1], qkv[b:b + 1, :1], None, [m + 1 + a], rope, f"q {b}")
        check_rope(Ks[b:b + 1, :, slot], qkv[b:b + 1, 1:2], rope.k_weight, [m + 1 + a], rope, f"k {b}")
        same(Vs[b, :, slot], f64(qkv[b, 2:]))
        if a:
            same(Ks[b, :, m + 1], f64(k[b, 0]))
            same(Vs[b, :, m + 1], f64(v[b, 0]))


@pytest.mark.parametrize("dtype,cap", [(BF, 20_000_000), (F32, 10_000_000)])
def test_offsets_beyond_32_bits(cuda_lib, dtype, cap):
    """A cache whose second sequence begins more than 2^32 bytes, and in bf16
    2^31 elements, behind the first: append, tree (tensor and CUDA cores) and
    commit of the same node twice."""
    rswa = cuda_lib
    m, t, n, H, d, N = [300, 170], [20, 65], 64, 2, 128, 21
    cache, states = make_cache(rswa, m, t, n, H, 1, d, dtype, 480, cap)
    Ks, Vs = cache.slabs()
    assert Ks[1].data_ptr() - Ks[0].data_ptr() > 2 ** 32
    rope = rswa.RswaRope(inv_freq(d), weight(d, 481, dtype), weight(d, 482, dtype))
    qkv = normal((2, H + 2, d), 483, dtype)
    qo = torch.empty(2, H, d, dtype=dtype, device="cuda")
    cache.append_kv_rope(rope, qkv[:, :H], qkv[:, H:H + 1], qkv[:, H + 1:], qo)
    pos = [a + b for a, b in zip(m, t)]
    check_rope(qo, qkv[:, :H], rope.q_weight, pos, rope, "q")
    for b in range(2):
        stored = Ks[b, :, cap + t[b] % n]
        check_rope(stored[None], qkv[b:b + 1, H:H + 1], rope.k_weight, pos[b:b + 1], rope, "k")
        states[b] = oracle.append_kv(states[b], f64(stored), f64(qkv[b, H + 1:]), n)
    q, k, v = normal((2, N, H, d), 484, dtype), normal((2, N, 1, d), 485, dtype), normal((2, N, 1, d), 486, dtype)
    par = [random_tree(N, 487), random_tree(N, 488)]
    path = torch.tensor([[0, 5, 5], [20, 20, 1]], dtype=torch.int32).cuda()
    acc = torch.tensor([3, 2], dtype=torch.int32).cuda()
    o, lse = torch.empty_like(q), torch.empty(2, N, H, device="cuda")
    cache.decode_tree(q, k, v, torch.tensor(par, dtype=torch.int32).cuda(), o, lse)
    cache.commit_tree(k, v, path, acc)
    assert cache.sync_status() == 0
    for b in range(2):
        check_tree(o[b], lse[b], q[b], k[b], v[b], states[b], par[b], n, f"{b}")
        states[b] = drafts.commit_tree(states[b], f64(k[b]), f64(v[b]), path[b, :int(acc[b])].tolist(), n)
        assert cache.get_t(b) == states[b]["t"]
        for slab, name in ((Ks, "Kr"), (Vs, "Vr")):
            got = f64(slab[b, :, cap:]).transpose(1, 0, 2)
            filled = sorted(oracle.ring_outputs(states[b]["t"], n))
            np.testing.assert_array_equal(got[filled], states[b][name][filled])


def test_two_graphs_share_a_workspace(cuda_lib):
    """Two captured calls of one cache, of different trees, replayed in turn on
    the workspace that the cache keeps."""
    rswa = cuda_lib
    m, n, H, Hkv, d = [1500, 900], 64, 8, 2, 128
    cache, states = make_cache(rswa, m, [40, 3], n, H, Hkv, d, BF, 490)
    calls = []
    for N in (60, 17):
        q, k, v = normal((2, N, H, d), 491 + N), normal((2, N, Hkv, d), 492 + N), normal((2, N, Hkv, d), 493 + N)
        par = [random_tree(N, 494), random_tree(N, 495)]
        calls.append((q, k, v, torch.tensor(par, dtype=torch.int32).cuda(), torch.empty_like(q),
                      torch.empty(2, N, H, device="cuda"), par))
    for c in calls:
        cache.decode_tree(*c[:6])
    graphs = []
    for c in calls:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            cache.decode_tree(*c[:6])
            cache.decode_tree(*c[:6])
    want = [(c[4].clone(), c[5].clone()) for c in calls]
    for _ in range(4):
        for c in calls:
            c[4].zero_(), c[5].zero_()
        for g in graphs:
            g.replay()
        for c, (o, lse) in zip(calls, want):
            assert torch.equal(c[4], o) and torch.equal(c[5], lse)
    for q, k, v, _, o, lse, par in calls:
        for b in range(2):
            check_tree(o[b], lse[b], q[b], k[b], v[b], states[b], par[b], n, f"{b}")
    assert cache.sync_status() == 0


def test_decode_tree_is_deterministic(cuda_lib):
    rswa = cuda_lib
    _, _, (q, k, v, par, o, lse) = run_tree(rswa, [1500], [90], 64, 4, 2, 128, 30, BF, 200)
    cache, _ = make_cache(rswa, [1500], [90], 64, 4, 2, 128, BF, 200)
    for _ in range(5):
        o2, l2 = torch.empty_like(o), torch.empty_like(lse)
        cache.decode_tree(q, k, v, torch.tensor(par, dtype=torch.int32).cuda(), o2, l2)
        assert torch.equal(o, o2) and torch.equal(lse, l2)
