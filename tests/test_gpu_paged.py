"""GPU parity of the paged-cache operators (append of a chunk, its attention, the
weights that cached tokens receive, eviction) against their float64 oracle.

Tolerances come from the arithmetic; a rounding to a type is off by at most half a
step, eps / 2 (bf16 2^-8, float32 2^-24) relative to the value.

A logit is a dot product of d terms, off by at most (d + 8) half steps of
sum |q k| / sqrt(d) (twice that on the tensor cores, which truncate); weights and
sums over S keys by S half steps more, and 2^-21 for the exponential.  That bounds
the log-sum-exp directly (with 2^-22 of its own size and of the logits' in base 2
for the products and the logarithm), and o relative to sum p |v|, twice (numerator
and denominator).  In bf16 the weights may be rounded to bf16 (2^-8 of sum p |v|)
and o is (2^-8 of |o|).  What a token receives is off by the same logit and
exponential relative to itself, and by the half steps of a sum of its rows.
Appended and evicted rows are copies and exact, and so are what stays and where.

Rows of pages that hold no token are NaN, and table entries without one are -1 or
far outside the pool: neither may be looked at.
"""

import numpy as np
import pytest
import torch

import workloads
from oracle import paged

pytestmark = pytest.mark.gpu

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
RSWA_EDEVICE = 6
BF, F32 = torch.bfloat16, torch.float32


def f64(t):
    return t.detach().double().cpu().numpy()


def normal(shape, seed, dtype=BF, std=1.0):
    return workloads.normal(shape, seed, std, dtype, "cuda")


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Case:
    """Sequences of L[b] tokens of which the last T[b] are the chunk, in pages in
    random order; rows without a token are NaN, entries without one `hole`.
    K, V: lists of [L][Hkv][d]; q, k, v: the chunk's rows."""

    def __init__(self, rswa, L, T, H, Hkv, d, P, dtype=BF, prefix=None, window=None, seed=0,
                 stored=True, spare=0, uniform=False, std=1.0, hole=-1):
        self.L, self.T, self.H, self.Hkv, self.d, self.P, self.dtype = L, T, H, Hkv, d, P, dtype
        self.m = prefix or [0] * len(L)
        self.n = window or 1 << 30
        g = np.random.default_rng(seed)
        need = [-(-x // P) for x in L]
        self.width = max(1, max(need)) + spare
        pool = sum(need) + 2
        ids = g.permutation(pool).tolist()
        table = [[ids.pop() for _ in range(c)] + [hole] * (self.width - c) for c in need]
        self.where = [list(r) for r in table]
        self.table, self.lens = ints(table), ints(L)
        self.start = np.concatenate([[0], np.cumsum(T)]).tolist()
        code = rswa.RSWA_F32 if dtype == F32 else rswa.RSWA_BF16
        self.pages = rswa.RswaPages(pool, P, H, d, code, kv_heads=Hkv)
        self.batch = rswa.RswaBatch(self.table, self.lens,
                                    starts=None if uniform else ints(self.start),
                                    prefix=None if prefix is None else ints(prefix), window=window)
        self.Kp, self.Vp = self.pages.slabs()
        self.Kp.fill_(float("nan"))
        self.Vp.fill_(float("nan"))
        rows = sum(T)
        self.q = normal((rows, H, d), 3 * seed + 1, dtype, std)
        kv = normal((2, sum(L), Hkv, d), 3 * seed + 2, dtype)
        at = np.concatenate([[0], np.cumsum(L)])
        self.K = [kv[0, at[b]:at[b + 1]] for b in range(len(L))]
        self.V = [kv[1, at[b]:at[b + 1]] for b in range(len(L))]
        self.k = torch.cat([x[l - t:] for x, l, t in zip(self.K, L, T)])
        self.v = torch.cat([x[l - t:] for x, l, t in zip(self.V, L, T)])
        for b in range(len(L)):
            self.write(b, L[b] if stored else L[b] - T[b])

    def write(self, b, upto):
        for p in range(-(-upto // self.P)):
            n = min(self.P, upto - p * self.P)
            for pool, rows in ((self.Kp, self.K[b]), (self.Vp, self.V[b])):
                pool[self.where[b][p], :, :n] = rows[p * self.P:p * self.P + n].transpose(0, 1)

    def tokens(self, pool, b, count, table=None):
        """[count][Hkv][d] as the pages hold them."""
        table = self.where if table is None else table
        if count == 0:
            return pool[:0, :, 0]
        x = pool[torch.tensor(table[b][:-(-count // self.P)], device="cuda")]
        return x.transpose(1, 2).reshape(-1, self.Hkv, self.d)[:count]

    def rows(self, b):
        return slice(self.start[b], self.start[b + 1])

    def attend(self, **kw):
        o = torch.full((sum(self.T), self.H, self.d), float("nan"), dtype=self.dtype, device="cuda")
        lse = torch.full((sum(self.T), self.H), float("nan"), device="cuda")
        self.pages.attend(self.batch, self.q, o, lse, **kw)
        return o, lse


def logit_error(c, size, S):
    u = 2.0 ** -24
    return (2 * (c.d + 8) * size + S + 4 * size) * u + 2.0 ** -21


def check_attend(c, o, lse, what="", rows_of=None):
    """rows_of: rows of a sequence's chunk to compare (None: all)."""
    worst = 0.0
    for b in range(len(c.L)):
        if c.T[b] == 0:
            continue
        pick = list(range(c.T[b])) if rows_of is None else sorted({r for r in rows_of if 0 <= r < c.T[b]})
        K, V = f64(c.K[b]), f64(c.V[b])
        for i in pick:
            row, L = c.start[b] + i, c.L[b] - c.T[b] + i + 1
            ro, rl, mass, size = paged.attend(f64(c.q[row:row + 1]), K[:L], V[:L], c.m[b], c.n)
            e = logit_error(c, size, min(L, c.n + c.m[b]))
            tol = 2 * e[..., None] * mass + 2.0 ** -24 * np.abs(ro)
            if c.dtype == BF:
                tol = tol + HALF[BF] * (mass + np.abs(ro) + tol)
            err = np.abs(f64(o[row:row + 1]) - ro)
            assert np.isfinite(err).all(), f"{what}: sequence {b} row {i}"
            worst = max(worst, (err / tol).max())
            assert (err <= tol).all(), f"{what}: sequence {b} row {i}: {(err / tol).max():.3g} of the bound"
            le = np.abs(f64(lse[row:row + 1]) - rl)
            assert (le <= e + 2.0 ** -22 * (np.abs(rl) + 1)).all(), f"{what}: lse of {b} row {i}"
    return worst


SHAPES = [
    # H, Hkv, d, P, dtype
    (10, 10, 128, 64, BF), (32, 8, 128, 16, BF), (8, 1, 64, 32, BF), (6, 2, 128, 128, BF),
    (5, 5, 64, 256, BF), (20, 5, 128, 32, BF), (28, 4, 64, 16, BF), (48, 2, 128, 64, BF),
    (4, 2, 64, 16, F32), (3, 3, 128, 128, F32), (12, 4, 128, 32, F32), (16, 1, 64, 256, F32),
]
LENGTHS = [
    # L, T, prefix, window
    ([1], [1], None, None),
    ([1, 2, 17, 16], [1, 1, 1, 1], None, None),
    ([130, 5, 0, 64, 33], [7, 5, 0, 0, 1], None, None),
    ([300, 129, 128, 127], [1, 1, 1, 1], [40, 129, 0, 127], 20),
    ([260, 90], [33, 90], [30, 16], 50),
    ([200, 333], [2, 1], [16, 0], 1),
    ([700], [70], [100], 128),
    ([389, 391], [200, 3], [4, 4], 7),
]


@pytest.mark.parametrize("H,Hkv,d,P,dtype", SHAPES)
@pytest.mark.parametrize("L,T,prefix,window", LENGTHS)
def test_attend(cuda_lib, H, Hkv, d, P, dtype, L, T, prefix, window):
    c = Case(cuda_lib, L, T, H, Hkv, d, P, dtype, prefix, window, seed=len(L) + H)
    o, lse = c.attend()
    check_attend(c, o, lse, rows_of=[0, 1, 31, 32, 63, 64, 127, 128, T[0] - 1, T[-1] - 1])
    assert c.pages.sync_status() == 0


@pytest.mark.parametrize("H,Hkv,d,P,dtype", [SHAPES[1], SHAPES[0], SHAPES[8]])
def test_attend_long_chunk(cuda_lib, H, Hkv, d, P, dtype):
    c = Case(cuda_lib, [1400, 1000, 640], [600, 1, 511], H, Hkv, d, P, dtype, [16, 500, 0], 333, seed=4)
    check_attend(c, *c.attend(), rows_of=[0, 5, 127, 128, 255, 256, 300, 510, 599])


@pytest.mark.parametrize("H,Hkv,d", [(10, 10, 128), (32, 8, 128), (16, 2, 64)])
@pytest.mark.parametrize("T", [1, 4])
def test_attend_many_sequences(cuda_lib, H, Hkv, d, T):
    """More sequences than a warp has lanes, uniform chunks, every length."""
    g = np.random.default_rng(T)
    L = [int(x) for x in g.integers(T, 900, 70)]
    c = Case(cuda_lib, L, [T] * 70, H, Hkv, d, 32, BF, uniform=True, seed=T)
    check_attend(c, *c.attend(), rows_of=[0, T - 1])
    c = Case(cuda_lib, L, [T] * 70, H, Hkv, d, 32, BF, [int(x) for x in g.integers(0, 900, 70)], 64, seed=T)
    c.m = [min(m, l) for m, l in zip(c.m, L)]          # prefixes past the length are cut
    check_attend(c, *c.attend(), rows_of=[0, T - 1])


def test_attend_long_cache(cuda_lib):
    for H, Hkv, T in ((10, 10, 1), (16, 2, 1), (8, 2, 40)):
        c = Case(cuda_lib, [10272], [T], H, Hkv, 128, 64, seed=T)
        check_attend(c, *c.attend(), rows_of=[0, 20, T - 1])


def test_attend_more_query_heads_than_a_tile(cuda_lib):
    c = Case(cuda_lib, [70, 20], [3, 20], 150, 1, 64, 16, BF, [3, 0], 30, seed=1)
    check_attend(c, *c.attend())


def test_attend_sharp_softmax(cuda_lib):
    """Logits of some hundred: the running maximum moves, weights vanish."""
    for dtype in (BF, F32):
        for T in (1, 150):
            c = Case(cuda_lib, [900], [T], 8, 2, 128, 32, dtype, [20], 300, seed=T, std=30.0)
            check_attend(c, *c.attend(), rows_of=[0, 77, T - 1])


@pytest.mark.parametrize("H,Hkv,d,T", [(10, 10, 128, 1), (32, 8, 128, 1), (16, 2, 64, 1), (10, 10, 64, 2),
                                       (10, 10, 128, 4), (8, 4, 128, 4)])
def test_attend_few_rows_keeps_its_weights(cuda_lib, H, Hkv, d, T):
    """In units of few rows the weights are two bf16 parts: a rounding takes 2^-8 of a weight
    off, and of that its second part all but 2^-8.  The output's own rounding is what is left."""
    g = np.random.default_rng(H * d + T)
    L = [int(x) for x in g.integers(T, 700, 64)]
    c = Case(cuda_lib, L, [T] * 64, H, Hkv, d, 32, BF, [40] * 64, 300, seed=T, uniform=H != 8)
    c.m = [min(40, l) for l in L]
    o, _ = c.attend()
    for b in range(64):
        K, V = f64(c.K[b]), f64(c.V[b])
        ro, _, mass, size = paged.attend(f64(c.q[c.rows(b)]), K, V, c.m[b], c.n)
        tol = (2 * logit_error(c, size, min(L[b], c.n + c.m[b]))[..., None] + HALF[BF] ** 2) * mass
        tol = tol + HALF[BF] * (np.abs(ro) + tol)
        err = np.abs(f64(o[c.rows(b)]) - ro)
        assert (err <= tol).all(), f"sequence {b}: {(err / tol).max():.3g} of the bound"


def test_attend_holes_are_not_read(cuda_lib):
    """Pages between the prefix and the window are gone, masked rows NaN."""
    for dtype, H, Hkv, T in ((BF, 32, 8, 1), (BF, 10, 10, 1), (BF, 32, 8, 37), (F32, 4, 2, 5),
                             (BF, 10, 10, 300)):
        c = Case(cuda_lib, [1000, 980], [T, T], H, Hkv, 128, 16, dtype, [21, 0], 100, seed=T,
                 hole=1 << 30)
        gone = 0
        for b in range(2):
            lo, hi = c.m[b], c.L[b] - T - 99           # tokens that no row sees
            for j in range(lo, hi):
                p = c.where[b][j // 16]
                c.Kp[p, :, j % 16] = float("nan")
                c.Vp[p, :, j % 16] = float("nan")
            for p in range(-(-lo // 16), hi // 16):
                c.table[b, p] = -1 - p
                gone += 1
        assert gone > 70
        check_attend(c, *c.attend(), rows_of=[0, T - 1])
        assert c.pages.sync_status() == 0


@pytest.mark.parametrize("H,Hkv,d,P", [(10, 10, 128, 64), (32, 8, 128, 16), (16, 2, 64, 128), (8, 4, 64, 256)])
@pytest.mark.parametrize("T", [1, 2, 0])
def test_attend_few_rows_of_many_sequences(cuda_lib, H, Hkv, d, P, T):
    """Prefixes, windows and lengths that meet inside tiles and 16-key steps; NaN in
    every row of a page that no row sees, pages that nobody sees gone; T 0: one to
    three rows each."""
    g = np.random.default_rng(H + T)
    B = 72
    T = [T] * B if T else [int(x) for x in g.integers(0, 4, B)]
    L = [int(x) for x in g.integers(4, 1500, B)]
    prefix = [int(x) for x in g.integers(0, 700, B)]
    window = 90
    c = Case(cuda_lib, L, T, H, Hkv, d, P, BF, prefix, window, seed=B, hole=1 << 30, uniform=T[0] == T[1] == T[2])
    c.m = [min(m, l) for m, l in zip(prefix, L)]
    for b in range(B):
        lo, hi = c.m[b], max(c.m[b], L[b] - T[b] - window + 1)
        hi = hi if T[b] else L[b]
        for p in range(lo // P, -(-hi // P)):
            a, z = max(lo, p * P), min(hi, (p + 1) * P)
            if a < z:
                c.Kp[c.where[b][p], :, a - p * P:z - p * P] = float("nan")
                c.Vp[c.where[b][p], :, a - p * P:z - p * P] = float("nan")
        for p in range(-(-lo // P), hi // P):
            c.table[b, p] = -3
    check_attend(c, *c.attend())
    assert c.pages.sync_status() == 0


@pytest.mark.parametrize("H,Hkv,d,P,L,T,m,n", [
    (10, 10, 128, 64, [1], [1], None, None), (32, 8, 128, 32, [2600], [1], None, None),
    (16, 2, 128, 16, [7000, 6500], [1, 1], [300, 0], 129), (10, 10, 128, 16, [7000], [8], None, None),
    (32, 8, 64, 64, [9000], [3], [5], 4000), (12, 4, 128, 128, [6700, 3], [9, 3], None, None),
])
def test_attend_wide_tables(cuda_lib, H, Hkv, d, P, L, T, m, n):
    """Tables that could hold long caches: few sequences on the tensor cores, units cut
    over many CTAs."""
    c = Case(cuda_lib, L, T, H, Hkv, d, P, BF, m, n, seed=5, spare=700)
    check_attend(c, *c.attend())
    assert c.pages.sync_status() == 0


@pytest.mark.parametrize("H,Hkv,d,P", [(10, 10, 128, 16), (12, 4, 64, 128), (20, 2, 128, 256), (6, 6, 64, 32)])
@pytest.mark.parametrize("T,prefix,window", [([300, 1, 0, 129], None, None), ([200, 90, 64, 3], [30, 0, 200, 5], 70)])
def test_float32_with_many_rows(cuda_lib, H, Hkv, d, P, T, prefix, window):
    """Tiles of 64 rows and keys; NaN in rows that nobody sees."""
    L = [433, 257, 90, 200]
    c = Case(cuda_lib, L, T, H, Hkv, d, P, F32, prefix, window, seed=H, hole=1 << 30)
    if window:
        for b in range(4):
            lo, hi = c.m[b], L[b] - T[b] - window + 1
            for j in range(lo, hi):
                c.Kp[c.where[b][j // P], :, j % P] = float("nan")
                c.Vp[c.where[b][j // P], :, j % P] = float("nan")
    o, lse = c.attend()
    check_attend(c, o, lse, rows_of=[0, 1, 20, 63, 64, 127, 128, 199, 299])
    old = torch.rand(4, Hkv, c.width * P, device="cuda")
    w = old.clone()
    c.pages.weigh(c.batch, c.q, lse, w, 0.5)
    check_weigh(c, lse, old, w, 0.5)
    q = c.q.clone()
    c.pages.attend(c.batch, q, q)
    assert torch.equal(q, o)
    assert c.pages.sync_status() == 0


@pytest.mark.parametrize("H,Hkv,d,T", [(10, 10, 128, 1), (32, 8, 128, 1), (32, 8, 128, 70), (10, 10, 64, 300)])
def test_waits_that_run_out(cuda_lib, H, Hkv, d, T):
    """A bound of 1 ns on every wait: the kernels give up, the flag says so, and with
    zeroed workspaces and the usual bound the next call is right."""
    rswa = cuda_lib
    c = Case(rswa, [900] * 40, [T] * 40, H, Hkv, d, 32, seed=1, uniform=True)
    ws = c.pages.attend_workspace(40 * T)
    w = torch.zeros(40, Hkv, c.width * 32, device="cuda")
    _, lse = c.attend(workspace=ws)
    for call in (lambda: c.attend(workspace=ws), lambda: c.pages.weigh(c.batch, c.q, lse, w)):
        rswa.rswa_debug_set_wait_limit_ns(1)
        try:
            call()
        finally:
            rswa.rswa_debug_set_wait_limit_ns(0)
        assert c.pages.sync_status() == RSWA_EDEVICE
        assert c.pages.sync_status() == 0
    ws.zero_()
    o, lse = c.attend(workspace=ws)
    c.L, c.T = c.L, [T] + [0] * 39
    check_attend(c, o, lse, rows_of=[0, T - 1])
    w.zero_()
    c.pages.weigh(c.batch, c.q, lse, w, 0.0)
    c.L = c.L[:1]
    c.T = c.T[:1]
    check_weigh(c, lse, torch.zeros_like(w), w, 0.0)
    assert c.pages.sync_status() == 0


@pytest.mark.parametrize("H,Hkv,T", [(10, 10, 1), (32, 8, 1), (32, 8, 70)])
def test_own_workspaces_after_waits_that_run_out(cuda_lib, H, Hkv, T):
    """The pool's own workspaces, of two streams and of a graph: sync_status leaves them
    fit for the next call."""
    rswa = cuda_lib
    c = Case(rswa, [900] * 40, [T] * 40, H, Hkv, 128, 32, seed=1, uniform=True)
    want, lse = c.attend()
    check_attend(c, want, lse, rows_of=[0])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o = torch.empty_like(want)
    with torch.cuda.stream(s):
        c.pages.attend(c.batch, c.q, o, lse)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            c.pages.attend(c.batch, c.q, o, lse)
    s.synchronize()
    told = 0
    for limit in [1] + [250 * x for x in range(1, 120)]:   # some CTAs give up, others have ended
        rswa.rswa_debug_set_wait_limit_ns(limit)
        try:
            c.attend()
            c.pages.attend(c.batch, c.q, o, lse, stream=s)
        finally:
            rswa.rswa_debug_set_wait_limit_ns(0)
        status = c.pages.sync_status()
        assert status in (0, RSWA_EDEVICE)
        told += status != 0
        assert torch.equal(c.attend()[0], want), limit
        o.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want), limit
        assert c.pages.sync_status() == 0
    assert told > 0


def test_attend_strided_queries_in_place_and_streams(cuda_lib):
    c = Case(cuda_lib, [200, 90], [30, 3], 10, 10, 128, 32, seed=2)
    qkv = torch.full((33, 30, 128), float("nan"), dtype=BF, device="cuda")
    qkv[:, :10] = c.q
    want, lse = c.attend()
    o = torch.empty_like(want)
    c.pages.attend(c.batch, qkv[:, :10], o)
    assert torch.equal(o, want)
    q = c.q.clone()
    c.pages.attend(c.batch, q, q)                      # in place, without lse
    assert torch.equal(q, want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o = torch.empty_like(want)
    c.pages.attend(c.batch, c.q, o, stream=s)
    s.synchronize()
    assert torch.equal(o, want)
    check_attend(c, want, lse, rows_of=[0, 29])


def test_rows_behind_the_last_sequence_stay(cuda_lib):
    for T in ([3, 2], [0, 0]):
        c = Case(cuda_lib, [50, 40], T, 8, 2, 128, 16, seed=3, stored=False)
        n = sum(T)
        pad = lambda x: torch.cat([x, torch.full((4, *x.shape[1:]), float("nan"), dtype=x.dtype, device="cuda")])
        c.pages.append(c.batch, pad(c.k), pad(c.v))
        for b in range(2):
            for pool, rows in ((c.Kp, c.K), (c.Vp, c.V)):
                assert torch.equal(c.tokens(pool, b, c.L[b]), rows[b])
        o = torch.full((n + 4, 8, 128), 7.0, dtype=BF, device="cuda")
        lse = torch.full((n + 4, 8), 7.0, device="cuda")
        c.pages.attend(c.batch, pad(c.q), o, lse)
        assert (o[n:] == 7).all() and (lse[n:] == 7).all()
        check_attend(c, o[:n], lse[:n])
        w = torch.zeros(2, 2, c.width * 16, device="cuda")
        c.pages.weigh(c.batch, pad(c.q), lse, w)
        assert torch.isfinite(w).all()
        assert c.pages.sync_status() == 0


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("H,Hkv,d,P,dtype", SHAPES)
@pytest.mark.parametrize("L,T,prefix,window", [LENGTHS[0], LENGTHS[1], LENGTHS[2], LENGTHS[7]])
@pytest.mark.parametrize("packed", [False, True])
def test_append(cuda_lib, H, Hkv, d, P, dtype, L, T, prefix, window, packed):
    c = Case(cuda_lib, L, T, H, Hkv, d, P, dtype, seed=5, stored=False, spare=1)
    before = c.Kp.clone(), c.Vp.clone()
    k, v = c.k, c.v
    if packed:
        kv = torch.stack((k, v), 1).reshape(len(k), 2 * Hkv, d).contiguous()
        k, v = kv[:, :Hkv], kv[:, Hkv:]
    c.pages.append(c.batch, k, v)
    for pool, old, rows in ((c.Kp, before[0], c.K), (c.Vp, before[1], c.V)):
        for b in range(len(L)):
            for p in range(-(-L[b] // P)):
                n = min(P, L[b] - p * P)
                old[c.where[b][p], :, :n] = rows[b][p * P:p * P + n].transpose(0, 1)
        assert torch.equal(torch.nan_to_num(pool.float(), 99.0), torch.nan_to_num(old.float(), 99.0))
    assert c.pages.sync_status() == 0


def test_append_of_many_sequences(cuda_lib):
    g = np.random.default_rng(1)
    T = [int(x) for x in g.integers(0, 4, 130)]
    L = [int(t + x) for t, x in zip(T, g.integers(0, 50, 130))]
    c = Case(cuda_lib, L, T, 4, 2, 64, 16, seed=6, stored=False)
    c.pages.append(c.batch, c.k, c.v)
    for b in range(130):
        assert torch.equal(c.tokens(c.Kp, b, L[b]), c.K[b]) and torch.equal(c.tokens(c.Vp, b, L[b]), c.V[b])


# ---------------------------------------------------------------------------
# weigh
# ---------------------------------------------------------------------------

def check_weigh(c, lse, old, got, decay, what=""):
    worst = 0.0
    for b in range(len(c.L)):
        L, rows = c.L[b], c.rows(b)
        ref = np.zeros((c.Hkv, L))
        size = np.zeros(1)
        if c.T[b]:
            ref = paged.weigh(f64(c.q[rows]), f64(c.K[b]), f64(lse[rows]), c.m[b], c.n)
            size = paged.attend(f64(c.q[rows]), f64(c.K[b]), f64(c.V[b]), c.m[b], c.n)[3]
        e = logit_error(c, size.max(), 0) + 2.0 ** -22 * np.abs(f64(lse[rows])).max(initial=0)
        want = ref + (decay * f64(old[b, :, :L]) if decay else 0)
        tol = e * ref + (c.T[b] * (c.H // c.Hkv) + 3) * 2.0 ** -24 * np.abs(want) + 1e-37
        err = np.abs(f64(got[b, :, :L]) - want)
        assert (err <= tol).all(), f"{what}: sequence {b}: {(err / tol).max():.3g} of the bound"
        worst = max(worst, (err / tol).max(initial=0))
        np.testing.assert_array_equal(f64(got[b, :, L:]), f64(old[b, :, L:]))
    return worst


@pytest.mark.parametrize("H,Hkv,d,P,dtype", SHAPES)
@pytest.mark.parametrize("L,T,prefix,window", LENGTHS)
@pytest.mark.parametrize("decay", [1.0, 0.0, 0.5])
def test_weigh(cuda_lib, H, Hkv, d, P, dtype, L, T, prefix, window, decay):
    if decay != 1.0 and len(L) not in (2, 5):
        pytest.skip("covered by the shorter lists")
    c = Case(cuda_lib, L, T, H, Hkv, d, P, dtype, prefix, window, seed=len(L) + H)
    _, lse = c.attend()
    old = torch.rand(len(L), Hkv, c.width * P, device="cuda")
    if decay == 0.0:
        old[:] = float("nan")                          # not read
    w = old.clone()
    c.pages.weigh(c.batch, c.q, lse, w, decay)
    check_weigh(c, lse, old, w, decay)
    again = old.clone()
    c.pages.weigh(c.batch, c.q, lse, again, decay)
    assert torch.equal(torch.nan_to_num(w, 9.0), torch.nan_to_num(again, 9.0))
    assert c.pages.sync_status() == 0


@pytest.mark.parametrize("H,Hkv,d,dtype", [(10, 10, 128, BF), (32, 8, 128, BF), (6, 2, 64, F32), (150, 1, 64, BF)])
def test_weigh_shapes(cuda_lib, H, Hkv, d, dtype):
    for L, T, m, n in (([700, 500], [300, 1], [16, 0], 100), ([1100], [9], None, None),
                       ([333] * 40, [1] * 40, None, None)):
        c = Case(cuda_lib, L, T, H, Hkv, d, 32, dtype, m, n, seed=9, uniform=m is None)
        _, lse = c.attend()
        old = torch.rand(len(L), Hkv, c.width * 32, device="cuda")
        w = old.clone()
        c.pages.weigh(c.batch, c.q, lse, w)
        check_weigh(c, lse, old, w, 1.0)


@pytest.mark.parametrize("H,Hkv", [(8, 8), (32, 8)])
@pytest.mark.parametrize("decay", [0.0, 0.5, 1.0])
@pytest.mark.parametrize("rows", [0, 1, 3])
def test_weigh_many_segments(cuda_lib, H, Hkv, decay, rows):
    """More (sequence, KV head) than the planner hands over at once to any CTA, most of
    which nobody sees, so that the warps that sum run ahead of those that fetch."""
    g = np.random.default_rng(rows)
    B = 400
    L = [int(x) for x in g.integers(rows + 1, 900, B)]
    live = set(g.choice(B, 25, replace=False).tolist()) if rows else set()
    T = [rows if b in live else 0 for b in range(B)]
    m = [int(x) for x in g.integers(0, 60, B)]
    c = Case(cuda_lib, L, T, H, Hkv, 64, 16, BF, m, 70, seed=rows, hole=1 << 30)
    c.m = [min(x, l) for x, l in zip(m, L)]
    lse = torch.empty(0, H, device="cuda")
    if rows:
        _, lse = c.attend()
    old = torch.rand(B, Hkv, c.width * 16, device="cuda")
    if decay == 0.0:
        old[:] = float("nan")                          # not read
    for _ in range(3):
        w = old.clone()
        c.pages.weigh(c.batch, c.q, lse, w, decay)
        assert c.pages.sync_status() == 0
        check_weigh(c, lse, old, w, decay)


def test_weigh_holes_are_not_read(cuda_lib):
    for dtype, T in ((BF, 1), (BF, 40), (F32, 3)):
        c = Case(cuda_lib, [600], [T], 8, 2, 128, 16, dtype, [5], 70, seed=T, hole=1 << 30)
        _, lse = c.attend()
        lo, hi = 5, 600 - T - 69
        for j in range(lo, hi):
            c.Kp[c.where[0][j // 16], :, j % 16] = float("nan")
        for p in range(-(-lo // 16), hi // 16):
            c.table[0, p] = -1
        old = torch.rand(1, 2, c.width * 16, device="cuda")
        w = old.clone()
        c.pages.weigh(c.batch, c.q, lse, w, 0.5)
        check_weigh(c, lse, old, w, 0.5)
        assert c.pages.sync_status() == 0


# ---------------------------------------------------------------------------
# evict
# ---------------------------------------------------------------------------

def run_evict(rswa, L, Hkv, d, P, dtype, budget, first, last, in_place, weights=None, seed=0, keep=True):
    B = len(L)
    c = Case(rswa, L, [0] * B, Hkv, Hkv, d, P, dtype, seed=seed, hole=-5)
    width = c.width * P
    w = torch.rand(B, Hkv, width, device="cuda") if weights is None else weights(B, Hkv, width)
    kept = torch.full((B, Hkv, budget), 77, dtype=torch.int32, device="cuda") if keep else None
    table_out, where = None, None
    if not in_place:
        # pages of its own: a larger pool
        need = [-(-min(x, budget) // P) for x in L]
        old = c.pages
        c.pages = rswa.RswaPages(old.pages + sum(need), P, Hkv, d, c.pages.dtype)
        K, V = c.pages.slabs()
        K.fill_(float("nan"))
        V.fill_(float("nan"))
        K[:old.pages], V[:old.pages] = c.Kp, c.Vp
        c.Kp, c.Vp = K, V
        ids = list(range(old.pages, old.pages + sum(need)))[::-1]
        where = [[ids.pop() for _ in range(x)] + [-9] * (c.width - x) for x in need]
        table_out = ints(where)
    before = c.Kp.clone(), c.Vp.clone()
    wo = w.clone() if in_place else torch.full_like(w, 5.0)
    src = wo if in_place else w
    c.pages.evict(c.batch, src, budget, first, last, table_out=table_out,
                  weights_out=None if in_place else wo, kept=kept)
    torch.cuda.synchronize()
    assert c.pages.sync_status() == 0
    wn = w.cpu().numpy()
    for b in range(B):
        n = min(L[b], budget)
        K, V = c.tokens(c.Kp, b, n, where), c.tokens(c.Vp, b, n, where)
        for h in range(Hkv):
            want = paged.evict(wn[b, h, :L[b]], budget, first, last)
            if keep:
                assert kept[b, h].tolist() == want + [-1] * (budget - n), (b, h)
            at = torch.tensor(want, dtype=torch.long, device="cuda")
            assert torch.equal(K[:, h], c.K[b][at, h]) and torch.equal(V[:, h], c.V[b][at, h]), (b, h)
            np.testing.assert_array_equal(wo[b, h, :n].cpu().numpy(), wn[b, h, want])
        assert (wo[b, :, n:] == 0).all()
    if not in_place:
        assert torch.equal(torch.nan_to_num(c.Kp[:old.pages].float(), 9.0),
                           torch.nan_to_num(before[0][:old.pages].float(), 9.0))


EVICT = [
    # L, budget, first, last
    ([1], 1, 0, 0), ([5, 0, 1, 9], 3, 1, 1), ([40, 17, 33], 16, 16, 0), ([40, 17, 33], 16, 0, 16),
    ([300, 64, 65, 129], 64, 3, 10), ([700], 1, 0, 0), ([700, 650], 333, 4, 128), ([90, 100], 200, 7, 9),
    ([1500], 1499, 0, 1), ([2500, 1100], 1025, 1, 700),
]


@pytest.mark.parametrize("L,budget,first,last", EVICT)
@pytest.mark.parametrize("Hkv,d,P,dtype", [(2, 128, 16, BF), (3, 64, 64, BF), (1, 64, 256, F32), (2, 128, 32, F32)])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict(cuda_lib, L, budget, first, last, Hkv, d, P, dtype, in_place):
    run_evict(cuda_lib, L, Hkv, d, P, dtype, budget, first, last, in_place, seed=len(L))


@pytest.mark.parametrize("in_place", [False, True])
def test_evict_ties_zeros_and_nan(cuda_lib, in_place):
    def few(*shape):
        return torch.randint(0, 3, shape, device="cuda").float()

    def zeros(*shape):
        return torch.randint(0, 2, shape, device="cuda").float() * -0.0

    def odd(*shape):
        x = torch.randn(shape, device="cuda")
        x[torch.rand(shape, device="cuda") < 0.3] = float("nan")
        x[torch.rand(shape, device="cuda") < 0.1] = float("inf")
        x[torch.rand(shape, device="cuda") < 0.1] = -float("inf")
        x[torch.rand(shape, device="cuda") < 0.1] = 1e-45
        return x

    for i, weights in enumerate((few, zeros, odd)):
        for budget in (1, 37, 300, 799):
            run_evict(cuda_lib, [800, 410], 2, 64, 16, BF, budget, min(budget, 5) // 2, budget // 3, in_place,
                      weights, seed=i)


def test_evict_long_sequences(cuda_lib):
    """More weights than shared memory holds, and rows that move far."""
    for in_place in (False, True):
        run_evict(cuda_lib, [60000], 1, 64, 256, BF, 9000, 16, 500, in_place, keep=False)
        run_evict(cuda_lib, [10272, 40], 2, 128, 64, BF, 2048, 16, 256, in_place)
    # the light ones first: every row moves, from behind its own chunk of rows
    run_evict(cuda_lib, [8000], 2, 128, 32, BF, 3500, 0, 0, True,
              lambda *s: torch.arange(s[-1], device="cuda").float().expand(*s).contiguous())


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("L,Hkv", [
    ([9000, 4097, 5], 2),             # clusters, weights in registers
    ([70000], 1),                     # more of them
    ([140000, 90000], 1),             # and read again
    ([4500] + [300] * 51, 3),         # a CTA for each head, in registers
    ([17000] + [40] * 51, 3),         # and read again
])
def test_evict_slices(cuda_lib, L, Hkv, in_place):
    """Ties and odd weights across the slices and rounds of long sequences."""
    def few(*shape):
        return torch.randint(0, 3, shape, device="cuda").float()

    def odd(*shape):
        x = torch.randn(shape, device="cuda")
        x[torch.rand(shape, device="cuda") < 0.3] = float("nan")
        x[torch.rand(shape, device="cuda") < 0.1] = float("inf")
        x[torch.rand(shape, device="cuda") < 0.1] = -0.0
        return x

    for i, weights in enumerate((few, odd, None)):
        for budget in (37, max(L) // 3, max(L) - 1):
            run_evict(cuda_lib, L, Hkv, 64, 256, BF, budget, budget // 5, budget // 3, in_place, weights, seed=i)


@pytest.mark.parametrize("L,spare", [([900, 30, 0], 0), ([900, 30, 0], 5), ([900, 30, 0], 60), ([700] * 80, 900),
                                     ([3000, 5], 1100)])
@pytest.mark.parametrize("budget", [1, 300, 2000])
def test_evict_wide_tables(cuda_lib, L, spare, budget):
    """Tables that could hold far more than the sequences: the weights' zeros behind what
    stays reach the table's end, over the weights and beside them."""
    B, Hkv, P = len(L), 2, 32
    for in_place in (True, False):
        c = Case(cuda_lib, L, [0] * B, Hkv, Hkv, 64, P, BF, seed=spare, spare=spare, hole=1 << 30)
        w = torch.rand(B, Hkv, c.width * P, device="cuda")
        wn, wo = w.cpu().numpy(), w if in_place else torch.full_like(w, 5.0)
        kept = torch.full((B, Hkv, budget), 77, dtype=torch.int32, device="cuda")
        K = c.Kp.clone()
        c.pages.evict(c.batch, w, budget, budget // 5, budget // 3, weights_out=wo, kept=kept)
        assert c.pages.sync_status() == 0
        for b in range(B):
            n = min(L[b], budget)
            assert (wo[b, :, n:] == 0).all()
            for h in range(Hkv):
                want = paged.evict(wn[b, h, :L[b]], budget, budget // 5, budget // 3)
                assert kept[b, h].tolist() == want + [-1] * (budget - n)
                at = torch.tensor(want, dtype=torch.long, device="cuda")
                assert torch.equal(c.tokens(c.Kp, b, n)[:, h], c.K[b][at, h])
                np.testing.assert_array_equal(wo[b, h, :n].cpu().numpy(), wn[b, h, want])
        if not in_place:
            assert torch.equal(w.cpu(), torch.from_numpy(wn))
        if budget >= max(L):
            assert torch.equal(torch.nan_to_num(c.Kp, 9.0), torch.nan_to_num(K, 9.0))


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("H,Hkv,d,P,dtype", [(10, 10, 128, 64, BF), (32, 8, 128, 16, BF), (4, 2, 64, 32, F32)])
def test_serving_run(cuda_lib, H, Hkv, d, P, dtype):
    """Prompts, single tokens, an eviction, more tokens: every step against the
    oracle on what the pages then are."""
    rswa = cuda_lib
    B, n, m, width = 3, 60, [5, 40, 0], 12 if P < 64 else 6
    pages = rswa.RswaPages(B * width, P, H, d, rswa.RSWA_F32 if dtype == F32 else rswa.RSWA_BF16, kv_heads=Hkv)
    where = np.random.default_rng(0).permutation(B * width).reshape(B, width)
    lens, starts = ints([0] * B), ints([0] * (B + 1))
    batch = rswa.RswaBatch(ints(where.tolist()), lens, starts, ints(m), n)
    weights = torch.zeros(B, Hkv, width * P, device="cuda")
    have = [(np.zeros((0, Hkv, d)), np.zeros((0, Hkv, d))) for _ in range(B)]
    total = np.zeros((B, Hkv, width * P))
    L = [0] * B
    steps = [[100, 57, 1], [1, 1, 1], [0, 20, 3], "evict", [1, 1, 1], [30, 0, 2], "evict", [1, 1, 1]]
    u = 2.0 ** -24
    for i, T in enumerate(steps):
        if T == "evict":
            budget = 48
            kept = torch.empty(B, Hkv, budget, dtype=torch.int32, device="cuda")
            w = weights.cpu().numpy()
            pages.evict(batch, weights, budget, 4, 16, kept=kept)
            for b in range(B):
                keep = [paged.evict(w[b, h, :L[b]], budget, 4, 16) for h in range(Hkv)]
                for h in range(Hkv):
                    assert kept[b, h, :len(keep[h])].tolist() == keep[h]
                have[b] = tuple(np.stack([x[keep[h], h] for h in range(Hkv)], 1) for x in have[b])
                new = np.zeros_like(total[b])
                for h in range(Hkv):
                    new[h, :len(keep[h])] = total[b, h, keep[h]]
                total[b] = new
                L[b] = min(L[b], budget)
            lens.clamp_(max=budget)
            continue
        rows = sum(T)
        at = np.concatenate([[0], np.cumsum(T)])
        lens += ints(T)
        starts.copy_(ints(at.tolist()))
        qkv = normal((rows, H + 2 * Hkv, d), 100 + i, dtype)
        q, k, v = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
        o = torch.empty(rows, H, d, dtype=dtype, device="cuda")
        lse = torch.empty(rows, H, device="cuda")
        pages.append(batch, k, v)
        pages.attend(batch, q, o, lse)
        pages.weigh(batch, q, lse, weights)
        for b in range(B):
            sl = slice(int(at[b]), int(at[b + 1]))
            have[b] = tuple(np.concatenate([x, f64(y[sl])]) for x, y in zip(have[b], (k, v)))
            L[b] += T[b]
            assert len(have[b][0]) == L[b] == int(lens[b])
            if T[b] == 0:
                continue
            ro, rl, mass, size = paged.attend(f64(q[sl]), *have[b], m[b], n)
            e = ((2 * (d + 8) + 4) * size + L[b]) * u + 2.0 ** -21
            tol = 2 * e[..., None] * mass + u * np.abs(ro)
            if dtype == BF:
                tol = tol + HALF[BF] * (mass + np.abs(ro) + tol)
            assert (np.abs(f64(o[sl]) - ro) <= tol).all(), (i, b)
            got = paged.weigh(f64(q[sl]), have[b][0], f64(lse[sl]), m[b], n)
            total[b, :, :L[b]] += got
            err = np.abs(f64(weights[b, :, :L[b]]) - total[b, :, :L[b]])
            # every step adds its own error to what was there
            bound = (e.max() + 2.0 ** -20 + 200 * u) * total[b, :, :L[b]] * (i + 1) + 1e-30
            assert (err <= bound).all(), (i, b, (err / bound).max())
    assert pages.sync_status() == 0


@pytest.mark.parametrize("H,Hkv", [(10, 10), (32, 8)])
def test_captured_step_replays_with_new_lengths(cuda_lib, H, Hkv):
    """A step of append, attention and weights in a graph: the lengths, pages and
    rows are read when it runs."""
    rswa = cuda_lib
    c = Case(rswa, [150, 90, 260], [1, 1, 1], H, Hkv, 128, 32, seed=8, spare=2, uniform=True)
    w = torch.zeros(3, Hkv, c.width * 32, device="cuda")
    o, lse = torch.empty_like(c.q), torch.empty(3, H, device="cuda")

    def step():
        c.pages.append(c.batch, c.k, c.v)
        c.pages.attend(c.batch, c.q, o, lse)
        c.pages.weigh(c.batch, c.q, lse, w, 0.0)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            step()
    s.synchronize()
    K, V = c.K, c.V
    for L in ([150, 90, 260], [33, 90, 1], [149, 2, 257]):
        c.L = L
        c.lens.copy_(ints(L))
        c.K = [x[:l] for x, l in zip(K, L)]
        c.V = [x[:l] for x, l in zip(V, L)]
        c.k.copy_(torch.stack([x[-1] for x in c.K]))
        c.v.copy_(torch.stack([x[-1] for x in c.V]))
        c.q.copy_(normal(c.q.shape, sum(L)))
        w.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        check_attend(c, o, lse)
        check_weigh(c, lse, w.clone(), w, 0.0)
    assert c.pages.sync_status() == 0


def test_captured_eviction_replays_with_new_weights(cuda_lib):
    """In place, in a graph: the lengths, weights and pages are read when it runs,
    and a call outside the graph on the same workspace leaves it as it was."""
    rswa = cuda_lib
    L0 = [700, 90, 4300]
    c = Case(rswa, L0, [0, 0, 0], 2, 2, 64, 32, seed=5)
    w = torch.rand(3, 2, c.width * 32, device="cuda")
    kept = torch.empty(3, 2, 128, dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c.pages.evict(c.batch, w, 128, 3, 20, kept=kept)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            c.pages.evict(c.batch, w, 128, 3, 20, kept=kept)
    s.synchronize()
    for i, L in enumerate((L0, [129, 40, 0], [699, 1, 4299], [128, 90, 4300])):
        assert all(x <= y for x, y in zip(L, L0))
        for b in range(3):
            c.write(b, L0[b])
        c.lens.copy_(ints(L))
        w.uniform_()
        wn = w.cpu().numpy()
        if i % 2:
            with torch.cuda.stream(s):
                s.wait_stream(torch.cuda.current_stream())
                c.pages.evict(c.batch, w, 128, 3, 20, kept=kept)
        else:
            graph.replay()
        torch.cuda.synchronize()
        for b in range(3):
            n = min(L[b], 128)
            for h in range(2):
                want = paged.evict(wn[b, h, :L[b]], 128, 3, 20)
                assert kept[b, h].tolist() == want + [-1] * (128 - n)
                at = torch.tensor(want, dtype=torch.long, device="cuda")
                assert torch.equal(c.tokens(c.Kp, b, n)[:, h], c.K[b][at, h])
                assert torch.equal(c.tokens(c.Vp, b, n)[:, h], c.V[b][at, h])
                np.testing.assert_array_equal(w[b, h, :n].cpu().numpy(), wn[b, h, want])
    assert c.pages.sync_status() == 0


def test_large_and_small_calls_overlap(cuda_lib):
    """Tiles of many rows, single tokens, weights and evictions of other pools on four
    streams at once."""
    rswa = cuda_lib
    big = Case(rswa, [3000, 700], [600, 1], 10, 10, 128, 64, seed=1)
    few = Case(rswa, [900] * 40, [1] * 40, 10, 10, 128, 32, seed=2)
    cut = Case(rswa, [5000, 60], [0, 0], 4, 4, 64, 16, seed=3)
    (ob, lb), (of, _) = big.attend(), few.attend()
    w0 = torch.rand(2, 4, cut.width * 16, device="cuda")
    w_big = torch.zeros(2, 10, big.width * 64, device="cuda")
    big.pages.weigh(big.batch, big.q, lb, w_big, 0.0)
    want = [paged.evict(w0[b, h, :n].cpu().numpy(), 300, 4, 30) for b, n in ((0, 5000), (1, 60)) for h in range(4)]
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    outs = []
    for _ in range(8):
        o1, o2 = torch.empty_like(ob), torch.empty_like(of)
        w1, w2 = torch.zeros_like(w_big), w0.clone()
        kept = torch.empty(2, 4, 300, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        big.pages.attend(big.batch, big.q, o1, stream=streams[0])
        few.pages.attend(few.batch, few.q, o2, stream=streams[1])
        big.pages.weigh(big.batch, big.q, lb, w1, 0.0, stream=streams[2])
        cut.pages.evict(cut.batch, w2, 300, 4, 30, kept=kept, stream=streams[3])
        big.pages.attend(big.batch, big.q, o1, stream=streams[0])
        outs.append((o1, o2, w1, kept))
    torch.cuda.synchronize()
    for o1, o2, w1, kept in outs:
        assert torch.equal(o1, ob) and torch.equal(o2, of)
        for b, n in ((0, 3000), (1, 700)):
            assert torch.equal(w1[b, :, :n], w_big[b, :, :n])
        got = [[x for x in row if x >= 0] for row in kept.flatten(0, 1).tolist()]
        assert got == want
    for c in (big, few, cut):
        assert c.pages.sync_status() == 0


def test_two_layers_share_a_batch_and_calls_overlap(cuda_lib):
    """Two pools, one description; two streams, each its own workspace."""
    rswa = cuda_lib
    a = Case(rswa, [500, 300], [40, 1], 32, 8, 128, 32, seed=1)
    b = Case(rswa, [500, 300], [40, 1], 32, 8, 128, 32, seed=1)
    b.batch = a.batch
    b.where, b.table = a.where, a.table
    want, _ = a.attend()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    outs = []
    for _ in range(20):
        for s, c in zip(streams, (a, b)):
            o = torch.empty_like(want)
            c.pages.attend(a.batch, a.q, o, stream=s)
            outs.append(o)
    # and both streams on one pool
    for s in streams:
        o = torch.empty_like(want)
        a.pages.attend(a.batch, a.q, o, stream=s)
        outs.append(o)
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, want)


def test_workspaces(cuda_lib):
    c = Case(cuda_lib, [900, 40], [1, 30], 32, 8, 128, 32, seed=1)
    want, _ = c.attend()
    ws = c.pages.attend_workspace(31)
    for _ in range(3):
        o, _ = c.attend(workspace=ws)
        assert torch.equal(o, want)
    with pytest.raises(cuda_lib.RswaError) as e:
        c.attend(workspace=ws[:256])
    assert e.value.status == 2
    big = c.pages.attend_workspace(5000)            # serves fewer rows
    assert torch.equal(c.attend(workspace=big)[0], want)
    with pytest.raises(ValueError):                    # a capture makes none
        s = torch.cuda.Stream()
        with torch.cuda.graph(torch.cuda.CUDAGraph(), stream=s):
            c.attend()


def test_eviction_with_a_workspace_of_its_own(cuda_lib):
    """On two streams at once, and in graphs that replay at the same time."""
    cases = [Case(cuda_lib, [700, 90, 4300], [0, 0, 0], 2, 2, 64, 32, seed=i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in cases]
    ws = [c.pages.evict_workspace(3, 128) for c in cases]
    ws[0].fill_(0x5a)                                  # any bits
    w = [torch.rand(3, 2, c.width * 32, device="cuda") for c in cases]
    kept = [torch.empty(3, 2, 128, dtype=torch.int32, device="cuda") for _ in cases]
    graphs = []
    capture = torch.cuda.Stream()
    for c, s, x, k in zip(cases, ws, w, kept):
        with torch.cuda.stream(capture):
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1], stream=capture):
                c.pages.evict(c.batch, x, 128, 3, 20, kept=k, workspace=s)
    for i in range(4):
        for c, x in zip(cases, w):
            x.uniform_()
            for b in range(3):
                c.write(b, c.L[b])
        wn = [x.cpu().numpy() for x in w]
        torch.cuda.synchronize()
        for c, s, x, k, st, g in zip(cases, ws, w, kept, streams, graphs):
            if i % 2:
                c.pages.evict(c.batch, x, 128, 3, 20, kept=k, workspace=s, stream=st)
            else:
                with torch.cuda.stream(st):
                    g.replay()
        torch.cuda.synchronize()
        for c, x, k in zip(cases, wn, kept):
            for b in range(3):
                for h in range(2):
                    want = paged.evict(x[b, h, :c.L[b]], 128, 3, 20)
                    assert k[b, h].tolist() == want + [-1] * (128 - len(want))
                    at = torch.tensor(want, dtype=torch.long, device="cuda")
                    assert torch.equal(c.tokens(c.Kp, b, len(want))[:, h], c.K[b][at, h])
            assert c.pages.sync_status() == 0


def test_one_workspace_serves_several_pools(cuda_lib):
    """Pools of unlike heads, one after the other and in a graph of all of them."""
    cases = [Case(cuda_lib, L, T, H, Hkv, d, 32, dtype, seed=H) for H, Hkv, d, dtype, L, T in (
        (10, 10, 128, BF, [900, 700], [300, 1]), (32, 8, 128, BF, [700] * 40, [1] * 40), (16, 2, 64, BF, [8000], [7]),
        (4, 2, 64, F32, [90, 700], [3, 1]), (10, 10, 128, BF, [300], [1]))]
    ws = max((c.pages.attend_workspace(sum(c.T)) for c in cases), key=torch.Tensor.numel)
    outs = [c.attend(workspace=ws) for c in cases]
    for c, (o, lse) in zip(cases, outs):
        check_attend(c, o, lse, rows_of=[0, 6, 299])
    again = [torch.empty_like(o) for o, _ in outs]
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=s):
        for c, o in zip(cases, again):
            c.pages.attend(c.batch, c.q, o, workspace=ws)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        for (o, _), x in zip(outs, again):
            assert torch.equal(o, x)
            x.zero_()
    for c in cases:
        assert not c.pages._attend_ws.all              # none made beside it
        assert c.pages.sync_status() == 0


def test_calls_by_handle(cuda_lib):
    """The functions that take a handle give what the class gives."""
    rswa = cuda_lib
    c = Case(rswa, [200, 90], [30, 3], 8, 2, 128, 32, seed=2, stored=False)
    need = rswa.rswa_pages_footprint(c.pages.pages, 32, 8, 2, 128, rswa.RSWA_BF16)
    buf = torch.zeros(need, dtype=torch.uint8, device="cuda")
    h = rswa.rswa_pages_create(c.pages.pages, 32, 8, 2, 128, rswa.RSWA_BF16, buf)
    assert rswa.rswa_pages_kv_offsets(h) == rswa.rswa_pages_kv_offsets(c.pages.handle)
    buf.copy_(c.pages.buf)
    c.pages.append(c.batch, c.k, c.v)
    rswa.rswa_pages_append(h, c.batch, c.k, 2 * 128, c.v, 2 * 128)
    assert torch.equal(buf, c.pages.buf)
    o, lse = c.attend()
    o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
    ws = torch.zeros(rswa.rswa_pages_attend_workspace(h, 33), dtype=torch.uint8, device="cuda")
    rswa.rswa_pages_attend(h, c.batch, c.q, 8 * 128, o2, ws, lse2)
    assert torch.equal(o2, o) and torch.equal(lse2, lse)
    w = torch.rand(2, 2, c.width * 32, device="cuda")
    w2 = w.clone()
    c.pages.weigh(c.batch, c.q, lse, w, 0.5)
    rswa.rswa_pages_weigh(h, c.batch, c.q, 8 * 128, lse, w2, 0.5)
    assert torch.equal(w2, w)
    kept, kept2 = (torch.empty(2, 2, 50, dtype=torch.int32, device="cuda") for _ in range(2))
    c.pages.evict(c.batch, w, 50, 4, 9, kept=kept)
    ws = torch.empty(rswa.rswa_pages_evict_workspace(h, 2, 50), dtype=torch.uint8, device="cuda")
    rswa.rswa_pages_evict(h, c.batch, w2, 50, 4, 9, w2, ws, kept=kept2)
    assert torch.equal(w2, w) and torch.equal(kept2, kept) and torch.equal(buf, c.pages.buf)
    assert rswa.rswa_pages_sync_status(h) == 0
    rswa.rswa_pages_destroy(h)
    with pytest.raises(rswa.RswaError):
        rswa.rswa_pages_append(h, c.batch, c.k, 2 * 128, c.v, 2 * 128)


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------

def test_bad_descriptions_are_flagged(cuda_lib):
    """A wrong sequence is left out, the others are served."""
    rswa = cuda_lib
    L, T = [100, 60, 30, 45], [3, 5, 2, 1]
    bad = [
        ("lens", 1, -1), ("lens", 1, 10 ** 6), ("lens", 1, 4),                  # fewer tokens than rows
        ("starts", 0, -2), ("starts", 4, 10 ** 6),
        ("table", 1, -1), ("table", 1, 10 ** 9),
    ]
    for what, b, value in bad:
        c = Case(rswa, L, T, 8, 2, 128, 16, seed=2)
        hit = {1} if what != "starts" else ({0} if b == 0 else {3})
        if what == "table":
            c.table[1, 0] = value
        else:
            (c.batch.lens if what == "lens" else c.batch.starts)[b] = value
        o, lse = c.attend()
        torch.cuda.synchronize()
        assert c.pages.sync_status() == RSWA_EDEVICE, (what, value)
        assert c.pages.sync_status() == 0
        for x in hit:
            if what != "table":
                assert torch.isnan(o[c.rows(x)]).all()
            c.T = [0 if y == x else t for y, t in enumerate(c.T)]
        check_attend(c, o, lse, what)
        w = torch.zeros(4, 2, c.width * 16, device="cuda")
        c.pages.weigh(c.batch, c.q, lse, w)
        assert c.pages.sync_status() == RSWA_EDEVICE, (what, value)
        before = c.Kp.clone()
        c.pages.append(c.batch, torch.zeros_like(c.k), torch.zeros_like(c.v))
        if what != "table":
            assert c.pages.sync_status() == RSWA_EDEVICE, (what, value)
            for x in hit:
                for p in range(-(-L[x] // 16)):
                    assert torch.equal(torch.nan_to_num(c.Kp[c.where[x][p]].float()),
                                       torch.nan_to_num(before[c.where[x][p]].float()))
        if what != "starts":
            c.pages.evict(c.batch, w, 20)
            assert (c.pages.sync_status() == RSWA_EDEVICE) == (value != 4), (what, value)


@pytest.mark.parametrize("H,Hkv,dtype", [(8, 2, BF), (4, 4, F32)])
@pytest.mark.parametrize("B,at", [(4, 1), (4, 2), (40, 5), (70, 33), (70, 64)])
@pytest.mark.parametrize("value", [10 ** 6, -7])
def test_a_wrong_range_in_the_middle_hides_no_other(cuda_lib, H, Hkv, dtype, B, at, value):
    """starts[at] out of range: the sequences before and behind it are empty, every other
    one is stored, attended and weighed."""
    g = np.random.default_rng(B + at)
    T = [int(x) for x in g.integers(1, 4, B)]
    L = [int(t + x) for t, x in zip(T, g.integers(0, 60, B))]
    c = Case(cuda_lib, L, T, H, Hkv, 64, 16, dtype, seed=at, stored=False)
    c.batch.starts[at] = value
    c.pages.append(c.batch, c.k, c.v)
    assert c.pages.sync_status() == RSWA_EDEVICE
    for b in range(B):
        old = L[b] - T[b]
        for pool, rows in ((c.Kp, c.K), (c.Vp, c.V)):
            got = c.tokens(pool, b, L[b])
            assert torch.equal(got[:old], rows[b][:old])
            if b in (at - 1, at):
                assert torch.isnan(got[old:]).all(), b
            else:
                assert torch.equal(got[old:], rows[b][old:]), b
    o, lse = c.attend()
    assert c.pages.sync_status() == RSWA_EDEVICE
    for b in (at - 1, at):
        assert torch.isnan(o[c.rows(b)]).all()
    c.T = [0 if b in (at - 1, at) else t for b, t in enumerate(T)]
    check_attend(c, o, lse)
    lse = torch.nan_to_num(lse)                        # of rows that nobody has
    w = torch.zeros(B, Hkv, c.width * 16, device="cuda")
    c.pages.weigh(c.batch, c.q, lse, w)
    assert c.pages.sync_status() == RSWA_EDEVICE
    check_weigh(c, lse, torch.zeros_like(w), w, 1.0)


@pytest.mark.parametrize("H,Hkv,dtype,rows", [(8, 2, BF, 1), (8, 2, BF, 300), (10, 10, BF, 40), (4, 4, F32, 2),
                                              (4, 4, F32, 900)])
@pytest.mark.parametrize("at,value", [(35, -1), (69, 10 ** 6), (64, -(1 << 31))])
def test_wrong_lengths_without_rows_are_flagged(cuda_lib, H, Hkv, dtype, rows, at, value):
    """All rows are the first sequence's; a length behind the first 32 is wrong."""
    L, T = [1000] + [20] * 69, [rows] + [0] * 69
    c = Case(cuda_lib, L, T, H, Hkv, 64, 16, dtype, seed=1)
    want, lse = c.attend()
    assert c.pages.sync_status() == 0
    c.lens[at] = value
    o, _ = c.attend()
    assert c.pages.sync_status() == RSWA_EDEVICE
    assert torch.equal(o, want)
    c.pages.append(c.batch, c.k, c.v)
    assert c.pages.sync_status() == RSWA_EDEVICE
    c.pages.weigh(c.batch, c.q, lse, torch.zeros(70, Hkv, c.width * 16, device="cuda"))
    assert c.pages.sync_status() == RSWA_EDEVICE


def test_refusals(cuda_lib):
    rswa = cuda_lib
    c = Case(rswa, [100, 60], [3, 2], 8, 2, 128, 16, seed=2)
    pages, batch = c.pages, c.batch
    o, lse = torch.empty_like(c.q), torch.empty(5, 8, device="cuda")
    w = torch.zeros(2, 2, c.width * 16, device="cuda")

    def refused(fn, kind=rswa.RswaError, status=1):
        with pytest.raises(kind) as e:
            fn()
        if kind is rswa.RswaError:
            assert e.value.status == status

    # shapes, types, devices
    refused(lambda: pages.attend(batch, c.q[:, :7], o), ValueError)
    refused(lambda: pages.attend(batch, c.q.float(), o), ValueError)
    refused(lambda: pages.attend(batch, c.q, o[:4]), ValueError)
    refused(lambda: pages.attend(batch, c.q, o, lse.double()), ValueError)
    refused(lambda: pages.attend(batch, c.q.cpu(), o), ValueError)
    refused(lambda: pages.append(batch, c.k, c.v[:4]), ValueError)
    refused(lambda: pages.append(batch, c.k, c.v.transpose(0, 1)), ValueError)
    refused(lambda: pages.weigh(batch, c.q, lse, w[:, :, :-1]), ValueError)
    refused(lambda: pages.evict(batch, w, 8, kept=torch.zeros(2, 2, 9, dtype=torch.int32, device="cuda")), ValueError)
    refused(lambda: pages.evict(batch, w, 8, table_out=c.table[:1]), ValueError)
    refused(lambda: rswa.RswaBatch(c.table, c.lens.long()), ValueError)
    refused(lambda: rswa.RswaBatch(c.table, c.lens, starts=c.lens), ValueError)
    refused(lambda: rswa.RswaBatch(c.table, c.lens, window=0), ValueError)
    refused(lambda: rswa.RswaBatch(c.table.t(), c.lens), ValueError)
    # rows that do not divide
    even = rswa.RswaBatch(c.table, c.lens)
    refused(lambda: pages.attend(even, c.q, o))
    refused(lambda: pages.append(even, c.k, c.v))
    refused(lambda: pages.weigh(even, c.q, lse, w))
    # alignment
    flat = torch.empty(5 * 8 * 128 + 8, dtype=BF, device="cuda")
    refused(lambda: pages.attend(batch, flat[4:4 + 5120].view(5, 8, 128), o))
    refused(lambda: pages.attend(batch, c.q, flat[4:4 + 5120].view(5, 8, 128)))
    # memory that is shared
    refused(lambda: pages.attend(batch, flat[:5120].view(5, 8, 128), flat[8:5128].view(5, 8, 128)))
    K, V = pages.slabs()
    refused(lambda: pages.attend(batch, c.q, K.reshape(-1)[:5120].view(5, 8, 128)))
    refused(lambda: pages.append(batch, V.reshape(-1)[:1280].view(5, 2, 128), c.v))
    refused(lambda: pages.attend(batch, c.q, o, o.view(torch.float32).reshape(-1)[:40].view(5, 8)))
    wide = torch.zeros(2, 2, 2 * c.width * 16, device="cuda").reshape(-1)
    half = w.numel()
    refused(lambda: pages.evict(batch, wide[:half].view(w.shape), 8, weights_out=wide[4:half + 4].view(w.shape)))
    refused(lambda: pages.evict(batch, w, 4, kept=w.reshape(-1)[:16].view(torch.int32).view(2, 2, 4)))
    refused(lambda: pages.weigh(batch, c.q, w.reshape(-1)[:40].view(5, 8), w))
    # numbers
    for kw in (dict(budget=0), dict(budget=-1), dict(budget=8, first=-1), dict(budget=8, last=-1),
               dict(budget=8, first=5, last=4), dict(budget=8, first=9), dict(budget=(1 << 30) + 1)):
        refused(lambda: pages.evict(batch, w, workspace=torch.zeros(1 << 16, dtype=torch.uint8, device="cuda"), **kw))
    for decay in (-0.1, 1.5, float("nan")):
        refused(lambda: pages.weigh(batch, c.q, lse, w, decay))
    small = torch.zeros(256, dtype=torch.uint8, device="cuda")
    refused(lambda: pages.evict(batch, w, 8, workspace=small), status=2)
    # CUDA failures
    for call in (lambda: pages.append(batch, c.k, c.v), lambda: pages.attend(batch, c.q, o),
                 lambda: pages.weigh(batch, c.q, lse, w), lambda: pages.evict(batch, w, 8)):
        rswa.rswa_debug_fail_next_cuda(1)
        refused(call, status=5)
    # a closed pool
    pages.close()
    refused(lambda: pages.append(batch, c.k, c.v), status=4)
    assert pages.sync_status() == 4


def test_eviction_workspaces_that_wrap(cuda_lib):
    """Heads times budget whose bytes pass 64 bits."""
    rswa = cuda_lib
    pages = rswa.RswaPages(1, 16, 4096, 64, rswa.RSWA_BF16)
    for batch, budget in ((1 << 20, 1 << 30), (1 << 20, 1), (1 << 19, 1 << 30)):
        with pytest.raises(rswa.RswaError) as e:
            rswa.rswa_pages_evict_workspace(pages.handle, batch, budget)
        assert e.value.status == 1
    for batch, budget in (((1 << 19) - 1, 1 << 30), (1000, 1 << 30), (3, 7)):
        # the kept tokens, and a word for every part of the move
        assert rswa.rswa_pages_evict_workspace(pages.handle, batch, budget) >= batch * 4096 * (budget + budget // 64) * 4


def test_a_pool_in_memory_that_is_still_written(cuda_lib):
    """Made on a stream whose queued work writes the block that the pool then gets."""
    rswa = cuda_lib
    need = rswa.rswa_pages_footprint(300, 16, 4, 4, 64, rswa.RSWA_BF16)
    s = torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s):
            old = torch.empty(need, dtype=torch.uint8, device="cuda")
            at = old.data_ptr()
            torch.cuda._sleep(100_000_000)             # some 50 ms
            old.fill_(1)
            del old
            pages = rswa.RswaPages(300, 16, 4, 64, rswa.RSWA_BF16)
        assert pages.buf.data_ptr() == at
        assert pages.sync_status() == 0
        pages.close()


def test_no_rows(cuda_lib):
    c = Case(cuda_lib, [100, 60], [0, 0], 8, 2, 128, 16, seed=2)
    c.pages.append(c.batch, c.k, c.v)
    c.pages.attend(c.batch, c.q, torch.empty_like(c.q))
    w = torch.ones(2, 2, c.width * 16, device="cuda")
    c.pages.weigh(c.batch, c.q, torch.empty(0, 8, device="cuda"), w, 0.5)
    for b in range(2):
        assert (w[b, :, :c.L[b]] == 0.5).all() and (w[b, :, c.L[b]:] == 1).all()
    assert c.pages.sync_status() == 0


def test_pool_beyond_32_bit_offsets(cuda_lib):
    """Pages whose elements lie past 2^32 bytes and 2^31 elements."""
    rswa = cuda_lib
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    H, Hkv, d, P = 8, 4, 128, 256
    count = (1 << 31) // (Hkv * d * P) + 40
    pages = rswa.RswaPages(count, P, H, d, rswa.RSWA_BF16, kv_heads=Hkv)
    K, V = pages.slabs()
    c = Case(rswa, [900, 300], [4, 1], H, Hkv, d, P, seed=3, stored=False)
    ids = [count - 1 - i for i in range(8)]
    where = [[ids.pop() for _ in range(c.width)] for _ in range(2)]
    c.table.copy_(ints(where))
    c.where, c.pages, c.Kp, c.Vp = where, pages, K, V
    for b in range(2):
        c.write(b, c.L[b] - c.T[b])
    pages.append(c.batch, c.k, c.v)
    check_attend(c, *c.attend())
    _, lse = c.attend()
    w = torch.zeros(2, Hkv, c.width * P, device="cuda")
    pages.weigh(c.batch, c.q, lse, w)
    check_weigh(c, lse, torch.zeros_like(w), w, 1.0)
    wn = w.cpu().numpy()
    pages.evict(c.batch, w, 200, 4, 50)
    for b in range(2):
        for h in range(Hkv):
            at = torch.tensor(paged.evict(wn[b, h, :c.L[b]], 200, 4, 50), device="cuda")
            assert torch.equal(c.tokens(K, b, 200)[:, h], c.K[b][at, h])
            assert torch.equal(c.tokens(V, b, 200)[:, h], c.V[b][at, h])


def test_refusals_of_counts_that_wrap(cuda_lib):
    """Rows and weights whose products pass 64 bits."""
    c = Case(cuda_lib, [100], [3], 16, 16, 64, 16, seed=3)
    pages, lib = c.pages, c.pages._lib
    o, lse, w = torch.empty_like(c.q), torch.empty(3, 16, device="cuda"), torch.zeros(1, 16, c.width * 16, device="cuda")
    ws = torch.zeros(cuda_lib.rswa_pages_attend_workspace(pages.handle, 3), dtype=torch.uint8, device="cuda")
    for rows in (1 << 60, 1 << 59, (1 << 63) - 1, (1 << 31) // 16):
        stride = 16 * 64
        assert lib.rswa_pages_append(pages.handle, c.batch.ref, rows, c.k.data_ptr(), stride, c.v.data_ptr(), stride,
                                     None) == 1
        assert lib.rswa_pages_attend(pages.handle, c.batch.ref, rows, c.q.data_ptr(), stride, o.data_ptr(),
                                     lse.data_ptr(), ws.data_ptr(), ws.numel(), None) == 1
        assert lib.rswa_pages_weigh(pages.handle, c.batch.ref, rows, c.q.data_ptr(), stride, lse.data_ptr(),
                                    w.data_ptr(), 1.0, None) == 1
    assert pages.sync_status() == 0
