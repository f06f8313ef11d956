"""Cases of the draft-and-verify operators: what they are timed on, and their plain forms.

Four operators that stand around the attention of a cache of a static prefix
(m_b tokens) and a ring of the last n outputs:

* ``norm_rope``: RMS norm of every query and key head, then the rotation by
  the row's position, in one pass.
* ``append``: the same for one new token per sequence at position m_b + t_b,
  whose key and value go to ring slot t_b mod n.
* ``tree``: attention of a tree of drafted tokens over the cache.  Node i has
  a parent before it (or -1) and counts as output t_b + depth(i); it sees the
  prefix, the cached outputs of its window and its own ancestors.
* ``commit``: the accepted path of a tree goes to the ring.

``own`` chooses between the plain forms (elementary torch operations) and the
package's kernels.
"""

import random

import torch

own = False

EPS = 1e-6
THETA = 10000.0
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    bf = {"dtype": "bf16", "d": 128, "rot": 128, "interleaved": False}
    one = {"B": 1, "H": 10, "Hkv": 10}
    batch = {"B": 64, "H": 10, "Hkv": 10}
    grouped = {"B": 64, "H": 32, "Hkv": 8}
    page = {"n": 128, "m_lo": 288, "m": 288, "t_lo": 200, "t": 200}
    ragged = {"n": 128, "m_lo": 256, "m": 2048, "t_lo": 40, "t": 200}
    return [
        # the prompt of one page (256 visual tokens and 32 of text) before its prefill
        dict(**bf, name="norm_rope page prompt", op="norm_rope", rows=288, H=10, Hkv=10, norm=True, packed=True, docs=1,
             pos0=0),
        # the 32K rows of a 40-page document, one layer
        dict(**bf, name="norm_rope 32K rows", op="norm_rope", rows=32768, H=10, Hkv=10, norm=True, packed=True, docs=1,
             pos0=0),
        # packed documents in float32 with grouped heads, a partial interleaved rotation, far positions, odd row count
        dict(name="norm_rope grouped f32", op="norm_rope", dtype="f32", d=64, rot=32, interleaved=True, rows=4099,
             H=32, Hkv=8, norm=True, packed=False, docs=5, pos0=100000),
        # the next token of one page: latency
        dict(**bf, **one, **page, name="append page", op="append"),
        # the next token of a served batch with grouped heads
        dict(**bf, **grouped, **ragged, name="append batch", op="append"),
        # 16 drafted tokens of one page: latency
        dict(**bf, **one, **page, name="tree page", op="tree", nodes=16, cnt_lo=16),
        # drafts of a served batch, trees of different sizes padded to one
        dict(**bf, **batch, **ragged, name="tree batch", op="tree", nodes=32, cnt_lo=9),
        # wide trees with grouped heads: 256 query rows for each key head
        dict(**bf, **grouped, **ragged, name="tree batch grouped", op="tree", nodes=64, cnt_lo=64),
        # one sequence after a 40-page document
        dict(**bf, **one, name="tree 40 pages", op="tree", n=128, m_lo=10272, m=10272, t_lo=150, t=150, nodes=61,
             cnt_lo=61),
        # the parity type
        dict(name="tree f32", op="tree", dtype="f32", d=64, rot=64, interleaved=False, B=2, H=4, Hkv=2, n=77,
             m_lo=290, m=310, t_lo=30, t=100, nodes=33, cnt_lo=20),
        # what is accepted of a page's draft
        dict(**bf, **one, **page, name="commit page", op="commit", nodes=16, path=5),
        # and of a batch's drafts, some of them rejected whole
        dict(**bf, **grouped, **ragged, name="commit batch", op="commit", nodes=64, path=9),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["norm_rope", "append", "tree", "tree", "commit"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    d = rng.choice([64, 128, 128])
    H, Hkv = rng.choice([(10, 10), (10, 10), (32, 8) if d == 128 else (20, 5), (8, 1), (12, 4), (5, 5), (6, 2),
                         (16, 2)])
    rot = rng.choice([d, d, d // 2, 16 * rng.randint(1, d // 16)])
    c = {"op": op, "dtype": dtype, "d": d, "rot": rot, "interleaved": rng.random() < 0.3, "H": H, "Hkv": Hkv}
    elt = 2 if dtype == "bf16" else 4
    if op == "norm_rope":
        most = 160_000_000 // ((H + Hkv) * d * elt)
        rows = _log(rng, 1, min(32768, most))
        return dict(c, rows=rows, norm=rng.random() < 0.8, packed=rng.random() < 0.5,
                    docs=rng.randint(1, min(rows, 9)), pos0=rng.choice([0, 0, 37, 100000]))
    if op in ("append", "commit"):
        m = _log(rng, 1, 1100)
        c = dict(c, B=_log(rng, 1, 96), n=_log(rng, 4, 300), m_lo=rng.randint(0, m), m=m)
        t = rng.randint(0, 2 * c["n"])
        c = dict(c, t_lo=rng.randint(0, t), t=t)
        if op == "commit":
            nodes = _log(rng, 1, 200)
            c = dict(c, nodes=nodes, path=rng.randint(1, min(nodes, 24)))
        return c
    if dtype == "f32":
        c = dict(c, B=rng.randint(1, 3), nodes=_log(rng, 1, 64))
        m = _log(rng, 1, 600)
    else:
        B = _log(rng, 1, 64)
        c = dict(c, B=B, nodes=_log(rng, 1, 256 if B < 16 else 64))
        m = _log(rng, 16, min(10272, 100_000_000 // (B * Hkv * d * 4)))
    n = _log(rng, 8, 300)
    t = rng.randint(0, 2 * n)
    return dict(c, n=n, m_lo=rng.randint(0, m), m=m, t_lo=rng.randint(0, t), t=t, cnt_lo=rng.randint(1, c["nodes"]))


def _lengths(case):
    """Prefix lengths, outputs so far, and live nodes or accepted tokens of
    each sequence: the same for every seed, so that the work of a case is."""
    rng = random.Random(7 * case["B"] + case["m"])
    B = case["B"]
    m = [rng.randint(case["m_lo"], case["m"]) for _ in range(B)]
    t = [rng.randint(case["t_lo"], case["t"]) for _ in range(B)]
    if case["op"] == "tree":
        return m, t, [rng.randint(case["cnt_lo"], case["nodes"]) for _ in range(B)]
    if case["op"] == "commit":
        return m, t, [rng.randint(0 if B > 1 else 1, case["path"]) for _ in range(B)]
    return m, t, [1] * B


def _device():
    return "cuda" if torch.cuda.is_available() else "cpu"


def _inv_freq(rot):
    """Radians a position for each rotated pair, in 64 bits."""
    i = torch.arange(rot // 2, dtype=torch.float64, device=_device())
    return THETA ** (-2.0 * i / rot)


def _inputs(case, seed):
    """The tensors of a case: drawn in 32 bits, rounded once."""
    dev, dt = _device(), DTYPES[case["dtype"]]
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=g, device=dev) * std).to(dt)

    H, Hkv, d, op = case["H"], case["Hkv"], case["d"], case["op"]
    x = {}
    if op in ("norm_rope", "append"):
        rows = case["rows"] if op == "norm_rope" else case["B"]
        if op == "append" or case["packed"]:
            # what one projection gives: the queries, keys and values of a row side by side
            qkv = normal(rows, H + 2 * Hkv, d)
            x["q"], x["k"], x["v"] = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
        else:
            x["q"], x["k"] = normal(rows, H, d), normal(rows, Hkv, d)
        x["inv_freq"] = _inv_freq(case["rot"])
        if op == "append" or case["norm"]:
            x["qw"] = (1 + 0.2 * torch.randn(d, generator=g, device=dev)).to(dt)
            x["kw"] = (1 + 0.2 * torch.randn(d, generator=g, device=dev)).to(dt)
        else:
            x["qw"] = x["kw"] = None
        if op == "norm_rope":
            each = -(-rows // case["docs"])
            x["pos"] = torch.arange(rows, device=dev) % each + case["pos0"]
            return x
    m, t, third = _lengths(case)
    B = case["B"]
    x["m"], x["t"] = m, t
    x["K"], x["V"] = normal(sum(m) + sum(t), Hkv, d), normal(sum(m) + sum(t), Hkv, d)
    if op == "append":
        return x
    N = case["nodes"]
    x["k"], x["v"] = normal(B, N, Hkv, d), normal(B, N, Hkv, d)
    rng = random.Random(seed)
    if op == "commit":
        path = [sorted(rng.sample(range(N), a)) + [0] * (case["path"] - a) for a in third]
        x["path"] = torch.tensor(path, dtype=torch.int32, device=dev)
        x["accepted"] = torch.tensor(third, dtype=torch.int32, device=dev)
        return x
    x["q"] = normal(B, N, H, d)
    # drafts: often the next token of a chain, else a branch from one of the last 16 nodes
    parents = [[-1 if i == 0 or rng.random() < 0.05 else i - 1 if rng.random() < 0.3 else
                rng.randrange(max(0, i - 16), i) for i in range(N)] for _ in range(B)]
    x["parents"] = torch.tensor(parents, dtype=torch.int32, device=dev)
    x["counts"] = torch.tensor(third, dtype=torch.int32, device=dev)
    return x


def prepare(case, seed):
    x = _inputs(case, seed)
    s = dict(x, op=case["op"], case=case)
    if own:
        import sliding_window_attention_02_gb300 as rswa
        if "inv_freq" in x:
            s["rope"] = rswa.RswaRope(x["inv_freq"], x["qw"], x["kw"], eps=EPS, interleaved=case["interleaved"])
        s["rswa"] = rswa
    if case["op"] != "norm_rope":
        B, Hkv, d, n, cap = case["B"], case["Hkv"], case["d"], case["n"], case["m"]
        K, V = s.pop("K"), s.pop("V")
        if own:
            dtype = rswa.RSWA_F32 if case["dtype"] == "f32" else rswa.RSWA_BF16
            s["cache"] = rswa.RswaCache(cap, n, case["H"], d, B, dtype, kv_heads=Hkv)
            s["cache"].prefill_varlen(None, K, V, None, x["m"], x["t"])
            s["Ks"], s["Vs"] = s["cache"].slabs()
        else:
            # the cache: prefix rows, then output j in row cap + j mod n
            s["Ks"] = torch.zeros(B, Hkv, cap + n, d, dtype=K.dtype, device=K.device)
            s["Vs"] = torch.zeros_like(s["Ks"])
            at = 0
            for b in range(B):
                m, t = x["m"][b], x["t"][b]
                keep = torch.arange(max(0, t - n), t, device=K.device)
                for slab, rows in ((s["Ks"], K), (s["Vs"], V)):
                    slab[b, :, :m] = rows[at:at + m].transpose(0, 1)
                    slab[b, :, cap + keep % n] = rows[at + m + keep].transpose(0, 1)
                at += m + t
            s["m"] = torch.tensor(x["m"], device=K.device)
            s["t"] = torch.tensor(x["t"], device=K.device)
        s["ring"] = (s["Ks"][:, :, cap:], s["Vs"][:, :, cap:])
    if case["op"] == "tree":
        s["o"] = torch.zeros_like(x["q"])
        s["lse"] = torch.zeros(x["q"].shape[:3], device=x["q"].device)
    elif "q" in x:
        s["q_out"] = torch.empty(x["q"].shape, dtype=x["q"].dtype, device=x["q"].device)
        s["k_out"] = torch.empty(x["k"].shape, dtype=x["k"].dtype, device=x["k"].device)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _normed_rotated(x, w, pos, inv_freq, interleaved):
    """RMS norm of each head of x [rows][heads][d] (where w is given), then the
    rotation of the first 2 len(inv_freq) elements.  The angles are taken in
    64 bits: a far position times a frequency does not fit 32."""
    y = x.float()
    if w is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + EPS) * w.float()
    rot = 2 * inv_freq.numel()
    ang = pos.double()[:, None, None] * inv_freq
    c, s = torch.cos(ang).float(), torch.sin(ang).float()
    z, rest = y[..., :rot], y[..., rot:]
    if interleaved:
        a, b = z[..., 0::2], z[..., 1::2]
        z = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    else:
        a, b = z[..., :rot // 2], z[..., rot // 2:]
        z = torch.cat((a * c - b * s, b * c + a * s), -1)
    return torch.cat((z, rest), -1).to(x.dtype)


def _norm_rope(s):
    il = s["case"]["interleaved"]
    return (_normed_rotated(s["q"], s["qw"], s["pos"], s["inv_freq"], il),
            _normed_rotated(s["k"], s["kw"], s["pos"], s["inv_freq"], il))


def _append(s):
    il, pos = s["case"]["interleaved"], s["m"] + s["t"]
    q = _normed_rotated(s["q"], s["qw"], pos, s["inv_freq"], il)
    k = _normed_rotated(s["k"], s["kw"], pos, s["inv_freq"], il)
    b, slot = torch.arange(len(pos), device=pos.device), s["t"] % s["case"]["n"]
    s["ring"][0][b, :, slot] = k
    s["ring"][1][b, :, slot] = s["v"]
    s["t"] += 1
    return q, s["ring"][0], s["ring"][1]


def _commit(s):
    """Slot x takes the last accepted token i with (t + i) mod n = x."""
    n = s["case"]["n"]
    x = torch.arange(n, device=s["t"].device)
    first = (x - s["t"][:, None]) % n
    acc = s["accepted"].long()[:, None]
    i = first + (acc - 1 - first).div(n, rounding_mode="floor") * n
    hit = first < acc
    node = s["path"].long().gather(1, i.clamp(0, s["path"].shape[1] - 1))
    for ring, rows in ((s["ring"][0], s["k"]), (s["ring"][1], s["v"])):
        new = rows.gather(1, node[:, :, None, None].expand(-1, -1, *rows.shape[2:])).transpose(1, 2)
        ring.copy_(torch.where(hit[:, None, :, None], new, ring))
    s["t"] += acc[:, 0]
    return s["ring"]


def _tree(s):
    c = s["case"]
    B, N, H, d = s["q"].shape
    Hkv, n, cap = c["Hkv"], c["n"], c["m"]
    dev = s["q"].device
    # reach[i, a]: a is i or an ancestor of i (paths of up to 2^k steps after k squarings)
    par = s["parents"].long()
    node = torch.arange(N, device=dev)
    reach = ((par[:, :, None] == node) | (node[:, None] == node)).float()
    for _ in range((N - 1).bit_length()):
        reach = (torch.bmm(reach, reach) > 0).float()
    depth = reach.sum(-1) - 1
    m, t = s["m"][:, None], s["t"][:, None]
    # cached outputs: slot x holds the output that is `age` older than the newest
    age = (t - 1 - torch.arange(n, device=dev)) % n
    lim = torch.minimum(t - 1, n - 2 - depth.long())
    sees_ring = age[:, None, :] <= lim[:, :, None]
    sees_prefix = (torch.arange(cap, device=dev) < m)[:, None, :].expand(-1, N, -1)
    sees_tree = (reach > 0) & (depth[:, :, None] - depth[:, None, :] < n)
    sees = torch.cat((sees_prefix, sees_ring, sees_tree), -1)[:, None, None]
    q = s["q"].float().view(B, N, Hkv, H // Hkv, d).permute(0, 2, 3, 1, 4)
    k = torch.cat((s["Ks"].float(), s["k"].float().transpose(1, 2)), 2)
    v = torch.cat((s["Vs"].float(), s["v"].float().transpose(1, 2)), 2)
    x = torch.matmul(q.reshape(B, Hkv, -1, d), k.transpose(-1, -2)) * d ** -0.5
    x = x.view(B, Hkv, H // Hkv, N, -1).masked_fill(~sees, float("-inf"))
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, Hkv, -1, p.shape[-1]), v).view(B, Hkv, H // Hkv, N, d) / total
    lse = (top + torch.log(total))[..., 0]
    live = (node < s["counts"][:, None])[:, :, None]
    s["o"] = torch.where(live[..., None], o.permute(0, 3, 1, 2, 4).reshape(B, N, H, d).to(s["o"].dtype), s["o"])
    s["lse"] = torch.where(live, lse.permute(0, 3, 1, 2).reshape(B, N, H), s["lse"])
    return s["o"], s["lse"]


def _own(s):
    if s["op"] == "norm_rope":
        s["rswa"].rswa_qk_norm_rope(s["rope"], s["q"], s["k"], s["pos"], s["q_out"], s["k_out"])
        return s["q_out"], s["k_out"]
    if s["op"] == "append":
        s["cache"].append_kv_rope(s["rope"], s["q"], s["k"], s["v"], s["q_out"])
        return s["q_out"], s["ring"][0], s["ring"][1]
    if s["op"] == "tree":
        s["cache"].decode_tree(s["q"], s["k"], s["v"], s["parents"], s["o"], s["lse"], counts=s["counts"])
        return s["o"], s["lse"]
    s["cache"].commit_tree(s["k"], s["v"], s["path"], s["accepted"])
    return s["ring"]


def run(s):
    if own:
        return _own(s)
    return {"norm_rope": _norm_rope, "append": _append, "tree": _tree, "commit": _commit}[s["op"]](s)


def work(case):
    H, Hkv, d = case["H"], case["Hkv"], case["d"]
    elt = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "norm_rope":
        return {"bytes": case["rows"] * ((H + Hkv) * d * elt * 2 + 8), "flops": case["rows"] * (H + Hkv) * d * 7}
    m, t, third = _lengths(case)
    if case["op"] == "append":
        return {"bytes": 2 * case["B"] * (H + 2 * Hkv) * d * elt, "flops": case["B"] * (H + Hkv) * d * 7}
    if case["op"] == "commit":
        return {"bytes": 4 * sum(third) * Hkv * d * elt, "flops": 0}
    keys = [a + min(case["n"], b) for a, b in zip(m, t)]
    return {"bytes": sum(2 * (a + c) * Hkv * d * elt + c * H * (2 * d * elt + 4) for a, c in zip(keys, third)),
            "flops": sum(4 * d * H * c * (a + 1) for a, c in zip(keys, third))}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_rotated(x, w, pos, inv_freq, interleaved):
    """Each pair as a complex number, turned by exp(i pos f)."""
    x = x.double()
    if w is not None:
        x = x * w.double() * ((x ** 2).sum(-1) / x.shape[-1] + EPS).rsqrt().unsqueeze(-1)
    half = inv_freq.numel()
    turn = torch.polar(torch.ones(len(pos), half, dtype=torch.float64, device=x.device),
                       torch.outer(pos.double(), inv_freq)).unsqueeze(1)
    out = x.clone()
    i = torch.arange(half, device=x.device)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    z = torch.complex(x[..., a], x[..., b]) * turn
    out[..., a], out[..., b] = z.real, z.imag
    return out


def exact(case, seed):
    x = _inputs(case, seed)
    op, il = case["op"], case["interleaved"]
    if op == "norm_rope":
        return tuple(_exact_rotated(x[i], x[i + "w"], x["pos"], x["inv_freq"], il) for i in "qk")
    m, t, third = _lengths(case)
    B, H, Hkv, d, n = case["B"], case["H"], case["Hkv"], case["d"], case["n"]
    dev = x["K"].device
    at, first = 0, []
    for b in range(B):
        first.append(at + m[b])                 # row of the sequence's output 0
        at += m[b] + t[b]
    if op in ("append", "commit"):
        ring = torch.zeros(2, B, Hkv, n, d, dtype=torch.float64, device=dev)
        if op == "append":
            pos = torch.tensor([i + j for i, j in zip(m, t)], device=dev)
            q = _exact_rotated(x["q"], x["qw"], pos, x["inv_freq"], il)
            k = _exact_rotated(x["k"], x["kw"], pos, x["inv_freq"], il)
            new = [[(k[b], x["v"][b])] for b in range(B)]
        else:
            path = x["path"].tolist()
            new = [[(x["k"][b, i], x["v"][b, i]) for i in path[b][:third[b]]] for b in range(B)]
        for b in range(B):
            for j in range(max(0, t[b] - n), t[b]):
                ring[0, b, :, j % n], ring[1, b, :, j % n] = x["K"][first[b] + j], x["V"][first[b] + j]
            for j, (kk, vv) in enumerate(new[b], t[b]):
                ring[0, b, :, j % n], ring[1, b, :, j % n] = kk, vv
        return (q, ring[0], ring[1]) if op == "append" else (ring[0], ring[1])
    N, G = case["nodes"], H // Hkv
    o = torch.zeros(B, N, H, d, dtype=torch.float64, device=dev)
    lse = torch.zeros(B, N, H, dtype=torch.float64, device=dev)
    parents = x["parents"].tolist()
    for b in range(B):
        rows = slice(first[b] - m[b], first[b] + t[b])
        K = torch.cat((x["K"][rows], x["k"][b])).double().transpose(0, 1)       # prefix, outputs, nodes
        V = torch.cat((x["V"][rows], x["v"][b])).double().transpose(0, 1)
        chains = []
        for i in range(third[b]):
            chains.append([i] + (chains[parents[b][i]] if parents[b][i] >= 0 else []))
        sees = torch.zeros(len(chains), K.shape[1], dtype=torch.bool)
        sees[:, :m[b]] = True
        for i, chain in enumerate(chains):
            here = t[b] + len(chain) - 1        # the output that the node stands for
            sees[i, m[b] + max(0, here - n + 1):m[b] + t[b]] = True
            sees[i, [m[b] + t[b] + a for a in chain[:n]]] = True
        c = len(chains)
        q = x["q"][b, :c].double().view(c, Hkv, G, d).permute(1, 2, 0, 3)
        logits = torch.einsum("hgcd,hsd->hgcs", q, K) / d ** 0.5
        logits = logits.masked_fill(~sees.to(dev), float("-inf"))
        l = torch.logsumexp(logits, -1)
        out = torch.einsum("hgcs,hsd->hgcd", torch.exp(logits - l.unsqueeze(-1)), V)
        o[b, :c] = out.permute(2, 0, 1, 3).reshape(c, H, d)
        lse[b, :c] = l.permute(2, 0, 1).reshape(c, H)
    return o, lse
