"""Cases of the paged-cache operators: what they are timed on, and their plain forms.

A paged cache keeps keys and values in a pool of pages, [pages][kv_heads][page
size][d]; a table names the pages of each sequence.  Four operators:

* ``append``: a chunk of new tokens of every sequence goes to its pages.
* ``attend``: attention of the chunk over the pages.  Token i sees token j <= i
  when j is one of the sequence's first m_b tokens (its prefix, or a few that
  stay visible) or j > i - n (the window; n of None: every token).
* ``weigh``: the attention weight that each cached token received from the
  chunk, summed over its rows and the query heads of the KV head, is added to
  what the token had.
* ``evict``: of every sequence and KV head the first tokens, the last ones and
  the heaviest of the others stay, up to a budget, in their order.

A chunk has ``starts[b + 1] - starts[b]`` rows of sequence b, the last of its
``lens[b]`` tokens.  ``own`` chooses between the plain forms (elementary torch
operations) and the package's kernels.
"""

import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    bf = {"dtype": "bf16", "d": 128}
    mha = {"H": 10, "Hkv": 10}
    grouped = {"H": 32, "Hkv": 8}
    tokens = {"T_lo": 1, "T": 1}
    # prefixes of 256..2048 tokens and some outputs, of which the last 128 count
    ragged = {"B": 64, "L_lo": 300, "L": 2300, "m_part": 0.9, "n": 128, "P": 64}
    everything = {"B": 64, "L_lo": 256, "L": 4096, "m_part": 0.0, "n": None, "P": 16}
    pages40 = {"B": 1, "L_lo": 10272, "L": 10272, "m_part": 0.0, "n": None, "P": 64}
    return [
        # the next token of a served batch: latency
        dict(**bf, **grouped, **tokens, **everything, name="append tokens", op="append"),
        # chunks of prompts of different lengths
        dict(**bf, **mha, name="append chunks", op="append", B=7, T_lo=300, T=2048, L_lo=2048, L=6000, m_part=0.0,
             n=None, P=32),
        # the next token of one page (288 prompt tokens, window of 128): latency
        dict(**bf, **mha, **tokens, name="attend page token", op="attend", B=1, L_lo=488, L=488, m_part=0.6, n=128,
             P=64),
        # the next token of a served batch
        dict(**bf, **mha, **tokens, **ragged, name="attend tokens", op="attend"),
        # the same with grouped heads, no window and small pages
        dict(**bf, **grouped, **tokens, **everything, name="attend tokens grouped", op="attend"),
        # a mixed step: single tokens and chunks of prompts, the first 16 tokens and a window of 1000 visible
        dict(**bf, **grouped, name="attend mixed", op="attend", B=24, T_lo=1, T=512, L_lo=512, L=4000, m_part=0.01,
             n=1000, P=128),
        # a chunk of a 40-page document's prompt, near its end
        dict(**bf, **mha, **pages40, name="attend 40 pages chunk", op="attend", T_lo=4096, T=4096),
        # the parity type
        dict(name="attend f32", op="attend", dtype="f32", d=64, H=4, Hkv=2, B=3, T_lo=1, T=90, L_lo=90, L=700,
             m_part=0.3, n=77, P=16),
        # weights of a batch's next tokens
        dict(**bf, **grouped, **tokens, **everything, name="weigh tokens", op="weigh"),
        # weights that the last 64 rows of a 40-page document's prompt give its tokens
        dict(**bf, **mha, **pages40, name="weigh prompt end", op="weigh", T_lo=64, T=64),
        # a 40-page document cut down after its prompt
        dict(**bf, **mha, **pages40, **tokens, name="evict 40 pages", op="evict", budget=2048, first=16, last=256,
             inplace=False),
        # a served batch, the short sequences copied whole
        dict(**bf, **grouped, **tokens, name="evict batch", op="evict", B=48, L_lo=400, L=2300, m_part=0.0, n=None,
             P=32, budget=700, first=4, last=128, inplace=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "attend", "weigh", "weigh", "evict"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    d = rng.choice([64, 128, 128])
    H, Hkv = rng.choice([(10, 10), (10, 10), (32, 8), (32, 8), (20, 5), (8, 1), (12, 4), (5, 5), (6, 2), (16, 2),
                         (28, 4), (48, 2)])
    c = {"op": op, "dtype": dtype, "d": d, "H": H, "Hkv": Hkv, "P": rng.choice([16, 16, 32, 64, 64, 128, 256])}
    if op in ("append", "evict"):
        B = _log(rng, 1, 64)
        L = _log(rng, 2, min(10272, 100_000_000 // (B * Hkv * d * 4)))
        c = dict(c, B=B, L_lo=rng.randint(1, L), L=L, m_part=0.0, n=None)
        if op == "append":
            T = _log(rng, 1, min(L, 2048, 16384 // B))
            return dict(c, L_lo=max(c["L_lo"], T), T_lo=rng.randint(0, T), T=T)
        budget = _log(rng, 1, L)
        first = rng.randint(0, budget) // rng.choice([1, 4, 50])
        last = rng.randint(0, budget - first) // rng.choice([1, 4])
        return dict(c, T_lo=1, T=1, budget=budget, first=first, last=last, inplace=rng.random() < 0.4)
    few = rng.random() < 0.5                    # single tokens or a few drafted ones
    B = _log(rng, 1, 64 if few else 24)
    T = rng.choice([1, 1, 1, 2, 5]) if few else _log(rng, 8, max(8, min(4096 // B, int((3e8 / (B * H)) ** 0.5))))
    lo = max(T, 2)
    if dtype == "f32":
        T, B = min(T, 96), min(B, 8)
        L = _log(rng, lo, max(lo, 900))
    else:
        L = _log(rng, lo, max(lo, min(10272, 100_000_000 // (B * Hkv * d * 4),
                                      400_000_000 // (B * T * H))))
    c = dict(c, B=B, T_lo=rng.choice([0, 1, T, T]), T=T, L_lo=rng.randint(max(T, L // 4), max(T, L)), L=max(T, L))
    return dict(c, m_part=rng.choice([0.0, 0.01, 0.3, 0.9]), n=rng.choice([None, None, _log(rng, 1, 2000)]))


def _lengths(case):
    """Tokens, chunk rows and prefix of each sequence: the same for every seed,
    so that the work of a case is."""
    rng = random.Random(11 * case["B"] + case["L"])
    L = [rng.randint(case["L_lo"], case["L"]) for _ in range(case["B"])]
    # half of the chunks are as short as the case has them
    T = [min(l, rng.choice([case["T_lo"], rng.randint(case["T_lo"], case["T"])])) for l in L]
    T[0] = max(T[0], 1)
    return L, T, [int(case["m_part"] * l) for l in L]


def _device():
    return "cuda" if torch.cuda.is_available() else "cpu"


def _inputs(case, seed):
    """The tensors of a case: drawn in 32 bits, rounded once."""
    dev, dt = _device(), DTYPES[case["dtype"]]
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev).to(dt)

    op, B, P, Hkv, d = case["op"], case["B"], case["P"], case["Hkv"], case["d"]
    L, T, m = _lengths(case)
    width = -(-max(L) // P)
    # pages in any order, some that no sequence has; an evicted cache may go to pages of its own
    need = [-(-l // P) for l in L]
    out = [-(-min(l, case["budget"]) // P) for l in L] if op == "evict" and not case["inplace"] else [0] * B
    pool = sum(need) + sum(out) + 3
    ids = list(range(pool))
    random.Random(seed).shuffle(ids)

    def table(counts, columns):
        rows = [[ids.pop() for _ in range(c)] for c in counts]
        return torch.tensor([r + [-1] * (columns - len(r)) for r in rows], dtype=torch.int32, device=dev)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    x = {"K": normal(pool, Hkv, P, d), "V": normal(pool, Hkv, P, d), "table": table(need, width), "lens": ints(L),
         "prefix": ints(m), "starts": None if T == [1] * B else ints([sum(T[:b]) for b in range(B + 1)])}
    rows = sum(T)
    if op == "append":
        x["k"], x["v"] = normal(rows, Hkv, d), normal(rows, Hkv, d)
    elif op in ("attend", "weigh"):
        x["q"] = normal(rows, case["H"], d)
    if op in ("weigh", "evict"):
        # what tokens have received so far: a few much, most little, some nothing
        w = torch.rand((B, Hkv, width * P), generator=g, device=dev)
        x["weights"] = (w ** 8 / (w + 0.01)) * (torch.rand(w.shape, generator=g, device=dev) > 0.1)
    if op == "evict":
        x["table_out"] = None if case["inplace"] else table(out, width)
    return x


def prepare(case, seed):
    x = _inputs(case, seed)
    s = dict(x, op=case["op"], case=case, rows=sum(_lengths(case)[1]))
    dev, H, Hkv, d = x["lens"].device, case["H"], case["Hkv"], case["d"]
    if own:
        import sliding_window_attention_02_gb300 as rswa
        dtype = rswa.RSWA_F32 if case["dtype"] == "f32" else rswa.RSWA_BF16
        s["pages"] = rswa.RswaPages(x["K"].shape[0], case["P"], H, d, dtype, kv_heads=Hkv)
        s["K"], s["V"] = s["pages"].slabs()
        s["K"].copy_(x["K"])
        s["V"].copy_(x["V"])
        s["batch"] = rswa.RswaBatch(x["table"], x["lens"], starts=x["starts"],
                                    prefix=x["prefix"] if case["n"] else None, window=case["n"])
    else:
        s["starts"] = torch.arange(case["B"] + 1, device=dev) if x["starts"] is None else x["starts"].long()
    if case["op"] == "attend":
        s["o"] = torch.empty_like(x["q"])
        s["lse"] = torch.empty(x["q"].shape[:2], device=dev)
    elif case["op"] == "weigh":
        # the softmax statistics of the chunk's attention, which comes first
        s["lse"] = _attention(dict(s, starts=torch.arange(case["B"] + 1, device=dev) if x["starts"] is None
                                   else x["starts"].long(), K=x["K"], V=x["V"]), "lse")
    elif case["op"] == "evict":
        s["weights_out"] = x["weights"] if case["inplace"] else torch.empty_like(x["weights"])
        s["kept"] = torch.empty(case["B"], Hkv, case["budget"], dtype=torch.int32, device=dev)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _append(s):
    P = s["case"]["P"]
    row = torch.arange(s["rows"], device=s["k"].device)
    b = torch.searchsorted(s["starts"], row, right=True) - 1
    token = s["lens"].long()[b] - s["starts"][b + 1] + row
    page = s["table"].long()[b, token // P]
    s["K"][page, :, token % P] = s["k"]
    s["V"][page, :, token % P] = s["v"]
    return s["K"], s["V"]


def _groups(s):
    """Runs of sequences whose padded scores fit 2 GB, with their longest chunk and length."""
    case = s["case"]
    L, T, _ = _lengths(case)
    b0 = 0
    while b0 < case["B"]:
        b1 = b0 + 1
        while b1 < case["B"] and (b1 + 1 - b0) * max(T[b0:b1 + 1]) * max(L[b0:b1 + 1]) * case["H"] < 1 << 29:
            b1 += 1
        if max(T[b0:b1]):
            yield slice(b0, b1), max(T[b0:b1]), max(L[b0:b1])
        b0 = b1


def _rows_of(s, name, bs, longest):
    """[sequences][kv_heads][longest][d] of a pool's rows in 32 bits."""
    P = s["case"]["P"]
    pages = s["table"][bs, :-(-longest // P)].long().clamp(min=0)
    x = s[name][pages].transpose(1, 2)
    return x.reshape(x.shape[0], x.shape[1], -1, x.shape[-1])[:, :, :longest].float()


def _scores(s, bs, T, L):
    """Scaled logits [sequences][kv_heads][group][T][L] of a run of sequences,
    -inf where a token is not seen, and the row of each (sequence, i), -1: none."""
    c = s["case"]
    H, Hkv, d = c["H"], c["Hkv"], c["d"]
    i = torch.arange(T, device=s["q"].device)
    lo, hi = s["starts"][:-1][bs, None], s["starts"][1:][bs, None]
    row = torch.where(lo + i < hi, lo + i, -1)
    token = (s["lens"].long()[bs, None] - (hi - lo) + i)[:, :, None]
    j = torch.arange(L, device=i.device)
    n = c["n"] or 1 << 40
    sees = (j <= token) & ((j < s["prefix"].long()[bs, None, None]) | (j > token - n))
    q = s["q"][row.clamp(min=0)].float().view(row.shape[0], T, Hkv, H // Hkv, d).permute(0, 2, 3, 1, 4)
    x = torch.matmul(q.reshape(row.shape[0], Hkv, -1, d), _rows_of(s, "K", bs, L).transpose(-1, -2)) * d ** -0.5
    return x.view(row.shape[0], Hkv, H // Hkv, T, L).masked_fill(~sees[:, None, None], float("-inf")), row


def _attention(s, what):
    c = s["case"]
    H, d = c["H"], c["d"]
    o = torch.empty(s["q"].shape, dtype=s["q"].dtype, device=s["q"].device)
    lse = torch.empty(s["q"].shape[:2], device=s["q"].device)
    for bs, T, L in _groups(s):
        x, row = _scores(s, bs, T, L)
        live = row >= 0
        top = x.amax(-1, keepdim=True).clamp(min=-1e30)
        p = torch.exp(x - top)
        total = p.sum(-1, keepdim=True)
        at = (top + torch.log(total))[..., 0]
        lse[row[live]] = at.permute(0, 3, 1, 2).reshape(*row.shape, H)[live]
        if what != "lse":
            y = torch.matmul(p.view(p.shape[0], p.shape[1], -1, L), _rows_of(s, "V", bs, L)).view(*p.shape[:4], d)
            y = (y / total).permute(0, 3, 1, 2, 4).reshape(*row.shape, H, d)
            o[row[live]] = y[live].to(o.dtype)
    return lse if what == "lse" else (o, lse)


def _weigh(s):
    c = s["case"]
    Hkv, G = c["Hkv"], c["H"] // c["Hkv"]
    for bs, T, L in _groups(s):
        x, row = _scores(s, bs, T, L)
        lse = s["lse"][row.clamp(min=0)].view(*row.shape, Hkv, G).permute(0, 2, 3, 1)[..., None]
        p = torch.exp(x - lse) * (row >= 0)[:, None, None, :, None]
        s["weights"][bs, :, :L] += p.sum((2, 3))
    return s["weights"]


def _evict(s):
    c = s["case"]
    P, budget = c["P"], c["budget"]
    w, lens = s["weights"], s["lens"].long()[:, None, None]
    j = torch.arange(w.shape[-1], device=w.device)
    kept_len = lens.clamp(max=budget)
    rank = torch.where((j < c["first"]) | (j >= lens - c["last"]), float("inf"), w)
    rank = torch.where(j < lens, rank, float("-inf"))
    order = rank.sort(stable=True, dim=-1, descending=True).indices[..., :budget]
    i = torch.arange(order.shape[-1], device=w.device)
    kept = torch.where(i < kept_len, order, 1 << 40).sort(-1).values
    live = (i < kept_len).expand_as(order)
    src = kept.clamp(max=w.shape[-1] - 1)
    b, h, dst = torch.where(live)
    at = src[live]
    table, table_out = s["table"].long(), (s["table"] if s["table_out"] is None else s["table_out"]).long()
    for pool in (s["K"], s["V"]):
        pool[table_out[b, dst // P], h, dst % P] = pool[table[b, at // P], h, at % P]
    new = torch.zeros_like(w)
    new[..., :order.shape[-1]] = torch.where(live, w.gather(-1, src), 0.0)
    s["weights_out"].copy_(new)
    s["kept"].fill_(-1)
    s["kept"][..., :order.shape[-1]] = torch.where(live, kept, -1).int()
    return s["K"], s["V"], s["weights_out"], s["kept"]


def _own(s):
    pages, batch = s["pages"], s["batch"]
    if s["op"] == "append":
        pages.append(batch, s["k"], s["v"])
        return s["K"], s["V"]
    if s["op"] == "attend":
        pages.attend(batch, s["q"], s["o"], s["lse"])
        return s["o"], s["lse"]
    if s["op"] == "weigh":
        pages.weigh(batch, s["q"], s["lse"], s["weights"])
        return s["weights"]
    c = s["case"]
    pages.evict(batch, s["weights"], c["budget"], first=c["first"], last=c["last"], table_out=s["table_out"],
                weights_out=s["weights_out"], kept=s["kept"])
    return s["K"], s["V"], s["weights_out"], s["kept"]


def run(s):
    if own:
        return _own(s)
    if s["op"] == "attend":
        s["o"], s["lse"] = _attention(s, "o")
        return s["o"], s["lse"]
    return {"append": _append, "weigh": _weigh, "evict": _evict}[s["op"]](s)


def work(case):
    H, Hkv, d, op = case["H"], case["Hkv"], case["d"], case["op"]
    elt = 2 if case["dtype"] == "bf16" else 4
    L, T, m = _lengths(case)
    if op == "append":
        return {"bytes": sum(T) * 4 * Hkv * d * elt, "flops": 0}
    if op == "evict":
        kept = [min(l, case["budget"]) for l in L]
        moved = [0 if case["inplace"] and l <= case["budget"] else k for l, k in zip(L, kept)]
        return {"bytes": sum(moved) * Hkv * 4 * d * elt + (sum(L) + 2 * sum(kept)) * Hkv * 4, "flops": 0}
    n = case["n"] or 1 << 40
    keys = pairs = 0
    for l, t, p in zip(L, T, m):
        if t == 0:
            continue
        lo = max(min(p, l), l - t - n + 1)              # the first token past the prefix that a row sees
        keys += min(p, l) + max(0, l - lo)
        # token i sees i + 1 tokens, less those between the prefix and its window
        pairs += sum(i + 1 - max(0, i - n + 1 - p) for i in range(l - t, l))
    rows = sum(T)
    if op == "attend":
        return {"bytes": keys * 2 * Hkv * d * elt + rows * H * (2 * d * elt + 4), "flops": 4 * d * H * pairs}
    return {"bytes": keys * Hkv * (d * elt + 8) + rows * H * (d * elt + 4), "flops": 2 * d * H * pairs}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    x = _inputs(case, seed)
    op, P, Hkv, d, H = case["op"], case["P"], case["Hkv"], case["d"], case["H"]
    L, T, m = _lengths(case)
    B, G = case["B"], H // Hkv
    dev = x["lens"].device
    table = x["table"].tolist()
    first = [sum(T[:b]) for b in range(B)]

    def pages_of(b, count):
        return torch.tensor(table[b][:-(-count // P)], device=dev)

    def tokens(pool, b):                                # [kv_heads][L][d]
        return pool[pages_of(b, L[b])].permute(1, 0, 2, 3).flatten(1, 2)[:, :L[b]]

    if op == "append":
        K, V = x["K"].double(), x["V"].double()
        for b in range(B):
            for pool, new in ((K, x["k"]), (V, x["v"])):
                for p in range((L[b] - T[b]) // P, -(-L[b] // P)):
                    lo, hi = max(p * P, L[b] - T[b]), min((p + 1) * P, L[b])
                    if lo < hi:
                        at = first[b] + lo - (L[b] - T[b])
                        pool[table[b][p], :, lo - p * P:hi - p * P] = new[at:at + hi - lo].double().transpose(0, 1)
        return K, V
    if op == "evict":
        K, V, budget = x["K"].clone(), x["V"].clone(), case["budget"]
        out_table = table if case["inplace"] else x["table_out"].tolist()
        weights = x["weights"].double().cpu()
        new_w = torch.zeros_like(weights)
        kept = torch.full((B, Hkv, budget), -1, dtype=torch.int32)
        for b in range(B):
            n = min(L[b], budget)
            oldK, oldV = tokens(x["K"], b), tokens(x["V"], b)
            dest = torch.tensor(out_table[b][:-(-n // P)], device=dev)
            for h in range(Hkv):
                w = weights[b, h].tolist()
                if L[b] <= budget:
                    keep = list(range(n))
                else:
                    lo, hi = case["first"], L[b] - case["last"]
                    heavy = sorted(range(lo, hi), key=lambda j: (-w[j], j))[:budget - lo - case["last"]]
                    keep = list(range(lo)) + sorted(heavy) + list(range(hi, L[b]))
                kept[b, h, :n] = torch.tensor(keep, dtype=torch.int32)
                new_w[b, h, :n] = weights[b, h, keep]
                rows = torch.tensor(keep, device=dev)
                where = torch.arange(n, device=dev)
                for pool, old in ((K, oldK), (V, oldV)):
                    pool[dest[where // P], h, where % P] = old[h, rows]
        return K.double(), V.double(), new_w.to(dev), kept.to(dev)
    n = case["n"] or max(L) + 1
    o = torch.zeros(sum(T), H, d, dtype=torch.float64, device=dev)
    lse = torch.zeros(sum(T), H, dtype=torch.float64, device=dev)
    weights = x["weights"].double() if op == "weigh" else None
    for b in range(B):
        if T[b] == 0:
            continue
        rows = slice(first[b], first[b] + T[b])
        K, V = tokens(x["K"], b).double(), tokens(x["V"], b).double()
        here = torch.arange(L[b] - T[b], L[b], device=dev).unsqueeze(1)
        there = torch.arange(L[b], device=dev)
        hidden = (there > here) | ((there >= m[b]) & (there <= here - n))
        for h in range(H):
            logits = (x["q"][rows, h].double() @ K[h // G].T / d ** 0.5).masked_fill(hidden, float("-inf"))
            if op == "attend":
                top = torch.logsumexp(logits, 1)
                o[rows, h], lse[rows, h] = torch.softmax(logits, 1) @ V[h // G], top
            else:
                weights[b, h // G, :L[b]] += torch.softmax(logits, 1).sum(0)
    return (o, lse) if op == "attend" else weights
