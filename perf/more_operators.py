"""The paged cache's operators for steps of several tokens and for long caches, timed: slots, positions and
ancestors of new tokens, attention of drafted token trees, keeping an accepted path, bounds of pages, and
attention over the pages that a score from the bounds picks.

``run`` computes each operator in its plain form (elementary torch operations in 32 bits), or, with ``own``
set, through the calls a user makes of the library.  Sizes are given per case; lengths and trees follow
from the case, values and page numbers from the seed.
"""
import math

import torch

own = False

DEV = "cuda:0"
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------------------
def listed():
    return [
        # a step of a server: 64 of 96 sequences draft small trees, padded to the step's fixed size
        dict(name="slots-trees", op="slots", n=64, seqs=96, page=32, lo=1, hi=16, have=4096, tree=True, pad=100),
        # the prompts of a batch on their way into pages
        dict(name="slots-prompts", op="slots", n=48, seqs=48, page=16, lo=17, hi=4099, have=0, tree=False, pad=0),
        # eight drafted tokens of one short request on a small model: all launch latency
        dict(name="tree-one-small", op="tree", B=1, n_lo=8, n_hi=8, Hq=4, Hkv=4, d=64, page=16, lo=256, hi=256, dtype="f16"),
        # a server's mixed batch, trees of 1 to 16 tokens on caches of every age
        dict(name="tree-batch", op="tree", B=32, n_lo=1, n_hi=16, Hq=32, Hkv=8, d=128, page=32, lo=64, hi=8192, dtype="bf16"),
        # wide trees on two long documents, eight queries to a key head: bound by the products
        dict(name="tree-wide-long", op="tree", B=2, n_lo=63, n_hi=64, Hq=32, Hkv=4, d=128, page=64, lo=65001, hi=65536,
             dtype="f16"),
        # three tokens of one request accepted
        dict(name="keep-one-small", op="keep", B=1, n=8, kept=3, layers=4, Hkv=4, d=64, page=16, hi=250, dtype="f16"),
        # a batch's accepted paths in every layer
        dict(name="keep-batch", op="keep", B=64, n=32, kept=8, layers=32, Hkv=8, d=128, page=32, hi=300, dtype="bf16"),
        # the page that each sequence of a batch has just written to
        dict(name="bounds-step", op="bounds", n=64, spare=192, Hkv=8, d=128, page=32, part=True, dtype="bf16"),
        # every page of the prompts of a batch
        dict(name="bounds-prompts", op="bounds", n=4000, spare=96, Hkv=8, d=128, page=16, part=False, dtype="f16"),
        # a quarter of one request's pages
        dict(name="picked-one-small", op="picked", B=1, Hq=8, Hkv=4, d=64, page=16, lo=1024, hi=1024, picks=16, dtype="f16"),
        # a server's batch, every sequence held to 2048 tokens
        dict(name="picked-batch", op="picked", B=64, Hq=32, Hkv=8, d=128, page=32, lo=100, hi=16384, picks=64, dtype="bf16"),
        # one long document: one page in 32
        dict(name="picked-long", op="picked", B=1, Hq=40, Hkv=8, d=128, page=16, lo=131071, hi=131071, picks=256, dtype="f16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["slots", "tree", "tree", "keep", "bounds", "picked", "picked"])
    dtype = rng.choice(["f16", "bf16"])
    d = rng.choice([64, 128, 128])
    page = rng.choice([8, 16, 24, 32, 64, 128])
    if op == "slots":
        tree = rng.random() < 0.5
        while True:
            n, have, hi = _log(rng, 1, 300), rng.choice([0, _log(rng, 1, 30000)]), _log(rng, 1, 64 if tree else 8000)
            lo = rng.choice([0, 1, hi])
            if n * hi <= 400000 and n * (have + hi) <= 10 ** 7:
                return dict(op=op, n=n, seqs=n + rng.choice([0, _log(rng, 1, 100)]), page=page, lo=min(lo, hi), hi=hi,
                            have=have, tree=tree, pad=rng.choice([0, _log(rng, 1, 200)]))
    if op == "tree":
        while True:
            B, Hkv, g = _log(rng, 1, 96), _log(rng, 1, 32), rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
            n, hi = _log(rng, 1, 64), _log(rng, 1, 65536)
            lo = rng.choice([1, max(1, hi // 2), hi])
            if B * hi * Hkv * d * 4 <= 10 ** 9 and Hkv * g <= 128 and B * Hkv * g * n * hi <= 1.3 * 10 ** 8:
                return dict(op=op, B=B, n_lo=rng.choice([0, 1, n]), n_hi=n, Hq=Hkv * g, Hkv=Hkv, d=d, page=page, lo=lo, hi=hi,
                            dtype=dtype)
    if op == "keep":
        while True:
            B, n, layers, Hkv = _log(rng, 1, 128), _log(rng, 1, 64), _log(rng, 1, 48), _log(rng, 1, 32)
            hi = _log(rng, 1, 2000)
            if layers * (B * (-(-(hi + n) // page) + 1)) * Hkv * page * d * 4 <= 3 * 10 ** 9 and \
                    layers * B * n * Hkv * d <= 10 ** 8:
                return dict(op=op, B=B, n=n, kept=rng.randint(0, n), layers=layers, Hkv=Hkv, d=d, page=page, hi=hi,
                            dtype=dtype)
    if op == "bounds":
        while True:
            n, Hkv = _log(rng, 1, 8000), _log(rng, 1, 40)
            if n * Hkv * page * d <= 2 * 10 ** 8:
                return dict(op=op, n=n, spare=_log(rng, 1, 300), Hkv=Hkv, d=d, page=page, part=rng.random() < 0.5,
                            dtype=dtype)
    while True:
        B, Hkv, g = _log(rng, 1, 96), _log(rng, 1, 32), rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
        hi, picks = _log(rng, 1, 131072), _log(rng, 4, 512)
        lo = rng.choice([0, hi // 2, hi])
        if B * hi * Hkv * d * 4 <= 3 * 10 ** 9 and Hkv * g <= 128 and B * Hkv * g * hi <= 6 * 10 ** 7 and \
                B * Hkv * picks * page * d <= 1.4 * 10 ** 8:
            return dict(op="picked", B=B, Hq=Hkv * g, Hkv=Hkv, d=d, page=page, lo=lo, hi=hi, picks=picks, dtype=dtype)


def _spread(B, lo, hi, by=0.6180339887):
    """B numbers spread over lo .. hi, hi among them."""
    return [hi if b == B - 1 else lo + int((hi + 1 - lo) * ((b * by) % 1.0)) for b in range(B)]


def _parents(n, salt):
    """A tree of n drafted tokens: each one's parent among those before it, -1 for the first level."""
    return [-1 if i == 0 else max(-1, i - 1 - (i * 7 + salt * 5) % 4) for i in range(n)]


def _ancestors(parents):
    """Bits of each token's ancestors and itself, as signed 64-bit numbers."""
    out = []
    for i, p in enumerate(parents):
        out.append((1 << i) | (out[p] if p >= 0 else 0))
    return [x - 2 ** 64 if x >= 2 ** 63 else x for x in out]


def _counts(c):
    """New tokens of each request (slots), or drafted ones (tree, with the lengths they are part of)."""
    if c["op"] == "slots":
        return _spread(c["n"], c["lo"], c["hi"])
    L = _spread(c["B"], c["lo"], c["hi"])
    return [min(n, x) for n, x in zip(_spread(c["B"], c["n_lo"], c["n_hi"], 0.7548776662), L)], L


def _rows(c):
    """Live rows of each page: whole pages, or 1 .. page."""
    return [c["page"] if not c["part"] else 1 + (7 * i + 4) % c["page"] for i in range(c["n"])]


def _path(c, b):
    """The drafted tokens of request b that are kept, ascending."""
    n, kept = c["n"], c["kept"]
    return sorted((b * 5 + i * n // max(kept, 1)) % n for i in range(kept))


# ---------------------------------------------------------------------------------------
# what a program has in hand before the call
# ---------------------------------------------------------------------------------------
def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _table(L, page, g, spare=3):
    """A page table of sequences of L tokens (pages in random order), and the number of pages."""
    mp = max(1, max(-(-x // page) for x in L))
    need = sum(-(-x // page) for x in L)
    perm = torch.randperm(need + spare, generator=g, device=DEV, dtype=torch.int32)
    used = torch.arange(mp, device=DEV)[None, :] < ((_i32(L) + page - 1) // page)[:, None]
    table = torch.full((len(L), mp), -1, dtype=torch.int32, device=DEV)
    table[used] = perm[:need]
    return table, need + spare


def _first(counts):
    out = [0]
    for x in counts:
        out.append(out[-1] + x)
    return out


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rand = lambda *shape, dt: torch.randn(*shape, generator=g, device=DEV, dtype=dt)  # noqa: E731
    s = dict(c=c)
    if c["op"] == "slots":
        counts = _counts(c)
        total = sum(counts)
        seq = torch.randperm(c["seqs"], generator=g, device=DEV)[:c["n"]]
        L = torch.randint(0, c["have"] + 1, (c["seqs"],), generator=g, device=DEV)
        L[seq] += torch.tensor(counts, device=DEV)
        s["table"], s["pages"] = _table(L.tolist(), c["page"], g)
        s["L"], s["seq"], s["counts"] = L.to(torch.int32), seq.to(torch.int32), _i32(counts)
        s["T"] = total + c["pad"]
        s["parents"] = s["masks"] = None
        if c["tree"]:
            flat = [p for i, n in enumerate(counts) for p in _parents(n, i + seed)]
            s["parents"] = _i32(flat + [-1] * c["pad"])
            s["masks"] = torch.empty(s["T"], dtype=torch.int64, device=DEV)
        s["first"] = torch.empty(c["n"] + 1, dtype=torch.int32, device=DEV)
        s["slots"] = torch.empty(s["T"], dtype=torch.int32, device=DEV)
        s["positions"] = torch.empty(s["T"], dtype=torch.int32, device=DEV)
        return s
    dt = DTYPES[c["dtype"]]
    Hkv, d, page = c["Hkv"], c["d"], c["page"]
    if c["op"] == "tree":
        counts, L = _counts(c)
        s["table"], n = _table(L, page, g)
        T = sum(counts)
        s["T"], s["n_hi"] = T, max(1, max(counts))
        s["L"], s["first"] = _i32(L), _i32(_first(counts))
        masks = [m for b, x in enumerate(counts) for m in _ancestors(_parents(x, b + seed))]
        s["masks"] = torch.tensor(masks, dtype=torch.int64, device=DEV)
        s["q"] = rand(T, c["Hq"], d, dt=dt) * 1.25
        s["K"] = rand(n, Hkv, page, d, dt=dt) * 1.25
        s["V"] = rand(n, Hkv, page, d, dt=dt)
        s["out"] = torch.empty(T, c["Hq"], d, dtype=dt, device=DEV)
        s["lse"] = torch.empty(T, c["Hq"], dtype=torch.float32, device=DEV)
        s["ws"] = None
    elif c["op"] == "keep":
        L = [x + c["n"] for x in _spread(c["B"], 0, c["hi"])]
        s["table"], n = _table(L, page, g)
        s["L"], s["first"] = _i32(L), _i32([c["n"] * b for b in range(c["B"] + 1)])
        paths = [_path(c, b) for b in range(c["B"])]
        s["path"] = _i32([p for x in paths for p in x + [0] * (c["n"] - len(x))])
        s["kept"] = _i32([len(x) for x in paths])
        s["K"] = rand(c["layers"], n, Hkv, page, d, dt=dt)
        s["V"] = rand(c["layers"], n, Hkv, page, d, dt=dt)
    elif c["op"] == "bounds":
        n = c["n"] + c["spare"]
        s["K"] = rand(n, Hkv, page, d, dt=dt) * 0.75 + rand(1, Hkv, 1, d, dt=dt) + rand(n, Hkv, 1, d, dt=dt) * 0.5
        pages = torch.randperm(n, generator=g, device=DEV, dtype=torch.int32)[:c["n"]]
        s["list"] = torch.stack([pages, _i32(_rows(c))], 1).contiguous()
        s["codes"] = torch.zeros(n, Hkv, 2, d, dtype=torch.int8, device=DEV)
        s["scales"] = torch.zeros(n, Hkv, dtype=torch.float32, device=DEV)
    else:
        L = _spread(c["B"], c["lo"], c["hi"])
        s["table"], n = _table(L, page, g)
        s["L"] = _i32(L)
        s["q"] = rand(c["B"], c["Hq"], d, dt=dt) * 1.25
        # keys lie around an offset of their head and of their page, as those of neighbouring tokens do
        s["K"] = rand(n, Hkv, page, d, dt=dt) * 0.75 + rand(1, Hkv, 1, d, dt=dt) + rand(n, Hkv, 1, d, dt=dt) * 0.5
        s["V"] = rand(n, Hkv, page, d, dt=dt)
        rows = torch.zeros(n, dtype=torch.int64, device=DEV)
        at = torch.arange(s["table"].shape[1], device=DEV)[None, :] * page
        live = (s["L"][:, None] - at).clamp(0, page)
        rows[s["table"][live > 0].long()] = live[live > 0]
        s["codes"], s["scales"] = _bounds(s["K"], rows)
        s["chosen"] = torch.empty(c["B"], Hkv, c["picks"], dtype=torch.int32, device=DEV)
        s["tokens"] = torch.empty(c["B"], Hkv, dtype=torch.int32, device=DEV)
        s["out"] = torch.empty(c["B"], c["Hq"], d, dtype=torch.float32, device=DEV)
        s["lse"] = torch.empty(c["B"], c["Hq"], dtype=torch.float32, device=DEV)
        s["ws"] = None
    return s


# ---------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------
def run(s):
    return (_own if own else _plain)[s["c"]["op"]](s)


def _slots_plain(s):
    c = s["c"]
    n, page, T = c["n"], c["page"], s["T"]
    seq, counts = s["seq"].long(), s["counts"].long()
    first = torch.cat([counts.new_zeros(1), torch.cumsum(counts, 0)])
    t = torch.arange(T, device=DEV)
    r = torch.searchsorted(first[1:].contiguous(), t, right=True)
    live = r < n
    r = r.clamp(max=n - 1)
    i = t - first[r]
    base = (s["L"].long()[seq] - counts)[r]
    at = torch.where(live, base + i, 0)
    slot = torch.where(live, s["table"].long()[seq[r], at // page] * page + at % page, -1)
    if not c["tree"]:
        return first.int(), slot.int(), torch.where(live, at, 0).int()
    mask = torch.where(live, torch.ones_like(i) << i.clamp(0, 63), 0)
    parent = torch.where(live & (s["parents"] >= 0), first[r] + s["parents"], -1)
    for _ in range(6):  # 1, 2, 4, .. ancestors
        up = parent.clamp(min=0)
        mask = torch.where(parent >= 0, mask | mask[up], mask)
        parent = torch.where(parent >= 0, parent[up], -1)
    bits = (mask[:, None] >> torch.arange(64, device=DEV)) & 1
    position = torch.where(live, base + bits.sum(1) - 1, 0)
    return first.int(), slot.int(), position.int(), mask


def _tree_plain(s):
    c = s["c"]
    B, Hq, Hkv, d, page, n = c["B"], c["Hq"], c["Hkv"], c["d"], c["page"], s["n_hi"]
    first = s["first"].long()
    counts = first[1:] - first[:-1]
    node = torch.arange(n, device=DEV)
    live = node[None, :] < counts[:, None]
    at = torch.where(live, first[:-1, None] + node, 0)
    pages = s["table"].clamp(min=0).long()
    keys = pages.shape[1] * page
    q = s["q"][at].float().view(B, n, Hkv, Hq // Hkv, d).transpose(1, 2).reshape(B, Hkv, -1, d)
    K = s["K"][pages].transpose(1, 2).reshape(B, Hkv, keys, d).float()
    z = torch.matmul(q, K.transpose(2, 3)) / math.sqrt(d)
    del K
    key = torch.arange(keys, device=DEV)[None, :]
    L = s["L"].long()[:, None]
    bit = key - (L - counts[:, None])
    seen = ((s["masks"][at][:, :, None] >> bit.clamp(0, 63)[:, None, :]) & 1).bool()
    seen = torch.where((bit < 0)[:, None, :], True, seen) & (key < L)[:, None, :]
    seen = seen[:, None, :, None, :]
    z = z.view(B, Hkv, n, Hq // Hkv, keys).masked_fill_(~seen, -math.inf)
    m = z.amax(-1, keepdim=True)
    p = torch.exp(z - m.masked_fill(m == -math.inf, 0.0))
    del z
    total = p.sum(-1, keepdim=True)
    V = s["V"][pages].transpose(1, 2).reshape(B, Hkv, keys, d).float().masked_fill((key >= L)[:, None, :, None], 0.0)
    o = torch.matmul(p.view(B, Hkv, -1, keys), V).view(B, Hkv, n, Hq // Hkv, d) / total.masked_fill(total == 0, 1.0)
    lse = (m + torch.log(total))[..., 0]
    o = o.permute(0, 2, 1, 3, 4).reshape(B, n, Hq, d)[live]
    return o.to(s["q"].dtype), lse.permute(0, 2, 1, 3).reshape(B, n, Hq)[live]


def _keep_plain(s):
    c = s["c"]
    n, page = c["n"], c["page"]
    path = s["path"].view(c["B"], n).long()
    i = torch.arange(n, device=DEV)
    base = s["L"].long()[:, None] - n
    on = i[None, :] < s["kept"][:, None]
    row = torch.arange(c["B"], device=DEV)[:, None].expand(-1, n)[on]
    src, dst = (base + path)[on], (base + i)[on]
    pages = s["table"].long()
    a, b = pages[row, src // page], pages[row, dst // page]
    for x in (s["K"], s["V"]):
        x[:, b, :, dst % page] = x[:, a, :, src % page]
    return s["K"], s["V"]


def _power(most):
    """The least power of two (from 2^-126 on) that ``most`` is at most 127 times of."""
    m, e = torch.frexp(most)
    e = torch.where(m > 127.0 / 128.0, e - 6, e - 7).clamp(min=-126)
    e = torch.where(most == 0, -126, e)
    return torch.ldexp(torch.ones_like(most), e)


def _bounds(K, rows):
    """Bounds of the first ``rows`` keys of each page, as whole numbers and the unit they are counted in."""
    K = K.float()
    live = (torch.arange(K.shape[2], device=DEV)[None, :] < rows[:, None])[:, None, :, None]
    none = (rows == 0)[:, None, None]
    lo = K.masked_fill(~live, math.inf).amin(2).masked_fill(none, 0.0)
    hi = K.masked_fill(~live, -math.inf).amax(2).masked_fill(none, 0.0)
    unit = _power(torch.maximum(lo.abs(), hi.abs()).amax(-1))
    codes = torch.stack([torch.floor(lo / unit[..., None]), torch.ceil(hi / unit[..., None])], 2)
    return codes.to(torch.int8), unit


def _bounds_plain(s):
    at = s["list"][:, 0].long()
    s["codes"][at], s["scales"][at] = _bounds(s["K"][at], s["list"][:, 1])
    return s["codes"] * s["scales"][:, :, None, None]


def _picked_plain(s):
    c = s["c"]
    B, Hq, Hkv, d, page, picks = c["B"], c["Hq"], c["Hkv"], c["d"], c["page"], c["picks"]
    pages = s["table"].clamp(min=0).long()
    mp = pages.shape[1]
    L = s["L"].long()[:, None]
    used = (L + page - 1) // page
    p = torch.arange(mp, device=DEV)[None, :]
    q = s["q"].float()
    unit = _power(q.abs().amax(-1))
    code = torch.round(q / unit[..., None]).view(B, Hkv, Hq // Hkv, d)
    both = torch.cat([code.clamp(max=0), code.clamp(min=0)], -1)
    bounds = s["codes"][pages].transpose(1, 2).reshape(B, Hkv, mp, 2 * d).float()
    score = torch.matmul(both, bounds.transpose(2, 3)) * unit.view(B, Hkv, -1, 1)
    score = (score.amax(2) * s["scales"][pages].transpose(1, 2)).clamp(max=torch.finfo(torch.float32).max)
    score = torch.where(((p < 1) | (p >= used - 2))[:, None, :], math.inf, score)
    score = torch.where((p < used)[:, None, :], score, -math.inf)
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :picks]
    if mp < picks:
        order = torch.nn.functional.pad(order, (0, picks - mp), value=mp)
    count = used.clamp(max=picks)[:, None, :]
    k = torch.arange(picks, device=DEV)
    order = torch.sort(torch.where(k < count, order, mp)).values
    inside = order < mp
    chosen = torch.where(inside, torch.gather(pages[:, None, :].expand(-1, Hkv, -1), 2, order.clamp(max=mp - 1)), -1)
    tokens = torch.where(used > 0, (used.clamp(max=picks) - 1) * page + L - (used - 1) * page, 0).expand(-1, Hkv)
    head = torch.arange(Hkv, device=DEV)[None, :, None]
    at = chosen.clamp(min=0)
    live = (torch.arange(picks * page, device=DEV) < tokens[..., None])[:, :, None, :]
    K = s["K"][at, head].reshape(B, Hkv, picks * page, d).float()
    z = torch.matmul(s["q"].float().view(B, Hkv, Hq // Hkv, d), K.transpose(2, 3)) / math.sqrt(d)
    z = z.masked_fill(~live, -math.inf)
    m = z.amax(-1, keepdim=True)
    w = torch.exp(z - m.masked_fill(m == -math.inf, 0.0))
    total = w.sum(-1, keepdim=True)
    V = s["V"][at, head].reshape(B, Hkv, picks * page, d).float().masked_fill(~live.transpose(2, 3), 0.0)
    o = torch.matmul(w, V) / total.masked_fill(total == 0, 1.0)
    return chosen.int(), tokens.int(), o.reshape(B, Hq, d), (m + torch.log(total)).reshape(B, Hq)


def _slots_own(s):
    from speculative_kv_cache_gb300 import ig

    c = s["c"]
    ig.ig_page_slots(None, c["n"], c["seqs"], c["page"], s["pages"], s["table"].shape[1], s["T"], s["table"], s["L"],
                     s["seq"], s["counts"], s["parents"], s["first"], s["slots"], s["positions"], s["masks"])
    return (s["first"], s["slots"], s["positions"]) + ((s["masks"],) if c["tree"] else ())


def _workspace(s, need):
    """The workspace, which a program keeps from its first call on."""
    if s["ws"] is None:
        s["ws"] = torch.empty(need, dtype=torch.uint8, device=DEV)
    return s["ws"]


def _tree_own(s):
    from speculative_kv_cache_gb300 import ig

    c = s["c"]
    B, Hq, Hkv, d = c["B"], c["Hq"], c["Hkv"], c["d"]
    ws = s["ws"] if s["ws"] is not None else _workspace(s, ig.ig_paged_tree_attend_workspace_bytes(B, s["n_hi"], Hq, Hkv, d))
    ig.ig_paged_tree_attend(None, ig.IG_F16 if c["dtype"] == "f16" else ig.IG_BF16, B, s["T"], s["n_hi"], Hq, Hkv, d, c["page"],
                            s["K"].shape[0], B, s["table"].shape[1], 1.0 / math.sqrt(d), s["q"], s["K"], s["V"], s["table"],
                            s["L"], None, s["first"], s["masks"], s["out"], s["lse"], ws, ws.numel())
    return s["out"], s["lse"]


def _keep_own(s):
    from speculative_kv_cache_gb300 import ig

    c = s["c"]
    ig.ig_tree_keep(None, c["layers"], s["K"].shape[1], c["Hkv"], c["page"], c["d"], list(s["K"]), list(s["V"]), c["B"], c["B"],
                    s["table"].shape[1], s["path"].numel(), s["table"], s["L"], None, s["first"], s["path"], s["kept"])
    return s["K"], s["V"]


def _bounds_own(s):
    from speculative_kv_cache_gb300 import ig

    c = s["c"]
    ig.ig_page_bounds(None, ig.IG_F16 if c["dtype"] == "f16" else ig.IG_BF16, s["K"].shape[0], c["Hkv"], c["page"], c["d"],
                      s["K"], c["n"], s["list"], s["codes"], s["scales"])
    return s["codes"] * s["scales"][:, :, None, None]


def _picked_own(s):
    from speculative_kv_cache_gb300 import ig

    c = s["c"]
    B, Hq, Hkv, d, page, picks = c["B"], c["Hq"], c["Hkv"], c["d"], c["page"], c["picks"]
    n, mp, dt = s["K"].shape[0], s["table"].shape[1], ig.IG_F16 if c["dtype"] == "f16" else ig.IG_BF16
    ws = s["ws"] if s["ws"] is not None else _workspace(s, ig.ig_paged_attend_workspace_bytes(B, Hq, Hkv, d))
    ig.ig_page_select(None, dt, B, Hq, Hkv, d, page, n, mp, picks, 1, 2, s["q"], s["codes"], s["scales"], s["table"], s["L"],
                      s["chosen"], s["tokens"])
    ig.ig_paged_attend_picked(None, dt, B, Hq, Hkv, d, page, n, picks, 1.0 / math.sqrt(d), s["q"], s["K"], s["V"], s["chosen"],
                              s["tokens"], s["out"], s["lse"], ws, ws.numel())
    return s["chosen"], s["tokens"], s["out"], s["lse"]


_plain = {"slots": _slots_plain, "tree": _tree_plain, "keep": _keep_plain, "bounds": _bounds_plain, "picked": _picked_plain}
_own = {"slots": _slots_own, "tree": _tree_own, "keep": _keep_own, "bounds": _bounds_own, "picked": _picked_own}


def work(case):
    c = case
    if c["op"] == "slots":
        counts = _counts(c)
        total = sum(counts)
        pages = sum(-(-x // c["page"]) for x in counts)
        return dict(bytes=12 * c["n"] + 4 * pages + (8 + (12 if c["tree"] else 0)) * (total + c["pad"]) + 4 * (c["n"] + 1), flops=0)
    if c["op"] == "tree":
        counts, L = _counts(c)
        keys = sum(x for x, n in zip(L, counts) if n)
        T = sum(counts)
        pairs = sum(x * n for x, n in zip(L, counts))
        return dict(bytes=keys * c["Hkv"] * c["d"] * 4 + T * c["Hq"] * (4 * c["d"] + 4) + 8 * T + 8 * c["B"] +
                    4 * sum(-(-x // c["page"]) for x in L), flops=4 * c["d"] * c["Hq"] * pairs)
    if c["op"] == "keep":
        moved = sum(p != i for b in range(c["B"]) for i, p in enumerate(_path(c, b)))
        return dict(bytes=2 * c["layers"] * 2 * c["Hkv"] * c["d"] * 2 * moved + 4 * c["B"] * (c["kept"] + 3), flops=0)
    if c["op"] == "bounds":
        rows, n = sum(_rows(c)), c["n"]
        return dict(bytes=c["Hkv"] * (rows * c["d"] * 2 + n * (2 * c["d"] + 4)) + 8 * n, flops=0)
    L = _spread(c["B"], c["lo"], c["hi"])
    pages = [-(-x // c["page"]) for x in L]
    read = sum(x if p <= c["picks"] else (c["picks"] - 1) * c["page"] + x - (p - 1) * c["page"] for x, p in zip(L, pages))
    scored = sum(p for p in pages if p > c["picks"])
    picked = sum(min(p, c["picks"]) for p in pages)
    q = c["B"] * c["Hq"] * c["d"]
    return dict(bytes=read * c["Hkv"] * c["d"] * 4 + scored * c["Hkv"] * (2 * c["d"] + 4) + 4 * sum(pages) +
                4 * c["Hkv"] * picked + q * (2 + 4) + c["B"] * c["Hq"] * 4,
                flops=4 * c["d"] * c["Hq"] * read + 4 * c["d"] * c["Hq"] * scored)


# ---------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------
def exact(case, seed):
    return _exact[case["op"]](case, prepare(case, seed))


def _slots_exact(c, s):
    table, L, seq, counts = s["table"].tolist(), s["L"].tolist(), s["seq"].tolist(), s["counts"].tolist()
    first, slots, positions, masks = [0], [], [], []
    for at, n in zip(seq, counts):
        base = L[at] - n
        slots += [table[at][x // c["page"]] * c["page"] + x % c["page"] for x in range(base, base + n)]
        if c["tree"]:
            bits, depth = [], []
            for i, p in enumerate(s["parents"][first[-1]:first[-1] + n].tolist()):
                bits.append(2 ** i + (bits[p] if p >= 0 else 0))
                depth.append(1 + depth[p] if p >= 0 else 0)
            masks += [x - 2 ** 64 if x >= 2 ** 63 else x for x in bits]
            positions += [base + x for x in depth]
        else:
            positions += range(base, base + n)
        first.append(first[-1] + n)
    slots += [-1] * c["pad"]
    positions += [0] * c["pad"]
    out = (_i32(first), _i32(slots), _i32(positions))
    return out + (torch.tensor(masks + [0] * c["pad"], dtype=torch.int64, device=DEV),) if c["tree"] else out


def _tree_exact(c, s):
    group, d, page = c["Hq"] // c["Hkv"], c["d"], c["page"]
    out = torch.zeros(s["T"], c["Hq"], d, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["T"], c["Hq"], dtype=torch.float64, device=DEV)
    table, first, masks = s["table"].tolist(), s["first"].tolist(), s["masks"].tolist()
    for b, n in enumerate(s["L"].tolist()):
        f, e = first[b], first[b + 1]
        if e == f:
            continue
        pages = torch.tensor(table[b][:-(-n // page)], device=DEV)
        hidden = torch.tensor([[not (masks[t] >> j) & 1 for j in range(e - f)] for t in range(f, e)], device=DEV)
        for h in range(c["Hkv"]):
            k = s["K"][pages, h].reshape(-1, d)[:n].double()
            v = s["V"][pages, h].reshape(-1, d)[:n].double()
            x = torch.einsum("tgd,nd->gtn", s["q"][f:e, h * group:(h + 1) * group].double(), k) * d ** -0.5
            x[:, :, n - (e - f):] = x[:, :, n - (e - f):].masked_fill(hidden, -math.inf)
            lse[f:e, h * group:(h + 1) * group] = torch.logsumexp(x, -1).T
            out[f:e, h * group:(h + 1) * group] = (torch.softmax(x, -1) @ v).transpose(0, 1)
    return out, lse


def _keep_exact(c, s):
    table = s["table"].tolist()
    for b, n in enumerate(s["L"].tolist()):
        base = n - c["n"]
        at = lambda i: (table[b][(base + i) // c["page"]], (base + i) % c["page"])  # noqa: E731,B023
        for i, p in enumerate(_path(c, b)):
            (x, r), (y, t) = at(p), at(i)
            for pages in (s["K"], s["V"]):
                pages[:, y, :, t] = pages[:, x, :, r]
    return s["K"], s["V"]


def _unit64(most):
    """The unit of bounds or queries whose largest magnitude is ``most``: exact, as logarithms of two are taken near no border."""
    e = torch.full_like(most, -126.0)
    for k in range(-126, 122):
        e = torch.where(most > 127.0 * 2.0 ** k, float(k + 1), e)
    return torch.exp2(e)


def _bounds_exact(c, s):
    out = torch.zeros(s["K"].shape[0], c["Hkv"], 2, c["d"], dtype=torch.float64, device=DEV)
    for page, rows in s["list"].tolist():
        k = s["K"][page, :, :rows].double()
        out[page, :, 0], out[page, :, 1] = k.min(1).values, k.max(1).values
    unit = _unit64(out.abs().amax((2, 3)))[:, :, None]
    out[:, :, 0] = torch.floor(out[:, :, 0] / unit) * unit
    out[:, :, 1] = torch.ceil(out[:, :, 1] / unit) * unit
    return out


def _picked_exact(c, s):
    B, Hkv, group, d, page, picks = c["B"], c["Hkv"], c["Hq"] // c["Hkv"], c["d"], c["page"], c["picks"]
    table = s["table"].tolist()
    chosen = torch.full((B, Hkv, picks), -1, dtype=torch.int32)
    tokens = torch.zeros(B, Hkv, dtype=torch.int32)
    out = torch.zeros(B, c["Hq"], d, dtype=torch.float64, device=DEV)
    lse = torch.full((B, c["Hq"]), -math.inf, dtype=torch.float64, device=DEV)
    for b, n in enumerate(s["L"].tolist()):
        if n == 0:
            continue
        pages = table[b][:-(-n // page)]
        at = torch.tensor(pages, device=DEV)
        for h in range(Hkv):
            q = s["q"][b, h * group:(h + 1) * group].double()
            unit = _unit64(q.abs().amax(1))[:, None]
            code = torch.round(q / unit)[:, None, :]
            lo, hi = (s["codes"][at, h, i].double() for i in (0, 1))
            score = (torch.maximum(code * lo, code * hi).sum(-1) * unit).amax(0) * s["scales"][at, h].double()
            score[:1] = score[-2:] = math.inf
            score = score.tolist()
            best = sorted(sorted(range(len(pages)), key=lambda i: (-score[i], i))[:picks])  # noqa: B023
            chosen[b, h, :len(best)] = torch.tensor([pages[i] for i in best], dtype=torch.int32)
            tokens[b, h] = (len(best) - 1) * page + n - (len(pages) - 1) * page
            some = torch.tensor([pages[i] for i in best], device=DEV)
            k = s["K"][some, h].reshape(-1, d)[:int(tokens[b, h])].double()
            v = s["V"][some, h].reshape(-1, d)[:int(tokens[b, h])].double()
            x = (q @ k.T) * d ** -0.5
            lse[b, h * group:(h + 1) * group] = torch.logsumexp(x, 1)
            out[b, h * group:(h + 1) * group] = torch.softmax(x, 1) @ v
    return chosen.to(DEV), tokens.to(DEV), out, lse


_exact = {"slots": _slots_exact, "tree": _tree_exact, "keep": _keep_exact, "bounds": _bounds_exact, "picked": _picked_exact}
