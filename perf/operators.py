"""The paged-cache operators, timed: attention of one new token over pages, the norm and rotation
of queries and keys on their way into the pages, and page copies.

``run`` computes each operator in its plain form (elementary torch operations in 32 bits, angles in
64), or, with ``own`` set, through the calls a user makes of the library.  Sizes are given per case;
lengths of sequences follow from the case, values and page numbers from the seed.
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
        # one short request on a small model: all launch latency
        dict(name="attend-one-small", op="attend", B=1, Hq=4, Hkv=4, d=64, page=16, lo=256, hi=256, dtype="f16"),
        # a full batch just past its prompt, every query head with its own keys
        dict(name="attend-batch", op="attend", B=8, Hq=32, Hkv=32, d=128, page=16, lo=1920, hi=2048, dtype="f16"),
        # a server's mixed batch: requests of every age, one of them empty, shared key heads
        dict(name="attend-ragged", op="attend", B=64, Hq=32, Hkv=8, d=128, page=32, lo=0, hi=8192, dtype="bf16"),
        # one long document: the whole GPU on eight key heads
        dict(name="attend-long", op="attend", B=1, Hq=40, Hkv=8, d=128, page=64, lo=131071, hi=131071, dtype="f16"),
        # one key head for all queries, pages that are no power of two
        dict(name="attend-one-key-head", op="attend", B=16, Hq=56, Hkv=1, d=128, page=24, lo=4001, hi=4099,
             dtype="bf16"),
        # one token of a small model on its way into its page
        dict(name="rope-one-small", op="rope", T=1, Hq=4, Hkv=4, d=64, rot=64, layout="half", norm=False, scaled="none",
             top=256, page=16, dtype="f16"),
        # a decode step of a batch, normed, into pages
        dict(name="rope-batch", op="rope", T=64, Hq=32, Hkv=8, d=128, rot=128, layout="half", norm=True, scaled="none",
             top=8192, page=32, dtype="bf16"),
        # the prompts of a batch (4 x 3968 tokens) into pages
        dict(name="rope-prompts", op="rope", T=15872, Hq=32, Hkv=32, d=128, rot=128, layout="half", norm=False,
             scaled="none", top=3968, page=16, dtype="f16"),
        # a chunk far into a long document: half of each head rotated, neighbours paired, scaled; dense output
        dict(name="rope-far", op="rope", T=4097, Hq=40, Hkv=8, d=128, rot=64, layout="pairs", norm=True, scaled="yarn",
             top=1000000, page=0, dtype="bf16"),
        # copy-on-write of one small page
        dict(name="copy-one-small", op="copy", layers=1, Hkv=4, d=64, page=16, pages=8, n=1, part=True, dtype="f16"),
        # eight requests forked inside a page, every layer
        dict(name="copy-forks", op="copy", layers=32, Hkv=8, d=128, page=16, pages=256, n=8, part=True, dtype="f16"),
        # a cache packed after many requests left
        dict(name="copy-pack", op="copy", layers=16, Hkv=8, d=128, page=64, pages=1100, n=500, part=False,
             dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "rope", "copy"])
    dtype = rng.choice(["f16", "bf16"])
    d = rng.choice([64, 128, 128])
    if op == "attend":
        while True:
            B, Hkv, g = _log(rng, 1, 192), _log(rng, 1, 40), rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16, 33])
            hi = _log(rng, 1, 131072)
            lo = rng.choice([0, hi // 2, hi])
            if B * hi * Hkv * d * 4 <= 10 ** 9 and Hkv * g <= 128 and B * Hkv * g * hi <= 6 * 10 ** 7:
                return dict(op=op, B=B, Hq=Hkv * g, Hkv=Hkv, d=d, page=rng.choice([8, 16, 24, 32, 64, 128]), lo=lo, hi=hi,
                            dtype=dtype)
    if op == "rope":
        while True:
            T, Hkv, g = _log(rng, 1, 20000), _log(rng, 1, 40), rng.choice([1, 2, 4, 5, 8])
            if T * Hkv * (g + 2) * d * 4 <= 7 * 10 ** 8:
                return dict(op=op, T=T, Hq=Hkv * g, Hkv=Hkv, d=d, rot=rng.choice([d, d, d // 2, 16]),
                            layout=rng.choice(["half", "pairs"]), norm=rng.random() < 0.5,
                            scaled=rng.choice(["none", "linear", "yarn"]), top=_log(rng, 256, 2000000),
                            page=rng.choice([0, 8, 16, 24, 64]), dtype=dtype)
    while True:
        layers, Hkv, page, n = _log(rng, 1, 48), _log(rng, 1, 40), rng.choice([8, 16, 24, 64, 128]), _log(rng, 1, 600)
        pages = 2 * n + _log(rng, 1, 100)
        if layers * pages * Hkv * page * d * 4 <= 4 * 10 ** 9:
            return dict(op=op, layers=layers, Hkv=Hkv, d=d, page=page, pages=pages, n=n, part=rng.random() < 0.5,
                        dtype=dtype)


def _lengths(c):
    """The sequences' lengths: spread over lo .. hi, both ends among them."""
    B, lo, hi = c["B"], c["lo"], c["hi"]
    return [hi if b == B - 1 else lo + int((hi - lo) * ((b * 0.6180339887) % 1.0)) for b in range(B)]


def _rows(c):
    """Rows copied by each move: whole pages, or 1 .. page rows."""
    return [c["page"] if not c["part"] else 1 + (7 * i + 4) % c["page"] for i in range(c["n"])]


# ---------------------------------------------------------------------------------------
# what a program has in hand before the call
# ---------------------------------------------------------------------------------------
def _frequencies(c):
    """Rotation per position of each pair (radians) and the factor on cos and sin."""
    rot = c["rot"]
    f = [10000.0 ** (-2.0 * j / rot) for j in range(rot // 2)]
    if c["scaled"] == "linear":
        return [x / 4.0 for x in f], 1.0
    if c["scaled"] == "yarn":  # factor 8 over 4096 positions, ramp between 32 and 1 turns
        at = lambda turns: rot * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(10000.0))  # noqa: E731
        a, b = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), rot - 1)
        out = []
        for j, x in enumerate(f):
            ramp = min(max((j - a) / max(b - a, 0.001), 0.0), 1.0)
            out.append(x / 8.0 * ramp + x * (1.0 - ramp))
        return out, 0.1 * math.log(8.0) + 1.0
    return f, 1.0


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    dt = DTYPES[c["dtype"]]
    s = dict(c=c)
    if c["op"] == "attend":
        B, Hq, Hkv, d, page = c["B"], c["Hq"], c["Hkv"], c["d"], c["page"]
        L = _lengths(c)
        mp = max(1, max(-(-x // page) for x in L))
        need = sum(-(-x // page) for x in L)
        n = need + 3
        s["q"] = torch.randn(B, Hq, d, generator=g, device=DEV, dtype=dt) * 1.25
        s["K"] = torch.randn(n, Hkv, page, d, generator=g, device=DEV, dtype=dt) * 1.25
        s["V"] = torch.randn(n, Hkv, page, d, generator=g, device=DEV, dtype=dt)
        perm = torch.randperm(n, generator=g, device=DEV, dtype=torch.int32)
        L = torch.tensor(L, dtype=torch.int32, device=DEV)
        used = torch.arange(mp, device=DEV)[None, :] < ((L + page - 1) // page)[:, None]
        s["table"] = torch.full((B, mp), -1, dtype=torch.int32, device=DEV)
        s["table"][used] = perm[:need]
        s["L"] = L
        s["out"] = torch.empty(B, Hq, d, dtype=torch.float32, device=DEV)
        s["lse"] = torch.empty(B, Hq, dtype=torch.float32, device=DEV)
        s["ws"] = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)
    elif c["op"] == "rope":
        T, Hq, Hkv, d, page = c["T"], c["Hq"], c["Hkv"], c["d"], c["page"]
        s["qkv"] = torch.randn(T, (Hq + 2 * Hkv) * d, generator=g, device=DEV, dtype=dt) * 1.25
        s["pos"] = torch.randint(0, c["top"], (T,), generator=g, device=DEV, dtype=torch.int32)
        s["wq"] = 1 + 0.1 * torch.randn(d, generator=g, device=DEV, dtype=dt) if c["norm"] else None
        s["wk"] = 1 + 0.1 * torch.randn(d, generator=g, device=DEV, dtype=dt) if c["norm"] else None
        f, s["factor"] = _frequencies(c)
        s["freq"] = torch.tensor(f, dtype=torch.float64, device=DEV)
        # the same as fractions of a turn in 64 bits, which the library's call takes
        turns = [int(x / (2 * math.pi) * 2.0 ** 64) for x in f]
        s["turns"] = torch.tensor([x - 2 ** 64 if x >= 2 ** 63 else x for x in turns], dtype=torch.int64, device=DEV)
        s["q_out"] = torch.empty(T, Hq, d, dtype=dt, device=DEV)
        if page:
            n = -(-T // page) + 2
            s["slot"] = torch.randperm(n * page, generator=g, device=DEV, dtype=torch.int32)[:T] if T < 512 else \
                torch.arange(T, dtype=torch.int32, device=DEV) + page
            s["K"] = torch.zeros(n, Hkv, page, d, dtype=dt, device=DEV)
            s["V"] = torch.zeros(n, Hkv, page, d, dtype=dt, device=DEV)
        else:
            n, s["slot"] = 0, None
            s["K"] = torch.empty(T, Hkv, d, dtype=dt, device=DEV)
            s["V"] = torch.empty(T, Hkv, d, dtype=dt, device=DEV)
        s["pages"] = n
    else:
        layers, Hkv, d, page, P, n = (c[x] for x in ("layers", "Hkv", "d", "page", "pages", "n"))
        s["K"] = torch.randn(layers, P, Hkv, page, d, generator=g, device=DEV, dtype=dt)
        s["V"] = torch.randn(layers, P, Hkv, page, d, generator=g, device=DEV, dtype=dt)
        perm = torch.randperm(P, generator=g, device=DEV)
        rows = torch.tensor(_rows(c), device=DEV)
        s["moves"] = torch.stack([perm[:n], perm[n:2 * n], rows], 1).to(torch.int32).contiguous()
    return s


# ---------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------
def run(s):
    return (_own if own else _plain)[s["c"]["op"]](s)


def _attend_plain(s):
    c = s["c"]
    B, Hq, Hkv, d, page = c["B"], c["Hq"], c["Hkv"], c["d"], c["page"]
    at = s["table"].clamp(min=0).long()
    n = at.shape[1] * page
    live = torch.arange(n, device=DEV)[None, None, None, :] < s["L"][:, None, None, None]
    K = s["K"][at].transpose(1, 2).reshape(B, Hkv, n, d).float()
    z = torch.matmul(s["q"].float().view(B, Hkv, Hq // Hkv, d), K.transpose(2, 3)) / math.sqrt(d)
    del K
    z = z.masked_fill(~live, -math.inf)
    m = z.amax(-1, keepdim=True)
    p = torch.exp(z - m.masked_fill(m == -math.inf, 0.0))
    total = p.sum(-1, keepdim=True)
    V = s["V"][at].transpose(1, 2).reshape(B, Hkv, n, d).float().masked_fill(~live.transpose(2, 3), 0.0)
    o = torch.matmul(p, V) / total.masked_fill(total == 0, 1.0)
    return o.reshape(B, Hq, d), (m + torch.log(total)).reshape(B, Hq)


def _rope_plain(s):
    c = s["c"]
    T, Hq, Hkv, d, rot, page = c["T"], c["Hq"], c["Hkv"], c["d"], c["rot"], c["page"]
    x = s["qkv"].view(T, Hq + 2 * Hkv, d)
    angle = s["pos"].double()[:, None, None] * s["freq"]
    cos, sin = (torch.cos(angle) * s["factor"]).float(), (torch.sin(angle) * s["factor"]).float()

    def turned(y, w):
        y = y.float()
        if w is not None:
            y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + 1e-6) * w.float()
        if c["layout"] == "half":
            a, b = y[..., :rot // 2], y[..., rot // 2:rot]
            r = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
        else:
            a, b = y[..., 0:rot:2], y[..., 1:rot:2]
            r = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
        return torch.cat([r, y[..., rot:]], -1).to(s["qkv"].dtype)

    s["q_out"].copy_(turned(x[:, :Hq], s["wq"]))
    k, v = turned(x[:, Hq:Hq + Hkv], s["wk"]), x[:, Hq + Hkv:]
    if page:
        at, row = (s["slot"] // page).long(), (s["slot"] % page).long()
        s["K"][at, :, row] = k
        s["V"][at, :, row] = v
    else:
        s["K"].copy_(k)
        s["V"].copy_(v)
    return s["q_out"], s["K"], s["V"]


def _copy_plain(s):
    page = s["c"]["page"]
    src, dst, rows = s["moves"].long().unbind(1)
    keep = (torch.arange(page, device=DEV)[None, :] < rows[:, None])[None, :, None, :, None]
    for x in (s["K"], s["V"]):
        x[:, dst] = torch.where(keep, x[:, src], x[:, dst])
    return s["K"], s["V"]


def _attend_own(s):
    from speculative_kv_cache_gb300 import ig

    c = s["c"]
    ig.ig_paged_attend(None, ig.IG_F16 if c["dtype"] == "f16" else ig.IG_BF16, c["B"], c["Hq"], c["Hkv"], c["d"], c["page"],
                       s["K"].shape[0], s["table"].shape[1], 1.0 / math.sqrt(c["d"]), s["q"], s["K"], s["V"], s["table"],
                       s["L"], s["out"], s["lse"], s["ws"], s["ws"].numel())
    return s["out"], s["lse"]


def _rope_own(s):
    from speculative_kv_cache_gb300 import ig

    c = s["c"]
    Hq, Hkv, d = c["Hq"], c["Hkv"], c["d"]
    x = s["qkv"]
    w = x.shape[1]
    q, k, v = x[:, :Hq * d], x[:, Hq * d:(Hq + Hkv) * d], x[:, (Hq + Hkv) * d:]
    ig.ig_qk_norm_rope(None, ig.IG_F16 if c["dtype"] == "f16" else ig.IG_BF16, c["T"], Hq, Hkv, d, c["rot"],
                       ig.IG_ROPE_HALF if c["layout"] == "half" else ig.IG_ROPE_PAIRS, q, w, k, w, v, w, s["wq"], s["wk"],
                       1e-6, s["pos"], s["turns"], s["factor"], s["q_out"], c["page"], s["pages"], s["slot"], s["K"],
                       s["V"])
    return s["q_out"], s["K"], s["V"]


def _copy_own(s):
    from speculative_kv_cache_gb300 import ig

    c = s["c"]
    ig.ig_page_copy(None, c["layers"], c["pages"], c["Hkv"], c["page"], c["d"], list(s["K"]), list(s["V"]), c["n"],
                    s["moves"])
    return s["K"], s["V"]


_plain = {"attend": _attend_plain, "rope": _rope_plain, "copy": _copy_plain}
_own = {"attend": _attend_own, "rope": _rope_own, "copy": _copy_own}


def work(case):
    c = case
    if c["op"] == "attend":
        tokens = sum(_lengths(c))
        q = c["B"] * c["Hq"] * c["d"]
        pages = sum(-(-x // c["page"]) for x in _lengths(c))
        return dict(bytes=tokens * c["Hkv"] * c["d"] * 4 + q * (2 + 4) + c["B"] * (c["Hq"] + 1) * 4 + pages * 4,
                    flops=4 * c["d"] * c["Hq"] * tokens)
    if c["op"] == "rope":
        values = c["T"] * (c["Hq"] + 2 * c["Hkv"]) * c["d"]
        return dict(bytes=4 * values + 8 * c["T"], flops=10 * c["T"] * (c["Hq"] + c["Hkv"]) * c["d"])
    return dict(bytes=2 * c["layers"] * 2 * c["Hkv"] * c["d"] * 2 * sum(_rows(c)) + 12 * c["n"], flops=0)


# ---------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------
def exact(case, seed):
    return {"attend": _attend_exact, "rope": _rope_exact, "copy": _copy_exact}[case["op"]](case, prepare(case, seed))


def _attend_exact(c, s):
    group, d = c["Hq"] // c["Hkv"], c["d"]
    out = torch.zeros(c["B"], c["Hq"], d, dtype=torch.float64, device=DEV)
    lse = torch.full((c["B"], c["Hq"]), -math.inf, dtype=torch.float64, device=DEV)
    table = s["table"].tolist()
    for b, n in enumerate(_lengths(c)):
        if n == 0:
            continue
        pages = torch.tensor(table[b][:-(-n // c["page"])], device=DEV)
        for h in range(c["Hkv"]):
            keys = s["K"][pages, h].reshape(-1, d)[:n].double()
            values = s["V"][pages, h].reshape(-1, d)[:n].double()
            q = s["q"][b, h * group:(h + 1) * group].double()
            logits = (q @ keys.T) * d ** -0.5
            lse[b, h * group:(h + 1) * group] = torch.logsumexp(logits, 1)
            out[b, h * group:(h + 1) * group] = torch.softmax(logits, 1) @ values
    return out, lse


def _rope_exact(c, s):
    T, Hq, Hkv, d, rot, page = c["T"], c["Hq"], c["Hkv"], c["d"], c["rot"], c["page"]
    half = rot // 2
    x = s["qkv"].double().view(T, Hq + 2 * Hkv, d)
    index = torch.arange(half, dtype=torch.float64, device=DEV)
    freq = torch.exp(index * (-math.log(10000.0) * 2 / rot))
    factor = 1.0
    if c["scaled"] == "linear":
        freq = freq / 4
    elif c["scaled"] == "yarn":
        where = [rot * math.log(4096 / (2 * math.pi * n)) / (2 * math.log(10000.0)) for n in (32, 1)]
        first, last = max(math.floor(where[0]), 0), min(math.ceil(where[1]), rot - 1)
        mix = ((index - first) / max(last - first, 0.001)).clamp(0, 1)
        freq = freq * (1 - mix + mix / 8)
        factor = 1 + math.log(8.0) / 10
    turn = torch.polar(torch.full((T, 1, half), factor, dtype=torch.float64, device=DEV),
                       s["pos"].double().view(T, 1, 1) * freq)
    first = list(range(half)) if c["layout"] == "half" else list(range(0, rot, 2))
    second = list(range(half, rot)) if c["layout"] == "half" else list(range(1, rot, 2))

    def heads(y, w):
        y = y.clone()
        if w is not None:
            y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * w.double()
        z = torch.complex(y[..., first], y[..., second]) * turn
        y[..., first], y[..., second] = z.real, z.imag
        return y

    q, k, v = heads(x[:, :Hq], s["wq"]), heads(x[:, Hq:Hq + Hkv], s["wk"]), x[:, Hq + Hkv:]
    if not page:
        return q, k, v.contiguous()
    out = []
    for y in (k, v):
        cache = torch.zeros(s["pages"] * page, Hkv, d, dtype=torch.float64, device=DEV)
        cache.index_copy_(0, s["slot"].long(), y.contiguous())
        out.append(cache.view(s["pages"], page, Hkv, d).transpose(1, 2).contiguous())
    return q, out[0], out[1]


def _copy_exact(c, s):
    for a, b, n in s["moves"].tolist():
        for x in (s["K"], s["V"]):
            x[:, b, :, :n] = x[:, a, :, :n]
    return s["K"], s["V"]
