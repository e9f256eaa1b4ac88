"""The paged cache's operators for drafted trees and picked pages against plain implementations in 64 bits.

Tolerances.  u = 2^-23 bounds one fp32 operation, truncation included; h is half a step of the type (bf16 2^-8, fp16 2^-11).
* tree attention: logits and weights as in the attention of one token (a logit is off by at most (d + 4) u A_t, a weight
  by e = exp(2 (d + 8) u max A + 2^-20) - 1); each weight is rounded to the type for the second product, h of it, in fp16
  at least half of the least step, 2^-25, where the largest weight, and so their sum, is at least 2^10 (the reference is 10
  below the logit that set it, and the largest is no lower): 2^-35 of the sum; the result is rounded once.  So with w
  the weights and v the values
  |o - o64| <= (2 e + h + (L + 64) u) sum w |v| + [fp16] 2^-35 sum |v| + h |o64| + least step / 2,
  lse: (d + 8) u max A + 2 e + (L + 64) u + 8 u |lse|.
* bounds, choices, slots, kept rows: equal (every number in them is exact).
* attention over picked pages: as the attention of one token over the same tokens.
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -23
DT = {"f16": torch.float16, "bf16": torch.bfloat16}
HALF = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}
LEAST = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134}  # half of the least step


@pytest.fixture(scope="module")
def ig():
    if not torch.cuda.is_available():
        pytest.fail("a CUDA GPU is required for the -m gpu tests")
    from speculative_kv_cache_gb300 import build

    build.build()
    from speculative_kv_cache_gb300 import ig as mod

    return mod


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def i64(x):
    return torch.tensor([v - 2 ** 64 if v >= 2 ** 63 else v for v in x], dtype=torch.int64, device=DEV)


def dtype_of(ig, dt):
    return ig.IG_F16 if dt == "f16" else ig.IG_BF16


def refused_on_device(ig):
    with pytest.raises(ig.IGError) as e:
        ig.ig_check()
    assert e.value.status == ig.IG_ERR_INVALID
    ig.ig_check()


def a_tree(rng, n, deep=False):
    return [-1 if i == 0 or (not deep and rng.random() < 0.2) else int(rng.integers(max(0, i - 4), i)) for i in range(n)]


def ancestors(parents):
    out = []
    for i, p in enumerate(parents):
        out.append(1 << i | (out[p] if p >= 0 else 0))
    return out


def layout(rng, lengths, page, spare=3, fill=2 ** 31 - 1):
    """Pages in random order: the table as lists (``fill`` where it is not used) and the number of pages."""
    count = [-(-n // page) for n in lengths]
    n = sum(count) + spare
    perm = rng.permutation(n).tolist()
    mp = max(1, max(count))
    table = [[perm.pop() for _ in range(c)] + [fill] * (mp - c) for c in count]
    return table, n, mp


# ---------------------------------------------------------------------------------------
# slots
# ---------------------------------------------------------------------------------------
def slots_by_loops(table, L, seq, counts, parents, page, T):
    first, slots, positions, masks = [0], [], [], []
    for s, n in zip(seq, counts):
        base = L[s] - n
        slots += [table[s][x // page] * page + x % page for x in range(base, base + n)]
        if n <= 64:
            bits = ancestors(parents[first[-1]:first[-1] + n] if parents else [i - 1 for i in range(n)])
            masks += bits
        else:
            bits = []
        positions += [base + bin(b).count("1") - 1 for b in bits] if parents else list(range(base, base + n))
        first.append(first[-1] + n)
    pad = T - first[-1]
    return first, slots + [-1] * pad, positions + [0] * pad, masks + [0] * pad


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("n,page,have,most,pad", [(1, 8, 0, 1, 0), (1, 16, 5, 64, 3), (3, 24, 100, 64, 0), (33, 16, 40, 33, 7),
                                                  (255, 32, 9, 17, 1), (256, 8, 0, 64, 0), (257, 64, 1000, 5, 300),
                                                  (5, 16, 3, 700, 9), (2000, 8, 70, 3, 50), (8192, 8, 20, 2, 1)])
def test_slots(ig, n, page, have, most, pad, tree):
    if tree:
        most = min(most, 64)
    rng = np.random.default_rng(n + page)
    seqs = n + 3
    seq = rng.permutation(seqs)[:n].tolist()
    counts = [most if i == n - 1 else int(rng.integers(0, most + 1)) for i in range(n)]
    L = [int(rng.integers(0, have + 1)) for _ in range(seqs)]
    for s, c in zip(seq, counts):
        L[s] += c
    table, pages, mp = layout(rng, L, page)
    parents = [p for c in counts for p in a_tree(rng, c)] if tree else None
    T = sum(counts) + pad
    first, slots, positions, masks = slots_by_loops(table, L, seq, counts, parents, page, T)
    dev = dict(table=i32(table), L=i32(L), seq=i32(seq), counts=i32(counts))
    up = i32(parents + [77] * pad) if tree else None  # (what lies behind is not read)
    for with_masks in ([True] if tree else [True, False]):
        if with_masks and max(counts) > 64:
            continue
        f, s, p = (torch.full((k,), -9, dtype=torch.int32, device=DEV) for k in (n + 1, T, T))
        m = torch.full((T,), -9, dtype=torch.int64, device=DEV) if with_masks else None
        ig.ig_page_slots(None, n, seqs, page, pages, mp, T, dev["table"], dev["L"], dev["seq"], dev["counts"], up, f, s, p, m)
        ig.ig_check()
        assert f.tolist() == first and s.tolist() == slots and p.tolist() == positions
        if with_masks:
            assert torch.equal(m, i64(masks))


def test_slots_in_the_sequences_own_order(ig):
    table, L, counts = [[3, 1], [0, 2], [4, 5]], [9, 16, 0], [2, 1, 0]
    f, s, p = (torch.empty(k, dtype=torch.int32, device=DEV) for k in (4, 3, 3))
    ig.ig_page_slots(None, 3, 3, 8, 6, 2, 3, i32(table), i32(L), None, i32(counts), None, f, s, p)
    assert f.tolist() == [0, 2, 3, 3] and s.tolist() == [31, 8, 23] and p.tolist() == [7, 8, 15]
    ig.ig_check()


def test_a_deep_tree_and_one_level(ig):
    for parents in ([i - 1 for i in range(64)], [-1] * 64, [max(-1, i - 2) for i in range(64)], [min(i - 1, 0) for i in range(64)]):
        m, s, p, f = (torch.empty(64, dtype=torch.int64, device=DEV), torch.empty(64, dtype=torch.int32, device=DEV),
                      torch.empty(64, dtype=torch.int32, device=DEV), torch.empty(2, dtype=torch.int32, device=DEV))
        ig.ig_page_slots(None, 1, 1, 64, 1, 1, 64, i32([[0]]), i32([64]), None, i32([64]), i32(parents), f, s, p, m)
        bits = ancestors(parents)
        assert torch.equal(m, i64(bits)) and p.tolist() == [bin(b).count("1") - 1 for b in bits]
    ig.ig_check()


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("bad", ["seq", "seq_low", "length", "length_low", "count", "many", "page", "room"])
def test_slots_leave_out_bad_requests_and_say_so(ig, bad, tree):
    """Request 1 of three cannot be; the others are as if it were not (it keeps its place, but for a count below zero)."""
    page, L, seq, counts = 8, [20, 9, 30], [0, 1, 2], [3, 2, 4]
    table = [[0, 1, 2, -1], [3, 4, -1, -1], [5, 6, 7, 8]]
    T = 9
    if bad == "seq":
        seq[1] = 3
    elif bad == "seq_low":
        seq[1] = -1
    elif bad == "length":
        L[1] = 33
    elif bad == "length_low":
        L[1] = -5
    elif bad == "count":
        counts[1] = -1
    elif bad == "many":
        L[1] = 1
    elif bad == "page":
        table[1][0], table[1][1] = 9, 9
    else:
        counts, T = [3, 2, 7], 9
    up = i32([-1] * T) if tree else None
    f, s, p = (torch.full((k,), -9, dtype=torch.int32, device=DEV) for k in (4, T, T))
    m = torch.full((T,), -9, dtype=torch.int64, device=DEV) if tree else None
    ig.ig_page_slots(None, 3, 3, page, 9, 4, T, i32(table), i32(L), i32(seq), i32(counts), up, f, s, p, m)
    refused_on_device(ig)
    flat = lambda base, n: [base] * n if tree else list(range(base, base + n))  # noqa: E731
    if bad == "room":
        assert f.tolist() == [0, 3, 5, 9]
        assert s.tolist() == [17, 18, 19, 3 * 8 + 7, 4 * 8, -1, -1, -1, -1]
        return
    c = 0 if bad == "count" else 2
    assert f.tolist() == [0, 3, 3 + c, 7 + c]
    assert s.tolist() == [17, 18, 19] + [-1] * c + [8 * 8 + 2 + i for i in range(4)] + [-1] * (2 - c)
    assert p.tolist() == flat(17, 3) + (flat(7, 2) if bad == "page" else [0] * c) + flat(26, 4) + [0] * (2 - c)


def test_slots_of_parents_out_of_range(ig):
    """They count as -1; more than 64 tokens with parents are left out."""
    f, s, p = (torch.empty(k, dtype=torch.int32, device=DEV) for k in (2, 4, 4))
    m = torch.empty(4, dtype=torch.int64, device=DEV)
    ig.ig_page_slots(None, 1, 1, 8, 1, 1, 4, i32([[0]]), i32([4]), None, i32([4]), i32([-2, 1, 0, 9]), f, s, p, m)
    refused_on_device(ig)
    assert m.tolist() == [1, 2, 5, 8] and p.tolist() == [0, 0, 1, 0] and s.tolist() == [0, 1, 2, 3]
    f, s, p = (torch.empty(k, dtype=torch.int32, device=DEV) for k in (2, 65, 65))
    ig.ig_page_slots(None, 1, 1, 8, 9, 9, 65, i32([list(range(9))]), i32([65]), None, i32([65]), i32([-1] * 65), f, s, p)
    refused_on_device(ig)
    assert s.tolist() == [-1] * 65 and p.tolist() == [0] * 65 and f.tolist() == [0, 65]


# ---------------------------------------------------------------------------------------
# tree attention
# ---------------------------------------------------------------------------------------
def make_tree(seed, dt, lengths, drafted, Hq, Hkv, d, page, masks=None, qs=1.25, seq=None, seqs=None, rows_behind=0, n_pages=None):
    """Every row past a sequence's end, and every spare page, is NaN."""
    rng = np.random.default_rng(seed)
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    B = len(lengths)
    seqs = seqs or B
    seq_of = seq if seq is not None else list(range(B))
    L = [0] * seqs
    for s, n in zip(seq_of, lengths):
        L[s] = n
    table, n, mp = layout(rng, L, page)
    K = torch.full((n, Hkv, page, d), float("nan"), dtype=DT[dt], device=DEV)
    V = torch.full((n, Hkv, page, d), float("nan"), dtype=DT[dt], device=DEV)
    for s, x in enumerate(L):
        for i in range(-(-x // page)):
            live = min(page, x - i * page)
            K[table[s][i], :, :live] = (torch.randn(Hkv, live, d, generator=g, device=DEV) * 1.25).to(DT[dt])
            V[table[s][i], :, :live] = torch.randn(Hkv, live, d, generator=g, device=DEV).to(DT[dt])
    first = np.concatenate([[0], np.cumsum(drafted)]).tolist()
    if masks is None:
        masks = [m for x in drafted for m in ancestors(a_tree(rng, x))]
    T = first[-1] + rows_behind
    q = (torch.randn(T, Hq, d, generator=g, device=DEV) * qs).to(DT[dt])
    return dict(dt=dt, B=B, Hq=Hq, Hkv=Hkv, d=d, page=page, n=n, mp=mp, seqs=seqs, seq=None if seq is None else i32(seq), seq_of=seq_of,
                q=q, K=K, V=V, table=i32(table), L=i32(L), lengths=list(lengths), drafted=list(drafted), first=first,
                dfirst=i32(first), bits=list(masks) + [0] * rows_behind, masks=i64(list(masks) + [0] * rows_behind), T=T,
                T_max=max([1] + list(drafted)), scale=1.0 / math.sqrt(d))


def attend_tree(ig, c, out=None, lse=None, ws=None, stream=None, want_lse=True):
    out = torch.full((c["T"], c["Hq"], c["d"]), 77.0, dtype=DT[c["dt"]], device=DEV) if out is None else out
    lse = torch.full((c["T"], c["Hq"]), 77.0, dtype=torch.float32, device=DEV) if lse is None and want_lse else lse
    if ws is None:  # arbitrary content
        ws = torch.full((ig.ig_paged_tree_attend_workspace_bytes(c["B"], c["T_max"], c["Hq"], c["Hkv"], c["d"]),), 0xff,
                        dtype=torch.uint8, device=DEV)
    ig.ig_paged_tree_attend(stream, dtype_of(ig, c["dt"]), c["B"], c["T"], c["T_max"], c["Hq"], c["Hkv"], c["d"], c["page"], c["n"],
                            c["seqs"], c["mp"], c["scale"], c["q"], c["K"], c["V"], c["table"], c["L"], c["seq"], c["dfirst"],
                            c["masks"], out, lse, ws, ws.numel())
    return out, lse


def check_tree(c, out, lse, drop=(), left=()):
    """Against the definition; drop: (request, table entry) whose tokens are left out; left: requests left as they were."""
    group, d, page, dt = c["Hq"] // c["Hkv"], c["d"], c["page"], c["dt"]
    table = c["table"].tolist()
    for b, (n, k) in enumerate(zip(c["lengths"], c["drafted"])):
        f = c["first"][b]
        if b in left:
            assert torch.all(out[f:f + k] == 77) and torch.all(lse[f:f + k] == 77)
            continue
        if k == 0:
            continue
        keep = [t for t in range(n) if (b, t // page) not in drop]
        s = c["seq_of"][b]
        p = torch.tensor([table[s][t // page] for t in keep], device=DEV, dtype=torch.long)
        r = torch.tensor([t % page for t in keep], device=DEV, dtype=torch.long)
        K, V = c["K"][p, :, r].double(), c["V"][p, :, r].double()  # [L, Hkv, d]
        q = c["q"][f:f + k].double().view(k, c["Hkv"], group, d)
        seen = torch.tensor([[t < n - k or bool(c["bits"][f + i] >> (t - n + k) & 1) for t in keep] for i in range(k)],
                            device=DEV).view(k, 1, 1, -1)
        z = torch.einsum("nhgd,thd->nhgt", q, K) * c["scale"]
        z = torch.where(seen, z, -math.inf)
        A = torch.where(seen, torch.einsum("nhgd,thd->nhgt", q.abs(), K.abs()) * abs(c["scale"]), 0.0)
        A = A.amax(-1) if keep else torch.zeros(k, c["Hkv"], group, device=DEV, dtype=torch.float64)
        none = ~seen.any(-1, keepdim=True).expand(k, c["Hkv"], group, 1)
        w = torch.where(none, 0.0, torch.softmax(z, -1)) if keep else z
        V = torch.where(seen.any(0).view(-1, 1, 1), V, 0.0)  # (rows that nobody sees)
        o = torch.einsum("nhgt,thd->nhgd", w, V)
        wv = torch.einsum("nhgt,thd->nhgd", w, V.abs())
        e = torch.exp(2 * (d + 8) * U * A + 2.0 ** -20) - 1
        add = (len(keep) + 64) * U
        tol = (2 * e + HALF[dt] + add)[..., None] * wv + HALF[dt] * o.abs() + LEAST[dt]
        if dt == "f16":
            tol = tol + 2.0 ** -35 * torch.einsum("nt,thd->nhd", seen[:, 0, 0].double(), V.abs())[:, :, None]
        diff = (out[f:f + k].double().view(o.shape) - o).abs()
        assert torch.all(diff <= tol), (b, float((diff / tol).max()))
        if lse is not None:
            ref = torch.logsumexp(z, -1) if keep else torch.full_like(A, -math.inf)
            got = lse[f:f + k].double().view(ref.shape)
            off = none[..., 0]
            assert torch.all(got[off] == -math.inf)
            dl = (got - ref).abs()[~off]
            assert torch.all(dl <= ((d + 8) * U * A + 2 * e + add + 8 * U * ref.abs())[~off])
    end = c["first"][-1]
    assert torch.all(out[end:] == 77) and (lse is None or torch.all(lse[end:] == 77))


EDGES = [1, 2, 7, 8, 9, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 190, 191, 192, 193, 255, 256, 257, 300, 1000]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [8, 16, 24, 40, 64, 128, 256])
def test_tree_lengths_and_pages(ig, dt, d, page):
    drafted = [min(n, 1 + (5 * i) % 64) for i, n in enumerate(EDGES)]
    c = make_tree(1, dt, EDGES, drafted, 4, 2, d, page)
    check_tree(c, *attend_tree(ig, c))
    ig.ig_check()


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (4, 1), (6, 2), (5, 1), (7, 1), (16, 2), (12, 1), (33, 1), (40, 8), (130, 1)])
@pytest.mark.parametrize("dt,d", [("f16", 128), ("bf16", 64)])
def test_tree_head_layouts(ig, Hq, Hkv, dt, d):
    c = make_tree(2, dt, [70, 1, 333, 20, 129], [5, 1, 31, 0, 64], Hq, Hkv, d, 16)
    check_tree(c, *attend_tree(ig, c))
    ig.ig_check()


@pytest.mark.parametrize("B,n,Hq,Hkv,d,page,dt,hi", [(1, 8, 8, 2, 128, 32, "f16", 20001), (2, 64, 16, 2, 128, 64, "bf16", 9001),
                                                     (40, 5, 8, 4, 64, 16, "f16", 1500), (3, 33, 32, 4, 128, 24, "f16", 5000),
                                                     (150, 3, 4, 2, 128, 32, "bf16", 300), (1, 64, 40, 8, 64, 128, "bf16", 30000),
                                                     (300, 2, 2, 1, 64, 8, "f16", 90)])
def test_tree_splits_over_length_and_batch(ig, B, n, Hq, Hkv, d, page, dt, hi):
    rng = np.random.default_rng(B + n)
    lengths = [hi if b == B - 1 else int(rng.integers(1, hi + 1)) for b in range(B)]
    drafted = [min(x, n if b == B - 1 else int(rng.integers(0, n + 1))) for b, x in enumerate(lengths)]
    c = make_tree(3, dt, lengths, drafted, Hq, Hkv, d, page)
    check_tree(c, *attend_tree(ig, c))
    ig.ig_check()


@pytest.mark.parametrize("dt,d", [("f16", 64), ("bf16", 128)])
@pytest.mark.parametrize("G,n", [(2, 64), (3, 43), (4, 64), (6, 43), (4, 32), (4, 33), (127, 1), (128, 1), (129, 1), (256, 1),
                                 (257, 1), (256, 3), (17, 31)])
def test_tree_rows_about_the_ends_of_blocks(ig, G, n, dt, d):
    """A key head's rows, n G of them, at 128 and 256 and one past them, in short sequences and in one that many CTAs share."""
    c = make_tree(21, dt, [n, 4001, n + 63, 300], [n, n, max(1, n - 1), n], 2 * G, 2, d, 32)
    check_tree(c, *attend_tree(ig, c))
    ig.ig_check()


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("lengths,n,G,Hkv", [([9000], 64, 8, 1), ([5000, 77, 2600], 64, 8, 2), ([4000, 64], 64, 12, 2),
                                             ([2500, 900, 43, 44, 3000], 43, 24, 1), ([1500, 70, 1300, 300], 64, 16, 8),
                                             ([6000, 6001], 64, 33, 1), ([130] * 30, 33, 8, 3)])
def test_tree_of_several_blocks_of_rows(ig, lengths, n, G, Hkv, dt):
    """All requests with as many blocks of rows (2 to 9 of them), which CTAs take side by side where that leaves few idle."""
    drafted = [n] * len(lengths)
    c = make_tree(28, dt, lengths + [40], drafted + [0], G * Hkv, Hkv, 128, 64)
    out = attend_tree(ig, c)
    check_tree(c, *out)
    again = attend_tree(ig, c)
    assert torch.equal(out[0], again[0]) and torch.equal(out[1], again[1])
    ig.ig_check()


@pytest.mark.parametrize("G", [1, 2, 3, 8])
@pytest.mark.parametrize("lengths,drafted", [([5], [1]), ([700, 90], [2, 3]), ([4000], [33])])
def test_tree_with_room_for_more_tokens(ig, lengths, drafted, G):
    """T_max above every count, and above all tokens."""
    for d in (64, 128):
        c = make_tree(29, "bf16", lengths, drafted, 2 * G, 2, d, 16)
        c["T_max"] = 64
        check_tree(c, *attend_tree(ig, c))
    ig.ig_check()


def test_tree_of_more_requests_than_threads(ig):
    rng = np.random.default_rng(22)
    lengths = [int(rng.integers(1, 40)) for _ in range(1000)]
    drafted = [min(x, int(rng.integers(0, 4))) for x in lengths]
    c = make_tree(22, "f16", lengths, drafted, 2, 1, 64, 8)
    check_tree(c, *attend_tree(ig, c))
    ig.ig_check()


@pytest.mark.parametrize("G", [1, 4])
@pytest.mark.parametrize("n", [1, 31, 32, 33, 63, 64])
def test_tree_without_an_earlier_token_and_with_any_mask(ig, n, G):
    """The whole sequence is drafted; masks are any bits, some of them none (bits past the tree say nothing)."""
    rng = np.random.default_rng(n)
    masks = [int(x) for x in rng.integers(0, 2 ** 64, n, dtype=np.uint64)]
    masks[0], masks[n // 2], masks[-1] = 2 ** 64 - 1, (2 ** 64 - 1) ^ (2 ** n - 1), 1 << (n - 1)
    c = make_tree(4, "f16", [n], [n], G, 1, 64, 16, masks=masks)
    check_tree(c, *attend_tree(ig, c))
    ig.ig_check()


def test_tree_of_named_sequences_and_rows_behind(ig):
    c = make_tree(5, "bf16", [50, 200, 7], [3, 9, 7], 8, 2, 128, 16, seq=[4, 0, 2], seqs=6, rows_behind=5)
    check_tree(c, *attend_tree(ig, c))
    out, _ = attend_tree(ig, c, want_lse=False)
    check_tree(c, out, None)
    ig.ig_check()


@pytest.mark.parametrize("scale", [-0.125, 0.0, 3.0])
def test_tree_other_scales(ig, scale):
    c = make_tree(6, "f16", [300, 64], [10, 64], 6, 3, 64, 8)
    c["scale"] = scale
    check_tree(c, *attend_tree(ig, c))


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("what", ["nan", "inf", "-inf"])
def test_tree_unseen_rows_may_be_anything(ig, dt, d, what):
    """A drafted row whose key and value are not finite reaches the tokens that see it, and no others."""
    lengths, drafted = [140, 64, 129], [20, 64, 3]
    masks = [m for x in drafted for m in ancestors([i - 1 if i % 2 else -1 for i in range(x)])]
    c = make_tree(7, dt, lengths, drafted, 4, 2, d, 16, masks=masks)
    rows = []
    for b, j in ((0, 2), (0, 19), (1, 0), (1, 63), (2, 1)):
        t = lengths[b] - drafted[b] + j
        at = (int(c["table"][b, t // 16]), t % 16)
        rows.append((b, j, at))
        c["V"][at[0], :, at[1], 3::7] = float(what)
        c["K"][at[0], :, at[1]] = float("nan") if what == "nan" else 0.0
    out, lse = attend_tree(ig, c)
    ig.ig_check()
    # as if those rows were zero, for the tokens that do not see them
    clean = dict(c, K=c["K"].clone(), V=c["V"].clone())
    for b, j, at in rows:
        clean["V"][at[0], :, at[1]] = 0
        clean["K"][at[0], :, at[1]] = 0
    want, wlse = attend_tree(ig, clean)
    for b, (f, k) in enumerate(zip(c["first"], drafted)):
        for i in range(k):
            hit = [j for bb, j, _ in rows if bb == b and c["bits"][f + i] >> j & 1]
            if not hit:
                assert torch.equal(out[f + i], want[f + i]) and torch.equal(lse[f + i], wlse[f + i])
            elif what == "nan":
                assert not torch.isfinite(out[f + i]).any()
            else:
                touched = torch.zeros(d, dtype=torch.bool, device=DEV)
                touched[3::7] = True
                assert torch.all(out[f + i][:, touched] == float(what)) and torch.isfinite(out[f + i][:, ~touched]).all()
                assert torch.equal(lse[f + i], wlse[f + i])


@pytest.mark.parametrize("dt,d", [("f16", 64), ("f16", 128), ("bf16", 64), ("bf16", 128)])
@pytest.mark.parametrize("what", ["nan", "inf", "-inf"])
@pytest.mark.parametrize("lengths,drafted,G,Hkv,page", [
    ([5000], [64], 2, 2, 16),                 # 128 rows, cut
    ([5000], [64], 4, 2, 24),                 # 256 rows, cut: one group clears for both
    ([5000], [64], 8, 1, 64),                 # 512 rows in CTAs side by side, cut
    ([5000, 3000], [64, 64], 5, 1, 32),       # 320 rows, the last 64 in a group's own unit
    ([5000, 3000, 64, 700], [64, 20, 64, 33], 8, 2, 8),  # of several numbers of blocks, so one after the other
    ([200, 64, 190, 321], [64, 64, 7, 64], 8, 3, 40)])   # few tiles, none cut
def test_tree_unseen_rows_may_be_anything_in_blocks_and_parts(ig, dt, d, what, lengths, drafted, G, Hkv, page):
    """As above, where a key head has more than 128 rows, and where several CTAs share a sequence's tiles: drafted rows on both
    sides of a tile's end, their keys and values not finite."""
    bad = [(b, j) for b, n in enumerate(drafted) for j in (2, 19, 55, 56, 63) if j < n]
    masks = [m for x in drafted for m in ancestors([i - 1 if i % 2 else -1 for i in range(x)])]
    c = make_tree(31, dt, lengths, drafted, G * Hkv, Hkv, d, page, masks=masks)
    clean = dict(c, K=c["K"].clone(), V=c["V"].clone())
    for b, j in bad:
        t = lengths[b] - drafted[b] + j
        at = (int(c["table"][b, t // page]), slice(None), t % page)
        c["V"][at][:, 3::7] = float(what)
        c["K"][at] = float("nan") if what == "nan" else 0.0
        clean["V"][at][:, 3::7] = 0
        clean["K"][at] = 0
    (out, lse), (want, wlse) = attend_tree(ig, c), attend_tree(ig, clean)
    ig.ig_check()
    check_tree(clean, want, wlse)
    touched = torch.zeros(d, dtype=torch.bool, device=DEV)
    touched[3::7] = True
    hit = torch.tensor([any(c["bits"][c["first"][b] + i] >> j & 1 for bb, j in bad if bb == b)
                        for b, n in enumerate(drafted) for i in range(n)], device=DEV)
    assert hit.any() and not hit.all()
    assert torch.equal(out[~hit], want[~hit]) and torch.equal(lse[~hit], wlse[~hit])
    if what == "nan":
        assert not torch.isfinite(out[hit]).any()
    else:
        assert torch.all(out[hit][:, :, touched] == float(what))
        assert torch.equal(out[hit][:, :, ~touched], want[hit][:, :, ~touched]) and torch.equal(lse[hit], wlse[hit])


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_tree_large_logits_and_small_weights_beside_a_large_one(ig, dt):
    """Logits up to some hundreds; and a first token whose value is zero takes nearly all the weight."""
    c = make_tree(8, dt, [700, 90], [12, 5], 4, 1, 128, 16, qs=30.0)
    check_tree(c, *attend_tree(ig, c))
    c = make_tree(9, dt, [3000], [6], 4, 1, 64, 16)
    page0 = int(c["table"][0, 0])
    c["K"][page0, 0, 0] = c["q"][:, :, :].float().mean((0, 1)).to(DT[dt])
    c["q"] = (c["q"].float() * 0.1 + c["K"][page0, 0, 0].float() * 24).to(DT[dt])
    c["V"][page0, 0, 0] = 0
    check_tree(c, *attend_tree(ig, c))


def test_tree_rises_and_falls(ig):
    """Logits that grow by steps along the sequence, so that the running maximum moves in most tiles, and then fall."""
    for dt in ("f16", "bf16"):
        for d, G in ((64, 1), (128, 5)):
            c = make_tree(10, dt, [4000, 2100], [7, 64], G, 1, d, 16)
            u = torch.ones(d, device=DEV) / math.sqrt(d)
            c["q"] = (c["q"].float() * 0.1 + 4 * u).to(DT[dt])
            for b, n in enumerate(c["lengths"]):
                for t in range(n):
                    up = (t // 100 if t < n // 2 else (n - t) // 100) * 1.5
                    p, r = int(c["table"][b, t // 16]), t % 16
                    c["K"][p, 0, r] = (c["K"][p, 0, r].float() * 0.1 + up * u * math.sqrt(d) / 4).to(DT[dt])
            check_tree(c, *attend_tree(ig, c))


def test_tree_leaves_out_bad_pages_and_bad_requests_and_says_so(ig):
    c = make_tree(11, "f16", [100, 300, 40], [6, 9, 4], 4, 2, 64, 16)
    c["table"][0, 2], c["table"][1, 0], c["table"][1, 18] = c["n"], -1, 2 ** 31 - 1
    out, lse = attend_tree(ig, c)
    refused_on_device(ig)
    check_tree(c, out, lse, drop=[(0, 2), (1, 0), (1, 18)])
    for b, (name, value) in enumerate([("L", 2), ("L", 10 ** 6), ("L", -1)]):
        c = make_tree(12, "bf16", [100, 300, 40], [6, 9, 4], 4, 2, 64, 16)
        c[name][b] = value
        out, lse = attend_tree(ig, c)
        refused_on_device(ig)
        check_tree(c, out, lse, left=[b])
    c = make_tree(13, "f16", [100, 300, 40], [6, 9, 4], 4, 2, 64, 16, seq=[0, 1, 2])
    c["seq"][1] = 3
    out, lse = attend_tree(ig, c)
    refused_on_device(ig)
    check_tree(c, out, lse, left=[1])
    c = make_tree(14, "f16", [100, 300, 40], [6, 9, 4], 4, 2, 64, 16)
    c["T_max"] = 8
    out, lse = attend_tree(ig, c)
    refused_on_device(ig)
    check_tree(c, out, lse, left=[1])
    c = make_tree(14, "f16", [100, 300, 40], [6, 9, 4], 4, 2, 64, 16)
    c["dfirst"][3] = 99
    c["T_max"] = 64
    out, lse = attend_tree(ig, c)
    refused_on_device(ig)
    check_tree(c, out, lse, left=[2])


def test_tree_offsets_past_32_bits(ig):
    """Pages whose bytes and elements lie past 2^32."""
    Hkv, page, d = 8, 64, 128
    n = (5 << 30) // (Hkv * page * d)
    K = torch.zeros((n, Hkv, page, d), dtype=torch.bfloat16, device=DEV)
    V = torch.zeros((n, Hkv, page, d), dtype=torch.bfloat16, device=DEV)
    c = make_tree(15, "bf16", [500], [7], 16, Hkv, d, page)
    far = [n - 1 - 3 * i for i in range(8)]
    for i in range(8):
        K[far[i]], V[far[i]] = c["K"][int(c["table"][0, i])], c["V"][int(c["table"][0, i])]
    c.update(K=K, V=V, n=n, table=i32([far]))
    check_tree(c, *attend_tree(ig, c))
    ig.ig_check()


@pytest.mark.parametrize("n,hi", [(5, 3000), (64, 9000)])
def test_tree_on_another_stream_and_replayed(ig, n, hi):
    c = make_tree(16, "f16", [hi, 33], [n, 9], 16, 2, 128, 32)
    want, wlse = attend_tree(ig, c)
    out, lse = torch.full_like(want, 77), torch.full_like(wlse, 77)
    ws = torch.empty(ig.ig_paged_tree_attend_workspace_bytes(2, c["T_max"], 16, 2, 128), dtype=torch.uint8, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    attend_tree(ig, c, out, lse, ws, s)
    s.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, wlse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        attend_tree(ig, c, out, lse, ws)
        attend_tree(ig, c, out, lse, ws)
    for length in (hi, 700, hi - 1):
        c["L"][0] = length
        c["lengths"][0] = length
        out.fill_(77)
        lse.fill_(77)
        g.replay()
        torch.cuda.synchronize()
        check_tree(c, out, lse)
        again = attend_tree(ig, c)
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    ig.ig_check()


def test_tree_two_calls_at_once(ig):
    cases = [make_tree(17, "f16", [4000, 50], [9, 9], 8, 2, 128, 16), make_tree(18, "bf16", [900] * 9, [64] * 9, 16, 4, 64, 32)]
    want = [attend_tree(ig, c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    ws = [torch.empty(ig.ig_paged_tree_attend_workspace_bytes(c["B"], c["T_max"], c["Hq"], c["Hkv"], c["d"]), dtype=torch.uint8,
                      device=DEV) for c in cases]
    got = [[(torch.full_like(o, 77), torch.full_like(x, 77)) for _ in range(5)] for o, x in want]
    torch.cuda.synchronize()
    for i in range(5):
        for c, s, w, o in zip(cases, streams, ws, got):
            attend_tree(ig, c, *o[i], w, s)
    torch.cuda.synchronize()
    for (o, x), runs in zip(want, got):
        for a, b in runs:
            assert torch.equal(a, o) and torch.equal(b, x)


def test_tree_of_a_chain_is_causal_attention(ig):
    """A chain's last token has what the attention of one token gives; drafting twice what one draft of both gives."""
    c = make_tree(19, "f16", [777], [40], 8, 2, 128, 16, masks=[(2 << i) - 1 for i in range(40)])
    out, lse = attend_tree(ig, c)
    one = torch.empty(1, 8, 128, dtype=torch.float32, device=DEV)
    ws = torch.empty(ig.ig_paged_attend_workspace_bytes(1, 8, 2, 128), dtype=torch.uint8, device=DEV)
    l1 = torch.empty(1, 8, dtype=torch.float32, device=DEV)
    ig.ig_paged_attend(None, ig.IG_F16, 1, 8, 2, 128, 16, c["n"], c["mp"], c["scale"], c["q"][39:], c["K"], c["V"], c["table"], c["L"],
                       one, l1, ws, ws.numel())
    A = float((c["q"][39].float().abs().sum(-1).max() * 6))  # (a loose bound of the logits' sums)
    assert torch.all((lse[39] - l1[0]).abs() <= 2 * (128 + 8) * U * A)
    assert torch.all((out[39].float() - one[0]).abs() <= 2 * 2.0 ** -11 * (one[0].abs() + 6))


# ---------------------------------------------------------------------------------------
# kept rows
# ---------------------------------------------------------------------------------------
@pytest.mark.parametrize("layers,Hkv,page,d,n,B", [(1, 1, 8, 64, 1, 1), (3, 2, 16, 128, 64, 5), (2, 5, 24, 64, 33, 9),
                                                   (128, 1, 8, 8, 9, 3), (4, 40, 32, 128, 16, 4), (2, 3, 8, 24, 64, 2)])
def test_kept_rows(ig, layers, Hkv, page, d, n, B):
    rng = np.random.default_rng(n + B)
    drafted = [n if b == 0 else int(rng.integers(0, n + 1)) for b in range(B)]
    L = [int(rng.integers(0, 70)) + x for x in drafted]
    seq = rng.permutation(B + 2)[:B].tolist()
    lengths = [0] * (B + 2)
    for s, x in zip(seq, L):
        lengths[s] = x
    table, pages, mp = layout(rng, lengths, page)
    K = torch.randint(0, 2 ** 15, (layers, pages, Hkv, page, d), dtype=torch.int16, device=DEV)
    V = torch.randint(0, 2 ** 15, (layers, pages, Hkv, page, d), dtype=torch.int16, device=DEV)
    paths = [sorted(rng.choice(x, int(rng.integers(0, x + 1)), replace=False).tolist()) if x else [] for x in drafted]
    paths[0] = list(range(n // 2, n)) if n > 1 else [0]
    first = np.concatenate([[0], np.cumsum(drafted)]).tolist()
    flat = [v for p, x in zip(paths, drafted) for v in p + [10 ** 6] * (x - len(p))]
    wk, wv = K.clone(), V.clone()
    for b, p in enumerate(paths):
        base = L[b] - drafted[b]
        for old, new in ((K, wk), (V, wv)):
            for i, j in enumerate(p):
                a, t = base + j, base + i
                new[:, table[seq[b]][t // page], :, t % page] = old[:, table[seq[b]][a // page], :, a % page]
    ig.ig_tree_keep(None, layers, pages, Hkv, page, d, list(K), list(V), B, B + 2, mp, max(1, len(flat)), i32(table), i32(lengths),
                    i32(seq), i32(first), i32(flat or [0]), i32([len(p) for p in paths]))
    ig.ig_check()
    assert torch.equal(K, wk) and torch.equal(V, wv)


@pytest.mark.parametrize("bad", ["path", "order", "twice", "low", "kept", "kept_low", "length", "long", "seq", "page", "first", "many"])
def test_kept_rows_of_bad_requests_stay_and_it_is_said(ig, bad):
    """Request 1 of three cannot be: none of its rows move, the others' do."""
    page, L, seq, first = 8, [12, 14, 9], [0, 1, 2], [0, 5, 10, 14]
    table = [[0, 1], [2, 3], [4, 5]]
    path, kept = [1, 3, 4, 0, 0, 2, 3, 4, 0, 0, 1, 2, 0, 0], [3, 3, 2]
    if bad == "path":
        path[7] = 5
    elif bad == "order":
        path[6], path[7] = 4, 3
    elif bad == "twice":
        path[7] = 3
    elif bad == "low":
        path[5] = -1
    elif bad == "kept":
        kept[1] = 6
    elif bad == "kept_low":
        kept[1] = -1
    elif bad == "length":
        L[1] = 4
    elif bad == "long":
        L[1] = 17
    elif bad == "seq":
        seq[1] = 3
    elif bad == "page":
        table[1][1] = 6
    elif bad == "first":
        first[1], first[2] = 10, 5
        first = [0, 5, 4, 8]  # request 1 has -1 tokens
        path = [1, 3, 4, 0, 1, 2, 0, 0, 0, 0, 0, 0, 0, 0]
    else:
        first = [0, 5, 75, 79]
        path = [1, 3, 4, 0, 0] + list(range(70)) + [1, 2, 0, 0]
        L[1], table[1] = 16, [2, 3]
    K = torch.randint(0, 2 ** 15, (2, 6, 2, page, 64), dtype=torch.int16, device=DEV)
    V = K.flip(0).contiguous()
    wk, wv = K.clone(), V.clone()
    for b, n in ((0, 5), (2, 4)):
        base = L[b] - n
        p = path[first[b]:first[b] + kept[b]]
        for old, new in ((K, wk), (V, wv)):
            for i, j in enumerate(p):
                a, t = base + j, base + i
                new[:, table[b][t // page], :, t % page] = old[:, table[b][a // page], :, a % page]
    ig.ig_tree_keep(None, 2, 6, 2, page, 64, list(K), list(V), 3, 3, 2, len(path), i32(table), i32(L), i32(seq), i32(first), i32(path),
                    i32(kept))
    refused_on_device(ig)
    assert torch.equal(K, wk) and torch.equal(V, wv)


def test_kept_rows_past_32_bits(ig):
    Hkv, page, d = 8, 64, 128
    n = (5 << 30) // (Hkv * page * d)
    K = torch.zeros((1, n, Hkv, page, d), dtype=torch.int16, device=DEV)
    K[0, n - 1] = torch.randint(0, 2 ** 15, (Hkv, page, d), dtype=torch.int16, device=DEV)
    want = K[0, n - 1].clone()
    want[:, 10] = want[:, 13]
    ig.ig_tree_keep(None, 1, n, Hkv, page, d, list(K), list(K), 1, 1, 1, 4, i32([[n - 1]]), i32([14]), None, i32([0, 4]),
                    i32([3, 0, 0, 0]), i32([1]))
    ig.ig_check()
    assert torch.equal(K[0, n - 1], want) and not K[0, :n - 1].any()


# ---------------------------------------------------------------------------------------
# bounds and choices
# ---------------------------------------------------------------------------------------
def unit_of(most):
    """Least power of two, from 2^-126 on, that `most` (float64) is at most 127 times of."""
    if most == 0:
        return 2.0 ** -126
    m, e = math.frexp(most)
    return 2.0 ** max(-126, e - 6 if m > 127 / 128 else e - 7)


def bounds_by_loops(K, rows):
    """Codes and unit of one page and head, K [rows.., d] in float64 on the host."""
    if rows == 0:
        lo = hi = np.zeros(K.shape[1])
    else:
        lo, hi = K[:rows].min(0), K[:rows].max(0)
    if not (np.isfinite(lo).all() and np.isfinite(hi).all()):
        return np.zeros((2, K.shape[1])), math.inf
    u = unit_of(max(np.abs(lo).max(), np.abs(hi).max()))
    return np.stack([np.floor(lo / u), np.ceil(hi / u)]), u


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page,Hkv", [(8, 3), (16, 1), (24, 2), (64, 5), (136, 2)])
def test_bounds(ig, dt, d, page, Hkv):
    g = torch.Generator(device=DEV)
    g.manual_seed(page)
    n = 40
    K = torch.randn(n, Hkv, page, d, generator=g, device=DEV) * torch.exp2(torch.randint(-14, 5, (n, 1, 1, 1), generator=g, device=DEV).float())
    K[1] = 0
    K[2, 0] = 127 / 128
    K[3, 0] = -127.0 / 128
    K[4] = 1.0
    K[5, 0, 0, 0], K[6, Hkv - 1, 1, d - 1], K[7, 0, 2, 5] = math.inf, -math.inf, math.nan
    K[8] = 2.0 ** -24 if dt == "f16" else 2.0 ** -133
    K[9] = -(2.0 ** -24 if dt == "f16" else 2.0 ** -130)
    K[10], K[11] = (65504.0, -65504.0) if dt == "f16" else (3e38, -3e38)
    K[12, :, :, 1] = (6e-8 if dt == "f16" else -1e-38)
    K = K.to(DT[dt])
    K[13, 0, page - 1] = math.nan  # behind the rows that count
    ids = torch.randperm(n, generator=torch.Generator().manual_seed(1)).tolist()[:-3]
    rows = [page if p not in (13, 14, 15, 16) else {13: page - 1, 14: 0, 15: 1, 16: 3}[p] for p in ids]
    entries = [[p, r] for p, r in zip(ids, rows)] + [[-1, 5]]
    codes = torch.full((n, Hkv, 2, d), 99, dtype=torch.int8, device=DEV)
    scales = torch.full((n, Hkv), 99.0, device=DEV)
    ig.ig_page_bounds(None, dtype_of(ig, dt), n, Hkv, page, d, K, len(entries), i32(entries), codes, scales)
    ig.ig_check()
    host, codes, scales = K.double().cpu().numpy(), codes.cpu().numpy(), scales.cpu().numpy()
    for p in range(n):
        for h in range(Hkv):
            if p not in ids:
                assert (codes[p, h] == 99).all() and scales[p, h] == 99
                continue
            c, u = bounds_by_loops(host[p, h], rows[ids.index(p)])
            assert scales[p, h] == u, (p, h, scales[p, h], u)
            assert (codes[p, h] == c).all(), (p, h)


def test_bounds_skip_bad_entries_and_say_so(ig):
    K = torch.ones((4, 2, 8, 64), dtype=torch.float16, device=DEV)
    for entry in ([4, 8], [1, 9], [1, -1]):
        codes = torch.full((4, 2, 2, 64), 99, dtype=torch.int8, device=DEV)
        scales = torch.full((4, 2), 99.0, device=DEV)
        ig.ig_page_bounds(None, 0, 4, 2, 8, 64, K, 2, i32([entry, [2, 8]]), codes, scales)
        refused_on_device(ig)
        assert torch.all(codes[[0, 1, 3]] == 99) and torch.all(codes[2] == 64) and scales[2].tolist() == [2.0 ** -6] * 2


def make_picked(seed, dt, lengths, Hq, Hkv, d, page, coarse=False):
    rng = np.random.default_rng(seed)
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    table, n, mp = layout(rng, lengths, page, fill=-1)
    K = torch.randn(n, Hkv, page, d, generator=g, device=DEV) * 0.75 + torch.randn(n, Hkv, 1, d, generator=g, device=DEV)
    q = torch.randn(len(lengths), Hq, d, generator=g, device=DEV)
    if coarse:  # few values: many equal scores
        K, q = K.sign(), q.sign()
        K[:, :, :, 3:], q[:, :, 4:] = 1, 0
    V = torch.randn(n, Hkv, page, d, generator=g, device=DEV)
    K, V, q = (x.to(DT[dt]) for x in (K, V, q))
    rows = [[table[b][i], min(page, x - i * page)] for b, x in enumerate(lengths) for i in range(-(-x // page))] or [[-1, 0]]
    for p, r in rows:
        K[p, :, r:] = math.nan
        V[p, :, r:] = math.nan
    codes = torch.zeros((n, Hkv, 2, d), dtype=torch.int8, device=DEV)
    scales = torch.zeros((n, Hkv), device=DEV)
    return dict(dt=dt, B=len(lengths), lengths=lengths, Hq=Hq, Hkv=Hkv, d=d, page=page, n=n, mp=mp, rows=rows, q=q, K=K, V=V,
                table=i32(table), L=i32(lengths), codes=codes, scales=scales, scale=1.0 / math.sqrt(d))


def bounds_of(ig, c):
    ig.ig_page_bounds(None, dtype_of(ig, c["dt"]), c["n"], c["Hkv"], c["page"], c["d"], c["K"], len(c["rows"]), i32(c["rows"]),
                      c["codes"], c["scales"])


def select(ig, c, picks, first, last, stream=None, out=None):
    chosen, tokens = out or (torch.full((c["B"], c["Hkv"], picks), -9, dtype=torch.int32, device=DEV),
                             torch.full((c["B"], c["Hkv"]), -9, dtype=torch.int32, device=DEV))
    ig.ig_page_select(stream, dtype_of(ig, c["dt"]), c["B"], c["Hq"], c["Hkv"], c["d"], c["page"], c["n"], c["mp"], picks, first, last,
                      c["q"], c["codes"], c["scales"], c["table"], c["L"], chosen, tokens)
    return chosen, tokens


def scores_of(c, b, h):
    """Scores of a sequence's pages for one key head, from the definition in 64 bits."""
    P = -(-c["lengths"][b] // c["page"])
    at = c["table"][b, :P].long()
    G = c["Hq"] // c["Hkv"]
    lo, hi = (c["codes"][at, h, i].double().cpu().numpy() for i in (0, 1))
    best = np.full(P, -math.inf)
    for q in c["q"][b, h * G:(h + 1) * G].double().cpu().numpy():
        v = unit_of(np.abs(q).max()) if np.isfinite(q).all() else 1.0
        code = np.round(q / v) if np.isfinite(q).all() else np.zeros_like(q)
        best = np.maximum(best, np.maximum(code * lo, code * hi).sum(1) * v)
    s = c["scales"][at, h].double().cpu().numpy()
    most = float(np.finfo(np.float32).max)
    return np.where(np.isinf(s), most, np.minimum(best * np.where(np.isinf(s), 1, s), most))


def check_choice(c, chosen, tokens, picks, first, last):
    chosen, tokens, table = chosen.tolist(), tokens.tolist(), c["table"].tolist()
    for b, x in enumerate(c["lengths"]):
        P = -(-x // c["page"])
        for h in range(c["Hkv"]):
            s = scores_of(c, b, h)
            always = [p for p in range(P) if p < first or p >= P - last]
            rest = sorted((p for p in range(P) if p not in set(always)), key=lambda p: (-s[p], p))
            take = list(range(P)) if P <= picks else sorted(always + rest[:picks - len(always)])
            assert chosen[b][h] == [table[b][p] for p in take] + [-1] * (picks - len(take)), (b, h)
            assert tokens[b][h] == (x - (P - len(take)) * c["page"] if P else 0)


@pytest.mark.parametrize("coarse", [False, True])
@pytest.mark.parametrize("dt,d", [("f16", 64), ("bf16", 128)])
@pytest.mark.parametrize("lengths,Hq,Hkv,page,picks,first,last",
                         [([0, 1, 7, 8, 9, 64, 65, 300], 4, 2, 8, 8, 1, 2), ([5000], 8, 1, 8, 100, 0, 1),
                          ([40000], 3, 1, 8, 7, 1, 2), ([16384, 16385], 10, 2, 16, 512, 4, 4), ([900] * 40, 14, 2, 16, 9, 1, 1),
                          ([3000, 2999, 17], 33, 1, 24, 3, 1, 2), ([2500] * 3, 4, 4, 8, 300, 100, 200), ([700], 256, 1, 8, 20, 0, 1)])
def test_choice(ig, lengths, Hq, Hkv, page, picks, first, last, dt, d, coarse):
    c = make_picked(len(lengths) + page, dt, lengths, Hq, Hkv, d, page, coarse)
    bounds_of(ig, c)
    check_choice(c, *select(ig, c, picks, first, last), picks, first, last)
    ig.ig_check()


def test_choice_of_a_very_long_table(ig):
    """More keys than one CTA holds: pages repeat (the choice only reads their bounds)."""
    c = make_picked(3, "f16", [8 * 4000], 2, 1, 64, 8)
    bounds_of(ig, c)
    ig.ig_check()
    c["table"] = c["table"].repeat(1, 65)[:, :250001].contiguous()
    c["mp"], c["lengths"], c["L"] = 250001, [250001 * 8 - 3], i32([250001 * 8 - 3])
    check_choice(c, *select(ig, c, 1000, 1, 2), 1000, 1, 2)
    ig.ig_check()


@pytest.mark.parametrize("d,Hq", [(64, 8), (64, 512), (128, 512)])
def test_choice_with_the_most_keys_and_queries(ig, d, Hq):
    """The longest table, whose pages repeat, with few queries a key head and with as many as there can be."""
    c = make_picked(27, "f16", [8 * 2000], Hq, 2, d, 8)
    bounds_of(ig, c)
    scores = [np.tile(scores_of(c, 0, h), 132)[:262144] for h in range(2)]
    c["table"] = c["table"].repeat(1, 132)[:, :262144].contiguous()
    c["mp"], c["L"] = 262144, i32([262144 * 8 - 3])
    chosen, tokens = select(ig, c, 700, 1, 2)
    ig.ig_check()
    for h in range(2):
        rest = 1 + np.argsort(-scores[h][1:-2], kind="stable")[:697]
        take = np.sort(np.concatenate([[0], rest, [262142, 262143]]))
        assert torch.equal(chosen[0, h], c["table"][0, torch.from_numpy(take).to(DEV)]) and int(tokens[0, h]) == 700 * 8 - 3


def test_choice_with_rows_that_are_not_finite_and_large_ones(ig):
    c = make_picked(4, "bf16", [1000, 1000], 4, 2, 64, 8)
    t = c["table"].tolist()
    c["K"][t[0][40], 0, 3, 7] = math.nan
    c["K"][t[0][50], 1, 0, 0] = math.inf
    c["K"][t[1][60]] = 3e38
    c["K"][t[1][61]] = -3e38
    c["q"][1, 0, 5] = math.nan
    c["q"][1, 1] = 3e38
    bounds_of(ig, c)
    chosen, tokens = select(ig, c, 10, 1, 2)
    check_choice(c, chosen, tokens, 10, 1, 2)
    assert t[0][40] in chosen[0, 0].tolist() and t[0][50] in chosen[0, 1].tolist()
    ig.ig_check()


def test_choice_bounds_bad_lengths_and_pages_and_says_so(ig):
    c = make_picked(5, "f16", [300, 200, 100], 4, 2, 64, 8)
    bounds_of(ig, c)
    good = select(ig, c, 12, 1, 2)
    c["L"][1] = -3
    chosen, tokens = select(ig, c, 12, 1, 2)
    refused_on_device(ig)
    assert torch.all(chosen[1] == -1) and torch.all(tokens[1] == 0)
    c["L"][1] = 10 ** 6
    select(ig, c, 12, 1, 2)
    refused_on_device(ig)
    c["L"][1] = 200
    c["table"][0, 20] = c["n"]
    chosen, tokens = select(ig, c, 12, 1, 2)
    refused_on_device(ig)
    assert torch.equal(chosen[1:], good[0][1:]) and not (chosen[0] == c["n"]).any()


@pytest.mark.parametrize("lengths,max_pages", [([40, 300, 0], 38), ([90, 60], 12), ([8], 3000)])
@pytest.mark.parametrize("entry", ["first", "last"])
def test_choice_of_all_pages_looks_at_their_numbers_too(ig, lengths, max_pages, entry):
    """A sequence with no more pages than are taken, in a CTA and in a cluster: its numbers go as they are, and it is said."""
    c = make_picked(8, "f16", lengths, 4, 2, 64, 8)
    bounds_of(ig, c)
    c["table"] = torch.cat([c["table"], torch.full((c["B"], max_pages - c["mp"]), -1, dtype=torch.int32, device=DEV)], 1).contiguous()
    c["mp"] = max_pages
    good = select(ig, c, 12, 1, 2)
    ig.ig_check()
    assert good[0][0, 0].tolist() == (c["table"][0].tolist() + [-1] * 12)[:12]
    at = 0 if entry == "first" else -(-lengths[0] // 8) - 1
    for number in (c["n"], -1, -(2 ** 31), 2 ** 31 - 1):
        c["table"][0, at] = number
        chosen, tokens = select(ig, c, 12, 1, 2)
        refused_on_device(ig)
        assert torch.equal(tokens, good[1]) and torch.equal(chosen[1:], good[0][1:])
        assert torch.all(chosen[0, :, at] == number)
        chosen[0, :, at] = good[0][0, 0, at]
        assert torch.equal(chosen, good[0])
    if len(lengths) > 1:  # entries past a sequence's pages are not looked at
        c["table"][0, at] = good[0][0, 0, at]
        c["table"][0, -(-lengths[0] // 8):] = c["n"]
        assert torch.equal(select(ig, c, 12, 1, 2)[0], good[0])
        ig.ig_check()


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("lengths,Hq,Hkv,d,page,picks", [([1000, 0, 17, 300], 4, 2, 64, 16, 6), ([9000], 40, 8, 128, 32, 33),
                                                         ([2000] * 50, 6, 3, 128, 8, 40), ([700, 701], 34, 2, 64, 24, 5),
                                                         ([129] * 3, 8, 8, 128, 64, 2)])
def test_attention_over_picked_pages(ig, lengths, Hq, Hkv, d, page, picks, dt):
    from test_gpu_paged import check_attend

    c = make_picked(6, dt, lengths, Hq, Hkv, d, page)
    bounds_of(ig, c)
    chosen, tokens = select(ig, c, picks, 1, 1)
    out = torch.full((c["B"], Hq, d), math.nan, device=DEV)
    lse = torch.full((c["B"], Hq), math.nan, device=DEV)
    ws = torch.full((ig.ig_paged_attend_workspace_bytes(c["B"], Hq, Hkv, d),), 0xff, dtype=torch.uint8, device=DEV)
    ig.ig_paged_attend_picked(None, dtype_of(ig, dt), c["B"], Hq, Hkv, d, page, c["n"], picks, c["scale"], c["q"], c["K"], c["V"], chosen,
                              tokens, out, lse, ws, ws.numel())
    ig.ig_check()
    G = Hq // Hkv
    for h in range(Hkv):  # a key head at a time, as a cache with one key head
        one = dict(Hq=G, Hkv=1, d=d, page=page, K=c["K"][:, h:h + 1], V=c["V"][:, h:h + 1], table=chosen[:, h], scale=c["scale"],
                   lengths=tokens[:, h].tolist(), q=c["q"][:, h * G:(h + 1) * G])
        check_attend(one, out[:, h * G:(h + 1) * G], lse[:, h * G:(h + 1) * G])


def test_choice_and_attention_replayed(ig):
    c = make_picked(7, "f16", [3000, 1700], 8, 2, 128, 16)
    bounds_of(ig, c)
    chosen, tokens = select(ig, c, 20, 1, 2)
    out = torch.empty(2, 8, 128, device=DEV)
    ws = torch.empty(ig.ig_paged_attend_workspace_bytes(2, 8, 2, 128), dtype=torch.uint8, device=DEV)

    def step():
        bounds_of_list()
        select(ig, c, 20, 1, 2, out=(chosen, tokens))
        ig.ig_paged_attend_picked(None, 0, 2, 8, 2, 128, 16, c["n"], 20, c["scale"], c["q"], c["K"], c["V"], chosen, tokens, out, None, ws,
                                  ws.numel())

    entries = i32(c["rows"])

    def bounds_of_list():
        ig.ig_page_bounds(None, 0, c["n"], 2, 16, 128, c["K"], len(c["rows"]), entries, c["codes"], c["scales"])

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    c["q"].copy_(torch.randn_like(c["q"]))
    g.replay()
    torch.cuda.synchronize()
    got = out.clone(), chosen.clone(), tokens.clone()
    check_choice(c, got[1], got[2], 20, 1, 2)
    step()
    assert torch.equal(out, got[0]) and torch.equal(chosen, got[1]) and torch.equal(tokens, got[2])
    ig.ig_check()


# ---------------------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------------------
def test_on_a_partition_of_the_sms(ig):
    """The same results, whatever the grid and the clusters: a tree's up to how its tiles are cut, a choice exactly."""
    c = make_tree(23, "f16", [9000, 40, 700], [16, 9, 64], 8, 2, 128, 32)
    p = make_picked(24, "bf16", [30000, 900], 8, 2, 64, 8)
    bounds_of(ig, p)
    want = select(ig, p, 50, 1, 2)
    counts, up = i32([5, 0, 7]), i32(a_tree(np.random.default_rng(25), 5) + a_tree(np.random.default_rng(26), 7))
    rows = i32(p["rows"])

    def room():  # what a call writes; nothing is made or freed while another stream is at work
        f, s, x = (torch.full((k,), -9, dtype=torch.int32, device=DEV) for k in (4, 12, 12))
        return f, s, x, torch.full((12,), -9, dtype=torch.int64, device=DEV)

    def slots(to, stream=None):
        ig.ig_page_slots(stream, 3, 3, 32, c["n"], c["mp"], 12, c["table"], c["L"], None, counts, up, *to)
        return to

    full, ws = slots(room()), torch.empty(ig.ig_paged_tree_attend_workspace_bytes(3, 64, 8, 2, 128), dtype=torch.uint8, device=DEV)
    codes, scales = p["codes"].clone(), p["scales"].clone()
    h, compute, fetch, _, _ = ig.ig_sm_split_create(0, 16)
    try:
        for stream in (compute, fetch):
            out, lse = (torch.full((c["T"], 8) + x, 77.0, dtype=t, device=DEV) for x, t in (((128,), torch.float16), ((), torch.float32)))
            got = [torch.full_like(x, -9) for x in want]
            part = room()
            p["codes"].fill_(0)
            torch.cuda.synchronize()
            attend_tree(ig, c, out, lse, ws, stream)
            ig.ig_page_bounds(stream, ig.IG_BF16, p["n"], 2, 8, 64, p["K"], len(p["rows"]), rows, p["codes"], p["scales"])
            select(ig, p, 50, 1, 2, stream, got)
            slots(part, stream)
            torch.cuda.synchronize()
            check_tree(c, out, lse)
            assert torch.equal(p["codes"], codes) and torch.equal(p["scales"], scales)
            assert all(torch.equal(x, y) for x, y in zip(got, want)) and all(torch.equal(x, y) for x, y in zip(part, full))
    finally:
        ig.ig_sm_split_destroy(h)
    ig.ig_check()


def test_buffers_on_another_gpu_than_the_current_one_are_refused(ig, monkeypatch):
    c = make_tree(30, "f16", [40], [4], 4, 2, 64, 16)
    p = make_picked(31, "f16", [90], 4, 2, 64, 16)
    path, kept = i32([0] * 4), i32([1])
    want, before = attend_tree(ig, c), c["K"].clone()
    codes = p["codes"].clone()
    torch.cuda.synchronize()
    n = ig.ig_launch_count()
    ws = torch.empty(1 << 25, dtype=torch.uint8, device=DEV)
    rows, out = i32(p["rows"]), (torch.empty(1, 2, 4, dtype=torch.int32, device=DEV), torch.empty(1, 2, dtype=torch.int32, device=DEV))
    calls = [lambda: attend_tree(ig, c, *want, ws, 0), lambda: select(ig, p, 4, 1, 2, 0, out),
             lambda: ig.ig_page_bounds(0, 0, p["n"], 2, 16, 64, p["K"], len(rows), rows, p["codes"], p["scales"]),
             lambda: ig.ig_page_slots(0, 1, 1, 16, c["n"], c["mp"], 4, c["table"], c["L"], None, kept, None, path, path, path),
             lambda: ig.ig_tree_keep(0, 1, c["n"], 2, 16, 64, [c["K"]], [c["V"]], 1, 1, c["mp"], 4, c["table"], c["L"], None, c["dfirst"],
                                     path, kept),
             lambda: ig.ig_paged_attend_picked(0, 0, 1, 4, 2, 64, 16, p["n"], 4, 0.125, p["q"], p["K"], p["V"], *out, want[1], None, ws,
                                               ws.numel())]
    with monkeypatch.context() as m:
        m.setattr(torch.cuda, "current_device", lambda: 1)  # as on a machine with two
        for call in calls:
            with pytest.raises(ValueError, match="cuda:0"):
                call()
    assert ig.ig_launch_count() == n
    torch.cuda.synchronize()
    assert torch.equal(c["K"].view(torch.int16), before.view(torch.int16)) and torch.equal(p["codes"], codes)
    ig.ig_check()


def test_cache_replays_the_choice_with_the_bounds_made_since(ig):
    from speculative_kv_cache_gb300.paged import PagedCache

    g = torch.Generator(device=DEV)
    g.manual_seed(9)
    rand = lambda *s: torch.randn(*s, generator=g, device=DEV).to(torch.float16)  # noqa: E731
    cache = PagedCache(layers=1, Hq=4, Hkv=2, d=64, n_pages=60, seqs=2, max_pages=25, page=16, bounds=True)
    slots, positions = cache.extend({0: 300, 1: 150})
    cache.write(0, rand(450, 4, 64), rand(450, 2, 64), rand(450, 2, 64), slots, positions)
    q = rand(2, 4, 64)
    out = torch.empty(2, 4, 64, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(ValueError, match="captured"):
        with torch.cuda.graph(graph):
            cache.attend_picked(0, q, 5, out=out)
    want = cache.attend_picked(0, q, 5)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.attend_picked(0, q, 5, out=out)
    graph.replay()
    assert torch.equal(out, want)
    for n in (1, 40, 17):
        slots, positions = cache.extend({0: n, 1: 2 * n})
        cache.write(0, rand(3 * n, 4, 64), rand(3 * n, 2, 64), rand(3 * n, 2, 64), slots, positions)
        q.copy_(rand(2, 4, 64))
        cache.summarise(0)
        graph.replay()
        got = out.clone()
        assert torch.equal(cache.attend_picked(0, q, 5), got)
    ig.ig_check()
    cache.close()


def test_cache_drafts_verifies_and_keeps(ig):
    """Rounds of drafting, checking and keeping, with forks and packing between: each attention is that of a sequence
    that grew token by token, and so are the rows that stay."""
    from speculative_kv_cache_gb300.paged import PagedCache

    Hq, Hkv, d, page, layers = 8, 2, 64, 16, 3
    rng = np.random.default_rng(0)
    g = torch.Generator(device=DEV)
    g.manual_seed(0)
    rand = lambda *s: torch.randn(*s, generator=g, device=DEV).to(torch.float16)  # noqa: E731
    cache = PagedCache(layers=layers, Hq=Hq, Hkv=Hkv, d=d, n_pages=120, seqs=5, max_pages=20, page=page, rot=d, bounds=True)
    kept = {s: [] for s in range(5)}  # per sequence, per token: every layer's (k, v) as projected

    def rows_of(seq, l):
        """What the pages should hold, from a dense rotation of the kept tokens at their positions."""
        n = len(kept[seq])
        k = torch.stack([x[l][0] for x in kept[seq]])
        v = torch.stack([x[l][1] for x in kept[seq]])
        q = torch.zeros(n, Hq, d, dtype=torch.float16, device=DEV)
        qo, ko, vo = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        ig.ig_qk_norm_rope(None, ig.IG_F16, n, Hq, Hkv, d, d, ig.IG_ROPE_HALF, q, Hq * d, k, Hkv * d, v, Hkv * d, None, None, 1e-6,
                           torch.arange(n, dtype=torch.int32, device=DEV), cache.turns, cache.rot_scale, qo, 0, 0, None, ko, vo)
        return ko, vo

    def check_rows():
        t, L = cache.table.tolist(), cache.L.tolist()
        assert L == [len(kept[s]) for s in range(5)]
        for s in range(5):
            for l in range(layers if kept[s] else 0):
                ko, vo = rows_of(s, l)
                at = torch.tensor([t[s][i // page] for i in range(L[s])], device=DEV)
                r = torch.arange(L[s], device=DEV) % page
                assert torch.equal(cache.K[l][at, :, r], ko) and torch.equal(cache.V[l][at, :, r], vo)

    prompt = {0: 37, 1: 3, 3: 100}
    slots, positions = cache.extend(prompt)
    T = len(slots)
    new = [(rand(T, Hkv, d), rand(T, Hkv, d)) for _ in range(layers)]
    for l in range(layers):
        cache.write(l, rand(T, Hq, d), *new[l], slots, positions)
    at = 0
    for s, n in prompt.items():
        kept[s] = [[(new[l][0][at + i], new[l][1][at + i]) for l in range(layers)] for i in range(n)]
        at += n
    check_rows()
    for round_ in range(5):
        if round_ == 1:
            cache.fork(0, 2)
            kept[2] = list(kept[0])
        if round_ == 3:
            cache.free(1)
            kept[1] = []
            assert cache.compact() > 0
        seqs = [s for s in rng.permutation(5).tolist() if kept[s] and rng.random() < 0.9] or [3]
        trees = {s: a_tree(rng, int(rng.integers(1, 20))) for s in seqs}
        draft = cache.draft(trees)
        assert draft.T == sum(map(len, trees.values()))
        new = [(rand(draft.T, Hkv, d), rand(draft.T, Hkv, d)) for _ in range(layers)]
        first, want = draft.first.tolist(), {}
        for l in range(layers):
            q = cache.write(l, rand(draft.T, Hq, d), *new[l], draft.slots, draft.positions)
            lse = torch.full((draft.T, Hq), 77.0, device=DEV)
            out = cache.attend_tree(l, q, draft, lse=lse)
            c = dict(dt="f16", Hq=Hq, Hkv=Hkv, d=d, page=page, q=q, K=cache.K[l], V=cache.V[l], table=cache.table, scale=cache.scale,
                     lengths=[len(kept[s]) + len(trees[s]) for s in trees], drafted=[len(x) for x in trees.values()], first=first,
                     seq_of=list(trees), bits=[m for x in trees.values() for m in ancestors(x)])
            check_tree(c, out, lse)
        paths = {}
        for s, tree in trees.items():
            path = []
            while rng.random() < 0.8:
                more = [i for i, p in enumerate(tree) if p == (path[-1] if path else -1)]
                if not more:
                    break
                path.append(int(rng.choice(more)))
            if path or rng.random() < 0.5:
                paths[s] = path
        if round_ == 2:  # bounds of drafted rows, which go again
            cache.summarise(0)
        cache.keep(draft, paths)
        with pytest.raises(ValueError, match="over"):
            cache.attend_tree(0, q, draft)
        for i, s in enumerate(trees):
            kept[s] = kept[s] + [[(new[l][0][first[i] + j], new[l][1][first[i] + j]) for l in range(layers)] for j in paths.get(s, [])]
        check_rows()
        # one more token each, over every page and over the picked ones
        grow = {s: 1 for s in range(5) if kept[s]}
        slots, positions = cache.extend(grow)
        new = [(rand(len(grow), Hkv, d), rand(len(grow), Hkv, d)) for _ in range(layers)]
        for i, s in enumerate(grow):
            kept[s] = kept[s] + [[(new[l][0][i], new[l][1][i]) for l in range(layers)]]
        for l in range(layers):
            cache.write(l, rand(len(grow), Hq, d), *new[l], slots, positions)
            q = rand(5, Hq, d)
            dense = cache.attend(l, q)
            all_of_it = cache.attend_picked(l, q, 1000)
            some = cache.attend_picked(l, q, 3)
            assert torch.all((dense - all_of_it).abs() <= 2.0 ** -16 * (dense.abs() + 1))
            for s in range(5):
                same = torch.equal(some[s], all_of_it[s])
                assert same or len(kept[s]) > 3 * page
            # the bounds are those of the pages as they are
            t = cache.table.tolist()
            host = cache.K[l].double().cpu().numpy()
            for s in range(5):
                for i in range(-(-len(kept[s]) // page)):
                    for h in range(Hkv):
                        codes, u = bounds_by_loops(host[t[s][i], h], min(page, len(kept[s]) - i * page))
                        assert float(cache.scales[l][t[s][i], h]) == u and (cache.codes[l][t[s][i], h].cpu().numpy() == codes).all()
        check_rows()
    ig.ig_check()
    cache.close()


def test_cache_refuses_what_cannot_be_drafted_or_kept(ig):
    from speculative_kv_cache_gb300.paged import PagedCache

    cache = PagedCache(layers=1, Hq=2, Hkv=2, d=64, n_pages=12, seqs=3, max_pages=5, page=8)
    cache.extend({0: 9})
    before = cache.L.tolist()
    for bad in ({0: [0]}, {0: [-1, 1]}, {0: [-2]}, {0: [-1] * 65}, {}, {7: [-1]}, {0: [1.5]}, {0: [-1] * 32}, {0: [-1], 1: [-1] * 41}):
        with pytest.raises((ValueError, TypeError, ig.IGError)):
            cache.draft(bad)
        assert cache.L.tolist() == before
    draft = cache.draft({0: [-1, 0, 0], 1: [-1]})
    q = torch.zeros(4, 2, 64, dtype=torch.float16, device=DEV)
    for bad in ({0: [1]}, {0: [0, 0]}, {0: [0, 3]}, {0: [0, 1, 2]}, {2: [0]}, {0: [-1]}):
        with pytest.raises(ValueError):
            cache.keep(draft, bad)
    with pytest.raises(ValueError):
        cache.attend_tree(0, q[:3], draft)
    with pytest.raises(ValueError, match="bounds"):
        cache.attend_picked(0, q[:3], 4)
    cache.fork(0, 2)
    for call in (lambda: cache.keep(draft, {}), lambda: cache.attend_tree(0, q, draft)):
        with pytest.raises(ValueError, match="over"):
            call()
    cache.close()



@pytest.mark.parametrize("limit", [0, 1, 2, 7])
@pytest.mark.parametrize("n,lengths", [(1, [100, 5]), (16, [100, 300]), (16, [20000, 40]), (64, [3000, 100]), (64, [64, 64])])
def test_tree_short_waits_are_reported_and_leave_the_next_call_right(ig, limit, n, lengths):
    """Short wait limits: the call ends by itself, its copies and products ended, ig_check names it, and the next one is right."""
    c = make_tree(20, "bf16", lengths, [n, 1], 12, 2, 128, 16)
    want = attend_tree(ig, c)
    ig.ig_check()
    ig.ig_set_wait_limit(limit)
    try:
        for fill in (0xff, 0, 1):
            size = ig.ig_paged_tree_attend_workspace_bytes(c["B"], c["T_max"], c["Hq"], c["Hkv"], c["d"])
            attend_tree(ig, c, ws=torch.full((size,), fill, dtype=torch.uint8, device=DEV))
        try:
            ig.ig_check()
            assert limit > 0  # logits may be there at the first probe
        except ig.IGError as e:
            assert e.status == ig.IG_ERR_TIMEOUT
    finally:
        ig.ig_set_wait_limit(-1)
    got = attend_tree(ig, c)
    ig.ig_check()
    check_tree(c, *got)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
