"""The paged-cache kernels against plain implementations in 64 bits.

Tolerances.  u = 2^-23 bounds one fp32 operation, truncation included.
* attention: a logit is a sum of d exact products, scaled: off by at most (d + 4) u A_t, with
  A_t = |scale| sum_i |q_i K_ti|.  Its difference from the running maximum, the exponential, and the
  weights' split into 16-bit parts add 2^-20 + u (A_t + max A) to the weight's relative error, so
  every weight is within e = exp(2 (d + 8) u max A + 2^-20) - 1, and so is their sum.  The sums over
  L tokens, in any order, are off by at most (L + 64) u sum_t w_t |v_t|.  Together
  |o - o64| <= (2 e + (L + 64) u) sum_t w_t |v_t|;  lse: (d + 8) u max A + 2 e + (L + 64) u + 8 u |lse|.
  As the roundings are not all of one sign, the error over a whole output is far smaller: its 2-norm
  is held to 1e-5 + 2 (d + 8) u max A of the output's where that is below 1e-2.
* norm and rotation: the sum of squares, root, quotient and products are off by (d + 12) u relative;
  an angle by 2^-24 of a turn's half (pi 2^-24) and sine and cosine by two units: 2^-21 in all; so
  |y - y64| <= rnd(y) + rot_scale (|a| + |b|) (2^-21 + (d + 16) u) for the pair (a, b) after the norm, with
  rnd(y) half a step of the type at |y| (bf16 2^-8 |y|, fp16 2^-11 |y|, or half its least step 2^-25).
* copies: equal.
"""
import math
import os
import subprocess
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -23
DT = {"f16": torch.float16, "bf16": torch.bfloat16}
STEP = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}


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


def dtype_of(ig, dt):
    return ig.IG_F16 if dt == "f16" else ig.IG_BF16


# ---------------------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------------------
def make_attend(seed, dt, lengths, Hq, Hkv, d, page, spare=3, qs=1.25, max_pages=None, n_pages=None):
    """Pages in random order; every row past a sequence's end, and every spare page, is NaN."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    B = len(lengths)
    count = [-(-n // page) for n in lengths]
    mp = max_pages or max(1, max(count))
    need = sum(count)
    n = n_pages or need + spare
    K = torch.full((n, Hkv, page, d), float("nan"), dtype=DT[dt], device=DEV)
    V = torch.full((n, Hkv, page, d), float("nan"), dtype=DT[dt], device=DEV)
    perm = torch.randperm(n, generator=g, device=DEV)[:need].tolist()
    table = torch.full((B, mp), 2 ** 31 - 1, dtype=torch.int32)
    at = 0
    for b, c in enumerate(count):
        for i in range(c):
            p = perm[at]
            at += 1
            table[b, i] = p
            live = min(page, lengths[b] - i * page)
            K[p, :, :live] = (torch.randn(Hkv, live, d, generator=g, device=DEV) * 1.25).to(DT[dt])
            V[p, :, :live] = torch.randn(Hkv, live, d, generator=g, device=DEV).to(DT[dt])
    q = (torch.randn(B, Hq, d, generator=g, device=DEV) * qs).to(DT[dt])
    return dict(dt=dt, B=B, Hq=Hq, Hkv=Hkv, d=d, page=page, n=n, mp=mp, q=q, K=K, V=V, table=table.to(DEV), L=i32(lengths),
                lengths=list(lengths), scale=1.0 / math.sqrt(d))


def attend(ig, c, out=None, lse=None, ws=None, stream=None):
    out = torch.full((c["B"], c["Hq"], c["d"]), float("nan"), dtype=torch.float32, device=DEV) if out is None else out
    lse = torch.full((c["B"], c["Hq"]), float("nan"), dtype=torch.float32, device=DEV) if lse is None else lse
    if ws is None:  # arbitrary content
        ws = torch.full((ig.ig_paged_attend_workspace_bytes(c["B"], c["Hq"], c["Hkv"], c["d"]),), 0xff, dtype=torch.uint8,
                        device=DEV)
    ig.ig_paged_attend(stream, dtype_of(ig, c["dt"]), c["B"], c["Hq"], c["Hkv"], c["d"], c["page"], c["n"], c["mp"],
                       c["scale"], c["q"], c["K"], c["V"], c["table"], c["L"], out, lse, ws, ws.numel())
    return out, lse


def check_attend(c, out, lse, drop=()):
    """Against the definition; drop: (sequence, table entry) whose tokens are left out."""
    group, d, page = c["Hq"] // c["Hkv"], c["d"], c["page"]
    table = c["table"].tolist()
    K, V = c["K"], c["V"]
    err = norm = 0.0
    worst = 0.0
    for b, n in enumerate(c["lengths"]):
        keep = [t for t in range(n) if (b, t // page) not in drop]
        if not keep:
            assert torch.all(out[b] == 0) and torch.all(lse[b] == -math.inf)
            continue
        p = torch.tensor([table[b][t // page] for t in keep], device=DEV)
        r = torch.tensor([t % page for t in keep], device=DEV)
        k, v = K[p, :, r].double(), V[p, :, r].double()  # [L, Hkv, d]
        q = c["q"][b].double().view(c["Hkv"], group, d)
        z = torch.einsum("hgd,thd->hgt", q, k) * c["scale"]
        A = (torch.einsum("hgd,thd->hgt", q.abs(), k.abs()) * abs(c["scale"])).amax(-1)
        w = torch.softmax(z, -1)
        o = torch.einsum("hgt,thd->hgd", w, v)
        wv = torch.einsum("hgt,thd->hgd", w, v.abs())
        e = torch.exp(2 * (d + 8) * U * A + 2.0 ** -20) - 1
        add = (len(keep) + 64) * U
        tol = (2 * e + add)[..., None] * wv
        diff = (out[b].double().view(o.shape) - o).abs()
        assert torch.all(diff <= tol), (b, float((diff / tol).max()))
        ref = torch.logsumexp(z, -1)
        dl = (lse[b].double().view(ref.shape) - ref).abs()
        assert torch.all(dl <= (d + 8) * U * A + 2 * e + add + 8 * U * ref.abs())
        err += float(diff.square().sum())
        norm += float(o.square().sum())
        worst = max(worst, float(A.max()))
    bound = 1e-5 + 2 * (d + 8) * U * worst
    if norm and bound < 1e-2:
        assert math.sqrt(err / norm) <= bound, math.sqrt(err / norm)


EDGES = [0, 1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 257, 1000]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [8, 16, 24, 40, 64, 128, 256])
def test_attend_lengths_and_pages(ig, dt, d, page):
    c = make_attend(page + d, dt, EDGES, 8, 2, d, page)
    out, lse = attend(ig, c)
    ig.ig_check()
    check_attend(c, out, lse)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (7, 1), (8, 1), (9, 1), (10, 2), (16, 1), (17, 1), (32, 2), (33, 1),
                                    (48, 1), (56, 1), (64, 1), (65, 1), (130, 1), (28, 4)])
@pytest.mark.parametrize("dt,d", [("f16", 128), ("bf16", 128), ("f16", 64), ("bf16", 64)])
def test_attend_head_layouts(ig, Hq, Hkv, dt, d):
    c = make_attend(Hq * 7 + d, dt, [300, 0, 65, 1], Hq, Hkv, d, 16)
    out, lse = attend(ig, c)
    ig.ig_check()
    check_attend(c, out, lse)


@pytest.mark.parametrize("B,Hq,Hkv,d,page,dt,hi", [(1, 8, 2, 128, 64, "f16", 70001), (1, 1, 1, 64, 8, "bf16", 20000),
                                                   (1, 64, 1, 128, 32, "bf16", 30011), (300, 4, 2, 64, 16, "f16", 40),
                                                   (5, 6, 3, 128, 48, "f16", 9000), (1500, 1, 1, 64, 8, "bf16", 9),
                                                   (48, 32, 8, 128, 32, "bf16", 5000), (40, 16, 8, 64, 16, "f16", 7000)])
def test_attend_splits_over_length_and_batch(ig, B, Hq, Hkv, d, page, dt, hi):
    lengths = [hi if b == B // 2 else (b * 7919) % (hi + 1) for b in range(B)]
    c = make_attend(B + hi, dt, lengths, Hq, Hkv, d, page)
    out, lse = attend(ig, c)
    ig.ig_check()
    check_attend(c, out, lse)
    again = attend(ig, c)  # the same bits, whatever the order the work ran in
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("B,Hkv,lo,hi", [(24, 8, 700, 720), (40, 5, 1, 190), (25, 8, 500, 700), (160, 1, 640, 660),
                                         (33, 9, 900, 990)])
@pytest.mark.parametrize("group,dt", [(1, "f16"), (5, "bf16"), (20, "f16")])
def test_attend_heads_with_a_cta_each(ig, B, Hkv, lo, hi, group, dt):
    """As many heads as CTAs or fewer: not cut where they are short or near even, cut otherwise; the first
    sequences are empty."""
    lengths = [0, 0] + [lo + (b * 37) % (hi - lo + 1) for b in range(B - 2)]
    c = make_attend(B + hi, dt, lengths, Hkv * group, Hkv, 64, 32)
    out, lse = attend(ig, c)
    ig.ig_check()
    check_attend(c, out, lse)


@pytest.mark.parametrize("B,live", [(3000, {0: 5000, 1200: 4001, 2999: 3333}), (700, {699: 20000}), (129, {3: 900, 128: 7}),
                                    (33, {32: 1})])
def test_attend_few_requests_in_many_slots(ig, B, live):
    """A batch of mostly empty slots: a CTA's share may go on hundreds of sequences further."""
    c = make_attend(B, "f16", [live.get(b, 0) for b in range(B)], 2, 1, 64, 296)
    out, lse = attend(ig, c)
    ig.ig_check()
    check_attend(c, out, lse)


def test_attend_without_lse_and_with_a_negative_scale(ig):
    c = make_attend(3, "f16", [100, 33], 4, 4, 64, 16)
    c["scale"] = -0.3
    out, lse = attend(ig, c)
    ig.ig_check()
    check_attend(c, out, lse)
    ws = torch.empty(ig.ig_paged_attend_workspace_bytes(2, 4, 4, 64), dtype=torch.uint8, device=DEV)
    only = torch.empty_like(out)
    ig.ig_paged_attend(None, ig.IG_F16, 2, 4, 4, 64, 16, c["n"], c["mp"], c["scale"], c["q"], c["K"], c["V"], c["table"],
                       c["L"], only, None, ws, ws.numel())
    ig.ig_check()
    assert torch.equal(only, out)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_attend_large_logits_and_wide_weights(ig, dt):
    # logits of thousands (one token takes all) in one sequence; weights over many decades in another;
    # equal logits in the third
    c = make_attend(5, dt, [200, 500, 333], 4, 2, 128, 16)
    c["q"][0] *= 60
    c["q"][1] *= 6
    c["q"][2] = 0
    big = c["table"][0, 3].item()
    c["V"][big] *= 1000
    out, lse = attend(ig, c)
    ig.ig_check()
    check_attend(c, out, lse)


@pytest.mark.parametrize("dt,d", [("f16", 64), ("f16", 128), ("bf16", 64), ("bf16", 128)])
@pytest.mark.parametrize("group", [1, 4, 12, 20, 40])
@pytest.mark.parametrize("gap", [9, 12, 16, 20, 25, 30, 60, 80])
def test_attend_small_weights_beside_a_large_one_without_a_value(ig, dt, d, group, gap):
    """One token of each sequence lies `gap` above the others and has a value of zero, so that the output
    is the small weights'; in the second half of the sequences the others fall off by up to `gap` more
    (up to 80 in all, which keeps every weight above 2^-126 of the largest)."""
    lengths = [40, 333, 700, 40, 150, 700]
    c = make_attend(gap + group + d, dt, lengths, 2 * group, 2, d, 16)
    c["q"] *= 0.5
    c["q"][..., 0] = 8.0
    unit = math.sqrt(d) / 8.0  # of key component 0 per unit of logit
    for b, n in enumerate(lengths):
        t = torch.arange(n, device=DEV)
        p, r = c["table"][b, t // 16].long(), t % 16
        fall = unit * min(gap, 80 - gap) * (t * 7 % 32) / 32 * (b >= 3)
        c["K"][p, :, r, 0] = -fall[:, None].expand(n, 2).to(DT[dt])
        sink = [0, n - 1, n // 2][b % 3]
        p, r = p[sink], r[sink]
        c["K"][p, :, r] = 0
        c["K"][p, :, r, 0] = unit * gap
        c["V"][p, :, r] = 0
    out, lse = attend(ig, c)
    ig.ig_check()
    check_attend(c, out, lse)
    assert torch.all(out.abs().amax(-1) > 0)


@pytest.mark.parametrize("dt,d", [("f16", 64), ("f16", 128), ("bf16", 128)])
@pytest.mark.parametrize("group,lengths", [(4, [3000]), (12, [700, 3000, 65]), (20, [3000, 300]), (40, [1000])])
@pytest.mark.parametrize("gap,period", [(15, 40), (15, 600), (40, 96), (75, 50), (75, 1000)])
def test_attend_logits_that_rise_and_fall(ig, dt, d, group, lengths, gap, period):
    """Logits between 0 and -gap, up and down within a tile or over many, parts of a sequence in several
    CTAs; the upper half's values are zero, so that the lower half's weights make the output."""
    c = make_attend(gap + period + group, dt, lengths, group, 1, d, 8)
    c["q"] *= 0.25
    c["q"][..., 0] = 8.0
    for b, n in enumerate(lengths):
        t = torch.arange(n, device=DEV)
        p, r = c["table"][b, t // 8].long(), t % 8
        fall = gap * ((t + 17 * b) % period - period / 2).abs() / (period / 2)
        c["K"][p, 0, r, 0] = (-fall * math.sqrt(d) / 8.0).to(DT[dt])
        c["V"][p[fall < gap / 2], 0, r[fall < gap / 2]] = 0
    out, lse = attend(ig, c)
    ig.ig_check()
    check_attend(c, out, lse)
    assert torch.all(out.abs().amax(-1) > 0)


def test_attend_logits_of_minus_infinity(ig):
    # every key of sequence 0, and all but one of sequence 1, gives -inf
    c = make_attend(6, "f16", [40, 40], 2, 1, 64, 8)
    c["q"][:] = 1.0
    for b in range(2):
        for t in range(40):
            if (b, t) != (1, 21):
                c["K"][c["table"][b, t // 8].item(), :, t % 8] = -math.inf
    out, lse = attend(ig, c)
    ig.ig_check()
    assert torch.all(out[0] == 0) and torch.all(lse[0] == -math.inf)
    v = c["V"][c["table"][1, 21 // 8].item(), 0, 21 % 8].float()
    assert torch.equal(out[1], v.expand(2, 64))


def test_attend_leaves_out_bad_pages_and_says_so(ig):
    c = make_attend(8, "f16", [200, 70, 16], 4, 2, 128, 16)
    c["table"][0, 2], c["table"][1, 0], c["table"][2, 0] = -1, c["n"], -2 ** 31
    out, lse = attend(ig, c)
    with pytest.raises(ig.IGError) as e:
        ig.ig_check()
    assert e.value.status == ig.IG_ERR_INVALID
    ig.ig_check()
    check_attend(c, out, lse, drop={(0, 2), (1, 0), (2, 0)})


def test_attend_bounds_bad_lengths_and_says_so(ig):
    c = make_attend(9, "bf16", [64, 32, 0], 4, 2, 64, 16, max_pages=4)
    c["L"] = i32([65, 32, -7])
    out, lse = attend(ig, c)
    with pytest.raises(ig.IGError) as e:
        ig.ig_check()
    assert e.value.status == ig.IG_ERR_INVALID
    check_attend(c, out, lse)


def test_attend_offsets_past_32_bits(ig):
    # pages whose bytes and elements lie past 2^32 and 2^31 (4.5 GB each of keys and values)
    Hkv, page, d = 8, 64, 128
    n = 35000
    K = torch.zeros(n, Hkv, page, d, dtype=torch.float16, device=DEV)
    V = torch.zeros_like(K)
    assert K.numel() > 2 ** 31 and K.numel() * 2 > 2 ** 32
    c = make_attend(10, "f16", [64 * 5 - 3, 64], Hkv * 2, Hkv, d, page)
    old = c["table"].clone()
    c["table"][0, :5] = i32([n - 1, 3, n - 777, 17000, 34000])
    c["table"][1, 0] = 32769
    for b, k in [(0, 5), (1, 1)]:
        for i in range(k):
            K[c["table"][b, i]] = c["K"][old[b, i]]
            V[c["table"][b, i]] = c["V"][old[b, i]]
    c.update(K=K, V=V, n=n)
    out, lse = attend(ig, c)
    ig.ig_check()
    check_attend(c, out, lse)


def test_attend_on_another_stream_and_replayed(ig):
    c = make_attend(11, "bf16", [500, 20, 0, 77], 8, 2, 128, 16)
    want = attend(ig, c)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = attend(ig, c)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    ws = torch.empty(ig.ig_paged_attend_workspace_bytes(4, 8, 2, 128), dtype=torch.uint8, device=DEV)
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    graphs = []
    for _ in range(2):  # two graphs share the workspace, replayed in turn
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            attend(ig, c, out, lse, ws)
        graphs.append(g)
    for i, lengths in enumerate([[500, 20, 0, 77], [499, 1, 0, 64], [3, 0, 0, 0], [500, 20, 0, 77]]):
        c["L"].copy_(i32(lengths))
        c["lengths"] = lengths
        out.fill_(float("nan"))
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        check_attend(c, out, lse)
    ig.ig_check()
    assert torch.equal(out, want[0])


def test_first_calls_of_a_process_can_be_captured():
    """No call outside a graph before: every operator captured, then replayed."""
    code = """
import math, sys
sys.path.insert(0, "tests")
import torch
from speculative_kv_cache_gb300 import ig
import test_gpu_paged as t
c = t.make_attend(1, "f16", [300, 0, 17], 8, 2, 128, 16)
r = t.make_rope(ig, 2, "bf16", 5, 4, 2, 64, 64, 0, True, 8)
K, V = torch.randn(4, 2, 8, 64, device="cuda").half(), torch.randn(4, 2, 8, 64, device="cuda").half()
moves = t.i32([[0, 1, 8]])
out = torch.zeros(3, 8, 128, device="cuda")
lse = torch.zeros(3, 8, device="cuda")
ws = torch.empty(ig.ig_paged_attend_workspace_bytes(3, 8, 2, 128), dtype=torch.uint8, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    t.attend(ig, c, out, lse, ws)
    t.rope(ig, r)
    ig.ig_page_copy(None, 1, 4, 2, 8, 64, [K], [V], 1, moves)
g.replay()
torch.cuda.synchronize()
ig.ig_check()
t.check_attend(c, out, lse)
t.check_rope(r, r["q"], r["k"], r["v"], r["qo"])
assert torch.equal(K[0], K[1]) and torch.equal(V[0], V[1])
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]


def test_attend_two_calls_at_once(ig):
    cases = [make_attend(20 + i, "f16", [3000 + i, 900], 16, 4, 128, 32) for i in range(2)]
    want = [attend(ig, c) for c in cases]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(attend(ig, cases[i]))
    torch.cuda.synchronize()
    ig.ig_check()
    for i in range(2):
        for o, l in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(l, want[i][1])


def test_attend_parts_join_by_their_lse(ig):
    c = make_attend(12, "f16", [640], 4, 2, 128, 16)
    whole, lse = attend(ig, c)
    parts = []
    for lo, hi in [(0, 16), (16, 40)]:
        p = dict(c, table=c["table"][:, lo:hi].contiguous(), mp=hi - lo, L=i32([(hi - lo) * 16]))
        parts.append(attend(ig, p))
    ig.ig_check()
    w = torch.softmax(torch.stack([p[1].double() for p in parts]), 0)
    joined = sum(w[i][..., None] * parts[i][0].double() for i in range(2))
    # each part within 1e-5 of its own (2-norm), as check_attend holds
    assert float((joined - whole.double()).norm() / whole.double().norm()) <= 4e-5
    assert torch.allclose(torch.logaddexp(parts[0][1].double(), parts[1][1].double()), lse.double(), rtol=0, atol=1e-4)


def test_attend_waits_that_run_out_are_reported(ig):
    """A wait limit of 0 makes every wait for a tile give up at once: the call ends by itself, ig_check
    names the timeout, and the next call is right again."""
    c = make_attend(13, "f16", [3000, 5], 8, 2, 128, 16)
    want = attend(ig, c)
    ig.ig_check()
    ig.ig_set_wait_limit(0)
    try:
        attend(ig, c)
        with pytest.raises(ig.IGError) as e:
            ig.ig_check()
        assert e.value.status == ig.IG_ERR_TIMEOUT
    finally:
        ig.ig_set_wait_limit(-1)
    got = attend(ig, c)
    ig.ig_check()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("limit", [0, 1, 2, 7])
@pytest.mark.parametrize("Hq,lengths", [(4, [100, 5]), (20, [100, 5]), (56, [100, 5]), (20, [3000, 40]), (56, [3000, 40])])
def test_attend_short_waits_leave_the_next_call_right(ig, limit, Hq, lengths):
    """Short wait limits with a CTA's tiles fewer and more than the stages that hold them, and queries that
    pass through shared memory: the call ends by itself, its copies landed, and the next one is right."""
    c = make_attend(15, "bf16", lengths, Hq, 1, 128, 16)
    want = attend(ig, c)
    ig.ig_check()
    ig.ig_set_wait_limit(limit)
    try:
        for _ in range(3):
            attend(ig, c)
        try:
            ig.ig_check()
            assert limit > 0  # a tile may have landed at the first probe
        except ig.IGError as e:
            assert e.status == ig.IG_ERR_TIMEOUT
    finally:
        ig.ig_set_wait_limit(-1)
    got = attend(ig, c)
    ig.ig_check()
    check_attend(c, *got)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_tensors_of_another_device_are_refused(ig, monkeypatch):
    c = make_attend(14, "f16", [5], 1, 1, 64, 8)
    args = make_rope(ig, 1, "f16", 1, 1, 1, 64, 0, 0, False, 0)
    n = ig.ig_launch_count()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)  # as on a machine with two
    ws = torch.empty(1 << 25, dtype=torch.uint8, device=DEV)
    with pytest.raises(ValueError):
        attend(ig, c, ws=ws, stream=0)
    with pytest.raises(ValueError):
        rope(ig, args, stream=0)
    with pytest.raises(ValueError):
        ig.ig_page_copy(0, 1, c["n"], 1, 8, 64, [c["K"]], [c["V"]], 0, None)
    assert ig.ig_launch_count() == n


# ---------------------------------------------------------------------------------------
# norm and rotation
# ---------------------------------------------------------------------------------------
def make_rope(ig, seed, dt, T, Hq, Hkv, d, rot, layout, norm, page, theta=10000.0, top=5000, fused=True, scale=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    turns = np.zeros(max(rot // 2, 2), dtype=np.int64)
    if rot:
        ig.ig_rope_turns(rot, theta, ig.IG_ROPE_PLAIN, 1.0, 0, 0.0, 0.0, turns)
    x = (torch.randn(T, Hq + 2 * Hkv + (1 if fused else 0), d, generator=g, device=DEV) * 1.5).to(DT[dt])
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:Hq + 2 * Hkv]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    n = -(-T // page) + 2 if page else 0
    w = lambda: (1 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(DT[dt]) if norm else None  # noqa: E731
    shape = (n, Hkv, page, d) if page else (T, Hkv, d)
    return dict(dt=dt, T=T, Hq=Hq, Hkv=Hkv, d=d, rot=rot, layout=layout, page=page, n=n, q=q, k=k, v=v, wq=w(), wk=w(),
                theta=theta, pos=torch.randint(0, top, (T,), generator=g, device=DEV, dtype=torch.int32),
                turns=torch.from_numpy(turns).to(DEV) if rot else None, rscale=scale,
                slot=torch.randperm(n * page, generator=g, device=DEV, dtype=torch.int32)[:T] if page else None,
                qo=torch.full((T, Hq, d), 7.0, dtype=DT[dt], device=DEV), ko=torch.full(shape, 7.0, dtype=DT[dt], device=DEV),
                vo=torch.full(shape, 7.0, dtype=DT[dt], device=DEV))


def rope(ig, c, stream=None):
    st = lambda x: x.stride(0)  # noqa: E731
    ig.ig_qk_norm_rope(stream, dtype_of(ig, c["dt"]), c["T"], c["Hq"], c["Hkv"], c["d"], c["rot"], c["layout"], c["q"],
                       st(c["q"]), c["k"], st(c["k"]), c["v"], st(c["v"]) if c["v"] is not None else 0, c["wq"], c["wk"],
                       1e-6, c["pos"] if c["rot"] else None, c["turns"], c["rscale"], c["qo"], c["page"], c["n"],
                       c["slot"], c["ko"], c["vo"])


def rope64(c, x, w):
    """(the rows in 64 bits, the tolerance)"""
    d, rot, T = c["d"], c["rot"], c["T"]
    y = x.double()
    if w is not None:
        y = y / torch.sqrt(y.square().mean(-1, keepdim=True) + 1e-6) * w.double()
    size = y.abs()
    y, bound = y.clone(), y.abs()
    if rot:
        j = torch.arange(rot // 2, dtype=torch.float64, device=DEV)
        # whole turns taken off in integers: positions up to 2^31 leave a double's angle 2^-21 exact
        f = c["theta"] ** (-2 * j / rot) / (2 * math.pi)
        turn = c["pos"].double()[:, None] * f
        a = (turn - turn.round()) * 2 * math.pi
        cos, sin = torch.cos(a)[:, None], torch.sin(a)[:, None]
        i0 = torch.arange(rot // 2, device=DEV) * (1 if c["layout"] == 0 else 2)
        i1 = i0 + (rot // 2 if c["layout"] == 0 else 1)
        a0, a1 = y[..., i0], y[..., i1]
        s = c["rscale"]
        r0, r1 = s * (a0 * cos - a1 * sin), s * (a0 * sin + a1 * cos)
        both = abs(s) * (size[..., i0] + size[..., i1])
        y[..., i0], y[..., i1] = r0, r1
        bound[..., i0], bound[..., i1] = both, both
    least = 2.0 ** -25 if c["dt"] == "f16" else 0.0
    rnd = torch.clamp(STEP[c["dt"]] * y.abs(), min=least)
    return y, rnd * (1 + 2.0 ** -8) + bound * (2.0 ** -21 + (d + 16) * U)


def check_rope(c, q, k, v, qo):
    y, tol = rope64(c, q, c["wq"])
    assert torch.all((qo.double() - y).abs() <= tol), float(((qo.double() - y).abs() / tol).max())
    y, tol = rope64(c, k, c["wk"])
    if not c["page"]:
        assert torch.all((c["ko"].double() - y).abs() <= tol)
        if v is not None:
            assert torch.equal(c["vo"], v)
        return
    page, rows = c["page"], c["n"] * c["page"]
    flat = lambda z: z.transpose(1, 2).reshape(rows, c["Hkv"], c["d"])  # noqa: E731
    slot = c["slot"].long()
    live = (slot >= 0) & (slot < rows)
    K, V = flat(c["ko"]), flat(c["vo"])
    assert torch.all((K[slot[live]].double() - y[live]).abs() <= tol[live])
    assert torch.equal(V[slot[live]], v[live])
    rest = torch.ones(rows, dtype=torch.bool, device=DEV)
    rest[slot[live]] = False
    assert torch.all(K[rest] == 7.0) and torch.all(V[rest] == 7.0)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("d,rot", [(64, 64), (64, 16), (64, 48), (64, 32), (64, 0), (128, 128), (128, 64), (128, 16),
                                   (128, 112), (128, 0)])
@pytest.mark.parametrize("norm,page", [(True, 16), (False, 0), (False, 24), (True, 0)])
def test_norm_and_rotation(ig, dt, layout, d, rot, norm, page):
    c = make_rope(ig, d + rot, dt, 37, 6, 2, d, rot, layout, norm, page)
    rope(ig, c)
    ig.ig_check()
    check_rope(c, c["q"], c["k"], c["v"], c["qo"])


@pytest.mark.parametrize("T,Hq,Hkv,page,fused", [(1, 1, 1, 8, True), (1, 4, 4, 16, False), (2, 56, 1, 32, True),
                                                 (3, 5, 5, 0, False), (700, 3, 1, 64, True), (5000, 8, 8, 16, True),
                                                 (1, 130, 13, 16, True), (257, 64, 8, 0, True)])
def test_norm_and_rotation_sizes(ig, T, Hq, Hkv, page, fused):
    c = make_rope(ig, T, "bf16", T, Hq, Hkv, 128, 128, 0, True, page, fused=fused)
    rope(ig, c)
    ig.ig_check()
    check_rope(c, c["q"], c["k"], c["v"], c["qo"])


def test_rotation_at_far_and_negative_positions(ig):
    c = make_rope(ig, 1, "f16", 8, 4, 2, 128, 128, 0, False, 0, scale=1.25)
    c["pos"] = i32([0, 1, -1, 2 ** 20 + 1, 2 ** 31 - 1, -2 ** 31, 123456789, 999999])
    rope(ig, c)
    ig.ig_check()
    # a double holds 2^31 f to 2^-22 of a turn's radian: 2^-20 more for the reference's own angle
    y, tol = rope64(c, c["q"], None)
    tol = tol + 2.0 ** -20 * 1.25 * 2 * c["q"].double().abs().amax()
    assert torch.all((c["qo"].double() - y).abs() <= tol)
    assert torch.equal(c["qo"][0, :, :], (c["q"][0].float() * 1.25).half())  # position 0: only the factor


def test_norm_weights_each_by_itself_and_rows_of_zeros(ig):
    c = make_rope(ig, 2, "bf16", 9, 4, 2, 64, 32, 1, True, 8)
    c["wk"] = None
    c["q"][3] = 0
    rope(ig, c)
    ig.ig_check()
    check_rope(c, c["q"], c["k"], c["v"], c["qo"])
    assert torch.all(c["qo"][3] == 0)


def test_rotation_in_place_and_without_values(ig):
    c = make_rope(ig, 4, "f16", 33, 4, 2, 128, 64, 0, True, 0, fused=False)
    was = c["q"].clone()
    c.update(qo=c["q"], v=None, vo=None)
    rope(ig, c)
    ig.ig_check()
    check_rope(c, was, c["k"], None, c["qo"])


def test_slots_skipped_and_out_of_range(ig):
    c = make_rope(ig, 5, "f16", 20, 4, 2, 128, 128, 0, False, 16)
    c["slot"][3], c["slot"][7] = -1, -2 ** 31
    rope(ig, c)
    ig.ig_check()
    check_rope(c, c["q"], c["k"], c["v"], c["qo"])
    c["ko"].fill_(7.0)
    c["vo"].fill_(7.0)
    c["slot"][5], c["slot"][6] = c["n"] * 16, 2 ** 31 - 1
    rope(ig, c)
    with pytest.raises(ig.IGError) as e:
        ig.ig_check()
    assert e.value.status == ig.IG_ERR_INVALID
    check_rope(c, c["q"], c["k"], c["v"], c["qo"])


def test_rotation_keeps_non_finite_values_in_their_rows(ig):
    c = make_rope(ig, 6, "f16", 4, 2, 1, 64, 64, 0, True, 8)
    c["q"][1, 0, 5] = float("inf")
    c["k"][2, 0, 1] = float("nan")
    clean = [c["q"].clone(), c["k"].clone()]
    rope(ig, c)
    ig.ig_check()
    assert torch.all(torch.isnan(c["qo"][1, 0]) | torch.isinf(c["qo"][1, 0]) | (c["qo"][1, 0] == 0))
    y, tol = rope64(c, clean[0], c["wq"])
    ok = torch.ones(4, 2, dtype=torch.bool, device=DEV)
    ok[1, 0] = False
    assert torch.all((c["qo"].double() - y).abs()[ok] <= tol[ok])


# ---------------------------------------------------------------------------------------
# page moves
# ---------------------------------------------------------------------------------------
@pytest.mark.parametrize("layers,Hkv,page,d,pages,n", [(1, 1, 8, 64, 2, 1), (3, 2, 16, 128, 40, 17), (48, 4, 24, 64, 12, 6),
                                                       (128, 1, 8, 8, 9, 4), (2, 7, 256, 128, 30, 15), (1, 1, 8, 8, 5000, 2500)])
def test_page_copies(ig, layers, Hkv, page, d, pages, n):
    g = torch.Generator(device=DEV)
    g.manual_seed(n)
    make = lambda: [torch.randn(pages, Hkv, page, d, generator=g, device=DEV).half() for _ in range(layers)]  # noqa: E731
    K, V = make(), make()
    want = [[x.clone() for x in K], [x.clone() for x in V]]
    perm = torch.randperm(pages, generator=g, device=DEV).tolist()
    moves = [[perm[i], perm[n + i], [page, 0, 1, page - 1, 5][i % 5]] for i in range(n)]
    if n > 4:
        moves[2][0] = moves[1][0]  # one page copied to two
        moves[3][0] = -1           # skipped
        moves[4] = [perm[4], perm[4], page]  # onto itself
    for a, b, r in moves:
        if a >= 0:
            for xs in want:
                for x in xs:
                    x[b, :, :r] = x[a, :, :r]
    ig.ig_page_copy(None, layers, pages, Hkv, page, d, K, V, n, i32(moves))
    ig.ig_check()
    for xs, ys in zip(want, (K, V)):
        for x, y in zip(xs, ys):
            assert torch.equal(x, y)


def test_page_copy_skips_bad_moves_and_says_so(ig):
    K, V = [torch.randn(6, 2, 8, 64, device=DEV).half()], [torch.randn(6, 2, 8, 64, device=DEV).half()]
    want = K[0].clone()
    want[5] = want[0]
    moves = [[6, 1, 8], [0, 6, 8], [0, -1, 8], [0, 2, 9], [0, 3, -1], [2 ** 31 - 1, 4, 8], [0, 5, 8]]
    ig.ig_page_copy(None, 1, 6, 2, 8, 64, K, V, len(moves), i32(moves))
    with pytest.raises(ig.IGError) as e:
        ig.ig_check()
    assert e.value.status == ig.IG_ERR_INVALID
    assert torch.equal(K[0], want)


def test_page_copy_offsets_past_32_bits(ig):
    n = 35000
    K = torch.zeros(n, 8, 64, 128, dtype=torch.float16, device=DEV)
    V = torch.zeros_like(K)
    K[n - 1], V[3] = 1.5, 2.5
    ig.ig_page_copy(None, 1, n, 8, 64, 128, [K], [V], 2, i32([[n - 1, 40, 64], [3, n - 2, 63]]))
    ig.ig_check()
    assert torch.all(K[40] == 1.5) and torch.all(V[n - 2, :, :63] == 2.5) and torch.all(V[n - 2, :, 63] == 0)
    assert torch.all(K[41] == 0) and torch.all(V[n - 1] == 0)


# ---------------------------------------------------------------------------------------
# all of them, as a server uses them
# ---------------------------------------------------------------------------------------
@pytest.mark.parametrize("dt,d,rot,layout,page", [("f16", 64, 64, 0, 8), ("bf16", 128, 64, 1, 24)])
def test_cache_of_forked_requests(ig, dt, d, rot, layout, page):
    """Prompts, forks, steps (some replayed as a graph), cuts and packing, two layers; every step's
    attention against the tokens each request has seen, as the pages' contents are checked against
    them too."""
    from speculative_kv_cache_gb300.paged import PagedCache

    layers, Hq, Hkv, seqs, theta = 2, 4, 2, 4, 10000.0
    cache = PagedCache(layers=layers, Hq=Hq, Hkv=Hkv, d=d, n_pages=60, seqs=seqs, max_pages=24, page=page, dtype=DT[dt],
                       rot=rot, layout=layout, theta=theta)
    g = torch.Generator(device=DEV)
    g.manual_seed(9)
    w = [(1 + 0.1 * torch.randn(d, generator=g, device=DEV)).to(DT[dt]) for _ in range(2)]
    seen = [[[] for _ in range(layers)] for _ in range(seqs)]  # per request and layer: (k, v, position)
    args = dict(dt=dt, d=d, rot=rot, layout=layout, theta=theta, rscale=1.0)

    def step(new, replay=None):
        T = sum(new.values())
        slots, pos = cache.extend(new)
        owner = [s for s, n in new.items() for _ in range(n)]
        last = {}
        for i, s in enumerate(owner):
            last[s] = i
        for l in range(layers):
            x = torch.randn(T, Hq + 2 * Hkv, d, generator=g, device=DEV).to(DT[dt])
            if replay is None:
                q = cache.write(l, x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], slots, pos, w[0], w[1])
                mine = torch.zeros(seqs, Hq, d, dtype=DT[dt], device=DEV)
                for s, i in last.items():
                    mine[s] = q[i]
                out = cache.attend(l, mine)
            else:  # one token per request, in request order
                replay["x"].copy_(x)
                replay["slots"].copy_(slots)
                replay["pos"].copy_(pos)
                replay["graphs"][l].replay()
                q, out = replay["q"], replay["out"]
            for i, s in enumerate(owner):
                seen[s][l].append((x[i, Hq:Hq + Hkv], x[i, Hq + Hkv:], int(pos[i])))
            check(l, x[:, :Hq], pos, q, out, last)
        ig.ig_check()

    def check(l, x, pos, q, out, last):
        y, tol = rope64(dict(args, pos=pos, T=len(pos)), x, w[0])
        assert torch.all((q.double() - y).abs() <= tol)
        table, L = cache.table.cpu(), cache.L.cpu()
        for s in range(seqs):
            n = int(L[s])
            assert n == len(seen[s][l])
            if n == 0:
                assert torch.all(out[s] == 0)
                continue
            at = table[s, torch.arange(n) // page].to(DEV).long()
            row = (torch.arange(n) % page).to(DEV)
            K, V = cache.K[l][at, :, row], cache.V[l][at, :, row]
            k = torch.stack([t[0] for t in seen[s][l]])
            assert torch.equal(V, torch.stack([t[1] for t in seen[s][l]]))
            p = torch.tensor([t[2] for t in seen[s][l]], device=DEV)
            assert p.tolist() == list(range(n))
            y, tol = rope64(dict(args, pos=p, T=n), k, w[1])
            assert torch.all((K.double() - y).abs() <= tol)
            if s in last:
                c = dict(Hq=Hq, Hkv=Hkv, d=d, page=n, q=q[last[s]][None], K=K.transpose(0, 1)[None],
                         V=V.transpose(0, 1)[None], table=torch.zeros(1, 1, dtype=torch.int32), lengths=[n],
                         scale=cache.scale)
                kk, qq = K.double(), q[last[s]].double().view(Hkv, Hq // Hkv, d)
                z = torch.einsum("hgd,thd->hgt", qq, kk) * cache.scale
                lse = torch.logsumexp(z, -1).reshape(1, Hq)
                check_attend(c, out[s][None], lse)

    try:
        step({0: 3 * page + 5, 1: 1})        # prompts
        for s in (2, 3):                      # forks inside a page
            cache.fork(0, s)
            seen[s] = [list(x) for x in seen[0]]
        for _ in range(3):
            step({0: 1, 1: 1, 2: 1, 3: 1})    # the forks part: copies on write
        replay = dict(x=torch.empty(seqs, Hq + 2 * Hkv, d, dtype=DT[dt], device=DEV), slots=i32([0] * seqs),
                      pos=i32([0] * seqs), q=torch.empty(seqs, Hq, d, dtype=DT[dt], device=DEV),
                      out=torch.empty(seqs, Hq, d, device=DEV), graphs=[])
        for l in range(layers):
            gr = torch.cuda.CUDAGraph()
            x = replay["x"]
            with torch.cuda.graph(gr):
                cache.write(l, x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], replay["slots"], replay["pos"], w[0], w[1],
                            q_out=replay["q"])
                cache.attend(l, replay["q"], replay["out"])
            replay["graphs"].append(gr)
        for _ in range(3):
            step({0: 1, 1: 1, 2: 1, 3: 1}, replay)
        cache.truncate(0, page + 3)           # a cut inside a page it shares
        seen[0] = [x[:page + 3] for x in seen[0]]
        cache.free(1)
        seen[1] = [[] for _ in range(layers)]
        step({0: 2, 3: 1})
        used = cache.n_pages - cache.free_pages()
        cache.compact()
        assert int(cache.table.max()) == used - 1
        step({0: 1, 2: 2, 3: 1})
        before = cache.free_pages(), cache.L.tolist()
        with pytest.raises(ValueError):
            cache.attend(0, torch.zeros(seqs, Hq, d, device=DEV))  # fp32
        with pytest.raises(ValueError):
            cache.write(0, *[torch.zeros(2, n, d, dtype=DT[dt], device=DEV) for n in (Hq, Hkv, Hkv)], i32([0]), i32([0, 0]))
        with pytest.raises(ig.IGError) as e:
            cache.extend({2: 1, 1: 25 * page})
        assert e.value.status == ig.IG_ERR_CAPACITY and cache.L.tolist() == before[1]
        step({1: page, 2: 1, 0: 1, 3: 1})
    finally:
        cache.close()


@pytest.mark.parametrize("bad", [{0: 1, 7: 1}, {0: 1, 2: -1}, {0: 1, 2: 1.5}, {0: 1, 2: 200}])
def test_cache_attends_right_after_a_refused_extension(ig, bad):
    """A sequence forked inside a page, whose extension is refused together with another's."""
    from speculative_kv_cache_gb300.paged import PagedCache

    cache = PagedCache(layers=1, Hq=4, Hkv=2, d=64, n_pages=20, seqs=3, max_pages=6, page=8)
    g = torch.Generator(device=DEV)
    g.manual_seed(4)
    seen = [[], [], []]

    def step(new):
        slots, pos = cache.extend(new)
        T = len(slots)
        k, v = (torch.randn(T, 2, 64, generator=g, device=DEV).half() for _ in range(2))
        cache.write(0, torch.zeros(T, 4, 64, dtype=torch.float16, device=DEV), k, v, slots, pos)
        for i, s in enumerate(s for s, n in new.items() for _ in range(n)):
            seen[s].append((k[i], v[i]))

    try:
        step({0: 13})
        cache.fork(0, 1)
        seen[1] = list(seen[0])
        with pytest.raises((ValueError, TypeError, ig.IGError)):
            cache.extend(bad)
        assert cache.L.tolist() == [13, 13, 0]
        step({0: 1, 1: 2})
        q = torch.randn(3, 4, 64, generator=g, device=DEV).half()
        lse = torch.empty(3, 4, device=DEV)
        out = cache.attend(0, q, lse=lse)
        ig.ig_check()
        K, V = (torch.zeros(3, 2, 16, 64, dtype=torch.float16, device=DEV) for _ in range(2))
        for s in range(3):
            for t, (k, v) in enumerate(seen[s]):
                K[s, :, t], V[s, :, t] = k, v
        check_attend(dict(Hq=4, Hkv=2, d=64, page=16, q=q, K=K, V=V, table=i32([[0], [1], [2]]), scale=cache.scale,
                          lengths=[len(x) for x in seen]), out, lse)
    finally:
        cache.close()


def test_rotation_keeps_a_nan_key_in_its_row(ig):
    c = make_rope(ig, 7, "f16", 6, 4, 3, 64, 64, 0, True, 8)
    clean = [c["q"].clone(), c["k"].clone(), c["v"].clone()]
    c["k"][2, 1, 5] = float("nan")
    c["k"][4, 0, 9] = float("inf")
    rope(ig, c)
    ig.ig_check()
    y, tol = rope64(c, clean[0], c["wq"])
    assert torch.all((c["qo"].double() - y).abs() <= tol)
    y, tol = rope64(c, clean[1], c["wk"])
    at, row = c["slot"].long() // 8, c["slot"].long() % 8
    K, V = c["ko"][at, :, row], c["vo"][at, :, row]
    ok = torch.ones(6, 3, dtype=torch.bool, device=DEV)
    ok[2, 1] = ok[4, 0] = False
    assert torch.all((K.double() - y).abs()[ok] <= tol[ok])
    assert torch.all(torch.isnan(K[2, 1])) and not torch.any(torch.isfinite(K[4, 0, 9:10]))
    assert torch.equal(V, clean[2])
    rest = torch.ones(c["n"], 8, dtype=torch.bool, device=DEV)
    rest[at, row] = False
    assert torch.all(c["ko"].transpose(1, 2)[rest] == 7.0) and torch.all(c["vo"].transpose(1, 2)[rest] == 7.0)


@pytest.mark.parametrize("scaling,factor,context,p0,p1", [(1, 4.0, 0, 0.0, 0.0), (2, 8.0, 0, 0.0, 0.0),
                                                          (3, 16.0, 4096, 32.0, 1.0), (4, 8.0, 8192, 1.0, 4.0)])
def test_rotation_by_scaled_frequencies(ig, scaling, factor, context, p0, p1):
    """What ig_rope_turns gives for each rule, through the kernel, against the rule's frequencies in doubles."""
    from test_pages_host import _frequencies

    c = make_rope(ig, 8, "f16", 50, 4, 2, 128, 128, 0, False, 0, top=60000)
    turns = np.zeros(64, dtype=np.int64)
    s = ig.ig_rope_turns(128, 10000.0, scaling, factor, context, p0, p1, turns)
    c.update(turns=torch.from_numpy(turns).to(DEV), rscale=s)
    rope(ig, c)
    ig.ig_check()
    f = torch.tensor(_frequencies(128, 10000.0, scaling, factor, context, p0, p1), dtype=torch.float64, device=DEV)
    a = (c["pos"].double()[:, None] * f)[:, None]
    for x, got in ((c["q"].double(), c["qo"]), (c["k"].double(), c["ko"])):
        x0, x1 = x[..., :64], x[..., 64:]
        y = s * torch.cat([x0 * a.cos() - x1 * a.sin(), x0 * a.sin() + x1 * a.cos()], -1)
        size = (s * (x0.abs() + x1.abs())).repeat(1, 1, 2)
        # as rope64's, and the reference's angle: up to 60000 radians in doubles, 2^-36
        tol = torch.clamp(STEP["f16"] * y.abs(), min=2.0 ** -25) * (1 + 2.0 ** -8) + size * (2.0 ** -21 + 144 * U + 2.0 ** -36)
        assert torch.all((got.double() - y).abs() <= tol), float(((got.double() - y).abs() / tol).max())


def test_cache_keeps_its_free_pages_when_an_extension_does_not_fit(ig):
    from speculative_kv_cache_gb300.paged import PagedCache

    cache = PagedCache(layers=1, Hq=2, Hkv=2, d=64, n_pages=6, seqs=3, max_pages=6, page=8)
    try:
        cache.extend({0: 12, 1: 8})
        for bad in ({0: 1, 2: 25}, {1: 9, 2: 17}, {2: 49}):
            with pytest.raises(ig.IGError) as e:
                cache.extend(bad)
            assert e.value.status == ig.IG_ERR_CAPACITY
            assert cache.free_pages() == 3 and cache.L.tolist() == [12, 8, 0]
        cache.fork(0, 2)
        with pytest.raises(ig.IGError):  # a page of its own stays with the sequence that parted
            cache.extend({2: 1, 1: 25})
        assert cache.free_pages() == 2 and cache.L.tolist() == [12, 8, 12]
        t = cache.table.tolist()
        assert t[0][0] == t[2][0] and t[0][1] != t[2][1]
    finally:
        cache.close()


@pytest.mark.parametrize("dt,d", [("f16", 64), ("f16", 128), ("bf16", 64), ("bf16", 128)])
@pytest.mark.parametrize("group", [1, 12, 20, 56])
def test_attend_non_finite_rows_stay_with_their_heads(ig, dt, d, group):
    """A logit that is NaN or +inf makes its heads' results non-finite, a value that is not finite its
    component, however small the weight; the other key head and the other sequences are right."""
    c = make_attend(31 + group, dt, [100, 333, 64, 700], 2 * group, 2, d, 16)
    c["q"][..., 0] = 1.0
    at = lambda b, t: (c["table"][b, t // 16].item(), 0, t % 16)  # noqa: E731
    c["K"][at(0, 70)] = float("nan")
    c["K"][at(1, 5) + (0,)] = float("inf")
    c["V"][at(2, 63) + (3,)] = float("-inf")
    c["K"][at(2, 63) + (0,)] = -200 * math.sqrt(d)  # a weight of zero
    out, lse = attend(ig, c)
    ig.ig_check()
    first = slice(0, group)
    assert not torch.any(torch.isfinite(out[:2, first])) and not torch.any(torch.isfinite(lse[:2, first]))
    assert not torch.any(torch.isfinite(out[2, first, 3])) and torch.all(torch.isfinite(lse[2, first]))
    assert torch.all(torch.isfinite(torch.cat([out[2, first, :3], out[2, first, 4:]], -1)))
    for b, keep in ((0, [1]), (1, [1]), (2, [1]), (3, [0, 1])):
        for h in keep:
            q = slice(h * group, (h + 1) * group)
            one = dict(c, Hq=group, Hkv=1, q=c["q"][b:b + 1, q], K=c["K"][:, h:h + 1], V=c["V"][:, h:h + 1],
                       table=c["table"][b:b + 1], lengths=c["lengths"][b:b + 1])
            check_attend(one, out[b:b + 1, q], lse[b:b + 1, q])
