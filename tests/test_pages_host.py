"""The paged cache on the host: the page manager against a plain model, the rotary frequencies
against their formulas, and what the paged calls refuse before any device work."""
import math
import random

import numpy as np
import pytest


@pytest.fixture(scope="module")
def ig():
    from speculative_kv_cache_gb300 import build

    build.build()
    from speculative_kv_cache_gb300 import ig as mod

    return mod


class Model:
    """Token contents instead of pages: what every sequence's tokens are, and the pages' rows."""

    def __init__(self, ig, n_pages, page, seqs, max_pages):
        self.ig, self.n_pages, self.page, self.seqs, self.max_pages = ig, n_pages, page, seqs, max_pages
        self.h = ig.ig_pages_create(n_pages, page, seqs, max_pages)
        self.rows = np.full((n_pages, page), -1, dtype=np.int64)
        self.want = [[] for _ in range(seqs)]
        self.next = 0

    def run(self, moves):
        for s, d, r in moves:
            self.rows[d, :r] = self.rows[s, :r]

    def extend(self, seq, n):
        slots = np.empty(n, dtype=np.int32)
        move = self.ig.ig_pages_extend(self.h, seq, n, slots)
        self.run([] if move is None else [move])
        for s in slots.tolist():
            self.rows[s // self.page, s % self.page] = self.next
            self.want[seq].append(self.next)
            self.next += 1

    def check(self):
        t = np.empty((self.seqs, self.max_pages), dtype=np.int32)
        n = np.empty(self.seqs, dtype=np.int32)
        self.ig.ig_pages_table(self.h, t, n)
        used = set()
        for s in range(self.seqs):
            assert n[s] == len(self.want[s])
            k = -(-int(n[s]) // self.page)
            assert np.all(t[s, k:] == -1) and np.all((t[s, :k] >= 0) & (t[s, :k] < self.n_pages))
            got = [self.rows[t[s, i // self.page], i % self.page] for i in range(n[s])]
            assert got == self.want[s]
            used.update(t[s, :k].tolist())
        assert self.ig.ig_pages_free_count(self.h) == self.n_pages - len(used)
        return used


@pytest.mark.parametrize("seed", range(6))
def test_page_manager_keeps_every_sequences_tokens(ig, seed):
    g = random.Random(seed)
    page = g.choice([8, 16, 24])
    m = Model(ig, g.choice([6, 20, 40]), page, 5, 7)
    refused = 0
    try:
        for _ in range(400):
            op, s, o = g.choice("eeeeftc"), g.randrange(5), g.randrange(5)
            if op == "e":
                n = g.choice([0, 1, 1, 3, page, 2 * page + 1])
                try:
                    m.extend(s, n)
                except ig.IGError as e:
                    assert e.status == ig.IG_ERR_CAPACITY
                    refused += 1
            elif op == "f" and s != o and not m.want[o]:
                ig.ig_pages_fork(m.h, s, o)
                m.want[o] = list(m.want[s])
            elif op == "t":
                n = g.choice([0, g.randint(0, len(m.want[s]))])
                ig.ig_pages_truncate(m.h, s, n)
                del m.want[s][n:]
            elif op == "c":
                moves = np.empty((m.n_pages // 2, 3), dtype=np.int32)
                n = ig.ig_pages_compact(m.h, moves, len(moves))
                src, dst = moves[:n, 0].tolist(), moves[:n, 1].tolist()
                assert len(set(dst)) == n and not set(dst) & set(src)
                m.run(moves[:n].tolist())
                used = m.check()
                assert used == set(range(len(used)))
            m.check()
        assert refused or m.n_pages == 40
    finally:
        ig.ig_pages_destroy(m.h)


def test_page_manager_refuses_and_changes_nothing(ig):
    m = Model(ig, 3, 8, 2, 2)
    try:
        m.extend(0, 10)
        for bad in [lambda: ig.ig_pages_extend(m.h, 0, 7), lambda: ig.ig_pages_extend(m.h, 1, 9),
                    lambda: ig.ig_pages_extend(m.h, 2, 1), lambda: ig.ig_pages_extend(m.h, 0, -1),
                    lambda: ig.ig_pages_fork(m.h, 1, 0), lambda: ig.ig_pages_fork(m.h, 0, 0),
                    lambda: ig.ig_pages_truncate(m.h, 0, 11), lambda: ig.ig_pages_truncate(m.h, 0, -1),
                    lambda: ig.ig_pages_extend(None, 0, 1)]:
            with pytest.raises(ig.IGError):
                bad()
            m.check()
        ig.ig_pages_fork(m.h, 0, 1)
        m.want[1] = list(m.want[0])
        m.extend(1, 1)  # takes the last free page for its copy
        m.extend(0, 1)  # page no longer shared
        m.check()
        assert ig.ig_pages_free_count(m.h) == 0
        ig.ig_pages_truncate(m.h, 0, 0)
        m.want[0] = []
        assert ig.ig_pages_free_count(m.h) == 1  # the first page is still the fork's
        m.check()
        with pytest.raises(ig.IGError) as e:  # page 2 would move to page 1
            ig.ig_pages_compact(m.h, None, 0)
        assert e.value.status == ig.IG_ERR_CAPACITY
        m.check()
    finally:
        ig.ig_pages_destroy(m.h)
    for args in [(0, 8, 1, 1), (1, 0, 1, 1), (1, 12, 1, 1), (1, 8, 0, 1), (1, 8, 1, 0), (1 << 28, 8, 1, 1)]:
        with pytest.raises(ig.IGError):
            ig.ig_pages_create(*args)


def _frequencies(rot, theta, kind, factor, context, p0, p1):
    if kind == 2:
        theta = theta * factor ** (rot / (rot - 2))
    f = [theta ** (-2 * j / rot) for j in range(rot // 2)]
    if kind == 1:
        return [x / factor for x in f]
    if kind == 3:
        x = lambda n: rot * math.log(context / (2 * math.pi * n)) / (2 * math.log(theta))  # noqa: E731
        lo, hi = max(math.floor(x(p0)), 0), min(math.ceil(x(p1)), rot - 1)
        r = [min(max((j - lo) / max(hi - lo, 0.001), 0), 1) for j in range(rot // 2)]
        return [a / factor * b + a * (1 - b) for a, b in zip(f, r)]
    if kind == 4:
        out = []
        for a in f:
            w = 2 * math.pi / a
            s = min(max((context / w - p0) / (p1 - p0), 0), 1)
            out.append(a * ((1 - s) / factor + s))
        return out
    return f


@pytest.mark.parametrize("rot,theta,kind,factor,context,p0,p1", [
    (128, 10000.0, 0, 1.0, 0, 0.0, 0.0), (2, 10000.0, 0, 1.0, 0, 0.0, 0.0), (64, 500000.0, 1, 4.0, 0, 0.0, 0.0),
    (16, 10000.0, 2, 8.0, 0, 0.0, 0.0), (128, 10000.0, 3, 16.0, 4096, 32.0, 1.0), (64, 1e6, 3, 1.0, 32768, 32.0, 1.0),
    (128, 500000.0, 4, 8.0, 8192, 1.0, 4.0), (32, 0.5, 0, 1.0, 0, 0.0, 0.0)])
def test_rope_turns_follow_their_formulas(ig, rot, theta, kind, factor, context, p0, p1):
    turns = np.zeros(rot // 2, dtype=np.uint64)
    scale = ig.ig_rope_turns(rot, theta, kind, factor, context, p0, p1, turns)
    for t, f in zip(turns.tolist(), _frequencies(rot, theta, kind, factor, context, p0, p1)):
        want = f / (2 * math.pi) % 1.0
        # both sides in doubles: a few roundings of pow, log and the products; and the fraction is cut to
        # a multiple of 2^-64, which takes off less than 2^-64
        assert abs(t / 2.0 ** 64 - want) <= 64 * 2.0 ** -52 * max(want, f) + 2.0 ** -64
    assert scale == pytest.approx(0.1 * math.log(factor) + 1 if kind == 3 else 1.0, rel=2 ** -23)


def test_rope_turns_refusals(ig):
    t = np.zeros(64, dtype=np.uint64)
    for args in [(0, 1e4, 0, 1, 0, 0, 0), (3, 1e4, 0, 1, 0, 0, 0), (16, 0.0, 0, 1, 0, 0, 0), (16, 1e4, 5, 1, 0, 0, 0),
                 (16, 1e4, 1, 0.5, 0, 0, 0), (2, 1e4, 2, 2, 0, 0, 0), (16, 1e4, 3, 2, 0, 32, 1), (16, 1e4, 3, 2, 4096, 1, 32),
                 (16, 1.0, 3, 2, 4096, 32, 1), (16, 1e4, 4, 2, 4096, 4, 1), (16, float("nan"), 0, 1, 0, 0, 0)]:
        with pytest.raises(ig.IGError) as e:
            ig.ig_rope_turns(*args, t)
        assert e.value.status == ig.IG_ERR_INVALID
    with pytest.raises(ig.IGError):
        ig.ig_rope_turns(16, 1e4, 0, 1, 0, 0, 0, None)


def _attend(ig, **k):
    a = dict(dtype=0, B=1, Hq=4, Hkv=2, d=64, page=16, n_pages=4, max_pages=2, scale=0.125, q=256, K=512, V=768,
             page_table=1024, L_valid=1280, out=1536, lse=None, workspace=1 << 20, nbytes=1 << 30)
    a.update(k)
    ig.ig_paged_attend(0, *a.values())


@pytest.mark.parametrize("bad", [dict(dtype=2), dict(dtype=-1), dict(B=0), dict(Hq=0), dict(Hkv=0), dict(Hq=3), dict(d=96),
                                 dict(page=12), dict(page=0), dict(page=-8), dict(n_pages=0), dict(max_pages=0),
                                 dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=2e38), dict(Hq=1 << 17), dict(q=None), dict(K=None),
                                 dict(V=None), dict(page_table=None), dict(L_valid=None), dict(out=None), dict(q=264),
                                 dict(K=520), dict(V=770), dict(out=1540), dict(page_table=1026), dict(lse=2),
                                 dict(workspace=(1 << 20) + 16), dict(n_pages=1 << 28), dict(max_pages=1 << 27),
                                 dict(B=1 << 30)])
def test_paged_attend_refusals(ig, bad):
    with pytest.raises(ig.IGError) as e:
        _attend(ig, **bad)
    assert e.value.status == ig.IG_ERR_INVALID


def test_paged_attend_workspace(ig):
    assert ig.ig_paged_attend_workspace_bytes(8, 32, 8, 128) >= 256
    assert ig.ig_paged_attend_workspace_bytes(8, 32, 5, 128) == 0
    assert ig.ig_paged_attend_workspace_bytes(0, 32, 8, 128) == 0
    assert ig.ig_paged_attend_workspace_bytes(8, 32, 8, 96) == 0
    for bad in [dict(nbytes=0), dict(workspace=None)]:
        with pytest.raises(ig.IGError) as e:
            _attend(ig, **bad)
        assert e.value.status == ig.IG_ERR_CAPACITY


def _rope(ig, **k):
    m = 1 << 20
    a = dict(dtype=0, T=4, Hq=4, Hkv=2, d=64, rot=64, layout=0, q=m, q_stride=512, k=m + 512, k_stride=512, v=m + 768,
             v_stride=512, q_weight=None, k_weight=None, eps=1e-6, positions=16, turns=32, rot_scale=1.0, q_out=2 * m,
             page=16, n_pages=4, slot=48, k_out=3 * m, v_out=4 * m)
    a.update(k)
    ig.ig_qk_norm_rope(0, *a.values())


@pytest.mark.parametrize("bad", [dict(dtype=7), dict(T=-1), dict(Hq=0), dict(Hkv=0), dict(d=80), dict(rot=8), dict(rot=80),
                                 dict(rot=-16), dict(layout=2), dict(q=None), dict(k=None), dict(v=None), dict(q_out=None),
                                 dict(k_out=None), dict(v_out=None), dict(positions=None), dict(turns=None), dict(page=12),
                                 dict(page=-16), dict(n_pages=0), dict(slot=None), dict(page=0), dict(q_stride=255),
                                 dict(q_stride=248), dict(k_stride=120), dict(v_stride=516), dict(q=(1 << 20) + 8),
                                 dict(k_out=(3 << 20) + 2), dict(q_weight=8, eps=-1.0), dict(q_weight=16, eps=-1.0),
                                 dict(rot_scale=float("inf")), dict(q_out=1 << 20), dict(q_out=(1 << 20) + 16),
                                 dict(k_out=1 << 20), dict(v_out=3 << 20), dict(q_out=3 << 20), dict(turns=24),
                                 dict(positions=18), dict(n_pages=1 << 28), dict(T=1 << 30)])
def test_qk_norm_rope_refusals(ig, bad):
    with pytest.raises(ig.IGError) as e:
        _rope(ig, **bad)
    assert e.value.status == ig.IG_ERR_INVALID


def test_no_tokens_and_no_moves_do_nothing(ig):
    n = ig.ig_launch_count()
    _rope(ig, T=0)
    ig.ig_page_copy(0, 1, 4, 2, 16, 64, [1 << 20], [2 << 20], 0, None)
    assert ig.ig_launch_count() == n


@pytest.mark.parametrize("bad", [dict(layers=0), dict(layers=129), dict(n_pages=0), dict(Hkv=0), dict(page=12), dict(page=0),
                                 dict(d=60), dict(d=0), dict(n=-1), dict(K=0), dict(V=8), dict(moves=None), dict(moves=2),
                                 dict(n_pages=1 << 28), dict(n_pages=1, page=1 << 23, d=512)])
def test_page_copy_refusals(ig, bad):
    a = dict(layers=2, n_pages=4, Hkv=2, page=16, d=64, K=1 << 20, V=2 << 20, n=1, moves=4)
    a.update(bad)
    a["K"], a["V"] = [1 << 20] * (a["layers"] - 1) + [a["K"]], [2 << 20] * (a["layers"] - 1) + [a["V"]]
    if a["layers"] == 0:
        a["K"], a["V"] = [], []
    with pytest.raises(ig.IGError) as e:
        ig.ig_page_copy(0, *a.values())
    assert e.value.status == ig.IG_ERR_INVALID


def test_strided_rows_are_checked(ig):
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 512, dtype=torch.float16)
    assert ig._rows(x[:, 64:128], 512) == x.data_ptr() + 128
    assert ig._rows(x.view(4, 8, 64)[:, 2:4], 512) == x.data_ptr() + 256
    for bad, stride in [(x[:, 64:128], 64), (x.t(), 4), (x[:, ::2], 512), (x.view(4, 8, 64)[:, ::2], 512)]:
        with pytest.raises(ValueError):
            ig._rows(bad, stride)


class HostCache:
    """A PagedCache on CPU tensors, its page copies by a plain loop, and the tokens its rows should hold."""

    def __init__(self, ig, monkeypatch, **k):
        torch = pytest.importorskip("torch")
        from speculative_kv_cache_gb300.paged import PagedCache

        def page_copy(stream, layers, n_pages, Hkv, page, d, K, V, n, moves):
            if self.fail:
                raise RuntimeError("no memory")
            for a, b, r in moves.tolist():
                for x in K + V:
                    x[b, :, :r] = x[a, :, :r].clone()

        self.fail = False
        monkeypatch.setattr(ig, "ig_page_copy", page_copy)
        monkeypatch.setattr(torch.cuda, "set_device", lambda d: None)
        monkeypatch.setattr(torch.cuda, "current_device", lambda: None)  # a CPU device's index
        a = dict(layers=2, Hq=2, Hkv=2, d=64, n_pages=12, seqs=4, max_pages=5, page=8, device="cpu")
        a.update(k)
        self.cache = PagedCache(**a)
        for x in self.cache.K + self.cache.V:
            x.fill_(-1)
        self.want, self.next = [[] for _ in range(self.cache.seqs)], 1

    def put(self, new):
        slots, positions = self.cache.extend(new)
        at = 0
        for seq, n in new.items():
            for _ in range(n):
                s, c = int(slots[at]), self.cache
                assert int(positions[at]) == len(self.want[seq])
                for x in c.K + c.V:
                    x[s // c.page, :, s % c.page] = self.next
                self.want[seq].append(self.next)
                self.next += 1
                at += 1
        assert at == len(slots) == len(positions)

    def check(self):
        """Device tables, manager and rows agree."""
        c = self.cache
        t, n = np.empty((c.seqs, c.max_pages), np.int32), np.empty(c.seqs, np.int32)
        import speculative_kv_cache_gb300.ig as ig

        ig.ig_pages_table(c.pages, t, n)
        assert np.array_equal(c.table.numpy(), t) and np.array_equal(c.L.numpy(), n)
        assert n.tolist() == [len(w) for w in self.want]
        assert c.free_pages() == c.n_pages - len(set(t[t >= 0].tolist()))
        for s, w in enumerate(self.want):
            for x in c.K + c.V:
                rows = [x[t[s, i // c.page], :, i % c.page] for i in range(len(w))]
                assert all(bool((r == v).all()) for r, v in zip(rows, w)), (s, w)


@pytest.mark.parametrize("bad", [{0: 1, 7: 1}, {0: 1, -1: 1}, {0: 1, 2: -1}, {0: 1, 2: 1.5}, {0: 1, 2: None}, {0: 1, "2": 1},
                                 {0: 1, 1: 1, 2: 10 ** 12}, {0: 1, 2: 41}, {0: 1, 2: 40, 3: 40}])
def test_cache_refuses_an_extension_and_keeps_every_sequence(ig, monkeypatch, bad):
    h = HostCache(ig, monkeypatch)
    h.put({0: 13})
    h.cache.fork(0, 1)
    h.want[1] = list(h.want[0])
    h.check()
    with pytest.raises((ValueError, TypeError, ig.IGError)) as e:
        h.cache.extend(bad)
    assert not isinstance(e.value, ig.IGError) or e.value.status == ig.IG_ERR_CAPACITY
    h.check()
    h.put({0: 1, 1: 4, 3: 9})
    h.check()
    h.cache.compact()
    h.check()


def test_cache_finishes_later_what_the_device_could_not_do(ig, monkeypatch):
    """Page moves that fail leave the sequences as they were, and run before anything else changes."""
    h = HostCache(ig, monkeypatch)
    h.put({0: 13, 2: 20})
    h.cache.fork(0, 1)
    h.want[1] = list(h.want[0])
    h.fail = True
    with pytest.raises(RuntimeError, match="no memory"):
        h.cache.extend({0: 2, 2: 1})
    for change in [lambda: h.cache.extend({1: 1}), lambda: h.cache.fork(0, 3), lambda: h.cache.free(2), h.cache.compact]:
        with pytest.raises(RuntimeError, match="no memory"):
            change()
    h.fail = False
    h.cache.truncate(2, 3)
    h.want[2] = h.want[2][:3]
    h.check()
    h.put({0: 1, 1: 1, 2: 9})
    h.check()
    h.cache.free(1)
    h.want[1] = []
    h.fail = True
    with pytest.raises(RuntimeError, match="no memory"):
        h.cache.compact()
    h.fail = False
    h.put({0: 1, 3: 2})
    h.check()


def test_buffers_on_the_cpu_are_refused(ig):
    """Where a call takes device buffers, a host tensor or array in any place is refused by the binding."""
    torch = pytest.importorskip("torch")
    host = torch.zeros(4096, dtype=torch.int64)
    n = ig.ig_launch_count()
    for bad in (host, host.numpy()):
        for name in ("q", "K", "V", "page_table", "L_valid", "out", "lse", "workspace"):
            with pytest.raises(ValueError, match="CPU"):
                _attend(ig, **{name: bad})
        for name in ("q", "k", "v", "q_weight", "k_weight", "positions", "turns", "q_out", "slot", "k_out", "v_out"):
            with pytest.raises(ValueError, match="CPU"):
                _rope(ig, **{name: bad})
        for K, V, moves in [([bad], [1 << 20], 4), ([1 << 20], [bad], 4), ([1 << 20], [1 << 20], bad), ([bad], [bad], 4)]:
            with pytest.raises(ValueError, match="CPU"):
                ig.ig_page_copy(0, 1, 4, 2, 16, 64, K, V, 1, moves)
    with pytest.raises(ValueError, match="CPU"):
        _rope(ig, q=host.view(64, 64)[:, :32], q_stride=64)
    assert ig.ig_launch_count() == n


def test_cache_works_on_its_own_gpu(ig, monkeypatch):
    """With another GPU as the current one (a stand-in), every call that does device work switches to the
    cache's, and back."""
    torch = pytest.importorskip("torch")
    h = HostCache(ig, monkeypatch)
    current, at = [1], []

    class On:
        def __init__(self, d):
            self.to = d.index

        def __enter__(self):
            self.was, current[0] = current[0], self.to

        def __exit__(self, *e):
            current[0] = self.was

    copies = ig.ig_page_copy
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "device", On)
    monkeypatch.setattr(ig, "ig_page_copy", lambda *a: (at.append(current[0]), copies(*a)))
    monkeypatch.setattr(ig, "ig_pages_table", lambda *a, f=ig.ig_pages_table: (at.append(current[0]), f(*a)))
    monkeypatch.setattr(ig, "ig_qk_norm_rope", lambda *a: at.append(current[0]))
    monkeypatch.setattr(ig, "ig_paged_attend", lambda *a: at.append(current[0]))
    c, z = h.cache, lambda *s: torch.zeros(*s, dtype=torch.float16)  # noqa: E731
    h.put({0: 13})
    c.fork(0, 1)
    h.want[1] = list(h.want[0])
    h.put({0: 1})
    c.write(0, z(2, 2, 64), z(2, 2, 64), z(2, 2, 64), *[torch.zeros(2, dtype=torch.int32)] * 2)
    c.attend(0, z(4, 2, 64))
    c.free(1)
    h.want[1] = []
    c.compact()
    assert len(at) >= 9 and set(at) == {None} and current == [1]
    h.check()


@pytest.mark.parametrize("args", [(64, 5e-324, 0, 1.0, 0, 0.0, 0.0), (64, 1e-320, 1, 4.0, 0, 0.0, 0.0),
                                  (4, 1e300, 2, 1e200, 0, 0.0, 0.0)])
def test_rope_turns_refuse_what_overflows(ig, args):
    turns = np.zeros(args[0] // 2, dtype=np.uint64)
    with pytest.raises(ig.IGError) as e:
        ig.ig_rope_turns(*args, turns)
    assert e.value.status == ig.IG_ERR_INVALID and not turns.any()
    ig.ig_rope_turns(64, 1e-300, 0, 1.0, 0, 0.0, 0.0, np.zeros(32, dtype=np.uint64))
