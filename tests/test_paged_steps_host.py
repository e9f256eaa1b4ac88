"""What the paged cache's operators for drafted trees and picked pages refuse, before any device work."""
import numpy as np
import pytest


@pytest.fixture(scope="module")
def ig():
    from speculative_kv_cache_gb300 import build

    build.build()
    from speculative_kv_cache_gb300 import ig as mod

    return mod


def _tree(ig, **k):
    a = dict(dtype=0, n=2, T=3, T_max=2, Hq=4, Hkv=2, d=64, page=16, n_pages=4, seqs=2, max_pages=2, scale=0.125, q=256, K=512, V=768,
             page_table=1024, L_valid=1280, seq=None, first=1536, masks=1792, out=2048, lse=None, workspace=1 << 20,
             nbytes=1 << 30)
    a.update(k)
    ig.ig_paged_tree_attend(0, *a.values())


def _slots(ig, **k):
    a = dict(n=2, seqs=2, page=16, n_pages=4, max_pages=2, T=3, page_table=1024, L_valid=1280, seq=None, counts=1536, parents=None,
             first=1792, slots=2048, positions=2304, masks=None)
    a.update(k)
    ig.ig_page_slots(0, *a.values())


def _keep(ig, **k):
    a = dict(layers=1, n_pages=4, Hkv=2, page=16, d=64, K=[512], V=[768], n=2, seqs=2, max_pages=2, T=3, page_table=1024, L_valid=1280,
             seq=None, first=1536, path=1792, kept=2048)
    a.update(k)
    ig.ig_tree_keep(0, *a.values())


def _bounds(ig, **k):
    a = dict(dtype=0, n_pages=4, Hkv=2, page=16, d=64, K=512, n=2, list=1024, codes=2048, scales=4096)
    a.update(k)
    ig.ig_page_bounds(0, *a.values())


def _select(ig, **k):
    a = dict(dtype=0, B=2, Hq=4, Hkv=2, d=64, page=16, n_pages=4, max_pages=2, picks=4, first=1, last=2, q=256, codes=512, scales=768,
             page_table=1024, L_valid=1280, chosen=1536, tokens=1792)
    a.update(k)
    ig.ig_page_select(0, *a.values())


def _picked(ig, **k):
    a = dict(dtype=0, B=1, Hq=4, Hkv=2, d=64, page=16, n_pages=4, picks=2, scale=0.125, q=256, K=512, V=768, chosen=1024, tokens=1280,
             out=1536, lse=None, workspace=1 << 20, nbytes=1 << 30)
    a.update(k)
    ig.ig_paged_attend_picked(0, *a.values())


_PAGES = [dict(page=12), dict(page=0), dict(page=-8), dict(n_pages=0)]
_TYPES = [dict(dtype=2), dict(dtype=-1), dict(d=96), dict(Hkv=0)]
_HEADS = [dict(Hq=0), dict(Hq=3)]


@pytest.mark.parametrize("bad", _PAGES + _TYPES + _HEADS + [
    dict(n=0), dict(n=3), dict(seqs=0), dict(T=-1), dict(T_max=0), dict(T_max=65), dict(max_pages=0), dict(scale=float("nan")),
    dict(scale=float("inf")), dict(scale=2e38), dict(Hq=1 << 17), dict(T=1 << 30), dict(n_pages=1 << 28), dict(max_pages=1 << 27),
    dict(q=None), dict(K=None), dict(V=None), dict(page_table=None), dict(L_valid=None), dict(first=None), dict(masks=None),
    dict(out=None), dict(q=264), dict(K=520), dict(V=770), dict(out=2056), dict(page_table=1026), dict(L_valid=2), dict(seq=2),
    dict(first=2), dict(masks=1796), dict(lse=2), dict(workspace=(1 << 20) + 16)])
def test_tree_attention_refusals(ig, bad):
    with pytest.raises(ig.IGError) as e:
        _tree(ig, **bad)
    assert e.value.status == ig.IG_ERR_INVALID


def test_tree_attention_workspace(ig):
    assert ig.ig_paged_tree_attend_workspace_bytes(8, 64, 32, 8, 128) >= 256
    for bad in [(0, 1, 4, 2, 64), (1, 0, 4, 2, 64), (1, 65, 4, 2, 64), (1, 1, 3, 2, 64), (1, 1, 4, 2, 96), (1, 1, 0, 2, 64)]:
        assert ig.ig_paged_tree_attend_workspace_bytes(*bad) == 0
    for bad in [dict(nbytes=0), dict(workspace=None)]:
        with pytest.raises(ig.IGError) as e:
            _tree(ig, **bad)
        assert e.value.status == ig.IG_ERR_CAPACITY


@pytest.mark.parametrize("bad", _PAGES + [
    dict(n=0), dict(n=8193, seqs=9000), dict(n=3), dict(seqs=0), dict(T=-1), dict(T=1 << 30), dict(max_pages=0), dict(max_pages=1 << 27),
    dict(n_pages=1 << 28), dict(page_table=None), dict(L_valid=None), dict(counts=None), dict(first=None), dict(slots=None),
    dict(positions=None), dict(page_table=2), dict(L_valid=2), dict(seq=2), dict(counts=2), dict(parents=2), dict(first=2),
    dict(slots=2), dict(positions=2), dict(masks=4)])
def test_slots_refusals(ig, bad):
    with pytest.raises(ig.IGError) as e:
        _slots(ig, **bad)
    assert e.value.status == ig.IG_ERR_INVALID


@pytest.mark.parametrize("bad", _PAGES + [
    dict(layers=0, K=[], V=[]), dict(layers=129, K=[512] * 129, V=[512] * 129), dict(Hkv=0), dict(d=0), dict(d=12), dict(n=-1), dict(n=3),
    dict(seqs=0), dict(max_pages=0), dict(max_pages=1 << 27), dict(T=-1), dict(n_pages=1 << 28), dict(K=[None]), dict(V=[None]),
    dict(K=[520]), dict(V=[770]), dict(page_table=None), dict(L_valid=None), dict(first=None), dict(path=None), dict(kept=None),
    dict(page_table=2), dict(L_valid=2), dict(seq=2), dict(first=2), dict(path=2), dict(kept=2)])
def test_kept_rows_refusals(ig, bad):
    with pytest.raises(ig.IGError) as e:
        _keep(ig, **bad)
    assert e.value.status == ig.IG_ERR_INVALID


@pytest.mark.parametrize("bad", _PAGES + _TYPES + [
    dict(n=-1), dict(n=1 << 30), dict(n_pages=1 << 28), dict(K=None), dict(list=None), dict(codes=None), dict(scales=None), dict(K=520),
    dict(list=2), dict(codes=2056), dict(scales=2)])
def test_bounds_refusals(ig, bad):
    with pytest.raises(ig.IGError) as e:
        _bounds(ig, **bad)
    assert e.value.status == ig.IG_ERR_INVALID


@pytest.mark.parametrize("bad", _PAGES + _TYPES + _HEADS + [
    dict(B=0), dict(Hq=514), dict(max_pages=0), dict(max_pages=262145), dict(picks=2), dict(picks=0), dict(picks=-1), dict(first=-1),
    dict(last=0), dict(first=3), dict(picks=1 << 27), dict(B=1 << 26), dict(n_pages=1 << 28), dict(first=2 ** 31 - 1), dict(q=None), dict(codes=None),
    dict(scales=None), dict(page_table=None), dict(L_valid=None), dict(chosen=None), dict(tokens=None), dict(q=264), dict(codes=520),
    dict(scales=2), dict(page_table=2), dict(L_valid=2), dict(chosen=2), dict(tokens=2)])
def test_choice_refusals(ig, bad):
    with pytest.raises(ig.IGError) as e:
        _select(ig, **bad)
    assert e.value.status == ig.IG_ERR_INVALID


@pytest.mark.parametrize("bad", _PAGES + _TYPES + _HEADS + [
    dict(B=0), dict(picks=0), dict(picks=1 << 27), dict(scale=float("nan")), dict(scale=2e38), dict(q=None), dict(K=None), dict(V=None),
    dict(chosen=None), dict(tokens=None), dict(out=None), dict(q=264), dict(K=520), dict(V=770), dict(out=1540), dict(chosen=1026),
    dict(tokens=2), dict(lse=2), dict(workspace=(1 << 20) + 16), dict(n_pages=1 << 28), dict(B=1 << 30)])
def test_picked_attention_refusals(ig, bad):
    with pytest.raises(ig.IGError) as e:
        _picked(ig, **bad)
    assert e.value.status == ig.IG_ERR_INVALID


def test_nothing_to_do_does_nothing(ig):
    n = ig.ig_launch_count()
    _tree(ig, T=0, q=None, K=None, out=None, workspace=None, nbytes=0)
    _keep(ig, n=0, path=None, kept=None)
    _bounds(ig, n=0, list=None)
    assert ig.ig_launch_count() == n


def test_buffers_on_the_cpu_are_refused(ig):
    torch = pytest.importorskip("torch")
    host = torch.zeros(4096, dtype=torch.int64)
    n = ig.ig_launch_count()
    for bad in (host, host.numpy()):
        for call, names in [
                (_tree, "q K V page_table L_valid seq first masks out lse workspace"),
                (_slots, "page_table L_valid seq counts parents first slots positions masks"),
                (_keep, "page_table L_valid seq first path kept"), (_bounds, "K list codes scales"),
                (_select, "q codes scales page_table L_valid chosen tokens"), (_picked, "q K V chosen tokens out lse workspace")]:
            for name in names.split():
                with pytest.raises(ValueError, match="CPU"):
                    call(ig, **{name: bad})
        for K, V in (([bad], [1 << 20]), ([1 << 20], [bad])):
            with pytest.raises(ValueError, match="CPU"):
                _keep(ig, K=K, V=V)
    with pytest.raises(ValueError, match="one K"):
        _keep(ig, K=[512, 512])
    assert ig.ig_launch_count() == n


class HostSteps:
    """A PagedCache on CPU tensors whose drafting, keeping and bounds are plain loops."""

    def __init__(self, ig, monkeypatch, **k):
        torch = pytest.importorskip("torch")
        from speculative_kv_cache_gb300.paged import PagedCache

        self.made, self.fail = [], False

        def page_copy(stream, layers, n_pages, Hkv, page, d, K, V, n, moves):
            for a, b, r in moves.tolist():
                for x in K + V:
                    x[b, :, :r] = x[a, :, :r].clone()

        def page_slots(stream, n, seqs, page, n_pages, max_pages, T, table, L, seq, counts, parents, first, slots, positions, masks):
            if self.fail:
                raise RuntimeError("no launch")
            at = 0
            for i in range(n):
                first[i] = at
                base = int(L[seq[i]]) - int(counts[i])
                for j in range(int(counts[i])):
                    p = int(parents[at + j])
                    masks[at + j] = (1 << j) | (int(masks[at + p]) if p >= 0 else 0)
                    slots[at + j] = int(table[seq[i], (base + j) // page]) * page + (base + j) % page
                    positions[at + j] = base + bin(int(masks[at + j])).count("1") - 1
                at += int(counts[i])
            first[n] = at

        def tree_keep(stream, layers, n_pages, Hkv, page, d, K, V, n, seqs, max_pages, T, table, L, seq, first, path, kept):
            if self.fail:
                raise RuntimeError("no launch")
            for i in range(n):
                base = int(L[seq[i]]) - int(first[i + 1] - first[i])
                at = lambda j: (int(table[seq[i], (base + j) // page]), (base + j) % page)  # noqa: E731,B023
                for k in range(int(kept[i])):
                    (a, r), (b, s) = at(int(path[first[i] + k])), at(k)
                    for x in K + V:
                        x[b, :, s] = x[a, :, r].clone()

        def page_bounds(stream, dt, n_pages, Hkv, page, d, K, n, pages, codes, scales):
            self.made.append([tuple(x) for x in pages.tolist()])
            for p, r in pages.tolist():
                codes[p, :, 0] = K[p, :, :r].amin(1).to(torch.int8)
                codes[p, :, 1] = K[p, :, :r].amax(1).to(torch.int8)

        for name, f in dict(ig_page_copy=page_copy, ig_page_slots=page_slots, ig_tree_keep=tree_keep, ig_page_bounds=page_bounds).items():
            monkeypatch.setattr(ig, name, f)
        monkeypatch.setattr(torch.cuda, "set_device", lambda d: None)
        monkeypatch.setattr(torch.cuda, "current_device", lambda: None)
        a = dict(layers=2, Hq=2, Hkv=2, d=64, n_pages=30, seqs=4, max_pages=9, page=8, device="cpu", bounds=True)
        a.update(k)
        self.cache, self.want, self.next = PagedCache(**a), [[] for _ in range(4)], 1
        for x in self.cache.K + self.cache.V:
            x.fill_(-1)

    def fill(self, slots):
        c, out = self.cache, []
        for s in slots.tolist():
            for x in c.K + c.V:
                x[s // c.page, :, s % c.page] = self.next
            out.append(self.next)
            self.next = self.next % 100 + 1
        return out

    def put(self, new):
        slots, _ = self.cache.extend(new)
        got = self.fill(slots)
        for seq, n in new.items():
            self.want[seq] += [got.pop(0) for _ in range(n)]

    def check(self):
        """Rows, and in every layer whose bounds are made the bounds of each page's live tokens (or of more: a page that was cut)."""
        c = self.cache
        t, L = c.table.tolist(), c.L.tolist()
        assert L == [len(w) for w in self.want]
        for s, w in enumerate(self.want):
            for i, v in enumerate(w):
                for x in c.K + c.V:
                    assert (x[t[s][i // c.page], :, i % c.page] == v).all()
        for layer in range(c.layers):
            c.summarise(layer)
            for s, w in enumerate(self.want):
                for i in range(0, len(w), c.page):
                    codes = c.codes[layer][t[s][i // c.page]]
                    assert (codes[:, 0] <= min(w[i:i + c.page])).all() and (codes[:, 1] >= max(w[i:i + c.page])).all()


def test_cache_drafts_and_keeps_on_the_host(ig, monkeypatch):
    h = HostSteps(ig, monkeypatch)
    c = h.cache
    h.put({0: 13, 1: 8})
    h.check()
    made = len(h.made)
    h.check()  # nothing is due
    assert len(h.made) == made
    draft = c.draft({1: [-1, 0, 0, 2, 2], 0: [-1, -1, 1]})
    assert draft.first.tolist() == [0, 5, 8] and draft.positions.tolist() == [8, 9, 9, 10, 10, 13, 13, 14]
    assert draft.masks.tolist() == [1, 3, 5, 13, 21, 1, 2, 6]
    rows = h.fill(draft.slots)
    h.want[1] += rows[:5]
    h.want[0] += rows[5:]
    h.check()  # bounds of the drafted rows too
    c.keep(draft, {1: [0, 2, 4], 0: [1]})
    h.want[1] = h.want[1][:8] + [rows[0], rows[2], rows[4]]
    h.want[0] = h.want[0][:13] + [rows[6]]
    h.check()
    t = c.table.tolist()  # kept rows have their own bounds, not those of the rows that went
    assert c.codes[0][t[1][1], 0, 1, 0] == max(h.want[1][8:])
    with pytest.raises(ValueError, match="over"):
        c.keep(draft, {})
    # forks that share a page: it has the bounds of what the longer one holds
    c.fork(0, 2)
    h.want[2] = list(h.want[0])
    c.truncate(2, 10)
    h.want[2] = h.want[2][:10]
    h.check()
    h.put({2: 3})
    h.check()
    c.free(0)
    h.want[0] = []
    assert c.compact() > 0
    h.check()
    h.put({0: 20, 1: 1})
    h.check()


def test_cache_takes_a_failed_draft_back(ig, monkeypatch):
    h = HostSteps(ig, monkeypatch)
    h.put({0: 13})
    free = h.cache.free_pages()
    h.fail = True
    with pytest.raises(RuntimeError, match="no launch"):
        h.cache.draft({0: [-1] * 20, 1: [-1]})
    h.fail = False
    assert h.cache.free_pages() == free
    h.check()
    draft = h.cache.draft({0: [-1, -1]})
    rows = h.fill(draft.slots)
    h.fail = True
    with pytest.raises(RuntimeError, match="no launch"):
        h.cache.keep(draft, {0: [1]})
    h.fail = False
    h.cache.keep(draft, {0: [1]})  # as if it had not been tried
    h.want[0].append(rows[1])
    h.check()


def test_cache_goes_on_with_a_keep_that_failed_between_its_layers(ig, monkeypatch):
    """Rows move 128 layers a call: those that have moved do not move again, and the draft stands for nothing else."""
    h = HostSteps(ig, monkeypatch, layers=300)
    c = h.cache
    h.put({0: 13, 1: 8})
    draft = c.draft({0: [-1, -1, 1, 2, 2], 1: [-1, -1]})
    rows = h.fill(draft.slots)
    keep, calls = ig.ig_tree_keep, []

    def now_and_then(*a):
        calls.append(a[1])
        if len(calls) in (2, 4):
            raise RuntimeError("no launch")
        keep(*a)

    monkeypatch.setattr(ig, "ig_tree_keep", now_and_then)
    for _ in range(2):
        with pytest.raises(RuntimeError, match="no launch"):
            c.keep(draft, {0: [1, 2, 4], 1: [1]})
        for other in ({}, {0: [1, 2, 4]}, {0: [1, 2, 3], 1: [1]}):
            with pytest.raises(ValueError, match="moved"):
                c.keep(draft, other)
        with pytest.raises(ValueError, match="moved"):
            c.attend_tree(0, None, draft)
    c.keep(draft, {1: [1], 0: (1, 2, 4)})
    assert calls == [128, 128, 128, 44, 44]
    h.want[0] += [rows[1], rows[2], rows[4]]
    h.want[1] += [rows[6]]
    h.check()


@pytest.mark.parametrize("end", ["extend", "fork", "truncate", "compact", "draft"])
def test_a_draft_is_over_when_its_sequences_change(ig, monkeypatch, end):
    h = HostSteps(ig, monkeypatch)
    c = h.cache
    h.put({3: 9, 0: 9})
    c.free(3)
    h.want[3] = []
    draft = c.draft({0: [-1, 0]})
    dict(extend=lambda: c.extend({0: 1}), fork=lambda: c.fork(0, 1), truncate=lambda: c.truncate(0, 10), compact=c.compact,
         draft=lambda: c.draft({0: [-1]}))[end]()
    with pytest.raises(ValueError, match="over"):
        c.keep(draft, {0: [0]})


def test_a_draft_is_over_when_one_of_its_sequences_becomes_a_copy(ig, monkeypatch):
    """An empty sequence with an empty tree is of the draft too: what is forked into it stays."""
    h = HostSteps(ig, monkeypatch)
    c = h.cache
    h.put({0: 9, 3: 4})
    draft = c.draft({3: [-1, 0], 1: []})
    h.want[3] += h.fill(draft.slots)
    c.fork(0, 1)
    h.want[1] = list(h.want[0])
    with pytest.raises(ValueError, match="over"):
        c.keep(draft, {3: [0]})
    with pytest.raises(ValueError, match="over"):
        c.attend_tree(0, None, draft)
    h.check()
    c.truncate(3, 4)  # the way out: the drafted tokens go
    h.want[3] = h.want[3][:4]
    h.check()


def test_a_draft_outlives_what_other_sequences_do(ig, monkeypatch):
    h = HostSteps(ig, monkeypatch)
    c = h.cache
    h.put({0: 9, 1: 9})
    draft = c.draft({0: [-1, 0]})
    rows = h.fill(draft.slots)
    h.put({1: 3})
    c.fork(1, 2)
    h.want[2] = list(h.want[1])
    c.keep(draft, {0: [0, 1]})
    h.want[0] += rows
    h.check()


def test_bounds_are_of_the_longer_of_two_sequences_that_share_a_page(ig, monkeypatch):
    h = HostSteps(ig, monkeypatch)
    c = h.cache
    slots, _ = c.extend({0: 12})
    rows = h.fill(slots)
    h.want[0] += rows
    c.fork(0, 1)
    c.truncate(1, 10)
    h.want[1] = rows[:10]
    h.check()
    assert np.array_equal(c.codes[0][int(c.table[0, 1]), 0, 1, :2], [max(rows[8:])] * 2)
