"""PagedCache: a paged KV cache in HBM over the C ABI (pages, page tables, forks, attention).

It owns the pages of every layer, the host-side page manager (``ig_pages_*``) and the device copy
of its tables, and runs a token's way through a layer: ``write`` (norm and rotation of q and k, the
rows into their pages: ``ig_qk_norm_rope``) and ``attend`` (``ig_paged_attend``).  Sequences can be
forked (pages shared until one writes), cut back, freed, and the pages packed (``ig_page_copy``).
Trees of drafted tokens go in together: ``draft`` (room, slots, positions and ancestors: ``ig_page_slots``), ``write``,
``attend_tree`` (``ig_paged_tree_attend``) and ``keep`` (the accepted path's rows: ``ig_tree_keep``).  With ``bounds=True`` the cache
keeps bounds of each page's keys (``summarise``: ``ig_page_bounds``), and ``attend_picked`` attends to the pages that
a score from the bounds picks (``ig_page_select``, ``ig_paged_attend_picked``).
All device work is queued on the current stream of the cache's GPU, whichever GPU is the current one.  The
device tensors ``table`` and ``L`` stay in place, so a captured ``write`` + ``attend`` replays with what
``extend`` put there since.  (A draft's slots, positions, masks and numbers of tokens are its own: a captured
``attend_tree`` replays that one draft, which has to be kept, and live, as long.)  A cache's calls share its
tables and one workspace, so they run one after another: on one stream, or on streams that wait for each other.
"""
from __future__ import annotations

import functools
import math
import operator

import numpy as np
import torch

from . import ig

_DTYPES = {torch.float16: ig.IG_F16, torch.bfloat16: ig.IG_BF16}


def _on_its_gpu(method):
    @functools.wraps(method)
    def call(self, *args, **kwargs):
        if torch.cuda.current_device() == self.dev.index:
            return method(self, *args, **kwargs)
        with torch.cuda.device(self.dev):
            return method(self, *args, **kwargs)

    return call


class Draft:
    """Drafted tokens of some sequences, packed in ``seqs``'s order (``first`` on the device: where each begins): their
    device ``slots`` and ``positions`` for ``write``, and the ``masks`` of their ancestors."""

    def __init__(self, seqs, parents, base):
        self.seqs, self.parents, self.base = seqs, parents, base
        self.n, self.T = len(seqs), sum(len(p) for p in parents)
        self.T_max = max([len(p) for p in parents] + [1])
        self.kept, self.moved = None, 0  # paths of a keep that has begun, and layers that have their rows


class PagedCache:
    def __init__(self, *, layers, Hq, Hkv, d, n_pages, seqs, max_pages, page=32, dtype=torch.float16, scale=None, rot=0,
                 layout=ig.IG_ROPE_HALF, theta=10000.0, scaling=ig.IG_ROPE_PLAIN, factor=1.0, context=0, p0=0.0, p1=0.0,
                 eps=1e-6, device="cuda:0", bounds=False):
        self.pages = None
        if dtype not in _DTYPES:
            raise ValueError(f"pages hold float16 or bfloat16, not {dtype}")
        self.layers, self.Hq, self.Hkv, self.d = layers, Hq, Hkv, d
        self.n_pages, self.seqs, self.max_pages, self.page = n_pages, seqs, max_pages, page
        self.dtype, self.dt = dtype, _DTYPES[dtype]
        self.scale = float(scale if scale is not None else 1.0 / math.sqrt(d))
        self.rot, self.layout, self.eps = rot, layout, eps
        self.dev = torch.device(device)
        torch.cuda.set_device(self.dev)
        self.pages = ig.ig_pages_create(n_pages, page, seqs, max_pages)
        shape = (n_pages, Hkv, page, d)
        self.K = [torch.empty(shape, dtype=dtype, device=self.dev) for _ in range(layers)]
        self.V = [torch.empty(shape, dtype=dtype, device=self.dev) for _ in range(layers)]
        self.turns, self.rot_scale = None, 1.0
        if rot:
            turns = np.zeros(rot // 2, dtype=np.int64)
            self.rot_scale = ig.ig_rope_turns(rot, theta, scaling, factor, context, p0, p1, turns)
            self.turns = torch.from_numpy(turns).to(self.dev)
        self.table_host = np.full((seqs, max_pages), -1, dtype=np.int32)
        self.L_host = np.zeros(seqs, dtype=np.int32)
        self._moves, self._stale = [], False  # page moves still to run; whether the device is behind the manager
        self.table = torch.full((seqs, max_pages), -1, dtype=torch.int32, device=self.dev)
        self.L = torch.zeros(seqs, dtype=torch.int32, device=self.dev)
        self.ws = torch.empty(ig.ig_paged_attend_workspace_bytes(seqs, Hq, Hkv, d), dtype=torch.uint8, device=self.dev)
        self.tree_ws = None  # from the first draft on
        self._drafts = {}  # the draft that each sequence ends with
        self.codes = self.scales = None
        if bounds:
            self.codes = [torch.zeros((n_pages, Hkv, 2, d), dtype=torch.int8, device=self.dev) for _ in range(layers)]
            self.scales = [torch.zeros((n_pages, Hkv), dtype=torch.float32, device=self.dev) for _ in range(layers)]
            self._seen = np.zeros((layers, seqs), dtype=np.int64)  # tokens whose pages have their bounds
            self._due = (None, None)  # the last list of pages, and what it was made for

    # ------------------------------------------------------------------ the sequences
    def _sync(self):
        """The device brought up to the manager: the moves that are due, then its tables and lengths
        (ordered on the current stream).  Where that fails, it stays due for the next call."""
        self._stale = True
        ig.ig_pages_table(self.pages, self.table_host, self.L_host)
        if len(self._moves):
            m = torch.from_numpy(np.ascontiguousarray(self._moves, dtype=np.int32)).to(self.dev)
            for l in range(0, self.layers, 128):
                K, V = self.K[l:l + 128], self.V[l:l + 128]
                ig.ig_page_copy(None, len(K), self.n_pages, self.Hkv, self.page, self.d, K, V, len(self._moves), m)
            if self.codes is not None:
                src, dst = m[:, 0].long(), m[:, 1].long()
                for x in self.codes + self.scales:
                    x[dst] = x[src]
        self._moves = []
        self.table.copy_(torch.from_numpy(self.table_host))
        self.L.copy_(torch.from_numpy(self.L_host))
        self._stale = False

    def _catch_up(self):
        if self._stale:
            self._sync()

    def _counts(self, new):
        """``new`` as pairs of whole numbers, all of them checked."""
        out = {}
        for seq, n in new.items():
            seq, n = operator.index(seq), operator.index(n)
            if not 0 <= seq < self.seqs or n < 0 or seq in out:
                raise ValueError(f"{n} tokens for sequence {seq}: the count must not be negative, the sequence one of "
                                 f"{self.seqs} and named once")
            out[seq] = min(n, self.max_pages * self.page + 1)  # one more than a table holds is refused below
        return out.items()

    def _check(self, name, x, *shape, dtype=None):
        if x is not None and (x.numel() != math.prod(shape) or x.shape[0] != shape[0] or x.dtype != (dtype or self.dtype)):
            raise ValueError(f"{name} must be {list(shape)} of {dtype or self.dtype}, got {list(x.shape)} of {x.dtype}")

    def _extend(self, new, answer):
        """Room for ``new[sequence]`` more tokens, and what ``answer`` makes of their slots and positions on the host;
        where any of it fails, every sequence as it was."""
        want = self._counts(new)
        self._catch_up()
        slots, positions, before = [], [], []
        try:
            for seq, n in want:
                s = np.empty(n, dtype=np.int32)
                had = int(self.L_host[seq])
                move = ig.ig_pages_extend(self.pages, seq, n, s)
                before.append((seq, had))
                if move is not None:
                    self._moves.append(move)
                slots.append(s)
                positions.append(np.arange(had, had + n, dtype=np.int32))
            self._sync()
            out = answer(slots, positions)
        except BaseException:
            for seq, had in before:
                ig.ig_pages_truncate(self.pages, seq, had)
            try:
                self._sync()
            except Exception:  # the first error is the one to name; what is due stays due
                pass
            raise
        for seq, n in want:
            if n:
                self._drafts.pop(seq, None)
        return out

    @_on_its_gpu
    def extend(self, new):
        """Room for ``new[sequence]`` more tokens of each named sequence; returns device int32 slots
        and positions of the tokens, in that order.  Raises ValueError or TypeError for a sequence or
        count that cannot be, and IGError (IG_ERR_CAPACITY) when the pages or a table run out, with
        every sequence as it was; only a page of its own that a sequence already got for the one it
        shared (copied on write) stays with it."""
        cat = lambda x: torch.from_numpy(np.concatenate(x) if x else np.empty(0, np.int32)).to(self.dev)  # noqa: E731
        return self._extend(new, lambda slots, positions: (cat(slots), cat(positions)))

    @_on_its_gpu
    def fork(self, src, dst):
        """Sequence ``dst`` (empty) becomes a copy of ``src``, sharing its pages."""
        self._catch_up()
        ig.ig_pages_fork(self.pages, src, dst)
        for seq in (src, dst):  # (an empty sequence with an empty tree is of its draft too)
            self._drafts.pop(seq, None)
        if self.codes is not None:
            self._seen[:, dst] = self._seen[:, src]
        self._sync()

    @_on_its_gpu
    def truncate(self, seq, n):
        """Keeps the first ``n`` tokens of a sequence.  (The bounds of the page that is cut stay those of what it held
        until tokens follow.)"""
        self._catch_up()
        self._cut(seq, n)
        self._sync()

    def _cut(self, seq, n):
        ig.ig_pages_truncate(self.pages, seq, n)
        self._drafts.pop(seq, None)
        if self.codes is not None:
            np.minimum(self._seen[:, seq], n, out=self._seen[:, seq])

    def free(self, seq):
        self.truncate(seq, 0)

    @_on_its_gpu
    def compact(self):
        """Moves the used pages to the lowest numbers; returns how many moved."""
        self._catch_up()
        moves = np.empty((self.n_pages // 2 + 1, 3), dtype=np.int32)
        n = ig.ig_pages_compact(self.pages, moves, len(moves))
        self._moves = moves[:n]
        if n:
            self._drafts.clear()  # their slots may be other ones now
        self._sync()
        return n

    def free_pages(self):
        return ig.ig_pages_free_count(self.pages)

    # ------------------------------------------------------------------ drafted trees
    @_on_its_gpu
    def draft(self, trees):
        """Room for trees of drafted tokens: ``trees[sequence]`` lists each token's parent among the sequence's drafted
        ones (a lower number than its own), or -1 (it follows the sequence's last token); at most 64 a
        sequence.  Returns a Draft: packed in that order, with its slots and positions (a sibling has its
        sibling's).  The sequences hold the drafted tokens until ``keep`` or ``truncate``.  Raises as ``extend``
        does, and ValueError for a tree that cannot be."""
        seqs, parents = [], []
        for seq, tree in trees.items():
            tree = [operator.index(p) for p in tree]
            if len(tree) > 64 or any(not -1 <= p < i for i, p in enumerate(tree)):
                raise ValueError(f"sequence {seq}: a tree has at most 64 tokens, each with a parent before it or -1")
            seqs.append(operator.index(seq))
            parents.append(tree)
        if not 1 <= len(seqs) <= 8192:
            raise ValueError(f"trees for 1 to 8192 sequences, not {len(seqs)}")
        if self.tree_ws is None:
            need = ig.ig_paged_tree_attend_workspace_bytes(self.seqs, 64, self.Hq, self.Hkv, self.d)
            self.tree_ws = torch.empty(need, dtype=torch.uint8, device=self.dev)

        def answer(slots, positions):
            x = Draft(seqs, parents, [int(self.L_host[s]) - len(p) for s, p in zip(seqs, parents)])
            up = np.array(seqs + [len(p) for p in parents] + [p for t in parents for p in t], dtype=np.int32)
            up = torch.from_numpy(up).to(self.dev)
            x.seq = up[:x.n]
            x.first = torch.empty(x.n + 1, dtype=torch.int32, device=self.dev)
            x.slots = torch.empty(x.T, dtype=torch.int32, device=self.dev)
            x.positions = torch.empty(x.T, dtype=torch.int32, device=self.dev)
            x.masks = torch.empty(x.T, dtype=torch.int64, device=self.dev)
            ig.ig_page_slots(None, x.n, self.seqs, self.page, self.n_pages, self.max_pages, x.T, self.table, self.L, x.seq,
                             up[x.n:2 * x.n], up[2 * x.n:], x.first, x.slots, x.positions, x.masks)
            return x

        x = self._extend({s: len(p) for s, p in zip(seqs, parents)}, answer)
        self._drafts.update((s, x) for s in seqs)
        return x

    def _drafted(self, draft, paths=None):
        if any(self._drafts.get(s) is not draft for s in draft.seqs):
            raise ValueError("the draft is over: its sequences have been extended, forked or cut since, or the pages packed")
        if draft.moved and paths != draft.kept:
            raise ValueError("rows of the draft have moved in some layers: a keep of the same paths goes on with the others")

    @_on_its_gpu
    def attend_tree(self, layer, q, draft, out=None, lse=None):
        """Attention of the drafted tokens, q [T, Hq, d], each over its sequence's tokens before the draft, its
        ancestors and itself: [T, Hq, d] of the cache's type."""
        self._drafted(draft)
        self._check("q", q, draft.T, self.Hq, self.d)
        self._check("out", out, draft.T, self.Hq, self.d)
        self._check("lse", lse, draft.T, self.Hq, dtype=torch.float32)
        if out is None:
            out = torch.empty((draft.T, self.Hq, self.d), dtype=self.dtype, device=self.dev)
        ig.ig_paged_tree_attend(None, self.dt, draft.n, draft.T, draft.T_max, self.Hq, self.Hkv, self.d, self.page, self.n_pages,
                                self.seqs, self.max_pages, self.scale, q, self.K[layer], self.V[layer], self.table, self.L,
                                draft.seq, draft.first, draft.masks, out, lse, self.tree_ws, self.tree_ws.numel())
        return out

    @_on_its_gpu
    def keep(self, draft, paths):
        """Keeps ``paths[sequence]`` of each of the draft's sequences, in every layer: the numbers of its accepted drafted tokens
        from the first level on, each the parent of the next (none where a sequence is not named).  The other
        drafted tokens go.  Where that fails, the sequences have their drafted tokens still, and it can be tried again: with
        other paths too, unless rows have moved already (in some of more than 128 layers)."""
        paths = {operator.index(s): [operator.index(i) for i in p] for s, p in paths.items()}
        if not set(paths) <= set(draft.seqs):
            raise ValueError("a path for a sequence that the draft does not have")
        paths = [paths.get(s, []) for s in draft.seqs]
        self._drafted(draft, paths)
        for seq, path, tree in zip(draft.seqs, paths, draft.parents):
            if any(not 0 <= i < len(tree) for i in path) or any(tree[i] != p for p, i in zip([-1] + path, path)):
                raise ValueError(f"sequence {seq}: {path} is no path of its tree from the first level on")
        self._catch_up()
        if any(i != k for path in paths for k, i in enumerate(path)):
            up = [len(path) for path in paths]
            for path, tree in zip(paths, draft.parents):
                up += path + [0] * (len(tree) - len(path))
            up = torch.from_numpy(np.array(up, dtype=np.int32)).to(self.dev)
            for l in range(draft.moved, self.layers, 128):  # (a second move would start from rows that are others by now)
                K, V = self.K[l:l + 128], self.V[l:l + 128]
                ig.ig_tree_keep(None, len(K), self.n_pages, self.Hkv, self.page, self.d, K, V, draft.n, self.seqs, self.max_pages,
                                draft.T, self.table, self.L, draft.seq, draft.first, up[draft.n:], up[:draft.n])
                draft.kept, draft.moved = paths, l + len(K)
        for seq, path, base in zip(draft.seqs, paths, draft.base):
            self._cut(seq, base + len(path))
            if self.codes is not None:
                np.minimum(self._seen[:, seq], base, out=self._seen[:, seq])
        self._sync()

    # ------------------------------------------------------------------ picked pages
    def _bounded(self):
        if self.codes is None:
            raise ValueError("the cache keeps no bounds: make it with bounds=True")

    @_on_its_gpu
    def summarise(self, layer):
        """The bounds of ``layer``'s pages that have got tokens since the last time, from what the pages hold now.  (Which ones is
        decided on the host: not while a graph is captured, which would repeat that one list.)"""
        self._bounded()
        self._catch_up()
        seen = self._seen[layer]
        stale = np.nonzero(seen < self.L_host)[0]
        if not len(stale):
            return
        if torch.cuda.is_initialized() and torch.cuda.is_current_stream_capturing():
            raise ValueError("bounds are due, and a graph is being captured: summarise the layer before")
        made_for = (seen.tobytes(), self.L_host.tobytes(), self.table_host[stale].tobytes())
        if self._due[0] != made_for:
            ids, rows = [], []
            for s in stale:
                at = np.arange(seen[s] // self.page, -(-int(self.L_host[s]) // self.page))
                ids.append(self.table_host[s, at])
                rows.append(np.minimum(self.L_host[s] - at * self.page, self.page))
            ids, rows = np.concatenate(ids), np.concatenate(rows)
            order = np.lexsort((rows, ids))  # a page that sequences share: with the most tokens it has in one of them
            ids, rows = ids[order], rows[order]
            last = np.append(ids[1:] != ids[:-1], True)
            pages = np.stack([ids[last], rows[last]], 1).astype(np.int32)
            self._due = (made_for, torch.from_numpy(pages).to(self.dev))
        pages = self._due[1]
        ig.ig_page_bounds(None, self.dt, self.n_pages, self.Hkv, self.page, self.d, self.K[layer], len(pages), pages,
                          self.codes[layer], self.scales[layer])
        seen[:] = self.L_host

    @_on_its_gpu
    def attend_picked(self, layer, q, picks, first=1, last=2, out=None, lse=None):
        """``attend`` over at most ``picks`` pages of each sequence and key head: its first ``first`` and last ``last`` ones, and
        those whose bounds allow its queries the largest logits.  Bounds that are due are made first; a captured call
        replays with those that ``summarise`` has made since."""
        self._bounded()
        self._check("q", q, self.seqs, self.Hq, self.d)
        self._check("out", out, self.seqs, self.Hq, self.d, dtype=torch.float32)
        self._check("lse", lse, self.seqs, self.Hq, dtype=torch.float32)
        self.summarise(layer)
        if out is None:
            out = torch.empty((self.seqs, self.Hq, self.d), dtype=torch.float32, device=self.dev)
        picks = min(operator.index(picks), max(self.max_pages, first + last))  # (more than a table holds are all of them)
        chosen = torch.empty((self.seqs, self.Hkv, max(picks, 0)), dtype=torch.int32, device=self.dev)
        tokens = torch.empty((self.seqs, self.Hkv), dtype=torch.int32, device=self.dev)
        ig.ig_page_select(None, self.dt, self.seqs, self.Hq, self.Hkv, self.d, self.page, self.n_pages, self.max_pages, picks, first,
                          last, q, self.codes[layer], self.scales[layer], self.table, self.L, chosen, tokens)
        ig.ig_paged_attend_picked(None, self.dt, self.seqs, self.Hq, self.Hkv, self.d, self.page, self.n_pages, picks, self.scale,
                                  q, self.K[layer], self.V[layer], chosen, tokens, out, lse, self.ws, self.ws.numel())
        return out

    # ------------------------------------------------------------------ a layer's step
    @_on_its_gpu
    def write(self, layer, q, k, v, slots, positions, q_weight=None, k_weight=None, q_out=None):
        """Norms and rotates the tokens' q [T, Hq, d] and k [T, Hkv, d] and puts k and v [T, Hkv, d]
        into ``layer``'s pages; returns the new q.  q, k and v may be slices of one projection
        [T, heads * d] (the first dimension's stride is taken as it is)."""
        T = q.shape[0]
        self._check("q", q, T, self.Hq, self.d)
        self._check("k", k, T, self.Hkv, self.d)
        self._check("v", v, T, self.Hkv, self.d)
        self._check("slots", slots, T, dtype=torch.int32)
        self._check("positions", positions, T, dtype=torch.int32)
        self._check("q_weight", q_weight, self.d)
        self._check("k_weight", k_weight, self.d)
        self._check("q_out", q_out, T, self.Hq, self.d)
        if q_out is None:
            q_out = torch.empty((T, self.Hq, self.d), dtype=self.dtype, device=self.dev)
        # a lone row's stride may be anything: it is never used
        qs, ks, vs = (x.stride(0) if T > 1 else h * self.d for x, h in ((q, self.Hq), (k, self.Hkv), (v, self.Hkv)))
        ig.ig_qk_norm_rope(None, self.dt, T, self.Hq, self.Hkv, self.d, self.rot, self.layout, q, qs, k, ks, v, vs,
                           q_weight, k_weight, self.eps, positions, self.turns, self.rot_scale, q_out, self.page,
                           self.n_pages, slots, self.K[layer], self.V[layer])
        return q_out

    @_on_its_gpu
    def attend(self, layer, q, out=None, lse=None):
        """Attention of one token per sequence, q [seqs, Hq, d], over all its tokens: fp32
        [seqs, Hq, d], zero for empty sequences."""
        self._check("q", q, self.seqs, self.Hq, self.d)
        self._check("out", out, self.seqs, self.Hq, self.d, dtype=torch.float32)
        self._check("lse", lse, self.seqs, self.Hq, dtype=torch.float32)
        if out is None:
            out = torch.empty((self.seqs, self.Hq, self.d), dtype=torch.float32, device=self.dev)
        ig.ig_paged_attend(None, self.dt, self.seqs, self.Hq, self.Hkv, self.d, self.page, self.n_pages, self.max_pages,
                           self.scale, q, self.K[layer], self.V[layer], self.table, self.L, out, lse, self.ws,
                           self.ws.numel())
        return out

    def close(self):
        if self.pages is not None:
            ig.ig_pages_destroy(self.pages)
            self.pages = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
