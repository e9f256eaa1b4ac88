"""PagedCache: a paged KV cache in HBM over the C ABI (pages, page tables, forks, attention).

It owns the pages of every layer, the host-side page manager (``ig_pages_*``) and the device copy
of its tables, and runs a token's way through a layer: ``write`` (norm and rotation of q and k, the
rows into their pages: ``ig_qk_norm_rope``) and ``attend`` (``ig_paged_attend``).  Sequences can be
forked (pages shared until one writes), cut back, freed, and the pages packed (``ig_page_copy``).
All device work is queued on the current stream of the cache's GPU, whichever GPU is the current one.  The
device tensors ``table`` and ``L`` stay in place, so a captured ``write`` + ``attend`` replays with what
``extend`` put there since.  A cache's calls share its tables and one workspace, so they run one after
another: on one stream, or on streams that wait for each other.
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


class PagedCache:
    def __init__(self, *, layers, Hq, Hkv, d, n_pages, seqs, max_pages, page=32, dtype=torch.float16, scale=None, rot=0,
                 layout=ig.IG_ROPE_HALF, theta=10000.0, scaling=ig.IG_ROPE_PLAIN, factor=1.0, context=0, p0=0.0, p1=0.0,
                 eps=1e-6, device="cuda:0"):
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

    @_on_its_gpu
    def extend(self, new):
        """Room for ``new[sequence]`` more tokens of each named sequence; returns device int32 slots
        and positions of the tokens, in that order.  Raises ValueError or TypeError for a sequence or
        count that cannot be, and IGError (IG_ERR_CAPACITY) when the pages or a table run out, with
        every sequence as it was; only a page of its own that a sequence already got for the one it
        shared (copied on write) stays with it."""
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
            cat = lambda x: torch.from_numpy(np.concatenate(x) if x else np.empty(0, np.int32)).to(self.dev)  # noqa: E731
            return cat(slots), cat(positions)
        except BaseException:
            for seq, had in before:
                ig.ig_pages_truncate(self.pages, seq, had)
            try:
                self._sync()
            except Exception:  # the first error is the one to name; what is due stays due
                pass
            raise

    @_on_its_gpu
    def fork(self, src, dst):
        """Sequence ``dst`` (empty) becomes a copy of ``src``, sharing its pages."""
        self._catch_up()
        ig.ig_pages_fork(self.pages, src, dst)
        self._sync()

    @_on_its_gpu
    def truncate(self, seq, n):
        """Keeps the first ``n`` tokens of a sequence."""
        self._catch_up()
        ig.ig_pages_truncate(self.pages, seq, n)
        self._sync()

    def free(self, seq):
        self.truncate(seq, 0)

    @_on_its_gpu
    def compact(self):
        """Moves the used pages to the lowest numbers; returns how many moved."""
        self._catch_up()
        moves = np.empty((self.n_pages // 2 + 1, 3), dtype=np.int32)
        n = ig.ig_pages_compact(self.pages, moves, len(moves))
        self._moves = moves[:n]
        self._sync()
        return n

    def free_pages(self):
        return ig.ig_pages_free_count(self.pages)

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
