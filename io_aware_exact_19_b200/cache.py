"""Serving over a paged key/value cache, and rotary positions for training.

:class:`PagedCache` keeps the buffers that the paged-cache entry points share and calls
them in the order of a serving step:

    cache.plan(new, parent)        pages, slots, positions, tree masks     (one launch)
    for each layer:
        q = cache.append(layer, q, k, v, rope)      rotate, write K and V   (one launch)
        o = cache.attend(layer, q)                  attention               (one or two)
    cache.commit(accepted, count)  or  cache.keep() the rows that stay      (one a layer; none)

Beside these launches plan, commit and keep run two or three, two and one small operations of torch.

Everything runs on the current stream. Lengths, tables and maps stay on the GPU, so a step can
be captured in a CUDA graph (after one run outside it) and replayed with other lengths in the
same buffers.
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import paged


def rope_tables(rot: int, sections=None, base: float = 10000.0, interleaved: bool = False, device="cuda"):
    """Frequencies and axes of the ``rot/2`` rotated pairs: ``base ** (-2 i / rot)`` for pair i;
    ``sections`` gives each axis (time, height, width) its number of pairs, in runs or, with
    ``interleaved``, taking turns while an axis has some left. None is a single axis."""
    half = rot // 2
    sections = [half] if sections is None else list(sections)
    if rot % 2 or sum(sections) != half or min(sections) < 0:
        raise ValueError(f"the sections {sections} do not share out {half} pairs")
    if interleaved:
        left, axis = list(sections), []
        while len(axis) < half:
            for a in range(len(sections)):
                if left[a] > 0:
                    left[a] -= 1
                    axis.append(a)
    else:
        axis = [a for a, n in enumerate(sections) for _ in range(n)]
    inv_freq = (float(base) ** (-torch.arange(half, dtype=torch.float64) * 2 / rot)).to(torch.float32)
    return inv_freq.to(device), torch.tensor(axis, dtype=torch.uint8, device=device)


@dataclass
class Rope:
    """A rotation: the tables of :func:`rope_tables`, the positions (int32 [axes, T] for a serving
    step, None: the plan's on every axis; [axes, B, N] or [axes, N] for training) and how pairs lie."""
    inv_freq: torch.Tensor
    axis: torch.Tensor
    positions: torch.Tensor | None = None
    pairs: bool = False

    def turn(self, x, out=None, inverse: bool = False, stream=None):
        """``x`` [B, H, N, d] rotated (into a new tensor unless ``out`` is given)."""
        if out is None:
            # Memory of the stream that writes it: the current stream's could still be in use there.
            with torch.cuda.stream(stream):
                out = torch.empty_like(x, memory_format=torch.contiguous_format)
            if stream is not None:
                out.record_stream(torch.cuda.current_stream(x.device))
        paged.fa_rope(x, out, self.positions, self.inv_freq, self.axis, inverse=inverse, pairs=self.pairs, stream=stream)
        return out


class PagedCache:
    """Key/value cache of ``layers`` layers in ``num_pages`` pages of ``page_size`` rows, for up to
    ``batch`` requests of ``max_len`` rows, ``max_rows`` new rows a step in all and ``max_new`` of one
    request. Request b's committed rows are counted in ``ctx_len[b]`` (0: the slot is free; its
    pages go back with the next plan)."""

    def __init__(self, num_pages: int, page_size: int, batch: int, max_len: int, H_kv: int, d: int, max_rows: int,
                 max_new: int, layers: int = 1, dtype=torch.bfloat16, device="cuda"):
        self.page_size, self.max_new, self.batch = page_size, max_new, batch
        self.k, self.v = (torch.empty((layers, num_pages, H_kv, page_size, d), dtype=dtype, device=device)
                          for _ in range(2))
        ints = lambda *shape: torch.zeros(shape, dtype=torch.int32, device=device)  # noqa: E731
        self.block_table = ints(batch, -(-max_len // page_size)).fill_(-1)
        self.n_pages, self.ctx_len, self.seq_len, self.new_len = ints(batch), ints(batch), ints(batch), ints(batch)
        self.free_list = torch.arange(num_pages, dtype=torch.int32, device=device)
        self.free_count = ints(1).fill_(num_pages)
        self.cu_new = ints(batch + 1)
        self.slot, self.position, self._parent = ints(max_rows), ints(max_rows), ints(max_rows)
        self._mask = torch.zeros(max_rows * -(-max_new // 64), dtype=torch.int64, device=device)
        self.tree_mask, self.most = None, max_new
        self._workspace = {}

    def plan(self, new, parent=None, most: int | None = None) -> None:
        """Start a step in which request b adds ``new[b]`` rows (an int32 tensor [batch] on the
        GPU, at most ``most`` each; the attention is quickest when that is close): their slots and
        positions, and with ``parent`` (int32, one for each new row) the masks of drafted trees.
        ``seq_len[b]`` is 0 where the pages did not suffice, and where a request's rows go beyond the
        step's ``max_rows``. Pages are granted in the order of the requests, and one that gets none holds up
        those behind it that need some: leave it out of the step (``new[b] = 0``) until pages are back."""
        self.most = self.max_new if most is None else most
        if not 1 <= self.most <= self.max_new:
            raise ValueError(f"most must lie in 1..{self.max_new}")
        self.cu_new[1:].copy_(new.cumsum(0))
        self.tree_mask = None
        if parent is not None:
            self._parent[:parent.numel()].copy_(parent)
            words = -(-self.most // 64)
            self.tree_mask = self._mask[:self.slot.numel() * words].view(-1, words)
        paged.fa_cache_plan(self.ctx_len, self.cu_new, self.block_table, self.n_pages, self.free_list, self.free_count,
                            self.seq_len, self.slot, self.position, page_size=self.page_size, max_new=self.most,
                            parent=None if parent is None else self._parent, tree_mask=self.tree_mask)

    def append(self, layer: int, q, k, v, rope: Rope | None = None, q_out=None):
        """Write the step's rows ``k`` and ``v`` [T, H_kv, d] to their slots; returns ``q`` rotated (and
        rotates ``k``) by ``rope``, in ``q_out`` if it is given. Without ``rope`` nothing is rotated: ``q`` is
        returned, or copied into ``q_out``. Rows past the step's last (a padded batch) are not written."""
        T = k.shape[0]
        if rope is None:
            paged.fa_rope_append(None if q_out is None else q, k, v, q_out, self.k[layer], self.v[layer], self.slot[:T])
            return q if q_out is None else q_out
        q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device) if q_out is None else q_out
        positions = rope.positions
        if positions is None:  # the plan's, on as many axes as the tables may name
            positions = self.position[:T].expand(8, T)
        paged.fa_rope_append(q, k, v, q_out, self.k[layer], self.v[layer], self.slot[:T], positions, rope.inv_freq,
                             rope.axis, pairs=rope.pairs)
        return q_out

    def attend(self, layer: int, q, o=None, lse=None, scale=None):
        """Attention of the step's rows ``q`` [T, Hq, d] over the cache; returns (o, lse)."""
        T, Hq, d = q.shape
        o = torch.empty((T, Hq, d), dtype=q.dtype, device=q.device) if o is None else o
        lse = torch.empty((T, Hq), dtype=torch.float32, device=q.device) if lse is None else lse
        # One for each number of heads, large enough for any step and never replaced: a graph captured
        # with a step of few rows goes on using it after one of many.
        workspace = self._workspace.get(Hq)
        if workspace is None:
            need = paged.fa_tree_fwd_workspace_size(self.batch, self.slot.numel(), self.max_new, Hq, self.k.shape[2], d)
            workspace = self._workspace[Hq] = torch.empty(need, dtype=torch.uint8, device=q.device)
        mask = None if self.tree_mask is None else self.tree_mask[:T]
        paged.fa_tree_fwd(q, self.k[layer], self.v[layer], self.block_table, self.seq_len, self.cu_new, o, lse,
                          workspace, max_q=self.most, tree_mask=mask, scale=scale)
        return o, lse

    def commit(self, accepted, n_accepted) -> None:
        """End a step of drafted trees: of each request's new rows keep the path ``accepted[b,
        :n_accepted[b]]`` (int32, strictly increasing), in every layer. A refused request, whose rows
        were not written, keeps its length whatever they say."""
        n_accepted = torch.where(self.seq_len > 0, n_accepted, 0)
        for layer in range(self.k.shape[0]):
            paged.fa_cache_commit(self.k[layer], self.v[layer], self.block_table, self.ctx_len, accepted, n_accepted,
                                  self.new_len)
        self.ctx_len.copy_(self.new_len)

    def keep(self) -> None:
        """End a step whose new rows all stay (decoding, prompt chunks); a refused request
        (``seq_len`` 0 although it has rows) keeps its length."""
        torch.where(self.seq_len > 0, self.seq_len, self.ctx_len, out=self.ctx_len)

    def release(self, b: int) -> None:
        """Request b is done: its pages go back with the next plan."""
        self.ctx_len[b] = 0
