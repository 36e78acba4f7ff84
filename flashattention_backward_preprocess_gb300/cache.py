"""A paged key/value cache over the library's paged calls: pages, tables and lengths of a fixed
set of request rows, for any number of attention layers.

One step of a model, for the new tokens of all requests (one each, or chunks of prompts):

    cache.begin(cu_q, tokens)                      # fa_page_slots: pages, slots, positions
    for layer in range(layers):
        O, LSE = cache.attend(layer, Q, K, V)      # fa_paged_write, fa_paged_fwd
Everything stays on the device and in stream order; nothing waits for the GPU but release().  A
step can be captured into a graph; every replay takes the step again, for the tokens and offsets
that its input tensors then hold.
"""
from __future__ import annotations

import torch

from . import packed
from .binding import FaError


class PagedKVCache:
    """layers x [num_pages, page_size, H_kv, d] K and V for up to `rows` requests.

    block_table [rows, max_pages], lens [rows] (tokens held), free_pages and free_start (the next
    unused entry of it) are device tensors; positions [tokens] of the step's new tokens are there
    after begin().  A request row that brings no token in a step (cu_q does not move) costs
    nothing.  When the pages run out, or a request outgrows max_pages, fa_check_device() raises, at
    every step until the row is released.  The tokens without a page are not cached: the row's later
    tokens see zeros in the place of those that found no page, and nothing of those behind the
    table's last column.  The other rows go on as ever.
    """

    def __init__(self, layers: int, num_pages: int, page_size: int, H_kv: int, d: int, rows: int, max_pages: int,
                 dtype=torch.bfloat16, device="cuda"):
        i32 = dict(dtype=torch.int32, device=device)
        self.page_size = int(page_size)
        self.K = [torch.zeros(num_pages, page_size, H_kv, d, dtype=dtype, device=device) for _ in range(layers)]
        self.V = [torch.zeros_like(k) for k in self.K]
        self.block_table = torch.full((rows, max_pages), -1, **i32)
        self.lens = torch.zeros(rows, **i32)
        self.free_pages = torch.arange(num_pages, **i32)
        self.free_start = torch.zeros(1, **i32)
        self.cu_q = self.slots = self.positions = None

    def begin(self, cu_q, tokens: int):
        """Takes the pages of the step's new tokens (int32 offsets cu_q [rows + 1], `tokens` rows in
        the step's tensors, padding behind cu_q[rows] included) and returns their positions."""
        self.cu_q = cu_q
        self.slots, self.positions, lens, start = packed.fa_page_slots(
            self.lens, cu_q, self.block_table, self.free_pages, self.free_start, self.page_size, tokens)
        # in place: the replays of a captured step go on from where the last one ended
        torch._foreach_copy_([self.lens, self.free_start], [lens, start])
        return self.positions

    def attend(self, layer: int, Q, K, V, scale: float | None = None, window_size: int = 0):
        """Caches K and V [tokens, H_kv, d] of the step and returns (O, LSE) of Q [tokens, H, d]."""
        if self.slots is None:
            raise FaError(1, "slots: attend() before the first begin()")
        packed.fa_paged_write(K, V, self.slots, self.K[layer], self.V[layer])
        return packed.fa_paged_fwd(Q, self.K[layer], self.V[layer], self.block_table, self.cu_q, self.lens, scale=scale,
                                   causal=True, window_size=window_size)

    def release(self, row: int):
        """Gives the pages of request row `row` back; the row is empty afterwards (waits for the GPU)."""
        held = -(-int(self.lens[row]) // self.page_size)
        pages = self.block_table[row, :held]
        # the unused end of the list, the row's pages behind it, in a list of the same length
        unused = self.free_pages[int(self.free_start):]
        back = torch.cat([unused, pages[pages >= 0]])
        self.free_pages[self.free_pages.numel() - back.numel():] = back
        self.free_start.fill_(self.free_pages.numel() - back.numel())
        self.block_table[row] = -1
        self.lens[row] = 0
