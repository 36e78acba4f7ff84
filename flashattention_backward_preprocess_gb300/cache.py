"""A paged key/value cache over the library's paged calls: pages, tables and lengths of a fixed
set of request rows, for any number of attention layers.

One step of a model, for the new tokens of all requests (one each, or chunks of prompts):

    cache.begin(cu_q, tokens)                      # fa_page_slots: pages, slots, positions
    for layer in range(layers):
        O, LSE = cache.attend(layer, Q, K, V)      # fa_paged_write, fa_paged_fwd
With drafted tokens (a tree for each request: begin()'s `parents`) the step ends once the accepted
ones are known:
    cache.accept(path, count)                      # fa_paged_keep, fa_page_trim
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

    quantised: the cache holds 8-bit rows (fa_paged_write_q8), K_exp and V_exp their exponents
    [num_pages, H_kv, page_size] in each layer; `dtype` is not used then, the steps' tensors have
    their own.  attend() chooses its kernel by the step's tokens per row then, idle rows included, so these
    do have a price in steps of prompts (one of 512 tokens over 8000 cached ones: 99 us with one row, 466
    with 64), and with 512 / (heads of a group) tokens per row or more it takes scratch for all that the
    tables have room for, 4 GB at most (fa_paged_workspace_bytes_ex).
    """

    def __init__(self, layers: int, num_pages: int, page_size: int, H_kv: int, d: int, rows: int, max_pages: int,
                 dtype=torch.bfloat16, device="cuda", quantised: bool = False):
        i32 = dict(dtype=torch.int32, device=device)
        self.page_size = int(page_size)
        self.K_exp = self.V_exp = None
        if quantised:
            dtype = torch.float8_e4m3fn
            self.K_exp, self.V_exp = ([torch.zeros(num_pages, H_kv, page_size, dtype=torch.uint8, device=device)
                                       for _ in range(layers)] for _ in "KV")
        self.K = [torch.zeros(num_pages, page_size, H_kv, d, dtype=dtype, device=device) for _ in range(layers)]
        self.V = [torch.zeros_like(k) for k in self.K]
        self.block_table = torch.full((rows, max_pages), -1, **i32)
        self.lens = torch.zeros(rows, **i32)
        self.free_pages = torch.arange(num_pages, **i32)
        self.free_start = torch.zeros(1, **i32)
        self.cu_q = self.slots = self.positions = self.tree = None

    def begin(self, cu_q, tokens: int, parents=None, words: int | None = None):
        """Takes the pages of the step's new tokens (int32 offsets cu_q [rows + 1], `tokens` rows in
        the step's tensors, padding behind cu_q[rows] included) and returns their positions.

        parents (int32 [tokens]): each request's new tokens are a tree, token i following the token
        parents[i] of the same request (an earlier one, counted from its first new token) or, at -1,
        the cached ones; its position counts its ancestors (attend() takes no window then).  words:
        64 tokens of the largest tree each (as many as the step's tokens may need unless given: a token's
        mask takes 8 bytes each, so give it where many requests share a step)."""
        # whatever is refused is refused before anything changes
        tree = depth = None
        if parents is not None:
            if parents.numel() != tokens:
                raise FaError(1, f"parents: expected one for each of {tokens} tokens, got {parents.numel()}")
            words = min(max(-(-int(tokens) // 64), 1), 1024) if words is None else words
            tree, depth = packed.fa_tree_mask(parents, cu_q, self.lens, words)
        self.slots, self.positions, lens, start = packed.fa_page_slots(
            self.lens, cu_q, self.block_table, self.free_pages, self.free_start, self.page_size, tokens)
        self.cu_q, self.tree = cu_q, tree
        if tree is not None:
            self.positions = depth
        # in place: the replays of a captured step go on from where the last one ended
        torch._foreach_copy_([self.lens, self.free_start], [lens, start])
        return self.positions

    def attend(self, layer: int, Q, K, V, scale: float | None = None, window_size: int = 0):
        """Caches K and V [tokens, H_kv, d] of the step and returns (O, LSE) of Q [tokens, H, d]."""
        if self.slots is None:
            raise FaError(1, "slots: attend() outside a step, begin() comes first")
        k_exp = v_exp = None
        if self.K_exp is None:
            packed.fa_paged_write(K, V, self.slots, self.K[layer], self.V[layer])
        else:
            k_exp, v_exp = self.K_exp[layer], self.V_exp[layer]
            packed.fa_paged_write_q8(K, V, self.slots, self.K[layer], self.V[layer], k_exp, v_exp)
        return packed.fa_paged_fwd(Q, self.K[layer], self.V[layer], self.block_table, self.cu_q, self.lens, scale=scale,
                                   causal=True, window_size=window_size, K_exp=k_exp, V_exp=v_exp, tree=self.tree)

    def accept(self, path, count):
        """Ends a step of drafted tokens: of request n's new tokens those numbered path[cu_q[n]] <
        path[cu_q[n] + 1] < ... (int32 [tokens], count[n] of them, from the request's first new token)
        stay, in this order; the others' pages are free again.  A request whose path or count does not fit
        keeps all its new tokens as they are, and fa_check_device() raises.  The next step begins with begin()."""
        if self.slots is None:
            raise FaError(1, "slots: accept() outside a step, begin() comes first")
        packed.fa_paged_keep(path, count, self.cu_q, self.lens, self.block_table, self.K, self.V, self.K_exp, self.V_exp)
        lens, start = packed.fa_page_trim(count, self.cu_q, self.lens, self.block_table, self.free_pages, self.free_start,
                                          self.page_size, path=path)
        torch._foreach_copy_([self.lens, self.free_start], [lens, start])
        self.slots = None

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
