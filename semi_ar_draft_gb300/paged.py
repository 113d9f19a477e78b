"""A paged key-value cache for the verify step, over the calls of `api`.

The cache of `requests` slots lives in pools of pages shared by all layers' tables: one block table, one page
stack, and per layer a pool of keys and one of values.  A round is

    plan(new_len, extra)      pages, slots and offsets of the step's new tokens
    append(layer, k, v)       a layer's new keys and values into their slots
    attend(layer, q)          a layer's attention of the new tokens
    commit(add_len, extra)    how many of them stay; pages past them go back

and nothing in it reads the device from the host.  plan and commit write their results to other tensors than
they read: plan goes from what the last commit left to what the next one reads, and commit writes there too.  So every
call reads the same addresses, and any sequence of calls can be captured into a graph and replayed; a plan that no
commit has followed is replaced by the next."""
from __future__ import annotations

import contextlib

import torch

from . import api
from . import binding as b


def _on(stream):
    """torch's current stream made the given one; None leaves it."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(b.torch_stream(stream))


class PagedCache:
    """requests slots of at most max_blocks pages each; num_pages pages of page_size tokens in all; max_tokens:
    the most new tokens of any step (a step may say that it has fewer: plan's tokens).  kv_dtype: dtype or
    torch.float8_e4m3fn, then with k_scale, v_scale [layers, Hk] fp32 (ones if not given)."""

    def __init__(self, requests, num_pages, page_size, max_blocks, layers, Hk, D, max_tokens, dtype=torch.bfloat16,
                 kv_dtype=None, k_scale=None, v_scale=None, device="cuda"):
        i32 = {"dtype": torch.int32, "device": device}
        shape = (layers, num_pages, page_size, Hk, D)
        self.k_pages = torch.zeros(shape, dtype=kv_dtype or dtype, device=device)
        self.v_pages = torch.zeros_like(self.k_pages)
        if kv_dtype == torch.float8_e4m3fn:
            ones = torch.ones((layers, Hk), device=device)
            k_scale, v_scale = (ones if s is None else s for s in (k_scale, v_scale))
        self.k_scale = [None] * layers if k_scale is None else k_scale
        self.v_scale = [None] * layers if v_scale is None else v_scale
        self.page_size, self.max_tokens = page_size, max_tokens
        self.block_table = torch.full((requests, max_blocks), -1, **i32)
        self.free_pages = torch.arange(num_pages - 1, -1, -1, **i32)
        # lengths, blocks held, pages free: [0] now, [1] as the last commit left them
        self._counts = [torch.zeros(2 * requests + 1, **i32) for _ in range(2)]
        self._len, self._blocks, self._free = ([x[a:b] for x in self._counts] for a, b in
                                               ((0, requests), (requests, 2 * requests), (2 * requests, 2 * requests + 1)))
        for x in self._free:
            x.fill_(num_pages)
        self.seq_len, self.offsets = torch.empty(requests, **i32), torch.empty(requests + 1, **i32)
        self._slots = torch.empty(max_tokens, dtype=torch.int64, device=device)
        self._positions = torch.empty(max_tokens, **i32)
        self.slots, self.positions = self._slots, self._positions
        self.ws = torch.zeros(256, dtype=torch.uint8, device=device)
        self._error = torch.zeros(1, **i32)  # the first device error since status() was last called
        self.max_new = 0

    @property
    def cache_len(self):
        """Tokens of each request in the cache [requests] (the tensor stays; commit changes what it holds)."""
        return self._len[0]

    @property
    def n_free(self):
        return self._free[0]

    def plan(self, new_len=None, extra=0, max_new=0, stream=None, tokens=None):
        """Pages and slots for new_len[j] + extra tokens of each request.  Sets seq_len, offsets, slots, positions.
        tokens: the most new tokens of this step, max_tokens if not given: the rows of slots, positions and of what
        append and attend take until the next plan (few rows a step are then few rows to copy, and attend's choice
        of kernel goes by their mean).  max_new: the most new tokens of one request, if known (for that choice too)."""
        if tokens is None:
            tokens = self.max_tokens
        if not 0 <= tokens <= self.max_tokens:
            raise ValueError(f"a step of {tokens} tokens; the cache was made for {self.max_tokens}")
        if tokens != len(self.slots):
            self.slots, self.positions = self._slots[:tokens], self._positions[:tokens]
        api.cache_plan(self._len[0], new_len, self.block_table, self._blocks[1], self.free_pages, self._free[1],
                       self.page_size, tokens, extra=extra, ws=self.ws, stream=stream, error=self._error,
                       out=(self.seq_len, self.offsets, self.slots, self.positions, self._blocks[0], self._free[0]))
        self.max_new = max_new

    def append(self, layer, k, v, stream=None):
        """k, v [the plan's tokens, Hk, D]: rows past offsets[-1] have no slot and are skipped."""
        api.cache_append(k, v, self.k_pages[layer], self.v_pages[layer], self.slots, self.k_scale[layer], self.v_scale[layer],
                         stream)

    def attend(self, layer, q, stream=None, **kw):
        """q [the plan's tokens, Hq, D]; kw as for api.paged_attention.  Returns (out, lse or None)."""
        out, lse, _ = api.paged_attention(q, self.k_pages[layer], self.v_pages[layer], self.block_table, self.seq_len,
                                          self.offsets, k_scale=self.k_scale[layer], v_scale=self.v_scale[layer],
                                          max_new=self.max_new, stream=stream, error=self._error, **kw)
        return out, lse

    def commit(self, add_len=None, extra=0, done=None, stream=None):
        """Keeps add_len[j] + extra of each request's new tokens (none of the whole request where done)."""
        api.cache_commit(self._len[0], add_len, self.block_table, self._blocks[0], self.free_pages, self._free[0],
                         self.page_size, extra=extra, done=done, ws=self.ws, stream=stream, error=self._error,
                         out=(self._len[1], self._blocks[1], self._free[1]), settled=self._counts[0])

    def status(self, stream=None):
        """The first device error of plan, attend and commit since this was last called, 0 if there was none
        (synchronises the stream; calls made on others count once they have run)."""
        code = b.dspark_get_device_status(self._error, stream)
        if code:
            with _on(stream):
                self._error.zero_()
        return code
