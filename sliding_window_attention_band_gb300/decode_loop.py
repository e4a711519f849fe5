"""A running batch that answers with the banded attention.

``DecodeLoop`` holds what a serving program keeps between steps -- the paged
cache, the block table, the free list, lengths, descriptors, workspace -- and
runs one step of it:

    loop = DecodeLoop(batch, h, hk, head_dim, w, max_new=4)
    loop.fill(qkv, n_new)               # prompts: into the cache
    loop.n_new.fill_(1)                 # one token for every request
    loop.qkv[:batch].copy_(projection)  # its Q, K, V heads side by side
    loop.step()                         # loop.out, loop.lse: rows loop.q_start[r] ..

A step needs no value on the host, so it can be captured once in a CUDA graph
and replayed.  Every computation is one of the library's calls: cache_slots,
rotary_append, band_decode (with ``norm`` norm_rotary_append; with ``bits=4``
rotary_append4, band_decode4).
"""
from __future__ import annotations

import operator

import torch

from . import cache4, norm as normed, serve


class DecodeLoop:
    """A batch of requests of h query and hk key heads under a window of ``w``
    keys on the left (dilation, ``n_sink`` leading global tokens), at most
    ``max_new`` tokens a request and step (one that adds more is left out of the
    step: its length stays, used[1] is not 0, the device status word says
    INVALID_ARG, its rows of the result mean nothing).  The blocks of a request are
    recycled as its window moves on, so the cache does not grow with the
    context.  Rotary positions turn the whole head unless ``rot_dim`` says
    less (0: none); ``turns`` and ``rotary_scale`` as rotary_frequencies gives
    them.  ``norm`` (a NormDesc; weights ``wq``, ``wk`` [head_dim], None: 1): queries
    and keys are normed first.  ``bits=4``: the cache holds K and V in 4 bits (codes
    Kc, Vc, scales Ks, Vs), head_dim a multiple of 32."""

    def __init__(self, batch, h, hk, head_dim, w, dilation=0, n_sink=0, max_new=1, page=64, rot_dim=None, turns=None,
                 rotary_scale=1.0, dtype=torch.bfloat16, device="cuda", bits=None, norm=None, wq=None, wk=None):
        if bits not in (None, 4):
            raise ValueError(f"bits: expected 4, or None for a cache of the tensors' type, got {bits!r}")
        for name, x in (("wq", wq), ("wk", wk)):
            if x is not None and (norm is None or x.dtype is not dtype or x.shape != (head_dim,)):
                raise ValueError(f"{name}: expected [{head_dim}] {dtype} with a norm, got {list(x.shape)} {x.dtype}")
        self.bits, self.norm = bits, norm
        self.batch, self.h, self.hk, self.head_dim, self.dtype = batch, h, hk, head_dim, dtype
        self.rot_dim, self.rotary_scale = head_dim if rot_dim is None else rot_dim, rotary_scale
        pinned = -(-n_sink // page)
        cols = pinned + -(-(w * (dilation + 1) + max_new - 1) // page) + 1
        self.cache = serve.CacheDesc(batch, page, batch * cols, cols, ring=True, pinned=pinned, max_new=max_new)
        self._prompts = serve.CacheDesc(batch, page, batch * cols, cols, ring=True, pinned=pinned, max_new=(1 << 31) - 1)
        if self.rot_dim and turns is None:
            turns, _ = serve.rotary_frequencies(self.rot_dim)
        if self.rot_dim and (turns.dtype is not torch.int64 or turns.shape != (self.rot_dim // 2,)):
            raise ValueError(f"turns: expected {self.rot_dim // 2} int64 values (rotary_frequencies), got {tuple(turns.shape)} "
                             f"{turns.dtype}")
        self.tokens = batch * max_new
        self._rotary = serve.RotaryDesc(1, self.tokens, h, hk, head_dim, self.rot_dim, scale=self.rotary_scale, dtype=dtype)
        self._decode = serve.DecodeDesc(self.cache, self.tokens, h, hk, head_dim, w=w, dilation=dilation, n_sink=n_sink,
                                        max_q=max_new, max_len=1 << 30, dtype=dtype)
        # (what the calls of a step would refuse is refused here: there the lengths would have moved on)
        serve.check_step(self.cache, self._rotary, self._decode)
        normed.check_norm(self._rotary, norm)
        cache4.check_step4(self.cache, self._rotary, self._decode, bits)
        self.turns = turns.contiguous().to(device) if self.rot_dim else None
        i32 = dict(dtype=torch.int32, device=device)
        new = dict(dtype=dtype, device=device)
        self.wq, self.wk = (None if x is None else x.contiguous().to(device) for x in (wq, wk))
        # (a slice of a larger tensor may start where the calls refuse it)
        self.wq, self.wk = (x.clone() if x is not None and x.data_ptr() % 16 else x for x in (self.wq, self.wk))
        if bits == 4:
            codes, scales = cache4.cache4_shapes(self.cache, hk, head_dim)
            self.Kc, self.Vc = (torch.zeros(codes, dtype=torch.uint8, device=device) for _ in range(2))
            self.Ks, self.Vs = (torch.zeros(scales, **new) for _ in range(2))
        else:
            self.Kc = torch.zeros(batch * cols, hk, page, head_dim, **new)
            self.Vc = torch.zeros_like(self.Kc)
        self.table = torch.full((batch, cols), -1, **i32)
        self.free_list = torch.arange(batch * cols, **i32)
        self.lens, self.used, self.q_start = torch.zeros(batch, **i32), torch.zeros(2, **i32), torch.zeros(batch + 1, **i32)
        self.n_new = torch.zeros(batch, **i32)
        self.slots, self.pos = torch.zeros(self.tokens, **i32), torch.zeros(self.tokens, **i32)
        self.qkv = torch.zeros(self.tokens, h + 2 * hk, head_dim, **new)
        self.q = torch.zeros(self.tokens, h, head_dim, **new)
        self.out = torch.zeros_like(self.q)
        self.lse = torch.zeros(self.tokens, h, dtype=torch.float32, device=device)
        need = cache4.band_decode4_workspace(self._decode) if bits == 4 else serve.band_decode_workspace(self._decode)
        self.workspace = torch.empty(need, dtype=torch.uint8, device=device) if need else None
        self.scale = head_dim ** -0.5

    def _place(self, cache, n_new, slots, pos):
        serve.cache_slots(cache, self.lens, n_new, self.table, self.free_list, self.used, self.lens, self.used, self.q_start,
                          slots, pos)

    def _append(self, d, qkv, pos, slots, out):
        q, k, v = qkv.split([self.h, self.hk, self.hk], dim=1)
        if self.bits == 4:
            cache4.rotary_append4(d, self.cache, self.turns, q, k, v, pos, slots, out, self.Kc, self.Ks, self.Vc, self.Vs, self.norm,
                                  self.wq, self.wk)
        elif self.norm is not None:
            normed.norm_rotary_append(d, self.norm, self.cache, self.turns, q, k, v, pos, slots, out, self.Kc, self.Vc, self.wq, self.wk)
        else:
            serve.rotary_append(d, self.cache, self.turns, q, k, v, pos, slots, out, self.Kc, self.Vc)

    def fill(self, qkv, n_new):
        """Prompts of n_new[r] tokens (int32 [batch]) into the cache: the rows of
        qkv [tokens, h + 2 hk, head_dim] request by request, at least as many as
        n_new adds up to (read from the device, unless the stream is being
        captured).  Returns the rotated queries [tokens, h, head_dim]; their
        attention over the whole prompt is left to the caller (band_attention
        where it takes the heads: hk = h and, in 16 bits, head_dim 64)."""
        T = qkv.shape[0]
        # (a refusal must come before the lengths move on)
        if T < 1 or qkv.shape[1:] != self.qkv.shape[1:] or qkv.dtype is not self.dtype or qkv.device != self.qkv.device:
            raise ValueError(f"qkv: expected [tokens, {self.h + 2 * self.hk}, {self.head_dim}] {self.dtype} on {self.qkv.device}, "
                             f"got {list(qkv.shape)} {qkv.dtype} on {qkv.device}")
        if qkv.stride(2) != 1 or qkv.stride(0) * qkv.element_size() % 16 or qkv.stride(1) * qkv.element_size() % 16 \
                or qkv.data_ptr() % 16:
            raise ValueError(f"qkv: adjacent channels and rows on 16 bytes expected, got strides {qkv.stride()}")
        captured = n_new.is_cuda and torch.cuda.is_current_stream_capturing()
        if not captured and int(n_new.clamp(min=0).sum()) > T:
            raise ValueError(f"n_new: adds up to more than the {T} rows of qkv")
        slots, pos = torch.empty(T, dtype=torch.int32, device=qkv.device), torch.empty(T, dtype=torch.int32, device=qkv.device)
        self._place(self._prompts, n_new, slots, pos)
        d = serve.RotaryDesc(1, T, self.h, self.hk, self.head_dim, self.rot_dim, scale=self.rotary_scale, dtype=self.dtype)
        out = torch.empty(T, self.h, self.head_dim, dtype=self.dtype, device=qkv.device)
        self._append(d, qkv, pos, slots, out)
        return out

    def step(self):
        """n_new[r] tokens for every request, their heads in the rows of ``qkv``;
        the attention in ``out`` and ``lse``."""
        self._place(self.cache, self.n_new, self.slots, self.pos)
        self._append(self._rotary, self.qkv, self.pos, self.slots, self.q)
        if self.bits == 4:
            cache4.band_decode4(self._decode, self.scale, self.q, self.Kc, self.Ks, self.Vc, self.Vs, self.table, self.lens, self.q_start,
                                self.out, self.lse, self.workspace)
            return
        serve.band_decode(self._decode, self.scale, self.q, self.Kc, self.Vc, self.table, self.lens, self.q_start, self.out,
                          self.lse, self.workspace)

    def restart(self, requests):
        """Empty the given requests (row numbers 0 .. batch - 1): their blocks go
        back to the free list.  Reads the number of blocks in use from the device."""
        wanted = sorted({operator.index(r) for r in requests})
        # (a negative number would name a row a second time and free its blocks twice)
        if wanted and not 0 <= wanted[0] <= wanted[-1] < self.batch:
            raise ValueError(f"requests: expected row numbers 0 .. {self.batch - 1}, got {wanted}")
        rows = torch.tensor(wanted, dtype=torch.long, device=self.table.device)
        held = self.table[rows]
        left = torch.cat((self.free_list[int(self.used[0]):], held[held >= 0]))
        start = self.free_list.numel() - left.numel()
        self.free_list[start:] = left
        self.used[0] = start
        self.table[rows] = -1
        self.lens[rows] = 0

    @classmethod
    def from_workload(cls, wl, batch=None, device="cuda", **more):
        """The loop that carries a named workload's sequences on: its heads,
        window on the left, dilation and global tokens, which have to be the
        leading ones.  ``more``: bits, norm, wq, wk."""
        n_sink = len(set(wl.global_idx))
        if sorted(set(wl.global_idx)) != list(range(n_sink)):
            raise ValueError(f"global tokens other than the leading ones: {tuple(wl.global_idx)}")
        return cls(wl.b if batch is None else batch, wl.h, wl.h, wl.head_dim, wl.w, wl.dilation, n_sink, dtype=wl.dtype, device=device,
                   **more)
