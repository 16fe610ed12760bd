"""Ragged batches over an 8-bit paged KV cache: the operators of
include/bytecross.h's section of that name on torch tensors, and RaggedCache,
which owns the buffers of such a cache.

Types, shapes and devices are checked here (ValueError), sizes and alignment
by the library (BCError).  A call runs on the given stream or on the current
stream of the tensors' device, whichever device is current, and does not wait.
"""
from __future__ import annotations

import ctypes as C

import torch

from . import (BC_BF16, BC_F32, KV8_TYPES, bc_block_tables, bc_block_tables_args, bc_kv8_append, bc_kv8_attention,
               bc_kv8_attention_args, bc_kv8_attention_scratch_bytes, bc_kv8_attention_status, bc_kv8_gather,
               bc_kv8_pool_bytes, bc_logits_adjust, bc_logits_args, check)

_DTYPES = {torch.float32: BC_F32, torch.bfloat16: BC_BF16}
_BLOCKS = {32 * hd + 32: hd for hd in (64, 128)}       # block bytes -> head_dim


_I32, _F32, _U8 = torch.int32, torch.float32, torch.uint8


# A call's checks are one expression over _is(); only when it fails do the
# checks below go through the arguments one by one to say which is wrong.
def _is(t, dtype, dev, n):
    """A contiguous tensor of dtype with n entries on device number dev."""
    return t.dtype is dtype and t.get_device() == dev and t.numel() == n and t.is_contiguous()


def _dense(who, dev, dtype, **tensors):
    """Raises for a tensor that is not contiguous, of dtype and on device
    number dev; None passes."""
    for name, t in tensors.items():
        if t is not None and (t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous()):
            raise ValueError(f"{who}: {name} must be a contiguous {dtype} tensor on cuda:{dev}")


def _sizes(who, **pairs):
    for name, (t, n) in pairs.items():
        if t is not None and t.numel() != n:
            raise ValueError(f"{who}: {name} must have {n} entries, not {t.numel()}")


def _dtype(who, t):
    try:
        return _DTYPES[t.dtype]
    except KeyError:
        raise ValueError(f"{who}: float32 or bfloat16 expected, not {t.dtype}") from None


def _code(who, code):
    try:
        return KV8_TYPES[code]
    except KeyError:
        raise ValueError(f"{who}: code must be one of {sorted(KV8_TYPES)}, not {code!r}") from None


def _pool(who, pool):
    """(n_pages, n_kv_heads, head_dim, device number) of a pool tensor."""
    if pool.dtype is not torch.uint8 or pool.dim() != 3 or not pool.is_cuda or not pool.is_contiguous() \
            or pool.shape[2] not in _BLOCKS:
        raise ValueError(f"{who}: the pool must be a contiguous CUDA uint8 tensor "
                         "[n_pages][n_kv_heads][32 head_dim + 32], head_dim 64 or 128")
    P, H, block = pool.shape
    return P, H, _BLOCKS[block], pool.get_device()


def _fits(who, *ints):
    """The argument blocks hold 32-bit integers; ctypes would cut longer ones."""
    if max(ints) > 0x7fffffff or min(ints) < -0x80000000:
        raise ValueError(f"{who}: a size beyond 2^31 - 1 ({ints})")


def _ptr(t):
    return None if t is None else t.data_ptr()


def _call(dev, stream, where, fn, *args):
    """fn(*args, stream) with device number dev current."""
    if torch._C._cuda_getDevice() != dev:
        with torch.cuda.device(dev):
            return _call(dev, stream, where, fn, *args)
    s = torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream
    check(fn(*args, s), where)


def block_tables(lens, delta, table, free_list, n_free, lens_out, n_free_out, q_start, slots, positions, ticket,
                 stream=None):
    """bc_block_tables: the plan of one step of a ragged batch.  int32 CUDA
    tensors: lens, delta, lens_out [B], table [B][max_blocks], free_list
    [n_pages], n_free, n_free_out, ticket [1], q_start [B + 1], slots and
    positions [max_tokens]."""
    who = "block_tables"
    if not table.is_cuda or table.dim() != 2:
        raise ValueError(f"{who}: table must be a CUDA tensor [batch][max_blocks]")
    dev = table.get_device()
    B, max_blocks = table.shape
    n, n_pages = slots.numel(), free_list.numel()
    if not (_is(lens, _I32, dev, B) and _is(delta, _I32, dev, B) and _is(table, _I32, dev, B * max_blocks)
            and _is(free_list, _I32, dev, n_pages) and _is(n_free, _I32, dev, 1) and _is(lens_out, _I32, dev, B)
            and _is(n_free_out, _I32, dev, 1) and _is(q_start, _I32, dev, B + 1) and _is(slots, _I32, dev, n)
            and _is(positions, _I32, dev, n) and _is(ticket, _I32, dev, 1)):
        _dense(who, dev, _I32, lens=lens, delta=delta, table=table, free_list=free_list, n_free=n_free,
               lens_out=lens_out, n_free_out=n_free_out, q_start=q_start, slots=slots, positions=positions,
               ticket=ticket)
        _sizes(who, lens=(lens, B), delta=(delta, B), lens_out=(lens_out, B), q_start=(q_start, B + 1),
               n_free=(n_free, 1), n_free_out=(n_free_out, 1), ticket=(ticket, 1), positions=(positions, n))
    _fits(who, B, max_blocks, n_pages, n)
    a = bc_block_tables_args(B, max_blocks, n_pages, n, lens.data_ptr(), delta.data_ptr(),
                             table.data_ptr(), free_list.data_ptr(), n_free.data_ptr(), lens_out.data_ptr(),
                             n_free_out.data_ptr(), q_start.data_ptr(), slots.data_ptr(), positions.data_ptr(),
                             ticket.data_ptr())
    _call(dev, stream, "bc_block_tables", bc_block_tables, C.byref(a))


def _rows(who, dev, shape, t, name, dtype):
    """Checks an [n][H][hd] tensor whose heads and dims are dense."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev:
        raise ValueError(f"{who}: {name} must be {dtype} {list(shape)} on cuda:{dev}")
    if not t.is_contiguous() and t.numel() and (t.stride(2) != 1 or (shape[1] > 1 and t.stride(1) != shape[2])):
        raise ValueError(f"{who}: heads and dims of {name} must be dense")


def kv8_append(k, v, slots, pool, code="e4m3", stream=None):
    """bc_kv8_append: k, v f32 or bf16 [n][n_kv_heads][hd], heads and dims
    dense (a token's stride is free); slots int32 [n]; pool uint8
    [n_pages][n_kv_heads][32 hd + 32]."""
    who = "kv8_append"
    P, H, hd, dev = _pool(who, pool)
    n = slots.numel()
    if not _is(slots, _I32, dev, n):
        _dense(who, dev, _I32, slots=slots)
    dt, typ = _dtype(who, k), _code(who, code)
    _rows(who, dev, (n, H, hd), k, "k", k.dtype)
    _rows(who, dev, (n, H, hd), v, "v", k.dtype)
    if n == 0:
        return
    ks, vs = (k.stride(0), v.stride(0)) if n > 1 else (H * hd, H * hd)
    _call(dev, stream, "bc_kv8_append", bc_kv8_append, k.data_ptr(), v.data_ptr(), dt, ks, vs, slots.data_ptr(), n,
          pool.data_ptr(), typ, P, H, hd)


def kv8_gather(pool, slots, k_out, v_out, code="e4m3", stream=None):
    """bc_kv8_gather: k_out, v_out f32 or bf16 [n][n_kv_heads][hd], contiguous,
    receive the tokens at slots (int32 [n])."""
    who = "kv8_gather"
    P, H, hd, dev = _pool(who, pool)
    n = slots.numel()
    if not _is(slots, _I32, dev, n):
        _dense(who, dev, _I32, slots=slots)
    dt, typ = _dtype(who, k_out), _code(who, code)
    _rows(who, dev, (n, H, hd), k_out, "k_out", k_out.dtype)
    _rows(who, dev, (n, H, hd), v_out, "v_out", k_out.dtype)
    if not (k_out.is_contiguous() and v_out.is_contiguous()):
        raise ValueError(f"{who}: k_out and v_out must be contiguous")
    if n == 0:
        return
    _call(dev, stream, "bc_kv8_gather", bc_kv8_gather, pool.data_ptr(), typ, P, H, hd, slots.data_ptr(), n,
          k_out.data_ptr(), v_out.data_ptr(), dt)


def kv8_attention(q, pool, lens, table, out, scratch, code="e4m3", q_start=None, max_q=1, pages=None, n_sel=None,
                  scale=None, cap=0.0, window=0, slopes=None, stream=None):
    """bc_kv8_attention: q f32 or bf16 [n_q][Hq][hd], heads and dims dense (a
    row's stride is free), out of the same type and shape, contiguous; lens
    int32 [B]; table int32 [B][max_blocks]; q_start int32 [B + 1] or None (one
    query a sequence); pages int32 [B][n_kv_heads][max_sel] with n_sel int32
    [B], or None; slopes f32 [Hq] or None; scale None for 1 / sqrt(hd); scratch
    uint8 of bc_kv8_attention_scratch_bytes(B, n_kv_heads, group, max_q, hd)
    bytes, zeroed before its first use."""
    who = "kv8_attention"
    P, H, hd, dev = _pool(who, pool)
    if q.dim() != 3 or q.shape[1] % H or q.shape[1] == 0:
        raise ValueError(f"{who}: q must be [n_q][a multiple of {H}][{hd}]")
    n_q, Hq, _ = q.shape
    dt, typ = _dtype(who, q), _code(who, code)
    _rows(who, dev, (n_q, Hq, hd), q, "q", q.dtype)
    _rows(who, dev, (n_q, Hq, hd), out, "out", q.dtype)
    if table.dim() != 2:
        raise ValueError(f"{who}: table must be [batch][max_blocks]")
    B, max_blocks = table.shape
    if not (out.is_contiguous() and _is(lens, _I32, dev, B) and _is(table, _I32, dev, B * max_blocks)
            and scratch.dtype is _U8 and scratch.get_device() == dev and scratch.is_contiguous()
            and (q_start is None or _is(q_start, _I32, dev, B + 1)) and (n_sel is None or _is(n_sel, _I32, dev, B))
            and (pages is None or (pages.dtype is _I32 and pages.get_device() == dev and pages.is_contiguous()))
            and (slopes is None or _is(slopes, _F32, dev, Hq))):
        _dense(who, dev, q.dtype, out=out)
        _dense(who, dev, _I32, lens=lens, table=table, q_start=q_start, pages=pages, n_sel=n_sel)
        _dense(who, dev, _U8, scratch=scratch)
        _dense(who, dev, _F32, slopes=slopes)
        _sizes(who, lens=(lens, B), q_start=(q_start, B + 1), n_sel=(n_sel, B), slopes=(slopes, Hq))
    if q_start is None and (max_q != 1 or n_q != B):
        raise ValueError(f"{who}: without q_start there is one query row per sequence")
    max_sel = 0
    if (pages is None) != (n_sel is None):
        raise ValueError(f"{who}: pages and n_sel go together")
    if pages is not None:
        if pages.dim() != 3 or pages.shape[0] != B or pages.shape[1] != H or pages.shape[2] == 0:
            raise ValueError(f"{who}: pages must be [batch][n_kv_heads][max_sel], max_sel at least 1")
        max_sel = pages.shape[2]
    _fits(who, n_q, B, max_blocks, max_sel, max_q, window)
    if cap and abs(cap) < 2.0 ** -126:                    # in 32 bits some of these are 0, which means none
        raise ValueError(f"{who}: cap must be 0 or a positive normal number, not {cap}")
    if n_q == 0:
        return
    a = bc_kv8_attention_args(q.data_ptr(), out.data_ptr(), dt, q.stride(0) if n_q > 1 else Hq * hd, n_q,
                              pool.data_ptr(), typ, P, H, Hq // H, hd, B, max_q, max_blocks, max_sel, lens.data_ptr(),
                              _ptr(q_start), table.data_ptr(), _ptr(pages), _ptr(n_sel),
                              hd ** -0.5 if scale is None else scale, cap, window, _ptr(slopes), scratch.data_ptr(),
                              scratch.numel())
    _call(dev, stream, "bc_kv8_attention", bc_kv8_attention, C.byref(a))


def logits_adjust(logits, out, hist=None, hist_start=None, prompt_len=None, repetition=None, frequency=None,
                  presence=None, bias_ids=None, bias_vals=None, bias_start=None, mask=None, mask_row=None,
                  stream=None):
    """bc_logits_adjust: logits f32 or bf16 [B][V] (a row's stride is free),
    out of the same type and shape (logits itself for an update in place);
    hist, bias_ids int32 with hist_start, bias_start int32 [B + 1]; prompt_len,
    mask_row int32 [B]; repetition, frequency, presence f32 [B]; bias_vals f32;
    mask int32 [n_masks][ceil(V / 32)]."""
    who = "logits_adjust"
    if not logits.is_cuda or logits.dim() != 2:
        raise ValueError(f"{who}: logits must be a CUDA tensor [B][V]")
    dev, dt = logits.get_device(), _dtype(who, logits)
    B, V = logits.shape
    if out.get_device() != dev or out.dtype is not logits.dtype or out.shape != logits.shape:
        raise ValueError(f"{who}: out must have the type, shape and device of logits")
    if V > 1 and (logits.stride(1) != 1 or out.stride(1) != 1):
        raise ValueError(f"{who}: rows of logits and out must be dense")
    if (hist is None) != (hist_start is None):
        raise ValueError(f"{who}: hist and hist_start go together")
    if not (bias_ids is None) == (bias_vals is None) == (bias_start is None):
        raise ValueError(f"{who}: bias_ids, bias_vals and bias_start go together")
    if mask is None and mask_row is not None:
        raise ValueError(f"{who}: mask_row needs mask")
    n_hist = 0 if hist is None else hist.numel()
    n_bias = 0 if bias_ids is None else bias_ids.numel()
    n_masks = 0
    if mask is not None:
        if mask.dim() != 2 or mask.shape[1] != (V + 31) // 32:
            raise ValueError(f"{who}: mask must be [n_masks][{(V + 31) // 32}]")
        n_masks = mask.shape[0]
        if mask_row is None and B > n_masks == 0:       # an empty tensor has no address: no masks at all
            raise ValueError(f"{who}: without mask_row there is a mask for each of the {B} rows, not 0")
    if not ((hist is None or (_is(hist, _I32, dev, n_hist) and _is(hist_start, _I32, dev, B + 1)))
            and (bias_ids is None or (_is(bias_ids, _I32, dev, n_bias) and _is(bias_vals, _F32, dev, n_bias)
                                      and _is(bias_start, _I32, dev, B + 1)))
            and (prompt_len is None or _is(prompt_len, _I32, dev, B))
            and (repetition is None or _is(repetition, _F32, dev, B))
            and (frequency is None or _is(frequency, _F32, dev, B))
            and (presence is None or _is(presence, _F32, dev, B))
            and (mask is None or (mask.dtype is _I32 and mask.get_device() == dev and mask.is_contiguous()))
            and (mask_row is None or _is(mask_row, _I32, dev, B))):
        _dense(who, dev, _I32, hist=hist, hist_start=hist_start, prompt_len=prompt_len, bias_ids=bias_ids,
               bias_start=bias_start, mask=mask, mask_row=mask_row)
        _dense(who, dev, _F32, repetition=repetition, frequency=frequency, presence=presence, bias_vals=bias_vals)
        _sizes(who, hist_start=(hist_start, B + 1), bias_start=(bias_start, B + 1), prompt_len=(prompt_len, B),
               mask_row=(mask_row, B), repetition=(repetition, B), frequency=(frequency, B), presence=(presence, B),
               bias_vals=(bias_vals, n_bias))
    _fits(who, B, V, n_hist, n_bias, n_masks)
    if B == 0 or V == 0:
        return
    a = bc_logits_args(logits.data_ptr(), out.data_ptr(), dt, B, V, logits.stride(0) if B > 1 else V,
                       out.stride(0) if B > 1 else V, _ptr(hist), _ptr(hist_start), _ptr(prompt_len), n_hist,
                       _ptr(repetition), _ptr(frequency), _ptr(presence), _ptr(bias_ids), _ptr(bias_vals),
                       _ptr(bias_start), n_bias, _ptr(mask), _ptr(mask_row), n_masks)
    _call(dev, stream, "bc_logits_adjust", bc_logits_adjust, C.byref(a))


class RaggedCache:
    """An 8-bit paged KV cache of `layers` layers that a batch of sequences of
    different lengths shares: owns the pools, block tables, free list and the
    step's plan (allocated with torch).  Per step: plan(delta), then per layer
    append(layer, k, v) and attend(layer, q, out).  Everything stays on the
    device, so a step can be captured into a graph.  Its methods share one
    scratch and its buffers are filled on the current stream when it is made:
    calls on several streams have to be ordered by the caller."""

    def __init__(self, layers: int, batch: int, n_pages: int, n_kv_heads: int, group: int, head_dim: int,
                 max_blocks: int, max_tokens: int, max_q: int = 1, code: str = "e4m3", device="cuda"):
        _code("RaggedCache", code)
        layer_bytes = bc_kv8_pool_bytes(n_pages, n_kv_heads, head_dim)
        scratch = bc_kv8_attention_scratch_bytes(batch, n_kv_heads, group, max_q, head_dim)
        if not (layer_bytes and scratch) or layers < 1 or max_blocks < 1 or max_tokens < 1:
            raise ValueError("bad sizes for an 8-bit ragged cache")
        self.layers, self.batch, self.group, self.max_q, self.code = layers, batch, group, max_q, code
        ints = lambda *s: torch.zeros(*s, dtype=torch.int32, device=device)
        self.pool = torch.empty(layers, n_pages, n_kv_heads, 32 * head_dim + 32, dtype=torch.uint8, device=device)
        self._pools = self.pool.unbind(0)
        self.table, self.lens, self.q_start = ints(batch, max_blocks), ints(batch), ints(batch + 1)
        self.free_list = torch.arange(n_pages, dtype=torch.int32, device=device)
        self.n_free = ints(1).fill_(n_pages)
        self.slots, self.positions, self.ticket = ints(max_tokens), ints(max_tokens), ints(1)
        self.scratch = torch.zeros(scratch, dtype=torch.uint8, device=device)

    def plan(self, delta, stream=None):
        """delta int32 [batch]: tokens each sequence takes (or, negative,
        drops); updates lens, table, free_list, q_start, slots, positions.  A
        dropped token's effect on the scales of a page that other tokens of
        its sequence keep stays: a rejected draft with an outlier leaves coarser
        codes there, one that is not finite NaN."""
        block_tables(self.lens, delta, self.table, self.free_list, self.n_free, self.lens, self.n_free, self.q_start,
                     self.slots, self.positions, self.ticket, stream)

    def append(self, layer: int, k, v, stream=None):
        """k, v [n][n_kv_heads][hd] of the step's new tokens in the plan's
        order; rows behind the last one do not reach the cache."""
        n = k.shape[0]
        if n > self.slots.numel():
            raise ValueError(f"RaggedCache.append: more than {self.slots.numel()} tokens")
        slots = self.slots if n == self.slots.numel() else self.slots[:n]
        kv8_append(k, v, slots, self._pools[layer], self.code, stream)

    def attend(self, layer: int, q, out, stream=None, **options):
        """q [n_q][Hq][hd], the queries of the step's new tokens; options as
        for kv8_attention.  Of a sequence with more than max_q of them (a prompt)
        only the first max_q rows of out are written, as kv8_attention has it;
        rows behind the plan's last token may pad q."""
        kv8_attention(q, self._pools[layer], self.lens, self.table, out, self.scratch, self.code, self.q_start,
                      self.max_q, stream=stream, **options)

    def read(self, layer: int, seq: int, n: int, dtype=torch.bfloat16):
        """The first n tokens of a sequence as (k, v), each [n][n_kv_heads][hd],
        on the current stream; zeros behind its last one."""
        H, hd = self.pool.shape[2], (self.pool.shape[3] - 32) // 32
        if not 0 <= n <= 16 * self.table.shape[1]:
            raise ValueError("RaggedCache.read: n outside the sequence's table")
        dev = self.pool.device
        pos = torch.arange(n, device=dev)
        slots = torch.where(pos < self.lens[seq], self.table[seq][pos // 16] * 16 + pos % 16, -1).int()
        k = torch.empty(n, H, hd, dtype=dtype, device=dev)
        v = torch.empty_like(k)
        kv8_gather(self._pools[layer], slots, k, v, self.code)
        return k, v

    def status(self, stream=None):
        """Waits for the stream; raises if a wait of an attention gave up."""
        _call(self.pool.get_device(), stream, "bc_kv8_attention_status", bc_kv8_attention_status,
              self.scratch.data_ptr())
