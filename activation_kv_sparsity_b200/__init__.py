"""Python binding of libbytecross (the C ABI in include/bytecross.h).

Argument marshalling only: every step of the decode path runs in the CUDA
kernels of libbytecross.so.  PyTorch is used for device memory and streams.
There is no fallback: if the shared library is missing the import fails.
Build it with ``python activation_kv_sparsity_b200/build.py``.
"""
from __future__ import annotations

import ctypes as C
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libbytecross.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with `python activation_kv_sparsity_b200/build.py`")
_lib = C.CDLL(LIB_PATH)

# ------------------------------------------------------------------ enums
BC_OK, BC_EINVAL, BC_ENOMEM, BC_ECAPACITY, BC_ECUDA, BC_ETIMEOUT = range(6)
BC_DENSE, BC_ACT, BC_KV, BC_BOTH, BC_SNAP, BC_MASKED = range(6)
MODES = {"dense": BC_DENSE, "act": BC_ACT, "kv": BC_KV, "both": BC_BOTH, "snap": BC_SNAP, "masked": BC_MASKED}
(BC_TRACE_XN, BC_TRACE_SEL_QKV, BC_TRACE_Q, BC_TRACE_ATTN, BC_TRACE_SEL_O, BC_TRACE_XN2,
 BC_TRACE_SEL_GU, BC_TRACE_H, BC_TRACE_SEL_D, BC_TRACE_X, BC_TRACE_PAGE_SCORES, BC_TRACE_PAGES,
 BC_TRACE_QKV, BC_TRACE_SNAP_SCORES, BC_TRACE_SNAP_PAGES) = range(15)


class bc_config(C.Structure):
    _fields_ = [(n, C.c_int) for n in ("n_layers", "hidden", "intermediate", "n_heads", "n_kv_heads",
                                       "head_dim", "vocab", "max_ctx", "page")] + \
               [("rms_eps", C.c_float), ("rope_theta", C.c_float)]


class bc_weights(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("embed", "lm_head", "final_norm", "attn_norm", "mlp_norm",
                                          "wqkv_t", "wo_t", "wgu_t", "wd_t")]


BC_F32, BC_BF16 = range(2)
BC_KV8_E4M3, BC_KV8_INT8 = range(2)
KV8_TYPES = {"e4m3": BC_KV8_E4M3, "int8": BC_KV8_INT8}
BC_RAGGED_MAX_BATCH = 2048


class bc_block_tables_args(C.Structure):
    _fields_ = [(n, C.c_int) for n in ("batch", "max_blocks", "n_pages", "max_tokens")] + \
               [(n, C.c_void_p) for n in ("lens", "delta", "table", "free_list", "n_free", "lens_out", "n_free_out",
                                          "q_start", "slots", "positions", "ticket")]


class bc_kv8_attention_args(C.Structure):
    _fields_ = [("q", C.c_void_p), ("out", C.c_void_p), ("dtype", C.c_int), ("q_stride", C.c_longlong),
                ("n_q", C.c_int), ("pool", C.c_void_p)] + \
               [(n, C.c_int) for n in ("type", "n_pages", "n_kv_heads", "group", "head_dim", "batch", "max_q",
                                       "max_blocks", "max_sel")] + \
               [(n, C.c_void_p) for n in ("lens", "q_start", "table", "pages", "n_sel")] + \
               [("scale", C.c_float), ("cap", C.c_float), ("window", C.c_int), ("slopes", C.c_void_p),
                ("scratch", C.c_void_p), ("scratch_bytes", C.c_size_t)]


class bc_logits_args(C.Structure):
    _fields_ = [("logits", C.c_void_p), ("out", C.c_void_p), ("dtype", C.c_int), ("batch", C.c_int),
                ("vocab", C.c_int), ("stride", C.c_longlong), ("out_stride", C.c_longlong), ("hist", C.c_void_p),
                ("hist_start", C.c_void_p), ("prompt_len", C.c_void_p), ("n_hist", C.c_int)] + \
               [(n, C.c_void_p) for n in ("repetition", "frequency", "presence", "bias_ids", "bias_vals",
                                          "bias_start")] + \
               [("n_bias", C.c_int), ("mask", C.c_void_p), ("mask_row", C.c_void_p), ("n_masks", C.c_int)]


class bc_bytes(C.Structure):
    _fields_ = [(n, C.c_double) for n in (
        "weight_bytes", "head_bytes", "kv_bytes_per_token", "dense_bytes", "saved_bytes", "bound",
        "n_star", "n_star_ff", "impl_weight_bytes", "impl_head_bytes", "impl_kv_read_bytes",
        "impl_meta_read_bytes", "impl_kv_write_bytes", "impl_other_bytes", "impl_total_bytes")] + \
        [("pages_total", C.c_longlong), ("pages_kept", C.c_longlong)]


_P = C.c_void_p
_SIGS = {
    "bc_kv_pool_bytes": (C.c_size_t, [C.POINTER(bc_config)]),
    "bc_meta_pool_bytes": (C.c_size_t, [C.POINTER(bc_config)]),
    "bc_workspace_bytes": (C.c_size_t, [C.POINTER(bc_config)]),
    "bc_model_create": (C.c_int, [C.POINTER(bc_config), C.POINTER(bc_weights), _P, _P, _P, C.c_size_t, _P,
                                  C.POINTER(_P)]),
    "bc_model_destroy": (C.c_int, [_P]),
    "bc_set_stream": (C.c_int, [_P, _P]),
    "bc_set_graphs": (C.c_int, [_P, C.c_int]),
    "bc_kv_length": (C.c_int, [_P]),
    "bc_launch_count": (C.c_longlong, [_P]),
    "bc_kv_reset": (C.c_int, [_P, C.c_int]),
    "bc_kv_append": (C.c_int, [_P, _P, _P, C.c_int]),
    "bc_kv_snap_select": (C.c_int, [_P, _P, C.c_int, C.c_double, C.c_int, C.c_int]),
    "bc_decode_step": (C.c_int, [_P, C.c_int, C.c_int, C.c_double, C.c_double, C.c_int, C.c_int, C.c_int, _P]),
    "bc_decode_step_host": (C.c_int, [_P, C.c_int, C.c_int, C.c_double, C.c_double, C.c_int, C.c_int, C.c_int, _P]),
    "bc_trace": (C.c_int, [_P, C.c_int, C.c_int, C.POINTER(_P), C.POINTER(C.c_int), C.POINTER(C.c_int)]),
    "bc_gemv_scratch_bytes": (C.c_size_t, [C.c_int]),
    "bc_gemv": (C.c_int, [_P, C.c_int, C.c_int, _P, _P, C.c_int, _P, _P, C.c_size_t, _P]),
    "bc_gemv_noalloc_max_dout": (C.c_int, []),
    "bc_gemv_noalloc": (C.c_int, [_P, C.c_int, C.c_int, _P, _P, C.c_int, _P, _P]),
    "bc_gemv_batch_scratch_bytes": (C.c_size_t, [C.c_int, C.c_int, C.c_int]),
    "bc_gemv_batch": (C.c_int, [_P, C.c_int, C.c_int, _P, _P, C.c_int, C.c_int, _P, _P, _P, C.c_size_t, _P]),
    "bc_select_topk": (C.c_int, [_P, C.c_int, C.c_int, _P, _P]),
    "bc_attention_scratch_bytes": (C.c_size_t, [C.c_int, C.c_int]),
    "bc_attention": (C.c_int, [_P, _P, C.c_int, C.c_int, C.c_int, C.c_int, _P, C.c_int, C.c_int, _P, _P,
                               C.c_size_t, _P]),
    "bc_byte_account": (C.c_int, [C.POINTER(bc_config), C.c_int, C.c_double, C.c_double, C.c_longlong, C.c_int,
                                  C.c_int, C.c_int, C.POINTER(bc_bytes)]),
    "bc_crossover_batch": (C.c_int, [C.POINTER(bc_config), C.c_double, C.c_double, C.c_int,
                                     C.POINTER(C.c_double)]),
    "bc_batch_workspace_bytes": (C.c_size_t, [C.POINTER(bc_config), C.c_int]),
    "bc_batch_create": (C.c_int, [C.POINTER(bc_config), C.POINTER(bc_weights), C.c_int, _P, _P, _P, C.c_size_t, _P,
                                  C.POINTER(_P)]),
    "bc_batch_destroy": (C.c_int, [_P]),
    "bc_batch_set_graphs": (C.c_int, [_P, C.c_int]),
    "bc_batch_length": (C.c_int, [_P]),
    "bc_batch_launch_count": (C.c_longlong, [_P]),
    "bc_batch_reset": (C.c_int, [_P, C.c_int]),
    "bc_batch_append": (C.c_int, [_P, _P, _P, C.c_int]),
    "bc_batch_step": (C.c_int, [_P, C.POINTER(C.c_int), C.c_int, C.c_double, C.c_double, C.c_int, C.c_int, C.c_int,
                                _P]),
    "bc_batch_trace": (C.c_int, [_P, C.c_int, C.c_int, C.c_int, C.POINTER(_P), C.POINTER(C.c_int),
                                 C.POINTER(C.c_int)]),
    "bc_kv8_pool_bytes": (C.c_size_t, [C.c_int, C.c_int, C.c_int]),
    "bc_block_tables": (C.c_int, [C.POINTER(bc_block_tables_args), _P]),
    "bc_kv8_append": (C.c_int, [_P, _P, C.c_int, C.c_longlong, C.c_longlong, _P, C.c_int, _P, C.c_int, C.c_int,
                                C.c_int, C.c_int, _P]),
    "bc_kv8_gather": (C.c_int, [_P, C.c_int, C.c_int, C.c_int, C.c_int, _P, C.c_int, _P, _P, C.c_int, _P]),
    "bc_kv8_attention_scratch_bytes": (C.c_size_t, [C.c_int, C.c_int, C.c_int, C.c_int, C.c_int]),
    "bc_kv8_attention": (C.c_int, [C.POINTER(bc_kv8_attention_args), _P]),
    "bc_kv8_attention_status": (C.c_int, [_P, _P]),
    "bc_logits_adjust": (C.c_int, [C.POINTER(bc_logits_args), _P]),
    "bc_last_error": (C.c_char_p, []),
    "bc_status_string": (C.c_char_p, [C.c_int]),
}
for _name, (_res, _args) in _SIGS.items():
    _f = getattr(_lib, _name)
    _f.restype = _res
    _f.argtypes = _args
    globals()[_name] = _f


class BCError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        msg = bc_last_error().decode(errors="replace")
        super().__init__(f"{where}: {bc_status_string(status).decode()} ({status}): {msg}")


def check(status, where=""):
    if status != BC_OK:
        raise BCError(status, where)


def config(d: dict, max_ctx: int) -> bc_config:
    return bc_config(d["n_layers"], d["hidden"], d["intermediate"], d["n_heads"], d["n_kv_heads"],
                     d["head_dim"], d["vocab"], max_ctx, d.get("page", 16), d.get("rms_eps", 1e-5),
                     d.get("rope_theta", 5e5))


def byte_account(cfg: dict, mode: str, n_ctx: int, rp=1.0, rkv=1.0, sinks=1, recent=16) -> dict:
    c = config(cfg, max(n_ctx + 1, 1))
    out = bc_bytes()
    check(bc_byte_account(C.byref(c), MODES[mode], rp, rkv, n_ctx, sinks, recent, c.page, C.byref(out)),
          "bc_byte_account")
    return {name: getattr(out, name) for name, _ in bc_bytes._fields_}


def crossover_batch(cfg: dict, union_keep: float, rkv: float, batch: int) -> float:
    """bc_crossover_batch: the batch byte crossover, in tokens."""
    c = config(cfg, 1)
    out = C.c_double()
    check(bc_crossover_batch(C.byref(c), union_keep, rkv, batch, C.byref(out)), "bc_crossover_batch")
    return out.value


def _stream_ptr(stream):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return C.c_void_p(s.cuda_stream)


class Model:
    """Owns the device buffers (allocated with torch) and the bc_model handle."""

    def __init__(self, cfg: dict, weights: dict, max_ctx: int, stream=None):
        import torch
        self.cfg = cfg
        self.c = config(cfg, max_ctx)
        self.weights = weights           # keep the tensors alive
        dev = weights["embed"].device
        self.stream = stream if stream is not None else torch.cuda.current_stream(dev)
        kvb = bc_kv_pool_bytes(C.byref(self.c))
        mb = bc_meta_pool_bytes(C.byref(self.c))
        wsb = bc_workspace_bytes(C.byref(self.c))
        if not (kvb and mb and wsb):
            raise ValueError("bad config for libbytecross")
        self.kv_pool = torch.empty(kvb, dtype=torch.uint8, device=dev)
        self.meta_pool = torch.empty(mb, dtype=torch.uint8, device=dev)
        self.workspace = torch.zeros(wsb, dtype=torch.uint8, device=dev)
        w = bc_weights(*(C.c_void_p(weights[k].data_ptr()) for k in (
            "embed", "lm_head", "final_norm", "attn_norm", "mlp_norm", "wqkv_t", "wo_t", "wgu_t", "wd_t")))
        h = C.c_void_p()
        check(bc_model_create(C.byref(self.c), C.byref(w), C.c_void_p(self.kv_pool.data_ptr()),
                              C.c_void_p(self.meta_pool.data_ptr()), C.c_void_p(self.workspace.data_ptr()),
                              wsb, C.c_void_p(self.stream.cuda_stream), C.byref(h)), "bc_model_create")
        self.h = h

    def close(self):
        if getattr(self, "h", None):
            bc_model_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __len__(self):
        return bc_kv_length(self.h)

    def set_graphs(self, enable: bool):
        check(bc_set_graphs(self.h, 1 if enable else 0), "bc_set_graphs")

    def launches(self) -> int:
        return bc_launch_count(self.h)

    def reset(self, n_ctx: int):
        check(bc_kv_reset(self.h, n_ctx), "bc_kv_reset")

    def append(self, k, v):
        """k, v: bf16 device tensors [L][Hkv][n][hd]."""
        k, v = k.contiguous(), v.contiguous()
        check(bc_kv_append(self.h, C.c_void_p(k.data_ptr()), C.c_void_p(v.data_ptr()), k.shape[2]),
              "bc_kv_append")

    def snap_select(self, q_obs, rkv, sinks=1, recent=16):
        """Once-after-prefill page selection; q_obs: f32 device tensor
        [L][n_obs][Hq][hd] of rotated observation queries."""
        q_obs = q_obs.contiguous()
        check(bc_kv_snap_select(self.h, C.c_void_p(q_obs.data_ptr()), q_obs.shape[1], rkv, sinks, recent),
              "bc_kv_snap_select")

    def step(self, token: int, mode: str, logits, rp=1.0, rkv=1.0, sinks=1, recent=16):
        check(bc_decode_step(self.h, int(token), MODES[mode], rp, rkv, sinks, recent, self.c.page,
                             C.c_void_p(logits.data_ptr())), "bc_decode_step")

    def step_host(self, token: int, mode: str, logits_host, rp=1.0, rkv=1.0, sinks=1, recent=16):
        check(bc_decode_step_host(self.h, int(token), MODES[mode], rp, rkv, sinks, recent, self.c.page,
                                  C.c_void_p(logits_host.data_ptr())), "bc_decode_step_host")

    def trace(self, layer: int, kind: int):
        """Device tensor view of a per-layer trace from the last step."""
        import torch
        ptr, cnt, stride = C.c_void_p(), C.c_int(), C.c_int()
        check(bc_trace(self.h, layer, kind, C.byref(ptr), C.byref(cnt), C.byref(stride)), "bc_trace")
        off = ptr.value - self.workspace.data_ptr()
        is_int = kind in (BC_TRACE_SEL_QKV, BC_TRACE_SEL_O, BC_TRACE_SEL_GU, BC_TRACE_SEL_D, BC_TRACE_PAGES,
                          BC_TRACE_SNAP_PAGES)
        dt = torch.int32 if is_int else torch.float32
        if stride.value:
            rows = self.cfg["n_kv_heads"]
            t = self.workspace[off:off + 4 * rows * stride.value].view(dt).view(rows, stride.value)
            return t[:, :cnt.value]
        return self.workspace[off:off + 4 * cnt.value].view(dt)


_INT_TRACES = (BC_TRACE_SEL_QKV, BC_TRACE_SEL_O, BC_TRACE_SEL_GU, BC_TRACE_SEL_D, BC_TRACE_PAGES, BC_TRACE_SNAP_PAGES)


class Batch:
    """A batch of sequences decoding in lock step (bc_batch_*): owns the
    sequences' KV and bound pools and the workspace (allocated with torch)."""

    def __init__(self, cfg: dict, weights: dict, batch: int, max_ctx: int, stream=None):
        import torch
        self.cfg = cfg
        self.B = batch
        self.c = config(cfg, max_ctx)
        self.weights = weights
        dev = weights["embed"].device
        self.stream = stream if stream is not None else torch.cuda.current_stream(dev)
        kvb = bc_kv_pool_bytes(C.byref(self.c))
        mb = bc_meta_pool_bytes(C.byref(self.c))
        wsb = bc_batch_workspace_bytes(C.byref(self.c), batch)
        if not (kvb and mb and wsb):
            raise ValueError("bad config or batch size for a libbytecross batch")
        self.kv_pool = torch.empty(batch * kvb, dtype=torch.uint8, device=dev)
        self.meta_pool = torch.empty(batch * mb, dtype=torch.uint8, device=dev)
        self.workspace = torch.zeros(wsb, dtype=torch.uint8, device=dev)
        w = bc_weights(*(C.c_void_p(weights[k].data_ptr()) for k in (
            "embed", "lm_head", "final_norm", "attn_norm", "mlp_norm", "wqkv_t", "wo_t", "wgu_t", "wd_t")))
        h = C.c_void_p()
        check(bc_batch_create(C.byref(self.c), C.byref(w), batch, C.c_void_p(self.kv_pool.data_ptr()),
                              C.c_void_p(self.meta_pool.data_ptr()), C.c_void_p(self.workspace.data_ptr()), wsb,
                              C.c_void_p(self.stream.cuda_stream), C.byref(h)), "bc_batch_create")
        self.h = h

    def close(self):
        if getattr(self, "h", None):
            bc_batch_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __len__(self):
        return bc_batch_length(self.h)

    def set_graphs(self, enable: bool):
        check(bc_batch_set_graphs(self.h, 1 if enable else 0), "bc_batch_set_graphs")

    def launches(self) -> int:
        return bc_batch_launch_count(self.h)

    def reset(self, n_ctx: int):
        check(bc_batch_reset(self.h, n_ctx), "bc_batch_reset")

    def append(self, k, v):
        """k, v: bf16 device tensors [batch][L][Hkv][n][hd]."""
        k, v = k.contiguous(), v.contiguous()
        check(bc_batch_append(self.h, C.c_void_p(k.data_ptr()), C.c_void_p(v.data_ptr()), k.shape[3]),
              "bc_batch_append")

    def step(self, tokens, mode: str, logits, rp=1.0, rkv=1.0, sinks=1, recent=16):
        """tokens: B ints; logits: f32 device tensor [B][vocab]."""
        toks = (C.c_int * self.B)(*[int(t) for t in tokens])
        check(bc_batch_step(self.h, toks, MODES[mode], rp, rkv, sinks, recent, self.c.page,
                            C.c_void_p(logits.data_ptr())), "bc_batch_step")

    def seq(self, b: int):
        """A view of sequence b with the trace() of a Model."""
        return _BatchSeq(self, b)


class _BatchSeq:
    def __init__(self, batch: Batch, b: int):
        self.batch, self.b, self.cfg = batch, b, batch.cfg

    def trace(self, layer: int, kind: int):
        import torch
        bt = self.batch
        ptr, cnt, stride = C.c_void_p(), C.c_int(), C.c_int()
        check(bc_batch_trace(bt.h, self.b, layer, kind, C.byref(ptr), C.byref(cnt), C.byref(stride)),
              "bc_batch_trace")
        off = ptr.value - bt.workspace.data_ptr()
        dt = torch.int32 if kind in _INT_TRACES else torch.float32
        if stride.value:
            rows = self.cfg["n_kv_heads"]
            t = bt.workspace[off:off + 4 * rows * stride.value].view(dt).view(rows, stride.value)
            return t[:, :cnt.value]
        return bt.workspace[off:off + 4 * cnt.value].view(dt)


# ------------------------------------------------------------------ single kernels

def gemv(W, x, idx, y, scratch, stream=None):
    d_in, d_out = W.shape
    k = d_in if idx is None else idx.numel()
    check(bc_gemv(C.c_void_p(W.data_ptr()), d_in, d_out, C.c_void_p(x.data_ptr()),
                  C.c_void_p(idx.data_ptr()) if idx is not None else None, k, C.c_void_p(y.data_ptr()),
                  C.c_void_p(scratch.data_ptr()), scratch.numel() * scratch.element_size(),
                  _stream_ptr(stream)), "bc_gemv")


def gemv_noalloc(W, x, idx, y, stream=None):
    """bc_gemv without a scratch argument (scratch is a static device array)."""
    d_in, d_out = W.shape
    k = d_in if idx is None else idx.numel()
    check(bc_gemv_noalloc(C.c_void_p(W.data_ptr()), d_in, d_out, C.c_void_p(x.data_ptr()),
                          C.c_void_p(idx.data_ptr()) if idx is not None else None, k, C.c_void_p(y.data_ptr()),
                          _stream_ptr(stream)), "bc_gemv_noalloc")


def gemv_batch(W, x, idx, y, scratch, n_union=None, stream=None):
    """bc_gemv_batch: x [B][d_in] f32, idx [B][k] int32 (or None for all
    channels), y [B][d_out] f32, n_union an int32 tensor of one element or None."""
    d_in, d_out = W.shape
    B = x.shape[0]
    k = d_in if idx is None else idx.shape[1]
    check(bc_gemv_batch(C.c_void_p(W.data_ptr()), d_in, d_out, C.c_void_p(x.data_ptr()),
                        C.c_void_p(idx.data_ptr()) if idx is not None else None, k, B,
                        C.c_void_p(y.data_ptr()), C.c_void_p(n_union.data_ptr()) if n_union is not None else None,
                        C.c_void_p(scratch.data_ptr()), scratch.numel() * scratch.element_size(),
                        _stream_ptr(stream)), "bc_gemv_batch")


def select_topk(v, k, idx, stream=None):
    check(bc_select_topk(C.c_void_p(v.data_ptr()), v.numel(), k, C.c_void_p(idx.data_ptr()),
                         _stream_ptr(stream)), "bc_select_topk")


def attention(q, kv, n_kv_heads, group, head_dim, Pmax, pages, n_pages, n_tok, out, scratch, stream=None):
    check(bc_attention(C.c_void_p(q.data_ptr()), C.c_void_p(kv.data_ptr()), n_kv_heads, group, head_dim, Pmax,
                       C.c_void_p(pages.data_ptr()) if pages is not None else None, n_pages, n_tok,
                       C.c_void_p(out.data_ptr()), C.c_void_p(scratch.data_ptr()),
                       scratch.numel() * scratch.element_size(), _stream_ptr(stream)), "bc_attention")


# ------------------------------------------------------------------ ragged batches over an 8-bit cache

def _need(ok, who, what):
    if not ok:
        raise ValueError(f"{who}: {what}")


def _ints(who, device, **tensors):
    """Checks contiguous int32 tensors of the device."""
    import torch
    for name, t in tensors.items():
        _need(t.dtype == torch.int32 and t.is_contiguous() and t.device == device, who,
              f"{name} must be a contiguous int32 tensor on {device}")


def _floats(who, device, **tensors):
    import torch
    for name, t in tensors.items():
        _need(t.dtype == torch.float32 and t.is_contiguous() and t.device == device, who,
              f"{name} must be a contiguous float32 tensor on {device}")


def _dtype(who, t):
    import torch
    if t.dtype == torch.float32:
        return BC_F32
    if t.dtype == torch.bfloat16:
        return BC_BF16
    raise ValueError(f"{who}: float32 or bfloat16 expected, not {t.dtype}")


def _kv8_type(who, code):
    _need(code in KV8_TYPES, who, f"code must be one of {sorted(KV8_TYPES)}, not {code!r}")
    return KV8_TYPES[code]


def _kv8_pool(who, pool):
    """(n_pages, n_kv_heads, head_dim) of a pool tensor uint8 [n_pages][n_kv_heads][32 hd + 32]."""
    import torch
    _need(pool.dtype == torch.uint8 and pool.dim() == 3 and pool.is_contiguous() and pool.is_cuda
          and (pool.shape[2] - 32) in (32 * 64, 32 * 128), who,
          "the pool must be a contiguous CUDA uint8 tensor [n_pages][n_kv_heads][32 head_dim + 32]")
    return pool.shape[0], pool.shape[1], (pool.shape[2] - 32) // 32


def _launch(device, stream, where, fn, *args):
    """Calls fn(*args, stream) with the tensors' device current, on `stream`
    or on that device's current stream."""
    import torch
    with torch.cuda.device(device):
        s = stream if stream is not None else torch.cuda.current_stream(device)
        check(fn(*args, s.cuda_stream), where)


def block_tables(lens, delta, table, free_list, n_free, lens_out, n_free_out, q_start, slots, positions, ticket,
                 stream=None):
    """bc_block_tables: the plan of one step of a ragged batch.  int32 CUDA
    tensors: lens, delta, lens_out [B], table [B][max_blocks], free_list
    [n_pages], n_free, n_free_out, ticket [1], q_start [B + 1], slots and
    positions [max_tokens]."""
    who, dev = "block_tables", table.device
    _need(table.is_cuda and table.dim() == 2, who, "table must be a CUDA tensor [batch][max_blocks]")
    _ints(who, dev, lens=lens, delta=delta, table=table, free_list=free_list, n_free=n_free, lens_out=lens_out,
          n_free_out=n_free_out, q_start=q_start, slots=slots, positions=positions, ticket=ticket)
    B = table.shape[0]
    _need(lens.numel() == delta.numel() == lens_out.numel() == B and q_start.numel() == B + 1, who,
          "lens, delta and lens_out need one entry per sequence, q_start one more")
    _need(n_free.numel() == n_free_out.numel() == ticket.numel() == 1, who, "n_free, n_free_out and ticket hold one word")
    _need(slots.numel() == positions.numel(), who, "slots and positions differ in length")
    a = bc_block_tables_args(B, table.shape[1], free_list.numel(), slots.numel(), lens.data_ptr(), delta.data_ptr(),
                             table.data_ptr(), free_list.data_ptr(), n_free.data_ptr(), lens_out.data_ptr(),
                             n_free_out.data_ptr(), q_start.data_ptr(), slots.data_ptr(), positions.data_ptr(),
                             ticket.data_ptr())
    _launch(dev, stream, "bc_block_tables", bc_block_tables, C.byref(a))


def _kv8_rows(who, dev, H, hd, n, dtype, **tensors):
    for name, t in tensors.items():
        _need(t.device == dev and t.dtype == dtype and tuple(t.shape) == (n, H, hd), who,
              f"{name} must be {dtype} [{n}][{H}][{hd}] on {dev}")


def kv8_append(k, v, slots, pool, code="e4m3", stream=None):
    """bc_kv8_append: k, v f32 or bf16 [n][n_kv_heads][hd], the last two
    dimensions dense (a token's stride is free); slots int32 [n]; pool uint8
    [n_pages][n_kv_heads][32 hd + 32]."""
    who = "kv8_append"
    P, H, hd = _kv8_pool(who, pool)
    n, dev = slots.numel(), pool.device
    _ints(who, dev, slots=slots)
    _kv8_rows(who, dev, H, hd, n, k.dtype, k=k, v=v)
    dt = _dtype(who, k)
    typ = _kv8_type(who, code)
    if n == 0:
        return
    for name, t in (("k", k), ("v", v)):
        _need(t.stride(2) == 1 and (H == 1 or t.stride(1) == hd), who, f"{name}: heads and dims must be dense")
    ks, vs = (t.stride(0) if n > 1 else max(t.stride(0), H * hd) for t in (k, v))
    _launch(dev, stream, "bc_kv8_append", bc_kv8_append, k.data_ptr(), v.data_ptr(), dt, ks, vs, slots.data_ptr(), n,
            pool.data_ptr(), typ, P, H, hd)


def kv8_gather(pool, slots, k_out, v_out, code="e4m3", stream=None):
    """bc_kv8_gather: k_out, v_out f32 or bf16 [n][n_kv_heads][hd] receive the
    tokens at slots (int32 [n])."""
    who = "kv8_gather"
    P, H, hd = _kv8_pool(who, pool)
    n, dev = slots.numel(), pool.device
    _ints(who, dev, slots=slots)
    _kv8_rows(who, dev, H, hd, n, k_out.dtype, k_out=k_out, v_out=v_out)
    _need(k_out.is_contiguous() and v_out.is_contiguous(), who, "k_out and v_out must be contiguous")
    dt = _dtype(who, k_out)
    typ = _kv8_type(who, code)
    if n == 0:
        return
    _launch(dev, stream, "bc_kv8_gather", bc_kv8_gather, pool.data_ptr(), typ, P, H, hd, slots.data_ptr(), n,
            k_out.data_ptr(), v_out.data_ptr(), dt)


def kv8_attention(q, pool, lens, table, out, scratch, code="e4m3", q_start=None, max_q=1, pages=None, n_sel=None,
                  scale=None, cap=0.0, window=0, slopes=None, stream=None):
    """bc_kv8_attention: q f32 or bf16 [n_q][Hq][hd] (a row's stride is free),
    out the same type and shape, contiguous; lens int32 [B]; table int32
    [B][max_blocks]; q_start int32 [B + 1] or None (one query a sequence);
    pages int32 [B][n_kv_heads][max_sel] with n_sel int32 [B], or None; slopes
    f32 [Hq] or None; scale None for 1 / sqrt(hd); scratch uint8 of
    bc_kv8_attention_scratch_bytes(B, n_kv_heads, group, max_q, hd) bytes,
    zeroed before its first use."""
    import torch
    who, dev = "kv8_attention", pool.device
    P, H, hd = _kv8_pool(who, pool)
    _need(q.dim() == 3 and q.shape[2] == hd and q.shape[1] % H == 0 and q.device == dev and q.stride(2) == 1
          and q.stride(1) == hd, who, f"q must be [n_q][group * {H}][{hd}] on {dev}, heads and dims dense")
    n_q, Hq = q.shape[0], q.shape[1]
    dt = _dtype(who, q)
    _need(out.dtype == q.dtype and out.shape == q.shape and out.is_contiguous() and out.device == dev, who,
          "out must be contiguous, of q's type and shape")
    _need(table.dim() == 2 and lens.numel() == table.shape[0], who, "table [batch][max_blocks], lens [batch] expected")
    B = table.shape[0]
    _ints(who, dev, lens=lens, table=table)
    _need(scratch.device == dev and scratch.dtype == torch.uint8 and scratch.is_contiguous(), who,
          "scratch must be a contiguous uint8 tensor on the pool's device")
    max_sel = 0
    if q_start is not None:
        _ints(who, dev, q_start=q_start)
        _need(q_start.numel() == B + 1, who, "q_start needs one entry more than the batch")
    else:
        _need(max_q == 1 and n_q == B, who, "without q_start there is one query row per sequence")
    _need((pages is None) == (n_sel is None), who, "pages and n_sel go together")
    if pages is not None:
        _ints(who, dev, pages=pages, n_sel=n_sel)
        _need(pages.dim() == 3 and pages.shape[0] == B and pages.shape[1] == H and pages.shape[2] >= 1
              and n_sel.numel() == B, who, "pages [batch][n_kv_heads][max_sel], n_sel [batch] expected")
        max_sel = pages.shape[2]
    if slopes is not None:
        _floats(who, dev, slopes=slopes)
        _need(slopes.numel() == Hq, who, "slopes needs one entry per query head")
    typ = _kv8_type(who, code)
    if n_q == 0:
        return
    a = bc_kv8_attention_args(
        q.data_ptr(), out.data_ptr(), dt, q.stride(0) if n_q > 1 else Hq * hd, n_q, pool.data_ptr(), typ, P, H,
        Hq // H, hd, B, max_q, table.shape[1], max_sel, lens.data_ptr(),
        q_start.data_ptr() if q_start is not None else None, table.data_ptr(),
        pages.data_ptr() if pages is not None else None, n_sel.data_ptr() if n_sel is not None else None,
        hd ** -0.5 if scale is None else scale, cap, window, slopes.data_ptr() if slopes is not None else None,
        scratch.data_ptr(), scratch.numel())
    _launch(dev, stream, "bc_kv8_attention", bc_kv8_attention, C.byref(a))


def logits_adjust(logits, out, hist=None, hist_start=None, prompt_len=None, repetition=None, frequency=None,
                  presence=None, bias_ids=None, bias_vals=None, bias_start=None, mask=None, mask_row=None,
                  stream=None):
    """bc_logits_adjust: logits f32 or bf16 [B][V] (a row's stride is free),
    out of the same type and shape (logits itself for an update in place);
    hist, bias_ids int32 with hist_start, bias_start int32 [B + 1]; prompt_len,
    mask_row int32 [B]; repetition, frequency, presence f32 [B]; bias_vals f32;
    mask int32 [n_masks][ceil(V / 32)]."""
    who, dev = "logits_adjust", logits.device
    _need(logits.is_cuda and logits.dim() == 2 and logits.stride(1) == 1, who, "logits must be a CUDA tensor [B][V]")
    dt = _dtype(who, logits)
    _need(out.device == dev and out.dtype == logits.dtype and out.shape == logits.shape and out.stride(1) == 1, who,
          "out must have the type, shape and device of logits")
    B, V = logits.shape
    _need((hist is None) == (hist_start is None), who, "hist and hist_start go together")
    _need((bias_ids is None) == (bias_vals is None) == (bias_start is None), who,
          "bias_ids, bias_vals and bias_start go together")
    _need(mask is not None or mask_row is None, who, "mask_row needs mask")
    ints = dict(hist=hist, hist_start=hist_start, prompt_len=prompt_len, bias_ids=bias_ids, bias_start=bias_start,
                mask=mask, mask_row=mask_row)
    floats = dict(repetition=repetition, frequency=frequency, presence=presence, bias_vals=bias_vals)
    _ints(who, dev, **{k: t for k, t in ints.items() if t is not None})
    _floats(who, dev, **{k: t for k, t in floats.items() if t is not None})
    for name, t, n in (("hist_start", hist_start, B + 1), ("bias_start", bias_start, B + 1),
                       ("prompt_len", prompt_len, B), ("mask_row", mask_row, B), ("repetition", repetition, B),
                       ("frequency", frequency, B), ("presence", presence, B)):
        _need(t is None or t.numel() == n, who, f"{name} needs {n} entries")
    n_bias = n_masks = 0
    if bias_ids is not None:
        n_bias = bias_ids.numel()
        _need(bias_vals.numel() == n_bias, who, "bias_ids and bias_vals differ in length")
    if mask is not None:
        _need(mask.dim() == 2 and mask.shape[1] == (V + 31) // 32, who, f"mask must be [n_masks][{(V + 31) // 32}]")
        n_masks = mask.shape[0]
    if B == 0 or V == 0:
        return
    ptr = lambda t: t.data_ptr() if t is not None else None
    a = bc_logits_args(logits.data_ptr(), out.data_ptr(), dt, B, V, logits.stride(0) if B > 1 else V,
                       out.stride(0) if B > 1 else V, ptr(hist), ptr(hist_start), ptr(prompt_len),
                       hist.numel() if hist is not None else 0, ptr(repetition), ptr(frequency), ptr(presence),
                       ptr(bias_ids), ptr(bias_vals), ptr(bias_start), n_bias, ptr(mask), ptr(mask_row), n_masks)
    _launch(dev, stream, "bc_logits_adjust", bc_logits_adjust, C.byref(a))


class RaggedCache:
    """An 8-bit paged KV cache of `layers` layers that a batch of sequences of
    different lengths shares: owns the pools, block tables, free list and the
    step's plan (allocated with torch).  Per step: plan(delta), then per layer
    append(layer, k, v) and attend(layer, q, out).  Everything stays on the
    device, so a step can be captured into a graph."""

    def __init__(self, layers: int, batch: int, n_pages: int, n_kv_heads: int, group: int, head_dim: int,
                 max_blocks: int, max_tokens: int, max_q: int = 1, code: str = "e4m3", device="cuda"):
        import torch
        _kv8_type("RaggedCache", code)
        layer_bytes = bc_kv8_pool_bytes(n_pages, n_kv_heads, head_dim)
        scratch = bc_kv8_attention_scratch_bytes(batch, n_kv_heads, group, max_q, head_dim)
        if not (layer_bytes and scratch) or layers < 1 or max_blocks < 1 or max_tokens < 1:
            raise ValueError("bad sizes for an 8-bit ragged cache")
        self.layers, self.batch, self.group, self.max_q, self.code = layers, batch, group, max_q, code
        ints = lambda *s: torch.zeros(*s, dtype=torch.int32, device=device)
        self.pool = torch.empty(layers, n_pages, n_kv_heads, 32 * head_dim + 32, dtype=torch.uint8, device=device)
        self.table, self.lens, self.q_start = ints(batch, max_blocks), ints(batch), ints(batch + 1)
        self.free_list = torch.arange(n_pages, dtype=torch.int32, device=device)
        self.n_free = ints(1).fill_(n_pages)
        self.slots, self.positions, self.ticket = ints(max_tokens), ints(max_tokens), ints(1)
        self.scratch = torch.zeros(scratch, dtype=torch.uint8, device=device)

    def plan(self, delta, stream=None):
        """delta int32 [batch]: tokens each sequence takes (or, negative,
        drops); updates lens, table, free_list, q_start, slots, positions."""
        block_tables(self.lens, delta, self.table, self.free_list, self.n_free, self.lens, self.n_free, self.q_start,
                     self.slots, self.positions, self.ticket, stream)

    def append(self, layer: int, k, v, stream=None):
        """k, v [n][n_kv_heads][hd] of the step's new tokens in the plan's
        order (rows behind the last one are not read into the cache)."""
        n = k.shape[0]
        _need(n <= self.slots.numel(), "RaggedCache.append", f"more than {self.slots.numel()} tokens")
        kv8_append(k, v, self.slots[:n], self.pool[layer], self.code, stream)

    def attend(self, layer: int, q, out, stream=None, **options):
        """q [n_q][Hq][hd], the queries of the step's new tokens; options as
        for kv8_attention."""
        kv8_attention(q, self.pool[layer], self.lens, self.table, out, self.scratch, self.code, self.q_start,
                      self.max_q, stream=stream, **options)

    def read(self, layer: int, seq: int, n: int, dtype=None, stream=None):
        """The first n tokens of a sequence as (k, v) [n][n_kv_heads][hd]
        (bf16, or dtype)."""
        import torch
        dtype = torch.bfloat16 if dtype is None else dtype
        H, hd = self.pool.shape[2], (self.pool.shape[3] - 32) // 32
        _need(0 <= n <= 16 * self.table.shape[1], "RaggedCache.read", "n outside the sequence's table")
        dev = self.pool.device
        with torch.cuda.device(dev), torch.cuda.stream(stream if stream is not None else torch.cuda.current_stream(dev)):
            pos = torch.arange(n, device=dev)
            slots = (self.table[seq][pos // 16] * 16 + pos % 16).int()
            k = torch.empty(n, H, hd, dtype=dtype, device=dev)
            v = torch.empty_like(k)
            kv8_gather(self.pool[layer], slots, k, v, self.code)
        return k, v

    def status(self, stream=None):
        """Waits for the stream; raises if a wait of an attention gave up."""
        import torch
        dev = self.pool.device
        _launch(dev, stream, "bc_kv8_attention_status", bc_kv8_attention_status, self.scratch.data_ptr())
