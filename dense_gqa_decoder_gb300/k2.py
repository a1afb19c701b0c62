"""Thin ctypes binding of libk2 (include/k2.h).

Argument marshalling only: every step of the decode path runs in the CUDA
kernels of libk2.so.  torch is used for device memory and streams.  If the
library is missing the import fails loudly -- there is no fallback.
"""
from __future__ import annotations

import ctypes as C
import os
import struct

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libk2.so")

K2_OK, K2_ERR_ARG, K2_ERR_SHAPE, K2_ERR_UNSUPPORTED, K2_ERR_TOKEN_RANGE, K2_ERR_CONTEXT_FULL, \
    K2_ERR_WORKSPACE, K2_ERR_CUDA, K2_ERR_DEVICE_GUARD, K2_ERR_STATE = range(10)
K2_STATE_HEADER_BYTES = 96
K2_F32, K2_BF16, K2_F16, K2_I8, K2_F8, K2_Q4 = range(6)
(K2_OPT_PDL, K2_OPT_GRAPH, K2_OPT_ATTN_SPLITS, K2_OPT_PERSISTENT, K2_OPT_TC_PREFILL, K2_OPT_TC_DECODE,
 K2_OPT_WAIT_LIMIT_US, K2_OPT_STALL_PHASE, K2_OPT_L2_AHEAD, K2_OPT_L2_AHEAD_PHASES, K2_OPT_TRACE,
 K2_OPT_PREFILL_ATTN, K2_OPT_PREFILL_SPLIT, K2_OPT_PREFILL_GEMM) = range(14)
KERNEL_CLASSES = ("embed", "qkv", "attn", "o_proj", "gate_up", "down", "lm_head", "step", "sample")
K2_PAGED_BAD_SLOT, K2_PAGED_BAD_BLOCK, K2_PAGED_BAD_LENGTH, K2_PAGED_TIMEOUT = 1, 2, 4, 8
K2_PLAN_BAD_LENGTH, K2_PLAN_TABLE_FULL, K2_PLAN_NO_BLOCKS, K2_PLAN_TOKENS_FULL = 1, 2, 4, 8
K2_PAGED_MAX_REQUESTS = 2048
DTYPES = {"f32": K2_F32, "bf16": K2_BF16, "f16": K2_F16, "i8": K2_I8, "f8": K2_F8, "q4": K2_Q4}


class K2Error(RuntimeError):
    def __init__(self, status, msg):
        super().__init__(f"k2 status {status}: {msg}")
        self.status = status


class Config(C.Structure):
    _fields_ = [(n, C.c_int32) for n in (
        "hidden", "n_layers", "n_heads", "n_kv_heads", "head_dim", "intermediate", "norm_groups", "vocab",
        "max_context", "max_batch")] + [("eps", C.c_float), ("rope_theta", C.c_float),
                                        ("weight_dtype", C.c_int32), ("kv_dtype", C.c_int32)]


_PP = C.POINTER(C.c_void_p)


class Weights(C.Structure):
    _fields_ = [("embed", C.c_void_p), ("lm_head", C.c_void_p), ("final_norm", C.c_void_p)] + [
        (n, _PP) for n in ("attn_norm", "wq", "wk", "wv", "wo", "mlp_norm", "w_gate", "w_up", "w_down")]


class Info(C.Structure):
    _fields_ = [("kv_capacity", C.c_int32), ("num_sms", C.c_int32), ("attn_splits", C.c_int32),
                ("gemv_grid", C.c_int32), ("kv_bytes", C.c_int64), ("repack_bytes", C.c_int64),
                ("scratch_bytes", C.c_int64), ("persistent_grid", C.c_int32), ("persistent_splits", C.c_int32),
                ("tc_prefill", C.c_int32), ("tc_batched", C.c_int32)]


class Sampling(C.Structure):
    _fields_ = [("temperature", C.c_float), ("top_k", C.c_int32), ("top_p", C.c_float), ("min_p", C.c_float),
                ("repetition_penalty", C.c_float), ("seed", C.c_uint64)]


def sampling(temperature=0.0, top_k=0, top_p=1.0, min_p=0.0, repetition_penalty=1.0, seed=0) -> Sampling:
    return Sampling(temperature=temperature, top_k=top_k, top_p=top_p, min_p=min_p,
                    repetition_penalty=repetition_penalty, seed=seed)


class PagedKv(C.Structure):
    _fields_ = [("k", C.c_void_p), ("v", C.c_void_p), ("k_scale", C.c_void_p), ("v_scale", C.c_void_p),
                ("n_blocks", C.c_int32), ("block_tokens", C.c_int32), ("n_kv_heads", C.c_int32),
                ("head_dim", C.c_int32), ("dtype", C.c_int32), ("wait_limit_us", C.c_int32), ("flags", C.c_void_p)]


class LogitRules(C.Structure):
    _fields_ = [("repetition", C.c_void_p), ("presence", C.c_void_p), ("frequency", C.c_void_p),
                ("ids", C.c_void_p), ("ids_stride", C.c_int64), ("ids_len", C.c_void_p), ("prompt_len", C.c_void_p),
                ("bias_offset", C.c_void_p), ("bias_ids", C.c_void_p), ("bias", C.c_void_p), ("n_bias", C.c_int32),
                ("mask", C.c_void_p), ("mask_stride", C.c_int64), ("n_masks", C.c_int32), ("mask_row", C.c_void_p)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libk2.so is not built ({LIB_PATH}); run dense_gqa_decoder_gb300.build")
    lib = C.CDLL(LIB_PATH)
    vp, i32, i64 = C.c_void_p, C.c_int32, C.c_int64
    sig = {
        "k2_workspace_bytes": (C.c_size_t, [C.POINTER(Config)]),
        "k2_init_weights": (C.c_int, [C.POINTER(Config), C.POINTER(Weights), vp, C.c_size_t, vp, C.POINTER(vp)]),
        "k2_free": (None, [vp]),
        "k2_last_error": (C.c_char_p, [vp]),
        "k2_get_info": (C.c_int, [vp, C.POINTER(Info)]),
        "k2_prefill": (C.c_int, [vp, i32, vp, i32, vp, vp, vp]),
        "k2_decode_step": (C.c_int, [vp, vp, i32, vp, vp, vp]),
        "k2_decode_layers": (C.c_int, [vp, vp, i32, vp]),
        "k2_kv_reset": (C.c_int, [vp, i32, vp]),
        "k2_kv_set_len": (C.c_int, [vp, i32, i32, vp]),
        "k2_kv_view": (C.c_int, [vp, i32, i32, C.POINTER(vp), C.POINTER(vp), C.POINTER(vp), C.POINTER(vp),
                                 C.POINTER(i32)]),
        "k2_hidden_view": (C.c_int, [vp, i32, C.POINTER(vp)]),
        "k2_sync_status": (C.c_int, [vp, vp]),
        "k2_clear_status": (C.c_int, [vp, vp]),
        "k2_set_option": (C.c_int, [vp, i32, i64]),
        "k2_profile_decode": (C.c_int, [vp, vp, i32, vp, C.POINTER(C.c_float), C.POINTER(i32), vp]),
        "k2_greedy_head_noalloc": (C.c_int, [C.POINTER(Config), vp, vp, vp, vp, vp, vp]),
        "k2_kv_state_bytes": (C.c_int, [vp, i32, i32, C.POINTER(C.c_size_t)]),
        "k2_kv_save": (C.c_int, [vp, i32, vp, i32, vp, C.c_size_t, C.POINTER(C.c_size_t), vp]),
        "k2_kv_peek": (C.c_int, [C.POINTER(Config), vp, C.c_size_t, C.POINTER(i32), C.POINTER(i32)]),
        "k2_kv_load": (C.c_int, [vp, i32, vp, C.c_size_t, vp, i32, vp]),
        "k2_set_sampling": (C.c_int, [vp, C.POINTER(Sampling)]),
        "k2_sample_logits": (C.c_int, [vp, vp, i32, vp, i32, vp, vp, i32, vp, vp]),
        "k2_philox": (C.c_int, [C.c_uint32, i32, C.c_uint32, C.c_uint32, C.c_uint32, C.c_uint64, vp, vp]),
        "k2_spec_draft": (i32, [vp, i32, i32, vp]),
        "k2_quantize_fp8": (C.c_int, [vp, i32, i32, vp, vp, vp]),
        "k2_quantize_q4": (C.c_int, [vp, i32, i32, vp, vp, vp]),
        "k2_decode_speculative": (C.c_int, [vp, i32, vp, i32, i32, vp, C.POINTER(i32), vp]),
        "k2_spec_logits_view": (C.c_int, [vp, C.POINTER(vp), C.POINTER(i32)]),
        "k2_paged_plan": (C.c_int, [vp, vp, i32, i32, vp, i32, vp, i32, vp, vp, vp, vp, vp, vp, i32, vp, vp]),
        "k2_paged_append": (C.c_int, [vp, vp, vp, i32, i64, i64, vp, i32, vp]),
        "k2_paged_workspace_bytes": (C.c_size_t, []),
        "k2_paged_attention": (C.c_int, [vp, vp, i32, i64, vp, vp, vp, i32, i32, i32, i32, i32, C.c_float, vp, i64, vp,
                                         C.c_size_t, vp]),
        "k2_paged_step": (C.c_int, [vp, vp, vp, vp, vp, i32, vp, vp, vp, i32, i32, i32, vp, vp, vp, C.c_size_t, vp]),
        "k2_adjust_logits": (C.c_int, [vp, vp, i64, vp, i64, i32, i32, vp]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    return lib


LIB = _load()
EXPORTED = ("k2_workspace_bytes", "k2_init_weights", "k2_free", "k2_last_error", "k2_get_info", "k2_prefill",
            "k2_decode_step", "k2_decode_layers", "k2_kv_reset", "k2_kv_set_len", "k2_kv_view", "k2_hidden_view",
            "k2_sync_status", "k2_clear_status", "k2_set_option", "k2_profile_decode", "k2_greedy_head_noalloc",
            "k2_kv_state_bytes", "k2_kv_save", "k2_kv_peek", "k2_kv_load", "k2_set_sampling", "k2_sample_logits",
            "k2_philox", "k2_spec_draft", "k2_decode_speculative", "k2_quantize_fp8",
            "k2_quantize_q4", "k2_spec_logits_view", "k2_paged_plan", "k2_paged_append",
            "k2_paged_workspace_bytes", "k2_paged_attention", "k2_paged_step", "k2_adjust_logits")


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def make_config(shape, max_context: int, max_batch: int = 1, kv_dtype: str = "f16", weights: str = None) -> Config:
    """weights: the stored weight dtype, default the shape's; "f8" stores the
    shape's bf16 weights as fp8 E4M3 rows with per-row scales, "q4" as int4
    codes with one scale per 64 weights of a row."""
    return Config(hidden=shape.hidden, n_layers=shape.n_layers, n_heads=shape.n_heads, n_kv_heads=shape.n_kv_heads,
                  head_dim=shape.head_dim, intermediate=shape.intermediate, norm_groups=shape.norm_groups,
                  vocab=shape.vocab, max_context=max_context, max_batch=max_batch, eps=shape.eps,
                  rope_theta=shape.rope_theta, weight_dtype=DTYPES[weights or shape.weight_dtype],
                  kv_dtype=DTYPES[kv_dtype])


def workspace_bytes(cfg: Config) -> int:
    return int(LIB.k2_workspace_bytes(C.byref(cfg)))


class Context:
    """Owns a k2_ctx plus the torch tensors whose memory it uses (workspace,
    weights).  Methods mirror the C calls of the same name (k2_ prefix dropped)."""

    def __init__(self, cfg: Config, weights: dict, stream=None):
        self.cfg = cfg
        self.weights = weights  # keeps device memory alive
        nbytes = workspace_bytes(cfg)
        if nbytes == 0:
            raise K2Error(K2_ERR_ARG, "invalid config: " + (LIB.k2_last_error(None) or b"").decode())
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        L = cfg.n_layers
        arrs = {}
        for n in ("attn_norm", "wq", "wk", "wv", "wo", "mlp_norm", "w_gate", "w_up", "w_down"):
            arrs[n] = (C.c_void_p * L)(*[_ptr(weights[n][l]) for l in range(L)])
        self._arrs = arrs
        w = Weights(embed=_ptr(weights["embed"]), lm_head=_ptr(weights["lm_head"]),
                    final_norm=_ptr(weights["final_norm"]),
                    **{n: C.cast(a, _PP) for n, a in arrs.items()})
        ctx = C.c_void_p()
        st = LIB.k2_init_weights(C.byref(cfg), C.byref(w), _ptr(self.workspace), nbytes, _stream(stream),
                                 C.byref(ctx))
        if st != K2_OK:
            raise K2Error(st, (LIB.k2_last_error(None) or b"").decode())
        self.ctx = ctx

    def __del__(self):
        ctx = getattr(self, "ctx", None)
        if ctx:
            LIB.k2_free(ctx)
            self.ctx = None

    def _check(self, st):
        if st != K2_OK:
            raise K2Error(st, LIB.k2_last_error(self.ctx).decode())

    def last_error(self) -> str:
        return LIB.k2_last_error(self.ctx).decode()

    def info(self) -> Info:
        i = Info()
        self._check(LIB.k2_get_info(self.ctx, C.byref(i)))
        return i

    def prefill(self, seq, tokens, next_token, logits=None, stream=None):
        self._check(LIB.k2_prefill(self.ctx, seq, _ptr(tokens), tokens.numel(), _ptr(next_token), _ptr(logits),
                                   _stream(stream)))

    def decode_step(self, tokens, batch, next_tokens, logits=None, stream=None):
        self._check(LIB.k2_decode_step(self.ctx, _ptr(tokens), batch, _ptr(next_tokens), _ptr(logits),
                                       _stream(stream)))

    def decode_layers(self, x, batch, stream=None):
        self._check(LIB.k2_decode_layers(self.ctx, _ptr(x), batch, _stream(stream)))

    def kv_reset(self, seq=-1, stream=None):
        self._check(LIB.k2_kv_reset(self.ctx, seq, _stream(stream)))

    def kv_set_len(self, seq, n, stream=None):
        self._check(LIB.k2_kv_set_len(self.ctx, seq, n, _stream(stream)))

    def kv_view(self, layer, seq):
        k, v, ks, vs = C.c_void_p(), C.c_void_p(), C.c_void_p(), C.c_void_p()
        n = C.c_int32()
        self._check(LIB.k2_kv_view(self.ctx, layer, seq, C.byref(k), C.byref(v), C.byref(ks), C.byref(vs),
                                   C.byref(n)))
        return k.value, v.value, ks.value, vs.value, n.value

    def hidden_view(self, b=0):
        p = C.c_void_p()
        self._check(LIB.k2_hidden_view(self.ctx, b, C.byref(p)))
        return p.value

    def spec_logits(self):
        """k2_spec_logits_view: the logits of the last speculative step as a
        [rows, vocab] float32 CUDA tensor view (not a copy)."""
        p, rows = C.c_void_p(), C.c_int32(0)
        self._check(LIB.k2_spec_logits_view(self.ctx, C.byref(p), C.byref(rows)))
        if rows.value == 0:
            return torch.empty(0, self.cfg.vocab, dtype=torch.float32, device="cuda")
        return device_view(p.value, rows.value * self.cfg.vocab, torch.float32).view(rows.value, self.cfg.vocab)

    def sync_status(self, stream=None):
        return LIB.k2_sync_status(self.ctx, _stream(stream))

    def clear_status(self, stream=None):
        self._check(LIB.k2_clear_status(self.ctx, _stream(stream)))

    def set_option(self, opt, value):
        self._check(LIB.k2_set_option(self.ctx, opt, value))

    def set_sampling(self, params=None):
        """k2_set_sampling: a Sampling (see sampling()) or None for greedy."""
        self._check(LIB.k2_set_sampling(self.ctx, C.byref(params) if params is not None else None))

    def sample_logits(self, logits, rows, positions, next_tokens, seen=None, seen_len=None, first_seq=0,
                      stream=None):
        """k2_sample_logits on device tensors: logits [rows, vocab] fp32, positions
        and next_tokens [rows] int32, seen [rows, stride] / seen_len [rows] int32."""
        stride = seen.shape[-1] if seen is not None else 0
        self._check(LIB.k2_sample_logits(self.ctx, _ptr(logits), rows, _ptr(seen), stride, _ptr(seen_len),
                                         _ptr(positions), first_seq, _ptr(next_tokens), _stream(stream)))

    def decode_speculative(self, seq, tokens, max_draft=8, stream=None):
        """k2_decode_speculative: `tokens` = the cached ids + the next input (a
        contiguous numpy int32 array is passed without a copy); returns the
        emitted greedy ids (the last one is the next input)."""
        import numpy as np
        if isinstance(tokens, np.ndarray) and tokens.dtype == np.int32 and tokens.flags.c_contiguous:
            ids, n_ids = tokens.ctypes.data, tokens.size
        else:
            arr = np.ascontiguousarray(np.asarray(tokens, dtype=np.int32))
            ids, n_ids = arr.ctypes.data, arr.size
        out = (C.c_int32 * (max(max_draft, 0) + 1))()
        n = C.c_int32(0)
        self._check(LIB.k2_decode_speculative(self.ctx, seq, ids, n_ids, max_draft, out, C.byref(n),
                                              _stream(stream)))
        return list(out[:n.value])

    def paged_step(self, caches, tokens, positions, slots, cu_new, kv_len, table, max_new, next_tokens, workspace,
                   logits=None, stream=None):
        """k2_paged_step: caches, one PagedCache per layer; tokens, positions, slots
        [tokens], cu_new [requests + 1], kv_len and next_tokens [requests], table
        [requests, columns] int32; logits [requests, vocab] float32 or None."""
        dev = _device(tokens)
        if len(caches) != self.cfg.n_layers or any(c.device != dev for c in caches):
            raise ValueError(f"a paged step needs {self.cfg.n_layers} caches on cuda:{dev}, one per layer")
        n, r, i32 = tokens.numel(), kv_len.numel(), torch.int32
        for what, t, shape in (("tokens", tokens, (n,)), ("positions", positions, (n,)), ("slots", slots, (n,)),
                               ("cu_new", cu_new, (r + 1,)), ("kv_len", kv_len, (r,)), ("table", table, (r, None)),
                               ("next_tokens", next_tokens, (r,))):
            _need(what, t, i32, shape, dev)
        if logits is not None:
            _need("logits", logits, torch.float32, (r, self.cfg.vocab), dev)
        _need("workspace", workspace, torch.uint8, (None,), dev)
        layers = (PagedKv * len(caches))(*[c.desc for c in caches])
        self._check(LIB.k2_paged_step(self.ctx, layers, tokens.data_ptr(), positions.data_ptr(), slots.data_ptr(), n,
                                      cu_new.data_ptr(), kv_len.data_ptr(), table.data_ptr(), table.size(1), r, max_new,
                                      next_tokens.data_ptr(), _ptr(logits), workspace.data_ptr(), workspace.numel(),
                                      _raw_stream(stream, dev)))

    def kv_state_bytes(self, seq, n_tokens=0):
        n = C.c_size_t()
        st = LIB.k2_kv_state_bytes(self.ctx, seq, n_tokens, C.byref(n))
        if st != K2_OK:
            raise K2Error(st, "kv_state_bytes: bad seq or n_tokens")
        return n.value

    def kv_save(self, seq, tokens=(), out=None, stream=None):
        """k2_kv_save into `out` (a uint8 CPU tensor, pinned copies fastest) or
        a new pinned buffer; returns the uint8 tensor holding the state."""
        ids = torch.as_tensor(list(tokens) if not torch.is_tensor(tokens) else tokens.cpu(),
                              dtype=torch.int32).contiguous()
        n = self.kv_state_bytes(seq, ids.numel())
        if out is None:
            out = torch.empty(n, dtype=torch.uint8).pin_memory()
        wrote = C.c_size_t()
        self._check(LIB.k2_kv_save(self.ctx, seq, ids.data_ptr() if ids.numel() else None, ids.numel(),
                                   out.data_ptr(), out.numel(), C.byref(wrote), _stream(stream)))
        return out[:wrote.value]

    def kv_load(self, seq, state, stream=None):
        """k2_kv_load from a uint8 CPU tensor; returns the saved token ids."""
        state = state.contiguous()
        cached, n_tok = peek_state(self.cfg, state)  # sizes the token buffer; the load re-checks
        ids = torch.empty(max(n_tok, 0), dtype=torch.int32)
        self._check(LIB.k2_kv_load(self.ctx, seq, state.data_ptr(), state.numel(),
                                   ids.data_ptr() if n_tok > 0 else None, max(n_tok, 0), _stream(stream)))
        return ids.tolist()

    def profile_decode(self, tokens, batch, next_tokens, stream=None):
        ms = (C.c_float * len(KERNEL_CLASSES))()
        n = (C.c_int32 * len(KERNEL_CLASSES))()
        self._check(LIB.k2_profile_decode(self.ctx, _ptr(tokens), batch, _ptr(next_tokens), ms, n,
                                          _stream(stream)))
        return dict(zip(KERNEL_CLASSES, ms)), dict(zip(KERNEL_CLASSES, n))


def greedy_head_noalloc(cfg: Config, lm_head, final_norm, x, logits, token, stream=None) -> int:
    """k2_greedy_head_noalloc: returns the k2 status (no context, no workspace).

    The tensors are checked here, since the C call reads raw pointers: x
    float32, logits float32 or None, token int32, lm_head and final_norm in
    the config's weight dtype, all contiguous CUDA tensors holding at least
    the elements the call touches (x and final_norm: hidden, lm_head:
    vocab * hidden, logits: vocab, token: 1); the call itself checks the
    config's shape.  A token of -1 after the call means a NaN logit or a
    bounded wait that ran out on the device.  ``x = None`` passes a null
    pointer through (the call refuses it)."""
    wdt = {K2_F32: torch.float32, K2_BF16: torch.bfloat16}.get(cfg.weight_dtype)

    def want(t, name, dtype, numel):
        if t is None:
            return
        if not (t.is_cuda and t.is_contiguous() and t.dtype == dtype and t.numel() >= numel):
            raise ValueError(f"greedy_head_noalloc: {name} must be a contiguous CUDA {dtype} tensor "
                             f"of at least {numel} elements, got {t.dtype} {tuple(t.shape)} on {t.device}")
    if wdt is not None:
        want(lm_head, "lm_head", wdt, cfg.vocab * cfg.hidden)
        want(final_norm, "final_norm", wdt, cfg.hidden)
    if cfg.hidden > 0 and cfg.vocab > 0:
        want(x, "x", torch.float32, cfg.hidden)
        want(logits, "logits", torch.float32, cfg.vocab)
    want(token, "token", torch.int32, 1)
    return LIB.k2_greedy_head_noalloc(C.byref(cfg), _ptr(lm_head), _ptr(final_norm), _ptr(x), _ptr(logits),
                                      _ptr(token), _stream(stream))


def philox(first: int, n: int, c1=0, c2=0, c3=0, key=0, stream=None) -> torch.Tensor:
    """k2_philox: [n, 4] uint32 words (as int64) of Philox4x32-10 for counters
    (first + i, c1, c2, c3) under the 64-bit key."""
    out = torch.empty(4 * n, dtype=torch.int32, device="cuda")
    st = LIB.k2_philox(first, n, c1, c2, c3, key, _ptr(out), _stream(stream))
    if st != K2_OK:
        raise K2Error(st, "k2_philox failed")
    return out.view(n, 4).cpu().to(torch.int64) & 0xFFFFFFFF


def quantize_fp8(src, stream=None):
    """k2_quantize_fp8 on a [rows, cols] bf16 device tensor: (codes uint8, scales fp32)."""
    rows, cols = src.shape
    codes = torch.empty(rows, cols, dtype=torch.uint8, device="cuda")
    scales = torch.empty(rows, dtype=torch.float32, device="cuda")
    st = LIB.k2_quantize_fp8(_ptr(src), rows, cols, _ptr(codes), _ptr(scales), _stream(stream))
    if st != K2_OK:
        raise K2Error(st, "k2_quantize_fp8 failed")
    return codes, scales


def quantize_q4(src, stream=None):
    """k2_quantize_q4 on a [rows, cols] bf16 device tensor: (codes int8 [rows, cols],
    scales fp32 [rows, ceil(cols / 64)])."""
    rows, cols = src.shape
    codes = torch.empty(rows, cols, dtype=torch.int8, device="cuda")
    scales = torch.empty(rows, (cols + 63) // 64, dtype=torch.float32, device="cuda")
    st = LIB.k2_quantize_q4(_ptr(src), rows, cols, _ptr(codes), _ptr(scales), _stream(stream))
    if st != K2_OK:
        raise K2Error(st, "k2_quantize_q4 failed")
    return codes, scales


# ---- a block-paged 8-bit cache for many requests -----------------------------------------------

_ROW_DTYPES = {torch.float32: K2_F32, torch.bfloat16: K2_BF16, torch.float16: K2_F16}


def _call(st):
    if st != K2_OK:
        raise K2Error(st, (LIB.k2_last_error(None) or b"").decode())


def _need(what, t, dtype, shape, device):
    """The C calls read raw pointers: a contiguous tensor of this type and shape
    (None: any extent) on the device (index) of the call."""
    if t.dtype is not dtype or t.get_device() != device or not t.is_contiguous() or len(t.shape) != len(shape) or any(
            n is not None and n != m for n, m in zip(shape, t.shape)):
        raise ValueError(f"{what} must be a contiguous {dtype} tensor of shape {tuple(shape)} on cuda:{device}, got "
                         f"{t.dtype} {tuple(t.shape)} on {t.device}")


# (a tensor on a CUDA device says that CUDA has been set up, which torch.cuda.current_device() checks every time)
_current_device, _current_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream


# The checks below run before every call of a serving loop, so they are written out with the cheapest tensor
# accessors (16 us of checks and marshalling per plan became 8); what fails one goes to _need, which says why.
def _device(t):
    """The call's device index: that of `t`, which has to be the current one (the
    C calls launch there)."""
    d = t.get_device()
    if d < 0 or d != _current_device():
        raise ValueError(f"the tensors must be on the current CUDA device, got {t.device}")
    return d


def _raw_stream(stream, dev):
    if stream is None:
        return _current_stream(dev)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


class PagedCache:
    """A pool of 8-bit blocks (k2_paged_kv) and the tensors that hold it: k and v
    [n_blocks, n_kv_heads, block_tokens, head_dim] (int8 or float8_e4m3fn codes),
    k_scale and v_scale [n_blocks, n_kv_heads] float32, and `flags`, an int32
    tensor of one word that device-side faults are OR-ed into (K2_PAGED_*)."""

    def __init__(self, n_blocks, block_tokens, n_kv_heads, head_dim, dtype="i8"):
        if dtype not in ("i8", "f8"):
            raise ValueError(f"a paged cache holds 'i8' or 'f8' codes, got {dtype!r}")
        shape = (n_blocks, n_kv_heads, block_tokens, head_dim)
        code = torch.int8 if dtype == "i8" else torch.float8_e4m3fn
        self._bind(torch.zeros(shape, dtype=torch.int8, device="cuda").view(code),
                   torch.zeros(shape, dtype=torch.int8, device="cuda").view(code),
                   torch.zeros(shape[:2], device="cuda"), torch.zeros(shape[:2], device="cuda"))

    @classmethod
    def of(cls, k, v, k_scale, v_scale):
        """A cache over tensors that the caller made (not copied)."""
        self = cls.__new__(cls)
        self._bind(k, v, k_scale, v_scale)
        return self

    def _bind(self, k, v, k_scale, v_scale):
        dev = _device(k)
        if k.dtype not in (torch.int8, torch.float8_e4m3fn) or k.dim() != 4:
            raise ValueError(f"k must be a 4-dimensional int8 or float8_e4m3fn tensor, got {k.dtype} {tuple(k.shape)}")
        _need("k", k, k.dtype, k.shape, dev)
        _need("v", v, k.dtype, k.shape, dev)
        _need("k_scale", k_scale, torch.float32, k.shape[:2], dev)
        _need("v_scale", v_scale, torch.float32, k.shape[:2], dev)
        self.k, self.v, self.k_scale, self.v_scale, self.device = k, v, k_scale, v_scale, dev
        self.flags = torch.zeros(1, dtype=torch.int32, device=dev)
        n, g, b, d = k.shape
        self.n_blocks, self.n_kv_heads, self.block_tokens, self.head_dim = n, g, b, d
        self.desc = PagedKv(k=k.data_ptr(), v=v.data_ptr(), k_scale=k_scale.data_ptr(), v_scale=v_scale.data_ptr(),
                            n_blocks=n, block_tokens=b, n_kv_heads=g, head_dim=d,
                            dtype=K2_I8 if k.dtype is torch.int8 else K2_F8, flags=self.flags.data_ptr())
        self._ref = C.addressof(self.desc)


def paged_plan(cached, fresh, table, free, free_count, block_tokens, *, kv_len, cu_new, slots, positions, status,
               free_count_out=None, stream=None):
    """k2_paged_plan on int32 device tensors: cached, fresh, kv_len [requests],
    table [requests, columns], free [blocks], free_count [1] (and free_count_out,
    default the same), cu_new [requests + 1], slots and positions [max_tokens],
    status [4].  kv_len may be cached."""
    dev = _device(cached)
    if free_count_out is None:
        free_count_out = free_count
    r, n = cached.numel(), slots.numel()
    i32 = torch.int32
    for t in (cached, fresh, table, free, free_count, free_count_out, kv_len, cu_new, slots, positions, status):
        if t.dtype is not i32 or t.get_device() != dev or not t.is_contiguous():
            break
    else:
        columns = table.shape
        if (cached.dim() == 1 and fresh.numel() == r and len(columns) == 2 and columns[0] == r and
                free_count.numel() == 1 and free_count_out.numel() == 1 and kv_len.numel() == r and
                cu_new.numel() == r + 1 and positions.numel() == n and status.numel() == 4):
            st = LIB.k2_paged_plan(cached.data_ptr(), fresh.data_ptr(), r, block_tokens, table.data_ptr(),
                                   columns[1], free.data_ptr(), free.numel(), free_count.data_ptr(),
                                   free_count_out.data_ptr(), kv_len.data_ptr(), cu_new.data_ptr(), slots.data_ptr(),
                                   positions.data_ptr(), n, status.data_ptr(), _raw_stream(stream, dev))
            if st:
                _call(st)
            return
    for what, t, shape in (("cached", cached, (r,)), ("fresh", fresh, (r,)), ("table", table, (r, None)),
                           ("free", free, (None,)), ("free_count", free_count, (1,)),
                           ("free_count_out", free_count_out, (1,)), ("kv_len", kv_len, (r,)),
                           ("cu_new", cu_new, (r + 1,)), ("slots", slots, (None,)),
                           ("positions", positions, (n,)), ("status", status, (4,))):
        _need(what, t, i32, shape, dev)
    raise ValueError("plan: tensors of another shape than the call's")


def _rows(what, t, dtype, heads, head_dim, device):
    """[tokens, heads, head_dim] rows whose tokens may be apart (a slice of packed rows): their number and distance"""
    if t.dtype is dtype and t.get_device() == device and t.dim() == 3:
        n, h, d = t.shape
        token, head, one = t.stride()
        if h == heads and d == head_dim and one == 1 and (heads == 1 or head == head_dim):
            return n, token
    raise ValueError(f"{what} must be [tokens, {heads}, {head_dim}] {dtype} rows on cuda:{device}, each row contiguous, "
                     f"got {t.dtype} {tuple(t.shape)} with strides {t.stride()} on {t.device}")


def paged_append(cache, k, v, slots, stream=None):
    """k2_paged_append: K and V rows [tokens, n_kv_heads, head_dim] (bf16, fp16 or
    fp32; tokens may be strided) to the int32 slots [tokens]."""
    dev = _device(k)
    if dev != cache.device:
        raise ValueError(f"the rows are on cuda:{dev}, the cache on cuda:{cache.device}")
    dtype = _ROW_DTYPES.get(k.dtype)
    if dtype is None:
        raise ValueError(f"k and v must be float32, bfloat16 or float16, got {k.dtype}")
    n, ks = _rows("k", k, k.dtype, cache.n_kv_heads, cache.head_dim, dev)
    m, vs = _rows("v", v, k.dtype, cache.n_kv_heads, cache.head_dim, dev)
    if m != n:
        raise ValueError(f"k has {n} rows, v {m}")
    if slots.dtype is not torch.int32 or slots.get_device() != dev or slots.numel() != n or not slots.is_contiguous():
        _need("slots", slots, torch.int32, (n,), dev)
    st = LIB.k2_paged_append(cache._ref, k.data_ptr(), v.data_ptr(), dtype, ks, vs, slots.data_ptr(), n,
                             _raw_stream(stream, dev))
    if st:
        _call(st)


def paged_workspace():
    """A zeroed workspace for paged_attention calls that do not overlap."""
    return torch.zeros(int(LIB.k2_paged_workspace_bytes()), dtype=torch.uint8, device="cuda")


def paged_attention(cache, q, out, cu_q, kv_len, table, max_q, workspace, scale=None, stream=None):
    """k2_paged_attention: q and out [tokens, n_heads, head_dim] (bf16 or fp16;
    tokens may be strided), cu_q [requests + 1], kv_len [requests], table
    [requests, columns] int32; max_q: the most queries of one request; scale:
    default head_dim ** -0.5."""
    dev = _device(q)
    if dev != cache.device:
        raise ValueError(f"the queries are on cuda:{dev}, the cache on cuda:{cache.device}")
    dtype = q.dtype
    if dtype is not torch.bfloat16 and dtype is not torch.float16:
        raise ValueError(f"q must be bfloat16 or float16, got {dtype}")
    heads, d = (q.shape[1] if q.dim() == 3 else 0), cache.head_dim
    n, qs = _rows("q", q, dtype, heads, d, dev)
    m, os_ = _rows("out", out, dtype, heads, d, dev)
    if m != n:
        raise ValueError(f"q has {n} rows, out {m}")
    r, i32 = kv_len.numel(), torch.int32
    for t in (cu_q, kv_len, table):
        if t.dtype is not i32 or t.get_device() != dev or not t.is_contiguous():
            break
    else:
        columns = table.shape
        if (cu_q.numel() == r + 1 and len(columns) == 2 and columns[0] == r and workspace.dtype is torch.uint8 and
                workspace.get_device() == dev and workspace.is_contiguous()):
            st = LIB.k2_paged_attention(cache._ref, q.data_ptr(), _ROW_DTYPES[dtype], qs, cu_q.data_ptr(),
                                        kv_len.data_ptr(), table.data_ptr(), columns[1], r, n, heads, max_q,
                                        d ** -0.5 if scale is None else scale, out.data_ptr(), os_,
                                        workspace.data_ptr(), workspace.numel(), _raw_stream(stream, dev))
            if st:
                _call(st)
            return
    _need("cu_q", cu_q, i32, (r + 1,), dev)
    _need("kv_len", kv_len, i32, (r,), dev)
    _need("table", table, i32, (r, None), dev)
    _need("workspace", workspace, torch.uint8, (None,), dev)
    raise ValueError("attention: tensors of another shape than the call's")


_RULES = struct.Struct("@PPPPqPPPPPiPqiP").pack  # a LogitRules, in a fifth of its constructor's time


def adjust_logits(logits, out=None, *, repetition=None, presence=None, frequency=None, ids=None, ids_len=None,
                  prompt_len=None, bias=None, mask=None, mask_row=None, stream=None):
    """k2_adjust_logits on logits [rows, vocab] fp32 (rows may be strided) into
    `out` (default: in place): repetition, presence, frequency [rows] fp32; ids
    [rows, n], ids_len, prompt_len [rows] int32; bias = (offsets [rows + 1], ids,
    values fp32); mask [masks, >= ceil(vocab / 32)] int32 words, mask_row [rows]."""
    dev = _device(logits)
    if out is None:
        out = logits
    f32, i32 = torch.float32, torch.int32
    rows, vocab = logits.shape if logits.dim() == 2 else (0, 0)
    ld, one = logits.stride() if logits.dim() == 2 else (0, 0)
    ld_out, one_out = (ld, one) if out is logits else out.stride() if out.dim() == 2 else (0, 0)
    if logits.dtype is not f32 or one != 1 or out is not logits and (
            out.dtype is not f32 or out.get_device() != dev or one_out != 1 or out.shape != logits.shape):
        raise ValueError(f"logits and out must be [rows, vocab] float32 rows on cuda:{dev}, got {logits.dtype} "
                         f"{tuple(logits.shape)} and {out.dtype} {tuple(out.shape)} on {out.device}")

    def fault(t, dtype, n):  # of a value per row
        return t.dtype is not dtype or t.get_device() != dev or t.numel() != n or not t.is_contiguous()
    rep = pres = freq = 0
    if repetition is not None:
        if fault(repetition, f32, rows):
            _need("repetition", repetition, f32, (rows,), dev)
        rep = repetition.data_ptr()
    if presence is not None:
        if fault(presence, f32, rows):
            _need("presence", presence, f32, (rows,), dev)
        pres = presence.data_ptr()
    if frequency is not None:
        if fault(frequency, f32, rows):
            _need("frequency", frequency, f32, (rows,), dev)
        freq = frequency.data_ptr()
    id_ptr = id_stride = id_len = id_prompt = 0
    if ids is not None:
        shape = ids.shape
        if ids.dtype is not i32 or ids.get_device() != dev or len(shape) != 2 or shape[0] != rows or \
                not ids.is_contiguous():
            _need("ids", ids, i32, (rows, None), dev)
        if ids_len is None:
            raise ValueError("ids need ids_len")
        if fault(ids_len, i32, rows):
            _need("ids_len", ids_len, i32, (rows,), dev)
        if prompt_len is not None:
            if fault(prompt_len, i32, rows):
                _need("prompt_len", prompt_len, i32, (rows,), dev)
            id_prompt = prompt_len.data_ptr()
        id_ptr, id_stride, id_len = ids.data_ptr(), shape[1], ids_len.data_ptr()
        if not rows * id_stride:  # no row holds a token: nothing to penalise
            rep = pres = freq = id_ptr = id_stride = id_len = id_prompt = 0
    b_off = b_ids = b_val = n_bias = 0
    if bias is not None:
        offset, bias_ids, values = bias
        n_bias = bias_ids.numel()
        if fault(offset, i32, rows + 1):
            _need("bias offsets", offset, i32, (rows + 1,), dev)
        if fault(bias_ids, i32, n_bias):
            _need("bias ids", bias_ids, i32, (n_bias,), dev)
        if fault(values, f32, n_bias):
            _need("bias values", values, f32, (n_bias,), dev)
        if n_bias:
            b_off, b_ids, b_val = offset.data_ptr(), bias_ids.data_ptr(), values.data_ptr()
    m_ptr = m_stride = n_masks = m_row = 0
    if mask is not None:
        if mask.dtype is not i32 or mask.get_device() != dev or mask.dim() != 2 or not mask.is_contiguous():
            _need("mask", mask, i32, (None, None), dev)
        m_ptr, (n_masks, m_stride) = mask.data_ptr(), mask.shape
        if m_stride < (vocab + 31) // 32 or (mask_row is None and n_masks < rows):
            raise ValueError(f"mask must have {(vocab + 31) // 32} words for each of its rows (and a row for each of the "
                             f"logits without mask_row), got {tuple(mask.shape)}")
        if mask_row is not None:
            if fault(mask_row, i32, rows):
                _need("mask_row", mask_row, i32, (rows,), dev)
            m_row = mask_row.data_ptr()
    u = _RULES(rep, pres, freq, id_ptr, id_stride, id_len, id_prompt, b_off, b_ids, b_val, n_bias, m_ptr, m_stride, n_masks,
               m_row)
    st = LIB.k2_adjust_logits(u, logits.data_ptr(), ld, out.data_ptr(), ld_out, rows, vocab, _raw_stream(stream, dev))
    if st:
        _call(st)


def spec_draft(tokens, max_draft=8) -> list:
    """k2_spec_draft (host only)."""
    ids = (C.c_int32 * max(len(tokens), 1))(*[int(t) for t in tokens])
    out = (C.c_int32 * 8)()
    n = LIB.k2_spec_draft(ids, len(tokens), max_draft, out)
    return list(out[:n])


def peek_state(cfg: Config, state) -> tuple:
    """k2_kv_peek: (cached rows, token ids) of a state in a uint8 CPU tensor,
    or (-1, -1) if it cannot be loaded into a context of cfg's model."""
    state = state.contiguous()
    cached, n_tok = C.c_int32(-1), C.c_int32(-1)
    if LIB.k2_kv_peek(C.byref(cfg), state.data_ptr(), state.numel(), C.byref(cached), C.byref(n_tok)) != K2_OK:
        return -1, -1
    return cached.value, n_tok.value


def save_state_file(path: str, state) -> None:
    with open(path, "wb") as f:
        f.write(state.numpy().tobytes())


def load_state_file(path: str) -> torch.Tensor:
    with open(path, "rb") as f:
        data = f.read()
    return torch.frombuffer(bytearray(data), dtype=torch.uint8)


def device_view(ptr: int, numel: int, dtype: torch.dtype) -> torch.Tensor:
    """A torch tensor over device memory inside a k2 workspace (test hooks)."""
    storage_bytes = numel * torch.empty((), dtype=dtype).element_size()

    class _Holder:
        __cuda_array_interface__ = {
            "shape": (storage_bytes,), "typestr": "|u1", "data": (ptr, False), "version": 3}
    return torch.as_tensor(_Holder(), device="cuda").view(dtype)[:numel]
