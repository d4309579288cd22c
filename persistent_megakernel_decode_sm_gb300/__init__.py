"""Python binding of the persistent decode megakernel's C ABI (include/mk.h).

Argument marshalling only: every step of the decode runs in the CUDA kernels of libmk.so.
PyTorch supplies device memory and the stream.  There is no fallback: if libmk.so is missing
or fails to load, importing this package raises.

Low level: the mk_* functions of the C ABI under the same names (``lib.mk_bind`` ...).
High level:
    sched = Schedule(cfg, sm_count)               # mk_build_schedule
    dec = Decoder(sched, weights, kv)             # allocates counters/scratch with torch, mk_bind
    dec.prefill([prompt[:-1]])                    # mk_prefill: the prompt into the KV cache
    nxt = dec.step(tokens, pos, logits)           # mk_decode_step (synchronous)
    dec.launch(tokens, pos, logits, next_dev)     # mk_launch_step (asynchronous)
Prompt operators (asynchronous on torch's current stream of the tensors' device):
    y = linear(x, w, bias, activation, residual)  # mk_linear
    o = attend(q, kv, q_lens, kv_lens, window=..) # mk_attend
    y = adapted_linear(x, w, adapters, index)     # mk_linear_adapted
    q = rope_append(qkv, kv, positions, slots, freqs)                             # mk_rope_append
    slots, positions, sequences, first = assign_pages(ring, ends, table, lens, new_lens, block_size, max_tokens)   # mk_assign_pages
"""
from __future__ import annotations

import array
import ctypes
import importlib.util
import os
import struct
from typing import List, Optional, Sequence

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmk.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it first (python -c 'import __graft_entry__ as g; g.build()')")
lib = ctypes.CDLL(LIB_PATH)
# Built where Python's headers are: without it linear() and attend() make their calls from Python.
_mk_call = importlib.import_module("._mk_call", __name__) if importlib.util.find_spec(__name__ + "._mk_call") else None

MK_OK, MK_ERR_ARG, MK_ERR_CAPACITY, MK_ERR_RESOURCES, MK_ERR_CUDA, MK_ERR_TIMEOUT, MK_ERR_OPCODE, \
    MK_ERR_BOUNDS, MK_ERR_POISONED = range(9)
STATUS_NAMES = ["MK_OK", "MK_ERR_ARG", "MK_ERR_CAPACITY", "MK_ERR_RESOURCES", "MK_ERR_CUDA", "MK_ERR_TIMEOUT",
                "MK_ERR_OPCODE", "MK_ERR_BOUNDS", "MK_ERR_POISONED"]
SYNC_TAGS, SYNC_COUNTERS = 0, 1   # mk_sync_mode
BF16, F32 = 0, 1                  # mk_dtype
ACTIVATIONS = {None: 0, "silu": 1, "gelu": 2, "swiglu": 3}   # mk_activation
ATTEND_MAX_BATCH = 256            # MK_ATTEND_MAX_BATCH
ADAPTERS_MAX_RANK = 256           # MK_ADAPTERS_MAX_RANK
PAGES_MAX_BATCH = 1024            # MK_PAGES_MAX_BATCH

EXPORTS = ["mk_build_schedule", "mk_schedule_queues", "mk_schedule_counters", "mk_schedule_patch",
           "mk_scratch_bytes", "mk_schedule_free", "mk_bind", "mk_set_timeout", "mk_decode_step",
           "mk_launch_step", "mk_ctx_status", "mk_device_sm_count", "mk_last_error", "mk_unbind", "mk_set_trace",
           "mk_decode_step_static", "mk_set_sync", "mk_decode_steps", "mk_bind_paged", "mk_schedule_attn_chunk",
           "mk_decode_persistent_start", "mk_decode_persistent_stop", "mk_decode_persistent_progress",
           "mk_decode_persistent_wait", "mk_rebind_schedule", "mk_linear", "mk_linear_plan", "mk_attend",
           "mk_attend_workspace", "mk_prefill", "mk_prefill_workspace", "mk_linear_adapted", "mk_linear_adapted_workspace",
           "mk_rope_append", "mk_assign_pages"]


class MkError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS_NAMES[status] if 0 <= status < 9 else status}: {msg}")
        self.status = status


class mk_model_cfg(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("n_layers", "hidden", "n_q_heads", "n_kv_heads", "head_dim",
                                              "ffn", "vocab", "tied_embeddings", "batch", "max_seq")] + \
               [("rms_eps", ctypes.c_double), ("rope_theta", ctypes.c_double)]


class mk_sched_opts(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("page_bytes", "tile_bytes", "attn_chunk", "rows_qkv", "rows_o",
                                              "pairs_up", "rows_down", "rows_lm")] + \
               [("shuffle_seed", ctypes.c_uint64), ("kv_limit", ctypes.c_int32 * 8)]


_P = ctypes.c_void_p


class mk_weights(ctypes.Structure):
    _fields_ = [("embed", _P), ("lm_head", _P), ("final_norm", _P), ("attn_norm", _P), ("wqkv", _P),
                ("wo", _P), ("mlp_norm", _P), ("wgate_up", _P), ("wdown", _P)]


class mk_kv(ctypes.Structure):
    _fields_ = [("k", _P), ("v", _P), ("batch_stride", ctypes.c_int64), ("layer_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


class mk_kv_pages(ctypes.Structure):
    _fields_ = [("block_table", _P), ("block_size", ctypes.c_int32), ("max_blocks", ctypes.c_int32),
                ("n_blocks", ctypes.c_int32)]


_I32P = ctypes.POINTER(ctypes.c_int32)


class mk_linear_args(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("rows", "n", "k", "activation")] + \
               [("x", _P), ("x_stride", ctypes.c_int64), ("w", _P), ("bias", _P), ("residual", _P),
                ("residual_stride", ctypes.c_int64), ("residual_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("out", _P), ("out_stride", ctypes.c_int64), ("status", _P)]


class mk_attend_args(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("n_q_heads", "n_kv_heads", "head_dim", "batch")] + \
               [("q_lens", _I32P), ("kv_lens", _I32P), ("q", _P), ("q_stride", ctypes.c_int64), ("out", _P),
                ("out_stride", ctypes.c_int64), ("kv", ctypes.POINTER(mk_kv)), ("pages", ctypes.POINTER(mk_kv_pages))] + \
               [(n, ctypes.c_int32) for n in ("layer", "max_seq", "window", "sinks", "shared_prefix")] + \
               [("scale", ctypes.c_float), ("status", _P)]


class mk_adapters(ctypes.Structure):
    _fields_ = [("n_adapters", ctypes.c_int32), ("rank", ctypes.c_int32), ("down", _P), ("up", _P), ("scale", _P), ("index", _P)]


class mk_rope_args(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("tokens", "n_q_heads", "n_kv_heads", "head_dim")] + \
               [("qkv", _P), ("qkv_stride", ctypes.c_int64), ("qkv_dtype", ctypes.c_int32), ("rotary", ctypes.c_int32),
                ("q_gain", _P), ("k_gain", _P), ("eps", ctypes.c_float), ("neighbours", ctypes.c_int32), ("n_axes", ctypes.c_int32),
                ("sections", _I32P), ("freqs", ctypes.POINTER(ctypes.c_double)), ("positions", _P),
                ("position_stride", ctypes.c_int64), ("slots", _P), ("kv", ctypes.POINTER(mk_kv)), ("layer", ctypes.c_int32),
                ("max_seq", ctypes.c_int32), ("sequences", ctypes.c_int32), ("q", _P), ("q_stride", ctypes.c_int64), ("status", _P)]


class mk_pages_args(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("batch", "block_size", "max_blocks", "n_blocks", "shared_prefix", "max_tokens")] + \
               [(n, _P) for n in ("ring", "ends", "ends_out", "table", "lens", "new_lens", "slots", "positions", "sequences",
                                  "first", "status")]


lib.mk_build_schedule.restype = ctypes.c_int
lib.mk_build_schedule.argtypes = [ctypes.POINTER(mk_model_cfg), ctypes.c_int32, ctypes.POINTER(mk_sched_opts),
                                  ctypes.POINTER(_P)]
lib.mk_schedule_queues.restype = ctypes.c_int
lib.mk_schedule_queues.argtypes = [_P, ctypes.POINTER(_I32P), _I32P, _I32P]
lib.mk_schedule_counters.restype = ctypes.c_int
lib.mk_schedule_counters.argtypes = [_P, ctypes.POINTER(ctypes.POINTER(ctypes.c_uint32)), _I32P]
lib.mk_schedule_attn_chunk.restype = ctypes.c_int
lib.mk_schedule_attn_chunk.argtypes = [_P, _I32P]
lib.mk_schedule_patch.restype = ctypes.c_int
lib.mk_schedule_patch.argtypes = [_P, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32]
lib.mk_scratch_bytes.restype = ctypes.c_size_t
lib.mk_scratch_bytes.argtypes = [_P]
lib.mk_schedule_free.restype = None
lib.mk_schedule_free.argtypes = [_P]
lib.mk_bind.restype = ctypes.c_int
lib.mk_bind.argtypes = [_P, ctypes.POINTER(mk_weights), ctypes.POINTER(mk_kv), _P, _P, _P, ctypes.POINTER(_P)]
lib.mk_bind_paged.restype = ctypes.c_int
lib.mk_bind_paged.argtypes = [_P, ctypes.POINTER(mk_weights), ctypes.POINTER(mk_kv), ctypes.POINTER(mk_kv_pages), _P,
                              _P, _P, ctypes.POINTER(_P)]
lib.mk_set_timeout.restype = ctypes.c_int
lib.mk_set_timeout.argtypes = [_P, ctypes.c_uint64]
lib.mk_decode_step.restype = ctypes.c_int
lib.mk_decode_step.argtypes = [_P, _I32P, _I32P, _P, _I32P]
lib.mk_launch_step.restype = ctypes.c_int
lib.mk_launch_step.argtypes = [_P, _I32P, _I32P, _P, _P]
lib.mk_decode_steps.restype = ctypes.c_int
lib.mk_decode_steps.argtypes = [_P, _I32P, _I32P, ctypes.c_int32, _P, _P, _I32P]
lib.mk_decode_persistent_start.restype = ctypes.c_int
lib.mk_decode_persistent_start.argtypes = [_P, _I32P, _I32P, ctypes.c_int32, _P, _P]
lib.mk_decode_persistent_stop.restype = ctypes.c_int
lib.mk_decode_persistent_stop.argtypes = [_P]
lib.mk_decode_persistent_progress.restype = ctypes.c_int
lib.mk_decode_persistent_progress.argtypes = [_P, _I32P]
lib.mk_decode_persistent_wait.restype = ctypes.c_int
lib.mk_decode_persistent_wait.argtypes = [_P, _I32P, _I32P]
lib.mk_rebind_schedule.restype = ctypes.c_int
lib.mk_rebind_schedule.argtypes = [_P, _P]
lib.mk_ctx_status.restype = ctypes.c_int
lib.mk_ctx_status.argtypes = [_P, _I32P]
lib.mk_device_sm_count.restype = ctypes.c_int
lib.mk_device_sm_count.argtypes = [_I32P]
lib.mk_last_error.restype = ctypes.c_char_p
lib.mk_last_error.argtypes = []
lib.mk_decode_step_static.restype = ctypes.c_int
lib.mk_decode_step_static.argtypes = [_P, _I32P, _I32P, _P, _I32P]
lib.mk_set_trace.restype = ctypes.c_int
lib.mk_set_trace.argtypes = [_P, _P]
lib.mk_set_sync.restype = ctypes.c_int
lib.mk_set_sync.argtypes = [_P, ctypes.c_int32]
lib.mk_linear.restype = ctypes.c_int
lib.mk_linear.argtypes = [_P, _P]   # (a packed mk_linear_args)
lib.mk_linear_plan.restype = ctypes.c_int
lib.mk_linear_plan.argtypes = [_P, _I32P]
lib.mk_attend_workspace.restype = ctypes.c_size_t
lib.mk_attend_workspace.argtypes = [_P]
lib.mk_attend.restype = ctypes.c_int
lib.mk_attend.argtypes = [_P, _P, ctypes.c_size_t, _P]
lib.mk_prefill_workspace.restype = ctypes.c_size_t
lib.mk_prefill_workspace.argtypes = [_P, _I32P, _I32P, ctypes.c_int32]
lib.mk_prefill.restype = ctypes.c_int
lib.mk_prefill.argtypes = [_P, _I32P, _I32P, _I32P, ctypes.c_int32, _P, ctypes.c_size_t]
lib.mk_linear_adapted_workspace.restype = ctypes.c_size_t
lib.mk_linear_adapted_workspace.argtypes = [_P, _P]   # (a packed mk_linear_args, a packed mk_adapters)
lib.mk_linear_adapted.restype = ctypes.c_int
lib.mk_linear_adapted.argtypes = [_P, _P, _P, ctypes.c_size_t, _P]
lib.mk_rope_append.restype = ctypes.c_int
lib.mk_rope_append.argtypes = [_P, _P]
lib.mk_assign_pages.restype = ctypes.c_int
lib.mk_assign_pages.argtypes = [_P, _P]
lib.mk_unbind.restype = None
lib.mk_unbind.argtypes = [_P]


def _check(st: int):
    if st != MK_OK:
        raise MkError(st, lib.mk_last_error().decode(errors="replace"))


def make_cfg(cfg) -> mk_model_cfg:
    """workload.ModelConfig (or any object with the same fields) -> mk_model_cfg."""
    return mk_model_cfg(cfg.n_layers, cfg.hidden, cfg.n_q_heads, cfg.n_kv_heads, cfg.head_dim, cfg.ffn, cfg.vocab,
                        int(cfg.tied_embeddings), cfg.batch, cfg.max_seq, float(cfg.rms_eps), float(cfg.rope_theta))


def device_sm_count() -> int:
    n = ctypes.c_int32()
    _check(lib.mk_device_sm_count(ctypes.byref(n)))
    return n.value


class Schedule:
    """Host schedule object (mk_build_schedule); frees itself."""

    def __init__(self, cfg, sm_count: int, page_bytes: int = 0, tile_bytes: int = 0, attn_chunk: int = 0,
                 rows_qkv: int = 0, rows_o: int = 0, pairs_up: int = 0, rows_down: int = 0, rows_lm: int = 0,
                 shuffle_seed: int = 0, kv_limit: Optional[Sequence[int]] = None):
        self.cfg = cfg
        self._c = make_cfg(cfg)
        lim = list(kv_limit or []) + [0] * (8 - len(kv_limit or []))
        o = mk_sched_opts(page_bytes, tile_bytes, attn_chunk, rows_qkv, rows_o, pairs_up, rows_down, rows_lm,
                          shuffle_seed, (ctypes.c_int32 * 8)(*lim))
        h = _P()
        _check(lib.mk_build_schedule(ctypes.byref(self._c), int(sm_count), ctypes.byref(o), ctypes.byref(h)))
        self.handle = h

    def __del__(self):
        if getattr(self, "handle", None):
            lib.mk_schedule_free(self.handle)
            self.handle = None

    def queues(self) -> np.ndarray:
        q, S, Q = _I32P(), ctypes.c_int32(), ctypes.c_int32()
        _check(lib.mk_schedule_queues(self.handle, ctypes.byref(q), ctypes.byref(S), ctypes.byref(Q)))
        return np.ctypeslib.as_array(q, shape=(S.value, Q.value, 32)).copy()

    def totals(self) -> np.ndarray:
        t, n = ctypes.POINTER(ctypes.c_uint32)(), ctypes.c_int32()
        _check(lib.mk_schedule_counters(self.handle, ctypes.byref(t), ctypes.byref(n)))
        return np.ctypeslib.as_array(t, shape=(n.value,)).copy()

    @property
    def n_counters(self) -> int:
        return int(self.totals().size)

    @property
    def attn_chunk(self) -> int:
        """KV positions per split-K attention tile (the block size of a paged KV cache)."""
        v = ctypes.c_int32()
        _check(lib.mk_schedule_attn_chunk(self.handle, ctypes.byref(v)))
        return v.value

    @property
    def scratch_bytes(self) -> int:
        return int(lib.mk_scratch_bytes(self.handle))

    def patch(self, sm: int, slot: int, word: int, value: int):
        _check(lib.mk_schedule_patch(self.handle, sm, slot, word, value))


def _ptr(t) -> int:
    return t.data_ptr()


class Decoder:
    """A bound context: borrows the weights / KV tensors, owns counters, scratch and logits (torch).

    ``pages`` (optional) binds a paged KV cache: a tuple (block_table, block_size, n_blocks) with
    block_table a CUDA int32 tensor [batch, max_blocks]; kv.k / kv.v are then the block pools,
    shaped [n_layers, n_kv_heads, n_blocks * block_size, head_dim].  ``scratch`` (optional) is the
    caller's device scratch (at least ``sched.scratch_bytes`` bytes, 256-byte aligned); by default
    one is allocated."""

    def __init__(self, sched: Schedule, weights, kv, stream=None, timeout_ns: Optional[int] = None, pages=None,
                 scratch=None):
        import torch
        cfg = sched.cfg
        dev = weights.embed.device
        assert dev.type == "cuda", "weights must be CUDA tensors"
        self.cfg, self.sched, self.weights, self.kv = cfg, sched, weights, kv
        L = cfg.n_layers
        self._tabs = {k: (_P * L)(*[_ptr(t) for t in getattr(weights, k)])
                      for k in ("attn_norm", "wqkv", "wo", "mlp_norm", "wgate_up", "wdown")}
        self._w = mk_weights(_ptr(weights.embed), _ptr(weights.lm_head), _ptr(weights.final_norm),
                             *[ctypes.cast(self._tabs[k], _P)
                               for k in ("attn_norm", "wqkv", "wo", "mlp_norm", "wgate_up", "wdown")])
        for t in (kv.k, kv.v):
            assert t.is_contiguous() and t.dtype == torch.bfloat16 and t.device == dev
        st = kv.k.stride()
        if pages is None:
            self._kv = mk_kv(_ptr(kv.k), _ptr(kv.v), st[0], st[1], st[2])
            self._pages = None
        else:
            table, block_size, n_blocks = pages
            assert table.dtype == torch.int32 and table.device == dev and table.is_contiguous()
            self._kv = mk_kv(_ptr(kv.k), _ptr(kv.v), 0, st[0], st[1])
            self._pages = mk_kv_pages(_ptr(table), int(block_size), int(table.shape[-1]), int(n_blocks))
            self._table = table
        self.counters = torch.zeros(sched.n_counters, dtype=torch.int32, device=dev)
        if scratch is None:
            scratch = torch.empty(sched.scratch_bytes // 4 + 64, dtype=torch.int32, device=dev)
        assert scratch.device == dev and scratch.numel() * scratch.element_size() >= sched.scratch_bytes
        self.scratch = scratch
        self.logits = torch.empty((cfg.batch, cfg.vocab), dtype=torch.float32, device=dev)
        self.stream = stream if stream is not None else torch.cuda.current_stream(dev)
        h = _P()
        _check(lib.mk_bind_paged(sched.handle, ctypes.byref(self._w), ctypes.byref(self._kv),
                                 ctypes.byref(self._pages) if self._pages is not None else None, _ptr(self.counters),
                                 _ptr(self.scratch), ctypes.c_void_p(self.stream.cuda_stream), ctypes.byref(h)))
        self.handle = h
        if timeout_ns is not None:
            self.set_timeout(timeout_ns)

    def close(self):
        if getattr(self, "handle", None):
            lib.mk_unbind(self.handle)
            self.handle = None

    def __del__(self):
        self.close()

    def set_timeout(self, ns: int):
        _check(lib.mk_set_timeout(self.handle, int(ns)))

    def _arrays(self, tokens, pos):
        B = self.cfg.batch
        t = (ctypes.c_int32 * B)(*[int(v) for v in tokens])
        p = (ctypes.c_int32 * B)(*[int(v) for v in pos])
        assert len(tokens) == B and len(pos) == B
        return t, p

    def step(self, tokens: Sequence[int], pos: Sequence[int], logits=None) -> List[int]:
        """mk_decode_step: one synchronous step; logits land in ``logits`` (default self.logits)."""
        lg = self.logits if logits is None else logits
        t, p = self._arrays(tokens, pos)
        out = (ctypes.c_int32 * self.cfg.batch)()
        _check(lib.mk_decode_step(self.handle, t, p, _ptr(lg), out))
        return list(out)

    def step_static(self, tokens: Sequence[int], pos: Sequence[int], logits=None) -> List[int]:
        """mk_decode_step_static: one synchronous step using the library's static device scratch."""
        lg = self.logits if logits is None else logits
        t, p = self._arrays(tokens, pos)
        out = (ctypes.c_int32 * self.cfg.batch)()
        _check(lib.mk_decode_step_static(self.handle, t, p, _ptr(lg), out))
        return list(out)

    def steps(self, tokens: Sequence[int], pos: Sequence[int], n_steps: int, logits=None,
              tokens_dev=None) -> List[List[int]]:
        """mk_decode_steps: n_steps chained greedy steps (each step's token feeds the next on the
        device), one host synchronisation.  Returns the greedy tokens per step ([n_steps][batch]);
        ``logits`` (default self.logits) holds the last step's logits."""
        import torch
        B = self.cfg.batch
        lg = self.logits if logits is None else logits
        if tokens_dev is None:
            tokens_dev = torch.empty(n_steps * B, dtype=torch.int32, device=lg.device)
        t, p = self._arrays(tokens, pos)
        out = (ctypes.c_int32 * (max(n_steps, 1) * B))()
        _check(lib.mk_decode_steps(self.handle, t, p, int(n_steps), _ptr(lg), _ptr(tokens_dev), out))
        return [list(out[i * B:(i + 1) * B]) for i in range(n_steps)]

    def prefill(self, tokens: Sequence[Sequence[int]], pos: Optional[Sequence[int]] = None, shared_prefix: int = 0,
                chunk: int = 4096, workspace=None):
        """mk_prefill: fills the KV cache with the prompt tokens of each sequence (lists, one per sequence,
        possibly empty) from position pos[b] on (default 0), in pieces of at most ``chunk`` tokens a
        sequence, and waits for it.  Leave a prompt's last token to ``step``: it gives the logits.
        shared_prefix: the first positions, the same for every sequence and already cached."""
        import torch
        B, dev = self.cfg.batch, self.counters.device
        pos = list(pos) if pos is not None else [0] * B
        if len(tokens) != B or len(pos) != B:
            raise ValueError(f"tokens and pos must have an entry for each of {B} sequences")
        if chunk < 1:
            raise ValueError("chunk must be positive")
        tokens = [array.array("i", t) for t in tokens]
        at = [0] * B
        with torch.cuda.device(dev):
            while any(a < len(t) for a, t in zip(at, tokens)):
                n = [min(chunk, len(t) - a) for a, t in zip(at, tokens)]
                flat = array.array("i")
                for a, k, t in zip(at, n, tokens):
                    flat.extend(t[a:a + k])
                c_t = (ctypes.c_int32 * len(flat)).from_buffer(flat)
                c_n, c_p = (ctypes.c_int32 * B)(*n), (ctypes.c_int32 * B)(*[p + a for p, a in zip(pos, at)])
                need = int(lib.mk_prefill_workspace(self.handle, c_n, c_p, int(shared_prefix)))
                ws = workspace
                if ws is None:   # (torch keeps it for this stream's later use: freed in stream order)
                    with torch.cuda.stream(self.stream):
                        ws = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
                _check(lib.mk_prefill(self.handle, c_t, c_n, c_p, int(shared_prefix), _ptr(ws), ws.numel() * ws.element_size()))
                at = [a + k for a, k in zip(at, n)]
            self.status()

    def rebind(self, sched: "Schedule"):
        """mk_rebind_schedule: continue on another schedule of the same model and SM count (new KV
        windows: the variable-length re-planning).  The schedule object must outlive its use."""
        _check(lib.mk_rebind_schedule(self.handle, sched.handle))
        self.sched = sched

    def persistent_start(self, tokens: Sequence[int], pos: Sequence[int], n_steps: int, logits=None,
                         tokens_dev=None):
        """mk_decode_persistent_start: one resident launch of up to n_steps chained greedy steps,
        enqueued on the bound stream.  Returns the device token buffer ([n_steps * batch] int32);
        keep it alive until persistent_wait."""
        import torch
        B = self.cfg.batch
        lg = self.logits if logits is None else logits
        if tokens_dev is None:
            tokens_dev = torch.empty(max(int(n_steps), 1) * B, dtype=torch.int32, device=lg.device)
        t, p = self._arrays(tokens, pos)
        _check(lib.mk_decode_persistent_start(self.handle, t, p, int(n_steps), _ptr(lg), _ptr(tokens_dev)))
        self._run = (int(n_steps), tokens_dev)
        return tokens_dev

    def persistent_stop(self):
        """mk_decode_persistent_stop: the launch in flight ends after the step it is deciding."""
        _check(lib.mk_decode_persistent_stop(self.handle))

    def persistent_progress(self) -> int:
        """mk_decode_persistent_progress: steps finished so far (no wait)."""
        out = ctypes.c_int32(0)
        _check(lib.mk_decode_persistent_progress(self.handle, ctypes.byref(out)))
        return out.value

    def persistent_wait(self) -> List[List[int]]:
        """mk_decode_persistent_wait: waits for the launch; returns the greedy tokens of the steps
        it ran ([steps][batch])."""
        B = self.cfg.batch
        n_steps = self._run[0] if getattr(self, "_run", None) else 1
        done = ctypes.c_int32(0)
        out = (ctypes.c_int32 * (n_steps * B))()
        st = lib.mk_decode_persistent_wait(self.handle, ctypes.byref(done), out)
        self._run = None
        _check(st)
        return [list(out[i * B:(i + 1) * B]) for i in range(done.value)]

    def persistent(self, tokens: Sequence[int], pos: Sequence[int], n_steps: int, logits=None,
                   tokens_dev=None) -> List[List[int]]:
        """One persistent launch of n_steps steps, waited for: the tokens per step."""
        self.persistent_start(tokens, pos, n_steps, logits, tokens_dev)
        return self.persistent_wait()

    def launch(self, tokens: Sequence[int], pos: Sequence[int], logits=None, next_dev=None):
        """mk_launch_step: enqueue one step on the bound stream."""
        lg = self.logits if logits is None else logits
        t, p = self._arrays(tokens, pos)
        _check(lib.mk_launch_step(self.handle, t, p, _ptr(lg), _ptr(next_dev) if next_dev is not None else None))

    def status(self) -> List[int]:
        """mk_ctx_status: waits for the stream; raises MkError on a device error. Returns the info words."""
        info = (ctypes.c_int32 * 8)()
        st = lib.mk_ctx_status(self.handle, info)
        if st != MK_OK:
            raise MkError(st, lib.mk_last_error().decode(errors="replace"))
        return list(info)

    def set_sync(self, mode: str):
        """mk_set_sync: "tags" (epoch-tagged activations, the default) or "counters" (every
        instruction waits its completion counters first)."""
        modes = {"tags": SYNC_TAGS, "counters": SYNC_COUNTERS}
        if mode not in modes:
            raise ValueError(f"sync mode {mode!r}: expected one of {sorted(modes)}")
        _check(lib.mk_set_sync(self.handle, modes[mode]))

    def set_trace(self, buf):
        """mk_set_trace: buf is a CUDA int64 tensor of S*Q*8 elements, or None to stop tracing."""
        _check(lib.mk_set_trace(self.handle, _ptr(buf) if buf is not None else None))

    def status_code(self):
        info = (ctypes.c_int32 * 8)()
        st = lib.mk_ctx_status(self.handle, info)
        return st, list(info)


# ---- prompt operators ------------------------------------------------------------------------
# A call's host time counts beside kernels of a few microseconds, so the common call is checked and made in C
# (csrc/mk_python.c).  What that does not take comes here: the same checks, which say what is wrong, and calls
# for another device than the current one.  Argument structs are packed in one go (native alignment, the layouts
# of mk_linear_args and mk_attend_args).  They record no gradients, whatever their operands' requires_grad: the
# framework runs models, it does not train them.

_LINEAR_ARGS = struct.Struct("@4iPqPPPq2iPqP")
_ATTEND_ARGS = struct.Struct("@4iPPPqPqPP5ifP")
_ADAPTERS = struct.Struct("@2i4P")
_ROPE_ARGS = struct.Struct("@4iPq2iPPf2iPPPqPP3iPqP")
_PAGES_ARGS = struct.Struct("@6i11P")
assert _ADAPTERS.size == ctypes.sizeof(mk_adapters) and _ROPE_ARGS.size == ctypes.sizeof(mk_rope_args)
assert _PAGES_ARGS.size == ctypes.sizeof(mk_pages_args)
assert _LINEAR_ARGS.size == ctypes.sizeof(mk_linear_args) and _ATTEND_ARGS.size == ctypes.sizeof(mk_attend_args)
assert ctypes.sizeof(mk_kv) == 40 and ctypes.sizeof(mk_kv_pages) == 24   # five 64-bit words, three (packed below)


def _operand(t, name, dtypes, device, dim):
    """(shape, strides) of an operand: a CUDA tensor of one of `dtypes` on `device` (an ordinal) with
    `dim` dimensions, the last one contiguous."""
    shape, strides = t.shape, t.stride()
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be one of {dtypes}, not {t.dtype}")
    if t.get_device() != device or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor on the first operand's device, not on {t.device}")
    if len(shape) != dim:
        raise ValueError(f"{name} must have {dim} dimensions, not {len(shape)}")
    if strides[-1] != 1 and shape[-1] > 1:
        raise ValueError(f"{name}: its last dimension must be contiguous")
    return shape, strides


class _NoCallModule:   # (leaves every call to Python)
    @staticmethod
    def linear(*args):
        return None

    attend = adapted_linear = rope_append = assign_pages = linear


_fast = None   # _mk_call, once it has torch's objects


def _setup():
    global _fast
    if _mk_call is None:
        _fast = _NoCallModule
        return _fast
    import torch
    c = torch._C
    _mk_call.setup(*(ctypes.cast(f, _P).value for f in (lib.mk_linear, lib.mk_attend, lib.mk_attend_workspace, lib.mk_linear_adapted,
                                                        lib.mk_linear_adapted_workspace, lib.mk_rope_append, lib.mk_assign_pages)),
                   torch.bfloat16, torch.float32, torch.float64, torch.int32, torch.empty, c._cuda_getCurrentRawStream, c._cuda_getDevice,
                   c._cuda_cudaCachingAllocator_raw_alloc, c._cuda_cudaCachingAllocator_raw_delete)
    _fast = _mk_call
    return _fast


def _status_ptr(status, device):
    if status is None:
        return 0
    import torch
    if _operand(status, "status", (torch.int32,), device, 1)[0][0] < 1:
        raise ValueError("status must hold one int32")
    return status.data_ptr()


def _launch(device: int, call, *args):
    """call(*args, stream) with `device` current and torch's current stream of it."""
    import torch
    stream = torch._C._cuda_getCurrentRawStream(device)
    if torch._C._cuda_getDevice() == device:
        st = call(*args, stream)
    else:
        with torch.cuda.device(device):
            st = call(*args, stream)
    if st:
        _check(st)


def linear(x, weight, bias=None, activation: Optional[str] = None, residual=None, out=None, out_dtype=None, status=None):
    """mk_linear: act(x @ weight.T + bias) + residual, in fp32, rounded once to the output's type.

    x [rows, k] bf16 (rows may be strided by a multiple of 8 elements), weight [n, k] bf16
    contiguous -- [2 n, k] with activation "swiglu": n gate rows, then n up rows, silu(gate) * up --
    bias bf16 [n] ([2 n]), residual bf16 or fp32 [rows, n] (or an expanded row).  activation: None,
    "silu", "gelu" (the erf form) or "swiglu".  out: a bf16 or fp32 [rows, n] tensor, which may be
    the residual itself; by default one of out_dtype (bf16) is allocated.  Returns out.

    status: a CUDA int32 tensor of one element, zeroed by the caller, that receives an mk_status when the
    device meets an error (MK_ERR_TIMEOUT: out is not valid).  Without it such an error leaves no trace.
    No gradients are recorded."""
    y = (_fast or _setup()).linear(x, weight, bias, activation, residual, out, out_dtype, status)
    if y is not None:
        return y
    dev, out, args = _linear_args(x, weight, bias, activation, residual, out, out_dtype, status)
    _launch(dev, lib.mk_linear, args)
    return out


def _linear_args(x, weight, bias, activation, residual, out, out_dtype, status):
    """(device, out, packed mk_linear_args) of a linear map's operands, which are checked."""
    import torch
    bf, f32 = torch.bfloat16, torch.float32
    dev = x.get_device()
    (rows, k), xs = _operand(x, "x", (bf,), dev, 2)
    (n, wk), ws = _operand(weight, "weight", (bf,), dev, 2)
    act = ACTIVATIONS.get(activation, -1)
    if act < 0:
        raise ValueError(f"activation {activation!r}: expected one of {list(ACTIVATIONS)}")
    if wk != k or (ws[0] != k and n > 1):
        raise ValueError(f"weight {tuple(weight.shape)} must be contiguous, with rows of {k}")
    if bias is not None and _operand(bias, "bias", (bf,), dev, 1)[0][0] != n:
        raise ValueError(f"bias must have {n} elements")
    if act == 3:
        if n % 2:
            raise ValueError("swiglu takes an even number of weight rows: gate rows, then up rows")
        n //= 2
    if out is None:
        if out_dtype is not None and out_dtype is not bf and out_dtype is not f32:
            raise ValueError(f"out_dtype must be torch.bfloat16 or torch.float32, not {out_dtype}")
        out, os = torch.empty((rows, n), dtype=out_dtype or bf, device=x.device), n
    else:
        if out_dtype is not None and out.dtype != out_dtype:
            raise ValueError(f"out is {out.dtype}, out_dtype {out_dtype}")
        shape, os = _operand(out, "out", (bf, f32), dev, 2)
        os = os[0]
        if shape[0] != rows or shape[1] != n:
            raise ValueError(f"out must be [{rows}, {n}], not {tuple(shape)}")
    rp = rs = rt = 0
    if residual is not None:
        shape, rs = _operand(residual, "residual", (bf, f32), dev, 2)
        if shape[0] != rows or shape[1] != n:
            raise ValueError(f"residual must be [{rows}, {n}], not {tuple(shape)}")
        rp, rs, rt = residual.data_ptr(), rs[0], F32 if residual.dtype is f32 else BF16
    return dev, out, _LINEAR_ARGS.pack(
        rows, n, k, act, x.data_ptr(), xs[0], weight.data_ptr(), 0 if bias is None else bias.data_ptr(), rp, rs, rt,
        F32 if out.dtype is f32 else BF16, out.data_ptr(), os, 0 if status is None else _status_ptr(status, dev))


def attend(q, kv, q_lens: Sequence[int], kv_lens: Sequence[int], layer: int = 0, window: int = 0, sinks: int = 0,
           shared_prefix: int = 0, scale: Optional[float] = None, pages=None, out=None, workspace=None, status=None):
    """mk_attend: attention of query tokens over one layer of a KV cache.

    q [tokens, n_q_heads, head_dim] bf16: the sequences' query tokens back to back, q_lens[b] of
    sequence b, which are the last of its kv_lens[b] positions (their K/V rows already in the
    cache).  kv, pages: the cache as Decoder takes it -- kv.k / kv.v [batch, layers, kv heads, max_seq,
    head_dim], or the pool [layers, kv heads, n_blocks * block_size, head_dim] with
    pages = (block_table, block_size, n_blocks).  A token at position t sees positions p <= t; with a
    window those with p > t - window or p < sinks.  shared_prefix: the first positions, the same
    for every sequence, read once through sequence 0.  out: bf16, shaped like q (allocated by
    default; rows behind the last sequence's are not written); workspace: at least mk_attend_workspace
    bytes (allocated by default).  Returns out.

    status: a CUDA int32 tensor of one element, zeroed by the caller, that receives an mk_status when the
    device meets an error: MK_ERR_BOUNDS (a table entry outside the pool; its positions count as not visible) or
    MK_ERR_TIMEOUT (out is not valid).  Without it such an error leaves no trace.  No gradients are recorded."""
    o = (_fast or _setup()).attend(q, kv.k, kv.v, q_lens, kv_lens, layer, window, sinks, shared_prefix, scale, pages, out, workspace,
                                   status)
    if o is not None:
        return o
    import torch
    bf = torch.bfloat16
    dev = q.get_device()
    (tokens, nq, d), qs = _operand(q, "q", (bf,), dev, 3)
    batch = len(q_lens)
    if len(kv_lens) != batch:
        raise ValueError("q_lens and kv_lens must have the same length")
    if sum(q_lens) > tokens:
        raise ValueError(f"q holds {tokens} tokens, q_lens add up to {sum(q_lens)}")
    if scale is not None and not scale > 1e-45:   # (what rounds to zero in fp32 would stand for the default)
        raise ValueError("scale must be positive")
    if out is None:
        out, os = torch.empty((tokens, nq, d), dtype=bf, device=q.device), (nq * d, d)
    else:
        shape, os = _operand(out, "out", (bf,), dev, 3)
        if shape != q.shape:
            raise ValueError("out must have q's shape")
    if nq > 1 and (qs[1] != d or os[1] != d):
        raise ValueError("q and out: a token's heads must be contiguous")
    k, v = kv.k, kv.v
    dims = 5 if pages is None else 4
    shape, ks = _operand(k, "kv.k", (bf,), dev, dims)
    if (v.shape != shape or v.stride() != ks or v.dtype is not bf or v.get_device() != dev or shape[-1] != d or
            (ks[-2] != d and shape[-2] > 1)):
        raise ValueError("kv.k and kv.v must be alike (shape, strides, type, device), with contiguous [positions, head_dim] rows of q's head_dim")
    layers, nkv, positions = shape[-4:-1]
    if not 0 <= layer < layers:
        raise ValueError(f"layer {layer} of {layers}")
    if pages is None:
        if shape[0] < batch:
            raise ValueError(f"the cache holds {shape[0]} sequences, q_lens name {batch}")
        cache = array.array("q", (k.data_ptr(), v.data_ptr(), ks[0], ks[1], ks[2]))
    else:
        table, block_size, n_blocks = pages
        tshape, ts = _operand(table, "the block table", (torch.int32,), dev, 2)
        if tshape[0] < batch or (ts[0] != tshape[1] and tshape[0] > 1):
            raise ValueError(f"the block table must be contiguous, with a row for each of {batch} sequences")
        if block_size < 1 or n_blocks < 1 or positions < n_blocks * block_size:
            raise ValueError(f"the pool holds {positions} positions a head, {n_blocks} blocks of {block_size} do not fit it")
        cache = array.array("q", (k.data_ptr(), v.data_ptr(), 0, ks[0], ks[1],
                                  table.data_ptr(), block_size | tshape[1] << 32, n_blocks))
        positions = tshape[1] * block_size
    lens = array.array("i", [*q_lens, *kv_lens])
    at, c_kv = lens.buffer_info()[0], cache.buffer_info()[0]
    a = _ATTEND_ARGS.pack(nq, nkv, d, batch, at, at + 4 * batch, q.data_ptr(), qs[0], out.data_ptr(), os[0],
                          c_kv, c_kv + 40 if pages is not None else 0, layer, min(positions, 1 << 30),
                          window, sinks, shared_prefix, scale or 0.0, 0 if status is None else _status_ptr(status, dev))
    _with_workspace(dev, workspace, lib.mk_attend, lib.mk_attend_workspace, a)
    return out


def _with_workspace(device: int, workspace, call, size, *args):
    """call(*args, workspace, bytes, stream) with `device` current, on the caller's workspace or one of torch's."""
    import torch
    if workspace is not None:
        if not workspace.is_cuda or workspace.get_device() != device or not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous, on the operands' device")
        _launch(device, call, *args, workspace.data_ptr(), workspace.numel() * workspace.element_size())
    elif torch._C._cuda_getDevice() == device:
        _allocating(device, call, size, *args)
    else:
        with torch.cuda.device(device):   # (the workspace's size depends on the device)
            _allocating(device, call, size, *args)


def _allocating(device: int, call, size, *args):
    """call(*args, workspace, bytes, stream) on the current device, with a workspace of size(*args) bytes from torch's
    allocator: taken for torch's current stream and given back at once, it is reused behind the call in stream order."""
    import torch
    stream, need = torch._C._cuda_getCurrentRawStream(device), size(*args)
    if not need:
        st = call(*args, 0, 0, stream)
    else:
        ws = torch._C._cuda_cudaCachingAllocator_raw_alloc(need, stream)
        try:
            st = call(*args, ws, need, stream)
        finally:
            torch._C._cuda_cudaCachingAllocator_raw_delete(ws)
    if st:
        _check(st)


# ---- around the paged cache of a serving step ---------------------------------------------------


def adapted_linear(x, weight, adapters, index, bias=None, activation: Optional[str] = None, residual=None, out=None, out_dtype=None,
                   workspace=None, status=None):
    """mk_linear_adapted: act(x @ weight.T + bias + scale[a] * (x @ down[a].T) @ up[a].T) + residual, a the token's adapter,
    in fp32, rounded once to the output's type.

    adapters: (down, up) or (down, up, scale) -- down bf16 [n_adapters, rank, k], up bf16 [n_adapters, n, rank] ([n_adapters,
    2 n, rank] with "swiglu": gate rows, then up rows), both contiguous, scale fp32 [n_adapters] or None (1).  index: int32
    [rows], each token's adapter, negative for none.  The other operands are linear()'s.  workspace: at least
    mk_linear_adapted_workspace bytes (allocated by default).  Returns out.

    The same call gives the same bits; a token's may differ in the last places where it stands in another row or beside others.
    status: as in linear(), and MK_ERR_BOUNDS for an index of n_adapters or more, which counts as none.  No gradients are
    recorded."""
    down, up, scale = adapters if len(adapters) == 3 else (*adapters, None)
    y = (_fast or _setup()).adapted_linear(x, weight, bias, activation, residual, out, out_dtype, status, down, up, scale, index, workspace)
    if y is not None:
        return y
    import torch
    bf = torch.bfloat16
    dev, out, args = _linear_args(x, weight, bias, activation, residual, out, out_dtype, status)
    (count, rank, k), ds = _operand(down, "down", (bf,), dev, 3)
    ushape, us = _operand(up, "up", (bf,), dev, 3)
    wide = weight.shape[0]
    if k != x.shape[1] or not down.is_contiguous():
        raise ValueError(f"down {tuple(down.shape)} must be contiguous, with rows of {x.shape[1]}")
    if tuple(ushape) != (count, wide, rank) or not up.is_contiguous():
        raise ValueError(f"up {tuple(ushape)} must be contiguous, [{count}, {wide}, {rank}]")
    if scale is not None and (_operand(scale, "scale", (torch.float32,), dev, 1)[0][0] != count or not scale.is_contiguous()):
        raise ValueError(f"scale must have {count} elements")
    if _operand(index, "index", (torch.int32,), dev, 1)[0][0] != x.shape[0] or not index.is_contiguous():
        raise ValueError(f"index must have {x.shape[0]} contiguous elements")
    ad = _ADAPTERS.pack(count, rank, down.data_ptr(), up.data_ptr(), 0 if scale is None else scale.data_ptr(), index.data_ptr())
    _with_workspace(dev, workspace, lib.mk_linear_adapted, lib.mk_linear_adapted_workspace, args, ad)
    return out


def rope_append(qkv, kv, positions, slots, freqs, layer: int = 0, sections: Optional[Sequence[int]] = None, neighbours: bool = False,
                q_gain=None, k_gain=None, eps: float = 1e-5, out=None, status=None):
    """mk_rope_append: norms of every q and k head (where their gain is given), rotation of q and k by the tokens' positions,
    q to its own buffer, k and v to the cache.

    qkv [tokens, (n_q_heads + 2 n_kv_heads) head_dim] bf16 or fp32: q, k, v heads in order (rows may be strided by 16 bytes);
    n_kv_heads and head_dim are the cache's.  kv: the cache as attend() takes it -- kv.k / kv.v [batch, layers, kv heads,
    max_seq, head_dim], or the pool [layers, kv heads, n_blocks * block_size, head_dim].  slots int32 [tokens]: b * max_seq + p
    in the first, block * block_size + offset in the second (assign_pages()); negative: not stored.
    freqs: float64 on the CPU, radians per position of each pair (theta ** (-2 p / rotary)); 2 len(freqs) elements of a head
    are rotated, pair p is elements p and p + len(freqs), or 2 p and 2 p + 1 with neighbours.  positions int32 [tokens], or
    [axes, tokens] with sections: the pairs of each axis in order, adding up to len(freqs).
    q_gain, k_gain bf16 [head_dim].  out: bf16 [tokens, n_q_heads, head_dim] (allocated by default; it may be the q part of a
    bf16 qkv).  Returns out.

    status: a CUDA int32 tensor of one element, zeroed by the caller, that receives MK_ERR_BOUNDS for a slot behind the
    cache (not stored), or MK_ERR_TIMEOUT where a copy did not arrive within its limit (out and the cache then lack heads).  No
    gradients are recorded."""
    q = (_fast or _setup()).rope_append(qkv, kv.k, kv.v, positions, slots, freqs, layer, sections, neighbours, q_gain, k_gain, eps, out,
                                        status)
    if q is not None:
        return q
    import torch
    bf, f32 = torch.bfloat16, torch.float32
    dev = qkv.get_device()
    (tokens, width), xs = _operand(qkv, "qkv", (bf, f32), dev, 2)
    k, v = kv.k, kv.v
    dims = k.dim()
    if dims not in (4, 5):
        raise ValueError(f"kv.k must have 5 dimensions, or 4 (a pool), not {dims}")
    shape, ks = _operand(k, "kv.k", (bf,), dev, dims)
    if v.shape != shape or v.stride() != ks or v.dtype is not bf or v.get_device() != dev or (ks[-2] != shape[-1] and shape[-2] > 1):
        raise ValueError("kv.k and kv.v must be alike (shape, strides, type, device), with contiguous [positions, head_dim] rows")
    layers, nkv, positions_of, d = shape[-4:]
    if not 0 <= layer < layers:
        raise ValueError(f"layer {layer} of {layers}")
    nq = width // d - 2 * nkv if d else 0
    if nq < 1 or (nq + 2 * nkv) * d != width:
        raise ValueError(f"qkv rows of {width} are not q heads and 2 x {nkv} kv heads of {d}")
    if freqs.dtype is not torch.float64 or freqs.is_cuda or freqs.dim() != 1 or not freqs.is_contiguous():
        raise ValueError("freqs must be a contiguous float64 tensor on the CPU")
    axes = 1 if sections is None else len(sections)
    pshape, ps = _operand(positions, "positions", (torch.int32,), dev, 1 if sections is None else 2)
    if pshape[-1] != tokens or (sections is not None and pshape[0] != axes):
        raise ValueError(f"positions must be [{tokens}]" if sections is None else f"positions must be [{axes}, {tokens}]")
    if _operand(slots, "slots", (torch.int32,), dev, 1)[0][0] != tokens:
        raise ValueError(f"slots must have {tokens} elements")
    for name, gain in (("q_gain", q_gain), ("k_gain", k_gain)):
        if gain is not None and _operand(gain, name, (bf,), dev, 1)[0][0] != d:
            raise ValueError(f"{name} must have {d} elements")
    if out is None:
        out, os = torch.empty((tokens, nq, d), dtype=bf, device=qkv.device), nq * d
    else:
        oshape, os = _operand(out, "out", (bf,), dev, 3)
        if tuple(oshape) != (tokens, nq, d) or (os[1] != d and nq > 1):
            raise ValueError(f"out must be [{tokens}, {nq}, {d}] with contiguous heads of a token")
        os = os[0]
    c_kv = mk_kv(k.data_ptr(), v.data_ptr(), ks[0] if dims == 5 else 0, ks[-4], ks[-3])
    c_sections = None if sections is None else (ctypes.c_int32 * axes)(*sections)
    args = _ROPE_ARGS.pack(tokens, nq, nkv, d, qkv.data_ptr(), xs[0], F32 if qkv.dtype is f32 else BF16, 2 * freqs.numel(),
                           0 if q_gain is None else q_gain.data_ptr(), 0 if k_gain is None else k_gain.data_ptr(), eps, bool(neighbours),
                           axes, 0 if sections is None else ctypes.addressof(c_sections), freqs.data_ptr(), positions.data_ptr(),
                           ps[0] if sections is not None else 0, slots.data_ptr(), ctypes.addressof(c_kv), layer, positions_of,
                           shape[0] if dims == 5 else 1, out.data_ptr(), os, 0 if status is None else _status_ptr(status, dev))
    _launch(dev, lib.mk_rope_append, args)
    return out


def assign_pages(ring, ends, table, lens, new_lens, block_size: int, max_tokens: int, shared_prefix: int = 0, ends_out=None, out=None,
                 status=None):
    """mk_assign_pages: blocks of a paged cache for requests that grow, shrink or end, and the slots of the step's tokens,
    worked out on the device.

    ring int32 [n_blocks] and ends int32 [3] (front, free blocks, 0): the free block ids, as a ring.  table int32 [batch,
    max_blocks].  lens, new_lens int32 [batch]: positions held and wanted; 0 ends a request.  Blocks no longer needed go to
    the back of the ring, new ones come from its front into table.  ends_out: receives the ends after the call (default: ends
    itself).  shared_prefix: positions whose whole blocks every row shares and no request owns.
    Returns (slots, positions, sequences, first): int32 [max_tokens] each (-1, 0, -1 behind the last token) and [batch + 1],
    or the four tensors of out.

    status: a CUDA int32 tensor of one element, zeroed by the caller: MK_ERR_CAPACITY (too few free blocks, more tokens than
    max_tokens) or MK_ERR_BOUNDS (lengths or ends that cannot be) where nothing was assigned and every slot is -1; MK_ERR_BOUNDS
    also for a block id outside the ring's n_blocks."""
    if ends_out is None:
        ends_out = ends
    if out is not None:
        out = tuple(out)
    taken = (_fast or _setup()).assign_pages(ring, ends, ends_out, table, lens, new_lens, block_size, max_tokens, shared_prefix, out,
                                             status)
    if taken is not None:
        return taken
    import torch
    dev, i32 = ring.get_device(), (torch.int32,)
    operands = dict(ring=(ring, 1), ends=(ends, 1), ends_out=(ends_out, 1), table=(table, 2), lens=(lens, 1), new_lens=(new_lens, 1))
    for name, (t, dim) in operands.items():
        _operand(t, name, i32, dev, dim)
    (batch, columns), n_blocks = table.shape, ring.shape[0]
    if not table.is_contiguous() or lens.shape[0] != batch or new_lens.shape[0] != batch:
        raise ValueError("table must be contiguous, with a row for each of lens and new_lens")
    if ends.shape[0] != 3 or ends_out.shape[0] != 3:
        raise ValueError("ends and ends_out must have 3 elements")
    if out is None:
        out = tuple(torch.empty(n, dtype=torch.int32, device=ring.device) for n in (max_tokens, max_tokens, max_tokens, batch + 1))
    else:
        for name, t, n in zip(("slots", "positions", "sequences", "first"), out, (max_tokens, max_tokens, max_tokens, batch + 1), strict=True):
            if _operand(t, name, i32, dev, 1)[0][0] != n:
                raise ValueError(f"{name} must have {n} elements")
    _launch(dev, lib.mk_assign_pages,
            _PAGES_ARGS.pack(batch, block_size, columns, n_blocks, shared_prefix, max_tokens, ring.data_ptr(), ends.data_ptr(),
                             ends_out.data_ptr(), table.data_ptr(), lens.data_ptr(), new_lens.data_ptr(), *(t.data_ptr() for t in out),
                             0 if status is None else _status_ptr(status, dev)))
    return out
