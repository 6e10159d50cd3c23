"""Thin ctypes binding over ``libtcd.so`` (the C ABI of ``include/tcd.h``).

Argument marshalling only: every step of the decode path runs in the CUDA
kernels behind the C ABI.  Device buffers are passed as torch CUDA tensors
(their ``data_ptr()``), streams as ``torch.cuda.Stream`` (default: the current
stream).  If the library is missing this module raises on import; there is no
CPU fallback.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional, Sequence

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.environ.get("TCD_LIB", os.path.join(_HERE, "libtcd.so"))

if not os.path.exists(LIB_PATH):
    raise ImportError(f"libtcd.so not found at {LIB_PATH}: build it with "
                      "`python -m trie_constrained_decoding_gb300.build` (no CPU fallback exists)")

_lib = ctypes.CDLL(LIB_PATH)

# Status codes and enums of include/tcd.h
TC_OK = 0
STATUS_NAMES = {}
RES_AUTO, RES_CONST, RES_GLOBAL = 0, 1, 2
BIND_LIVE_COUNTS = 0x10        # or-ed into bind's residency: per-sequence live-count arrays for every k
HEAD_SPARSE, HEAD_DENSE, HEAD_UNION_GEMM, HEAD_DENSE_GEMM = 0, 1, 2, 3
FLAG_JUMP_FORWARD = 0x100      # or-ed into `head` of decode / decode_graph: forced tokens skip the head
FLAG_FORCED_LOGITS = 0x200     # with FLAG_JUMP_FORWARD: forced tokens still get their logits
FLAG_ROOT_GEMM = 0x400         # with HEAD_SPARSE in decodes: the first (root) step on the tcgen05 GEMM
STAT_SLOTS = 6
TC_ERR_EMPTY_MASK, TC_ERR_NO_LIVE_EDGE, TC_ERR_MAX_STEPS, TC_ERR_BOUNDS = 16, 17, 18, 19
TC_ERR_DEVICE_TIMEOUT = 20
CONST_CAPACITY_BYTES = 63 * 1024

_i32p = ctypes.POINTER(ctypes.c_int32)
_i64p = ctypes.POINTER(ctypes.c_int64)
_vp = ctypes.c_void_p


class _TrieInfo(ctypes.Structure):
    _fields_ = [("n_nodes", ctypes.c_int32), ("n_edges", ctypes.c_int32), ("n_strings", ctypes.c_int32),
                ("max_fanout", ctypes.c_int32), ("root_fanout", ctypes.c_int32), ("max_depth", ctypes.c_int32),
                ("vocab", ctypes.c_int32), ("sep_id", ctypes.c_int32), ("stop_id", ctypes.c_int32),
                ("header_bytes", ctypes.c_int32), ("total_tokens", ctypes.c_int64),
                ("walk_image_bytes", ctypes.c_int64)]


class Sampling(ctypes.Structure):
    """tc_sampling_t: temperature > 0, top_k >= 0 (0: off), top_p in [0, 1] (1: off)."""
    _fields_ = [("temperature", ctypes.c_float), ("top_k", ctypes.c_int32), ("top_p", ctypes.c_float)]


def _decl(name, restype, argtypes):
    f = getattr(_lib, name)
    f.restype = restype
    f.argtypes = argtypes
    return f


_compile = _decl("tc_compile_trie", ctypes.c_int, [_i32p, _i64p, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                                   ctypes.c_int32, ctypes.c_int32, ctypes.POINTER(_vp)])
_compile_chars = _decl("tc_compile_char_trie", ctypes.c_int,
                       [_vp, _i64p, ctypes.c_int32, _i32p, _vp, _i64p, ctypes.c_int32, ctypes.c_int32,
                        ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.POINTER(_vp)])
_info = _decl("tc_trie_info", ctypes.c_int, [_vp, ctypes.POINTER(_TrieInfo)])
_export = _decl("tc_trie_export", ctypes.c_int, [_vp] + [_i32p] * 7)
_trie_free = _decl("tc_trie_free", None, [_vp])
_export_ranks = _decl("tc_trie_export_ranks", ctypes.c_int, [_vp, _i32p, _i32p])
_ctx_create = _decl("tc_ctx_create", ctypes.c_int, [ctypes.c_int32, _vp, ctypes.c_int32, ctypes.c_int32,
                                                   ctypes.c_int32, ctypes.c_int32, ctypes.POINTER(_vp)])
_ctx_destroy = _decl("tc_ctx_destroy", None, [_vp])
_bind = _decl("tc_bind_grammar", ctypes.c_int, [_vp, _vp, ctypes.c_int32, _vp])
_bound_res = _decl("tc_bound_residency", ctypes.c_int, [_vp, _i32p])
_reset = _decl("tc_reset", ctypes.c_int, [_vp, ctypes.c_int32, ctypes.c_int32, _vp])
_step = _decl("tc_step", ctypes.c_int, [_vp, _vp, ctypes.c_int32, _vp, _vp, _vp, _vp])
_decode_args = [_vp, _vp, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                _vp, _vp, _vp, _vp]
_decode = _decl("tc_decode", ctypes.c_int, _decode_args + [_vp])
_decode_host = _decl("tc_decode_host", ctypes.c_int, _decode_args + [_vp])
_graph_create = _decl("tc_decode_graph_create", ctypes.c_int, _decode_args + [ctypes.POINTER(_vp)])
_graph_launch = _decl("tc_graph_launch", ctypes.c_int, [_vp, _vp])
_graph_destroy = _decl("tc_graph_destroy", None, [_vp])
_first_error = _decl("tc_first_error", ctypes.c_int, [_vp, _vp, _i32p, _i32p])
_read_state = _decl("tc_read_seq_state", ctypes.c_int, [_vp, _vp] + [_i32p] * 5)
_read_stats = _decl("tc_read_stats", ctypes.c_int, [_vp, _vp, _i64p, ctypes.c_int32])
_decode_sample = _decl("tc_decode_sample", ctypes.c_int,
                       [_vp, _vp, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                        ctypes.POINTER(Sampling), _vp, _vp, _vp, _vp, _vp, _vp])
_step_sample = _decl("tc_step_sample", ctypes.c_int, [_vp, _vp, ctypes.c_int32, ctypes.POINTER(Sampling), _vp, _vp,
                                                      _vp, _vp, _vp])
_loop_floor = _decl("tc_loop_floor", ctypes.c_int, [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, _vp,
                                                    ctypes.POINTER(ctypes.c_float), _i64p])
_gemm_wait_test = _decl("tc_gemm_wait_test", ctypes.c_int, [_vp, ctypes.c_int32, ctypes.c_int64])
_status_str = _decl("tc_status_str", ctypes.c_char_p, [ctypes.c_int])
_last_msg = _decl("tc_last_error_message", ctypes.c_char_p, [])


def status_name(code: int) -> str:
    return _status_str(int(code)).decode()


class TcError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = int(code)
        self.name = status_name(code)
        msg = _last_msg().decode()
        super().__init__(f"{where}: {self.name}" + (f" ({msg})" if msg else ""))


def _check(code: int, where: str):
    if code != TC_OK:
        raise TcError(code, where)


def _stream_ptr(stream) -> Optional[int]:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


class Trie:
    """A compiled catalog (host object)."""

    def __init__(self, handle):
        self._h = handle

    @classmethod
    def compile(cls, catalog: Sequence[Sequence[int]], sep_id: int, stop_id: int, vocab: int,
                max_fanout: int = 256) -> "Trie":
        lens = [len(s) for s in catalog]
        offsets = np.zeros(len(catalog) + 1, dtype=np.int64)
        offsets[1:] = np.cumsum(lens)
        ids = np.array([t for s in catalog for t in s], dtype=np.int32) if offsets[-1] else np.zeros(1, np.int32)
        h = _vp()
        code = _compile(ids.ctypes.data_as(_i32p), offsets.ctypes.data_as(_i64p), len(catalog), sep_id, stop_id,
                        vocab, max_fanout, ctypes.byref(h))
        _check(code, "tc_compile_trie")
        return cls(h)

    @classmethod
    def compile_chars(cls, strings: Sequence[bytes], vocab: Sequence[tuple], sep_id: int, stop_id: int,
                      vocab_size: int, max_fanout: int = 4096) -> "Trie":
        """tc_compile_char_trie: byte strings and a byte vocabulary [(token id, bytes)]."""
        offs = np.zeros(len(strings) + 1, dtype=np.int64)
        offs[1:] = np.cumsum([len(x) for x in strings])
        chars = np.frombuffer(b"".join(strings), dtype=np.uint8).copy()
        ids = np.array([i for i, _ in vocab], dtype=np.int32)
        toff = np.zeros(len(vocab) + 1, dtype=np.int64)
        toff[1:] = np.cumsum([len(b) for _, b in vocab])
        tchars = np.frombuffer(b"".join(b for _, b in vocab), dtype=np.uint8).copy()
        h = _vp()
        code = _compile_chars(chars.ctypes.data, offs.ctypes.data_as(_i64p), len(strings),
                              ids.ctypes.data_as(_i32p), tchars.ctypes.data, toff.ctypes.data_as(_i64p), len(vocab),
                              sep_id, stop_id, vocab_size, max_fanout, ctypes.byref(h))
        _check(code, "tc_compile_char_trie")
        return cls(h)

    def info(self) -> dict:
        inf = _TrieInfo()
        _check(_info(self._h, ctypes.byref(inf)), "tc_trie_info")
        return {name: getattr(inf, name) for name, _ in _TrieInfo._fields_}

    def export(self) -> dict:
        i = self.info()
        N, E, K, T = i["n_nodes"], i["n_edges"], i["n_strings"], i["total_tokens"]
        arrs = {"node_begin": N + 1, "edge_tok": E, "edge_child": E, "node_ptr": N, "static_cnt": E,
                "path_off": K + 1, "path": max(T, 1)}
        out = {k: np.zeros(n, dtype=np.int32) for k, n in arrs.items()}
        _check(_export(self._h, *[out[k].ctypes.data_as(_i32p) for k in arrs]), "tc_trie_export")
        out["path"] = out["path"][:T]
        return out

    def ranks(self) -> dict:
        """Depth-first pointer ranks (tc_trie_export_ranks): ptr_rank[K], edge_lo[E]."""
        i = self.info()
        out = {"ptr_rank": np.zeros(i["n_strings"], dtype=np.int32), "edge_lo": np.zeros(i["n_edges"], np.int32)}
        _check(_export_ranks(self._h, out["ptr_rank"].ctypes.data_as(_i32p), out["edge_lo"].ctypes.data_as(_i32p)),
               "tc_trie_export_ranks")
        return out

    def close(self):
        if self._h:
            _trie_free(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Graph:
    def __init__(self, ctx, handle, keep):
        self._ctx, self._h, self._keep = ctx, handle, keep

    def launch(self, stream=None):
        _check(_graph_launch(self._h, _stream_ptr(stream)), "tc_graph_launch")

    def close(self):
        if self._h:
            _graph_destroy(self._h)
            self._h = None


class Context:
    """A decoding context over a bf16 tied embedding held in a torch CUDA tensor."""

    def __init__(self, emb, max_batch: int, cand_cap: int = 256, device: Optional[int] = None):
        import torch
        if not (emb.is_cuda and emb.dtype == torch.bfloat16 and emb.dim() == 2 and emb.is_contiguous()):
            raise ValueError("emb must be a contiguous 2-D bfloat16 CUDA tensor [vocab, hidden]")
        self.emb = emb                   # keep the embedding alive
        self.vocab, self.hidden = emb.shape
        self.device = emb.device.index if device is None else device
        self.max_batch = max_batch
        h = _vp()
        _check(_ctx_create(self.device, emb.data_ptr(), self.vocab, self.hidden, max_batch, cand_cap,
                           ctypes.byref(h)), "tc_ctx_create")
        self._h = h
        self._graphs = []

    def bind(self, trie: Trie, residency: int = RES_AUTO, stream=None):
        _check(_bind(self._h, trie._h, residency, _stream_ptr(stream)), "tc_bind_grammar")

    def residency(self) -> int:
        r = ctypes.c_int32()
        _check(_bound_res(self._h, ctypes.byref(r)), "tc_bound_residency")
        return r.value

    def reset(self, batch: int, k: int, stream=None):
        _check(_reset(self._h, batch, k, _stream_ptr(stream)), "tc_reset")

    def step(self, hidden, tok_out, logit_out=None, status_out=None, head: int = HEAD_SPARSE, stream=None):
        _check(_step(self._h, hidden.data_ptr(), head, tok_out.data_ptr(), _ptr(logit_out), _ptr(status_out),
                     _stream_ptr(stream)), "tc_step")

    def _dargs(self, hidden_steps, k, max_steps, head, toks, logits, lens, status):
        S, B, H = hidden_steps.shape
        return (self._h, hidden_steps.data_ptr(), S, B, k, max_steps, head, toks.data_ptr(), logits.data_ptr(),
                lens.data_ptr(), status.data_ptr())

    def decode(self, hidden_steps, k, max_steps, toks, logits, lens, status, head=HEAD_SPARSE, stream=None):
        _check(_decode(*self._dargs(hidden_steps, k, max_steps, head, toks, logits, lens, status),
                       _stream_ptr(stream)), "tc_decode")

    def decode_sample(self, hidden_steps, k, max_steps, uniforms, toks, logits, lens, status, temperature=1.0,
                      top_k=0, top_p=1.0, head=HEAD_SPARSE, stream=None):
        """tc_decode_sample: uniforms is a device float32 [batch, max_steps] tensor."""
        S, B, H = hidden_steps.shape
        sp = Sampling(float(temperature), int(top_k), float(top_p))
        _check(_decode_sample(self._h, hidden_steps.data_ptr(), S, B, k, max_steps, head, ctypes.byref(sp),
                              uniforms.data_ptr(), toks.data_ptr(), logits.data_ptr(), lens.data_ptr(),
                              status.data_ptr(), _stream_ptr(stream)), "tc_decode_sample")

    def step_sample(self, hidden, uniforms, tok_out, logit_out=None, status_out=None, temperature=1.0, top_k=0,
                    top_p=1.0, head: int = HEAD_SPARSE, stream=None):
        sp = Sampling(float(temperature), int(top_k), float(top_p))
        _check(_step_sample(self._h, hidden.data_ptr(), head, ctypes.byref(sp), uniforms.data_ptr(),
                            tok_out.data_ptr(), _ptr(logit_out), _ptr(status_out), _stream_ptr(stream)),
               "tc_step_sample")

    def decode_host(self, hidden_steps, k, max_steps, toks, logits, lens, status, head=HEAD_SPARSE, stream=None):
        _check(_decode_host(*self._dargs(hidden_steps, k, max_steps, head, toks, logits, lens, status),
                            _stream_ptr(stream)), "tc_decode_host")

    def decode_graph(self, hidden_steps, k, max_steps, toks, logits, lens, status, head=HEAD_SPARSE) -> Graph:
        h = _vp()
        _check(_graph_create(*self._dargs(hidden_steps, k, max_steps, head, toks, logits, lens, status),
                             ctypes.byref(h)), "tc_decode_graph_create")
        g = Graph(self, h, (hidden_steps, toks, logits, lens, status))
        self._graphs.append(g)
        return g

    def first_error(self, stream=None):
        seq, code = ctypes.c_int32(), ctypes.c_int32()
        _check(_first_error(self._h, _stream_ptr(stream), ctypes.byref(seq), ctypes.byref(code)), "tc_first_error")
        return seq.value, code.value

    def raise_on_error(self, stream=None):
        seq, code = self.first_error(stream)
        if code != TC_OK:
            raise TcError(code, f"sequence {seq}")

    def seq_state(self, batch: int, stream=None) -> dict:
        out = {k: np.zeros(batch, dtype=np.int32) for k in ("node", "emitted", "len", "status", "done")}
        _check(_read_state(self._h, _stream_ptr(stream), *[out[k].ctypes.data_as(_i32p) for k in
                                                           ("node", "emitted", "len", "status", "done")]),
               "tc_read_seq_state")
        return out

    def stats(self, reset: bool = False, stream=None) -> dict:
        out = np.zeros(STAT_SLOTS, dtype=np.int64)
        _check(_read_stats(self._h, _stream_ptr(stream), out.ctypes.data_as(_i64p), int(reset)), "tc_read_stats")
        return {"step_launches": int(out[0]), "seq_steps": int(out[1]), "cand_rows": int(out[2]),
                "reset_launches": int(out[3]), "forced": int(out[4]), "union_rows": int(out[5])}

    def gemm_wait_test(self, withhold: bool, wait_polls: int = 0):
        """tc_gemm_wait_test: make the GEMM heads' first pipeline stage never
        arrive (withhold) with waits of `wait_polls` polls; (False, 0) restores."""
        _check(_gemm_wait_test(self._h, int(bool(withhold)), int(wait_polls)), "tc_gemm_wait_test")

    def close(self):
        for g in self._graphs:
            g.close()
        self._graphs = []
        if self._h:
            _ctx_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def loop_floor(device: int, batch: int, iterations: int, stream=None):
    """Milliseconds and kernel launches of the decode loop's graph shape with
    do-nothing kernels in the steps' place (tc_loop_floor)."""
    ms = ctypes.c_float()
    n = ctypes.c_int64()
    _check(_loop_floor(device, batch, iterations, _stream_ptr(stream), ctypes.byref(ms), ctypes.byref(n)),
           "tc_loop_floor")
    return float(ms.value), int(n.value)


# ------------------------------------------------- paged cache (include/tcd_cache.h)

DT_BF16, DT_F16 = 0, 1
TREE_MAX_WORDS, PATH_MAX, KV_MAX_BATCH = 4, 256, 65536


class _Kv(ctypes.Structure):
    _fields_ = [("pool", _vp), ("device", ctypes.c_int32), ("dtype", ctypes.c_int32), ("layers", ctypes.c_int32),
                ("pages", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("keep_status", ctypes.c_int32)]


class _Tokens(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("n_tokens", ctypes.c_int32), ("cu_tokens", _vp), ("ctx_lens", _vp),
                ("page_table", _vp), ("table_width", ctypes.c_int32)]


class _Append(ctypes.Structure):
    _fields_ = [("qkv", _vp), ("qkv_stride", ctypes.c_int64), ("q_heads", ctypes.c_int32), ("q_weight", _vp),
                ("k_weight", _vp), ("eps", ctypes.c_float), ("rope", _vp), ("rope_len", ctypes.c_int32),
                ("positions", _vp), ("interleaved", ctypes.c_int32), ("q_out", _vp), ("q_out_stride", ctypes.c_int64)]


class _Attend(ctypes.Structure):
    _fields_ = [("q", _vp), ("q_stride", ctypes.c_int64), ("q_heads", ctypes.c_int32), ("max_tokens", ctypes.c_int32),
                ("scale", ctypes.c_float), ("tree", _vp), ("tree_words", ctypes.c_int32), ("out", _vp),
                ("out_stride", ctypes.c_int64), ("lse", _vp), ("wait_polls", ctypes.c_int64),
                ("withhold", ctypes.c_int32)]


_kvp, _tokp = ctypes.POINTER(_Kv), ctypes.POINTER(_Tokens)
_kv_append = _decl("tc_kv_append", ctypes.c_int, [_kvp, ctypes.c_int32, _tokp, ctypes.POINTER(_Append), _vp, _vp])
_attend = _decl("tc_attend", ctypes.c_int, [_kvp, ctypes.c_int32, _tokp, ctypes.POINTER(_Attend), _vp, ctypes.c_int64,
                                            _vp, _vp])
_attend_workspace = _decl("tc_attend_workspace", ctypes.c_int, [_kvp, _i64p])
_tree_masks = _decl("tc_tree_masks", ctypes.c_int, [_tokp, _vp, ctypes.c_int32, _vp, _vp, _vp, _vp])
_kv_copy_pages = _decl("tc_kv_copy_pages", ctypes.c_int, [_kvp, _vp, _vp, ctypes.c_int32, _vp, _vp])
_kv_compact = _decl("tc_kv_compact", ctypes.c_int, [_kvp, _tokp, _vp, ctypes.c_int32, _vp, _vp, _vp, _vp])
_pages_create = _decl("tc_pages_create", ctypes.c_int, [ctypes.c_int32, ctypes.c_int32, ctypes.POINTER(_vp)])
_pages_destroy = _decl("tc_pages_destroy", None, [_vp])
_pages_open = _decl("tc_pages_open", ctypes.c_int, [_vp, _i32p])
_pages_close = _decl("tc_pages_close", ctypes.c_int, [_vp, ctypes.c_int32])
_pages_reserve = _decl("tc_pages_reserve", ctypes.c_int, [_vp, ctypes.c_int32, ctypes.c_int64, ctypes.c_int64, _i32p,
                                                          _i32p, _i32p])
_pages_fork = _decl("tc_pages_fork", ctypes.c_int, [_vp, ctypes.c_int32, ctypes.c_int64, _i32p])
_pages_trim = _decl("tc_pages_trim", ctypes.c_int, [_vp, ctypes.c_int32, ctypes.c_int64])
_pages_row = _decl("tc_pages_row", ctypes.c_int, [_vp, ctypes.c_int32, _i32p, ctypes.c_int32, _i32p])
_pages_free_count = _decl("tc_pages_free_count", ctypes.c_int, [_vp, _i32p])
_capture_id = _decl("tc_capture_id", ctypes.c_int, [_vp, ctypes.POINTER(ctypes.c_uint64)])
_capture_watch = _decl("tc_capture_watch", ctypes.c_int, [_vp, ctypes.POINTER(_i32p)])
_capture_unwatch = _decl("tc_capture_unwatch", None, [_i32p])
_capture_mode = _decl("tc_capture_mode", ctypes.c_int, [_i32p])
_clear_now = _decl("tc_clear_now", ctypes.c_int, [_vp, ctypes.c_int64, _vp])


def _rows(t, dtype, device, what: str, heads: int, head_dim: int):
    """Address and row stride (elements) of packed rows [n, heads * head_dim] or [n, heads, head_dim]; the rows may
    be slices of wider ones."""
    shape, stride = t.shape, t.stride()
    if len(shape) == 3:
        ok = shape[1] == heads and shape[2] == head_dim and stride[2] == 1 and (heads == 1 or stride[1] == head_dim)
    else:
        ok = len(shape) == 2 and shape[1] == heads * head_dim and stride[1] == 1
    if not ok or t.dtype is not dtype or t.device != device:
        raise ValueError(f"{what} must hold rows of {heads} heads of {head_dim} contiguous {dtype} elements on {device}")
    # (the stride of a single row says nothing: torch keeps whatever it was)
    return t.data_ptr(), stride[0] if shape[0] > 1 else heads * head_dim


def _empty(n: int, dtype, device, stream: int, zero: bool = False):
    """A buffer that belongs to the stream its kernels run on: memory of another stream may still be in use there."""
    import torch
    make = torch.zeros if zero else torch.empty
    if stream == torch.cuda.current_stream(device).cuda_stream:
        return make(n, dtype=dtype, device=device)
    own = torch.cuda.ExternalStream(stream, device=device) if stream else torch.cuda.default_stream(device)
    with torch.cuda.stream(own):
        return make(n, dtype=dtype, device=device)


class _Codes:
    """Gathered error codes: of sequences, then of pairs of pages."""

    def __init__(self, codes):
        self.codes, self.at = codes, codes.data_ptr()
        self.used = [0, 0]  # entries that a call may have written


class _Own:
    """What calls use where the caller gives nothing: of one stream, or of one graph that it is captured into."""

    def __init__(self, codes: _Codes, stream: int, gone=None):
        self.codes, self.workspace, self.place, self.stream = codes, None, None, stream  # (whose memory it is)
        self.gone = gone                     # (captured) a word: 1 when the graph is gone

    def idle(self) -> bool:
        return bool(self.gone) and self.gone[0] != 0

    def __del__(self):
        try:
            if self.idle():
                _capture_unwatch(self.gone)
        except Exception:
            pass


_held = []  # of captured calls: they stay while their graph does, whatever becomes of the KvCache
_held_lock = threading.Lock()


def _hold(own: _Own):
    with _held_lock:
        _held[:] = [o for o in _held if not o.idle()]
        _held.append(own)


def _stream_aside(device) -> int:
    """A stream that is not part of a capture."""
    import torch
    n = ctypes.c_uint64()
    for _ in range(64):
        s = torch.cuda.Stream(device).cuda_stream
        _check(_capture_id(s, ctypes.byref(n)), "tc_capture_id")
        if not n.value:
            return s
    raise RuntimeError("every stream is being captured")


def _empty_aside(n: int, dtype, device, stream: int, clear: bool):
    """A buffer for captured calls, out of the memory of a stream aside.  What that memory was used for before is
    over when it is returned (and it is cleared): a graph waits for nothing on that stream."""
    mode = ctypes.c_int32(2)                 # (the allocator may have to ask the driver for memory)
    _check(_capture_mode(ctypes.byref(mode)), "tc_capture_mode")
    try:
        t = _empty(n, dtype, device, stream)
    finally:
        _check(_capture_mode(ctypes.byref(mode)), "tc_capture_mode")
    _check(_clear_now(t.data_ptr(), n * t.element_size() if clear else 0, stream), "tc_clear_now")
    return t


class KvCache:
    """A paged key-value cache over a torch CUDA tensor
    [layers, pages, 2 (keys, values), kv_heads, page_size, head_dim], bf16 or f16.

    The object holds no cache state: the caller owns the pool, the page tables
    and the lengths.  ``status`` arguments are int32 tensors, one code per
    sequence (per pair for copy_pages), written whole by the call; left out,
    errors are gathered in a buffer of the object, the first of each sequence
    (or pair), until raise_on_error() raises and clears them.  attend's
    ``workspace`` is a tensor of at least ``workspace_bytes`` bytes that belongs
    to one call at a time; left out, it is a buffer of the object as well, one
    per stream, and one per stream of every capture: a captured graph shares
    none with other graphs or with calls on a stream, and its buffers stay while
    it exists.  Calls on one object belong to one host thread.
    """

    def __init__(self, pool):
        import torch
        types = {torch.bfloat16: DT_BF16, torch.float16: DT_F16}
        if not (pool.is_cuda and pool.dtype in types and pool.dim() == 6 and pool.shape[2] == 2 and
                pool.is_contiguous()):
            raise ValueError("pool must be a contiguous bfloat16 or float16 CUDA tensor "
                             "[layers, pages, 2, kv_heads, page_size, head_dim]")
        self.pool, self.dtype, self.device = pool, pool.dtype, pool.device
        self.layers, self.pages, _, self.kv_heads, self.page_size, self.head_dim = pool.shape
        self._kv = _Kv(pool.data_ptr(), pool.device.index, types[pool.dtype], self.layers, self.pages, self.kv_heads,
                       self.page_size, self.head_dim)
        self._kvp = ctypes.byref(self._kv)
        self._kv_keep = _Kv.from_buffer_copy(self._kv)   # for calls whose errors are gathered
        self._kv_keep.keep_status = 1
        self._kvp_keep = ctypes.byref(self._kv_keep)
        self._i32, self._i64, self._f32, self._u8 = torch.int32, torch.int64, torch.float32, torch.uint8
        # (a decode step's calls are a few microseconds long: asking for the stream object would be a good part)
        index, raw = pool.device.index, getattr(torch._C, "_cuda_getCurrentRawStream", None)
        self._current = (lambda: raw(index)) if raw else (lambda: torch.cuda.current_stream(index).cuda_stream)
        need = ctypes.c_int64()
        _check(_attend_workspace(self._kvp, ctypes.byref(need)), "tc_attend_workspace")
        self.workspace_bytes = need.value
        self._wait_test = (0, 0)
        self._own = {}                       # _Own per stream
        self._captured, self._graph_codes = {}, None   # _Own per capture and stream; their common codes
        self._capture = ctypes.c_uint64()
        self._capture_ref = ctypes.byref(self._capture)

    def _stream(self, stream):
        if stream is None:
            return self._current()
        return stream if isinstance(stream, int) else stream.cuda_stream

    def _ints(self, t, shape, what: str):
        if t.dtype is not self._i32 or t.shape != shape or t.device != self.device or not t.is_contiguous():
            raise ValueError(f"{what} must be a contiguous int32 tensor of shape {tuple(shape)} on {self.device}")
        return t.data_ptr()

    def _buffers(self, stream: int):
        if stream:                           # (the default stream cannot be captured)
            _check(_capture_id(stream, self._capture_ref), "tc_capture_id")
            if self._capture.value:
                return self._captured.get((self._capture.value, stream)) or \
                    self._capture_buffers(self._capture.value, stream)
        own = self._own.get(stream)
        if own is None:
            codes = _empty(2 * KV_MAX_BATCH, self._i32, self.device, stream, zero=True)
            own = self._own[stream] = _Own(_Codes(codes), stream)
        return own

    def _capture_buffers(self, capture: int, stream: int):
        """Their memory is no graph's own and the codes are cleared outside of the capture: a launch must not clear
        what the one before has left.  (Only errors are written: all graphs of the object share the codes.)"""
        for key in [k for k, o in self._captured.items() if o.idle()]:
            del self._captured[key]
        aside = _stream_aside(self.device)
        if self._graph_codes is None:
            self._graph_codes = _Codes(_empty_aside(2 * KV_MAX_BATCH, self._i32, self.device, aside, clear=True))
        gone = _i32p()
        if _capture_watch(stream, ctypes.byref(gone)) != TC_OK:
            gone = None                      # (never known to be gone: kept)
        own = self._captured[capture, stream] = _Own(self._graph_codes, aside, gone)
        _hold(own)
        return own

    def _codes(self, status, n: int, stream: int, pairs: int = 0, own=None):
        """Where a call's codes go, behind the description of the cache that says how."""
        if status is not None:
            return self._kvp, self._ints(status, (n,), "status")
        codes = (own or self._buffers(stream)).codes
        if n > codes.used[pairs]:
            codes.used[pairs] = min(n, KV_MAX_BATCH)
        return self._kvp_keep, codes.at + 4 * KV_MAX_BATCH * pairs

    def _workspace(self, workspace, stream: int, own=None):
        if workspace is None:
            own = own or self._buffers(stream)
            if own.place is None:
                if own.stream == stream:
                    own.workspace = _empty(self.workspace_bytes, self._u8, self.device, stream)
                else:
                    own.workspace = _empty_aside(self.workspace_bytes, self._u8, self.device, own.stream, clear=False)
                own.place = own.workspace.data_ptr(), self.workspace_bytes
            return own.place
        if workspace.device != self.device or not workspace.is_contiguous():
            raise ValueError(f"workspace must be a contiguous tensor on {self.device}")
        return workspace.data_ptr(), workspace.numel() * workspace.element_size()

    def _tokens(self, n, cu, ctx_lens, page_table):
        batch, width = page_table.shape
        return _Tokens(batch, n, None if cu is None else self._ints(cu, (batch + 1,), "cu_tokens"),
                       self._ints(ctx_lens, (batch,), "ctx_lens"), self._ints(page_table, (batch, width), "page_table"),
                       width)

    def append(self, layer: int, qkv, cu_tokens, ctx_lens, page_table, q_out, q_weight=None, k_weight=None,
               eps: float = 1e-6, rope=None, positions=None, interleaved: bool = False, status=None, stream=None):
        """tc_kv_append: qkv [n, (q_heads + 2 kv_heads) * head_dim], q_out [n, q_heads, head_dim]; rope float32
        [positions, head_dim / 2, 2] (cosine, sine)."""
        d, n = self.head_dim, qkv.shape[0]
        out = q_out.shape
        if out[0] != n:
            raise ValueError("q_out must have as many rows as qkv")
        hq = out[1] if len(out) == 3 else out[1] // d
        dtype, device = self.dtype, self.device
        for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
            if w is not None and (w.dtype is not dtype or w.shape != (d,) or w.device != device or
                                  not w.is_contiguous()):
                raise ValueError(f"{name} must be a contiguous {dtype} tensor of {d} elements")
        angles = 0
        if rope is not None:
            angles = rope.shape[0]
            if rope.dtype is not self._f32 or rope.shape != (angles, d // 2, 2) or rope.device != device or \
                    not rope.is_contiguous():
                raise ValueError(f"rope must be a contiguous float32 tensor [positions, {d // 2}, 2]")
        a = _Append(*_rows(qkv, dtype, device, "qkv", hq + 2 * self.kv_heads, d), hq,
                    None if q_weight is None else q_weight.data_ptr(),
                    None if k_weight is None else k_weight.data_ptr(), eps,
                    None if rope is None else rope.data_ptr(), angles,
                    None if positions is None else self._ints(positions, (n,), "positions"), bool(interleaved),
                    *_rows(q_out, dtype, device, "q_out", hq, d))
        t = self._tokens(n, cu_tokens, ctx_lens, page_table)
        s = self._stream(stream)
        kv, codes = self._codes(status, t.batch, s)
        _check(_kv_append(kv, layer, t, a, codes, s), "tc_kv_append")

    def attend(self, layer: int, q, cu_tokens, ctx_lens, page_table, out, max_tokens: int, scale=None, tree=None,
               lse=None, status=None, stream=None, workspace=None):
        """tc_attend: q and out [n, q_heads, head_dim]; tree int64 [n, words] (tree_masks) or None for the causal
        mask; scale defaults to head_dim ** -0.5; lse float32 [n, q_heads] or None."""
        d, shape = self.head_dim, q.shape
        n = shape[0]
        if out.shape[0] != n:
            raise ValueError("out must have as many rows as q")
        hq = shape[1] if len(shape) == 3 else shape[1] // d
        dtype, device = self.dtype, self.device
        masks, words = None, 0
        if tree is not None:
            if tree.dtype is not self._i64 or tree.dim() != 2 or tree.shape[0] != n or tree.device != device or \
                    not tree.is_contiguous():
                raise ValueError("tree must be a contiguous int64 tensor [tokens, words]")
            # (a call without tokens has no mask to point at)
            masks, words = tree.data_ptr() or None, tree.shape[1]
        sums = None
        if lse is not None:
            if lse.dtype is not self._f32 or lse.shape != (n, hq) or lse.device != device or not lse.is_contiguous():
                raise ValueError("lse must be a contiguous float32 tensor [tokens, q_heads]")
            sums = lse.data_ptr()
        a = _Attend(*_rows(q, dtype, device, "q", hq, d), hq, max_tokens, d ** -0.5 if scale is None else scale, masks,
                    words, *_rows(out, dtype, device, "out", hq, d), sums, *self._wait_test)
        t = self._tokens(n, cu_tokens, ctx_lens, page_table)
        s = self._stream(stream)
        own = None if workspace is not None else self._buffers(s)
        kv, codes = self._codes(status, t.batch, s, own=own)
        _check(_attend(kv, layer, t, a, *self._workspace(workspace, s, own), codes, s), "tc_attend")

    def attend_wait_test(self, withhold: bool, wait_polls: int = 0):
        """Make attend's kernel leave out its first load (withhold) with waits of `wait_polls` polls; (False, 0)
        restores."""
        self._wait_test = (int(wait_polls), int(bool(withhold)))

    def copy_pages(self, src, dst, status=None, stream=None):
        """tc_kv_copy_pages: page dst[i] becomes page src[i] in every layer."""
        n, s = src.shape[0], self._stream(stream)
        kv, codes = self._codes(status, n, s, pairs=1)
        _check(_kv_copy_pages(kv, self._ints(src, (n,), "src"), self._ints(dst, (n,), "dst"), n, codes, s),
               "tc_kv_copy_pages")

    def compact(self, page_table, ctx_lens, path, n_path, lens_out, status=None, stream=None):
        """tc_kv_compact: slot ctx_lens[b] + i takes what slot ctx_lens[b] + path[b, i] holds, i < n_path[b];
        lens_out = ctx_lens + n_path."""
        t = self._tokens(0, None, ctx_lens, page_table)
        b, wide, s = t.batch, path.shape[-1], self._stream(stream)
        kv, codes = self._codes(status, b, s)
        _check(_kv_compact(kv, t, self._ints(path, (b, wide), "path"), wide, self._ints(n_path, (b,), "n_path"),
                           self._ints(lens_out, (b,), "lens_out"), codes, s), "tc_kv_compact")

    def raise_on_error(self):
        """Wait for the device, and if a call made without `status` since the last error raised has failed, clear
        all codes and raise one of the first errors."""
        import torch
        gathered = [o.codes for o in self._own.values()]
        if self._graph_codes:
            gathered.append(self._graph_codes)
        if not gathered:
            return
        torch.cuda.synchronize(self.device)
        found = None
        for own in gathered:
            for pairs, what in enumerate(("sequence", "page copy")):
                codes = own.codes[KV_MAX_BATCH * pairs:][:own.used[pairs]]
                for i, code in enumerate(codes.tolist()):
                    if code != TC_OK:
                        found = found or (code, f"{what} {i}")
                        codes.zero_()
                        break
        if found:
            torch.cuda.synchronize(self.device)
            raise TcError(*found)


def _int_tensor(t, shape, device, what: str):
    import torch
    if t.dtype is not torch.int32 or t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous int32 tensor of shape {tuple(shape)} on {device}")
    return t.data_ptr()


def tree_masks(parents, cu_tokens, ctx_lens, masks, positions=None, status=None, stream=None):
    """tc_tree_masks: parents int32 [n] -> masks int64 [n, words] and positions int32 [n]."""
    import torch
    n, dev, batch = parents.shape[0], parents.device, ctx_lens.shape[0]
    if masks.dtype is not torch.int64 or masks.device != dev or masks.dim() != 2 or masks.shape[0] != n or \
            not masks.is_contiguous():
        raise ValueError("masks must be a contiguous int64 tensor [tokens, words]")
    with torch.cuda.device(dev):
        s = _stream_ptr(stream)
        if status is None:
            status = _empty(batch, torch.int32, dev, s)
    t = _Tokens(batch, n, _int_tensor(cu_tokens, (batch + 1,), dev, "cu_tokens"),
                _int_tensor(ctx_lens, (batch,), dev, "ctx_lens"), None, 0)
    with torch.cuda.device(dev):
        _check(_tree_masks(ctypes.byref(t), _int_tensor(parents, (n,), dev, "parents"), masks.shape[1], masks.data_ptr(),
                           None if positions is None else _int_tensor(positions, (n,), dev, "positions"),
                           _int_tensor(status, (batch,), dev, "status"), s), "tc_tree_masks")
    return status


class PagePool:
    """Which pages of a cache belong to which sequence (tc_pages; host only)."""

    def __init__(self, pages: int, page_size: int):
        self._h = None
        h = _vp()
        _check(_pages_create(pages, page_size, ctypes.byref(h)), "tc_pages_create")
        self._h, self.page_size = h, page_size

    def open(self) -> int:
        seq = ctypes.c_int32()
        _check(_pages_open(self._h, ctypes.byref(seq)), "tc_pages_open")
        return seq.value

    def close_seq(self, seq: int):
        _check(_pages_close(self._h, seq), "tc_pages_close")

    def reserve(self, seq: int, start: int, end: int) -> list:
        """Room for slots [start, end); returns the copies to make first: [(source page, new page)]."""
        src, dst, n = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32()
        _check(_pages_reserve(self._h, seq, start, end, ctypes.byref(src), ctypes.byref(dst), ctypes.byref(n)),
               "tc_pages_reserve")
        return [(src.value, dst.value)] if n.value else []

    def fork(self, seq: int, length: int) -> int:
        child = ctypes.c_int32()
        _check(_pages_fork(self._h, seq, length, ctypes.byref(child)), "tc_pages_fork")
        return child.value

    def trim(self, seq: int, length: int):
        _check(_pages_trim(self._h, seq, length), "tc_pages_trim")

    def row(self, seq: int, width: int) -> np.ndarray:
        out, n = np.zeros(max(width, 1), dtype=np.int32), ctypes.c_int32()
        _check(_pages_row(self._h, seq, out.ctypes.data_as(_i32p), width, ctypes.byref(n)), "tc_pages_row")
        return out[:width]

    @property
    def free(self) -> int:
        n = ctypes.c_int32()
        _check(_pages_free_count(self._h, ctypes.byref(n)), "tc_pages_free_count")
        return n.value

    def close(self):
        if self._h:
            _pages_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
