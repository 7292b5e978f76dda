"""Python binding of libkvq (ctypes): argument marshalling only.

Every step of the quantize / append / decode path runs in the CUDA library;
PyTorch supplies device memory and the current stream.  The library must be
built (``python -m asymmetric_kv_cache_b200.build``); importing this module
without it raises ImportError, there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
from array import array
from contextlib import nullcontext
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# KVQ_LIBRARY=debug selects libkvq_debug.so, the same library with the
# decode kernels' range checks compiled in (a failed check is reported by
# kvq_workspace_status instead of faulting)
_NAME = "libkvq_debug.so" if os.environ.get("KVQ_LIBRARY") == "debug" else "libkvq.so"
LIB_PATH = os.path.join(_HERE, _NAME)

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{_NAME} not found at {LIB_PATH}; build it with "
                      "`python -m asymmetric_kv_cache_b200.build`")
_lib = ctypes.CDLL(LIB_PATH)

KVQ_OK = 0
STATUS_NAMES = {
    0: "KVQ_OK", 1: "KVQ_ERR_NULL", 2: "KVQ_ERR_CONFIG", 3: "KVQ_ERR_BUFFER_TOO_SMALL",
    4: "KVQ_ERR_CAPACITY", 5: "KVQ_ERR_EMPTY", 6: "KVQ_ERR_DTYPE", 7: "KVQ_ERR_CUDA",
    8: "KVQ_ERR_ALIGN", 9: "KVQ_ERR_ARG", 10: "KVQ_ERR_DEVICE",
}
DTYPE_CODES = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}
LAYOUT_VERSION = 2


class KvqConfig(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "k_bits", "v_bits", "group", "head_dim", "n_q_heads", "n_kv_heads",
        "max_seqs", "max_tokens", "layout_version", "window", "sink", "rotate", "akvq_delta")]


class KvqLayout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_uint64) for n in (
        "total_bytes", "lens_offset", "counters_offset", "blocks_offset", "block_bytes", "max_groups",
        "tails_offset", "tail_bytes", "kcodes_offset", "kscale_offset", "kmin_offset",
        "vcodes_offset", "vscale_offset", "vmin_offset", "tail_slots", "sinks_offset",
        "sink_bytes", "sink_slots", "akvq_block_bytes", "akvq_kscale_offset", "akvq_kmin_offset",
        "akvq_vcodes_offset", "akvq_vscale_offset", "akvq_vmin_offset")]


_NOWHERE = nullcontext()


def _on(stream):
    """Where a call allocates its outputs: on the stream that writes them.  The current stream's allocator may hand out memory
    that kernels of the current stream still read, and would take it back before another stream's have written it."""
    return _NOWHERE if stream is None else torch.cuda.stream(stream)


def _int32s(values, name: str):
    """The integers as an array of int32 (ctypes would cut off the upper bits of those that do not fit)."""
    try:
        return array("i", values)
    except OverflowError:
        raise ValueError(f"{name} must be 32-bit integers") from None


class KvqScores(ctypes.Structure):
    _fields_ = [("scale", ctypes.c_float), ("cap", ctypes.c_float), ("window", ctypes.c_int32),
                ("slopes", ctypes.c_void_p), ("prefix", ctypes.c_void_p)]


class KvqRotary(ctypes.Structure):
    _fields_ = [("inv_freq", ctypes.c_void_p), ("n_pairs", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("positions", ctypes.c_void_p),
                ("n_axes", ctypes.c_int32), ("sections", ctypes.c_int32 * 4),
                ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p),
                ("eps", ctypes.c_float)]


_c_status = ctypes.c_int32
_vp = ctypes.c_void_p
_P = ctypes.POINTER


def _sig(name, args, res=_c_status):
    fn = getattr(_lib, name)
    fn.argtypes = args
    fn.restype = res
    return fn


kvq_status_string = _sig("kvq_status_string", [_c_status], ctypes.c_char_p)
kvq_last_error = _sig("kvq_last_error", [], ctypes.c_char_p)
kvq_layout_for = _sig("kvq_layout_for", [_P(KvqConfig), _P(KvqLayout)])
kvq_cache_required_bytes = _sig("kvq_cache_required_bytes",
                                [_P(KvqConfig), _P(ctypes.c_size_t), _P(ctypes.c_size_t)])
kvq_cache_create = _sig("kvq_cache_create", [_P(KvqConfig), _vp, ctypes.c_size_t, _P(_vp)])
kvq_cache_destroy = _sig("kvq_cache_destroy", [_vp])
kvq_reset = _sig("kvq_reset", [_vp, _vp])
kvq_append = _sig("kvq_append", [_vp, _vp, _vp, ctypes.c_int32, _P(ctypes.c_int32),
                                 ctypes.c_int32, _vp])
kvq_decode = _sig("kvq_decode", [_vp, _vp, ctypes.c_int32, _vp, ctypes.c_int32, _vp,
                                 ctypes.c_size_t, _vp])
kvq_attend = _sig("kvq_attend", [_vp, _vp, ctypes.c_int32, _vp, ctypes.c_int32,
                                 _P(KvqScores), _vp, _vp, ctypes.c_size_t, _vp])
kvq_norm_rotary = _sig("kvq_norm_rotary",
                       [_vp, _vp, ctypes.c_int64, _vp, ctypes.c_int64, _vp, ctypes.c_int64,
                        ctypes.c_int32, _vp, ctypes.c_int32, _P(KvqRotary), _vp, _vp, _vp,
                        ctypes.c_int32, _vp])
kvq_reorder = _sig("kvq_reorder", [_vp, _vp, ctypes.c_int32, ctypes.c_int32, _vp])
kvq_workspace_init = _sig("kvq_workspace_init", [_vp, ctypes.c_size_t, _vp])
kvq_workspace_status = _sig("kvq_workspace_status", [_vp, _vp])
kvq_cache_config = _sig("kvq_cache_config", [_vp, _P(KvqConfig)])
kvq_cache_layout = _sig("kvq_cache_layout", [_vp, _P(KvqLayout)])
kvq_get_lengths = _sig("kvq_get_lengths", [_vp, _P(ctypes.c_int32), ctypes.c_int32])
kvq_sync_lengths = _sig("kvq_sync_lengths", [_vp, _vp])
kvq_decode_noalloc = _sig("kvq_decode_noalloc", [_vp, _vp, ctypes.c_int32, _vp, ctypes.c_int32, _vp])
kvq_noalloc_scratch_bytes = _sig("kvq_noalloc_scratch_bytes", [], ctypes.c_size_t)
kvq_fp16_workspace_bytes = _sig("kvq_fp16_workspace_bytes",
                                [ctypes.c_int32] * 4 + [ctypes.POINTER(ctypes.c_size_t)])
kvq_decode_fp16 = _sig("kvq_decode_fp16",
                       [_vp, _vp, _vp, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                        ctypes.c_int32, ctypes.c_int32, _vp, ctypes.c_int32, _vp, _vp,
                        ctypes.c_size_t, _vp])

EXPORTED = ["kvq_status_string", "kvq_last_error", "kvq_layout_for", "kvq_cache_required_bytes",
            "kvq_cache_create", "kvq_cache_destroy", "kvq_reset", "kvq_append", "kvq_decode",
            "kvq_workspace_init", "kvq_workspace_status", "kvq_cache_config",
            "kvq_cache_layout", "kvq_get_lengths", "kvq_sync_lengths", "kvq_decode_noalloc",
            "kvq_noalloc_scratch_bytes", "kvq_fp16_workspace_bytes", "kvq_decode_fp16",
            "kvq_attend", "kvq_norm_rotary", "kvq_reorder"]


class KvqError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        detail = kvq_last_error().decode(errors="replace")
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}: {detail}")


def check(status: int, where: str) -> None:
    if status != KVQ_OK:
        raise KvqError(status, where)


def make_config(k_bits, v_bits, group, head_dim, n_q_heads, n_kv_heads, max_seqs,
                max_tokens, window=0, sink=0, rotate=0, akvq_delta=0) -> KvqConfig:
    return KvqConfig(k_bits, v_bits, group, head_dim, n_q_heads, n_kv_heads, max_seqs,
                     max_tokens, LAYOUT_VERSION, window, sink, int(rotate), int(akvq_delta))


def required_bytes(cfg: KvqConfig) -> tuple[int, int]:
    c, w = ctypes.c_size_t(), ctypes.c_size_t()
    check(kvq_cache_required_bytes(ctypes.byref(cfg), ctypes.byref(c), ctypes.byref(w)),
          "kvq_cache_required_bytes")
    return c.value, w.value


def layout_for(cfg: KvqConfig) -> dict:
    lay = KvqLayout()
    check(kvq_layout_for(ctypes.byref(cfg), ctypes.byref(lay)), "kvq_layout_for")
    return {n: int(getattr(lay, n)) for n, _ in KvqLayout._fields_}


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _dev_ptr(t: torch.Tensor, name: str) -> int:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


@dataclass
class CacheSpec:
    k_bits: int
    v_bits: int
    group: int
    head_dim: int
    n_q_heads: int
    n_kv_heads: int
    max_seqs: int
    max_tokens: int
    window: int = 0     # R: recent tokens kept in fp16 beyond the partial group
    sink: int = 0       # S: first tokens of each sequence kept in fp16
    rotate: int = 0     # 1: tokens, q and the output rotated by H / sqrt(d)
    akvq_delta: int = 0  # Delta > 0: position-adaptive key bits (4 early/recent, 2 middle)


class KVQCache:
    """A quantized KV cache in a torch-owned device buffer.

    ``append(k, v, n_new)`` adds tokens (prefill, per-step append, flush);
    ``decode(q)`` returns fp16 attention outputs [n_seq, n_q_heads, d].
    """

    def __init__(self, spec: CacheSpec, device="cuda"):
        self.spec = spec
        self.cfg = make_config(spec.k_bits, spec.v_bits, spec.group, spec.head_dim,
                               spec.n_q_heads, spec.n_kv_heads, spec.max_seqs, spec.max_tokens,
                               spec.window, spec.sink, spec.rotate, spec.akvq_delta)
        cache_bytes, ws_bytes = required_bytes(self.cfg)
        self.buffer = torch.empty(cache_bytes, dtype=torch.uint8, device=device)
        self._device = self.buffer.get_device()
        self.workspace = torch.zeros(ws_bytes, dtype=torch.uint8, device=device)
        torch.cuda.synchronize(self.buffer.device)
        h = _vp()
        check(kvq_cache_create(ctypes.byref(self.cfg), self.buffer.data_ptr(), cache_bytes,
                               ctypes.byref(h)), "kvq_cache_create")
        self._h = h
        self.layout = self._layout()

    def _layout(self) -> dict:
        lay = KvqLayout()
        check(kvq_cache_layout(self._h, ctypes.byref(lay)), "kvq_cache_layout")
        return {n: int(getattr(lay, n)) for n, _ in KvqLayout._fields_}

    def close(self):
        if getattr(self, "_h", None):
            kvq_cache_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def lengths(self, n=None) -> list:
        n = self.spec.max_seqs if n is None else n
        arr = (ctypes.c_int32 * n)()
        check(kvq_get_lengths(self._h, arr, n), "kvq_get_lengths")
        return list(arr)

    def sync_lengths(self, stream=None):
        check(kvq_sync_lengths(self._h, _stream(stream)), "kvq_sync_lengths")

    def reset(self, stream=None):
        check(kvq_reset(self._h, _stream(stream)), "kvq_reset")

    def append(self, k: torch.Tensor, v: torch.Tensor, n_new, stream=None):
        """k, v: [sum(n_new), n_kv_heads, d] device tensors (fp16/bf16/fp32)."""
        if k.dtype != v.dtype or k.dtype not in DTYPE_CODES:
            raise ValueError("k and v must share one of fp16/bf16/fp32")
        n_new = [int(x) for x in n_new]
        rows = sum(n_new)
        want = (rows, self.spec.n_kv_heads, self.spec.head_dim)
        if tuple(k.shape) != want or tuple(v.shape) != want:
            raise ValueError(f"k and v must be {want}, got {tuple(k.shape)} and {tuple(v.shape)}")
        arr = (ctypes.c_int32 * len(n_new))(*n_new)
        kp = _dev_ptr(k, "k") if k.numel() else None
        vp = _dev_ptr(v, "v") if v.numel() else None
        check(kvq_append(self._h, kp, vp, DTYPE_CODES[k.dtype], arr, len(n_new), _stream(stream)),
              "kvq_append")

    def decode(self, q: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """q: [n_seq, n_q_heads, d] device tensor; returns fp16 [n_seq, n_q_heads, d]."""
        if q.dtype not in DTYPE_CODES:
            raise ValueError("q must be fp16, bf16 or fp32")
        if q.dim() != 3 or tuple(q.shape[1:]) != (self.spec.n_q_heads, self.spec.head_dim):
            raise ValueError(f"q must be [n_seq, {self.spec.n_q_heads}, {self.spec.head_dim}], "
                             f"got {tuple(q.shape)}")
        n_seq = q.shape[0]
        if out is None:
            out = torch.empty(q.shape, dtype=torch.float16, device=q.device)
        elif out.dtype != torch.float16 or out.shape != q.shape:
            raise ValueError("out must be an fp16 tensor shaped like q")
        check(kvq_decode(self._h, _dev_ptr(q, "q"), DTYPE_CODES[q.dtype], _dev_ptr(out, "out"),
                         n_seq, self.workspace.data_ptr(), self.workspace.numel(),
                         _stream(stream)), "kvq_decode")
        return out

    def decode_noalloc(self, q: torch.Tensor, out: torch.Tensor, stream=None) -> torch.Tensor:
        """kvq_decode_noalloc: decode into a caller-given ``out`` using the
        library's fixed device scratch (no allocation, no workspace)."""
        if q.dtype not in DTYPE_CODES:
            raise ValueError("q must be fp16, bf16 or fp32")
        if q.dim() != 3 or tuple(q.shape[1:]) != (self.spec.n_q_heads, self.spec.head_dim):
            raise ValueError(f"q must be [n_seq, {self.spec.n_q_heads}, {self.spec.head_dim}]")
        if out.dtype != torch.float16 or out.shape != q.shape:
            raise ValueError("out must be an fp16 tensor shaped like q")
        check(kvq_decode_noalloc(self._h, _dev_ptr(q, "q"), DTYPE_CODES[q.dtype],
                                 _dev_ptr(out, "out"), q.shape[0], _stream(stream)),
              "kvq_decode_noalloc")
        return out

    # ---- several new tokens per sequence, positions, reordering ----
    def _ptr(self, t: torch.Tensor, name: str, dtype=None, shape=None) -> int:
        """The address of a contiguous tensor on the cache's device, of the type and shape given."""
        if t.get_device() != self._device:
            raise ValueError(f"{name} must be on {self.buffer.device}, got {t.device}")
        if dtype is not None and t.dtype != dtype:
            raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
        if shape is not None and t.shape != shape:
            raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        return t.data_ptr()

    def _launch(self, name, fn, stream, *args):
        """fn(*args, stream) on the cache's device; without a stream, on that device's current one."""
        if torch.cuda.current_device() == self._device:
            raw = torch._C._cuda_getCurrentRawStream(self._device) if stream is None else stream.cuda_stream
            status = fn(*args, raw)
        else:
            with torch.cuda.device(self._device):
                status = fn(*args, _stream(stream))
        if status != KVQ_OK:
            raise KvqError(status, name)

    def attend(self, q: torch.Tensor, n_q, scale: float = 0.0, cap: float = 0.0, window: int = 0,
               slopes: torch.Tensor | None = None, prefix: torch.Tensor | None = None,
               out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """Attention of the newest ``n_q[b]`` tokens of each sequence (kvq_attend).

        q: [sum(n_q), n_q_heads, d]; scale (0: 1 / sqrt(d)), cap, window: numbers, 0 for none;
        slopes: fp32 [n_q_heads], prefix: int32 [n_seq], on the device.  Returns fp16 like q, written to
        ``out`` if given, else to a new tensor of ``stream``.
        """
        dt = DTYPE_CODES.get(q.dtype)
        if dt is None:
            raise ValueError("q must be fp16, bf16 or fp32")
        if not -2 ** 31 <= window < 2 ** 31:
            raise ValueError("window must be a 32-bit integer")
        sp, n_seq = self.spec, len(n_q)
        arr = _int32s(n_q, "n_q")
        shape = (sum(n_q), sp.n_q_heads, sp.head_dim)
        qp = self._ptr(q, "q", None, shape)
        sc = KvqScores(scale, cap, window,
                       None if slopes is None else self._ptr(slopes, "slopes", torch.float32, (sp.n_q_heads,)),
                       None if prefix is None else self._ptr(prefix, "prefix", torch.int32, (n_seq,)))
        if out is None:
            with _on(stream):
                out = torch.empty(shape, dtype=torch.float16, device=q.device)
        self._launch("kvq_attend", kvq_attend, stream, self._h, qp, dt, arr.buffer_info()[0], n_seq, ctypes.byref(sc),
                     self._ptr(out, "out", torch.float16, shape), self.workspace.data_ptr(),
                     self.workspace.numel())
        return out

    def _rows(self, t: torch.Tensor, name: str, dtype, shape) -> tuple[int, int]:
        """Address of t [rows, heads, d] with each row's heads side by side, and elements between rows."""
        if t.get_device() != self._device or t.dtype != dtype:
            raise ValueError(f"{name} must be {dtype} on {self.buffer.device}, got {t.dtype} on {t.device}")
        if t.shape != shape:
            raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
        st = t.stride()
        if t.numel() and (st[2] != 1 or (shape[1] > 1 and st[1] != shape[2])):
            raise ValueError(f"{name}: a row's heads must lie side by side")
        return t.data_ptr(), st[0] if shape[0] > 1 else shape[1] * shape[2]

    def norm_rotary(self, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor | None, n_new,
                    inv_freq: torch.Tensor, q_weight: torch.Tensor | None = None,
                    k_weight: torch.Tensor | None = None, eps: float = 1e-6,
                    positions: torch.Tensor | None = None, sections=None, interleaved: bool = False,
                    out_dtype=torch.float16, out=None, stream=None):
        """Norms and position rotation of new tokens' rows (kvq_norm_rotary): what ``append``,
        ``decode`` and ``attend`` take.  Called before the append.

        q, k, v: [sum(n_new), heads, d] of one type, heads side by side, any row stride (slices of
        one projection output); inv_freq: fp32 [pairs]; q_weight, k_weight: [d] of the rows' type,
        None for no norm; positions: None (the cache's lengths + 0, 1, ..) or int32 [rows] or
        [axes, rows] with the pairs of each axis in ``sections``.  Returns contiguous (q, k, v) of
        ``out_dtype`` (v None if it was), written to ``out`` if three tensors are given, else to new
        tensors of ``stream``.
        """
        dt, odt = DTYPE_CODES.get(q.dtype), DTYPE_CODES.get(out_dtype)
        if dt is None or odt is None:
            raise ValueError("rows and outputs must be fp16, bf16 or fp32")
        sp, n, n_seq, d, kind = self.spec, sum(n_new), len(n_new), self.spec.head_dim, q.dtype
        arr = _int32s(n_new, "n_new")
        q_shape, k_shape = (n, sp.n_q_heads, d), (n, sp.n_kv_heads, d)
        qp, qs = self._rows(q, "q", kind, q_shape)
        kp, ks = self._rows(k, "k", kind, k_shape)
        vp, vs = (None, 0) if v is None else self._rows(v, "v", kind, k_shape)
        if inv_freq.dim() != 1:
            raise ValueError("inv_freq must be [pairs]")
        pairs = inv_freq.numel()
        rot = KvqRotary(self._ptr(inv_freq, "inv_freq", torch.float32), pairs, int(interleaved), None, 0,
                        (0, 0, 0, 0),
                        None if q_weight is None else self._ptr(q_weight, "q_weight", kind, (d,)),
                        None if k_weight is None else self._ptr(k_weight, "k_weight", kind, (d,)), eps)
        if positions is not None:
            axes = positions.shape[0] if positions.dim() == 2 else 1
            if positions.dim() not in (1, 2) or positions.shape[-1] != n or not 1 <= axes <= 4:
                raise ValueError(f"positions must be [{n}] or [1 to 4 axes, {n}]")
            sections = [pairs] if sections is None and axes == 1 else list(sections or [])
            if len(sections) != axes:
                raise ValueError(f"sections must give the pairs of {axes} axes")
            rot.positions = self._ptr(positions, "positions", torch.int32)
            rot.n_axes = axes
            rot.sections[:axes] = _int32s(sections, "sections")[:axes]
        elif sections is not None:
            raise ValueError("sections go with positions")
        if out is None:
            dev = q.device
            with _on(stream):
                out = (torch.empty(q_shape, dtype=out_dtype, device=dev), torch.empty(k_shape, dtype=out_dtype, device=dev),
                       None if v is None else torch.empty(k_shape, dtype=out_dtype, device=dev))
        qo, ko, vo = out
        if qo is None or ko is None or (vo is None) != (v is None):
            raise ValueError("out must hold a tensor for each of q, k and v")
        self._launch("kvq_norm_rotary", kvq_norm_rotary, stream, self._h, qp, qs, kp, ks, vp, vs, dt,
                     arr.buffer_info()[0], n_seq, ctypes.byref(rot), self._ptr(qo, "q output", out_dtype, q_shape),
                     self._ptr(ko, "k output", out_dtype, k_shape),
                     None if vo is None else self._ptr(vo, "v output", out_dtype, k_shape), odt)
        return qo, ko, vo

    def reorder(self, parent, shared: int = 0, stream=None):
        """Sequence b takes over sequence ``parent[b]``, all at once (kvq_reorder); the first
        ``shared`` tokens of moving sequences and their parents are the same already."""
        if not -2 ** 31 <= shared < 2 ** 31:
            raise ValueError("shared must be a 32-bit integer")
        arr = _int32s(parent, "parent")
        self._launch("kvq_reorder", kvq_reorder, stream, self._h, arr.buffer_info()[0], len(arr), int(shared))

    def workspace_status(self, stream=None) -> int:
        return kvq_workspace_status(self.workspace.data_ptr(), _stream(stream))

    # ---- views of the raw buffer (tests, checkpointing) ----
    def block_bytes(self, seq: int, kv_head: int, n_groups: int) -> torch.Tensor:
        L = self.layout
        base = L["blocks_offset"] + ((seq * self.spec.n_kv_heads + kv_head) * L["max_groups"]) * L["block_bytes"]
        return self.buffer[base: base + n_groups * L["block_bytes"]].view(n_groups, L["block_bytes"])

    def tail_halves(self, seq: int, kv_head: int) -> tuple[torch.Tensor, torch.Tensor]:
        L = self.layout
        W, d = L["tail_slots"], self.spec.head_dim
        base = L["tails_offset"] + (seq * self.spec.n_kv_heads + kv_head) * L["tail_bytes"]
        raw = self.buffer[base: base + L["tail_bytes"]].view(torch.float16)
        return raw[: W * d], raw[W * d: 2 * W * d]

    def sink_halves(self, seq: int, kv_head: int) -> tuple[torch.Tensor, torch.Tensor]:
        L = self.layout
        SW, d = L["sink_slots"], self.spec.head_dim
        base = L["sinks_offset"] + (seq * self.spec.n_kv_heads + kv_head) * L["sink_bytes"]
        raw = self.buffer[base: base + L["sink_bytes"]].view(torch.float16)
        return raw[: SW * d], raw[SW * d: 2 * SW * d]

    def device_lengths(self) -> torch.Tensor:
        L = self.layout
        return self.buffer[L["lens_offset"]: L["lens_offset"] + 4 * self.spec.max_seqs].view(torch.int32)


def decode_fp16(k: torch.Tensor, v: torch.Tensor, lens: torch.Tensor, q: torch.Tensor,
                out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                stream=None) -> torch.Tensor:
    """kvq_decode_fp16, the unquantized comparison kernel: k, v fp16 CUDA
    tensors [n_seq, n_kv_heads, max_tokens, head_dim], lens int32 CUDA
    [n_seq], q [n_seq, n_q_heads, head_dim] fp16/bf16/fp32."""
    if k.dtype != torch.float16 or v.dtype != torch.float16 or k.shape != v.shape or k.dim() != 4:
        raise ValueError("k and v must be fp16 [n_seq, n_kv_heads, max_tokens, head_dim]")
    n_seq, hkv, max_tokens, d = k.shape
    if q.dtype not in DTYPE_CODES or q.dim() != 3 or q.shape[0] != n_seq or q.shape[2] != d:
        raise ValueError("q must be [n_seq, n_q_heads, head_dim] fp16/bf16/fp32")
    if lens.dtype != torch.int32 or tuple(lens.shape) != (n_seq,):
        raise ValueError("lens must be int32 [n_seq]")
    hq = q.shape[1]
    if out is None:
        out = torch.empty(q.shape, dtype=torch.float16, device=q.device)
    nbytes = ctypes.c_size_t()
    check(kvq_fp16_workspace_bytes(n_seq, hq, hkv, d, ctypes.byref(nbytes)), "kvq_fp16_workspace_bytes")
    if workspace is None or workspace.numel() < nbytes.value:
        workspace = torch.zeros(nbytes.value, dtype=torch.uint8, device=q.device)
    check(kvq_decode_fp16(_dev_ptr(k, "k"), _dev_ptr(v, "v"), _dev_ptr(lens, "lens"), max_tokens,
                          n_seq, hq, hkv, d, _dev_ptr(q, "q"), DTYPE_CODES[q.dtype],
                          _dev_ptr(out, "out"), workspace.data_ptr(), workspace.numel(),
                          _stream(stream)), "kvq_decode_fp16")
    return out
