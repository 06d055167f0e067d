"""ctypes binding of libkvq (include/kvq.h), plus a small cache holder.

Argument marshalling only: every step of append, decode attention and
dequantization runs in the library's CUDA kernels.  PyTorch provides device
memory and streams.  Importing this module without a built libkvq.so raises.
"""

from __future__ import annotations

import contextlib
import ctypes
import os
from typing import Optional, Tuple

from .config import (AXIS_CHANNEL, AXIS_TOKEN, DEV_BOUNDS, DEV_CAPACITY, DEV_LENGTH, DEV_PAGE,  # noqa: F401
                     DEV_RANGE, DEV_SEQ, DEV_STALL, DT_BF16, DT_F16, K_PRE_ROPE, ROPE_BANDS, ROPE_LINEAR, ROPE_NONE,
                     ROPE_NTK, ROPE_YARN, ROTATE_K, ROTATE_V, TBQ4_K, TBQ4_V, ZP_K, ZP_V, Config, Fmt)

_PKG = os.path.dirname(os.path.abspath(__file__))
# KVQ_LIBRARY selects another build of the same ABI (the tests use it for the
# bounds-checked libkvq_checked.so).
LIB_PATH = os.environ.get("KVQ_LIBRARY") or os.path.join(_PKG, "libkvq.so")

STATUS_NAMES = {0: "OK", 1: "ERR_ARG", 2: "ERR_UNSUPPORTED", 3: "ERR_CUDA", 4: "ERR_CAPACITY", 5: "ERR_WORKSPACE"}


class KvqError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


class _Fmt(ctypes.Structure):
    _fields_ = [("bits", ctypes.c_int32), ("group", ctypes.c_int32), ("axis", ctypes.c_int32)]


class _Config(ctypes.Structure):
    _fields_ = [
        ("L", ctypes.c_int32), ("H_kv", ctypes.c_int32), ("H_q", ctypes.c_int32), ("D", ctypes.c_int32),
        ("batch", ctypes.c_int32), ("max_T", ctypes.c_int32), ("in_dtype", ctypes.c_int32),
        ("k_fmt", _Fmt), ("v_fmt", _Fmt), ("k_cold", _Fmt), ("v_cold", _Fmt),
        ("hot_window", ctypes.c_int32), ("residual_window", ctypes.c_int32),
        ("flags", ctypes.c_uint32), ("rope_theta", ctypes.c_float), ("sign_seed", ctypes.c_uint64),
        ("page_tokens", ctypes.c_int32), ("n_pages", ctypes.c_int32), ("max_pages_per_seq", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
    ]


class _Cache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k_main", "v_main", "k_cold", "v_cold", "k_resid", "v_resid",
                                                  "block_table")]


class _RopeParams(ctypes.Structure):
    _fields_ = [
        ("D", ctypes.c_int32), ("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("scaling", ctypes.c_int32),
        ("theta", ctypes.c_double), ("factor", ctypes.c_double), ("low", ctypes.c_double), ("high", ctypes.c_double),
        ("original_len", ctypes.c_int32), ("reserved", ctypes.c_int32), ("attn_factor", ctypes.c_double),
    ]


class RopePlan(ctypes.Structure):
    """kvq_rope_plan: a prepared rotary turn (rope_plan), host data."""

    _fields_ = [
        ("D", ctypes.c_int32), ("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("reserved", ctypes.c_int32),
        ("scale", ctypes.c_float), ("unused", ctypes.c_float), ("turns", ctypes.c_uint64 * 128),
    ]


def _to_c(cfg: Config) -> _Config:
    """kvq_config of a Config."""
    def f(x: Optional[Fmt]) -> _Fmt:
        return _Fmt() if x is None else _Fmt(x.bits, x.group, x.axis)

    return _Config(cfg.L, cfg.H_kv, cfg.H_q, cfg.D, cfg.batch, cfg.max_T, cfg.in_dtype, f(cfg.k_fmt), f(cfg.v_fmt),
                   f(cfg.k_cold), f(cfg.v_cold), cfg.hot_window, cfg.residual_window, cfg.flags, cfg.rope_theta,
                   cfg.sign_seed, cfg.page_tokens, cfg.n_pages, cfg.max_pages_per_seq, 0)


def _load():
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -c 'import __graft_entry__ as g; g.build()'`")
    lib = ctypes.CDLL(LIB_PATH)
    P = ctypes.POINTER
    vp, i32, i64, u32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32, ctypes.c_size_t
    cfgp, cachep = P(_Config), P(_Cache)
    sig = {
        "kvq_version": ([], ctypes.c_char_p),
        "kvq_last_error": ([], ctypes.c_char_p),
        "kvq_validate_config": ([cfgp], ctypes.c_int),
        "kvq_block_bytes": ([i32, i32, P(i32)], ctypes.c_int),
        "kvq_bytes_per_token": ([cfgp, P(i64)], ctypes.c_int),
        "kvq_cache_bytes": ([cfgp, i64, P(i64)], ctypes.c_int),
        "kvq_buffer_sizes": ([cfgp, P(sz)], ctypes.c_int),
        "kvq_workspace_bytes": ([cfgp, P(sz)], ctypes.c_int),
        "kvq_workspace_init": ([cfgp, vp, sz, vp], ctypes.c_int),
        "kvq_append": ([cfgp, cachep, i32, i32, vp, vp, vp, vp, i32, i32, vp, sz, vp], ctypes.c_int),
        "kvq_commit_lengths": ([cfgp, vp, vp, vp], ctypes.c_int),
        "kvq_decode_attention": ([cfgp, cachep, i32, i32, vp, vp, vp, i32, vp, sz, vp], ctypes.c_int),
        "kvq_decode_splits": ([cfgp, i32, P(i32)], ctypes.c_int),
        "kvq_decode_step": ([cfgp, cachep, i32, i32, vp, vp, vp, vp, vp, i32, vp, sz, vp], ctypes.c_int),
        "kvq_step_launches": ([cfgp, P(i32)], ctypes.c_int),
        "kvq_launch_counts": ([cfgp, P(i32), P(i32)], ctypes.c_int),
        "kvq_tbq4_codebook": ([P(ctypes.c_float), P(ctypes.c_float)], ctypes.c_int),
        "kvq_decode_attention_static": ([cfgp, cachep, i32, i32, vp, vp, vp, i32, vp], ctypes.c_int),
        "kvq_dequantize": ([cfgp, cachep, i32, i32, i32, i32, vp, vp, vp, vp, sz, vp], ctypes.c_int),
        "kvq_test_force_stall": ([i32], ctypes.c_int),
        "kvq_test_shrink_bounds": ([i32], ctypes.c_int),
        "kvq_rope_plan_init": ([P(_RopeParams), P(RopePlan)], ctypes.c_int),
        "kvq_qk_norm_rope": ([cfgp, P(RopePlan), vp, i64, i64, vp, i64, i64, vp, vp, ctypes.c_float, vp, i32, vp, vp,
                              vp], ctypes.c_int),
        "kvq_pages_workspace_bytes": ([cfgp, P(sz)], ctypes.c_int),
        "kvq_pages_init": ([cfgp, vp, vp, vp, sz, vp], ctypes.c_int),
        "kvq_pages_release": ([cfgp, vp, vp, vp, vp, i32, vp, sz, vp], ctypes.c_int),
        "kvq_pages_fork": ([cfgp, cachep, vp, vp, vp, vp, vp, i32, vp, sz, vp], ctypes.c_int),
        "kvq_pages_reserve": ([cfgp, cachep, vp, vp, vp, vp, vp, i32, vp, sz, vp], ctypes.c_int),
        "kvq_pages_compact": ([cfgp, cachep, vp, vp, vp, vp, vp, sz, vp], ctypes.c_int),
        "kvq_chunk_workspace_bytes": ([cfgp, P(sz)], ctypes.c_int),
        "kvq_chunk_workspace_init": ([cfgp, vp, sz, vp], ctypes.c_int),
        "kvq_chunk_attention": ([cfgp, cachep, i32, i32, vp, vp, i32, i32, vp, i32, i32, vp, vp, sz, vp], ctypes.c_int),
        "kvq_read_device_status": ([vp, P(u32), vp], ctypes.c_int),
        "kvq_clear_device_status": ([vp, vp], ctypes.c_int),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    return lib


LIB = _load()

# C-ABI names declared in include/kvq.h (checked by the tests).
EXPORTED = ("kvq_version", "kvq_last_error", "kvq_validate_config", "kvq_block_bytes", "kvq_bytes_per_token",
            "kvq_cache_bytes", "kvq_buffer_sizes", "kvq_workspace_bytes", "kvq_workspace_init", "kvq_append",
            "kvq_commit_lengths", "kvq_decode_attention", "kvq_decode_splits", "kvq_decode_attention_static",
            "kvq_dequantize", "kvq_launch_counts", "kvq_tbq4_codebook", "kvq_decode_step", "kvq_step_launches",
            "kvq_read_device_status", "kvq_clear_device_status", "kvq_test_force_stall",
            "kvq_test_shrink_bounds", "kvq_rope_plan_init", "kvq_qk_norm_rope", "kvq_pages_workspace_bytes",
            "kvq_pages_init", "kvq_pages_release", "kvq_pages_fork", "kvq_pages_reserve", "kvq_pages_compact",
            "kvq_chunk_workspace_bytes", "kvq_chunk_workspace_init", "kvq_chunk_attention")


def _check(st: int):
    if st != 0:
        raise KvqError(st, LIB.kvq_last_error().decode())


# ---- thin wrappers, same names as the C ABI --------------------------------


def kvq_version() -> str:
    return LIB.kvq_version().decode()


def kvq_validate_config(cfg: Config) -> None:
    _check(LIB.kvq_validate_config(ctypes.byref(_to_c(cfg))))


def kvq_block_bytes(bits: int, group: int) -> int:
    out = ctypes.c_int32()
    _check(LIB.kvq_block_bytes(bits, group, ctypes.byref(out)))
    return out.value


def kvq_bytes_per_token(cfg: Config) -> int:
    out = ctypes.c_int64()
    _check(LIB.kvq_bytes_per_token(ctypes.byref(_to_c(cfg)), ctypes.byref(out)))
    return out.value


def kvq_cache_bytes(cfg: Config, T: int) -> int:
    out = ctypes.c_int64()
    _check(LIB.kvq_cache_bytes(ctypes.byref(_to_c(cfg)), T, ctypes.byref(out)))
    return out.value


def kvq_buffer_sizes(cfg: Config) -> Tuple[int, ...]:
    arr = (ctypes.c_size_t * 6)()
    _check(LIB.kvq_buffer_sizes(ctypes.byref(_to_c(cfg)), arr))
    return tuple(arr)


def kvq_tbq4_codebook():
    """(16 centroids, 15 thresholds) of the TBQ4 format, fp32 lists."""
    c = (ctypes.c_float * 16)()
    t = (ctypes.c_float * 15)()
    _check(LIB.kvq_tbq4_codebook(c, t))
    return list(c), list(t)


def kvq_launch_counts(cfg: Config):
    """(kernel launches of one kvq_append call, of one kvq_decode_attention call)."""
    a, d = ctypes.c_int32(), ctypes.c_int32()
    _check(LIB.kvq_launch_counts(ctypes.byref(_to_c(cfg)), ctypes.byref(a), ctypes.byref(d)))
    return a.value, d.value


def kvq_step_launches(cfg: Config) -> int:
    """Kernel launches of one kvq_decode_step call (1 when fused)."""
    n = ctypes.c_int32()
    _check(LIB.kvq_step_launches(ctypes.byref(_to_c(cfg)), ctypes.byref(n)))
    return n.value


def kvq_workspace_bytes(cfg: Config) -> int:
    out = ctypes.c_size_t()
    _check(LIB.kvq_workspace_bytes(ctypes.byref(_to_c(cfg)), ctypes.byref(out)))
    return out.value


def kvq_decode_splits(cfg: Config, n_layers: int) -> int:
    out = ctypes.c_int32()
    _check(LIB.kvq_decode_splits(ctypes.byref(_to_c(cfg)), n_layers, ctypes.byref(out)))
    return out.value


def kvq_pages_workspace_bytes(cfg: Config) -> int:
    out = ctypes.c_size_t()
    _check(LIB.kvq_pages_workspace_bytes(ctypes.byref(_to_c(cfg)), ctypes.byref(out)))
    return out.value


def kvq_chunk_workspace_bytes(cfg: Config) -> int:
    out = ctypes.c_size_t()
    _check(LIB.kvq_chunk_workspace_bytes(ctypes.byref(_to_c(cfg)), ctypes.byref(out)))
    return out.value


def kvq_test_shrink_bounds(rows: int) -> None:
    """Bounds-checked build: treat the last `rows` rows of every cache segment
    as outside it (0 = off)."""
    _check(LIB.kvq_test_shrink_bounds(rows))


def kvq_test_force_stall(polls: int) -> None:
    """Failure-detection test mode of the tensor-core decode (0 = off)."""
    _check(LIB.kvq_test_force_stall(polls))


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch

        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


def _on(stream):
    """The given stream (None: the current one) as torch's current one.  Memory
    made in here belongs to it: the allocator hands out no block that another
    stream's pending work still writes."""
    import torch

    if stream is None:
        return contextlib.nullcontext()
    return torch.cuda.stream(stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(stream))


BUFFER_NAMES = ("k_main", "v_main", "k_cold", "v_cold", "k_resid", "v_resid")


def _here(index, *tensors) -> None:
    """The tensors live on GPU `index`, and that is the current one: streams and launches belong to it."""
    for t in tensors:
        if t is not None and t.get_device() != index:
            raise ValueError(f"a tensor is on {t.device}, not on device {index}")
    if index < 0:
        raise ValueError("tensors must be on a GPU")
    if index != _current_device():
        raise ValueError(f"device {index} is not the current one")


def _current_device() -> int:
    import torch

    return torch.cuda.current_device()


class KVCache:
    """Device buffers (torch tensors) of one quantized cache plus its workspace."""

    def __init__(self, cfg: Config, device="cuda", block_table=None, buffers=None):
        import torch

        self.cfg = cfg
        self.c_cfg = _to_c(cfg)
        self.device = torch.device(device)
        sizes = kvq_buffer_sizes(cfg)
        self.buffers = {}
        for name, n in zip(BUFFER_NAMES, sizes):
            given = None if buffers is None else buffers.get(name)
            if given is not None and given.numel() * given.element_size() < n:
                raise ValueError(f"{name}: {given.numel() * given.element_size()} bytes, {n} needed")
            if buffers is not None and n and given is None:
                raise ValueError(f"{name} is needed")
            if given is not None:
                if not given.is_contiguous():
                    raise ValueError(f"{name} must be contiguous")
                self.buffers[name] = given
            else:
                self.buffers[name] = torch.zeros(n, dtype=torch.uint8, device=self.device) if n else None
        self.block_table = None
        if block_table is not None:
            self.block_table = torch.as_tensor(block_table, dtype=torch.int32).to(self.device).contiguous()
        if buffers is not None:
            if len({t.device for t in (*self.buffers.values(), self.block_table) if t is not None}) > 1:
                raise ValueError("buffers and block table are on one device")
            if cfg.page_tokens:
                self._check_table()
        self.ws_bytes = kvq_workspace_bytes(cfg)
        self.workspace = torch.empty(self.ws_bytes, dtype=torch.uint8, device=self.device)
        self.index = self.workspace.get_device()
        self.c_cache = _Cache(*[_ptr(self.buffers[n]) for n in BUFFER_NAMES], _ptr(self.block_table))
        _check(LIB.kvq_workspace_init(ctypes.byref(self.c_cfg), _ptr(self.workspace), self.ws_bytes,
                                      _stream(None)))
        self.chunk_ws_bytes = kvq_chunk_workspace_bytes(cfg)
        self.chunk_workspace = None  # the last one that chunk_attention chose by itself
        self._chunk_workspaces = {}  # by stream

    @classmethod
    def from_buffers(cls, cfg: Config, buffers: dict, block_table=None) -> "KVCache":
        """A cache over the caller's filled buffers (contiguous tensors by
        BUFFER_NAMES, in the layout of include/kvq.h); they are used as they
        are, and so is an int32 block table on their device."""
        return cls(cfg, next(iter(buffers.values())).device, block_table, buffers)

    def _check_table(self):
        if self.block_table is None or self.block_table.numel() < self.cfg.batch * self.cfg.max_pages_per_seq:
            raise ValueError("a paged cache needs a block table [batch, max_pages_per_seq]")

    # -- the C calls ----------------------------------------------------------

    def append(self, layer0, n_layers, k, v, cu_new, seq_lens, total_new, max_new, stream=None):
        _check(LIB.kvq_append(ctypes.byref(self.c_cfg), ctypes.byref(self.c_cache), layer0, n_layers,
                              _ptr(k), _ptr(v), _ptr(cu_new), _ptr(seq_lens), total_new, max_new,
                              _ptr(self.workspace), self.ws_bytes, _stream(stream)))

    def commit_lengths(self, cu_new, seq_lens, stream=None):
        _check(LIB.kvq_commit_lengths(ctypes.byref(self.c_cfg), _ptr(cu_new), _ptr(seq_lens), _stream(stream)))

    def decode(self, layer0, n_layers, q, seq_lens, out, num_splits=0, stream=None):
        _check(LIB.kvq_decode_attention(ctypes.byref(self.c_cfg), ctypes.byref(self.c_cache), layer0, n_layers,
                                        _ptr(q), _ptr(seq_lens), _ptr(out), num_splits,
                                        _ptr(self.workspace), self.ws_bytes, _stream(stream)))

    def decode_step(self, layer0, n_layers, k_new, v_new, q, seq_lens, out, num_splits=0, stream=None):
        _check(LIB.kvq_decode_step(ctypes.byref(self.c_cfg), ctypes.byref(self.c_cache), layer0, n_layers,
                                   _ptr(k_new), _ptr(v_new), _ptr(q), _ptr(seq_lens), _ptr(out), num_splits,
                                   _ptr(self.workspace), self.ws_bytes, _stream(stream)))

    def make_chunk_workspace(self, stream=None):
        """A prepared workspace for chunk_attention, made on `stream`.  Calls that may run at
        the same time (other streams, graphs replayed side by side) each need one; calls in
        order may share one, also those of other caches of the same head size (62 MB for each)."""
        import torch

        with _on(stream):
            ws = torch.empty(self.chunk_ws_bytes, dtype=torch.uint8, device=self.device)
        _check(LIB.kvq_chunk_workspace_init(ctypes.byref(self.c_cfg), _ptr(ws), self.chunk_ws_bytes, _stream(stream)))
        return ws

    def chunk_attention(self, layer0, n_layers, q, cu_q, total_q, max_q, seq_lens, out, window=0, sinks=0, stream=None,
                        workspace=None):
        """Attention of the last cu_q[b+1] - cu_q[b] cached tokens of every sequence (kvq_chunk_attention).

        Without a workspace the cache keeps one for each stream (chunk_ws_bytes,
        made by the stream's first call).  A captured call without one takes the capturing stream's, else the one
        of the cache's last call: its replays then must not run beside other calls with that workspace."""
        import torch

        cfg = self.cfg
        dt = torch.float16 if cfg.in_dtype == DT_F16 else torch.bfloat16
        for t in (q, out):
            if t.dtype != dt or t.shape != (n_layers, total_q, cfg.H_q, cfg.D) or not t.is_contiguous():
                raise ValueError("q and out are contiguous [n_layers, total_q, H_q, D] tensors of the cache's dtype")
        for t, n in ((cu_q, cfg.batch + 1), (seq_lens, cfg.batch)):
            if t.dtype != torch.int32 or t.numel() != n or not t.is_contiguous():
                raise ValueError("cu_q [batch + 1] and seq_lens [batch] are contiguous int32 tensors")
        _here(self.index, q, out, cu_q, seq_lens, workspace)
        if cfg.page_tokens:
            self._check_table()
        if workspace is None:
            workspace = self.chunk_workspace = self._chunk_workspace_of(stream)
        _check(LIB.kvq_chunk_attention(ctypes.byref(self.c_cfg), ctypes.byref(self.c_cache), layer0, n_layers,
                                       _ptr(q), _ptr(cu_q), total_q, max_q, _ptr(seq_lens), window, sinks, _ptr(out),
                                       _ptr(workspace), workspace.numel(), _stream(stream)))

    def chunk_status(self, workspace=None, stream=None) -> int:
        """KVQ_DEV_* bits that chunk_attention has set in a workspace since they
        were cleared, read on `stream`; without a workspace those of all that the cache has
        made by itself, when the device has finished its work."""
        bits, out = 0, ctypes.c_uint32()
        for ws, s in self._chunk_words(workspace, stream):
            _check(LIB.kvq_read_device_status(_ptr(ws), ctypes.byref(out), s))
            bits |= out.value
        return bits

    def clear_chunk_status(self, workspace=None, stream=None):
        for ws, s in self._chunk_words(workspace, stream):
            _check(LIB.kvq_clear_device_status(_ptr(ws), s))

    def _chunk_words(self, workspace, stream):
        if workspace is not None:
            return [(workspace, _stream(stream))]
        import torch

        torch.cuda.synchronize(self.device)  # of every stream; some may not exist any more
        return [(ws, _stream(stream)) for ws in list(self._chunk_workspaces.values())]

    def _chunk_workspace_of(self, stream):
        import torch

        handle = _stream(stream)
        if handle not in self._chunk_workspaces:
            with _on(stream):
                capturing = torch.cuda.is_current_stream_capturing()
            if capturing:  # nothing can be prepared in here once and for all
                if self.chunk_workspace is None:
                    raise RuntimeError("the first chunk_attention prepares its workspace: make it before the capture")
                return self.chunk_workspace
            self._chunk_workspaces[handle] = self.make_chunk_workspace(stream)
        return self._chunk_workspaces[handle]

    def dequantize(self, layer, seq, t0, t1, seq_lens, k_out, v_out, stream=None):
        _check(LIB.kvq_dequantize(ctypes.byref(self.c_cfg), ctypes.byref(self.c_cache), layer, seq, t0, t1,
                                  _ptr(seq_lens), _ptr(k_out), _ptr(v_out), _ptr(self.workspace), self.ws_bytes,
                                  _stream(stream)))

    def device_status(self, stream=None) -> int:
        out = ctypes.c_uint32()
        _check(LIB.kvq_read_device_status(_ptr(self.workspace), ctypes.byref(out), _stream(stream)))
        return out.value

    def clear_status(self, stream=None):
        _check(LIB.kvq_clear_device_status(_ptr(self.workspace), _stream(stream)))

    def buffer_numpy(self) -> dict:
        """Host copies of the buffers shaped as the oracle expects (tests only)."""
        import numpy as np

        out = {}
        for n in BUFFER_NAMES:
            t = self.buffers[n]
            if t is not None:
                a = t.cpu().numpy()
                out[n] = a.view(np.uint16) if n.endswith("resid") else a
        return out


def rope_plan(D, rot_dim=None, interleaved=False, theta=10000.0, scaling=ROPE_NONE, factor=1.0, low=1.0, high=32.0,
              original_len=0, attn_factor=0.0) -> RopePlan:
    """A prepared rotary turn for qk_norm_rope (kvq_rope_plan_init)."""
    p = _RopeParams(D, D if rot_dim is None else rot_dim, int(interleaved), scaling, theta, factor, low, high,
                    original_len, 0, attn_factor)
    plan = RopePlan()
    _check(LIB.kvq_rope_plan_init(ctypes.byref(p), ctypes.byref(plan)))
    return plan


def qk_norm_rope(cfg: Config, q, k, positions, q_out, k_out, plan=None, q_weight=None, k_weight=None, eps=1e-6,
                 stream=None) -> None:
    """RMS norm and rotary turn of queries and keys in one pass
    (kvq_qk_norm_rope).  q, k: [tokens, heads, D], any token and head stride;
    q_out, k_out contiguous; either pair may be None."""
    import torch

    some = q if q is not None else k
    if some is None:
        raise ValueError("q and k are both None")
    dt = torch.float16 if cfg.in_dtype == DT_F16 else torch.bfloat16
    n = some.shape[0]
    for t, o, w, h in ((q, q_out, q_weight, cfg.H_q), (k, k_out, k_weight, cfg.H_kv)):
        if t is not None and (t.shape != (n, h, cfg.D) or t.stride(2) != 1 or t.dtype != dt or o is None or
                              o.shape != t.shape or o.dtype != dt or not o.is_contiguous()):
            raise ValueError("tensors are [tokens, heads, D] of the configuration with contiguous channels, outputs "
                             "contiguous and alike")
        if w is not None and (w.numel() != cfg.D or w.dtype != dt or not w.is_contiguous()):
            raise ValueError("a weight is a contiguous [D] tensor of the same dtype")
    if plan is not None and (positions is None or positions.dtype != torch.int32 or positions.numel() != n or
                             not positions.is_contiguous()):
        raise ValueError("positions is a contiguous int32 tensor, one of each token")
    if n == 0:  # empty tensors have no address
        return
    _here(some.get_device(), q, k, q_out, k_out, q_weight, k_weight, positions)
    qs = (0, 0) if q is None else q.stride()
    ks = (0, 0) if k is None else k.stride()
    _check(LIB.kvq_qk_norm_rope(ctypes.byref(_to_c(cfg)), None if plan is None else ctypes.byref(plan), _ptr(q), qs[0],
                                qs[1], _ptr(k), ks[0], ks[1], _ptr(q_weight), _ptr(k_weight), eps, _ptr(positions),
                                n, _ptr(q_out), _ptr(k_out), _stream(stream)))


class PagePool:
    """The pages of a paged KVCache: reader counts and the calls that share,
    copy, move and free pages (kvq_pages_*).  Works on the cache's block table."""

    def __init__(self, cache: KVCache, refs=None, stream=None):
        import torch

        cache._check_table()
        self.cache, self.index = cache, cache.index
        self.ws_bytes = kvq_pages_workspace_bytes(cache.cfg)
        with _on(stream):
            self.workspace = torch.empty(self.ws_bytes, dtype=torch.uint8, device=cache.device)
            self.refs = refs if refs is not None else torch.empty(cache.cfg.n_pages, dtype=torch.int32, device=cache.device)
        if self.refs.dtype != torch.int32 or self.refs.numel() != cache.cfg.n_pages or not self.refs.is_contiguous():
            raise ValueError("refs is a contiguous int32 tensor of n_pages")
        _here(self.index, self.refs)
        _check(LIB.kvq_pages_init(self._cfg(), _ptr(cache.block_table), _ptr(self.refs), *self._ws(stream)))

    def _cfg(self):
        return ctypes.byref(self.cache.c_cfg)

    def _ws(self, stream):
        return _ptr(self.workspace), self.ws_bytes, _stream(stream)

    def _lists(self, seq_lens, *lists):
        import torch

        for t in (seq_lens, *lists):
            if t.dtype != torch.int32 or not t.is_contiguous():
                raise ValueError("lengths and lists are contiguous int32 tensors")
        if seq_lens.numel() != self.cache.cfg.batch or len({t.numel() for t in lists}) != 1:
            raise ValueError("seq_lens is [batch]; lists have one length")
        _here(self.index, seq_lens, *lists)

    def release(self, seqs, seq_lens, stream=None):
        """Frees the listed sequences."""
        self._lists(seq_lens, seqs)
        _check(LIB.kvq_pages_release(self._cfg(), _ptr(self.cache.block_table), _ptr(self.refs), _ptr(seq_lens),
                                     _ptr(seqs), seqs.numel(), *self._ws(stream)))

    def fork(self, src, dst, seq_lens, stream=None):
        """Sequence dst[i] becomes a copy of src[i] that shares its pages."""
        self._lists(seq_lens, src, dst)
        _check(LIB.kvq_pages_fork(self._cfg(), ctypes.byref(self.cache.c_cache), _ptr(self.cache.block_table),
                                  _ptr(self.refs), _ptr(seq_lens), _ptr(src), _ptr(dst), src.numel(),
                                  *self._ws(stream)))

    def reserve(self, seqs, n_new, seq_lens, stream=None):
        """Pages for n_new[i] more tokens of seqs[i], and its own copy of a partly filled shared page."""
        self._lists(seq_lens, seqs, n_new)
        _check(LIB.kvq_pages_reserve(self._cfg(), ctypes.byref(self.cache.c_cache), _ptr(self.cache.block_table),
                                     _ptr(self.refs), _ptr(seq_lens), _ptr(seqs), _ptr(n_new), seqs.numel(),
                                     *self._ws(stream)))

    def compact(self, refs_out=None, table_out=None, stream=None):
        """Moves the used pages together.  Without outputs the cache's table and the counts are changed in place.  With
        them the pages have moved all the same, and nothing may use the cache until the caller has copied table_out into
        its block table and refs_out into the counts."""
        import torch

        table = self.cache.block_table
        for t, like in ((refs_out, self.refs), (table_out, table)):
            if t is not None and (t.dtype != torch.int32 or t.numel() != like.numel() or not t.is_contiguous()):
                raise ValueError("outputs are contiguous int32 tensors like the inputs")
        _here(self.index, refs_out, table_out)
        _check(LIB.kvq_pages_compact(self._cfg(), ctypes.byref(self.cache.c_cache), _ptr(table), _ptr(self.refs),
                                     _ptr(table if table_out is None else table_out),
                                     _ptr(self.refs if refs_out is None else refs_out), *self._ws(stream)))

    def device_status(self, stream=None) -> int:
        out = ctypes.c_uint32()
        _check(LIB.kvq_read_device_status(_ptr(self.workspace), ctypes.byref(out), _stream(stream)))
        return out.value

    def clear_status(self, stream=None):
        _check(LIB.kvq_clear_device_status(_ptr(self.workspace), _stream(stream)))
