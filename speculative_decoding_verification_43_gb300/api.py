"""Python binding of the C ABI: argument marshalling only.

Every step of the verifier runs in the CUDA kernels of libspecverify.so. PyTorch supplies
device memory and the stream; this module fills the C structs with tensor pointers, allocates
output tensors on request, and raises when a call returns an error status.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch

from . import _lib
from ._lib import SpecAttendArgs, SpecCompactArgs, SpecKvAppendArgs, SpecVerifyArgs, check, lib

_DTYPE = {torch.float32: _lib.SPEC_F32, torch.bfloat16: _lib.SPEC_BF16}


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_handle(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _run_stream(obj, stream):
    """Handle of the stream a prepared call runs on (None: the current one). The caching allocator takes a tensor
    to be in use on the stream it was allocated on; where the call's outputs and workspace are used on another, it
    is told, once for each stream, so that it gives their memory to nobody while the kernels are at work."""
    if stream is None:
        stream = torch.cuda.current_stream()
    handle = stream.cuda_stream
    if handle not in obj._streams:
        for t in (*vars(obj.out).values(), getattr(obj, "workspace", None)):
            if t is not None:
                t.record_stream(stream)
        obj._streams.add(handle)
    return ctypes.c_void_p(handle)


def _hand_over(out, stream):
    """Outputs that were allocated and written on `stream` (None: the current one), for the current stream."""
    if stream is not None:
        here = torch.cuda.current_stream()
        if here.cuda_stream != stream.cuda_stream:
            for t in out if isinstance(out, tuple) else vars(out).values():
                if t is not None:
                    t.record_stream(here)
    return out


def _choice(dev, stream):
    """Outputs of a gamma choice on `stream`: int32[1], float64[1]."""
    with torch.cuda.stream(stream):
        out = torch.empty(1, dtype=torch.int32, device=dev), torch.empty(1, dtype=torch.float64, device=dev)
    return _hand_over(out, stream)


def _i32(t):
    assert t.dtype == torch.int32 and t.is_contiguous() and t.is_cuda, "int32 CUDA tensor expected"
    return t


def workspace_size(B: int, V: int, total_rows: int, dtype: torch.dtype) -> int:
    return int(lib.spec_verify_workspace_size(B, V, total_rows, _DTYPE[dtype]))


def verify_plan(B: int, V: int, total_rows: int, dtype: torch.dtype):
    """(kernel name, CTAs per cluster, CTAs) that spec_verify launches for this shape on the
    current device, or None when the device cannot host it (or the shape is invalid)."""
    c, n = ctypes.c_int32(0), ctypes.c_int32(0)
    name = lib.spec_verify_plan(B, V, total_rows, _DTYPE[dtype], ctypes.byref(c), ctypes.byref(n))
    return None if name is None else (name.decode(), c.value, n.value)


@dataclass
class VerifyOutputs:
    accept_len: torch.Tensor
    n_emitted: torch.Tensor
    out_tokens: torch.Tensor
    req_status: torch.Tensor
    alpha_rows: torch.Tensor
    alpha_sum: torch.Tensor
    alpha_count: torch.Tensor
    rho_rows: torch.Tensor | None = None
    resid_rows: torch.Tensor | None = None
    frontier_prob: torch.Tensor | None = None
    frontier_margin: torch.Tensor | None = None
    fallback: torch.Tensor | None = None
    depth_reached: torch.Tensor | None = None   # [K_max] requests that reached depth j
    depth_accepted: torch.Tensor | None = None  # [K_max] requests that accepted depth j


class Verifier:
    """A prepared spec_verify call for one batch shape.

    Holds the C struct, the workspace and the output tensors, so that repeated rounds on the
    same buffers cost one ctypes call each. Inputs are bound with ``bind``; ``run`` enqueues
    the verifier's kernel on the given (or current) stream and returns without synchronising.
    The workspace is zero-filled once, here: every call leaves it ready for the next one.
    """

    def __init__(self, B: int, V: int, total_rows: int, dtype: torch.dtype, *, K_max: int = 64,
                 device=None, diagnostics: bool = False):
        device = torch.device(device or "cuda")
        self.B, self.V, self.T, self.dtype, self.K_max = B, V, total_rows, dtype, K_max
        nd = max(total_rows - B, 1)
        i32 = dict(dtype=torch.int32, device=device)
        f32 = dict(dtype=torch.float32, device=device)
        self.out = VerifyOutputs(
            accept_len=torch.empty(B, **i32), n_emitted=torch.empty(B, **i32),
            out_tokens=torch.empty(total_rows, **i32), req_status=torch.empty(B, **i32),
            alpha_rows=torch.empty(nd, **f32),
            alpha_sum=torch.empty(1, dtype=torch.float64, device=device),
            alpha_count=torch.empty(1, **i32),
            depth_reached=torch.empty(max(K_max, 1), **i32), depth_accepted=torch.empty(max(K_max, 1), **i32))
        if diagnostics:
            self.out.rho_rows = torch.empty(nd, **f32)
            self.out.resid_rows = torch.empty(nd, **f32)
            self.out.frontier_prob = torch.empty(B, **f32)
            self.out.frontier_margin = torch.empty(B, **f32)
            self.out.fallback = torch.empty(B, **i32)
        self.ws_bytes = workspace_size(B, V, total_rows, dtype)
        # 256-byte aligned (the caching allocator hands out 512-byte aligned blocks) and zeroed
        self.workspace = torch.zeros(self.ws_bytes, dtype=torch.uint8, device=device)
        self.args = SpecVerifyArgs()
        a = self.args
        a.B, a.V, a.K_max, a.total_rows, a.dtype = B, V, K_max, total_rows, _DTYPE[dtype]
        o = self.out
        for name in ("accept_len", "n_emitted", "out_tokens", "req_status", "alpha_rows", "alpha_sum",
                     "alpha_count", "rho_rows", "resid_rows", "frontier_prob", "frontier_margin",
                     "fallback", "depth_reached", "depth_accepted"):
            setattr(a, name, _ptr(getattr(o, name)))
        self._streams, self._keep = set(), ()

    def bind(self, target, draft, row_off, draft_tokens, uniforms, temperature=1.0, *,
             stop_token=None, max_new=None, top_k=None, top_p=None):
        B, V, T = self.B, self.V, self.T
        assert target.dtype == self.dtype and target.is_cuda and target.is_contiguous()
        assert target.shape == (T, V), (target.shape, (T, V))
        if T > B:
            assert draft is not None and draft.dtype == self.dtype and draft.is_contiguous()
            assert draft.shape == (T - B, V)
            _i32(draft_tokens)
        _i32(row_off)
        assert row_off.shape == (B + 1,)
        assert uniforms.dtype == torch.float64 and uniforms.is_cuda and uniforms.numel() >= T
        a = self.args
        a.target_logits = _ptr(target)
        a.draft_logits = _ptr(draft) if T > B else None
        a.row_off = _ptr(row_off)
        a.draft_tokens = _ptr(draft_tokens) if T > B else None
        a.uniforms = _ptr(uniforms)
        if isinstance(temperature, torch.Tensor):
            assert temperature.dtype == torch.float32 and temperature.is_cuda and temperature.numel() == B
            a.temperature = _ptr(temperature)
            a.temperature_scalar = 1.0
        else:
            a.temperature = None
            a.temperature_scalar = float(temperature)
        a.stop_token = _ptr(_i32(stop_token)) if stop_token is not None else None
        a.max_new = _ptr(_i32(max_new)) if max_new is not None else None
        # top-k / top-p of the target law, per request (None: no truncation)
        if top_p is not None:
            assert top_p.dtype == torch.float32 and top_p.is_cuda and top_p.numel() == B
        a.top_k = _ptr(_i32(top_k)) if top_k is not None else None
        a.top_p = _ptr(top_p) if top_p is not None else None
        self._keep = (target, draft, row_off, draft_tokens, uniforms, temperature, stop_token, max_new,
                      top_k, top_p)
        return self

    def time_rows_with(self, begin, end, stats_end=None):
        """On each following run, record torch.cuda.Event `begin` before the verifier's first
        kernel, `end` after its last and `stats_end` after the statistics kernel (each may be
        None; all None: stop)."""
        ev = lambda e: ctypes.c_void_p(e.cuda_event) if e is not None else None  # noqa: E731
        self.args.rows_event_begin = ev(begin)
        self.args.rows_event_end = ev(end)
        self.args.stats_event_end = ev(stats_end)
        self._events = (begin, end, stats_end)

    def run(self, stream=None) -> VerifyOutputs:
        rc = lib.spec_verify(ctypes.byref(self.args), ctypes.c_void_p(self.workspace.data_ptr()),
                             self.ws_bytes, _run_stream(self, stream))
        check(rc, "spec_verify")
        return self.out


def verify(target, draft, row_off, draft_tokens, uniforms, temperature=1.0, *, K_max: int = 64,
           stop_token=None, max_new=None, top_k=None, top_p=None, diagnostics: bool = False,
           stream=None) -> VerifyOutputs:
    """One verifier round on device tensors (see include/spec_verify.h for the layout). With a stream, workspace
    and outputs are allocated and written there; who uses the outputs elsewhere waits for it first."""
    T, V = target.shape
    B = row_off.numel() - 1
    with torch.cuda.stream(stream):
        v = Verifier(B, V, T, target.dtype, K_max=K_max, device=target.device, diagnostics=diagnostics)
        v.bind(target, draft, row_off, draft_tokens, uniforms, temperature, stop_token=stop_token,
               max_new=max_new, top_k=top_k, top_p=top_p)
        out = v.run(stream)
    return _hand_over(out, stream)


@dataclass
class CompactOutputs:
    out_off: torch.Tensor
    packed_tokens: torch.Tensor
    packed_pos: torch.Tensor
    kv_off: torch.Tensor
    kv_src: torch.Tensor
    kv_dst: torch.Tensor
    new_seq_len: torch.Tensor
    new_kv_len: torch.Tensor
    new_draft_len: torch.Tensor
    compact_status: torch.Tensor


class Compactor:
    """A prepared spec_compact call for one batch shape."""

    def __init__(self, B: int, total_rows: int, device=None):
        device = torch.device(device or "cuda")
        i32 = dict(dtype=torch.int32, device=device)
        nd = max(total_rows - B, 1)
        self.B, self.T = B, total_rows
        self.out = CompactOutputs(
            out_off=torch.empty(B + 1, **i32), packed_tokens=torch.empty(total_rows, **i32),
            packed_pos=torch.empty(total_rows, **i32), kv_off=torch.empty(B + 1, **i32),
            kv_src=torch.empty(nd, **i32), kv_dst=torch.empty(nd, **i32),
            new_seq_len=torch.empty(B, **i32), new_kv_len=torch.empty(B, **i32),
            new_draft_len=torch.empty(B, **i32), compact_status=torch.empty(B, **i32))
        self.args = SpecCompactArgs()
        a = self.args
        a.B, a.total_rows = B, total_rows
        for name in ("out_off", "packed_tokens", "packed_pos", "kv_off", "kv_src", "kv_dst",
                     "new_seq_len", "new_kv_len", "new_draft_len", "compact_status"):
            setattr(a, name, _ptr(getattr(self.out, name)))
        self._streams, self._keep = set(), ()

    def bind(self, row_off, accept_len, n_emitted, out_tokens, req_status, prefix_len, cand_kv_rows,
             block_table, page_size: int):
        a = self.args
        assert block_table.dim() == 2 and block_table.shape[0] == self.B
        a.page_size = int(page_size)
        a.max_blocks = int(block_table.shape[1])
        for name, t in (("row_off", row_off), ("accept_len", accept_len), ("n_emitted", n_emitted),
                        ("out_tokens", out_tokens), ("req_status", req_status),
                        ("prefix_len", prefix_len), ("cand_kv_rows", cand_kv_rows),
                        ("block_table", block_table)):
            setattr(a, name, _ptr(_i32(t)) if t is not None else None)
        self._keep = (row_off, accept_len, n_emitted, out_tokens, req_status, prefix_len,
                      cand_kv_rows, block_table)
        return self

    def run(self, stream=None) -> CompactOutputs:
        check(lib.spec_compact(ctypes.byref(self.args), _run_stream(self, stream)), "spec_compact")
        return self.out


def compact(row_off, accept_len, n_emitted, out_tokens, req_status, prefix_len, cand_kv_rows,
            block_table, page_size: int, stream=None) -> CompactOutputs:
    with torch.cuda.stream(stream):
        c = Compactor(row_off.numel() - 1, out_tokens.numel(), device=out_tokens.device)
        c.bind(row_off, accept_len, n_emitted, out_tokens, req_status, prefix_len, cand_kv_rows,
               block_table, page_size)
        out = c.run(stream)
    return _hand_over(out, stream)


def run_round(verifier: "Verifier", compactor: "Compactor", alpha_prev: float, c: float, gamma_min: int = 0,
              gamma_max: int = 8, *, out=None, stream=None):
    """One round through spec_verify_round: the bound verifier, the bound compactor and the gamma
    choice in one call (the same results as verifier.run(), compactor.run() and choose_gamma()).
    Returns (verify outputs, compaction outputs, (gamma int32[1], alpha float64[1]))."""
    dev = verifier.out.alpha_sum.device
    if out is None:
        out = _choice(dev, stream)
    g, a = out
    _run_stream(compactor, stream)
    rc = lib.spec_verify_round(ctypes.byref(verifier.args), ctypes.c_void_p(verifier.workspace.data_ptr()),
                               verifier.ws_bytes, ctypes.byref(compactor.args), float(alpha_prev), float(c),
                               int(gamma_min), int(gamma_max), _ptr(g), _ptr(a), _run_stream(verifier, stream))
    check(rc, "spec_verify_round")
    return verifier.out, compactor.out, (g, a)


def choose_gamma(alpha_sum, alpha_count, alpha_prev: float, c: float, gamma_min: int = 0,
                 gamma_max: int = 8, *, out=None, stream=None):
    """Device-side gamma choice; returns (gamma int32[1], alpha float64[1]) device tensors."""
    dev = alpha_sum.device
    if out is None:
        out = _choice(dev, stream)
    g, a = out
    rc = lib.spec_choose_gamma(_ptr(alpha_sum), _ptr(alpha_count), float(alpha_prev), float(c),
                               int(gamma_min), int(gamma_max), _ptr(g), _ptr(a), _stream_handle(stream))
    check(rc, "spec_choose_gamma")
    return g, a


def choose_gamma_depth(depth_reached, depth_accepted, alpha_prev: float, c: float, gamma_min: int = 0,
                       gamma_max: int = 8, *, out=None, stream=None):
    """Device-side gamma choice from per-depth counts (as spec_verify writes them); returns
    (gamma int32[1], E[A] float64[1]) device tensors."""
    dev = depth_reached.device
    _i32(depth_reached)
    _i32(depth_accepted)
    assert depth_reached.numel() == depth_accepted.numel()
    if out is None:
        out = _choice(dev, stream)
    g, ea = out
    rc = lib.spec_choose_gamma_depth(_ptr(depth_reached), _ptr(depth_accepted), int(depth_reached.numel()),
                                     float(alpha_prev), float(c), int(gamma_min), int(gamma_max), _ptr(g),
                                     _ptr(ea), _stream_handle(stream))
    check(rc, "spec_choose_gamma_depth")
    return g, ea


def depth_objective(n_reached, n_accepted, alpha_prev: float, c: float, gamma: int) -> float:
    """Host evaluation (double) of the depth-aware objective from host integer arrays."""
    import numpy as np
    nr = np.ascontiguousarray(n_reached, np.int32)
    na = np.ascontiguousarray(n_accepted, np.int32)
    assert nr.shape == na.shape
    return float(lib.spec_depth_objective(nr.ctypes.data_as(ctypes.c_void_p), na.ctypes.data_as(ctypes.c_void_p),
                                          int(nr.size), float(alpha_prev), float(c), int(gamma)))


def _rows_of(t, T: int, heads: int, D: int, dtype):
    """Pointer and row stride (elements) of [T][heads][D] rows whose heads are contiguous."""
    assert t.dtype == dtype and t.is_cuda and t.shape == (T, heads, D), (t.dtype, t.shape, (T, heads, D))
    assert (D == 1 or t.stride(2) == 1) and (heads == 1 or t.stride(1) == D), "a row's heads must be contiguous"
    return _ptr(t), (t.stride(0) if T > 1 else heads * D)


def _bind_cache(a, k_cache, v_cache, Hkv: int, D: int, dtype):
    """The paged cache as [n_pages, page_size, Hkv, D] tensors of any strides (elements of a head
    contiguous), the same for keys and values."""
    assert k_cache.dtype == dtype and v_cache.dtype == dtype and k_cache.is_cuda and v_cache.is_cuda
    assert k_cache.dim() == 4 and k_cache.shape[2:] == (Hkv, D), (k_cache.shape, (Hkv, D))
    assert k_cache.shape == v_cache.shape and k_cache.stride() == v_cache.stride(), "keys and values alike"
    assert D == 1 or k_cache.stride(3) == 1
    a.n_pages, a.page_size = int(k_cache.shape[0]), int(k_cache.shape[1])
    a.page_stride, a.slot_stride, a.head_stride = k_cache.stride()[:3]
    a.k_cache, a.v_cache = _ptr(k_cache), _ptr(v_cache)


def _bind_requests(a, B: int, row_off, kv_len, block_table):
    assert _i32(row_off).shape == (B + 1,) and _i32(kv_len).shape == (B,)
    assert _i32(block_table).dim() == 2 and block_table.shape[0] == B
    a.row_off, a.kv_len, a.block_table = _ptr(row_off), _ptr(kv_len), _ptr(block_table)
    a.max_blocks = int(block_table.shape[1])


@dataclass
class AppendOutputs:
    q: torch.Tensor           # [T, Hq, D] rotated queries
    req_status: torch.Tensor


class KvAppender:
    """A prepared spec_kv_append call for one batch shape: a round's keys (rotated) and values go to
    the paged cache, its queries (rotated) to ``out.q``. rot_dim None rotates whole heads."""

    def __init__(self, B: int, total_rows: int, Hq: int, Hkv: int, D: int, dtype: torch.dtype, *,
                 rot_dim: int | None = None, interleaved: bool = False, device=None):
        device = torch.device(device or "cuda")
        self.B, self.T, self.Hq, self.Hkv, self.D, self.dtype = B, total_rows, Hq, Hkv, D, dtype
        self.out = AppendOutputs(q=torch.empty(total_rows, Hq, D, dtype=dtype, device=device),
                                 req_status=torch.empty(B, dtype=torch.int32, device=device))
        self._streams = set()
        self.args = SpecKvAppendArgs()
        a = self.args
        a.B, a.total_rows, a.n_q_heads, a.n_kv_heads, a.head_dim = B, total_rows, Hq, Hkv, D
        a.rot_dim, a.interleaved, a.dtype = D if rot_dim is None else rot_dim, int(interleaved), _DTYPE[dtype]
        a.req_status = _ptr(self.out.req_status)
        self._keep = ()

    def bind(self, q, k, v, cos_sin, row_off, kv_len, k_cache, v_cache, block_table, *, q_out=None):
        """q [T, Hq, D], k and v [T, Hkv, D] (slices of one projection are fine), cos_sin
        [n_pos, rot_dim] float32 (cosines, then sines), k_cache and v_cache [n_pages, page_size, Hkv,
        D], block_table [B, max_blocks]. q_out may be q itself."""
        a, T, D = self.args, self.T, self.D
        if q_out is not None:
            self.out.q = q_out
        if self.Hq:
            a.q, a.q_stride = _rows_of(q, T, self.Hq, D, self.dtype)
            a.q_out, a.q_out_stride = _rows_of(self.out.q, T, self.Hq, D, self.dtype)
        a.k, a.k_stride = _rows_of(k, T, self.Hkv, D, self.dtype)
        a.v, a.v_stride = _rows_of(v, T, self.Hkv, D, self.dtype)
        if a.rot_dim:
            assert cos_sin.dtype == torch.float32 and cos_sin.is_cuda and cos_sin.is_contiguous()
            assert cos_sin.dim() == 2 and cos_sin.shape[1] == a.rot_dim, (cos_sin.shape, a.rot_dim)
            a.cos_sin, a.n_pos = _ptr(cos_sin), int(cos_sin.shape[0])
        _bind_cache(a, k_cache, v_cache, self.Hkv, D, self.dtype)
        _bind_requests(a, self.B, row_off, kv_len, block_table)
        self._keep = (q, k, v, cos_sin, row_off, kv_len, k_cache, v_cache, block_table, q_out)
        return self

    def run(self, stream=None) -> AppendOutputs:
        check(lib.spec_kv_append(ctypes.byref(self.args), _run_stream(self, stream)), "spec_kv_append")
        return self.out


def kv_append(q, k, v, cos_sin, row_off, kv_len, k_cache, v_cache, block_table, *, rot_dim: int | None = None,
              interleaved: bool = False, q_out=None, stream=None) -> AppendOutputs:
    """Appends a round's rows to the paged cache (see include/spec_attend.h). With a stream, the outputs are
    allocated and written there; who uses them elsewhere waits for it first."""
    T, Hkv, D = k.shape
    with torch.cuda.stream(stream):
        c = KvAppender(row_off.numel() - 1, T, q.shape[1] if q is not None else 0, Hkv, D, k.dtype, rot_dim=rot_dim,
                       interleaved=interleaved, device=k.device)
        c.bind(q, k, v, cos_sin, row_off, kv_len, k_cache, v_cache, block_table, q_out=q_out)
        out = c.run(stream)
    return _hand_over(out, stream)


@dataclass
class AttendOutputs:
    out: torch.Tensor         # [T, Hq, D]
    lse: torch.Tensor         # [T, Hq] float32, natural logarithm
    req_status: torch.Tensor


class Attention:
    """A prepared spec_attend call for one batch shape: attention of the round's rows over the paged
    cache. window 0: every earlier position; n_sink first positions stay visible behind a window;
    the first shared_len positions of all requests lie in the pages of the shared table."""

    def __init__(self, B: int, total_rows: int, Hq: int, Hkv: int, D: int, dtype: torch.dtype, *, window: int = 0,
                 n_sink: int = 0, shared_len: int = 0, scale: float | None = None, device=None):
        self.device = torch.device(device or "cuda")
        self.B, self.T, self.Hq, self.Hkv, self.D, self.dtype = B, total_rows, Hq, Hkv, D, dtype
        self.out = AttendOutputs(out=torch.empty(total_rows, Hq, D, dtype=dtype, device=self.device),
                                 lse=torch.empty(total_rows, Hq, dtype=torch.float32, device=self.device),
                                 req_status=torch.empty(B, dtype=torch.int32, device=self.device))
        self.args = SpecAttendArgs()
        a = self.args
        a.B, a.total_rows, a.n_q_heads, a.n_kv_heads, a.head_dim = B, total_rows, Hq, Hkv, D
        a.window, a.n_sink, a.shared_len, a.dtype = window, n_sink, shared_len, _DTYPE[dtype]
        a.scale = D ** -0.5 if scale is None else scale
        a.lse, a.req_status = _ptr(self.out.lse), _ptr(self.out.req_status)
        self.workspace, self.ws_bytes = None, 0
        self._streams, self._keep = set(), ()

    def bind(self, q, k_cache, v_cache, row_off, kv_len, block_table, *, shared_table=None, out=None):
        """q [T, Hq, D], k_cache and v_cache [n_pages, page_size, Hkv, D] of any strides, block_table
        [B, max_blocks], shared_table [ceil(shared_len / page_size)]."""
        a = self.args
        if out is not None:
            self.out.out = out
        a.q, a.q_stride = _rows_of(q, self.T, self.Hq, self.D, self.dtype)
        a.out, a.out_stride = _rows_of(self.out.out, self.T, self.Hq, self.D, self.dtype)
        _bind_cache(a, k_cache, v_cache, self.Hkv, self.D, self.dtype)
        _bind_requests(a, self.B, row_off, kv_len, block_table)
        if a.shared_len:
            assert _i32(shared_table).numel() * a.page_size >= a.shared_len
        a.shared_table = _ptr(shared_table)
        self.ws_bytes = int(lib.spec_attend_workspace_size(ctypes.byref(a)))
        if self.workspace is None or self.workspace.numel() < self.ws_bytes:
            self.workspace = torch.empty(max(self.ws_bytes, 256), dtype=torch.uint8, device=self.device)
            self._streams = set()
        self._keep = (q, k_cache, v_cache, row_off, kv_len, block_table, shared_table, out)
        return self

    def plan(self) -> str | None:
        """The kernel that serves the bound call's own positions, or None when its sizes are invalid."""
        name = lib.spec_attend_plan(ctypes.byref(self.args))
        return None if name is None else name.decode()

    def run(self, stream=None) -> AttendOutputs:
        rc = lib.spec_attend(ctypes.byref(self.args), ctypes.c_void_p(self.workspace.data_ptr()),
                             self.workspace.numel(), _run_stream(self, stream))
        check(rc, "spec_attend")
        return self.out


def attend(q, k_cache, v_cache, row_off, kv_len, block_table, *, window: int = 0, n_sink: int = 0,
           shared_len: int = 0, shared_table=None, scale: float | None = None, stream=None) -> AttendOutputs:
    """Attention of a round's rows over the paged cache (see include/spec_attend.h). With a stream, workspace and
    outputs are allocated and written there; who uses the outputs elsewhere waits for it first."""
    T, Hq, D = q.shape
    with torch.cuda.stream(stream):
        a = Attention(row_off.numel() - 1, T, Hq, k_cache.shape[2], D, q.dtype, window=window, n_sink=n_sink,
                      shared_len=shared_len, scale=scale, device=q.device)
        a.bind(q, k_cache, v_cache, row_off, kv_len, block_table, shared_table=shared_table)
        out = a.run(stream)
    return _hand_over(out, stream)


def gamma_objective(alpha: float, c: float, gamma: int) -> float:
    return float(lib.spec_gamma_objective(float(alpha), float(c), int(gamma)))


def version() -> str:
    return lib.spec_version().decode()
