"""kv_cache_analyzer_b200 -- Python binding of libjano, the B200 (sm_100a)
library for the data-parallel hot path of Jano (block-wise complexity
analyzer, three-level token schedule, KV-cache scatter and active-query
attention).

The functions named ``jano_*`` mirror the C ABI in ``include/jano.h`` one to
one: they only marshal torch tensors (device memory) and the current CUDA
stream into the C call and turn a non-OK status into ``JanoError``.  The
lower-case helpers below them allocate outputs with torch and call those.
Every step of the path runs in the library's CUDA kernels; there is no CPU
or PyTorch fallback, and importing a function fails loudly when the library
is not built.
"""
from __future__ import annotations

import ctypes as C
import os
import struct
from dataclasses import dataclass

import torch

__all__ = [
    "JanoError", "jano_geom", "jano_sched_cfg", "lib", "library_path",
    "jano_block_scores", "jano_classify", "jano_build_schedule_workspace_bytes",
    "jano_build_schedule", "jano_build_schedule_noalloc", "jano_kv_scatter", "jano_active_attention",
    "jano_active_attention_split", "jano_active_attention_workspace_bytes", "jano_active_attention_splits",
    "jano_active_attention_splits_on", "jano_get_device_error", "jano_status_str", "jano_version",
    "Geometry", "Schedule", "block_scores", "classify", "build_schedule",
    "kv_scatter", "active_attention", "device_error",
    "jano_rope_cfg", "jano_page_pool", "jano_page_seqs", "jano_rope_table_floats", "jano_rope_table",
    "jano_axis_rope", "jano_rope_scatter", "jano_paged_append", "jano_paged_attention",
    "jano_paged_attention_splits_on", "Rope", "rope_table", "axis_rope", "rope_scatter", "page_pool",
    "paged_append", "paged_attention",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
# JANO_LIBRARY may point at another build of the same library (e.g. a
# variant compiled with different tuning macros).
library_path = os.environ.get("JANO_LIBRARY") or os.path.join(_HERE, "libjano.so")

STATUS_NAMES = {0: "JANO_OK", 1: "JANO_EINVAL", 2: "JANO_ESHAPE", 3: "JANO_EALIGN",
                4: "JANO_EUNSUPPORTED", 5: "JANO_ENONFINITE", 6: "JANO_EINDEX",
                7: "JANO_ETIMEOUT", 8: "JANO_ECUDA"}
EXPORTS = ("jano_block_scores", "jano_block_scores_literal", "jano_classify", "jano_build_schedule_workspace_bytes",
           "jano_build_schedule", "jano_build_schedule_noalloc", "jano_kv_scatter", "jano_active_attention",
           "jano_active_attention_split", "jano_active_attention_workspace_bytes", "jano_active_attention_splits",
           "jano_active_attention_splits_on", "jano_gather_gemm", "jano_qkv_project", "jano_random_scores", "jano_fft_scores",
           "jano_stream_sum", "jano_rope_table_floats", "jano_rope_table", "jano_axis_rope", "jano_rope_scatter",
           "jano_paged_append", "jano_paged_attention", "jano_paged_attention_splits_on",
           "jano_get_device_error", "jano_status_str", "jano_version")


class JanoError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} failed: {STATUS_NAMES.get(code, code)}")
        self.code = code


class jano_geom(C.Structure):
    _fields_ = [(n, C.c_int) for n in ("F", "H", "W", "bf", "bh", "bw", "pf", "ph", "pw")]


class jano_sched_cfg(C.Structure):
    _fields_ = [(n, C.c_int) for n in ("T", "warmup", "cooldown", "period_moderate", "period_static")]


class jano_rope_cfg(C.Structure):
    _fields_ = [("axes", C.c_int * 3), ("n_pos", C.c_int * 3), ("grid_h", C.c_int), ("grid_w", C.c_int),
                ("halves", C.c_int)]


class jano_page_pool(C.Structure):
    _fields_ = [("k", C.c_void_p), ("v", C.c_void_p), ("n_pages", C.c_int), ("page_size", C.c_int),
                ("kv_heads", C.c_int), ("d", C.c_int), ("page_stride", C.c_longlong),
                ("token_stride", C.c_longlong), ("head_stride", C.c_longlong)]


class jano_page_seqs(C.Structure):
    _fields_ = [("page_table", C.c_void_p), ("seq_lens", C.c_void_p), ("cu_rows", C.c_void_p),
                ("n_seqs", C.c_int), ("max_pages", C.c_int)]


_lib = None


def lib() -> C.CDLL:
    """Load libjano.so (built in-tree by ``python -m kv_cache_analyzer_b200.build``)."""
    global _lib
    if _lib is None:
        if not os.path.exists(library_path):
            raise RuntimeError(f"libjano.so is not built at {library_path}; "
                               "run `python -m kv_cache_analyzer_b200.build`")
        L = C.CDLL(library_path)
        P, i, f, z = C.c_void_p, C.c_int, C.c_float, C.c_size_t
        G, S = C.POINTER(jano_geom), C.POINTER(jano_sched_cfg)
        L.jano_block_scores.argtypes = [P, i, i, G, f, f, P, P]
        L.jano_block_scores_literal.argtypes = [P, i, i, G, f, f, P, P]
        L.jano_classify.argtypes = [P, i, f, f, P, P]
        L.jano_build_schedule_workspace_bytes.argtypes = [G]
        L.jano_build_schedule_workspace_bytes.restype = z
        L.jano_build_schedule.argtypes = [P, G, S, P, P, z, P, P, z, P]
        L.jano_build_schedule_noalloc.argtypes = [P, G, S, P, P, z, P, P]
        L.jano_kv_scatter.argtypes = [P, P, P, i, i, i, P, P, i, P]
        L.jano_active_attention.argtypes = [P, P, P, P, i, i, i, i, f, P, P]
        L.jano_active_attention_split.argtypes = [P, P, P, P, i, i, i, i, f, i, P, z, P, P]
        L.jano_active_attention_workspace_bytes.argtypes = [i, i, i, i]
        L.jano_active_attention_workspace_bytes.restype = z
        L.jano_active_attention_splits.argtypes = [i, i, i, i]
        L.jano_active_attention_splits.restype = C.c_int
        L.jano_active_attention_splits_on.argtypes = [i, i, i, i, i]
        L.jano_active_attention_splits_on.restype = C.c_int
        L.jano_gather_gemm.argtypes = [P, i, P, i, P, i, i, P, P, i, P]
        L.jano_qkv_project.argtypes = [P, i, P, i, P, i, i, P, P, P, P]
        L.jano_random_scores.argtypes = [i, C.c_uint64, P, P]
        L.jano_fft_scores.argtypes = [P, i, G, i, P, P]
        L.jano_stream_sum.argtypes = [P, C.c_longlong, P, i, P]
        ll, R = C.c_longlong, C.POINTER(jano_rope_cfg)
        pool, seqs = C.POINTER(jano_page_pool), C.POINTER(jano_page_seqs)
        L.jano_rope_table_floats.argtypes = [R]
        L.jano_rope_table_floats.restype = z
        L.jano_rope_table.argtypes = [R, C.c_double, i, P, P]
        L.jano_axis_rope.argtypes = [P, ll, P, P, i, i, i, R, P, P, ll, P]
        L.jano_rope_scatter.argtypes = [P, ll, P, ll, P, ll, P, P, i, i, i, i, R, P, P, ll, P, P, i, P]
        L.jano_paged_append.argtypes = [pool, seqs, P, ll, P, ll, P, ll, P, P, P, i, i, R, P, P, ll, P]
        L.jano_paged_attention.argtypes = [pool, seqs, P, ll, P, i, i, i, i, f, i, P, ll, P]
        L.jano_paged_attention_splits_on.argtypes = [i, i, i, i, i, i, i]
        L.jano_get_device_error.argtypes = [P]
        L.jano_status_str.argtypes = [i]
        L.jano_status_str.restype = C.c_char_p
        L.jano_version.argtypes = []
        for fn in ("jano_block_scores", "jano_block_scores_literal", "jano_classify", "jano_build_schedule",
                   "jano_build_schedule_noalloc", "jano_kv_scatter", "jano_active_attention",
                   "jano_active_attention_split", "jano_get_device_error",
                   "jano_gather_gemm", "jano_qkv_project", "jano_random_scores", "jano_fft_scores",
                   "jano_stream_sum", "jano_rope_table", "jano_axis_rope", "jano_rope_scatter",
                   "jano_paged_append", "jano_paged_attention", "jano_paged_attention_splits_on",
                   "jano_version"):
            getattr(L, fn).restype = C.c_int
        _lib = L
    return _lib


def _torch_stream(stream):
    """The torch stream object for `stream` (None: the current stream; a raw
    cudaStream_t handle is wrapped), for allocator bookkeeping."""
    if stream is None:
        return torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return stream
    return torch.cuda.ExternalStream(int(stream))


def _stream(stream) -> int:
    """The cudaStream_t of a launch (None: the current stream; read as a raw
    handle, a stream object per call costs 3 us)."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _dev(t: torch.Tensor | None, name: str, dtype=None) -> int | None:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def _addr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


def _here(**tensors) -> None:
    """Every given tensor lies on the current CUDA device (the kernels are
    launched there)."""
    cur = None
    for name, t in tensors.items():
        if t is None:
            continue
        dev = t.get_device()                 # -1 on the CPU
        if dev == cur:
            continue
        if dev < 0:
            raise ValueError(f"{name} must be a CUDA tensor")
        if cur is None:
            cur = torch.cuda.current_device()
        if dev != cur:
            raise ValueError(f"{name} is on cuda:{dev}, the current device is cuda:{cur}")


def _rows(t: torch.Tensor, name: str, heads: int | None = None, d: int | None = None) -> int:
    """Row distance of a BF16 tensor [rows][heads][d] whose heads and columns
    are adjacent (rows may be slices of a wider buffer)."""
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be torch.bfloat16, got {t.dtype}")
    if t.dim() != 3:
        raise ValueError(f"{name} must be [rows][heads][d], got {tuple(t.shape)}")
    n, h, c = t.shape
    if (heads is not None and h != heads) or (d is not None and c != d):
        raise ValueError(f"{name} must be [rows][{heads}][{d}], got {tuple(t.shape)}")
    s0, s1, s2 = t.stride()
    if (c > 1 and s2 != 1) or (h > 1 and s1 != c):
        raise ValueError(f"the heads and columns of {name}'s rows must be adjacent")
    if n <= 1:
        return h * c if h * c % 8 == 0 else -(-h * c // 8) * 8
    return s0


def _count(t: torch.Tensor | None, name: str, n: int) -> None:
    if t is not None and t.numel() != n:
        raise ValueError(f"{name} must have {n} elements, got {t.numel()}")


def _on_stream(stream, shape, like: torch.Tensor) -> torch.Tensor:
    """A new tensor for a launch on `stream` (allocated there, so the memory's
    earlier uses are ordered before it)."""
    if stream is None:
        return like.new_empty(shape)
    with torch.cuda.stream(_torch_stream(stream)):
        return like.new_empty(shape)


def _check(fn: str, code: int) -> None:
    if code != 0:
        raise JanoError(fn, code)


# ---------------------------------------------------------------- C ABI mirror
def jano_block_scores(lat, K, C_, geom, w_temporal, w_spatial, scores, stream=None):
    _check("jano_block_scores", lib().jano_block_scores(
        _dev(lat, "lat", torch.float32), K, C_, C.byref(geom), w_temporal, w_spatial,
        _dev(scores, "scores", torch.float32), _stream(stream)))


def jano_block_scores_literal(lat, K, C_, geom, w_temporal, w_spatial, scores, stream=None):
    _check("jano_block_scores_literal", lib().jano_block_scores_literal(
        _dev(lat, "lat", torch.float32), K, C_, C.byref(geom), w_temporal, w_spatial,
        _dev(scores, "scores", torch.float32), _stream(stream)))


def jano_classify(scores, n_blocks, frac_active, frac_static, levels, stream=None):
    _check("jano_classify", lib().jano_classify(
        _dev(scores, "scores", torch.float32), n_blocks, frac_active, frac_static,
        _dev(levels, "levels", torch.uint8), _stream(stream)))


def jano_build_schedule_workspace_bytes(geom) -> int:
    return int(lib().jano_build_schedule_workspace_bytes(C.byref(geom)))


def jano_build_schedule(block_levels, geom, cfg, offsets, idx, idx_capacity, token_levels,
                        workspace, ws_bytes, stream=None):
    _check("jano_build_schedule", lib().jano_build_schedule(
        _dev(block_levels, "block_levels", torch.uint8), C.byref(geom), C.byref(cfg),
        _dev(offsets, "offsets", torch.int32), _dev(idx, "idx", torch.int32), idx_capacity,
        _dev(token_levels, "token_levels", torch.uint8), _dev(workspace, "workspace"),
        ws_bytes, _stream(stream)))


def jano_build_schedule_noalloc(block_levels, geom, cfg, offsets, idx, idx_capacity, token_levels,
                                stream=None):
    """jano_build_schedule without a workspace argument: for callers that
    cannot allocate device memory.  The library's own 1 MiB device array
    serves as scratch (geometries of at most 1,036,416 tokens); calls
    overlapping on the GPU race on it, and the first call on a device should
    come before any stream capture."""
    _check("jano_build_schedule_noalloc", lib().jano_build_schedule_noalloc(
        _dev(block_levels, "block_levels", torch.uint8), C.byref(geom), C.byref(cfg),
        _dev(offsets, "offsets", torch.int32), _dev(idx, "idx", torch.int32), idx_capacity,
        _dev(token_levels, "token_levels", torch.uint8), _stream(stream)))


def jano_kv_scatter(k_act, v_act, idx, n_act, heads, d, k_cache, v_cache, n_tokens, stream=None):
    _check("jano_kv_scatter", lib().jano_kv_scatter(
        _dev(k_act, "k_act", torch.bfloat16), _dev(v_act, "v_act", torch.bfloat16),
        _dev(idx, "idx", torch.int32), n_act, heads, d,
        _dev(k_cache, "k_cache", torch.bfloat16), _dev(v_cache, "v_cache", torch.bfloat16),
        n_tokens, _stream(stream)))


def jano_active_attention(q_act, k_cache, v_cache, idx, n_act, n_tokens, heads, d, scale, out,
                          stream=None):
    _check("jano_active_attention", lib().jano_active_attention(
        _dev(q_act, "q_act", torch.bfloat16), _dev(k_cache, "k_cache", torch.bfloat16),
        _dev(v_cache, "v_cache", torch.bfloat16), _dev(idx, "idx", torch.int32), n_act,
        n_tokens, heads, d, scale, _dev(out, "out", torch.bfloat16), _stream(stream)))


def jano_active_attention_split(q_act, k_cache, v_cache, idx, n_act, n_tokens, heads, d, scale,
                                n_split, workspace, ws_bytes, out, stream=None):
    _check("jano_active_attention_split", lib().jano_active_attention_split(
        _dev(q_act, "q_act", torch.bfloat16), _dev(k_cache, "k_cache", torch.bfloat16),
        _dev(v_cache, "v_cache", torch.bfloat16), _dev(idx, "idx", torch.int32), n_act,
        n_tokens, heads, d, scale, n_split, _dev(workspace, "workspace"), ws_bytes,
        _dev(out, "out", torch.bfloat16), _stream(stream)))


def jano_active_attention_workspace_bytes(n_act, heads, d, n_split) -> int:
    return int(lib().jano_active_attention_workspace_bytes(n_act, heads, d, n_split))


def jano_active_attention_splits(n_act, n_tokens, heads, d) -> int:
    return int(lib().jano_active_attention_splits(n_act, n_tokens, heads, d))


def jano_active_attention_splits_on(n_act, n_tokens, heads, d, sm_count) -> int:
    return int(lib().jano_active_attention_splits_on(n_act, n_tokens, heads, d, sm_count))


def jano_gather_gemm(x, n_x, gather, m, w, n, k, scatter, out, n_out, stream=None):
    _check("jano_gather_gemm", lib().jano_gather_gemm(
        _dev(x, "x", torch.bfloat16), n_x, _dev(gather, "gather", torch.int32), m,
        _dev(w, "w", torch.bfloat16), n, k, _dev(scatter, "scatter", torch.int32),
        _dev(out, "out", torch.bfloat16), n_out, _stream(stream)))


def jano_qkv_project(x, n_tokens, idx, n_act, w_qkv, hd, k, q_act, k_cache, v_cache, stream=None):
    _check("jano_qkv_project", lib().jano_qkv_project(
        _dev(x, "x", torch.bfloat16), n_tokens, _dev(idx, "idx", torch.int32), n_act,
        _dev(w_qkv, "w_qkv", torch.bfloat16), hd, k, _dev(q_act, "q_act", torch.bfloat16),
        _dev(k_cache, "k_cache", torch.bfloat16), _dev(v_cache, "v_cache", torch.bfloat16),
        _stream(stream)))


def jano_random_scores(n_blocks, seed, scores, stream=None):
    _check("jano_random_scores", lib().jano_random_scores(
        n_blocks, C.c_uint64(seed), _dev(scores, "scores", torch.float32), _stream(stream)))


def jano_fft_scores(x, C_, geom, cutoff, scores, stream=None):
    _check("jano_fft_scores", lib().jano_fft_scores(
        _dev(x, "x", torch.float32), C_, geom, cutoff, _dev(scores, "scores", torch.float32),
        _stream(stream)))


def jano_stream_sum(x, n, partial, n_partial, stream=None):
    _check("jano_stream_sum", lib().jano_stream_sum(
        _dev(x, "x", torch.float32), n, _dev(partial, "partial", torch.float32), n_partial,
        _stream(stream)))


def stream_sum(x: torch.Tensor, n_partial: int | None = None, out=None, stream=None) -> torch.Tensor:
    """Partial sums of one streaming pass over the fp32 tensor x (the read-rate
    calibration the analyzer is compared with); one CTA per SM by default."""
    if n_partial is None:
        n_partial = torch.cuda.get_device_properties(x.device).multi_processor_count
    if out is None:
        out = torch.empty(n_partial, dtype=torch.float32, device=x.device)
    jano_stream_sum(x, x.numel(), out, n_partial, stream)
    return out


def jano_rope_table_floats(cfg) -> int:
    return int(lib().jano_rope_table_floats(C.byref(cfg)))


def jano_rope_table(cfg, theta, shared_freq, table, stream=None):
    _check("jano_rope_table", lib().jano_rope_table(
        C.byref(cfg), theta, shared_freq, _dev(table, "table", torch.float32), _stream(stream)))


def jano_axis_rope(x, x_ld, ids, coords, n_rows, heads, d, cfg, table, out, out_ld, stream=None):
    """x and out as (device address, row distance) or tensors whose rows lie x_ld / out_ld elements apart."""
    _check("jano_axis_rope", lib().jano_axis_rope(
        _addr(x), x_ld, _dev(ids, "ids", torch.int32), _dev(coords, "coords", torch.int32), n_rows, heads, d,
        C.byref(cfg), _dev(table, "table", torch.float32), _addr(out), out_ld, _stream(stream)))


def jano_rope_scatter(q, q_ld, k, k_ld, v, v_ld, idx, coords, n_act, heads, kv_heads, d, cfg, table, q_out, q_out_ld,
                      k_cache, v_cache, n_tokens, stream=None):
    _check("jano_rope_scatter", lib().jano_rope_scatter(
        _addr(q), q_ld, _addr(k), k_ld, _addr(v), v_ld, _dev(idx, "idx", torch.int32),
        _dev(coords, "coords", torch.int32), n_act, heads, kv_heads, d, C.byref(cfg),
        _dev(table, "table", torch.float32), _addr(q_out), q_out_ld, _dev(k_cache, "k_cache", torch.bfloat16),
        _dev(v_cache, "v_cache", torch.bfloat16), n_tokens, _stream(stream)))


def jano_paged_append(pool, seqs, q, q_ld, k, k_ld, v, v_ld, pos, coords, grids, n_rows, heads, cfg, table, q_out,
                      q_out_ld, stream=None):
    _check("jano_paged_append", lib().jano_paged_append(
        C.byref(pool), C.byref(seqs), _addr(q), q_ld, _addr(k), k_ld, _addr(v), v_ld, _dev(pos, "pos", torch.int32),
        _dev(coords, "coords", torch.int32), _dev(grids, "grids", torch.int32), n_rows, heads,
        None if cfg is None else C.byref(cfg), _dev(table, "table", torch.float32), _addr(q_out), q_out_ld,
        _stream(stream)))


def jano_paged_attention(pool, seqs, q, q_ld, limits, n_rows, max_rows, max_len, heads, scale, n_split, out, out_ld,
                         stream=None):
    _check("jano_paged_attention", lib().jano_paged_attention(
        C.byref(pool), C.byref(seqs), _addr(q), q_ld, _dev(limits, "limits", torch.int32), n_rows, max_rows, max_len,
        heads, scale, n_split, _addr(out), out_ld, _stream(stream)))


def jano_paged_attention_splits_on(n_rows, max_rows, max_len, n_seqs, heads, kv_heads, sm_count) -> int:
    return int(lib().jano_paged_attention_splits_on(n_rows, max_rows, max_len, n_seqs, heads, kv_heads, sm_count))


def jano_get_device_error(stream=None) -> int:
    return int(lib().jano_get_device_error(_stream(stream)))


def jano_status_str(code: int) -> str:
    return lib().jano_status_str(code).decode()


def jano_version() -> int:
    return int(lib().jano_version())


# ---------------------------------------------------------------- helpers
@dataclass(frozen=True)
class Geometry:
    """Latent dims, analyzer block and token patch (latent elements)."""
    F: int
    H: int
    W: int
    block: tuple = (1, 4, 4)
    patch: tuple = (1, 2, 2)

    def c(self) -> jano_geom:
        return jano_geom(self.F, self.H, self.W, *self.block, *self.patch)

    @property
    def n_blocks(self) -> int:
        bf, bh, bw = self.block
        return (-(-self.F // bf)) * (-(-self.H // bh)) * (-(-self.W // bw))

    @property
    def n_tokens(self) -> int:
        pf, ph, pw = self.patch
        return (self.F // pf) * (self.H // ph) * (self.W // pw)


@dataclass(frozen=True)
class Schedule:
    T: int = 50
    warmup: int = 5
    cooldown: int = 5
    period_moderate: int = 2
    period_static: int = 4

    def c(self) -> jano_sched_cfg:
        return jano_sched_cfg(self.T, self.warmup, self.cooldown, self.period_moderate,
                              self.period_static)


def block_scores(lat: torch.Tensor, geom: Geometry, w_temporal=0.5, w_spatial=0.5,
                 out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    K1, Cc = lat.shape[0], lat.shape[1]
    if out is None:
        out = torch.empty(geom.n_blocks, dtype=torch.float32, device=lat.device)
    jano_block_scores(lat, K1 - 1, Cc, geom.c(), w_temporal, w_spatial, out, stream)
    return out


def block_scores_literal(lat: torch.Tensor, geom: Geometry, w_temporal=0.5, w_spatial=0.5,
                         out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The literal reading: second differences over the steps of the gradients."""
    K1, Cc = lat.shape[0], lat.shape[1]
    if out is None:
        out = torch.empty(geom.n_blocks, dtype=torch.float32, device=lat.device)
    jano_block_scores_literal(lat, K1 - 1, Cc, geom.c(), w_temporal, w_spatial, out, stream)
    return out


def classify(scores: torch.Tensor, frac_active: float, frac_static: float,
             out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    if out is None:
        out = torch.empty(scores.numel(), dtype=torch.uint8, device=scores.device)
    jano_classify(scores, scores.numel(), frac_active, frac_static, out, stream)
    return out


def build_schedule(block_levels: torch.Tensor, geom: Geometry, sched: Schedule,
                   stream=None, workspace: torch.Tensor | None = None):
    """-> (offsets int32 [T+1], idx int32 [T*N capacity], token_levels uint8 [N])."""
    dev = block_levels.device
    g = geom.c()
    N = geom.n_tokens
    ws_bytes = jano_build_schedule_workspace_bytes(g)
    if workspace is None:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    offsets = torch.empty(sched.T + 1, dtype=torch.int32, device=dev)
    idx = torch.empty(sched.T * N, dtype=torch.int32, device=dev)
    tl = torch.empty(N, dtype=torch.uint8, device=dev)
    jano_build_schedule(block_levels, g, sched.c(), offsets, idx, idx.numel(), tl, workspace,
                        workspace.numel(), stream)
    return offsets, idx, tl


def kv_scatter(k_act, v_act, idx, k_cache, v_cache, stream=None) -> None:
    n_act = idx.numel()
    N, H, d = k_cache.shape
    jano_kv_scatter(k_act, v_act, idx, n_act, H, d, k_cache, v_cache, N, stream)


def active_attention(q_act, k_cache, v_cache, idx, out, scale=None, stream=None, split=None,
                     workspace=None) -> None:
    """out[idx[i]] = attention of q_act[i] over the whole cache.  split: the
    number of key ranges per query tile (None: the library's choice for this
    shape on the current device, 1 for large due sets); with split > 1 the
    partials go to `workspace` (a device uint8 tensor of at least
    jano_active_attention_workspace_bytes bytes), allocated here if None."""
    n_act = idx.numel()
    N, H, d = k_cache.shape
    if scale is None:
        scale = d ** -0.5
    if split is None:
        split = jano_active_attention_splits(n_act, N, H, d) if n_act > 0 else 1
    if split <= 1:
        jano_active_attention(q_act, k_cache, v_cache, idx, n_act, N, H, d, scale, out, stream)
        return
    ws_bytes = jano_active_attention_workspace_bytes(n_act, H, d, split)
    temporary = workspace is None
    if temporary:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=k_cache.device)
    jano_active_attention_split(q_act, k_cache, v_cache, idx, n_act, N, H, d, scale, split,
                                workspace, workspace.numel() * workspace.element_size(), out, stream)
    if temporary:
        # freed on return: the allocator must not hand it out again before the
        # launch on `stream` has finished with it
        workspace.record_stream(_torch_stream(stream))


class SplitWorkspace:
    """Device workspaces of key-split attention, one per stream, each grown
    on demand.  Launches on one stream are ordered, so reusing that stream's
    buffer is safe; a launch on another stream gets a buffer of its own, so
    concurrent split launches never share partials."""

    def __init__(self, device):
        self.device = torch.device(device)
        self.bufs = {}

    def get(self, nbytes: int, stream) -> torch.Tensor:
        ts = _torch_stream(stream)
        key = int(ts.cuda_stream)
        buf = self.bufs.get(key)
        if buf is None or buf.numel() < nbytes:
            with torch.cuda.stream(ts):
                buf = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
            self.bufs[key] = buf
        return buf


def attention_auto(q_act, k_cache, v_cache, idx, n_act, n_tokens, heads, d, out, stream,
                   ws: SplitWorkspace) -> int:
    """jano_active_attention, or its key-split form when the library's choice
    for this shape on this device is a split (small due sets, few heads);
    returns the split count used."""
    split = jano_active_attention_splits(n_act, n_tokens, heads, d) if n_act > 0 else 1
    if split <= 1:
        jano_active_attention(q_act, k_cache, v_cache, idx, n_act, n_tokens, heads, d, d ** -0.5,
                              out, stream)
        return 1
    buf = ws.get(jano_active_attention_workspace_bytes(n_act, heads, d, split), stream)
    jano_active_attention_split(q_act, k_cache, v_cache, idx, n_act, n_tokens, heads, d, d ** -0.5,
                                split, buf, buf.numel(), out, stream)
    return split


def gather_gemm(x, w, out, gather=None, scatter=None, stream=None) -> None:
    """out[scatter[r] or r] = x[gather[r] or r] @ w^T for r < m (BF16 tensors
    x [n_x][k], w [n][k], out [n_out][n]; m = len(gather or scatter or x))."""
    n_x, k = x.shape
    n = w.shape[0]
    m = gather.numel() if gather is not None else (scatter.numel() if scatter is not None else n_x)
    jano_gather_gemm(x, n_x, gather, m, w, n, k, scatter, out, out.shape[0], stream)


def qkv_project(x, idx, w_qkv, q_act, k_cache, v_cache, stream=None) -> None:
    """Q/K/V of the active tokens idx from the hidden states x [N][k]:
    q_act [n_act][hd] and the rows idx of k_cache, v_cache [N][hd] (also
    accepted as [N][heads][d])."""
    N, k = x.shape
    hd = w_qkv.shape[0] // 3
    jano_qkv_project(x, N, idx, idx.numel(), w_qkv, hd, k, q_act, k_cache, v_cache, stream)


def random_scores(n_blocks: int, seed: int, out=None, stream=None) -> torch.Tensor:
    """Uniform scores of the random-masking ablation (classify them for a
    random level map with the analyzer's level counts)."""
    if out is None:
        out = torch.empty(n_blocks, dtype=torch.float32, device="cuda")
    jano_random_scores(n_blocks, seed, out, stream)
    return out


def fft_scores(x: torch.Tensor, geom: Geometry, cutoff: int = 1, out=None, stream=None) -> torch.Tensor:
    """High-band spectral energy per block of one snapshot x [C][F][H][W]
    (the FFT baseline score)."""
    if out is None:
        out = torch.empty(geom.n_blocks, dtype=torch.float32, device=x.device)
    jano_fft_scores(x, x.shape[0], geom.c(), cutoff, out, stream)
    return out


def device_error(stream=None) -> int:
    return jano_get_device_error(stream)


# ---------------------------------------------------------------- rotary positions and the paged cache
@dataclass(frozen=True)
class Rope:
    """Rotary positions with up to three axes (frame, row, column).

    axes    columns of a head that each axis turns (even; their sum at most d);
    n_pos   positions per axis that the table holds;
    grid    (rows, columns) of the token grid, for token ids without explicit
            coordinates;
    pairing "interleaved": columns (2s, 2s + 1); "halves": (s, s + rot / 2);
    shared  one frequency series over all slots instead of one per axis."""
    axes: tuple
    n_pos: tuple
    grid: tuple = (0, 0)
    theta: float = 10000.0
    pairing: str = "interleaved"
    shared: bool = False

    def __post_init__(self):
        if self.pairing not in ("interleaved", "halves"):
            raise ValueError(f"pairing must be 'interleaved' or 'halves', got {self.pairing!r}")
        if len(self.axes) != 3 or len(self.n_pos) != 3 or len(self.grid) != 2:
            raise ValueError("axes and n_pos have three entries, grid has two")

    @classmethod
    def of(cls, geom: "Geometry", axes, **kw) -> "Rope":
        """The rotation over a geometry's token grid."""
        pf, ph, pw = geom.patch
        n = (geom.F // pf, geom.H // ph, geom.W // pw)
        return cls(axes=tuple(axes), n_pos=n, grid=n[1:], **kw)

    def c(self) -> jano_rope_cfg:
        return jano_rope_cfg.from_buffer_copy(_ROPE(*self.axes, *self.n_pos, *self.grid, self.pairing == "halves"))

    @property
    def table_shape(self) -> tuple:
        return (sum(n * (a // 2) for a, n in zip(self.axes, self.n_pos)), 2)


def _table(rope: Rope, table: torch.Tensor) -> None:
    (a, b, c), (x, y, z) = rope.axes, rope.n_pos
    _count(table, "table", 2 * (x * (a // 2) + y * (b // 2) + z * (c // 2)))


def rope_table(rope: Rope, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The (cos, sin) table of a rotation, fp32 [entries][2]: axis 0's
    positions x slots, then axis 1's, then axis 2's."""
    if out is None:
        dev = torch.empty(0, dtype=torch.float32, device="cuda")
        out = _on_stream(stream, rope.table_shape, dev)
    _here(out=out)
    _table(rope, out)
    jano_rope_table(rope.c(), rope.theta, int(rope.shared), out, stream)
    return out


def axis_rope(x, rope: Rope, table, ids=None, coords=None, out=None, stream=None) -> torch.Tensor:
    """x [rows][heads][d] rotated by each row's position: of token ids[r]
    (default r) on the rope's grid, or at coords [rows][3].  out may be x."""
    ld = _rows(x, "x")
    n, h, d = x.shape
    _here(x=x, table=table, ids=ids, coords=coords, out=out)
    _table(rope, table)
    _count(ids, "ids", n)
    _count(coords, "coords", 3 * n)
    if out is None:
        out = _on_stream(stream, (n, h, d), x)
    elif out.shape[0] != n:
        raise ValueError(f"out must have {n} rows, got {out.shape[0]}")
    jano_axis_rope(x, ld, ids, coords, n, h, d, rope.c(), table, out, _rows(out, "out", h, d), stream)
    return out


def _queries(q, q_out, n, d, stream):
    """(q, its row distance, q_out, its row distance, heads) of an append; q may be None."""
    if q is None:
        if q_out is not None:
            raise ValueError("q_out without q")
        return None, 0, None, 0, 1
    ld = _rows(q, "q", None, d)
    if q.shape[0] != n:
        raise ValueError(f"q must have {n} rows, got {q.shape[0]}")
    h = q.shape[1]
    if q_out is None:
        q_out = _on_stream(stream, (n, h, d), q)
    elif q_out.shape[0] != n:
        raise ValueError(f"q_out must have {n} rows, got {q_out.shape[0]}")
    return q, ld, q_out, _rows(q_out, "q_out", h, d), h


def rope_scatter(k, v, idx, k_cache, v_cache, rope: Rope, table, q=None, q_out=None, coords=None, stream=None):
    """kv_scatter with the rotation on the way: rows idx of the caches
    [N][kv_heads][d] become the rotated k and v; the queries q [n][heads][d]
    are rotated in the same launch (into q_out, which may be q; returned)."""
    n = idx.numel()
    N, h, d = k_cache.shape
    _here(k=k, v=v, idx=idx, k_cache=k_cache, v_cache=v_cache, table=table, q=q, q_out=q_out, coords=coords)
    k_ld, v_ld = _rows(k, "k", h, d), _rows(v, "v", h, d)
    if k.shape[0] != n or v.shape[0] != n or v_cache.shape != k_cache.shape:
        raise ValueError("k, v and idx must have as many rows, and both caches one shape")
    _table(rope, table)
    _count(coords, "coords", 3 * n)
    q, q_ld, q_out, o_ld, heads = _queries(q, q_out, n, d, stream)
    jano_rope_scatter(q, q_ld, k, k_ld, v, v_ld, idx, coords, n, heads, h, d, rope.c(), table, q_out, o_ld,
                      k_cache, v_cache, N, stream)
    return q_out


def page_pool(n_pages: int, page_size: int, kv_heads: int, d: int, head_major: bool = False, device="cuda"):
    """Empty K and V pages, each [n_pages][page_size][kv_heads][d] (head_major:
    a head's places are adjacent in memory)."""
    shape = (n_pages, kv_heads, page_size, d) if head_major else (n_pages, page_size, kv_heads, d)
    k, v = (torch.empty(shape, dtype=torch.bfloat16, device=device) for _ in range(2))
    return (k.transpose(1, 2), v.transpose(1, 2)) if head_major else (k, v)


# the C structures packed in one step (a third of the time of their constructors)
_ROPE = struct.Struct("9i").pack
_POOL = struct.Struct("PP4i3q").pack
_SEQS = struct.Struct("PPP2i").pack


def _pool(k_pages, v_pages) -> jano_page_pool:
    for t, name in ((k_pages, "k_pages"), (v_pages, "v_pages")):
        if t.dtype != torch.bfloat16:
            raise TypeError(f"{name} must be torch.bfloat16, got {t.dtype}")
        if t.dim() != 4:
            raise ValueError(f"{name} must be [pages][page_size][kv_heads][d], got {tuple(t.shape)}")
    if k_pages.shape != v_pages.shape or k_pages.stride() != v_pages.stride():
        raise ValueError("k_pages and v_pages must have one shape and the same strides")
    n, p, h, d = k_pages.shape
    s0, s1, s2, s3 = k_pages.stride()
    if d > 1 and s3 != 1:
        raise ValueError("the columns of a head must be adjacent")
    # the stride of a dimension of one element is any number: one that passes the checks
    return jano_page_pool.from_buffer_copy(_POOL(k_pages.data_ptr(), v_pages.data_ptr(), n, p, h, d,
                                                 s0 if n > 1 else p * h * d, s1, s2 if h > 1 else d))


def _seqs(page_table, seq_lens, cu_rows) -> jano_page_seqs:
    if page_table.dim() != 2:
        raise ValueError(f"page_table must be [sequences][pages], got {tuple(page_table.shape)}")
    n = page_table.shape[0]
    _count(seq_lens, "seq_lens", n)
    _count(cu_rows, "cu_rows", n + 1)
    return jano_page_seqs.from_buffer_copy(_SEQS(
        _dev(page_table, "page_table", torch.int32), _dev(seq_lens, "seq_lens", torch.int32),
        _dev(cu_rows, "cu_rows", torch.int32), n, page_table.shape[1]))


def paged_append(k, v, pos, k_pages, v_pages, page_table, seq_lens, cu_rows, rope: Rope | None = None, table=None,
                 q=None, q_out=None, coords=None, grids=None, stream=None):
    """Write new K/V rows [n][kv_heads][d] at positions pos of their sequences
    (sequence s owns rows cu_rows[s]:cu_rows[s+1]; seq_lens counts them in),
    K rotated on the way when a rope and its table are given, and the queries
    q [n][heads][d] with it (into q_out, which may be q; returned).  A row's
    coordinates come from coords [n][3], or from pos on its sequence's grid
    (grids [sequences][2], or the rope's)."""
    n = pos.numel()
    h, d = k_pages.shape[-2:]
    _here(k=k, v=v, pos=pos, k_pages=k_pages, v_pages=v_pages, page_table=page_table, seq_lens=seq_lens,
          cu_rows=cu_rows, table=table, q=q, q_out=q_out, coords=coords, grids=grids)
    k_ld, v_ld = _rows(k, "k", h, d), _rows(v, "v", h, d)
    if k.shape[0] != n or v.shape[0] != n:
        raise ValueError("k, v and pos must have as many rows")
    if rope is None and (table is not None or coords is not None or grids is not None):
        raise ValueError("table, coords and grids need a rope")
    if rope is not None:
        if table is None:
            raise ValueError("a rope needs its table")
        _table(rope, table)
    _count(coords, "coords", 3 * n)
    _count(grids, "grids", 2 * page_table.shape[0])
    q, q_ld, q_out, o_ld, heads = _queries(q, q_out, n, d, stream)
    jano_paged_append(_pool(k_pages, v_pages), _seqs(page_table, seq_lens, cu_rows), q, q_ld, k, k_ld, v, v_ld, pos,
                      coords, grids, n, heads, None if rope is None else rope.c(), table, q_out, o_ld, stream)
    return q_out


def paged_attention(q, k_pages, v_pages, page_table, seq_lens, cu_rows, out=None, limits=None, max_rows=None,
                    max_len=None, scale=None, split=0, stream=None) -> torch.Tensor:
    """Attention of the rows q [n][heads][d] of several sequences over their
    pages; row r sees the first min(seq_lens[s], limits[r]) positions (all of
    them without limits; none: zeros).  max_rows / max_len: upper bounds of a
    sequence's rows and length, if known (they size the grid and choose the
    split); split: CTAs that share one query tile's keys (0: the library's
    choice).  Rows past cu_rows[-1] of out are left as they are."""
    q_ld = _rows(q, "q")
    n, h, d = q.shape
    _here(q=q, k_pages=k_pages, v_pages=v_pages, page_table=page_table, seq_lens=seq_lens, cu_rows=cu_rows, out=out,
          limits=limits)
    if k_pages.shape[-1] != d:
        raise ValueError(f"q and the pages must have one head size, got {d} and {k_pages.shape[-1]}")
    _count(limits, "limits", n)
    if out is None:
        out = _on_stream(stream, (n, h, d), q)
    elif out.shape[0] != n:
        raise ValueError(f"out must have {n} rows, got {out.shape[0]}")
    if max_rows is None:
        max_rows = n
    if max_len is None:
        max_len = page_table.shape[1] * k_pages.shape[1]
    jano_paged_attention(_pool(k_pages, v_pages), _seqs(page_table, seq_lens, cu_rows), q, q_ld, limits, n, max_rows,
                         max_len, h, d ** -0.5 if scale is None else scale, split, out, _rows(out, "out", h, d),
                         stream)
    return out
