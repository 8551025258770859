"""Rotary positions with several axes, and a KV cache in pages shared by
several generations: the torch side of jano_axis_rope, jano_rope_scatter,
jano_paged_append and jano_paged_attention.

These calls are made for small work too (a token per generation), where the
host's share is most of their time, so each argument is looked at once: type,
device, shape and layout in one expression, the reasons only where it fails.
Tensors live on the current CUDA device; rows are BF16 [rows][heads][d] whose
heads and columns are adjacent (rows may be slices of a wider buffer), lists
are contiguous int32.
"""
from __future__ import annotations

import ctypes as C
import functools
import struct
from dataclasses import dataclass

import torch

from . import (Geometry, _stream, _torch_stream, jano_axis_rope, jano_paged_append, jano_paged_attention,
               jano_paged_attention_workspace_bytes, jano_rope_cfg, jano_rope_scatter, jano_rope_table)

_current_device, _current_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
_BF16, _I32, _F32 = torch.bfloat16, torch.int32, torch.float32
# the C structures, packed in one step (a fifth of the time of their constructors)
_ROPE = struct.Struct("9i").pack            # jano_rope_cfg
_POOL = struct.Struct("PP4i3q").pack        # jano_page_pool
_SEQS = struct.Struct("PPP2i").pack         # jano_page_seqs


# ---------------------------------------------------------------- arguments
def _device(t: torch.Tensor, name: str) -> int:
    """The device of a call's first tensor: the current one."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    cur = _current_device()
    if dev != cur:
        raise ValueError(f"{name} is on cuda:{dev}, the current device is cuda:{cur}")
    return dev


def _wrong(t: torch.Tensor, name: str, dev: int, dtype, shape: str) -> Exception:
    if t.dtype is not dtype:
        return TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        return ValueError(f"{name} must be a CUDA tensor on cuda:{dev}, got {t.device}")
    return ValueError(f"{name} must be {shape}, got {tuple(t.shape)} with strides {t.stride()}")


def _list(t: torch.Tensor | None, name: str, n: int, dev: int, dtype=_I32) -> int | None:
    """Address of a contiguous tensor of n elements."""
    if t is None:
        return None
    if t.dtype is not dtype or t.get_device() != dev or t.numel() != n or not t.is_contiguous():
        raise _wrong(t, name, dev, dtype, f"contiguous with {n} elements")
    return t.data_ptr()


def _rows(t: torch.Tensor, name: str, dev: int, n: int, heads: int, d: int) -> tuple:
    """(address, row distance) of rows [n][heads][d]."""
    if t.dtype is _BF16 and t.get_device() == dev and t.shape == (n, heads, d):
        if t.is_contiguous():                  # (a single row too, whatever its stride)
            return t.data_ptr(), heads * d
        strides = t.stride()
        if (strides[2] == 1 or d == 1) and (strides[1] == d or heads == 1):
            return t.data_ptr(), strides[0] if n > 1 else heads * d
    raise _wrong(t, name, dev, _BF16, f"[{n}][{heads}][{d}], its heads and columns adjacent")


def _shape3(t: torch.Tensor, name: str) -> tuple:
    if t.dim() != 3:
        raise ValueError(f"{name} must be [rows][heads][d], got {tuple(t.shape)}")
    return t.shape


def _new(stream, shape, like: torch.Tensor) -> torch.Tensor:
    """A new tensor of like's type for a launch on `stream` (allocated there, so
    that the memory's earlier uses are ordered before it)."""
    if stream is None:
        return torch.empty_like(like) if like.shape == shape and like.is_contiguous() else like.new_empty(shape)
    with torch.cuda.stream(_torch_stream(stream)):
        return like.new_empty(shape)


def _launch_stream(stream, dev: int) -> int:
    """The cudaStream_t of a launch on the current device `dev`."""
    return _current_stream(dev) if stream is None else _stream(stream)


def _pool(k_pages: torch.Tensor, v_pages: torch.Tensor, dev: int) -> bytes:
    """jano_page_pool of pages [n][page_size][kv_heads][d]."""
    shape, strides = k_pages.shape, k_pages.stride()
    if (len(shape) != 4 or k_pages.dtype is not _BF16 or v_pages.dtype is not _BF16 or v_pages.shape != shape or
            v_pages.stride() != strides or (strides[3] != 1 and shape[3] > 1) or k_pages.get_device() != dev or
            v_pages.get_device() != dev):
        for t, name in ((k_pages, "k_pages"), (v_pages, "v_pages")):
            if t.dtype is not _BF16 or t.get_device() != dev or t.dim() != 4 or (t.stride(3) != 1 and t.shape[3] > 1):
                raise _wrong(t, name, dev, _BF16, "[pages][page_size][kv_heads][d], its columns adjacent")
        raise ValueError("k_pages and v_pages must have one shape and the same strides, got "
                         f"{tuple(shape)} {strides} and {tuple(v_pages.shape)} {v_pages.stride()}")
    n, p, h, d = shape
    # the stride of a dimension of one element is any number: one that passes the checks
    return _POOL(k_pages.data_ptr(), v_pages.data_ptr(), n, p, h, d, strides[0] if n > 1 else p * h * d,
                 strides[1], strides[2] if h > 1 else d)


def _seqs(page_table: torch.Tensor, seq_lens: torch.Tensor, cu_rows: torch.Tensor, dev: int) -> bytes:
    if page_table.dim() != 2:
        raise ValueError(f"page_table must be [sequences][pages], got {tuple(page_table.shape)}")
    n, pages = page_table.shape
    return _SEQS(_list(page_table, "page_table", n * pages, dev), _list(seq_lens, "seq_lens", n, dev),
                 _list(cu_rows, "cu_rows", n + 1, dev), n, pages)


# ---------------------------------------------------------------- rotary positions
@dataclass(frozen=True, init=False)
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

    def __init__(self, axes, n_pos, grid=(0, 0), theta=10000.0, pairing="interleaved", shared=False):
        if pairing not in ("interleaved", "halves"):
            raise ValueError(f"pairing must be 'interleaved' or 'halves', got {pairing!r}")
        if len(axes) != 3 or len(n_pos) != 3 or len(grid) != 2:
            raise ValueError("axes and n_pos have three entries, grid has two")
        # past the frozen class's __setattr__: 0.7 us, not 1.2 (a call of few rows costs the host 12)
        self.__dict__.update(axes=axes, n_pos=n_pos, grid=grid, theta=theta, pairing=pairing, shared=shared)

    @classmethod
    def of(cls, geom: Geometry, axes, **kw) -> "Rope":
        """The rotation over a geometry's token grid."""
        pf, ph, pw = geom.patch
        n = (geom.F // pf, geom.H // ph, geom.W // pw)
        return cls(axes=tuple(axes), n_pos=n, grid=n[1:], **kw)

    def packed(self) -> bytes:
        return _ROPE(*self.axes, *self.n_pos, *self.grid, self.pairing == "halves")

    def c(self) -> jano_rope_cfg:
        return jano_rope_cfg.from_buffer_copy(self.packed())

    @property
    def entries(self) -> int:
        """(cos, sin) pairs of the table."""
        (a, b, c), (x, y, z) = self.axes, self.n_pos
        return x * (a // 2) + y * (b // 2) + z * (c // 2)


def rope_table(rope: Rope, out: torch.Tensor | None = None, stream=None, device="cuda") -> torch.Tensor:
    """The (cos, sin) table of a rotation, fp32 [entries][2]: axis 0's
    positions x slots, then axis 1's, then axis 2's.  Without out it is made
    on `device` (default: the current one), on its stream `stream`."""
    if out is None:
        with torch.cuda.device(device):
            out = _new(stream, (rope.entries, 2), torch.empty(0, dtype=_F32, device="cuda"))
            return rope_table(rope, out, stream)
    _list(out, "out", 2 * rope.entries, _device(out, "out"), _F32)
    jano_rope_table(rope.c(), rope.theta, int(rope.shared), out, stream)
    return out


def axis_rope(x, rope: Rope, table, ids=None, coords=None, out=None, stream=None) -> torch.Tensor:
    """x [rows][heads][d] rotated by each row's position: of token ids[r]
    (default r) on the rope's grid, or at coords [rows][3].  out may be x."""
    n, h, d = _shape3(x, "x")
    dev = _device(x, "x")
    x_ptr, x_ld = _rows(x, "x", dev, n, h, d)
    if out is None:
        out = _new(stream, (n, h, d), x)
    o_ptr, o_ld = _rows(out, "out", dev, n, h, d)
    jano_axis_rope(x_ptr, x_ld, _list(ids, "ids", n, dev), _list(coords, "coords", 3 * n, dev), n, h, d,
                   rope.packed(), _list(table, "table", 2 * rope.entries, dev, _F32), o_ptr, o_ld,
                   _launch_stream(stream, dev))
    return out


def _queries(q, q_out, n, d, dev, stream) -> tuple:
    """(q, its row distance, q_out, its row distance, heads, the q_out tensor) of an append; q may be None."""
    if q is None:
        if q_out is not None:
            raise ValueError("q_out without q")
        return None, 0, None, 0, 1, None
    h = _shape3(q, "q")[1]
    ptr, ld = _rows(q, "q", dev, n, h, d)
    if q_out is None:
        q_out = _new(stream, (n, h, d), q)
        return ptr, ld, q_out.data_ptr(), h * d, h, q_out
    o_ptr, o_ld = _rows(q_out, "q_out", dev, n, h, d)
    return ptr, ld, o_ptr, o_ld, h, q_out


def rope_scatter(k, v, idx, k_cache, v_cache, rope: Rope, table, q=None, q_out=None, coords=None, stream=None):
    """kv_scatter with the rotation on the way: rows idx of the caches
    [N][kv_heads][d] become the rotated k and v; the queries q [n][heads][d]
    are rotated in the same launch (into q_out, which may be q; returned)."""
    n = idx.numel()
    N, h, d = _shape3(k_cache, "k_cache")
    dev = _device(k_cache, "k_cache")
    size = N * h * d
    k_ptr, k_ld = _rows(k, "k", dev, n, h, d)
    v_ptr, v_ld = _rows(v, "v", dev, n, h, d)
    q_ptr, q_ld, o_ptr, o_ld, heads, q_out = _queries(q, q_out, n, d, dev, stream)
    jano_rope_scatter(q_ptr, q_ld, k_ptr, k_ld, v_ptr, v_ld, _list(idx, "idx", n, dev),
                      _list(coords, "coords", 3 * n, dev), n, heads, h, d, rope.packed(),
                      _list(table, "table", 2 * rope.entries, dev, _F32), o_ptr, o_ld,
                      _list(k_cache, "k_cache", size, dev, _BF16), _list(v_cache, "v_cache", size, dev, _BF16), N,
                      _launch_stream(stream, dev))
    return q_out


# ---------------------------------------------------------------- the paged cache
def page_pool(n_pages: int, page_size: int, kv_heads: int, d: int, head_major: bool = False, device="cuda"):
    """Empty K and V pages, each [n_pages][page_size][kv_heads][d] (head_major:
    a head's places are adjacent in memory)."""
    shape = (n_pages, kv_heads, page_size, d) if head_major else (n_pages, page_size, kv_heads, d)
    k, v = (torch.empty(shape, dtype=_BF16, device=device) for _ in range(2))
    return (k.transpose(1, 2), v.transpose(1, 2)) if head_major else (k, v)


def paged_append(k, v, pos, k_pages, v_pages, page_table, seq_lens, cu_rows, rope: Rope | None = None, table=None,
                 q=None, q_out=None, coords=None, grids=None, stream=None):
    """Write new K/V rows [n][kv_heads][d] at positions pos of their sequences
    (sequence s owns rows cu_rows[s]:cu_rows[s+1]; seq_lens counts them in),
    K rotated on the way when a rope and its table are given, and the queries
    q [n][heads][d] with it (into q_out, which may be q; returned).  A row's
    coordinates come from coords [n][3], or from pos on its sequence's grid
    (grids [sequences][2], or the rope's)."""
    n = pos.numel()
    if k_pages.dim() != 4:
        raise ValueError(f"k_pages must be [pages][page_size][kv_heads][d], got {tuple(k_pages.shape)}")
    _, _, h, d = k_pages.shape
    dev = _device(k_pages, "k_pages")
    k_ptr, k_ld = _rows(k, "k", dev, n, h, d)
    v_ptr, v_ld = _rows(v, "v", dev, n, h, d)
    cfg = None
    if rope is not None:
        if table is None:
            raise ValueError("a rope needs its table")
        cfg, table = rope.packed(), _list(table, "table", 2 * rope.entries, dev, _F32)
    elif table is not None or coords is not None or grids is not None:
        raise ValueError("table, coords and grids need a rope")
    seqs = _seqs(page_table, seq_lens, cu_rows, dev)
    q_ptr, q_ld, o_ptr, o_ld, heads, q_out = _queries(q, q_out, n, d, dev, stream)
    jano_paged_append(_pool(k_pages, v_pages, dev), seqs, q_ptr, q_ld, k_ptr, k_ld, v_ptr, v_ld,
                      _list(pos, "pos", n, dev), _list(coords, "coords", 3 * n, dev),
                      None if grids is None else _list(grids, "grids", 2 * page_table.shape[0], dev), n, heads, cfg,
                      table, o_ptr, o_ld,
                      _launch_stream(stream, dev))
    return q_out


@functools.lru_cache(maxsize=None)
def _decode_bytes(device: int, max_rows: int, heads: int, kv_heads: int, d: int) -> int:
    """jano_paged_attention_workspace_bytes on the current device `device`."""
    return jano_paged_attention_workspace_bytes(max_rows, heads, kv_heads, d)


def paged_attention(q, k_pages, v_pages, page_table, seq_lens, cu_rows, out=None, limits=None, max_rows=None,
                    max_len=None, scale=None, split=0, workspace=None, stream=None) -> torch.Tensor:
    """Attention of the rows q [n][heads][d] of several sequences over their
    pages; row r sees the first min(seq_lens[s], limits[r]) positions (all of
    them without limits; none: zeros).  max_rows / max_len: upper bounds of a
    sequence's rows and length, if known (they size the grid and choose the
    form: give max_rows where it is small); split: CTAs that share one query
    tile's keys (0: the library's choice).  workspace: a device uint8 tensor
    of jano_paged_attention_workspace_bytes bytes, allocated here if None and
    needed; calls that may overlap (streams, captured graphs) must not share
    one.  K and V below a sequence's length must be finite.  Rows past
    cu_rows[-1] of out are left as they are."""
    n, h, d = _shape3(q, "q")
    dev = _device(q, "q")
    q_ptr, q_ld = _rows(q, "q", dev, n, h, d)
    pool = _pool(k_pages, v_pages, dev)
    _, page_size, kv_heads, pool_d = k_pages.shape
    if pool_d != d:
        raise ValueError(f"q and the pages must have one head size, got {d} and {pool_d}")
    if out is None:
        out = _new(stream, (n, h, d), q)
        o_ptr, o_ld = out.data_ptr(), h * d
    else:
        o_ptr, o_ld = _rows(out, "out", dev, n, h, d)
    if max_rows is None:
        max_rows = n
    if max_len is None:
        max_len = min(page_table.shape[1] * page_size, 1 << 26)          # the longest that a call takes
    ws, ws_bytes = None, 0
    if workspace is not None:
        ws, ws_bytes = _list(workspace, "workspace", workspace.numel(), dev, torch.uint8), workspace.numel()
    elif split == 0 and 0 < max_rows * h <= 32 * kv_heads:
        ws_bytes = _decode_bytes(dev, max_rows, h, kv_heads, d)
        if ws_bytes:
            workspace = _new(stream, (ws_bytes // 2,), q)        # BF16 elements
            ws = workspace.data_ptr()
    jano_paged_attention(pool, _seqs(page_table, seq_lens, cu_rows, dev), q_ptr, q_ld,
                         _list(limits, "limits", n, dev), n, max_rows, max_len, h,
                         d ** -0.5 if scale is None else scale, split, ws, ws_bytes, o_ptr, o_ld,
                         _launch_stream(stream, dev))
    return out
