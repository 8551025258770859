"""A wait that spans many key tiles does not run out while the tiles go on.

The test-only build of the library (``-DJANO_WAIT_CYCLES=2097152``) bounds its
waits at about a millisecond, where the product's stand at about a second: what
takes the product 2^26 keys (a CTA's own tiles for about a second) it meets at a
few hundred thousand.  Each wait ends, by its bound or by the copy it waits for."""
import ctypes as C
import os

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def hasty():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from kv_cache_analyzer_b200 import build
    L = C.CDLL(build.build(out=os.path.join(ROOT, "_build", "hasty", "libjano_hasty.so"),
                           defines=("JANO_WAIT_CYCLES=2097152",)))
    P, i, ll = C.c_void_p, C.c_int, C.c_longlong
    L.jano_paged_attention.argtypes = [P, P, P, ll, P, i, i, i, i, C.c_float, i, P, C.c_size_t, P, ll, P]
    L.jano_get_device_error.argtypes = [P]
    return L


@pytest.mark.parametrize("rows,length,heads,split", [
    (256, 2 ** 19 - 5, 1, 1),              # two tiles a CTA; the last V tile's clearing waits from the first
    (100, 2 ** 20 - 100, 1, 1),            # one tile, two streams
    (1, 2 ** 18 - 28, 888, 0),             # few rows: six long items a CTA, each with a ragged end
    (1, 2 ** 18, 888, 0),                  # ... and without: warps that have nothing to do run ahead
])
def test_a_long_items_waits_outlast_its_tiles(hasty, rows, length, heads, split):
    import kv_cache_analyzer_b200 as J
    import kv_cache_analyzer_b200.paged as PG
    d, page = 128, 16
    gen = torch.Generator("cuda").manual_seed(length)
    k, v = (torch.randn((8, page, heads, d), generator=gen, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn((rows, heads, d), generator=gen, device="cuda").bfloat16()
    ints = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()
    table = ints(np.arange(-(-length // page))[None] % 8)
    lens, cu = ints([length]), ints([0, rows])
    need = J.jano_paged_attention_workspace_bytes(rows, heads, heads, d) if split == 0 else 0
    assert (need > 0) == (split == 0)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    out = torch.full_like(q, 0.25)
    stream = torch.cuda.current_stream().cuda_stream
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    assert hasty.jano_paged_attention(
        PG._pool(k, v, 0), PG._seqs(table, lens, cu, 0), q.data_ptr(), heads * d, None, rows, rows, length, heads,
        d ** -0.5, split, ws.data_ptr() if need else None, need, out.data_ptr(), heads * d, stream) == 0
    end.record()
    assert hasty.jano_get_device_error(stream) == 0
    # it did last longer than one bound (at no more than 2 GHz), an item of the few-rows form too
    assert begin.elapsed_time(end) * 2e6 / (6 if split == 0 else 1) > 2097152
    want = J.paged_attention(q, k, v, table, lens, cu, max_rows=rows, split=split)
    assert J.device_error() == 0
    assert torch.equal(out, want) and torch.isfinite(out.float()).all()
