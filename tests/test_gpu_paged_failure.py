"""Failure detection of the paged attention, without a fault: bounded waits
run out.

The test-only build of the library (``-DJANO_INJECT_DROP_LOAD=2``) never
issues a CTA's third K tile, so the MMA thread's wait for it runs out after
about a second.  The CTA records JANO_ETIMEOUT, its other warps see the abort
flag, copies in flight land, tensor memory is freed, a cluster's barriers are
kept, and rows with a missing part are not written.  The context stays usable:
the product library then computes the same attention.
"""
import ctypes as C
import os

import numpy as np
import pytest
import torch

from paged_tools import Paged

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ETIMEOUT = 7


@pytest.fixture(scope="module")
def inject():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from kv_cache_analyzer_b200 import build
    L = C.CDLL(build.build(out=os.path.join(ROOT, "_build", "inject", "libjano_inject.so"),
                           defines=("JANO_INJECT_DROP_LOAD=2",)))
    P, i, ll = C.c_void_p, C.c_int, C.c_longlong
    L.jano_paged_attention.argtypes = [P, P, P, ll, P, i, i, i, i, C.c_float, i, P, C.c_size_t, P, ll, P]
    L.jano_get_device_error.argtypes = [P]
    return L


CASES = [  # rows, lengths, heads, kv_heads, d, split (0: with a workspace): pair, single, cluster, few rows
    ([200], [512], 2, 2, 128, 1),
    ([40, 3], [512, 128], 2, 1, 64, 1),
    ([40], [1000], 2, 2, 128, 2),
    ([1, 1], [16384, 100], 16, 8, 64, 0),
]


@pytest.mark.parametrize("rows,lens,heads,kv_heads,d,split", CASES)
def test_wait_runs_out_reports_and_leaves_rows(inject, rows, lens, heads, kv_heads, d, split):
    import kv_cache_analyzer_b200 as J
    import kv_cache_analyzer_b200.paged as PG
    p = Paged(rows, lens, heads, kv_heads, d, 64, seed=7)
    n = p.n
    out = torch.full_like(p.dev_q, 0.25)
    stream = torch.cuda.current_stream().cuda_stream
    ws = torch.full((J.jano_paged_attention_workspace_bytes(max(rows), heads, kv_heads, d) // 4 if split == 0 else 4,),
                    float("nan"), dtype=torch.float32, device="cuda")
    assert inject.jano_paged_attention(
        PG._pool(p.dev_k, p.dev_v, 0), PG._seqs(p.dev_table, p.dev_lens, p.dev_cu, 0), p.dev_q.data_ptr(), heads * d,
        None, n, max(rows), max(lens), heads, d ** -0.5, split, ws.data_ptr() if split == 0 else None, ws.numel() * 4,
        out.data_ptr(), heads * d, stream) == 0
    assert inject.jano_get_device_error(stream) == ETIMEOUT
    assert inject.jano_get_device_error(stream) == 0              # read and cleared
    assert bool((out[:rows[0]] == 0.25).all())
    # the product library on the same device
    good = torch.empty_like(p.dev_q)
    J.paged_attention(p.dev_q, p.dev_k, p.dev_v, p.dev_table, p.dev_lens, p.dev_cu, out=good, max_rows=max(rows),
                      split=split)
    assert J.device_error() == 0
    if max(lens) <= 1000:
        p.check(good)
    else:
        assert torch.isfinite(good.float()).all()
    # a sequence whose tiles all arrived is right, or not written where it shared a CTA
    for s in range(1, len(rows)):
        a, b = int(p.cu[s]), int(p.cu[s + 1])
        assert torch.equal(out[a:b], good[a:b]) or bool((out[a:b] == 0.25).any())
