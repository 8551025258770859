"""GPU parity of the paged attention where its masks and its softmax can go
wrong, against the fp64 oracle.  Tolerances: tests/paged_tools.py.  Places that
nobody owns or that lie past a sequence's length hold NaN throughout."""
import numpy as np
import pytest
import torch

from paged_tools import Paged

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def J():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from kv_cache_analyzer_b200 import build
    build.build()
    import kv_cache_analyzer_b200 as j
    j.lib()
    return j


def no_device_error(J):
    code = J.device_error()
    assert code == 0, J.jano_status_str(code)


def ints(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def attend(J, p, limits=None, **kw):
    return J.paged_attention(p.dev_q, p.dev_k, p.dev_v, p.dev_table, p.dev_lens, p.dev_cu,
                             limits=None if limits is None else ints(limits), **kw)


LOWEST = -2 ** 31
FAR_BELOW = [LOWEST, LOWEST + 1, LOWEST + 127, LOWEST + 128, LOWEST + 300, -2 ** 30, -1, 0]
FORMS = [  # rows, lengths, heads, kv_heads, splits (None: few rows, with a workspace)
    ([8, 5, 3, 2], [300, 130, 257, 140], 4, 2, (None,)),
    ([16, 1, 9, 1], [700, 64, 513, 1], 2, 1, (None,)),
    ([40, 3, 30, 9], [300, 130, 513, 200], 2, 1, (1, 2, 4, 8)),        # one tile each
    ([150, 30, 140, 5], [400, 300, 140, 100], 2, 2, (1, 2, 8)),        # two tiles and one
]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows,lens,heads,kv_heads,splits", FORMS)
def test_limits_down_to_the_lowest_int(J, rows, lens, heads, kv_heads, splits, d):
    # rows that see nothing by any limit from 0 to the lowest int32, among rows with causal limits (in the
    # same warp), and whole sequences of them
    p = Paged(rows, lens, heads, kv_heads, d, 32, seed=sum(lens))
    causal = np.concatenate([np.arange(m - r, m) + 1 for r, m in zip(rows, lens)]).astype(np.int64)
    for every in (3, 1):
        limits = causal.copy()
        dark = np.arange(every - 1, len(limits), every)
        limits[dark] = [FAR_BELOW[i % len(FAR_BELOW)] for i in range(len(dark))]
        limits[p.cu[3]:] = LOWEST                                     # the last sequence sees nothing
        for split in splits:
            kw = dict(max_rows=max(rows)) if split is None else dict(split=split)
            out = torch.full_like(p.dev_q, 3.0)
            attend(J, p, limits, out=out, **kw)
            no_device_error(J)
            p.check(out, limits)
