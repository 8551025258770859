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


@pytest.mark.parametrize("tiles", [73999, 74000, 74001])
def test_few_rows_of_two_items_cut_at_a_thousand_tiles(J, tiles):
    # Parts of some thousand key tiles, one tile less and more than a multiple: every part must be found again
    # by the merge.  The sequences go through 64 pages one after another, and page c has its V in column c
    # alone, so column c is the weight of a 64th of the keys: a lost or doubled part (a 74th) shows there.
    gen = np.random.default_rng(tiles)
    lens = [tiles * 128, 73556 * 128]
    page, d, n_pages = 256, 64, 64
    per = [-(-m // page) for m in lens]
    table = np.zeros((2, max(per)), dtype=np.int64)
    for s in range(2):
        table[s, :per[s]] = np.arange(per[s]) * n_pages // per[s]
    k = torch.from_numpy(gen.standard_normal((n_pages, page, 1, d))).bfloat16()
    v = torch.zeros_like(k)
    for c in range(n_pages):
        v[c, :, 0, c] = 1.0
    q = torch.from_numpy(gen.standard_normal((2, 1, d))).bfloat16()
    out = J.paged_attention(q.cuda(), k.cuda(), v.cuda(), ints(table), ints(lens), ints([0, 1, 2]), max_rows=1)
    no_device_error(J)
    for s in range(2):
        times = np.bincount(table[s, :per[s]], minlength=n_pages).astype(np.float64)[:, None] * np.ones(page)
        last = per[s] * page - lens[s]                               # places of the last page past the length
        if last:
            times[table[s, per[s] - 1], page - last:] -= 1.0
        kk, qq = k[:, :, 0].double().numpy(), q[s, 0].double().numpy()
        z = kk @ qq * d ** -0.5
        w = times * np.exp(z - z.max())
        want = w.sum(1) / w.sum()
        top = (np.abs(kk) @ np.abs(qq)).max() * d ** -0.5
        # as check_attention, and the fp32 sums of a share's O: 8 additions a tile, each off by at most 2^-23
        bound = (2.0 ** -8 + 2.0 ** -8 + 2.0 ** -15 * top + 2.0 ** -12 + 8 * 1002 * 2.0 ** -23) * want
        err = np.abs(out[s, 0].double().cpu().numpy() - want)
        assert np.all(err <= bound), (s, float((err / want).max()), float((bound / want).max()))
        assert float((bound / want).max()) < 0.5 * 64 / 75            # below what half of a part would move
