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


@pytest.mark.parametrize("rows,n,heads,kv_heads,d,kw", [
    ([130, 2], 640, 2, 2, 64, {}),                                      # a pair of tiles; some exponentials by polynomial
    ([130, 2], 640, 2, 2, 64, dict(split=2)),
    ([40, 1], 640, 2, 1, 64, dict(split=1)),                            # one tile, two streams of keys
    ([40, 1], 1500, 2, 1, 128, dict(split=4)),
    ([1, 2], 640, 2, 2, 64, dict(max_rows=2)),                          # few rows
    ([2, 1], 2300, 2, 2, 128, dict(max_rows=2)),                        # ... an item in many parts
    ([7, 9], 900, 3, 1, 64, dict(max_rows=9)),
])
def test_maxima_that_grow_in_every_form(J, rows, n, heads, kv_heads, d, kw):
    # logits up to some hundreds that rise key by key (every tile makes the running maximum grow by more than the
    # lazy rescale allows), fall (all but the first keys below the polynomial's clamp) and come in no order
    for seed, order in enumerate((np.arange(n), np.arange(n)[::-1], np.random.default_rng(1).permutation(n))):
        p = Paged(rows, [n, n], heads, kv_heads, d, 64, seed=seed)
        scale_of = (0.25 * 2.0 ** (np.arange(n) * 6.4 / n))[order].astype(np.float32)
        for s in range(2):
            for j in range(n):
                p.k[p.table[s, j // 64], j % 64] = p.q[0, :1] * float(scale_of[j])
        p.dev_k = p.k.cuda()
        out = attend(J, p, **kw)
        no_device_error(J)
        p.check(out)


AT_SIZE = [  # rows, lengths, heads, kv_heads, d, page, limits ("token", a frame's tokens, or none)
    ([4680], [32760], 12, 12, 128, 128, 1560),
    ([16380], [32760], 12, 12, 128, 256, None),
    ([1228, 1004, 0, 779], [4096, 3000, 2000, 3555], 24, 24, 128, 64, None),
    ([4096], [16384], 24, 24, 64, 64, None),
    ([2500, 700, 1, 40], [8192, 5000, 9000, 777], 24, 8, 64, 16, "token"),
    ([2100, 3000], [8000, 3000], 10, 2, 128, 32, "token"),
]


@pytest.mark.parametrize("rows,lens,heads,kv_heads,d,page,mask", AT_SIZE)
def test_long_chunks_at_size_on_sampled_rows(J, rows, lens, heads, kv_heads, d, page, mask):
    # more CTAs than SMs, the library's split; sampled rows (the tiles' first and last ones among them) of every
    # head against fp64 on the device
    gen = torch.Generator("cuda").manual_seed(sum(rows))
    n, per = sum(rows), [-(-m // page) for m in lens]
    k, v = (torch.full((sum(per) + 1, page, kv_heads, d), float("nan"), dtype=torch.bfloat16, device="cuda")
            for _ in range(2))
    order = torch.randperm(sum(per) + 1, generator=gen, device="cuda").int()
    table = torch.full((len(rows), max(per)), 2 ** 30, dtype=torch.int32, device="cuda")
    own = []
    for s, m in enumerate(lens):
        pages = order[sum(per[:s]):sum(per[:s + 1])]
        table[s, :per[s]] = pages
        kv = torch.randn((2, m, kv_heads, d), generator=gen, device="cuda").bfloat16()
        at = torch.arange(m, device="cuda")
        for t, x in zip((k, v), kv):
            t[pages.long()[at // page], at % page] = x
        own.append(kv)
    q = torch.randn((n, heads, d), generator=gen, device="cuda").bfloat16()
    cu = np.concatenate([[0], np.cumsum(rows)])
    pos = np.concatenate([np.arange(m - r, m) for r, m in zip(rows, lens)])
    limits = None if mask is None else pos + 1 if mask == "token" else (pos // mask + 1) * mask
    out = J.paged_attention(q, k, v, table, ints(lens), ints(cu), limits=None if limits is None else ints(limits))
    no_device_error(J)
    pick = np.random.default_rng(n)
    step, g, scale = 128 // (heads // kv_heads), heads // kv_heads, d ** -0.5
    for s, (r, m) in enumerate(zip(rows, lens)):
        if not r:
            continue
        edges = np.arange(0, r, step)
        take = np.unique(np.concatenate([pick.choice(edges, min(len(edges), 12), replace=False), pick.integers(0, r, 24),
                                         [0, min(step, r) - 1, r - 1]]))
        at = torch.from_numpy(cu[s] + take).cuda()
        lim = torch.full((len(take),), m, device="cuda")
        if limits is not None:
            lim = torch.from_numpy(np.minimum(limits[cu[s] + take], m)).cuda()
        hidden = torch.arange(m, device="cuda") >= lim[:, None]
        for h in range(heads):
            x, (kk, vv) = q[at, h].double(), own[s][:, :, h // g].double()
            w = torch.softmax((x @ kk.T * scale).masked_fill_(hidden, -torch.inf), 1)
            want, pv = w @ vv, w @ vv.abs()
            top = (x.abs() @ kk.abs().T).masked_fill_(hidden, 0.0).amax(1, keepdim=True) * scale
            # as check_attention, and the sums of O: 8 additions a key tile, each off by at most 2^-23
            bound = 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -15 * top + 2.0 ** -12 + m / 128 * 8 * 2.0 ** -23) * pv
            over = (out[at, h].double() - want).abs() - bound
            assert bool((over <= 0).all()), (s, h, float(over.max()), take[int(over.amax(1).argmax())])
