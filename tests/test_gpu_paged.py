"""GPU parity of the paged KV cache (append with the rotation on the way,
attention of a chunk of rows over the pages) against the fp64 oracle, through
the Python binding of the C ABI.  Tolerances: tests/paged_tools.py.  Places
that nobody owns or that lie past a sequence's length hold NaN throughout."""
import numpy as np
import pytest
import torch

import oracle.paged as op
import synth
from paged_tools import Paged, bits, check_attention, check_rope, f64

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


# ------------------------------------------------------------------ append
APPEND = [  # rows per sequence, lengths, heads, kv_heads, d, page, axes, halves, head_major, one_buffer
    ([1], [1], 2, 2, 64, 16, (16, 24, 24), False, False, False),
    ([5, 0, 130, 1], [77, 9, 130, 401], 6, 2, 128, 32, (44, 42, 42), False, False, True),
    ([3, 17], [100, 17], 24, 8, 128, 16, (16, 56, 56), True, True, False),
    ([40, 2], [300, 2], 3, 3, 96, 256, (12, 10, 20), False, True, False),
    ([9], [64], 4, 1, 64, 64, (16, 24, 24), False, False, True),
    ([64, 64, 64], [128, 64, 200], 8, 4, 128, 128, None, False, False, False),
    ([1] * 70, list(range(1, 71)), 2, 1, 64, 16, (20, 22, 22), False, False, False),
]


@pytest.mark.parametrize("rows,lens,heads,kv_heads,d,page,axes,halves,head_major,one_buffer", APPEND)
def test_append_matches_oracle_and_keeps_the_rest(J, rows, lens, heads, kv_heads, d, page, axes, halves, head_major,
                                                  one_buffer):
    p = Paged(rows, lens, heads, kv_heads, d, page, seed=sum(rows), head_major=head_major, one_buffer=one_buffer,
              pad_rows=3)
    gen = np.random.default_rng(7)
    n = int(p.cu[-1])
    # any rising positions of each sequence, the last one among them
    pos = np.concatenate([np.sort(np.append(gen.choice(m - 1, r - 1, replace=False), m - 1)) if r else []
                          for r, m in zip(rows, lens)] + [[0] * 3]).astype(np.int64)
    kv = synth.normal_bf16((n + 3, 2 * kv_heads, d), seed=n)
    k, v = kv.split(kv_heads, 1)
    dk, dv = kv.cuda().split(kv_heads, 1)
    r = table = coords = None
    if axes:
        r = J.Rope(axes=axes, n_pos=(5, 9, 16), grid=(9, 16), pairing="halves" if halves else "interleaved")
        table = J.rope_table(r)
        coords = op.grid_coords(pos, 9, 16)
    before = bits(p.dev_k), bits(p.dev_v)
    q_out = torch.full_like(p.dev_q, 5.0)
    got = J.paged_append(dk, dv, ints(pos), p.dev_k, p.dev_v, p.dev_table, p.dev_lens, p.dev_cu, rope=r, table=table,
                         q=p.dev_q, q_out=q_out)
    no_device_error(J)
    assert got is q_out
    assert bool((q_out[n:] == 5.0).all())                         # rows behind the last sequence
    seq = np.repeat(np.arange(len(rows)), rows)
    at = p.table[seq, pos[:n] // page], pos[:n] % page
    after = bits(p.dev_k), bits(p.dev_v)
    np.testing.assert_array_equal(after[1][at], bits(v)[:n])
    written = torch.from_numpy(after[0][at].view(np.int16)).view(torch.bfloat16)
    if axes:
        check_rope(written, k[:n], coords[:n], axes, halves=halves)
        check_rope(q_out[:n], p.q[:n], coords[:n], axes, halves=halves)
    else:
        np.testing.assert_array_equal(after[0][at], bits(k)[:n])
        np.testing.assert_array_equal(bits(q_out)[:n], bits(p.q)[:n])
    for old, new in zip(before, after):
        old[at] = new[at]
        np.testing.assert_array_equal(old, new)                   # every other place as it was


def test_append_takes_each_sequences_own_grid_and_the_queries_in_place(J):
    rows, lens = [4, 6], [40, 60]
    p = Paged(rows, lens, 4, 2, 64, 16, seed=3)
    pos = np.concatenate([np.arange(36, 40), np.arange(54, 60)])
    grids = np.array([[2, 5], [6, 3]])
    coords = np.concatenate([op.grid_coords(pos[:4], 2, 5), op.grid_coords(pos[4:], 6, 3)])
    r = J.Rope(axes=(16, 24, 24), n_pos=(5, 6, 5))
    table = J.rope_table(r)
    k = synth.normal_bf16((10, 2, 64), seed=4)
    kw = dict(rope=r, table=table)
    args = (k.cuda(), k.cuda(), ints(pos), p.dev_k, p.dev_v, p.dev_table, p.dev_lens, p.dev_cu)
    q = p.dev_q.clone()
    assert J.paged_append(*args, q=q, q_out=q, grids=ints(grids), **kw) is q
    no_device_error(J)
    check_rope(q, p.q, coords, (16, 24, 24))
    same = J.paged_append(*args, q=p.dev_q, coords=ints(coords), **kw)
    assert torch.equal(same, q)
    J.paged_append(*args, grids=ints([[2, 5], [6, 0]]), **kw)     # a grid without columns
    assert J.device_error() == 6


def test_append_finds_the_sequence_among_many(J):
    # 1,100 sequences (two levels of the search), empty ones among them
    rows = [(s * 7 + 3) % 4 for s in range(1100)]
    lens = [max(1, r) for r in rows]
    p = Paged(rows, lens, 1, 1, 64, 16, seed=11)
    n = int(p.cu[-1])
    pos = np.concatenate([np.arange(r) for r in rows])
    v = synth.normal_bf16((n, 1, 64), seed=12)
    J.paged_append(v.cuda(), v.cuda(), ints(pos), p.dev_k, p.dev_v, p.dev_table, p.dev_lens, p.dev_cu)
    no_device_error(J)
    seq = np.repeat(np.arange(len(rows)), rows)
    np.testing.assert_array_equal(bits(p.dev_v)[p.table[seq, pos // 16], pos % 16], bits(v))


def test_append_skips_and_reports_bad_rows(J):
    p = Paged([6, 2], [40, 20], 2, 2, 64, 16, seed=5)
    table = p.table.copy()
    table[1, 1] = p.n_pages                                       # sequence 1's second page: outside the pool
    pos = [3, 3, 2, 5, 40, -1, 4, 18]                             # duplicate, step back, past the length, negative, bad page
    k = synth.normal_bf16((8, 2, 64), seed=6).cuda()
    before = p.dev_k.clone()
    q_out = torch.full((8, 2, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    J.paged_append(k, k, ints(pos), p.dev_k, p.dev_v, ints(table), p.dev_lens, p.dev_cu, q=k, q_out=q_out)
    assert J.device_error() == 6
    assert [i for i in range(8) if bool((q_out[i] == 5.0).all())] == [1, 2, 4, 5, 7]
    changed = (p.dev_k.view(torch.int16) != before.view(torch.int16)).any(-1).any(-1).nonzero().cpu().numpy()
    want = sorted((int(p.table[s, x // 16]), x % 16) for s, x in ((0, 3), (0, 5), (1, 4)))
    assert [tuple(c) for c in changed.tolist()] == want
    # row lists that do not rise from 0
    for cu in ([1, 6, 8], [0, 7, 5], [-3, 6, 8]):
        J.paged_append(k, k, ints([0, 1, 2, 3, 4, 5, 6, 7]), p.dev_k, p.dev_v, p.dev_table, p.dev_lens, ints(cu))
        assert J.device_error() == 6, cu


# ------------------------------------------------------------------ attention
ATTEND = [  # rows, lengths, heads, kv_heads, d, page, limits, options
    ([1], [1], 1, 1, 64, 16, None, {}),
    ([1], [129], 4, 4, 128, 16, None, {}),
    ([1, 1, 1], [1, 128, 700], 8, 2, 128, 16, None, {}),
    ([3, 0, 7], [130, 50, 31], 6, 2, 64, 16, "token", {}),
    ([61, 44], [777, 44], 6, 6, 64, 32, "token", {}),
    ([130], [400], 2, 2, 128, 64, "token", {}),
    ([300, 5], [300, 1000], 2, 1, 128, 128, "token", {}),
    ([257, 1], [513, 2049], 3, 3, 128, 128, None, {}),
    ([40], [640], 3, 3, 64, 256, "random", {}),
    ([50, 30], [256, 383], 6, 1, 128, 64, "random", {}),          # 21 rows of 6 heads in a tile
    ([9, 90], [90, 300], 10, 2, 64, 32, "token", {}),             # 25 rows of 5 heads
    ([3, 2], [200, 150], 128, 1, 64, 16, None, {}),               # one row fills a tile
    ([2, 3], [140, 260], 65, 1, 128, 16, "token", {}),            # 65 of 128 tile rows
    ([20, 20], [300, 200], 4, 2, 128, 32, "token", dict(head_major=True)),
    ([20, 140], [300, 200], 4, 4, 64, 64, None, dict(one_buffer=True, pad_rows=5)),
    ([4, 0, 3], [0, 0, 12], 2, 2, 64, 16, None, dict(pad_rows=2)),     # an empty cache
]


def limits_of(kind, rows, lens, seed=0):
    if kind is None:
        return None
    gen = np.random.default_rng(seed)
    if kind == "token":
        return np.concatenate([np.arange(m - r, m) + 1 for r, m in zip(rows, lens)]).astype(np.int64)
    # any order, rows that see nothing (0 and below) and more than there is
    out = np.concatenate([gen.integers(-3, m + 9, r) for r, m in zip(rows, lens)])
    out[::7] = 0
    return out


@pytest.mark.parametrize("split", [0, 1, 2, 4, 8])
@pytest.mark.parametrize("rows,lens,heads,kv_heads,d,page,kind,opt", ATTEND)
def test_attention_matches_oracle(J, rows, lens, heads, kv_heads, d, page, kind, opt, split):
    p = Paged(rows, lens, heads, kv_heads, d, page, seed=sum(lens), **opt)
    limits = limits_of(kind, rows, lens)
    if limits is not None and opt.get("pad_rows"):
        limits = np.concatenate([limits, np.zeros(opt["pad_rows"], dtype=limits.dtype)])
    out = torch.full_like(p.dev_q, 3.0)
    got = attend(J, p, limits, out=out, split=split)
    no_device_error(J)
    assert got is out
    p.check(out, limits)
    assert bool((out[int(p.cu[-1]):] == 3.0).all())               # rows behind the last sequence


FEW = [  # at most 32 packed rows per sequence: the form in which every SM takes an equal share of the key tiles
    ([1], [1], 1, 1, 64, 16, None, {}),
    ([1], [128], 1, 1, 128, 128, None, {}),
    ([1], [129], 3, 3, 128, 16, None, {}),
    ([1], [5000], 2, 2, 64, 64, None, {}),                             # two items cut over some twenty CTAs each
    ([1, 1, 1], [700, 128, 1], 8, 2, 128, 16, None, {}),
    ([2, 0, 2, 1], [130, 50, 31, 2000], 10, 1, 64, 32, "token", {}),   # 20 of 32 rows, one sequence without any
    ([1, 1], [3, 300], 32, 1, 128, 256, None, {}),
    ([32, 5, 17], [257, 383, 40], 2, 2, 128, 64, "random", {}),
    ([8, 8], [600, 90], 12, 3, 64, 16, "random", dict(head_major=True)),
    ([1] * 70, [(s * 97) % 400 + 1 for s in range(70)], 4, 2, 64, 16, None, dict(pad_rows=3)),   # three looks of 32
    ([1] * 40, [1] * 40, 2, 2, 128, 16, None, {}),                     # fewer tiles than SMs
    ([1] * 20, [(s * 331) % 2200 + 1 for s in range(20)], 16, 8, 64, 16, None, {}),   # 160 items: shares go across them
    ([1, 2, 1, 1, 3], [4000, 1, 700, 2300, 129], 6, 3, 128, 64, "random", {}),        # shares that end with their item
    ([1] * 9, [1300] * 8 + [3], 32, 2, 64, 32, None, {}),              # 16 rows: MMAs of 64 rows
    ([17], [3000], 1, 1, 64, 64, "random", {}),                        # 17: of 128
    ([2, 1, 1], [0, 0, 5], 2, 2, 64, 16, None, dict(one_buffer=True, pad_rows=2)),
    ([3, 3], [300, 200], 6, 2, 128, 32, "dark", {}),                   # a sequence whose rows all see nothing
]


@pytest.mark.parametrize("rows,lens,heads,kv_heads,d,page,kind,opt", FEW)
def test_few_rows_match_oracle(J, rows, lens, heads, kv_heads, d, page, kind, opt):
    p = Paged(rows, lens, heads, kv_heads, d, page, seed=sum(lens), **opt)
    n = int(p.cu[-1])
    limits = limits_of(None if kind == "dark" else kind, rows, lens)
    if kind == "dark":
        limits = np.array([5, 300, 77, 0, -4, 0])
    if limits is not None and opt.get("pad_rows"):
        limits = np.concatenate([limits, np.zeros(opt["pad_rows"], dtype=limits.dtype)])
    need = J.jano_paged_attention_workspace_bytes(max(rows), heads, kv_heads, d)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert need == 2 * sms * max(rows) * heads // kv_heads * (d + 2) * 4
    # garbage in the workspace, as a reused buffer would hold
    ws = torch.full((need // 4,), float("nan"), dtype=torch.float32, device="cuda").view(torch.uint8)
    outs = []
    for kw in (dict(workspace=ws), dict(workspace=ws, max_len=max(max(lens), 1)), {}):
        out = torch.full_like(p.dev_q, 3.0)
        attend(J, p, limits, out=out, max_rows=max(rows), **kw)
        no_device_error(J)
        p.check(out, limits)
        assert bool((out[n:] == 3.0).all())
        outs.append(out)
    assert all(torch.equal(o, outs[0]) for o in outs)             # the same sums in the same order


@pytest.mark.parametrize("split", [0, 1, 2])
def test_a_bad_sequence_late_in_a_long_list_is_reported(J, split):
    n = 300                                             # sequences; the 128-at-a-time search crosses three groups
    p = Paged([1 + s % 2 for s in range(n)], [(s * 37) % 150 + 1 for s in range(n)], 2, 1, 64, 16, seed=5)
    want = attend(J, p, max_rows=2, split=split).clone()
    no_device_error(J)
    p.check(want)
    lens = np.array(p.lens)
    lens[283] = -1
    out = torch.full_like(p.dev_q, 3.0)
    J.paged_attention(p.dev_q, p.dev_k, p.dev_v, p.dev_table, ints(lens), p.dev_cu, out=out, max_rows=2, split=split)
    assert J.device_error() == 6
    bad = slice(int(p.cu[283]), int(p.cu[284]))
    assert bool((out[bad] == 3.0).all())
    out[bad] = want[bad]
    p.check(out)


def test_few_rows_report_bad_lists_and_need_their_workspace(J):
    p = Paged([1, 2], [100, 200], 2, 2, 64, 16, seed=12)
    out = torch.full_like(p.dev_q, 3.0)
    want = attend(J, p, max_rows=2).clone()
    for kw, dark in ((dict(lens=[100, -1]), slice(1, 3)), (dict(lens=[10 ** 9, 200]), slice(0, 1)),
                     (dict(cu=[0, 1, 4]), slice(1, 3)), (dict(cu=[2, 3, 3]), slice(0, 2))):
        out.fill_(3.0)
        J.paged_attention(p.dev_q, p.dev_k, p.dev_v, p.dev_table, ints(kw["lens"]) if "lens" in kw else p.dev_lens,
                          ints(kw["cu"]) if "cu" in kw else p.dev_cu, out=out, max_rows=2)
        assert J.device_error() == 6, kw
        assert bool((out[dark] == 3.0).all()), kw
    table = p.table.copy()
    table[0, 2] = p.n_pages
    J.paged_attention(p.dev_q, p.dev_k, p.dev_v, ints(table), p.dev_lens, p.dev_cu, out=out, max_rows=2)
    assert J.device_error() == 6
    assert torch.equal(out[1:], want[1:]) and torch.isfinite(out.float()).all()
    with pytest.raises(J.JanoError, match="EINVAL"):
        attend(J, p, max_rows=2, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(TypeError, match="uint8"):
        attend(J, p, max_rows=2, workspace=torch.empty(10 ** 6, device="cuda"))
    no_device_error(J)


def test_few_rows_calls_at_once_on_streams_and_replayed(J):
    cases = [Paged([1, 1, 1], [1500 + 300 * i, 77, 900], 4, 2, 128, 32, seed=20 + i) for i in range(4)]
    want = [attend(J, p, max_rows=1).clone() for p in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [[attend(J, p, max_rows=1, stream=s) for p, s in zip(cases, streams)] for _ in range(5)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for r in outs for o, w in zip(r, want))
    # two graphs, captured one after the other, replayed together
    graphs, res = [], []
    for p, s in zip(cases[:2], streams):
        o = torch.zeros_like(p.dev_q)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            for _ in range(3):
                attend(J, p, max_rows=1, out=o)
        graphs.append(g)
        res.append(o)
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    no_device_error(J)
    assert torch.equal(res[0], want[0]) and torch.equal(res[1], want[1])
    del graphs, g


def test_attention_takes_strided_rows_and_bounds(J):
    p = Paged([33, 70], [210, 333], 4, 2, 64, 32, seed=8)
    wide = torch.zeros(p.n, 3 * 4, 64, dtype=torch.bfloat16, device="cuda")
    wide[:, 4:8] = p.dev_q
    out = torch.full_like(wide, 2.0)
    J.paged_attention(wide[:, 4:8], p.dev_k, p.dev_v, p.dev_table, p.dev_lens, p.dev_cu, out=out[:, 8:],
                      max_rows=70, max_len=333, scale=0.3)
    no_device_error(J)
    p.check(out[:, 8:].contiguous(), scale=0.3)
    assert bool((out[:, :8] == 2.0).all())


def test_logits_over_many_binades(J):
    # rising maxima: every tile makes the running maximum grow by more than the
    # lazy rescale allows, in order, reversed and shuffled
    for seed, order in enumerate((np.arange(640), np.arange(640)[::-1], np.random.default_rng(1).permutation(640))):
        p = Paged([130, 2], [640, 640], 2, 2, 128, 64, seed=seed)
        scale_of = (0.25 * 2.0 ** (np.arange(640) / 100.0))[order].astype(np.float32)
        for s in range(2):
            for j in range(640):
                p.k[p.table[s, j // 64], j % 64] = p.q[0, :1] * float(scale_of[j])
        p.dev_k = p.k.cuda()
        out = attend(J, p)
        no_device_error(J)
        p.check(out)


def test_places_past_the_length_may_hold_anything(J):
    p = Paged([5, 140], [131, 260], 4, 2, 128, 64, seed=9)
    want = attend(J, p)
    for fill in (float("inf"), -float("inf"), 0.0, 3e38):
        k, v = p.k.clone(), p.v.clone()
        for t in (k, v):
            t[torch.isnan(t)] = fill
        got = J.paged_attention(p.dev_q, k.cuda(), v.cuda(), p.dev_table, p.dev_lens, p.dev_cu)
        assert torch.equal(got, want), fill
    # and past what the rows' limits let the tile see
    limits = np.minimum(np.arange(145) % 60, 37)
    want = attend(J, p, limits)
    k, v = p.k.clone(), p.v.clone()
    for s in range(2):
        for j in range(37, p.lens[s]):
            k[p.table[s, j // 64], j % 64] = float("nan")
            v[p.table[s, j // 64], j % 64] = float("nan")
    got = J.paged_attention(p.dev_q, k.cuda(), v.cuda(), p.dev_table, p.dev_lens, p.dev_cu, limits=ints(limits))
    no_device_error(J)
    assert torch.equal(got, want)
    p.check(want, limits)


def test_sequences_may_share_pages(J):
    p = Paged([3, 3], [200, 128], 2, 2, 64, 64, seed=10)
    table = p.table.copy()
    table[1, :2] = table[0, :2]                                   # a common prefix of 128 positions
    out = J.paged_attention(p.dev_q, p.dev_k, p.dev_v, ints(table), p.dev_lens, p.dev_cu)
    no_device_error(J)
    k, v = p.seq(0)
    check_attention(out[:3], f64(p.q[:3]), k, v, np.full(3, 200), 0.125)
    check_attention(out[3:], f64(p.q[3:]), k[:128], v[:128], np.full(3, 128), 0.125)


def test_bad_lists_raise_eindex_and_write_no_row(J):
    p = Paged([4, 4], [100, 200], 2, 2, 64, 16, seed=11)
    call = lambda **kw: J.paged_attention(*[kw.get(n, x) for n, x in (
        ("q", p.dev_q), ("k", p.dev_k), ("v", p.dev_v), ("table", p.dev_table), ("lens", p.dev_lens),
        ("cu", p.dev_cu))], out=out, max_rows=kw.get("max_rows"), max_len=kw.get("max_len"))
    out = torch.full_like(p.dev_q, 3.0)
    want = call().clone()
    no_device_error(J)
    for kw, dark in ((dict(lens=ints([100, -1])), [1]), (dict(lens=ints([2 ** 30, 200])), [0]), (dict(max_len=150), [1]),
                     (dict(max_rows=3), [0, 1]), (dict(cu=ints([0, 4, 9])), [1]), (dict(cu=ints([0, -4, 8])), [0, 1]),
                     (dict(cu=ints([0, 8, 4])), [])):              # sequence 0 owns all eight rows here
        out.fill_(3.0)
        call(**kw)
        assert J.device_error() == 6, kw
        for s in dark:
            assert bool((out[4 * s:4 * s + 4] == 3.0).all()), kw
        if dark == [1]:
            assert torch.equal(out[:4], want[:4]), kw
    # a page id outside the pool: reported, reads as zeros, the other sequence is right
    table = p.table.copy()
    table[1, 3] = -5
    table[1, 4] = 2 ** 31 - 1
    call(table=ints(table))
    assert J.device_error() == 6
    assert torch.equal(out[:4], want[:4]) and torch.isfinite(out.float()).all()


def test_pool_past_32_bit_offsets(J):
    # the last pages of a pool of 2^31 + elements per buffer
    page, h, d = 256, 8, 128
    n_pages = 2 ** 31 // (page * h * d) + 6
    k, v = J.page_pool(n_pages, page, h, d)
    lens, rows = [700, 300], [2, 1]
    ids = np.full((2, 4), -1, dtype=np.int32)
    ids[0, :3] = [n_pages - 1, 0, n_pages - 3]
    ids[1, :2] = [n_pages - 2, n_pages - 4]
    cu, ln, table = ints([0, 2, 3]), ints(lens), ints(ids)
    kv = synth.normal_bf16((1000, 2 * h, d), seed=13)
    pos = np.concatenate([np.arange(700), np.arange(300)])
    dk, dv = kv.cuda().split(h, 1)
    J.paged_append(dk, dv, ints(pos), k, v, table, ln, ints([0, 700, 1000]))
    q = synth.normal_bf16((3, h, d), seed=14)
    out = J.paged_attention(q.cuda(), k, v, table, ln, cu)
    no_device_error(J)
    for a, b, rows_ in ((0, 700, slice(0, 2)), (700, 1000, slice(2, 3))):
        check_attention(out[rows_], f64(q[rows_]), f64(kv[a:b, :h]), f64(kv[a:b, h:]),
                        np.full(rows_.stop - rows_.start, b - a), d ** -0.5)


def test_runs_are_bit_identical_and_streams_independent(J):
    p = Paged([1, 200, 33], [1500, 700, 33], 4, 2, 128, 32, seed=15)
    limits = limits_of("token", [1, 200, 33], [1500, 700, 33])
    want = attend(J, p, limits)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    lim = ints(limits)
    torch.cuda.synchronize()
    outs = [J.paged_attention(p.dev_q, p.dev_k, p.dev_v, p.dev_table, p.dev_lens, p.dev_cu, limits=lim, stream=s)
            for _ in range(4) for s in streams]
    torch.cuda.synchronize()
    no_device_error(J)
    assert all(torch.equal(o, want) for o in outs)


def test_replayed_graph_follows_its_lists(J):
    # one captured launch pair (append, attention); between replays the lengths,
    # positions, page table and rows change on the device
    p = Paged([2, 2], [90, 140], 4, 2, 64, 32, seed=16)
    rows = np.array([2, 2])
    r = J.Rope(axes=(16, 24, 24), n_pos=(4, 8, 16), grid=(8, 16))
    table = J.rope_table(r)
    pos, k = torch.zeros(4, dtype=torch.int32, device="cuda"), synth.normal_bf16((4, 2, 64), seed=17).cuda()
    q, out = torch.empty_like(p.dev_q), torch.empty_like(p.dev_q)
    lens = p.dev_lens.clone()
    run = lambda: (J.paged_append(k, k, pos, p.dev_k, p.dev_v, p.dev_table, lens, p.dev_cu, rope=r, table=table,
                                  q=p.dev_q, q_out=q),
                   J.paged_attention(q, p.dev_k, p.dev_v, p.dev_table, lens, p.dev_cu, out=out))
    pos.copy_(ints([88, 89, 138, 139]))
    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for step, ln in enumerate(([90, 140], [33, 160], [2, 2])):
        k.copy_(synth.normal_bf16((4, 2, 64), seed=20 + step).cuda())
        new = np.concatenate([np.arange(m - n, m) for n, m in zip(rows, ln)])
        if ln[1] == 160:
            p.table[1, 4] = p.table[1, 0]                         # a fifth page for the second sequence
            p.table[1, 0] = [x for x in range(p.n_pages) if x not in p.table[:, :5]][0]
            fill = synth.normal_bf16((32, 2, 64), seed=30).cuda()
            p.dev_k[int(p.table[1, 0])], p.dev_v[int(p.table[1, 0])] = fill, fill
            p.dev_table.copy_(ints(p.table))
        pos.copy_(ints(new))
        lens.copy_(ints(ln))
        g.replay()
        torch.cuda.synchronize()
        no_device_error(J)
        kc, vc = p.dev_k.cpu(), p.dev_v.cpu()
        for s in range(2):
            ks, vs = (op.gather(f64(t), p.table[s], ln[s]) for t in (kc, vc))
            check_attention(out[2 * s:2 * s + 2], f64(q[2 * s:2 * s + 2]), ks, vs, np.full(2, ln[s]), 0.125)
    del g


@pytest.mark.parametrize("page,d", [(16, 128), (128, 64)])
def test_paged_path_equals_the_contiguous_one(J, page, d):
    # a generation's due tokens through both caches: rope_scatter and
    # active_attention, paged_append and paged_attention
    gen = np.random.default_rng(1)
    N, heads, n = 1000, 4, 301
    axes = (16, 24, 24) if d == 64 else (44, 42, 42)
    r = J.Rope(axes=axes, n_pos=(2, 20, 25), grid=(20, 25))
    table = J.rope_table(r)
    idx = ints(np.sort(gen.choice(N, n, replace=False)))
    q, k, v = (synth.normal_bf16((n, heads, d), seed=s).cuda() for s in (1, 2, 3))
    kc, vc = (synth.normal_bf16((N, heads, d), seed=s).cuda() for s in (4, 5))
    n_pages = -(-N // page)
    kp, vp = J.page_pool(n_pages + 2, page, heads, d)
    kp.fill_(float("nan")), vp.fill_(float("nan"))
    order = gen.permutation(n_pages + 2)[:n_pages]
    pages, lens = ints(order[None]), ints([N])
    everyone = torch.arange(N, dtype=torch.int32, device="cuda")
    J.paged_append(kc, vc, everyone, kp, vp, pages, lens, ints([0, N]))
    qr = J.rope_scatter(k, v, idx, kc, vc, r, table, q=q)
    qp = J.paged_append(k, v, idx, kp, vp, pages, lens, ints([0, n]), rope=r, table=table, q=q)
    assert torch.equal(qr, qp)
    flat = kp[torch.from_numpy(order).cuda()].reshape(-1, heads, d)[:N]
    assert torch.equal(flat.view(torch.int16), kc.view(torch.int16))
    out = torch.zeros(N, heads, d, dtype=torch.bfloat16, device="cuda")
    J.active_attention(qr, kc, vc, idx, out)
    got = J.paged_attention(qp, kp, vp, pages, lens, ints([0, n]))
    no_device_error(J)
    check_attention(got, f64(qp), f64(kc), f64(vc), np.full(n, N), d ** -0.5)
    check_attention(out[idx.long()], f64(qr), f64(kc), f64(vc), np.full(n, N), d ** -0.5)
