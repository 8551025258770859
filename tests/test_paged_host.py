"""The rotary and paged entry points refuse bad calls on the host, before any
launch; and the fp64 oracle they are tested against is pinned by hand-worked
values.  No GPU is needed."""
import ctypes as C
import os

import numpy as np
import pytest
import torch

import kv_cache_analyzer_b200.paged as P
import oracle.paged as op
from paged_tools import Paged

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
EINVAL, ESHAPE, EALIGN, EUNSUPPORTED = 1, 2, 3, 4


@pytest.fixture(scope="module")
def J():
    from kv_cache_analyzer_b200 import build
    build.build()
    import kv_cache_analyzer_b200 as j
    return j


fake, nil = C.c_void_p(256), None          # never dereferenced: validation fails first
odd = C.c_void_p(264)


def cfg(J, axes=(16, 24, 24), n_pos=(2, 5, 7), grid=(5, 7), halves=0):
    return bytes(J.jano_rope_cfg((C.c_int * 3)(*axes), (C.c_int * 3)(*n_pos), *grid, halves))


def test_rope_table_refusals(J):
    L = J.lib()
    assert L.jano_rope_table_floats(cfg(J)) == 2 * 16 + 5 * 24 + 7 * 24
    for bad in (dict(axes=(15, 24, 24)), dict(axes=(-2, 24, 24)), dict(axes=(0, 0, 0)), dict(n_pos=(0, 5, 7)),
                dict(n_pos=(2 ** 30, 2 ** 30, 7)), dict(axes=(4, 2, 2), halves=1)):
        assert L.jano_rope_table_floats(cfg(J, **bad)) == 0, bad
        assert L.jano_rope_table(cfg(J, **bad), 10000.0, 0, fake, nil) in (EINVAL, EUNSUPPORTED), bad
    for theta in (0.0, -1.0, float("nan"), float("inf")):
        assert L.jano_rope_table(cfg(J), theta, 0, fake, nil) == EINVAL
    assert L.jano_rope_table(cfg(J), 10000.0, 0, nil, nil) == EINVAL
    assert L.jano_rope_table(cfg(J), 10000.0, 0, C.c_void_p(260), nil) == EALIGN
    assert L.jano_rope_table(None, 10000.0, 0, fake, nil) == EINVAL


def test_axis_rope_refusals(J):
    L = J.lib()
    call = lambda x=fake, x_ld=256, ids=fake, coords=nil, n=8, heads=4, d=64, c=None, table=fake, out=fake, o_ld=256: \
        L.jano_axis_rope(x, x_ld, ids, coords, n, heads, d, c or cfg(J), table, out, o_ld, nil)
    assert call(n=0, x=nil, out=nil, table=nil) == 0
    assert call(n=-1) == EINVAL and call(heads=0) == EINVAL and call(d=0) == EINVAL
    assert call(x=nil) == EINVAL and call(out=nil) == EINVAL and call(table=nil) == EINVAL
    assert call(x_ld=248) == ESHAPE and call(o_ld=255) == ESHAPE
    assert call(x_ld=260) == EUNSUPPORTED and call(o_ld=257) == EUNSUPPORTED
    assert call(x=odd) == EALIGN and call(out=odd) == EALIGN and call(table=C.c_void_p(260)) == EALIGN
    assert call(d=32, x_ld=128, o_ld=128) == EINVAL                      # more rotated columns than a head has
    assert call(d=68, x_ld=272, o_ld=272) == EUNSUPPORTED                # not whole 16-byte vectors
    assert call(d=2048, x_ld=8192, o_ld=8192) == EUNSUPPORTED
    assert call(c=cfg(J, grid=(0, 7))) == EINVAL                         # ids without a grid
    assert call(c=cfg(J, axes=(4, 2, 2), halves=1)) == EUNSUPPORTED      # 8 rotated columns cannot be split in vectors


def test_rope_scatter_refusals(J):
    L = J.lib()
    a = dict(q=fake, q_ld=256, k=fake, k_ld=128, v=fake, v_ld=128, idx=fake, coords=nil, n=8, heads=4, kv=2, d=64, c=None,
             table=fake, q_out=fake, o_ld=256, kc=fake, vc=fake, N=100)

    def call(**kw):
        b = {**a, **kw}
        return L.jano_rope_scatter(b["q"], b["q_ld"], b["k"], b["k_ld"], b["v"], b["v_ld"], b["idx"], b["coords"], b["n"],
                                   b["heads"], b["kv"], b["d"], b["c"] or cfg(J), b["table"], b["q_out"], b["o_ld"],
                                   b["kc"], b["vc"], b["N"], nil)
    assert call(n=0, k=nil, idx=nil) == 0
    for kw in (dict(n=-1), dict(N=0), dict(kv=0), dict(k=nil), dict(v=nil), dict(idx=nil), dict(table=nil), dict(kc=nil),
               dict(q=nil), dict(q_out=nil), dict(c=cfg(J, axes=(32, 32, 32)))):
        assert call(**kw) == EINVAL, kw
    for kw in (dict(q_ld=248), dict(k_ld=120), dict(v_ld=64), dict(o_ld=0)):
        assert call(**kw) == ESHAPE, kw
    for kw in (dict(k=odd), dict(v=odd), dict(q=odd), dict(kc=odd), dict(vc=odd)):
        assert call(**kw) == EALIGN, kw
    assert call(v_ld=132) == EUNSUPPORTED


def pool(J, **kw):
    a = dict(k=256, v=256, n_pages=9, page_size=16, kv_heads=2, d=64, page_stride=2048, token_stride=128,
             head_stride=64)
    a.update(kw)
    return bytes(J.jano_page_pool(*a.values()))


def seqs(J, **kw):
    a = dict(page_table=256, seq_lens=256, cu_rows=256, n_seqs=3, max_pages=8)
    a.update(kw)
    return bytes(J.jano_page_seqs(*a.values()))


POOLS = [(dict(k=None), EINVAL), (dict(n_pages=0), EINVAL), (dict(kv_heads=0), EINVAL), (dict(page_size=8), EUNSUPPORTED),
         (dict(page_size=48), EUNSUPPORTED), (dict(page_size=512), EUNSUPPORTED), (dict(token_stride=32), ESHAPE),
         (dict(head_stride=-64), ESHAPE), (dict(page_stride=2052), EUNSUPPORTED),
         (dict(page_stride=1 << 40), EUNSUPPORTED), (dict(v=264), EALIGN)]
SEQS = [(dict(page_table=None), EINVAL), (dict(seq_lens=None), EINVAL), (dict(cu_rows=None), EINVAL),
        (dict(n_seqs=0), EINVAL), (dict(max_pages=0), EINVAL), (dict(max_pages=2 ** 28), EUNSUPPORTED)]


def test_paged_append_refusals(J):
    L = J.lib()

    def call(p=None, s=None, q=fake, q_ld=256, k=fake, k_ld=128, v=fake, v_ld=128, pos=fake, grids=nil, n=8, heads=4,
             c=cfg(J), table=fake, q_out=fake, o_ld=256):
        return L.jano_paged_append(p or pool(J), s or seqs(J), q, q_ld, k, k_ld, v, v_ld, pos, nil, grids, n, heads, c,
                                   table, q_out, o_ld, nil)
    assert call(n=0, k=nil) == 0 and call(n=-1) == EINVAL
    for kw, code in POOLS:
        assert call(p=pool(J, **kw)) == code, kw
    for kw, code in SEQS:
        assert call(s=seqs(J, **kw)) == code, kw
    for kw in (dict(c=None), dict(table=nil), dict(pos=nil), dict(k=nil), dict(q=nil), dict(c=cfg(J, grid=(0, 0)))):
        assert call(**kw) == EINVAL, kw
    assert call(k_ld=64) == ESHAPE and call(v=odd) == EALIGN and call(q_ld=252) == ESHAPE
    assert call(p=pool(J, d=60, token_stride=120, head_stride=64)) == EINVAL          # rotates more than a head
    assert call(p=pool(J, d=68, token_stride=144, head_stride=72), k_ld=144) == EUNSUPPORTED


def test_paged_attention_refusals(J):
    L = J.lib()

    def call(p=None, s=None, q=fake, q_ld=256, n=8, max_rows=8, max_len=128, heads=4, scale=0.125, split=0, ws=nil,
             out=fake, o_ld=256):
        return L.jano_paged_attention(p or pool(J), s or seqs(J), q, q_ld, nil, n, max_rows, max_len, heads, scale, split,
                                      ws, 0, out, o_ld, nil)
    assert call(n=0, q=nil) == 0 and call(n=-1) == EINVAL and call(max_len=-1) == EINVAL and call(max_rows=-1) == EINVAL
    assert call(max_len=2 ** 26 + 1) == EUNSUPPORTED
    for kw, code in POOLS:
        assert call(p=pool(J, **kw)) == code, kw
    for kw, code in SEQS:
        assert call(s=seqs(J, **kw)) == code, kw
    for kw in (dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(split=3), dict(split=16),
               dict(split=-1), dict(q=nil), dict(out=nil), dict(heads=0)):
        assert call(**kw) == EINVAL, kw
    assert call(heads=3, q_ld=192, o_ld=192) == ESHAPE                    # not a multiple of the K/V heads
    assert call(heads=258, q_ld=258 * 64, o_ld=258 * 64) == EUNSUPPORTED  # 129 query heads per K/V head
    assert call(p=pool(J, d=96, token_stride=192, head_stride=96), q_ld=384, o_ld=384) == EUNSUPPORTED
    assert call(q_ld=128) == ESHAPE and call(o_ld=260) == EUNSUPPORTED and call(q=odd) == EALIGN
    assert call(ws=odd) == EALIGN


def test_split_choice_is_host_only(J):
    f = J.jano_paged_attention_splits_on
    assert f(75600, 75600, 75600, 1, 40, 40, 148) == 1            # enough query tiles to fill the SMs
    assert f(1, 1, 128, 1, 24, 24, 148) == 1                      # one key tile
    assert f(1, 1, 75600, 1, 8, 8, 148) == 8                      # eight heads, 591 key tiles
    # the best of the measured splits: 12 heads over 32,760 keys, 4 heads over 8,192
    assert [f(n, n, 32760, 1, 12, 12, 148) for n in (1638, 3276, 4680, 16380)] == [4, 4, 4, 2]
    assert f(1000, 1000, 8192, 1, 4, 4, 148) == 4 and f(4 * 256, 256, 2048, 4, 12, 12, 148) == 2
    assert f(0, 1, 128, 1, 4, 4, 148) == 1 and f(1, 1, 128, 1, 4, 3, 148) == 1 and f(1, 1, 128, 1, 129, 1, 148) == 1
    for n in (1, 33, 1000):
        for length in (1, 200, 5000, 75600):
            for kv in (1, 8, 40):
                z = f(n, n, length, 1, kv, kv, 148)
                assert z in (1, 2, 4, 8) and z <= -(-length // 128)


def test_python_refusals_need_no_gpu(J):
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    r = J.Rope(axes=(16, 24, 24), n_pos=(2, 5, 7), grid=(5, 7))
    table = torch.zeros(r.entries, 2)
    with pytest.raises(ValueError, match="CUDA tensor"):
        J.axis_rope(x, r, table)
    with pytest.raises(ValueError, match=r"\[rows\]\[heads\]\[d\]"):
        J.axis_rope(x[0], r, table)
    rows = lambda t, n=4, h=2, d=64: P._rows(t, "x", -1, n, h, d)         # as on device -1
    with pytest.raises(TypeError, match="bfloat16"):
        rows(x.float())
    with pytest.raises(ValueError, match="adjacent"):
        rows(x.transpose(1, 2), h=64, d=2)
    with pytest.raises(ValueError, match=r"\[4\]\[3\]\[64\]"):
        rows(x, h=3)
    with pytest.raises(TypeError, match="int32"):
        P._list(torch.zeros(4), "ids", 4, -1)
    with pytest.raises(ValueError, match="5 elements"):
        P._list(torch.zeros(4, dtype=torch.int32), "ids", 5, -1)
    with pytest.raises(ValueError, match="contiguous"):
        P._list(torch.zeros(8, dtype=torch.int32)[::2], "ids", 4, -1)
    with pytest.raises(ValueError, match="cuda:3"):                       # another device than the first tensor's
        P._list(torch.zeros(4, dtype=torch.int32), "ids", 4, 3)
    with pytest.raises(ValueError, match="pairing"):
        J.Rope(axes=(16, 24, 24), n_pos=(2, 5, 7), pairing="quarters")
    with pytest.raises(ValueError, match="three entries"):
        J.Rope(axes=(16, 24), n_pos=(2, 5, 7))
    p = Paged([2, 2], [20, 30], 2, 2, 64, 16, dev=None)
    ints = lambda a: torch.from_numpy(np.asarray(a, dtype=np.int32))
    with pytest.raises(ValueError, match="CUDA tensor"):
        J.paged_attention(p.q, p.k, p.v, ints(p.table), ints(p.lens), ints(p.cu))
    with pytest.raises(ValueError, match="CUDA tensor"):
        J.paged_append(p.q, p.q, ints([0, 1, 2, 3]), p.k, p.v, ints(p.table), ints(p.lens), ints(p.cu))
    with pytest.raises(ValueError, match="same strides"):
        P._pool(p.k, p.v.transpose(1, 2).contiguous().transpose(1, 2), -1)
    with pytest.raises(TypeError, match="v_pages must be torch.bfloat16"):
        P._pool(p.k, p.v.float(), -1)


def test_size_one_dimensions_take_any_stride(J):
    # a pool of one page or one K/V head: torch reports whatever stride made the view
    k = torch.zeros(5, 32, 1, 64, dtype=torch.bfloat16)[:1]
    k = k.as_strided(k.shape, (7, 64, 3, 1))
    c = J.jano_page_pool.from_buffer_copy(P._pool(k, k, -1))
    assert (c.page_stride, c.token_stride, c.head_stride) == (32 * 64, 64, 64)
    assert (c.k, c.n_pages, c.page_size, c.kv_heads, c.d) == (k.data_ptr(), 1, 32, 1, 64)
    wide = torch.zeros(3, 9, 64, dtype=torch.bfloat16)[:, 2:3]
    assert P._rows(wide[:1], "x", -1, 1, 1, 64)[1] == 64 and P._rows(wide, "x", -1, 3, 1, 64)[1] == 576


def test_rope_of_a_geometry(J):
    r = J.Rope.of(J.Geometry(21, 60, 104), (44, 42, 42))
    assert r.n_pos == (21, 30, 52) and r.grid == (30, 52) and r.entries == 21 * 22 + 30 * 21 + 52 * 21
    c = r.c()
    assert (list(c.axes), list(c.n_pos), c.grid_h, c.grid_w, c.halves) == ([44, 42, 42], [21, 30, 52], 30, 52, 0)


# ------------------------------------------------------------------ page bookkeeping
def test_pages_are_handed_out_returned_and_never_shared():
    from kv_cache_analyzer_b200.serving import PagedBatch
    b = PagedBatch(n_pages=10, page_size=16, heads=4, kv_heads=2, d=64, device="cpu")
    a, c = b.open(33), b.open(64)                                  # 3 and 4 pages
    assert b.free_pages == 3 and b.k_pages.shape == (10, 16, 2, 64)
    with pytest.raises(RuntimeError, match="exhausted: 4 pages needed, 3 free"):
        b.open(50)
    assert b.free_pages == 3
    b.extend(a, 48)                                                # still 3 pages
    b.extend(a, 49)
    assert b.free_pages == 2
    with pytest.raises(RuntimeError, match="exhausted"):
        b.extend(a, 200)
    with pytest.raises(ValueError, match="cannot shrink"):
        b.extend(a, 10)
    p = b.plan([(c, 5), (a, 1)])
    t = p.lists["page_table"]
    assert t.shape == (2, 4) and len(set(t.flatten().tolist())) == 8
    assert p.lists["seq_lens"].tolist() == [64, 49] and p.lists["cu_rows"].tolist() == [0, 5, 6]
    assert (p.max_rows, p.max_len, p.n_rows) == (5, 64, 6)
    with pytest.raises(ValueError, match="once"):
        b.plan([(a, 1), (a, 2)])
    with pytest.raises(ValueError, match="at least one"):
        b.plan([])
    with pytest.raises(ValueError, match="negative"):
        b.plan([(a, -1)])
    rows = torch.zeros(5, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="plan has 6 rows, got 5"):
        b.step(p, rows, rows[:, :2], rows[:, :2], torch.zeros(5, dtype=torch.int32))
    b.close(a)
    with pytest.raises(ValueError, match="grew or closed"):
        b.step(p, rows, rows[:, :2], rows[:, :2], torch.zeros(6, dtype=torch.int32))
    p = b.plan([(c, 1)])
    b.extend(c, 65)
    with pytest.raises(ValueError, match="grew or closed"):
        b.step(p, rows, rows[:, :2], rows[:, :2], torch.zeros(1, dtype=torch.int32))
    assert b.free_pages == 5
    d = b.open(80)
    t = b.plan([(c, 1), (d, 1)]).lists["page_table"]
    assert t.shape == (2, 5) and len(set(t.flatten().tolist())) == 10


# ------------------------------------------------------------------ the polynomial 2^x
def test_paged_kernels_use_the_tested_polynomial():
    # tests/test_exp2_poly.py bounds the error of attention.cu's; the paged kernels' is the same text
    src = os.path.join(ROOT, "kv_cache_analyzer_b200", "csrc")
    body = [open(os.path.join(src, f)).read().split("void exp2_poly2(")[1].split("\n}\n")[0]
            for f in ("attention.cu", "paged_tile.cuh")]
    assert body[0] == body[1]


# ------------------------------------------------------------------ oracle pins
def test_oracle_rope_by_hand():
    # one head of 8 columns, axes of 2, 2 and 4: slots at 1, 1, 1 and theta^-1/2 = 1/100
    assert op.slots((2, 2, 4), 10000.0, False) == [(0, 1.0), (1, 1.0), (2, 1.0), (2, 0.01)]
    assert [a for a, _ in op.slots((2, 2, 4), 16.0, True)] == [0, 1, 2, 2]
    np.testing.assert_allclose([f for _, f in op.slots((2, 2, 4), 16.0, True)], [1.0, 0.5, 0.25, 0.125])
    x = np.array([[[1.0, 0.0, 0.0, 1.0, 2.0, 0.0, 3.0, 4.0]]])
    y = op.rope(x, np.array([[1, 2, 3]]), (2, 2, 4))
    c = np.cos
    s = np.sin
    np.testing.assert_allclose(y[0, 0], [c(1), s(1), -s(2), c(2), 2 * c(3), 2 * s(3), 3 * c(.03) - 4 * s(.03),
                                         3 * s(.03) + 4 * c(.03)])
    y = op.rope(x, np.array([[1, 2, 3]]), (2, 2, 4), halves=True)       # pairs (0, 4), (1, 5), (2, 6), (3, 7)
    np.testing.assert_allclose(y[0, 0, [0, 4]], [c(1) - 2 * s(1), s(1) + 2 * c(1)])
    np.testing.assert_allclose(y[0, 0, [3, 7]], [c(.03) - 4 * s(.03), s(.03) + 4 * c(.03)])


def test_oracle_rope_keeps_lengths_and_relative_positions():
    gen = np.random.default_rng(0)
    q, k = gen.standard_normal((2, 1, 1, 64))
    for halves in (False, True):
        turn = lambda x, p: op.rope(x, np.array([p]), (16, 24, 24), halves=halves)[0, 0]
        np.testing.assert_allclose(np.linalg.norm(turn(q, (3, 9, 4))), np.linalg.norm(q))
        # a dot product depends on the difference of the positions only
        np.testing.assert_allclose(turn(q, (3, 9, 4)) @ turn(k, (1, 2, 3)), turn(q, (5, 8, 14)) @ turn(k, (3, 1, 13)))


def test_oracle_table_and_grid():
    t = op.table((2, 4, 0), (2, 3, 1))
    assert t.shape == (2 * 1 + 3 * 2, 2)
    np.testing.assert_allclose(t[0], [1, 0])
    np.testing.assert_allclose(t[2 + 2 * 2 + 1], [np.cos(0.02), np.sin(0.02)])
    np.testing.assert_array_equal(op.grid_coords([0, 6, 7, 35, 69], 5, 7),
                                  [[0, 0, 0], [0, 0, 6], [0, 1, 0], [1, 0, 0], [1, 4, 6]])


def test_oracle_gather_and_attention_by_hand():
    pages = np.arange(4 * 2, dtype=np.float64).reshape(4, 2, 1, 1)
    np.testing.assert_array_equal(op.gather(pages, [3, 0, 9], 3)[:, 0, 0], [6, 7, 0])
    # logits 0 and ln 3 with scale 1: weights 1/4 and 3/4; a limit of one key; none
    q = np.full((3, 1, 1), np.log(3.0))
    k = np.array([0.0, 1.0]).reshape(2, 1, 1)
    v = np.array([4.0, 8.0]).reshape(2, 1, 1)
    out, pv, top = op.attention(q, k, v, [9, 1, 0], 1.0)
    np.testing.assert_allclose(out[:, 0, 0], [7.0, 4.0, 0.0])
    np.testing.assert_allclose(pv[:, 0, 0], [7.0, 4.0, 0.0])
    np.testing.assert_allclose(top[:2, 0, 0], [np.log(3.0), 0.0])
    # two query heads share a K/V head
    q2 = np.concatenate([q, q], 1)
    np.testing.assert_allclose(op.attention(q2, k, v, [9, 9, 9], 1.0)[0][:, 1], op.attention(q, k, v, [9] * 3, 1.0)[0][:, 0])
