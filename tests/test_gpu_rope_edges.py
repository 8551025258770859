"""Rows that the rotations skip: with a bad coordinate, grid or list nothing of
the row is written, neither K nor V nor its query, through the Python binding
of the C ABI."""
import numpy as np
import pytest
import torch

import synth

pytestmark = pytest.mark.gpu

EINDEX = 6


@pytest.fixture(scope="module")
def J():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from kv_cache_analyzer_b200 import build
    build.build()
    import kv_cache_analyzer_b200 as j
    j.lib()
    return j


def ints(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def changed(t, fill):
    """Which of t's first-dimension rows differ from the fill they had."""
    return (t != fill).flatten(1).any(1).cpu().numpy()


# (rows, heads, kv_heads, d, axes, halves): whole rows and parts of rows per warp, both pairings, heads whose
# units divide 32 and not
SHAPES = [(12, 3, 2, 64, (16, 24, 24), False), (12, 4, 4, 128, (32, 48, 48), True), (12, 2, 1, 96, (12, 10, 20), False),
          (9000, 1, 1, 64, (0, 32, 32), False)]


def ropes(J, axes, halves):
    # an axis without columns has no bound: the frames of a (0, ...) rotation are never bad
    r = J.Rope(axes=axes, n_pos=(3, 5, 7), grid=(5, 7), pairing="halves" if halves else "interleaved")
    return r, J.rope_table(r)


def bad_coords(n, axes, gen):
    c = np.stack([gen.integers(0, m, n) for m in (3, 5, 7)], 1)
    bad = gen.random(n) < 0.4
    bad[:2] = True, False
    for i in np.nonzero(bad)[0]:
        a = int(gen.choice([x for x in range(3) if axes[x]]))
        c[i, a] = gen.choice([-1, (3, 5, 7)[a], 2 ** 31 - 1, -2 ** 31])
    return c, bad


@pytest.mark.parametrize("n,heads,kv_heads,d,axes,halves", SHAPES)
def test_scatter_writes_nothing_of_a_row_with_bad_coordinates(J, n, heads, kv_heads, d, axes, halves):
    r, table = ropes(J, axes, halves)
    gen = np.random.default_rng(n + d)
    q = synth.normal_bf16((n, heads, d), seed=1).cuda()
    k, v = (synth.normal_bf16((n, kv_heads, d), seed=s).cuda() for s in (2, 3))
    coords, bad = bad_coords(n, axes, gen)
    idx = np.arange(n)
    cases = [(dict(coords=ints(coords)), idx, bad)]
    if axes[0]:                                                   # ids behind the last frame: 3 frames of 5 x 7 tokens
        ids = np.sort(gen.choice(n + 120, n, replace=False))
        cases.append((dict(), ids, ids >= 105))
        assert cases[-1][2].any()
    for kw, ids, bad in cases:
        N = int(ids.max()) + 1
        kc, vc = (torch.full((N, kv_heads, d), 100.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        q_out = torch.full_like(q, 100.0)
        J.rope_scatter(k, v, ints(ids), kc, vc, r, table, q=q, q_out=q_out, **kw)
        assert J.device_error() == EINDEX
        np.testing.assert_array_equal(changed(q_out, 100.0), ~bad)
        for t in (kc, vc):
            want = np.zeros(N, dtype=bool)
            want[ids[~bad]] = True
            np.testing.assert_array_equal(changed(t, 100.0), want)
        good = torch.from_numpy(ids[~bad]).cuda()
        assert torch.equal(vc[good], v[torch.from_numpy(~bad).cuda()])


@pytest.mark.parametrize("n,heads,kv_heads,d,axes,halves", SHAPES)
def test_append_writes_nothing_of_a_row_with_bad_coordinates(J, n, heads, kv_heads, d, axes, halves):
    r, table = ropes(J, axes, halves)
    gen = np.random.default_rng(n + d + 1)
    q = synth.normal_bf16((n, heads, d), seed=1).cuda()
    k, v = (synth.normal_bf16((n, kv_heads, d), seed=s).cuda() for s in (2, 3))
    coords, bad = bad_coords(n, axes, gen)
    half = n // 2
    cu, lens = ints([0, half, n]), ints([half, n - half])
    pos = np.concatenate([np.arange(half), np.arange(n - half)])
    per = -(-n // 16)
    pages = ints(np.arange(2 * per).reshape(2, per))
    seq = np.arange(n) >= half
    cases = [(dict(coords=ints(coords)), bad)]
    if n < 100:                                                   # a grid of its own without rows or columns
        cases += [(dict(grids=ints([(5, 7), grid])), seq) for grid in ((0, 7), (7, 0), (-1, 7))]
    for kw, bad in cases:
        kp, vp = (torch.full((2 * per, 16, kv_heads, d), 100.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        q_out = torch.full_like(q, 100.0)
        J.paged_append(k, v, ints(pos), kp, vp, pages, lens, cu, rope=r, table=table, q=q, q_out=q_out, **kw)
        assert J.device_error() == EINDEX
        np.testing.assert_array_equal(changed(q_out, 100.0), ~bad)
        at = seq * per * 16 + pos
        for t in (kp, vp):
            want = np.zeros(2 * per * 16, dtype=bool)
            want[at[~bad]] = True
            np.testing.assert_array_equal(changed(t.flatten(0, 1), 100.0), want)


def test_append_without_a_rope_has_no_coordinates_to_check(J):
    k = synth.normal_bf16((6, 2, 64), seed=1).cuda()
    kp, vp = (torch.full((2, 16, 2, 64), 100.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    J.paged_append(k, k, ints(range(6)), kp, vp, ints([[1]]), ints([6]), ints([0, 6]))
    assert J.device_error() == 0
    assert torch.equal(kp[1, :6], k) and torch.equal(vp[1, :6], k)


@pytest.mark.parametrize("cu", [[-3, 0, 4], [-1, 0, 0, 4], [-2 ** 31, 0, 4]])
def test_append_reports_a_row_list_that_does_not_begin_at_zero(J, cu):
    # the rows lie in a later sequence, whose own bounds are good
    k = synth.normal_bf16((4, 2, 64), seed=1).cuda()
    kp, vp = (torch.full((8, 16, 2, 64), 100.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    n = len(cu) - 1
    q_out = torch.full_like(k, 100.0)
    J.paged_append(k, k, ints(range(4)), kp, vp, ints(np.arange(n)[:, None]), ints([4] * n), ints(cu), q=k, q_out=q_out)
    assert J.device_error() == EINDEX
    assert not changed(kp, 100.0).any() and not changed(vp, 100.0).any() and not changed(q_out, 100.0).any()
    # sequences without rows in front of it are no fault
    J.paged_append(k, k, ints(range(4)), kp, vp, ints([[0], [1], [2]]), ints([4, 4, 4]), ints([0, 0, 0, 4]))
    assert J.device_error() == 0
    assert torch.equal(kp[2, :4], k) and torch.equal(vp[2, :4], k)
