"""GPU parity of the rotary positions (table, rows alone, rows on the way
into the token-ordered cache) against the fp64 oracle, through the Python
binding of the C ABI.  Tolerances: tests/paged_tools.py."""
import numpy as np
import pytest
import torch

import oracle.paged as op
import synth
from paged_tools import bits, check_rope

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


@pytest.mark.parametrize("axes,n_pos,theta,shared", [((44, 42, 42), (21, 45, 80), 10000.0, False),
                                                     ((0, 2, 6), (1, 100000, 3), 500.0, False),
                                                     ((16, 24, 24), (70001, 5, 9), 1e6, True),
                                                     ((2, 0, 0), (1, 1, 1), 10000.0, True)])
def test_table_matches_fp64(J, axes, n_pos, theta, shared):
    r = J.Rope(axes=axes, n_pos=n_pos, theta=theta, shared=shared)
    got = J.rope_table(r).cpu().numpy().astype(np.float64)
    ref = op.table(axes, n_pos, theta, shared)
    assert got.shape == ref.shape == (r.entries, 2)
    # cos and sin are rounded once to fp32 (2^-24 of at most 1); the angle, up
    # to 1e5, comes from a pow and a product in fp64 (a few 2^-53 of it)
    assert np.abs(got - ref).max() <= 2.0 ** -24 + 1e5 * 2.0 ** -50


CASES = [  # rows, heads, d, axes, halves, shared, wide buffer
    (1, 1, 64, (16, 24, 24), False, False, False),
    (1, 40, 128, (44, 42, 42), False, False, True),
    (37, 12, 128, (16, 56, 56), False, False, False),
    (700, 3, 64, (20, 22, 22), False, False, True),
    (53, 5, 128, (32, 48, 48), True, True, False),
    (1, 24, 64, (16, 24, 24), True, False, True),
    (29, 7, 96, (12, 10, 20), False, False, False),       # 12 vectors a head, columns 42.. kept
    (31, 3, 96, (16, 16, 32), True, False, False),        # 12 vectors, 4 units of split pairs and 4 kept vectors
    (19, 2, 72, (4, 2, 8), False, True, True),            # a vector with rotated and kept pairs
    (260, 1, 8, (2, 4, 2), False, False, False),
    (9, 2, 256, (0, 128, 128), True, False, False),
    (5, 3, 200, (0, 0, 200), False, False, False),
    (7, 2, 128, (16, 8, 8), True, False, False),          # rotated columns 0..31 only
]


@pytest.mark.parametrize("n,heads,d,axes,halves,shared,wide", CASES)
def test_axis_rope_matches_oracle(J, n, heads, d, axes, halves, shared, wide):
    gen = np.random.default_rng(n + d)
    n_pos = (6, 9, 31)
    r = J.Rope(axes=axes, n_pos=n_pos, grid=n_pos[1:], pairing="halves" if halves else "interleaved", shared=shared)
    table = J.rope_table(r)
    x = synth.normal_bf16((n, heads * (3 if wide else 1), d), seed=n)[:, :heads]
    xd = synth.normal_bf16((n, heads * (3 if wide else 1), d), seed=n).cuda()[:, :heads]
    ids = gen.integers(0, 6 * 9 * 31, size=n)                     # any order, repeats
    coords = op.grid_coords(ids, 9, 31)
    got = J.axis_rope(xd, r, table, ids=ints(ids))
    check_rope(got, x, coords, axes, halves=halves, shared=shared)
    # explicit coordinates and the rows in place give the same bits
    same = J.axis_rope(xd, r, table, coords=ints(coords))
    assert torch.equal(got.view(torch.int16), same.view(torch.int16))
    before = xd.clone()
    J.axis_rope(xd, r, table, ids=ints(ids), out=xd)
    no_device_error(J)
    assert torch.equal(xd.contiguous().view(torch.int16), got.view(torch.int16))
    assert not torch.equal(before, got) or n == 1


def test_rows_without_ids_are_their_own_tokens(J):
    r = J.Rope(axes=(16, 24, 24), n_pos=(2, 5, 7), grid=(5, 7))
    x = synth.normal_bf16((70, 4, 64), seed=3)
    got = J.axis_rope(x.cuda(), r, J.rope_table(r))
    no_device_error(J)
    check_rope(got, x, op.grid_coords(np.arange(70), 5, 7), (16, 24, 24))


def test_kept_columns_and_other_heads_never_meet_nan(J):
    # columns past the rotated ones hold NaN and infinities: moved bit for bit,
    # and no rotated column becomes NaN by them
    axes = (4, 6, 4)                                              # columns 0..13 of 24: inside a 16-byte vector
    r = J.Rope(axes=axes, n_pos=(3, 3, 3), grid=(3, 3))
    x = synth.normal_bf16((27, 3, 24), seed=5)
    x[..., 14:] = torch.tensor([float("nan"), float("inf"), -float("inf"), float("nan"), 0.0] * 2)
    got = J.axis_rope(x.cuda(), r, J.rope_table(r))
    no_device_error(J)
    assert torch.isfinite(got[..., :14].float()).all()
    np.testing.assert_array_equal(bits(got)[..., 14:], bits(x)[..., 14:])


def test_bad_ids_and_coordinates_raise_eindex_and_skip_the_row(J):
    r = J.Rope(axes=(16, 24, 24), n_pos=(2, 5, 7), grid=(5, 7))
    table = J.rope_table(r)
    x = synth.normal_bf16((6, 2, 64), seed=6).cuda()
    out = torch.full_like(x, 7.0)
    J.axis_rope(x, r, table, ids=ints([0, -1, 3, 70, 69, 2 ** 31 - 1]), out=out)
    assert J.device_error() == 6
    assert all(bool((out[i] == 7.0).all()) == (i in (1, 3, 5)) for i in range(6))
    out.fill_(7.0)
    J.axis_rope(x, r, table, out=out, coords=ints([[0, 0, 0], [2, 0, 0], [0, 5, 0], [0, 0, 7], [1, 4, 6], [0, -1, 0]]))
    assert J.device_error() == 6
    assert all(bool((out[i] == 7.0).all()) == (i in (1, 2, 3, 5)) for i in range(6))
    # an axis without columns has no bound to break
    flat = J.Rope(axes=(0, 32, 32), n_pos=(1, 5, 7), grid=(5, 7))
    J.axis_rope(x, flat, J.rope_table(flat), coords=ints([[9, 0, 0]] * 6), out=out)
    no_device_error(J)


@pytest.mark.parametrize("n,N,heads,kv_heads,d,axes,halves,fused", [
    (1, 64, 4, 4, 64, (16, 24, 24), False, False),
    (33, 1024, 4, 4, 64, (16, 24, 24), True, False),
    (301, 1000, 12, 3, 128, (44, 42, 42), False, True),
    (90, 90, 2, 2, 96, (12, 10, 20), False, True),
    (45, 77, 3, 1, 96, (16, 16, 32), True, True),
])
def test_rope_scatter_matches_oracle_and_keeps_other_rows(J, n, N, heads, kv_heads, d, axes, halves, fused):
    gen = np.random.default_rng(n)
    n_pos = (5, 10, 21)
    r = J.Rope(axes=axes, n_pos=n_pos, grid=n_pos[1:], pairing="halves" if halves else "interleaved")
    table = J.rope_table(r)
    idx = np.sort(gen.choice(N, size=n, replace=False))
    coords = op.grid_coords(idx, 10, 21)
    whole = synth.normal_bf16((n, heads + 2 * kv_heads, d), seed=n + 1)
    q, k, v = whole.split([heads, kv_heads, kv_heads], 1)
    dq, dk, dv = whole.cuda().split([heads, kv_heads, kv_heads], 1)
    if not fused:
        dq, dk, dv = dq.contiguous(), dk.contiguous(), dv.contiguous()
    kc0, vc0 = (synth.normal_bf16((N, kv_heads, d), seed=s) for s in (8, 9))
    kc, vc = kc0.cuda(), vc0.cuda()
    got = J.rope_scatter(dk, dv, ints(idx), kc, vc, r, table, q=dq)
    no_device_error(J)
    check_rope(got, q, coords, axes, halves=halves)
    check_rope(kc[torch.from_numpy(idx).cuda()], k, coords, axes, halves=halves)
    np.testing.assert_array_equal(bits(vc)[idx], bits(v))
    rest = np.setdiff1d(np.arange(N), idx)
    np.testing.assert_array_equal(bits(kc)[rest], bits(kc0)[rest])
    np.testing.assert_array_equal(bits(vc)[rest], bits(vc0)[rest])
    # the same bits as rotating first and scattering then
    kc2, vc2 = kc0.cuda(), vc0.cuda()
    rk = J.axis_rope(dk, r, table, ids=ints(idx))
    if kv_heads * d % 8 == 0:
        J.kv_scatter(rk, dv.contiguous(), ints(idx), kc2, vc2)
        assert torch.equal(kc.view(torch.int16), kc2.view(torch.int16))
        assert torch.equal(vc.view(torch.int16), vc2.view(torch.int16))
    # without queries, coordinates given
    kc3, vc3 = kc0.cuda(), vc0.cuda()
    assert J.rope_scatter(dk, dv, ints(idx), kc3, vc3, r, table, coords=ints(coords)) is None
    no_device_error(J)
    assert torch.equal(kc.view(torch.int16), kc3.view(torch.int16))


def test_rope_scatter_rejects_duplicate_descending_and_far_ids(J):
    r = J.Rope(axes=(16, 24, 24), n_pos=(4, 4, 4), grid=(4, 4))
    table = J.rope_table(r)
    idx = [0, 2, 2, 5, 4, 9, 40, 63]
    skipped = [2, 4, 6]                                           # duplicate, step back, past the 40-row cache
    k = synth.normal_bf16((8, 2, 64), seed=1).cuda()
    kc = torch.full((40, 2, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    vc = kc.clone()
    q = torch.full_like(k, 9.0)
    J.rope_scatter(k, k, ints(idx), kc, vc, r, table, q=k, q_out=q)
    assert J.device_error() == 6
    assert [i for i in range(8) if bool((q[i] == 9.0).all())] == [2, 4, 6, 7]
    assert bool((kc[4] == 3.0).all()) and bool((vc[4] == 3.0).all())
    assert torch.equal(vc[[0, 2, 5, 9]], k[[0, 1, 3, 5]])


def test_empty_calls_do_nothing(J):
    r = J.Rope(axes=(16, 24, 24), n_pos=(4, 4, 4), grid=(4, 4))
    table = J.rope_table(r)
    none = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    assert J.axis_rope(none, r, table).shape == (0, 2, 64)
    kc = torch.ones(8, 2, 64, dtype=torch.bfloat16, device="cuda")
    J.rope_scatter(none, none, ints([]), kc, kc.clone(), r, table)
    no_device_error(J)
    assert bool((kc == 1).all())


def test_side_stream_and_graph_replay(J):
    r = J.Rope(axes=(44, 42, 42), n_pos=(2, 16, 16), grid=(16, 16))
    table = J.rope_table(r)
    x = synth.normal_bf16((512, 12, 128), seed=2).cuda()
    want = J.axis_rope(x, r, table)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = J.axis_rope(x, r, table, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    out = torch.zeros_like(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        J.axis_rope(x, r, table, out=out)
    assert bool((out == 0).all())
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    x.mul_(2.0)                                                   # the graph reads its inputs anew
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want * 2.0)                           # a power of two: exact
    no_device_error(J)
    del g
