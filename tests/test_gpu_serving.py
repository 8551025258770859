"""Several generations over one page pool (PagedBatch) against the fp64 oracle
and against each generation's own contiguous cache; the hot path's step with
the rotation on the way."""
import numpy as np
import pytest
import torch

import oracle.paged as op
import synth
from paged_tools import check_attention, check_rope, f64

pytestmark = pytest.mark.gpu


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


@pytest.mark.parametrize("page,heads,kv_heads,d,axes", [(32, 4, 4, 64, (16, 24, 24)), (64, 6, 2, 128, (44, 42, 42))])
def test_batch_of_generations_equals_each_ones_own_cache(J, page, heads, kv_heads, d, axes):
    from kv_cache_analyzer_b200.serving import PagedBatch
    # three generations of different grids: a video of 2 frames, an image, a
    # larger image that takes the pages a closed one left (their contents: NaN)
    grids = [(2, 10, 12), (1, 9, 21), (1, 17, 19)]
    sizes = [f * h * w for f, h, w in grids]
    rope = J.Rope(axes=axes, n_pos=(2, 17, 21), grid=(10, 12))
    need = sum(-(-n // page) for n in sizes)
    b = PagedBatch(n_pages=need + 1, page_size=page, heads=heads, kv_heads=kv_heads, d=d, rope=rope)
    b.k_pages.fill_(float("nan"))
    b.v_pages.fill_(float("nan"))
    gone = b.open(3 * page)
    gens = [b.open(sizes[0], grids[0][1:]), b.open(sizes[1], grids[1][1:])]
    b.close(gone)
    gens.append(b.open(sizes[2], grids[2][1:]))
    gen = np.random.default_rng(d)
    own = [[np.zeros((n, kv_heads, d)) for _ in range(2)] for n in sizes]          # each one's cache, fp64
    ours = [[torch.zeros(n, heads, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)] for n in sizes]
    for step in range(3):
        # step 0 writes every token, later ones the due tokens of some generations
        who = [0, 1, 2] if step != 1 else [2, 0]
        due = [np.arange(sizes[g]) if step == 0 else np.sort(gen.choice(sizes[g], 1 + 40 * g, replace=False))
               for g in who]
        n = sum(len(x) for x in due)
        q = synth.normal_bf16((n, heads, d), seed=10 * step)
        k, v = (synth.normal_bf16((n, kv_heads, d), seed=10 * step + s) for s in (1, 2))
        plan = b.plan([(gens[g], len(x)) for g, x in zip(who, due)])
        out = b.step(plan, q.cuda(), k.cuda(), v.cuda(), ints(np.concatenate(due)))
        assert J.device_error() == 0
        at = 0
        for g, x in zip(who, due):
            sl = slice(at, at + len(x))
            at += len(x)
            _, h, w = grids[g]
            coords = op.grid_coords(x, h, w)
            table = J.rope_table(rope)
            kr, qr = (J.axis_rope(t[sl].cuda(), rope, table, coords=ints(coords)) for t in (k, q))
            check_rope(kr, k[sl], coords, axes)
            own[g][0][x], own[g][1][x] = f64(kr), f64(v[sl])
            if step:
                check_attention(out[sl], f64(qr), own[g][0], own[g][1], np.full(len(x), sizes[g]), d ** -0.5)
            if kv_heads == heads:                     # the contiguous path of the same generation
                mine = J.Rope(axes=axes, n_pos=(2, 17, 21), grid=(h, w))
                qc = J.rope_scatter(k[sl].cuda(), v[sl].cuda(), ints(x), *ours[g], mine, table, q=q[sl].cuda())
                assert torch.equal(qc, qr)
                o = torch.zeros(sizes[g], heads, d, dtype=torch.bfloat16, device="cuda")
                J.active_attention(qc, *ours[g], ints(x), o)
                if step:
                    check_attention(o[torch.from_numpy(x).cuda()], f64(qr), own[g][0], own[g][1],
                                    np.full(len(x), sizes[g]), d ** -0.5)
    assert J.device_error() == 0


def test_streamed_generation_grows_frame_by_frame(J):
    # frames of 6 x 9 tokens: each new frame is appended and sees the frames up to its own
    from kv_cache_analyzer_b200.serving import PagedBatch
    heads, d, per = 4, 64, 54
    rope = J.Rope(axes=(16, 24, 24), n_pos=(5, 6, 9), grid=(6, 9))
    b = PagedBatch(n_pages=40, page_size=16, heads=heads, d=d, rope=rope)
    g = b.open(0)
    q, k, v = (synth.normal_bf16((5 * per, heads, d), seed=s) for s in (1, 2, 3))
    table = J.rope_table(rope)
    kr, qr = (f64(J.axis_rope(t.cuda(), rope, table)) for t in (k, q))
    for first, last in ((0, 1), (1, 2), (2, 5)):
        b.extend(g, last * per)
        sl = slice(first * per, last * per)
        pos = np.arange(first * per, last * per)
        limits = (pos // per + 1) * per
        plan = b.plan([(g, len(pos))])
        out = b.step(plan, q[sl].cuda(), k[sl].cuda(), v[sl].cuda(), ints(pos), limits=ints(limits))
        assert J.device_error() == 0
        check_attention(out, qr[sl], kr[:last * per], f64(v[:last * per]), limits, d ** -0.5)


def test_layers_keep_their_own_pages(J):
    from kv_cache_analyzer_b200.serving import PagedBatch
    b = PagedBatch(n_pages=8, page_size=16, heads=2, d=64, layers=2)
    one = PagedBatch(n_pages=8, page_size=16, heads=2, d=64)
    g, h = b.open(90), one.open(90)
    pos = ints(np.arange(90))
    plan, alone = b.plan([(g, 90)]), one.plan([(h, 90)])
    rows = [[synth.normal_bf16((90, 2, 64), seed=3 * layer + s).cuda() for s in range(3)] for layer in range(2)]
    outs = [b.step(plan, *rows[layer], pos, layer=layer) for layer in range(2)]
    for layer in range(2):                                 # without a rope: the rows as they are
        assert torch.equal(one.step(alone, *rows[layer], pos), outs[layer])
    # a second step of layer 0 still finds its own keys
    few = b.plan([(g, 1)])
    q, k, v = (x[:1].contiguous() for x in rows[0])
    got = b.step(few, q, k, v, ints([0]))
    assert J.device_error() == 0
    check_attention(got, f64(q), f64(rows[0][1]), f64(rows[0][2]), np.array([90]), 64 ** -0.5)
    with pytest.raises(IndexError):
        b.step(few, q, k, v, ints([0]), layer=2)


def test_batch_step_replays_as_a_graph_on_a_side_stream(J):
    from kv_cache_analyzer_b200.serving import PagedBatch
    s = torch.cuda.Stream()
    rope = J.Rope(axes=(16, 24, 24), n_pos=(1, 16, 16), grid=(16, 16))
    with torch.cuda.stream(s):
        b = PagedBatch(n_pages=20, page_size=32, heads=4, d=64, rope=rope, stream=s)
        x, y = b.open(256), b.open(200)
        rows = torch.cat([torch.arange(256), torch.arange(200)]).int().cuda()
        fill = [synth.normal_bf16((456, 4, 64), seed=i).cuda() for i in range(3)]
        b.step(b.plan([(x, 256), (y, 200)]), *fill, rows)
        plan = b.plan([(x, 3), (y, 1)])
        q, k, v = (synth.normal_bf16((4, 4, 64), seed=i).cuda() for i in range(5, 8))
        pos, out = ints([1, 7, 255, 199]), torch.empty_like(q)
        want = b.step(plan, q, k, v, pos).clone()
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            b.step(plan, q, k, v, pos, out=out)
        out.zero_()
        b.plan([(y, 7), (x, 2)])                      # another plan in between changes nothing
        g.replay()
        s.synchronize()
    assert J.device_error(s) == 0
    assert torch.equal(out, want)
    del g


def test_hot_path_with_a_rope_equals_its_parts(J):
    from kv_cache_analyzer_b200.pipeline import HotPath
    w = synth.WORKLOADS["tiny"]
    stream = torch.cuda.Stream()
    geom = J.Geometry(w.F, w.H, w.W, w.patch, w.patch)
    rope = J.Rope.of(geom, (16, 24, 24))
    hp = HotPath(K=w.K, C=w.C, latent_geom=J.Geometry(w.F, w.H, w.W, w.block, w.patch), token_geom=geom,
                 heads=w.heads, d=w.d, frac_active=w.frac_active, frac_static=w.frac_static,
                 sched=J.Schedule(w.T, w.warmup, w.cooldown, w.period_moderate, w.period_static), stream=stream,
                 rope=rope)
    hp.set_activations(w.n_tokens)
    n = w.n_tokens
    q, k, v, kc, vc = (synth.normal_bf16((n, w.heads, w.d), seed=s).cuda() for s in range(5))
    with torch.cuda.stream(stream):
        hp.lat.copy_(torch.from_numpy(synth.latent_history(w.K, w.C, w.F, w.H, w.W, seed=w.seed)))
        hp.field.copy_(torch.from_numpy(synth.token_field(*w.grid, seed=3, sigma=w.field_sigma)))
        hp.q_act.copy_(q), hp.k_act.copy_(k), hp.v_act.copy_(v), hp.k_cache.copy_(kc), hp.v_cache.copy_(vc)
    hp.plan()
    n_act = hp.run_step_kernels(w.warmup)
    stream.synchronize()
    assert J.device_error(stream) == 0
    start, _ = hp.due(w.warmup)
    idx = hp.idx[start:start + n_act]
    table = J.rope_table(rope)
    qr = J.axis_rope(q[:n_act], rope, table, ids=idx)
    kr = J.axis_rope(k[:n_act], rope, table, ids=idx)
    J.kv_scatter(kr, v[:n_act].contiguous(), idx, kc, vc)
    assert torch.equal(hp.k_cache, kc) and torch.equal(hp.v_cache, vc) and torch.equal(hp.q_rot[:n_act], qr)
    out = torch.zeros_like(kc)
    J.active_attention(qr, kc, vc, idx, out)
    assert J.device_error() == 0
    assert torch.equal(hp.out[idx.long()], out[idx.long()])
    # the unrotated rows stay, so the step can be captured and replayed
    assert torch.equal(hp.q_act, q) and torch.equal(hp.k_act, k)
    # two head-sharded ranks of the same step
    from kv_cache_analyzer_b200.sharding import ShardedHotPath
    for rank in range(2):
        sh = ShardedHotPath(rank=rank, world=2, K=w.K, C=w.C, latent_geom=hp.lg, token_geom=geom, heads=w.heads, d=w.d,
                            frac_active=w.frac_active, frac_static=w.frac_static, sched=hp.sched, stream=stream,
                            rope=rope)
        sh.set_activations(n)
        with torch.cuda.stream(stream):
            for name, t in (("q_act", q), ("k_act", k), ("v_act", v), ("k_cache", kc), ("v_cache", vc)):
                getattr(sh, name).copy_(sh.head_slice(t))
        sh.idx, sh.host_offsets = hp.idx, hp.host_offsets
        sh.run_head_kernels(w.warmup)
        stream.synchronize()
        assert J.device_error(stream) == 0
        assert torch.equal(sh.out[idx.long()], sh.head_slice(out)[idx.long()])
    first = hp.out.clone()
    g = hp.capture_step(w.warmup)
    hp.out.zero_()
    with torch.cuda.stream(stream):
        g.replay()
    stream.synchronize()
    assert torch.equal(hp.out[idx.long()], first[idx.long()])
    del g


@pytest.mark.parametrize("rows", [1, 40])
def test_calls_in_a_row_see_what_the_ones_before_wrote(J, rows):
    # each kernel sets itself up while the one in front ends: a chain in which every call reads the last
    # one's output (rows, lengths, cache) gives bit for bit what it gives with a wait after every call
    from kv_cache_analyzer_b200.serving import PagedBatch
    rope = J.Rope(axes=(16, 24, 24), n_pos=(8, 16, 16), grid=(16, 16))
    start = synth.normal_bf16((rows, 4, 64), seed=1).cuda()

    def chain(wait):
        b = PagedBatch(n_pages=80, page_size=16, heads=4, d=64, rope=rope)
        g = b.open(1200)
        b.k_pages.fill_(0.25)
        b.v_pages.fill_(0.5)
        plan = b.plan([(g, rows)])
        x, outs = start.clone(), []
        for i in range(60):
            pos = torch.arange(i * 7, i * 7 + rows, device="cuda", dtype=torch.int32)
            plan.lists["seq_lens"].fill_(100 + 17 * i)             # written by a kernel in front
            if wait:
                torch.cuda.synchronize()
            y = J.axis_rope(x, rope, b.table, ids=pos)
            if wait:
                torch.cuda.synchronize()
            x = b.step(plan, y, x, y, pos, limits=pos + 60)
            if wait:
                torch.cuda.synchronize()
            outs.append(x)
        torch.cuda.synchronize()
        assert J.device_error() == 0
        return torch.stack(outs)

    want = chain(True)
    for _ in range(5):
        assert torch.equal(chain(False), want)
