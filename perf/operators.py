"""Measured cases of the rotated and paged cache operators.

Four operators: the rotation of rows by their (frame, row, column) position
(`axis_rope`), the scatter of due K/V rows into the token-ordered cache with
the rotation on the way (`rope_scatter`), the append to a page pool shared by
several generations (`paged_append`) and the attention of a chunk of rows over
such pages (`paged_attention`).

`run` computes them in plain torch operations, in 32 bits with one rounding at
the end; where `own` is true it makes the calls of this package instead.
`exact` gives the same outputs from the definition in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
THETA = 10000.0


# ------------------------------------------------------------------ cases
def listed():
    return [
        # every token of an image DiT step (64 x 64 tokens, 24 heads), its queries rotated in one call
        dict(name="rope image", op="rope", rows=4096, of=4096, heads=24, d=128, axes="16,56,56", grid="1,64,64",
             halves=False, fused=False),
        # the Active tokens of a large video step (75,600 tokens, 40 heads), read from a fused projection's columns
        dict(name="rope large video", op="rope", rows=18900, of=75600, heads=40, d=128, axes="44,42,42",
             grid="21,45,80", halves=False, fused=True),
        # the smallest due sets: a few tokens of a tiny latent, where the call's latency is what counts
        dict(name="scatter few", op="scatter", rows=33, of=1024, heads=4, kv_heads=4, d=64, axes="16,24,24",
             grid="4,16,16", halves=False, fused=False),
        # 35% due tokens of a small video step, Q, K and V as columns of the fused projection
        dict(name="scatter small video", op="scatter", rows=11466, of=32760, heads=12, kv_heads=12, d=128,
             axes="44,42,42", grid="21,30,52", halves=False, fused=True),
        # one new token for each of sixteen running generations, small pages, grouped heads, paired by halves
        dict(name="append one each", op="append", seqs=16, rows=1, length=4096, heads=24, kv_heads=8, d=128, page=16,
             axes="16,56,56", grid="1,64,64", halves=True, fused=False, head_major=False),
        # three streamed videos each append about three frames of 30 x 52 tokens
        dict(name="append frames", op="append", seqs=3, rows=4680, length=32760, heads=12, kv_heads=12, d=128, page=64,
             axes="44,42,42", grid="21,30,52", halves=False, fused=True, head_major=False),
        # a single row over one image's cache: latency
        dict(name="attend one token", op="attend", seqs=1, rows=1, length=4096, heads=24, kv_heads=24, d=128, page=16,
             mask="none", frame=1, head_major=False),
        # one row for each of many generations of different lengths, grouped heads: the cache's bytes count
        dict(name="attend one each of 32", op="attend", seqs=32, rows=1, length=32760, heads=40, kv_heads=8, d=128,
             page=64, mask="none", frame=1, head_major=True),
        # short, odd, ragged sequences (one of them without rows), heads of 64, each row sees what came before it
        dict(name="attend odd ragged", op="attend", seqs=5, rows=61, length=777, heads=6, kv_heads=2, d=64, page=16,
             mask="token", frame=1, head_major=False),
        # the due sets (30% and less) of four images in one call
        dict(name="attend four images", op="attend", seqs=4, rows=1228, length=4096, heads=24, kv_heads=24, d=128,
             page=64, mask="none", frame=1, head_major=False),
        # three new frames of a streamed video: every row sees the frames up to its own
        dict(name="attend new frames", op="attend", seqs=1, rows=4680, length=32760, heads=12, kv_heads=12, d=128,
             page=128, mask="frame", frame=1560, head_major=False),
        # half of a small video's tokens due at once: the matrix products count
        dict(name="attend half of a video", op="attend", seqs=1, rows=16380, length=32760, heads=12, kv_heads=12,
             d=128, page=128, mask="none", frame=1, head_major=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "scatter", "append", "append", "attend", "attend", "attend"])
    d = rng.choice([64, 128, 128])
    axes = rng.choice({64: ["16,24,24", "20,22,22", "0,32,32"], 128: ["16,56,56", "44,42,42", "32,48,48"]}[d])
    halves = rng.random() < 0.4
    if halves:
        axes = {64: "16,24,24", 128: "32,48,48"}[d]
    grid = (rng.randint(1, 21), rng.randint(8, 45), rng.randint(8, 80))
    of = grid[0] * grid[1] * grid[2]
    text = "%d,%d,%d" % grid
    if op == "rope":
        return dict(op=op, rows=_log(rng, 1, min(of, 18900)), of=of, heads=rng.randint(1, 40), d=d, axes=axes, grid=text,
                    halves=halves, fused=rng.random() < 0.5)
    kv_heads = rng.randint(1, 12)
    heads = kv_heads * rng.choice([1, 1, 2, 3, 5, 8])
    if op == "scatter":
        return dict(op=op, rows=_log(rng, 1, min(of, 11466)), of=of, heads=min(heads, 40) // kv_heads * kv_heads,
                    kv_heads=kv_heads, d=d, axes=axes, grid=text, halves=halves, fused=rng.random() < 0.5)
    page = rng.choice([16, 32, 64, 128])
    seqs = _log(rng, 1, 24)
    if op == "append":
        return dict(op=op, seqs=seqs, rows=max(1, min(_log(rng, 1, 4680), 9000 // seqs, of)), length=of, heads=heads,
                    kv_heads=kv_heads, d=d, page=page, axes=axes, grid=text, halves=halves, fused=rng.random() < 0.5,
                    head_major=rng.random() < 0.3)
    length = _log(rng, 1, 32760)
    # as many scores as the largest listed case at most
    rows = max(1, min(_log(rng, 1, 4680), length, int(2.0e9 / (length * heads * seqs))))
    return dict(op=op, seqs=seqs, rows=rows, length=length, heads=heads, kv_heads=kv_heads, d=d, page=page,
                mask=rng.choice(["none", "token", "frame"]), frame=rng.choice([1, 60, 256, 1560]),
                head_major=rng.random() < 0.3)


def _ints(text):
    return [int(x) for x in text.split(",")]


def _rows_of(case):
    """Rows of each sequence: the case's count for the first, fewer for the others (none for one of five)."""
    return [case["rows"] - (s * 37 % 101) * case["rows"] // 202 if s % 5 != 3 or case["rows"] == 1 else 0
            for s in range(case["seqs"])]


def _lens_of(case):
    """Length of each sequence after the append: the case's for the first, down to a quarter of it for the others,
    and at least its rows."""
    return [max(n, case["length"] - (s * 53 % 97) * case["length"] * 3 // (4 * 97), 1)
            for s, n in enumerate(_rows_of(case))]


# ------------------------------------------------------------------ inputs
def _angles(case):
    """Per axis the 64-bit angles [positions][slots]."""
    return [torch.arange(n, dtype=torch.float64, device=DEV)[:, None]
            * THETA ** (-2.0 * torch.arange(a // 2, dtype=torch.float64, device=DEV) / max(a, 1))
            for a, n in zip(_ints(case["axes"]), _ints(case["grid"]))]


def _table(case):
    """The rotation table that a program makes once: cos and sin of every (position, slot), axis after axis."""
    a = torch.cat([x.reshape(-1) for x in _angles(case)])
    return torch.stack([a.cos(), a.sin()], 1).float().contiguous()


def _columns(gen, n, parts, d, fused):
    """[n][heads][d] tensors: columns of one fused buffer, or buffers of their own."""
    def randn(*shape):
        return torch.randn(shape, generator=gen, device=DEV).bfloat16()
    if not fused:
        return [randn(n, h, d) for h in parts]
    whole = randn(n, sum(parts) * d)
    return [x.view(n, h, d) for x, h in zip(whole.split([h * d for h in parts], 1), parts)]


def _pages(gen, case, lens):
    """A pool with its pages handed out in no order, a quarter of them to nobody."""
    p, h, d = case["page"], case["kv_heads"], case["d"]
    per = [-(-n // p) for n in lens]
    n_pages = sum(per) + sum(per) // 4 + 1
    shape = (n_pages, h, p, d) if case["head_major"] else (n_pages, p, h, d)
    k, v = (torch.randn(shape, generator=gen, device=DEV).bfloat16() for _ in range(2))
    if case["head_major"]:
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    order = torch.randperm(n_pages, generator=gen, device=DEV).int()
    table = torch.zeros(len(lens), max(per), dtype=torch.int32, device=DEV)
    at = 0
    for s, n in enumerate(per):
        table[s, :n] = order[at:at + n]
        at += n
    return k, v, table


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    gen = torch.Generator(DEV).manual_seed(seed)
    st = dict(case)
    d = case["d"]
    if case["op"] in ("rope", "scatter"):
        st["ids"] = torch.randperm(case["of"], generator=gen, device=DEV)[:case["rows"]].sort().values.int()
        st["table"] = _table(case)
        if case["op"] == "rope":
            # with `fused` the rows are the query columns of a projection with as many key and value columns
            h = case["heads"]
            st["x"] = _columns(gen, case["rows"], [h, h, h] if case["fused"] else [h], d, case["fused"])[0]
        else:
            st["q"], st["k"], st["v"] = _columns(gen, case["rows"], [case["heads"]] + 2 * [case["kv_heads"]], d,
                                                 case["fused"])
            st["k_cache"], st["v_cache"] = _columns(gen, case["of"], 2 * [case["kv_heads"]], d, False)
        return st
    rows, lens = _rows_of(case), _lens_of(case)
    n = sum(rows)
    st["max_rows"], st["max_len"] = max(rows), max(lens)
    st["lens"] = _int32(lens)
    st["cu_rows"] = _int32([sum(rows[:s]) for s in range(len(rows) + 1)])
    st["k_pages"], st["v_pages"], st["page_table"] = _pages(gen, case, lens)
    if case["op"] == "append":
        st["table"] = _table(case)
        # the rows are the last of their sequence
        st["pos"] = torch.cat([torch.arange(m - r, m, device=DEV) for r, m in zip(rows, lens)]).int()
        st["q"], st["k"], st["v"] = _columns(gen, n, [case["heads"]] + 2 * [case["kv_heads"]], d, case["fused"])
    else:
        st["q"], = _columns(gen, n, [case["heads"]], d, False)
        pos = torch.cat([torch.arange(m - r, m, device=DEV) for r, m in zip(rows, lens)])
        f = case["frame"]
        st["limits"] = {"none": None, "token": (pos + 1).int(), "frame": ((pos // f + 1) * f).int()}[case["mask"]]
    return st


# ------------------------------------------------------------------ plain forms
def _seq_of_row(cu_rows, n):
    return torch.searchsorted(cu_rows[1:].long(), torch.arange(n, device=DEV), right=True)


def _cos_sin(st, ids):
    """cos and sin [rows][slots] of the rows at token ids."""
    _, th, tw = _ints(st["grid"])
    ids = ids.long()
    coords = (ids // (th * tw), ids // tw % th, ids % tw)
    sizes = [n * (a // 2) for a, n in zip(_ints(st["axes"]), _ints(st["grid"]))]
    parts = [t.view(n, a // 2, 2)[c] for t, a, n, c in
             zip(st["table"].split(sizes), _ints(st["axes"]), _ints(st["grid"]), coords)]
    cs = torch.cat(parts, 1)
    return cs[:, None, :, 0], cs[:, None, :, 1]


def _rotate(x, c, s, halves):
    """Rows [n][heads][d] rotated in the precision of c and s; columns past the rotated ones are kept."""
    n = c.shape[-1]
    x = x.to(c.dtype)
    rot, rest = x[..., :2 * n], x[..., 2 * n:]
    a, b = (rot[..., :n], rot[..., n:]) if halves else (rot[..., 0::2], rot[..., 1::2])
    y = (a * c - b * s, a * s + b * c)
    y = torch.cat(y, -1) if halves else torch.stack(y, -1).flatten(-2)
    return torch.cat([y, rest], -1)


def _slots(st, pos, n):
    """Page and place in it of the rows at positions pos of their sequences."""
    seq = _seq_of_row(st["cu_rows"], n)
    pos = pos.long()
    return st["page_table"][seq, pos // st["page"]].long(), pos % st["page"]


def _padded(st, dtype):
    """Queries [seqs][kv_heads][group][rows][d] and the cache [seqs][kv_heads][length][d] of every sequence, padded,
    the visible length of each row, and where the rows came from."""
    q, cu, lens = st["q"], st["cu_rows"].long(), st["lens"].long()
    h, d = st["kv_heads"], st["d"]
    g = st["heads"] // h
    r = torch.arange(st["max_rows"], device=DEV)
    at = cu[:-1, None] + r
    real = at < cu[1:, None]
    at = at.clamp(max=max(q.shape[0] - 1, 0))
    qp = q[at].to(dtype).view(len(lens), st["max_rows"], h, g, d).permute(0, 2, 3, 1, 4)
    j = torch.arange(st["max_len"], device=DEV)
    page = st["page_table"].long()[:, (j // st["page"])].clamp(0, st["k_pages"].shape[0] - 1)
    # the pages of a shorter sequence end before the padded length: what is read there is masked, as finite values
    live = (j < lens[:, None])[..., None, None]
    zero = torch.zeros((), dtype=dtype, device=DEV)
    k, v = (torch.where(live, x[page, j % st["page"]].to(dtype), zero).transpose(1, 2)
            for x in (st["k_pages"], st["v_pages"]))
    seen = lens[:, None].expand(-1, st["max_rows"])
    if st["limits"] is not None:
        seen = torch.minimum(seen, st["limits"].long()[at])
    return qp, k, v, seen, at, real


def _attend(st, dtype):
    qp, k, v, seen, at, real = _padded(st, dtype)
    n, h, g, r, d = qp.shape
    scores = torch.matmul(qp.reshape(n, h, g * r, d), k.transpose(2, 3)).mul_(d ** -0.5).view(n, h, g, r, -1)
    masked = torch.arange(k.shape[2], device=DEV) >= seen[:, None, None, :, None]
    scores.masked_fill_(masked, -math.inf)
    top = scores.amax(-1, keepdim=True).clamp(min=-3e38)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(n, h, g * r, -1), v).view(n, h, g, r, d)
    o = torch.where(total > 0, o / total, torch.zeros((), dtype=dtype, device=DEV))
    o = o.permute(0, 3, 1, 2, 4).reshape(n, r, h * g, d)
    out = torch.zeros(st["q"].shape, dtype=dtype, device=DEV)
    out[at[real]] = o[real]
    return out


def run(state):
    st = state
    if own:
        return _run_own(st)
    if st["op"] == "rope":
        c, s = _cos_sin(st, st["ids"])
        return _rotate(st["x"], c, s, st["halves"]).bfloat16()
    if st["op"] == "attend":
        return _attend(st, torch.float32).bfloat16()
    if st["op"] == "scatter":
        c, s = _cos_sin(st, st["ids"])
        at = st["ids"].long()
        st["k_cache"][at] = _rotate(st["k"], c, s, st["halves"]).bfloat16()
        st["v_cache"][at] = st["v"]
        return _rotate(st["q"], c, s, st["halves"]).bfloat16(), st["k_cache"], st["v_cache"]
    c, s = _cos_sin(st, st["pos"])
    page, place = _slots(st, st["pos"], st["q"].shape[0])
    st["k_pages"][page, place] = _rotate(st["k"], c, s, st["halves"]).bfloat16()
    st["v_pages"][page, place] = st["v"]
    return _rotate(st["q"], c, s, st["halves"]).bfloat16(), st["k_pages"], st["v_pages"]


# ------------------------------------------------------------------ this package's calls
def _run_own(st):
    import kv_cache_analyzer_b200 as J
    if st["op"] == "attend":
        return J.paged_attention(st["q"], st["k_pages"], st["v_pages"], st["page_table"], st["lens"], st["cu_rows"],
                                 limits=st["limits"], max_rows=st["max_rows"], max_len=st["max_len"])
    frames, th, tw = _ints(st["grid"])
    rope = J.Rope(axes=tuple(_ints(st["axes"])), n_pos=(frames, th, tw), grid=(th, tw), theta=THETA,
                  pairing="halves" if st["halves"] else "interleaved")
    if st["op"] == "rope":
        return J.axis_rope(st["x"], rope, st["table"], ids=st["ids"])
    if st["op"] == "scatter":
        q = J.rope_scatter(st["k"], st["v"], st["ids"], st["k_cache"], st["v_cache"], rope, st["table"], q=st["q"])
        return q, st["k_cache"], st["v_cache"]
    q = J.paged_append(st["k"], st["v"], st["pos"], st["k_pages"], st["v_pages"], st["page_table"], st["lens"],
                       st["cu_rows"], rope=rope, table=st["table"], q=st["q"])
    return q, st["k_pages"], st["v_pages"]


# ------------------------------------------------------------------ what a pass cannot do without
def _visible(case):
    """Per sequence its rows' visible keys, summed, and the keys that any row sees."""
    f = {"none": 0, "token": 1, "frame": case["frame"]}[case["mask"]]
    total, keys = 0, 0
    for r, m in zip(_rows_of(case), _lens_of(case)):
        seen = [m if f == 0 else min(m, (p // f + 1) * f) for p in range(m - r, m)]
        total += sum(seen)
        keys += max(seen, default=0)
    return total, keys


def work(case):
    d = case["d"]
    if case["op"] == "attend":
        total, keys = _visible(case)
        n = sum(_rows_of(case))
        return {"bytes": 2.0 * d * (2 * n * case["heads"] + 2 * keys * case["kv_heads"]),
                "flops": 4.0 * d * case["heads"] * total}
    rows = sum(_rows_of(case)) if case["op"] == "append" else case["rows"]
    rotated = case["heads"] + (case["kv_heads"] if case["op"] != "rope" else 0)
    moved = rotated + (case["kv_heads"] if case["op"] != "rope" else 0)
    return {"bytes": 2.0 * 2.0 * rows * moved * d + 4.0 * rows, "flops": 3.0 * rows * rotated * sum(_ints(case["axes"]))}


# ------------------------------------------------------------------ the definition in 64 bits
def _turned(case, x, ids):
    """Rows x [n][heads][d] at token ids: every pair as a complex number, times exp(i angle)."""
    _, th, tw = _ints(case["grid"])
    ids = ids.double()
    row = torch.floor(ids / tw)
    at = (torch.floor(row / th), row - th * torch.floor(row / th), ids - tw * row)
    angle = torch.cat([p[:, None] / THETA ** (torch.arange(0, a, 2, dtype=torch.float64, device=DEV) / max(a, 1))
                       for p, a in zip(at, _ints(case["axes"]))], 1)[:, None, :]
    x = x.double()
    n = angle.shape[-1]
    first = list(range(n)) if case["halves"] else list(range(0, 2 * n, 2))
    second = [i + n if case["halves"] else i + 1 for i in first]
    z = torch.complex(x[..., first], x[..., second]) * torch.polar(torch.ones_like(angle), angle)
    y = x.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rope":
        return _turned(case, st["x"], st["ids"])
    if case["op"] == "scatter":
        k, v = st["k_cache"].double(), st["v_cache"].double()
        k.index_copy_(0, st["ids"].long(), _turned(case, st["k"], st["ids"]))
        v.index_copy_(0, st["ids"].long(), st["v"].double())
        return _turned(case, st["q"], st["ids"]), k, v
    cu, table = st["cu_rows"].tolist(), st["page_table"].tolist()
    if case["op"] == "append":
        k, v = st["k_pages"].double(), st["v_pages"].double()
        kt, p = _turned(case, st["k"], st["pos"]), case["page"]
        seq = [s for s in range(len(cu) - 1) for _ in range(cu[s + 1] - cu[s])]
        pos = st["pos"].tolist()
        page = torch.tensor([table[s][i // p] for s, i in zip(seq, pos)], device=DEV)
        place = torch.tensor([i % p for i in pos], device=DEV)
        k.index_put_((page, place), kt)
        v.index_put_((page, place), st["v"].double())
        return _turned(case, st["q"], st["pos"]), k, v
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV)
    g = case["heads"] // case["kv_heads"]
    for s, m in enumerate(_lens_of(case)):
        a, b = cu[s], cu[s + 1]
        pages = torch.tensor(table[s][:-(-m // case["page"])], device=DEV)
        k, v = (x[pages].flatten(0, 1)[:m].double() for x in (st["k_pages"], st["v_pages"]))
        lim = torch.full((b - a,), m, device=DEV) if st["limits"] is None else st["limits"][a:b].long()
        hidden = torch.arange(m, device=DEV)[None, :] >= lim[:, None]
        for h in range(case["heads"]):
            z = st["q"][a:b, h].double() @ k[:, h // g].T / math.sqrt(case["d"])
            w = torch.softmax(z.masked_fill(hidden, -math.inf), 1)
            out[a:b, h] = torch.nan_to_num(w, nan=0.0) @ v[:, h // g]
    return out
