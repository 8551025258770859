"""Shared by the tests of the rotary positions and the paged cache: seeded
problems, and the tolerances that the arithmetic allows."""
import numpy as np
import torch

import oracle.paged as op
import synth


def f64(t):
    return synth.bf16_to_f32(synth.bits_of(t.detach().cpu().contiguous())).astype(np.float64)


def bits(t):
    return synth.bits_of(t.detach().cpu().contiguous())


def check_rope(got, x, coords, axes, theta=10000.0, halves=False, shared=False):
    """got, x BF16 tensors [n][heads][d].  Per element: the output's rounding,
    2^-8 |y|, and in fp32 the rounding of cos and sin, of one product and of
    the fused sum, each at most 2^-24 of |x0| + |x1|: together below
    2^-22 (|x0| + |x1|), itself rounded up by the output's step."""
    xf = f64(x)
    ref = op.rope(xf, coords, axes, theta, halves, shared)
    bound = 2.0 ** -8 * np.abs(ref) + 2.0 ** -21 * op.rope_partner(xf, axes, halves)
    err = np.abs(f64(got) - ref)
    assert np.all(err <= bound), float((err - bound).max())
    rot = sum(axes)
    np.testing.assert_array_equal(bits(got)[..., rot:], bits(x)[..., rot:])


def check_attention(got, q, k, v, limits, scale):
    """got BF16 [n][heads][d]; q, k, v fp64 of one sequence.  Per element
    2^-8 |o| (output rounding) + sum p |v| times: 2^-8 (P rounded to BF16),
    2^-15 A (the logits' fp32 sums of d BF16 products, off by at most 2^-16 of
    A = max scale * sum |q| |k|, move a weight by twice that), 2^-12 (exp2,
    scale and the fp32 sums over the keys)."""
    ref, pv, top = op.attention(q, k, v, limits, scale)
    bound = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -15 * top + 2.0 ** -12) * pv
    err = np.abs(f64(got) - ref)
    assert np.all(err <= bound), (float((err - bound).max()), np.argwhere(err > bound)[:3].tolist())
    dark = np.asarray(limits) <= 0
    assert not np.any(bits(got)[dark]), "a row that sees nothing is 0"


class Paged:
    """Sequences of given rows and lengths over a pool whose pages are handed
    out in a seeded order; places past a sequence's length and pages that
    nobody owns hold NaN."""

    def __init__(self, rows, lens, heads, kv_heads, d, page, seed=0, head_major=False, pad_rows=0, dev="cuda",
                 one_buffer=False, spare=3):
        gen = np.random.default_rng(seed)
        self.rows, self.lens, self.heads, self.kv_heads, self.d, self.page = rows, lens, heads, kv_heads, d, page
        per = [-(-n // page) for n in lens]
        self.n_pages = sum(per) + spare
        order = gen.permutation(self.n_pages).astype(np.int32)
        self.max_pages = max(per + [1]) + 1
        # entries past a sequence's pages are never read: an id outside the pool stands there
        self.table = np.full((len(lens), self.max_pages), 2 ** 30, dtype=np.int32)
        at = 0
        for s, n in enumerate(per):
            self.table[s, :n] = order[at:at + n]
            at += n
        self.cu = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        self.n = int(self.cu[-1]) + pad_rows
        tg = torch.Generator().manual_seed(seed)
        self.q = torch.randn((self.n, heads, d), generator=tg).bfloat16()
        k, v = (torch.full((self.n_pages, page, kv_heads, d), float("nan"), dtype=torch.bfloat16) for _ in range(2))
        for s, m in enumerate(lens):
            for i in range(per[s]):
                c = min(page, m - i * page)
                for t in (k, v):
                    t[self.table[s, i], :c] = torch.randn((c, kv_heads, d), generator=tg).bfloat16()
        self.k, self.v = k, v
        if dev is None:
            return
        put = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)
        self.dev_q = self.q.to(dev)
        if one_buffer:                       # [page][2][place][head][d]
            both = torch.stack([k, v], 1).to(dev)
            self.dev_k, self.dev_v = both[:, 0], both[:, 1]
        elif head_major:
            self.dev_k, self.dev_v = (t.transpose(1, 2).contiguous().to(dev).transpose(1, 2) for t in (k, v))
        else:
            self.dev_k, self.dev_v = k.to(dev), v.to(dev)
        self.dev_table, self.dev_cu = put(self.table), put(self.cu)
        self.dev_lens = put(np.asarray(lens, dtype=np.int32))

    def seq(self, s):
        """fp64 K and V of sequence s."""
        m = self.lens[s]
        shape = (m, self.kv_heads, self.d)
        if m == 0:
            return np.zeros(shape), np.zeros(shape)
        return tuple(op.gather(f64(t), self.table[s], m) for t in (self.k, self.v))

    def check(self, out, limits=None, scale=None):
        scale = self.d ** -0.5 if scale is None else scale
        for s in range(len(self.lens)):
            a, b = int(self.cu[s]), int(self.cu[s + 1])
            if a == b:
                continue
            k, v = self.seq(s)
            lim = np.full(b - a, 2 ** 31 - 1) if limits is None else limits[a:b]
            lim = np.minimum(lim, self.lens[s])
            check_attention(out[a:b], f64(self.q[a:b]), k, v, lim, scale)
