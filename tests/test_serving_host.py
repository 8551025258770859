"""PagedBatch's bookkeeping of generations on the host.  No GPU is needed."""
import contextlib

import numpy as np
import pytest
import torch

import kv_cache_analyzer_b200.paged as P
from kv_cache_analyzer_b200.serving import PagedBatch


@pytest.fixture
def batch():
    return PagedBatch(n_pages=10, page_size=16, heads=4, kv_heads=2, d=64, device="cpu")


@pytest.mark.parametrize("n,error", [(-1, ValueError), (161, RuntimeError), (2.5, TypeError), (32.0, TypeError),
                                     ("32", TypeError), (None, TypeError), (float("nan"), TypeError)])
def test_a_refused_generation_leaves_nothing_behind(batch, n, error):
    kept = batch.open(20)
    state = dict(batch._gens[kept], pages=list(batch._gens[kept]["pages"]))
    free = list(batch._free)
    with pytest.raises(error):
        batch.open(n)
    assert list(batch._gens) == [kept] and batch._free == free
    # and a refused growth leaves the generation as it was
    with pytest.raises(error):
        batch.extend(kept, n)
    assert batch._gens[kept] == state and batch._free == free
    with pytest.raises(KeyError):
        batch.extend(kept + 1, 40)
    assert batch.open(32) != kept and batch.free_pages == 10 - 2 - 2


def test_token_counts_may_be_numpy_integers(batch):
    g = batch.open(np.int64(33))
    batch.extend(g, np.int32(49))
    assert batch.free_pages == 6
    assert batch.plan([(g, 3)]).lists["seq_lens"].tolist() == [49]


def test_a_rotations_table_is_made_on_the_batchs_device(monkeypatch):
    # (another device than the current one: pools and table have to meet in one call)
    rope = P.Rope(axes=(16, 24, 24), n_pos=(2, 5, 7), grid=(5, 7))
    inside, seen = [], []

    @contextlib.contextmanager
    def on_device(device):
        inside.append(torch.device(device))
        yield
        inside.pop()

    monkeypatch.setattr(torch.cuda, "device", on_device)
    monkeypatch.setattr(P, "_new", lambda stream, shape, like: seen.append(("made", list(inside))) or torch.empty(shape))
    monkeypatch.setattr(P, "_device", lambda t, name: -1)
    monkeypatch.setattr(P, "jano_rope_table", lambda *a: seen.append(("filled", list(inside))))
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: empty(*a, **{**kw, "device": "cpu"}))
    b = PagedBatch(n_pages=4, page_size=16, heads=4, d=64, rope=rope, device="cuda:3")
    assert b.table.shape == (rope.entries, 2)
    assert seen == [("made", [torch.device("cuda:3")]), ("filled", [torch.device("cuda:3")])]
    seen.clear()
    P.rope_table(rope, device="cuda:1")
    assert seen == [("made", [torch.device("cuda:1")]), ("filled", [torch.device("cuda:1")])]
    # a table that the caller brings stays where it is
    seen.clear()
    P.rope_table(rope, torch.zeros(rope.entries, 2))
    assert seen == [("filled", [])]
