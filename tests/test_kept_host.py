"""Trees of drafted tokens, accumulated weight and the cutting of a cache: what is refused, and the oracle's pins (no GPU)."""
import math

import numpy as np
import pytest

import oracle
from test_paged_host import BAD_BATCHES, BAD_CACHES, BAD_ROWS, batch_of, cache_of, rows_of, sp  # noqa: F401

BIG = 1 << 40
WS = 65536


def tree_attend(sp, rows, cache, batch, **over):
    a = dict(H=4, scale=0.125, window=0, seen=512, stride=1, words=1, out=rows, lse=None, ws=WS, size=BIG)
    a.update(over)
    return sp.sp_attend_tree(rows, cache, batch, a["H"], a["scale"], a["window"], a["seen"], a["stride"], a["words"], a["out"],
                             a["lse"], 0, 0, a["ws"], a["size"], 0)


def weights(sp, rows, cache, batch, **over):
    a = dict(H=4, scale=0.125, window=0, lse=1024, decay=1.0, weights=2048, ws=WS, size=BIG)
    a.update(over)
    return sp.sp_attend_weights(rows, cache, batch, a["H"], a["scale"], a["window"], a["lse"], 1, 10, a["decay"], a["weights"],
                                a["ws"], a["size"], 0)


def choose(sp, cache, batch, **over):
    a = dict(weights=2048, shared=0, budget=8, first=1, last=2, kept=4096, seq=16, head=8, n=8192, ws=WS, size=BIG)
    a.update(over)
    return sp.sp_cache_choose(cache, batch, a["weights"], a["shared"], a["budget"], a["first"], a["last"], a["kept"], a["seq"],
                              a["head"], a["n"], a["ws"], a["size"], 0)


def keep(sp, cache, batch, **over):
    a = dict(kept=4096, heads=2, seq=16, head=8, n=8192, most=8, drafted=0, to=None, width=0, to_stride=0, weights=None, out=8448,
             ws=WS, size=BIG)
    a.update(over)
    return sp.sp_cache_keep(cache, batch, a["kept"], a["heads"], a["seq"], a["head"], a["n"], a["most"], a["drafted"], a["to"],
                            a["width"], a["to_stride"], a["weights"], a["out"], a["ws"], a["size"], 0)


def seen(sp, batch, **over):
    a = dict(parent=512, seen=1024, stride=1, words=1, pos=2048, ws=WS, size=BIG)
    a.update(over)
    return sp.sp_tree_seen(batch, a["parent"], a["seen"], a["stride"], a["words"], a["pos"], a["ws"], a["size"], 0)


def accept(sp, batch, **over):
    a = dict(parent=512, draft=1024, target=1536, path=2048, stride=5, n=4096, next=None, ws=WS, size=BIG)
    a.update(over)
    return sp.sp_tree_accept(batch, a["parent"], a["draft"], a["target"], a["path"], a["stride"], a["n"], a["next"], a["ws"],
                             a["size"], 0)


@pytest.mark.parametrize("over,status", BAD_CACHES)
def test_bad_caches_are_refused(sp, over, status):  # noqa: F811
    c, b, r = cache_of(sp, **over), batch_of(sp), rows_of(sp)
    for name, s in (("tree", tree_attend(sp, r, c, b)), ("weights", weights(sp, r, c, b)), ("choose", choose(sp, c, b)), ("keep", keep(sp, c, b))):
        assert sp.sp_status_string(s) == status, name
    assert sp.sp_attend_tree_workspace_size(c, b, 4) == 0 and sp.sp_attend_weights_workspace_size(c, b, 4) == 0


@pytest.mark.parametrize("over", BAD_BATCHES)
def test_bad_batches_are_refused(sp, over):  # noqa: F811
    c, b, r = cache_of(sp), batch_of(sp, **over), rows_of(sp)
    for name, s in (("tree", tree_attend(sp, r, c, b)), ("weights", weights(sp, r, c, b)), ("choose", choose(sp, c, b)), ("keep", keep(sp, c, b)),
                    ("seen", seen(sp, b)), ("accept", accept(sp, b))):
        assert s == sp.SP_EINVAL, name


@pytest.mark.parametrize("over", BAD_ROWS)
def test_bad_rows_are_refused(sp, over):  # noqa: F811
    bad, c, b, good = None if over is None else rows_of(sp, **over), cache_of(sp), batch_of(sp), rows_of(sp)
    assert tree_attend(sp, bad, c, b) == sp.SP_EINVAL
    assert tree_attend(sp, good, c, b, out=bad) == sp.SP_EINVAL
    assert weights(sp, bad, c, b) == sp.SP_EINVAL


@pytest.mark.parametrize("over", [
    dict(seen=None), dict(seen=514), dict(words=0), dict(stride=-1), dict(H=3), dict(H=0), dict(scale=0.0), dict(scale=math.nan),
    dict(window=-1), dict(lse=6), dict(ws=None), dict(ws=65544),
])
def test_attend_tree_refusals(sp, over):  # noqa: F811
    assert tree_attend(sp, rows_of(sp), cache_of(sp), batch_of(sp), **over) == sp.SP_EINVAL
    assert sp.sp_last_error()


def test_words_must_hold_the_new_tokens(sp):  # noqa: F811
    b = batch_of(sp, max_new=33, T=70)
    assert tree_attend(sp, rows_of(sp), cache_of(sp), b) == sp.SP_EINVAL
    assert seen(sp, b, words=1) == sp.SP_EINVAL
    assert seen(sp, b, words=2, stride=1) == sp.SP_EINVAL           # rows that overlap
    assert tree_attend(sp, rows_of(sp), cache_of(sp), b, words=2, stride=2, size=100) == sp.SP_ENOMEM


@pytest.mark.parametrize("over", [
    dict(lse=None), dict(lse=1026), dict(weights=None), dict(weights=2050), dict(decay=-0.1), dict(decay=1.5), dict(decay=math.nan), dict(H=5),
    dict(scale=-1.0), dict(window=-2), dict(ws=None),
])
def test_weights_refusals(sp, over):  # noqa: F811
    assert weights(sp, rows_of(sp), cache_of(sp), batch_of(sp), **over) == sp.SP_EINVAL
    assert weights(sp, rows_of(sp), cache_of(sp), batch_of(sp), size=64) == sp.SP_ENOMEM


@pytest.mark.parametrize("over", [
    dict(weights=None), dict(budget=-1), dict(budget=1 << 31), dict(first=-1), dict(last=-1), dict(first=5, last=4), dict(first=9, last=0),
    dict(kept=None), dict(kept=4098), dict(n=None), dict(n=8196), dict(head=4), dict(seq=8), dict(seq=0), dict(ws=None),
])
def test_choose_refusals(sp, over):  # noqa: F811
    assert choose(sp, cache_of(sp), batch_of(sp), **over) == sp.SP_EINVAL
    assert choose(sp, cache_of(sp), batch_of(sp), size=64) == sp.SP_ENOMEM
    assert choose(sp, cache_of(sp, H_kv=60000, stride_head=1024, stride_page=60000 * 1024), batch_of(sp, B=60000)) == sp.SP_EUNSUPPORTED


@pytest.mark.parametrize("over", [
    dict(kept=None), dict(kept=4099), dict(heads=3), dict(heads=0), dict(n=None), dict(most=-1), dict(most=1 << 31), dict(out=None), dict(out=8449),
    dict(out=128), dict(out=8192), dict(to=514, width=4), dict(to=512, width=0), dict(to=512, width=4, to_stride=-1), dict(weights=3), dict(ws=None),
])
def test_keep_refusals(sp, over):  # noqa: F811
    assert keep(sp, cache_of(sp), batch_of(sp), **over) == sp.SP_EINVAL
    assert keep(sp, cache_of(sp), batch_of(sp), size=64) == sp.SP_ENOMEM
    for c in (dict(stride_page=0), dict(stride_head=0), dict(stride_page=1024)):        # places that overlap
        assert keep(sp, cache_of(sp, **c), batch_of(sp)) == sp.SP_EINVAL


@pytest.mark.parametrize("over", [
    dict(parent=None), dict(parent=513), dict(seen=None, pos=None), dict(seen=1026), dict(pos=2050), dict(ws=None), dict(words=0), dict(stride=0),
])
def test_tree_seen_refusals(sp, over):  # noqa: F811
    assert seen(sp, batch_of(sp), **over) == sp.SP_EINVAL
    assert seen(sp, batch_of(sp), size=64) == sp.SP_ENOMEM


@pytest.mark.parametrize("over", [
    dict(parent=None), dict(draft=None), dict(target=1537), dict(path=None), dict(path=2049), dict(stride=4), dict(n=None), dict(n=4100), dict(next=3),
    dict(ws=None),
])
def test_tree_accept_refusals(sp, over):  # noqa: F811
    assert accept(sp, batch_of(sp), **over) == sp.SP_EINVAL
    assert accept(sp, batch_of(sp), size=64) == sp.SP_ENOMEM


def test_outputs_in_the_place_of_what_is_read_are_refused(sp):  # noqa: F811
    c, b = cache_of(sp), batch_of(sp)           # cu_new at 64 (24 bytes), kv_len at 128 (16), rows of 40 bytes
    for s in (choose(sp, c, b, n=128), choose(sp, c, b, n=136), choose(sp, c, b, n=120), choose(sp, c, b, n=80),
              keep(sp, c, b, out=128), keep(sp, c, b, out=136), keep(sp, c, b, out=8200), keep(sp, c, b, out=8184), keep(sp, c, b, out=64),
              seen(sp, b, pos=512), seen(sp, b, pos=548), seen(sp, b, seen=476), seen(sp, b, seen=None, pos=128),
              accept(sp, b, path=512), accept(sp, b, path=1024), accept(sp, b, path=1572), accept(sp, b, path=1500), accept(sp, b, n=128),
              accept(sp, b, n=1568), accept(sp, b, next=1024), accept(sp, b, next=80)):
        assert s == sp.SP_EINVAL and "read meanwhile" in sp.sp_last_error()


def test_python_checks(sp):  # noqa: F811
    import torch
    i64 = lambda *v: torch.tensor(v, dtype=torch.int64)                                         # noqa: E731
    batch = sp.Batch(i64(0, 3, 5), i64(9, 7), torch.zeros(2, 1, dtype=torch.int32), rows=5, max_new=3)
    cache = sp.Cache(torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16), torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16))
    q, ids = torch.zeros(5, 4, 64, dtype=torch.bfloat16), torch.zeros(5, dtype=torch.int32)
    bits = torch.zeros(5, 1, dtype=torch.int32)
    lse, w = torch.zeros(4, 5), torch.zeros(4, 2, 16)
    lists, n = torch.zeros(2, 2, 8, dtype=torch.int32), i64(1, 1)
    bad = [
        lambda: sp.tree_seen(batch, ids[:4]), lambda: sp.tree_seen(batch, ids.long()), lambda: sp.tree_seen(batch, ids, seen=bits[:3]),
        lambda: sp.tree_seen(batch, ids, positions=torch.zeros(10, dtype=torch.int32)[::2]),
        lambda: sp.attend_tree(q, cache, batch, bits[:3]), lambda: sp.attend_tree(q, cache, batch, bits.long()),
        lambda: sp.attend_tree(q, cache, batch, torch.zeros(5, 4, dtype=torch.int32)[:, ::2]), lambda: sp.attend_tree(q[:4], cache, batch, bits),
        lambda: sp.tree_accept(batch, ids, ids, ids[:2]), lambda: sp.tree_accept(batch, ids, ids, ids, path=torch.zeros(2, 4, dtype=torch.int32)),
        lambda: sp.tree_accept(batch, ids, ids, ids, n_path=n.int()), lambda: sp.tree_accept(batch, ids, ids, ids, next_token=n),
        lambda: sp.attend_weights(q, cache, batch, lse[:, :4], w), lambda: sp.attend_weights(q, cache, batch, lse.double(), w),
        lambda: sp.attend_weights(q, cache, batch, lse, w[:3]), lambda: sp.attend_weights(q, cache, batch, lse, w.transpose(1, 2)),
        lambda: sp.attend_weights(q[..., :32], cache, batch, lse, w),
        lambda: sp.cache_choose(cache, batch, w.double(), 8), lambda: sp.cache_choose(cache, batch, w, 8, kept=lists[:, :1]),
        lambda: sp.cache_choose(cache, batch, w, 8, shared=True, kept=lists), lambda: sp.cache_choose(cache, batch, w, 8, n_kept=n.int()),
        lambda: sp.cache_keep(cache, batch, lists[:1], n), lambda: sp.cache_keep(cache, batch, lists, n[:1]),
        lambda: sp.cache_keep(cache, batch, lists.long(), n), lambda: sp.cache_keep(cache, batch, lists, n, to=ids),
        lambda: sp.cache_keep(cache, batch, lists, n, weights=w[:1]), lambda: sp.cache_keep(cache, batch, lists, n, kv_len=n.int()),
        # on the CPU all along
        lambda: sp.tree_seen(batch, ids), lambda: sp.cache_choose(cache, batch, w, 8), lambda: sp.attend_weights(q, cache, batch, lse, w),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()


def test_oracle_of_a_tree():
    parent = [-1, 0, 0, 1, 3, -1]
    see, depth = oracle.kept.tree_seen(parent)
    assert depth.tolist() == [0, 1, 1, 2, 3, 0]
    assert [np.flatnonzero(s).tolist() for s in see] == [[0], [0, 1], [0, 2], [0, 1, 3], [0, 1, 3, 4], [5]]
    assert oracle.kept.words(see, 1)[:, 0].tolist() == [1, 3, 5, 11, 27, 32]
    assert oracle.kept.words(np.ones((1, 40), bool), 2).tolist() == [[0xffffffff, 0xff]]
    v = oracle.kept.visible(6, 9, 2, see)
    # places 3 4 4 5 6 3: a window of two hides all but the place before, if that is a cached token
    assert [np.flatnonzero(x).tolist() for x in v] == [[2, 3], [3, 4], [3, 5], [3, 4, 6], [3, 4, 6, 7], [2, 8]]
    assert oracle.kept.visible(2, 4).tolist() == [[True] * 3 + [False], [True] * 4]
    assert oracle.kept.accept(parent, [7, 5, 6, 8, 9, 1], [6, 0, 4, 0, 0, 0]) == ([0, 2], 4)
    assert oracle.kept.accept(parent, [7, 5, 5, 8, 9, 1], [5, 8, 4, 9, 3, 0]) == ([0, 1, 3, 4], 3)
    assert oracle.kept.accept([], [], []) == ([], -1)


def test_oracle_of_a_chain_is_causal():
    rng = np.random.default_rng(0)
    q, k, v = rng.standard_normal((5, 4, 8)), rng.standard_normal((2, 9, 8)), rng.standard_normal((2, 9, 8))
    see = oracle.kept.visible(5, 9, 0, oracle.kept.tree_seen(np.arange(5) - 1)[0])
    for a, b in zip(oracle.kept.attend(q, k, v, 0.3, see), oracle.paged.attend(q, k, v, 0.3)):
        assert np.allclose(a, b, rtol=1e-12, atol=1e-12)
    # the weights of each row add up to one
    lse = oracle.paged.attend(q, k, v, 0.3)[1]
    w, bound = oracle.kept.weights(q, k, lse, 0.3, see)
    assert np.allclose(w.sum(), 5 * 4) and np.all(bound < 1e-4 * w + 1e-30) and w.shape == (2, 9)
    # by hand: one row, equal keys
    w, _ = oracle.kept.weights(np.ones((1, 1, 8)), np.ones((1, 4, 8)), np.full((1, 1), 8 + np.log(4)), 1.0, np.ones((1, 4), bool))
    assert np.allclose(w, 0.25)


def test_oracle_of_the_choice():
    w = np.array([1, 5, 3, 5, 0, 2], np.float32)
    assert oracle.kept.choose(w, 2, 0, 0).tolist() == [1, 3]
    assert oracle.kept.choose(w, 3, 1, 1).tolist() == [0, 1, 5]
    assert oracle.kept.choose(w, 6, 1, 1).tolist() == list(range(6)) and oracle.kept.choose(w, 0, 0, 0).tolist() == []
    odd = np.array([np.nan, -np.inf, 0.0, -0.0, 1.0], np.float32)
    assert oracle.kept.choose(odd, 2, 0, 0).tolist() == [2, 4]
    assert oracle.kept.choose(odd, 4, 0, 0).tolist() == [1, 2, 3, 4]
