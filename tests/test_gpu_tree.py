"""Trees of drafted tokens on the GPU, against the 64-bit oracle: their bits and positions, the attention, the accepted path."""
import numpy as np
import pytest

import oracle
from paged_helpers import attend_bounds, make_batch, make_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sp():
    import torch
    assert torch.cuda.is_available(), "the GPU tests need a CUDA device"
    from speculative_prefill_token_sp_gb300 import build
    build.build()
    import speculative_prefill_token_sp_gb300 as m
    m.lib()
    return m


def torch_dtype(name):
    import torch
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def f64(t):
    return t.detach().double().cpu().numpy()


def i32(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a).astype(np.int32)).cuda()


def tree(rng, n, shape):
    """Parents of n tokens: a chain, a star, roots alone, or one after the other at random."""
    if shape == "chain":
        return np.arange(n) - 1
    if shape == "star":
        return np.where(np.arange(n) == 0, -1, 0)
    if shape == "roots":
        return np.full(n, -1)
    return np.array([rng.integers(-1 if t % 7 == 0 else 0, t) if t else -1 for t in range(n)], dtype=np.int64)


def plain_batch(sp, new, kv, *, first=0, behind=0, max_new=None):
    """A batch whose table is never read."""
    import torch
    cu = np.concatenate([[first], first + np.cumsum(new)]).astype(np.int64)
    return sp.Batch(torch.from_numpy(cu).cuda(), torch.tensor(kv, dtype=torch.int64, device="cuda"),
                    torch.full((len(new), 1), -5, dtype=torch.int32, device="cuda"), rows=int(cu[-1]) + behind,
                    max_new=max(new) if max_new is None else max_new), cu


@pytest.mark.parametrize("shape", ["chain", "star", "roots", "random"])
@pytest.mark.parametrize("new,kv,max_new", [
    ([1], [1], None), ([5, 0, 33], [700, 0, 40], None), ([64, 31, 32, 1], [64, 5, 1 << 30, 9], 70), ([1000], [131072], None),
    ([3] * 300, [10] * 300, None),
])
def test_tree_seen(sp, new, kv, max_new, shape):
    import torch
    rng = np.random.default_rng(1)
    batch, cu = plain_batch(sp, new, kv, first=2, behind=3, max_new=max_new)
    parent = np.full(batch.rows, 77)
    for b, n in enumerate(new):
        parent[cu[b]:cu[b + 1]] = tree(rng, n, shape)
    words = -(-batch.max_new // 32) + 1
    seen = torch.full((batch.rows, words + 2), 7, dtype=torch.int32, device="cuda")
    pos = torch.full((batch.rows,), 7, dtype=torch.int32, device="cuda")
    sp.tree_seen(batch, i32(parent), seen=seen[:, :words], positions=pos, check=True)
    got, got_pos = seen.cpu().numpy(), pos.cpu().numpy()
    want, want_pos = np.full_like(got, 7), np.full_like(got_pos, 7)
    for b, n in enumerate(new):
        see, depth = oracle.kept.tree_seen(parent[cu[b]:cu[b + 1]])
        want[cu[b]:cu[b + 1], :words] = oracle.kept.words(see, words).view(np.int32)
        want_pos[cu[b]:cu[b + 1]] = kv[b] - n + depth
    assert np.array_equal(got, want) and np.array_equal(got_pos, want_pos)
    alone, p2 = sp.tree_seen(batch, i32(parent), check=True)
    rows = slice(2, 2 + sum(new))
    assert np.array_equal(alone.cpu().numpy()[rows], want[rows, :words - 1]) and np.array_equal(p2.cpu().numpy()[rows], want_pos[rows])


def test_bad_parents_are_roots_and_reported(sp):
    import torch
    batch, _ = plain_batch(sp, [6], [20])
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    seen, pos = sp.tree_seen(batch, i32([-1, 1, 0, 1 << 30, -(1 << 31), 4]), ws=ws)
    assert sp.sp_workspace_status(ws) == sp.SP_EDEVICE
    assert seen[:, 0].tolist() == [1, 2, 5, 8, 16, 48] and pos.tolist() == [14, 14, 15, 14, 14, 15]
    tok = i32([5, 5, 5, 5, 5, 5])
    path, n, nxt = sp.tree_accept(batch, i32([-1, 1, 0, 1 << 30, -(1 << 31), 4]), tok, tok, ws=ws)
    assert sp.sp_workspace_status(ws) == sp.SP_EDEVICE
    assert path[0].tolist() == [0, 2, -1, -1, -1, -1] and n.item() == 2 and nxt.item() == 5
    sp.tree_seen(batch, i32([-1, 0, 0, 1, 2, 4]), ws=ws)
    assert sp.sp_workspace_status(ws) == sp.SP_OK
    # impossible offsets: the sequence is left out
    batch, _ = plain_batch(sp, [3, 2], [20, 9], max_new=2)
    seen = torch.full((5, 1), 7, dtype=torch.int32, device="cuda")
    sp.tree_seen(batch, i32([-1, 0, 1, -1, 0]), seen=seen, ws=ws)
    assert sp.sp_workspace_status(ws) == sp.SP_EDEVICE and seen[:, 0].tolist() == [7, 7, 7, 1, 3]
    path, n, nxt = sp.tree_accept(batch, i32([-1, 0, 1, -1, 0]), i32([1] * 5), i32([1] * 5), ws=ws)
    assert sp.sp_workspace_status(ws) == sp.SP_EDEVICE
    assert n.tolist() == [0, 2] and path.tolist() == [[-1, -1], [0, 1]] and nxt.tolist() == [-1, 1]


def test_the_longest_chain_and_one_more(sp):
    import torch
    batch, cu = plain_batch(sp, [4096, 4097, 2], [5000, 4097, 9])
    parent = np.concatenate([np.arange(n) - 1 for n in (4096, 4097, 2)])
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    seen = torch.full((batch.rows, 129), 7, dtype=torch.int32, device="cuda")
    pos = torch.full((batch.rows,), 7, dtype=torch.int32, device="cuda")
    sp.tree_seen(batch, i32(parent), seen=seen, positions=pos, ws=ws)
    assert sp.sp_workspace_status(ws) == sp.SP_EDEVICE
    assert pos[:4096].tolist() == list(range(904, 5000)) and torch.all(pos[4096:8193] == 7) and pos[8193:].tolist() == [7, 8]
    assert torch.all(seen[4096:8193] == 7) and seen[8193:, 0].tolist() == [1, 3] and not seen[8193:, 1:].any()
    bits = seen[:4096, :128].cpu().numpy().view(np.uint32)
    t = np.arange(4096)[:, None]
    inside = np.clip(t + 1 - 32 * np.arange(128), 0, 32).astype(np.uint64)
    assert np.array_equal(bits, ((np.uint64(1) << inside) - np.uint64(1)).astype(np.uint32))


@pytest.mark.parametrize("new", [[1], [0, 7, 33, 64, 0], [1, 31, 32, 100], [1000], [24] * 40])
@pytest.mark.parametrize("agree", [0.0, 0.5, 1.0])
def test_tree_accept(sp, new, agree):
    import torch
    rng = np.random.default_rng(3)
    batch, cu = plain_batch(sp, new, [5 + n for n in new], first=1, behind=2, max_new=max(new) + 3)
    T = batch.rows
    parent = np.zeros(T, dtype=np.int64)
    draft, target = rng.integers(-5, 5, T), rng.integers(100, 105, T)
    for b, n in enumerate(new):
        parent[cu[b]:cu[b + 1]] = tree(rng, n, "chain" if agree == 1.0 else "random")
        for t in range(cu[b], cu[b + 1]):
            if parent[t] >= 0 and rng.random() < agree:
                target[cu[b] + parent[t]] = draft[t]           # several children may hold the same token
    path = torch.full((len(new), max(new) + 5), 9, dtype=torch.int32, device="cuda")
    p, n_path, nxt = sp.tree_accept(batch, i32(parent), i32(draft), i32(target), path=path[:, :max(new) + 3], check=True)
    assert torch.all(path[:, max(new) + 3:] == 9)
    for b, n in enumerate(new):
        lo, hi = cu[b], cu[b + 1]
        want, then = oracle.kept.accept(parent[lo:hi], draft[lo:hi], target[lo:hi])
        assert p[b].tolist() == want + [-1] * (max(new) + 3 - len(want))
        assert n_path[b].item() == len(want) and nxt[b].item() == then


def check_tree(sp, *, H, H_kv, d, page, new, kv, dtype="bf16", kind="same", window=0, shape="random", layout="hnd", before=1,
               behind=2, seed=0, seen=None, scale=None):
    import torch
    rng = np.random.default_rng(seed)
    td = torch_dtype(dtype)
    cache, table, kval, vval = make_cache(sp, rng, H_kv=H_kv, d=d, page=page, kv=kv, kind=kind, dtype=td, layout=layout,
                                          junk=float("nan"))
    T = before + sum(new) + behind
    batch, cu = make_batch(sp, new, kv, table, rows=T, first=before, max_new=max(new))
    see = []
    for b, n in enumerate(new):
        if seen == "any":           # bits of all kinds, rows without one among them
            s = rng.random((n, n)) < rng.choice([0.0, 0.1, 0.9], (n, 1))
        else:
            s = oracle.kept.tree_seen(tree(rng, n, shape))[0]
        see.append(s)
    words = max(1, -(-max(new) // 32)) + 1
    bits = np.full((T, words), 0xffffffff, dtype=np.uint32)     # also behind a sequence's last token: ignored there
    for b, n in enumerate(new):
        w = oracle.kept.words(see[b], words)
        for k in range(words):
            inside = min(max(n - 32 * k, 0), 32)
            w[:, k] |= np.uint32((0xffffffff << inside) & 0xffffffff)
        bits[cu[b]:cu[b + 1]] = w
    q = torch.from_numpy(rng.standard_normal((T, H, d))).to(td)
    real = np.zeros(T, dtype=bool)
    real[before:before + sum(new)] = True
    q[~torch.from_numpy(real)] = float("nan")
    out = torch.full((T, H, d), 7.0, dtype=td, device="cuda")
    lse = torch.full((H, T), 7.0, dtype=torch.float32, device="cuda")
    sp.attend_tree(q.cuda(), cache, batch, i32(bits.view(np.int32)), scale=scale, window=window, out=out, lse=lse, check=True)
    got, got_lse = f64(out), f64(lse)
    assert np.all(got[~real] == 7) and np.all(got_lse[:, ~real] == 7)
    qd = q.double().numpy()
    for b, n in enumerate(new):
        lo, hi = int(cu[b]), int(cu[b + 1])
        if not n:
            continue
        ref, ref_lse, top, spread = oracle.kept.attend(qd[lo:hi], kval[b], vval[b], d ** -0.5 if scale is None else scale,
                                                       oracle.kept.visible(n, kv[b], window, see[b]))
        bound, lse_bound = attend_bounds(dtype, d, max(kv[b], 1), ref, spread, top, ref_lse)
        err = np.abs(got[lo:hi] - ref)
        assert np.all(err <= bound), f"sequence {b}: out off by {np.nanmax(err / bound)} of its bound"
        empty = np.isneginf(ref_lse)
        assert np.array_equal(np.isneginf(got_lse[:, lo:hi]), empty)
        assert np.all(got[lo:hi][empty.T] == 0)
        with np.errstate(invalid="ignore"):
            assert np.all((np.abs(got_lse[:, lo:hi] - ref_lse) <= lse_bound) | empty)


@pytest.mark.parametrize("kind", ["same", "e4m3", "int8"])
@pytest.mark.parametrize("H,H_kv,d,page", [
    (4, 2, 64, 16), (8, 2, 128, 64), (3, 1, 64, 32), (16, 1, 128, 8), (7, 7, 64, 48), (5, 1, 40, 7), (2, 1, 256, 16), (3, 3, 8, 5),
])
@pytest.mark.parametrize("new,kv,window,shape", [
    ([1], [1], 0, "random"), ([4, 3, 0, 2], [4, 300, 0, 129], 0, "random"), ([16, 5], [500, 33], 0, "random"),
    ([2, 4], [40, 260], 33, "chain"), ([16], [300], 9, "random"),
])
def test_attend_tree_of_few(sp, H, H_kv, d, page, new, kv, window, shape, kind):
    check_tree(sp, H=H, H_kv=H_kv, d=d, page=page, new=new, kv=kv, kind=kind, window=window, shape=shape)


@pytest.mark.parametrize("kind", ["same", "e4m3", "int8"])
@pytest.mark.parametrize("H,H_kv,d,page", [(4, 2, 64, 16), (8, 2, 128, 64), (3, 1, 64, 8), (12, 1, 128, 256), (2, 2, 72, 7)])
@pytest.mark.parametrize("new,kv,window,shape", [
    ([33], [33], 0, "random"), ([64, 1, 65, 0], [64, 400, 200, 0], 0, "random"), ([100, 40], [260, 40], 37, "random"),
    ([130, 31], [131, 700], 0, "star"), ([50, 64], [1000, 129], 128, "chain"), ([200], [1200], 0, "roots"),
])
def test_attend_tree_of_many(sp, H, H_kv, d, page, new, kv, window, shape, kind):
    check_tree(sp, H=H, H_kv=H_kv, d=d, page=page, new=new, kv=kv, kind=kind, window=window, shape=shape)


@pytest.mark.parametrize("kind", ["same", "e4m3"])
@pytest.mark.parametrize("new,kv,window", [([8], [512], 0), ([5, 0, 40], [3, 0, 90], 0), ([33, 2], [300, 2], 21)])
@pytest.mark.parametrize("H,H_kv,d,page", [(4, 2, 64, 16), (3, 1, 128, 5)])
def test_attend_tree_in_single_precision(sp, H, H_kv, d, page, new, kv, window, kind):
    check_tree(sp, H=H, H_kv=H_kv, d=d, page=page, new=new, kv=kv, kind=kind, window=window, dtype="f32")


@pytest.mark.parametrize("kind", ["same", "int8"])
@pytest.mark.parametrize("H,H_kv,d,dtype", [(4, 2, 64, "bf16"), (8, 2, 128, "bf16"), (2, 1, 64, "f32"), (2, 1, 96, "bf16")])
@pytest.mark.parametrize("new,kv", [([4, 2], [4, 90]), ([8, 4], [3, 1]), ([70, 150], [70, 900]), ([90, 40], [30, 40])])
@pytest.mark.parametrize("window", [0, 50])
def test_any_bits_will_do(sp, H, H_kv, d, dtype, new, kv, kind, window):
    """Bits that are no tree's: later tokens, none at all (a row that then sees nothing gives 0), and sequences of fewer
    cached tokens than new ones."""
    check_tree(sp, H=H, H_kv=H_kv, d=d, page=16, new=new, kv=kv, kind=kind, dtype=dtype, seen="any", window=window)


@pytest.mark.parametrize("d,n,H", [(64, 4, 4), (64, 60, 8), (128, 16, 1), (128, 300, 4)])
def test_a_chain_is_causal_attention(sp, d, n, H):
    """Every token hanging on the one before it sees what sp_attend's does: the same bits come out."""
    import torch
    rng = np.random.default_rng(4)
    kv = [n + 1000, n]
    cache, table, _, _ = make_cache(sp, rng, H_kv=1, d=d, page=16, kv=kv)
    batch, _ = make_batch(sp, [n, n], kv, table)
    q = torch.from_numpy(rng.standard_normal((2 * n, H, d))).to(torch.bfloat16).cuda()
    seen, pos = sp.tree_seen(batch, i32(np.tile(np.arange(n) - 1, 2)), check=True)
    assert pos.tolist() == list(range(1000, 1000 + n)) + list(range(n))
    out, lse = sp.attend_tree(q, cache, batch, seen, check=True)
    want, want_lse = sp.attend(q, cache, batch, check=True)
    assert torch.equal(lse, want_lse) and torch.equal(out, want)


def test_trees_of_many_sequences_and_a_long_cache(sp):
    check_tree(sp, H=8, H_kv=2, d=128, page=64, new=[48], kv=[20000], kind="e4m3")
    check_tree(sp, H=4, H_kv=2, d=64, page=16, new=[1, 9, 30, 2] * 20, kv=[100, 9, 64, 257] * 20)


@pytest.mark.parametrize("n,dtype", [(4, "bf16"), (60, "bf16"), (5, "f32")])
def test_a_captured_tree_follows_its_bits(sp, n, dtype):
    import torch
    rng = np.random.default_rng(6)
    td = torch_dtype(dtype)
    H, H_kv, d, page, kv = 4, 2, 64, 16, [700, 90]
    cache, table, kval, vval = make_cache(sp, rng, H_kv=H_kv, d=d, page=page, kv=kv, dtype=td)
    batch, cu = make_batch(sp, [n, n], kv, table, max_new=n)
    q = torch.from_numpy(rng.standard_normal((2 * n, H, d))).to(td).cuda()
    parent = i32(np.zeros(2 * n))
    draft, target = i32(np.zeros(2 * n)), i32(np.zeros(2 * n))

    def call(o):
        sp.tree_seen(batch, parent, seen=o["seen"], positions=o["pos"], ws=o["w1"])
        sp.attend_tree(q, cache, batch, o["seen"], out=o["out"], lse=o["lse"], ws=o["ws"])
        sp.tree_accept(batch, parent, draft, target, path=o["path"], n_path=o["n"], next_token=o["next"], ws=o["w2"])

    def space():
        z = lambda *s, t=torch.int32: torch.zeros(*s, dtype=t, device="cuda")                     # noqa: E731
        return dict(seen=z(2 * n, -(-n // 32)), pos=z(2 * n), out=torch.zeros_like(q), lse=z(H, 2 * n, t=torch.float32), path=z(2, n),
                    n=z(2, t=torch.int64), next=z(2), w1=z(64), w2=z(64),
                    ws=z(sp.attend_tree_workspace_size(q, cache, batch), t=torch.uint8))

    runs = []
    for _ in range(2):
        o = space()
        call(o)
        torch.cuda.synchronize()
        graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph, stream=stream):
            call(o)
        runs.append((graph, stream, o))
    for shape in ("chain", "star", "random"):
        p = np.concatenate([tree(rng, n, shape) for _ in range(2)])
        parent.copy_(torch.from_numpy(p.astype(np.int32)))
        draft.copy_(torch.from_numpy(rng.integers(0, 3, 2 * n).astype(np.int32)))
        target.copy_(torch.from_numpy(rng.integers(0, 3, 2 * n).astype(np.int32)))
        torch.cuda.synchronize()
        for graph, stream, _ in runs:
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for _, _, o in runs:
            assert all(sp.sp_workspace_status(o[w]) == sp.SP_OK for w in ("w1", "w2", "ws"))
            for b in range(2):
                rows = slice(b * n, (b + 1) * n)
                see, depth = oracle.kept.tree_seen(p[rows])
                assert np.array_equal(o["pos"][rows].cpu().numpy(), kv[b] - n + depth)
                ref = oracle.kept.attend(f64(q[rows]), kval[b], vval[b], d ** -0.5, oracle.kept.visible(n, kv[b], 0, see))
                bound, _ = attend_bounds(dtype, d, kv[b], ref[0], ref[3], ref[2], ref[1])
                assert np.all(np.abs(f64(o["out"][rows]) - ref[0]) <= bound)
                want, then = oracle.kept.accept(p[rows], draft[rows].tolist(), target[rows].tolist())
                assert o["path"][b].tolist() == want + [-1] * (n - len(want)) and o["next"][b].item() == then


def test_a_tree_over_a_cache_beyond_2_31_entries(sp):
    import torch
    for d, n in ((64, 4), (128, 70), (96, 5)):
        far = 5 * (1 << 29)
        buf = torch.zeros(far + 8192 * 8, dtype=torch.bfloat16, device="cuda")
        shape, stride = (2, 1, 64, d), (far, 64 * d, d, 1)
        k, v = buf.as_strided(shape, stride), buf.as_strided(shape, stride, 64 * d)
        g = torch.Generator(device="cuda").manual_seed(d)
        for t in (k, v):
            t.copy_(torch.randn(shape, generator=g, device="cuda"))
        cache = sp.Cache(k, v)
        batch, _ = make_batch(sp, [n], [110], np.array([[1, 0]], np.int32))
        q = torch.randn(n, 2, d, generator=g, device="cuda").to(torch.bfloat16)
        parent = tree(np.random.default_rng(d), n, "random")
        seen, _ = sp.tree_seen(batch, i32(parent), check=True)
        out, _ = sp.attend_tree(q, cache, batch, seen, check=True)
        kk, vv = (f64(torch.cat([t[1], t[0]], 1))[:, :110] for t in (k, v))
        see = oracle.kept.tree_seen(parent)[0]
        ref, ref_lse, top, spread = oracle.kept.attend(f64(q), kk, vv, d ** -0.5, oracle.kept.visible(n, 110, 0, see))
        bound, _ = attend_bounds("bf16", d, 110, ref, spread, top, ref_lse)
        assert np.all(np.abs(f64(out) - ref) <= bound)


@pytest.mark.parametrize("handle", [False, True])
def test_a_round_on_another_stream(sp, handle):
    """All calls of a round on a stream of their own, by object and by handle, give what they give on the current one."""
    import torch
    rng = np.random.default_rng(16)
    cache, table, _, _ = make_cache(sp, rng, H_kv=2, d=64, page=16, kv=[300, 90])
    batch, _ = make_batch(sp, [6, 20], [300, 90], table, max_new=20)
    q = torch.from_numpy(rng.standard_normal((26, 4, 64))).to(torch.bfloat16).cuda()
    parent = i32(np.concatenate([tree(rng, 6, "random"), tree(rng, 20, "random")]))
    tok = i32(rng.integers(0, 2, 26))

    def round_(stream):
        c = sp.Cache(cache.k.clone(), cache.v.clone())
        torch.cuda.synchronize()
        a = dict(stream=stream)
        seen, pos = sp.tree_seen(batch, parent, **a)
        out, lse = sp.attend_tree(q, c, batch, seen, **a)
        w = sp.attend_weights(q, c, batch, lse, torch.zeros(c.pages, 2, 16, device="cuda"), **a)
        path, n, nxt = sp.tree_accept(batch, parent, tok, tok, **a)
        length = sp.cache_keep(c, batch, path, n, drafted=True, weights=w, **a)
        kept, m = sp.cache_choose(c, batch, w, 40, first=2, last=3, **a)
        torch.cuda.synchronize()
        return [seen, pos, out, lse, w, path, n, nxt, length, kept, m, c.k, c.v]

    s = torch.cuda.Stream()
    for a, b in zip(round_(None), round_(s.cuda_stream if handle else s)):
        assert torch.equal(a, b)
