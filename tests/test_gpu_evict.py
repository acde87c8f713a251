"""Accumulated attention weight and the cutting of a cache on the GPU, against the 64-bit oracle."""
import numpy as np
import pytest

import oracle
from paged_helpers import attend_bounds, make_batch, make_cache
from test_gpu_tree import f64, i32, sp, torch_dtype, tree  # noqa: F401

pytestmark = pytest.mark.gpu


def place(table, b, i, page):
    return table[b, i // page], i % page


# ----------------------------------------------------------------------------
# Weights
# ----------------------------------------------------------------------------

def check_weights(sp, *, H, H_kv, d, page, new, kv, dtype="bf16", kind="same", window=0, decay=1.0, layout="hnd", before=1,
                  behind=2, seed=0, scale=None, lse_shift=0.0):
    import torch
    rng = np.random.default_rng(seed)
    td = torch_dtype(dtype)
    cache, table, kval, _ = make_cache(sp, rng, H_kv=H_kv, d=d, page=page, kv=kv, kind=kind, dtype=td, layout=layout,
                                       junk=float("nan"))
    T = before + sum(new) + behind
    batch, cu = make_batch(sp, new, kv, table, rows=T, first=before, max_new=max(new))
    q = torch.from_numpy(rng.standard_normal((T, H, d))).to(td)
    scale_ = d ** -0.5 if scale is None else scale
    lse = np.full((H, T), np.nan, dtype=np.float32)             # rows of no token hold NaN
    real = np.zeros(T, dtype=bool)
    real[before:before + sum(new)] = True
    q[~torch.from_numpy(real)] = float("nan")
    qd = q.double().numpy()
    see = [oracle.kept.visible(n, c, window) for n, c in zip(new, kv)]
    for b, n in enumerate(new):
        if n:
            rows = slice(cu[b], cu[b + 1])
            x = oracle.kept.attend(qd[rows], kval[b], kval[b], scale_, see[b])[1]
            lse[:, rows] = (x + lse_shift).astype(np.float32)
    old = rng.standard_normal((cache.pages, H_kv, page)).astype(np.float32) ** 2
    if decay == 0:
        old[rng.random(old.shape) < 0.5] = np.nan               # not read then
    lse_t = torch.from_numpy(np.ascontiguousarray(lse.T)).cuda().T if layout == "nhd" else torch.from_numpy(lse).cuda()
    w = torch.from_numpy(old.copy()).cuda()
    got_w = sp.attend_weights(q.cuda(), cache, batch, lse_t, w, scale=scale, window=window, decay=decay, check=True)
    assert got_w is w
    got = f64(w)
    touched = np.zeros(old.shape, dtype=bool)
    for b, n in enumerate(new):
        if not n:
            continue
        want, bound = oracle.kept.weights(qd[cu[b]:cu[b + 1]], kval[b], lse[:, cu[b]:cu[b + 1]].astype(np.float64), scale_, see[b])
        for i in range(max(0, kv[b] - n - window + 1) if window else 0, kv[b]):
            pg, slot = place(table, b, i, page)
            before_ = decay * old[pg, :, slot].astype(np.float64) if i < kv[b] - n and decay else np.zeros(H_kv)
            touched[pg, :, slot] = True
            err = np.abs(got[pg, :, slot] - (want[:, i] + before_))
            # the product with decay and the sum are rounded once each
            assert np.all(err <= bound[:, i] + 2.0 ** -23 * (want[:, i] + before_)), (b, i, err, bound[:, i])
    assert np.array_equal(got[~touched], old[~touched].astype(np.float64), equal_nan=True)
    return w, cache, batch, q, lse_t


@pytest.mark.parametrize("kind", ["same", "e4m3", "int8"])
@pytest.mark.parametrize("H,H_kv,d,page", [
    (4, 2, 64, 16), (32, 8, 128, 64), (7, 7, 64, 32), (6, 2, 128, 128), (8, 1, 64, 48), (5, 1, 40, 7), (2, 1, 256, 16),
    (16, 1, 128, 1), (3, 3, 8, 5), (24, 1, 64, 256),
])
@pytest.mark.parametrize("new,kv,decay", [([1], [1], 1.0), ([1, 1, 0, 1, 1], [17, 300, 0, 128, 129], 0.5), ([2, 3, 1], [2, 5, 523], 0.0)])
def test_weights_of_steps(sp, H, H_kv, d, page, new, kv, decay, kind):
    check_weights(sp, H=H, H_kv=H_kv, d=d, page=page, new=new, kv=kv, kind=kind, decay=decay)


@pytest.mark.parametrize("kind", ["same", "e4m3", "int8"])
@pytest.mark.parametrize("H,H_kv,d,page", [(4, 2, 64, 16), (8, 2, 128, 64), (3, 1, 64, 32), (7, 1, 128, 48), (2, 2, 40, 7), (2, 1, 128, 8)])
@pytest.mark.parametrize("new,kv,window,decay", [
    ([33], [33], 0, 0.0), ([64, 1, 65, 0], [64, 400, 200, 0], 0, 1.0), ([129, 5], [300, 2], 0, 0.75), ([100, 40], [260, 40], 37, 1.0),
    ([1, 70], [500, 128], 128, 0.0), ([300], [513], 0, 0.5),
])
def test_weights_of_chunks(sp, H, H_kv, d, page, new, kv, window, decay, kind):
    check_weights(sp, H=H, H_kv=H_kv, d=d, page=page, new=new, kv=kv, kind=kind, window=window, decay=decay)


@pytest.mark.parametrize("kind", ["same", "e4m3", "int8"])
@pytest.mark.parametrize("new,kv,window", [([1], [512], 0), ([1, 1], [1, 300], 9), ([5, 0, 40], [3, 0, 90], 0), ([130], [131], 64)])
@pytest.mark.parametrize("H,H_kv,d,page", [(4, 2, 64, 16), (3, 1, 128, 5), (2, 2, 256, 32)])
def test_weights_in_single_precision(sp, H, H_kv, d, page, new, kv, window, kind):
    check_weights(sp, H=H, H_kv=H_kv, d=d, page=page, new=new, kv=kv, kind=kind, window=window, dtype="f32", decay=0.25)


@pytest.mark.parametrize("new,kv", [([1, 1], [2000, 40]), ([90, 1, 20], [700, 900, 30])])
@pytest.mark.parametrize("layout,scale,shift", [("nhd", None, 0.0), ("hnd", 1.0, 0.0), ("nhd", 1e-4, 0.0), ("nhd", None, 60.0), ("hnd", None, -60.0)])
@pytest.mark.parametrize("d,page", [(64, 16), (128, 64)])
@pytest.mark.parametrize("kind", ["same", "int8"])
def test_weights_layouts_scales_and_normalisers(sp, new, kv, layout, scale, shift, d, page, kind):
    check_weights(sp, H=4, H_kv=2, d=d, page=page, new=new, kv=kv, layout=layout, scale=scale, lse_shift=shift, kind=kind)


@pytest.mark.parametrize("d,kind,n,kv", [(128, "e4m3", 32, 60000), (64, "same", 24, 90000), (128, "same", 700, 30000), (64, "int8", 1, 120000),
                                         (128, "int8", 90, 50000)])
def test_weights_of_a_long_cache(sp, d, kind, n, kv):
    """Every CTA has dozens of items: all tokens' weights against 64-bit products of the rows as they read back."""
    import torch
    H, H_kv, page = 16, 4, 64
    g = torch.Generator(device="cuda").manual_seed(n)
    pages = -(-kv // page)
    cache = sp.cache_alloc(pages, H_kv, page, d, kind=kind)
    table = torch.randperm(pages, generator=g, device="cuda").int()[None]
    i64 = lambda *v: torch.tensor(v, dtype=torch.int64, device="cuda")                          # noqa: E731
    full = sp.Batch(i64(0, kv), i64(kv), table, rows=kv)
    new = lambda h, m: torch.randn(m, h, d, generator=g, device="cuda").to(torch.bfloat16)      # noqa: E731
    sp.cache_write(cache, full, new(H_kv, kv), new(H_kv, kv), check=True)
    k, _ = sp.cache_read(cache, full, check=True)
    q = new(H, n)
    batch = sp.Batch(i64(0, n), i64(kv), table, rows=n)
    lse = np.log(kv) + 0.5 + 0.1 * torch.randn(H, n, generator=g, device="cuda")
    w = sp.attend_weights(q, cache, batch, lse, sp.weights_alloc(cache).fill_(3.0), decay=0.5, check=True)
    i = torch.arange(kv, device="cuda")
    got = w[table[0].long()[i // page], :, i % page].double().T                                  # [H_kv, kv]
    seen = i <= torch.arange(kv - n, kv, device="cuda")[:, None]
    for h in range(H_kv):
        want = torch.where(i < kv - n, 1.5, 0.0).double()
        for f in range(4 * h, 4 * h + 4):
            x = q[:, f].double() @ k[h].double().T * d ** -0.5 - lse[f].double()[:, None]
            want += torch.where(seen, x.exp(), 0.0).sum(0)
        # |logits| below 12, of products that sum to at most 100: each weight within 2^-17 (oracle.kept.weights' bound), and sums of n * 4
        assert torch.all((got[h] - want).abs() <= want * (2.0 ** -17 + 4 * n * 2.0 ** -24))


@pytest.mark.parametrize("n,d,dtype,page", [(1, 64, "bf16", 16), (1, 128, "bf16", 16), (40, 64, "bf16", 16), (40, 128, "bf16", 64), (5, 64, "f32", 16),
                                            (3, 64, "bf16", 7), (30, 128, "bf16", 7)])
@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_weights_over_a_cache_of_any_scales(sp, kind, n, d, dtype, page):
    """Scales that are no powers of two, tiny, negative and zero ones, as another program may have filled them in."""
    import torch
    rng = np.random.default_rng(18)
    kv, H, H_kv = 200, 4, 2
    cache, table, _, _ = make_cache(sp, rng, H_kv=H_kv, d=d, page=page, kv=[kv], kind=kind, dtype=torch_dtype(dtype))
    scale = rng.uniform(0.5, 1.5, cache.k_scale.shape) * (1 / 64 if kind == "int8" else 1 / 128)
    scale[rng.random(scale.shape) < 0.1] = 0
    scale[rng.random(scale.shape) < 0.1] *= -1
    scale[rng.random(scale.shape) < 0.1] *= 1e-20
    cache.k_scale.copy_(torch.from_numpy(scale))
    i = np.arange(kv)
    codes = f64(cache.k.float())[table[0, i // page], :, i % page]
    k = (codes * f64(cache.k_scale)[table[0, i // page], :, i % page][..., None]).transpose(1, 0, 2)
    batch, _ = make_batch(sp, [n], [kv], table)
    q = torch.from_numpy(rng.standard_normal((n, H, d))).to(torch_dtype(dtype)).cuda()
    lse = torch.from_numpy(rng.uniform(4, 6, (H, n))).float().cuda()
    w = sp.attend_weights(q, cache, batch, lse, sp.weights_alloc(cache), decay=0, check=True)
    want, bound = oracle.kept.weights(f64(q), k, f64(lse), d ** -0.5, oracle.kept.visible(n, kv))
    got = f64(w)[table[0, i // page], :, i % page].T
    assert np.all(np.abs(got - want) <= bound + 2.0 ** -23 * want)


@pytest.mark.parametrize("kind", ["same", "int8"])
@pytest.mark.parametrize("n,d,dtype", [(1, 64, "bf16"), (40, 64, "bf16"), (40, 128, "bf16"), (2, 64, "f32")])
def test_a_key_that_is_nan_has_a_weight_that_is_nan(sp, n, d, dtype, kind):
    """And no other token's weight knows of it; a row whose normaliser is NaN reaches all that it sees."""
    import torch
    rng = np.random.default_rng(19)
    kv, H, H_kv, page = 300, 4, 2, 16
    cache, table, kval, _ = make_cache(sp, rng, H_kv=H_kv, d=d, page=page, kv=[kv], kind=kind, dtype=torch_dtype(dtype))
    at = [5, 130, kv - 1]
    for i in at:
        if kind == "same":
            cache.k[int(table[0, i // page]), 1, i % page, 3] = float("nan")
        else:
            cache.k_scale[int(table[0, i // page]), 1, i % page] = float("nan")
    batch, _ = make_batch(sp, [n], [kv], table)
    q = torch.from_numpy(rng.standard_normal((n, H, d))).to(torch_dtype(dtype)).cuda()
    lse = torch.full((H, n), 6.0, device="cuda")
    i = np.arange(kv)
    got = f64(sp.attend_weights(q, cache, batch, lse, sp.weights_alloc(cache), decay=0, check=True))[table[0, i // page], :, i % page].T
    nan = np.isnan(got)
    assert not nan[0].any() and np.flatnonzero(nan[1]).tolist() == at
    want, bound = oracle.kept.weights(f64(q), kval[0], f64(lse), d ** -0.5, oracle.kept.visible(n, kv))
    assert np.all((np.abs(got - want) <= bound + 2.0 ** -23 * want) | nan)
    lse[0, 0] = float("nan")
    got = f64(sp.attend_weights(q, cache, batch, lse, sp.weights_alloc(cache), decay=0, check=True))[table[0, i // page], :, i % page].T
    assert np.isnan(got[0, :kv - n + 1]).all() and not np.isnan(got[0, kv - n + 1:]).any()


def test_weights_of_a_cache_beyond_2_31_entries(sp):
    import torch
    for d, n in ((64, 2), (128, 40), (96, 3)):
        far = 5 * (1 << 29)
        buf = torch.zeros(far + 8192 * 8, dtype=torch.bfloat16, device="cuda")
        shape, stride = (2, 1, 64, d), (far, 64 * d, d, 1)
        k, v = buf.as_strided(shape, stride), buf.as_strided(shape, stride, 64 * d)
        g = torch.Generator(device="cuda").manual_seed(d)
        k.copy_(torch.randn(shape, generator=g, device="cuda"))
        batch, _ = make_batch(sp, [n], [110], np.array([[1, 0]], np.int32))
        q = torch.randn(n, 2, d, generator=g, device="cuda").to(torch.bfloat16)
        lse = torch.full((2, n), 5.0, device="cuda")
        w = sp.attend_weights(q, sp.Cache(k, v), batch, lse, torch.full((2, 1, 64), 2.0, device="cuda"), check=True)
        kk = f64(torch.cat([k[1], k[0]], 1))[:, :110]
        want, bound = oracle.kept.weights(f64(q), kk, f64(lse), d ** -0.5, oracle.kept.visible(n, 110))
        want[:, :110 - n] += 2
        got = f64(torch.cat([w[1], w[0]], 1))
        assert np.all(np.abs(got[:, :110] - want) <= bound + 2.0 ** -23 * want) and np.all(got[:, 110:] == 2)


def test_weights_sum_to_the_rows(sp):
    """With lse as attend returns it, the weights of a sequence add up to its rows, whatever the batch."""
    import torch
    rng = np.random.default_rng(2)
    for d, H, new, kv in ((64, 4, [1, 40], [3000, 700]), (128, 8, [300, 1], [1000, 20])):
        cache, table, _, _ = make_cache(sp, rng, H_kv=2, d=d, page=16, kv=kv)
        batch, cu = make_batch(sp, new, kv, table)
        q = torch.from_numpy(rng.standard_normal((sum(new), H, d))).to(torch.bfloat16).cuda()
        _, lse = sp.attend(q, cache, batch, check=True)
        w = sp.attend_weights(q, cache, batch, lse, sp.weights_alloc(cache), decay=0, check=True)
        for b, n in enumerate(new):
            i = np.arange(kv[b])
            total = f64(w)[table[b, i // 16], :, i % 16].sum(0)
            # lse and each weight are off by about 2^-20 each
            assert np.all(np.abs(total - n * H / 2) <= n * H / 2 * 2.0 ** -17)
        again = sp.attend_weights(q, cache, batch, lse, sp.weights_alloc(cache), decay=0, check=True)
        for b in range(2):
            i = np.arange(kv[b])
            assert np.array_equal(f64(w)[table[b, i // 16], :, i % 16], f64(again)[table[b, i // 16], :, i % 16])


@pytest.mark.parametrize("n,d,dtype", [(1, 64, "bf16"), (40, 128, "bf16"), (3, 64, "f32")])
def test_weights_of_a_bad_batch(sp, n, d, dtype):
    """A page out of range, impossible lengths and a row without a normaliser: reported, and nothing else is touched."""
    import torch
    rng = np.random.default_rng(7)
    td = torch_dtype(dtype)
    page, kv = 16, [200, 90]
    cache, table, _, _ = make_cache(sp, rng, H_kv=2, d=d, page=page, kv=kv, dtype=td)
    q = torch.from_numpy(rng.standard_normal((2 * n, 4, d))).to(td).cuda()
    good, _ = make_batch(sp, [n, n], kv, table)
    _, lse = sp.attend(q, cache, good, check=True)
    fresh = lambda: torch.full((cache.pages, 2, page), 5.0, device="cuda")             # noqa: E731
    want = sp.attend_weights(q, cache, good, lse, fresh(), check=True)
    ws = torch.empty(sp.attend_weights_workspace_size(q, cache, good), dtype=torch.uint8, device="cuda")
    bad_table = table.copy()
    bad_table[0, 3] = cache.pages
    batch, _ = make_batch(sp, [n, n], kv, bad_table)
    got = sp.attend_weights(q, cache, batch, lse, fresh(), ws=ws)
    assert sp.sp_workspace_status(ws) == sp.SP_EDEVICE
    same = np.ones(cache.pages, dtype=bool)
    same[table[0, 3]] = False
    assert torch.equal(got[torch.from_numpy(same)], want[torch.from_numpy(same)]) and torch.all(got[int(table[0, 3])] == 5)
    batch, _ = make_batch(sp, [n, n], [200, 16 * table.shape[1] + 1], table)
    got = sp.attend_weights(q, cache, batch, lse, fresh(), ws=ws)
    assert sp.sp_workspace_status(ws) == sp.SP_EDEVICE
    mine = table[0, :13].astype(np.int64)
    others = np.setdiff1d(np.arange(cache.pages), mine)
    assert torch.equal(got[mine], want[mine]) and torch.all(got[others] == 5)
    none = torch.full_like(lse, float("-inf"))
    got = sp.attend_weights(q, cache, good, none, fresh(), ws=ws)
    assert sp.sp_workspace_status(ws) == sp.SP_OK
    i = np.arange(200 - n)
    assert torch.all(got[table[0, i // page].astype(np.int64), :, i % page] == 5)
    i = np.arange(200 - n, 200)
    assert torch.all(got[table[0, i // page].astype(np.int64), :, i % page] == 0)


# ----------------------------------------------------------------------------
# Choosing
# ----------------------------------------------------------------------------

def lists_of(rng, shape, how):
    w = rng.standard_normal(shape).astype(np.float32)
    if how == "few":            # many ties
        w = np.round(w * 2) / 2
    elif how == "zeros":
        w = np.zeros(shape, dtype=np.float32)
        w[rng.random(shape) < 0.2] *= -1
    elif how == "odd":
        w[rng.random(shape) < 0.1] = np.nan
        w[rng.random(shape) < 0.1] = np.inf
        w[rng.random(shape) < 0.1] = -np.inf
        w[rng.random(shape) < 0.1] = -0.0
        w[rng.random(shape) < 0.1] = 0.0
        w[rng.random(shape) < 0.1] = 1e-45
    elif how == "sums":
        w = np.exp(2 * w - 5).astype(np.float32)
    return w


@pytest.mark.parametrize("how", ["normal", "few", "zeros", "odd", "sums"])
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("H_kv,page,kv,budget,first,last", [
    (1, 16, [1], 1, 0, 0), (2, 16, [100, 0, 7, 33], 20, 2, 5), (3, 7, [5000, 3], 700, 0, 0), (8, 64, [1000], 999, 4, 995),
    (2, 128, [4096, 4097, 2048], 2048, 0, 2048), (1, 1, [300], 10, 10, 0), (4, 32, [70, 64], 0, 0, 0), (2, 48, [20000], 1, 0, 0),
])
def test_cache_choose(sp, H_kv, page, kv, budget, first, last, shared, how):
    import torch
    rng = np.random.default_rng(budget)
    cache, table, _, _ = make_cache(sp, rng, H_kv=H_kv, d=8, page=page, kv=kv)
    batch, _ = make_batch(sp, [0] * len(kv), kv, table)
    w = lists_of(rng, (cache.pages, H_kv, page), how)
    kept, n = sp.cache_choose(cache, batch, torch.from_numpy(w).cuda(), budget, first=first, last=last, shared=shared, check=True)
    assert n.tolist() == [min(c, budget) for c in kv]
    for b, c in enumerate(kv):
        i = np.arange(c)
        mine = w[table[b, i // page], :, i % page]
        if shared:
            mine = np.fmax.reduce(mine, 1)[:, None] if c else mine[:, :1]
        for h in range(1 if shared else H_kv):
            want = oracle.kept.choose(mine[:, h], budget, first, last)
            assert np.array_equal(kept[b, h].cpu().numpy(), np.concatenate([want, np.full(budget - len(want), -1)]))


@pytest.mark.parametrize("kv,budget", [([131072], 8192), ([900000], 5), ([600001, 20], 599999)])
def test_cache_choose_of_long_caches(sp, kv, budget):
    """Also more tokens than a cluster holds, which are read again in each pass."""
    import torch
    page = 64
    per = [-(-c // page) for c in kv]
    pages = sum(per)
    k = torch.zeros(pages, 1, page, 8, dtype=torch.bfloat16, device="cuda")
    cache = sp.Cache(k, k)
    table = np.zeros((len(kv), max(per)), np.int32)
    order = np.random.default_rng(3).permutation(pages)
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = order[at:at + n]
        at += n
    batch, _ = make_batch(sp, [0] * len(kv), kv, table)
    w = torch.rand(pages, 1, page, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    w = (w * 1000).round() / 1000           # ties
    kept, n = sp.cache_choose(cache, batch, w, budget, first=1, last=3, check=True)
    host = w.cpu().numpy()
    for b, c in enumerate(kv):
        i = np.arange(c)
        mine = host[table[b, i // page], 0, i % page].astype(np.float64)
        m = min(c, budget)
        if m < c:
            mine[0] = mine[-3:] = np.inf
        want = np.sort(np.lexsort((i, -mine))[:m])
        assert n[b].item() == m and np.array_equal(kept[b, 0, :m].cpu().numpy(), want) and torch.all(kept[b, 0, m:] == -1)


# ----------------------------------------------------------------------------
# Keeping
# ----------------------------------------------------------------------------

def check_keep(sp, *, H_kv, d, page, new, kv, dtype="bf16", kind="same", layout="hnd", shared=False, drafted=False, to=False,
               with_weights=True, keep=0.3, seed=0):
    import torch
    rng = np.random.default_rng(seed)
    td = torch_dtype(dtype)
    spare = 2 + (sum(-(-c // page) for c in kv) if to else 0)
    cache, table, _, _ = make_cache(sp, rng, H_kv=H_kv, d=d, page=page, kv=kv, kind=kind, dtype=td, layout=layout, spare=spare)
    batch, _ = make_batch(sp, new, kv, table, max_new=max(new))
    B, heads = len(kv), 1 if shared else H_kv
    base = [c - n if drafted else 0 for n, c in zip(new, kv)]
    most = max(c - o for c, o in zip(kv, base)) + 3
    kept, n_kept = np.full((B, heads, most), 1 << 30), np.zeros(B, np.int64)
    for b in range(B):
        avail = kv[b] - base[b]
        n_kept[b] = rng.integers(0, avail + 1) if keep is None else int(round(keep * avail))
        for h in range(heads):
            kept[b, h, :n_kept[b]] = np.sort(rng.permutation(avail)[:n_kept[b]])
    to_table = None
    if to:
        free = np.setdiff1d(np.arange(cache.pages), table[table >= 0])
        to_table, at = np.full((B, max(1, table.shape[1])), -9), 0
        for b in range(B):
            need = -(-kv[b] // page)
            to_table[b, :need] = rng.permutation(free)[:0] if need == 0 else free[at:at + need]
            at += need
    w = torch.from_numpy(rng.standard_normal((cache.pages, H_kv, page)).astype(np.float32)).cuda() if with_weights else None
    raw = lambda t: t.view(torch.uint8) if t.element_size() == 1 else t                         # noqa: E731
    parts = [raw(cache.k), raw(cache.v)] + [t for t in (cache.k_scale, cache.v_scale, w) if t is not None]
    old = [t.cpu().clone() for t in parts]
    got = sp.cache_keep(cache, batch, i32(kept) if not shared else i32(kept[:, 0]), torch.from_numpy(n_kept).cuda(), drafted=drafted,
                        to=None if to_table is None else i32(to_table), weights=w, check=True)
    assert got.tolist() == [o + int(n) for o, n in zip(base, n_kept)]
    for t, was in zip(parts, old):
        want = was.clone()
        for b in range(B):
            for h in range(H_kv):
                for j in range(n_kept[b]):
                    i = base[b] + int(kept[b, 0 if shared else h, j])
                    src, dst = place(table, b, i, page), place(to_table if to else table, b, base[b] + j, page)
                    want[dst[0], h, dst[1]] = was[src[0], h, src[1]]
        assert torch.equal(t.cpu().view(torch.uint8), want.view(torch.uint8))


@pytest.mark.parametrize("to", [False, True])
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("kind,dtype", [("same", "bf16"), ("e4m3", "bf16"), ("int8", "f32"), ("same", "f32")])
@pytest.mark.parametrize("H_kv,d,page,kv,layout", [
    (2, 64, 16, [40, 0, 17], "hnd"), (1, 256, 7, [50], "nhd"), (3, 8, 5, [30, 1], "hnd"), (2, 128, 64, [300, 64], "nhd"),
    (2, 40, 1, [9, 20], "hnd"), (1, 72, 48, [1500], "hnd"),
])
def test_cache_keep(sp, H_kv, d, page, kv, layout, kind, dtype, shared, to):
    check_keep(sp, H_kv=H_kv, d=d, page=page, new=[0] * len(kv), kv=kv, kind=kind, dtype=dtype, layout=layout, shared=shared, to=to)


@pytest.mark.parametrize("keep", [0.0, 0.05, 0.9, 1.0, None])
def test_cache_keep_of_few_and_many(sp, keep):
    check_keep(sp, H_kv=2, d=64, page=16, new=[0, 0], kv=[1400, 130], keep=keep, seed=3)


@pytest.mark.parametrize("kind", ["same", "e4m3"])
@pytest.mark.parametrize("shared", [False, True])
def test_cache_keep_of_drafted_tokens(sp, kind, shared):
    check_keep(sp, H_kv=2, d=64, page=16, new=[30, 1, 0, 64], kv=[100, 1, 40, 64], drafted=True, kind=kind, shared=shared, keep=None)


def test_rows_move_within_a_cache_as_if_all_were_read_first(sp):
    """In place, thousands of rows over several rounds of a cluster: every source slot is another row's destination."""
    import torch
    rng = np.random.default_rng(5)
    H_kv, page, kv = 1, 64, 30000
    pages = -(-kv // page)
    for d, drop in ((128, 1), (64, 300), (8, 7)):
        k = torch.randn(pages, H_kv, page, d, dtype=torch.bfloat16, device="cuda", generator=torch.Generator(device="cuda").manual_seed(d))
        v = -k
        table = rng.permutation(pages).astype(np.int32)[None]
        batch, _ = make_batch(sp, [0], [kv], table)
        gone = np.sort(rng.permutation(kv)[:drop])
        kept = np.setdiff1d(np.arange(kv), gone)
        where = torch.from_numpy(table[0].astype(np.int64)).cuda()
        flat = lambda t: t[where, 0].reshape(-1, d)                                             # noqa: E731
        want = flat(k)[torch.from_numpy(kept).cuda()].clone()
        cache = sp.Cache(k, v)
        n = sp.cache_keep(cache, batch, i32(kept[None]), torch.tensor([len(kept)], device="cuda"), check=True)
        assert n.item() == len(kept)
        assert torch.equal(flat(k)[:len(kept)], want) and torch.equal(flat(v)[:len(kept)], -want)


def test_lists_that_are_wrong_are_reported(sp):
    import torch
    rng = np.random.default_rng(8)
    page, kv = 16, [40, 30]
    cache, table, _, _ = make_cache(sp, rng, H_kv=2, d=64, page=page, kv=kv)
    batch, _ = make_batch(sp, [2, 3], kv, table)
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    old = cache.k.clone()
    count = lambda *n: torch.tensor(n, dtype=torch.int64, device="cuda")                        # noqa: E731
    two = i32([[3, 5, 7], [1, 2, 9]])
    for n, bad in (((4, 3), 0), ((-1, 0), 0), ((3, 1 << 40), 1)):
        cache.k.copy_(old)
        out = sp.cache_keep(cache, batch, two, count(*n), ws=ws)
        assert sp.sp_workspace_status(ws) == sp.SP_EDEVICE
        assert out[bad].item() == kv[bad] and out[1 - bad].item() == n[1 - bad]
        mine = table[bad][table[bad] >= 0].astype(np.int64)
        assert torch.equal(cache.k[mine], old[mine])
    for entries in ([3, 3, 7], [5, 3, 7], [3, 5, 40], [-1, 5, 7]):
        cache.k.copy_(old)
        sp.cache_keep(cache, batch, i32([entries, [1, 2, 9]]), count(3, 3), ws=ws)
        assert sp.sp_workspace_status(ws) == sp.SP_EDEVICE
        mine = table[1][table[1] >= 0].astype(np.int64)
        i = np.array([1, 2, 9])
        assert torch.equal(cache.k[mine[0], :, :3], old[table[1, i // page].astype(np.int64), :, i % page].transpose(0, 1))
    # a page to go to that is none: those rows stay where they are; and too few pages
    to = i32([[cache.pages, 0], [-1, 0]])
    cache.k.copy_(old)
    sp.cache_keep(cache, batch, two, count(3, 3), to=to, ws=ws)
    assert sp.sp_workspace_status(ws) == sp.SP_EDEVICE and torch.equal(cache.k, old)
    sp.cache_keep(cache, batch, i32(np.tile(np.arange(20), (2, 1))), count(20, 5), to=i32([[0], [1]]), ws=ws)
    assert sp.sp_workspace_status(ws) == sp.SP_EDEVICE
    w = torch.zeros(cache.pages, 2, page, device="cuda")
    bad_table = table.copy()
    bad_table[1, 1] = cache.pages
    kept, n = sp.cache_choose(cache, make_batch(sp, [0, 0], kv, bad_table)[0], w + 1, 20, ws=ws)
    assert sp.sp_workspace_status(ws) == sp.SP_EDEVICE
    assert kept[0, 0].tolist() == list(range(20)) and kept[1, 1].tolist() == list(range(16)) + [16, 17, 18, 19]
    kept, n = sp.cache_choose(cache, make_batch(sp, [0, 0], [40, 999], table)[0], w, 20, ws=ws)
    assert sp.sp_workspace_status(ws) == sp.SP_EDEVICE and n.tolist() == [20, 0] and torch.all(kept[1] == -1)


def test_tokens_beyond_2_31_entries_are_moved(sp):
    import torch
    far = 5 * (1 << 30)
    buf = torch.zeros(far + 4096, dtype=torch.int8, device="cuda")
    k = buf.as_strided((2, 1, 16, 64), (far, 1024, 64, 1))
    v = buf.as_strided((2, 1, 16, 64), (far, 1024, 64, 1), 2048)
    s = [torch.rand(2, 1, 16, device="cuda") for _ in range(2)]
    k[1, 0] = torch.arange(16, device="cuda")[:, None].to(torch.int8)
    v[0, 0] = -torch.arange(16, device="cuda")[:, None].to(torch.int8)
    cache = sp.Cache(k, v, *s, dtype=torch.bfloat16)
    batch, _ = make_batch(sp, [0], [32], np.array([[0, 1]], np.int32))
    sp.cache_keep(cache, batch, i32([[7, 16, 31]]), torch.tensor([3], device="cuda"), check=True)
    assert k[0, 0, :4, 5].tolist() == [0, 0, 15, 0] and v[0, 0, :4, 5].tolist() == [-7, 0, 0, -3]


# ----------------------------------------------------------------------------
# Together
# ----------------------------------------------------------------------------

@pytest.mark.parametrize("kind", ["same", "int8"])
def test_a_prompt_is_cut_and_drafted_tokens_are_verified_over_it(sp, kind):
    """A prompt's chunks with the weights they give it, its cache cut to the heaviest tokens, then rounds of drafted tokens: their
    positions, attention, acceptance, and the cache that holds the accepted ones; every round's attention against the
    oracle's over the tokens that are still there."""
    import torch
    rng = np.random.default_rng(13)
    H, H_kv, d, page, M, budget = 8, 2, 64, 16, 500, 120
    plan = sp.rotary_plan(d)
    dev = lambda *s: torch.from_numpy(rng.standard_normal(s)).to(torch.bfloat16).cuda()          # noqa: E731
    i64 = lambda *v: torch.tensor(v, dtype=torch.int64, device="cuda")                          # noqa: E731
    pages = -(-(M + 64) // page)
    cache = sp.cache_alloc(pages, H_kv, page, d, kind=kind)
    weights = sp.weights_alloc(cache)
    table = torch.from_numpy(rng.permutation(pages).astype(np.int32))[None].cuda()
    total = np.zeros((H_kv, 0))
    for lo, hi in ((0, 300), (300, M)):
        q, k = sp.rotary(dev(hi - lo, H, d), dev(hi - lo, H_kv, d), torch.arange(lo, hi, dtype=torch.int32, device="cuda"), plan)
        batch = sp.Batch(i64(0, hi - lo), i64(hi), table, rows=hi - lo)
        sp.cache_write(cache, batch, k, dev(hi - lo, H_kv, d), check=True)
        _, lse = sp.attend(q, cache, batch, check=True)
        sp.attend_weights(q, cache, batch, lse, weights, decay=0.5, check=True)
        kk, _ = sp.cache_read(cache, sp.Batch(i64(0, hi), i64(hi), table, rows=hi), check=True)
        w, _ = oracle.kept.weights(f64(q), f64(kk), f64(lse), d ** -0.5, oracle.kept.visible(hi - lo, hi))
        total = 0.5 * np.pad(total, ((0, 0), (0, hi - lo))) + w
    full = sp.Batch(i64(0, M), i64(M), table, rows=M)
    k_all, v_all = (f64(t) for t in sp.cache_read(cache, full, check=True))
    kept, n_kept = sp.cache_choose(cache, full, weights, budget, first=4, last=32, check=True)
    i = np.arange(M)
    got = f64(weights)[table[0].cpu().numpy()[i // page], :, i % page].T
    assert np.all(np.abs(got - total) <= 1e-4 * total + 1e-7)
    length = sp.cache_keep(cache, full, kept, n_kept, weights=weights, check=True)
    lists = kept[0].cpu().numpy()
    k_now, v_now = (np.stack([x[h][lists[h]] for h in range(H_kv)]) for x in (k_all, v_all))
    w_now = np.stack([got[h][lists[h]] for h in range(H_kv)])
    i = np.arange(budget)
    assert np.array_equal(f64(weights)[table[0].cpu().numpy()[i // page], :, i % page].T, w_now)
    next_position = M                           # positions go on behind the whole prompt
    for n in (12, 3):
        parent = tree(rng, n, "random")
        parent[1:] = np.maximum(parent[1:], 0)
        batch = sp.Batch(i64(0, n), length + n, table, rows=n)
        seen, pos = sp.tree_seen(batch, i32(parent), check=True)
        held = int(length.item())
        pos = pos + (next_position - held)
        q, k = sp.rotary(dev(n, H, d), dev(n, H_kv, d), pos.int(), plan)
        sp.cache_write(cache, batch, k, dev(n, H_kv, d), check=True)
        out, _ = sp.attend_tree(q, cache, batch, seen, check=True)
        kk, vv = (f64(t) for t in sp.cache_read(cache, sp.Batch(i64(0, held + n), length + n, table, rows=held + n), check=True))
        assert np.array_equal(kk[:, :held], k_now) and np.array_equal(vv[:, :held], v_now)
        see, depth = oracle.kept.tree_seen(parent)
        assert np.array_equal(pos.cpu().numpy(), next_position + depth)
        ref, ref_lse, top, spread = oracle.kept.attend(f64(q), kk, vv, d ** -0.5, oracle.kept.visible(n, held + n, 0, see))
        bound, _ = attend_bounds("bf16", d, held + n, ref, spread, top, ref_lse)
        assert np.all(np.abs(f64(out) - ref) <= bound)
        draft, target = rng.integers(0, 9, n), rng.integers(0, 9, n)
        for t in range(1, n):
            if rng.random() < 0.7:
                target[parent[t]] = draft[t]
        path, n_path, nxt = sp.tree_accept(batch, i32(parent), i32(draft), i32(target), check=True)
        want, then = oracle.kept.accept(parent, draft, target)
        assert path[0, :len(want)].tolist() == want and nxt.item() == then
        length = sp.cache_keep(cache, batch, path, n_path, drafted=True, check=True)
        assert length.item() == held + len(want)
        rows = list(range(held)) + [held + t for t in want]
        k_now, v_now = kk[:, rows], vv[:, rows]
        next_position += len(want)
    kk, vv = (f64(t) for t in sp.cache_read(cache, sp.Batch(i64(0, len(rows)), length, table, rows=len(rows)), check=True))
    assert np.array_equal(kk, k_now) and np.array_equal(vv, v_now)


def test_the_positions_that_select_keeps_cut_a_cache(sp):
    import torch
    rng = np.random.default_rng(14)
    M, page = 700, 16
    cache, table, kval, vval = make_cache(sp, rng, H_kv=2, d=64, page=page, kv=[M], kind="e4m3")
    batch, _ = make_batch(sp, [0], [M], table)
    kept, n_kept = sp.select(torch.rand(M, device="cuda"), 32, 3, "topk", 0.3, trim=False)
    n = sp.cache_keep(cache, batch, kept[None], n_kept, check=True)
    n = int(n.item())
    rows = kept[:n].cpu().numpy()
    back, _ = make_batch(sp, [n], [n], table)
    k, v = sp.cache_read(cache, back, check=True)
    assert 0 < n < M and np.array_equal(f64(k), kval[0][:, rows]) and np.array_equal(f64(v), vval[0][:, rows])


def test_a_captured_cut_follows_the_arrays(sp):
    import torch
    rng = np.random.default_rng(15)
    page, H_kv, d, budget = 16, 2, 64, 50
    cache, table, kval, vval = make_cache(sp, rng, H_kv=H_kv, d=d, page=page, kv=[400, 300])
    batch, _ = make_batch(sp, [1, 1], [400, 300], table)
    q = torch.from_numpy(rng.standard_normal((2, 4, d))).to(torch.bfloat16).cuda()
    keep0 = [cache.k.clone(), cache.v.clone()]
    weights = torch.zeros(cache.pages, H_kv, page, device="cuda")
    kept = torch.zeros(2, H_kv, budget, dtype=torch.int32, device="cuda")
    n, out_len = (torch.zeros(2, dtype=torch.int64, device="cuda") for _ in range(2))
    lse = torch.zeros(4, 2, device="cuda")
    ws = [torch.zeros(sp.attend_weights_workspace_size(q, cache, batch), dtype=torch.uint8, device="cuda")] + \
         [torch.zeros(256, dtype=torch.uint8, device="cuda") for _ in range(2)]

    def call():
        sp.attend_weights(q, cache, batch, lse, weights, decay=0, ws=ws[0])
        sp.cache_choose(cache, batch, weights, budget, first=1, last=2, kept=kept, n_kept=n, ws=ws[1])
        sp.cache_keep(cache, batch, kept, n, weights=weights, kv_len=out_len, ws=ws[2])

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for lens in ([400, 300], [51, 1], [50, 299]):
        cache.k.copy_(keep0[0])
        cache.v.copy_(keep0[1])
        batch.kv_len.copy_(torch.tensor(lens))
        _, z = sp.attend(q, cache, batch)
        lse.copy_(z)
        graph.replay()
        torch.cuda.synchronize()
        assert all(sp.sp_workspace_status(w) == sp.SP_OK for w in ws)
        assert out_len.tolist() == [min(c, budget) for c in lens]
        k_now = cache.k.clone()
        for b, c in enumerate(lens):
            w, bound = oracle.kept.weights(f64(q[b:b + 1]), kval[b][:, :c], f64(z[:, b:b + 1]), d ** -0.5, np.ones((1, c), bool))
            for h in range(H_kv):
                mine = kept[b, h, :min(c, budget)].cpu().numpy()
                middle = [i for i in mine if 1 <= i < c - 2]
                if c > budget:
                    assert mine[0] == 0 and list(mine[-2:]) == [c - 2, c - 1]
                    left = np.setdiff1d(np.arange(1, c - 2), middle)
                    worst = np.argmin(w[h][middle])
                    assert np.all(w[h][left] <= w[h][middle][worst] + bound[h][left] + bound[h][middle][worst])
                for j, i in enumerate(mine):
                    assert np.array_equal(f64(k_now[int(table[b, j // page]), h, j % page]), kval[b][h, i])
