"""Rotary positions, the paged cache and the attention over it on the GPU, against the 64-bit oracle."""
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


# ----------------------------------------------------------------------------
# Rotary positions
# ----------------------------------------------------------------------------

# a pair's result is two products and a sum of fp32 values rounded to the type: half a step of the type, plus the
# sine and cosine (fp32: 2 units of 2^-24, and 2^-24 * pi from the angle's fp32 conversion) and the fp32 products and sum (2 more)
def rotary_bound(x, dtype, pairs, interleaved):
    turned = x[..., :2 * pairs]
    a, b = (turned[..., 0::2], turned[..., 1::2]) if interleaved else (turned[..., :pairs], turned[..., pairs:])
    size = np.abs(a) + np.abs(b)
    size = np.stack([size, size], -1).reshape(turned.shape) if interleaved else np.concatenate([size, size], -1)
    full = np.abs(x).copy()
    full[..., :2 * pairs] = size
    return full * ((2.0 ** -8 if dtype == "bf16" else 2.0 ** -24) + 8 * 2.0 ** -24)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,H,H_kv,d,rot,sections", [
    (1, 4, 2, 64, 64, None), (5, 32, 8, 128, 128, (16, 24, 24)), (131, 3, 1, 96, 32, None), (33, 2, 2, 16, 16, (1, 3, 4)),
    (3, 1, 1, 256, 256, None), (700, 16, 4, 64, 64, (8, 12, 12)), (2, 5, 0, 24, 16, None), (9, 0, 3, 40, 32, None),
])
def test_rotary_matches_the_oracle(sp, dtype, interleaved, T, H, H_kv, d, rot, sections):
    import torch
    rng = np.random.default_rng(T * 1000 + d)
    axes = len(sections) if sections else 1
    pos = rng.integers(-(1 << 31), 1 << 31, (axes, T)).astype(np.int32)
    pos[:, : T // 2] = rng.integers(0, 131072, (axes, T // 2))
    plan = sp.rotary_plan(rot, base=500000.0, sections=sections, interleaved=interleaved)
    freq = [500000.0 ** (-i / (rot // 2)) for i in range(rot // 2)]
    axis = [a for a, n in enumerate(sections) for _ in range(n)] if sections else [0] * (rot // 2)
    mk = lambda h: torch.from_numpy(rng.standard_normal((T, h, d))).to(torch_dtype(dtype)).cuda() if h else None  # noqa: E731
    q, k = mk(H), mk(H_kv)
    p = torch.from_numpy(pos if axes > 1 else pos[0]).cuda()
    for inverse in (False, True):
        for x, got in zip((q, k), sp.rotary(q, k, p, plan, inverse=inverse)):
            if x is None:
                assert got is None
                continue
            ref = oracle.paged.rotary(f64(x), pos, freq, axis, interleaved, inverse)
            # 2^31 * 2^-53 of a turn from the 64-bit fraction's own double: below 2^-24
            assert np.all(np.abs(f64(got) - ref) <= rotary_bound(f64(x), dtype, rot // 2, interleaved) + 1e-30)
            assert np.array_equal(f64(got)[..., rot:], f64(x)[..., rot:])


def test_rotary_in_place_on_slices_of_a_fused_projection(sp):
    import torch
    T, H, H_kv, d = 77, 6, 2, 64
    g = torch.Generator().manual_seed(3)
    qkv = torch.randn(T, H + 2 * H_kv, d, generator=g).to(torch.bfloat16).cuda()
    pos = torch.arange(1000, 1000 + T, dtype=torch.int32).cuda()
    plan = sp.rotary_plan(d)
    want_q, want_k = sp.rotary(qkv[:, :H].contiguous(), qkv[:, H:H + H_kv].contiguous(), pos, plan)
    before = qkv.clone()
    q, k = qkv[:, :H], qkv[:, H:H + H_kv]
    sp.rotary(q, k, pos, plan, q_out=q, k_out=k)
    assert torch.equal(qkv[:, :H], want_q) and torch.equal(qkv[:, H:H + H_kv], want_k)
    assert torch.equal(qkv[:, H + H_kv:], before[:, H + H_kv:])


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_inverse_is_its_gradient(sp, interleaved):
    import torch
    T, H, d = 9, 3, 32
    rng = np.random.default_rng(5)
    pos = rng.integers(0, 5000, (1, T)).astype(np.int32)
    x, g, e = (torch.from_numpy(rng.standard_normal((T, H, d))).float().cuda() for _ in range(3))
    plan = sp.rotary_plan(d, interleaved=interleaved)
    p = torch.from_numpy(pos).cuda()
    grad, _ = sp.rotary(g, None, p, plan, inverse=True)
    # the formula's gradient: the transpose of the rotation, by its matrix' columns
    freq, axis = [10000.0 ** (-i / (d // 2)) for i in range(d // 2)], [0] * (d // 2)
    columns = np.stack([oracle.paged.rotary(np.broadcast_to(np.eye(d)[j], (T, 1, d)), pos, freq, axis, interleaved)[:, 0]
                        for j in range(d)], -1)                          # [T, out, in]
    want = np.einsum("toi,tho->thi", columns, f64(g))
    assert np.all(np.abs(f64(grad) - want) <= rotary_bound(f64(g), "f32", d // 2, interleaved))
    # differences: the map is linear, so a difference of any size has the gradient's product.  Each result is off
    # by 9 * 2^-24 of at most sqrt(2) * |pair|: summed over T H d entries against g, in quadrature and six times that
    up, _ = sp.rotary(x + e, None, p, plan)
    down, _ = sp.rotary(x, None, p, plan)
    lhs = ((f64(up) - f64(down)) * f64(g)).sum()
    rhs = (f64(x + e) - f64(x)).ravel() @ f64(grad).ravel()
    assert abs(lhs - rhs) <= 6 * np.sqrt(T * H * d) * 3 * 9 * 2.0 ** -24 * 10


def test_rotary_of_no_tokens(sp):
    import torch
    q = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    out, k = sp.rotary(q, None, torch.empty(0, dtype=torch.int32, device="cuda"), sp.rotary_plan(64))
    assert out.shape == q.shape and k is None


# ----------------------------------------------------------------------------
# The cache
# ----------------------------------------------------------------------------

SHAPES = [  # H_kv, d, page, new, kv, rows before and behind
    (2, 64, 16, [1], [1], 0, 0), (8, 128, 64, [70, 0, 1], [200, 0, 64], 0, 3), (3, 72, 7, [20, 5], [20, 33], 2, 1),
    (1, 256, 1, [9], [12], 0, 0), (4, 8, 48, [100], [100], 0, 0), (2, 40, 128, [5, 6, 7], [3, 300, 7], 1, 0),
]


def rows_with_edges(rng, T, H_kv, d, dtype):
    """Rows of all sizes: normal ones, zeros, tiny and huge ones, halfway values, and some that hold NaN and infinity."""
    import torch
    x = rng.standard_normal((T, H_kv, d)) * 2.0 ** rng.integers(-8, 8, (T, H_kv, 1))
    for i in range(T):
        kind = i % 9
        if kind == 1:
            x[i] = 0
        elif kind == 2:
            x[i] *= 2.0 ** -110
        elif kind == 3:
            x[i] *= 2.0 ** 110
        elif kind == 4:
            x[i] = rng.integers(-254, 255, (H_kv, d)) / 2       # half steps of the 8-bit integers
            x[i, :, 0] = 127
        elif kind == 5:
            x[i, 0, d // 2] = np.nan
        elif kind == 6:
            x[i, -1, d - 1] = -np.inf
        elif kind == 7:
            x[i, :, 0] = 448 * 2.0 ** -3                        # the largest code exactly, and one step above
            x[i, :, 1:] = np.clip(x[i, :, 1:], -50, 50)
    return torch.from_numpy(x).to(torch_dtype(dtype))


@pytest.mark.parametrize("layout", ["hnd", "nhd"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["same", "e4m3", "int8"])
@pytest.mark.parametrize("H_kv,d,page,new,kv,before,behind", SHAPES)
def test_cache_write_and_read(sp, H_kv, d, page, new, kv, before, behind, kind, dtype, layout):
    import torch
    rng = np.random.default_rng(d * page)
    cache, table, kval, vval = make_cache(sp, rng, H_kv=H_kv, d=d, page=page, kv=kv, kind=kind, dtype=torch_dtype(dtype),
                                          layout=layout)
    T = before + sum(new) + behind
    batch, cu = make_batch(sp, new, kv, table, rows=T, first=before, max_new=max(new))
    k_new, v_new = (rows_with_edges(rng, T, H_kv, d, dtype) for _ in range(2))
    raw = lambda t: t.contiguous().view(torch.uint8 if kind != "same" else t.dtype).cpu()        # noqa: E731
    sides = [(cache.k, cache.k_scale), (cache.v, cache.v_scale)]
    old = [(raw(t), None if s is None else s.cpu()) for t, s in sides]
    sp.cache_write(cache, batch, k_new.cuda(), v_new.cuda(), check=True)
    places = oracle.paged.places(cu, kv)
    read = sp.cache_read(cache, batch, out_k=torch.full((H_kv, T, d), 7.0, dtype=torch_dtype(dtype), device="cuda"),
                         out_v=torch.full((H_kv, T, d), 7.0, dtype=torch_dtype(dtype), device="cuda"), check=True)
    for x, (t, s), (was, was_scale), got in zip((k_new, v_new), sides, old, read):
        now = raw(t)
        touched = torch.zeros(t.shape[:3], dtype=torch.bool)
        for r, (b, i) in enumerate(places):
            row = x[before + r].double().numpy()
            back = f64(got[:, before + r])
            if i < 0:
                assert np.all(back == 0)
                continue
            pg, slot = table[b, i // page], i % page
            touched[pg, :, slot] = True
            if kind == "same":
                assert np.array_equal(f64(t[pg, :, slot]), row, equal_nan=True)
                assert np.array_equal(back, row, equal_nan=True)
                continue
            codes, scale = oracle.paged.quantise(row, kind)
            held = f64(t[pg, :, slot].float())
            assert np.array_equal(f64(s[pg, :, slot]), scale, equal_nan=True)
            assert np.array_equal(held, codes)
            with np.errstate(invalid="ignore"):
                assert np.array_equal(back, f64(torch.from_numpy(codes * scale[:, None]).to(torch_dtype(dtype))), equal_nan=True)
        assert torch.equal(now[~touched], was[~touched])
        if s is not None:
            assert torch.equal(s.cpu()[~touched], was_scale[~touched])
        left = f64(got)
        assert np.all(left[:, :before] == 7) and np.all(left[:, before + sum(new):] == 7)


def test_cache_read_one_side_into_a_layer_of_k_prompt(sp):
    import torch
    rng = np.random.default_rng(8)
    kv = [37, 64, 5]
    cache, table, kval, _ = make_cache(sp, rng, H_kv=2, d=64, page=16, kv=kv, kind="e4m3")
    batch, cu = make_batch(sp, kv, kv, table)
    K = torch.zeros(3, 2, sum(kv), 64, dtype=torch.bfloat16, device="cuda")
    k, v = sp.cache_read(cache, batch, out_k=K[1], check=True)
    assert v is None and k.data_ptr() == K[1].data_ptr()
    for b in range(3):
        assert np.array_equal(f64(K[1][:, cu[b]:cu[b + 1]]), kval[b])
    assert not K[0].any() and not K[2].any()


def test_every_code_reads_back_as_its_value(sp):
    import torch
    codes = torch.arange(256, dtype=torch.uint8).view(1, 1, 2, 128)
    for held in (torch.float8_e4m3fn, torch.int8):
        for scale in (1.0, 2.0 ** -100, 2.0 ** 119):
            k = codes.view(held).cuda()
            s = torch.full((1, 1, 2), scale, device="cuda")
            cache = sp.Cache(k, k.clone(), s, s.clone())
            batch, _ = make_batch(sp, [2], [2], np.zeros((1, 1), np.int32))
            got, _ = sp.cache_read(cache, batch, check=True)
            want = (codes.view(held).double() * scale).view(1, 2, 128)
            assert np.array_equal(f64(got), want.numpy(), equal_nan=True)


def test_rows_of_a_cache_beyond_2_31_entries(sp):
    import torch
    # two pages, 5 * 2^30 bytes apart
    far = 5 * (1 << 30)
    buf = torch.zeros(far + 4096, dtype=torch.int8, device="cuda")
    k = buf.as_strided((2, 1, 16, 64), (far, 1024, 64, 1))
    v = buf.as_strided((2, 1, 16, 64), (far, 1024, 64, 1), 2048)
    s = [torch.zeros(2, 1, 16, device="cuda") for _ in range(2)]
    cache = sp.Cache(k, v, *s, dtype=torch.bfloat16)
    batch, _ = make_batch(sp, [20], [20], np.array([[1, 0]], np.int32))
    x = torch.randn(20, 1, 64, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    sp.cache_write(cache, batch, x.cuda(), (-x).cuda(), check=True)
    got, gotv = sp.cache_read(cache, batch, check=True)
    codes, scale = oracle.paged.quantise(x[:, 0].double().numpy(), "int8")
    assert np.array_equal(f64(got)[0], codes * scale[:, None]) and np.array_equal(f64(gotv)[0], -codes * scale[:, None])
    out, lse = sp.attend(x.cuda(), cache, batch, check=True)
    ref = oracle.paged.attend(x.double().numpy(), f64(got), f64(gotv), 0.125)
    bound, lse_bound = attend_bounds("bf16", 64, 20, ref[0], ref[3], ref[2], ref[1])
    assert np.all(np.abs(f64(out) - ref[0]) <= bound) and np.all(np.abs(f64(lse) - ref[1]) <= lse_bound)


# ----------------------------------------------------------------------------
# Attention
# ----------------------------------------------------------------------------

def check_attend(sp, *, H, H_kv, d, page, new, kv, dtype="bf16", kind="same", window=0, layout="hnd", before=0, behind=0,
                 scale=None, seed=0, junk=float("nan"), q_gain=1.0):
    import torch
    rng = np.random.default_rng(seed + 17 * d + page)
    td = torch_dtype(dtype)
    cache, table, kval, vval = make_cache(sp, rng, H_kv=H_kv, d=d, page=page, kv=kv, kind=kind, dtype=td, layout=layout,
                                          junk=junk)
    T = before + sum(new) + behind
    batch, cu = make_batch(sp, new, kv, table, rows=T, first=before, max_new=max(new))
    q = torch.from_numpy(rng.standard_normal((T, H, d)) * q_gain).to(td)
    # rows of no token hold NaN, and what they would write to must stay
    real = np.zeros(T, dtype=bool)
    real[before:before + sum(new)] = True
    q[~torch.from_numpy(real)] = float("nan")
    out = torch.full((T, H, d), 7.0, dtype=td, device="cuda")
    lse = torch.full((H, T), 7.0, dtype=torch.float32, device="cuda")
    sp.attend(q.cuda(), cache, batch, scale=scale, window=window, out=out, lse=lse, check=True)
    got, got_lse = f64(out), f64(lse)
    assert np.all(got[~real] == 7) and np.all(got_lse[:, ~real] == 7)
    qd = q.double().numpy()
    for b in range(len(new)):
        lo, hi = int(cu[b]), int(cu[b + 1])
        if lo == hi:
            continue
        ref, ref_lse, top, spread = oracle.paged.attend(qd[lo:hi], kval[b], vval[b], d ** -0.5 if scale is None else scale,
                                                        window)
        bound, lse_bound = attend_bounds(dtype, d, kv[b], ref, spread, top, ref_lse)
        err = np.abs(got[lo:hi] - ref)
        assert np.all(err <= bound), f"sequence {b}: out off by {np.nanmax(err / bound)} of its bound"
        empty = np.isneginf(ref_lse)
        assert np.array_equal(np.isneginf(got_lse[:, lo:hi]), empty)
        assert np.all(got[lo:hi][empty.T] == 0)
        with np.errstate(invalid="ignore"):
            assert np.all((np.abs(got_lse[:, lo:hi] - ref_lse) <= lse_bound) | empty)


@pytest.mark.parametrize("kind", ["same", "e4m3", "int8"])
@pytest.mark.parametrize("H,H_kv,d,page", [
    (4, 2, 64, 16), (32, 8, 128, 64), (7, 7, 64, 32), (6, 2, 128, 128), (8, 1, 64, 48), (5, 1, 40, 7), (2, 1, 256, 16),
    (16, 1, 128, 1), (3, 3, 8, 5), (24, 1, 64, 256),
])
@pytest.mark.parametrize("new,kv", [
    ([1], [1]), ([1, 1, 0, 1, 1], [17, 300, 0, 128, 129]), ([2, 3, 1], [2, 5, 1023]),
])
def test_attend_decode_steps(sp, H, H_kv, d, page, new, kv, kind):
    check_attend(sp, H=H, H_kv=H_kv, d=d, page=page, new=new, kv=kv, kind=kind, behind=2)


@pytest.mark.parametrize("kind", ["same", "e4m3", "int8"])
@pytest.mark.parametrize("H,H_kv,d,page", [
    (4, 2, 64, 16), (8, 2, 128, 64), (3, 1, 64, 32), (6, 2, 128, 128), (7, 1, 64, 48), (2, 2, 40, 7), (2, 1, 128, 8),
    (12, 1, 128, 256),
])
@pytest.mark.parametrize("new,kv,window", [
    ([33], [33], 0), ([64, 1, 65, 0], [64, 400, 200, 0], 0), ([129, 5], [300, 2], 0), ([100, 40], [260, 40], 37),
    ([1, 70], [500, 128], 128),
])
def test_attend_chunks(sp, H, H_kv, d, page, new, kv, window, kind):
    check_attend(sp, H=H, H_kv=H_kv, d=d, page=page, new=new, kv=kv, kind=kind, window=window, before=1, behind=3)


@pytest.mark.parametrize("kind", ["same", "e4m3", "int8"])
@pytest.mark.parametrize("new,kv,window", [
    ([1], [512], 0), ([1, 1], [1, 700], 9), ([5, 0, 40], [3, 0, 90], 0), ([130], [131], 64),
])
@pytest.mark.parametrize("H,H_kv,d,page", [(4, 2, 64, 16), (3, 1, 128, 5), (2, 2, 256, 32)])
def test_attend_single_precision(sp, H, H_kv, d, page, new, kv, window, kind):
    check_attend(sp, H=H, H_kv=H_kv, d=d, page=page, new=new, kv=kv, kind=kind, window=window, dtype="f32", behind=1)


@pytest.mark.parametrize("new,kv", [([1, 1], [5000, 40]), ([300, 1, 20], [1300, 2000, 30])])
@pytest.mark.parametrize("layout,q_gain,scale", [("nhd", 1.0, None), ("hnd", 12.0, None), ("nhd", 1.0, 3.0), ("hnd", 1.0, 1e-4)])
@pytest.mark.parametrize("d,page", [(64, 16), (128, 64)])
@pytest.mark.parametrize("kind", ["same", "int8"])
def test_attend_layouts_and_scales(sp, new, kv, layout, q_gain, scale, d, page, kind):
    check_attend(sp, H=4, H_kv=2, d=d, page=page, new=new, kv=kv, layout=layout, q_gain=q_gain, scale=scale, kind=kind)


@pytest.mark.parametrize("fill", [float("inf"), float("-inf"), 3e38])
@pytest.mark.parametrize("new", [[1], [200]])
def test_unwritten_slots_have_no_effect(sp, fill, new):
    check_attend(sp, H=4, H_kv=2, d=128, page=64, new=new, kv=[205], junk=fill)


@pytest.mark.parametrize("kind", ["same", "e4m3"])
@pytest.mark.parametrize("d,dtype", [(64, "bf16"), (128, "bf16"), (64, "f32")])
@pytest.mark.parametrize("n", [1, 6, 150])
@pytest.mark.parametrize("shape", ["up", "down", "late", "spike"])
def test_logits_that_leave_the_running_maximum_behind(sp, shape, n, d, dtype, kind):
    """Logits that climb or fall by hundreds from one end of the cache to the other, or jump in one place."""
    import torch
    rng = np.random.default_rng(21)
    td = torch_dtype(dtype)
    H, H_kv, page, kv = 4, 2, 16, 700
    along = np.arange(kv) / kv
    level = {"up": 300 * along, "down": 300 - 300 * along, "late": np.where(np.arange(kv) % 128 == 127, 40.0, -40.0),
             "spike": np.where(np.arange(kv) == 250, 90.0, 0.0)}[shape]
    cache, table, kval, vval = make_cache(sp, rng, H_kv=H_kv, d=d, page=page, kv=[kv], dtype=td, kind=kind)
    k = rng.standard_normal((kv, H_kv, d)) * 0.3
    k[:, :, 0] = level[:, None] * 4         # times q[0] = 4 and the scale 1 / 16
    new = torch.from_numpy(k).to(td)
    v = torch.from_numpy(rng.standard_normal((kv, H_kv, d))).to(td)
    fill, _ = make_batch(sp, [kv], [kv], table)
    sp.cache_write(cache, fill, new.cuda(), v.cuda(), check=True)
    kk, vv = sp.cache_read(cache, fill, check=True)
    q = torch.from_numpy(rng.standard_normal((n, H, d))).to(td)
    q[:, :, 0] = 4
    batch, _ = make_batch(sp, [n], [kv], table)
    out, lse = sp.attend(q.cuda(), cache, batch, scale=1 / 16, check=True)
    ref, ref_lse, top, spread = oracle.paged.attend(q.double().numpy(), f64(kk), f64(vv), 1 / 16)
    bound, lse_bound = attend_bounds(dtype, d, kv, ref, spread, top, ref_lse)
    assert np.all(np.abs(f64(out) - ref) <= bound) and np.all(np.abs(f64(lse) - ref_lse) <= lse_bound)


@pytest.mark.parametrize("kind", ["same", "e4m3", "int8"])
@pytest.mark.parametrize("d,dtype", [(64, "bf16"), (128, "bf16"), (64, "f32")])
@pytest.mark.parametrize("n", [1, 150])
@pytest.mark.parametrize("size", [2.0 ** 9, 2.0 ** 14, 2.0 ** 40, -2.0 ** 12, -2.0 ** 40])
def test_logits_beyond_single_precision_steps(sp, size, n, d, dtype, kind):
    """Logits of 2^18 to 2^88, where neighbouring fp32 values are up to 2^64 apart: the largest one takes all (tokens
    whose keys are equal share it)."""
    import torch
    rng = np.random.default_rng(25)
    td = torch_dtype(dtype)
    H, H_kv, page, kv = 4, 2, 16, 200
    cache, table, _, _ = make_cache(sp, rng, H_kv=H_kv, d=d, page=page, kv=[kv], dtype=td, kind=kind)
    k = torch.zeros(kv, H_kv, d, dtype=td)
    k[:, :, 0] = ((torch.arange(kv) + 1) * abs(size))[:, None].to(td)
    v = torch.from_numpy(rng.standard_normal((kv, H_kv, d))).to(td)
    fill, _ = make_batch(sp, [kv], [kv], table)
    sp.cache_write(cache, fill, k.cuda(), v.cuda(), check=True)
    kk, vv = sp.cache_read(cache, fill, check=True)
    q = torch.zeros(n, H, d, dtype=td)
    q[:, :, 0] = size
    batch, _ = make_batch(sp, [n], [kv], table)
    out, lse = sp.attend(q.cuda(), cache, batch, scale=1.0, check=True)
    ref, ref_lse, _, spread = oracle.paged.attend(q.double().numpy(), f64(kk), f64(vv), 1.0)
    # the keys are 2^-8 apart or equal, so a weight is 0 or 1 exactly; sums of equal weights as fp32 and bf16 allow
    assert np.all(np.abs(f64(out) - ref) <= (2.0 ** -7 if dtype == "bf16" else 2.0 ** -20) * spread)
    assert np.all(np.abs(f64(lse) - ref_lse) <= 2.0 ** -20 * np.abs(ref_lse))


@pytest.mark.parametrize("kind", ["same", "e4m3", "int8"])
@pytest.mark.parametrize("d,dtype", [(64, "bf16"), (128, "bf16"), (64, "f32")])
@pytest.mark.parametrize("n", [1, 150])
@pytest.mark.parametrize("spread", [1e4, 1e10, 1e30])
def test_rows_of_all_sizes_stay_finite(sp, spread, n, d, dtype, kind):
    """Keys whose sizes spread over many decades: every output is a mean of values."""
    import torch
    rng = np.random.default_rng(26)
    td = torch_dtype(dtype)
    H, H_kv, page, kv = 4, 2, 16, 400
    cache, table, _, _ = make_cache(sp, rng, H_kv=H_kv, d=d, page=page, kv=[kv], dtype=td, kind=kind)
    size = spread ** rng.uniform(-1, 1, (kv, H_kv, 1))
    k = torch.from_numpy(rng.standard_normal((kv, H_kv, d)) * size).to(td)
    v = torch.from_numpy(rng.standard_normal((kv, H_kv, d))).to(td)
    fill, _ = make_batch(sp, [kv], [kv], table)
    sp.cache_write(cache, fill, k.cuda(), v.cuda(), check=True)
    _, vv = sp.cache_read(cache, fill, check=True)
    q = torch.from_numpy(rng.standard_normal((n, H, d))).to(td)
    batch, _ = make_batch(sp, [n], [kv], table)
    out, lse = sp.attend(q.cuda(), cache, batch, check=True)
    got = f64(out)
    assert np.all(np.isfinite(got)) and np.all(np.isfinite(f64(lse)))
    assert np.abs(got).max() <= np.abs(f64(vv)).max() * (1 + 2.0 ** -7)


@pytest.mark.parametrize("d,dtype", [(64, "bf16"), (40, "f32")])
def test_a_batch_without_rows(sp, d, dtype):
    import torch
    cache = sp.cache_alloc(2, 1, 16, d, dtype=torch_dtype(dtype))
    batch, _ = make_batch(sp, [0, 0], [5, 0], np.array([[0], [1]]), rows=0, max_new=700)
    empty = torch.empty(0, 2, d, dtype=torch_dtype(dtype), device="cuda")
    out, lse = sp.attend(empty, cache, batch, check=True)
    assert out.shape == (0, 2, d) and lse.shape == (2, 0)
    sp.cache_write(cache, batch, empty[:, :1], empty[:, :1], check=True)
    assert sp.cache_read(cache, batch, check=True)[0].shape == (1, 0, d)


@pytest.mark.parametrize("kind", ["same", "int8"])
def test_many_sequences_of_all_kinds_at_once(sp, kind):
    rng = np.random.default_rng(22)
    new = [int(x) for x in rng.choice([0, 1, 1, 1, 2, 4, 5, 33, 70], 90)]
    kv = [n + int(rng.integers(0, 300)) for n in new]
    kv[3] = 0
    check_attend(sp, H=4, H_kv=1, d=64, page=16, new=new, kv=kv, kind=kind, behind=4)


@pytest.mark.parametrize("n", [1, 100])
def test_two_streams_at_once(sp, n):
    import torch
    rng = np.random.default_rng(23)
    runs = []
    for i in range(2):
        cache, table, _, _ = make_cache(sp, rng, H_kv=2, d=128, page=16, kv=[3000 + n])
        batch, _ = make_batch(sp, [n], [3000 + n], table)
        q = torch.from_numpy(rng.standard_normal((n, 8, 128))).to(torch.bfloat16).cuda()
        runs.append((cache, batch, q, sp.attend(q, cache, batch, check=True)[0], torch.cuda.Stream()))
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(8):
        for i, (cache, batch, q, _, stream) in enumerate(runs):
            outs[i].append(sp.attend(q, cache, batch, stream=stream)[0])
    torch.cuda.synchronize()
    for i in range(2):
        for o in outs[i]:
            assert torch.equal(o, runs[i][3])


def test_a_chunk_over_a_cache_beyond_2_31_entries(sp):
    import torch
    far = 3 * (1 << 30)         # entries between two pages
    buf = torch.zeros(far + 8192, dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(24)
    pages = [buf.as_strided((2, 1, 64, 64), (far, 4096, 64, 1), at) for at in (0, 4096)]
    cache = sp.Cache(*pages)
    x, y = (torch.from_numpy(rng.standard_normal((100, 1, 64))).to(torch.bfloat16) for _ in range(2))
    batch, _ = make_batch(sp, [100], [100], np.array([[1, 0]], np.int32))
    sp.cache_write(cache, batch, x.cuda(), y.cuda(), check=True)
    out, lse = sp.attend(x.cuda(), cache, batch, check=True)
    ref = oracle.paged.attend(x.double().numpy(), x.double().numpy().transpose(1, 0, 2), y.double().numpy().transpose(1, 0, 2), 0.125)
    bound, lse_bound = attend_bounds("bf16", 64, 100, ref[0], ref[3], ref[2], ref[1])
    assert np.all(np.abs(f64(out) - ref[0]) <= bound) and np.all(np.abs(f64(lse) - ref[1]) <= lse_bound)


@pytest.mark.parametrize("d,dtype,n", [(64, "bf16", 1), (128, "bf16", 3), (64, "f32", 2), (128, "bf16", 90), (40, "bf16", 5)])
def test_pages_behind_the_window_may_be_gone(sp, d, dtype, n):
    import torch
    rng = np.random.default_rng(13)
    td = torch_dtype(dtype)
    H, H_kv, page, kv, window = 4, 2, 16, 700, 100
    cache, table, kval, vval = make_cache(sp, rng, H_kv=H_kv, d=d, page=page, kv=[kv], dtype=td)
    first = kv - n - window + 1
    cache.k[table[0, first // page], :, :first % page] = float("nan")       # in the window's first page, before it
    cache.v[table[0, first // page], :, :first % page] = float("nan")
    table[0, :first // page] = -1
    batch, _ = make_batch(sp, [n], [kv], table)
    q = torch.from_numpy(rng.standard_normal((n, H, d))).to(td).cuda()
    out, lse = sp.attend(q, cache, batch, window=window, check=True)
    ref, ref_lse, top, spread = oracle.paged.attend(f64(q), kval[0], vval[0], d ** -0.5, window)
    bound, lse_bound = attend_bounds(dtype, d, window, ref, spread, top, ref_lse)
    assert np.all(np.abs(f64(out) - ref) <= bound) and np.all(np.abs(f64(lse) - ref_lse) <= lse_bound)


def test_a_long_cache(sp):
    check_attend(sp, H=2, H_kv=1, d=64, page=16, new=[1, 17], kv=[70001, 9001])


@pytest.mark.parametrize("H,H_kv,d,page", [(4, 2, 64, 16), (3, 1, 256, 7), (2, 1, 8, 32)])
@pytest.mark.parametrize("kind", ["same", "int8"])
def test_items_cut_into_hundreds_of_parts(sp, H, H_kv, d, page, kind):
    check_attend(sp, H=H, H_kv=H_kv, d=d, page=page, new=[1, 2], kv=[20000, 9000], dtype="f32", kind=kind)


@pytest.mark.parametrize("d,dtype", [(64, "bf16"), (128, "bf16"), (48, "bf16"), (64, "f32")])
@pytest.mark.parametrize("n", [1, 150])
def test_strided_queries_and_outputs(sp, d, dtype, n):
    import torch
    rng = np.random.default_rng(4)
    td = torch_dtype(dtype)
    H, H_kv, page, kv = 4, 2, 16, [n + 20]
    cache, table, kval, vval = make_cache(sp, rng, H_kv=H_kv, d=d, page=page, kv=kv, dtype=td)
    batch, _ = make_batch(sp, [n], kv, table)
    qkv = torch.from_numpy(rng.standard_normal((n, H + 2 * H_kv, d))).to(td).cuda()
    q = qkv[:, :H]
    want, want_lse = sp.attend(q.contiguous(), cache, batch, check=True)
    out = torch.zeros(H, n, d, dtype=td, device="cuda").transpose(0, 1)
    lse = torch.zeros(3, n, 5, H, device="cuda")[1, :, 2].T
    sp.attend(q, cache, batch, out=out, lse=lse, check=True)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 40), ("f32", 64)])
@pytest.mark.parametrize("n", [1, 140])
def test_what_the_arrays_get_wrong_is_reported_and_does_no_harm(sp, dtype, d, n):
    import torch
    rng = np.random.default_rng(6)
    td = torch_dtype(dtype)
    H, H_kv, page = 4, 2, 16
    new, kv = [n, n, n], [n + 50, n + 40, n + 30]
    cache, table, kval, vval = make_cache(sp, rng, H_kv=H_kv, d=d, page=page, kv=kv, dtype=td)
    good, cu = make_batch(sp, new, kv, table)
    T = 3 * n
    q = torch.from_numpy(rng.standard_normal((T, H, d))).to(td).cuda()
    x = torch.from_numpy(rng.standard_normal((T, H_kv, d))).to(td).cuda()
    bad_page = table.copy()
    bad_page[1, 1] = cache.pages
    negative = table.copy()
    negative[1, 0] = -1
    far = torch.tensor([n + 50, 16 * table.shape[1] + 1, n + 30]).cuda()
    cases = [make_batch(sp, new, kv, bad_page)[0], sp.Batch(good.cu_new, good.kv_len, torch.from_numpy(np.where(negative < 0, -1, negative)).cuda(), rows=T),
             sp.Batch(good.cu_new, far, good.table, rows=T), sp.Batch(good.cu_new, -good.kv_len, good.table, rows=T),
             sp.Batch(good.cu_new, good.kv_len, good.table, rows=T, max_new=n - 1),
             sp.Batch(good.cu_new + 1, good.kv_len, good.table, rows=T)]
    for i, batch in enumerate(cases):
        out = torch.full((T, H, d), 7.0, dtype=td, device="cuda")
        ws = torch.empty(sp.attend_workspace_size(q, cache, batch), dtype=torch.uint8, device="cuda")
        sp.attend(q, cache, batch, out=out, ws=ws)
        assert sp.sp_workspace_status(ws) == sp.SP_EDEVICE, i
        for b in (0, 2) if i < 3 else ():
            # the sequences around the bad one are right.  (Not to the bit what they are without it: where the keys are
            # cut, and so the order of the sums, goes by the whole batch.  The bound holds for every order.)
            ref, ref_lse, top, spread = oracle.paged.attend(f64(q[b * n:(b + 1) * n]), kval[b], vval[b], d ** -0.5)
            bound, _ = attend_bounds(dtype, d, kv[b], ref, spread, top, ref_lse)
            assert np.all(np.abs(f64(out[b * n:(b + 1) * n]) - ref) <= bound)
        if i in (2, 3, 4):
            assert torch.all(out[n:2 * n] == 7)
    # writing and reading: a bad page among the new tokens' own
    tail = table.copy()
    tail[1, (kv[1] - 1) // page] = 0x7ffffff0
    batch = make_batch(sp, new, kv, tail)[0]
    before = cache.k.clone()
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    sp.cache_write(cache, batch, x, x, ws=ws)
    assert sp.sp_workspace_status(ws) == sp.SP_EDEVICE
    for r, (b, i) in enumerate(oracle.paged.places(cu, kv)):
        pg = tail[b, i // page]
        if pg < cache.pages:
            before[pg, :, i % page] = x[r]
    assert torch.equal(cache.k, before)
    k, _ = sp.cache_read(cache, batch, ws=ws)
    assert sp.sp_workspace_status(ws) == sp.SP_EDEVICE
    gone = [r for r, (b, i) in enumerate(oracle.paged.places(cu, kv)) if tail[b, i // page] >= cache.pages]
    assert gone and torch.all(k[:, gone] == 0)
    sp.cache_read(cache, good, ws=ws)
    assert sp.sp_workspace_status(ws) == sp.SP_OK


@pytest.mark.parametrize("n,dtype", [(1, "bf16"), (200, "bf16"), (1, "f32")])
def test_a_captured_call_follows_the_arrays_and_two_of_them_do_not_meet(sp, n, dtype):
    import torch
    rng = np.random.default_rng(9)
    td = torch_dtype(dtype)
    H, H_kv, d, page = 4, 2, 64, 16
    cap = [n + 600, n + 300]
    cache, table, kval, vval = make_cache(sp, rng, H_kv=H_kv, d=d, page=page, kv=cap, dtype=td)
    runs = []
    for g in range(2):
        batch, cu = make_batch(sp, [n, n], cap, table)
        q = torch.from_numpy(rng.standard_normal((2 * n, H, d))).to(td).cuda()
        out = torch.zeros_like(q)
        lse = torch.zeros(H, 2 * n, device="cuda")
        ws = torch.empty(sp.attend_workspace_size(q, cache, batch), dtype=torch.uint8, device="cuda")
        sp.attend(q, cache, batch, out=out, lse=lse, ws=ws)
        torch.cuda.synchronize()
        graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph, stream=stream):
            sp.attend(q, cache, batch, out=out, lse=lse, ws=ws)
        runs.append((graph, stream, batch, q, out, lse, ws))
    torch.cuda.synchronize()
    for lens in ([n + 600, n + 300], [n + 13, n], [n - 1, n + 299]):
        for graph, stream, batch, q, out, lse, ws in runs:
            batch.kv_len.copy_(torch.tensor(lens))
            out.fill_(7)
        torch.cuda.synchronize()
        for _ in range(3):
            for graph, stream, *_ in runs:
                with torch.cuda.stream(stream):
                    graph.replay()
        torch.cuda.synchronize()
        for graph, stream, batch, q, out, lse, ws in runs:
            assert sp.sp_workspace_status(ws) == sp.SP_OK
            want, want_lse = sp.attend(q, cache, batch, check=True)
            assert torch.equal(out, want) and torch.equal(lse, want_lse)
            for b in range(2):
                ref = oracle.paged.attend(f64(q[b * n:(b + 1) * n]), kval[b][:, :lens[b]], vval[b][:, :lens[b]], d ** -0.5)
                bound, _ = attend_bounds(dtype, d, max(lens[b], 1), ref[0], ref[3], ref[2], ref[1])
                assert np.all(np.abs(f64(out[b * n:(b + 1) * n]) - ref[0]) <= bound)


def test_calls_on_another_stream(sp):
    import torch
    rng = np.random.default_rng(10)
    cache, table, kval, vval = make_cache(sp, rng, H_kv=2, d=64, page=16, kv=[300])
    batch, _ = make_batch(sp, [1], [300], table)
    q = torch.from_numpy(rng.standard_normal((1, 4, 64))).to(torch.bfloat16).cuda()
    want, _ = sp.attend(q, cache, batch, check=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for handle in (s, s.cuda_stream):
        out, _ = sp.attend(q, cache, batch, stream=handle)
        s.synchronize()
        assert torch.equal(out, want)


def test_the_same_call_gives_the_same_bits(sp):
    import torch
    rng = np.random.default_rng(11)
    for d, new, kv in ((64, [1, 1, 1], [9000, 20, 3000]), (128, [900, 3], [5000, 8000])):
        cache, table, _, _ = make_cache(sp, rng, H_kv=2, d=d, page=16, kv=kv)
        batch, _ = make_batch(sp, new, kv, table)
        q = torch.from_numpy(rng.standard_normal((sum(new), 8, d))).to(torch.bfloat16).cuda()
        first = sp.attend(q, cache, batch)
        for _ in range(3):
            again = sp.attend(q, cache, batch)
            assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


# ----------------------------------------------------------------------------
# Together
# ----------------------------------------------------------------------------

@pytest.mark.parametrize("kind", ["same", "e4m3"])
def test_from_the_speculators_cache_to_the_targets_sparse_prefill(sp, kind):
    """Chunked prefill into a paged cache, look-ahead steps whose lse goes to score_lse, selection, and the target's
    attention of the kept tokens at their original positions."""
    import torch
    rng = np.random.default_rng(12)
    L, H, H_kv, d, M, N, page = 2, 8, 2, 64, 700, 3, 16
    plan = sp.rotary_plan(d)
    freq, axis = [10000.0 ** (-i / (d // 2)) for i in range(d // 2)], [0] * (d // 2)
    dev = lambda *s: torch.from_numpy(rng.standard_normal(s)).to(torch.bfloat16).cuda()          # noqa: E731
    pages = -(-(M + N) // page)
    table = torch.from_numpy(rng.permutation(pages).astype(np.int32))[None].cuda()
    i64 = lambda *v: torch.tensor(v, dtype=torch.int64, device="cuda")                          # noqa: E731
    caches = [sp.cache_alloc(pages, H_kv, page, d, kind=kind) for _ in range(L)]
    Q_la = torch.zeros(N, L, H, d, dtype=torch.bfloat16, device="cuda")
    K_prompt = torch.zeros(L, H_kv, M, d, dtype=torch.bfloat16, device="cuda")
    K_la = torch.zeros(L, H_kv, N, d, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(L, H, N, device="cuda")
    for layer in range(L):
        for lo, hi in ((0, 400), (400, M)):
            pos = torch.arange(lo, hi, dtype=torch.int32, device="cuda")
            q, k = sp.rotary(dev(hi - lo, H, d), dev(hi - lo, H_kv, d), pos, plan)
            batch = sp.Batch(i64(0, hi - lo), i64(hi), table, rows=hi - lo)
            sp.cache_write(caches[layer], batch, k, dev(hi - lo, H_kv, d), check=True)
            sp.attend(q, caches[layer], batch, check=True)
        for j in range(N):
            pos = torch.tensor([M + j], dtype=torch.int32, device="cuda")
            q, k = sp.rotary(dev(1, H, d), dev(1, H_kv, d), pos, plan)
            step = sp.Batch(i64(0, 1), i64(M + j + 1), table, rows=1)
            sp.cache_write(caches[layer], step, k, dev(1, H_kv, d), check=True)
            sp.attend(q, caches[layer], step, lse=lse[layer, :, j:j + 1], check=True)
            Q_la[j, layer] = q[0]
        sp.cache_read(caches[layer], sp.Batch(i64(0, M), i64(M), table, rows=M), out_k=K_prompt[layer], check=True)
        sp.cache_read(caches[layer], sp.Batch(i64(0, N), i64(M + N), table, rows=N), out_k=K_la[layer], check=True)
    ref_lse = oracle.row_lse(f64(Q_la), f64(K_prompt), f64(K_la))
    assert np.all(np.abs(f64(lse) - np.asarray(ref_lse).reshape(L, H, N)) <= 1e-4)
    imp = sp.score_lse(Q_la, K_prompt, lse, check=True)
    full = sp.score(Q_la, K_prompt, K_la, check=True)
    ref = oracle.importance(f64(Q_la), f64(K_prompt), f64(K_la))
    for got in (imp, full):         # the scoring's own tolerance
        assert np.all(np.abs(f64(got) - ref) <= np.minimum(1e-3, 1e-2 * np.abs(ref) + 1e-9))
    kept, n_kept = sp.select(imp, 32, 3, "topk", 0.3, trim=False)
    tokens, positions, cu_kept = sp.gather_kept(torch.arange(M, dtype=torch.int32, device="cuda"), [0, M], kept, n_kept)
    # the target: the kept tokens' rows, packed, with capacity for the whole prompt
    q0, k0, v0 = dev(M, H, d), dev(M, H_kv, d), dev(M, H_kv, d)
    batch = sp.Batch(cu_kept, n_kept, table, rows=M)
    q, k = sp.rotary(q0, k0, positions, plan)
    target = sp.cache_alloc(pages, H_kv, page, d, kind=kind)
    sp.cache_write(target, batch, k, v0, check=True)
    out, _ = sp.attend(q, target, batch, check=True)
    n = int(n_kept.item())
    assert 0 < n < M
    pos = positions[:n].cpu().numpy()[None]
    qr = f64(torch.from_numpy(oracle.paged.rotary(f64(q0[:n]), pos, freq, axis)).to(torch.bfloat16))
    assert np.all(np.abs(f64(q[:n]) - qr) <= 2.0 ** -7 * np.abs(qr) + 1e-6)     # a rounding may fall the other way
    kk, vv = (f64(t).transpose(1, 0, 2) for t in (k[:n], v0[:n]))
    if kind != "same":
        kk, vv = (c * s[..., None] for c, s in (oracle.paged.quantise(t, kind) for t in (kk, vv)))
    ref, ref_l, top, spread = oracle.paged.attend(f64(q[:n]), kk, vv, d ** -0.5)
    bound, _ = attend_bounds("bf16", d, n, ref, spread, top, ref_l)
    assert np.all(np.abs(f64(out[:n]) - ref) <= bound)


@pytest.mark.parametrize("T,H", [(1, 4), (1, 32), (5, 1)])
def test_the_stride_of_one_row_or_head_is_not_looked_at(sp, T, H):
    """Every operator on tensors whose stride is odd along an axis with one entry, against the same rows contiguous."""
    import torch
    d, page = 64, 16
    stride = (3, d, 1) if T == 1 else (d, 3, 1)
    odd = lambda like: torch.zeros(like.numel(), dtype=like.dtype, device="cuda").as_strided(like.shape, stride)  # noqa: E731
    g = torch.Generator(device="cuda").manual_seed(5)
    q, v = (torch.randn(T, H, d, dtype=torch.bfloat16, device="cuda", generator=g) for _ in range(2))
    q2, v2 = odd(q), odd(v)
    q2.copy_(q)
    v2.copy_(v)
    plan, pos = sp.rotary_plan(d), torch.arange(7, 7 + T, dtype=torch.int32, device="cuda")
    want, _ = sp.rotary(q, None, pos, plan)
    got, _ = sp.rotary(q2, None, pos, plan, q_out=odd(q))
    assert torch.equal(got, want)
    H_kv = 1 if H == 32 else H
    cu, kv = (torch.tensor(x, dtype=torch.int64, device="cuda") for x in ([0, T], [T]))
    table = torch.tensor([[1]], dtype=torch.int32, device="cuda")
    batch = sp.Batch(cu, kv, table, rows=T)
    outs = []
    for a, b in ((q, v), (q2, v2)):
        cache = sp.cache_alloc(2, H_kv, page, d)
        sp.cache_write(cache, batch, a[:, :H_kv], b[:, :H_kv], check=True)
        outs.append(sp.attend(a, cache, batch, out=None if a is q else odd(q), check=True))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


@pytest.mark.parametrize("stride", [(0, 0, 0), (3, 5, 7)])
def test_the_strides_of_an_empty_tensor_are_not_looked_at(sp, stride):
    import torch
    H, d = 4, 64
    none = torch.empty(0, dtype=torch.bfloat16, device="cuda").as_strided((0, H, d), stride)
    cache = sp.cache_alloc(2, H, 16, d)
    batch = sp.Batch(torch.zeros(2, dtype=torch.int64, device="cuda"), torch.tensor([5], device="cuda"),
                     torch.zeros(1, 1, dtype=torch.int32, device="cuda"), rows=0)
    sp.cache_write(cache, batch, none, none, check=True)
    sp.cache_read(cache, batch, out_k=none.transpose(0, 1), check=True)
    out, lse = sp.attend(none, cache, batch, check=True)
    assert out.shape == (0, H, d) and lse.shape == (H, 0)
    q, k = sp.rotary(none, none, torch.empty(0, dtype=torch.int32, device="cuda"), sp.rotary_plan(d), q_out=none)
    assert q.shape == k.shape == (0, H, d)


def test_more_pairs_of_sequence_and_head_than_a_grid_has_blocks(sp):
    """65535 sequences of 40000 KV heads, two of which have a new token each."""
    import torch
    B, H, d = 65535, 40000, 64
    assert B * H > 2 ** 31
    rng = np.random.default_rng(31)
    cache = sp.cache_alloc(2, H, 2, d)
    x = [torch.from_numpy(rng.standard_normal((3, H, d))).to(torch.bfloat16) for _ in range(2)]
    i64 = lambda a: torch.tensor(a, dtype=torch.int64, device="cuda")                          # noqa: E731
    table = torch.zeros(B, 1, dtype=torch.int32, device="cuda")
    table[B - 1] = 1
    fill = sp.Batch(i64([0, 1, 3]), i64([1, 2]), table[[0, B - 1]], rows=3)
    sp.cache_write(cache, fill, x[0].cuda(), x[1].cuda(), check=True)
    new, kv = np.zeros(B, np.int64), np.zeros(B, np.int64)
    new[[0, -1]], kv[[0, -1]] = 1, [1, 2]
    batch = sp.Batch(i64(np.concatenate([[0], np.cumsum(new)])), i64(kv), table, rows=2, max_new=1)
    q = torch.from_numpy(rng.standard_normal((2, H, d))).to(torch.bfloat16)
    out, lse = sp.attend(q.cuda(), cache, batch, check=True)
    # the first token sees itself alone, the last one two keys: every head by itself, so the heads are the oracle's rows
    k, v = f64(x[0]), f64(x[1])
    assert np.array_equal(f64(out[0]), v[0])
    logits = np.einsum("hd,khd->hk", f64(q[1]), k[1:]) / 8
    top = np.einsum("hd,khd->hk", np.abs(f64(q[1])), np.abs(k[1:])).max(1) / 8
    m = logits.max(1)
    w = np.exp(logits - m[:, None])
    z = w.sum(1)
    w /= z[:, None]
    ref, spread = np.einsum("hk,khd->hd", w, v[1:]), np.einsum("hk,khd->hd", w, np.abs(v[1:]))
    ref_lse = m + np.log(z)
    bound, lse_bound = attend_bounds("bf16", d, 2, ref, spread, top, ref_lse)
    assert np.all(np.abs(f64(out[1]) - ref) <= bound) and np.all(np.abs(f64(lse[:, 1]) - ref_lse) <= lse_bound)


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("factor", ["any", "some", 1 + (2 ** 16 - 1) * 2.0 ** -23, 1.5, -1.25])
@pytest.mark.parametrize("d,dtype", [(64, "bf16"), (128, "bf16"), (40, "bf16"), (64, "f32")])
def test_scales_of_another_cache_that_are_no_powers_of_two(sp, kind, factor, d, dtype):
    """A cache that another program has filled, with scales of largest magnitude / 127 for instance."""
    import torch
    rng = np.random.default_rng(32)
    td = torch_dtype(dtype)
    H, H_kv, page = 4, 2, 16
    new, kv = [1, 150, 6], [300, 400, 6]
    cache, table, _, _ = make_cache(sp, rng, H_kv=H_kv, d=d, page=page, kv=kv, dtype=td, kind=kind)
    rows = []
    for codes, scale in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        times = 1 + rng.integers(0, 1 << 23, tuple(scale.shape)) * 2.0 ** -23 if factor in ("any", "some") else factor
        if factor == "some":        # one slot of the long sequences
            rest = times != 1
            rest[table[0, 7], :, 3] = rest[table[1, 9], 0, 15] = False
            times[rest] = 1
        scale.copy_(torch.from_numpy(scale.double().cpu().numpy() * times))
        rows.append(f64(codes.float()) * f64(scale)[..., None])
    sequence = lambda x, b: np.stack([x[table[b, i // page], :, i % page] for i in range(kv[b])], 1)       # noqa: E731
    whole, cu = make_batch(sp, kv, kv, table)
    read = sp.cache_read(cache, whole, check=True)
    batch, at = make_batch(sp, new, kv, table, max_new=max(new))
    q = torch.from_numpy(rng.standard_normal((sum(new), H, d))).to(td)
    out, lse = sp.attend(q.cuda(), cache, batch, check=True)
    for b in range(len(kv)):
        held = [sequence(x, b) for x in rows]
        got = [f64(x[:, cu[b]:cu[b + 1]]) for x in read]
        for x, y in zip(held, got):
            # rounded once to the type; as a product in fp32 first, whose own half step moves a rounding by 2^-24 at most
            assert np.all(np.abs(y - x) <= ((2.0 ** -8 if dtype == "bf16" else 0) + 2.0 ** -24) * np.abs(x))
        # chunks attend the rows as they are read back, the other kernels as they are held
        if d in (64, 128) and dtype == "bf16" and new[b] * H // H_kv > 16:
            held = got
        ref, ref_lse, top, spread = oracle.paged.attend(f64(q[at[b]:at[b + 1]]), *held, d ** -0.5)
        bound, lse_bound = attend_bounds(dtype, d, kv[b], ref, spread, top, ref_lse)
        assert np.all(np.abs(f64(out[at[b]:at[b + 1]]) - ref) <= bound)
        assert np.all(np.abs(f64(lse[:, at[b]:at[b + 1]]) - ref_lse) <= lse_bound)


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("d,dtype", [(64, "bf16"), (128, "bf16"), (40, "bf16"), (64, "f32")])
@pytest.mark.parametrize("n", [1, 6, 150])
def test_the_smallest_codes_in_attention(sp, kind, d, dtype, n):
    """Caches that hold nothing but e4m3's subnormal codes, -7 to 7 times 2^-9, or int8's -7 to 7: keys, values, or both."""
    import torch
    rng = np.random.default_rng(33)
    td = torch_dtype(dtype)
    H, H_kv, page, kv = 4, 2, 16, 300
    for small in ("k", "v", "kv"):
        cache, table, kval, vval = make_cache(sp, rng, H_kv=H_kv, d=d, page=page, kv=[kv], dtype=td, kind=kind)
        held = [kval[0], vval[0]]
        for i, (name, codes, scale) in enumerate((("k", cache.k, cache.k_scale), ("v", cache.v, cache.v_scale))):
            if name not in small:
                continue
            c = rng.integers(-7, 8, tuple(codes.shape))
            bits = np.where(c < 0, 128 - c, c) if kind == "e4m3" else c & 255       # sign and magnitude, or two's complement
            codes.view(torch.uint8).copy_(torch.from_numpy(bits.astype(np.uint8)))
            size = 2.0 ** 7 if kind == "e4m3" else 2.0 ** -2        # values up to 7 / 4
            scale.fill_(size)
            x = c * (2.0 ** -9 if kind == "e4m3" else 1.0) * size
            held[i] = np.stack([x[table[0, t // page], :, t % page] for t in range(kv)], 1)
        batch, _ = make_batch(sp, [n], [kv], table)
        q = torch.from_numpy(rng.standard_normal((n, H, d))).to(td)
        out, lse = sp.attend(q.cuda(), cache, batch, check=True)
        ref, ref_lse, top, spread = oracle.paged.attend(f64(q), *held, d ** -0.5)
        bound, lse_bound = attend_bounds(dtype, d, kv, ref, spread, top, ref_lse)
        assert np.all(np.abs(f64(out) - ref) <= bound) and np.all(np.abs(f64(lse) - ref_lse) <= lse_bound), small


@pytest.mark.parametrize("kind", ["same", "e4m3", "int8"])
@pytest.mark.parametrize("d,dtype", [(64, "bf16"), (128, "bf16"), (40, "bf16"), (64, "f32")])
@pytest.mark.parametrize("new", [[1, 140, 2], [140, 1, 150], [1, 2, 1], [150, 130, 140]])
@pytest.mark.parametrize("bad", [0, 1, 2])
def test_a_bad_page_of_any_sequence_harms_no_other(sp, kind, d, dtype, new, bad):
    """Steps and chunks in one batch, over every kind of cache; the sequence with the bad page among them."""
    import torch
    rng = np.random.default_rng(34)
    td = torch_dtype(dtype)
    H, H_kv, page = 4, 2, 16
    kv = [n + 60 for n in new]
    cache, table, kval, vval = make_cache(sp, rng, H_kv=H_kv, d=d, page=page, kv=kv, dtype=td, kind=kind, junk=float("nan"))
    T = sum(new)
    q = torch.from_numpy(rng.standard_normal((T, H, d))).to(td).cuda()
    x = torch.from_numpy(rng.standard_normal((T, H_kv, d))).to(td).cuda()
    wrong = table.copy()
    wrong[bad, 1] = 0                           # (make_batch takes negative entries for unused ones)
    batch, cu = make_batch(sp, new, kv, wrong, max_new=max(new))
    batch.table[bad, 1] = (cache.pages, -1, 0x7fffffff)[bad]
    out = torch.full((T, H, d), 7.0, dtype=td, device="cuda")
    lse = torch.full((H, T), 7.0, device="cuda")
    ws = torch.empty(sp.attend_workspace_size(q, cache, batch), dtype=torch.uint8, device="cuda")
    sp.attend(q, cache, batch, out=out, lse=lse, ws=ws)
    assert sp.sp_workspace_status(ws) == sp.SP_EDEVICE
    for b in range(3):
        rows = slice(int(cu[b]), int(cu[b + 1]))
        k, v = kval[b].copy(), vval[b].copy()
        sides = [(k, v)]
        if b == bad:                            # its page's tokens count as zeros, or not at all
            k[:, page:2 * page] = v[:, page:2 * page] = 0
            there = np.arange(kv[b]) // page != 1
            sides.append((k[:, there], v[:, there]))
        fits = []
        for k, v in sides:
            ref, ref_lse, top, spread = oracle.paged.attend(f64(q[rows]), k, v, d ** -0.5)
            bound, lse_bound = attend_bounds(dtype, d, kv[b], ref, spread, top, ref_lse)
            fits.append(np.all(np.abs(f64(out[rows]) - ref) <= bound) and np.all(np.abs(f64(lse[:, rows]) - ref_lse) <= lse_bound))
        assert any(fits), b
    # the bad page among the tokens that are written and read back
    last = (kv[bad] - 1) // page
    wrong = table.copy()
    wrong[bad, last] = 0x7ffffff0
    batch, cu = make_batch(sp, new, kv, wrong, max_new=max(new))
    sides = [(cache.k, cache.k_scale), (cache.v, cache.v_scale)]
    raw = lambda t: t.contiguous().view(torch.uint8 if kind != "same" else t.dtype).cpu().clone()         # noqa: E731
    old = [(raw(t), None if s is None else s.cpu().clone()) for t, s in sides]
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    sp.cache_write(cache, batch, x, -x, ws=ws)
    assert sp.sp_workspace_status(ws) == sp.SP_EDEVICE
    touched = torch.zeros(cache.k.shape[:3], dtype=torch.bool)
    places = oracle.paged.places(cu, kv)
    for b, i in places:
        if wrong[b, i // page] < cache.pages:
            touched[wrong[b, i // page], :, i % page] = True
    for (t, s), (was, was_scale) in zip(sides, old):
        assert np.array_equal(f64(raw(t)[~touched]), f64(was[~touched]), equal_nan=True)
        if s is not None:
            assert np.array_equal(f64(s.cpu()[~touched]), f64(was_scale[~touched]), equal_nan=True)
    k, v = sp.cache_read(cache, batch, ws=ws)
    assert sp.sp_workspace_status(ws) == sp.SP_EDEVICE
    for r, (b, i) in enumerate(places):
        row = f64(x[r])
        if wrong[b, i // page] >= cache.pages:
            row = row * 0
        elif kind != "same":
            codes, scale = oracle.paged.quantise(row, kind)
            row = f64(torch.from_numpy(codes * scale[:, None]).to(td))
        assert np.array_equal(f64(k[:, r]), row) and np.array_equal(f64(v[:, r]), -row)


@pytest.mark.parametrize("kind", ["same", "e4m3", "int8"])
@pytest.mark.parametrize("d,dtype", [(64, "bf16"), (128, "bf16"), (40, "bf16"), (64, "f32")])
@pytest.mark.parametrize("n,kv,at", [(1, 300, 5), (6, 300, 297), (150, 700, 620), (150, 5000, 4990), (40, 3000, 100)])
def test_a_key_that_is_nan_reaches_the_rows_that_see_it(sp, kind, d, dtype, n, kv, at):
    """And no others: neither the tokens before it nor another sequence."""
    import torch
    rng = np.random.default_rng(35)
    td = torch_dtype(dtype)
    H, H_kv, page = 4, 2, 16
    new, lens = [n, 2], [kv, 90]
    cache, table, kval, vval = make_cache(sp, rng, H_kv=H_kv, d=d, page=page, kv=lens, dtype=td, kind=kind)
    one, _ = make_batch(sp, [1], [at + 1], table[:1])
    x = torch.from_numpy(rng.standard_normal((1, H_kv, d))).to(td)
    x[:, :, d // 3] = float("nan")
    v = torch.from_numpy(vval[0][:, at][None]).to(td)           # what is there already
    sp.cache_write(cache, one, x.cuda(), v.cuda(), check=True)
    batch, cu = make_batch(sp, new, lens, table, max_new=max(new))
    q = torch.from_numpy(rng.standard_normal((n + 2, H, d))).to(td)
    out, lse = (f64(t) for t in sp.attend(q.cuda(), cache, batch, check=True))
    sees = np.arange(kv - n, kv) >= at
    assert np.all(np.isnan(out[:n][sees])) and np.all(np.isnan(lse[:, :n][:, sees]))
    for b, rows in ((0, np.flatnonzero(~sees)), (1, np.arange(n, n + 2))):
        if len(rows) == 0:
            continue
        # the rows before the NaN are the last ones of a sequence that ends there
        end = lens[1] if b else at
        ref, ref_lse, top, spread = oracle.paged.attend(f64(q[rows]), kval[b][:, :end], vval[b][:, :end], d ** -0.5)
        bound, lse_bound = attend_bounds(dtype, d, end, ref, spread, top, ref_lse)
        assert np.all(np.abs(out[rows] - ref) <= bound) and np.all(np.abs(lse[:, rows] - ref_lse) <= lse_bound)


def test_scoring_steps_and_chunks_on_streams_of_their_own(sp):
    """A mixed batch, a decode step, a single-precision call and a scoring call, each again and again beside the others."""
    import torch
    rng = np.random.default_rng(36)
    dev = lambda *s, t=torch.bfloat16: torch.from_numpy(rng.standard_normal(s)).to(t).cuda()            # noqa: E731
    calls = []
    for new, kv, dtype, kind in (([1, 200, 3], [3000, 2500, 700], "bf16", "e4m3"), ([1] * 5, [9000, 20, 4000, 1, 600], "bf16", "same"),
                                 ([2, 30], [900, 1000], "f32", "int8")):
        cache, table, _, _ = make_cache(sp, rng, H_kv=2, d=64, page=16, kv=kv, dtype=torch_dtype(dtype), kind=kind)
        batch, _ = make_batch(sp, new, kv, table, max_new=max(new))
        q = dev(sum(new), 8, 64, t=torch_dtype(dtype))
        calls.append(lambda s=None, q=q, c=cache, b=batch: sp.attend(q, c, b, stream=s))
    Q, K, K_la = dev(8, 2, 32, 128), dev(2, 8, 8192, 128), dev(2, 8, 8, 128)
    ws = torch.empty(sp.sp_score_workspace_size(2, 32, 8, 128, 8192, 8, sp.SP_BF16), dtype=torch.uint8, device="cuda")
    calls.append(lambda s=None: (sp.score(Q, K, K_la, ws=ws, stream=s),))
    want = [call() for call in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = [[call(s) for call, s in zip(calls, streams)] for _ in range(20)]
    torch.cuda.synchronize()
    for one in got:
        for mine, right in zip(one, want):
            assert all(torch.equal(a, b) for a, b in zip(mine, right))
