"""Rotary positions, the paged cache and the attention over it: what is refused, and what the host works out (no GPU)."""
import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest

import oracle


@pytest.fixture(scope="module")
def sp():
    from speculative_prefill_token_sp_gb300 import build
    build.build()
    import speculative_prefill_token_sp_gb300 as m
    m.lib()
    return m


def cache_of(sp, **over):
    a = dict(k=4096, v=8192, k_scale=None, v_scale=None, stride_page=2 * 16 * 64, stride_head=16 * 64, stride_slot=64,
             pages=10, page=16, H_kv=2, d=64, dtype=sp.SP_BF16, kind=sp.SP_CACHE_SAME)
    a.update(over)
    return sp.SpCache(*[a[n] for n, _ in sp.SpCache._fields_])


def batch_of(sp, **over):
    a = dict(B=2, max_new=5, T=10, cu_new=64, kv_len=128, table=256, table_width=4, table_stride=4)
    a.update(over)
    return sp.SpBatch(*[a[n] for n, _ in sp.SpBatch._fields_])


def rows_of(sp, **over):
    a = dict(data=4096, stride_row=256, stride_head=64)
    a.update(over)
    return sp.SpRows(*[a[n] for n, _ in sp.SpRows._fields_])


BAD_CACHES = [
    (dict(k=None), "SP_EINVAL"), (dict(v=None), "SP_EINVAL"), (dict(d=12), "SP_EUNSUPPORTED"), (dict(d=264), "SP_EUNSUPPORTED"),
    (dict(d=0), "SP_EINVAL"), (dict(dtype=3), "SP_EINVAL"), (dict(kind=5), "SP_EINVAL"), (dict(kind=1), "SP_EINVAL"),
    (dict(kind=2, k_scale=64), "SP_EINVAL"), (dict(page=0), "SP_EINVAL"), (dict(pages=0), "SP_EINVAL"), (dict(H_kv=0), "SP_EINVAL"),
    (dict(k=4104), "SP_EINVAL"), (dict(stride_slot=68), "SP_EINVAL"), (dict(stride_slot=32), "SP_EINVAL"),
    (dict(stride_page=-2048), "SP_EINVAL"), (dict(H_kv=65536), "SP_EUNSUPPORTED"), (dict(stride_head=1028), "SP_EINVAL"), (dict(pages=1 << 31), "SP_EINVAL"),
]
BAD_BATCHES = [dict(B=0), dict(T=-1), dict(T=1 << 31), dict(max_new=-1), dict(table_width=0), dict(cu_new=None), dict(kv_len=None),
               dict(table=None), dict(cu_new=68), dict(table=258), dict(table_stride=-4)]
BAD_ROWS = [None, dict(data=None), dict(data=4104), dict(stride_row=257), dict(stride_head=60)]


def calls(sp, cache, batch, rows, ws=65536, ws_bytes=1 << 40):
    yield "write", sp.sp_cache_write(cache, batch, rows, rows, ws, ws_bytes, 0)
    yield "read", sp.sp_cache_read(cache, batch, rows, rows, ws, ws_bytes, 0)
    yield "attend", sp.sp_attend(rows, cache, batch, 4, 0.125, 0, rows, None, 0, 0, ws, ws_bytes, 0)


@pytest.mark.parametrize("over,status", BAD_CACHES)
def test_bad_caches_are_refused(sp, over, status):
    for name, s in calls(sp, cache_of(sp, **over), batch_of(sp), rows_of(sp)):
        assert sp.sp_status_string(s) == status, name
        assert sp.sp_last_error()
    assert sp.sp_attend_workspace_size(cache_of(sp, **over), batch_of(sp), 4) == 0


@pytest.mark.parametrize("over", BAD_BATCHES)
def test_bad_batches_are_refused(sp, over):
    for name, s in calls(sp, cache_of(sp), batch_of(sp, **over), rows_of(sp)):
        assert s == sp.SP_EINVAL, name


@pytest.mark.parametrize("over", BAD_ROWS)
def test_bad_rows_are_refused(sp, over):
    bad = None if over is None else rows_of(sp, **over)
    c, b, good = cache_of(sp), batch_of(sp), rows_of(sp)
    big = 1 << 40
    assert sp.sp_cache_write(c, b, bad, good, 65536, big, 0) == sp.SP_EINVAL
    assert sp.sp_cache_write(c, b, good, bad, 65536, big, 0) == sp.SP_EINVAL
    if over is not None:
        assert sp.sp_cache_read(c, b, bad, good, 65536, big, 0) == sp.SP_EINVAL
        assert sp.sp_cache_read(c, b, good, bad, 65536, big, 0) == sp.SP_EINVAL
    assert sp.sp_attend(bad, c, b, 4, 0.125, 0, good, None, 0, 0, 65536, big, 0) == sp.SP_EINVAL
    assert sp.sp_attend(good, c, b, 4, 0.125, 0, bad, None, 0, 0, 65536, big, 0) == sp.SP_EINVAL


def test_overlapping_rows_are_refused(sp):
    c, b, good = cache_of(sp), batch_of(sp), rows_of(sp)
    big = 1 << 40
    for over in (dict(stride_row=0), dict(stride_head=0), dict(stride_head=32), dict(stride_row=-256), dict(stride_row=1 << 39)):
        bad = rows_of(sp, **over)
        assert sp.sp_attend(bad, c, b, 4, 0.125, 0, good, None, 0, 0, 65536, big, 0) == sp.SP_EINVAL
        assert sp.sp_attend(good, c, b, 4, 0.125, 0, bad, None, 0, 0, 65536, big, 0) == sp.SP_EINVAL
        assert sp.sp_cache_read(c, b, bad, None, 65536, big, 0) == sp.SP_EINVAL
        assert sp.sp_cache_read(c, b, None, bad, 65536, big, 0) == sp.SP_EINVAL
    s = sp.sp_cache_write(c, batch_of(sp, B=65536), good, good, 65536, big, 0)
    assert s == sp.SP_EUNSUPPORTED


def test_other_arguments_that_are_refused(sp):
    c, b, r = cache_of(sp), batch_of(sp), rows_of(sp)
    big = 1 << 40
    assert sp.sp_cache_read(c, b, None, None, 65536, big, 0) == sp.SP_EINVAL
    for H in (0, 3, -2):
        assert sp.sp_attend(r, c, b, H, 0.125, 0, r, None, 0, 0, 65536, big, 0) == sp.SP_EINVAL
    for scale in (0.0, -1.0, math.nan, math.inf, 1e300):
        assert sp.sp_attend(r, c, b, 4, scale, 0, r, None, 0, 0, 65536, big, 0) == sp.SP_EINVAL
    assert sp.sp_attend(r, c, b, 4, 0.125, -1, r, None, 0, 0, 65536, big, 0) == sp.SP_EINVAL
    assert sp.sp_attend(r, c, b, 4, 0.125, 0, r, 6, 1, 1, 65536, big, 0) == sp.SP_EINVAL
    for ws, size, status in ((None, big, sp.SP_EINVAL), (65544, big, sp.SP_EINVAL), (65536, 100, sp.SP_ENOMEM)):
        assert all(s == status for _, s in calls(sp, c, b, r, ws, size))
    for null in (dict(cache=None), dict(batch=None)):
        for name, s in calls(sp, null.get("cache", c), null.get("batch", b), r):
            assert s == sp.SP_EINVAL, name


def test_rotary_refusals(sp):
    plan = sp.SpRotaryPlan()
    f = [1.0] * 32
    for rot, freq, axis, axes, status in ((60, f, None, 1, "SP_EUNSUPPORTED"), (0, f, None, 1, "SP_EINVAL"),
                                          (512, [1.0] * 256, None, 1, "SP_EUNSUPPORTED"), (64, None, None, 1, "SP_EINVAL"),
                                          (64, f, [3] * 32, 3, "SP_EINVAL"), (64, f, None, 9, "SP_EINVAL"),
                                          (64, f, None, 0, "SP_EINVAL"), (64, [math.inf] + f[1:], None, 1, "SP_EINVAL"),
                                          (64, [math.nan] + f[1:], None, 1, "SP_EINVAL")):
        assert sp.sp_status_string(sp.sp_rotary_plan_init(plan, rot, freq, axis, axes, 0)) == status
    r = rows_of(sp)
    blank = sp.SpRotaryPlan()
    go = lambda plan=plan, pos=64, T=4, d=64, dtype=0, q=r, qo=r, H=2, k=r, ko=r, H_kv=1: sp.sp_rotary(  # noqa: E731
        plan, pos, 0, T, d, dtype, 0, q, qo, H, k, ko, H_kv, 0)
    assert go(plan=blank) == sp.SP_EINVAL and go(plan=None) == sp.SP_EINVAL
    assert sp.sp_rotary_plan_init(plan, 64, f, None, 1, 0) == sp.SP_OK
    assert go(d=32) == sp.SP_EINVAL and go(d=68) == sp.SP_EUNSUPPORTED and go(dtype=2) == sp.SP_EINVAL
    assert go(T=-1) == sp.SP_EINVAL and go(H=-1) == sp.SP_EINVAL and go(pos=None) == sp.SP_EINVAL and go(pos=66) == sp.SP_EINVAL
    for over in BAD_ROWS:
        bad = None if over is None else rows_of(sp, **over)
        assert go(q=bad) == go(qo=bad) == go(k=bad) == go(ko=bad) == sp.SP_EINVAL


def test_rotary_plan_holds_exact_fractions_of_a_turn(sp):
    plan = sp.rotary_plan(128, base=500000.0, sections=(16, 24, 24))
    assert list(plan.axis)[:64] == [0] * 16 + [1] * 24 + [2] * 24 and plan.axes == 3
    for i in range(64):
        turns = np.longdouble(500000.0 ** (-i / 64)) / (2 * np.arctan2(np.longdouble(0), np.longdouble(-1)))
        # the quotient is taken in double: half a unit of 2^-53 of it, twice over; and the fraction has 64 bits, so
        # it holds a frequency to 2^-64 of a turn
        assert abs(np.longdouble(plan.turns[i]) / np.longdouble(2) ** 64 - turns) <= float(turns) * 2.0 ** -51 + 2.0 ** -64
    back = sp.rotary_plan(16, inv_freq=[-1.0, 0.0, 2 * math.pi, -1e-300, 7.0, 1e6, 0.5, 3.0])
    assert back.turns[1] == 0 and back.turns[3] == 0 and back.turns[0] > 1 << 63


def test_python_checks(sp):
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError):
        sp.rotary_plan(64, sections=(8, 8))
    with pytest.raises(ValueError):
        sp.rotary_plan(64, inv_freq=[1.0])
    with pytest.raises(ValueError):
        sp.rotary_plan(64, sections=(32,), axis_of_pair=[0] * 32)
    k = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        sp.Cache(k, k[:3])
    with pytest.raises(ValueError):
        sp.Cache(k.transpose(2, 3), k.transpose(2, 3))
    with pytest.raises(ValueError):
        sp.Cache(k.to(torch.int8), k.to(torch.int8))
    with pytest.raises(ValueError):
        sp.Cache(k, k, dtype=torch.float32)
    with pytest.raises(TypeError):
        sp.Cache(k.half(), k.half())
    cu, kv, table = torch.tensor([0, 1]), torch.tensor([5]), torch.zeros(1, 4, dtype=torch.int32)
    with pytest.raises(TypeError):
        sp.Batch(cu.int(), kv, table, rows=1)
    with pytest.raises(ValueError):
        sp.Batch(cu, kv, table[0], rows=1)
    cache, batch = sp.Cache(k, k), sp.Batch(cu, kv, table, rows=1)
    with pytest.raises(ValueError):         # not on a GPU
        sp.attend(torch.zeros(1, 4, 64, dtype=torch.bfloat16), cache, batch)
    with pytest.raises(ValueError):
        sp.attend(torch.zeros(2, 4, 64, dtype=torch.bfloat16), cache, batch)
    with pytest.raises(ValueError):
        sp.cache_write(cache, batch, torch.zeros(1, 2, 64), torch.zeros(1, 2, 64))


def test_struct_layouts_match_the_header(sp):
    # natural C layout: the offsets a 64-bit C compiler gives these members
    assert ctypes.sizeof(sp.SpRows) == 24 and ctypes.sizeof(sp.SpBatch) == 56 and ctypes.sizeof(sp.SpCache) == 88
    assert sp.SpRotaryPlan.turns.offset == 16 and sp.SpRotaryPlan.axis.offset == 16 + 1024
    assert ctypes.sizeof(sp.SpRotaryPlan) == 16 + 1024 + 128


def test_oracle_of_the_cache_and_the_attention():
    codes, scale = oracle.paged.quantise(np.array([[448.0, 1.0, 0.0], [449.0, -1.0, 18.0]]), "e4m3")
    assert scale.tolist() == [1.0, 2.0] and codes.tolist() == [[448.0, 1.0, 0.0], [224.0, -0.5, 9.0]]
    codes, scale = oracle.paged.quantise(np.array([[127.0, 2.5, 3.5], [1.0, 0.5, 0.25]]), "int8")
    assert scale.tolist() == [1.0, 2.0 ** -6] and codes.tolist() == [[127.0, 2.0, 4.0], [64.0, 32.0, 16.0]]
    q = np.zeros((2, 1, 8))
    v = np.arange(24.0).reshape(1, 3, 8)
    out, lse, _, _ = oracle.paged.attend(q, np.zeros((1, 3, 8)), v, 1.0)
    assert np.allclose(out[0, 0], v[0, :2].mean(0)) and np.allclose(out[1, 0], v[0].mean(0))
    assert np.allclose(lse, np.log([[2.0, 3.0]]))


def test_many_heads_and_misaligned_scales_are_refused(sp):
    plan, r = sp.SpRotaryPlan(), rows_of(sp)
    assert sp.sp_rotary_plan_init(plan, 64, [1.0] * 32, None, 1, 0) == sp.SP_OK
    for H, H_kv in ((65536, 1), (1, 65536), ((1 << 31) - 1, (1 << 31) - 1)):
        assert sp.sp_rotary(plan, 64, 0, 4, 64, 0, 0, r, r, H, r, r, H_kv, 0) == sp.SP_EUNSUPPORTED
    for over in (dict(k_scale=66, v_scale=64), dict(k_scale=64, v_scale=66)):
        for name, s in calls(sp, cache_of(sp, kind=sp.SP_CACHE_INT8, **over), batch_of(sp), r):
            assert s == sp.SP_EINVAL, name
    with pytest.raises(ValueError):
        sp.cache_alloc(1, 1, 16, 64, kind="int4", device="cpu")


PI = Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")


@pytest.mark.parametrize("freq", [
    [1.0, -1.0, 0.1, -0.1, 1e-5, -1e-5, 3e-9, -3e-9], [6.0, -6.0, 7.0, 100.0, -1000.0, 1e6, 2.0 ** 40, -2.0 ** 40],
    [2 * math.pi, -2 * math.pi, 0.0, -0.0, 1e-300, -1e-300, 5e-324, -5e-324],
])
def test_rotary_plan_is_exact_for_fast_and_negative_frequencies(sp, freq):
    """A position of 2^31 multiplies the error of a fraction: at 2^-62 of a turn the angle is off by 2^-31 of one."""
    plan = sp.rotary_plan(16, inv_freq=freq)
    for i, f in enumerate(freq):
        turns = Fraction(f) / (2 * PI)          # off by 2^-256 of itself
        off = (Fraction(plan.turns[i], 1 << 64) - turns) % 1
        # cut off once and rounded once, to 2^-64 of a turn each; the product with 1 / 2 pi in two doubles is off by 2^-105 of it
        assert min(off, 1 - off) <= Fraction(3, 1 << 65) + abs(turns) / (1 << 105), f


def test_rotary_frequencies_beyond_2_40_are_refused(sp):
    plan = sp.SpRotaryPlan()
    for f in (2.0 ** 40 * (1 + 2.0 ** -52), -1e300):
        assert sp.sp_rotary_plan_init(plan, 16, [1.0] * 7 + [f], None, 1, 0) == sp.SP_EUNSUPPORTED
        assert sp.sp_last_error()


def test_scales_that_single_precision_does_not_hold_are_refused(sp):
    """The kernels take logits to base 2: scale * log2(e) has to be a normal fp32 number."""
    c, b, r = cache_of(sp), batch_of(sp), rows_of(sp)
    for scale in (5e-324, 1e-46, 1e-40, 8.1e-39, 2.4e38, 3e38, 1e39):
        assert sp.sp_attend(r, c, b, 4, scale, 0, r, None, 0, 0, 65536, 1 << 40, 0) == sp.SP_EINVAL, scale
        assert "scale" in sp.sp_last_error()


# 10 rows of 4 (H) or 2 (H_kv) heads of 64; each stride by itself is at least a row
CROSSED = [dict(stride_row=64, stride_head=64), dict(stride_row=128, stride_head=64), dict(stride_row=64, stride_head=576),
           dict(stride_row=120, stride_head=64), dict(stride_row=(1 << 38), stride_head=(1 << 38))]


@pytest.mark.parametrize("over", CROSSED)
def test_rows_of_one_head_that_meet_those_of_another_are_refused(sp, over):
    c, b, good, bad = cache_of(sp), batch_of(sp), rows_of(sp), rows_of(sp, **over)
    big = 1 << 40
    assert sp.sp_attend(good, c, b, 4, 0.125, 0, bad, None, 0, 0, 65536, big, 0) == sp.SP_EINVAL
    assert "overlap" in sp.sp_last_error()
    assert sp.sp_attend(bad, c, b, 4, 0.125, 0, good, None, 0, 0, 65536, big, 0) == sp.SP_EINVAL
    plan = sp.SpRotaryPlan()
    assert sp.sp_rotary_plan_init(plan, 64, [1.0] * 32, None, 1, 0) == sp.SP_OK
    assert sp.sp_rotary(plan, 64, 0, 10, 64, 0, 0, good, bad, 4, None, None, 0, 0) == sp.SP_EINVAL
    assert sp.sp_rotary(plan, 64, 0, 10, 64, 0, 0, None, None, 0, good, bad, 4, 0) == sp.SP_EINVAL
    if over["stride_row"] != 128:       # two heads of 64 do fit there
        assert sp.sp_cache_read(c, b, bad, None, 65536, big, 0) == sp.SP_EINVAL
        assert sp.sp_cache_read(c, b, None, bad, 65536, big, 0) == sp.SP_EINVAL


@pytest.mark.parametrize("over", [dict(stride_row=256, stride_head=64), dict(stride_row=64, stride_head=640),
                                  dict(stride_row=1 << 38, stride_head=64), dict(stride_row=264, stride_head=64)])
def test_rows_apart_are_taken(sp, over):
    """An empty workspace is refused behind the rows: that is how far these calls come."""
    c, b, r = cache_of(sp), batch_of(sp), rows_of(sp, **over)
    assert sp.sp_attend(r, c, b, 4, 0.125, 0, r, None, 0, 0, 65536, 0, 0) == sp.SP_ENOMEM
    assert sp.sp_cache_read(c, b, r, r, 65536, 0, 0) == sp.SP_ENOMEM


def test_a_cache_whose_places_overlap_is_not_written(sp):
    """Two heads, pages or slots in one place: reading such a cache is fine, writing it is refused."""
    b, r = batch_of(sp), rows_of(sp)
    slot, head, page = 64, 16 * 64, 2 * 16 * 64
    for over in (dict(stride_head=0), dict(stride_page=0), dict(stride_page=page - 8), dict(stride_head=head - 8),
                 dict(stride_slot=slot, stride_head=slot), dict(stride_slot=head, stride_head=slot, stride_page=page - 8),
                 dict(stride_page=slot, stride_head=10 * slot, stride_slot=slot),
                 dict(kind=sp.SP_CACHE_INT8, k_scale=64, v_scale=64, stride_head=0)):
        c = cache_of(sp, **over)
        assert sp.sp_cache_write(c, b, r, r, 65536, 1 << 40, 0) == sp.SP_EINVAL, over
        assert "overlap" in sp.sp_last_error()
        assert sp.sp_cache_read(c, b, r, r, 65536, 0, 0) == sp.SP_ENOMEM, over         # an empty workspace
        assert sp.sp_attend(r, c, b, 4, 0.125, 0, r, None, 0, 0, 65536, 0, 0) == sp.SP_ENOMEM, over


def test_caches_of_every_order_are_written(sp):
    """Pages, heads and slots in any order of their strides, with gaps; and a stride along an axis with one entry."""
    b, r = batch_of(sp), rows_of(sp)
    for over in (dict(stride_slot=64, stride_head=1024, stride_page=2048), dict(stride_slot=128, stride_head=64, stride_page=2048),
                 dict(stride_page=64, stride_head=640, stride_slot=1280), dict(stride_slot=136, stride_head=64, stride_page=4096),
                 dict(H_kv=1, stride_head=0, stride_page=1024), dict(pages=1, stride_page=0), dict(page=1, stride_slot=64, stride_head=64)):
        assert sp.sp_cache_write(cache_of(sp, **over), b, r, r, 65536, 0, 0) == sp.SP_ENOMEM, over
