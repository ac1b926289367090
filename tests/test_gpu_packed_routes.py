"""Ragged steps on each of their kernels, told apart by their launches: small steps in narrow
tables work on whole pairs (one launch), or cut them and join (two); more sequences than a warp
plans have a plan kernel in front (three)."""
import numpy as np
import pytest
import torch

import paged_kv_cache_267_gb300 as pa
from test_gpu_packed import DIMS, Step, U, flagged, values

pytestmark = pytest.mark.gpu

WHOLE, CUT, PLANNED = 1, 2, 3
# How the plan kernel deals a step out: whole pairs, or cut ones.
ROUTES = ["cut", "planned whole", "planned cut"]


def launches(st, window=0, **over):
    """(out, launches) of a step."""
    n = pa.launch_count()
    out = st.run(window, **over)
    return out, pa.launch_count() - n


@pytest.mark.parametrize("R,n,ctx,route", [(4, 1, 1000, WHOLE), (19, 16, 1000, WHOLE), (32, 16, 1000, WHOLE), (16, 48, 1000, WHOLE),
                                           (28, 48, 1000, WHOLE), (20, 48, 1000, CUT), (24, 48, 1000, CUT), (20, 48, 600, CUT),
                                           (4, 48, 1000, CUT), (4, 1, 1800, CUT), (33, 1, 100, PLANNED)])
def test_rounds_of_whole_pairs(R, n, ctx, route):
    """Whole pairs are taken where their last round is full enough to be worth it."""
    if torch.cuda.get_device_properties(0).multi_processor_count != 152:
        pytest.skip("rounds of 152 CTAs")
    st = Step([n] * R, [ctx] * R, Hq=32, Hkv=8, seed=R)
    out, got = launches(st)
    assert got == route
    st.check(got=out)


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("D,fp8", [(64, False), (128, False), (128, True), (256, False)])
def test_padded_steps_repeat_their_bits(D, fp8, tree):
    """Other paddings of the rows, the batch and the tables may cut a step elsewhere: each gives the
    same bits every time, and all of them values within the tolerance."""
    new, ctx = [40, 3, 17], [600, 900, 0] if D < 256 else [300, 200, 0]
    ways = set()
    for pad, wide, empty in ((0, 0, 0), (64, 0, 0), (5000, 0, 0), (0, 40, 0), (64, 200, 0), (0, 0, 20), (0, 0, 31), (300, 90, 40)):
        st = Step(new + [0] * empty, ctx + [0] * empty, D=D, fp8=fp8, seed=50, tree=tree, pad=pad, wide=wide)
        out, route = launches(st)
        ways.add(route)
        st.check(got=out)
        n = sum(new)
        for _ in range(2):
            assert torch.equal(st.run()[:n], out[:n])
    assert ways == {WHOLE, CUT, PLANNED}


def plan_is_whole(st, window=0):
    """What the plan kernel chooses for a step."""
    D, Hkv, ctas = st.q.shape[2], st.Hkv, torch.cuda.get_device_properties(0).multi_processor_count
    tpg, kv = 128 // (st.q.shape[1] // Hkv), 64 if D == 256 else 128
    tpu = tpg if D == 256 else 2 * tpg
    costs = []
    for n, L in zip(st.new, st.lens):
        L = max(L, 0)
        for t in range(0, n, tpu):
            m, first = min(n - t, tpu), L - n
            hi = first + (min(n, 64) if st.mask is not None else t + m) - 1
            start = first if st.mask is not None else first + t + 1
            lo = start - window if 0 < window < start else 0
            nt = -(-(hi + 1 - lo // 16 * 16) // kv) if hi >= lo else 0
            costs.append(8 + max(nt, 1) * (4 if m > tpg else 3))
    longest, mean = max(costs), -(-sum(costs) * Hkv // ctas)
    bins = [0] * 256
    for c in costs:
        bins[min(int(np.float32(longest - c) * (np.float32(256) / np.float32(longest))), 255)] += 1
    most = upto = 0
    for i, k in enumerate(bins):
        r0, upto = upto * Hkv, upto + k
        turn = (upto * Hkv - 1) // ctas
        if k and turn * ctas >= r0:
            most = max(most, (turn + 1) * (longest - int(i * (np.float32(longest) / np.float32(256)))))
    return max(mean, most) <= mean + 16


def on(route, new, ctx, lens=None, Hkv=2, D=128, **kw):
    """A step of these sequences that takes the route: wide tables, or other sequences behind them."""
    extra = ([], [])
    if route == "planned whole":
        extra = ([8] * (100 // Hkv) + [0] * 33, [1000 if D < 256 else 500] * (100 // Hkv) + [0] * 33)
    elif route == "planned cut":
        extra = ([1, 0, 2] * 11 + [5], [3, 0, 20] * 11 + [6000])
    if lens is not None:
        lens = lens + [n + c for n, c in zip(*extra)]
    st = Step(new + extra[0], ctx + extra[1], lens=lens, Hkv=Hkv, D=D, wide=88 if route == "cut" else 0, **kw)
    st.route = route
    return st


def checked(st, window=0, whole=None):
    """Runs and checks a step, and that it took its route."""
    out, got = launches(st, window)
    assert got == (CUT if st.route == "cut" else PLANNED)
    if got == PLANNED and whole is not False:
        assert plan_is_whole(st, window) == (st.route == "planned whole")
    return st.check(window, got=out)


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("D,fp8", DIMS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_prompts_and_trees(D, fp8, dtype, route):
    checked(on(route, [1, 7, 64, 65, 130, 0, 33], [0] * 7, D=D, fp8=fp8, dtype=dtype, seed=60))
    checked(on(route, [3, 50, 90], [70, 0, 200], D=D, fp8=fp8, dtype=dtype, seed=61))
    checked(on(route, [1, 7, 64, 33, 0, 5], [0, 100, 300, 40, 9, 290], D=D, fp8=fp8, dtype=dtype, seed=62, tree=True))


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("D,fp8", DIMS)
@pytest.mark.parametrize("Hq,Hkv", [(8, 8), (6, 2), (16, 1), (10, 2), (24, 8)])
def test_heads(D, fp8, Hq, Hkv, route):
    checked(on(route, [3, 50, 60], [70, 0, 100], Hq=Hq, Hkv=Hkv, D=D, fp8=fp8, seed=63))
    checked(on(route, [3, 50, 60], [70, 0, 100], Hq=Hq, Hkv=Hkv, D=D, fp8=fp8, seed=64, tree=True))


@pytest.mark.parametrize("D,fp8", DIMS)
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("route,window", [("cut", 1000), ("cut", 2000), ("planned cut", 1000), ("planned whole", 300),
                                          ("planned", 1), ("planned", 16), ("planned", 64), ("planned", 100)])
def test_windows(D, fp8, tree, route, window):
    """(Steps of short windows have few tiles: small ones are whole, of many sequences whole, too.)"""
    if tree and window < 64:
        pytest.skip("a window of trees is at least 64")
    ctx = [0, 2500, 777] if route != "planned whole" else [0, 400, 290]
    st = on("planned cut" if route == "planned" else route, [40, 60, 1], ctx, D=D, fp8=fp8, seed=65, tree=tree)
    checked(st, window, whole=False if route == "planned" else None)


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("D,fp8", DIMS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_values_that_are_not_attended(D, fp8, dtype, route):
    """Infinities and NaN in later tokens, before a window and in other branches; rows that attend
    to them have them, in whichever of the parts of a cut unit they are."""
    odd = [0x7F] if fp8 else [float("inf"), float("-inf"), float("nan")]
    st = on(route, [100, 40, 1], [30, 200, 128], D=D, fp8=fp8, dtype=dtype, seed=66)
    for i, x in enumerate(odd):
        st.poke(0, 60 + 3 * i, v=x, d=slice(5, 9))
        st.poke(1, 225 + i, v=x, head=1)
    st.poke(0, 129, v=odd[0], k=odd[-1])
    st.poke(2, 128, k=odd[-1])
    checked(st)
    W = 1000 if route == "cut" else 300
    st = on(route, [64, 9], [W + 100, 0], D=D, fp8=fp8, dtype=dtype, seed=67)
    for i, x in enumerate(odd):
        st.poke(0, 130 + i, v=x, k=x)                    # leaves the window on the way
        st.poke(0, W + 120 + i, v=x, d=slice(0, 1))
        st.poke(0, W + 50 + i, v=x, d=slice(7 + i, 8 + i))  # seen by all rows
    checked(st, W, whole=False)  # (the window leaves few tiles)
    st = on(route, [64, 20, 3], [100, 1, 260], D=D, fp8=fp8, dtype=dtype, seed=68, tree=True)
    for i, x in enumerate(odd):
        st.poke(0, 100 + 11 * i, v=x, d=slice(2, 3))
        st.poke(1, 1 + 5 * i, v=x, head=0)
        st.poke(2, 17 + i, v=x, d=slice(0, 2))
    checked(st)


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("D,fp8", DIMS)
def test_rows_that_attend_to_nothing(D, fp8, route):
    st = on(route, [10, 5, 40], [0, 0, 0], D=D, fp8=fp8, seed=69, lens=[4, 0, 40])
    out, got = launches(st)
    assert got == (CUT if route == "cut" else PLANNED)
    assert not out[:6].any() and not out[10:15].any() and out[6:10].any()
    ref, A = st.expect()
    tol = (2.0 ** -8 + 2.0 ** -14) * A + 2.0 ** -8 * ref.abs() + 2.0 ** -24
    assert ((out[15:].double() - ref[15:]).abs() <= tol[15:]).all()
    st = on(route, [4, 4, 64], [0, 50, 0], D=D, fp8=fp8, seed=70, tree=True)
    st.mask[1] = 0
    st.mask[5] = 0
    st.mask[3] = -1
    st.mask[6] = (1 << 40) | 1
    st.mask[20] = 0
    out = checked(st)
    assert not out[1].any() and not out[20].any() and out[5].any()
    # units without tiles beside long ones
    st = on(route, [6, 1, 90], [0, 900, 0], D=D, fp8=fp8, seed=71, lens=[0, 901, 3])
    out = launches(st)[0]
    assert not out[:6].any() and not out[7:94].any() and out[6].any() and out[94:97].any()


@pytest.mark.parametrize("tree", [False, True])
def test_bad_starts_lengths_and_blocks_where_pairs_are_cut(tree):
    B = 3
    st = Step([5] * B, [60] * B, seed=72, tree=tree, wide=88)
    good, got = launches(st)
    assert got == CUT
    s = list(st.starts)
    s[2], s[1] = s[1], s[2]                              # decreases: raised to the one before
    out, bits = flagged(st, starts=st.ints(s))
    assert bits == pa.DEVERR_QUERY
    s = st.starts[:-1] + [5 * B + 9]                     # leaves [0, T]: clamped
    out, bits = flagged(st, starts=st.ints(s))
    assert bits == pa.DEVERR_QUERY and torch.equal(out, good)
    out, bits = flagged(st, starts=st.ints([-7] + st.starts[1:]))
    assert bits == pa.DEVERR_QUERY and torch.equal(out, good)
    assert flagged(st, starts=st.ints([2 ** 31 - 1] * (B + 1)))[1] == pa.DEVERR_QUERY
    assert flagged(st, starts=st.ints([-2 ** 31] * (B + 1)))[1] == pa.DEVERR_QUERY
    n = list(st.lens)
    n[1] = 2 ** 31 - 1                                   # clamped to the table, whose end has no blocks
    assert flagged(st, lens=st.ints(n))[1] == pa.DEVERR_SEQ_LEN | pa.DEVERR_BLOCK_ID
    n[1] = -5
    out, bits = flagged(st, lens=st.ints(n))
    assert bits == pa.DEVERR_SEQ_LEN and not out[5:10].any() and torch.equal(out[:5], good[:5]) and torch.equal(out[10:], good[10:])
    t = st.tables.clone()
    t[0, 1], t[1, 0] = 1 << 30, -9
    out, bits = flagged(st, tables=t)
    assert bits == pa.DEVERR_BLOCK_ID and torch.equal(out[10:], good[10:])


@pytest.mark.parametrize("route", ["cut", "planned cut"])
@pytest.mark.parametrize("D,fp8", DIMS)
def test_scales_and_large_scores(D, fp8, route):
    for scale, spread in ((-D ** -0.5, 1.0), (0.0, 1.0), (D ** -0.5, 8.0), (1e-30, 1.0)):
        checked(on(route, [40, 3], [700, 150], D=D, fp8=fp8, scale=scale, spread=spread, seed=73))
    checked(on(route, [20, 3], [700, 150], D=D, fp8=fp8, scale=-0.02, spread=3.0, seed=74, tree=True))


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D", [128, 256])
def test_query_ranges_on_an_e4m3_cache(D, dtype, route):
    """Rows whose largest magnitudes go from 2 to 2^26 (f16 has infinities there), values down to 2^-24
    of them, zeros, subnormals, NaN. Next to a row's largest magnitude m an element may be off by
    2^-17 m, and so a score by 2^-17 m sum |k| scale, a weight by twice that of its own value."""
    st = on(route, [70, 9, 33], [40, 300, 0], D=D, fp8=True, dtype=dtype, seed=75)
    g = torch.Generator(device="cuda").manual_seed(76)
    T, Hq = st.q.shape[:2]
    small = torch.exp2(-24 * torch.rand(T, Hq, D, generator=g, device="cuda"))
    sign = torch.where(torch.rand(T, Hq, D, generator=g, device="cuda") < 0.5, -1.0, 1.0)
    row = torch.exp2(-torch.arange(T, device="cuda").float() % 26 - 25)[:, None, None]
    st.q = (sign * small * 2.0 ** 26 * row).to(dtype)
    st.q[3] = 0
    st.q[5] = torch.finfo(dtype).smallest_normal / 4
    st.q[7, 0, 5] = float("inf")
    st.q[8, 1, 6] = float("nan")
    st.q[9, 2, 7] = float("-inf")
    out, got = launches(st)
    assert got == (CUT if route == "cut" else PLANNED)
    out, (ref, A) = out.double(), st.expect()
    bad = ~st.q.isfinite().all(-1)
    assert bad.sum() >= 3 and out[bad].isnan().all() and ref[bad].isnan().all()
    ks = max(float(values(k, st.k_scale, True).abs().sum(-1).max()) for k in st.k if k.numel())
    ds = st.scale * ks * 2.0 ** -17 * st.q.double().abs().amax(-1, keepdim=True)
    tol = (2.0 ** -11 + 2.0 ** -14 + 2 * ds) * A + U[dtype] * ref.abs() + 2.0 ** -24
    err = ((out - ref).abs() / tol)[~bad]
    assert err.max() <= 1, err.max()
