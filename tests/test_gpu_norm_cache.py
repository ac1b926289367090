"""pa_norm_rope_and_cache against the formulas in 64 bits.

Tolerances. A result is rounded once, by at most half a step: eps / 2 of its
value (2^-11 f16, 2^-8 bf16, 2^-4 e4m3), or half the smallest step near zero.
Before that, fp32: the sum of D squares is off by at most (D + 2) 2^-24 of
itself, its root and quotient add three roundings, the products with the weight
and the angles and their sum four more, all relative to |a c| + |b s| <=
|a| + |b|: in all less than (D / 2 + 12) 2^-24 (|a| + |b|).
"""
import numpy as np
import pytest
import torch

from conftest import have_gpu

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a GPU")]

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "e4m3": 2.0 ** -4}
TINY = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25, "e4m3": 2.0 ** -10}


def angles(P, R, base=10000.0):
    i = np.arange(0, R, 2, dtype=np.float64) / max(R, 1)
    a = np.arange(P, dtype=np.float64)[:, None] * base ** -i
    return torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], 1)).float().cuda()


def reference(x, w, cs, pos, R, interleaved, eps):
    """(value, bound on the fp32 error) in 64 bits; x [T, H, D]."""
    x = x.double().cpu()
    D = x.shape[-1]
    if w is not None:
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * w.double().cpu()
    cs = cs.double().cpu()[pos.long().cpu()]
    c, s = cs[:, None, : R // 2], cs[:, None, R // 2:]
    i = torch.arange(R // 2)
    lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
    y, size = x.clone(), x.abs().clone()
    y[..., lo] = x[..., lo] * c - x[..., hi] * s
    y[..., hi] = x[..., hi] * c + x[..., lo] * s
    size[..., lo] = size[..., hi] = x[..., lo].abs() + x[..., hi].abs()
    return y, size * ((D / 2 + 12) * 2.0 ** -24)


def check(got, ref, slack, kind, what):
    err = (got.double().cpu() - ref).abs()
    bound = HALF[kind] * (ref.abs() + slack) + slack + TINY[kind]
    assert torch.isfinite(got.double()).all(), what
    worst = (err - bound).max().item()
    assert worst <= 0, f"{what}: beyond the bound by {worst:.3e} (largest error {err.max():.3e})"


def make(T, Hq, Hkv, D, dt, fp8, bs=16, seed=0, skipped=0.15, spread=1.0, P=5000, R=None,
         extra_cols=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    H = Hq + 2 * Hkv
    packed = (torch.randn(T, H * D + extra_cols, generator=g, device="cuda") * spread).to(DT[dt])
    q, k, v = packed[:, :H * D].unflatten(1, (H, D)).split([Hq, Hkv, Hkv], dim=1)
    NB = -(-T // bs) + 3
    slots = torch.randperm(NB * bs, generator=g, device="cuda")[:T]
    slots = torch.where(torch.rand(T, generator=g, device="cuda") < skipped, -1 - slots, slots)
    cache = torch.full((NB, Hkv, bs, D), 3 if fp8 else 2.5, device="cuda",
                       dtype=torch.uint8 if fp8 else DT[dt])
    pos = torch.randint(0, P, (T,), generator=g, device="cuda", dtype=torch.int32)
    if T > 1:
        pos[0], pos[-1] = 0, P - 1
    w = [(1 + 0.3 * torch.randn(D, generator=g, device="cuda")).to(DT[dt]) for _ in range(2)]
    return packed, q, k, v, cache, cache.clone(), slots, pos, angles(P, D if R is None else R), w


def check_cache(got, before, ref, slack, slots, kind, scale, what):
    NB, H, bs, D = got.shape
    live = (slots >= 0).cpu()
    at = slots.cpu()[live]
    flat = got.transpose(1, 2).reshape(NB * bs, H, D).cpu()
    old = before.transpose(1, 2).reshape(NB * bs, H, D).cpu()
    rows = flat[at]
    if kind == "e4m3":
        rows = rows.view(torch.float8_e4m3fn).float()
        # the quotient by the fp32 scale adds one rounding; saturation at 448
        sc = float(np.float32(scale))
        ref, slack = (ref / sc).clamp(-448, 448), slack / sc + (ref / sc).abs() * 2.0 ** -23
    check(rows, ref[live], slack[live], kind, what)
    rest = torch.ones(NB * bs, dtype=torch.bool)
    rest[at] = False
    assert torch.equal(flat[rest], old[rest]), f"{what}: a slot of no row was written"


CASES = [
    # T, Hq, Hkv, D, R, dtype, fp8, interleaved, norm
    (1, 8, 2, 64, 64, "f16", False, False, True),
    (1, 1, 1, 16, 16, "bf16", False, False, True),
    (7, 5, 3, 48, 32, "bf16", False, True, True),
    (33, 4, 4, 80, 48, "f16", False, False, True),
    (64, 32, 8, 128, 128, "bf16", False, False, True),
    (64, 32, 8, 128, 128, "bf16", True, False, True),
    (129, 6, 1, 96, 96, "f16", True, True, True),
    (100, 8, 2, 256, 128, "bf16", False, False, True),
    (51, 16, 16, 256, 256, "f16", True, False, False),
    (2049, 32, 8, 128, 64, "bf16", False, False, True),   # four heads a thread
    (4100, 8, 2, 64, 32, "f16", False, True, True),
    (1500, 12, 4, 256, 256, "f16", False, False, True),
    (3001, 7, 3, 112, 0, "bf16", True, False, True),      # no rotation
    (40, 0, 4, 128, 128, "bf16", False, False, True),     # keys only
    (40, 4, 0, 128, 128, "bf16", False, False, True),     # queries only
]


@pytest.mark.parametrize("T,Hq,Hkv,D,R,dt,fp8,inter,norm", CASES)
def test_against_the_formulas(T, Hq, Hkv, D, R, dt, fp8, inter, norm, pa_lib):
    packed, q, k, v, kc, vc, slots, pos, cs, (wq, wk) = make(T, Hq, Hkv, D, dt, fp8, seed=T + D, R=R)
    if not norm:
        wq = wk = None
    ks, vs = (0.0371, 0.0123) if fp8 else (1.0, 1.0)
    before = packed.clone()
    k0, v0 = kc.clone(), vc.clone()
    out = pa_lib.norm_rope_and_cache(q, k, v, kc, vc, slots, pos, cs, q_weight=wq, k_weight=wk,
                                     eps=1e-5, interleaved=inter, kv_dtype="fp8" if fp8 else "auto",
                                     k_scale=ks, v_scale=vs)
    assert pa_lib.check_device_error() == 0
    assert torch.equal(packed, before)
    eps = float(np.float32(1e-5))
    if Hq:
        check(out, *reference(q, wq, cs, pos, R, inter, eps), dt, "q")
    if not Hkv:
        return
    kind = "e4m3" if fp8 else dt
    ref, slack = reference(k, wk, cs, pos, R, inter, eps)
    check_cache(kc, k0, ref, slack, slots, kind, ks, "k")
    # v: as the plain write path stores it, bit for bit
    kp, vp = k0.clone(), v0.clone()
    pa_lib.reshape_and_cache(k.contiguous(), v.contiguous(), kp, vp, slots,
                             "fp8" if fp8 else "auto", ks, vs)
    assert torch.equal(vc, vp)


@pytest.mark.parametrize("src", ["bf16", "f16"])
@pytest.mark.parametrize("scale", [1.0, 0.0123, 3.7, 1e-3, 300.0, 0.7499999, 2.0 ** -60, 1.1e-19, 1e-30, 1e30, 3e38])
def test_v_codes_equal_the_plain_write_paths_for_every_pattern(src, scale, pa_lib):
    """All 65,536 16-bit inputs, infinities and NaNs among them."""
    bits = torch.from_numpy(np.arange(65536, dtype=np.uint32).astype(np.uint16).view(np.int16).copy())
    for H, D in ((2, 128), (4, 64)):
        T = 65536 // (H * D)
        v = bits.view(DT[src]).reshape(T, H, D).cuda()
        k = torch.zeros_like(v)
        NB = -(-T // 16)
        a = [torch.zeros(NB, H, 16, D, dtype=torch.uint8, device="cuda") for _ in range(4)]
        slots = torch.arange(T, device="cuda")
        pos = torch.zeros(T, dtype=torch.int32, device="cuda")
        pa_lib.norm_rope_and_cache(k, k, v, a[0], a[1], slots, pos, angles(1, D), kv_dtype="fp8", v_scale=scale)
        pa_lib.reshape_and_cache(k, v, a[2], a[3], slots, "fp8", 1.0, scale)
        nan = torch.isnan(v.float()).reshape(-1, H, D).cpu()
        x, y = (c.transpose(1, 2).reshape(NB * 16, H, D)[:T].cpu() for c in (a[1], a[3]))
        assert torch.equal(x[~nan], y[~nan])
        assert ((x[nan] & 0x7F) == 0x7F).all()


@pytest.mark.parametrize("src", ["bf16", "f16"])
@pytest.mark.parametrize("scale", [1.0, 0.0123, 3.7, 7.0, 1e-3, 300.0, 0.7499999, 2.0 ** -60, 1.1e-19, 1e-30, 1e30, 3e38])
def test_key_codes_equal_the_plain_write_paths_for_every_pattern(src, scale, pa_lib):
    """All 65,536 16-bit keys, without a weight or a rotation: nothing comes between
    the key and its code, so ties of the quotient fall alike."""
    bits = torch.from_numpy(np.arange(65536, dtype=np.uint32).astype(np.uint16).view(np.int16).copy())
    for H, D in ((2, 128), (4, 64)):
        for many in (1, 20):            # 20: four heads a thread
            T = 65536 // (H * D)
            k = bits.view(DT[src]).reshape(T, H, D).cuda().repeat(many, 1, 1)
            T *= many
            v = torch.zeros_like(k)
            NB = -(-T // 16)
            a = [torch.zeros(NB, H, 16, D, dtype=torch.uint8, device="cuda") for _ in range(4)]
            slots = torch.arange(T, device="cuda")
            pos = torch.zeros(T, dtype=torch.int32, device="cuda")
            pa_lib.norm_rope_and_cache(v, k, v, a[0], a[1], slots, pos, angles(1, 0), kv_dtype="fp8", k_scale=scale)
            pa_lib.reshape_and_cache(k, v, a[2], a[3], slots, "fp8", scale, 1.0)
            nan = torch.isnan(k.float()).cpu()
            x, y = (c.transpose(1, 2).reshape(NB * 16, H, D)[:T].cpu() for c in (a[0], a[2]))
            assert torch.equal(x[~nan], y[~nan])
            assert ((x[nan] & 0x7F) == 0x7F).all()


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("T", [5, 2100])
@pytest.mark.parametrize("scale", [1e-40, 1e-25, 0.02, 1e25, 3e38])
def test_keys_at_any_scale(scale, T, norm, pa_lib):
    """Keys of up to about 448 times the scale, inside fp32's range with a
    factor of 30 for the products and sums on the way."""
    D = 128
    packed, q, k, v, kc, vc, slots, pos, cs, (_, wk) = make(T, 8, 2, D, "bf16", True, skipped=0, seed=3)
    sc = float(np.float32(scale))
    size = min(100 * sc, 1e37)
    if norm:
        wk = (wk.double() * size).to(torch.bfloat16)
    else:
        wk = None
        k.copy_(k.double() * size / 5)
    k[0].zero_()
    k0 = kc.clone()
    pa_lib.norm_rope_and_cache(q, k, v, kc, vc, slots, pos, cs, k_weight=wk, eps=1e-5, kv_dtype="fp8", k_scale=sc)
    ref, slack = reference(k, wk, cs, pos, D, False, float(np.float32(1e-5)))
    # a product below fp32's least normal number is off by 2^-149, four of them a pair
    check_cache(kc, k0, ref, slack + 2.0 ** -146, slots, "e4m3", sc, f"k at {scale}")


@pytest.mark.parametrize("T", [3, 3000])
def test_in_place_and_strided_outputs(T, pa_lib):
    packed, q, k, v, kc, vc, slots, pos, cs, (wq, wk) = make(T, 8, 2, 128, "bf16", False, extra_cols=24)
    kw = dict(q_weight=wq, k_weight=wk)
    want = pa_lib.norm_rope_and_cache(q, k, v, kc, vc, slots, pos, cs, **kw)
    kc2, vc2 = torch.full_like(kc, 2.5), torch.full_like(vc, 2.5)
    wide = torch.full((T, 8 * 128 + 16), 9.0, dtype=q.dtype, device="cuda")
    strided = wide[:, :1024].unflatten(1, (8, 128))
    pa_lib.norm_rope_and_cache(q, k, v, kc2, vc2, slots, pos, cs, out=strided, **kw)
    assert torch.equal(strided, want) and torch.equal(kc2, kc) and torch.equal(vc2, vc)
    assert (wide[:, 1024:] == 9).all()
    rest = packed[:, 1024:].clone()
    kc2.fill_(2.5), vc2.fill_(2.5)
    got = pa_lib.norm_rope_and_cache(q, k, v, kc2, vc2, slots, pos, cs, out=q, **kw)
    assert got.data_ptr() == q.data_ptr() and torch.equal(q, want)
    assert torch.equal(packed[:, 1024:], rest) and torch.equal(kc2, kc) and torch.equal(vc2, vc)


def test_one_weight_only_and_zero_rows(pa_lib):
    T = 6
    packed, q, k, v, kc, vc, slots, pos, cs, (wq, wk) = make(T, 4, 2, 64, "f16", False, skipped=0)
    packed[2].zero_()                # a row of zeros stays one
    out = pa_lib.norm_rope_and_cache(q, k, v, kc, vc, slots, pos, cs, k_weight=wk, eps=0.5)
    check(out, *reference(q, None, cs, pos, 64, False, 0.5), "f16", "q without a weight")
    ref, slack = reference(k, wk, cs, pos, 64, False, 0.5)
    check_cache(kc, torch.full_like(kc, 2.5), ref, slack, slots, "f16", 1.0, "k")
    assert (out[2] == 0).all()
    empty = q[:0]
    got = pa_lib.norm_rope_and_cache(empty, k[:0], v[:0], kc, vc, slots[:0], pos[:0], cs)
    assert got.shape == (0, 4, 64)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("R", [0, 32])
@pytest.mark.parametrize("T", [9, 2100])
def test_an_infinity_behind_the_rotation_stays_its_own(T, R, inter, norm, fp8, pa_lib):
    """One infinite element a head, where nothing is rotated: without a weight the
    others pass as they are (as the plain write path stores them), with one they
    are zeros, x / sqrt(inf)."""
    H, D = 4, 96
    packed, q, k, v, kc, vc, slots, pos, cs, (wq, wk) = make(T, 8, H, D, "f16", fp8, skipped=0, R=R, seed=R + T)
    at = torch.randint(R, D, (T, 8 + H), generator=torch.Generator(device="cuda").manual_seed(T), device="cuda")
    for h, x in enumerate([*q.unbind(1), *k.unbind(1)]):
        x.scatter_(1, at[:, h:h + 1], float("inf") if h % 2 else float("-inf"))
    hit = torch.zeros(T, 8 + H, D, dtype=torch.bool, device="cuda").scatter_(2, at[:, :, None], True)
    kw = dict(kv_dtype="fp8", k_scale=0.25) if fp8 else {}
    kp, vp = kc.clone(), vc.clone()
    out = pa_lib.norm_rope_and_cache(q, k, v, kc, vc, slots, pos, cs, interleaved=inter,
                                     **(dict(q_weight=wq, k_weight=wk) if norm else {}), **kw)
    stored = lambda c: c.transpose(1, 2).reshape(-1, H, D)[slots]  # noqa: E731
    keys = stored(kc)
    if fp8:
        keys = keys.view(torch.float8_e4m3fn).float()
    if norm:
        assert (out[~hit[:, :8]] == 0).all() and (keys[~hit[:, 8:]] == 0).all()
        return
    pa_lib.reshape_and_cache(k.contiguous(), v.contiguous(), kp, vp, slots, kw.get("kv_dtype", "auto"),
                             kw.get("k_scale", 1.0), 1.0)
    assert torch.equal(out[..., R:], q[..., R:]) and torch.equal(stored(kc)[..., R:], stored(kp)[..., R:])
    assert torch.isfinite(out[..., :R]).all() and torch.isfinite(keys[..., :R].float()).all()


@pytest.mark.parametrize("dt,spread", [("bf16", 1e18), ("bf16", 1e-18), ("f16", 1e4), ("f16", 1e-6)])
def test_large_and_small_rows(dt, spread, pa_lib):
    """Sums of squares that leave 16 bits (1e36 D is inside fp32's range)."""
    T = 20
    packed, q, k, v, kc, vc, slots, pos, cs, (wq, wk) = make(T, 4, 2, 128, dt, False, skipped=0,
                                                             spread=spread)
    eps = 0.0 if spread > 1 else 1e-30 if dt == "bf16" else 1e-12
    out = pa_lib.norm_rope_and_cache(q, k, v, kc, vc, slots, pos, cs, q_weight=wq, k_weight=wk, eps=eps)
    check(out, *reference(q, wq, cs, pos, 128, False, float(np.float32(eps))), dt, "q")


def test_bad_slots_and_positions_are_flagged_and_safe(pa_lib):
    T, P = 5, 100
    packed, q, k, v, kc, vc, slots, pos, cs, (wq, wk) = make(T, 4, 2, 64, "bf16", False, skipped=0, P=P)
    good = pa_lib.norm_rope_and_cache(q, k, v, kc, vc, slots, pos, cs)
    assert pa_lib.check_device_error() == 0
    bad = pos.clone()
    bad[1], bad[3] = -1, P
    near = pos.clone()
    near[1], near[3] = 0, P - 1
    got = pa_lib.norm_rope_and_cache(q, k, v, kc, vc, slots, bad, cs)
    assert pa_lib.check_device_error() == pa_lib.DEVERR_POSITION
    assert torch.equal(got, pa_lib.norm_rope_and_cache(q, k, v, kc, vc, slots, near, cs))
    kc.fill_(2.5), vc.fill_(2.5)
    over = slots.clone()
    over[2] = kc.shape[0] * 16
    got = pa_lib.norm_rope_and_cache(q, k, v, kc, vc, over, pos, cs)
    assert pa_lib.check_device_error() == pa_lib.DEVERR_SLOT
    assert torch.equal(got, good)
    ref, slack = reference(k, None, cs, pos, 64, False, 0.0)
    over[2] = -1
    check_cache(kc, torch.full_like(kc, 2.5), ref, slack, over, "bf16", 1.0, "k")


def test_another_stream_and_a_graph(pa_lib):
    packed, q, k, v, kc, vc, slots, pos, cs, (wq, wk) = make(40, 8, 2, 128, "bf16", False)
    want = pa_lib.norm_rope_and_cache(q, k, v, kc, vc, slots, pos, cs, q_weight=wq, k_weight=wk)
    out = torch.empty_like(want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
        pa_lib.norm_rope_and_cache(q, k, v, kc, vc, slots, pos, cs, q_weight=wq, k_weight=wk, out=out)
    k1 = kc.clone()
    kc.zero_(), out.zero_()
    kc.copy_(torch.where(k1 == 2.5, 2.5, kc))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(kc, k1)
