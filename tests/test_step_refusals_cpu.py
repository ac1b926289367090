"""What pa_norm_rope_and_cache, pa_pool_extend and pa_pool_release refuse, on
the host: each call differs from a fine one in one respect and comes back with
the documented status before any device is touched (the descriptors point at
made-up addresses, so this runs without a GPU only)."""
import ctypes

import pytest
import torch

from test_lib_cpu import _desc

pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="host-only: descriptors point at made-up addresses")

BASE = 0x10000000
ARG, UNSUP, LAYOUT = -1, -2, -3


def strided(pa, dtype, shape, strides, data):
    d = _desc(pa, dtype, shape, data)
    for i, s in enumerate(strides):
        d.strides[i] = s
    return d


def refs(ts):
    return [None if t is None else ctypes.byref(t) for t in ts]


@pytest.fixture
def norm(pa_lib):
    pa = pa_lib
    T, Hq, Hkv, D, NB, bs = 5, 4, 2, 128, 6, 16
    W = (Hq + 2 * Hkv) * D

    def call(eps=1e-6, kv=0, ks=1.0, vs=1.0, **over):
        rows = lambda h, off: strided(pa, pa.PA_BF16, (T, h, D), (W, D, 1), BASE + 2 * off)  # noqa: E731
        a = dict(out=_desc(pa, pa.PA_BF16, (T, Hq, D), BASE + 0x100000), q=rows(Hq, 0),
                 k=rows(Hkv, Hq * D), v=rows(Hkv, (Hq + Hkv) * D),
                 kc=_desc(pa, pa.PA_BF16, (NB, Hkv, bs, D), BASE + 0x200000),
                 vc=_desc(pa, pa.PA_BF16, (NB, Hkv, bs, D), BASE + 0x400000),
                 slots=_desc(pa, pa.PA_I64, (T,), BASE + 0x600000),
                 pos=_desc(pa, pa.PA_I32, (T,), BASE + 0x610000),
                 cs=_desc(pa, pa.PA_F32, (50, D), BASE + 0x620000),
                 wq=_desc(pa, pa.PA_BF16, (D,), BASE + 0x700000),
                 wk=_desc(pa, pa.PA_BF16, (D,), BASE + 0x710000))
        a.update(over)
        return pa.lib().pa_norm_rope_and_cache(*refs(a.values()), eps, 0, kv, ks, vs, None)

    call.pa, call.rows = pa, lambda h, D, w, off, dt=None: strided(
        pa, pa.PA_BF16 if dt is None else dt, (T, h, D), (w, D, 1), BASE + 2 * off)
    return call


def test_norm_refusals(norm):
    pa = norm.pa
    d = lambda dt, shape, at: _desc(pa, dt, shape, BASE + at)  # noqa: E731
    bf, f16, f32, i32, i64, e4 = pa.PA_BF16, pa.PA_F16, pa.PA_F32, pa.PA_I32, pa.PA_I64, pa.PA_FP8_E4M3
    assert norm() == -4, pa.last_error()      # fine: stopped by the missing device only
    W = 8 * 128
    for want, over in [
        (ARG, dict(q=None)), (ARG, dict(out=None)), (ARG, dict(slots=None)), (ARG, dict(cs=None)),
        (UNSUP, dict(q=norm.rows(4, 128, W, 0, f32))),
        (ARG, dict(k=norm.rows(2, 128, W, 512, f16))),
        (ARG, dict(out=d(f16, (5, 4, 128), 0x100000))),
        (ARG, dict(out=d(bf, (5, 3, 128), 0x100000))),
        (ARG, dict(v=norm.rows(1, 128, W, 768))),
        (ARG, dict(kc=d(bf, (6, 3, 16, 128), 0x200000))),
        (ARG, dict(kc=d(bf, (7, 2, 16, 128), 0x200000))),
        (ARG, dict(kv=2)),                                     # e4m3 asked, bf16 caches
        (ARG, dict(kv=1)),
        (ARG, dict(kv=2, ks=0.0, kc=d(e4, (6, 2, 16, 128), 0x200000), vc=d(e4, (6, 2, 16, 128), 0x400000))),
        (ARG, dict(kv=2, vs=float("nan"), kc=d(e4, (6, 2, 16, 128), 0x200000), vc=d(e4, (6, 2, 16, 128), 0x400000))),
        (ARG, dict(slots=d(i32, (5,), 0x600000))), (ARG, dict(slots=d(i64, (4,), 0x600000))),
        (ARG, dict(pos=d(i64, (5,), 0x610000))), (ARG, dict(pos=d(i32, (6,), 0x610000))),
        (ARG, dict(cs=d(bf, (50, 128), 0x620000))),
        (UNSUP, dict(cs=d(f32, (50, 144), 0x620000))),         # R > D
        (UNSUP, dict(cs=d(f32, (50, 24), 0x620000))),
        (ARG, dict(cs=d(f32, (0, 128), 0x620000))),            # no row to clamp to
        (LAYOUT, dict(cs=strided(pa, f32, (50, 128), (256, 1), BASE + 0x620000))),
        (LAYOUT, dict(cs=d(f32, (50, 128), 0x620004))),
        (ARG, dict(wq=d(f32, (128,), 0x700000))), (ARG, dict(wk=d(bf, (64,), 0x710000))),
        (LAYOUT, dict(wq=d(bf, (128,), 0x700002))),
        (LAYOUT, dict(wk=strided(pa, bf, (128,), (2,), BASE + 0x710000))),
        (ARG, dict(eps=-1.0)), (ARG, dict(eps=float("inf"))),
        (LAYOUT, dict(kc=d(bf, (6, 2, 16, 128), 0x200008))),
        (LAYOUT, dict(q=norm.rows(4, 128, W + 4, 0))),         # rows not 16-byte aligned
        (LAYOUT, dict(q=norm.rows(4, 128, W, 4))),
        (LAYOUT, dict(q=strided(pa, bf, (5, 4, 128), (W, 256, 1), BASE))),
        (LAYOUT, dict(k=strided(pa, bf, (5, 2, 128), (W, 128, 2), BASE + 1024))),
        (LAYOUT, dict(out=strided(pa, bf, (5, 4, 128), (256, 128, 1), BASE + 0x100000))),
        (LAYOUT, dict(out=strided(pa, bf, (5, 4, 128), (0, 128, 1), BASE + 0x100000))),
        (ARG, dict(out=norm.rows(4, 128, W, 512))),            # over k
        (ARG, dict(out=d(bf, (5, 4, 128), 0x200000))),         # over a cache
        (ARG, dict(out=d(bf, (5, 4, 128), 0x610000 - 16))),    # over the positions
        (ARG, dict(vc=d(bf, (6, 2, 16, 128), 0x200000))),
        (ARG, dict(vc=d(bf, (6, 2, 16, 128), 0x200000 + 256))),
        (ARG, dict(kc=d(bf, (6, 2, 16, 128), 0))),             # over q
    ]:
        got = norm(**over)
        assert got == want, (got, want, sorted(over), pa.last_error())
    # q's own place is fine, but not where k or v are rows of q themselves
    own = norm.rows(4, 128, W, 0)
    assert norm(out=own) == -4
    assert norm(out=own, k=norm.rows(2, 128, W, 768), v=norm.rows(2, 128, W, 512)) == -4
    assert norm(out=own, k=norm.rows(2, 128, W, 256)) == ARG
    assert norm(out=own, v=norm.rows(2, 128, W, 2 * W + 128)) == ARG
    assert norm(out=own, v=norm.rows(2, 128, W, W - 128)) == ARG      # ends in the next row's q
    assert norm(out=own, v=norm.rows(2, 128, 2 * W, 768)) == ARG      # another stride
    assert norm(out=own, v=norm.rows(2, 128, W, 9 * W + 384)) == -4   # beyond the last row
    for D in (8, 264, 272):
        assert norm(q=norm.rows(4, D, 8 * D, 0), out=d(bf, (5, 4, D), 0x100000), k=norm.rows(2, D, 8 * D, 4 * D),
                    v=norm.rows(2, D, 8 * D, 6 * D), kc=d(bf, (6, 2, 16, D), 0x200000), vc=d(bf, (6, 2, 16, D), 0x400000),
                    cs=d(f32, (50, 0), 0x620000), wq=None, wk=None) == UNSUP
    # no rows: nothing to do, before any device
    none = dict(q=d(bf, (0, 4, 128), 0), out=d(bf, (0, 4, 128), 0x100000), k=d(bf, (0, 2, 128), 0), v=d(bf, (0, 2, 128), 0),
                slots=d(i64, (0,), 0), pos=d(i32, (0,), 0))
    assert norm(**none) == 0


@pytest.fixture
def pool(pa_lib):
    pa = pa_lib
    B, MB, NB, T = 3, 4, 12, 20

    def base():
        i = lambda shape, at: _desc(pa, pa.PA_I32, shape, BASE + at)  # noqa: E731
        return dict(tables=i((B, MB), 0), lens=i((B,), 0x1000), free=i((NB,), 0x3000), state=i((2,), 0x4000),
                    lens_out=i((B,), 0x5000), state_out=i((2,), 0x6000)), i

    def extend(bs=16, **over):
        a, i = base()
        a.update(new=i((B,), 0x2000), start=i((B + 1,), 0x7000), slots=_desc(pa, pa.PA_I64, (T,), BASE + 0x8000),
                 pos=i((T,), 0x9000))
        a.update(over)
        return pa.lib().pa_pool_extend(*refs(a[n] for n in ("tables", "lens", "new", "free", "state", "lens_out", "state_out",
                                                            "start", "slots", "pos")), bs, None)

    def release(bs=16, **over):
        a, i = base()
        a.update(gone=i((B,), 0x2000), shared=i((B,), 0x7000))
        a.update(over)
        return pa.lib().pa_pool_release(*refs(a[n] for n in ("tables", "lens", "gone", "shared", "free", "state", "lens_out",
                                                             "state_out")), bs, None)

    return pa, extend, release


def test_pool_refusals(pool):
    pa, extend, release = pool
    i = lambda shape, at: _desc(pa, pa.PA_I32, shape, BASE + at)  # noqa: E731
    l64 = lambda shape, at: _desc(pa, pa.PA_I64, shape, BASE + at)  # noqa: E731
    assert extend() == -4 and release() == -4 and release(shared=None) == -4
    both = [
        (ARG, dict(tables=None)), (ARG, dict(lens=None)), (ARG, dict(free=None)), (ARG, dict(state=None)),
        (ARG, dict(lens_out=None)), (ARG, dict(state_out=None)),
        (ARG, dict(tables=l64((3, 4), 0))), (ARG, dict(lens=l64((3,), 0x1000))), (ARG, dict(lens=i((2,), 0x1000))),
        (ARG, dict(free=l64((12,), 0x3000))), (ARG, dict(state=i((1,), 0x4000))), (ARG, dict(state_out=i((3,), 0x6000))),
        (ARG, dict(lens_out=i((4,), 0x5000))), (ARG, dict(tables=i((3, 0), 0))),
        (LAYOUT, dict(tables=strided(pa, pa.PA_I32, (3, 4), (8, 1), BASE))),
        (LAYOUT, dict(lens=strided(pa, pa.PA_I32, (3,), (2,), BASE + 0x1000))),
        (LAYOUT, dict(free=i((12,), 0x3002))), (LAYOUT, dict(tables=i((3, 4), 1))),
        (UNSUP, dict(bs=24)), (UNSUP, dict(bs=0)), (UNSUP, dict(bs=-16)), (UNSUP, dict(bs=2048)),
        (UNSUP, dict(tables=i((3, 1 << 28), 0x10000000), bs=16)),
        (UNSUP, dict(free=i((2**31 - 100,), 0x10000000))),
        (ARG, dict(lens_out=i((3,), 0x1004))),      # over the lengths, but not in their place
        (ARG, dict(state_out=i((2,), 0x4004))),
        (ARG, dict(lens_out=i((3,), 0x3000))),      # over the free list
        (ARG, dict(state_out=i((2,), 0x5008))),     # two outputs
        (ARG, dict(state_out=i((2,), 0))),          # over the tables
    ]
    for call in (extend, release):
        for want, over in both:
            got = call(**over)
            assert got == want, (call.__name__, got, want, sorted(over), pa.last_error())
    for want, over in [
        (ARG, dict(new=None)), (ARG, dict(start=None)), (ARG, dict(slots=None)), (ARG, dict(pos=None)),
        (ARG, dict(start=i((3,), 0x7000))), (ARG, dict(slots=i((20,), 0x8000))), (ARG, dict(pos=i((19,), 0x9000))),
        (ARG, dict(new=i((4,), 0x2000))), (UNSUP, dict(slots=l64(((1 << 30) + 1,), 1 << 33), pos=i(((1 << 30) + 1,), 1 << 35))),
        (ARG, dict(pos=i((20,), 0x8000))), (ARG, dict(start=i((4,), 0x2000))), (LAYOUT, dict(slots=l64((20,), 0x8004))),
    ]:
        got = extend(**over)
        assert got == want, (got, want, sorted(over), pa.last_error())
    for want, over in [(ARG, dict(gone=None)), (ARG, dict(gone=i((2,), 0x2000))), (ARG, dict(shared=i((2,), 0x7000))),
                       (ARG, dict(free=i((12,), 0)))]:
        assert release(**over) == want, (want, sorted(over), pa.last_error())
    # in place is fine
    assert extend(lens_out=i((3,), 0x1000), state_out=i((2,), 0x4000)) == -4
    assert release(lens_out=i((3,), 0x1000), state_out=i((2,), 0x4000)) == -4
    too_many = dict(tables=i((4097, 4), 1 << 30), lens=i((4097,), 1 << 31), lens_out=i((4097,), 1 << 32))
    assert extend(new=i((4097,), 1 << 33), start=i((4098,), 1 << 34), **too_many) == UNSUP


@pytest.fixture
def shared(pa_lib):
    pa = pa_lib
    B, Hq, Hkv, D, NB, bs, MB, NG = 6, 8, 2, 128, 20, 16, 9, 2

    def call(heads=Hkv, scale=0.1, bs=bs, window=0, kv=0, ks=1.0, vs=1.0, **over):
        d = lambda dt, shape, at: _desc(pa, dt, shape, BASE + at)  # noqa: E731
        a = dict(out=d(pa.PA_BF16, (B, Hq, D), 0x100000), q=d(pa.PA_BF16, (B, Hq, D), 0),
                 kc=d(pa.PA_BF16, (NB, Hkv, bs, D), 0x200000), vc=d(pa.PA_BF16, (NB, Hkv, bs, D), 0x400000),
                 tables=d(pa.PA_I32, (B, MB), 0x600000), lens=d(pa.PA_I32, (B,), 0x610000),
                 prefix=d(pa.PA_I32, (NG,), 0x620000), starts=d(pa.PA_I32, (NG + 1,), 0x630000))
        a.update(over)
        return pa.lib().pa_decode_shared(*refs(a.values()), heads, scale, bs, window, kv, ks, vs, None)

    return pa, call


@pytest.mark.parametrize("path", [0, 1, 2])
def test_shared_refusals(shared, path):
    """The same answers whichever kernels the call would take."""
    pa, call = shared
    d = lambda dt, shape, at: _desc(pa, dt, shape, BASE + at)  # noqa: E731
    bf, f16, i32, i64, e4 = pa.PA_BF16, pa.PA_F16, pa.PA_I32, pa.PA_I64, pa.PA_FP8_E4M3
    pa.set_shared_path(path)
    try:
        assert call() == -4, pa.last_error()       # fine: stopped by the missing device only
        none = dict(prefix=d(i32, (0,), 0x620000), starts=d(i32, (1,), 0x630000))
        assert call(**none) == -4
        for want, over in [
            (ARG, {n: None}) if isinstance(n, str) else n for n in [
                "out", "q", "kc", "vc", "tables", "lens", "prefix", "starts",
                (ARG, dict(prefix=d(i64, (2,), 0x620000))), (ARG, dict(starts=d(i64, (3,), 0x630000))),
                (ARG, dict(starts=d(i32, (2,), 0x630000))), (ARG, dict(prefix=d(i32, (3,), 0x620000))),
                (ARG, dict(prefix=d(i32, (2, 1), 0x620000))),
                (LAYOUT, dict(prefix=strided(pa, i32, (2,), (2,), BASE + 0x620000))),
                (LAYOUT, dict(starts=strided(pa, i32, (3,), (0,), BASE + 0x630000))),
                (LAYOUT, dict(starts=d(i32, (3,), 0x630002))),
                (UNSUP, dict(prefix=d(i32, (4097,), 0x1000000), starts=d(i32, (4098,), 0x2000000))),
                (ARG, dict(prefix=d(i32, (2,), 0x100000 + 8))),           # under out
                (ARG, dict(starts=d(i32, (3,), 0x100000 - 8))),
                (ARG, dict(out=d(bf, (6, 8, 128), 0x610000 - 16))),       # over the lengths
                (ARG, dict(out=d(bf, (6, 8, 128), 0x200000))),
                (ARG, dict(out=d(f16, (6, 8, 128), 0x100000))), (ARG, dict(out=d(bf, (6, 7, 128), 0x100000))),
                (ARG, dict(heads=4)), (ARG, dict(scale=float("nan"))), (ARG, dict(kv=1)),
                (ARG, dict(tables=d(i32, (5, 9), 0x600000))), (ARG, dict(lens=d(i64, (6,), 0x610000))),
                (ARG, dict(tables=d(i32, (6, 0), 0x600000))),
                (LAYOUT, dict(q=d(bf, (6, 8, 128), 4))),
                (LAYOUT, dict(tables=strided(pa, i32, (6, 9), (12, 1), BASE + 0x600000))),
                (ARG, dict(kv=2)),                                        # e4m3 asked, bf16 caches
                (ARG, dict(kv=2, vs=0.0, kc=d(e4, (20, 2, 16, 128), 0x200000),
                           vc=d(e4, (20, 2, 16, 128), 0x400000))),
                (UNSUP, dict(q=d(bf, (6, 8, 96), 0), out=d(bf, (6, 8, 96), 0x100000),
                             kc=d(bf, (20, 2, 16, 96), 0x200000), vc=d(bf, (20, 2, 16, 96), 0x400000))),
            ]]:
            got = call(**over)
            assert got == want, (got, want, sorted(over), pa.last_error())
        # no sequences: nothing to do, before any device
        assert call(q=d(bf, (0, 8, 128), 0), out=d(bf, (0, 8, 128), 0x100000), tables=d(i32, (0, 9), 0x600000),
                    lens=d(i32, (0,), 0x610000)) == 0
    finally:
        pa.set_shared_path(0)


def test_shared_settings(shared):
    pa, _ = shared
    for bad in (-1, 3):
        with pytest.raises(pa.PAError):
            pa.set_shared_path(bad)
    for bad in (dict(num_groups=-1), dict(num_groups=4097), dict(batch=4097), dict(head_dim=96), dict(num_kv_heads=3)):
        with pytest.raises(pa.PAError):
            pa.decode_shared_workspace_size(**{**dict(batch=4, num_groups=1, num_q_heads=8, num_kv_heads=2, head_dim=128),
                                               **bad})
