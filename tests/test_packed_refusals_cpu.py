"""What pa_prefill_packed, pa_decode_tree, pa_copy_blocks and pa_compact_cache refuse, on
the host: each call differs from a fine one in one respect and comes back with the
documented status before any device is touched (the descriptors point at made-up
addresses, so this runs without a GPU only)."""
import ctypes

import pytest
import torch

from test_lib_cpu import _desc
from test_step_refusals_cpu import ARG, BASE, LAYOUT, UNSUP, refs, strided

pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="host-only: descriptors point at made-up addresses")

T, B, Hq, Hkv, D, NB, bs, MB = 11, 3, 8, 2, 128, 20, 16, 9


@pytest.fixture
def attend(pa_lib):
    pa = pa_lib

    def call(tree, heads=Hkv, scale=0.1, block=bs, window=0, kv=0, ks=1.0, vs=1.0, **over):
        a = dict(out=_desc(pa, pa.PA_BF16, (T, Hq, D), BASE + 0x100000), q=_desc(pa, pa.PA_BF16, (T, Hq, D), BASE),
                 kc=_desc(pa, pa.PA_BF16, (NB, Hkv, bs, D), BASE + 0x200000),
                 vc=_desc(pa, pa.PA_BF16, (NB, Hkv, bs, D), BASE + 0x400000),
                 bt=_desc(pa, pa.PA_I32, (B, MB), BASE + 0x600000), sl=_desc(pa, pa.PA_I32, (B,), BASE + 0x610000),
                 qs=_desc(pa, pa.PA_I32, (B + 1,), BASE + 0x620000))
        if tree:
            a["mask"] = _desc(pa, pa.PA_I64, (T,), BASE + 0x630000)
        a.update(over)
        fn = pa.lib().pa_decode_tree if tree else pa.lib().pa_prefill_packed
        return fn(*refs(a.values()), heads, scale, block, window, kv, ks, vs, None)

    call.pa = pa
    return call


@pytest.mark.parametrize("tree", [False, True])
def test_attention_refusals(attend, tree):
    pa = attend.pa
    d = lambda dt, shape, at: _desc(pa, dt, shape, BASE + at)  # noqa: E731
    bf, f16, f32, i32, i64, e4 = pa.PA_BF16, pa.PA_F16, pa.PA_F32, pa.PA_I32, pa.PA_I64, pa.PA_FP8_E4M3
    codes = dict(kc=d(e4, (NB, Hkv, bs, D), 0x200000), vc=d(e4, (NB, Hkv, bs, D), 0x400000))
    assert attend(tree) == -4, pa.last_error()          # fine: stopped by the missing device only
    assert attend(tree, kv=2, **codes) == -4
    assert attend(tree, window=64) == -4
    assert attend(tree, q=strided(pa, bf, (T, Hq, D), (2000, D, 1), BASE)) == -4
    assert attend(tree, out=strided(pa, bf, (T, Hq, D), (2000, D, 1), BASE + 0x100000)) == -4
    shape = lambda x, **o: dict(q=d(bf, x, 0), out=d(bf, x, 0x100000), **o)  # noqa: E731
    pool = lambda h, dim, dt=bf: dict(kc=d(dt, (NB, h, bs, dim), 0x200000), vc=d(dt, (NB, h, bs, dim), 0x400000))  # noqa: E731
    for want, over in [
        (ARG, dict(q=None)), (ARG, dict(out=None)), (ARG, dict(kc=None)), (ARG, dict(vc=None)), (ARG, dict(bt=None)),
        (ARG, dict(sl=None)), (ARG, dict(qs=None)),
        (UNSUP, dict(q=d(f32, (T, Hq, D), 0))), (ARG, dict(out=d(f16, (T, Hq, D), 0x100000))),
        (ARG, dict(out=d(bf, (T + 1, Hq, D), 0x100000))), (ARG, dict(q=d(bf, (1, T, Hq, D), 0))),
        (ARG, dict(kc=d(f16, (NB, Hkv, bs, D), 0x200000))), (ARG, dict(vc=d(bf, (NB + 1, Hkv, bs, D), 0x400000))),
        (ARG, dict(heads=1)), (ARG, dict(block=32)), (ARG, dict(kv=2)), (ARG, dict(kv=1)), (ARG, dict(**codes)),
        (ARG, dict(scale=float("nan"))), (ARG, dict(scale=float("inf"))),
        (ARG, dict(kv=2, ks=0.0, **codes)), (ARG, dict(kv=2, vs=float("inf"), **codes)),
        (ARG, dict(sl=d(i32, (B + 1,), 0x610000))), (ARG, dict(sl=d(i64, (B,), 0x610000))),
        (ARG, dict(qs=d(i32, (B,), 0x620000))), (ARG, dict(qs=d(i64, (B + 1,), 0x620000))),
        (ARG, dict(bt=d(i64, (B, MB), 0x600000))), (ARG, dict(bt=d(i32, (B, 0), 0x600000))),
        (LAYOUT, dict(bt=strided(pa, i32, (B, MB), (16, 1), BASE + 0x600000))),
        (LAYOUT, dict(qs=strided(pa, i32, (B + 1,), (2,), BASE + 0x620000))),
        (LAYOUT, dict(qs=d(i32, (B + 1,), 0x620002))), (LAYOUT, dict(bt=d(i32, (B, MB), 0x600001))),
        (LAYOUT, dict(kc=d(bf, (NB, Hkv, bs, D), 0x200008))),
        (LAYOUT, dict(kc=strided(pa, bf, (NB, Hkv, bs, D), (2 * Hkv * bs * D, bs * D, D, 1), BASE + 0x200000))),
        (LAYOUT, dict(q=d(bf, (T, Hq, D), 8))),
        (LAYOUT, dict(q=strided(pa, bf, (T, Hq, D), (Hq * D + 4, D, 1), BASE))),
        (LAYOUT, dict(q=strided(pa, bf, (T, Hq, D), (2 * Hq * D, 2 * D, 1), BASE))),
        (LAYOUT, dict(out=strided(pa, bf, (T, Hq, D), (Hq * D, D, 2), BASE + 0x100000))),
        (LAYOUT, dict(out=strided(pa, bf, (T, Hq, D), (512, D, 1), BASE + 0x100000))),
        (LAYOUT, dict(q=strided(pa, bf, (T, Hq, D), (0, D, 1), BASE))),
        (UNSUP, dict(q=strided(pa, bf, (T, Hq, D), (1 << 23, D, 1), 1 << 40))),
        (ARG, dict(out=d(bf, (T, Hq, D), 0))), (ARG, dict(out=d(bf, (T, Hq, D), 0x200000))),
        (ARG, dict(out=d(bf, (T, Hq, D), 0x620000 - 16))),
        (UNSUP, dict(heads=Hkv, **shape((T, 34, D)))),           # 17 heads a KV head
        (ARG, dict(**shape((T, 7, D)))),
        (UNSUP, dict(**shape((T, Hq, 96), **pool(Hkv, 96)))),
        (UNSUP, dict(kv=2, **shape((T, Hq, 64), **pool(Hkv, 64, e4)))),
        (ARG, dict(kc=d(bf, (0, Hkv, bs, D), 0x200000), vc=d(bf, (0, Hkv, bs, D), 0x400000))),
        (UNSUP, dict(bt=d(i32, (B, 1 << 27), 1 << 33))),
        (UNSUP, dict(kc=d(bf, (1 << 26, Hkv, bs, D), 1 << 45), vc=d(bf, (1 << 26, Hkv, bs, D), 1 << 46))),
        (UNSUP, dict(bt=d(i32, (4097, MB), 0x600000), sl=d(i32, (4097,), 1 << 33), qs=d(i32, (4098,), 1 << 34))),
    ]:
        got = attend(tree, **over)
        assert got == want, (got, want, sorted(over), pa.last_error())
    for size in (0, 8, 24, 2048):
        over = dict(block=size, **{n: d(bf, (NB, Hkv, size, D), at) for n, at in (("kc", 0x200000), ("vc", 0x400000))})
        assert attend(tree, **over) == UNSUP
    # no rows or no sequences: nothing to do, before any device
    none = dict(q=d(bf, (0, Hq, D), 0), out=d(bf, (0, Hq, D), 0x100000))
    if tree:
        none["mask"] = d(i64, (0,), 0x630000)
    assert attend(tree, **none) == 0
    assert attend(tree, bt=d(i32, (0, MB), 0x600000), sl=d(i32, (0,), 0x610000), qs=d(i32, (1,), 0x620000)) == 0


def test_tree_refusals(attend):
    pa = attend.pa
    assert attend(True, mask=None) == ARG
    assert attend(True, mask=_desc(pa, pa.PA_I32, (T,), BASE + 0x630000)) == ARG
    assert attend(True, mask=_desc(pa, pa.PA_I64, (T - 1,), BASE + 0x630000)) == ARG
    assert attend(True, mask=_desc(pa, pa.PA_I64, (T,), BASE + 0x630004)) == LAYOUT
    assert attend(True, out=_desc(pa, pa.PA_BF16, (T, Hq, D), BASE + 0x630000)) == ARG
    assert attend(True, window=63) == ARG and attend(False, window=63) == -4
    assert attend(True, window=-1) == -4


@pytest.fixture
def moves(pa_lib):
    pa = pa_lib

    def cache(at, shape=(NB, Hkv, bs, D), dt=None):
        return _desc(pa, pa.PA_BF16 if dt is None else dt, shape, BASE + at)

    def copy(**over):
        a = dict(kc=cache(0), vc=cache(0x400000), pairs=_desc(pa, pa.PA_I32, (5, 2), BASE + 0x800000))
        a.update(over)
        return pa.lib().pa_copy_blocks(*refs(a.values()), None)

    def compact(block=bs, **over):
        i = lambda shape, at: _desc(pa, pa.PA_I32, shape, BASE + at)  # noqa: E731
        a = dict(kc=cache(0), vc=cache(0x400000), bt=i((B, MB), 0x800000), sl=i((B,), 0x810000), qs=i((B + 1,), 0x820000),
                 kept=i((B, 4), 0x830000), num=i((B,), 0x840000), lens=i((B,), 0x850000), tokens=i((B,), 0x860000))
        a.update(over)
        return pa.lib().pa_compact_cache(*refs(a.values()), block, None)

    return pa, cache, copy, compact


def test_move_refusals(moves):
    pa, cache, copy, compact = moves
    i = lambda shape, at: _desc(pa, pa.PA_I32, shape, BASE + at)  # noqa: E731
    l64 = lambda shape, at: _desc(pa, pa.PA_I64, shape, BASE + at)  # noqa: E731
    layers = lambda at, stride: strided(pa, pa.PA_BF16, (3, NB, Hkv, bs, D), (stride, Hkv * bs * D, bs * D, D, 1), BASE + at)  # noqa: E731
    block = Hkv * bs * D
    assert copy() == -4 and compact() == -4 and compact(tokens=None) == -4
    five = lambda s: dict(kc=layers(0, s), vc=layers(0x4000000, s))  # noqa: E731
    for call in (copy, compact):
        far = dict(pairs=i((5, 2), 0x8000000)) if call is copy else dict(
            bt=i((B, MB), 0x8000000), sl=i((B,), 0x8010000), qs=i((B + 1,), 0x8020000), kept=i((B, 4), 0x8030000),
            num=i((B,), 0x8040000), lens=i((B,), 0x8050000), tokens=None)
        assert call(**five(NB * block), **far) == -4 and call(**five(NB * block + 64), **far) == -4
        for want, over in [
            (ARG, dict(kc=None)), (ARG, dict(vc=None)), (ARG, dict(kc=cache(0, (NB, Hkv, D)), vc=cache(0x400000, (NB, Hkv, D)))),
            (ARG, dict(vc=cache(0x400000, (NB, Hkv, bs, D), pa.PA_F16))), (ARG, dict(vc=cache(0x400000, (NB + 1, Hkv, bs, D)))),
            (UNSUP, dict(kc=cache(0, dt=pa.PA_F32), vc=cache(0x400000, dt=pa.PA_F32))),
            (LAYOUT, dict(kc=cache(8))), (ARG, dict(vc=cache(0))), (ARG, dict(vc=cache(block))),
            (LAYOUT, dict(kc=strided(pa, pa.PA_BF16, (NB, Hkv, bs, D), (2 * block, bs * D, D, 1), BASE))),
            (LAYOUT, dict(kc=strided(pa, pa.PA_BF16, (NB, Hkv, bs, D), (block, D, Hkv * D, 1), BASE))),
            (UNSUP, dict(kc=cache(0, (NB, Hkv, bs, 4)), vc=cache(0x400000, (NB, Hkv, bs, 4)))),
        ]:
            got = call(**over)
            assert got == want, (call.__name__, got, want, sorted(over), pa.last_error())
        assert call(**five(NB * block - 8), **far) == LAYOUT      # layers overlap
        assert call(**five(NB * block + 4), **far) == LAYOUT      # not 16-byte aligned
    for want, over in [
        (ARG, dict(pairs=None)), (ARG, dict(pairs=l64((5, 2), 0x800000))), (ARG, dict(pairs=i((5, 3), 0x800000))),
        (ARG, dict(pairs=i((10,), 0x800000))), (LAYOUT, dict(pairs=strided(pa, pa.PA_I32, (5, 2), (4, 1), BASE + 0x800000))),
        (LAYOUT, dict(pairs=i((5, 2), 0x800004))), (ARG, dict(pairs=i((5, 2), 0x400000))),
        (UNSUP, dict(pairs=i((1 << 30, 2), 1 << 33))),
    ]:
        assert copy(**over) == want, (want, sorted(over), pa.last_error())
    assert copy(pairs=i((0, 2), 0x800000)) == 0
    for want, over in [
        (ARG, dict(bt=None)), (ARG, dict(sl=None)), (ARG, dict(qs=None)), (ARG, dict(kept=None)), (ARG, dict(num=None)),
        (ARG, dict(lens=None)), (ARG, dict(bt=l64((B, MB), 0x800000))), (ARG, dict(bt=i((B, 0), 0x800000))),
        (ARG, dict(sl=i((B + 1,), 0x810000))), (ARG, dict(qs=i((B,), 0x820000))), (ARG, dict(kept=i((B + 1, 4), 0x830000))),
        (ARG, dict(kept=l64((B, 4), 0x830000))), (ARG, dict(kept=i((B,), 0x830000))), (ARG, dict(num=i((1,), 0x840000))),
        (ARG, dict(lens=l64((B,), 0x850000))), (ARG, dict(tokens=i((B - 1,), 0x860000))),
        (LAYOUT, dict(kept=strided(pa, pa.PA_I32, (B, 4), (8, 1), BASE + 0x830000))), (LAYOUT, dict(kept=i((B, 4), 0x830002))),
        (LAYOUT, dict(bt=strided(pa, pa.PA_I32, (B, MB), (16, 1), BASE + 0x800000))),
        (ARG, dict(block=32)), (ARG, dict(lens=i((B,), 0x810000))), (ARG, dict(lens=i((B,), 0x830008))),
        (ARG, dict(tokens=i((B,), 0x850000))), (ARG, dict(tokens=i((B,), 0x840004))), (ARG, dict(lens=i((B,), 0x400000))),
        (ARG, dict(kept=i((B, 4), 0))), (UNSUP, dict(bt=i((B, 1 << 27), 1 << 33))),
    ]:
        got = compact(**over)
        assert got == want, (got, want, sorted(over), pa.last_error())
    none = dict(bt=i((0, MB), 0x800000), sl=i((0,), 0x810000), qs=i((1,), 0x820000), kept=i((0, 4), 0x830000),
                num=i((0,), 0x840000), lens=i((0,), 0x850000), tokens=i((0,), 0x860000))
    assert compact(**none) == 0


def test_layers_in_turn(moves):
    """K and V as every other layer of one tensor; layers that touch another's are refused."""
    pa, _, copy, _ = moves
    block = Hkv * bs * D
    layers = lambda at, stride: strided(pa, pa.PA_BF16, (3, NB, Hkv, bs, D), (stride, block, bs * D, D, 1), BASE + at)  # noqa: E731
    size, pairs = 2 * NB * block, _desc(pa, pa.PA_I32, (5, 2), BASE + 0x8000000)
    for vk, step, want in [(size, size, -4), (-size, size, -4), (3 * size, size, -4), (size, size + 32, -4),
                           (size - 16, size, ARG), (size + 16, size, ARG), (2 * size, size, ARG), (size, size - 8, ARG)]:
        at = 0x1000000
        assert copy(kc=layers(at, step), vc=layers(at + vk, step), pairs=pairs) == want, (vk, step, pa.last_error())
    assert copy(kc=layers(0, size), vc=layers(size, size + 8), pairs=pairs) == ARG


def test_workspace_query_refusals(pa_lib):
    pa = pa_lib
    n = ctypes.c_size_t(0)
    q = pa.lib().pa_packed_workspace_size
    assert q(10, 2, 8, 2, 128, None) == ARG
    assert q(-1, 2, 8, 2, 128, ctypes.byref(n)) == UNSUP and q((1 << 30) + 1, 2, 8, 2, 128, ctypes.byref(n)) == UNSUP
    assert q(10, 4097, 8, 2, 128, ctypes.byref(n)) == UNSUP and q(10, -1, 8, 2, 128, ctypes.byref(n)) == UNSUP
    assert q(10, 2, 7, 2, 128, ctypes.byref(n)) == ARG and q(10, 2, 34, 2, 128, ctypes.byref(n)) == UNSUP
    assert q(10, 2, 8, 2, 96, ctypes.byref(n)) == UNSUP


def test_both_routes(pa_lib):
    """The compiled binding and the ctypes route: same statuses and messages."""
    pa = pa_lib
    binding = pytest.importorskip("paged_kv_cache_267_gb300._pa_torch")
    i32 = torch.int32
    q, lens, starts = torch.zeros(T, Hq, D, dtype=torch.bfloat16), torch.zeros(B, dtype=i32), torch.zeros(B + 1, dtype=i32)
    kc, vc = (torch.zeros(2, NB, Hkv, bs, D, dtype=torch.bfloat16) for _ in range(2))
    tables, tail = torch.zeros(B, MB, dtype=i32), [Hkv, 0.1, bs, 0, 0, 1.0, 1.0]
    attend = [torch.empty_like(q), q, kc[0], vc[0], tables, lens, starts]
    calls = dict(pa_prefill_packed=attend + tail, pa_decode_tree=attend + [torch.zeros(T, dtype=torch.int64)] + tail,
                 pa_copy_blocks=[kc, vc, torch.zeros(4, 2, dtype=i32)],
                 pa_compact_cache=[kc, vc, tables, lens, starts, torch.zeros(B, 4, dtype=i32), lens.clone(), lens.clone(),
                                   None, bs])
    for name, args in calls.items():
        seen = set()
        for i, x in enumerate(args):
            for other in ([x, None, x.flatten()[1:], x.unsqueeze(0)] if isinstance(x, torch.Tensor) else [x]):
                got = []
                for route in (binding, pa._CtypesCalls()):
                    got.append((getattr(route, name)(*args[:i], other, *args[i + 1:], 0), pa.last_error()))
                assert got[0] == got[1], (name, i, got)
                seen.add(got[0][0])
        assert {-1, -4} <= seen, (name, seen)
