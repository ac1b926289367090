"""The compiled binding of the hot calls and the ctypes route reach the same
library: same statuses and messages for the same arguments, on the host."""
import pytest
import torch

import paged_kv_cache_267_gb300 as pa

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="host tensors, stopped by the missing device")


@pytest.fixture(scope="module")
def routes(pa_lib):
    binding = pytest.importorskip("paged_kv_cache_267_gb300._pa_torch")
    return binding, pa._CtypesCalls()


def call_args():
    B, Hq, Hkv, D, NB, bs, MB, T = 3, 8, 2, 128, 10, 16, 4, 5
    bf, i32 = torch.bfloat16, torch.int32
    cache = lambda: torch.zeros(NB, Hkv, bs, D, dtype=bf)  # noqa: E731
    q = torch.zeros(B, Hq, D, dtype=bf)
    tables, lens = torch.zeros(B, MB, dtype=i32), torch.zeros(B, dtype=i32)
    row = torch.zeros(T, (Hq + 2 * Hkv) * D, dtype=bf)
    qkv = [t.view(T, -1, D) for t in row.split([Hq * D, Hkv * D, Hkv * D], 1)]
    slots, pos = torch.zeros(T, dtype=torch.int64), torch.zeros(T, dtype=i32)
    free, state = torch.zeros(NB, dtype=i32), torch.zeros(2, dtype=i32)
    attend = [torch.empty_like(q), q, cache(), cache(), tables, lens]
    return dict(
        pa_decode=attend + [Hkv, 0.1, bs, 0, 0, 1.0, 1.0],
        pa_decode_shared=attend + [torch.zeros(1, dtype=i32), torch.zeros(2, dtype=i32), Hkv, 0.1, bs, 0, 0, 1.0, 1.0],
        pa_prefill_chunk=[t.unsqueeze(1) for t in attend[:2]] + attend[2:] + [Hkv, 0.1, bs, 0, 0, 1.0, 1.0],
        pa_reshape_and_cache=[qkv[1], qkv[2], cache(), cache(), slots, 0, 1.0, 1.0],
        pa_norm_rope_and_cache=[torch.empty(T, Hq, D, dtype=bf), *qkv, cache(), cache(), slots, pos,
                                torch.zeros(9, 64), None, torch.zeros(D, dtype=bf), 1e-6, 1, 0, 1.0, 1.0],
        pa_pool_extend=[tables, lens, lens.clone(), free, state, lens.clone(), state.clone(),
                        torch.zeros(B + 1, dtype=i32), slots, pos, bs],
        pa_pool_release=[tables, lens, lens.clone(), None, free, state, lens.clone(), state.clone(), bs])


@pytest.mark.parametrize("name", list(call_args()))
def test_routes_agree(routes, name):
    args = call_args()[name]
    seen = {}
    for i, x in enumerate(args):
        for other in ([None, x.to(torch.float64) if x.dtype != torch.float64 else x, x.flatten()[1:], x.unsqueeze(0)]
                      if isinstance(x, torch.Tensor) else [x]):
            if isinstance(other, torch.Tensor) and other.dtype not in pa._TORCH_TO_PA:
                continue
            got = []
            for route in routes:
                status = getattr(route, name)(*args[:i], other, *args[i + 1:], 0)
                got.append((status, pa.last_error()))
            assert got[0] == got[1], (name, i, got)
            seen[got[0][0]] = seen.get(got[0][0], 0) + 1
    assert -1 in seen and -4 in seen, seen      # refusals, and fine calls stopped by the missing device


def test_unknown_type(routes):
    args = call_args()["pa_decode"]
    args[1] = args[1].to(torch.float64)
    for route in routes:
        with pytest.raises((TypeError, KeyError)):
            getattr(route, "pa_decode")(*args, 0)


@pytest.mark.parametrize("stamp", [None, "2.1.0 cpython-312-x86_64-linux-gnu", ""])
def test_a_binding_of_another_torch_is_not_loaded(pa_lib, monkeypatch, tmp_path, stamp):
    """Its symbols may resolve and the layout of tensors differ all the same."""
    from paged_kv_cache_267_gb300 import build
    monkeypatch.setattr(pa, "_calls", None)
    assert not isinstance(pa._native(), pa._CtypesCalls)
    path = tmp_path / "stamp"
    if stamp is not None:
        path.write_text(stamp)
    monkeypatch.setattr(build, "BINDING_STAMP", str(path))
    monkeypatch.setattr(pa, "_calls", None)
    assert isinstance(pa._native(), pa._CtypesCalls)


def test_descriptors_for_the_library_itself(pa_lib):
    """As a PaTensor, by reference, as a pointer or as bytes; nothing else."""
    import ctypes
    t = call_args()["pa_decode"][:6]
    forms = [pa.tensor_desc, lambda x: ctypes.byref(pa.tensor_desc(x)), lambda x: ctypes.pointer(pa.tensor_desc(x)), pa._desc]
    seen = set()
    for form in forms:
        seen.add((pa.lib().pa_decode(*[form(x) for x in t], 2, 0.1, 16, 0, 0, 1.0, 1.0, None), pa.last_error()))
        assert pa.lib().pa_decode(None, *[form(x) for x in t[1:]], 2, 0.1, 16, 0, 0, 1.0, 1.0, None) == -1
    assert len(seen) == 1
    for bad in (t[0].data_ptr(), 0, "x", t[0], 1.5):
        with pytest.raises(ctypes.ArgumentError):
            pa.lib().pa_decode(bad, *[pa.tensor_desc(x) for x in t[1:]], 2, 0.1, 16, 0, 0, 1.0, 1.0, None)


@pytest.mark.parametrize("window", [2**31 - 1, 2**31, 2**32 + 5, 2**63 - 1, -1, -2**31 - 1])
def test_windows_beyond_32_bits(routes, window, monkeypatch):
    """They reach the library (and are stopped by the missing device only), as the
    largest window or none."""
    args = call_args()
    kw = dict(num_kv_heads=2, scale=0.1, block_size=16, window=window, stream=0)
    for route in routes:
        sent = []

        class Spy:
            def __getattr__(self, name):
                return lambda *a: (sent.append(a), getattr(route, name)(*a))[1]

        monkeypatch.setattr(pa, "_calls", Spy())
        for name in ("decode", "decode_shared", "prefill_chunk", "decode_noalloc"):
            out, *rest = args["pa_" + name if name != "decode_noalloc" else "pa_decode"]
            rest = [x for x in rest if isinstance(x, torch.Tensor)]
            with pytest.raises(pa.PAError) as e:
                getattr(pa, name)(*rest, out=out, **kw)
            assert e.value.status == -4
        windows = [[x for x in a if isinstance(x, int)][2] for a in sent]  # kv heads, block size, window
        assert windows == [2**31 - 1 if window > 0 else -1] * 4
