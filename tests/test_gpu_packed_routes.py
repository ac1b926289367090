"""Ragged steps on each of their kernels, told apart by their launches: small steps in narrow
tables work on whole pairs (one launch), or cut them and join (two); more sequences than a warp
plans have a plan kernel in front (three)."""
import pytest
import torch

import paged_kv_cache_267_gb300 as pa
from test_gpu_packed import Step

pytestmark = pytest.mark.gpu

WHOLE, CUT, PLANNED = 1, 2, 3


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
