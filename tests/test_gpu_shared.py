"""pa_decode_shared against the fp64 oracle's plain decode of the same batch.

The pool holds NaN wherever no sequence has a token, so reading a table entry,
a tail slot or a window's outside that nobody attends to shows in the result.

Tolerance. With weights w_j (summing to 1) and A = sum_j w_j |v_j|, element by
element (the oracle's decode over |V|):
  - the output is rounded once: h |out|, h = 2^-8 (bf16) or 2^-11 (f16);
  - the weights enter the second product in 16 bits, bf16 for bf16 caches and
    f16 for the others: p A with p = 2^-8 or 2^-11, and, where f16 weights are
    subnormal, 2^-25 each against a sum of at least 2^-8 (the lazy reference):
    n 2^-17 mean |v|, which is below n 2^-17 max |v| over n tokens; weights that
    small stay below 2^-6 A of the total for the sizes here, so 2^-11 A more;
  - scores: fp32 sums of D products, off by D 2^-24 sum |q k| scale log2(e); with
    sum |q k| scale below 64 here that is a relative error of each weight of at
    most 256 * 2^-24 * 64 * 1.45 < 2^-9; the exponential adds 2^-21.
Bound: h |ref| + (p + 2^-11 + 2^-9) A + 1e-6.
"""
import subprocess
import sys

import numpy as np
import pytest
import torch

import oracle
from conftest import ROOT, have_gpu
from pa_testutil import host_copy, out_f64
from workloads.layout import shuffled_free_list

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a GPU")]

DT = {"bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(autouse=True)
def shared_path(pa_lib):
    """These batches are small: by default they would be decoded plainly."""
    pa_lib.set_shared_path(2)
    yield
    pa_lib.set_shared_path(0)


class Batch:
    """Groups of (prefix tokens, tails) and rows of no group, over a shuffled
    pool whose unused slots hold NaN."""

    def __init__(self, groups, loose_before=(), loose_after=(), *, heads=(8, 2), D=128, bs=16,
                 dt="bf16", fp8=False, idle=(), seed=0, extra_blocks=3, qmul=1.0, kmul=1.0):
        rng = np.random.default_rng(seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        Hq, Hkv = heads
        self.heads, self.D, self.bs, self.dt, self.fp8 = heads, D, bs, dt, fp8
        lens, starts, pre, owner = list(loose_before), [], [], [None] * len(loose_before)
        for gi, (P, tails) in enumerate(groups):
            starts.append(len(lens))
            pre.append(P)
            lens += [P + t if t is not None else 0 for t in tails]
            owner += [gi] * len(tails)
        starts.append(len(lens))
        lens += list(loose_after)
        owner += [None] * len(loose_after)
        for b in idle:
            lens[b] = 0
        B = len(lens)
        self.MB = max(1, max(-(-n // bs) for n in lens), *[-(-p // bs) for p in pre]) + 1
        shared = [p // bs for p in pre]
        need = sum(shared) + sum(-(-n // bs) for n in lens) + extra_blocks
        ids = shuffled_free_list(need, seed + 1)
        tables = np.full((B, self.MB), -1, np.int32)
        blocks = [[ids.pop() for _ in range(n)] for n in shared]
        used = np.zeros((need, bs), bool)
        for b, n in enumerate(lens):
            nb = -(-n // bs)
            t = (blocks[owner[b]] if owner[b] is not None else [])[:nb]
            t = t + [ids.pop() for _ in range(nb - len(t))]
            tables[b, :nb] = t
            for j, blk in enumerate(t):
                used[blk, :min(bs, n - j * bs)] = True
        self.lens = np.asarray(lens, np.int32)
        self.tables, self.prefix, self.starts, self.B = tables, np.asarray(pre, np.int32), np.asarray(starts, np.int32), B
        self.ks, self.vs = (0.031, 0.017) if fp8 else (1.0, 1.0)
        u = torch.from_numpy(used).cuda()[:, None, :, None]
        shape = (need, Hkv, bs, D)

        def values(mul):
            x = torch.randn(shape, generator=g, device="cuda") * mul
            return torch.where(u, x, torch.nan)

        k, v = values(kmul), values(1.0)
        if fp8:
            enc = lambda x, s: torch.where(u, (x / s).to(torch.float8_e4m3fn).view(torch.uint8), 0x7F)  # noqa: E731
            self.kc, self.vc = enc(k, self.ks).to(torch.uint8), enc(v, self.vs).to(torch.uint8)
            self.va = self.vc & 0x7F
        else:
            self.kc, self.vc = k.to(DT[dt]), v.to(DT[dt])
            self.va = self.vc.abs()
        self.q = (torch.randn(B, Hq, D, generator=g, device="cuda") * qmul).to(DT[dt])
        self.scale = D ** -0.5

    def args(self):
        i = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
        return (self.q, self.kc, self.vc, i(self.tables), i(self.lens), i(self.prefix), i(self.starts))

    def kw(self, window=0):
        return dict(num_kv_heads=self.heads[1], scale=self.scale, block_size=self.bs, window=window,
                    kv_dtype="fp8" if self.fp8 else "auto", k_scale=self.ks, v_scale=self.vs)

    def reference(self, window=0):
        kw = dict(num_kv_heads=self.heads[1], scale=self.scale, block_size=self.bs, window=window,
                  q_dtype=self.dt, cache_dtype="fp8" if self.fp8 else self.dt, k_scale=self.ks, v_scale=self.vs)
        q, kc = host_copy(self.q), host_copy(self.kc)
        return [oracle.decode(q, kc, host_copy(v), self.tables, self.lens, **kw) for v in (self.vc, self.va)]

    def check(self, out, window=0, what=""):
        ref, A = self.reference(window)
        got = out_f64(out)
        assert np.isfinite(got).all(), f"{what}: non-finite outputs in rows {sorted(set(np.argwhere(~np.isfinite(got))[:, 0]))}"
        h = 2.0 ** -8 if self.dt == "bf16" else 2.0 ** -11
        p = 2.0 ** -8 if self.dt == "bf16" and not self.fp8 else 2.0 ** -11
        bound = h * np.abs(ref) + (p + 2.0 ** -11 + 2.0 ** -9) * A + 1e-6
        err = np.abs(got - ref)
        over = (err - bound).max(axis=(1, 2))
        assert over.max() <= 0, f"{what}: rows {np.argwhere(over > 0).ravel()[:8]} beyond the bound by {over.max():.3e}"
        # a wrong or missing token would be far outside this
        assert err.mean() <= 2e-3 * max(A.mean(), 1e-9), f"{what}: mean error {err.mean():.3e}"

    def run(self, pa, window=0):
        out = torch.full_like(self.q, float("nan"))
        pa.decode_shared(*self.args(), out=out, **self.kw(window))
        torch.cuda.synchronize()
        return out


CASES = {
    # one small group, both halves on the same rows
    "two_rows": dict(groups=[(128, [1, 5])]),
    "one_tile": dict(groups=[(16, [1, 2, 40])]),
    "odd_prefix": dict(groups=[(1040, [1, 17, 300, 2])]),
    "no_tails": dict(groups=[(272, [0, 0, 0])]),
    "partial_block": dict(groups=[(261, [3, 30, 9])]),     # 256 tokens are shared
    "below_a_block": dict(groups=[(15, [3, 30])]),         # nothing is
    "single_row_groups": dict(groups=[(256, [5]), (128, [7]), (64, [9])]),
    "idle_rows": dict(groups=[(512, [4, 9, 1, 80, 2])], idle=(0, 3)),
    "one_left": dict(groups=[(512, [4, 9, 1])], idle=(0, 2)),
    "loose_rows": dict(groups=[(384, [1, 2, 3]), (640, [9, 8])], loose_before=(5, 700, 0), loose_after=(33, 1)),
    "empty_groups": dict(groups=[(0, []), (300, [1, 2]), (128, []), (0, [9, 8]), (512, [3, 3, 3])]),
    "many_groups": dict(groups=[(64 + 16 * i, [1 + i, 2]) for i in range(40)]),
    "uneven": dict(groups=[(2048, [3] * 70), (48, [100, 2]), (1008, [1] * 9)], heads=(32, 8)),
    # units of more than 128 rows, the last ones partly filled
    "dual": dict(groups=[(640, [5] * 40)], heads=(8, 2)),
    "dual_129": dict(groups=[(400, [1] * 129)], heads=(2, 2)),
    "dual_units": dict(groups=[(656, [2] * 131)], heads=(8, 2)),
    "group_of_3": dict(groups=[(528, [7] * 90)], heads=(6, 2)),
    "group_of_7": dict(groups=[(528, [7] * 50)], heads=(7, 1)),
    "group_of_16": dict(groups=[(304, [7] * 20)], heads=(32, 2)),
    "group_of_12": dict(groups=[(304, [7] * 11)], heads=(24, 2)),
    "f16": dict(groups=[(1200, [9, 200, 1, 44])], dt="f16", heads=(16, 4)),
    "f16_dual": dict(groups=[(1200, [9] * 48)], dt="f16", heads=(16, 4)),
    "d64": dict(groups=[(720, [9, 2, 130])], D=64, dt="f16"),
    "d64_dual": dict(groups=[(720, [9] * 50)], D=64, heads=(8, 2)),
    "d256": dict(groups=[(720, [9, 2, 130])], D=256),
    "d256_units": dict(groups=[(336, [9] * 70)], D=256, dt="f16", heads=(4, 1)),
    "fp8": dict(groups=[(848, [9, 2, 130])], fp8=True, heads=(8, 2)),
    "fp8_dual": dict(groups=[(848, [3] * 45)], fp8=True, dt="f16", heads=(8, 2)),
    "fp8_d256": dict(groups=[(336, [3] * 45)], fp8=True, D=256, heads=(4, 1)),
    "fp8_d256_f16": dict(groups=[(1008, [3, 60])], fp8=True, dt="f16", D=256, heads=(8, 2)),
    "blocks_of_32": dict(groups=[(992, [9, 2, 130])], bs=32),
    "blocks_of_48": dict(groups=[(48 * 13, [9, 2, 130])], bs=48),
    "blocks_of_1024": dict(groups=[(2048, [9, 1025])], bs=1024),
    "long": dict(groups=[(20000, [50, 1, 700])], heads=(8, 1)),
    "large_scores": dict(groups=[(1504, [9, 70, 300])], qmul=4.0, kmul=1.5),
    "large_scores_dual": dict(groups=[(1504, [9] * 40)], qmul=4.0, kmul=1.5, dt="f16"),
}


@pytest.mark.parametrize("name", list(CASES))
def test_against_the_oracle(name, pa_lib):
    b = Batch(seed=len(name) * 7 + 1, **CASES[name])
    out = b.run(pa_lib)
    assert pa_lib.check_device_error() == 0
    b.check(out, what=name)


@pytest.mark.parametrize("window", [1, 100, 512, 530, 5000])
def test_windows_that_cut_some_rows_off_the_prefix(window, pa_lib):
    b = Batch([(512, [1, 18, 300, 2, 0]), (96, [4, 900])], loose_after=(700, 3), seed=5)
    out = b.run(pa_lib, window)
    assert pa_lib.check_device_error() == 0
    b.check(out, window, f"window {window}")


def poison_outside_windows(b, window):
    """NaN at every position that no sequence attends to, and no table entry of a
    block wholly before a sequence's window."""
    bs = b.bs
    seen = np.zeros((b.kc.shape[0], bs), bool)
    for r, L in enumerate(b.lens):
        p = np.arange(max(0, L - window), L)
        seen[b.tables[r, p // bs], p % bs] = True
        b.tables[r, :max(0, L - window) // bs] = -1
    out = torch.from_numpy(~seen).cuda()[:, None, :, None]
    for x in (b.kc, b.vc):
        x.copy_(torch.where(out, torch.full_like(x, 0x7F if b.fp8 else float("nan")), x))
    b.va = b.vc & 0x7F if b.fp8 else b.vc.abs()


WINDOWED = [
    # groups, windows: prefixes that the windows cut at many places
    (dict(groups=[(1600, [1, 18, 300, 2, 0])], loose_after=(900, 3)), (17, 40, 599, 601, 800, 1599, 1600, 1601, 1700)),
    (dict(groups=[(640, [9] * 40), (2048, [1, 700, 3])], heads=(8, 2)), (330, 1000, 1409)),
    (dict(groups=[(1040, [5, 5, 6])], bs=80, dt="f16"), (250, 1039)),
    (dict(groups=[(848, [9, 2, 130])], fp8=True), (300, 777)),
    (dict(groups=[(720, [9, 2, 130])], D=256, dt="f16"), (288,)),
    (dict(groups=[(720, [9, 2, 30])], D=64), (333,)),
    (dict(groups=[(512, [1, 2]), (256, [1, 1]), (64, [4, 4])] * 12), (200, 511)),
    (dict(groups=[(2048, [9, 1025, 5, 6])], bs=1024, loose_before=(1500,)), (1500, 2049)),
]


@pytest.mark.parametrize("kw,window", [(k, w) for k, ws in WINDOWED for w in ws])
def test_windows_that_end_inside_the_prefix(kw, window, pa_lib):
    b = Batch(seed=window, **kw)
    poison_outside_windows(b, window)
    out = b.run(pa_lib, window)
    assert pa_lib.check_device_error() == 0
    b.check(out, window, f"window {window}")


def test_a_nan_in_one_sequences_window_stays_its_own(pa_lib):
    """The shortest sequence of a group attends to positions that no other one's
    window reaches."""
    b = Batch([(1600, [40, 1, 60, 33])], dt="f16", seed=3)
    window = 900                    # from 701 on for the shortest (1601 - 900), from 733 for the others
    out0 = b.run(pa_lib, window)
    b.check(out0, window)
    b.vc[int(b.tables[1, 732 // 16]), :, 732 % 16] = float("nan")
    b.kc[int(b.tables[1, 705 // 16]), :, 705 % 16] = float("nan")
    out = b.run(pa_lib, window)
    assert out[1].isnan().all()
    rest = [0, 2, 3]
    assert torch.equal(out[rest], out0[rest])
    assert pa_lib.check_device_error() == 0


@pytest.mark.parametrize("dt,fp8", [("bf16", False), ("f16", True)])
def test_negative_and_zero_scale(dt, fp8, pa_lib):
    for scale in (-0.09, 0.0):
        b = Batch([(400, [1, 18, 30]), (256, [4] * 40)], dt=dt, fp8=fp8, seed=6)
        b.scale = scale
        b.check(b.run(pa_lib), what=f"scale {scale}")
    assert pa_lib.check_device_error() == 0


@pytest.mark.parametrize("shape", ["climb", "jump", "fall"])
def test_scores_that_grow_along_the_prefix(shape, pa_lib):
    """The reference maximum moves in some tiles, by more and by less than 8."""
    b = Batch([(1600, [40] * 3), (1600, [5] * 40)], dt="f16", seed=8)
    n = 1600
    t = torch.arange(n, device="cuda", dtype=torch.float32)
    m = {"climb": 0.2 + t / 200, "jump": torch.where(t > 900, 6.0, 0.1), "fall": 8 - t / 250}[shape]
    for gi, row in ((0, 0), (1, 3)):
        blocks = torch.from_numpy(b.tables[row, :n // 16].astype(np.int64)).cuda()
        # K along the mean query, so scores follow m
        for h in range(2):
            d = b.q[row:row + 3, 4 * h:4 * h + 4].float().mean((0, 1))
            d = d / d.norm()
            b.kc[blocks, h] = (m.view(-1, 16, 1) * d * 4).to(torch.float16)
    b.check(b.run(pa_lib), what=shape)
    assert pa_lib.check_device_error() == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("heavy", [0, 1])
def test_halves_of_a_unit_whose_weights_vanish_for_some_rows(heavy, fp8, pa_lib):
    """K along one query on every other tile of 128: for its row one half of the
    unit outweighs the other by more than fp32's range, for the other rows not.
    |score| <= 120 with D = 128 keeps the bound on the scores' error above."""
    b = Batch([(1200, [4, 30, 1])], dt="f16", fp8=fp8, seed=9)
    blocks = torch.from_numpy(b.tables[0, :75].astype(np.int64)).cuda()
    on = blocks[(torch.arange(75, device="cuda") // 8) % 2 == heavy]
    for h in range(2):
        d = b.q[1, 4 * h + 2].float()
        d = d * (119 / b.scale / d.square().sum())
        row = d.to(torch.float16)
        if fp8:
            row = (d / b.ks).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        b.kc[on, h] = row
    b.check(b.run(pa_lib), what=f"heavy {heavy}")
    assert pa_lib.check_device_error() == 0


@pytest.mark.parametrize("fp8,D", [(False, 64), (True, 128)])
@pytest.mark.parametrize("log2,bound", [(25.05, 55296 * 2.0 ** -25.05 + 2.0 ** -12), (19.5, 2.0 ** -11)])
def test_many_small_weights_behind_one_large_one(log2, bound, fp8, D, pa_lib):
    """The first of 131072 shared keys outweighs each of the others by 2^log2; every
    value is 1, and so is the output. A segment has at most 64 * 1024 tiles / 152
    = 432, 55296 tokens. The second product adds 16 weights at a time to an fp32
    sum, which starts with the large one (2^7 with the lift): it drops what is
    below 2^-16, its last place there.
    2^-25.05 each: 16 of them are 2^-14.05, and each alone below the last place, so
    all may go: 55296 2^-25.05, and half a step of f16, 2^-12.
    2^-19.5: 16 are 2^-8.5, off by 2^-7.5 of themselves at most, as is their part
    of the whole, 55296 2^-19.5 = 0.0744: 2^-11.2; their f16 rounding adds 2^-11 of
    that part, the output's 2^-12: below 0.0008, so at most one step from 1."""
    P, Hkv, B, bs = 131072, 64, 2, 16
    k, v = torch.zeros(3, Hkv, bs, D, device="cuda"), torch.ones(3, Hkv, bs, D, device="cuda")
    k[0, :, 0] = 1.0
    k, v = (x.to(torch.float8_e4m3fn).view(torch.uint8) if fp8 else x.to(torch.float16) for x in (k, v))
    tables = torch.ones(B, P // bs + 1, dtype=torch.int32, device="cuda")
    tables[:, 0], tables[:, -1] = 0, 2
    i = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    out = pa_lib.decode_shared(torch.ones(B, Hkv, D, dtype=torch.float16, device="cuda"), k, v, tables, i(P + 3, P + 5),
                               i(P), i(0, B), num_kv_heads=Hkv, scale=log2 * np.log(2.0) / D, block_size=bs,
                               kv_dtype="fp8" if fp8 else "auto")
    assert pa_lib.check_device_error() == 0
    assert (out.double() - 1).abs().max() <= bound, (out.min(), out.max())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("where", ["k", "v"])
@pytest.mark.parametrize("tile", [0, 1, 9])
@pytest.mark.parametrize("rows", [3, 40])
def test_a_nan_that_is_attended_to_shows(rows, tile, where, fp8, pa_lib):
    """One NaN among the shared keys or values of KV head 1: its heads' outputs
    are NaN (one element of them, for a value), the other heads' are as ever."""
    b = Batch([(1200, [4] * rows)], loose_after=(50,), dt="f16", fp8=fp8, seed=9)
    block = int(b.tables[0, tile * 8 + 2])
    cache = b.kc if where == "k" else b.vc
    cache[block, 1, 5, 77] = 0x7F if fp8 else float("nan")
    out = b.run(pa_lib)
    bad = torch.zeros(out.shape, dtype=torch.bool, device="cuda")
    bad[:rows, 4:, slice(None) if where == "k" else slice(77, 78)] = True
    assert torch.equal(out.isnan(), bad)
    cache[block, 1, 5, 77] = 0          # and the rest is what it is without it
    clean = b.run(pa_lib)
    b.check(clean)
    heads = ~bad.any(-1)
    assert (out[heads].float() - clean[heads].float()).abs().max() <= 2.0 ** -6
    assert pa_lib.check_device_error() == 0


def test_agrees_with_decode_and_no_groups_is_decode(pa_lib):
    b = Batch([(640, [9, 3, 100]), (128, [1, 1])], seed=11)
    a = b.args()
    out = b.run(pa_lib)
    plain = pa_lib.decode(*a[:5], **b.kw())
    assert (out.float() - plain.float()).abs().max() <= 2.0 ** -6
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa_lib.set_decode_tuning(pool_permille=-1)  # bit-reproducible
    try:
        x = pa_lib.decode_shared(*a[:5], none, zero, **b.kw())
        assert torch.equal(x, pa_lib.decode(*a[:5], **b.kw()))
        y = [b.run(pa_lib) for _ in range(3)]
        assert torch.equal(y[0], y[1]) and torch.equal(y[0], y[2])
    finally:
        pa_lib.set_decode_tuning()


def test_windows_longer_than_any_sequence(pa_lib):
    """2^31 - 1 and all that is beyond 32 bits cut nothing off."""
    b = Batch([(640, [9, 3, 100]), (128, [1, 1])], seed=11)
    args, kw = b.args(), {k: v for k, v in b.kw().items() if k != "window"}
    q4 = torch.stack([b.q, b.q], 1)
    calls = [lambda w: pa_lib.decode_shared(*args, window=w, **kw), lambda w: pa_lib.decode(*args[:5], window=w, **kw),
             lambda w: pa_lib.prefill_chunk(q4, *args[1:5], window=w, **kw)]
    pa_lib.set_decode_tuning(pool_permille=-1)  # bit-reproducible
    try:
        for call in calls:
            want = call(0)
            for w in (2**31 - 1, 2**31, 2**32 + 5, 2**63 - 1, -1, -2**40):
                assert torch.equal(call(w), want), w
    finally:
        pa_lib.set_decode_tuning()
    assert pa_lib.check_device_error() == 0


def test_small_steps_are_decoded_plainly_by_default(pa_lib):
    b = Batch([(640, [9, 3, 100]), (128, [1, 1])], seed=21)
    big = Batch([(8192, [9] * 70)], seed=22)  # 70 rows of 8200 tokens: 590 MB
    for path, small_kernels, big_kernels in ((0, 2, 4), (1, 2, 2), (2, 4, 4)):
        pa_lib.set_shared_path(path)
        for x, kernels in ((b, small_kernels), (big, big_kernels)):
            n = pa_lib.launch_count()
            out = x.run(pa_lib)
            assert pa_lib.launch_count() - n == kernels
            x.check(out)
    with pytest.raises(pa_lib.PAError):
        pa_lib.set_shared_path(3)


def test_empty_batch(pa_lib):
    b = Batch([(640, [9, 3, 100])], seed=11)
    a = list(b.args())
    out = pa_lib.decode_shared(a[0][:0], a[1], a[2], a[3][:0], a[4][:0], a[5], a[6], **b.kw())
    assert out.shape == (0, 8, 128)


def test_data_errors_are_flagged_and_safe(pa_lib):
    b = Batch([(512, [9, 3, 100]), (256, [4, 4])], seed=12)
    a = list(b.args())
    i = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    assert pa_lib.check_device_error() == 0
    # group starts that leave the batch, or decrease: clamped; rows still right
    for starts, pre in (([-4, 3, 5], [512, 256]), ([0, 3, 99], [512, 256]), ([3, 0, 5], [512, 256]),
                        ([0, 3, 5], [512, -7])):
        out = pa_lib.decode_shared(*a[:5], i(pre), i(starts), **b.kw())
        assert pa_lib.check_device_error() == pa_lib.DEVERR_GROUP
        if starts == [3, 0, 5]:
            continue  # rows 3, 4 become one group with the first prefix
        b.check(out, what=str(starts))
    # beyond the tables: no row is that long
    out = pa_lib.decode_shared(*a[:5], i([512, 2**31 - 1]), i([0, 3, 5]), **b.kw())
    assert pa_lib.check_device_error() == pa_lib.DEVERR_GROUP
    b.check(out, what="prefix")
    # a bad block id in the prefix, a bad length
    bad = a[3].clone()
    bad[0, 7] = 10**6
    pa_lib.decode_shared(*a[:3], bad, *a[4:], **b.kw())
    assert pa_lib.check_device_error() & pa_lib.DEVERR_BLOCK_ID
    lens = a[4].clone()
    lens[1] = 10**7
    pa_lib.decode_shared(*a[:4], lens, *a[5:], **b.kw())
    assert pa_lib.check_device_error() & pa_lib.DEVERR_SEQ_LEN
    b.check(b.run(pa_lib), what="after the errors")
    assert pa_lib.check_device_error() == 0


def test_own_workspace_of_the_stated_size(pa_lib):
    b = Batch([(640, [9] * 40), (128, [1, 1])], seed=13)
    n = pa_lib.decode_shared_workspace_size(b.B, 2, 8, 2, 128)
    ws = torch.empty(n + 256, dtype=torch.uint8, device="cuda")
    ws[n:] = 77
    try:
        pa_lib.set_workspace(ws[:n])
        for _ in range(2):
            b.check(b.run(pa_lib))
        assert (ws[n:] == 77).all()
        pa_lib.set_workspace(ws[:4096])
        with pytest.raises(pa_lib.PAError):
            b.run(pa_lib)
    finally:
        pa_lib.set_workspace(None)


@pytest.mark.parametrize("fp8", [False, True])
def test_large_batches_after_small_ones(fp8, pa_lib):
    """The shared memory that a large batch needs stays granted."""
    kw = dict(dt="f16", fp8=fp8, heads=(2, 1))
    big, mid, small = (Batch([(64, [3] * n)], seed=n, **kw) for n in (1500, 300, 2))
    for b in (big, small, mid, big, small, big):
        b.check(b.run(pa_lib))
        a = b.args()
        b.check(pa_lib.decode(*a[:5], **b.kw()))
    assert pa_lib.check_device_error() == 0


def test_many_groups_of_many_rows(pa_lib):
    """More groups than one warp scans, up to the limits of the call."""
    b = Batch([(16, [1])] * 4000 + [(32, [2] * 96)], dt="f16", heads=(1, 1), D=64, seed=5)
    assert b.B == 4096
    out = b.run(pa_lib)
    assert pa_lib.check_device_error() == 0
    b.check(out)
    few = Batch([(16, [1, 1])] * 40, dt="f16", heads=(1, 1), D=64, seed=6)
    few.check(few.run(pa_lib))
    b.check(b.run(pa_lib))


def group_plan(ws, g):
    """Group g's record in the plan of the last shared step in the workspace ws."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    at = (256 + -(-(8 + 4097) * 4 // 256) * 256) // 4 + 8 + 16 * sms + 12 * g
    names = "r0 n table_row prefix f0 nt nut up base dual wfirst first".split()
    return dict(zip(names, ws.view(torch.int32)[at:at + 12].tolist()))


@pytest.mark.parametrize("rows,live,units,kw", [
    (256, [100, 103], 1, {}),                        # 4 units for all rows of the group
    (256, range(10), 1, {}),                         # a padded batch
    (256, range(200, 256), 1, {}),
    (256, range(100, 190), 2, {}),
    (256, [0, 255], 0, {}),                          # two rows would read the prefix four times
    (256, [0, 100, 180, 255], 0, {}),
    (256, [0, 100, 180, 200, 255], 4, {}),
    (130, [7, 9, 128], 0, dict(D=256)),              # 4 units of at most 32 rows
    (130, [1, 33, 34], 2, dict(D=256)),
    (200, [0, 70, 199], 0, dict(fp8=True)),
    (200, range(150, 199), 1, dict(fp8=True)),
])
def test_idle_rows_make_no_units(rows, live, units, kw, pa_lib):
    """Every unit reads the prefix: a batch that is mostly idle has no more of them
    than its live rows need."""
    b = Batch([(640, [5 + i % 7 for i in range(rows)])], heads=(8, 2), seed=rows,
              idle=[i for i in range(rows) if i not in live], **kw)
    ws = torch.zeros(pa_lib.decode_shared_workspace_size(b.B, 1, 8, 2, b.D), dtype=torch.uint8, device="cuda")
    try:
        pa_lib.set_workspace(ws)
        b.check(b.run(pa_lib))
    finally:
        pa_lib.set_workspace(None)
    p = group_plan(ws, 0)
    assert (p["nut"] if p["nt"] else 0) == units, p
    if units:
        assert (p["r0"], p["n"], p["table_row"]) == (min(live), max(live) - min(live) + 1, min(live))
    assert pa_lib.check_device_error() == 0


@pytest.mark.parametrize("B,heads,D", [(2, (8, 2), 128), (300, (2, 1), 64), (40, (16, 1), 256)])
def test_the_stated_workspace_serves_both_paths(B, heads, D, pa_lib):
    b = Batch([(320, [3 + i % 40 for i in range(B)])], dt="f16", heads=heads, D=D, seed=B)
    n = pa_lib.decode_shared_workspace_size(b.B, 1, *heads, D)
    ws = torch.empty(n + 256, dtype=torch.uint8, device="cuda")
    ws[n:] = 77
    try:
        pa_lib.set_workspace(ws[:n])
        for path in (1, 2, 0, 2, 1):
            pa_lib.set_shared_path(path)
            b.check(b.run(pa_lib), what=f"path {path}")
        assert (ws[n:] == 77).all()
    finally:
        pa_lib.set_workspace(None)


@pytest.mark.parametrize("tuning", [dict(max_ctas=1), dict(max_ctas=7, min_tiles=5), dict(min_tiles=1 << 20),
                                    dict(pool_permille=900, piece_tiles=1)])
def test_any_split_of_the_tails(tuning, pa_lib):
    bs = [Batch([(640, [9, 1, 70, 300, 1, 16, 17])], loose_after=(0, 33), seed=41),
          Batch([(1600, [40, 1, 60, 33]), (64, [1] * 30)], dt="f16", fp8=True, seed=42)]
    try:
        pa_lib.set_decode_tuning(**tuning)
        for b in bs:
            for window in (0, 700):
                b.check(b.run(pa_lib, window), window, f"{tuning} window {window}")
    finally:
        pa_lib.set_decode_tuning()
    assert pa_lib.check_device_error() == 0


def test_other_streams_and_shapes_in_turn(pa_lib):
    """Calls of several shapes on two streams at once, each with its own
    library workspace, and plain decodes between them."""
    bs = [Batch([(640, [9] * 40)], seed=14), Batch([(64, [2, 3]), (1600, [7, 8, 9])], seed=15)]
    streams = [torch.cuda.Stream() for _ in bs]
    torch.cuda.synchronize()
    args = [b.args() for b in bs]
    outs = [[], []]
    torch.cuda.synchronize()
    for rnd in range(6):
        for k, (b, s) in enumerate(zip(bs, streams)):
            with torch.cuda.stream(s):
                if rnd % 3 == 2:
                    outs[k].append(pa_lib.decode(*args[k][:5], **b.kw()))
                else:
                    outs[k].append(pa_lib.decode_shared(*args[k], **b.kw()))
    torch.cuda.synchronize()
    for k, b in enumerate(bs):
        for o in outs[k]:
            b.check(o)
    assert pa_lib.check_device_error() == 0


def test_steps_that_follow_one_another_without_a_gap(pa_lib):
    """A step may plan while the one before is still being joined: steps of very
    different shapes in one workspace, enqueued back to back, shared and plain."""
    bs = [Batch([(640, [9] * 40), (1600, [7, 8, 9])], seed=31), Batch([(16, [1])] * 2000 + [(32, [2] * 96)], heads=(2, 1), seed=32),
          Batch([(64, [2, 3])] * 30, dt="f16", seed=33), Batch([(2048, [5, 9, 300])], heads=(32, 8), seed=34)]
    args = [b.args() for b in bs]
    want = [b.run(pa_lib) for b in bs]
    for b, w in zip(bs, want):
        b.check(w)
    order = [0, 1, 0, 2, 3, 1, 3, 2, 0, 3, 1, 2] * 4
    outs = [torch.empty_like(bs[k].q) for k in order]
    plain = [torch.empty_like(bs[k].q) for k in order]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for rep in range(2):
        with torch.cuda.stream(s):
            for i, k in enumerate(order):
                pa_lib.decode_shared(*args[k], out=outs[i], stream=s, **bs[k].kw())
                if i % 3 == rep:
                    pa_lib.decode(*args[k][:5], out=plain[i], stream=s, **bs[k].kw())
        torch.cuda.synchronize()
        for i, k in enumerate(order):
            assert torch.equal(outs[i], want[k]), (rep, i, k)
            if i % 3 == rep:
                bs[k].check(plain[i])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        for i, k in enumerate(order):
            pa_lib.decode_shared(*args[k], out=outs[i], stream=s, **bs[k].kw())
    for _ in range(3):
        for o in outs:
            o.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        for i, k in enumerate(order):
            assert torch.equal(outs[i], want[k]), (i, k)
    assert pa_lib.check_device_error() == 0


def test_threads_calling_on_one_stream(pa_lib):
    """Steps of different shapes from two host threads on the same stream: their
    launches must not mix in the stream's one workspace."""
    import threading
    bs = [Batch([(640, [9] * 40)], seed=14), Batch([(64, [2, 3]), (1600, [7, 8, 9])], seed=15)]
    args = [b.args() for b in bs]
    s = torch.cuda.Stream()
    outs = [[torch.empty_like(b.q) for _ in range(60)] for b in bs]
    torch.cuda.synchronize()
    for b, a, o in zip(bs, args, outs):  # the workspace grows here
        pa_lib.decode_shared(*a, out=o[0], stream=s, **b.kw())
    errors = []

    def calls(k):
        try:
            for i, o in enumerate(outs[k]):
                if (i + k) % 5 == 4:
                    pa_lib.decode(*args[k][:5], out=o, stream=s, **bs[k].kw())
                else:
                    pa_lib.decode_shared(*args[k], out=o, stream=s, **bs[k].kw())
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=calls, args=(k,)) for k in range(2)]
    pa_lib.set_shared_path(2)
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    assert pa_lib.check_device_error() == 0
    for k, b in enumerate(bs):
        ref = torch.stack(outs[k]).float()
        b.check(outs[k][0])
        # the same values up to the order of summation
        assert (ref - ref[0]).abs().max() <= 2.0 ** -6


def test_a_thread_that_waits_on_its_stream_holds_up_no_other(pa_lib):
    """A host function keeps one stream from going on (for at most 20 s), a thread
    fills it with steps until its launches wait; a step on another stream, from
    another thread, is enqueued all the same, and releases the first."""
    import ctypes
    import threading
    import time
    cu = ctypes.CDLL("libcuda.so.1")
    b = Batch([(64, [3, 4])], seed=1)
    args = b.args()[:5]
    outs = [torch.empty_like(b.q) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for o, s in zip(outs, streams):
        pa_lib.decode(*args, out=o, stream=s, **b.kw())
    torch.cuda.synchronize()
    went_on, freed, count = threading.Event(), [], [0]
    hold = ctypes.CFUNCTYPE(None, ctypes.c_void_p)(lambda _: freed.append(went_on.wait(20)))
    assert cu.cuLaunchHostFunc(ctypes.c_void_p(streams[0].cuda_stream), hold, None) == 0

    def many():
        for _ in range(3000):
            pa_lib.decode(*args, out=outs[0], stream=streams[0], **b.kw())
            count[0] += 1

    def other():
        pa_lib.decode(*args, out=outs[1], stream=streams[1], **b.kw())
        went_on.set()

    threads = [threading.Thread(target=f) for f in (many, other)]
    threads[0].start()
    last = -1
    while count[0] != last and not freed:       # until it no longer gets on
        last = count[0]
        time.sleep(1)
    threads[1].start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert freed == [True]
    b.check(outs[0])
    b.check(outs[1])


def test_a_graph_outlives_a_larger_step_on_its_stream(pa_lib):
    small, large = Batch([(640, [9, 30, 1, 60])], seed=16), Batch([(512, [9] * 200)], heads=(16, 8), seed=17)
    args = small.args()
    out = torch.empty_like(small.q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        pa_lib.decode_shared(*args, out=out, **small.kw())
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            pa_lib.decode_shared(*args, out=out, **small.kw())
        for _ in range(3):
            large.check(large.run(pa_lib))      # the stream's workspace grows
            out.fill_(float("nan"))
            graph.replay()
            torch.cuda.synchronize()
            small.check(out)
    assert pa_lib.check_device_error() == 0


def test_a_workspace_that_grows_is_not_kept_twice(pa_lib):
    """A stream whose steps get larger holds what one with the large step alone holds;
    only one that a graph was captured with stays beside the larger one."""
    D, Hq, Hkv = 256, 16, 8
    kc = torch.zeros(4, Hkv, 16, D, dtype=torch.bfloat16, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    steps = []
    for B in (1024, 4096):
        q = torch.ones(B, Hq, D, dtype=torch.bfloat16, device="cuda")
        steps.append((q, kc, kc.clone(), torch.zeros(B, 2, **i32), torch.ones(B, **i32), torch.empty_like(q)))

    def call(k, s):
        *args, out = steps[k]
        pa_lib.decode(*args, num_kv_heads=Hkv, scale=1.0, block_size=16, out=out, stream=s)

    def held(ks, capture=False):
        s = torch.cuda.Stream()
        torch.cuda.synchronize()
        before = torch.cuda.mem_get_info()[0]
        for n, k in enumerate(ks):
            call(k, s)
            if capture and n == 0:
                torch.cuda.synchronize()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph, stream=s):
                    call(k, s)
                graphs.append(graph)
        torch.cuda.synchronize()
        return before - torch.cuda.mem_get_info()[0]

    graphs = []
    held([0, 1], capture=True)                  # whatever a first call sets up
    small, large = held([0]), held([1])
    slack = 4 << 20
    assert small > 2 * slack
    assert held([0, 1, 0, 1]) <= large + slack
    assert held([0, 1], capture=True) >= small + large - slack
    want = [o.clone() for *_, o in steps]
    for *_, o in steps:
        o.fill_(float("nan"))
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(steps[0][-1], want[0])


def test_captured_step_follows_new_lengths_and_groups(pa_lib):
    b = Batch([(640, [9, 30, 1, 60]), (640, [200, 3, 4, 5])], seed=16)
    args = b.args()
    out = torch.empty_like(b.q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        pa_lib.decode_shared(*args, out=out, **b.kw())  # workspace before the capture
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            pa_lib.decode_shared(*args, out=out, **b.kw())
    full = b.lens.copy()
    for lens, pre in ((full, b.prefix), (np.maximum(full - 1, 0), [320, 640]), (full * [1, 0, 1, 1, 0, 1, 1, 1], [640, 16]),
                      (full, [0, 0])):
        b.lens = np.asarray(lens, np.int32)
        args[4].copy_(torch.from_numpy(b.lens))
        args[5].copy_(torch.tensor(pre, dtype=torch.int32))
        out.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        b.check(out)
    assert pa_lib.check_device_error() == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_queries_written_by_the_call_just_before(fp8, pa_lib):
    """norm_rope_and_cache lets the shared step start before it has written q and the
    caches: steps in a row, in place in one buffer, without anything between them and
    in a graph, give what they give one by one."""
    b = Batch([(640, [9] * 40), (1600, [7, 8, 9])], dt="f16", fp8=fp8, seed=51)
    Hq, Hkv = b.heads
    D, n, steps = b.D, b.B, 8
    g = torch.Generator(device="cuda").manual_seed(1)
    rows = torch.randn(steps, n, Hq + 2 * Hkv, D, generator=g, device="cuda").to(torch.float16)
    last = torch.from_numpy(b.lens.astype(np.int64) - 1).cuda()
    _, kc, vc, tables, lens, prefix, starts = b.args()
    slots = tables.gather(1, (last // b.bs)[:, None])[:, 0].long() * b.bs + last % b.bs
    a = torch.arange(2000, dtype=torch.float64)[:, None] * 10000.0 ** -(torch.arange(0, D, 2, dtype=torch.float64) / D)
    cs = torch.cat([a.cos(), a.sin()], 1).float().cuda()
    position = last.int()
    w = torch.ones(D, dtype=torch.float16, device="cuda")
    kv = dict(kv_dtype="fp8" if fp8 else "auto", k_scale=b.ks, v_scale=b.vs)
    kw = dict(b.kw(), **kv)
    q = torch.empty(n, Hq, D, dtype=torch.float16, device="cuda")
    outs = torch.empty(steps, n, Hq, D, dtype=torch.float16, device="cuda")

    def run(between=lambda: None):
        for i in range(steps):
            x = rows[i]
            pa_lib.norm_rope_and_cache(*x.split([Hq, Hkv, Hkv], 1), kc, vc, slots, position, cs, q_weight=w, k_weight=w,
                                       out=q, **kv)
            between()
            pa_lib.decode_shared(q, kc, vc, tables, lens, prefix, starts, out=outs[i], **kw)
            between()

    run(torch.cuda.synchronize)
    want = outs.clone()
    for _ in range(5):
        outs.fill_(float("nan"))
        run()
        assert torch.equal(outs, want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            run()
    for _ in range(5):
        outs.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs, want)
    assert pa_lib.check_device_error() == 0


def test_a_whole_step_from_lengths_to_attention(pa_lib):
    """pool_extend, norm_rope_and_cache and decode_shared in one captured step,
    replayed: a batch that forks one prompt grows by one token a step, its new
    keys rotated at the positions the pool gave. The reference keeps its own
    keys and values per sequence in 64 bits, from the same 16-bit inputs."""
    B, P, Hq, Hkv, D, bs, steps = 6, 96, 8, 2, 128, 16, 20
    dt = torch.float16
    NB, MB = 64, 10
    g = torch.Generator(device="cuda").manual_seed(3)
    kc = torch.full((NB, Hkv, bs, D), float("nan"), dtype=dt, device="cuda")
    vc = torch.full((NB, Hkv, bs, D), float("nan"), dtype=dt, device="cuda")
    ids = shuffled_free_list(NB, 4)
    pre = [ids.pop() for _ in range(P // bs)]
    kp, vp = (torch.randn(P, Hkv, D, generator=g, device="cuda").to(dt) for _ in range(2))
    slots = (torch.tensor(pre, device="cuda")[:, None] * bs + torch.arange(bs, device="cuda")).reshape(-1)
    pa_lib.reshape_and_cache(kp, vp, kc, vc, slots)
    tables = torch.full((B, MB), -1, dtype=torch.int32, device="cuda")
    tables[:, :P // bs] = torch.tensor(pre, dtype=torch.int32, device="cuda")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    free = torch.tensor(ids + pre, dtype=torch.int32, device="cuda")
    state = i32(len(ids), 0)
    lens, new = i32(*[P] * B), i32(*[1] * B)
    new[4] = 0                                          # this one pauses
    T = B + 2
    slot, pos, start = (torch.zeros(n, dtype=d, device="cuda") for n, d in ((T, torch.int64), (T, torch.int32), (B + 1, torch.int32)))
    qkv = torch.zeros(T, (Hq + 2 * Hkv) * D, dtype=dt, device="cuda")
    q, k, v = qkv.view(T, Hq + 2 * Hkv, D).split([Hq, Hkv, Hkv], dim=1)
    w = [(1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(dt) for _ in range(2)]
    a = torch.arange(200, dtype=torch.float64)[:, None] * 10000.0 ** -(torch.arange(0, D, 2, dtype=torch.float64) / D)
    cs = torch.cat([a.cos(), a.sin()], 1).float().cuda()
    qr = torch.zeros(T, Hq, D, dtype=dt, device="cuda")
    out = torch.zeros(B, Hq, D, dtype=dt, device="cuda")
    prefix, groups = i32(P), i32(0, B)

    def step():
        pa_lib.pool_extend(tables, lens, new, free, state, block_size=bs, slot_mapping=slot, positions=pos, query_start=start)
        pa_lib.norm_rope_and_cache(q, k, v, kc, vc, slot, pos, cs, q_weight=w[0], k_weight=w[1], out=qr)
        # rows of the step to rows of the batch (a paused row keeps an older query)
        qb.copy_(qr[torch.minimum(start[:B], last)])
        pa_lib.decode_shared(qb, kc, vc, tables, lens, prefix, groups, num_kv_heads=Hkv, scale=D ** -0.5, block_size=bs, out=out)

    qb = torch.zeros(B, Hq, D, dtype=dt, device="cuda")
    last = torch.full((B,), T - 1, dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    keep = [x.clone() for x in (tables, lens, state, kc, vc)]
    with torch.cuda.stream(s):
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            step()
    for x, y in zip((tables, lens, state, kc, vc), keep):
        x.copy_(y)
    keys = [kp.double().cpu().numpy().copy() for _ in range(B)]
    vals = [vp.double().cpu().numpy().copy() for _ in range(B)]
    cs64 = cs.double().cpu().numpy()

    def turned(x, wt, p):
        x = x.double().cpu().numpy()
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6) * wt.double().cpu().numpy()
        c, sn = cs64[p, :D // 2], cs64[p, D // 2:]
        return np.concatenate([x[..., :D // 2] * c - x[..., D // 2:] * sn, x[..., D // 2:] * c + x[..., :D // 2] * sn], -1)

    for n in range(steps):
        qkv.copy_(torch.randn(qkv.shape, generator=g, device="cuda"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = out_f64(out)
        row = 0
        for b in range(B):
            if b == 4:
                assert lens[b].item() == P
                continue
            p = P + n
            keys[b] = np.concatenate([keys[b], turned(k[row], w[1], p)[None]])
            vals[b] = np.concatenate([vals[b], v[row].double().cpu().numpy()[None]])
            qq = turned(q[row], w[0], p).reshape(Hkv, Hq // Hkv, D)
            sc = np.einsum("kgd,tkd->kgt", qq, keys[b]) * D ** -0.5
            e = np.exp(sc - sc.max(-1, keepdims=True))
            e /= e.sum(-1, keepdims=True)
            ref = np.einsum("kgt,tkd->kgd", e, vals[b]).reshape(Hq, D)
            size = np.einsum("kgt,tkd->kgd", e, np.abs(vals[b])).reshape(Hq, D)
            # besides the bound above: q and k are themselves rounded, 2^-11 of each
            # element, so a score moves by at most 2^-10 sum |q k| scale (below 16
            # here), a weight by 2^-10 * 16 of itself against the others'
            bound = 2.0 ** -11 * np.abs(ref) + (2.0 ** -10 * 16 * 2 + 2.0 ** -8) * size + 1e-6
            assert (np.abs(got[b] - ref) <= bound).all(), (n, b)
            # and far closer on average
            assert np.abs(got[b] - ref).mean() <= 2e-3 * size.mean(), (n, b)
            row += 1
        assert start.tolist() == [0, 1, 2, 3, 4, 4, 5]
    assert pa_lib.check_device_error() == 0


FRESH = """
import sys
sys.path[:0] = [{root!r}, {root!r} + "/tests"]
import paged_kv_cache_267_gb300 as pa
from test_gpu_shared import Batch
pa.set_shared_path(2)
for n in {sizes}:
    b = Batch([(16, [1])] * (n - 1) + [(32, [2, 5, 1])], dt="f16", heads=(1, 1), D=64, seed=n)
    b.check(b.run(pa), what=str(n))
assert pa.check_device_error() == 0
"""


@pytest.mark.parametrize("sizes", [[853, 930, 931], [1023, 1024, 1025], [1109, 1110, 1111], [1117, 1118], [4000, 1111]])
def test_group_counts_whose_plan_just_fits_the_shared_memory(sizes, pa_lib):
    """In a process of their own: more groups before them would raise the limit."""
    r = subprocess.run([sys.executable, "-c", FRESH.format(root=ROOT, sizes=sizes)], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
