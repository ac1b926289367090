"""Attention of ragged steps (pa_prefill_packed, pa_decode_tree) against their
definition in 64 bits.

Tolerances, per element: with A the softmax-weighted sum of |V|, the weights are rounded
once to the products' 16-bit type (u_p A: 2^-8 for bf16 caches, 2^-11 else) and the
output once to its own (u_o |out|); scores and sums are held in fp32 (a score of up to
2^6 is off by less than 2^-15 after D products, which the weight of 2^-14 A covers), and
an f16 output or weight may be subnormal (2^-25).
"""
import math

import pytest
import torch

import paged_kv_cache_267_gb300 as pa

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def values(cache, scale, fp8):
    return (cache.view(torch.float8_e4m3fn).double() if fp8 else cache.double()) * scale


class Step:
    """A ragged step over a shuffled pool; whatever no sequence holds is NaN."""

    def __init__(self, new, ctx, Hq=8, Hkv=2, D=128, bs=16, dtype=torch.bfloat16, fp8=False, pad=0, seed=0, tree=False,
                 scale=None, spread=1.0, wide=0, q_gap=0, lens=None):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.new, self.bs, self.fp8, self.Hkv, self.dtype = new, bs, fp8, Hkv, dtype
        self.lens = [n + c for n, c in zip(new, ctx)] if lens is None else lens
        B = len(new)
        self.starts = [0]
        for n in new:
            self.starts.append(self.starts[-1] + n)
        T = self.starts[-1] + pad
        rows = torch.randn(T, Hq * D + q_gap, generator=g, device="cuda").mul_(spread).to(dtype)
        self.q = rows[:, q_gap // 16 * 8: q_gap // 16 * 8 + Hq * D].unflatten(1, (Hq, D))
        width = max(1, max((-(-x // bs) for x in self.lens), default=1)) + wide
        used = [-(-max(x, 0) // bs) for x in self.lens]
        pool = sum(used) + 5
        ids = torch.randperm(pool, generator=g, device="cuda").int()
        tables = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
        nan = 0x7F if fp8 else float("nan")
        cache = dict(device="cuda", dtype=torch.uint8 if fp8 else dtype)
        self.kc, self.vc = (torch.full((pool, Hkv, bs, D), nan, **cache) for _ in range(2))
        self.k_scale, self.v_scale = (0.03125, 0.02) if fp8 else (1.0, 1.0)
        self.k, self.v = [], []
        at = 0
        for b, L in enumerate(self.lens):
            blocks = ids[at: at + used[b]].long()
            at += used[b]
            tables[b, : used[b]] = blocks.int()
            pair = []
            for c, s in ((self.kc, self.k_scale), (self.vc, self.v_scale)):
                x = torch.randn(max(L, 0), Hkv, D, generator=g, device="cuda")
                x = (x / s).to(torch.float8_e4m3fn).view(torch.uint8) if fp8 else x.to(dtype)
                pos = torch.arange(max(L, 0), device="cuda")
                c[blocks[pos // bs], :, pos % bs] = x
                pair.append(x)
            self.k.append(pair[0])
            self.v.append(pair[1])
        self.tables = tables
        self.scale = D ** -0.5 if scale is None else scale
        self.mask = None
        if tree:
            bits = []
            for n in new:
                for j in range(n):
                    up = int(torch.randint(0, 5, (1,), generator=g, device="cuda")) + 1
                    m = 1 << min(j, 63)
                    if up < 5 and j - up >= 0:
                        m |= bits[len(bits) - up]
                    bits.append(m)
            bits += [0] * pad
            self.mask = torch.tensor([b - (1 << 64) if b >> 63 else b for b in bits], dtype=torch.int64, device="cuda")

    def poke(self, b, pos, v=None, k=None, d=slice(None), head=slice(None)):
        """Other keys or values at a position (e4m3 codes for such caches)."""
        block = int(self.tables[b, pos // self.bs])
        for x, c, rows in ((k, self.kc, self.k), (v, self.vc, self.v)):
            if x is not None:
                c[block, head, pos % self.bs, d] = x
                rows[b][pos, head, d] = x

    def ints(self, x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    def run(self, window=0, out=None, **over):
        kw = dict(num_kv_heads=self.Hkv, scale=self.scale, block_size=self.bs, window=window,
                  kv_dtype="fp8" if self.fp8 else "auto", k_scale=self.k_scale, v_scale=self.v_scale, out=out)
        kw.update(over)
        args = [self.q, self.kc, self.vc, self.tables, self.ints(self.lens), self.ints(self.starts)]
        out = pa.prefill_packed(*args, **kw) if self.mask is None else pa.decode_tree(*args, self.mask, **kw)
        torch.cuda.synchronize()
        assert pa.check_device_error() == 0
        return out

    def attends(self, b, window):
        """[n, L] which positions each row attends to."""
        n, L = self.new[b], self.lens[b]
        j = torch.arange(L, device="cuda")[None, :]
        first = L - n
        if self.mask is None:
            p = first + torch.arange(n, device="cuda")[:, None]
            seen = j <= p
        else:
            m = self.mask[self.starts[b]: self.starts[b] + n, None]
            nb = min(n, 64)
            m = m & (-1 if nb == 64 else (1 << nb) - 1)
            p = first - 1 + ((m >> torch.arange(64, device="cuda")) & 1).sum(1, keepdim=True)
            d = j - first
            seen = (d < 0) | ((d < 64) & ((m >> d.clamp(0, 63)) & 1 == 1))
        if window > 0:
            cut = j >= p + 1 - window
            seen = seen & (cut if self.mask is None else cut | (j >= first))
        return seen

    def expect(self, window=0):
        """(out, A) in 64 bits, a sequence and KV head at a time."""
        T, Hq, D = self.q.shape
        G = Hq // self.Hkv
        out = torch.zeros(T, Hq, D, dtype=torch.float64, device="cuda")
        A = torch.zeros_like(out)
        for b, n in enumerate(self.new):
            if n == 0 or self.lens[b] <= 0:
                continue
            seen = self.attends(b, window)
            k, v = values(self.k[b], self.k_scale, self.fp8), values(self.v[b], self.v_scale, self.fp8)
            r = slice(self.starts[b], self.starts[b] + n)
            for h in range(self.Hkv):
                q = self.q[r, h * G: (h + 1) * G].double()
                s = torch.einsum("tgd,ld->tgl", q, k[:, h]) * self.scale
                s = s.masked_fill(~seen[:, None, :], -math.inf)
                w = torch.softmax(s, -1).masked_fill(~seen.any(1)[:, None, None], 0.0)
                vv = v[:, h]
                clean = torch.where(vv.isfinite(), vv, 0)
                o = torch.einsum("tgl,ld->tgd", w, clean)
                for i in (~vv.isfinite()).any(1).nonzero()[:, 0].tolist():  # only rows that attend to it
                    o = o + torch.where(seen[:, i, None, None], w[:, :, i, None] * torch.where(vv[i].isfinite(), 0, vv[i]), 0)
                out[r, h * G: (h + 1) * G] = o
                A[r, h * G: (h + 1) * G] = torch.einsum("tgl,ld->tgd", w, clean.abs())
        return out, A

    def check(self, window=0, out=None, got=None, **over):
        got = self.run(window, out, **over) if got is None else got
        ref, A = self.expect(window)
        n = self.starts[-1]
        up = U[torch.bfloat16 if self.dtype == torch.bfloat16 and not self.fp8 else torch.float16]
        tol = (up + 2.0 ** -14) * A + U[self.dtype] * ref.abs().nan_to_num(0, 0, 0) + 2.0 ** -24
        g, e = got[:n].double(), ref[:n]
        fin = e.isfinite()
        assert torch.equal(g.isnan(), e.isnan())
        assert torch.equal(g[~fin & ~e.isnan()], e[~fin & ~e.isnan()])
        err = ((g - e).abs() / tol[:n])[fin]
        assert err.numel() == 0 or err.max() <= 1, f"{err.max()} tolerances"
        return got


DIMS = [(64, False), (128, False), (256, False), (128, True), (256, True)]


@pytest.mark.parametrize("D,fp8", DIMS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_prompts(D, fp8, dtype):
    Step([1, 7, 64, 65, 130, 0, 33], [0] * 7, D=D, fp8=fp8, dtype=dtype, seed=1).check()


@pytest.mark.parametrize("D,fp8", DIMS)
def test_one_token(D, fp8):
    for ctx in (0, 1, 15, 16, 127, 128, 500):
        Step([1], [ctx], D=D, fp8=fp8, seed=ctx).check()


@pytest.mark.parametrize("D,fp8", DIMS)
@pytest.mark.parametrize("Hq,Hkv", [(8, 8), (6, 2), (16, 1), (10, 2), (24, 8)])
def test_heads(D, fp8, Hq, Hkv):
    Step([3, 50, 90], [70, 0, 200], Hq=Hq, Hkv=Hkv, D=D, fp8=fp8, seed=2).check()


@pytest.mark.parametrize("D,fp8", DIMS)
@pytest.mark.parametrize("window", [1, 16, 100, 1000])
def test_window(D, fp8, window):
    Step([40, 300, 1], [0, 250, 777], D=D, fp8=fp8, seed=3).check(window=window)


@pytest.mark.parametrize("D,fp8", DIMS)
def test_long_cache_split(D, fp8):
    """Few rows, long caches: units cut between many CTAs."""
    Step([4, 1], [9000, 3001], D=D, fp8=fp8, seed=4).check()


@pytest.mark.parametrize("D,fp8", DIMS)
def test_many_units(D, fp8):
    """More units than CTAs: whole units, dealt out."""
    Step([700, 1500, 33, 900], [0, 64, 500, 0], Hq=32, Hkv=8, D=D, fp8=fp8, seed=5).check()


@pytest.mark.parametrize("D,fp8", DIMS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_tree(D, fp8, dtype):
    Step([1, 7, 64, 33, 0, 5], [0, 100, 513, 40, 9, 2000], D=D, fp8=fp8, dtype=dtype, seed=6, tree=True).check()


@pytest.mark.parametrize("D,fp8", DIMS)
@pytest.mark.parametrize("window", [64, 100, 1000])
def test_tree_window(D, fp8, window):
    Step([20, 64, 1], [0, 250, 777], Hq=24, Hkv=8, D=D, fp8=fp8, seed=7, tree=True).check(window=window)


# ---------------------------------------------------- how the work is cut and dealt out

@pytest.mark.parametrize("D,fp8", DIMS)
def test_planned_whole(D, fp8):
    """More sequences than a warp plans, more pairs than CTAs: whole pairs, dealt out."""
    Step([70, 1, 0, 129, 256, 3, 64, 65] * 5, [0, 500, 0, 64, 0, 9, 1, 300] * 5, Hq=32, Hkv=8, D=D, fp8=fp8, seed=8).check()


@pytest.mark.parametrize("D,fp8", DIMS)
def test_planned_split(D, fp8):
    """One long sequence among many short ones: cut between CTAs by the plan kernel."""
    Step([1] * 20 + [90] + [2] * 20, [3] * 20 + [6000] + [17] * 20, Hq=8, Hkv=1, D=D, fp8=fp8, seed=9).check()


def test_more_units_than_a_block_plans():
    """Several passes of the plan kernel over units and over sequences, whole and cut."""
    Step([3, 1, 0, 2] * 400, [5, 0, 0, 40] * 400, Hq=4, Hkv=2, D=64, seed=10).check()
    Step([1] * 1500 + [40], [2] * 1500 + [30000], Hq=1, Hkv=1, D=64, bs=64, seed=11).check()
    Step([1100 * 64 + 7], [0], Hq=2, Hkv=1, D=64, bs=64, dtype=torch.float16, seed=12).check(window=100)


@pytest.mark.parametrize("bs", [16, 48, 128, 1024])
def test_block_sizes(bs):
    Step([100, 1, 17], [333, 1025, 0], bs=bs, seed=13).check()
    Step([30, 1, 17], [333, 1025, 0], bs=bs, seed=13, tree=True).check()


def test_same_bits_again():
    """Results depend on nothing but the inputs: whole, split and small steps."""
    for st in (Step([700] * 20, [0] * 20, Hq=32, Hkv=8, seed=14), Step([5, 9], [20000, 333], seed=14),
               Step([1] * 40 + [64], [5] * 40 + [9000], seed=14)):
        a = st.run()
        for _ in range(3):
            assert torch.equal(st.run(), a)


def test_as_the_chunk_step():
    """Equal numbers of queries: what pa_prefill_chunk gives, up to its weights' rounding."""
    st = Step([64, 64, 64], [100, 0, 700], seed=15)
    st.check()
    out = pa.prefill_chunk(st.q.contiguous().view(3, 64, 8, 128), st.kc, st.vc, st.tables, st.ints(st.lens), num_kv_heads=2,
                           scale=st.scale, block_size=16)
    st.check(got=out.view(192, 8, 128))


# ------------------------------------------------------------- masks, odd values, layouts

@pytest.mark.parametrize("D,fp8", DIMS)
def test_values_that_are_not_attended(D, fp8):
    """Infinities and NaN in keys and values of later tokens, of tokens before a window and of
    other branches leave a row as it is; rows that attend to them have them."""
    odd = [0x7F] if fp8 else [float("inf"), float("-inf"), float("nan")]
    st = Step([100, 40, 1], [30, 200, 128], D=D, fp8=fp8, seed=16)
    for i, x in enumerate(odd):
        st.poke(0, 60 + 3 * i, v=x, d=slice(5, 9))       # seen by the later tokens of the same tile
        st.poke(1, 225 + i, v=x, head=1)
    st.poke(0, 129, v=odd[0], k=odd[-1])                 # the very last token
    st.poke(2, 128, k=odd[-1])
    st.check()
    st = Step([64, 9], [500, 0], D=D, fp8=fp8, seed=17)
    for i, x in enumerate(odd):
        st.poke(0, 430 + i, v=x, k=x)                    # leaves the window on the way
        st.poke(0, 520 + i, v=x, d=slice(0, 1))
    st.check(window=77)
    st = Step([64, 20, 3], [100, 1, 260], D=D, fp8=fp8, seed=18, tree=True)
    for i, x in enumerate(odd):
        st.poke(0, 100 + 11 * i, v=x, d=slice(2, 3))
        st.poke(1, 1 + 5 * i, v=x, head=0)
        st.poke(2, 17 + i, v=x, d=slice(0, 2))           # seen by all of this sequence's rows
    st.check()
    st.check(window=64)


@pytest.mark.parametrize("D,fp8", DIMS)
def test_rows_that_attend_to_nothing(D, fp8):
    # fewer tokens in the cache than new ones; none at all
    st = Step([10, 5, 40], [0, 0, 0], D=D, fp8=fp8, seed=19, lens=[4, 0, 40])
    out = st.run()
    assert not out[:6].any() and not out[10:15].any() and out[6:10].any()
    st = Step([6, 70], [0, 0], D=D, fp8=fp8, seed=20, tree=False)
    st.check()
    # trees: no bit and nothing cached; no bit and something cached; bits beyond the drafted tokens
    st = Step([4, 4, 64], [0, 50, 0], D=D, fp8=fp8, seed=21, tree=True)
    st.mask[1] = 0
    st.mask[5] = 0
    st.mask[3] = -1
    st.mask[6] = (1 << 40) | 1
    st.mask[20] = 0
    out = st.check()
    assert not out[1].any() and not out[20].any() and out[5].any()
    st.check(window=64)


def test_tree_of_many_tokens():
    """More than 64 drafted tokens: rows are computed against the first 64, and flagged."""
    st = Step([80, 3], [20, 5], seed=22, tree=True)
    with pytest.raises(AssertionError):
        st.run()
    kw = dict(num_kv_heads=2, scale=st.scale, block_size=16)
    out = pa.decode_tree(st.q, st.kc, st.vc, st.tables, st.ints(st.lens), st.ints(st.starts), st.mask, **kw)
    assert pa.check_device_error() == pa.DEVERR_QUERY
    st.check(got=out)


def test_padded_and_strided_rows():
    for dtype in (torch.bfloat16, torch.float16):
        st = Step([5, 130, 1], [3, 0, 200], dtype=dtype, pad=9, q_gap=48, seed=23)
        assert not st.q.is_contiguous()
        full = torch.full((st.q.shape[0], 8 * 128 + 16), 3.25, device="cuda", dtype=dtype)
        out = full[:, :1024].view(-1, 8, 128) if full.stride(0) == 1024 else full[:, :1024].unflatten(1, (8, 128))
        st.check(out=out)
        assert (full[:, 1024:] == 3.25).all() and (out[136:] == 3.25).all()
    st = Step([4, 3], [0, 100], pad=5, seed=24, tree=True)
    out = torch.full((12, 8, 128), 3.25, device="cuda", dtype=torch.bfloat16)
    st.check(out=out)
    assert (out[7:] == 3.25).all()
    # rows before the first sequence
    st = Step([6, 4], [10, 0], seed=25)
    q = torch.cat([torch.full((3, 8, 128), float("nan"), device="cuda", dtype=torch.bfloat16), st.q])
    out = torch.full((13, 8, 128), 3.25, device="cuda", dtype=torch.bfloat16)
    pa.prefill_packed(q, st.kc, st.vc, st.tables, st.ints(st.lens), st.ints([3, 9, 13]), num_kv_heads=2, scale=st.scale,
                      block_size=16, out=out)
    assert (out[:3] == 3.25).all()
    st.check(got=out[3:])


@pytest.mark.parametrize("D,fp8", DIMS)
def test_scales_and_large_scores(D, fp8):
    for scale, spread in ((-D ** -0.5, 1.0), (0.0, 1.0), (D ** -0.5, 8.0), (1e-30, 1.0)):
        Step([40, 3], [700, 150], D=D, fp8=fp8, scale=scale, spread=spread, seed=26).check()
    st = Step([20, 3], [700, 150], D=D, fp8=fp8, scale=-0.02, spread=3.0, seed=27, tree=True)
    st.check()


@pytest.mark.parametrize("D,fp8", [(128, False), (256, False), (128, True)])
def test_scores_that_grow(D, fp8):
    """Every tile beats the last one's reference: the accumulated output is rescaled each time."""
    st = Step([40, 2], [1500, 600], Hq=2, Hkv=1, D=D, fp8=fp8, scale=1.0, seed=28)
    st.q.zero_()
    st.q[:, :, 0] = 1.0
    for b, L in enumerate(st.lens):
        x = torch.arange(L, device="cuda") / L * 60
        x = (x / st.k_scale).clamp(max=448).to(torch.float8_e4m3fn).view(torch.uint8) if fp8 else x.bfloat16()
        pos = torch.arange(L, device="cuda")
        blocks = st.tables[b].long()[pos // 16]
        st.kc[blocks, 0, pos % 16, 0] = x
        st.k[b][:, 0, 0] = x
    st.check()


def test_offsets_beyond_32_bits():
    """Blocks whose elements lie more than 2^32 from the pool's start."""
    Hkv, bs, D = 8, 64, 128
    st = Step([70, 3], [100, 3000], Hq=8, Hkv=Hkv, bs=bs, seed=29)
    NB = (1 << 32) // (Hkv * bs * D) + 200
    at = NB - st.kc.shape[0]
    pools = []
    for c in (st.kc, st.vc):
        big = torch.empty(NB, Hkv, bs, D, device="cuda", dtype=torch.bfloat16)
        big[at:] = c
        pools.append(big)
    st.tables = torch.where(st.tables >= 0, st.tables + at, -1)
    st.kc, st.vc = pools
    st.check()
    st.mask = torch.tensor([1 << min(i, 63) for i in range(62)] * 2, device="cuda")[:73]
    st.new, st.starts = [60, 13], [0, 60, 73]
    st.check()


# --------------------------------------------------------------------- bad data, safe

def flagged(st, **over):
    a = dict(tables=st.tables, lens=st.ints(st.lens), starts=st.ints(st.starts))
    a.update(over)
    kw = dict(num_kv_heads=st.Hkv, scale=st.scale, block_size=16)
    args = (st.q, st.kc, st.vc, a["tables"], a["lens"], a["starts"])
    out = pa.prefill_packed(*args, **kw) if st.mask is None else pa.decode_tree(*args, st.mask, **kw)
    torch.cuda.synchronize()
    return out, pa.check_device_error()


@pytest.mark.parametrize("B", [3, 40])
@pytest.mark.parametrize("tree", [False, True])
def test_bad_starts_lengths_and_blocks(B, tree):
    st = Step([5] * B, [60] * B, seed=30, tree=tree)
    T = 5 * B
    good, bits = flagged(st)
    assert bits == 0
    s = list(st.starts)
    s[2], s[1] = s[1], s[2]                              # decreases: raised to the one before
    assert flagged(st, starts=st.ints(s))[1] == pa.DEVERR_QUERY
    s = list(st.starts)
    s[-1] = T + 9                                        # leaves [0, T]: clamped
    out, bits = flagged(st, starts=st.ints(s))
    assert bits == pa.DEVERR_QUERY and torch.equal(out[: T - 5], good[: T - 5])
    s = [-7] + st.starts[1:]
    out, bits = flagged(st, starts=st.ints(s))
    assert bits == pa.DEVERR_QUERY and torch.equal(out, good)
    assert flagged(st, starts=st.ints([2 ** 31 - 1] * (B + 1)))[1] == pa.DEVERR_QUERY
    assert flagged(st, starts=st.ints([-2 ** 31] * (B + 1)))[1] == pa.DEVERR_QUERY
    n = list(st.lens)
    n[1] = 2 ** 31 - 1
    assert flagged(st, lens=st.ints(n))[1] & pa.DEVERR_SEQ_LEN
    n[1] = -5
    out, bits = flagged(st, lens=st.ints(n))
    assert bits == pa.DEVERR_SEQ_LEN and not out[5:10].any() and torch.equal(out[:5], good[:5])
    t = st.tables.clone()
    t[0, 1], t[1, 0] = 1 << 30, -9
    out, bits = flagged(st, tables=t)
    assert bits == pa.DEVERR_BLOCK_ID and torch.equal(out[10:], good[10:])


# ------------------------------------------------------------- streams, graphs, workspaces

def test_graph_replays_with_other_inputs():
    """Small, split and whole steps captured and replayed on new lengths and values."""
    for new, ctx in (([4, 3, 20], [900, 50, 0]), ([1] * 40, [3000] + [9] * 39), ([300] * 30, [0] * 30)):
        st = Step(new, ctx, Hq=32, Hkv=8, seed=31)
        other = Step(list(reversed(new)), list(reversed(ctx)), Hq=32, Hkv=8, seed=32)
        fixed = dict(q=st.q.clone(), kc=torch.zeros(max(st.kc.shape[0], other.kc.shape[0]), 8, 16, 128, device="cuda", dtype=torch.bfloat16))
        fixed["vc"] = fixed["kc"].clone()
        width = max(st.tables.shape[1], other.tables.shape[1])
        fixed["tables"] = torch.full((len(new), width), -1, device="cuda", dtype=torch.int32)
        lens, starts, out = st.ints(st.lens), st.ints(st.starts), torch.empty_like(fixed["q"])

        def load(x):
            fixed["q"].copy_(x.q)
            fixed["kc"][: x.kc.shape[0]] = x.kc
            fixed["vc"][: x.vc.shape[0]] = x.vc
            fixed["tables"].fill_(-1)
            fixed["tables"][:, : x.tables.shape[1]] = x.tables
            lens.copy_(x.ints(x.lens))
            starts.copy_(x.ints(x.starts))

        def step():
            pa.prefill_packed(fixed["q"], fixed["kc"], fixed["vc"], fixed["tables"], lens, starts, num_kv_heads=8, scale=st.scale,
                              block_size=16, out=out)

        load(st)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
        for x in (other, st, other):
            load(x)
            out.fill_(7.0)
            graph.replay()
            torch.cuda.synchronize()
            x.check(got=out)
        assert pa.check_device_error() == 0


def test_two_streams_at_once():
    a, b = Step([3, 40], [9000, 0], seed=33), Step([64, 1], [300, 4000], seed=34)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = []
    torch.cuda.synchronize()
    for _ in range(6):
        for st, stream in zip((a, b), streams):
            outs.append(pa.prefill_packed(st.q, st.kc, st.vc, st.tables, st.ints(st.lens), st.ints(st.starts), num_kv_heads=2,
                                          scale=st.scale, block_size=16, stream=stream))
    torch.cuda.synchronize()
    for i, st in enumerate((a, b)):
        st.check(got=outs[i])
        for o in outs[i::2]:
            assert torch.equal(o, outs[i])


def test_workspace_of_the_caller():
    st = Step([4, 1], [9000, 3001], seed=35)
    want = st.run()
    n = pa.packed_workspace_size(5, 2, 8, 2, 128)
    buf = torch.empty(n, dtype=torch.uint8, device="cuda")
    try:
        pa.set_workspace(buf)
        assert torch.equal(st.run(), want)
        # a decode step in the same workspace, before and after
        kw = dict(num_kv_heads=2, scale=st.scale, block_size=16)
        q = st.q[:2].contiguous()
        big = torch.empty(max(n, pa.workspace_size(2, 8, 2, 128)), dtype=torch.uint8, device="cuda")
        pa.set_workspace(big)
        d0 = pa.decode(q, st.kc, st.vc, st.tables, st.ints(st.lens), **kw)
        for _ in range(3):
            assert torch.equal(st.run(), want)
            d1 = pa.decode(q, st.kc, st.vc, st.tables, st.ints(st.lens), **kw)
        torch.testing.assert_close(d0, d1, rtol=2.0 ** -7, atol=1e-3)
        pa.set_workspace(torch.empty(4096, dtype=torch.uint8, device="cuda"))
        with pytest.raises(pa.PAError, match="workspace too small"):
            st.run()
    finally:
        pa.set_workspace(None)


def test_nothing_to_do():
    st = Step([0, 0], [0, 0], pad=3, seed=36)
    out = torch.full((3, 8, 128), 2.5, device="cuda", dtype=torch.bfloat16)
    st.run(out=out)
    assert (out == 2.5).all()
    st = Step([0], [0], seed=37)
    n0 = pa.launch_count()
    assert st.run().numel() == 0 and pa.launch_count() == n0


@pytest.mark.parametrize("B", [1365, 2700, 4096])
def test_large_batches(B):
    """Batches around and at the most, whose lists the plan keeps in shared memory."""
    new = [(7 * b) % 4 for b in range(B)]
    Step(new, [(5 * b) % 23 for b in range(B)], Hq=2, Hkv=1, D=64, seed=38).check()
    Step(new, [(5 * b) % 23 for b in range(B)], Hq=2, Hkv=1, D=64, seed=38, tree=True).check()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D", [128, 256])
def test_query_ranges_on_an_e4m3_cache(D, dtype):
    """Rows of small and large values side by side (up to 2^27: f16 has infinities there), of
    subnormal ones, zeros, NaN. Next to a row's largest magnitude m an element may be off by
    2^-17 m, and so a score by 2^-17 m sum |k| scale, a weight by twice that of its own value."""
    st = Step([70, 9, 33], [40, 300, 0], D=D, fp8=True, dtype=dtype, seed=39)
    g = torch.Generator(device="cuda").manual_seed(40)
    T, Hq = st.q.shape[:2]
    small = torch.exp2(-24 * torch.rand(T, Hq, D, generator=g, device="cuda"))
    sign = torch.where(torch.rand(T, Hq, D, generator=g, device="cuda") < 0.5, -1.0, 1.0)
    row = torch.exp2(-torch.arange(T, device="cuda").float() % 26)[:, None, None]
    st.q = (sign * small * 4 * row).to(dtype)
    st.q[3] = 0
    st.q[5] = torch.finfo(dtype).smallest_normal / 4
    st.q[7, 0, 5] = float("inf")
    st.q[8, 1, 6] = float("nan")
    st.q[9, 2, 7] = float("-inf")
    out, (ref, A) = st.run().double(), st.expect()
    bad = ~st.q.isfinite().all(-1)
    assert bad.sum() >= 3 and out[bad].isnan().all() and ref[bad].isnan().all()
    ks = max(float(values(k, st.k_scale, True).abs().sum(-1).max()) for k in st.k)
    ds = st.scale * ks * 2.0 ** -17 * st.q.double().abs().amax(-1, keepdim=True)
    tol = (2.0 ** -11 + 2.0 ** -14 + 2 * ds) * A + U[dtype] * ref.abs() + 2.0 ** -24
    err = ((out - ref).abs() / tol)[~bad]
    assert err.max() <= 1, err.max()
