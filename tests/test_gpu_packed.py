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
