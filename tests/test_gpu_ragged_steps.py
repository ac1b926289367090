"""Whole steps of ragged and drafted requests as a server runs them: tables grown on the
GPU, rows normalised, rotated and written, the attention of prompts and of drafted trees,
the accepted tokens moved together, the blocks behind them given back; enqueued, and
captured as one graph. Against a plain model that keeps every request's rows in a list."""
import math

import pytest
import torch

import paged_kv_cache_267_gb300 as pa

pytestmark = pytest.mark.gpu

HQ, HKV, D, BS = 8, 2, 128, 16


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Server:
    """B requests over a pool of blocks on the GPU, and their rows as the model knows them."""

    def __init__(self, B, NB, MB, rows, seed):
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.B, self.NB, self.rows = B, NB, rows
        self.kc, self.vc = (torch.full((NB, HKV, BS, D), float("nan"), device="cuda", dtype=torch.bfloat16) for _ in range(2))
        self.tables = torch.full((B, MB), -1, device="cuda", dtype=torch.int32)
        self.lens, self.kept_lens, self.scratch, self.tokens = (torch.zeros(B, device="cuda", dtype=torch.int32) for _ in range(4))
        self.free = torch.randperm(NB, generator=self.g, device="cuda").int()
        self.state = ints([NB, 0])
        self.starts = ints([0] * (B + 1))
        self.slots = torch.zeros(rows, device="cuda", dtype=torch.int64)
        self.positions = torch.zeros(rows, device="cuda", dtype=torch.int32)
        self.new, self.released = ints([0] * B), ints([1] * B)
        self.x = torch.zeros(rows, (HQ + 2 * HKV) * D, device="cuda", dtype=torch.bfloat16)
        self.q, self.out = (torch.zeros(rows, HQ, D, device="cuda", dtype=torch.bfloat16) for _ in range(2))
        self.mask = torch.zeros(rows, device="cuda", dtype=torch.int64)
        self.kept, self.count = ints([[0] * 64] * B), ints([0] * B)
        angle = torch.arange(4096, device="cuda", dtype=torch.float64)[:, None] * 1e4 ** (-torch.arange(0, D, 2, device="cuda") / D)
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float()
        self.weight = (1 + 0.2 * torch.randn(D, generator=self.g, device="cuda")).bfloat16()
        self.model = [(torch.zeros(0, HKV, D, device="cuda"), torch.zeros(0, HKV, D, device="cuda")) for _ in range(B)]

    def project(self, new):
        """This step's projected rows; returns them by request."""
        self.new.copy_(ints(new))
        self.x.copy_(torch.randn(self.x.shape, generator=self.g, device="cuda").bfloat16())

    def grow(self):
        pa.pool_extend(self.tables, self.lens, self.new, self.free, self.state, block_size=BS, slot_mapping=self.slots,
                       positions=self.positions, query_start=self.starts)
        q, k, v = self.x.view(self.rows, -1, D).split([HQ, HKV, HKV], 1)
        pa.norm_rope_and_cache(q, k, v, self.kc, self.vc, self.slots, self.positions, self.cos_sin, q_weight=self.weight,
                               k_weight=self.weight, out=self.q)

    def kw(self):
        return dict(num_kv_heads=HKV, scale=D ** -0.5, block_size=BS, out=self.out)

    def prompt_step(self):
        self.grow()
        pa.prefill_packed(self.q, self.kc, self.vc, self.tables, self.lens, self.starts, **self.kw())

    def tree_step(self):
        self.grow()
        pa.decode_tree(self.q, self.kc, self.vc, self.tables, self.lens, self.starts, self.mask, **self.kw())
        pa.compact_cache(self.kc, self.vc, self.tables, self.lens, self.starts, self.kept, self.count, block_size=BS,
                         seq_lens_out=self.kept_lens, kept_tokens=self.tokens)
        pa.pool_release(self.tables, self.lens, self.released, self.free, self.state, block_size=BS, shared_tokens=self.tokens,
                        seq_lens_out=self.scratch)
        self.lens.copy_(self.kept_lens)

    # ------------------------------------------------------------------ the model

    def rotated(self, x, p):
        y = x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt() * self.weight.double()
        c, s = self.cos_sin[p].double()[:, None].chunk(2, -1)
        a, b = y.chunk(2, -1)
        return torch.cat([a * c - b * s, b * c + a * s], -1)

    def expect(self, new, masks=None, kept=None):
        """Checks the step's outputs, then moves the model on."""
        r = 0
        for b, n in enumerate(new):
            K, V = self.model[b]
            if n == 0:
                continue
            L = K.shape[0]
            x = self.x[r: r + n].view(n, -1, D).double()
            p = torch.arange(L, L + n, device="cuda")
            q, k, v = x.split([HQ, HKV, HKV], 1)
            q = self.rotated(q, p).bfloat16().double()
            K = torch.cat([K, self.rotated(k, p).bfloat16().float()])
            V = torch.cat([V, v.float()])
            seen = torch.ones(n, L + n, dtype=torch.bool, device="cuda")
            j = torch.arange(n, device="cuda")
            seen[:, L:] = j[None] <= j[:, None] if masks is None else (masks[b][:, None] >> j) & 1 == 1
            s = torch.einsum("thgd,lhd->thgl", q.view(n, HKV, -1, D), K.double()) * D ** -0.5
            w = torch.softmax(s.masked_fill(~seen[:, None, None], -math.inf), -1)
            want = torch.einsum("thgl,lhd->thgd", w, V.double()).reshape(n, HQ, D)
            A = torch.einsum("thgl,lhd->thgd", w, V.double().abs()).reshape(n, HQ, D)
            # weights and outputs rounded to bf16; q and k may be off by a step of bf16 where the
            # norm's fp32 arithmetic lands beside the 64-bit value: a score (sums of |q k| up to
            # 4 sqrt(D), and few elements differ) by at most 2^-6
            tol = (2.0 ** -8 + 2 * 2.0 ** -6) * A + 2.0 ** -8 * want.abs() + 1e-6
            err = ((self.out[r: r + n].double() - want).abs() / tol).max()
            assert err <= 1, f"request {b}: {err} tolerances"
            if kept is not None:
                stay = list(range(L)) + [L + i for i in kept[b]]
                K, V = K[stay], V[stay]
            self.model[b] = (K, V)
            r += n
        torch.cuda.synchronize()
        assert pa.check_device_error() == 0
        assert self.lens.tolist() == [k.shape[0] for k, _ in self.model]
        used = sum(-(-k.shape[0] // BS) for k, _ in self.model)
        assert self.state.tolist() == [self.NB - used, 0]
        held = [i for b in range(self.B) for i in self.tables[b, : -(-self.model[b][0].shape[0] // BS)].tolist()]
        assert sorted(held + self.free[: self.NB - used].tolist()) == list(range(self.NB))

    def draft(self, new):
        """Random trees, and a path of each that is accepted."""
        masks, kept = [], []
        for n in new:
            bits, parent = [], []
            for j in range(n):
                up = int(torch.randint(0, 5, (1,), generator=self.g, device="cuda"))
                p = j - 1 - up if up < 4 and j - 1 - up >= 0 else -1
                parent.append(p)
                bits.append((bits[p] if p >= 0 else 0) | 1 << j)
            path, j = [], n - 1 - int(torch.randint(0, max(n // 2, 1), (1,), generator=self.g, device="cuda")) if n else -1
            while j >= 0:
                path.insert(0, j)
                j = parent[j]
            masks.append(torch.tensor([x - (1 << 64) if x >> 63 else x for x in bits], dtype=torch.int64, device="cuda"))
            kept.append(path)
        flat = torch.cat(masks)
        self.mask.zero_()
        self.mask[: flat.numel()] = flat
        self.kept.copy_(ints([k + [0] * (64 - len(k)) for k in kept]))
        self.count.copy_(ints([len(k) for k in kept]))
        return masks, kept


def test_prompts_then_drafted_steps():
    s = Server(B=5, NB=120, MB=40, rows=420, seed=1)
    for new in ([100, 1, 0, 257, 33], [3, 64, 16, 0, 1]):
        s.project(new)
        s.prompt_step()
        s.expect(new)
    for new in ([8, 8, 8, 8, 8], [64, 1, 0, 17, 30], [5, 0, 0, 0, 64], [16, 16, 16, 16, 16]):
        s.project(new)
        masks, kept = s.draft(new)
        s.tree_step()
        s.expect(new, masks, kept)
    # plain decode over what is left in the cache
    new = [1] * 5
    s.project(new)
    s.grow()
    s.out[:5] = pa.decode(s.q[:5], s.kc, s.vc, s.tables, s.lens, num_kv_heads=HKV, scale=D ** -0.5, block_size=BS)
    s.expect(new)


def test_drafted_steps_as_a_graph():
    s = Server(B=4, NB=200, MB=50, rows=256, seed=2)
    new = [90, 16, 1, 140]
    s.project(new)
    s.prompt_step()
    s.expect(new)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    new = [6, 6, 6, 6]
    s.project(new)
    masks, kept = s.draft(new)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        s.tree_step()
    torch.cuda.synchronize()
    s.expect(new, masks, kept)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        s.tree_step()
    for new in ([6, 6, 6, 6], [64, 3, 0, 20], [1, 1, 1, 1], [12, 64, 5, 64]):
        s.project(new)
        masks, kept = s.draft(new)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        s.expect(new, masks, kept)


def test_forked_requests_copy_their_partial_block():
    """The host allocator's copy-on-write, carried out by copy_blocks; both forks decode what they should."""
    host = pa.BlockAllocator(40, BS, 3)
    g = torch.Generator(device="cuda").manual_seed(3)
    kc, vc = (torch.randn(2, 40, HKV, BS, D, generator=g, device="cuda").bfloat16() for _ in range(2))
    a = host.add(50)
    forks = [host.fork(a) for _ in range(3)]
    pairs = [host.append(f, 1) for f in forks]
    assert all(x >= 0 and y >= 0 for x, y in pairs)
    before = kc.clone(), vc.clone()
    pa.copy_blocks(kc, vc, ints(pairs + [host.append(a, 1)]))
    for c, w in zip((kc, vc), before):
        for x, y in pairs:
            assert torch.equal(c[:, y], w[:, x])
    tables, lens = host.fill_tables([a, *forks], 8)
    tables, lens = torch.from_numpy(tables).cuda(), torch.from_numpy(lens).cuda()
    q = torch.randn(1, HQ, D, generator=g, device="cuda").bfloat16().expand(4, HQ, D).contiguous()
    for layer in range(2):
        out = pa.decode(q, kc[layer], vc[layer], tables, lens - 1, num_kv_heads=HKV, scale=D ** -0.5, block_size=BS)
        torch.testing.assert_close(out, out[:1].expand(4, HQ, D), rtol=0, atol=2.0 ** -8)
    assert pa.check_device_error() == 0
