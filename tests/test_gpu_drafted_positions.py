"""Drafted steps with the positions of a tree: siblings share a place in the sequence, so a
drafted token is rotated for the place behind its ancestors, not for its row's. Then the
accepted path is, in the cache and in the outputs, what the same tokens give one after the
other."""
import math

import pytest
import torch

import paged_kv_cache_267_gb300 as pa
from test_gpu_ragged_steps import BS, D, HKV, HQ, Server, ints

pytestmark = pytest.mark.gpu


class TreeServer(Server):
    """`back`: a drafted row's ancestors less its place among the drafted rows (else 0)."""

    def __init__(self, *args, **kw):
        super().__init__(*args, **kw)
        self.back = torch.zeros(self.rows, device="cuda", dtype=torch.int32)

    def project(self, new, x=None):
        super().project(new)
        self.back.zero_()
        if x is not None:
            self.x.zero_()
            self.x[: x.shape[0]] = x

    def grow(self):
        pa.pool_extend(self.tables, self.lens, self.new, self.free, self.state, block_size=BS, slot_mapping=self.slots,
                       positions=self.positions, query_start=self.starts)
        self.positions.add_(self.back)
        q, k, v = self.x.view(self.rows, -1, D).split([HQ, HKV, HKV], 1)
        pa.norm_rope_and_cache(q, k, v, self.kc, self.vc, self.slots, self.positions, self.cos_sin, q_weight=self.weight,
                               k_weight=self.weight, out=self.q)

    def draft(self, new):
        masks, kept = super().draft(new)
        self.depths = [((m[:, None] >> torch.arange(64, device="cuda")) & 1).sum(1) - 1 for m in masks]
        back = torch.cat([d - torch.arange(d.numel(), device="cuda") for d in self.depths])
        self.back[: back.numel()] = back
        return masks, kept

    def rows_of(self, cache, b, n):
        pos = torch.arange(n, device="cuda")
        return cache[self.tables[b].long()[pos // BS], :, pos % BS]

    def expect(self, new, masks=None, kept=None):
        r = 0
        for b, n in enumerate(new):
            K, V = self.model[b]
            L = K.shape[0]
            if n:
                x = self.x[r: r + n].view(n, -1, D).double()
                j = torch.arange(n, device="cuda")
                p = L + (j if masks is None else self.depths[b])
                q, k, v = x.split([HQ, HKV, HKV], 1)
                q = self.rotated(q, p).bfloat16().double()
                K = torch.cat([K, self.rotated(k, p).bfloat16().float()])
                V = torch.cat([V, v.float()])
                seen = torch.ones(n, L + n, dtype=torch.bool, device="cuda")
                seen[:, L:] = j[None] <= j[:, None] if masks is None else (masks[b][:, None] >> j) & 1 == 1
                s = torch.einsum("thgd,lhd->thgl", q.view(n, HKV, -1, D), K.double()) * D ** -0.5
                w = torch.softmax(s.masked_fill(~seen[:, None, None], -math.inf), -1)
                want = torch.einsum("thgl,lhd->thgd", w, V.double()).reshape(n, HQ, D)
                A = torch.einsum("thgl,lhd->thgd", w, V.double().abs()).reshape(n, HQ, D)
                # (as in the parent: q and k may be off by a step of bf16, a score by 2^-6)
                tol = (2.0 ** -8 + 2 * 2.0 ** -6) * A + 2.0 ** -8 * want.abs() + 1e-6
                err = ((self.out[r: r + n].double() - want).abs() / tol).max()
                assert err <= 1, f"request {b}: {err} tolerances"
                if kept is not None:
                    assert [int(d) for d in self.depths[b][kept[b]]] == list(range(len(kept[b])))
                    stay = list(range(L)) + [L + i for i in kept[b]]
                    K, V = K[stay], V[stay]
                self.model[b] = (K, V)
                r += n
            # every row in its place: values bit for bit; keys, rounded from fp32 here and from
            # 64 bits there, within one step of bf16 (2^-7) and fp32's error of the sum of two
            # products of at most 2^4 (2^-18)
            assert torch.equal(self.rows_of(self.vc, b, V.shape[0]).float(), V)
            off = (self.rows_of(self.kc, b, K.shape[0]).float() - K).abs()
            assert (off <= 2.0 ** -7 * K.abs() + 2.0 ** -18).all()
        torch.cuda.synchronize()
        assert pa.check_device_error() == 0
        assert self.lens.tolist() == [k.shape[0] for k, _ in self.model]
        used = sum(-(-k.shape[0] // BS) for k, _ in self.model)
        assert self.state.tolist() == [self.NB - used, 0]


def test_drafted_steps_against_the_model():
    s = TreeServer(B=5, NB=120, MB=40, rows=420, seed=11)
    new = [100, 1, 0, 257, 33]
    s.project(new)
    s.prompt_step()
    s.expect(new)
    for new in ([8, 8, 8, 8, 8], [64, 1, 0, 17, 30], [5, 0, 0, 0, 64], [16, 16, 16, 16, 16]):
        s.project(new)
        masks, kept = s.draft(new)
        s.tree_step()
        s.expect(new, masks, kept)
    new = [1] * 5
    s.project(new)
    s.grow()
    s.out[:5] = pa.decode(s.q[:5], s.kc, s.vc, s.tables, s.lens, num_kv_heads=HKV, scale=D ** -0.5, block_size=BS)
    s.expect(new)


def test_drafted_steps_as_a_graph():
    s = TreeServer(B=4, NB=200, MB=50, rows=256, seed=12)
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
    for new in ([6, 6, 6, 6], [64, 3, 0, 20], [12, 64, 5, 64]):
        s.project(new)
        masks, kept = s.draft(new)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        s.expect(new, masks, kept)


def test_an_accepted_path_is_the_same_tokens_in_order():
    """Three rounds of trees beside a server that is given the accepted tokens alone: equal caches,
    bit for bit, and outputs that differ by the order of summation and the weights' rounding."""
    B = 4
    a, b = (TreeServer(B=B, NB=200, MB=50, rows=256, seed=s) for s in (13, 14))
    b.weight = a.weight
    new = [90, 16, 1, 140]
    a.project(new)
    b.project(new, a.x[: sum(new)])
    a.prompt_step()
    b.prompt_step()
    for new in ([40, 7, 64, 20], [5, 64, 1, 33], [64, 64, 16, 2]):
        a.project(new)
        masks, kept = a.draft(new)
        starts = [sum(new[:i]) for i in range(B)]
        rows = [starts[i] + j for i in range(B) for j in kept[i]]
        b.project([len(k) for k in kept], a.x[rows])
        a.tree_step()
        b.prompt_step()
        torch.cuda.synchronize()
        assert pa.check_device_error() == 0
        assert torch.equal(a.lens, b.lens)
        for i, n in enumerate(a.lens.tolist()):
            assert torch.equal(a.rows_of(a.kc, i, n), b.rows_of(b.kc, i, n))
            assert torch.equal(a.rows_of(a.vc, i, n), b.rows_of(b.vc, i, n))
        assert torch.equal(a.q[rows], b.q[: len(rows)])
        # each side's weights are rounded to bf16, by at most 2^-8 of a mean of |v|, which no |v|
        # exceeds, and its output once
        x, y = a.out[rows].double(), b.out[: len(rows)].double()
        top = max(float(a.rows_of(a.vc, i, n).abs().max()) for i, n in enumerate(a.lens.tolist()))
        assert ((x - y).abs() <= 2 * 2.0 ** -8 * top + 2 * 2.0 ** -8 * y.abs() + 1e-6).all()
