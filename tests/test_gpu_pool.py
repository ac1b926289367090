"""The block pool on the GPU (pa_pool_extend, pa_pool_release) against a plain
model of it, entry for entry: lengths from zero up, odd requests, sequences
that want nothing, padded rows, one CTA and many, in place and not, refused
steps, captured steps, and the host allocator's tables for the same requests.
"""
import subprocess
import sys

import numpy as np
import pytest
import torch

from conftest import ROOT, have_gpu
from workloads.layout import shuffled_free_list

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not have_gpu(), reason="needs a GPU")]


class Pool:
    """The plain model, on the host."""

    def __init__(self, B, MB, bs, NB, seed):
        self.B, self.MB, self.bs, self.NB = B, MB, bs, NB
        self.tables = np.full((B, MB), -1, np.int32)
        self.lens = np.zeros(B, np.int32)
        self.free = np.asarray(shuffled_free_list(NB, seed), np.int32)
        self.count = NB

    def blocks(self, n):
        return -(-n // self.bs)

    def extend(self, new, T):
        L = self.lens.astype(np.int64)
        new = np.asarray(new, np.int64)
        had, has = self.blocks(L), self.blocks(L + new)
        slots, pos = np.full(T, -1, np.int64), np.zeros(T, np.int32)
        start = np.zeros(self.B + 1, np.int32)
        if ((new < 0).any() or (L + new > self.MB * self.bs).any() or new.sum() > T
                or (has - had).sum() > self.count):
            return start, slots, pos
        t = 0
        for b in range(self.B):
            for j in range(had[b], has[b]):
                self.count -= 1
                self.tables[b, j] = self.free[self.count]
            p = np.arange(L[b], L[b] + new[b])
            slots[t:t + new[b]] = self.tables[b, p // self.bs].astype(np.int64) * self.bs + p % self.bs
            pos[t:t + new[b]] = p
            t += new[b]
            start[b + 1] = t
        self.lens = (L + new).astype(np.int32)
        return start, slots, pos

    def release(self, gone, shared=None):
        give = []
        for b in range(self.B):
            if gone[b]:
                keep = 0 if shared is None else int(shared[b]) // self.bs
                give += list(self.tables[b, keep:self.blocks(int(self.lens[b]))])
        if self.count + len(give) > self.NB:
            return
        self.free[self.count:self.count + len(give)] = give
        self.count += len(give)
        self.lens = np.where(np.asarray(gone) != 0, 0, self.lens).astype(np.int32)


class Gpu:
    """The same state on the GPU, and the calls."""

    def __init__(self, pa, m: Pool):
        self.pa, self.bs = pa, m.bs
        self.tables = torch.from_numpy(m.tables.copy()).cuda()
        self.lens = torch.from_numpy(m.lens.copy()).cuda()
        self.free = torch.from_numpy(m.free.copy()).cuda()
        self.state = torch.tensor([m.count, 0], dtype=torch.int32, device="cuda")

    def step(self, T):
        self.slots = torch.full((T,), 7, dtype=torch.int64, device="cuda")
        self.pos = torch.full((T,), 7, dtype=torch.int32, device="cuda")
        self.start = torch.full((self.tables.shape[0] + 1,), 7, dtype=torch.int32, device="cuda")

    def extend(self, new, in_place=True):
        kw = {} if in_place else dict(seq_lens_out=torch.full_like(self.lens, -9),
                                      pool_state_out=torch.full_like(self.state, -9))
        before = self.lens.clone(), self.state.clone()
        self.pa.pool_extend(self.tables, self.lens, new, self.free, self.state,
                            block_size=self.bs, slot_mapping=self.slots, positions=self.pos,
                            query_start=self.start, **kw)
        if not in_place:
            assert torch.equal(self.lens, before[0]) and torch.equal(self.state, before[1])
            self.lens, self.state = kw["seq_lens_out"], kw["pool_state_out"]

    def release(self, gone, shared=None, in_place=True):
        kw = {} if in_place else dict(seq_lens_out=torch.full_like(self.lens, -9),
                                      pool_state_out=torch.full_like(self.state, -9))
        self.pa.pool_release(self.tables, self.lens, gone, self.free, self.state,
                             block_size=self.bs, shared_tokens=shared, **kw)
        if not in_place:
            self.lens, self.state = kw["seq_lens_out"], kw["pool_state_out"]

    def same_state(self, m: Pool):
        assert self.state.tolist() == [m.count, 0]
        assert np.array_equal(self.lens.cpu().numpy(), m.lens)
        assert np.array_equal(self.tables.cpu().numpy(), m.tables)
        assert np.array_equal(self.free.cpu().numpy(), m.free)

    def same_step(self, want):
        start, slots, pos = want
        assert np.array_equal(self.start.cpu().numpy(), start)
        assert np.array_equal(self.slots.cpu().numpy(), slots)
        assert np.array_equal(self.pos.cpu().numpy(), pos)


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("B,bs,MB,top,T", [
    (1, 16, 4, 64, 64),            # one sequence, exactly its table
    (3, 16, 9, 40, 121),           # odd rows
    (64, 32, 20, 2, 64 * 2 + 5),   # a decode-like step with padded rows
    (257, 48, 11, 60, 257 * 60),   # a block size that is no power of two, several CTAs
    (4096, 16, 8, 30, 4096 * 30),  # the largest batch
    (5, 16, 700, 2300, 5 * 2300 + 3),
])
def test_rounds_of_requests_follow_the_model(B, bs, MB, top, T, in_place, pa_lib):
    rng = np.random.default_rng(B * 1000 + bs)
    NB = B * MB
    m = Pool(B, MB, bs, NB, seed=B + bs)
    g = Gpu(pa_lib, m)
    for rnd in range(5):
        room = np.minimum(top, MB * bs - m.lens)
        new = rng.integers(0, room + 1)
        new[rng.random(B) < 0.2] = 0
        if rnd == 0:
            new[0] = min(top, MB * bs)
        g.step(T)
        g.extend(i32(new), in_place)
        g.same_step(m.extend(new, T))
        g.same_state(m)
        gone = (rng.random(B) < 0.4).astype(np.int32) * (rnd + 1)  # any nonzero value
        shared = rng.integers(0, 3, B).astype(np.int32) * bs + 5
        g.release(i32(gone), i32(shared) if rnd % 2 else None, in_place)
        m.release(gone, shared if rnd % 2 else None)
        g.same_state(m)
    assert pa_lib.check_device_error() == 0


def test_rows_end_inside_every_vector_of_four(pa_lib):
    """Totals of 0..9 rows in tables of odd length, with unaligned views."""
    for total in range(10):
        for off in (0, 1):
            m = Pool(2, 3, 16, 6, seed=total)
            g = Gpu(pa_lib, m)
            T = 9
            big_s = torch.full((T + off,), 7, dtype=torch.int64, device="cuda")
            big_p = torch.full((T + off,), 7, dtype=torch.int32, device="cuda")
            g.slots, g.pos = big_s[off:], big_p[off:]
            g.start = torch.full((3,), 7, dtype=torch.int32, device="cuda")
            new = [total // 3, total - total // 3]
            g.extend(i32(new))
            g.same_step(m.extend(new, T))
            g.same_state(m)


def test_empty_batch_and_no_rows(pa_lib):
    m = Pool(0, 4, 16, 8, seed=1)
    g = Gpu(pa_lib, m)
    g.step(5)
    g.extend(i32([]))
    g.same_step((np.zeros(1, np.int32), np.full(5, -1), np.zeros(5, np.int32)))
    g.release(i32([]))
    g.same_state(m)
    m = Pool(2, 4, 16, 8, seed=1)
    g = Gpu(pa_lib, m)
    g.step(0)
    g.extend(i32([0, 0]))
    g.same_step(m.extend([0, 0], 0))
    g.same_state(m)


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("B,new,T,bit", [
    (3, [20, 33, 64], 200, "DEVERR_POOL"),        # 2 + 3 + 4 blocks, 8 are free
    (3, [5, -1, 5], 200, "DEVERR_TOKENS"),
    (3, [5, 6, 7], 17, "DEVERR_TOKENS"),          # 18 tokens, 17 rows
    (3, [5, 65, 7], 200, "DEVERR_SEQ_LEN"),       # a table holds 64
    (3, [5, 2**31 - 1, 7], 200, "DEVERR_SEQ_LEN"),
    (300, [16] * 300, 40000, "DEVERR_POOL"),      # several CTAs
])
def test_a_step_that_does_not_fit_changes_nothing(B, new, T, bit, in_place, pa_lib):
    m = Pool(B, 4, 16, 8, seed=3)
    g = Gpu(pa_lib, m)
    assert pa_lib.check_device_error() == 0
    g.step(T)
    g.extend(i32(new), in_place)
    g.same_step((np.zeros(B + 1, np.int32), np.full(T, -1), np.zeros(T, np.int32)))
    g.same_state(m)
    assert pa_lib.check_device_error() == getattr(pa_lib, bit)
    # the pool works on
    small = [1] * min(B, 8) + [0] * max(0, B - 8)
    g.step(T)
    g.extend(i32(small), in_place)
    g.same_step(m.extend(small, T))
    g.same_state(m)
    assert pa_lib.check_device_error() == 0


@pytest.mark.parametrize("which", ["seq_lens_out", "pool_state_out"])
@pytest.mark.parametrize("B", [5, 700])
def test_only_one_of_lengths_and_state_in_place(B, which, pa_lib):
    """The other one's input stays as it was, so it can be used again."""
    bs, MB, T = 16, 4, 64 * B
    new = [(7 * b) % 30 for b in range(B)]
    gone = [b % 3 == 0 for b in range(B)]
    g = Gpu(pa_lib, Pool(B, MB, bs, 4 * B, seed=5))
    for _ in range(3):
        m = Pool(B, MB, bs, 4 * B, seed=5)
        g.tables.fill_(-1)
        g.lens.copy_(torch.from_numpy(m.lens)), g.free.copy_(torch.from_numpy(m.free)), g.state.copy_(i32([m.count, 0]))
        for step in range(2):
            for call in ("extend", "release"):
                out = torch.full_like(g.lens if which == "seq_lens_out" else g.state, -9)
                before = g.lens.clone(), g.state.clone()
                g.step(T)
                if call == "extend":
                    pa_lib.pool_extend(g.tables, g.lens, i32(new), g.free, g.state, block_size=bs, slot_mapping=g.slots,
                                       positions=g.pos, query_start=g.start, **{which: out})
                    g.same_step(m.extend(new, T))
                else:
                    pa_lib.pool_release(g.tables, g.lens, i32(gone), g.free, g.state, block_size=bs, **{which: out})
                    m.release(gone)
                if which == "seq_lens_out":
                    assert torch.equal(g.lens, before[0])
                    g.lens = out
                else:
                    assert torch.equal(g.state, before[1])
                    g.state = out
                g.same_state(m)
    assert pa_lib.check_device_error() == 0


def test_release_beyond_the_free_list_and_bad_lengths_change_nothing(pa_lib):
    m = Pool(2, 4, 16, 8, seed=3)
    m.extend([40, 40], 80)
    g = Gpu(pa_lib, m)
    g.state[0] = 5     # six blocks are in use, the list has room for three more
    g.release(i32([1, 1]))
    assert pa_lib.check_device_error() == pa_lib.DEVERR_POOL
    assert g.state.tolist() == [5, 0] and g.lens.tolist() == [40, 40]
    g.state[0] = m.count
    for bad in (-1, 65):
        g.lens[1] = bad
        g.release(i32([1, 1]))
        assert pa_lib.check_device_error() == pa_lib.DEVERR_SEQ_LEN
        assert g.state.tolist() == [m.count, 0] and g.lens.tolist() == [40, bad]
    g.lens[1] = 40
    g.release(i32([1, 1]))
    m.release([1, 1])
    g.same_state(m)
    assert pa_lib.check_device_error() == 0


def test_bad_ids_are_flagged_and_get_no_slot(pa_lib):
    m = Pool(2, 4, 16, 8, seed=3)
    g = Gpu(pa_lib, m)
    g.free[7] = 8       # popped first, by sequence 0
    g.step(40)
    g.extend(i32([20, 16]))
    assert pa_lib.check_device_error() == pa_lib.DEVERR_BLOCK_ID
    s = g.slots.tolist()
    f = m.free
    assert s[:16] == [-1] * 16 and s[16:20] == [f[6] * 16 + i for i in range(4)]
    assert s[20:36] == [f[5] * 16 + i for i in range(16)] and s[36:] == [-1] * 4
    assert g.tables[0, :2].tolist() == [8, f[6]] and g.lens.tolist() == [20, 16]


def test_tables_equal_the_host_allocators(pa_lib):
    bs, NB, seed = 16, 200, 77
    lens = [1, 16, 17, 300, 0, 48, 1000]
    host = pa_lib.BlockAllocator(NB, bs, seed)
    ids = [host.add(n) for n in lens]
    m = Pool(len(lens), 70, bs, NB, seed)
    g = Gpu(pa_lib, m)
    g.step(sum(lens))
    g.extend(i32(lens))
    tables, want = host.fill_tables(ids, 70)
    assert np.array_equal(g.tables.cpu().numpy(), tables)
    assert g.lens.tolist() == want.tolist()
    assert g.state[0].item() == host.num_free()


def test_captured_steps_replay_in_place(pa_lib):
    """A decode loop's growth as one graph: every replay adds one token."""
    B, bs, MB = 37, 16, 6
    m = Pool(B, MB, bs, B * MB, seed=9)
    start = np.random.default_rng(0).integers(0, 40, B)
    m.extend(start, int(start.sum()))
    g = Gpu(pa_lib, m)
    new = torch.ones(B, dtype=torch.int32, device="cuda")
    g.step(B + 3)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            g.extend(new)
    for _ in range(40):
        graph.replay()
        torch.cuda.synchronize()
        g.same_step(m.extend([1] * B, B + 3))
        g.same_state(m)
    assert pa_lib.check_device_error() == 0


FRESH = """
import sys
sys.path[:0] = [{root!r}, {root!r} + "/tests"]
import numpy as np
import paged_kv_cache_267_gb300 as pa
from test_gpu_pool import Gpu, Pool, i32
for B in {sizes}:
    m = Pool(B, 2, 16, 2 * B, seed=B)
    g = Gpu(pa, m)
    new = np.arange(B) % 19
    g.step(int(new.sum()) + 3)
    g.extend(i32(new))
    g.same_step(m.extend(new, int(new.sum()) + 3))
    g.same_state(m)
    gone = np.arange(B) % 3 == 0
    g.release(i32(gone))
    m.release(gone)
    g.same_state(m)
assert pa.check_device_error() == 0
"""


@pytest.mark.parametrize("sizes", [[3400], [4077, 4078], [4079, 4095], [4096, 3413, 4079]])
def test_batches_whose_prefixes_just_fit_the_shared_memory(sizes, pa_lib):
    """In a process of their own: a larger batch before them would raise the limit."""
    r = subprocess.run([sys.executable, "-c", FRESH.format(root=ROOT, sizes=sizes)], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
