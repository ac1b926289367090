"""Compaction of many planes (a layer's K or V) a CTA, of caches without elements, and moves in
layers and blocks that lie more than 2^31 bytes from the caches' start."""
import pytest
import torch

import paged_kv_cache_267_gb300 as pa
from test_gpu_cache_moves import bits, caches, compact_model, ints

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [(0, 8, 2, 16, 64), (3, 8, 0, 16, 64), (3, 8, 2, 16, 0), (8, 0, 16, 64), (8, 2, 16, 0)])
def test_compact_without_elements(shape):
    """Lists with a gap over caches of no layers, no heads, no elements: nothing to move, nothing to flag."""
    kc, vc = (torch.empty(shape, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    tokens = ints([-1, -1])
    args = (ints([20, 30]), ints([0, 6, 12]), ints([[1, 3], [0, 5]]), ints([2, 2]))
    lens = pa.compact_cache(kc, vc, ints([[1, 2], [4, 5]]), *args, block_size=16, kept_tokens=tokens)
    assert pa.check_device_error() == 0
    assert lens.tolist() == [16, 26] and tokens.tolist() == [16, 32]
    # a list or a table that is wrong is flagged all the same
    lens = pa.compact_cache(kc, vc, ints([[1, 2], [4, 5]]), ints([20, 30]), ints([0, 6, 12]), ints([[3, 1], [0, 5]]), ints([2, 2]),
                            block_size=16)
    assert pa.check_device_error() == pa.DEVERR_QUERY and lens.tolist() == [20, 26]
    lens = pa.compact_cache(kc, vc, ints([[1, 8], [4, 5]]), *args, block_size=16)
    assert pa.check_device_error() == pa.DEVERR_BLOCK_ID and lens.tolist() == [16, 26]


def test_compact_in_an_empty_pool():
    """No blocks: every entry of a table is outside of the pool."""
    kc, vc = (torch.empty(0, 2, 16, 64, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    lens = pa.compact_cache(kc, vc, ints([[0, 1]]), ints([20]), ints([0, 6]), ints([[1, 3]]), ints([2]), block_size=16)
    assert pa.check_device_error() == pa.DEVERR_BLOCK_ID and lens.tolist() == [16]
    lens = pa.compact_cache(kc, vc, ints([[-1, -1]]), ints([20]), ints([0, 6]), ints([[0, 1]]), ints([2]), block_size=16)
    assert pa.check_device_error() == 0 and lens.tolist() == [16]


@pytest.mark.parametrize("B,layers,Hkv,bs,D,dtype", [(256, 16, 1, 16, 64, torch.bfloat16),  # 3 of 32 planes a CTA, the last has 2
                                                     (300, 25, 3, 16, 64, torch.uint8),     # 6 of 50, the last has 2
                                                     (4096, 1, 1, 16, 64, torch.float16),   # both planes in one
                                                     (700, 40, 1, 16, 128, torch.uint8)])   # 23 of 80, the last has 11
def test_compact_many_planes(B, layers, Hkv, bs, D, dtype):
    """Lists of differing lengths, with and without gaps, against plain indexing, bit for bit."""
    g = torch.Generator(device="cuda").manual_seed(20)
    r = torch.Generator().manual_seed(21)
    new = torch.randint(0, 25, (B,), generator=r).tolist()
    ctx = torch.randint(0, 24, (B,), generator=r).tolist()
    kept = [sorted(torch.randperm(n, generator=r)[: int(torch.randint(0, n + 1, (1,), generator=r))].tolist()) for n in new]
    width = 3
    NB = B * width + 3
    table = torch.randperm(NB, generator=g, device="cuda")[: B * width].view(B, width)
    kc, vc = caches((layers, NB, Hkv, bs, D), dtype, g, gap=1 if layers > 1 else 0)
    # all moves at once: (sequence, from, to) of every kept token
    b, src, dst = (torch.tensor(x, device="cuda") for x in zip(*[(i, ctx[i] + k, ctx[i] + j) for i in range(B) for j, k in enumerate(kept[i])]))
    want = []
    for c in (kc, vc):
        w = bits(c).clone()
        w[:, table[b, dst // bs], :, dst % bs] = w[:, table[b, src // bs], :, src % bs].clone()
        want.append(w)
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    lists = ints([k + [-7] * (25 - len(k)) for k in kept])
    got = pa.compact_cache(kc, vc, table.int(), ints([n + c for n, c in zip(new, ctx)]), ints(starts), lists,
                           ints([len(k) for k in kept]), block_size=bs)
    assert pa.check_device_error() == 0
    assert got.tolist() == [c + len(k) for c, k in zip(ctx, kept)]
    for c, w in zip((kc, vc), want):
        assert torch.equal(bits(c), w)


def test_moves_beyond_32_bits():
    """Layers 2^31 bytes and more from the start, blocks 2^31 bytes from their layer's, and rows and
    blocks beside them as they were."""
    g = torch.Generator(device="cuda").manual_seed(22)
    bs, D = 16, 64
    NB = (1 << 20) + 70                                  # of 2 KB
    kc, vc = (torch.empty(3, NB, 1, bs, D, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    used = torch.tensor([0, 1, 5, 70, (1 << 19) + 3, (1 << 20) - 1, 1 << 20, (1 << 20) + 1, NB - 2, NB - 1], device="cuda")
    want = []
    for c in (kc, vc):
        w = torch.randn(3, used.numel(), 1, bs, D, generator=g, device="cuda").bfloat16()
        c[:, used] = w
        want.append(bits(w).clone())
    at = {int(x): i for i, x in enumerate(used.tolist())}
    pairs = [(NB - 1, 1), (5, (1 << 20) + 1), (70, 1 << 20)]
    pa.copy_blocks(kc, vc, ints(pairs))
    for w in want:
        for s, t in pairs:
            w[:, at[t]] = w[:, at[s]].clone()
    for c, w in zip((kc, vc), want):
        assert torch.equal(bits(c[:, used]), w)
    tables = [[NB - 2, (1 << 20) - 1], [0, (1 << 19) + 3]]
    pa.compact_cache(kc, vc, ints(tables), ints([32, 29]), ints([0, 20, 36]), ints([[1, 3, 19], [0, 14, 15]]), ints([3, 3]), block_size=bs)
    assert pa.check_device_error() == 0
    for w in want:
        compact_model(w, [at[t] for t in tables[0]], bs, 12, [1, 3, 19])
        compact_model(w, [at[t] for t in tables[1]], bs, 13, [0, 14, 15])
    for c, w in zip((kc, vc), want):
        assert torch.equal(bits(c[:, used]), w)
