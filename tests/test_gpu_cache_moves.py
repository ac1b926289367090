"""Block copies and compaction of accepted tokens (pa_copy_blocks, pa_compact_cache):
bit for bit what plain indexing gives, everything else in the caches as it was."""
import pytest
import torch

import paged_kv_cache_267_gb300 as pa

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16, torch.uint8]


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def bits(t):
    return t.view(torch.uint8)


def caches(shape, dtype, g, gap=0):
    """K and V caches of random bits; with a gap, layers that do not touch."""
    out = []
    for _ in range(2):
        full = list(shape)
        if gap:
            full[1] += gap
        x = torch.randint(0, 256, (*full[:-1], full[-1] * dtype.itemsize), generator=g, device="cuda", dtype=torch.uint8)
        x = x.view(dtype)
        out.append(x[:, : shape[1]] if gap else x)
    return out


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("Hkv,bs,D", [(8, 16, 128), (1, 16, 64), (5, 32, 256), (2, 1024, 128)])
@pytest.mark.parametrize("layers", [0, 1, 3])
def test_copy(dtype, Hkv, bs, D, layers):
    g = torch.Generator(device="cuda").manual_seed(1)
    NB = 23
    shape = (NB, Hkv, bs, D) if layers == 0 else (layers, NB, Hkv, bs, D)
    kc, vc = caches(shape, dtype, g, gap=2 if layers > 1 else 0)
    want = [bits(c).clone() for c in (kc, vc)]
    pairs = [(3, 7), (3, 8), (-1, 4), (5, -1), (22, 0), (11, 11), (6, 21)]
    for w in want:
        d = w if layers else w[None]
        for s, t in pairs:
            if s >= 0 and t >= 0:
                d[:, t] = d[:, s].clone()
    pa.copy_blocks(kc, vc, ints(pairs))
    assert pa.check_device_error() == 0
    for c, w in zip((kc, vc), want):
        assert torch.equal(bits(c), w)


def test_layers_in_turn():
    """K and V as every other layer of one tensor."""
    g = torch.Generator(device="cuda").manual_seed(11)
    pool = torch.randn(4, 2, 12, 2, 16, 64, generator=g, device="cuda").bfloat16()
    want = pool.clone()
    want[:, :, 5] = pool[:, :, 1]
    pa.copy_blocks(pool[:, 0], pool[:, 1], ints([(1, 5)]))
    assert torch.equal(pool, want)
    want[:, :, 7, :, 3] = pool[:, :, 7, :, 5]
    pa.compact_cache(pool[:, 0], pool[:, 1], ints([[2, 7]]), ints([24]), ints([0, 5]), ints([[2]]), ints([1]), block_size=16)
    assert torch.equal(pool, want)
    assert pa.check_device_error() == 0


def test_copy_beyond_the_pool():
    g = torch.Generator(device="cuda").manual_seed(2)
    kc, vc = caches((9, 2, 16, 64), torch.bfloat16, g)
    want = [bits(c).clone() for c in (kc, vc)]
    for w in want:
        w[1] = w[2]
    pa.copy_blocks(kc, vc, ints([(9, 3), (4, 1000000), (2, 1)]))
    assert pa.check_device_error() == pa.DEVERR_BLOCK_ID
    for c, w in zip((kc, vc), want):
        assert torch.equal(bits(c), w)


def test_copy_nothing():
    g = torch.Generator(device="cuda").manual_seed(2)
    kc, vc = caches((9, 2, 16, 64), torch.bfloat16, g)
    n0 = pa.launch_count()
    pa.copy_blocks(kc, vc, torch.empty(0, 2, dtype=torch.int32, device="cuda"))
    assert pa.launch_count() == n0


def compact_model(cache, table, bs, base, kept):
    """cache [layers, NB, Hkv, bs, bytes] after one sequence's move."""
    rows = [cache[:, table[(base + k) // bs], :, (base + k) % bs].clone() for k in kept]
    for i, r in enumerate(rows):
        cache[:, table[(base + i) // bs], :, (base + i) % bs] = r


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("Hkv,bs,D,layers", [(8, 16, 128, 0), (2, 32, 64, 1), (5, 16, 256, 3), (1, 64, 128, 2)])
def test_compact(dtype, Hkv, bs, D, layers):
    g = torch.Generator(device="cuda").manual_seed(3)
    new = [0, 1, 5, 16, 40, 64, 300, 3]
    ctx = [0, 15, 16, 3, 100, 0, 7, 31]
    kept = [[], [0], [1, 4], [0, 1, 2, 9], [3, 4, 5, 39], list(range(64)),
            sorted(torch.randperm(300, generator=torch.Generator().manual_seed(4))[:280].tolist()), []]
    B, M = len(new), max(len(k) for k in kept) + 1
    lens = [n + c for n, c in zip(new, ctx)]
    width = max(-(-x // bs) for x in lens) + 1
    NB = B * width + 3
    table = torch.randperm(NB, generator=g, device="cuda")[: B * width].view(B, width)
    shape = (NB, Hkv, bs, D) if layers == 0 else (layers, NB, Hkv, bs, D)
    kc, vc = caches(shape, dtype, g, gap=1 if layers > 1 else 0)
    want = [bits(c).clone() for c in (kc, vc)]
    for w in want:
        d = w if layers else w[None]
        for b in range(B):
            compact_model(d, table[b].tolist(), bs, ctx[b], kept[b])
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    pad = [k + [-7] * (M - len(k)) for k in kept]
    tokens = torch.full((B,), -1, dtype=torch.int32, device="cuda")
    got = pa.compact_cache(kc, vc, table.int(), ints(lens), ints(starts), ints(pad), ints([len(k) for k in kept]),
                           block_size=bs, kept_tokens=tokens)
    assert pa.check_device_error() == 0
    left = [c + len(k) for c, k in zip(ctx, kept)]
    assert got.tolist() == left
    assert tokens.tolist() == [-(-x // bs) * bs for x in left]
    for c, w in zip((kc, vc), want):
        assert torch.equal(bits(c), w)


@pytest.mark.parametrize("kept,count", [([2, 1], 2), ([1, 1], 2), ([0, 6], 2), ([-1, 2], 2), ([0, 1], 7), ([0, 1], -1), ([0, 1], 3)])
def test_compact_refuses_a_bad_list(kept, count):
    """A list that does not ascend inside the drafted tokens, or a count beyond it: the sequence stays."""
    g = torch.Generator(device="cuda").manual_seed(5)
    kc, vc = caches((8, 2, 16, 64), torch.bfloat16, g)
    want = [bits(c).clone() for c in (kc, vc)]
    for w in want:
        compact_model(w[None], [4, 5], 16, 14, [1, 3])
    lens = pa.compact_cache(kc, vc, ints([[1, 2], [4, 5]]), ints([20, 20]), ints([0, 6, 12]), ints([kept, [1, 3]]),
                            ints([count, 2]), block_size=16)
    assert pa.check_device_error() == pa.DEVERR_QUERY
    assert lens.tolist() == [20, 16]
    for c, w in zip((kc, vc), want):
        assert torch.equal(bits(c), w)


def test_compact_bad_blocks_and_lengths():
    """Table entries outside of the pool move nothing; a length outside of the tables is clamped."""
    g = torch.Generator(device="cuda").manual_seed(6)
    kc, vc = caches((8, 2, 16, 64), torch.float16, g)
    want = [bits(c).clone() for c in (kc, vc)]
    args = (ints([[1, 99], [-1, 3]]), ints([20, 20]), ints([0, 6, 12]), ints([[3, 5], [3, 5]]), ints([2, 2]))
    lens = pa.compact_cache(kc, vc, *args, block_size=16)
    assert pa.check_device_error() == pa.DEVERR_BLOCK_ID
    assert lens.tolist() == [16, 16]
    for c, w in zip((kc, vc), want):
        assert torch.equal(bits(c), w)
    lens = pa.compact_cache(kc, vc, ints([[1, 2]]), ints([50]), ints([0, 4]), ints([[0, 1]]), ints([2]), block_size=16)
    assert pa.check_device_error() == pa.DEVERR_SEQ_LEN
    assert lens.tolist() == [30]
    lens = pa.compact_cache(kc, vc, ints([[1, 2]]), ints([3]), ints([0, 4]), ints([[0, 1]]), ints([2]), block_size=16)
    assert pa.check_device_error() == pa.DEVERR_QUERY  # more new tokens than there are tokens
    assert lens.tolist() == [3]
