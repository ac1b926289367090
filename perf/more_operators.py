"""The operators of ragged and drafted steps over the paged KV cache, as they are measured.

pool_extend lays a step out as packed rows: sequence b's new tokens are rows [query_start[b], query_start[b + 1]). The
attention of such a step is prefill_packed (prompts and chunks of different lengths, causal) or decode_tree (drafted tokens
that form a tree: each attends to the cache and to its ancestors). Of a tree, compact_cache moves the accepted tokens'
keys and values together; copy_blocks copies the blocks that forked requests stop sharing.

`run` with `own` false computes each in elementary torch operations; with `own` true it calls the
framework. `exact` computes the two attentions in 64 bits from their definition; the other two move values unchanged.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # a few short prompts: the latency of one call
        dict(name="packed_tiny", op="packed", batch=4, q_heads=8, kv_heads=2, head_dim=64, block_size=16, new_lo=1, new_hi=24,
             ctx_lo=0, ctx_hi=0, dtype="f16", fp8=False, window=0, idle=0.0, pad=0),
        # a prompt batch, ragged, nothing cached before
        dict(name="packed_prompts", op="packed", batch=16, q_heads=32, kv_heads=8, head_dim=128, block_size=16, new_lo=128,
             new_hi=2048, ctx_lo=0, ctx_hi=0, dtype="bf16", fp8=False, window=0, idle=0.0, pad=0),
        # a mixed step on an e4m3 cache: chunks of prompts beside requests that decode, some rows padded
        dict(name="packed_mixed", op="packed", batch=48, q_heads=32, kv_heads=8, head_dim=128, block_size=16, new_lo=1,
             new_hi=512, ctx_lo=0, ctx_hi=8192, dtype="bf16", fp8=True, window=0, idle=0.1, pad=77),
        # one long prompt
        dict(name="packed_long", op="packed", batch=1, q_heads=32, kv_heads=8, head_dim=128, block_size=16, new_lo=16384,
             new_hi=16384, ctx_lo=0, ctx_hi=0, dtype="bf16", fp8=False, window=0, idle=0.0, pad=0),
        # two requests with a few drafted tokens each: the latency of one call
        dict(name="tree_tiny", op="tree", batch=2, q_heads=8, kv_heads=2, head_dim=64, block_size=16, new_lo=5, new_hi=8,
             ctx_lo=100, ctx_hi=400, dtype="f16", fp8=False, window=0, idle=0.0, pad=0),
        # a decode batch whose requests have 16 drafted tokens each
        dict(name="tree_batch", op="tree", batch=32, q_heads=32, kv_heads=8, head_dim=128, block_size=16, new_lo=16, new_hi=16,
             ctx_lo=512, ctx_hi=4095, dtype="bf16", fp8=False, window=0, idle=0.0, pad=0),
        # wide trees of different sizes on an e4m3 cache
        dict(name="tree_fp8", op="tree", batch=64, q_heads=32, kv_heads=8, head_dim=128, block_size=16, new_lo=8, new_hi=64,
             ctx_lo=1, ctx_hi=8192, dtype="bf16", fp8=True, window=0, idle=0.05, pad=0),
        # one request on a long document
        dict(name="tree_long", op="tree", batch=1, q_heads=64, kv_heads=8, head_dim=128, block_size=32, new_lo=32, new_hi=32,
             ctx_lo=131072, ctx_hi=131072, dtype="bf16", fp8=False, window=0, idle=0.0, pad=0),
        # the blocks that a few forked requests stop sharing, one layer
        dict(name="copy_fork", op="copy", pairs=8, layers=1, blocks=512, kv_heads=8, head_dim=128, block_size=16, dtype="bf16",
             fp8=False, skipped=0.0),
        # the same of a large batch, all layers of a cache
        dict(name="copy_layers", op="copy", pairs=256, layers=32, blocks=640, kv_heads=8, head_dim=128, block_size=16,
             dtype="bf16", fp8=False, skipped=0.1),
        # accepted tokens of a decode batch, one layer
        dict(name="compact_step", op="compact", batch=32, layers=1, new_lo=16, new_hi=16, most=8, ctx_hi=1000, kv_heads=8,
             head_dim=128, block_size=16, dtype="bf16", fp8=False),
        # of wide trees of a large batch, all layers of an e4m3 cache
        dict(name="compact_layers", op="compact", batch=256, layers=32, new_lo=32, new_hi=64, most=16, ctx_hi=100, kv_heads=8,
             head_dim=128, block_size=16, dtype="bf16", fp8=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["packed", "packed", "packed", "packed", "tree", "tree", "tree", "copy", "compact"])
    bs = rng.choice([16, 32, 64])
    if op in ("packed", "tree"):
        fp8 = rng.random() < 0.3
        D = rng.choice([128, 128, 256] if fp8 else [64, 128, 128, 256])
        Hq, Hkv = rng.choice([(8, 2), (32, 8), (64, 8), (24, 8), (5, 5), (16, 1)])
        c = dict(op=op, q_heads=Hq, kv_heads=Hkv, head_dim=D, block_size=bs, dtype=rng.choice(["bf16", "f16"]), fp8=fp8,
                 idle=rng.choice([0.0, 0.2]), pad=rng.choice([0, 0, 1, 131]))
        if op == "packed":
            new_hi = _log_int(rng, 1, 8192)
            c.update(batch=_log_int(rng, 1, 64), new_hi=new_hi, new_lo=rng.choice([1, (new_hi + 1) // 2, new_hi]),
                     ctx_lo=0, ctx_hi=rng.choice([0, 0, _log_int(rng, 1, 16384)]))
        else:
            new_hi = rng.randint(1, 64)
            c.update(batch=_log_int(rng, 1, 64), new_hi=new_hi, new_lo=rng.choice([1, new_hi]), ctx_lo=0,
                     ctx_hi=_log_int(rng, 1, 65536))
        # not more than the largest listed ones: operations of the longest prompt, bytes of the widest trees' caches
        while c["batch"] > 1 and (4 * c["batch"] * c["new_hi"] * (c["ctx_hi"] + c["new_hi"] / 2) * Hq * D > 2.1e12
                                  or c["batch"] * (c["ctx_hi"] + c["new_hi"]) * Hkv * D > 64 * 8192 * 8 * 128):
            c["batch"] = (c["batch"] + 1) // 2
        while 4 * c["new_hi"] * (c["ctx_hi"] + c["new_hi"] / 2) * Hq * D > 2.1e12:
            c["new_hi"] = (c["new_hi"] + 1) // 2
            c["ctx_hi"] //= 2
        c["new_lo"] = min(c["new_lo"], c["new_hi"])
        c["window"] = rng.choice([0, 0, 0, 64 + (c["ctx_hi"] + c["new_hi"]) // 3])
        return c
    dtype, fp8 = rng.choice(["bf16", "f16"]), rng.random() < 0.3
    Hkv, D = rng.choice([(8, 128), (2, 64), (8, 256), (5, 128)])
    layers = _log_int(rng, 1, 32)
    if op == "copy":
        pairs = _log_int(rng, 1, 256)
        while pairs > 1 and pairs * layers * Hkv * D * bs > 256 * 32 * 8 * 128 * 16:
            pairs //= 2
        return dict(op=op, pairs=pairs, layers=layers, blocks=2 * pairs + rng.randint(1, 64), kv_heads=Hkv, head_dim=D,
                    block_size=bs, dtype=dtype, fp8=fp8, skipped=rng.choice([0.0, 0.3]))
    new_hi = rng.randint(1, 64)
    batch = _log_int(rng, 1, 256)
    while batch > 1 and batch * layers * Hkv * D > 256 * 32 * 8 * 128 // 2:
        batch //= 2
    return dict(op=op, batch=batch, layers=layers, new_lo=rng.choice([1, new_hi]), new_hi=new_hi, most=rng.randint(1, new_hi),
                ctx_hi=rng.choice([0, 50, 100]), kv_heads=Hkv, head_dim=D, block_size=bs, dtype=dtype, fp8=fp8)


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _ints(g, lo, hi, n):
    return torch.randint(lo, hi + 1, (n,), generator=g, device="cuda", dtype=torch.int32)


def _tables(g, lens, bs, width, pool):
    """[B, width] tables of `lens` tokens over a shuffled pool, and a block that none of them has."""
    ids = torch.randperm(pool, generator=g, device="cuda").int()
    n = (lens.long() + bs - 1) // bs
    start = torch.cumsum(n, 0) - n
    j = torch.arange(width, device="cuda")
    at = (start[:, None] + j[None, :]).clamp(max=pool - 1)
    return torch.where(j[None, :] < n[:, None], ids[at], -1).int(), ids[-1].long()


def _tokens(c):
    """New tokens of a step: the mean of what is drawn for the requests that are not idle."""
    live = c["batch"] - int(c["idle"] * c["batch"])
    return live * (c["new_lo"] + c["new_hi"]) // 2


def _lengths(c, seed):
    """New tokens of every request, 0 for the idle ones, that add up to the step's."""
    rng, B = random.Random(seed), c["batch"]
    lo, hi = c["new_lo"], c["new_hi"]
    live = sorted(rng.sample(range(B), B - int(c["idle"] * B)))
    new = [rng.randint(lo, hi) if b in live else 0 for b in range(B)]
    left = _tokens(c) - sum(new)
    while left:
        b = rng.choice(live)
        more = max(lo - new[b], min(hi - new[b], left))
        new[b] += rng.randint(min(0, more), max(0, more))
        left = _tokens(c) - sum(new)
    return new


def _starts(new):
    return torch.cat([torch.zeros_like(new[:1]), torch.cumsum(new, 0)]).int()


def _cache(g, shape, c, scale):
    """Values of a cache of the case's type: e4m3 codes of x / scale, or 16-bit x."""
    if not c["fp8"]:
        return torch.randn(shape, generator=g, device="cuda", dtype=DTYPES[c["dtype"]])
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
    return (x / scale).to(torch.float8_e4m3fn).view(torch.uint8)


def _tree(g, new):
    """Ancestor bits of random trees, one row a drafted token: its parent is one of the four drafted before it, or it hangs
    at the root (the cached token). Bit j of a row: drafted token j of the same request, itself among them."""
    B, N = new.numel(), int(new.max()) if new.numel() else 0
    back = torch.randint(1, 6, (B, max(N, 1)), generator=g, device="cuda")
    bits = torch.zeros(B, max(N, 1), dtype=torch.int64, device="cuda")
    one = torch.ones((), dtype=torch.int64, device="cuda")
    for j in range(N):
        parent = torch.where(back[:, j] == 5, -1, j - back[:, j])
        above = torch.where(parent >= 0, bits.gather(1, parent.clamp(min=0)[:, None])[:, 0], 0)
        bits[:, j] = above | (one << j)
    j = torch.arange(bits.shape[1], device="cuda")
    return bits[j[None, :] < new[:, None]]


def _prepare_attend(c, g):
    B, Hq, Hkv, D, bs = (c[k] for k in ("batch", "q_heads", "kv_heads", "head_dim", "block_size"))
    new = torch.tensor(_lengths(c, g.initial_seed()), dtype=torch.int32, device="cuda")
    lens = torch.where(new > 0, new + _ints(g, c["ctx_lo"], c["ctx_hi"], B), 0).int()
    width = max(1, -(-(c["new_hi"] + c["ctx_hi"]) // bs))
    # the pool holds what the requests use, and some blocks that none of them does
    pool = int(((lens.long() + bs - 1) // bs).sum()) + 16
    ks, vs = (0.03125, 0.02) if c["fp8"] else (1.0, 1.0)
    starts = _starts(new)
    T = _tokens(c) + c["pad"]
    q = torch.randn(T, Hq, D, generator=g, device="cuda").to(DTYPES[c["dtype"]])
    s = dict(q=q, kc=_cache(g, (pool, Hkv, bs, D), c, ks), vc=_cache(g, (pool, Hkv, bs, D), c, vs),
             tables=_tables(g, lens, bs, width, pool)[0], lens=lens, starts=starts, scale=D ** -0.5, k_scale=ks, v_scale=vs,
             out=torch.zeros_like(q), host_lens=lens.tolist(), host_starts=starts.tolist(), mask=None)
    if c["op"] == "tree":
        s["mask"] = torch.cat([_tree(g, new), torch.zeros(c["pad"], dtype=torch.int64, device="cuda")])
    return s


def _prepare_copy(c, g):
    n, NB = c["pairs"], c["blocks"]
    shape = (c["layers"], NB, c["kv_heads"], c["block_size"], c["head_dim"])
    ids = torch.randperm(NB, generator=g, device="cuda").int()
    # targets are blocks of their own; a source may have several
    source = ids[n + torch.randint(0, NB - n, (n,), generator=g, device="cuda")]
    target = torch.where(torch.rand(n, generator=g, device="cuda") < c["skipped"], -1, ids[:n])
    return dict(kc=_cache(g, shape, c, 0.03125), vc=_cache(g, shape, c, 0.02), pairs=torch.stack([source, target], 1).int().contiguous())


def _prepare_compact(c, g):
    B, bs, M = c["batch"], c["block_size"], c["most"]
    new = _ints(g, c["new_lo"], c["new_hi"], B)
    lens = (new + _ints(g, 0, c["ctx_hi"], B)).int()
    width = max(1, -(-(c["new_hi"] + c["ctx_hi"]) // bs))
    pool = B * width + 8
    shape = (c["layers"], pool, c["kv_heads"], bs, c["head_dim"])
    # of the accepted tokens the first few were drafted in a row; the others come from a branch behind as many places as
    # are accepted (so that a second pass over the same cache finds the same rows)
    count = torch.minimum(_ints(g, 0, M, B), new)
    chain = (torch.rand(B, generator=g, device="cuda") * (count + 1)).int().minimum(count)
    order = torch.rand(B, c["new_hi"], generator=g, device="cuda")
    j = torch.arange(c["new_hi"], device="cuda")[None, :]
    order = torch.where((j >= count[:, None]) & (j < new[:, None]), order, 2.0)
    rank = order.argsort(1).argsort(1)
    count = torch.minimum(count, chain + (new - count))
    picked = (j < chain[:, None]) | ((order < 1) & (rank < (count - chain)[:, None]))
    slot = torch.where(picked, torch.cumsum(picked, 1) - 1, M)
    kept = torch.full((B, M + 1), -1, device="cuda").scatter(1, slot.clamp(max=M), j.expand(B, -1))[:, :M]
    kept = torch.where(torch.arange(M, device="cuda")[None, :] < count[:, None], kept, -1).int().contiguous()
    tables, spare = _tables(g, lens, bs, width, pool)
    return dict(kc=_cache(g, shape, c, 0.03125), vc=_cache(g, shape, c, 0.02), tables=tables, spare=spare, lens=lens, starts=_starts(new),
                kept=kept, count=count.int(), lens_out=torch.empty_like(lens), kept_tokens=torch.empty_like(lens))


def prepare(case, seed):
    make = {"packed": _prepare_attend, "tree": _prepare_attend, "copy": _prepare_copy, "compact": _prepare_compact}[case["op"]]
    return dict(make(case, _gen(seed)), case=case)


# ------------------------------------------------------------- plain forms

def _attend(s):
    c = s["case"]
    bs, W, Hkv = c["block_size"], c["window"], c["kv_heads"]
    T, Hq, D = s["q"].shape
    G = Hq // Hkv
    out = torch.zeros(T, Hkv, G, D, device="cuda")
    starts, lens = s["host_starts"], s["host_lens"]
    tree = s["mask"] is not None
    for b in range(c["batch"]):
        n, L = starts[b + 1] - starts[b], lens[b]
        if n == 0:
            continue
        blocks = s["tables"][b, : -(-L // bs)].long()

        def rows(cache, scale):
            x = cache[blocks].transpose(0, 1).flatten(1, 2)[:, :L]
            return x.view(torch.float8_e4m3fn).float().mul_(scale) if c["fp8"] else x.float()

        k, v = rows(s["kc"], s["k_scale"]).transpose(1, 2), rows(s["vc"], s["v_scale"])
        j = torch.arange(L, device="cuda")
        step = max(1, min(n, (1 << 28) // (Hq * L)))  # rows at once: a gigabyte of scores
        for t0 in range(0, n, step):
            t1 = min(n, t0 + step)
            r0, r1 = starts[b] + t0, starts[b] + t1
            if tree:
                bits = s["mask"][r0:r1, None]
                seen = (bits >> (j - (L - n)).clamp(0, 63)) & 1 == 1
                pos = L - n - 1 + ((bits >> torch.arange(min(n, 64), device="cuda")) & 1).sum(1, keepdim=True)
                seen = torch.where(j < L - n, True, seen & (j < L - n + 64))
            else:
                pos = L - n + torch.arange(t0, t1, device="cuda")[:, None]
                seen = j <= pos
            if W > 0:
                seen = seen & ((j > pos - W) | (j >= L - n if tree else False))
            q = s["q"][r0:r1].float().view(t1 - t0, Hkv, G, D).permute(1, 2, 0, 3).reshape(Hkv, -1, D)
            score = (q @ k * s["scale"]).view(Hkv, G, t1 - t0, L).masked_fill_(~seen, -torch.inf)
            top = score.amax(-1, keepdim=True).clamp(min=-1e30)
            p = torch.exp(score - top)
            del score
            total = p.sum(-1, keepdim=True)
            o = (p.view(Hkv, -1, L) @ v).view(Hkv, G, t1 - t0, D)
            out[r0:r1] = torch.where(total > 0, o / total, 0).permute(2, 0, 1, 3)
    return out.view(T, Hq, D).to(s["q"].dtype)


def _copy(s):
    src, dst = s["pairs"][:, 0].long(), s["pairs"][:, 1].long()
    live = dst >= 0
    dst = torch.where(live, dst, src)  # a skipped pair: its source stays as it is
    for cache in (s["kc"], s["vc"]):
        cache[:, dst] = cache[:, src]
    return _caches(s)


def _caches(s):
    kc, vc = s["kc"], s["vc"]
    return dict(kc=kc.view(torch.float8_e4m3fn), vc=vc.view(torch.float8_e4m3fn)) if s["case"]["fp8"] else dict(kc=kc, vc=vc)


def _compact(s):
    bs, NL = s["case"]["block_size"], s["case"]["layers"]
    lens, count = s["lens"].long(), s["count"].long()
    new = s["starts"].diff().long()
    base = (lens - new)[:, None]
    i = torch.arange(s["kept"].shape[1], device="cuda")[None, :]
    live = i < count[:, None]
    # places behind the accepted ones move rows of a block that nothing uses onto themselves
    src, dst = torch.where(live, base + s["kept"].long(), 0), torch.where(live, base + i, 0)
    blocks = s["tables"].long()
    sb = torch.where(live, blocks.gather(1, src // bs), s["spare"]).flatten()
    db = torch.where(live, blocks.gather(1, dst // bs), s["spare"]).flatten()
    so, do = (src % bs).flatten(), (dst % bs).flatten()
    layer = torch.arange(NL, device="cuda")[:, None]
    for cache in (s["kc"], s["vc"]):
        cache[layer, db, :, do] = cache[layer, sb, :, so]
    kept = (lens - new + count).int()
    return dict(_caches(s), lens=kept, kept_tokens=(kept + bs - 1) // bs * bs)


# --------------------------------------------------------------------- run

def run(state):
    s, c = state, state["case"]
    if own:
        import paged_kv_cache_267_gb300 as pa
        kw = dict(num_kv_heads=c["kv_heads"], block_size=c["block_size"], window=c.get("window", 0),
                  kv_dtype="fp8" if c["fp8"] else "auto", scale=s.get("scale"), k_scale=s.get("k_scale"), v_scale=s.get("v_scale"))
        if c["op"] == "packed":
            return pa.prefill_packed(s["q"], s["kc"], s["vc"], s["tables"], s["lens"], s["starts"], out=s["out"], **kw)
        if c["op"] == "tree":
            return pa.decode_tree(s["q"], s["kc"], s["vc"], s["tables"], s["lens"], s["starts"], s["mask"], out=s["out"], **kw)
        if c["op"] == "copy":
            pa.copy_blocks(s["kc"], s["vc"], s["pairs"])
            return _caches(s)
        pa.compact_cache(s["kc"], s["vc"], s["tables"], s["lens"], s["starts"], s["kept"], s["count"], block_size=c["block_size"],
                         seq_lens_out=s["lens_out"], kept_tokens=s["kept_tokens"])
        return dict(_caches(s), lens=s["lens_out"], kept_tokens=s["kept_tokens"])
    return {"packed": _attend, "tree": _attend, "copy": _copy, "compact": _compact}[c["op"]](s)


# -------------------------------------------------------------------- work

def work(case):
    c = case
    elt = 1 if c["fp8"] else 2
    if c["op"] == "copy":
        return {"bytes": 4 * c["pairs"] * (1 - c["skipped"]) * c["layers"] * c["kv_heads"] * c["block_size"] * c["head_dim"] * elt,
                "flops": 0}
    if c["op"] == "compact":
        # half of the most that may be accepted, half of those in their place already
        moved = c["batch"] * min(c["most"], (c["new_lo"] + c["new_hi"]) / 2) / 4
        return {"bytes": 4 * moved * c["layers"] * c["kv_heads"] * c["head_dim"] * elt + 16 * c["batch"], "flops": 0}
    B, Hq, Hkv, D = c["batch"] * (1 - c["idle"]), c["q_heads"], c["kv_heads"], c["head_dim"]
    # means over the lengths that are drawn: tokens, tokens squared, tokens before them
    lo, hi = c["new_lo"], c["new_hi"]
    n, n2 = (lo + hi) / 2, (lo * lo + lo * hi + hi * hi) / 3
    ctx = (c["ctx_lo"] + c["ctx_hi"]) / 2
    W = c["window"] or 10 ** 9
    if c["op"] == "tree":
        # a drafted token has five ancestors in the mean, itself among them, where there are as many
        seen, pairs = min(ctx, W) + n, n * (min(ctx, W) + min((n + 1) / 2, 5))
    else:
        seen, pairs = min(ctx, W) + n, min(n * ctx + n2 / 2, n * W)
    return {"bytes": B * (seen * 2 * Hkv * D * elt + 4 * n * Hq * D + 4 * seen / c["block_size"]), "flops": 4 * B * pairs * Hq * D}


# ------------------------------------------------------------------- exact

def exact(case, seed):
    """The attentions from their definition in 64 bits, one (request, KV head) at a time."""
    if case["op"] in ("copy", "compact"):
        return None
    c, s = case, prepare(case, seed)
    bs, W, Hkv = c["block_size"], c["window"], c["kv_heads"]
    T, Hq, D = s["q"].shape
    G = Hq // Hkv
    out = torch.zeros(T, Hq, D, dtype=torch.float64, device="cuda")
    for b, L in enumerate(s["host_lens"]):
        r0, r1 = s["host_starts"][b], s["host_starts"][b + 1]
        n = r1 - r0
        if n == 0:
            continue
        first = L - n
        place = torch.arange(L, device="cuda")
        for h in range(Hkv):
            def values(cache, scale):
                x = cache[s["tables"][b, : (L + bs - 1) // bs].long(), h].reshape(-1, D)[:L]
                return (x.view(torch.float8_e4m3fn).float() if c["fp8"] else x).double() * scale

            k, v = values(s["kc"], s["k_scale"]), values(s["vc"], s["v_scale"])
            for t0 in range(0, n, 1024):
                t1 = min(n, t0 + 1024)
                # one row a token: which positions it attends to
                if s["mask"] is None:
                    p = torch.arange(first + t0, first + t1, device="cuda")
                    lo = torch.clamp(p - (W - 1), min=0) if W > 0 else torch.zeros_like(p)
                    attends = (place[None, :] >= lo[:, None]) & (place[None, :] <= p[:, None])
                else:
                    m = s["mask"][r0 + t0: r0 + t1]
                    bit = ((m[:, None] >> torch.arange(min(n, 64), device="cuda")) & 1).bool()
                    p = first + bit.sum(1) - 1
                    lo = torch.clamp(p - (W - 1), min=0) if W > 0 else torch.zeros_like(p)
                    attends = (place[None, :] >= lo[:, None]) & (place[None, :] < first)
                    attends[:, first: first + bit.shape[1]] = bit
                q = s["q"][r0 + t0: r0 + t1, h * G: (h + 1) * G].double()
                a = torch.einsum("tgd,ld->tgl", q, k) * s["scale"]
                a.masked_fill_(~attends[:, None, :], -math.inf)
                w = torch.softmax(a, -1).nan_to_num_(0.0)
                out[r0 + t0: r0 + t1, h * G: (h + 1) * G] = torch.einsum("tgl,ld->tgd", w, v)
    return out
