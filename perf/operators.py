"""The serving-step operators over the paged KV cache, as they are measured.

A decode or chunk step over the cache is four calls: grow every request's block table on the GPU and
get the slots of its new tokens (pool_extend), give the blocks of finished requests back (pool_release),
normalise and rotate the heads of the projected rows while writing them to the cache
(norm_rope_and_cache), and attend, reading a prefix that several requests share once for all of them
(decode_shared).

`run` with `own` false computes each in elementary torch operations; with `own` true it calls the
framework. `exact` computes the floating-point ones in 64 bits from their definitions.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # one decode step of 64 requests: one new token each, a block popped by every 16th
        dict(name="extend_decode", op="extend", batch=64, block_size=16, len_lo=512, len_hi=4095, new_lo=1, new_hi=1,
             max_tokens=64, zero_rows=0.0),
        # a prompt batch from empty tables: half a million ragged tokens, padded to 2^20 rows
        dict(name="extend_prompts", op="extend", batch=256, block_size=32, len_lo=0, len_hi=0, new_lo=1, new_hi=4096,
             max_tokens=1 << 20, zero_rows=0.05),
        # a few finished requests of a decode batch
        dict(name="release_some", op="release", batch=256, block_size=16, len_lo=1, len_hi=8192, share=0.06, shared=0),
        # the end of a large batch whose requests share a prefix that stays
        dict(name="release_all", op="release", batch=4096, block_size=16, len_lo=1024, len_hi=8192, share=1.0, shared=1024),
        # one decode step's rows
        dict(name="norm_decode", op="norm", tokens=64, q_heads=32, kv_heads=8, head_dim=128, rotary=128, block_size=16,
             dtype="bf16", fp8=False, interleaved=False, norm=True, skipped=0.0),
        # an odd number of rows, small heads, part of each head rotated in neighbouring pairs, padded rows
        dict(name="norm_partial", op="norm", tokens=4099, q_heads=8, kv_heads=2, head_dim=64, rotary=32, block_size=16,
             dtype="f16", fp8=False, interleaved=True, norm=True, skipped=0.1),
        # a prompt batch into an e4m3 cache
        dict(name="norm_prompts_fp8", op="norm", tokens=16384, q_heads=32, kv_heads=8, head_dim=128, rotary=128,
             block_size=16, dtype="bf16", fp8=True, interleaved=False, norm=True, skipped=0.0),
        # four short requests: the latency of one call
        dict(name="shared_tiny", op="shared", batch=4, groups=1, q_heads=8, kv_heads=2, head_dim=64, block_size=16,
             prefix=208, tail_lo=1, tail_hi=64, dtype="f16", fp8=False, window=0, idle=0.0),
        # a system prompt of 4096 tokens under 64 short conversations
        dict(name="shared_prompt", op="shared", batch=64, groups=1, q_heads=32, kv_heads=8, head_dim=128, block_size=16,
             prefix=4096, tail_lo=1, tail_hi=512, dtype="bf16", fp8=False, window=0, idle=0.0),
        # four prompts, longer conversations, some rows of the batch idle
        dict(name="shared_groups", op="shared", batch=128, groups=4, q_heads=32, kv_heads=8, head_dim=128, block_size=16,
             prefix=2048, tail_lo=128, tail_hi=2048, dtype="bf16", fp8=False, window=0, idle=0.05),
        # a large batch on an e4m3 cache
        dict(name="shared_fp8", op="shared", batch=256, groups=1, q_heads=32, kv_heads=8, head_dim=128, block_size=16,
             prefix=8192, tail_lo=1, tail_hi=1024, dtype="bf16", fp8=True, window=0, idle=0.0),
        # a few requests about one long document
        dict(name="shared_document", op="shared", batch=16, groups=1, q_heads=64, kv_heads=8, head_dim=128, block_size=32,
             prefix=65536, tail_lo=256, tail_hi=2048, dtype="bf16", fp8=False, window=0, idle=0.0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["extend", "release", "norm", "norm", "shared", "shared", "shared"])
    bs = rng.choice([16, 32, 64])
    if op == "extend":
        batch = _log_int(rng, 1, 1024)
        new_hi = _log_int(rng, 1, max(1, min(4096, (1 << 19) // batch)))
        return dict(op=op, batch=batch, block_size=bs, len_lo=0, len_hi=_log_int(rng, 1, 4096), new_lo=rng.choice([1, new_hi]),
                    new_hi=new_hi, max_tokens=batch * new_hi + rng.choice([0, 1, 77]), zero_rows=rng.choice([0.0, 0.1, 0.5]))
    if op == "release":
        return dict(op=op, batch=_log_int(rng, 1, 4096), block_size=bs, len_lo=rng.randint(0, 512), len_hi=_log_int(rng, 512, 8192),
                    share=rng.choice([0.02, 0.1, 0.5, 1.0]), shared=rng.choice([0, 0, 4 * bs]))
    if op == "norm":
        D = rng.choice([64, 128, 128, 256])
        Hq, Hkv = rng.choice([(8, 2), (32, 8), (64, 8), (24, 8), (5, 5)])
        most = int(16384 * 48 * 128 / ((Hq + 2 * Hkv) * D))
        return dict(op=op, tokens=_log_int(rng, 1, min(most, 16384)), q_heads=Hq, kv_heads=Hkv, head_dim=D,
                    rotary=rng.choice([D, D, D // 2]), block_size=bs, dtype=rng.choice(["bf16", "f16"]),
                    fp8=rng.random() < 0.3, interleaved=rng.random() < 0.3, norm=rng.random() < 0.8, skipped=rng.choice([0.0, 0.2]))
    fp8 = rng.random() < 0.3
    D = rng.choice([128, 128, 256] if fp8 else [64, 128, 128, 256])
    Hq, Hkv = rng.choice([(8, 2), (32, 8), (64, 8), (24, 8), (8, 8)])
    batch = _log_int(rng, 2, 256)
    groups = rng.randint(1, max(1, min(6, batch // 2)))
    tail_hi = _log_int(rng, 1, 1024)
    prefix = _log_int(rng, 64, 16384)
    while prefix > 64 and batch * (prefix + tail_hi) * Hkv * D > 256 * 9216 * 8 * 128:
        prefix //= 2
    prefix = max(bs, prefix // bs * bs)
    return dict(op=op, batch=batch, groups=groups, q_heads=Hq, kv_heads=Hkv, head_dim=D, block_size=bs, prefix=prefix,
                tail_lo=1, tail_hi=tail_hi, dtype=rng.choice(["bf16", "f16"]), fp8=fp8,
                window=rng.choice([0, 0, 0, prefix // 2 + 1, 2 * prefix + tail_hi]), idle=rng.choice([0.0, 0.1]))


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _ints(g, lo, hi, n):
    return torch.randint(lo, hi + 1, (n,), generator=g, device="cuda", dtype=torch.int32)


def _blocks_of(lens, bs):
    return (lens + (bs - 1)) // bs


def _tables(g, lens, bs, width, pool):
    """[B, width] tables of `lens` tokens over a shuffled pool, and the ids that are left."""
    ids = torch.randperm(pool, generator=g, device="cuda").int()
    n = _blocks_of(lens, bs).long()
    start = torch.cumsum(n, 0) - n
    j = torch.arange(width, device="cuda")
    used = j[None, :] < n[:, None]
    at = (start[:, None] + j[None, :]).clamp(max=pool - 1)
    return torch.where(used, ids[at], -1).int(), ids[int(n.sum()):]


def _prepare_pool(c, g):
    B, bs = c["batch"], c["block_size"]
    lens = _ints(g, c["len_lo"], c["len_hi"], B)
    most = c["len_hi"] + (c["new_hi"] if c["op"] == "extend" else 0)
    width = max(1, -(-most // bs))
    pool = B * width + 64
    tables, left = _tables(g, lens, bs, width, pool)
    free = torch.full((pool,), -1, dtype=torch.int32, device="cuda")
    free[: left.numel()] = left
    state = torch.tensor([left.numel(), 0], dtype=torch.int32, device="cuda")
    s = dict(tables=tables, lens=lens, free=free, state=state, lens_out=torch.empty_like(lens),
             state_out=torch.zeros_like(state))
    if c["op"] == "extend":
        new = _ints(g, c["new_lo"], c["new_hi"], B)
        s["new"] = torch.where(torch.rand(B, generator=g, device="cuda") < c["zero_rows"], 0, new).int()
        T = c["max_tokens"]
        s.update(slots=torch.empty(T, dtype=torch.int64, device="cuda"), positions=torch.empty(T, dtype=torch.int32, device="cuda"),
                 query_start=torch.empty(B + 1, dtype=torch.int32, device="cuda"))
    else:
        s["released"] = (torch.rand(B, generator=g, device="cuda") < c["share"]).int()
        s["shared"] = torch.full((B,), c["shared"], dtype=torch.int32, device="cuda") if c["shared"] else None
    return s


def _prepare_norm(c, g):
    T, Hq, Hkv, D, R, bs = (c[k] for k in ("tokens", "q_heads", "kv_heads", "head_dim", "rotary", "block_size"))
    dt = DTYPES[c["dtype"]]
    # one projection's output row holds the q, k and v heads of a token
    qkv = torch.randn(T, (Hq + 2 * Hkv) * D, generator=g, device="cuda").to(dt)
    q, k, v = qkv.view(T, Hq + 2 * Hkv, D).split([Hq, Hkv, Hkv], dim=1)
    nb = -(-T // bs) + 8
    cache = dict(dtype=torch.uint8 if c["fp8"] else dt, device="cuda")
    slots = torch.randperm(nb * bs, generator=g, device="cuda")[:T]
    slots = torch.where(torch.rand(T, generator=g, device="cuda") < c["skipped"], -1, slots)
    angle = torch.arange(8192, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (
        -torch.arange(0, R, 2, device="cuda", dtype=torch.float64) / R)
    s = dict(q=q, k=k, v=v, slots=slots, positions=_ints(g, 0, 8191, T),
             cos_sin=torch.cat([angle.cos(), angle.sin()], 1).float(), kc=torch.zeros(nb, Hkv, bs, D, **cache),
             vc=torch.zeros(nb, Hkv, bs, D, **cache), out=torch.empty(T, Hq, D, dtype=dt, device="cuda"), wq=None, wk=None,
             k_scale=0.03125 if c["fp8"] else 1.0, v_scale=0.02 if c["fp8"] else 1.0)
    if c["norm"]:
        s["wq"] = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(dt)
        s["wk"] = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(dt)
    return s


def _prepare_shared(c, g):
    B, NG, Hq, Hkv, D, bs, P = (c[k] for k in ("batch", "groups", "q_heads", "kv_heads", "head_dim", "block_size", "prefix"))
    dt = DTYPES[c["dtype"]]
    tails = _ints(g, c["tail_lo"], c["tail_hi"], B)
    width = -(-(P + c["tail_hi"]) // bs)
    pb = P // bs
    pool = NG * pb + B * (width - pb) + 32
    ids = torch.randperm(pool, generator=g, device="cuda").int()
    starts = torch.arange(NG + 1, device="cuda") * B // NG
    group = torch.searchsorted(starts[1:], torch.arange(B, device="cuda"), right=True)
    pre = ids[: NG * pb].view(NG, pb)[group]
    own_blocks = ids[NG * pb: NG * pb + B * (width - pb)].view(B, width - pb)
    used = torch.arange(width - pb, device="cuda")[None, :] < _blocks_of(tails, bs)[:, None]
    tables = torch.cat([pre, torch.where(used, own_blocks, -1)], 1).int().contiguous()
    lens = torch.where(torch.rand(B, generator=g, device="cuda") < c["idle"], 0, tails + P).int()
    kw = dict(generator=g, device="cuda", dtype=torch.float32 if c["fp8"] else dt)
    shape = (pool, Hkv, bs, D)
    ks, vs = (0.03125, 0.02) if c["fp8"] else (1.0, 1.0)
    kc, vc = torch.randn(shape, **kw), torch.randn(shape, **kw)
    if c["fp8"]:
        kc, vc = ((x / sc).to(torch.float8_e4m3fn).view(torch.uint8) for x, sc in ((kc, ks), (vc, vs)))
    q = torch.randn(B, Hq, D, generator=g, device="cuda").to(dt)
    return dict(q=q, kc=kc, vc=vc, tables=tables, lens=lens, prefix_lens=torch.full((NG,), P, dtype=torch.int32, device="cuda"),
                group_starts=starts.int(), scale=D ** -0.5, k_scale=ks, v_scale=vs, out=torch.empty_like(q))


def prepare(case, seed):
    g = _gen(seed)
    make = {"extend": _prepare_pool, "release": _prepare_pool, "norm": _prepare_norm, "shared": _prepare_shared}[case["op"]]
    return dict(make(case, g), case=case)


# ------------------------------------------------------------- plain forms

def _extend(s):
    c = s["case"]
    B, bs, T = c["batch"], c["block_size"], c["max_tokens"]
    lens, new, free, tables = s["lens"].long(), s["new"].long(), s["free"], s["tables"]
    count = s["state"][0].long()
    width = tables.shape[1]
    had, has = _blocks_of(lens, bs), _blocks_of(lens + new, bs)
    need = has - had
    end = torch.cumsum(need, 0)
    stop = torch.cumsum(new, 0)
    # all or nothing: enough free blocks, table columns and rows of slots
    ok = (end[-1] <= count) & (stop[-1] <= T) & ((lens + new) <= width * bs).all() & (new >= 0).all()
    new = torch.where(ok, new, 0)
    stop = torch.where(ok, stop, 0)
    j = torch.arange(width, device="cuda")[None, :]
    at = count - 1 - ((end - need)[:, None] + j - had[:, None])
    fresh = (j >= had[:, None]) & (j < has[:, None]) & ok
    tables = torch.where(fresh, free[at.clamp(0, free.numel() - 1)], tables)
    t = torch.arange(T, device="cuda")
    row = torch.searchsorted(stop, t, right=True).clamp(max=B - 1)
    live = t < stop[-1]
    pos = torch.where(live, lens[row] + t - (stop - new)[row], 0)
    slots = torch.where(live, tables[row, (pos // bs).clamp(0, width - 1)].long() * bs + pos % bs, -1)
    left = torch.where(ok, count - end[-1], count)
    return dict(tables=tables, lens=(lens + new).int(), state=torch.stack([left, torch.zeros_like(left)]).int(),
                query_start=torch.cat([torch.zeros_like(stop[:1]), stop]).int(), slots=slots, positions=pos.int())


def _release(s):
    bs = s["case"]["block_size"]
    lens, free, tables, gone = s["lens"].long(), s["free"], s["tables"], s["released"] != 0
    count = s["state"][0].long()
    had = _blocks_of(lens, bs)
    keep = s["shared"].long() // bs if s["shared"] is not None else torch.zeros_like(had)
    give = torch.where(gone, (had - keep).clamp(min=0), 0)
    end = torch.cumsum(give, 0)
    j = torch.arange(tables.shape[1], device="cuda")[None, :]
    mine = (j >= keep[:, None]) & (j < had[:, None]) & gone[:, None]
    at = torch.where(mine, count + (end - give)[:, None] + j - keep[:, None], free.numel())
    free = torch.cat([free, free[:1]]).scatter(0, at.reshape(-1), tables.reshape(-1))[:-1]
    total = count + end[-1]
    return dict(free=free, lens=torch.where(gone, 0, lens).int(), state=torch.stack([total, torch.zeros_like(total)]).int())


def _rms(x, w):
    return x if w is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.float()


def _rotate(x, cos, sin, R, interleaved):
    if interleaved:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., : R // 2], x[..., R // 2: R]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., R:]], -1)


def _norm(s):
    c = s["case"]
    R, bs = c["rotary"], c["block_size"]
    cs = s["cos_sin"][s["positions"].long()]
    cos, sin = cs[:, None, : R // 2], cs[:, None, R // 2:]
    q = _rotate(_rms(s["q"].float(), s["wq"]), cos, sin, R, c["interleaved"])
    k = _rotate(_rms(s["k"].float(), s["wk"]), cos, sin, R, c["interleaved"])
    v = s["v"].float()
    nb, Hkv, _, D = s["kc"].shape
    # padded rows go to one spare block behind the pool, which is dropped
    slots = torch.where(s["slots"] < 0, nb * bs, s["slots"])

    def store(cache, x, scale):
        if c["fp8"]:
            x = (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            x = x.to(cache.dtype)
        rows = torch.cat([cache, cache[:1]])
        rows[slots // bs, :, slots % bs, :] = x
        return rows[:-1]

    return dict(q=q.to(s["q"].dtype), **_caches(c, store(s["kc"], k, s["k_scale"]), store(s["vc"], v, s["v_scale"])))


def _caches(c, kc, vc):
    return dict(kc=kc.view(torch.float8_e4m3fn), vc=vc.view(torch.float8_e4m3fn)) if c["fp8"] else dict(kc=kc, vc=vc)


def _shared(s):
    c = s["case"]
    bs, W, Hkv = c["block_size"], c["window"], c["kv_heads"]
    B, Hq, D = s["q"].shape
    L = s["tables"].shape[1] * bs
    pos = torch.arange(L, device="cuda")
    block = s["tables"].clamp(min=0).long()[:, pos // bs]

    def rows(cache, scale):
        x = cache[block, :, pos % bs, :]
        return x.view(torch.float8_e4m3fn).float().mul_(scale) if c["fp8"] else x.float()

    lens = s["lens"].long()[:, None]
    first = (lens - W).clamp(min=0) if W > 0 else torch.zeros_like(lens)
    seen = ((pos >= first) & (pos < lens))[:, None, None, :]
    q = s["q"].float().view(B, Hkv, Hq // Hkv, D)
    score = torch.einsum("bkgd,blkd->bkgl", q, rows(s["kc"], s["k_scale"])) * s["scale"]
    score = score.masked_fill(~seen, -torch.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    o = torch.einsum("bkgl,blkd->bkgd", p, rows(s["vc"], s["v_scale"]).masked_fill(~seen.view(B, L, 1, 1), 0))
    return torch.where(total > 0, o / total, 0).view(B, Hq, D).to(s["q"].dtype)


# --------------------------------------------------------------------- run

def run(state):
    s, c = state, state["case"]
    if own:
        import paged_kv_cache_267_gb300 as pa
        kv = "fp8" if c.get("fp8") else "auto"
        if c["op"] == "extend":
            pa.pool_extend(s["tables"], s["lens"], s["new"], s["free"], s["state"], block_size=c["block_size"],
                           slot_mapping=s["slots"], positions=s["positions"], query_start=s["query_start"],
                           seq_lens_out=s["lens_out"], pool_state_out=s["state_out"])
            return dict(tables=s["tables"], lens=s["lens_out"], state=s["state_out"], query_start=s["query_start"],
                        slots=s["slots"], positions=s["positions"])
        if c["op"] == "release":
            pa.pool_release(s["tables"], s["lens"], s["released"], s["free"], s["state"], block_size=c["block_size"],
                            shared_tokens=s["shared"], seq_lens_out=s["lens_out"], pool_state_out=s["state_out"])
            return dict(free=s["free"], lens=s["lens_out"], state=s["state_out"])
        if c["op"] == "norm":
            pa.norm_rope_and_cache(s["q"], s["k"], s["v"], s["kc"], s["vc"], s["slots"], s["positions"], s["cos_sin"],
                                   q_weight=s["wq"], k_weight=s["wk"], eps=1e-6, interleaved=c["interleaved"], kv_dtype=kv,
                                   k_scale=s["k_scale"], v_scale=s["v_scale"], out=s["out"])
            return dict(q=s["out"], **_caches(c, s["kc"], s["vc"]))
        return pa.decode_shared(s["q"], s["kc"], s["vc"], s["tables"], s["lens"], s["prefix_lens"], s["group_starts"],
                                num_kv_heads=c["kv_heads"], scale=s["scale"], block_size=c["block_size"], window=c["window"],
                                kv_dtype=kv, k_scale=s["k_scale"], v_scale=s["v_scale"], out=s["out"])
    return {"extend": _extend, "release": _release, "norm": _norm, "shared": _shared}[c["op"]](s)


# -------------------------------------------------------------------- work

def work(case):
    c = case
    if c["op"] in ("extend", "release"):
        B, bs = c["batch"], c["block_size"]
        mean = (c["len_lo"] + c["len_hi"]) / 2
        if c["op"] == "extend":
            new = (1 - c["zero_rows"]) * (c["new_lo"] + c["new_hi"]) / 2
            # lengths and requests in, lengths and starts out; a block id moved per block; a slot and a position per row
            return {"bytes": B * 16 + 8 * B * new / bs + 12 * c["max_tokens"], "flops": 0}
        return {"bytes": B * 12 + 8 * B * c["share"] * max(0, mean - c["shared"]) / bs, "flops": 0}
    if c["op"] == "norm":
        T, Hq, Hkv, D, R = (c[k] for k in ("tokens", "q_heads", "kv_heads", "head_dim", "rotary"))
        live = 1 - c["skipped"]
        b = T * Hq * D * 4 + live * T * 2 * Hkv * D * (3 if c["fp8"] else 4) + T * 12 + min(T, 8192) * R * 4
        return {"bytes": b, "flops": T * (Hq + Hkv) * (4 * D + 3 * R)}
    B, NG, Hq, Hkv, D, bs, P = (c[k] for k in ("batch", "groups", "q_heads", "kv_heads", "head_dim", "block_size", "prefix"))
    live = B * (1 - c["idle"])
    tail = (c["tail_lo"] + c["tail_hi"]) / 2
    W = c["window"] or 10 ** 9
    unique = NG * min(P, max(0, W - c["tail_lo"])) + live * min(tail, W)
    kv = unique * Hkv * D * (2 if c["fp8"] else 4)
    return {"bytes": kv + 4 * B * Hq * D + 4 * unique / bs, "flops": 4 * live * Hq * D * min(P + tail, W)}


# ------------------------------------------------------------------- exact

def exact(case, seed):
    """From the definitions in 64 bits, a row at a time; whole-number outputs need none."""
    if case["op"] in ("extend", "release"):
        return None
    s, c = prepare(case, seed), case
    if c["op"] == "norm":
        R, D = c["rotary"], c["head_dim"]
        cs = s["cos_sin"].double().index_select(0, s["positions"].long())
        i = torch.arange(R // 2, device="cuda")
        lo, hi = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + R // 2)

        def turned(x, w):
            y = x.double()
            if w is not None:
                y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / D + 1e-6) * w.double()
            z = y.clone()
            co, si = cs[:, None, : R // 2], cs[:, None, R // 2:]
            z[..., lo] = y[..., lo] * co - y[..., hi] * si
            z[..., hi] = y[..., lo] * si + y[..., hi] * co
            return z

        def stored(cache, x, scale):
            flat = torch.zeros(cache.shape, dtype=torch.float64, device="cuda").transpose(1, 2).flatten(0, 1).contiguous()
            live = s["slots"] >= 0
            flat[s["slots"][live]] = (x[live] / scale).clamp(-448, 448) if c["fp8"] else x[live]
            return flat.view(cache.shape[0], cache.shape[2], cache.shape[1], cache.shape[3]).transpose(1, 2).contiguous()

        return dict(q=turned(s["q"], s["wq"]), kc=stored(s["kc"], turned(s["k"], s["wk"]), s["k_scale"]),
                    vc=stored(s["vc"], s["v"].double(), s["v_scale"]))
    bs, Hkv, W = c["block_size"], c["kv_heads"], c["window"]
    B, Hq, D = s["q"].shape
    out = torch.zeros(B, Hkv, Hq // Hkv, D, dtype=torch.float64, device="cuda")
    lens, tables = s["lens"].tolist(), s["tables"].long()
    for b in range(B):
        L = lens[b]
        if L == 0:
            continue
        lo = max(0, L - W) if W > 0 else 0

        def heads(cache, scale):
            x = cache[tables[b, lo // bs: -(-L // bs)]].transpose(0, 1).flatten(1, 2)[:, lo % bs: lo % bs + L - lo]
            return (x.view(torch.float8_e4m3fn).float() if c["fp8"] else x).double() * scale

        a = s["q"][b].double().view(Hkv, Hq // Hkv, D) @ heads(s["kc"], s["k_scale"]).transpose(1, 2) * s["scale"]
        out[b] = torch.softmax(a, -1) @ heads(s["vc"], s["v_scale"])
    return out.view(B, Hq, D)
