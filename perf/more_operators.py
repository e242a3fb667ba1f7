"""Cases of the codec LM's cache in 4 bits, of its pages, and of beam search: store, step, fork, compact, beams.

A server that keeps many long streams holds their keys and values in 4 bits:
`store` writes new rows and reads a context back for the attention of a prompt,
`step` attends over the cache as it lies. With beams, one selection per step
(`beams`) says which beams go on; `fork` gives each its pages, and `compact`
moves the pages that are held together when streams have ended.

`own` false computes them in elementary torch operations, `own` true calls
the library.

The cache in 4 bits: uint8 [blocks][kv_heads][block * dim * 5 / 8], in tiles of
16 positions of a head (10 * dim bytes). A value is low + scale * code, with
code 0 .. 15 and an fp16 pair (scale, low) for 32 values of a head; `_k_views`
and `_v_views` say where each lies.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DEVICE = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---- cases ------------------------------------------------------------------

def listed():
    return [
        # one token for each of 64 streams, five of them idle
        {"name": "store 64 rows", "op": "store", "requests": 64, "lo": 1, "hi": 1, "ctx_lo": 0, "ctx_hi": 0,
         "spread": 1, "idle": 5, "kv_heads": 8, "dim": 128, "type": "bf16", "in_type": "bf16", "block": 16},
        # new texts behind cached voice prompts, whose contexts are read back for their attention
        {"name": "store 16 behind contexts", "op": "store", "requests": 16, "lo": 1, "hi": 200, "ctx_lo": 1000,
         "ctx_hi": 4000, "spread": 2, "idle": 0, "kv_heads": 16, "dim": 64, "type": "fp16", "in_type": "fp32",
         "block": 32},
        # a full batch of prompts
        {"name": "store 24 prompts", "op": "store", "requests": 24, "lo": 700, "hi": 2000, "ctx_lo": 0, "ctx_hi": 0,
         "spread": 3, "idle": 0, "kv_heads": 8, "dim": 128, "type": "bf16", "in_type": "bf16", "block": 64},
        # the first stream of an empty server, 700 tokens in
        {"name": "step 1 alone", "op": "step", "requests": 1, "lo": 700, "hi": 700, "spread": 4, "shared": 0,
         "idle": 0, "q_heads": 16, "kv_heads": 8, "dim": 128, "type": "fp16", "block": 16},
        # 64 streams of an LM with 64-wide heads behind one voice prompt, five of them idle
        {"name": "step 64 shared", "op": "step", "requests": 64, "lo": 1, "hi": 1500, "spread": 5, "shared": 1024,
         "idle": 5, "q_heads": 16, "kv_heads": 16, "dim": 64, "type": "bf16", "block": 32},
        # 256 long-form streams behind a long voice prompt
        {"name": "step 256 long", "op": "step", "requests": 256, "lo": 500, "hi": 4000, "spread": 6, "shared": 8192,
         "idle": 0, "q_heads": 32, "kv_heads": 8, "dim": 128, "type": "bf16", "block": 64},
        # four utterances of four beams, two layers
        {"name": "fork 4 x 4", "op": "fork", "groups": 4, "beams": 4, "lo": 100, "hi": 400, "spread": 7, "ended": 0,
         "shared": 0, "short": 0, "kv_heads": 8, "dim": 128, "type": "bf16", "block": 16, "layers": 2},
        # 64 utterances of eight beams behind one voice prompt, three of them done, four layers
        {"name": "fork 64 x 8", "op": "fork", "groups": 64, "beams": 8, "lo": 200, "hi": 2000, "spread": 8, "ended": 3,
         "shared": 512, "short": 0, "kv_heads": 8, "dim": 128, "type": "bf16", "block": 32, "layers": 4},
        # a small server whose pages lie apart, one layer
        {"name": "compact 16", "op": "compact", "requests": 16, "lo": 100, "hi": 700, "spread": 9, "shared": 0,
         "held": 0.6, "kv_heads": 8, "dim": 128, "type": "fp16", "block": 16, "layers": 1},
        # 256 streams behind one voice prompt give a third of a pool back, two layers
        {"name": "compact 256", "op": "compact", "requests": 256, "lo": 200, "hi": 4000, "spread": 10, "shared": 1024,
         "held": 0.65, "kv_heads": 8, "dim": 128, "type": "bf16", "block": 32, "layers": 2},
        # one codebook's scores for four utterances of four beams
        {"name": "beams 4 x 4 of 2048", "op": "beams", "groups": 4, "beams": 4, "vocab": 2048, "in_type": "fp32",
         "ended": 2, "first": False},
        # 128 utterances of eight beams over a text vocabulary, of odd size
        {"name": "beams 128 x 8 of 65537", "op": "beams", "groups": 128, "beams": 8, "vocab": 65537, "in_type": "bf16",
         "ended": 60, "first": False},
    ]


def _log(rng, lo, hi):
    """A whole number of lo .. hi, even over its logarithm (lo may be 0)."""
    return min(hi, int((lo + 1) * math.exp(rng.random() * math.log((hi + 1) / (lo + 1)) + 1e-9) - 1 + rng.random()))


def draw(rng):
    heads = rng.choice([(16, 16, 64), (16, 8, 128), (32, 8, 128), (8, 1, 64), (12, 4, 128), (10, 2, 64), (7, 1, 128),
                        (16, 1, 128)])
    kind = rng.choice(["bf16", "fp16"])
    head = {"kv_heads": heads[1], "dim": heads[2], "type": kind}
    block = rng.choice([16, 32, 64, 128])
    spread = rng.randrange(1 << 20)
    op = rng.choice(["store", "step", "fork", "compact", "beams"])
    if op == "store":
        n, hi, ctx = _log(rng, 1, 48), _log(rng, 1, 1000), rng.choice([0, _log(rng, 10, 4000)])
        hi = min(hi, 1 + 40000 // n)
        ctx = min(ctx, 60000 // n)
        return {"op": op, "requests": n, "lo": rng.choice([1, 1 + hi // 3]), "hi": hi, "ctx_lo": ctx // 4,
                "ctx_hi": ctx, "spread": spread, "idle": rng.choice([0, 1]), **head,
                "in_type": rng.choice(["fp32", kind]), "block": block}
    if op == "step":
        hi = _log(rng, 1, 4000)
        return {"op": op, "requests": _log(rng, 1, 128), "lo": 1 + rng.choice([0, hi // 3]), "hi": max(hi, 2),
                "spread": spread, "shared": block * rng.choice([0, _log(rng, 0, 8192 // block)]), "idle": 0,
                "q_heads": heads[0], **head, "block": block}
    if op == "fork":
        g, k, hi = _log(rng, 1, 60), _log(rng, 1, 16), _log(rng, 1, 2000)
        return {"op": op, "groups": g, "beams": k, "lo": 1 + hi // 4, "hi": hi, "spread": spread,
                "ended": rng.choice([0, g // 5]), "shared": block * rng.choice([0, _log(rng, 1, 8)]),
                "short": rng.choice([0, 0, 3]), **head, "block": block, "layers": rng.choice([1, 2, 3])}
    if op == "compact":
        n, hi = _log(rng, 1, 250), _log(rng, 1, 3500)
        return {"op": op, "requests": n, "lo": 1 + hi // 8, "hi": hi, "spread": spread,
                "shared": block * rng.choice([0, _log(rng, 1, 30)]), "held": rng.choice([0.35, 0.7, 0.9, 0.99]), **head,
                "block": block, "layers": rng.choice([1, 2])}
    g, k, v = _log(rng, 1, 100), _log(rng, 1, 16), _log(rng, 40, 130000)
    v = max(k + 1, min(v, 60_000_000 // (g * k)))
    return {"op": op, "groups": g, "beams": k, "vocab": v, "in_type": rng.choice(["bf16", "fp16", "fp32"]),
            "ended": rng.choice([0, g * k // 8]), "first": rng.random() < 0.2}


def _lengths(case, lo, hi, salt=0, n=None):
    rng = random.Random(case["spread"] * 7 + salt)
    got = [_log(rng, case[lo], case[hi]) for _ in range(n or case["requests"])]
    got[rng.randrange(len(got))] = case[hi]
    return got


def _store_lengths(case):
    new, ctx = _lengths(case, "lo", "hi"), _lengths(case, "ctx_lo", "ctx_hi", 1)
    return new, [a + b for a, b in zip(new, ctx)]


def _step_lengths(case):
    lens = [case["shared"] + n for n in _lengths(case, "lo", "hi")]
    for i in random.Random(case["spread"]).sample(range(len(lens)), min(case["idle"], len(lens) - 1)):
        lens[i] = 0
    return lens


def _fork_rows(case):
    """Host lists of a group of beams each: length, blocks of its own that all
    its beams hold, and each row's parent row (-1: the utterance is done)."""
    rng = random.Random(case["spread"])
    g, k, blk, sh = case["groups"], case["beams"], case["block"], case["shared"]
    own_len = _lengths(case, "lo", "hi", n=g)
    trunk = [rng.randrange(n // blk + 1) for n in own_len]
    done = set(rng.sample(range(g), min(case["ended"], g - 1)))
    parents = []
    for i in range(g):
        # beams are chosen by score: the better ones have more children
        picked = sorted(min(int(rng.expovariate(3.0 / k)), k - 1) for _ in range(k))
        parents += [-1 if i in done else i * k + p for p in picked]
    return [sh + n for n in own_len], trunk, parents


def _copies(case):
    """Copies that a fork asks for: children, but the first, of a row whose last block is not full."""
    lens, _, parents = _fork_rows(case)
    k, seen, n = case["beams"], set(), 0
    for p in parents:
        if p >= 0 and p in seen and lens[p // k] % case["block"]:
            n += 1
        seen.add(p)
    return max(0, n - case["short"]) if case["short"] else n


def _block_bytes(case):
    return 2 * case["block"] * case["kv_heads"] * case["dim"]


def _compact_blocks(case):
    """Lengths, blocks held, blocks of the pool."""
    lens = [case["shared"] + n for n in _lengths(case, "lo", "hi")]
    sh = case["shared"] // case["block"]
    held = sh + sum(-(-n // case["block"]) - sh for n in lens)
    return lens, held, held + max(1, int(held * (1 / case["held"] - 1)))


def work(case):
    op = case["op"]
    if op == "beams":
        rows = case["groups"] * case["beams"]
        live = case["groups"] if case["first"] else rows - case["ended"]
        n = live * case["vocab"]
        return {"bytes": n * (4 if case["in_type"] == "fp32" else 2) + rows * 24, "flops": 4 * n}
    blk = case["block"]
    if op == "fork":
        lens, _, parents = _fork_rows(case)
        entries = sum(-(-lens[p // case["beams"]] // blk) for p in parents if p >= 0)
        return {"bytes": 8 * entries + 20 * len(parents) + 4 * case["layers"] * _copies(case) * _block_bytes(case),
                "flops": entries}
    if op == "compact":
        lens, held, pool = _compact_blocks(case)
        moved = held * (pool - held) / pool         # as many as chance puts behind the held ones' number
        entries = sum(-(-n // blk) for n in lens)
        return {"bytes": 8 * entries + 12 * pool + 4 * case["layers"] * moved * _block_bytes(case), "flops": entries}
    hk, d = case["kv_heads"], case["dim"]
    if op == "store":
        new, lens = _store_lengths(case)
        size = 4 if case["in_type"] == "fp32" else 2
        back = sum(-(-n // blk) for n in lens) * blk
        rows = sum(new) - min(case["idle"], sum(new) - 1)
        return {"bytes": 2 * hk * d * (rows * (size + 0.625) + back * (0.625 + 2)) + 4 * rows,
                "flops": 2 * hk * d * (4 * rows + 2 * back)}
    lens = _step_lengths(case)
    hq = case["q_heads"]
    keys = sum(n - case["shared"] for n in lens if n) + case["shared"]
    return {"bytes": len(lens) * 4 * hq * d + keys * hk * d * 1.25 + 4 * keys // blk, "flops": 4 * d * hq * sum(lens)}


# ---- the cache in 4 bits ----------------------------------------------------

def _k_views(cache, d):
    """Codes uint8 [block][head][tile][16 positions][4 words][group][4 bytes] (word t of a group holds its values
    8 t .. 8 t + 7, the lower half of a byte first) and fp16 [..][16 positions][group][scale, low]."""
    tiles = cache.unflatten(-1, (-1, 10 * d))
    return (tiles[..., : 8 * d].unflatten(-1, (16, 4, d // 32, 4)),
            tiles[..., 8 * d:].view(torch.float16).unflatten(-1, (16, d // 32, 2)))


def _v_views(cache, d):
    """Position p = 8 a + 2 t + b of a tile: codes uint8 [block][head][tile][a 2][r 8][t 4][group][b 2][2 bytes]
    (a group's values 4 r .. 4 r + 3) and fp16 [..][scale, low][t 4][group][a 2][b 2]."""
    tiles = cache.unflatten(-1, (-1, 10 * d))
    return (tiles[..., : 8 * d].unflatten(-1, (2, 8, 4, d // 32, 2, 2)),
            tiles[..., 8 * d:].view(torch.float16).unflatten(-1, (2, 4, d // 32, 2, 2)))


def _coded(x):
    """Codes uint8 [..][dim], scales and lows fp16 [..][groups] of x [..][dim] in 32 bits, step by step in 32 bits:
    the codes lie next to borders, so both sides take the same steps."""
    x = x.unflatten(-1, (-1, 32))
    good = x.isfinite().all(-1)
    x = x.clamp(-65504, 65504)
    lo, hi = x.amin(-1), x.amax(-1)
    low = lo.half()
    scale = ((hi - lo) * (1 / 15)).half()
    code = ((x - low.float()[..., None]) * (1 / scale.float())[..., None]).round().clamp(0, 15)
    code = torch.where((good & (scale > 0))[..., None], code, 0.0).to(torch.uint8).flatten(-2)
    nan = torch.full_like(low, math.nan)
    return code, torch.where(good, scale, nan), torch.where(good, low, nan)


def _bytes(code):
    return code[..., 0::2] | code[..., 1::2] << 4


def _write(k_cache, v_cache, blk, at, k, v):
    """Rows k, v [n][heads][dim] in 32 bits to position `at` of block `blk`."""
    d = k.shape[-1]
    tile, p = at // 16, at % 16
    code, scale, low = _coded(k)
    codes, params = _k_views(k_cache, d)
    codes[blk, :, tile, p] = _bytes(code).unflatten(-1, (-1, 4, 4)).transpose(-3, -2)
    params[blk, :, tile, p] = torch.stack([scale, low], -1)
    code, scale, low = _coded(v)
    codes, params = _v_views(v_cache, d)
    codes[blk, :, tile, p // 8, :, p // 2 % 4, :, p % 2] = _bytes(code).unflatten(-1, (-1, 8, 2)).transpose(-3, -2)
    params[blk, :, tile, :, p // 2 % 4, :, p // 8, p % 2] = torch.stack([scale, low], -2)


def _nibbles(b):
    return torch.stack([b & 15, b >> 4], -1).float()


def _k_values(cache, d):
    """[block][position][head][dim] in 32 bits."""
    codes, params = _k_views(cache, d)
    code = _nibbles(codes).permute(0, 2, 3, 1, 5, 4, 6, 7).flatten(5)       # block, tile, p, head, group, 32
    scale, low = params.permute(0, 2, 3, 1, 4, 5).float().unbind(-1)
    return (code * scale[..., None] + low[..., None]).flatten(4).flatten(1, 2)


def _v_values(cache, d):
    codes, params = _v_views(cache, d)
    code = _nibbles(codes).permute(0, 2, 3, 5, 7, 1, 6, 4, 8, 9).flatten(7)  # block, tile, a, t, b, head, group, 32
    scale, low = params.permute(0, 2, 6, 4, 7, 1, 5, 3).float().unbind(-1)   # block, tile, a, t, b, head, group
    return (code * scale[..., None] + low[..., None]).flatten(6).flatten(1, 4)


# ---- inputs -----------------------------------------------------------------

def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEVICE)


def _tables(gen, counts, width, n_blocks, shared=0):
    """Block tables [requests][width] of counts[b] blocks, each of its own in
    any order; the first `shared` blocks are the same ones for everybody."""
    perm = torch.randperm(n_blocks, generator=gen, device=DEVICE)
    c = torch.tensor([max(0, n - shared) for n in counts], device=DEVICE)
    first = shared + torch.cumsum(c, 0) - c
    j = torch.arange(width, device=DEVICE)
    at = torch.where(j < shared, j, first[:, None] + j - shared)
    held = j < torch.tensor(counts, device=DEVICE)[:, None]
    return torch.where(held, perm[at.clamp(max=n_blocks - 1)], 0).to(torch.int32), perm


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEVICE)


def _zeros(*shape):
    return torch.zeros(*shape, dtype=torch.int32, device=DEVICE)


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE).manual_seed(seed)
    s = {"case": case}
    conf = {"dtype": case.get("type", "bf16"), "q_heads": case.get("q_heads", case.get("kv_heads", 1)),
            "kv_heads": case.get("kv_heads", 1), "head_dim": case.get("dim", 64), "max_rows": 1, "max_requests": 1,
            "block_size": case.get("block", 16), "n_blocks": 1, "table_blocks": 1}
    {"store": _prepare_store, "step": _prepare_step, "fork": _prepare_fork, "compact": _prepare_compact,
     "beams": _prepare_beams}[case["op"]](case, gen, s, conf)
    if own:
        from streaming_tts_vocoder_gb300 import codec
        s["lm"] = codec.Lm(**conf)
    return s


def _caches4(case, blocks):
    shape = (blocks, case["kv_heads"], case["block"] * case["dim"] * 5 // 8)
    return (torch.zeros(shape, dtype=torch.uint8, device=DEVICE) for _ in range(2))


def _fill4(case, gen, s):
    """All positions of the cache, a part at a time. Keys as a norm and a rotation leave them, with a few strong
    channels; values with a spread of their own for each head."""
    n, hk, d, blk = s["k_cache"].shape[0], case["kv_heads"], case["dim"], case["block"]
    strong = 1 + 3 * (torch.rand(hk, d, generator=gen, device=DEVICE) < 0.03)
    spread = 0.2 + torch.rand(hk, 1, generator=gen, device=DEVICE)
    part = max(1, 32_000_000 // (blk * hk * d))
    for a in range(0, n, part):
        ids = torch.arange(a, min(a + part, n), device=DEVICE).repeat_interleave(blk)
        at = torch.arange(len(ids), device=DEVICE) % blk
        _write(s["k_cache"], s["v_cache"], ids, at, _normal(gen, len(ids), hk, d) * strong,
               _normal(gen, len(ids), hk, d) * spread)


def _prepare_store(case, gen, s, conf):
    new, lens = _store_lengths(case)
    hk, d, blk = case["kv_heads"], case["dim"], case["block"]
    counts = [-(-n // blk) for n in lens]
    rows, blocks, width = sum(new), sum(counts) + 3, max(counts)
    tables, _ = _tables(gen, counts, width, blocks)
    s["k_cache"], s["v_cache"] = _caches4(case, blocks)
    _fill4(case, gen, s)
    # one fused projection's output; k and v are views of it
    kv = _normal(gen, rows, 2 * hk * d).mul_(2).to(TYPES[case["in_type"]])
    s["k"], s["v"] = (t.unflatten(1, (hk, d)) for t in kv.split([hk * d, hk * d], 1))
    owner = torch.repeat_interleave(torch.arange(len(new), device=DEVICE), torch.tensor(new, device=DEVICE))
    starts = torch.tensor([sum(new[:i]) - (n - m) for i, (m, n) in enumerate(zip(new, lens))], device=DEVICE)
    pos = torch.arange(rows, device=DEVICE) - starts[owner]
    s["slots"] = (tables[owner, pos // blk] * blk + pos % blk).to(torch.int32)
    if case["idle"] and rows > case["idle"]:
        s["slots"][-case["idle"]:] = -1
    held = torch.arange(width, device=DEVICE) < torch.tensor(counts, device=DEVICE)[:, None]
    s["src"] = tables[held]                         # the contexts' blocks, request by request
    s["dst"] = torch.arange(sum(counts), device=DEVICE, dtype=torch.int32)
    s["k_out"], s["v_out"] = (torch.zeros(sum(counts), blk, hk, d, dtype=TYPES[case["type"]], device=DEVICE)
                              for _ in range(2))
    conf |= {"max_rows": rows, "n_blocks": blocks}


def _prepare_step(case, gen, s, conf):
    lens = _step_lengths(case)
    blk, hq, d = case["block"], case["q_heads"], case["dim"]
    counts = [-(-n // blk) for n in lens]
    sh = case["shared"] // blk
    blocks = sh + sum(max(0, c - sh) for c in counts) + 5
    width = max(counts) + 1
    s["k_cache"], s["v_cache"] = _caches4(case, blocks)
    _fill4(case, gen, s)
    s["tables"], perm = _tables(gen, counts, width, blocks, sh)
    s["shared_table"] = perm[:sh].to(torch.int32)
    s["kv_len"] = _i32(lens)
    s["q"] = _normal(gen, len(lens), hq, d).mul_(1.5).to(TYPES[case["type"]])
    s["o"] = torch.zeros_like(s["q"])
    conf |= {"max_requests": len(lens), "max_rows": len(lens), "n_blocks": blocks, "table_blocks": width}


def _caches16(case, gen, blocks, s):
    """Keys and values of all layers, [layers * 2][blocks][block][heads][dim], and a list of each."""
    s["caches"] = torch.empty(2 * case["layers"], blocks, case["block"], case["kv_heads"], case["dim"],
                              dtype=TYPES[case["type"]], device=DEVICE).normal_(generator=gen)
    s["layers"] = list(s["caches"])


def _prepare_fork(case, gen, s, conf):
    lens, trunk, parents = _fork_rows(case)
    g, k, blk = case["groups"], case["beams"], case["block"]
    sh = case["shared"] // blk
    counts = [-(-n // blk) for n in lens]
    held = sh + sum(t + k * (c - sh - t) for t, c in zip(trunk, counts))
    need = _copies(case)
    blocks = held + need + (0 if case["short"] else 9)
    free, width = blocks - held, max(counts) + 2
    perm = torch.randperm(blocks, generator=gen, device=DEVICE)
    # group i: `trunk` blocks of all its beams, then the beams' own ones
    c, t = (torch.tensor(v, device=DEVICE) for v in (counts, trunk))
    each = t + k * (c - sh - t)
    first = sh + torch.cumsum(each, 0) - each
    j = torch.arange(width, device=DEVICE) - sh
    i = torch.arange(k, device=DEVICE)[:, None]
    at = torch.where(j < t[:, None, None], j, t[:, None, None] + i * (c - sh - t)[:, None, None] + j - t[:, None, None])
    at = torch.where(j < 0, j + sh, first[:, None, None] + at)
    s["tables"] = torch.where(j + sh < c[:, None, None], perm[at.clamp(max=blocks - 1)], 0).flatten(0, 1).to(torch.int32)
    s["tables_out"] = torch.zeros_like(s["tables"])
    s["owners"] = _zeros(blocks)
    common = (j >= 0) & (j < t[:, None])
    s["owners"][s["tables"].unflatten(0, (g, k))[:, 0][common].long()] = k - 1
    head = 5 * blocks + 3                   # the ring of free blocks has been round a few times
    ring = _zeros(blocks)
    ring[(head + torch.arange(free, device=DEVICE)) % blocks] = perm[held:].to(torch.int32)
    s["free_list"], s["free"] = ring, torch.tensor([head, head + free], device=DEVICE)
    s["free_out"] = torch.zeros(2, dtype=torch.int64, device=DEVICE)
    s["parents"], s["kv_len"] = _i32(parents), _i32(lens).repeat_interleave(k)
    rows = g * k
    for name, size in (("kv_out", rows), ("status", rows), ("owners_out", blocks), ("src", rows), ("dst", rows),
                       ("count", 1)):
        s[name] = _zeros(size)
    _caches16(case, gen, blocks, s)
    conf |= {"max_requests": rows, "n_blocks": blocks, "table_blocks": width}


def _prepare_compact(case, gen, s, conf):
    lens, held, blocks = _compact_blocks(case)
    blk = case["block"]
    sh = case["shared"] // blk
    counts = [-(-n // blk) for n in lens]
    width = max(counts) + 2
    s["tables"], perm = _tables(gen, counts, width, blocks, sh)
    s["tables_out"] = torch.zeros_like(s["tables"])
    s["shared_table"] = perm[:sh].to(torch.int32)
    s["shared_out"] = torch.zeros_like(s["shared_table"])
    s["kv_len"] = _i32(lens)
    s["free_out"] = torch.zeros(2, dtype=torch.int64, device=DEVICE)
    for name, size in (("owners", blocks), ("owners_out", blocks), ("free_list", blocks), ("src", blocks // 2),
                       ("dst", blocks // 2), ("count", 1)):
        s[name] = _zeros(size)
    _caches16(case, gen, blocks, s)
    conf |= {"max_requests": len(lens), "n_blocks": blocks, "table_blocks": width}


def _prepare_beams(case, gen, s, conf):
    rows, v = case["groups"] * case["beams"], case["vocab"]
    x = torch.empty(rows, v, dtype=TYPES[case["in_type"]], device=DEVICE).normal_(generator=gen).mul_(2.5)
    s["logits"] = x
    s["sums"] = _normal(gen, rows).abs_().mul_(-4).sub_(20)
    s["ended"] = _zeros(rows)
    if case["first"]:                       # one beam of each utterance is there yet
        s["sums"].view(-1, case["beams"])[:, 1:] = -math.inf
    else:
        s["ended"][torch.randperm(rows, generator=gen, device=DEVICE)[: case["ended"]]] = 1
    s["end"] = v - 1
    s["sums_out"] = torch.zeros(rows, device=DEVICE)
    s["parents"], s["tokens"], s["ended_out"] = _zeros(rows), _zeros(rows), _zeros(rows)
    conf |= {"max_requests": rows}


# ---- one pass ---------------------------------------------------------------

def run(s):
    return {"store": _store, "step": _step, "fork": _fork, "compact": _compact, "beams": _beams}[s["case"]["op"]](s)


def _store(s):
    if own:
        s["lm"].store_q4(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"])
        s["lm"].load_q4(s["k_cache"], s["v_cache"], s["src"], s["dst"], s["k_out"], s["v_out"])
        return {"k": s["k_out"], "v": s["v_out"]}
    d, blk, dt = s["case"]["dim"], s["case"]["block"], s["k_out"].dtype
    held = s["slots"] >= 0
    to = s["slots"][held].long()
    _write(s["k_cache"], s["v_cache"], to // blk, to % blk, s["k"][held].float(), s["v"][held].float())
    src, dst = s["src"].long(), s["dst"].long()
    s["k_out"][dst] = _k_values(s["k_cache"][src], d).to(dt)
    s["v_out"][dst] = _v_values(s["v_cache"][src], d).to(dt)
    return {"k": s["k_out"], "v": s["v_out"]}


def _step(s):
    if own:
        s["lm"].step_q4(s["q"], s["k_cache"], s["v_cache"], s["tables"], s["kv_len"], s["o"],
                        shared_table=s["shared_table"])
        return s["o"]
    q, d = s["q"].float(), s["case"]["dim"]
    k = _k_values(s["k_cache"], d)[s["tables"].long()].flatten(1, 2)
    v = _v_values(s["v_cache"], d)[s["tables"].long()].flatten(1, 2)
    b, m, hk = k.shape[:3]
    x = (q.view(b, hk, -1, d) @ k.permute(0, 2, 3, 1)).mul_(1 / math.sqrt(d))
    seen = torch.arange(m, device=q.device) < s["kv_len"][:, None]
    x = x.masked_fill_(~seen[:, None, None], -math.inf)
    x = x.sub_(x.amax(-1, keepdim=True).clamp(min=-1e30)).exp_()
    o = (x @ v.permute(0, 2, 1, 3)) / x.sum(-1, keepdim=True).clamp(min=1e-30)
    return o.reshape(q.shape).to(s["o"].dtype)


def _fork(s):
    if own:
        shared = s["case"]["shared"] // s["case"]["block"]
        s["lm"].fork(s["parents"], s["kv_len"], s["tables"], s["tables_out"], s["owners"], s["owners_out"],
                     s["free_list"], s["free"], s["free_out"], s["kv_out"], s["status"], s["src"], s["dst"],
                     s["count"], shared_blocks=shared)
        s["lm"].copy_blocks(s["layers"], s["src"], s["dst"], s["count"])
        return {k: s[k] for k in ("tables_out", "owners_out", "free_list", "free_out", "kv_out", "status", "src",
                                  "dst", "count", "caches")}
    blk, sh = s["case"]["block"], s["case"]["shared"] // s["case"]["block"]
    tables, ring, n = s["tables"].long(), s["free_list"], s["free_list"].numel()
    b, width = tables.shape
    parents, lens = s["parents"].long(), s["kv_len"].long()
    row, j = torch.arange(b, device=DEVICE), torch.arange(width, device=DEVICE)
    good = (parents >= -1) & (parents < b)
    live = good & (parents >= 0)
    p = parents.clamp(0, b - 1)
    count = (lens + blk - 1) // blk
    part = (lens % blk != 0) & (count > sh)             # the last block is the row's own and not full
    first = torch.full_like(row, b).scatter_reduce(0, torch.where(live, p, 0), torch.where(live, row, b), "amin")
    needs = live & part[p] & (first[p] != row)
    upto = torch.cumsum(needs, 0)
    head, tail = s["free"][0], s["free"][1]
    ok = live & (~needs | (upto <= tail - head))
    taken = (needs & ok).sum()
    children = torch.zeros_like(row).scatter_add(0, p, ok.long())
    last = part[:, None] & (j == count[:, None] - 1)
    more = torch.where(last, children.clamp(max=1)[:, None], children[:, None]) - 1
    more = torch.where((j >= sh) & (j < count[:, None]), more, 0)
    owners = s["owners"].long().index_add(0, tables.flatten(), more.flatten())
    freed = owners < 0
    ids = torch.arange(n, device=DEVICE)
    to = torch.where(freed, (tail + torch.cumsum(freed, 0) - 1) % n, n)
    new = ring[((head + upto - 1) % n)]
    copy = needs & ok
    end = count[p] - 1
    old = tables[p, end.clamp(min=0)]
    out = torch.where(ok[:, None] & (j < count[p][:, None]), tables[p], s["tables_out"].long())
    out = torch.where(copy[:, None] & (j == end[:, None]), new[:, None].long(), out)
    ring = torch.nn.functional.pad(ring, (0, 1)).scatter(0, to, ids.int())[:n]
    at = torch.where(copy, upto - 1, b)
    src = torch.nn.functional.pad(s["src"], (0, 1)).scatter(0, at, old.int())[:b]
    dst = torch.nn.functional.pad(s["dst"], (0, 1)).scatter(0, at, new)[:b]
    s["caches"][:, new[copy].long()] = s["caches"][:, old[copy]]
    return {"tables_out": out.int(), "owners_out": owners.clamp(min=0).int(), "free_list": ring,
            "free_out": torch.stack([head + taken, tail + freed.sum()]),
            "kv_out": torch.where(ok, lens[p], 0).int(),
            "status": torch.where(~good, 2, torch.where(live & ~ok, 1, 0)).int(), "src": src, "dst": dst,
            "count": taken.int().view(1), "caches": s["caches"]}


def _compact(s):
    if own:
        s["lm"].compact(s["kv_len"], s["tables"], s["tables_out"], s["owners"], s["owners_out"], s["free_list"],
                        s["free_out"], s["src"], s["dst"], s["count"], shared_table=s["shared_table"],
                        shared_out=s["shared_out"])
        s["lm"].copy_blocks(s["layers"], s["src"], s["dst"], s["count"])
        return {k: s[k] for k in ("tables_out", "shared_out", "owners_out", "free_list", "free_out", "src", "dst",
                                  "count", "caches")}
    blk, sh = s["case"]["block"], s["shared_table"].numel()
    tables, n, m = s["tables"].long(), s["free_list"].numel(), s["src"].numel()
    j = torch.arange(tables.shape[1], device=DEVICE)
    held = j < ((s["kv_len"] + blk - 1) // blk)[:, None]
    used = torch.zeros(n + 1, dtype=torch.bool, device=DEVICE)
    used[torch.where(held & (j >= sh), tables, n).flatten()] = True
    used[s["shared_table"].long()] = True
    used = used[:n]
    ids, most = torch.arange(n, device=DEVICE), used.sum()
    away, room = used & (ids >= most), ~used & (ids < most)
    k, to = torch.cumsum(away, 0) - 1, torch.cumsum(room, 0) - 1
    src = torch.nn.functional.pad(s["src"], (0, 1)).scatter(0, torch.where(away, k, m), ids.int())[:m]
    dst = torch.nn.functional.pad(s["dst"], (0, 1)).scatter(0, torch.where(room, to, m), ids.int())[:m]
    moved = away.sum()
    where = torch.where(away, torch.nn.functional.pad(dst, (0, 1)).long()[k.clamp(0, m)], ids)
    owners = torch.zeros(n + 1, dtype=torch.int32, device=DEVICE).scatter(0, torch.where(used, where, n), s["owners"])
    free = torch.where(ids < n - most, most + ids, s["free_list"].long())
    take = torch.arange(m, device=DEVICE) < moved
    s["caches"][:, dst[take].long()] = s["caches"][:, src[take].long()]
    return {"tables_out": torch.where(held, where[tables], s["tables_out"].long()).int(),
            "shared_out": where[s["shared_table"].long()].int(), "owners_out": owners[:n], "free_list": free.int(),
            "free_out": torch.stack([torch.zeros_like(most), n - most]), "src": src, "dst": dst,
            "count": moved.int().view(1), "caches": s["caches"]}


def _beams(s):
    if own:
        s["lm"].beams(s["logits"], s["case"]["beams"], s["sums"], s["ended"], s["end"], s["sums_out"], s["parents"],
                      s["tokens"], s["ended_out"])
        return {k: s[k] for k in ("sums_out", "parents", "tokens", "ended_out")}
    k, end = s["case"]["beams"], s["end"]
    x = s["logits"].double()            # candidates of two beams may lie closer than 32 bits tell
    rows, v = x.shape
    top = x.amax(-1, keepdim=True)
    x = x - (top + (x - top).exp().sum(-1, keepdim=True).log()) + s["sums"].double()[:, None]
    ended = s["ended"][:, None] != 0
    only = torch.arange(v, device=x.device) == end
    x = torch.where(ended, torch.where(only, s["sums"].double()[:, None], -math.inf), x)
    x = torch.where(x.isfinite(), x, -math.inf).view(-1, k * v)
    best, at = (t[:, :k] for t in torch.sort(x, dim=-1, descending=True, stable=True))
    there = best > -math.inf
    base = torch.arange(0, rows, k, device=x.device)[:, None]
    token = torch.where(there, at % v, -1)
    return {"sums_out": best.float().flatten(), "parents": torch.where(there, base + at // v, -1).int().flatten(),
            "tokens": token.int().flatten(), "ended_out": (~there | (token == end)).int().flatten()}


# ---- the definition in 64 bits ----------------------------------------------

def exact(case, seed):
    if case["op"] in ("fork", "compact"):
        return None         # whole numbers and moved blocks: equal, or not
    s = prepare(case, seed)
    return {"store": _exact_store, "step": _exact_step, "beams": _exact_beams}[case["op"]](case, s)


def _places(d, keys):
    """For each position p of a tile and element i of a head: which byte of the tile, whether the upper half, and
    the bytes of its scale and low."""
    p, i = torch.arange(16, device=DEVICE)[:, None], torch.arange(d, device=DEVICE)
    g, e = i // 32, i % 32
    if keys:
        byte = p * (d // 2) + (e // 8 * (d // 32) + g) * 4 + e % 8 // 2
        scale = 8 * d + p * (d // 8) + g * 4
        return byte, e % 2, scale, scale + 2
    t, a, b = p % 8 // 2, p // 8, p % 2
    byte = a * 4 * d + (e // 4 * 4 + t) * (d // 8) + g * 4 + b * 2 + e % 4 // 2
    scale = 8 * d + ((t * (d // 32) + g) * 4 + 2 * a + b) * 2
    return byte, e % 2, scale, scale + d


def _half(tiles, at):
    """The fp16 numbers at bytes `at`, taken apart: sign, exponent, fraction."""
    bits = tiles[..., at].long() + 256 * tiles[..., at + 1].long()
    e, f = bits // 1024 % 32, bits % 1024
    x = torch.where(e == 0, f * 2.0 ** -24, (1024 + f) * torch.pow(2.0, e.double() - 25))
    return torch.where(bits >= 32768, -x, x)


def _exact_values(cache, d, keys):
    """[blocks][positions][heads][dim] of uint8 [blocks][heads][bytes] in 64 bits."""
    byte, upper, scale, low = _places(d, keys)
    tiles = cache.unflatten(-1, (-1, 10 * d))
    code = tiles[..., byte].long()
    code = torch.where(upper == 1, code // 16, code % 16).double()
    return (_half(tiles, low) + _half(tiles, scale) * code).permute(0, 2, 3, 1, 4).flatten(1, 2)


def _rounded(x):
    """x [..][dim] in 64 bits as what its 4 bits stand for. The steps whose rounding the format fixes are rounded."""
    x = x.unflatten(-1, (-1, 32)).clamp(-65504, 65504)
    lo, hi = x.min(-1, keepdim=True).values, x.max(-1, keepdim=True).values
    third = torch.tensor(1 / 15, dtype=torch.float32).double().item()
    scale = ((hi - lo).float().double() * third).float().half().double()
    low = lo.half().double()
    inverse = (1 / scale).float().double()
    steps = ((x - low).float().double() * inverse).float().round().clamp(0, 15).double()
    return torch.where(scale > 0, low + scale * steps, low.expand_as(x)).flatten(-2)


def _exact_store(case, s):
    d, blk = case["dim"], case["block"]
    new = {"k": s["k"], "v": s["v"]}
    row = torch.full((s["k_cache"].shape[0] * blk,), -1, dtype=torch.long, device=DEVICE)
    slots = s["slots"].long()
    row[slots[slots >= 0]] = torch.arange(len(slots), device=DEVICE)[slots >= 0]
    got = {}
    for name in ("k", "v"):
        out = torch.zeros(s["k_out"].shape, dtype=torch.float64, device=DEVICE)
        for a in range(0, len(s["src"]), 200):
            ids = s["src"][a:a + 200].long()
            was = _exact_values(s[name + "_cache"][ids], d, name == "k")
            here = row.view(-1, blk)[ids]
            now = _rounded(new[name].double()[here.clamp(min=0)])
            out[s["dst"][a:a + 200].long()] = torch.where((here >= 0)[..., None, None], now, was)
        got[name] = out
    return got


def _exact_step(case, s):
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEVICE)
    d, hk, blk = case["dim"], case["kv_heads"], case["block"]
    for i, n in enumerate(s["kv_len"].tolist()):
        if n:
            ids = s["tables"][i, : -(-n // blk)].long()
            k, v = (_exact_values(s[c][ids], d, c == "k_cache").flatten(0, 1)[:n] for c in ("k_cache", "v_cache"))
            x = torch.einsum("hgd,mhd->hgm", s["q"][i].double().view(hk, -1, d), k) / math.sqrt(d)
            o[i] = torch.einsum("hgm,mhd->hgd", torch.softmax(x, -1), v).reshape(-1, d)
    return o


def _exact_beams(case, s):
    """The sums alone: what goes on where is whole numbers."""
    k = case["beams"]
    sums = s["sums"].double()
    got = torch.full((len(sums), k), -math.inf, dtype=torch.float64, device=DEVICE)
    for r, ended in enumerate(s["ended"].tolist()):
        if ended:
            got[r, 0] = sums[r]
        else:
            got[r, : min(k, case["vocab"])] = sums[r] + torch.topk(
                torch.log_softmax(s["logits"][r].double(), -1), min(k, case["vocab"])).values
    best = torch.topk(got.view(-1, k * k), k).values.flatten()
    return {"sums_out": best, "parents": None, "tokens": None, "ended_out": None}
