"""Cases of the codec LM's attention operators: plan, rotate, prompt and step.

A codec LM reads a prompt (text and a voice sample) and then makes one code
frame per step for every stream; the decoder turns the frames into audio.
One attention layer of it is, per call: `plan` (which cache blocks the new
tokens go to), `rotate` (norms of queries and keys, position rotation, store
into the cache), and `prompt` or `step` (the attention over it).

`own` false computes them in elementary torch operations, `own` true calls
the library.
"""
from __future__ import annotations

import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
THETA, EPS = 1e6, 1e-6


# ---- cases ------------------------------------------------------------------

def listed():
    return [
        # every stream of a 64-stream server gets its next token: the smallest call, once per step
        {"name": "plan 64 x 1", "op": "plan", "requests": 64, "old_lo": 40, "old_hi": 2000, "new_lo": 1, "new_hi": 1,
         "spread": 1, "done": 3, "shared": 0, "block": 16, "short": 0},
        # a queue of 1000 requests behind one voice prompt is admitted at once
        {"name": "plan 1000 prompts", "op": "plan", "requests": 1000, "old_lo": 0, "old_hi": 0, "new_lo": 25,
         "new_hi": 2000, "spread": 2, "done": 0, "shared": 512, "block": 32, "short": 0},
        # one token for each of 64 streams, five of them idle (rows kept so that one graph serves all steps)
        {"name": "rotate 64 rows", "op": "rotate", "rows": 64, "idle": 5, "q_heads": 16, "kv_heads": 8, "dim": 128,
         "type": "bf16", "in_type": "bf16", "pairs": False, "norm": True, "far": 4000, "block": 16},
        # prompts of an LM with 64-wide heads whose projections come in fp32
        {"name": "rotate 4097 rows", "op": "rotate", "rows": 4097, "idle": 0, "q_heads": 16, "kv_heads": 16,
         "dim": 64, "type": "fp16", "in_type": "fp32", "pairs": True, "norm": True, "far": 30000, "block": 32},
        # a full batch of prompts
        {"name": "rotate 32768 rows", "op": "rotate", "rows": 32768, "idle": 0, "q_heads": 32, "kv_heads": 8,
         "dim": 128, "type": "bf16", "in_type": "bf16", "pairs": False, "norm": True, "far": 32768, "block": 64},
        # eight short texts of 1 to 97 tokens
        {"name": "prompt 8 short", "op": "prompt", "requests": 8, "lo": 1, "hi": 97, "spread": 3, "q_heads": 16,
         "kv_heads": 16, "dim": 64, "type": "fp16"},
        # a ragged batch of texts with voice samples
        {"name": "prompt 24 ragged", "op": "prompt", "requests": 24, "lo": 60, "hi": 1500, "spread": 4, "q_heads": 16,
         "kv_heads": 8, "dim": 128, "type": "bf16"},
        # long-form texts: 9000 tokens, with a shorter one beside it
        {"name": "prompt 2 long", "op": "prompt", "requests": 2, "lo": 5001, "hi": 9000, "spread": 5, "q_heads": 32,
         "kv_heads": 8, "dim": 128, "type": "bf16"},
        # new texts behind a cached voice prompt, in cache blocks
        {"name": "prompt 16 paged", "op": "paged", "requests": 16, "lo": 1, "hi": 200, "ctx_lo": 1000, "ctx_hi": 4000,
         "spread": 6, "q_heads": 16, "kv_heads": 8, "dim": 128, "type": "bf16", "block": 16},
        # the first stream of an empty server, 700 tokens in
        {"name": "step 1 alone", "op": "step", "requests": 1, "lo": 700, "hi": 700, "spread": 7, "shared": 0,
         "idle": 0, "q_heads": 16, "kv_heads": 8, "dim": 128, "type": "fp16", "block": 16},
        # 64 streams behind one voice prompt
        {"name": "step 64 shared", "op": "step", "requests": 64, "lo": 1, "hi": 500, "spread": 8, "shared": 1024,
         "idle": 5, "q_heads": 16, "kv_heads": 8, "dim": 128, "type": "bf16", "block": 16},
        # 256 long-form streams behind a long voice prompt
        {"name": "step 256 long", "op": "step", "requests": 256, "lo": 500, "hi": 4000, "spread": 9, "shared": 8192,
         "idle": 0, "q_heads": 32, "kv_heads": 8, "dim": 128, "type": "bf16", "block": 64},
    ]


def _log(rng, lo, hi):
    """A whole number of lo .. hi, even over its logarithm (lo may be 0)."""
    return min(hi, int((lo + 1) * math.exp(rng.random() * math.log((hi + 1) / (lo + 1)) + 1e-9) - 1 + rng.random()))


def draw(rng):
    heads = rng.choice([(16, 16, 64), (16, 8, 128), (32, 8, 128), (8, 1, 64), (12, 4, 128), (10, 2, 64), (7, 1, 128)])
    head = {"q_heads": heads[0], "kv_heads": heads[1], "dim": heads[2], "type": rng.choice(["bf16", "fp16"])}
    block = rng.choice([16, 32, 64, 128])
    spread = rng.randrange(1 << 20)
    op = rng.choice(["plan", "rotate", "prompt", "paged", "step"])
    if op == "plan":
        new = _log(rng, 1, 1000)
        old = rng.choice([0, _log(rng, 10, 2000)])
        return {"op": op, "requests": _log(rng, 1, 900), "old_lo": old // 3, "old_hi": old, "new_lo": 1 + new // 9,
                "new_hi": new, "spread": spread, "done": rng.randrange(4) if old else 0,
                "shared": block * _log(rng, 0, 8), "block": block, "short": rng.choice([0, 0, _log(rng, 1, 30)])}
    if op == "rotate":
        return {"op": op, "rows": _log(rng, 1, 16000), "idle": rng.choice([0, 1]), **head,
                "in_type": rng.choice(["fp32", head["type"]]), "pairs": rng.random() < 0.5, "norm": rng.random() < 0.8,
                "far": _log(rng, 100, 60000), "block": block}
    if op == "prompt":
        n, hi = _log(rng, 1, 32), _log(rng, 1, 5000)
        hi = min(hi, max(1, int(8000 / math.sqrt(n))))
        return {"op": op, "requests": n, "lo": rng.choice([0, 1 + hi // 3]) if n > 1 else hi, "hi": hi,
                "spread": spread, **head}
    if op == "paged":
        n, hi, ctx = _log(rng, 1, 24), _log(rng, 1, 1000), _log(rng, 1, 6000)
        hi = min(hi, max(1, 40_000_000 // (n * (ctx + hi))))
        return {"op": op, "requests": n, "lo": rng.choice([1, 1 + hi // 3]), "hi": hi,
                "ctx_lo": ctx // 4, "ctx_hi": ctx, "spread": spread, **head, "block": block}
    hi = _log(rng, 1, 4000)
    return {"op": op, "requests": _log(rng, 1, 128), "lo": 1 + rng.choice([0, hi // 3]), "hi": max(hi, 2),
            "spread": spread, "shared": block * rng.choice([0, _log(rng, 0, 8192 // block)]), "idle": 0, **head,
            "block": block}


def _lengths(case, lo, hi, salt=0):
    rng = random.Random(case["spread"] * 7 + salt)
    got = [_log(rng, case[lo], case[hi]) for _ in range(case["requests"])]
    got[rng.randrange(len(got))] = case[hi]
    return got


def _plan_lengths(case):
    """Host lists: length of each request before and after the call. A
    request that ends goes to 0; the others grow."""
    before = [case["shared"] + n if n else case["shared"] for n in _lengths(case, "old_lo", "old_hi")]
    after = [b + n for b, n in zip(before, _lengths(case, "new_lo", "new_hi", 1))]
    ends = random.Random(case["spread"]).sample(range(len(after)), min(case["done"], len(after)))
    return before, [0 if i in ends else a for i, a in enumerate(after)]


def _owned(n, case):
    return max(0, -(-n // case["block"]) - case["shared"] // case["block"])


def work(case):
    op = case["op"]
    if op == "plan":
        before, after = _plan_lengths(case)
        rows = sum(max(0, a - b) for a, b in zip(after, before))
        moved = sum(abs(_owned(a, case) - _owned(b, case)) for a, b in zip(after, before))
        return {"bytes": 20 * len(after) + 8 * rows + 8 * moved, "flops": 4 * rows}
    hq, hk, d = case["q_heads"], case["kv_heads"], case["dim"]
    if op == "rotate":
        per = (hq + 2 * hk) * d
        size = 4 if case["in_type"] == "fp32" else 2
        n = case["rows"] - case["idle"] if case["rows"] > case["idle"] else case["rows"]
        return {"bytes": n * (per * (size + 2) + 8) + 8 * d, "flops": n * (hq + hk) * d * 7}
    if op == "prompt":
        lens = _lengths(case, "lo", "hi")
        return {"bytes": sum(lens) * 4 * (hq + hk) * d, "flops": 2 * d * hq * sum(n * (n + 1) for n in lens)}
    if op == "paged":
        lens, ctx = _lengths(case, "lo", "hi"), _lengths(case, "ctx_lo", "ctx_hi", 1)
        keys = sum(lens) + sum(ctx)
        pairs = sum(n * c + n * (n + 1) // 2 for n, c in zip(lens, ctx))
        return {"bytes": sum(lens) * 4 * hq * d + keys * (4 * hk * d) + 4 * keys // case["block"],
                "flops": 4 * d * hq * pairs}
    lens = _step_lengths(case)
    keys = sum(n - case["shared"] for n in lens if n) + case["shared"]
    return {"bytes": len(lens) * 4 * hq * d + keys * 4 * hk * d + 4 * keys // case["block"],
            "flops": 4 * d * hq * sum(lens)}


def _step_lengths(case):
    lens = [case["shared"] + n for n in _lengths(case, "lo", "hi")]
    for i in random.Random(case["spread"]).sample(range(len(lens)), min(case["idle"], len(lens) - 1)):
        lens[i] = 0
    return lens


# ---- inputs -----------------------------------------------------------------

def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _tables(gen, counts, width, n_blocks, shared=0):
    """Block tables [requests][width] of counts[b] blocks, each of its own in
    any order; the first `shared` blocks are the same ones for everybody."""
    perm = torch.randperm(n_blocks, generator=gen, device="cuda")
    c = torch.tensor([max(0, n - shared) for n in counts], device="cuda")
    first = shared + torch.cumsum(c, 0) - c
    j = torch.arange(width, device="cuda")
    at = torch.where(j < shared, j, first[:, None] + j - shared)
    held = j < torch.tensor(counts, device="cuda")[:, None]
    return torch.where(held, perm[at.clamp(max=n_blocks - 1)], 0).to(torch.int32), perm


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    s = {"case": case}
    conf = {"dtype": "bf16", "q_heads": 16, "kv_heads": 8, "head_dim": 128, "max_rows": 1, "max_requests": 1,
            "block_size": case.get("block", 16), "n_blocks": 1, "table_blocks": 1}
    if op == "plan":
        _prepare_plan(case, gen, s, conf)
    else:
        conf |= {"dtype": case["type"], "q_heads": case["q_heads"], "kv_heads": case["kv_heads"],
                 "head_dim": case["dim"]}
        {"rotate": _prepare_rotate, "prompt": _prepare_prompt, "paged": _prepare_paged,
         "step": _prepare_step}[op](case, gen, s, conf)
    if own:
        from streaming_tts_vocoder_gb300 import codec
        s["lm"] = codec.Lm(**conf)
    return s


def _prepare_plan(case, gen, s, conf):
    before, after = _plan_lengths(case)
    blk, sh = case["block"], case["shared"] // case["block"]
    counts = [-(-b // blk) if b > case["shared"] else 0 for b in before]  # fresh requests have nothing yet
    need = sum(max(0, _owned(a, case) - _owned(b, case)) for a, b in zip(after, before))
    held = sh + sum(max(0, c - sh) for c in counts)
    free = max(0, need - case["short"]) if case["short"] else need + 40
    n = held + free
    width = max(-(-max(max(a, b) for a, b in zip(after, before)) // blk), sh) + 3
    s["tables"], perm = _tables(gen, counts, width, n, sh)
    s["shared_table"] = perm[:sh].to(torch.int32)
    head = 5 * n + 3                        # the ring of free blocks has been round a few times
    ring = torch.zeros(n, dtype=torch.int32, device="cuda")
    ring[(head + torch.arange(free, device="cuda")) % n] = perm[held:].to(torch.int32)
    s["free_list"], s["free"] = ring, torch.tensor([head, head + free], device="cuda")
    rows = sum(max(0, a - b) for a, b in zip(after, before)) + 7
    s["before"], s["after"] = _i32(before), _i32(after)
    b = case["requests"]
    s["free_out"] = torch.zeros(2, dtype=torch.int64, device="cuda")
    for name, size in (("row_start", b + 1), ("kv_len", b), ("status", b), ("slots", rows), ("positions", rows)):
        s[name] = torch.zeros(size, dtype=torch.int32, device="cuda")
    conf |= {"max_requests": b, "max_rows": rows, "n_blocks": n, "table_blocks": width}


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _prepare_rotate(case, gen, s, conf):
    n, hq, hk, d, blk = case["rows"], case["q_heads"], case["kv_heads"], case["dim"], case["block"]
    dt = TYPES[case["type"]]
    # one fused projection's output; q, k and v are views of it
    qkv = _normal(gen, n, (hq + 2 * hk) * d).mul_(3).to(TYPES[case["in_type"]])
    s["q"], s["k"], s["v"] = (t.unflatten(1, (-1, d)) for t in qkv.split([hq * d, hk * d, hk * d], 1))
    s["q_gain"], s["k_gain"] = ((1 + 0.1 * _normal(gen, d)) if case["norm"] else None for _ in range(2))
    s["positions"] = torch.randint(case["far"], (n,), generator=gen, device="cuda", dtype=torch.int32)
    blocks = -(-n // blk) + 2
    s["slots"] = torch.randperm(blocks * blk, generator=gen, device="cuda")[:n].to(torch.int32)
    if case["idle"] and n > case["idle"]:
        s["slots"][-case["idle"]:] = -1
    s["k_cache"], s["v_cache"] = (torch.zeros(blocks, blk, hk, d, dtype=dt, device="cuda") for _ in range(2))
    s["q_out"] = torch.zeros(n, hq, d, dtype=dt, device="cuda")
    conf |= {"max_rows": n, "n_blocks": blocks, "max_positions": case["far"], "rope_theta": THETA,
             "rope_pairs": case["pairs"], "rms_eps": EPS}


def _prepare_prompt(case, gen, s, conf):
    lens = _lengths(case, "lo", "hi")
    n, hq, hk, d, dt = sum(lens), case["q_heads"], case["kv_heads"], case["dim"], TYPES[case["type"]]
    s["q"] = _normal(gen, n, hq, d).mul_(1.5).to(dt)
    s["k"] = _normal(gen, n, hk, d).to(dt)
    s["v"] = _normal(gen, n, hk, d).to(dt)
    s["row_start"] = _i32([sum(lens[:i]) for i in range(len(lens) + 1)])
    s["o"] = torch.zeros(n, hq, d, dtype=dt, device="cuda")
    s["longest"] = max(lens)
    conf |= {"max_requests": len(lens), "max_rows": n}


def _cache(case, gen, s, conf, lens, shared=0):
    blk, hk, d, dt = case["block"], case["kv_heads"], case["dim"], TYPES[case["type"]]
    counts = [-(-n // blk) for n in lens]
    sh = shared // blk
    blocks = sh + sum(max(0, c - sh) for c in counts) + 5
    width = max(counts) + 1
    s["k_cache"], s["v_cache"] = (torch.empty(blocks, blk, hk, d, dtype=dt, device="cuda").normal_(generator=gen)
                                  for _ in range(2))
    s["tables"], perm = _tables(gen, counts, width, blocks, sh)
    s["shared_table"] = perm[:sh].to(torch.int32)
    s["kv_len"] = _i32(lens)
    conf |= {"max_requests": len(lens), "n_blocks": blocks, "table_blocks": width}


def _prepare_paged(case, gen, s, conf):
    lens, ctx = _lengths(case, "lo", "hi"), _lengths(case, "ctx_lo", "ctx_hi", 1)
    n, hq, d, dt = sum(lens), case["q_heads"], case["dim"], TYPES[case["type"]]
    _cache(case, gen, s, conf, [a + b for a, b in zip(lens, ctx)])
    s["q"] = _normal(gen, n, hq, d).mul_(1.5).to(dt)
    s["row_start"] = _i32([sum(lens[:i]) for i in range(len(lens) + 1)])
    s["o"] = torch.zeros(n, hq, d, dtype=dt, device="cuda")
    s["longest"] = max(lens)
    conf |= {"max_rows": n}


def _prepare_step(case, gen, s, conf):
    lens = _step_lengths(case)
    hq, d, dt = case["q_heads"], case["dim"], TYPES[case["type"]]
    _cache(case, gen, s, conf, lens, case["shared"])
    s["q"] = _normal(gen, len(lens), hq, d).mul_(1.5).to(dt)
    s["o"] = torch.zeros(len(lens), hq, d, dtype=dt, device="cuda")
    conf |= {"max_rows": len(lens)}


# ---- one pass ---------------------------------------------------------------

def run(s):
    return {"plan": _plan, "rotate": _rotate, "prompt": _prompt, "paged": _paged, "step": _step}[s["case"]["op"]](s)


def _plan(s):
    if own:
        s["lm"].plan(s["before"], s["after"], s["tables"], s["free_list"], s["free"], s["free_out"], s["row_start"],
                     s["kv_len"], s["status"], s["slots"], s["positions"], shared_table=s["shared_table"])
        return {k: s[k] for k in ("tables", "free_list", "free_out", "row_start", "kv_len", "status", "slots",
                                  "positions")}
    blk, sh = s["case"]["block"], s["shared_table"].numel()
    tables, ring, n = s["tables"], s["free_list"], s["free_list"].numel()
    b, width = tables.shape
    most = s["slots"].numel()
    before, after = s["before"].long(), s["after"].long()
    head, tail = s["free"][0], s["free"][1]
    good = (before >= 0) & (after >= 0) & (before <= width * blk) & (after <= width * blk)
    rows = torch.where(good, (after - before).clamp(min=0), 0)
    ends = torch.cumsum(rows, 0)
    fits = good & (ends <= most)
    n0 = ((before + blk - 1) // blk - sh).clamp(min=0)
    n1 = ((after + blk - 1) // blk - sh).clamp(min=0)
    need = torch.where(fits, (n1 - n0).clamp(min=0), 0)
    upto = torch.cumsum(need, 0)
    room = (need == 0) | (upto <= tail - head)
    ok = fits & room
    back = torch.where(ok, (n0 - n1).clamp(min=0), 0)
    kept = torch.cumsum(back, 0) - back
    j = torch.arange(width, device="cuda")
    lo, hi = (sh + n0)[:, None], (sh + n1)[:, None]
    new = torch.where((ok & (before <= sh * blk) & (after > before))[:, None] & (j < sh),
                      torch.nn.functional.pad(s["shared_table"], (0, width - sh)), tables)
    ids = ring[(head + (upto - need)[:, None] + j - lo).remainder(n)]
    new = torch.where(ok[:, None] & (j >= lo) & (j < hi), ids, new)
    freed = ok[:, None] & (j >= hi) & (j < lo)
    to = torch.where(freed, (tail + kept[:, None] + j - hi).remainder(n), n)
    ring = torch.nn.functional.pad(ring, (0, 1)).scatter(0, to.flatten(), tables.flatten())[:n]
    row_start = torch.cat([ends.new_zeros(1), ends]).clamp(max=most)
    t = torch.arange(most, device="cuda")
    at = torch.searchsorted(ends, t, right=True).clamp(max=b - 1)
    pos = before[at] + t - (ends - rows)[at]
    held = t < ends[-1]
    slot = new[at, (pos // blk).clamp(0, width - 1)] * blk + pos % blk
    taken = torch.where(ok & (need > 0), upto, 0).max()
    return {"tables": new, "free_list": ring, "free_out": torch.stack([head + taken, tail + back.sum()]),
            "row_start": row_start.int(), "kv_len": torch.where(ok, after, 0).int(),
            "status": torch.where(ok, 0, torch.where(~good, 2, torch.where(~fits, 3, 1))).int(),
            "slots": torch.where(held & ok[at], slot, -1).int(), "positions": torch.where(held, pos, 0).int()}


def _turned(x, gain, cos, sin, pairs):
    """Norm over the head, then the rotation; x [rows][heads][dim] in 32 bits."""
    if gain is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * gain
    if pairs:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    a, b = x.chunk(2, -1)
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _rotate(s):
    if own:
        s["lm"].rotate(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["q_out"], s["k_cache"], s["v_cache"],
                       q_gain=s["q_gain"], k_gain=s["k_gain"])
        return {k: s[k] for k in ("q_out", "k_cache", "v_cache")}
    d, dt = s["case"]["dim"], s["q_out"].dtype
    freq = THETA ** (torch.arange(0, d, 2, device="cuda", dtype=torch.float64) / -d)
    angle = s["positions"][:, None, None] * freq
    cos, sin = angle.cos().float(), angle.sin().float()
    q = _turned(s["q"].float(), s["q_gain"], cos, sin, s["case"]["pairs"]).to(dt)
    k = _turned(s["k"].float(), s["k_gain"], cos, sin, s["case"]["pairs"]).to(dt)
    held = s["slots"] >= 0
    s["q_out"].copy_(torch.where(held[:, None, None], q, s["q_out"]))
    to = s["slots"][held].long()
    s["k_cache"].flatten(0, 1)[to] = k[held]
    s["v_cache"].flatten(0, 1)[to] = s["v"][held].to(dt)
    return {k: s[k] for k in ("q_out", "k_cache", "v_cache")}


def _attend(q, k, v, allowed):
    """q [b][n][hq][d], k and v [b][m][hk][d] in 32 bits, allowed [b][n][m]."""
    b, n, hq, d = q.shape
    m, hk = k.shape[1:3]
    q = q.reshape(b, n, hk, hq // hk, d).permute(0, 2, 3, 1, 4).reshape(b, hk, -1, d)
    x = (q @ k.permute(0, 2, 3, 1)).mul_(1 / math.sqrt(d)).view(b, hk, hq // hk, n, m)
    x = x.masked_fill_(~allowed[:, None, None], -math.inf)
    x = x.sub_(x.amax(-1, keepdim=True).clamp(min=-1e30)).exp_()
    p = x.view(b, hk, -1, m)
    o = (p @ v.permute(0, 2, 1, 3)) / p.sum(-1, keepdim=True).clamp(min=1e-30)
    return o.view(b, hk, hq // hk, n, d).permute(0, 3, 1, 2, 4).reshape(b, n, hq, d)


def _padded(s):
    """Rows of the packed queries by request, [requests][longest], and which of them are there."""
    start = s["row_start"].long()
    at = start[:-1, None] + torch.arange(s["longest"], device="cuda")
    return at.clamp(max=s["q"].shape[0] - 1), at < start[1:, None]


def _prompt(s):
    if own:
        s["lm"].prompt(s["q"], s["k"], s["v"], s["row_start"], s["o"])
        return s["o"]
    at, there = _padded(s)
    i = torch.arange(s["longest"], device="cuda")
    allowed = (i <= i[:, None]) & there[:, None]
    o = _attend(s["q"].float()[at], s["k"].float()[at], s["v"].float()[at], allowed)
    return o[there].to(s["o"].dtype)


def _pages(cache, tables):
    return cache[tables.long()].flatten(1, 2).float()


def _paged(s):
    if own:
        s["lm"].prompt_paged(s["q"], s["k_cache"], s["v_cache"], s["row_start"], s["tables"], s["kv_len"], s["o"])
        return s["o"]
    at, there = _padded(s)
    k, v = _pages(s["k_cache"], s["tables"]), _pages(s["v_cache"], s["tables"])
    start = s["row_start"]
    last = (s["kv_len"] - (start[1:] - start[:-1]))[:, None] + torch.arange(s["longest"], device="cuda")
    allowed = torch.arange(k.shape[1], device="cuda") <= last[:, :, None]
    return _attend(s["q"].float()[at], k, v, allowed)[there].to(s["o"].dtype)


def _step(s):
    if own:
        s["lm"].step(s["q"], s["k_cache"], s["v_cache"], s["tables"], s["kv_len"], s["o"],
                     shared_table=s["shared_table"])
        return s["o"]
    k, v = _pages(s["k_cache"], s["tables"]), _pages(s["v_cache"], s["tables"])
    allowed = torch.arange(k.shape[1], device="cuda") < s["kv_len"][:, None]
    return _attend(s["q"].float()[:, None], k, v, allowed[:, None])[:, 0].to(s["o"].dtype)


# ---- the definition in 64 bits ----------------------------------------------

def exact(case, seed):
    if case["op"] == "plan":
        return None         # whole numbers: equal, or not
    s = prepare(case, seed)
    return {"rotate": _exact_rotate, "prompt": _exact_prompt, "paged": _exact_paged,
            "step": _exact_step}[case["op"]](case, s)


def _exact_rotate(case, s):
    d = case["dim"]
    i = torch.arange(d // 2, device="cuda")
    first, second = (2 * i, 2 * i + 1) if case["pairs"] else (i, i + d // 2)
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                       s["positions"].double()[:, None] / THETA ** (2.0 * i / d))[:, None]
    got = {}
    for name, gain in (("q", s["q_gain"]), ("k", s["k_gain"])):
        x = s[name].double()
        if gain is not None:
            x = x / ((x * x).sum(-1, keepdim=True) / d + EPS).sqrt() * gain.double()
        z = torch.complex(x[..., first], x[..., second]) * turn
        y = torch.empty_like(x)
        y[..., first], y[..., second] = z.real, z.imag
        got[name] = y
    rows = [r for r, slot in enumerate(s["slots"].tolist()) if slot >= 0]
    to = s["slots"][rows].long()
    out = {k: s[k].double() for k in ("q_out", "k_cache", "v_cache")}
    out["q_out"][rows] = got["q"][rows]
    out["k_cache"].view(-1, *out["k_cache"].shape[2:])[to] = got["k"][rows]
    out["v_cache"].view(-1, *out["v_cache"].shape[2:])[to] = s["v"][rows].double()
    return out


def _exact_rows(q, k, v, first):
    """Attention of q [n][hq][d] over k, v [m][hk][d]: query i sees keys 0 .. first + i."""
    n, hq, d = q.shape
    group = hq // k.shape[1]
    o = torch.zeros(n, hq, d, dtype=torch.float64, device="cuda")
    for h in range(hq):
        kh, vh = k[:, h // group].double(), v[:, h // group].double()
        for a in range(0, n, 2048):
            x = q[a:a + 2048, h].double() @ kh.T / math.sqrt(d)
            seen = torch.arange(len(kh), device="cuda") <= first + a + torch.arange(len(x), device="cuda")[:, None]
            o[a:a + 2048, h] = torch.softmax(x.masked_fill(~seen, -math.inf), -1) @ vh
    return o


def _exact_prompt(case, s):
    b = s["row_start"].tolist()
    parts = [_exact_rows(s["q"][x:y], s["k"][x:y], s["v"][x:y], 0) for x, y in zip(b, b[1:]) if y > x]
    return torch.cat(parts) if parts else s["q"].double()


def _keys(case, s, i, n):
    ids = s["tables"][i, : -(-n // case["block"])].long()
    return (s[c][ids].flatten(0, 1)[:n] for c in ("k_cache", "v_cache"))


def _exact_paged(case, s):
    b, lens = s["row_start"].tolist(), s["kv_len"].tolist()
    return torch.cat([_exact_rows(s["q"][b[i]:b[i + 1]], *_keys(case, s, i, n), n - (b[i + 1] - b[i]))
                      for i, n in enumerate(lens) if b[i + 1] > b[i]])


def _exact_step(case, s):
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    d, hk = case["dim"], case["kv_heads"]
    for i, n in enumerate(s["kv_len"].tolist()):
        if n:
            k, v = _keys(case, s, i, n)
            x = torch.einsum("hgd,mhd->hgm", s["q"][i].double().view(hk, -1, d), k.double()) / math.sqrt(d)
            o[i] = torch.einsum("hgm,mhd->hgd", torch.softmax(x, -1), v.double()).reshape(-1, d)
    return o
