"""The codec LM's attention operators against their definitions in 64 bits
(whole numbers for the plan): both types, head widths and rotation forms,
lengths from none to several tiles, strided inputs, poisoned places that no
row may see, device data that is wrong, and a layer's run of them together."""
from __future__ import annotations

import random
import threading

import numpy as np
import pytest
import torch

import lm_ref as R
from streaming_tts_vocoder_gb300 import codec as C

pytestmark = pytest.mark.gpu
NAN = float("nan")


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def f64(t):
    return t.detach().cpu().double().numpy()


# ---- plan -------------------------------------------------------------------

def plan_case(seed, B, bs, sh, width, max_rows, free, old, new, bad=False):
    rng = random.Random(seed)
    before = [rng.choice([0, rng.randrange(old + 1)]) + sh * bs for _ in range(B)]
    after = [rng.choice([0, n, n + 1, n + rng.randrange(new + 1), n // 2]) for n in before]
    if bad:
        for i in range(0, B, 7):
            before[i] = rng.choice([-1, -2 ** 31, width * bs + 1, 2 ** 31 - 1])
        for i in range(3, B, 7):
            after[i] = rng.choice([-5, width * bs + 1, 2 ** 31 - 1])
    counts = [max(0, -(-n // bs) - sh) if 0 <= n <= width * bs else 0 for n in before]
    n_blocks = sh + sum(counts) + free
    ids = list(range(n_blocks))
    rng.shuffle(ids)
    shared, ids = ids[:sh], ids[sh:]
    tables = [[-7] * width for _ in range(B)]
    for b, c in enumerate(counts):
        if before[b] > sh * bs and c:
            tables[b][:sh] = shared
        tables[b][sh:sh + c], ids = ids[:c], ids[c:]
    head = rng.randrange(10 * n_blocks + 1)
    ring = [-9] * n_blocks
    for i, x in enumerate(ids):
        ring[(head + i) % n_blocks] = x
    return before, after, tables, ring, (head, head + len(ids)), shared, n_blocks


def run_plan(lm, before, after, tables, ring, free, shared, max_rows):
    B = len(before)
    t = dict(tables=i32(tables), free_list=i32(ring), free_out=torch.full((2,), -1, dtype=torch.int64, device="cuda"),
             row_start=i32([-3] * (B + 1)), kv_len=i32([-3] * B), status=i32([-3] * B), slots=i32([-3] * max_rows),
             positions=i32([-3] * max_rows))
    free_in = torch.tensor(free, dtype=torch.int64, device="cuda")
    for _ in range(2):      # a repeated call writes the same
        lm.plan(i32(before), i32(after), t["tables"], t["free_list"], free_in, t["free_out"], t["row_start"],
                t["kv_len"], t["status"], t["slots"], t["positions"], shared_table=i32(shared) if shared else None)
    return {k: v.tolist() for k, v in t.items()}


@pytest.mark.parametrize("seed,B,bs,sh,width,max_rows,free,old,new,bad", [
    (0, 1, 16, 0, 4, 1, 3, 0, 1, False),
    (1, 7, 16, 0, 20, 600, 90, 200, 40, False),
    (2, 64, 16, 3, 40, 5000, 400, 500, 60, False),
    (3, 64, 32, 0, 40, 5000, 30, 500, 200, False),       # the blocks run out
    (4, 33, 128, 2, 9, 200, 100, 300, 100, False),       # the rows run out
    (5, 700, 64, 1, 12, 30000, 900, 400, 100, True),     # more requests than threads, wrong lengths
    (6, 40, 16, 5, 5, 300, 0, 0, 0, False),              # nothing free, table all shared
])
def test_plan(seed, B, bs, sh, width, max_rows, free, old, new, bad):
    before, after, tables, ring, fr, shared, n_blocks = plan_case(seed, B, bs, sh, width, max_rows, free, old, new, bad)
    lm = C.Lm(8, 8, 64, block_size=bs, n_blocks=n_blocks, table_blocks=width, max_requests=B, max_rows=max_rows)
    got = run_plan(lm, before, after, tables, ring, fr, shared, max_rows)
    want = R.plan(before, after, tables, ring, fr, shared, bs, max_rows)
    for k in want:
        assert got[k] == want[k], k
    assert lm.errors() == 0


def test_plan_wrong_free_counts_take_nothing():
    lm = C.Lm(8, 8, 64, n_blocks=8, table_blocks=4, max_requests=2, max_rows=40)
    for free in [(5, 3), (-1, 2), (0, 9)]:
        got = run_plan(lm, [0, 3], [20, 5], [[0] * 4, [1] * 4], list(range(8)), free, [], 40)
        assert got["status"] == [1, 0] and got["free_out"] == list(free)
        assert got["slots"][20:22] == [19, 20] and got["slots"][:20] == [-1] * 20
        assert lm.errors() == C.LM_ERR_FREE


def test_plan_give_back_then_take():
    """Blocks go round: a request ends, the next takes its blocks."""
    lm = C.Lm(8, 8, 64, n_blocks=3, table_blocks=3, max_requests=1, max_rows=48)
    tables, ring, free = [[-1] * 3], [2, 0, 1], (0, 3)
    seen = []
    for before, after in [(0, 40), (40, 0), (0, 17), (17, 48), (48, 16), (16, 0)]:
        want = R.plan([before], [after], tables, ring, free, [], 16, 48)
        got = run_plan(lm, [before], [after], tables, ring, free, [], 48)
        assert got == want and got["status"] == [0]
        tables, ring, free = got["tables"], got["free_list"], tuple(got["free_out"])
        seen.append(free[1] - free[0])
    assert seen == [0, 3, 1, 0, 2, 3]


# ---- rotate -----------------------------------------------------------------

@pytest.mark.parametrize("rows,hq,hk,d,dt,it,pairs,norm,far", [
    (1, 16, 8, 128, "bf16", "bf16", False, True, 50),
    (5, 7, 1, 128, "fp16", "fp32", True, True, 60000),
    (67, 10, 2, 64, "bf16", "fp32", False, False, 1000),
    (300, 3, 3, 64, "fp16", "fp16", True, False, 9),
    (2500, 16, 16, 64, "bf16", "bf16", True, True, 30000),
    (2600, 12, 4, 128, "fp16", "fp16", False, True, 30000),
])
def test_rotate(rows, hq, hk, d, dt, it, pairs, norm, far):
    gen = torch.Generator(device="cuda").manual_seed(rows)
    lm = C.Lm(hq, hk, d, dt, block_size=16, n_blocks=rows // 16 + 3, max_rows=rows, max_positions=far,
              rope_theta=1e4, rope_pairs=pairs, rms_eps=1e-5)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    fused = (r(rows, (hq + 2 * hk) * d + 8) * 3).to(R.DTYPES[it])      # rows further apart than they are wide
    q, k, v, _ = fused.split([hq * d, hk * d, hk * d, 8], 1)
    q, k, v = (x.unflatten(1, (-1, d)) for x in (q, k, v))
    gq, gk = (1 + 0.1 * r(d), 1 + 0.1 * r(d)) if norm else (None, None)
    pos = torch.randint(far, (rows,), generator=gen, device="cuda", dtype=torch.int32)
    n_slots = (rows // 16 + 3) * 16
    slots = torch.randperm(n_slots, generator=gen, device="cuda")[:rows].to(torch.int32)
    skip = torch.arange(0, rows, 5, device="cuda") if rows > 5 else torch.arange(0, device="cuda")
    slots[skip] = -1
    T = R.DTYPES[dt]
    qo = torch.full((rows, hq, d), 7.0, dtype=T, device="cuda")
    kc, vc = (torch.full((n_slots // 16, 16, hk, d), 7.0, dtype=T, device="cuda") for _ in range(2))
    lm.rotate(q, k, v, pos, slots, qo, kc, vc, q_gain=gq, k_gain=gk)
    assert lm.errors() == 0
    held = (slots >= 0).cpu().numpy()
    to = slots.cpu().numpy()[held]
    want = {}
    for name, x, g in (("q", q, gq), ("k", k, gk)):
        y = R.rotate(x, g, pos, 1e4, 1e-5, pairs)
        # a rotation adds two products: their sizes bound its rounding
        size = np.abs(f64(x)).max(-1, keepdims=True)
        if g is not None:
            size = size / np.sqrt((f64(x) ** 2).mean(-1, keepdims=True) + 1e-5) * 1.6
        want[name] = y, torch.finfo(T).eps / 2 * np.abs(y) + 2 * size * 2.0 ** -20 + (2.0 ** -25 if dt == "fp16" else 0)
    full_q = np.full((rows, hq, d), 7.0)
    full_q[held] = want["q"][0][held]
    tol = np.zeros_like(full_q)
    tol[held] = np.broadcast_to(want["q"][1], full_q.shape)[held]
    assert (np.abs(f64(qo) - full_q) <= tol).all()
    kw, kt = np.full((n_slots, hk, d), 7.0), np.zeros((n_slots, hk, d))
    kw[to], kt[to] = want["k"][0][held], want["k"][1][held]
    assert (np.abs(f64(kc).reshape(kw.shape) - kw) <= kt).all()
    vw = torch.full((n_slots, hk, d), 7.0, dtype=T, device="cuda")
    vw[torch.from_numpy(to).cuda().long()] = v.to(T)[torch.from_numpy(held).cuda()]
    assert torch.equal(vc.view(vw.shape), vw)
    # rows that stay where they are; in place where the type allows it
    pk = torch.empty(rows, hk, d, dtype=T, device="cuda")
    qp = q.contiguous() if it == dt else torch.empty(rows, hq, d, dtype=T, device="cuda")
    lm.rotate(qp if it == dt else q, k, None, pos, None, qp, pk, None, q_gain=gq, k_gain=gk)
    assert torch.equal(qp[torch.from_numpy(held).cuda()], qo[torch.from_numpy(held).cuda()])
    assert torch.equal(pk[torch.from_numpy(held).cuda()], kc.view(-1, hk, d)[torch.from_numpy(to).cuda().long()])


def test_rotate_wrong_slots_and_positions_are_skipped():
    lm = C.Lm(2, 2, 64, n_blocks=2, max_rows=8, max_positions=10)
    x = torch.randn(6, 2, 64, device="cuda")
    q = torch.zeros(6, 2, 64, dtype=torch.bfloat16, device="cuda")
    kc, vc = (torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lm.rotate(x, x, x, i32([0, 1, 2, 3, 4, 5]), i32([0, 32, -2, 2 ** 31 - 1, -2 ** 31, 31]), q, kc, vc)
    assert lm.errors() == C.LM_ERR_SLOT and lm.errors() == 0
    assert [bool(r.any()) for r in q] == [True, False, False, False, False, True]
    assert [bool(r.any()) for r in vc.view(32, -1)] == [True] + [False] * 30 + [True]
    q.zero_()
    lm.rotate(x, x, x, i32([0, 10, -1, 2 ** 31 - 1, -2 ** 31, 9]), i32([0, 1, 2, 3, 4, 5]), q, kc, vc)
    assert lm.errors() == C.LM_ERR_POSITION
    assert [bool(r.any()) for r in q] == [True, False, False, False, False, True]


# ---- prompt -----------------------------------------------------------------

HEADS = [(16, 16, 64), (16, 8, 128), (7, 1, 128), (10, 2, 64), (12, 4, 128), (16, 1, 64), (3, 3, 128)]


def prompt_inputs(seed, lens, hq, hk, d, dt, extra=3, pad=8):
    """Packed q, k, v whose rows lie `pad` elements further apart than they are
    wide, with `extra` poisoned rows behind the last request."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    n = sum(lens) + extra
    T = R.DTYPES[dt]
    mk = lambda h, f: (torch.randn(n, h * d + pad, generator=gen, device="cuda") * f).to(T)[:, :h * d].unflatten(1, (h, d))
    q, k, v = mk(hq, 1.5), mk(hk, 1.0), mk(hk, 1.0)
    for t in (q, k, v):
        t[sum(lens):] = NAN
    starts = [sum(lens[:i]) for i in range(len(lens) + 1)]
    return q, k, v, starts


def check_prompt(lens, hq, hk, d, dt, scale=0.0, seed=0, mul=1.0):
    q, k, v, starts = prompt_inputs(seed, lens, hq, hk, d, dt)
    q.mul_(mul)
    n = q.shape[0]
    lm = C.Lm(hq, hk, d, dt, max_requests=len(lens), max_rows=n, scale=scale)
    o = torch.full((n, hq, d + 8), 5.0, dtype=q.dtype, device="cuda")
    o = o.view(n, -1)[:, :hq * d].unflatten(1, (hq, d)) if hq > 1 else o[:, :, :d]
    lse = torch.full((n, hq), 5.0, device="cuda")
    lm.prompt(q, k, v, i32(starts), o, lse=lse)
    assert lm.errors() == 0
    live = sum(lens)
    assert (o[live:] == 5).all() and (lse[live:] == 5).all()
    q6, k6, v6 = f64(q)[:live], f64(k), f64(v)
    where = [(s, i) for s, e in zip(starts, starts[1:]) for i in range(e - s)]
    ref = R.attention(q6, range(live), lambda r: (k6[where[r][0]:r + 1], v6[where[r][0]:r + 1]), hk,
                      scale or d ** -0.5)
    R.assert_attention(o[:live], lse[:live], ref, dt, [w[1] + 1 for w in where], d, 5.0)
    o2 = torch.empty_like(o)
    lm.prompt(q, k, v, i32(starts), o2)
    assert torch.equal(o2[:live], o[:live])


@pytest.mark.parametrize("hq,hk,d", HEADS)
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_prompt_heads(hq, hk, d, dt):
    check_prompt([1, 0, 37, 130], hq, hk, d, dt)


@pytest.mark.parametrize("lens", [[1], [2], [127], [128], [129], [255], [256], [257], [0, 0, 1], [64] * 9, [383, 1, 300],
                                  [640]])
def test_prompt_lengths(lens):
    check_prompt(lens, 4, 2, 128, "bf16")
    check_prompt(lens, 2, 2, 64, "fp16", seed=1)


def test_prompt_scale_and_large_scores():
    check_prompt([200], 4, 4, 64, "bf16", scale=0.7)
    check_prompt([200, 50], 4, 2, 128, "fp16", mul=20.0)     # nearly one-hot rows


def test_prompt_a_later_token_never_reaches_an_earlier_row():
    """NaN and infinities from position 100 on leave rows 0 .. 99 the bits they had."""
    for d, dt in ((128, "bf16"), (64, "fp16")):
        q, k, v, starts = prompt_inputs(5, [300, 90], 4, 2, d, dt)
        lm = C.Lm(4, 2, d, dt, max_requests=2, max_rows=q.shape[0])
        o, o2 = (torch.zeros(q.shape, dtype=q.dtype, device="cuda") for _ in range(2))
        lm.prompt(q, k, v, i32(starts), o)
        k[100:300:3] = NAN
        v[101:300:3] = NAN
        v[100] = float("inf")
        k[102] = float("-inf")
        lm.prompt(q, k, v, i32(starts), o2)
        assert torch.equal(o[:100], o2[:100]) and torch.equal(o[300:390], o2[300:390])
        assert o2[102:300].isnan().all()


def test_prompt_row_start_out_of_range_is_bent():
    q, k, v, _ = prompt_inputs(6, [20], 2, 2, 64, "bf16", extra=0)
    lm = C.Lm(2, 2, 64, max_requests=3, max_rows=20)
    o = torch.zeros(20, 2, 64, dtype=q.dtype, device="cuda")
    want = torch.zeros_like(o)
    lm.prompt(q, k, v, i32([0, 20]), want)
    assert lm.errors() == 0
    for starts in ([0, 2 ** 31 - 1], [-4, 20], [-2 ** 31, 2 ** 31 - 1]):
        lm.prompt(q, k, v, i32(starts), o.zero_())
        assert lm.errors() == C.LM_ERR_LENGTH and torch.equal(o, want)
    lm.prompt(q, k, v, i32([20, 0, -1, 5]), o.zero_())
    assert lm.errors() == C.LM_ERR_LENGTH


# ---- cache ------------------------------------------------------------------

def cache_case(seed, lens, hk, d, dt, bs, sh=0, rows=None, mul=1.0):
    """Caches in which every place behind a length is NaN; tables whose entries
    behind a length are out of range."""
    rng = random.Random(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    T = R.DTYPES[dt]
    counts = [max(0, -(-n // bs) - sh) for n in lens]
    n_blocks = sh + sum(counts) + 3
    width = max(1, sh + max(counts) + 1)
    ids = list(range(n_blocks))
    rng.shuffle(ids)
    shared, ids = ids[:sh], ids[sh:]
    tables = [[2 ** 31 - 1] * width for _ in lens]
    kc, vc = (torch.full((n_blocks, bs, hk, d), NAN, dtype=T, device="cuda") for _ in range(2))
    for i in shared:
        for c in (kc, vc):
            c[i] = torch.randn(bs, hk, d, generator=gen, device="cuda").to(T)
    for b, n in enumerate(lens):
        tables[b][:sh] = shared
        mine, ids = ids[:counts[b]], ids[counts[b]:]
        tables[b][sh:sh + counts[b]] = mine
        for j, blk in enumerate(mine):
            left = min(bs, n - (sh + j) * bs)
            for c in (kc, vc):
                c[blk, :left] = torch.randn(left, hk, d, generator=gen, device="cuda").to(T) * mul
    return kc, vc, tables, shared, n_blocks, width, gen


def gathered(cache, table, n, bs):
    ids = [table[j] for j in range(-(-n // bs))]
    return f64(cache[ids].flatten(0, 1)[:n]) if n else np.zeros((0,) + tuple(cache.shape[2:]))


def check_paged(new, kv, hq, hk, d, dt, bs, seed=0):
    kc, vc, tables, _, n_blocks, width, gen = cache_case(seed, kv, hk, d, dt, bs)
    n = sum(new) + 2
    q = (torch.randn(n, hq, d, generator=gen, device="cuda") * 1.5).to(R.DTYPES[dt])
    q[sum(new):] = NAN
    starts = [sum(new[:i]) for i in range(len(new) + 1)]
    lm = C.Lm(hq, hk, d, dt, block_size=bs, n_blocks=n_blocks, table_blocks=width, max_requests=len(new), max_rows=n)
    o = torch.full((n, hq, d), 5.0, dtype=q.dtype, device="cuda")
    lse = torch.full((n, hq), 5.0, device="cuda")
    lm.prompt_paged(q, kc, vc, i32(starts), i32(tables), i32(kv), o, lse=lse)
    assert lm.errors() == 0
    live = sum(new)
    assert (o[live:] == 5).all() and (lse[live:] == 5).all()
    ks = [(gathered(kc, tables[b], kv[b], bs), gathered(vc, tables[b], kv[b], bs)) for b in range(len(new))]
    where = [(b, max(0, kv[b] - new[b] + i + 1)) for b in range(len(new)) for i in range(new[b])]
    ref = R.attention(f64(q)[:live], range(live), lambda r: tuple(x[:where[r][1]] for x in ks[where[r][0]]), hk, d ** -0.5)
    R.assert_attention(o[:live], lse[:live], ref, dt, [w[1] for w in where], d, 5.0)


@pytest.mark.parametrize("hq,hk,d", HEADS)
@pytest.mark.parametrize("bs", [16, 32, 64, 128])
def test_prompt_paged(hq, hk, d, bs):
    dt = "bf16" if bs in (16, 64) else "fp16"
    # whole prompt, one token behind a context, several, none, more rows than keys, keys but no rows
    check_paged([33, 1, 70, 0, 9, 0], [33, 150, 200, 0, 4, 40], hq, hk, d, dt, bs)


def test_prompt_paged_rows_without_keys():
    check_paged([5, 200], [0, 64], 4, 2, 128, "bf16", 16)
    check_paged([300], [300], 4, 1, 64, "fp16", 32)


@pytest.mark.parametrize("new,kv,hq,hk,d,bs", [
    ([3], [9000], 4, 2, 128, 16),               # one request behind a long context: cut along the keys
    ([70, 1, 33], [5000, 8200, 700], 4, 1, 64, 64),
    ([260], [4100], 2, 2, 128, 128),            # several pairs of tiles, each cut
    ([40, 5], [3, 6000], 16, 1, 64, 32),        # one with rows that see nothing, one cut
])
def test_prompt_paged_long_context(new, kv, hq, hk, d, bs):
    check_paged(new, kv, hq, hk, d, "bf16", bs, seed=3)
    check_paged(new, kv, hq, hk, d, "fp16", bs, seed=4)


def test_prompt_cut_along_the_keys():
    """Packed prompts whose items are few and long."""
    check_prompt([2100], 4, 1, 64, "fp16")
    check_prompt([1500, 30, 1], 2, 2, 128, "bf16")


def check_step(kv, sh, hq, hk, d, dt, bs, seed=0, mul=1.0):
    kc, vc, tables, shared, n_blocks, width, gen = cache_case(seed, kv, hk, d, dt, bs, sh)
    B = len(kv)
    q = (torch.randn(B, hq * d + 16, generator=gen, device="cuda") * 1.5 * mul).to(R.DTYPES[dt])[:, :hq * d].unflatten(1, (hq, d))
    lm = C.Lm(hq, hk, d, dt, block_size=bs, n_blocks=n_blocks, table_blocks=width, max_requests=B, max_rows=B)
    o = torch.full((B, hq, d), 5.0, dtype=q.dtype, device="cuda")
    lse = torch.full((B, hq), 5.0, device="cuda")
    own = [[-1] * sh + t[sh:] for t in tables]      # the entries of the shared blocks are not read
    lm.step(q, kc, vc, i32(own), i32(kv), o, shared_table=i32(shared) if sh else None, lse=lse)
    assert lm.errors() == 0
    ks = [(gathered(kc, tables[b], n, bs), gathered(vc, tables[b], n, bs)) for b, n in enumerate(kv)]
    ref = R.attention(f64(q), range(B), lambda r: ks[r], hk, d ** -0.5)
    R.assert_attention(o, lse, ref, dt, kv, d, 5.0)
    return lm, q, kc, vc, own, shared, o


@pytest.mark.parametrize("hq,hk,d", HEADS)
@pytest.mark.parametrize("bs", [16, 32, 64, 128])
def test_step(hq, hk, d, bs):
    dt = "fp16" if bs in (16, 64) else "bf16"
    check_step([1, 0, 17, 128, 129, 260], 0, hq, hk, d, dt, bs)
    # behind a shared part: nothing, one, several blocks; shorter than the shared part; idle
    check_step([2 * bs, 2 * bs + 1, 2 * bs + 70, 0, bs + 3, 1], 2, hq, hk, d, dt, bs, seed=1)


@pytest.mark.parametrize("kv,sh,bs", [([1000], 0, 16), ([2100, 5, 700], 0, 64), ([1500] * 3, 64, 16), ([700] * 70, 9, 64),
                                      ([4200], 32, 128)])
def test_step_long(kv, sh, bs):
    check_step(kv, sh, 4, 2, 128, "bf16", bs)
    check_step(kv, sh, 4, 1, 64, "fp16", bs, seed=2, mul=8.0)


def test_step_result_does_not_depend_on_the_batch():
    lm, q, kc, vc, own, shared, o = check_step([40 + 13 * i for i in range(20)], 2, 8, 2, 128, "bf16", 16)
    for b in (0, 7, 19):
        kv = i32([40 + 13 * b])
        o1 = torch.zeros(1, 8, 128, dtype=q.dtype, device="cuda")
        lm.step(q[b:b + 1], kc, vc, i32(own[b:b + 1]), kv, o1, shared_table=i32(shared))
        assert torch.equal(o1[0], o[b])


@pytest.mark.parametrize("hq,hk,d,dt", [(8, 2, 128, "bf16"), (4, 4, 64, "fp16")])
def test_step_behind_many_shared_tiles_does_not_depend_on_the_batch(hq, hk, d, dt):
    """Scores large enough that running references move in every tile: each
    request's must move for its own sake alone."""
    kv = [1100 + 37 * i for i in range(30)] + [700, 0, 3]
    lm, q, kc, vc, own, shared, o = check_step(kv, 66, hq, hk, d, dt, 16, seed=5, mul=8.0)
    for b in (0, 11, 29, 30, 32):
        o1 = torch.zeros(1, hq, d, dtype=q.dtype, device="cuda")
        lm.step(q[b:b + 1], kc, vc, i32(own[b:b + 1]), i32([kv[b]]), o1, shared_table=i32(shared))
        assert torch.equal(o1[0], o[b])
    back = list(range(len(kv)))[::-1]           # other neighbours, other order
    o2 = torch.zeros_like(o)
    lm.step(q[back], kc, vc, i32([own[b] for b in back]), i32([kv[b] for b in back]), o2, shared_table=i32(shared))
    assert torch.equal(o2, o[back])


def test_step_short_request_does_not_see_the_rest_of_the_shared_part():
    kc, vc, tables, shared, n_blocks, width, gen = cache_case(7, [300, 300, 300], 2, 128, "bf16", 16, 12)
    q = torch.randn(3, 4, 128, generator=gen, device="cuda").to(torch.bfloat16)
    lm = C.Lm(4, 2, 128, n_blocks=n_blocks, table_blocks=width, max_requests=3, max_rows=3)
    o, o2 = torch.zeros_like(q), torch.zeros_like(q)
    lm.step(q, kc, vc, i32(tables), i32([50, 300, 130]), o, shared_table=i32(shared))
    kc[shared[10]] = NAN
    vc[shared[10], ::2] = float("inf")
    vc[shared[10], 1::2] = NAN
    lm.step(q, kc, vc, i32(tables), i32([50, 300, 130]), o2, shared_table=i32(shared))
    assert torch.equal(o2[::2], o[::2]) and o2[1].isnan().all()


def test_many_requests():
    rng = random.Random(1)
    check_prompt([rng.choice([0, 1, 2, 5, 9, 40]) for _ in range(700)], 4, 2, 64, "bf16")       # too many to sort
    lens = [0] * 1000
    for i in rng.sample(range(1000), 20):
        lens[i] = rng.randrange(1, 5)
    check_prompt(lens, 2, 2, 64, "fp16")        # fewer rows than requests
    check_step([rng.choice([0, 1, 7, 90]) for _ in range(600)], 0, 2, 1, 64, "bf16", 16)
    check_step([32 + rng.choice([0, 1, 7, 90]) for _ in range(1500)], 2, 2, 1, 64, "fp16", 16)


def test_graph_of_prompts_follows_the_lengths():
    """One captured call, replayed with other lengths in the same rows: packed
    with a list of items, and behind the cache with pieces."""
    q, k, v, _ = prompt_inputs(8, [3000], 4, 2, 64, "bf16", extra=0)
    for paged in (False, True):
        bs, width = 64, 60
        lm = C.Lm(4, 2, 64, block_size=bs, n_blocks=60, table_blocks=width, max_requests=3, max_rows=3000)
        eager = C.Lm(4, 2, 64, block_size=bs, n_blocks=60, table_blocks=width, max_requests=3, max_rows=3000)
        gen = torch.Generator(device="cuda").manual_seed(0)
        kc, vc = (torch.randn(60, bs, 2, 64, generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2))
        tables = torch.randint(60, (3, width), generator=gen, device="cuda", dtype=torch.int32)
        rows, kv, o = i32([0, 0, 0, 0]), i32([0, 0, 0]), torch.zeros(3000, 4, 64, dtype=q.dtype, device="cuda")

        def call(lm, o):
            if paged:
                lm.prompt_paged(q[:200], kc, vc, rows, tables, kv, o[:200])
            else:
                lm.prompt(q, k, v, rows, o)

        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(lm, o)
        for starts, lens in (([0, 1, 1, 100], [3000, 9, 3840]), ([0, 70, 71, 200], [70, 1, 2500]),
                             ([0, 0, 0, 0], [5, 5, 5])):
            rows.copy_(i32(starts))
            kv.copy_(i32(lens))
            want = torch.full_like(o, 3.0)
            call(eager, want)
            o.fill_(3.0)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(o, want) and lm.errors() == 0 and eager.errors() == 0
            assert (o[starts[-1]:] == 3).all() and not (o[:starts[-1]] == 3).all(-1).any()


def test_cache_beyond_32_bits():
    """Blocks whose elements lie past 2^32, and a slot to the last of them."""
    hq, hk, d, bs = 16, 8, 128, 128
    n_blocks = 2 ** 32 // (bs * hk * d) + 40
    T = torch.bfloat16
    kc, vc = (torch.empty(n_blocks, bs, hk, d, dtype=T, device="cuda") for _ in range(2))
    kc[:8], vc[:8] = NAN, NAN                   # where a wrapped offset would read
    ids = [n_blocks - 1, n_blocks - 30, n_blocks - 2]
    gen = torch.Generator(device="cuda").manual_seed(4)
    for i in ids:
        for c in (kc, vc):
            c[i] = torch.randn(bs, hk, d, generator=gen, device="cuda").to(T)
    lm = C.Lm(hq, hk, d, block_size=bs, n_blocks=n_blocks, table_blocks=3, max_requests=2, max_rows=64)
    x = (torch.randn(1, (hq + 2 * hk) * d, generator=gen, device="cuda")).to(T)
    q, k, v = (t.unflatten(1, (-1, d)) for t in x.split([hq * d, hk * d, hk * d], 1))
    qo = torch.zeros(1, hq, d, dtype=T, device="cuda")
    last = n_blocks * bs - 1
    lm.rotate(q, k, v, i32([0]), i32([last]), qo, kc, vc)       # position 0 turns by nothing
    assert torch.equal(kc.view(-1, hk, d)[last], k[0]) and torch.equal(vc.view(-1, hk, d)[last], v[0])
    kv, tables = [384, 200], [ids, ids]
    ks, vs = (f64(c[ids].flatten(0, 1)) for c in (kc, vc))
    q = torch.randn(12, hq, d, generator=gen, device="cuda").to(T)
    o = torch.zeros_like(q)
    lm.prompt_paged(q, kc, vc, i32([0, 10, 12]), i32(tables), i32(kv), o)
    n = [375 + i for i in range(10)] + [199, 200]
    ref = R.attention(f64(q), range(12), lambda r: (ks[:n[r]], vs[:n[r]]), hk, d ** -0.5)
    R.assert_attention(o, None, ref, "bf16", n, d, 5.0)
    for sh in (0, 1):
        lm.step(q[:2], kc, vc, i32(tables), i32(kv), o[:2], shared_table=i32(ids[:sh]) if sh else None)
        ref = R.attention(f64(q[:2]), range(2), lambda r: (ks[:kv[r]], vs[:kv[r]]), hk, d ** -0.5)
        R.assert_attention(o[:2], None, ref, "bf16", kv, d, 5.0)
    assert lm.errors() == 0


def test_bad_blocks_read_as_zeros():
    """A table entry out of range: score 0 and value 0 for its positions, and the bit."""
    hq, hk, d, bs = 4, 2, 64, 16
    for bad in (-1, 7, 2 ** 31 - 1, -2 ** 31):
        kc, vc, tables, _, n_blocks, width, gen = cache_case(9, [50, 20], hk, d, "bf16", bs)
        if bad == 7:
            bad = n_blocks
        q = torch.randn(2, hq, d, generator=gen, device="cuda").to(torch.bfloat16)
        blk = tables[0][1]
        lm = C.Lm(hq, hk, d, block_size=bs, n_blocks=n_blocks, table_blocks=width, max_requests=2, max_rows=2)
        o, o2 = (torch.zeros(2, hq, d, dtype=q.dtype, device="cuda") for _ in range(2))
        wrong = [list(t) for t in tables]
        wrong[0][1] = bad
        run = [lambda t, o: lm.step(q, kc, vc, i32(t), i32([50, 20]), o),
               lambda t, o: lm.prompt_paged(q, kc, vc, i32([0, 1, 2]), i32(t), i32([50, 20]), o)]
        outs = []
        for f in run:
            f(wrong, o)
            assert lm.errors() == C.LM_ERR_BLOCK
            outs.append(o.clone())
        kc[blk], vc[blk] = 0, 0
        for f, got in zip(run, outs):
            f(tables, o2)
            assert lm.errors() == 0 and torch.equal(got, o2)


def test_lengths_past_the_table_are_bent():
    kc, vc, tables, _, n_blocks, width, gen = cache_case(3, [48], 2, 64, "bf16", 16)
    tables[0][3] = tables[0][0]
    full = width * 16
    kc[tables[0][0]], vc[tables[0][0]] = 1, 1
    q = torch.randn(1, 4, 64, generator=gen, device="cuda").to(torch.bfloat16)
    lm = C.Lm(4, 2, 64, n_blocks=n_blocks, table_blocks=width, max_requests=1, max_rows=1)
    o, want = (torch.zeros(1, 4, 64, dtype=q.dtype, device="cuda") for _ in range(2))
    for f in (lambda n, o: lm.step(q, kc, vc, i32(tables), i32([n]), o),
              lambda n, o: lm.prompt_paged(q, kc, vc, i32([0, 1]), i32(tables), i32([n]), o)):
        f(full, want)
        assert lm.errors() == 0
        for n in (full + 1, 2 ** 31 - 1):
            f(n, o)
            assert lm.errors() == C.LM_ERR_LENGTH and torch.equal(o, want)
        f(-5, o)
        assert lm.errors() == C.LM_ERR_LENGTH and not o.any()


# ---- together ---------------------------------------------------------------

def test_layer_prompts_then_steps():
    """As a server uses them: a shared voice prompt, requests of different
    lengths behind it, then tokens one by one, with one captured graph for
    every step; each step's attention against 64 bits over all keys so far."""
    hq, hk, d, bs, B, sh = 8, 2, 128, 16, 5, 3
    width, n_blocks, max_rows = 12, 70, 128
    T = torch.bfloat16
    lm = C.Lm(hq, hk, d, "bf16", block_size=bs, n_blocks=n_blocks, table_blocks=width, max_requests=B,
              max_rows=max_rows, rope_theta=1e4)
    gen = torch.Generator(device="cuda").manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    gq, gk = 1 + 0.1 * r(d), 1 + 0.1 * r(d)
    kc, vc = (torch.full((n_blocks, bs, hk, d), NAN, dtype=T, device="cuda") for _ in range(2))
    z = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")
    tables = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    shared = i32([69, 5, 33])
    ids = [i for i in range(n_blocks) if i not in (69, 5, 33)]
    ring = i32(ids + [-1] * (n_blocks - len(ids)))
    free = [torch.tensor([0, len(ids)], device="cuda"), torch.zeros(2, dtype=torch.int64, device="cuda")]
    keys, vals = [[] for _ in range(B)], [[] for _ in range(B)]

    def project(n):
        return (r(n, (hq + 2 * hk) * d) * 2).to(T)

    def split(x):
        return [t.unflatten(1, (-1, d)) for t in x.split([hq * d, hk * d, hk * d], 1)]

    # the voice prompt: packed attention, keys and values into the shared blocks
    n = sh * bs
    q, k, v = split(project(n))
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    slots = (shared.repeat_interleave(bs) * bs + pos % bs).int()
    qo, ko = torch.zeros(n, hq, d, dtype=T, device="cuda"), torch.zeros(n, hk, d, dtype=T, device="cuda")
    lm.rotate(q, k, None, pos, None, qo, ko, None, q_gain=gq, k_gain=gk)
    lm.rotate(q, k, v, pos, slots, qo, kc, vc, q_gain=gq, k_gain=gk)
    o, o2 = torch.zeros_like(qo), torch.zeros_like(qo)
    lm.prompt(qo, ko, v, i32([0, n]), o)
    one = C.Lm(hq, hk, d, "bf16", block_size=bs, n_blocks=n_blocks, table_blocks=sh, max_requests=1, max_rows=n)
    one.prompt_paged(qo, kc, vc, i32([0, n]), shared.view(1, -1), i32([n]), o2)
    assert torch.equal(o, o2)
    ks, vs = f64(ko), f64(v)

    def check(o, qo, rows_of):
        ref = R.attention(f64(qo), range(qo.shape[0]),
                          lambda row: tuple(np.concatenate([s] + x[rows_of[row][0]])[:rows_of[row][1]]
                                            for s, x in ((ks, keys), (vs, vals))), hk, d ** -0.5)
        R.assert_attention(o, None, ref, "bf16", [n for _, n in rows_of], d, 8.0)

    def collect(qo_rows, k, v, starts, slots):
        kk = kc.view(-1, hk, d)[slots.long()]
        for b in range(B):
            a, e = starts[b], starts[b + 1]
            if e > a:
                keys[b].append(f64(kk[a:e]))
                vals[b].append(f64(v[a:e]))

    # the requests' own prompts
    new = [20, 1, 33, 16, 7]
    before, after = i32([n] * B), i32([n + x for x in new])
    row_start, kv_len, status, slots, pos = z(B + 1), z(B), z(B), z(max_rows), z(max_rows)
    lm.plan(before, after, tables, ring, free[0], free[1], row_start, kv_len, status, slots, pos, shared_table=shared)
    q, k, v = split(project(max_rows))      # padded: the rows behind the last request are not ours
    qo = torch.zeros(max_rows, hq, d, dtype=T, device="cuda")
    lm.rotate(q, k, v, pos, slots, qo, kc, vc, q_gain=gq, k_gain=gk)
    o = torch.full_like(qo, 5.0)
    lm.prompt_paged(qo, kc, vc, row_start, tables, kv_len, o)
    assert status.tolist() == [0] * B and (o[sum(new):] == 5).all() and not qo[sum(new):].any()
    starts = row_start.tolist()
    collect(qo, k, v, starts, slots)
    rows_of = [(b, n + i + 1) for b in range(B) for i in range(new[b])]
    check(o[:sum(new)], qo[:sum(new)], rows_of)

    # one token each per step, from one graph
    x = project(B)
    q, k, v = split(x)
    slots, pos, row_start = z(B), z(B), z(B + 1)
    qo, o = torch.zeros(B, hq, d, dtype=T, device="cuda"), torch.zeros(B, hq, d, dtype=T, device="cuda")
    before.copy_(after)
    side = torch.cuda.Stream()

    def layer():
        lm.plan(before, after, tables, ring, free[1], free[0], row_start, kv_len, status, slots, pos,
                shared_table=shared)
        lm.rotate(q, k, v, pos, slots, qo, kc, vc, q_gain=gq, k_gain=gk)
        lm.step(qo, kc, vc, tables, kv_len, o, shared_table=shared)

    after.add_(1)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        layer()
    lens = [n + v for v in new]
    for step in range(20):
        x.copy_(project(B))
        graph.replay()
        torch.cuda.synchronize()
        assert status.tolist() == [0] * B and lm.errors() == 0
        st = row_start.tolist()
        assert st == list(range(B + 1))
        collect(qo, k, v, st, slots)
        lens = [v + 1 for v in lens]
        check(o, qo, [(b, lens[b]) for b in range(B)])
        free[1].copy_(free[0])
        before.copy_(after)
        after.add_(1)


def test_two_streams_and_other_current_stream():
    """Calls go to the stream they are given, ordered with its other work."""
    lm = C.Lm(4, 2, 64, max_requests=1, max_rows=64)
    q, k, v, starts = prompt_inputs(1, [64], 4, 2, 64, "bf16", extra=0)
    want = torch.zeros(64, 4, 64, dtype=q.dtype, device="cuda")
    lm.prompt(q, k, v, i32(starts), want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    q2, o, rs = torch.zeros_like(q), torch.zeros_like(want), i32(starts)
    with torch.cuda.stream(side):
        torch.cuda._sleep(10_000_000)
        q2.copy_(q)
        lm.prompt(q2, k, v, rs, o)
    side.synchronize()
    assert torch.equal(o, want)
    o.zero_()
    torch.cuda.synchronize()
    lm.prompt(q2, k, v, rs, o, stream=side)
    side.synchronize()
    assert torch.equal(o, want)


# ---- refusals ---------------------------------------------------------------

def test_refusals():
    lm = C.Lm(4, 2, 64, block_size=16, n_blocks=4, table_blocks=3, max_requests=2, max_rows=8)
    T = torch.bfloat16
    q = torch.zeros(8, 4, 64, dtype=T, device="cuda")
    k = torch.zeros(8, 2, 64, dtype=T, device="cuda")
    kc = torch.zeros(4, 16, 2, 64, dtype=T, device="cuda")
    o, rs, tb, kv = torch.zeros_like(q), i32([0, 4, 8]), i32([[0] * 3] * 2), i32([8, 8])
    pos, slots = i32([0] * 8), i32(list(range(8)))

    def refused(kind, f, *a, **kw):
        with pytest.raises(kind):
            f(*a, **kw)

    V, E = ValueError, C.CodecError
    refused(V, lm.prompt, q.half(), k, k, rs, o)                        # another type
    refused(V, lm.prompt, q.cpu(), k, k, rs, o)                         # another device
    refused(V, lm.prompt, q[:, :2], k, k, rs, o)                        # heads missing
    refused(V, lm.prompt, q.transpose(1, 2).contiguous().transpose(1, 2), k, k, rs, o)   # heads apart
    refused(V, lm.prompt, q, k[:4], k, rs, o)                           # rows missing
    refused(V, lm.prompt, q, k, k, rs.long(), o)
    refused(V, lm.prompt, q, k, k, rs, o, lse=torch.zeros(8, 2, device="cuda"))
    wide = torch.zeros(8 * 260 + 8, dtype=T, device="cuda")
    refused(E, lm.prompt, wide[:8 * 260].view(8, 260)[:, :256].unflatten(1, (4, 64)), k, k, rs, o)    # stride of 520 bytes
    refused(E, lm.prompt, wide[4:4 + 2048].view(8, 4, 64), k, k, rs, o)  # 8-byte address
    refused(E, lm.prompt, torch.zeros(9, 4, 64, dtype=T, device="cuda"), torch.zeros(9, 2, 64, dtype=T, device="cuda"),
            torch.zeros(9, 2, 64, dtype=T, device="cuda"), rs, torch.zeros(9, 4, 64, dtype=T, device="cuda"))
    refused(E, lm.prompt, q, k, k, i32([0, 1, 2, 3]), o)                # three requests
    refused(V, lm.prompt_paged, q, kc[:3], kc, rs, tb, kv, o)
    refused(V, lm.prompt_paged, q, kc, kc, rs, tb[:, :2], kv, o)
    refused(V, lm.prompt_paged, q, kc, kc, rs, tb, kv[:1], o)
    refused(V, lm.step, q[:2], kc, kc.float(), tb, kv, o[:2])
    refused(V, lm.step, q[:1], kc, kc, tb, kv, o[:1])
    refused(E, lm.step, q[:2], kc, kc, tb, kv, o[:2], shared_table=i32([0] * 4))
    refused(E, lm.step, q[:3], kc, kc, i32([[0] * 3] * 3), i32([1] * 3), o[:3])
    refused(E, lm.rotate, q, k, k, pos, slots, o, kc, kc.clone(), q_gain=torch.ones(64, device="cuda"))
    refused(E, lm.rotate, q, k, None, pos, slots, o, kc, None)          # slots without values
    refused(V, lm.rotate, q, k.float(), k, pos, slots, o, kc, kc.clone())
    refused(V, lm.rotate, q.half(), k.half(), k.half(), pos, slots, o, kc, kc.clone())
    refused(V, lm.rotate, q, k, k, pos, slots, o[:, :2], kc, kc.clone())
    free = torch.tensor([0, 4], device="cuda")
    out = [i32([0] * 3), i32([0] * 2), i32([0] * 2), i32([0] * 8), i32([0] * 8)]
    refused(E, lm.plan, kv, kv, tb, i32([0] * 4), free, free, *out)     # counts in place
    refused(V, lm.plan, kv, kv, tb, i32([0] * 3), free, free.clone(), *out)
    refused(E, lm.plan, kv, kv, tb, i32([0] * 4), free, free.clone(), *out[:3], i32([0] * 9), i32([0] * 9))
    torch.cuda.synchronize()
    assert lm.errors() == 0 and not o.any() and not kc.any()
    lm.prompt(q[:0], k[:0], k[:0], rs, o[:0])                           # no rows: nothing to do
    for bad in (dict(head_dim=96), dict(q_heads=3), dict(q_heads=34), dict(block_size=24), dict(block_size=8),
                dict(n_blocks=0), dict(table_blocks=0), dict(max_requests=0), dict(max_requests=5000),
                dict(max_rows=0), dict(rope_theta=1.0), dict(rms_eps=-1.0), dict(scale=NAN), dict(n_blocks=2 ** 27)):
        with pytest.raises(C.CodecError) as e:
            C.Lm(**{**dict(q_heads=4, kv_heads=2, head_dim=64), **bad})
        assert e.value.status == 2, bad
    with pytest.raises(ValueError):
        C.Lm(4, 2, 64, "fp32")


# ---- places that a user may share, and scores without a finite one -----------

def test_outputs_in_place_are_refused_or_right():
    lm = C.Lm(4, 2, 64, block_size=16, n_blocks=4, table_blocks=3, max_requests=2, max_rows=8)
    T = torch.bfloat16
    x = torch.randn(8, 8, 64, device="cuda").to(T)
    q, k, v = x[:, :4].contiguous(), x[:, 4:6].contiguous(), x[:, 6:].contiguous()
    kc = torch.zeros(4, 16, 2, 64, dtype=T, device="cuda")
    before, after, kv = i32([0, 0]), i32([4, 4]), i32([0, 0])
    pos, slots = i32(list(range(8))), i32(list(range(8)))
    free = torch.tensor([0, 4], device="cuda")
    for a, b, c in ((before, after, before), (before, after, after), (kv, kv, kv)):
        with pytest.raises(C.CodecError) as e:
            lm.plan(a, b, i32([[0] * 3] * 2), i32(range(4)), free, free.clone(), i32([0] * 3), c, i32([0] * 2),
                    i32([0] * 8), i32([0] * 8))
        assert e.value.status == 4
    square = C.Lm(2, 2, 64, block_size=16, n_blocks=4, table_blocks=3, max_requests=2, max_rows=8)
    rs, tb = i32([0, 4, 8]), i32([[0] * 3] * 2)
    for call in (lambda: lm.prompt(q, k, v, rs, q), lambda: square.prompt(q[:, :2].contiguous(), k, v, rs, k),
                 lambda: square.prompt(q[:, :2].contiguous(), k, v, rs, v),
                 lambda: lm.prompt_paged(q, kc, kc, rs, tb, i32([8, 8]), q),
                 lambda: lm.step(q[:2], kc, kc, tb, i32([8, 8]), q[:2]),
                 lambda: lm.rotate(q, kc.view(-1, 2, 64)[:8], v, pos, slots, torch.empty_like(q), kc, kc.clone()),
                 lambda: lm.rotate(q, k, kc.view(-1, 2, 64)[:8], pos, slots, torch.empty_like(q), kc.clone(), kc)):
        with pytest.raises(C.CodecError) as e:
            call()
        assert e.value.status == 4
    # without slots in place
    qo, ko, vo = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    lm.rotate(q, k, v, pos, None, qo, ko, vo)
    lm.rotate(q, k, v, pos, None, q, k, v)
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(v, vo)
    for bad in (dict(table_blocks=2 ** 21 + 1, n_blocks=4, block_size=16),):
        with pytest.raises(C.CodecError) as e:
            C.Lm(4, 2, 64, **bad)
        assert e.value.status == 2


def test_length_out_of_range_is_told_without_rows_too():
    lm = C.Lm(4, 2, 64, block_size=16, n_blocks=4, table_blocks=3, max_requests=2, max_rows=8)
    q = torch.zeros(8, 4, 64, dtype=torch.bfloat16, device="cuda")
    kc = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16, device="cuda")
    lm.prompt_paged(q, kc, kc, i32([0, 8, 8]), i32([[0] * 3] * 2), i32([8, 49]), torch.zeros_like(q))
    assert lm.errors() == C.LM_ERR_LENGTH


@pytest.mark.parametrize("n,hq,hk,d,cut", [(300, 4, 2, 128, False), (2100, 4, 1, 64, True)])
def test_scores_of_minus_infinity_have_no_weight(n, hq, hk, d, cut):
    """Keys that score -inf for every row, more than a tile of them, in front of
    keys whose scores lie far below zero: only the latter count."""
    T, skip, bs = torch.bfloat16, 130, 16
    gen = torch.Generator(device="cuda").manual_seed(n)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    q = (2 + 0.1 * r(n, hq, d)).to(T)
    k, v = (-12 + 0.1 * r(n, hk, d)).to(T), r(n, hk, d).to(T)
    k[:skip] = -float("inf")
    k6, v6 = f64(k), f64(v)

    def check(o, rows):         # rows: of q
        ref = R.attention(f64(q)[rows], range(len(rows)), lambda i: (k6[skip:rows[i] + 1], v6[skip:rows[i] + 1]), hk, d ** -0.5)
        R.assert_attention(o, None, ref, "bf16", [x + 1 for x in rows], d, 5.0)

    blocks = -(-n // bs)
    lm = C.Lm(hq, hk, d, block_size=bs, n_blocks=blocks, table_blocks=blocks, max_requests=3, max_rows=n)
    rows = list(range(skip, n)) if not cut else list(range(skip, n, 61))
    o, o2 = torch.zeros_like(q), torch.zeros_like(q)
    lm.prompt(q, k, v, i32([0, n]), o)
    check(o[rows], rows)
    assert o[:skip].isnan().all()
    kc, vc = (torch.zeros(blocks, bs, hk, d, dtype=T, device="cuda") for _ in range(2))
    kc.view(-1, hk, d)[:n], vc.view(-1, hk, d)[:n] = k, v
    table = i32([list(range(blocks))])
    lm.prompt_paged(q, kc, vc, i32([0, n]), table, i32([n]), o2)
    check(o2[rows], rows)
    three = i32([n - 1, n - 100, skip])
    for shared in (None, table[0, :10].contiguous()):
        o3 = torch.zeros(3, hq, d, dtype=T, device="cuda")
        qs = q[[n - 2, n - 101, skip - 1]].contiguous()
        lm.step(qs, kc, vc, table.expand(3, -1).contiguous(), three, o3, shared_table=shared)
        check(o3[:2], [n - 2, n - 101])
        assert o3[2].isnan().all()
    assert lm.errors() == 0


@pytest.mark.parametrize("kv,sh,bs,hq,hk", [
    ([700], 40, 16, 4, 2),                                  # one request shares with nobody: many blocks read as its own
    ([2000, 10, 1030, 0, 33], 64, 16, 4, 1),                # up to 1,024 shared positions of few heads
    ([300] * 20 + [100, 256, 257, 0, 255], 2, 128, 8, 2),   # short shared part
    ([260 + i for i in range(40)], 16, 16, 16, 8),          # one more head, and it is a part of its own
    ([520 + i for i in range(17)], 32, 16, 8, 4),
])
def test_step_short_and_long_shared_parts(kv, sh, bs, hq, hk):
    lm, q, kc, vc, own, shared, o = check_step(kv, sh, hq, hk, 128, "bf16", bs, seed=len(kv))
    check_step(kv, sh, hq, hk, 64, "fp16", bs, seed=len(kv) + 1, mul=4.0)
    b = len(kv) // 2
    o1 = torch.zeros(1, hq, 128, dtype=q.dtype, device="cuda")
    lm.step(q[b:b + 1], kc, vc, i32(own[b:b + 1]), i32([kv[b]]), o1, shared_table=i32(shared))
    assert torch.equal(o1[0], o[b])
    # a block of the shared part that is none reads as zeros wherever it is read from
    wrong = list(shared)
    wrong[0] = -1
    kc2, vc2 = kc.clone(), vc.clone()
    kc2[shared[0]], vc2[shared[0]] = 0, 0
    o2, o3 = torch.zeros_like(o), torch.zeros_like(o)
    lm.step(q, kc, vc, i32(own), i32(kv), o2, shared_table=i32(wrong))
    assert lm.errors() == C.LM_ERR_BLOCK
    lm.step(q, kc2, vc2, i32(own), i32(kv), o3, shared_table=i32(shared))
    assert torch.equal(o2, o3) and lm.errors() == 0


@pytest.mark.parametrize("B,width", [(1, 1), (33, 1), (153, 30), (1025, 2), (1100, 40), (4096, 2)])
def test_step_many_requests_of_few_positions(B, width):
    """Units are looked up 32 requests at a time: one, two and three rounds of it,
    with tables that are split and tables that are not."""
    rng = random.Random(B)
    kv = [rng.choice([0, 1, 15, 16, 17, width * 16]) if rng.random() < 0.2 else rng.randrange(1, 30) % (width * 16 + 1)
          for _ in range(B)]
    n_blocks, d = 64, 64
    gen = torch.Generator(device="cuda").manual_seed(B)
    kc, vc = (torch.randn(n_blocks, 16, 2, d, generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2))
    tables = [[rng.randrange(n_blocks) for _ in range(width)] for _ in range(B)]     # requests may share blocks
    q = (torch.randn(B, 4, d, generator=gen, device="cuda") * 1.5).to(torch.bfloat16)
    lm = C.Lm(4, 2, d, n_blocks=n_blocks, table_blocks=width, max_requests=B, max_rows=B)
    o, lse = torch.full_like(q, 5.0), torch.full((B, 4), 5.0, device="cuda")
    lm.step(q, kc, vc, i32(tables), i32(kv), o, lse=lse)
    assert lm.errors() == 0
    k6, v6 = f64(kc), f64(vc)
    rows = sorted({0, B - 1, *rng.sample(range(B), min(B, 200))})

    def keys_of(i):
        b = rows[i]
        ids = tables[b][:-(-kv[b] // 16)]
        return tuple(x[ids].reshape(-1, 2, d)[:kv[b]] for x in (k6, v6))

    ref = R.attention(f64(q)[rows], range(len(rows)), keys_of, 2, d ** -0.5)
    R.assert_attention(o[rows], lse[rows], ref, "bf16", [kv[b] for b in rows], d, 5.0)


@pytest.mark.parametrize("new,kv,hq,hk,d,bs", [
    ([64, 64], [1200, 1100], 4, 2, 128, 16),            # just long enough to be cut, four tiles a piece
    ([33, 1, 70, 9], [497, 1990, 0, 1200], 10, 2, 64, 128),
    ([300, 2], [1300, 515], 7, 1, 128, 32),
    ([130], [1024], 4, 1, 128, 64),                     # just not
])
def test_prompt_paged_middling_context(new, kv, hq, hk, d, bs):
    check_paged(new, kv, hq, hk, d, "bf16", bs, seed=5)
    check_paged(new, kv, hq, hk, d, "fp16", bs, seed=6)


def tile_pairs(lens, hq, hk):
    """Pairs of query tiles that the prompts make, over all K/V heads."""
    pair = 2 * (128 // (hq // hk))
    return hk * sum(-(-n // pair) for n in lens)


@pytest.mark.parametrize("B", [33, 64, 200, 511, 512])
def test_prompt_list_of_many_sorted_requests(B):
    """More items than SMs and more requests than a warp has lanes, few enough to
    be ordered by their keys: whichever warp wrote a request's place in the
    list, each request's rows come out as alone."""
    rng = random.Random(B)
    hq, hk, d = 16, 8, 64
    lens = [rng.choice([0, 1, 2, 7, 30, 90]) for _ in range(B)]
    lens[rng.randrange(B)] = 300
    assert tile_pairs(lens, hq, hk) > 152
    check_prompt(lens, 2, 2, d, "fp16", seed=B)         # the definition, few heads
    q, k, v, starts = prompt_inputs(B, lens, hq, hk, d, "bf16", extra=2)
    n = q.shape[0]
    lm = C.Lm(hq, hk, d, max_requests=B, max_rows=n)
    one = C.Lm(hq, hk, d, max_requests=1, max_rows=300)
    o, lse = torch.full((n, hq, d), 5.0, dtype=q.dtype, device="cuda"), torch.full((n, hq), 5.0, device="cuda")
    lm.prompt(q, k, v, i32(starts), o, lse=lse)
    for b in range(B):
        x, y = starts[b], starts[b + 1]
        if y > x:
            want, want_lse = torch.zeros_like(o[x:y]), torch.zeros_like(lse[x:y])
            one.prompt(q[x:y], k[x:y], v[x:y], i32([0, y - x]), want, lse=want_lse)
            assert torch.equal(o[x:y], want) and torch.equal(lse[x:y], want_lse), b
    assert (o[starts[-1]:] == 5).all() and (lse[starts[-1]:] == 5).all() and lm.errors() == 0


@pytest.mark.parametrize("B,bs", [(33, 16), (150, 64), (512, 32)])
def test_prompt_paged_list_of_many_sorted_requests(B, bs):
    rng = random.Random(B)
    kv = [rng.choice([1, 5, 40, 130, 260]) for _ in range(B)]
    new = [min(n, rng.choice([0, 1, 3, 20])) for n in kv]
    assert tile_pairs([1] * B, 8, 8) > 152
    check_paged(new, kv, 8, 8, 64, "bf16", bs, seed=B)


@pytest.mark.parametrize("paged", [False, True])
def test_row_starts_that_overlap_stay_inside_the_outputs(paged):
    """Row starts that go back and forth name rows many times over: more items
    than a call can have.  The bit, and nothing written outside."""
    hq, hk, d, B, rows = 4, 4, 64, 60, 700
    T = torch.bfloat16
    gen = torch.Generator(device="cuda").manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(T)
    q, k, v = r(rows, hq, d), r(rows, hk, d), r(rows, hk, d)
    kc, vc = r(64, 16, hk, d), r(64, 16, hk, d)
    tables = torch.randint(64, (B, 50), generator=gen, device="cuda", dtype=torch.int32)
    lm = C.Lm(hq, hk, d, n_blocks=64, table_blocks=50, max_requests=B, max_rows=rows)
    guard = torch.full((3 * rows, hq, d), 5.0, dtype=T, device="cuda")
    lse = torch.full((3 * rows, hq), 5.0, device="cuda")
    for starts in ([0, rows] * 30 + [0], [rows - i for i in range(B + 1)], [2 ** 31 - 1, -2 ** 31] * 30 + [rows]):
        call = ((lambda: lm.prompt_paged(q, kc, vc, i32(starts), tables, i32([800] * B), guard[rows:2 * rows],
                                         lse=lse[rows:2 * rows])) if paged else
                (lambda: lm.prompt(q, k, v, i32(starts), guard[rows:2 * rows], lse=lse[rows:2 * rows])))
        call()
        assert lm.errors() == C.LM_ERR_LENGTH
        assert (guard[:rows] == 5).all() and (guard[2 * rows:] == 5).all()
        assert (lse[:rows] == 5).all() and (lse[2 * rows:] == 5).all()


# ---- values that are not finite, where they are seen -------------------------

def check_not_finite(got, q, rows, keys_of, hk, dt, n_keys, d):
    """NaN and infinities exactly where the definition has them (probabilities
    that are zero for the type do not occur here), all else within the bound."""
    with np.errstate(invalid="ignore"):
        want = R.attention(q, rows, keys_of, hk, d ** -0.5)[0]
    clean = R.attention(q, rows, lambda i: tuple(np.nan_to_num(x, nan=0.0, posinf=0.0, neginf=0.0) for x in keys_of(i)),
                        hk, d ** -0.5)
    g = f64(got)
    odd = ~np.isfinite(want)
    assert odd.any() and (~odd).any()
    wrong = ~(np.isfinite(g) == ~odd) | (np.isnan(g) != np.isnan(want)) | (np.isinf(want) & (g != want))
    assert not wrong.any(), f"{wrong.sum()} of {odd.sum()}, first {np.argwhere(wrong)[:4].tolist()}: {g[wrong][:4]} for {want[wrong][:4]}"
    patched = torch.from_numpy(np.where(odd, clean[0], g)).to(got.dtype)
    R.assert_attention(patched, None, clean, dt, n_keys, d, 6.0)


def poison(v, at):
    """Values of an early and a late key: one column NaN early and an infinity
    late, one with both infinities, one with the same twice, some with one."""
    inf = float("inf")
    early, late = at
    v[early, ..., 0], v[late, ..., 0] = NAN, inf
    v[early, ..., 1], v[late, ..., 1] = inf, -inf
    v[early, ..., 2], v[late, ..., 2] = -inf, -inf
    v[late, ..., 3] = NAN
    v[early, ..., 4] = inf
    v[late, ..., 5] = inf
    v[late - 1, ..., 6], v[late, ..., 6] = -inf, inf


@pytest.mark.parametrize("dt,d,hq,hk,lens", [
    ("bf16", 128, 4, 2, [300, 290]),            # an item per CTA
    ("fp16", 64, 3, 3, [300, 290]),
    ("bf16", 128, 8, 8, [290] * 12),            # a list
    ("fp16", 64, 4, 1, [2100, 290]),            # cut along the keys
])
@pytest.mark.parametrize("paged", [False, True])
def test_values_that_are_not_finite_come_out_as_defined(dt, d, hq, hk, lens, paged):
    bs = 16
    q, k, v, starts = prompt_inputs(11, lens, hq, hk, d, dt, extra=0)
    q.mul_(0.5)
    for b, x in enumerate(starts[:-1]):
        n = lens[b]
        poison(v[x:x + n], (5, n - 20))
    k[starts[1] + 9] = NAN                      # every row of the second request from its tenth on
    n = sum(lens)
    blocks = sum(-(-x // bs) for x in lens)
    lm = C.Lm(hq, hk, d, dt, block_size=bs, n_blocks=blocks, table_blocks=max(130, -(-max(lens) // bs)),
              max_requests=len(lens), max_rows=n)
    o = torch.zeros(n, hq, d, dtype=q.dtype, device="cuda")
    if paged:
        kc, vc = (torch.full((blocks, bs, hk, d), NAN, dtype=q.dtype, device="cuda") for _ in range(2))
        tables = torch.full((len(lens), lm._width), -1, dtype=torch.int32)
        at = 0
        for b, x in enumerate(starts[:-1]):
            kc.view(-1, hk, d)[at * bs:at * bs + lens[b]] = k[x:x + lens[b]]
            vc.view(-1, hk, d)[at * bs:at * bs + lens[b]] = v[x:x + lens[b]]
            c = -(-lens[b] // bs)
            tables[b, :c] = torch.arange(at, at + c)
            at += c
        lm.prompt_paged(q.contiguous(), kc, vc, i32(starts), tables.cuda(), i32(lens), o)
    else:
        lm.prompt(q, k, v, i32(starts), o)
    assert lm.errors() == 0
    where = [(s, s + i + 1) for s, e in zip(starts, starts[1:]) for i in range(e - s)]
    rows = sorted({r for s, e in zip(starts, starts[1:]) for r in (s, s + 4, s + 5, s + 12, s + 127, s + 128, e - 23, e - 22,
                                                                    e - 21, e - 20, e - 19, e - 1)})
    k6, v6 = f64(k), f64(v)
    check_not_finite(o[rows], f64(q)[rows], range(len(rows)),
                     lambda i: (k6[where[rows[i]][0]:where[rows[i]][1]], v6[where[rows[i]][0]:where[rows[i]][1]]), hk, dt,
                     [where[r][1] - where[r][0] for r in rows], d)


@pytest.mark.parametrize("dt,d,hq,hk", [("bf16", 128, 4, 2), ("fp16", 64, 3, 3)])
@pytest.mark.parametrize("sh", [0, 128])
def test_step_values_that_are_not_finite_come_out_as_defined(dt, d, hq, hk, sh):
    """The shared part as rows of one product (some requests end inside it), and
    each request's own part."""
    bs = 16
    kv = [2100, 2300, 2048, 1000, 40, 2040, 3, 0, 2200]
    kc, vc, tables, shared, n_blocks, width, gen = cache_case(21, kv, hk, d, dt, bs, sh)
    if sh:
        flat = vc[shared].flatten(0, 1)
        poison(flat, (5, 990))
        poison(flat, (1500, 2044))
        vc[shared] = flat.unflatten(0, (sh, bs))
    for b in (0, 8):                                            # in their own parts too
        blk = tables[b][kv[b] // bs - 1]
        vc[blk, 3, :, 1], vc[blk, 4, :, 7], vc[blk, 4, :, 8] = -float("inf"), NAN, float("inf")
    kc[tables[1][2200 // bs], 2] = NAN
    q = torch.randn(len(kv), hq, d, generator=gen, device="cuda").mul_(0.75).to(R.DTYPES[dt])
    lm = C.Lm(hq, hk, d, dt, block_size=bs, n_blocks=n_blocks, table_blocks=width, max_requests=len(kv), max_rows=9)
    o = torch.zeros_like(q)
    lm.step(q, kc, vc, i32(tables), i32(kv), o, shared_table=i32(shared) if sh else None)
    assert lm.errors() == 0
    ks = [(gathered(kc, tables[b], n, bs), gathered(vc, tables[b], n, bs)) for b, n in enumerate(kv)]
    check_not_finite(o, f64(q), range(len(kv)), lambda b: ks[b], hk, dt, kv, d)


def test_one_infinity_among_many_shared_positions_costs_little():
    """A request that ends inside the shared part makes all behind it places
    that some row may not see; an infinity there is found again in one pass
    (0.4 ms with it and 0.1 without; row by row it was 48)."""
    hq, hk, d, bs, sh, B = 32, 8, 128, 64, 128, 64
    T, width, n_blocks = torch.bfloat16, 132, 300
    gen = torch.Generator(device="cuda").manual_seed(2)
    kc, vc = (torch.randn(n_blocks, bs, hk, d, generator=gen, device="cuda").to(T) for _ in range(2))
    q = torch.randn(B, hq, d, generator=gen, device="cuda").to(T)
    o = torch.zeros_like(q)
    tables = torch.randint(sh, n_blocks, (B, width), generator=gen, device="cuda", dtype=torch.int32)
    shared, kv = torch.arange(sh, device="cuda", dtype=torch.int32), i32([8400] * (B - 1) + [5])
    lm = C.Lm(hq, hk, d, block_size=bs, n_blocks=n_blocks, table_blocks=width, max_requests=B, max_rows=B)

    def ms():
        times = []
        for _ in range(4):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            lm.step(q, kc, vc, tables, kv, o, shared_table=shared)
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b))
        return min(times)

    without = ms()
    vc[7, 3, :, 0] = float("inf")
    assert ms() < 40 * without
    assert o[:-1, :, 0].isposinf().all() and o[:, :, 1:].isfinite().all() and o[-1].isfinite().all()


@pytest.mark.parametrize("dt,hq,hk,d", [("bf16", 16, 8, 128), ("fp16", 32, 8, 64)])
def test_step_a_head_does_not_depend_on_the_others_of_its_group(dt, hq, hk, d):
    """Units of eight tiles in which running references move often: a head's
    moves for its own scores alone, so its bits are the same beside others."""
    B, bs = 20, 32
    kv = [500 - 7 * i for i in range(B)]
    kc, vc, tables, _, n_blocks, width, gen = cache_case(31, kv, hk, d, dt, bs)
    assert width * bs > 500 and width * bs <= 512 + bs
    tables = [t[:16] for t in tables]
    r = lambda: torch.randn(B, hk, hq // hk, d, generator=gen, device="cuda")
    q, q2 = r() * 12, r() * 12
    q2[:, :, 0] = q[:, :, 0]
    lm = C.Lm(hq, hk, d, dt, block_size=bs, n_blocks=n_blocks, table_blocks=16, max_requests=B, max_rows=B)
    outs = []
    for x in (q, q2):
        x = x.to(R.DTYPES[dt]).view(B, hq, d)
        o, lse = torch.zeros_like(x), torch.zeros(B, hq, device="cuda")
        lm.step(x, kc, vc, i32(tables), i32(kv), o, lse=lse)
        outs.append((o.view(B, hk, -1, d)[:, :, 0], lse.view(B, hk, -1)[:, :, 0]))
    assert lm.errors() == 0
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


# ---- waits that run out -------------------------------------------------------

@pytest.mark.parametrize("form", ["prompt", "list", "cut", "step joined inside", "step joined after", "shared"])
def test_bounded_waits_run_out_report_and_recover(form):
    """One warp per CTA waits for a barrier that nothing arrives on while the
    other roles are at work: the kernels stop cleanly, the bit is set, and after
    it is cleared the same call gives its bits again."""
    T, hq, hk, d, bs = torch.bfloat16, 8, 4, 128, 16
    gen = torch.Generator(device="cuda").manual_seed(6)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(T)
    if form in ("prompt", "list"):
        lens = [400, 30] if form == "prompt" else [150] * 60
        n = sum(lens)
        q, k, v = r(n, hq, d), r(n, hk, d), r(n, hk, d)
        starts = i32([sum(lens[:i]) for i in range(len(lens) + 1)])
        lm = C.Lm(hq, hk, d, max_requests=len(lens), max_rows=n)
        call = lambda o: lm.prompt(q, k, v, starts, o)
    else:
        B, width = (1, 313) if form == "step joined inside" else (2, 300) if form == "cut" else (40, 120)
        kc, vc = r(400, bs, hk, d), r(400, bs, hk, d)
        tables = torch.randint(400, (B, width), generator=gen, device="cuda", dtype=torch.int32)
        kv = i32([width * bs - 5 * b for b in range(B)])
        n = 70 if form == "cut" else B
        q = r(n, hq, d)
        lm = C.Lm(hq, hk, d, n_blocks=400, table_blocks=width, max_requests=B, max_rows=n)
        shared = tables[0, :80].contiguous() if form == "shared" else None
        starts = i32([0, 40, 70])
        call = ((lambda o: lm.prompt_paged(q, kc, vc, starts, tables, kv, o)) if form == "cut" else
                (lambda o: lm.step(q, kc, vc, tables, kv, o, shared_table=shared)))
    want, o = torch.zeros_like(q), torch.zeros_like(q)
    call(want)
    assert lm.errors() == 0 and want.any()
    for _ in range(2):
        lm.set_unarrived_wait(1000)
        call(o)
        bits = lm.errors()
        lm.set_unarrived_wait(0)
        assert bits == C.LM_ERR_TIMEOUT
        call(o.zero_())
        assert lm.errors() == 0 and torch.equal(o, want)


# ---- plans of more requests than a CTA has threads -----------------------------

@pytest.mark.parametrize("seed,B,bs,sh,width,max_rows,free,old,new,bad", [
    (10, 1024, 16, 0, 30, 20000, 3000, 300, 40, False),
    (11, 1025, 16, 2, 30, 20000, 3000, 300, 40, False),
    (12, 2049, 32, 1, 20, 90000, 400, 400, 60, True),       # the blocks run out behind the first thousand
    (13, 3000, 16, 0, 12, 11000, 9000, 100, 40, False),     # the rows run out in the third
    (14, 4096, 128, 3, 9, 400000, 9000, 500, 300, True),
])
def test_plan_of_many_requests(seed, B, bs, sh, width, max_rows, free, old, new, bad):
    before, after, tables, ring, fr, shared, n_blocks = plan_case(seed, B, bs, sh, width, max_rows, free, old, new, bad)
    lm = C.Lm(8, 8, 64, block_size=bs, n_blocks=n_blocks, table_blocks=width, max_requests=B, max_rows=max_rows)
    got = run_plan(lm, before, after, tables, ring, fr, shared, max_rows)
    want = R.plan(before, after, tables, ring, fr, shared, bs, max_rows)
    for k in want:
        assert got[k] == want[k], k
    assert lm.errors() == 0
    stop = {12: 1, 13: 3}.get(seed)
    if stop:
        assert want["status"].index(stop) > 1024


def test_plan_rows_that_do_not_fit_leave_all_behind_them():
    """The third request's rows pass max_rows: it, one that ended, one that did
    not change and one that grows are all left as they were."""
    lm = C.Lm(8, 8, 64, n_blocks=12, table_blocks=4, max_requests=6, max_rows=20)
    before, after = [16, 30, 0, 40, 20, 5], [17, 16, 20, 0, 20, 6]
    tables = [[0, -1, -1, -1], [1, 2, -1, -1], [-1] * 4, [3, 4, 5, -1], [6, 7, -1, -1], [8, -1, -1, -1]]
    got = run_plan(lm, before, after, tables, [9, 10, 11] + [-1] * 9, (0, 3), [], 20)
    assert got["status"] == [0, 0, 3, 3, 3, 3] and got["kv_len"] == [17, 16, 0, 0, 0, 0]
    assert got["free_out"] == [1, 4] and got["free_list"][3] == 2
    assert got["row_start"] == [0, 1, 1, 20, 20, 20, 20]
    assert got["tables"] == [[0, 9, -1, -1]] + tables[1:] and lm.errors() == 0
    assert got["slots"] == [9 * 16] + [-1] * 19 and got["positions"] == [16] + list(range(19))


@pytest.mark.parametrize("call", ["plan", "rotate", "prompt", "prompt_paged", "step", "errors"])
def test_first_call_of_a_new_host_thread(call):
    """A thread that has made no CUDA call before has no context bound yet."""
    hq, hk, d = 4, 2, 64
    T = torch.bfloat16
    gen = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(T)
    q, k, v, kc, vc = r(20, hq, d), r(20, hk, d), r(20, hk, d), r(8, 16, hk, d), r(8, 16, hk, d)
    starts, tables, kv = i32([0, 9, 20]), i32([[0, 1, 2], [3, 4, 5]]), i32([33, 48])
    lm = C.Lm(hq, hk, d, n_blocks=8, table_blocks=3, max_requests=2, max_rows=20)
    stream = torch.cuda.current_stream()
    free = torch.tensor([0, 8], device="cuda")

    def run(o):
        z = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")
        out, ring = [z(3), z(2), z(2), z(20), z(20)], i32(range(8))
        qo, kd, vd, t = torch.zeros_like(q), torch.zeros_like(kc), torch.zeros_like(vc), tables.clone()
        pos, before, after, counts = i32(range(20)), i32([5, 0]), i32([9, 7]), torch.zeros_like(free)
        torch.cuda.synchronize()
        return {"plan": lambda: (lm.plan(before, after, t, ring, free, counts, *out, stream=stream), out[3]),
                "rotate": lambda: (lm.rotate(q, k, v, pos, pos, qo, kd, vd, stream=stream), qo),
                "prompt": lambda: (lm.prompt(q, k, v, starts, o, stream=stream), o),
                "prompt_paged": lambda: (lm.prompt_paged(q, kc, vc, starts, tables, kv, o, stream=stream), o),
                "step": lambda: (lm.step(q[:2], kc, vc, tables, kv, o[:2], stream=stream), o),
                "errors": lambda: (None, torch.tensor(lm.errors(stream=stream)))}[call]

    want = run(torch.zeros_like(q))()[1]
    got, f = [], run(torch.zeros_like(q))

    def work():
        try:
            got.append(f()[1])
        except Exception as e:      # told by the other thread
            got.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert torch.is_tensor(got[0]), got[0]
    assert torch.equal(got[0], want) and lm.errors() == 0


# ---- captured calls and several streams ----------------------------------------

def test_graph_of_steps_behind_a_long_shared_part_follows_the_lengths():
    """Rotation, shared part, own parts and join in one graph: nothing of the
    last replay's queries, lengths or cache may be seen by the next."""
    hq, hk, d, bs, sh, B = 16, 8, 128, 16, 96, 40
    T, width, n_blocks = torch.bfloat16, sh + 12, 200
    gen = torch.Generator(device="cuda").manual_seed(12)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    kc, vc = r(n_blocks, bs, hk, d).to(T), r(n_blocks, bs, hk, d).to(T)
    tables = torch.randint(n_blocks, (B, width), generator=gen, device="cuda", dtype=torch.int32)
    shared = torch.randperm(n_blocks, generator=gen, device="cuda")[:sh].to(torch.int32)
    mk = lambda: C.Lm(hq, hk, d, n_blocks=n_blocks, table_blocks=width, max_requests=B, max_rows=B)
    lm, eager = mk(), mk()
    x = torch.zeros(B, (hq + 2 * hk) * d, dtype=T, device="cuda")
    q, k, v = (t.unflatten(1, (-1, d)) for t in x.split([hq * d, hk * d, hk * d], 1))
    pos, slots, kv = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(3))
    qo, o = torch.zeros(B, hq, d, dtype=T, device="cuda"), torch.zeros(B, hq, d, dtype=T, device="cuda")

    def layer(lm, kc, vc, qo, o):
        lm.rotate(q, k, v, pos, slots, qo, kc, vc)
        lm.step(qo, kc, vc, tables, kv, o, shared_table=shared)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer(lm, kc, vc, qo, o)
    for i in range(12):
        x.copy_((r(B, (hq + 2 * hk) * d) * 3).to(T))
        kv.copy_(torch.randint(0, width * bs + 1, (B,), generator=gen, device="cuda") * (torch.arange(B, device="cuda") % 5 != i % 5))
        pos.copy_(torch.randint(width * bs, (B,), generator=gen, device="cuda"))
        slots.copy_(torch.randperm(n_blocks * bs, generator=gen, device="cuda")[:B])
        kc2, vc2, want = kc.clone(), vc.clone(), torch.zeros_like(o)
        torch.cuda.synchronize()
        layer(eager, kc2, vc2, torch.zeros_like(qo), want)
        torch.cuda.synchronize()
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(kc, kc2) and torch.equal(vc, vc2) and torch.equal(o, want), i
    assert lm.errors() == 0 and eager.errors() == 0


def test_objects_on_streams_of_their_own_run_at_once():
    """Prompts, steps behind a shared part and prompts behind the cache, each
    object on its own stream and host thread: each gives the bits it gives alone."""
    hq, hk, d = 16, 8, 128
    T = torch.bfloat16
    gen = torch.Generator(device="cuda").manual_seed(8)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(T)
    lens = [60, 900, 300, 500] * 3
    n = sum(lens)
    q, k, v, starts = r(n, hq, d), r(n, hk, d), r(n, hk, d), i32([sum(lens[:i]) for i in range(13)])
    kc, vc = r(300, 16, hk, d), r(300, 16, hk, d)
    tables = torch.randint(300, (30, 110), generator=gen, device="cuda", dtype=torch.int32)
    shared, kv = tables[0, :80].contiguous(), i32([1281 + 11 * i for i in range(30)])
    mk = lambda: C.Lm(hq, hk, d, n_blocks=300, table_blocks=110, max_requests=30, max_rows=n)
    two, tables2, kv2 = i32([0, 40, 90]), tables[:2].contiguous(), kv[:2].contiguous()
    calls = [lambda lm, o, s: lm.prompt(q, k, v, starts, o, stream=s),
             lambda lm, o, s: lm.step(q[:30], kc, vc, tables, kv, o[:30], shared_table=shared, stream=s),
             lambda lm, o, s: lm.prompt_paged(q[:90], kc, vc, two, tables2, kv2, o[:90], stream=s)]
    wants, lms = [], [mk() for _ in calls]
    for f, lm in zip(calls, lms):
        wants.append(torch.zeros_like(q))
        f(lm, wants[-1], torch.cuda.current_stream())
    outs = [[torch.zeros_like(q) for _ in range(8)] for _ in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()

    def work(i):
        for o in outs[i]:
            calls[i](lms[i], o, streams[i])

    threads = [threading.Thread(target=work, args=(i,)) for i in range(3)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    torch.cuda.synchronize()
    for want, out, lm in zip(wants, outs, lms):
        assert want.any() and all(torch.equal(o, want) for o in out) and lm.errors() == 0
