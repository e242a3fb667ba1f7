"""The codec LM's cache in 4 bits, forked and compacted blocks, and beam search
against their definitions: bytes and whole numbers equal, attention within what
its arithmetic allows."""
from __future__ import annotations

import random

import numpy as np
import pytest
import torch

import lm_q4_ref as Q
from streaming_tts_vocoder_gb300 import codec as C

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")
T = Q.DTYPES


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def f64(t):
    return t.detach().cpu().double().numpy()


def gpu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


# ---- store and load ---------------------------------------------------------

def rows_of_kinds(rows, hk, d, seed):
    """float32 rows with flat, tiny, huge and not finite groups among ordinary ones."""
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(rows, hk, d)).astype(np.float32)
    x *= (10.0 ** rng.integers(-4, 4, size=(rows, hk, 1))).astype(np.float32)
    f = x.reshape(rows, hk, -1, 32)
    kind = rng.integers(0, 12, size=f.shape[:3])
    f[kind == 0] = 0.0
    f[kind == 1] = 0.1
    f[kind == 2] += 300.0
    f[kind == 3] *= 1e-7
    for r, h, g in np.argwhere(kind == 4)[:4]:
        f[r, h, g, rng.integers(32)] = [np.nan, np.inf, -np.inf, 3e38][r % 4]
    return x


@pytest.mark.parametrize("rows,hk,d,dt,it,bs", [
    (1, 8, 128, "bf16", "bf16", 16), (5, 1, 64, "fp16", "fp32", 32), (33, 3, 128, "fp16", "fp16", 64),
    (70, 2, 64, "bf16", "fp32", 128), (300, 5, 64, "bf16", "bf16", 16), (2700, 8, 128, "bf16", "fp32", 64),
])
def test_store_and_load(rows, hk, d, dt, it, bs):
    n_blocks = -(-rows // bs) + 3
    lm = C.Lm(hk, hk, d, dt, block_size=bs, n_blocks=n_blocks, max_rows=rows)
    rng = np.random.default_rng(rows)
    both = torch.from_numpy(np.concatenate([rows_of_kinds(rows, hk, d, s).reshape(rows, -1) for s in (1, 2)], 1))
    if it == "fp16":
        both = both.clamp(-65504, 65504)
    both = both.to(T[it]).cuda()
    wide = torch.zeros(rows, 2 * hk * d + 8, dtype=T[it], device="cuda")
    wide[:, :2 * hk * d] = both                     # rows further apart than they are wide
    k, v = (t.unflatten(1, (hk, d)) for t in wide[:, :2 * hk * d].split(hk * d, 1))
    slots = rng.permutation(n_blocks * bs)[:rows]
    if n_blocks * bs - 1 not in slots:
        slots[rows // 2] = n_blocks * bs - 1
    if rows > 4:
        slots[::5] = -1
    fill = rng.integers(0, 256, size=(2, n_blocks, hk, bs * d * 5 // 8), dtype=np.uint8)
    kc, vc = gpu(fill[0]), gpu(fill[1])
    lm.store_q4(k, v, i32(slots.tolist()), kc, vc)
    assert lm.errors() == 0
    for t, c, want, keys in ((k, kc, fill[0], True), (v, vc, fill[1], False)):
        Q.store(want, t.float().cpu().numpy(), slots, bs, keys)
        got = c.cpu().numpy()
        # a NaN's bits and a zero's sign are free
        if not np.array_equal(got, want):
            a, b = (Q.values(x, bs, d, keys) for x in (got, want))
            assert np.array_equal(a, b, equal_nan=True)
            assert (got != want).sum() <= 2 * (np.isnan(b).sum() + (b == 0).sum())
    # back: some blocks, in another order, others left as they were
    src = rng.permutation(n_blocks)
    dst = rng.permutation(n_blocks + 4)[:n_blocks]
    src[::4] = -1
    kd, vd = (torch.full((n_blocks + 4, bs, hk, d), 7.0, dtype=T[dt], device="cuda") for _ in range(2))
    lm.load_q4(kc, vc, i32(src.tolist()), i32(dst.tolist()), kd, vd)
    assert lm.errors() == 0
    for c, out, keys in ((kc, kd, True), (vc, vd, False)):
        want = np.full(out.shape, 7.0)
        with np.errstate(all="ignore"):
            y = Q.values(c.cpu().numpy(), bs, d, keys).astype(np.float32)
            if dt == "fp16":
                y = np.where(y > 65504, np.float32(65504), y)
        y = torch.from_numpy(y).to(T[dt]).double().numpy()
        for s, e in zip(src, dst):
            if s >= 0:
                want[e] = y[s]
        assert np.array_equal(f64(out), want, equal_nan=True)


def test_store_and_load_leave_wrong_places_out():
    lm = C.Lm(2, 2, 64, n_blocks=2, max_rows=8)
    x = torch.randn(6, 2, 64, device="cuda")
    kc, vc = (torch.zeros(2, 2, 640, dtype=torch.uint8, device="cuda") for _ in range(2))
    lm.store_q4(x, x, i32([0, 32, -2, 2 ** 31 - 1, -2 ** 31, 31]), kc, vc)
    assert lm.errors() == C.LM_ERR_SLOT and lm.errors() == 0
    for c, keys in ((kc, True), (vc, False)):
        y = Q.values(c.cpu().numpy(), 16, 64, keys).reshape(32, -1)
        assert [bool(r.any()) for r in y] == [True] + [False] * 30 + [True]
    kd, vd = (torch.zeros(3, 16, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lm.load_q4(kc, vc, i32([0, 2, -2, 0, 0, 2 ** 31 - 1]), i32([1, 0, 0, 3, -1, 0]), kd, vd)
    assert lm.errors() == C.LM_ERR_BLOCK
    assert [bool(b.any()) for b in kd] == [False, True, False] == [bool(b.any()) for b in vd]


# ---- single tokens ----------------------------------------------------------

HEADS = [(16, 16, 64), (16, 8, 128), (7, 1, 128), (10, 2, 64), (12, 4, 128), (16, 1, 64), (3, 3, 128), (9, 1, 128)]


def cache_q4(seed, lens, hk, d, bs, sh=0, v_mul=1.0):
    """Caches whose bytes behind a length are 0xFF (scales and lows NaN); tables
    whose entries behind a length are out of range."""
    rng = np.random.default_rng(seed)
    counts = [max(0, -(-n // bs) - sh) for n in lens]
    n_blocks, width = sh + sum(counts) + 3, max(1, sh + max(counts) + 1)
    ids = rng.permutation(n_blocks).tolist()
    shared, ids = ids[:sh], ids[sh:]
    kc, vc = (torch.full((n_blocks, hk, bs * d * 5 // 8), 255, dtype=torch.uint8, device="cuda") for _ in range(2))
    tables = [[2 ** 31 - 1] * width for _ in lens]
    slots = [i * bs + p for i in shared for p in range(bs)]
    for b, n in enumerate(lens):
        tables[b][:sh] = shared
        mine, ids = ids[:counts[b]], ids[counts[b]:]
        tables[b][sh:sh + counts[b]] = mine
        slots += [tables[b][p // bs] * bs + p % bs for p in range(sh * bs, n)]
    if slots:
        k = rng.normal(size=(len(slots), hk, d)) * (1 + 2 * (rng.random((hk, d)) < 0.05))
        v = rng.normal(size=(len(slots), hk, d)) * v_mul
        one = C.Lm(hk, hk, d, block_size=bs, n_blocks=n_blocks, max_rows=len(slots))
        one.store_q4(gpu(k.astype(np.float32)), gpu(v.astype(np.float32)), i32(slots), kc, vc)
        assert one.errors() == 0
    return kc, vc, tables, shared, n_blocks, width


def as_halves(dt, most, hq, hk, shared_len):
    """Positions of the shared part that the batch has in common as halves: none
    where it is units of the step's own kernel (fp16, or by tiles of 16 keys x 8 or
    16 columns of an object for `most` requests) or read by every request."""
    wide = 16 if hq // hk > 8 else 8
    return 0 if dt != torch.bfloat16 or most == 1 or most * hq // wide * (shared_len // 16) <= 16384 else min(shared_len, 32768)


def step_reference(q, kc, vc, tables, lens, shared, hk, d, bs, scale=None, most=1):
    sh = len(shared)
    parts = [Q.values(c.cpu().numpy(), bs, d, keys, parts=True) for c, keys in ((kc, True), (vc, False))]
    halves = as_halves(q.dtype, most, q.shape[1], hk, sh * bs)

    def keys_of(b):
        n = lens[b]
        ids = [(shared + tables[b][sh:])[j] for j in range(-(-n // bs))]
        got = []
        for low, rest in parts:
            low, rest = (x[ids].reshape(-1, hk, d)[:n].copy() for x in (low, rest))
            rest[:halves] = (low[:halves] + rest[:halves]).astype(np.float16).astype(np.float64) - low[:halves]
            got += [low, rest]
        return got

    return Q.step(f64(q), keys_of, hk, scale or d ** -0.5)


def check_step(lens, sh, hq, hk, d, dt, bs, seed=0, mul=1.0, v_mul=1.0, most=None, scale=0.0):
    kc, vc, tables, shared, n_blocks, width = cache_q4(seed, lens, hk, d, bs, sh, v_mul=v_mul)
    B = len(lens)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    q = (torch.randn(B, hq * d + 16, generator=gen, device="cuda") * 1.5 * mul).to(T[dt])[:, :hq * d].unflatten(1, (hq, d))
    lm = C.Lm(hq, hk, d, dt, block_size=bs, n_blocks=n_blocks, table_blocks=width, max_requests=most or B, max_rows=B,
              scale=scale)
    o = torch.full((B, hq * d + 8), 5.0, dtype=q.dtype, device="cuda")
    o = o[:, :hq * d].unflatten(1, (hq, d))
    lse = torch.full((B, hq), 5.0, device="cuda")
    own = [[-1] * sh + t[sh:] for t in tables]      # the entries of the shared blocks are not read
    run = lambda o, lse: lm.step_q4(q, kc, vc, i32(own), i32(lens), o, shared_table=i32(shared) if sh else None, lse=lse)
    run(o, lse)
    assert lm.errors() == 0
    ref = step_reference(q, kc, vc, tables, lens, shared, hk, d, bs, scale, most or B)
    Q.assert_step(o, lse, ref, dt, d, 6.0 * v_mul)
    o2 = torch.zeros(B, hq, d, dtype=q.dtype, device="cuda")
    run(o2, None)
    assert torch.equal(o2, o)
    return lm, q, kc, vc, own, shared, o


@pytest.mark.parametrize("hq,hk,d", HEADS)
@pytest.mark.parametrize("bs", [16, 32, 64, 128])
def test_step(hq, hk, d, bs):
    dt = "fp16" if bs in (16, 64) else "bf16"
    check_step([1, 0, 17, 128, 129, 260], 0, hq, hk, d, dt, bs)
    # behind a shared part: nothing, one, several blocks; shorter than the shared part; idle
    check_step([2 * bs, 2 * bs + 1, 2 * bs + 70, 0, bs + 3, 1], 2, hq, hk, d, dt, bs, seed=1)
    # the same behind more of it, for a few and for many requests
    lens = [11 * bs, 11 * bs + 1, 11 * bs + 70, 0, 11 * bs - 1, bs + 3, 1]
    check_step(lens, 11, hq, hk, d, dt, bs, seed=2)
    assert as_halves(T["bf16"], 4096, hq, hk, 11 * bs)
    check_step(lens, 11, hq, hk, d, dt, bs, seed=3, most=4096)


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 255, 257, 500])
def test_step_lengths(n):
    check_step([n], 0, 4, 2, 128, "bf16", 16, seed=n)
    check_step([n, 3], 0, 2, 2, 64, "fp16", 128, seed=n)


@pytest.mark.parametrize("lens,sh,bs", [([1000], 0, 16), ([2100, 5, 700], 0, 64), ([1500] * 3, 64, 16),
                                        ([700] * 70, 9, 64), ([4200], 32, 128), ([1100 + 37 * i for i in range(24)], 66, 16)])
def test_step_long(lens, sh, bs):
    check_step(lens, sh, 4, 2, 128, "bf16", bs)
    check_step(lens, sh, 4, 1, 64, "fp16", bs, seed=2, mul=8.0)


@pytest.mark.parametrize("dt,sh", [("bf16", 0), ("fp16", 0), ("fp16", 520), ("bf16", 520)])
def test_step_units_of_many_positions(dt, sh):
    """Tables of more than 65,536 positions: units of 2,048, looked up in more than one turn."""
    check_step([68000, 66561, 0] if sh else [68000, 2049], sh, 2, 1, 64, dt, 128, seed=5)


@pytest.mark.parametrize("v_mul", [3e-4, 40.0, 4000.0])
def test_step_values_of_other_sizes(v_mul):
    check_step([300, 40, 1], 0, 4, 2, 128, "bf16", 32, seed=3, v_mul=v_mul)
    check_step([70, 500], 1, 16, 1, 64, "fp16", 32, seed=4, v_mul=v_mul)


def test_step_scales_that_grow_along_the_keys():
    """Each tile's values are larger than all before it, and the last ones small again."""
    hq, hk, d, bs, n = 8, 2, 128, 16, 400
    kc, vc, tables, shared, n_blocks, width = cache_q4(5, [n], hk, d, bs)
    gen = torch.Generator(device="cuda").manual_seed(0)
    grow = (2.0 ** (torch.arange(n, device="cuda") % 330 / 25)).view(-1, 1, 1)
    v = torch.randn(n, hk, d, generator=gen, device="cuda") * grow
    k = torch.randn(n, hk, d, generator=gen, device="cuda") * 0.3
    slots = i32([tables[0][p // bs] * bs + p % bs for p in range(n)])
    lm = C.Lm(hq, hk, d, "bf16", block_size=bs, n_blocks=n_blocks, table_blocks=width, max_requests=1, max_rows=n)
    lm.store_q4(k, v, slots, kc, vc)
    q = torch.randn(1, hq, d, generator=gen, device="cuda").bfloat16()
    o, lse = torch.zeros_like(q), torch.zeros(1, hq, device="cuda")
    lm.step_q4(q, kc, vc, i32(tables), i32([n]), o, lse=lse)
    Q.assert_step(o, lse, step_reference(q, kc, vc, tables, [n], [], hk, d, bs), "bf16", d, float(v.abs().max()))


def test_step_queries_of_any_size():
    """Whole rows of queries a power of two larger or smaller, with the scale that
    undoes it: the scores are the same."""
    lens, hq, hk, d, bs = [200, 31], 6, 2, 64, 16
    kc, vc, tables, _, n_blocks, width = cache_q4(6, lens, hk, d, bs)
    q = torch.randn(2, hq, d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(6)).bfloat16()
    outs = []
    for e in (-60, -20, 0, 20, 60):
        lm = C.Lm(hq, hk, d, "bf16", block_size=bs, n_blocks=n_blocks, table_blocks=width, max_requests=2, max_rows=2,
                  scale=0.125 * 2.0 ** -e)
        o = torch.zeros_like(q)
        lm.step_q4(q * 2.0 ** e, kc, vc, i32(tables), i32(lens), o)
        outs.append(o)
    assert all(torch.equal(o, outs[2]) for o in outs)
    zero = torch.zeros_like(q)
    lm.step_q4(zero, kc, vc, i32(tables), i32(lens), outs[0])      # every key alike
    Q.assert_step(outs[0], None, step_reference(zero, kc, vc, tables, lens, [], hk, d, bs), "bf16", d, 6.0)
    # the same behind a shared part, as units and as halves
    lens = [500, 420]
    kc, vc, tables, shared, n_blocks, width = cache_q4(6, lens, hk, d, bs, 25)
    for most in (2, 4096):
        outs = []
        for e in (-60, 0, 60):
            lm = C.Lm(hq, hk, d, "bf16", block_size=bs, n_blocks=n_blocks, table_blocks=width, max_requests=most,
                      max_rows=2, scale=0.125 * 2.0 ** -e)
            outs.append(torch.zeros_like(q))
            lm.step_q4(q * 2.0 ** e, kc, vc, i32(tables), i32(lens), outs[-1], shared_table=i32(shared))
        assert torch.equal(outs[0], outs[1]) and torch.equal(outs[2], outs[1])
        # a query that is not finite stays its own row's and head's
        for what in (NAN, INF, -INF):
            bad, o = q.clone(), torch.zeros_like(q)
            bad[1, 4, 9] = what
            lm.step_q4((bad * 2.0 ** 60), kc, vc, i32(tables), i32(lens), o, shared_table=i32(shared))
            rest = torch.ones(2, hq, dtype=torch.bool, device="cuda")
            rest[1, 4] = False
            assert torch.equal(o[rest], outs[1][rest]) and o[1, 4].isnan().all() and lm.errors() == 0


def test_step_result_does_not_depend_on_the_batch():
    for hq, hk, d, dt, sh, mul, most in (
            (8, 2, 128, "bf16", 2, 1.0, None), (8, 2, 128, "bf16", 66, 8.0, None), (4, 4, 64, "fp16", 66, 8.0, None),
            (16, 1, 64, "fp16", 66, 4.0, None), (8, 2, 128, "bf16", 66, 8.0, 1024), (16, 1, 64, "fp16", 66, 4.0, 1024)):
        lens = [sh * 16 + 3 + 37 * i for i in range(20)] + [sh * 8, 0, 3]
        lm, q, kc, vc, own, shared, o = check_step(lens, sh, hq, hk, d, dt, 16, seed=7, mul=mul, most=most)
        for b in (0, 7, 19, 20, 22):
            o1 = torch.zeros(1, hq, d, dtype=q.dtype, device="cuda")
            lm.step_q4(q[b:b + 1], kc, vc, i32(own[b:b + 1]), i32(lens[b:b + 1]), o1, shared_table=i32(shared))
            assert torch.equal(o1[0], o[b])
        back = list(range(len(lens)))[::-1]
        o2 = torch.zeros(o.shape, dtype=o.dtype, device="cuda")
        lm.step_q4(q[back], kc, vc, i32([own[b] for b in back]), i32([lens[b] for b in back]), o2,
                   shared_table=i32(shared))
        assert torch.equal(o2, o[back])


def test_step_many_requests():
    rng = random.Random(1)
    check_step([rng.choice([0, 1, 7, 90]) for _ in range(600)], 0, 2, 1, 64, "bf16", 16)
    check_step([32 + rng.choice([0, 1, 7, 90]) for _ in range(1500)], 2, 2, 1, 64, "fp16", 16)
    check_step([96 + rng.choice([-96, -50, 0, 1, 7, 90]) for _ in range(4096)], 6, 3, 1, 64, "bf16", 16)
    check_step([400 + rng.choice([-400, -50, 0, 1, 7, 90]) for _ in range(1000)], 25, 12, 1, 128, "bf16", 16)
    check_step([40, 700, 3], 0, 8, 2, 128, "bf16", 16, most=4096)


@pytest.mark.parametrize("most", [3, 4096])      # every request reads the shared part, or it is worked on for all
def test_step_what_is_not_finite_reaches_its_own_rows(most):
    """A NaN in a request's own key makes its results NaN, one in a value its
    group's columns; one in the shared part reaches those who see it."""
    hq, hk, d, bs, sh = 4, 2, 128, 16, 12
    lens = [300, 50, 200]
    kc, vc, tables, shared, n_blocks, width = cache_q4(8, lens, hk, d, bs, sh)
    q = torch.randn(3, hq, d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(8)).bfloat16()
    lm = C.Lm(hq, hk, d, block_size=bs, n_blocks=n_blocks, table_blocks=width, max_requests=most, max_rows=8)

    def run():
        o = torch.zeros_like(q)
        lm.step_q4(q, kc, vc, i32(tables), i32(lens), o, shared_table=i32(shared))
        return o

    want = run()
    at = tables[0][14] * bs + 5                     # position 229 of request 0
    x = torch.randn(1, hk, d, device="cuda")
    y = x.clone()
    y[0, 1, 70] = INF                               # group 2 of head 1
    lm.store_q4(x, y, i32([at]), kc, vc)
    got = run()
    assert torch.equal(got[1:], want[1:])
    bad = got[0].isnan()
    assert bad[2:, 64:96].all() and bad.sum() == 2 * 32
    lm.store_q4(x, x, i32([at]), kc, vc)
    want = run()
    x[0, 0, 3] = NAN
    lm.store_q4(x, torch.ones_like(x), i32([at]), kc, vc)
    got = run()
    assert torch.equal(got[1:], want[1:]) and got[0, :2].isnan().all() and not got[0, 2:].isnan().any()
    lm.store_q4(y, y, i32([at]), kc, vc)
    y[0, 1, 70] = 1.0
    lm.store_q4(y, y, i32([at]), kc, vc)
    place, want = i32([shared[5] * bs + 1]), run()              # position 81: behind request 1's end
    lm.store_q4(x, torch.ones_like(x), place, kc, vc)
    got = run()
    assert torch.equal(got[1], want[1]) and got[::2, :2].isnan().all() and not got[::2, 2:].isnan().any()
    x[0, 0, 3], y[0, 0, 100] = 1.0, -INF                        # group 3 of head 0
    lm.store_q4(x, y, place, kc, vc)
    bad = run().isnan()
    assert torch.equal(run()[1], want[1]) and bad[::2, :2, 96:].all() and bad.sum() == 2 * 2 * 32
    assert lm.errors() == 0


def test_step_bad_blocks_read_as_zeros():
    """A table entry out of range: score 0 and value 0 for its positions, and the bit."""
    for hq, hk, d, bs, lens in ((4, 2, 64, 16, [50, 20]), (4, 2, 128, 128, [400, 20])):
        kc, vc, tables, _, n_blocks, width = cache_q4(9, lens, hk, d, bs)
        q = torch.randn(2, hq, d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(9)).bfloat16()
        lm = C.Lm(hq, hk, d, block_size=bs, n_blocks=n_blocks, table_blocks=width, max_requests=2, max_rows=2)
        outs = []
        for bad in (-1, n_blocks, 2 ** 31 - 1, -2 ** 31):
            wrong = [list(t) for t in tables]
            wrong[0][1] = bad
            outs.append(torch.zeros_like(q))
            lm.step_q4(q, kc, vc, i32(wrong), i32(lens), outs[-1])
            assert lm.errors() == C.LM_ERR_BLOCK
        kc[tables[0][1]], vc[tables[0][1]] = 0, 0
        want = torch.zeros_like(q)
        lm.step_q4(q, kc, vc, i32(tables), i32(lens), want)
        assert lm.errors() == 0 and all(torch.equal(o, want) for o in outs)


@pytest.mark.parametrize("most", [2, 4096])
def test_step_bad_shared_blocks_read_as_zeros(most):
    hq, hk, d, bs, lens = 8, 2, 64, 32, [300, 200]
    kc, vc, tables, shared, n_blocks, width = cache_q4(12, lens, hk, d, bs, 6)
    q = torch.randn(2, hq, d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(9)).bfloat16()
    lm = C.Lm(hq, hk, d, block_size=bs, n_blocks=n_blocks, table_blocks=width, max_requests=most, max_rows=2)
    o, want = torch.zeros_like(q), torch.zeros_like(q)
    for bad in (-1, n_blocks, 2 ** 31 - 1):
        lm.step_q4(q, kc, vc, i32(tables), i32(lens), o, shared_table=i32(shared[:3] + [bad] + shared[4:]))
        assert lm.errors() == C.LM_ERR_BLOCK
    kc[shared[3]], vc[shared[3]] = 0, 0
    lm.step_q4(q, kc, vc, i32(tables), i32(lens), want, shared_table=i32(shared))
    assert lm.errors() == 0 and torch.equal(o, want)


def test_step_behind_more_than_is_worked_on_for_all():
    """A shared part of more positions than the workspace holds: the rest is read
    by every request."""
    hq, hk, d, bs, sh = 2, 1, 64, 128, 32768 // 128 + 3
    check_step([sh * bs + 5, sh * bs + 300, 33000, 20000, 0], sh, hq, hk, d, "bf16", bs, seed=13, most=64)


def test_step_lengths_past_the_table_are_bent():
    kc, vc, tables, _, n_blocks, width = cache_q4(3, [64], 2, 64, 16)
    tables[0][4] = tables[0][0]
    q = torch.randn(1, 4, 64, device="cuda").bfloat16()
    lm = C.Lm(4, 2, 64, n_blocks=n_blocks, table_blocks=width, max_requests=1, max_rows=1)
    o, want = torch.zeros_like(q), torch.zeros_like(q)
    lm.step_q4(q, kc, vc, i32(tables), i32([width * 16]), want)
    assert lm.errors() == 0
    for n in (width * 16 + 1, 2 ** 31 - 1):
        lm.step_q4(q, kc, vc, i32(tables), i32([n]), o)
        assert lm.errors() == C.LM_ERR_LENGTH and torch.equal(o, want)
    lm.step_q4(q, kc, vc, i32(tables), i32([-5]), o)
    assert lm.errors() == C.LM_ERR_LENGTH and not o.any()


def test_step_graph_follows_the_lengths():
    hq, hk, d, bs, sh, B = 8, 2, 128, 16, 70, 5
    lens = [1300, 1500, 1800, 1200, 2400]
    kc, vc, tables, shared, n_blocks, width = cache_q4(10, lens, hk, d, bs, sh)
    q = torch.randn(B, hq, d, device="cuda").bfloat16()
    make = lambda: C.Lm(hq, hk, d, block_size=bs, n_blocks=n_blocks, table_blocks=width, max_requests=B, max_rows=B)
    lm, eager = make(), make()
    kv, t, st, o = i32(lens), i32(tables), i32(shared), torch.zeros_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lm.step_q4(q, kc, vc, t, kv, o, shared_table=st)
        lm.step_q4(q, kc, vc, t, kv, o, shared_table=st)
    for now in (lens, [1, 0, 1800, 1120, 1121], [0] * 5, [5, 1119, 1300, 16, 2400]):
        kv.copy_(i32(now))
        want = torch.full_like(o, 3.0)
        now = [min(n, m) for n, m in zip(now, lens)]
        kv.copy_(i32(now))
        eager.step_q4(q, kc, vc, t, kv, want, shared_table=st)
        o.fill_(4.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want) and lm.errors() == 0 == eager.errors()
        assert not o.isnan().any()


@pytest.mark.parametrize("most,sh", [(256, 0), (256, 40), (2048, 40)])
def test_step_waits_are_bounded(most, sh):
    """With one warp waiting for nothing the call stops, reports it, and is right again."""
    lens = [900, 300, 1500, 1200]
    lm, q, kc, vc, own, shared, o = check_step(lens, sh, 8, 2, 128, "bf16", 16, seed=11, most=most)
    lm.set_unarrived_wait(2000)
    lm.step_q4(q, kc, vc, i32(own), i32(lens), torch.zeros(o.shape, dtype=o.dtype, device="cuda"),
               shared_table=i32(shared) if sh else None)
    assert lm.errors() == C.LM_ERR_TIMEOUT
    lm.set_unarrived_wait(0)
    o2 = torch.zeros(o.shape, dtype=o.dtype, device="cuda")
    lm.step_q4(q, kc, vc, i32(own), i32(lens), o2, shared_table=i32(shared) if sh else None)
    assert lm.errors() == 0 and torch.equal(o2, o)


@pytest.mark.parametrize("most", [6, 4096])
def test_two_objects_at_once(most):
    """Objects of their own on streams of their own, calls behind one another on each."""
    hq, hk, d, bs, sh, lens = 8, 2, 128, 16, 40, [700, 640, 900, 1500, 0, 641]
    lm, q, kc, vc, own, shared, want = check_step(lens, sh, hq, hk, d, "bf16", bs, seed=4, most=most)
    n, width = kc.shape[0], len(own[0])
    lms = [C.Lm(hq, hk, d, block_size=bs, n_blocks=n, table_blocks=width, max_requests=most, max_rows=8) for _ in range(3)]
    streams = [torch.cuda.Stream() for _ in lms]
    outs = [[torch.zeros(want.shape, dtype=q.dtype, device="cuda") for _ in range(20)] for _ in lms]
    x, rows = logits(2, 24, 30001, "bf16"), 24
    sums, ended = torch.zeros(rows, device="cuda"), i32([0] * rows)
    picks = [[[torch.zeros(rows, device="cuda"), *(i32([0] * rows) for _ in range(3))] for _ in range(20)] for _ in lms]
    own, lens, shared = i32(own), i32(lens), i32(shared)
    big = [C.Lm(1, 1, 64, max_requests=rows) for _ in lms]
    torch.cuda.synchronize()
    for turn in range(20):
        for i, s in enumerate(streams):
            lms[i].step_q4(q, kc, vc, own, lens, outs[i][turn], shared_table=shared, stream=s)
            big[i].beams(x, 8, sums, ended, 1, *picks[i][turn], stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for of in outs for o in of)
    assert all(torch.equal(a, b) for of in picks for got in of for a, b in zip(got, picks[0][0]))
    assert picks[0][0][1].tolist() == Q.beams(f64(x), 8, np.zeros(rows), [0] * rows, 1)["parents"]
    assert all(l.errors() == 0 for l in lms + big)


def test_streams_and_cache_beyond_32_bits():
    """Bytes past 2^32 of a cache, on a stream of its own behind its work."""
    hq, hk, d, bs = 8, 8, 128, 128
    n_blocks = 2 ** 32 // (bs * hk * d * 5 // 8) + 40
    kc, vc = (torch.empty(n_blocks, hk, bs * d * 5 // 8, dtype=torch.uint8, device="cuda") for _ in range(2))
    kc[:8], vc[:8] = 255, 255                   # where a wrapped offset would read
    ids, lens = [n_blocks - 1, n_blocks - 30, n_blocks - 2], [384, 200]
    lm = C.Lm(hq, hk, d, block_size=bs, n_blocks=n_blocks, table_blocks=3, max_requests=2, max_rows=384)
    gen = torch.Generator(device="cuda").manual_seed(4)
    k, v = (torch.randn(384, hk, d, generator=gen, device="cuda") for _ in range(2))
    slots = i32([ids[p // bs] * bs + p % bs for p in range(384)])
    q = torch.randn(2, hq, d, generator=gen, device="cuda").bfloat16()
    o, kd, vd = torch.zeros_like(q), *(torch.zeros(3, bs, hk, d, dtype=q.dtype, device="cuda") for _ in range(2))
    tables, kv, src, dst = i32([ids, ids]), i32(lens), i32(ids), i32([0, 1, 2])
    side, late = torch.cuda.Stream(), torch.zeros_like(k)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(10_000_000)
        late.copy_(k)
        lm.store_q4(late, v, slots, kc, vc)
        lm.step_q4(q, kc, vc, tables, kv, o)
    lm.load_q4(kc, vc, src, dst, kd, vd, stream=side)
    side.synchronize()
    small = [c[ids].clone() for c in (kc, vc)]
    y = Q.values(small[0].cpu().numpy(), bs, d, True)
    assert np.array_equal(y.reshape(384, hk, d), Q.decoded(k.cpu().numpy())) and lm.errors() == 0
    assert torch.equal(kd, torch.from_numpy(y).float().bfloat16().cuda())
    ref = step_reference(q, *small, [[0, 1, 2]] * 2, lens, [], hk, d, bs)
    Q.assert_step(o, None, ref, "bf16", d, 6.0)


# ---- forks, compaction, copies ----------------------------------------------

def fork_case(seed, B, bs, sh, width, free, bad=False):
    """Rows that share full blocks from the front, as forks leave them."""
    rng = random.Random(seed)
    lens, tables, ids = [], [[-7] * width for _ in range(B)], sh
    names = list(range(sh))
    for b in range(B):
        n = rng.choice([0, rng.randrange(width * bs + 1), bs * rng.randrange(width + 1), rng.randrange(width * bs + 1)])
        lens.append(n)
        blocks = -(-n // bs)
        tables[b][:min(sh, blocks)] = names[:min(sh, blocks)]
        keep = 0
        if b and rng.random() < 0.6:
            o = rng.randrange(b)
            keep = max(0, min(n // bs, lens[o] // bs) - sh)
            keep = rng.randrange(keep + 1)
            tables[b][sh:sh + keep] = tables[o][sh:sh + keep]
        for j in range(sh + keep, blocks):
            tables[b][j] = ids
            ids += 1
    n = ids + free
    owners = [-1] * n
    for b in range(B):
        for j in range(sh, -(-lens[b] // bs)):
            owners[tables[b][j]] += 1
    owners = [max(0, c) for c in owners]
    perm = list(range(n))
    rng.shuffle(perm)
    tables = [[perm[x] if x >= 0 else x for x in t] for t in tables]
    moved = [0] * n
    for i, c in enumerate(owners):
        moved[perm[i]] = c
    head = rng.randrange(10 * n + 1)
    ring = [-9] * n
    for i in range(free):
        ring[(head + i) % n] = perm[ids + i]
    parents = [rng.choice([-1, rng.randrange(B), rng.randrange(max(1, B // 3))]) for _ in range(B)]
    if bad:
        for i in range(0, B, 5):
            parents[i] = rng.choice([B, -2, 2 ** 31 - 1, -2 ** 31])
        for i in range(2, B, 6):
            lens[i] = rng.choice([-1, width * bs + 1, 2 ** 31 - 1, -2 ** 31])
    return parents, lens, tables, moved, ring, (head, head + free), perm[:sh], n


def run_fork(lm, parents, lens, tables, owners, ring, free, sh, width):
    B, n = len(parents), len(owners)
    t = dict(tables_out=i32([[-3] * width] * B), owners_out=i32([-3] * n), free_list=i32(ring),
             free_out=torch.zeros(2, dtype=torch.int64, device="cuda"), kv_out=i32([-3] * B), status=i32([-3] * B),
             copy_src=i32([-3] * B), copy_dst=i32([-3] * B), copies=i32([-3]))
    free_in = torch.tensor(free, dtype=torch.int64, device="cuda")
    for _ in range(2):          # a repeated call writes the same
        lm.fork(i32(parents), i32(lens), i32(tables), t["tables_out"], i32(owners), t["owners_out"], t["free_list"],
                free_in, t["free_out"], t["kv_out"], t["status"], t["copy_src"], t["copy_dst"], t["copies"],
                shared_blocks=sh)
    return {k: v.tolist() for k, v in t.items()}


def same(got, want):
    for k in want:
        if k.startswith("copy_"):
            assert got[k][:len(want[k])] == want[k] and all(x == -3 for x in got[k][len(want[k]):]), k
        else:
            assert got[k] == want[k], k


@pytest.mark.parametrize("seed,B,bs,sh,width,free,bad", [
    (0, 1, 16, 0, 4, 3, False), (1, 8, 16, 0, 9, 20, False), (2, 40, 32, 2, 30, 60, False), (3, 40, 16, 0, 12, 5, False),
    (4, 300, 128, 1, 7, 400, True), (5, 1500, 64, 0, 5, 900, True), (6, 33, 16, 6, 6, 0, False),
    (7, 512, 16, 3, 90, 600, False), (8, 4096, 16, 0, 3, 5000, False),
])
def test_fork(seed, B, bs, sh, width, free, bad):
    parents, lens, tables, owners, ring, fr, shared, n = fork_case(seed, B, bs, sh, width, free, bad)
    lm = C.Lm(2, 2, 64, block_size=bs, n_blocks=n, table_blocks=width, max_requests=B, max_rows=8)
    got = run_fork(lm, parents, lens, tables, owners, ring, fr, sh, width)
    same(got, Q.fork(parents, lens, tables, [[-3] * width] * B, owners, ring, fr, bs, sh))
    wrong = any(0 <= p < B and not 0 <= lens[p] <= width * bs for p in parents)
    assert lm.errors() == (C.LM_ERR_LENGTH if wrong else 0)


def test_fork_wrong_counts_and_blocks():
    lm = C.Lm(2, 2, 64, n_blocks=8, table_blocks=4, max_requests=2, max_rows=40)
    tables, owners = [[0, 1, -1, -1], [2, -1, -1, -1]], [0] * 8
    for free in [(5, 3), (-1, 2), (0, 9)]:       # nothing is taken or given back
        got = run_fork(lm, [0, 0], [20, 5], tables, owners, list(range(8)), free, 0, 4)
        assert got["status"] == [0, 1] and got["free_out"] == list(free) and lm.errors() == C.LM_ERR_FREE
        same(got, Q.fork([0, 0], [20, 5], tables, [[-3] * 4] * 2, owners, list(range(8)), free, 16, 0))
    # two rows hold block 0, and its count says one
    both = [[0, 1, -1, -1], [0, 3, -1, -1]]
    got = run_fork(lm, [-1, -1], [32, 32], both, owners, [4, 5, 6, 7, 2, 0, 0, 0], (0, 5), 0, 4)
    assert lm.errors() == C.LM_ERR_OWNERS and got["free_list"][5:] == [0, 1, 3] and got["free_out"] == [0, 8]
    got = run_fork(lm, [-1, 1], [32, 20], [[9, -1, -1, -1], [2, 3, -1, -1]], owners, [4, 5, 6, 7, 1, 0, 0, 0], (0, 5), 0, 4)
    assert lm.errors() == C.LM_ERR_BLOCK and got["free_out"] == [0, 5] and got["tables_out"][1] == [2, 3, -3, -3]


@pytest.mark.parametrize("seed,B,bs,sh,width,free", [(0, 1, 16, 0, 4, 3), (1, 8, 16, 2, 9, 20), (2, 40, 32, 0, 30, 600),
                                                     (3, 300, 128, 1, 7, 1), (4, 700, 16, 3, 60, 9000), (5, 9, 16, 0, 5, 0)])
def test_compact(seed, B, bs, sh, width, free):
    _, lens, tables, owners, ring, fr, shared, n = fork_case(seed, B, bs, sh, width, free)
    lm = C.Lm(2, 2, 64, block_size=bs, n_blocks=n, table_blocks=width, max_requests=B, max_rows=8)
    t = dict(tables_out=i32([[-3] * width] * B), shared_out=i32([-3] * sh), owners_out=i32([-3] * n), free_list=i32(ring),
             free_out=torch.zeros(2, dtype=torch.int64, device="cuda"), copy_src=i32([-3] * (n // 2)),
             copy_dst=i32([-3] * (n // 2)), copies=i32([-3]))
    for counted in (True, False, True):
        lm.compact(i32(lens), i32(tables), t["tables_out"], i32(owners) if counted else None,
                   t["owners_out"] if counted else None, t["free_list"], t["free_out"], t["copy_src"], t["copy_dst"],
                   t["copies"], shared_table=i32(shared) if sh else None, shared_out=t["shared_out"] if sh else None)
    assert lm.errors() == 0
    same({k: v.tolist() for k, v in t.items()}, Q.compact(lens, tables, [[-3] * width] * B, shared, owners, ring, bs))


def test_one_block():
    lm = C.Lm(2, 2, 64, n_blocks=1, table_blocks=1, max_requests=2, max_rows=8)
    got = run_fork(lm, [0, 0], [5, 0], [[0], [-1]], [0], [0], (1, 1), 0, 1)       # no block for the copy
    same(got, Q.fork([0, 0], [5, 0], [[0], [-1]], [[-3]] * 2, [0], [0], (1, 1), 16, 0))
    got = run_fork(lm, [1, -1], [5, 0], [[0], [-1]], [0], [0], (1, 1), 0, 1)      # it is given back
    same(got, Q.fork([1, -1], [5, 0], [[0], [-1]], [[-3]] * 2, [0], [0], (1, 1), 16, 0))
    assert got["free_out"] == [1, 2] and got["free_list"] == [0]
    none, t = i32([]), [i32([[-3]] * 2), i32([-3]), i32([0]), torch.zeros(2, dtype=torch.int64, device="cuda")]
    for lens, want in (([16, 0], [0, 0]), ([0, 0], [0, 1])):
        count = i32([-3])
        lm.compact(i32(lens), i32([[0], [-1]]), t[0], i32([0]), t[1], t[2], t[3], none, none.clone(), count)
        assert t[3].tolist() == want and count.item() == 0 and t[1].item() == 0
    assert t[0].tolist() == [[0], [-3]] and lm.errors() == 0


def test_compact_wrong_blocks_and_lengths():
    n, width = 9, 3
    lm = C.Lm(2, 2, 64, n_blocks=n, table_blocks=width, max_requests=3, max_rows=8)
    lens, tables = [40, 10 ** 9, -4], [[7, 9, -1], [8, 2 ** 31 - 1, 3], [5, 5, 5]]
    t = [i32([[-3] * width] * 3), i32(list(range(n))), torch.zeros(2, dtype=torch.int64, device="cuda"), i32([-3] * 4),
         i32([-3] * 4), i32([-3])]
    lm.compact(i32(lens), i32(tables), t[0], None, None, *t[1:])
    assert lm.errors() == C.LM_ERR_BLOCK | C.LM_ERR_LENGTH
    same(dict(zip(("tables_out", "free_list", "free_out", "copy_src", "copy_dst", "copies"), [x.tolist() for x in t])),
         {k: v for k, v in Q.compact(lens, tables, [[-3] * width] * 3, [], [0] * n, list(range(n)), 16).items()
          if k not in ("owners_out", "shared_out")})


@pytest.mark.parametrize("n,blocks,shape,dt,caches", [
    (1, 3, (16, 1, 64), "bf16", 1), (5, 40, (2, 640), "u8", 3), (200, 500, (16, 2, 64), "fp16", 2), (7, 20, (4,), "i32", 256),
    (90, 300, (128, 8, 128), "bf16", 2), (3, 9, (3, 16), "u8", 2)])
def test_copy_blocks(n, blocks, shape, dt, caches):
    kind = {"bf16": torch.bfloat16, "fp16": torch.float16, "u8": torch.uint8, "i32": torch.int32}[dt]
    gen = torch.Generator(device="cuda").manual_seed(n)
    all_of = [torch.randint(0, 200, (blocks, *shape), generator=gen, device="cuda").to(kind) for _ in range(caches)]
    perm = torch.randperm(blocks, generator=gen, device="cuda").int()
    src, dst = perm[:n].clone(), perm[n:2 * n].clone()
    lm = C.Lm(1, 1, 64, n_blocks=blocks)
    for count in (0, n // 2, n, n + 5, -3, None):
        want = [c.clone() for c in all_of]
        m = n if count is None else min(max(count, 0), n)
        for c in want:
            c[dst[:m].long()] = c[src[:m].long()]
        lm.copy_blocks(all_of, src, dst, None if count is None else i32([count]))
        assert all(torch.equal(a, b) for a, b in zip(all_of, want)) and lm.errors() == 0
    want = [c.clone() for c in all_of]
    for c in want:
        c[dst[1:-1].long()] = c[src[1:-1].long()]
    src[0], dst[-1] = blocks, -1
    lm.copy_blocks(all_of, src, dst)
    assert lm.errors() == C.LM_ERR_BLOCK
    assert all(torch.equal(a, b) for a, b in zip(all_of, want))


# ---- beams ------------------------------------------------------------------

def check_beams(x, k, sums, ended, end, most=None):
    """x: logits on the GPU; sums may be off by the result's rounding and 2e-6."""
    rows = x.shape[0]
    lm = C.Lm(1, 1, 64, max_requests=most or rows)
    out = [torch.full((rows,), 9.0, device="cuda"), *(i32([9] * rows) for _ in range(3))]
    lm.beams(x, k, gpu(np.asarray(sums, np.float32)), i32(ended), end, *out)
    want = Q.beams(f64(x), k, np.asarray(sums, np.float32), ended, end)
    got = [t.tolist() for t in out]
    assert got[1] == want["parents"] and got[2] == want["tokens"] and got[3] == want["ended_out"]
    s = np.array(want["sums_out"])
    none = np.isinf(s)
    off = np.abs(np.where(none, 0, got[0]) - np.where(none, 0, s))
    assert np.array_equal(np.isinf(got[0]), none) and (off <= np.abs(np.where(none, 0, s)) * 2.0 ** -24 + 2e-6).all()
    assert lm.errors() == 0
    return got


def logits(seed, rows, vocab, dt, spread=2.5, pad=0, at=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    flat = torch.empty(rows * (vocab + pad) + at + 1, dtype=T[dt], device="cuda").normal_(generator=gen).mul_(spread)
    return flat[at:at + rows * (vocab + pad)].view(rows, vocab + pad)[:, :vocab]


@pytest.mark.parametrize("groups,k,vocab,dt,pad,at", [
    (1, 1, 2, "fp32", 0, 0), (3, 2, 5, "bf16", 3, 1), (2, 4, 33, "fp16", 0, 0), (4, 4, 2048, "fp32", 0, 0),
    (3, 8, 2047, "bf16", 0, 0), (2, 32, 1025, "fp16", 7, 3), (1, 32, 70001, "bf16", 0, 0), (5, 5, 4099, "fp32", 1, 1),
    (70, 4, 513, "bf16", 0, 0), (1, 1, 1000003, "fp32", 1, 1), (128, 32, 40, "fp16", 0, 0),
    (40, 32, 3001, "bf16", 1, 0), (2, 3, 131072, "fp16", 0, 0), (1, 17, 9000, "fp32", 0, 0), (1, 4, 1000003, "bf16", 0, 0),
])
def test_beams(groups, k, vocab, dt, pad, at):
    rows = groups * k
    rng = np.random.default_rng(rows)
    x = logits(rows, rows, vocab, dt, pad=pad, at=at)
    sums = -20 - 4 * np.abs(rng.normal(size=rows))
    check_beams(x, k, sums, [0] * rows, vocab - 1)
    check_beams(x, k, sums, (rng.random(rows) < 0.4).astype(int).tolist(), int(x[0].argmax()), most=4096)
    first = np.where(np.arange(rows) % k == 0, 0.0, -np.inf)
    check_beams(x, k, first, [0] * rows, 0)


@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
def test_beams_ties_go_to_the_lowest(dt):
    """Few different logits; whole rows alike; all alike; ties across the parts of a row."""
    for seed, (k, vocab) in enumerate([(4, 50), (8, 3000), (32, 40), (5, 9001)]):
        x = (logits(seed, 2 * k, vocab, dt) / 2).round()
        check_beams(x, k, -np.arange(2 * k) / 3.0, [0] * (2 * k), 3)
        x[1] = x[0]
        check_beams(x, k, [0.0] * (2 * k), [0] * (2 * k), 3)
        check_beams(torch.zeros_like(x), k, [-1.0] * (2 * k), [0] * (2 * k), -1)
        check_beams(torch.full_like(x, -3.0), k, [-1.0] * (2 * k), [1] * k + [0] * k, 7)


@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
def test_beams_masked_by_the_lowest_value(dt):
    """The type's lowest value, and others far from zero, in places, in whole rows, in
    whole stretches of a row; zeros of both signs are equal."""
    k, vocab = 4, 9001
    low = torch.finfo(T[dt]).min
    x = logits(8, 4 * k, vocab, dt)
    x[0], x[1, 3:], x[2, ::2], x[3, 4000:] = low, low, low, low
    for b, far in enumerate([-1e9, -3e10, 1e10, 1e30]):
        far = max(min(far, 6e4), -6e4) if dt == "fp16" else far
        x[4 + b, 20:7000] = far
        x[8 + b] = far
        x[8 + b, 5 + b] = far + abs(far) / 16
    x[12:] = 0.0
    x[12:, ::3] = -0.0
    sums = -np.arange(4 * k) / 7.0
    check_beams(x, k, sums, [0] * (4 * k), 3)
    check_beams(x, k, [0.0] * (4 * k), [0] * (4 * k), 3, most=4096)


def test_beams_infinities_and_nan():
    k, vocab = 4, 3001
    x = logits(5, 3 * k, vocab, "fp32")
    x[0, :] = -INF                      # nothing
    x[1, 7:] = -INF                     # seven tokens
    x[2, 5] = NAN
    x[3, 9] = INF
    x[4:8] = -INF                       # a group with two candidates
    x[5, 2990], x[6, 0] = -5.0, 80.0
    x[8:, 100:] = -INF
    sums = [-1.0] * (3 * k)
    sums[9], sums[10] = NAN, -INF
    got = check_beams(x, k, sums, [0] * (3 * k), 2)
    assert got[1][4:8] == [5, 6, -1, -1] and got[2][6:8] == [-1, -1] and got[3][6:8] == [1, 1]
    got = check_beams(x, k, sums, [0, 0, 0, 0, 1, 0, 0, 1, 0, 1, 1, 0], 2)
    assert set(got[1][:4]) == {1} and sorted(got[1][4:8]) == [4, 5, 6, 7]
    check_beams(x.bfloat16(), k, sums, [0] * (3 * k), 2)


def test_beams_that_lie_closer_than_32_bits_tell():
    """Two beams whose next sums differ by 1e-7 or so, both ways: the order is
    that of 64 bits."""
    k, vocab = 2, 5000
    rng = np.random.default_rng(0)
    for trial in range(40):
        x = torch.from_numpy(rng.normal(size=(k, vocab)) * 2).float()
        x[:, 17] = 14.0                                     # the best of both by far
        for _ in range(4):                                  # logit of beam 1 that brings the two together, in fp32
            lse = torch.logsumexp(x.double(), 1)
            x[1, 17] = float(14.0 - lse[0] + lse[1] + rng.choice([-1, 1]) * rng.uniform(0, 1e-7))
        check_beams(x.cuda(), k, [0.0, 0.0], [0, 0], 3)
        check_beams(x.flip(0).cuda(), k, [0.0, 0.0], [0, 0], 3)


def test_beams_in_a_graph():
    k, rows = 4, 24
    x, lm = logits(3, rows, 5001, "bf16"), C.Lm(1, 1, 64, max_requests=rows)
    sums, ended = torch.zeros(rows, device="cuda"), i32([0] * rows)
    out = [torch.zeros(rows, device="cuda"), *(i32([0] * rows) for _ in range(3))]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lm.beams(x, k, sums, ended, 5, *out)
    for turn in range(4):
        x.copy_(logits(turn, rows, 5001, "bf16"))
        sums.copy_(-torch.rand(rows, device="cuda"))
        ended.copy_(torch.rand(rows, device="cuda") < 0.2)
        graph.replay()
        torch.cuda.synchronize()
        want = Q.beams(f64(x), k, sums.cpu().numpy(), ended.tolist(), 5)
        assert out[1].tolist() == want["parents"] and out[2].tolist() == want["tokens"]


# ---- together ---------------------------------------------------------------

def test_beam_search_over_the_cache_in_4_bits():
    """As a server uses them: a voice prompt, one prompt a group behind it, then
    steps of selection, fork, copy, plan, store and attention in one captured
    graph; after each, every row's attention against 64 bits over the keys of its
    own history; at last the blocks are moved together and nothing changes."""
    hq, hk, d, bs, sh, G, k, vocab = 4, 2, 64, 16, 2, 3, 4, 300
    B, width, n_blocks, layers = G * k, 8, 120, 2
    lm = C.Lm(hq, hk, d, "bf16", block_size=bs, n_blocks=n_blocks, table_blocks=width, max_requests=B, max_rows=128)
    gen = torch.Generator(device="cuda").manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    caches = [torch.full((n_blocks, hk, bs * d * 5 // 8), 255, dtype=torch.uint8, device="cuda") for _ in range(2 * layers)]
    z = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    shared = i32([100, 7])
    ids = [i for i in range(n_blocks) if i not in (100, 7)]
    ring = i32(ids + [-1] * (n_blocks - len(ids)))
    free = [torch.tensor([0, len(ids)], device="cuda"), *(torch.zeros(2, dtype=torch.int64, device="cuda") for _ in range(2))]
    tables, owners = [z(B, width), z(B, width)], [z(n_blocks), z(n_blocks)]

    def store(rows, slots):
        kv = [(r(rows, hk, d), r(rows, hk, d)) for _ in range(layers)]
        for l, (a, b) in enumerate(kv):
            lm.store_q4(a, b, slots, caches[2 * l], caches[2 * l + 1])
        return kv

    hist = [[[] for _ in range(layers)] for _ in range(B)]      # per row and layer: each position's parts, as stored

    def remember(rows, kv):
        for l, pair in enumerate(kv):
            coded = [Q.encode(x.cpu().numpy()) for x in pair]
            for i, row in enumerate(rows):
                parts = []
                for c, s, low in coded:
                    parts += [np.repeat(low[i].astype(np.float64), 32, -1),
                              np.repeat(s[i].astype(np.float64), 32, -1) * c[i]]
                for b in row:
                    hist[b][l].append(parts)

    pos = torch.arange(sh * bs, device="cuda")
    slots = (shared.repeat_interleave(bs) * bs + pos % bs).int()
    firsts = list(range(0, B, k))
    remember([firsts] * (sh * bs), store(sh * bs, slots))
    # one prompt for each group, in its first row
    new = [5, 16, 20]
    before = i32([sh * bs if b % k == 0 else 0 for b in range(B)])
    after = i32([sh * bs + new[b // k] if b % k == 0 else 0 for b in range(B)])
    row_start, kv_len, status, slot, at = z(B + 1), z(B), z(B), z(128), z(128)
    lm.plan(before, after, tables[0], ring, free[0], free[1], row_start, kv_len, status, slot, at, shared_table=shared)
    remember([[g * k] for g in range(G) for _ in range(new[g])], store(128, slot))
    sums = torch.full((B,), -INF, device="cuda")
    sums[::k] = 0.0
    ended, tokens, parents, sums2, ended2 = z(B), z(B), z(B), torch.zeros(B, device="cuda"), z(B)
    x, q = torch.zeros(B, vocab, device="cuda"), [torch.zeros(B, hq, d, dtype=torch.bfloat16, device="cuda") for _ in range(layers)]
    kv_in, kv_out, src, dst, count = kv_len.clone(), z(B), z(B), z(B), z(1)
    fk = [torch.zeros(B, hk, d, device="cuda") for _ in range(2 * layers)]
    o = [torch.zeros_like(t) for t in q]
    slot1, at1 = z(B), z(B)

    def step():
        lm.beams(x, k, sums, ended, 3, sums2, parents, tokens, ended2)
        lm.fork(parents, kv_in, tables[0], tables[1], owners[0], owners[1], ring, free[1], free[2], kv_out, status, src,
                dst, count, shared_blocks=sh)
        lm.copy_blocks(caches, src, dst, count)
        after.copy_(torch.where((ended2 == 0) & (kv_out > 0), kv_out + 1, kv_out))
        lm.plan(kv_out, after, tables[1], ring, free[2], free[0], row_start, kv_len, status, slot1, at1, shared_table=shared)
        for l in range(layers):
            lm.store_q4(fk[2 * l], fk[2 * l + 1], slot1, caches[2 * l], caches[2 * l + 1])
            lm.step_q4(q[l], caches[2 * l], caches[2 * l + 1], tables[1], kv_len, o[l], shared_table=shared)
        for a, b in ((sums, sums2), (ended, ended2), (tables[0], tables[1]), (owners[0], owners[1]), (free[1], free[0]),
                     (kv_in, kv_len)):
            a.copy_(b)

    def check(o, l):
        lens = kv_len.tolist()
        assert [len(h[l]) for h in hist] == lens
        ref = Q.step(f64(q[l]), lambda b: [np.stack([p[i] for p in hist[b][l]]) if lens[b] else np.zeros((0, hk, d))
                                           for i in range(4)], hk, d ** -0.5)
        Q.assert_step(o, None, ref, "bf16", d, 6.0)

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    for turn in range(40):
        x.copy_(r(B, vocab) * 2)
        x[:, 3] += 2.5 if turn > 10 else -9.0
        if turn == 30:
            sums[k:2 * k] = -INF                # the second group is given up
        for t in q + fk:
            t.copy_(r(*t.shape))
        want = Q.beams(f64(x), k, sums.cpu().numpy(), ended.tolist(), 3)
        graph.replay()
        torch.cuda.synchronize()
        assert parents.tolist() == want["parents"] and tokens.tolist() == want["tokens"] and lm.errors() == 0
        assert not status.any()
        hist = [[list(h) for h in hist[p]] if p >= 0 else [[] for _ in range(layers)] for p in want["parents"]]
        grown = [b for b in range(B) if want["parents"][b] >= 0 and not want["ended_out"][b]]
        assert row_start[-1] == len(grown)
        remember([[b] for b in grown], [(fk[2 * l][:len(grown)], fk[2 * l + 1][:len(grown)]) for l in range(layers)])
        for l in range(layers):
            check(o[l], l)
        count_of = [0] * n_blocks
        for row, n in zip(tables[0].tolist(), kv_len.tolist()):
            for j in range(sh, -(-n // bs)):
                count_of[row[j]] += 1
        assert owners[0].tolist() == [max(0, c - 1) for c in count_of]
        head, tail = free[0].tolist()
        loose = [ring[i % n_blocks].item() for i in range(head, tail)]
        assert sorted(loose + [i for i, c in enumerate(count_of) if c] + [100, 7]) == list(range(n_blocks))
    moved, so, oo = torch.zeros_like(tables[0]), torch.zeros_like(shared), torch.zeros_like(owners[0])
    src, dst = z(n_blocks // 2), z(n_blocks // 2)
    lm.compact(kv_len, tables[0], moved, owners[0], oo, ring, free[2], src, dst, count, shared_table=shared, shared_out=so)
    lm.copy_blocks(caches, src, dst, count)
    used = n_blocks - free[2][1].item()
    assert count.item() > 0 and max(so.tolist()) < used
    for l in range(layers):
        o2 = torch.zeros_like(o[l])
        lm.step_q4(q[l], caches[2 * l], caches[2 * l + 1], moved, kv_len, o2, shared_table=so)
        assert torch.equal(o2, o[l])
    # a prompt's attention behind the context: back to 16 bits, and its rows there
    b = int(kv_len.argmax())
    n = kv_len[b].item()
    blocks = -(-n // bs)
    kd, vd = (torch.zeros(blocks, bs, hk, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    order = torch.arange(blocks, device="cuda", dtype=torch.int32)
    lm.load_q4(caches[0], caches[1], moved[b, :blocks].contiguous(), order, kd, vd)
    one = C.Lm(hq, hk, d, "bf16", block_size=bs, n_blocks=blocks, table_blocks=blocks, max_requests=1, max_rows=1)
    o3 = torch.zeros(1, hq, d, dtype=torch.bfloat16, device="cuda")
    one.prompt_paged(q[0][b:b + 1], kd, vd, i32([0, 1]), order.view(1, -1), i32([n]), o3)
    # keys rounded to bf16 move a score by sum |q k| 2^-9 / 8 (about 0.1), values by 2^-9
    assert (o3[0].float() - o[0][b].float()).abs().max() < 0.1 and lm.errors() == 0


# ---- refusals ---------------------------------------------------------------

def test_refusals():
    lm = C.Lm(4, 2, 64, block_size=16, n_blocks=4, table_blocks=3, max_requests=2, max_rows=8)
    bf = torch.bfloat16
    k = torch.zeros(8, 2, 64, dtype=bf, device="cuda")
    kc, vc = (torch.zeros(4, 2, 640, dtype=torch.uint8, device="cuda") for _ in range(2))
    slots, tb, kv = i32(list(range(8))), i32([[0] * 3] * 2), i32([8, 8])
    V, E = ValueError, C.CodecError

    def refused(kind, f, *a, **kw):
        with pytest.raises(kind):
            f(*a, **kw)

    refused(V, lm.store_q4, k.half(), k.half(), slots, kc, vc)              # another type
    refused(V, lm.store_q4, k, k.float(), slots, kc, vc)
    refused(V, lm.store_q4, k, k, slots[:4], kc, vc)
    refused(V, lm.store_q4, k, k, slots, kc[:3], vc)
    refused(V, lm.store_q4, k, k, slots, kc.int(), vc)
    refused(V, lm.store_q4, k.cpu(), k, slots, kc, vc)
    refused(E, lm.store_q4, k, k, slots, kc, kc)                            # one cache for both
    nine = torch.zeros(9, 2, 64, dtype=bf, device="cuda")
    refused(E, lm.store_q4, nine, nine, i32([0] * 9), kc, vc)
    odd = torch.zeros(8 * 132 + 8, dtype=bf, device="cuda")
    refused(E, lm.store_q4, odd[:8 * 132].view(8, 132)[:, :128].unflatten(1, (2, 64)), k, slots, kc, vc)    # 264 bytes
    lm.store_q4(k[:0], k[:0], slots[:0], kc, vc)
    kd, vd = (torch.zeros(5, 16, 2, 64, dtype=bf, device="cuda") for _ in range(2))
    refused(V, lm.load_q4, kc, vc, slots[:2], slots[:3], kd, vd)
    refused(V, lm.load_q4, kc, vc, slots[:2], slots[:2], kd, vd[:4])
    refused(V, lm.load_q4, kc, vc, slots[:2], slots[:2], kd.half(), vd.half())
    refused(E, lm.load_q4, kc, vc, slots[:2], slots[:2], kd, kd)
    q = torch.zeros(2, 4, 64, dtype=bf, device="cuda")
    o = torch.zeros_like(q)
    refused(V, lm.step_q4, q, kc, vc.float(), tb, kv, o)
    refused(V, lm.step_q4, q[:1], kc, vc, tb, kv, o[:1])
    refused(V, lm.step_q4, q.float(), kc, vc, tb, kv, o)
    refused(E, lm.step_q4, q, kc, vc, tb, kv, q)
    refused(E, lm.step_q4, q, kc, vc, tb, kv, o, shared_table=i32([0] * 4))
    q3 = torch.zeros(3, 4, 64, dtype=bf, device="cuda")
    refused(E, lm.step_q4, q3, kc, vc, i32([[0] * 3] * 3), i32([1] * 3), torch.zeros_like(q3))
    x, s, e = torch.zeros(2, 9, device="cuda"), torch.zeros(2, device="cuda"), i32([0, 0])
    out = lambda: (torch.zeros(2, device="cuda"), i32([0, 0]), i32([0, 0]), i32([0, 0]))
    refused(V, lm.beams, x.double(), 2, s, e, 1, *out())
    refused(V, lm.beams, x.t().contiguous().t(), 2, s, e, 1, *out())
    refused(V, lm.beams, x, 3, s, e, 1, *out())
    refused(V, lm.beams, x, 0, s, e, 1, *out())
    refused(V, lm.beams, x, 2, s, e.long(), 1, *out())
    refused(E, lm.beams, x, 2, s, e, 9, *out())
    refused(E, lm.beams, x, 2, s, e, -2, *out())
    refused(E, lm.beams, x[:, :1], 2, s, e, 0, *out())
    refused(E, lm.beams, x, 2, s, e, 1, s, *out()[1:])
    refused(E, lm.beams, x, 2, s, e, 1, out()[0], e, *out()[2:])
    refused(E, lm.beams, x, 2, s, e, 1, *out()[:2], *[i32([0, 0])] * 2)
    refused(E, lm.beams, x[:1].expand(2, 9), 2, s, e, 1, *out())            # both rows in one place
    refused(E, lm.beams, torch.zeros(4, 9, device="cuda"), 2, torch.zeros(4, device="cuda"), i32([0] * 4), 1,
            torch.zeros(4, device="cuda"), i32([0] * 4), i32([0] * 4), i32([0] * 4))     # more rows than requests
    f2 = lambda: torch.zeros(2, dtype=torch.int64, device="cuda")
    ow, ring, one = i32([0] * 4), i32([0] * 4), i32([0])
    fork = lambda **kw: lm.fork(**{**dict(parents=i32([0, 0]), kv_len=kv, tables=tb, tables_out=tb.clone(), owners=ow,
                                          owners_out=ow.clone(), free_list=ring, free_in=f2(), free_out=f2(),
                                          kv_out=i32([0, 0]), status=i32([0, 0]), copy_src=i32([0, 0]),
                                          copy_dst=i32([0, 0]), copies=one), **kw})
    fork()
    refused(E, fork, tables_out=tb)
    refused(E, fork, owners_out=ow)
    refused(E, fork, kv_out=kv)
    two = i32([0, 0])
    for pair in (("parents", "status"), ("parents", "copy_src"), ("kv_out", "status"), ("copy_src", "copy_dst"),
                 ("kv_len", "copy_dst")):
        refused(E, fork, **{name: two for name in pair})
    refused(E, fork, owners=ring)
    refused(E, fork, owners_out=ring)
    refused(E, fork, **(lambda t: dict(free_in=t, free_out=t))(f2()))
    refused(E, fork, shared_blocks=4)
    refused(E, fork, shared_blocks=-1)
    refused(V, fork, owners=ow[:3])
    refused(V, fork, copies=i32([0, 0]))
    refused(V, fork, parents=i32([0, 0, 0]))
    comp = lambda **kw: lm.compact(**{**dict(kv_len=kv, tables=tb, tables_out=tb.clone(), owners=ow, owners_out=ow.clone(),
                                             free_list=ring, free_out=f2(), copy_src=i32([0, 0]), copy_dst=i32([0, 0]),
                                             copies=one), **kw})
    comp()
    refused(E, comp, tables_out=tb)
    refused(E, comp, copy_src=two, copy_dst=two)
    refused(E, comp, kv_len=two, copy_dst=two)
    refused(E, comp, owners=ring)
    refused(E, comp, owners=None)
    refused(V, comp, copy_src=i32([0]))
    refused(V, comp, shared_table=i32([1]), shared_out=i32([1, 2]))
    refused(E, comp, **(lambda t: dict(shared_table=t, shared_out=t))(i32([1])))
    refused(V, lm.copy_blocks, [kc, vc[:3]], slots[:1], slots[1:2])
    refused(V, lm.copy_blocks, [kc, torch.zeros(4, 16, device="cuda")], slots[:1], slots[1:2])
    refused(V, lm.copy_blocks, [kc.transpose(1, 2)], slots[:1], slots[1:2])
    refused(E, lm.copy_blocks, [], slots[:1], slots[1:2])
    refused(E, lm.copy_blocks, [kc] * 257, slots[:1], slots[1:2])
    refused(E, lm.copy_blocks, [torch.zeros(4, 2, device="cuda")], slots[:1], slots[1:2])      # 8 bytes
    lm.errors()                         # the tables above share a block
