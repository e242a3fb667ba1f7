"""Corners of the 4-bit cache and of the selection: candidates closer than 32 bits tell
where a list ends, values past fp16's largest, values far below one, parts without
weight, nothing to copy, and what an object allocates."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import lm_q4_ref as Q
from streaming_tts_vocoder_gb300 import codec as C
from test_gpu_lm_q4 import as_halves, cache_q4, check_beams, f64, gpu, i32, step_reference

pytestmark = pytest.mark.gpu
T = Q.DTYPES


# ---- selection --------------------------------------------------------------

def log_sums(x):
    return torch.logsumexp(x.double(), 1).numpy()


def test_beams_one_rows_candidates_at_the_cut():
    """The last one chosen and the first left out are of one row, and another row's
    candidate lies 3e-8 to 2e-7 before or behind them."""
    k, vocab = 3, 5000
    rng = np.random.default_rng(0)
    for trial in range(60):
        x = torch.from_numpy(rng.normal(size=(k, vocab)) * 2).float()
        x[2, 40] = 30.0                                     # first by far
        x[1, [5, 100, 2000, 4000]] = 14.0
        x[0, [17, 1000, 1001, 1002]] = torch.tensor([14.0, 13.5, 13.5, 13.5])
        for _ in range(20):
            lse = log_sums(x)
            x[0, 17] = float(14.0 - lse[1] + lse[0])
        lse = log_sums(x)
        off = rng.choice([-1, 1]) * rng.uniform(3e-8, 2e-7)
        assert abs((14.0 - lse[1]) - (float(x[0, 17]) - lse[0])) < 1e-5
        sums = [np.float32((14.0 - lse[1]) - (float(x[0, 17]) - lse[0]) + off), 0.0, 0.0]
        got = check_beams(x.cuda(), k, sums, [0] * k, 3)
        assert got[1] == ([2, 0, 1] if off > 0 else [2, 1, 1])
        got = check_beams(x.flip(0).cuda(), k, sums[::-1], [0] * k, 3)
        assert got[1] == ([0, 2, 1] if off > 0 else [0, 1, 1])


@pytest.mark.parametrize("dt,vocab", [("fp32", 9001), ("bf16", 9001), ("fp16", 2049), ("fp32", 300)])
@pytest.mark.parametrize("k", [2, 5, 32])
def test_beams_rows_of_one_value(dt, vocab, k):
    """All beams alike, all logits one constant: the first beam's first tokens."""
    for c in np.random.default_rng(vocab + k).normal(size=24) * 4:
        x = torch.full((k, vocab), c, dtype=T[dt], device="cuda")
        got = check_beams(x, k, [0.0] * k, [0] * k, -1)
        assert got[1] == [0] * k and got[2] == list(range(k))


@pytest.mark.parametrize("dt,vocab", [("fp32", 5000), ("bf16", 9001), ("fp32", 301)])
@pytest.mark.parametrize("k", [2, 3, 8])
def test_beams_many_candidates_closer_than_32_bits_tell(dt, vocab, k):
    """Rows of a few different logits whose best are a rounding of the sums apart, some
    of them many times; an ended beam among them."""
    rng = np.random.default_rng(vocab + k)
    groups = 12
    x = torch.from_numpy(rng.integers(-6, 3, size=(groups * k, vocab)) * 0.5).to(T[dt])
    for r in range(groups * k):
        x[r, torch.from_numpy(rng.permutation(vocab)[:rng.integers(1, 5)])] = 9.0
    lse = log_sums(x)
    sums, best = np.zeros(groups * k, np.float32), np.zeros(groups * k)
    for r in rng.permutation(groups * k):               # steps of 32 bits away from the others of its group
        mates = [i for i in range(r // k * k, r // k * k + k) if best[i] != 0.0] + [r // k * k]
        for step in rng.permutation(np.arange(-4, 5)):
            sums[r] = np.float32(lse[r] - 12.0)
            sums[r] += step * np.spacing(sums[r])
            best[r] = float(sums[r]) + 9.0 - lse[r]
            if all(abs(best[r] - best[i]) > 2e-8 for i in mates if i != r):
                break
        else:
            raise AssertionError("no room")
    ended = [0] * (groups * k)
    check_beams(x.cuda(), k, sums, ended, 3)
    ended[k] = 1                                        # itself alone, as near
    sums[k] = next(c for c in np.float32(-3.0) + np.arange(9) * np.spacing(np.float32(3.0))
                   if np.abs(best[k + 1:2 * k] - c).min() > 2e-8)
    check_beams(x.cuda(), k, sums, ended, 3)


@pytest.mark.parametrize("dt,vocab", [("fp32", 9001), ("bf16", 9001), ("fp16", 2049), ("fp32", 300), ("fp32", 130001)])
@pytest.mark.parametrize("k", [2, 5, 32])
def test_beams_rows_of_a_value_each(dt, vocab, k):
    """Rows of a constant of their own, whose roundings are all of one sign, and sums 3e-8
    to 5e-6 apart: the best sum's tokens."""
    rng = np.random.default_rng(vocab + k)
    for trial in range(12):
        x = torch.from_numpy(rng.normal(size=(k, 1)) * 4).to(T[dt]).expand(k, vocab).contiguous().cuda()
        sums = rng.permutation((3e-8 + rng.random() * (5e-6 / k - 3e-8)) * np.arange(1, k + 1)).astype(np.float32)
        got = check_beams(x, k, sums, [0] * k, -1)
        assert got[1] == [int(sums.argmax())] * k and got[2] == list(range(k))


@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
def test_beams_sums_of_zero_of_either_sign(dt):
    """0 and -0 are equal: ended beams, and ones whose one token is certain, in order of beams."""
    k, vocab = 5, 40
    x = torch.full((2 * k, vocab), -float("inf"), dtype=T[dt], device="cuda")
    x[:, 7], x[3, 7], x[8, 7] = 0.0, -0.0, -2.0
    for sums in ([0.0, -0.0, 0.0, -0.0, 0.0, -0.0, 0.0, -0.0, 0.0, -0.0], [-0.0] * 3 + [0.0] * 4 + [-0.0] * 3):
        for ended in ([0, 0, 1, 0, 1, 1, 0, 1, 0, 0], [1] * 10, [0] * 10):
            got = check_beams(x, k, sums, ended, 7)
            assert got[1] == list(range(2 * k))


# ---- store ------------------------------------------------------------------

@pytest.mark.parametrize("hk,d,dt", [(3, 128, "bf16"), (2, 64, "fp16")])
def test_store_groups_past_the_largest_half(hk, d, dt):
    """fp32 groups whose values lie around 65,504 on both sides of it, of either sign,
    and far beyond: to the byte."""
    rows, bs = 60, 16
    rng = np.random.default_rng(d)
    both = []
    for _ in range(2):
        x = rng.uniform(65300, 65503, size=(rows, hk, d // 32, 32))
        x[:, :, :, ::3] = rng.uniform(65504, 66000, size=x[:, :, :, ::3].shape)
        x[::4, :, :, 7] = 10.0 ** rng.uniform(4.9, 38, size=x[::4, :, :, 7].shape)
        x[1::4, :, 0, :31], x[1::4, :, 0, 31] = 65490, 70000
        x[2::4, :, 0, 1:], x[2::4, :, 0, 0] = 65400, 70000
        x[3::4, :, 0, 5] = -7e4
        x[rows // 2:] *= np.where(rng.random((rows - rows // 2, hk, 1, 1)) < 0.5, -1, 1)
        both.append(x.reshape(rows, hk, d).astype(np.float32))
    lm = C.Lm(hk, hk, d, dt, block_size=bs, n_blocks=4, max_rows=rows)
    slots = rng.permutation(4 * bs)[:rows]
    caches = [torch.zeros(4, hk, bs * d * 5 // 8, dtype=torch.uint8, device="cuda") for _ in range(2)]
    lm.store_q4(*(gpu(x) for x in both), i32(slots.tolist()), *caches)
    assert lm.errors() == 0
    for x, c, keys in zip(both, caches, (True, False)):
        want = np.zeros(c.shape, np.uint8)
        Q.store(want, x, slots, bs, keys)
        assert np.array_equal(c.cpu().numpy(), want)


# ---- single tokens ----------------------------------------------------------

def near(got, ref, dt, d, low, scale):
    """Elementwise.  As Q.assert_step, but with what is held in fixed steps relative to the
    values.  A split's largest probability is 2^6 at least, 2^6 / scale where its largest
    step `scale` passes 1, and halves' steps are 2^-24: a probability is off by 2^-31 of the
    largest, twice where it is two halves, times the largest `low`.  Its product with a step
    is taken times the power of two that brings the split's largest below 2 where that lies
    below 2^-6 (2^15 at most), and off by 2^-31 over that, three times (a rounding each of
    the product, of what it leaves off, of their sum), times a code of 15."""
    o, _, al, ac, s, n = ref
    half = torch.finfo(T[dt]).eps / 2
    ds = (4 * d * 2.0 ** -23 * (s + 1))[..., None]
    n = n[:, None, None]
    fine = dt == "fp16"
    tol = half * np.abs(o) * 1.01 + (al * 2.0 ** -11 + ac * 2.0 ** -10) * (2.0 ** -10 if fine else 1.01)
    tol = tol + (al + ac) * (2 * ds + (n / (4 if fine else 8) + 16) * 2.0 ** -23)
    unit = max(scale, 2.0 ** -15) if scale < 2.0 ** -6 else max(scale, 1.0)
    tol = tol + n * 2.0 ** -31 * (2 * low * max(scale, 1.0) + 3 * 15 * unit) + 2.0 ** -25 * fine
    off = np.abs(f64(got) - o) / tol
    worst = off.max()
    assert worst <= 1, f"{worst:.3g} x the bound"


@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("size", [3e-6, 1e-5, 1e-4, 1e-3, 0.03, 1.0, 200.0])
@pytest.mark.parametrize("sh,most", [(0, 1), (60, 2)])
def test_step_values_far_below_one(dt, size, sh, most):
    """One key at the reference and, in the same split, 7,680 to 8,000 that lie 9 nats
    below and weigh as much: values of any size come out as close, relative to them."""
    hk, d, bs, n, width = 2, 64, 128, 8001, 4100         # splits of 8,192 positions
    gen = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    lm = C.Lm(hk, hk, d, dt, block_size=bs, n_blocks=70, table_blocks=width, max_requests=most, max_rows=n)
    kc, vc = (torch.full((70, hk, bs * d * 5 // 8), 255, dtype=torch.uint8, device="cuda") for _ in range(2))
    ids = torch.randperm(70, generator=gen, device="cuda")[:63].int()
    pos = torch.arange(n, device="cuda")
    q = r(1, hk, d).to(T[dt])
    k, v = r(n, hk, d) * 0.02, r(n, hk, d) * size
    k[0] += q[0].float() * (9 * d ** 0.5 / q[0].float().square().sum(-1, keepdim=True))
    lm.store_q4(k, v, (ids[pos // bs] * bs + pos % bs).int(), kc, vc)
    tables, o = torch.full((1, width), -1, dtype=torch.int32, device="cuda"), torch.zeros_like(q)
    tables[0, :63] = ids
    lm.step_q4(q, kc, vc, tables, i32([n]), o, shared_table=ids[:sh].contiguous() if sh else None)
    assert lm.errors() == 0
    ref = step_reference(q, kc, vc, tables.tolist(), [n], ids[:sh].tolist(), hk, d, bs)
    low, rest = (x.reshape(-1, hk, d)[:n] for x in Q.values(vc[ids.long()].cpu().numpy(), bs, d, False, parts=True))
    near(o, ref, dt, d, np.abs(low).max(), rest.max() / 15)


@pytest.mark.parametrize("dt,sh,most", [("bf16", 0, 1), ("fp16", 0, 1), ("fp16", 8, 64), ("bf16", 8, 64), ("bf16", 64, 4096)])
def test_step_nan_of_no_weight_reaches_its_row(dt, sh, most):
    """A group that stands for NaN among keys hundreds of nats below the rest, in the same
    split or in another: 0 times NaN is NaN."""
    hk, d, bs, n = 1, 64, 16, 64 * 16 + 200
    for where, heavy in ((3, 67), (3, 4), (100, 164), (700, 5), (700, 701), (n - 1, 5)):
        lens = [n]
        kc, vc, tables, shared, n_blocks, width = cache_q4(3, lens, hk, d, bs, sh)
        lm = C.Lm(hk, hk, d, dt, block_size=bs, n_blocks=n_blocks, table_blocks=width, max_requests=most, max_rows=n)
        table = i32((shared + tables[0][sh:])[:-(-n // bs)])
        pos = torch.arange(n, device="cuda")
        k = torch.full((n, hk, d), -1.5, device="cuda")
        k[heavy] = 1.5                                      # all the weight: 12 * 64 * 3 / 8 = 288 nats above
        v = torch.randn(n, hk, d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2))
        v[where, 0, 40] = float("nan")                      # group 1
        lm.store_q4(k, v, (table[pos // bs] * bs + pos % bs).int(), kc, vc)
        q, o = torch.full((1, hk, d), 12.0, dtype=T[dt], device="cuda"), torch.zeros(1, hk, d, dtype=T[dt], device="cuda")
        lm.step_q4(q, kc, vc, i32(tables), i32(lens), o, shared_table=i32(shared) if sh else None)
        assert lm.errors() == 0
        assert o[0, 0, 32:].isnan().all() and o[0, 0, :32].isfinite().all(), (where, heavy)


@pytest.mark.parametrize("hq,hk,d,bs,sh,mul", [(8, 2, 128, 16, 66, 1.0), (16, 1, 64, 32, 40, 3.0), (4, 4, 128, 128, 20, 1.0)])
def test_step_long_shared_part_against_its_own_values(hq, hk, d, bs, sh, mul):
    """What a long shared part's halves put off, against the cache's values as they are.
    A key rounded to fp16 moves a score by sum |q| |k| 2^-11 of scale, at most as much of
    which is common to all keys, so a probability by twice that; a value moves by 2^-11."""
    assert as_halves(torch.bfloat16, 4096, hq, hk, sh * bs) == sh * bs
    lens = [sh * bs, sh * bs + 1, sh * bs + 333, sh * bs - 5, 40, 0]
    kc, vc, tables, shared, n_blocks, width = cache_q4(21, lens, hk, d, bs, sh)
    gen = torch.Generator(device="cuda").manual_seed(21)
    q = (torch.randn(len(lens), hq, d, generator=gen, device="cuda") * mul).bfloat16()
    o, lse = torch.zeros_like(q), torch.zeros(len(lens), hq, device="cuda")
    lm = C.Lm(hq, hk, d, "bf16", block_size=bs, n_blocks=n_blocks, table_blocks=width, max_requests=4096, max_rows=8)
    lm.step_q4(q, kc, vc, i32(tables), i32(lens), o, shared_table=i32(shared), lse=lse)
    assert lm.errors() == 0
    ref = step_reference(q, kc, vc, tables, lens, shared, hk, d, bs)            # nothing of it rounded
    want, want_lse, al, ac, s, n = ref
    moved = (s * 2.0 ** -11)[..., None]
    ds = (4 * d * 2.0 ** -23 * (s + 1))[..., None]
    n = n[:, None, None]
    tol = 2.0 ** -9 * np.abs(want) * 1.01 + al * 2.0 ** -11 * 1.01 + ac * 2.0 ** -10 * 1.01
    tol = tol + (al + ac) * (np.exp(2 * (moved + ds)) - 1 + 2.0 ** -11 + (n / 8 + 16) * 2.0 ** -23)
    tol = tol + n * 2.0 ** -31 * (15 + 12.0) * 6.0 + 1e-30
    off = np.abs(f64(o) - want)
    assert (off <= tol).all(), f"{(off / tol).max():.3g} x the bound"
    seen = ~np.isneginf(want_lse)
    far = np.abs(f64(lse) - np.where(seen, want_lse, 0))[seen]
    assert (far <= ((moved + ds)[..., 0] + (np.abs(np.where(seen, want_lse, 0)) + 4) * 2.0 ** -20)[seen]).all()
    # in all: the result's own rounding is 2^-9 / sqrt(3) on average (0.0011); the keys' move a
    # score by 2^-11 / sqrt(3) of the root of the sum of scale^2 (q k)^2, 4 at most (0.0011)
    rel = np.linalg.norm(f64(o) - want) / np.linalg.norm(want)
    assert rel < 2.0 ** -8, rel


# ---- blocks -----------------------------------------------------------------

def test_copy_of_nothing():
    """No entries: nothing is copied, and what a pool of one block's compaction leaves can
    be handed on.  Caches are looked at all the same."""
    lm = C.Lm(2, 2, 64, n_blocks=1, table_blocks=1, max_requests=1, max_rows=8)
    cache = torch.arange(2 * 640, device="cuda").to(torch.uint8).view(1, 2, 640)
    want, none, count = cache.clone(), i32([]), i32([7])
    lm.compact(i32([16]), i32([[0]]), i32([[0]]), None, None, i32([0]), torch.zeros(2, dtype=torch.int64, device="cuda"),
               none, none.clone(), count)
    lm.copy_blocks([cache], none, none.clone(), count)
    lm.copy_blocks([cache, cache.clone()], none, none.clone())
    assert torch.equal(cache, want) and lm.errors() == 0 and count.item() == 0
    with pytest.raises(C.CodecError):
        lm.copy_blocks([], none, none.clone())
    with pytest.raises(ValueError):
        lm.copy_blocks([cache], none, i32([0]))


# ---- objects ----------------------------------------------------------------

def taken(**kw):
    torch.cuda.synchronize()
    before = torch.cuda.mem_get_info()[0]
    lm = C.Lm(8, 8, 128, n_blocks=2, max_rows=8, **kw)
    return before - torch.cuda.mem_get_info()[0], lm


@pytest.mark.parametrize("kw,much", [
    (dict(table_blocks=2048, max_requests=1), False),       # the way is closed to one request
    (dict(table_blocks=200, max_requests=64), False),       # 64 sets of 8 columns x 200 tiles of 16 keys: below 16,384
    (dict(table_blocks=2048, max_requests=64), True),
])
def test_workspace_of_a_long_shared_part(kw, much):
    """An object has room for a long shared part as halves only where its shape can come to
    that: one of bf16 takes what one of fp16 takes, which never does."""
    kw = dict(block_size=16, **kw)
    taken(dtype="fp16", **kw)
    halves, _ = taken(dtype="fp16", **kw)
    wide, _ = taken(dtype="bf16", **kw)
    more = 2 * 2 * min(kw["table_blocks"] * 16, 32768) * 8 * 128
    slack = 4 << 20                     # small arrays share what is handed out at once, 2 MB
    assert abs(wide - halves - (more if much else 0)) <= slack, (wide, halves)
