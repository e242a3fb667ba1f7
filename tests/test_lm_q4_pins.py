"""CPU pins of the 4-bit cache's, the forks' and the beams' references, and what
the library refuses without a device."""
from __future__ import annotations

import random

import numpy as np
import pytest

import lm_q4_ref as Q
from streaming_tts_vocoder_gb300 import build as B
from streaming_tts_vocoder_gb300 import codec as C


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("keys", [True, False])
def test_every_byte_of_a_tile_has_one_use(d, keys):
    code, upper, scale, low = Q.places(d, keys)
    halves = sorted(zip(code.ravel().tolist(), upper.ravel().tolist()))
    assert halves == [(b, h) for b in range(8 * d) for h in (0, 1)]
    pairs = sorted(scale.ravel().tolist() + low.ravel().tolist())
    assert pairs == list(range(8 * d, 10 * d, 2))


def test_a_value_is_off_by_half_a_step():
    rng = np.random.default_rng(0)
    x = (rng.normal(size=(50, 4, 128)) * rng.uniform(1e-3, 1e3, size=(50, 4, 1))).astype(np.float32)
    c, s, l = Q.encode(x)
    y = Q.decoded(x)
    group = lambda t: np.repeat(t.astype(np.float64), 32, -1)
    # half a step; a step more than 15 or a low above the least value: what their roundings (2^-11) moved
    tol = group(s) * (0.5 + 15 * 2.0 ** -11 + 2.0 ** -20) + np.abs(group(l)) * 2.0 ** -11 + 2.0 ** -24
    assert (np.abs(y - x) <= tol).all() and c.max() == 15 and c.min() == 0


def test_groups_that_are_flat_large_or_not_finite():
    x = np.zeros((6, 1, 64), np.float32)
    x[1] = 0.1
    x[2, 0, :32], x[2, 0, 5] = 7e4, -1e9
    x[3, 0, 40] = np.nan
    x[4, 0, 3] = np.inf
    x[5, 0, 1] = 1e-9
    y = Q.decoded(x)
    assert (y[0] == 0).all() and (y[1] == np.float64(np.float16(0.1))).all()
    assert y[2, 0, 5] == -65504 and abs(y[2, 0, 0] - 65504) < 65504 * 2 * 2.0 ** -10
    assert np.isnan(y[3, 0, 32:]).all() and (y[3, 0, :32] == 0).all()
    assert np.isnan(y[4, 0, :32]).all() and (y[4, 0, 32:] == 0).all() and (y[5] == 0).all()


@pytest.mark.parametrize("keys", [True, False])
def test_stored_rows_read_back(keys):
    rng = np.random.default_rng(1)
    x = rng.normal(size=(9, 2, 64)).astype(np.float32)
    cache = np.full((3, 2, 32 * 40), 0xA5, np.uint8)
    slots = [0, 15, 16, 31, 95, 40, -1, 96, 41]
    Q.store(cache, x, slots, 32, keys)
    want = Q.decoded(x)
    got = Q.values(cache, 32, 64, keys).reshape(96, 2, 64)
    for r, slot in enumerate(slots):
        if 0 <= slot < 96:
            assert np.array_equal(got[slot], want[r])


def holders(tables, lens, bs, sh, n):
    count = [0] * n
    for row, x in zip(tables, lens):
        for j in range(sh, -(-x // bs)):
            count[row[j]] += 1
    return count


def test_forks_keep_count_of_who_holds_what():
    """Many forks in a row: owners are what counting the tables finds, no block is
    lost, none is both free and held, and a last, unfilled block has one holder."""
    rng = random.Random(3)
    bs, sh, B, width, n = 4, 1, 6, 9, 40
    ring, free = list(range(1, n)) + [-1], (0, n - 1)
    owners, tables, lens = [0] * n, [[0] * width for _ in range(B)], [0] * B
    for r in range(B):
        lens[r] = rng.randrange(0, 12) + sh * bs
        for j in range(sh, -(-lens[r] // bs)):
            tables[r][j] = ring[free[0]]
            free = (free[0] + 1, free[1])
    for turn in range(60):
        parents = [rng.choice([-1] + list(range(B)) * 2) for _ in range(B)]
        got = Q.fork(parents, lens, tables, [[0] * width for _ in range(B)], owners, ring, free, bs, sh)
        tables, lens, owners, ring = got["tables_out"], got["kv_out"], got["owners_out"], got["free_list"]
        free = tuple(got["free_out"])
        count = holders(tables, lens, bs, sh, n)
        assert owners == [max(0, c - 1) for c in count]
        loose = [ring[i % n] for i in range(*free)]
        assert len(set(loose)) == len(loose) and not any(count[x] for x in loose)
        assert len(loose) + sum(c > 0 for c in count) == n - 1
        for row, x in zip(tables, lens):
            if x > sh * bs and x % bs:
                assert count[row[-(-x // bs) - 1]] == 1
        for r in range(B):                      # grow, as the plan would
            for _ in range(rng.randrange(4)):
                if lens[r] >= sh * bs and lens[r] < width * bs and (lens[r] % bs or free[0] < free[1]):
                    if lens[r] % bs == 0:
                        tables[r][lens[r] // bs] = ring[free[0] % n]
                        free = (free[0] + 1, free[1])
                    lens[r] += 1


def test_beams_by_all_candidates():
    rng = np.random.default_rng(2)
    k, v = 3, 11
    x = np.round(rng.normal(size=(6, v)) * 2) / 2
    sums, ended = -np.abs(rng.normal(size=6)).astype(np.float32), [0, 1, 0, 0, 0, 0]
    got = Q.beams(x, k, sums, ended, 4)
    lp = x - np.log(np.exp(x).sum(-1, keepdims=True))
    for g in range(2):
        every = sorted([(-(sums[r] + lp[r, t]), r, t) for r in range(3 * g, 3 * g + 3) for t in range(v) if not ended[r]] +
                       [(-float(sums[r]), r, 4) for r in range(3 * g, 3 * g + 3) if ended[r]])[:k]
        assert got["parents"][3 * g:3 * g + 3] == [c[1] for c in every]
        assert got["tokens"][3 * g:3 * g + 3] == [c[2] for c in every]
        assert np.allclose(got["sums_out"][3 * g:3 * g + 3], [-c[0] for c in every], atol=1e-12)


def test_null_pointers_are_refused_without_a_device():
    B.build()
    lib, n = C._lib(), None
    assert lib.codec_lm_store_q4(n, n, 0, n, 0, 0, 1, n, n, n, n) == 1
    assert lib.codec_lm_load_q4(n, n, n, n, n, 1, n, n, 1, n) == 1
    assert lib.codec_lm_step_q4(n, n, 0, 1, n, n, n, n, n, 0, n, 0, n, n) == 1
    assert lib.codec_lm_beams(n, n, 0, 0, 1, 1, 2, n, n, 0, n, n, n, n, n) == 1
    assert lib.codec_lm_fork(n, n, n, 1, n, n, 0, n, n, n, n, n, n, n, n, n, n, n) == 1
    assert lib.codec_lm_compact(n, n, 1, n, n, n, n, 0, n, n, n, n, n, n, n, n) == 1
    assert lib.codec_lm_copy(n, n, 1, 16, n, n, 1, n, n) == 1
