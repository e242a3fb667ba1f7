"""The codec LM's cache in 4 bits, forked and compacted blocks, and beam search
from their definitions: numpy, whole numbers and 64 bits.  Test infrastructure only."""
from __future__ import annotations

import numpy as np
import torch

import lm_ref as R

DTYPES = R.DTYPES


# ---- the format -------------------------------------------------------------

def encode(x):
    """float32 [..][d] -> codes uint8 [..][d], scale, low float16 [..][d / 32], each step in 32 bits."""
    x = np.asarray(x, np.float32)
    x = x.reshape(*x.shape[:-1], -1, 32)
    good = np.isfinite(x).all(-1)
    with np.errstate(all="ignore"):
        x = np.clip(x, np.float32(-65504), np.float32(65504))
        lo, hi = x.min(-1), x.max(-1)
        scale = ((hi - lo) * np.float32(1 / 15)).astype(np.float16)
        low = lo.astype(np.float16)
        inverse = np.float32(1) / scale.astype(np.float32)
        steps = np.rint((x - low.astype(np.float32)[..., None]) * inverse[..., None])
        steps = np.clip(np.where((good & (scale > 0))[..., None], steps, 0), 0, 15)
    codes = steps.astype(np.uint8).reshape(*x.shape[:-2], -1)
    nan = np.float16(np.nan)
    return codes, np.where(good, scale, nan), np.where(good, low, nan)


def decoded(x):
    """What rows [..][d] stand for once stored, float64."""
    c, s, l = encode(x)
    return np.repeat(l.astype(np.float64), 32, -1) + np.repeat(s.astype(np.float64), 32, -1) * c


def places(d, keys):
    """For position p and element i: byte of the code in a tile and whether its
    upper half; for position p and group g: bytes of scale and low."""
    G = d // 32
    code, upper = np.zeros((16, d), int), np.zeros((16, d), int)
    scale, low = np.zeros((16, G), int), np.zeros((16, G), int)
    for p in range(16):
        a, t, b = p // 8, p % 8 // 2, p % 2
        for i in range(d):
            g, e = i // 32, i % 32
            upper[p, i] = e % 2
            if keys:
                code[p, i] = p * d // 2 + (e // 8 * G + g) * 4 + e % 8 // 2
            else:
                code[p, i] = a * 4 * d + (e // 4 * 4 + t) * 4 * G + g * 4 + b * 2 + e % 4 // 2
        for g in range(G):
            if keys:
                scale[p, g] = 8 * d + (p * G + g) * 4
                low[p, g] = scale[p, g] + 2
            else:
                scale[p, g] = 8 * d + ((t * G + g) * 4 + 2 * a + b) * 2
                low[p, g] = scale[p, g] + d
    return code, upper, scale, low


def store(cache, rows, slots, bs, keys):
    """cache uint8 [blocks][heads][bytes] (in place), rows float32 [n][heads][d]."""
    n, hk, d = rows.shape
    code, upper, scale, low = places(d, keys)
    c, s, l = encode(rows)
    for r in range(n):
        if not 0 <= slots[r] < cache.shape[0] * bs:
            continue
        blk, at = divmod(int(slots[r]), bs)
        tile, p = divmod(at, 16)
        for h in range(hk):
            t = cache[blk, h, tile * 10 * d:(tile + 1) * 10 * d]
            for half in (0, 1):
                i = np.flatnonzero(upper[p] == half)
                keep = 0x0F if half else 0xF0
                t[code[p, i]] = (t[code[p, i]] & keep) | (c[r, h, i] << (4 * half))
            for g in range(d // 32):
                t[scale[p, g]:scale[p, g] + 2] = np.frombuffer(s[r, h, g].tobytes(), np.uint8)
                t[low[p, g]:low[p, g] + 2] = np.frombuffer(l[r, h, g].tobytes(), np.uint8)


def values(cache, bs, d, keys, parts=False):
    """float64 [blocks][bs][heads][d] that the bytes stand for (parts: low, and scale * code)."""
    code, upper, scale, low = places(d, keys)
    n, hk = cache.shape[:2]
    t = cache.reshape(n, hk, bs // 16, 10 * d)
    c = t[..., code]
    c = np.where(upper == 1, c >> 4, c & 15).astype(np.float64)
    with np.errstate(invalid="ignore"):
        pick = lambda at: np.ascontiguousarray(t[..., np.stack([at, at + 1], -1)]).view(np.float16)[..., 0].astype(np.float64)
        sc, lo = (np.repeat(pick(at), 32, -1) for at in (scale, low))
    put = lambda x: np.moveaxis(x, 1, 3).reshape(n, bs, hk, d)
    with np.errstate(invalid="ignore"):
        return (put(lo), put(sc * c)) if parts else put(lo + sc * c)


# ---- attention --------------------------------------------------------------

def step(q, keys_of, hk, scale):
    """q float64 [B][hq][d]; keys_of(b): (k low, k rest, v low, v rest), float64
    [n][hk][d].  Results and the sums that bound their rounding."""
    B, hq, d = q.shape
    o, lse = np.zeros(q.shape), np.full((B, hq), -np.inf)
    al, ac, s, n_keys = np.zeros(q.shape), np.zeros(q.shape), np.zeros((B, hq)), np.zeros(B)
    for b in range(B):
        kl, kc, vl, vc = keys_of(b)
        n_keys[b] = len(kl)
        if len(kl) == 0:
            continue
        for h in range(hq):
            g = h // (hq // hk)
            x = ((kl + kc)[:, g] @ q[b, h]) * scale
            p = np.exp(x - x.max())
            l = p.sum()
            p, lse[b, h] = p / l, x.max() + np.log(l)
            o[b, h] = p @ (vl + vc)[:, g]
            al[b, h], ac[b, h] = p @ np.abs(vl[:, g]), p @ np.abs(vc[:, g])
            s[b, h] = ((np.abs(kl) + np.abs(kc))[:, g] @ np.abs(q[b, h])).max() * scale
    return o, lse, al, ac, s, n_keys


def assert_step(got, got_lse, ref, dtype, d, v_max):
    """Elementwise, from the arithmetic.  The result is rounded once, to its type.
    A probability is rounded to fp16 (half a step, 2^-11) and its product with a
    group's scale once more; the sum over lows takes it with the first alone.
    Scores are sums of 2 d products in fp32 (codes' and lows') whose additions may
    truncate, 2 d steps of 2^-23 of sum |q| (|low| + scale code), as much again for
    the sum of a query's group in 22 bits and the exponent's argument; that moves a
    probability by as much relatively, twice with the normaliser.  Sums over keys may
    truncate at each of their steps of 16 keys.  Probabilities are held as multiples
    of 2^-24 with the row's largest at 2^6 at least (2^6 / v_max where scales pass 2),
    so each, and each product with a scale, may be off by 2^-31 of it, times a code
    of 15 or a low.
    fp16: a probability is two halves, what is rounded and what that leaves off, rounded:
    2^-22 of it.  Its product with a scale as well: the rounded product's rest is exact,
    the second half's product and their sum are rounded (2^-22 and 2^-21).  Sums take
    two steps for 16 keys."""
    o, lse, al, ac, s, n = ref
    half = torch.finfo(DTYPES[dtype]).eps / 2
    ds = (4 * d * 2.0 ** -23 * (s + 1))[..., None]
    n = n[:, None, None]
    a, fine = al + ac, dtype == "fp16"
    tol = half * np.abs(o) * 1.01 + (al * 2.0 ** -11 + ac * 2.0 ** -10) * (2.0 ** -10 if fine else 1.01)
    tol = tol + a * (2 * ds + (n / (4 if fine else 8) + 16) * 2.0 ** -23)
    tol = tol + n * 2.0 ** -31 * (15 + 2 * v_max) * max(1.0, v_max) + 2.0 ** -25 * (dtype == "fp16") + 1e-30
    g = got.detach().cpu().double().numpy()
    bad = ~(np.abs(g - o) <= tol)
    assert not bad.any(), (f"{bad.sum()} of {bad.size} off, worst {np.nanmax(np.abs(g - o) / tol):.3g} x the bound "
                           f"at {np.argwhere(bad)[:4].tolist()}, NaN {np.isnan(g).sum()}")
    if got_lse is not None:
        gl = got_lse.detach().cpu().double().numpy()
        empty = np.isneginf(lse)
        assert np.array_equal(np.isneginf(gl), empty)
        off = np.abs(np.where(empty, 0, gl) - np.where(empty, 0, lse))
        assert (off <= ds[..., 0] + (np.abs(np.where(empty, 0, lse)) + 4) * 2.0 ** -20).all(), f"lse off by {off.max():.3g}"


# ---- blocks -----------------------------------------------------------------

def fork(parents, lens, tables, tables_out, owners, ring, free, bs, sh):
    """Row by row.  tables_out, ring: what is there before."""
    B, width, n = len(parents), len(tables[0]), len(owners)
    head, tail = free
    good_ring = 0 <= head <= tail <= head + n
    left = tail - head if good_ring else 0
    out, ring, count = [list(r) for r in tables_out], list(ring), list(owners)
    there = [0 <= x <= width * bs for x in lens]
    blocks = [-(-x // bs) if ok else 0 for x, ok in zip(lens, there)]
    unfilled = [blocks[r] > sh and lens[r] % bs != 0 for r in range(B)]
    status, kv, src, dst, children, asked, seen = [], [], [], [], [0] * B, 0, set()
    for b, p in enumerate(parents):
        if p == -1 or not (0 <= p < B) or not there[p]:
            status.append(0 if p == -1 else 2)
            kv.append(0)
            continue
        row = list(tables[p][:blocks[p]])
        if p in seen and unfilled[p]:           # not its first child
            asked += 1
            if asked > left:
                status.append(1)
                kv.append(0)
                continue
            fresh = ring[(head + asked - 1) % n]
            src.append(row[-1])
            dst.append(fresh)
            row[-1] = fresh
        seen.add(p)
        children[p] += 1
        out[b][:blocks[p]] = row
        status.append(0)
        kv.append(lens[p])
    for r in range(B):
        for j in range(sh, blocks[r]):
            own = unfilled[r] and j == blocks[r] - 1
            if 0 <= tables[r][j] < n:
                count[tables[r][j]] += (min(children[r], 1) if own else children[r]) - 1
    back = 0
    for i in range(n):
        if count[i] < 0:
            if good_ring and back < n - left:
                ring[(tail + back) % n] = i
                back += 1
            count[i] = 0
    return dict(tables_out=out, owners_out=count, free_list=ring, free_out=[head + len(src), tail + back], kv_out=kv,
                status=status, copies=[len(src)], copy_src=src, copy_dst=dst)


def compact(lens, tables, tables_out, shared, owners, ring, bs):
    B, width, n, sh = len(lens), len(tables[0]), len(owners), len(shared)
    blocks = [-(-min(max(x, 0), width * bs) // bs) for x in lens]
    used = {x for r in range(B) for x in tables[r][sh:blocks[r]] if 0 <= x < n} | {x for x in shared if 0 <= x < n}
    U = len(used)
    src, dst = sorted(x for x in used if x >= U), [x for x in range(U) if x not in used]
    move = dict(zip(src, dst))
    to = lambda x: move.get(x, x)
    out = [list(r) for r in tables_out]
    for r in range(B):
        for j in range(blocks[r]):
            out[r][j] = to(shared[j] if j < sh else tables[r][j])
    count = [0] * n
    for x in used:
        count[to(x)] = owners[x]
    ring = list(range(U, n)) + list(ring[n - U:])
    return dict(tables_out=out, shared_out=[to(x) for x in shared], owners_out=count, free_list=ring,
                free_out=[0, n - U], copies=[len(src)], copy_src=src, copy_dst=dst)


# ---- beam search ------------------------------------------------------------

def beams(logits, k, sums, ended, end):
    """logits float64 [rows][vocab]."""
    rows, vocab = logits.shape
    out = dict(sums_out=[], parents=[], tokens=[], ended_out=[])
    for g0 in range(0, rows, k):
        got = []
        for r in range(g0, g0 + k):
            if not np.isfinite(sums[r]):
                continue
            if ended[r]:
                got.append((-float(sums[r]), r, end, True))
                continue
            x = logits[r]
            if np.isnan(x).any() or not np.isfinite(x.max()):
                continue
            m = x.max()
            base = float(sums[r]) - np.log(np.exp(x - m).sum())
            for v in np.argsort(-x, kind="stable")[:k]:
                if x[v] > -np.inf:
                    got.append((-(base + (x[v] - m)), r, int(v), False))
        got.sort(key=lambda c: c[:3])
        for i in range(k):
            s, r, v, itself = got[i] if i < len(got) else (np.inf, -1, -1, False)
            out["sums_out"].append(-s)
            out["parents"].append(r)
            out["tokens"].append(v)
            out["ended_out"].append(int(r < 0 or itself or v == end))
    return out
