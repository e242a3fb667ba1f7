"""The codec LM's attention operators from their definitions, in 64 bits or in
whole numbers, one request and one row at a time.  Test infrastructure only."""
from __future__ import annotations

import numpy as np
import torch

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def plan(before, after, tables, free_list, free, shared_table, bs, max_rows):
    """Sequential statement of the block plan; returns every output."""
    tables, ring = [list(r) for r in tables], list(free_list)
    n, width, sh = len(ring), len(tables[0]), len(shared_table)
    head, tail = free
    if not (0 <= head <= tail <= head + n):
        left, room = 0, 0
    else:
        left, room = tail - head, n - (tail - head)
    owned = lambda x: max(0, -(-x // bs) - sh)
    row_start, kv_len, status, slots, positions = [0], [], [], [], []
    taken = asked = back = total = 0
    for b, (n0, n1) in enumerate(zip(before, after)):
        st, rows = 0, 0
        if min(n0, n1) < 0 or max(n0, n1) > width * bs:
            st = 2
        else:
            rows = max(0, n1 - n0)
            total += rows
            if total > max_rows:
                st = 3
        need = max(0, owned(n1) - owned(n0)) if st == 0 else 0
        asked += need
        if need and asked > left:
            st = 1
        if st == 0:
            if n0 <= sh * bs and n1 > n0:
                tables[b][:sh] = shared_table
            for j in range(need):
                tables[b][sh + owned(n0) + j] = ring[(head + taken) % n]
                taken += 1
            for j in range(sh + owned(n1), sh + owned(n0)):
                if back < room:
                    ring[(tail + back) % n] = tables[b][j]
                    back += 1
        for p in range(n0, n0 + rows):
            if len(slots) < max_rows:
                slots.append(tables[b][p // bs] * bs + p % bs if st == 0 else -1)
                positions.append(p)
        row_start.append(min(total, max_rows))
        kv_len.append(n1 if st == 0 else 0)
        status.append(st)
    pad = max_rows - len(slots)
    return dict(tables=tables, free_list=ring, free_out=[head + taken, tail + back], row_start=row_start,
                kv_len=kv_len, status=status, slots=slots + [-1] * pad, positions=positions + [0] * pad)


def rotate(x, gain, positions, theta, eps, pairs):
    """x [rows][heads][d] -> normed and turned, float64."""
    x = x.detach().cpu().double().numpy()
    d = x.shape[-1]
    if gain is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * gain.cpu().double().numpy()
    out = np.empty_like(x)
    for i in range(d // 2):
        a, b = (2 * i, 2 * i + 1) if pairs else (i, i + d // 2)
        angle = positions.cpu().double().numpy() * float(theta) ** (-2.0 * i / d)
        c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
        out[..., a] = x[..., a] * c - x[..., b] * s
        out[..., b] = x[..., b] * c + x[..., a] * s
    return out


def attend_row(q, k, v, scale):
    """One query [d] over keys [n][d]: (o, lse, sum p|v|, largest sum |q k| scale)."""
    if len(k) == 0:
        return np.zeros(v.shape[1]), -np.inf, np.zeros(v.shape[1]), 0.0
    x = (k @ q) * scale
    m = x.max()
    p = np.exp(x - m)
    l = p.sum()
    return p @ v / l, m + np.log(l), p @ np.abs(v) / l, float((np.abs(k) @ np.abs(q)).max() * scale)


def attention(q, rows_of, keys_of, hk, scale):
    """q float64 [rows][hq][d]; rows_of: list of (row, keys, values) with keys,
    values [n][hk][d] the ones that row may see."""
    hq, d = q.shape[1:]
    o = np.full(q.shape, np.nan)
    a, lse, s = np.zeros(q.shape), np.full(q.shape[:2], np.nan), np.zeros(q.shape[:2])
    for row in rows_of:
        k, v = keys_of(row)
        for h in range(hq):
            g = h // (hq // hk)
            o[row, h], lse[row, h], a[row, h], s[row, h] = attend_row(q[row, h], k[:, g], v[:, g], scale)
    return o, lse, a, s


def assert_attention(got, got_lse, ref, dtype, n_keys, d, v_max):
    """Elementwise, from the arithmetic: the result is rounded once (half a step
    of its type), every probability once (half a step, so sum p |v| half a step);
    scores are sums of d products in fp32 whose every addition may truncate
    (d steps of 2^-23 of sum |q k|, and as much again for the scale and the
    exponent's argument), which moves a probability by as much relatively, twice
    with the normaliser; sums over keys may truncate at each of their steps of 16
    keys.  fp16 probabilities below 2^-24 of the row's largest may vanish."""
    o, lse, a, s = ref
    half = torch.finfo(DTYPES[dtype]).eps / 2
    ds = (2 * d * 2.0 ** -23 * (s + 1))[..., None]
    keys = np.asarray(n_keys)
    while keys.ndim < 3:
        keys = keys[..., None]
    tol = half * (np.abs(o) + a * 1.01) + a * (2 * ds + (keys / 8 + 16) * 2.0 ** -23) + 1e-30
    if dtype == "fp16":
        tol = tol + 2.0 ** -25 * (1 + keys * v_max)
    g = got.detach().cpu().double().numpy()
    bad = ~(np.abs(g - o) <= tol)
    assert not bad.any(), (f"{bad.sum()} of {bad.size} off, worst {np.nanmax(np.abs(g - o) / tol):.3g} x the bound "
                           f"at {np.argwhere(bad)[:4].tolist()}, NaN {np.isnan(g).sum()}")
    if got_lse is not None:
        gl = got_lse.detach().cpu().double().numpy()
        empty = np.isneginf(lse)
        assert np.array_equal(np.isneginf(gl), empty)
        tl = ds[..., 0] + (np.abs(np.where(empty, 0, lse)) + 4) * 2.0 ** -20
        off = np.abs(np.where(empty, 0, gl) - np.where(empty, 0, lse))
        assert (off <= tl).all(), f"lse off by {off.max():.3g}"
