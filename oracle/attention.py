"""CPU oracle of the attention operators: plain definitions in 64 bits (test
infrastructure, like the rest of this package; it shares no code with the HIP
library).

  attention          out_i = sum_{j<=i} p_ij v_j, p_i = softmax_j(scale q_i . k_j), per packed sequence
  cache_append       per block of 64 tokens and head: s' = max(s, max|x|, 1e-30), codes rint(x (127/s')),
                     earlier codes rint(c (s/s')); every step rounded to fp32 as the definition says
  attention_cached   the same softmax over the values c (s/127) of a paged cache
  cache_evict        which blocks a sequence keeps

Codes are held in natural order here ([pages][heads][64 tokens][d]); stored() and
natural() go by the storage rule, byte by byte.
"""
from __future__ import annotations

import numpy as np

BLOCK = 64
_f32 = np.float32


def code_places(d: int):
    """(K, V) byte of every (token, dim) inside a page and head."""
    tok, dim = np.meshgrid(np.arange(BLOCK), np.arange(d), indexing="ij")
    k = ((tok % 4) * (d // 16) + dim // 16) * 256 + (tok // 4) * 16 + dim % 16
    v = ((dim // 16) * 4 + tok // 16) * 256 + (dim % 16) * 16 + tok % 16
    return k, v


def stored(codes: np.ndarray, place: np.ndarray) -> np.ndarray:
    out = np.empty(codes.shape[:2] + (place.size,), np.int8)
    out[:, :, place.ravel()] = codes.reshape(codes.shape[0], codes.shape[1], -1)
    return out


def natural(codes: np.ndarray, place: np.ndarray) -> np.ndarray:
    return codes[:, :, place.ravel()].reshape(codes.shape[:2] + place.shape)


def _rows(cu, m, seqs):
    if cu is None:
        return [(s, s + 1) for s in range(seqs)]
    c = np.clip(np.asarray(cu, np.int64), 0, m)
    return [(int(a), int(max(a, b))) for a, b in zip(c[:-1], c[1:])]


def _softmax(s, seen):
    """Rows of weights over the seen entries (a row that sees none: zeros)."""
    s = np.where(seen, s, -np.inf)
    top = s.max(1, keepdims=True, initial=-np.inf)
    p = np.where(seen, np.exp(s - np.where(np.isfinite(top), top, 0.0)), 0.0)
    total = p.sum(1, keepdims=True)
    return np.divide(p, total, out=np.zeros_like(p), where=total > 0)


def attention(q, k, v, cu, scale):
    """q [m][hq][d], k, v [m][hkv][d] -> (out [m][hq][d], spread, reach): spread = sum_j p_ij |v_j|, by which
    relative errors of p count, and reach = max_j scale sum |q_i||k_j|, by which rounding of the logits does."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    m, hq, d = q.shape
    group = hq // k.shape[1]
    out, spread, reach = np.zeros_like(q), np.zeros_like(q), np.zeros((m, hq, 1))
    for a, b in _rows(cu, m, None):
        seen = np.tril(np.ones((b - a, b - a), bool))
        for h in range(hq if b > a else 0):
            kk, vv = k[a:b, h // group], v[a:b, h // group]
            p = _softmax(scale * (q[a:b, h] @ kk.T), seen)
            out[a:b, h], spread[a:b, h] = p @ vv, p @ np.abs(vv)
            reach[a:b, h, 0] = np.where(seen, abs(scale) * (np.abs(q[a:b, h]) @ np.abs(kk).T), 0).max(1)
    return out, spread, reach


def cache_append(codes, scales, x, table, lens, cu):
    """Appends x [m][heads][d] to codes [pages][heads][64][d], scales [pages][heads], in place."""
    x = np.asarray(x, _f32)
    x = np.where(np.isnan(x), _f32(0), np.clip(x, -np.finfo(_f32).max, np.finfo(_f32).max))
    for s, (a, b) in enumerate(_rows(cu, x.shape[0], len(lens))):
        have = int(lens[s])
        if have < 0:
            continue
        for block in range(have // BLOCK, min(-(-(have + b - a) // BLOCK), table.shape[1])):
            page = int(table[s, block])
            lo, hi = max(have, block * BLOCK), min(have + b - a, (block + 1) * BLOCK)
            if hi <= lo or not 0 <= page < codes.shape[0]:
                continue
            used, new = lo - block * BLOCK, x[a + lo - have:a + hi - have]
            for h in range(x.shape[1]):
                old = scales[page, h] if used else _f32(0)
                big = max(old, np.abs(new[:, h]).max(), _f32(1e-30))
                codes[page, h, :used] = np.rint(codes[page, h, :used].astype(_f32) * _f32(old / big)).astype(np.int8)
                codes[page, h, used:used + hi - lo] = np.rint(new[:, h] * _f32(_f32(127) / big)).astype(np.int8)
                scales[page, h] = big


def tokens(codes, scales, table_row, first, last):
    """Values [last - first][heads][d] (fp32 products) of a sequence's tokens, and which of them have a page."""
    heads, d = codes.shape[1], codes.shape[3]
    out, there = np.zeros((last - first, heads, d), _f32), np.zeros(last - first, bool)
    for t in range(first, last):
        block = t // BLOCK
        page = int(table_row[block]) if block < len(table_row) else -1
        if 0 <= page < codes.shape[0]:
            out[t - first] = codes[page, :, t % BLOCK].astype(_f32) * (scales[page] / _f32(127))[:, None]
            there[t - first] = True
    return out, there


def attention_cached(q, kc, ks, vc, vs, table, lens, cu, scale):
    """-> (out, weights to add [seqs][max_blocks], spread, reach, grain): grain is the size by which errors of p
    relative to its block's largest count, per output."""
    q = np.asarray(q, np.float64)
    m, hq, d = q.shape
    group, seqs, wide = hq // kc.shape[1], table.shape[0], table.shape[1]
    out, spread, grain = (np.zeros_like(q) for _ in range(3))
    reach, weights = np.zeros((m, hq, 1)), np.zeros((seqs, wide))
    for s, (a, b) in enumerate(_rows(cu, m, seqs)):
        have = int(lens[s])
        if have < 0 or b <= a:
            continue
        last = min(have + b - a, wide * BLOCK)
        k, there = tokens(kc, ks, table[s], 0, last)
        v, _ = tokens(vc, vs, table[s], 0, last)
        k, v = k.astype(np.float64), v.astype(np.float64)
        blocks = -(-last // BLOCK)
        seen = there[None, :] & (np.arange(last)[None, :] <= (have + np.arange(b - a))[:, None])
        for h in range(hq):
            kk, vv = k[:, h // group], v[:, h // group]
            p = _softmax(scale * (q[a:b, h] @ kk.T), seen)
            out[a:b, h], spread[a:b, h] = p @ vv, p @ np.abs(vv)
            qmax = np.abs(q[a:b, h]).max(1, keepdims=True)
            reach[a:b, h, 0] = (abs(scale) * (np.abs(q[a:b, h]) @ np.abs(kk).T + qmax * np.abs(kk).sum(1)[None])).max(1, initial=0)
            full = np.pad(p, ((0, 0), (0, blocks * BLOCK - last))).reshape(b - a, blocks, BLOCK)
            sums = np.pad(np.abs(vv), ((0, blocks * BLOCK - last), (0, 0))).reshape(blocks, BLOCK, d).sum(1)
            grain[a:b, h] = full.max(2, initial=0) @ sums
            weights[s, :blocks] += full.sum((0, 2))
    return out, weights, spread, reach, grain


def cache_evict(table, lens, weights, keep, first, recent):
    seqs, wide = table.shape
    out = [np.full((seqs, wide), -1, np.int32), lens.copy(), np.zeros((seqs, wide), _f32), np.full((seqs, wide), -1, np.int32),
           np.zeros(seqs, np.int32)]
    for s in range(seqs):
        used = min(-(-max(int(lens[s]), 0) // BLOCK), wide)
        held = [b for b in range(used) if b < first or b >= used - recent]
        value = lambda b: np.inf if np.isnan(weights[s, b]) else float(weights[s, b])  # noqa: E731
        rest = sorted((b for b in range(used) if b not in set(held)), key=lambda b: (-value(b), b))
        stays = sorted(held + rest[:max(0, keep - len(held))])
        gone = [b for b in range(used) if b not in set(stays)]
        out[0][s, :len(stays)] = table[s, stays]
        out[2][s, :len(stays)] = weights[s, stays]
        out[3][s, :len(gone)] = table[s, gone]
        out[1][s] -= BLOCK * len(gone)
        out[4][s] = len(gone)
    return out
