"""CPU oracle of what stands before and beside attention over the cache: plain definitions in 64 bits (test
infrastructure, like the rest of this package; it shares no code with the HIP library).

  rotate              every pair (a, b) of a head times magnitude * e^(i position frequency), an RMS norm before
  attention_shared    the softmax over a prefix's tokens and the sequence's own together
  cache_bounds        the largest and the smallest K code of a block's tokens
  block_select        the blocks with the largest upper bound of the products with a row's queries
  attention_selected  the softmax over the tokens of listed blocks

Caches and tables are held as in oracle/attention.py.
"""
from __future__ import annotations

import numpy as np

from oracle.attention import BLOCK, _rows, _softmax, tokens

_f32 = np.float32


def positions(begin, cu, m):
    """Position of every row (-1: in no sequence, or in an unused slot)."""
    out = np.full(m, -1, np.int64)
    for s, (a, b) in enumerate(_rows(cu, m, len(begin))):
        if begin[s] >= 0:
            out[a:b] = int(begin[s]) + np.arange(b - a)
    return out


def rotate(x, position, inv_freq, interleaved, gain, eps, magnitude):
    """x [m][heads][d] -> (y, size): size is |a| + |b| of an element's pair before the rotation (of the element itself
    behind the rotated ones), by which rounding of the cosines and sines counts. Angles in extended precision: a
    position below 2^31 times an fp32 frequency is exact there."""
    x = np.asarray(x, np.float64)
    if gain is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(gain, np.float64)
    y, size = x.copy(), np.abs(x)
    n = len(inv_freq)
    angle = np.asarray(position, np.longdouble)[:, None] * np.asarray(inv_freq, np.longdouble)[None]
    co, si = (np.asarray(f(angle), np.float64)[:, None] * magnitude for f in (np.cos, np.sin))
    first = np.arange(n) * 2 if interleaved else np.arange(n)
    second = first + 1 if interleaved else first + n
    a, b = x[..., first], x[..., second]
    y[..., first], y[..., second] = a * co - b * si, b * co + a * si
    size[..., first] = size[..., second] = np.abs(a) + np.abs(b)
    return y, size


def _attend(q, k, v, seen, scale, out, spread, reach, grain):
    """One kv head's rows q [rows][d] over keys k, v [n][d]; results into the given views. n is a multiple of 64."""
    p = _softmax(scale * (q @ k.T), seen)
    out[:], spread[:] = p @ v, p @ np.abs(v)
    qmax = np.abs(q).max(1, keepdims=True)
    reach[:, 0] = np.where(seen, abs(scale) * (np.abs(q) @ np.abs(k).T + qmax * np.abs(k).sum(1)[None]), 0).max(1, initial=0)
    if len(k):
        counted = np.where(seen.any(0)[:, None], np.abs(v), 0.0)
        grain[:] = p.reshape(len(q), -1, BLOCK).max(2) @ counted.reshape(-1, BLOCK, v.shape[1]).sum(1)


def _block_tokens(kc, ks, vc, vs, pages):
    """K and V values [blocks * 64][heads][d] of pages (-1: none), and which tokens have one."""
    row = np.asarray(pages, np.int64)
    k, there = tokens(kc, ks, row, 0, BLOCK * len(row))
    return k.astype(np.float64), tokens(vc, vs, row, 0, BLOCK * len(row))[0].astype(np.float64), there


def attention_shared(q, kc, ks, vc, vs, prefix, length, table, lens, cu, scale):
    """-> (out, spread, reach, grain) as attention_cached's"""
    q = np.asarray(q, np.float64)
    m, hq, d = q.shape
    group = hq // kc.shape[1]
    out, spread, grain = (np.zeros_like(q) for _ in range(3))
    reach = np.zeros((m, hq, 1))
    kp, vp, there_p = _block_tokens(kc, ks, vc, vs, prefix)
    seen_p = there_p & (np.arange(len(kp)) < length)
    for s, (a, b) in enumerate(_rows(cu, m, table.shape[0])):
        have = int(lens[s])
        if have < 0 or b <= a:
            continue
        k, v, there = _block_tokens(kc, ks, vc, vs, table[s])
        seen = there[None] & (np.arange(len(k))[None] <= (have + np.arange(b - a))[:, None])
        k, v = np.concatenate((kp, k)), np.concatenate((vp, v))
        seen = np.concatenate((np.broadcast_to(seen_p, (b - a, len(seen_p))), seen), 1)
        for h in range(hq):
            _attend(q[a:b, h], k[:, h // group], v[:, h // group], seen, scale, *(x[a:b, h] for x in (out, spread, reach, grain)))
    return out, spread, reach, grain


def cache_bounds(kc, bounds, table, lens, cu, m):
    """Writes bounds [pages][heads][2][d] of the blocks that the rows reach, in place."""
    for s, (a, b) in enumerate(_rows(cu, m, table.shape[0])):
        have = int(lens[s])
        if have < 0 or b <= a:
            continue
        for block in range(have // BLOCK, min(-(-(have + b - a) // BLOCK), table.shape[1])):
            page = int(table[s, block])
            if 0 <= page < kc.shape[0]:
                held = kc[page, :, :min(BLOCK, have + b - a - block * BLOCK)]
                bounds[page, :, 0], bounds[page, :, 1] = held.max(1), held.min(1)


def block_select(q, bounds, ks, table, lens, keep, cu, first, recent, fill):
    """-> [m][heads][keep]; rows that are not written keep `fill`."""
    q = np.asarray(q, _f32)
    m, hq, d = q.shape
    heads, wide = bounds.shape[1], table.shape[1]
    out = np.full((m, heads, keep), fill, np.int32)
    most = np.finfo(_f32).max
    for s, (a, b) in enumerate(_rows(cu, m, table.shape[0])):
        for r in range(a, b if lens[s] >= 0 else a):
            used = min((int(lens[s]) + r - a) // BLOCK + 1, wide)
            for g in range(heads):
                x = q[r, g * (hq // heads):(g + 1) * (hq // heads)]
                x = np.where(np.isnan(x), _f32(0), np.clip(x, -most, most))
                c = np.rint(x * _f32(_f32(127) / max(np.abs(x).max(), _f32(1e-30)))).astype(np.int64)
                score = np.full(used, -np.inf)
                for i in range(used):
                    page = int(table[s, i])
                    if 0 <= page < bounds.shape[0]:
                        high, low = bounds[page, g].astype(np.int64)
                        with np.errstate(over="ignore"):
                            score[i] = _f32(np.maximum(high * c, low * c).sum()) * ks[page, g]
                score = np.where(np.isnan(score), np.inf, score)
                held = [i for i in range(used) if i < first or i >= used - recent]
                rest = sorted(set(range(used)) - set(held), key=lambda i: (-score[i], i))
                stays = sorted(held + rest[:keep - len(held)]) if used > keep else list(range(used))
                out[r, g] = stays + [-1] * (keep - len(stays))
    return out


def attention_selected(q, kc, ks, vc, vs, table, lens, selected, cu, scale):
    """-> (out, spread, reach, grain) as attention_cached's"""
    q = np.asarray(q, np.float64)
    m, hq, d = q.shape
    heads = kc.shape[1]
    group = hq // heads
    out, spread, grain = (np.zeros_like(q) for _ in range(3))
    reach = np.zeros((m, hq, 1))
    for s, (a, b) in enumerate(_rows(cu, m, table.shape[0])):
        have = int(lens[s])
        for r in range(a, b if have >= 0 else a):
            for g in range(heads):
                blocks = np.array([i for i in selected[r, g] if 0 <= i < table.shape[1]], np.int64)
                k, v, there = _block_tokens(kc, ks, vc, vs, table[s][blocks])
                token = (blocks[:, None] * BLOCK + np.arange(BLOCK)).ravel()
                seen = (there & (token <= have + r - a))[None]
                at = slice(g * group, (g + 1) * group)
                _attend(q[r, at], k[:, g], v[:, g], np.broadcast_to(seen, (group, len(k))), scale,
                        *(x[r, at] for x in (out, spread, reach, grain)))
    return out, spread, reach, grain
