"""Paged 8-bit KV cache -- test infrastructure only.

A pool of blocks of `bs` tokens; block b holds, for every key/value head, bs x d
8-bit codes and one fp32 scale for the keys and one for the values.  Three rules:

  plan    request lengths -> block tables, starts and slots (a ring of free blocks,
          taken from the front in request order, given back at the end).
  append  s = max(s_old, max |x| / qmax) over the block's new tokens (s_old = 0 in a
          block whose first row is new); code = round(x / s); the block's earlier
          codes, when s grew, become round(code (s_old / s)).  fp32, nearest even.
  attend  softmax(scale q k^T) v over the cached tokens, in float64.

The source of the 8-bit cache is "VAR-Compressor：在边缘GPU上实现80亿参数视觉自回归模型的
高效量化部署", INT8 KV缓存量化; it says nothing about pages, so the rules above are this
project's own.
"""
from __future__ import annotations

import numpy as np

F32 = np.float32
QMAX = {"int8": F32(127.0), "e4m3": F32(448.0)}
NORMAL = {2.0 ** -8: 2.0 ** -126, 2.0 ** -11: 2.0 ** -14}   # smallest normal number by half a step: bf16, fp16


def e4m3_values() -> np.ndarray:
    """The 256 values of the E4M3 codes (NaN for 0x7f and 0xff)."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m / 8.0 * 2.0 ** -6, (1 + m / 8.0) * 2.0 ** (e - 7.0))
    v = np.where((e == 15) & (m == 7), np.nan, v)
    return np.where(c & 0x80, -v, v)


E4M3 = e4m3_values()


def to_codes(x: np.ndarray, fmt: str) -> np.ndarray:
    """fp32 values to the nearest code (ties to even), saturating; uint8 bit patterns."""
    x = np.asarray(x, dtype=np.float64)
    if fmt == "int8":
        return np.clip(np.rint(x), -127, 127).astype(np.int8).view(np.uint8)
    a = np.abs(x)
    step = 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(a, 2.0 ** -20))), -6) - 3)
    a = np.minimum(np.rint(a / step) * step, 448.0)
    pos = E4M3[:0x7F]                                     # increasing
    return (np.searchsorted(pos, a) | np.where(np.signbit(x), 0x80, 0)).astype(np.uint8)


def values(codes: np.ndarray, fmt: str) -> np.ndarray:
    return codes.view(np.int8).astype(np.float64) if fmt == "int8" else E4M3[codes]


def plan(prev, target, table, ring, head, count, bs, n_tokens, max_new, max_len):
    """Returns dict(table, lens, cu, slots, ring, state); inputs are not changed."""
    prev, target = [int(v) for v in prev], [int(v) for v in target]
    table, ring, n = np.array(table), np.array(ring), len(ring)
    blocks = lambda t: -(-t // bs)  # noqa: E731
    room = table.shape[1] * bs
    bad = not (0 <= head < n and 0 <= count <= n)
    for p, t in zip(prev, target):
        bad = bad or p < 0 or t < 0 or t > max_len or p > room or t > room or t - p > max_new
    new = [max(0, t - p) for p, t in zip(prev, target)]
    bad = bad or sum(new) > n_tokens
    lacking = -1
    if not bad:
        take = sum(max(0, blocks(t) - blocks(p)) for p, t in zip(prev, target))
        give = sum(max(0, blocks(p) - blocks(t)) for p, t in zip(prev, target))
        lacking = -1 if count + give > n else max(0, take - count)
    slots = np.full(n_tokens, -1, np.int32)
    if lacking != 0:
        return dict(table=table, lens=np.array(prev, np.int32), cu=np.zeros(len(prev) + 1, np.int32), slots=slots,
                    ring=ring, state=np.array([head, count, lacking, 0], np.int32))
    front, back = head, (head + count) % n
    cu, given = [0], []
    for i, (p, t) in enumerate(zip(prev, target)):
        for c in range(blocks(p), blocks(t)):
            table[i, c] = ring[front]
            front = (front + 1) % n
        given += [table[i, c] for c in range(blocks(t), blocks(p))]
        for k, pos in enumerate(range(p, t)):
            blk = table[i, pos // bs]
            slots[cu[-1] + k] = blk * bs + pos % bs if 0 <= blk < n else -1
        cu.append(cu[-1] + max(0, t - p))
    for k, b in enumerate(given):
        ring[(back + k) % n] = b
    return dict(table=table, lens=np.array(target, np.int32), cu=np.array(cu, np.int32), slots=slots, ring=ring,
                state=np.array([front, count - take + len(given), 0, cu[-1]], np.int32))


def append(x, slots, cu, codes, scale, fmt):
    """x: tokens x heads x d (fp32-exact values); codes: blocks x heads x bs x d uint8; scale: blocks x heads fp32.
    Returns new (codes, scale)."""
    codes, scale = codes.copy(), scale.copy()
    n_blocks, heads, bs, _ = codes.shape
    x = np.asarray(x).astype(F32)
    for a, e in zip(cu[:-1], cu[1:]):
        t = int(a)
        while t < e:
            if slots[t] < 0:
                t += 1
                continue
            blk, off = divmod(int(slots[t]), bs)
            r = 1
            while t + r < e and slots[t + r] == slots[t] + r and off + r < bs:
                r += 1
            for h in range(heads):
                rows = x[t:t + r, h]
                s_old = scale[blk, h] if off > 0 else F32(0)
                s = max(s_old, F32(np.abs(rows).max() / QMAX[fmt]))
                if s > s_old and off > 0:
                    ratio = F32(s_old / s)
                    old = values(codes[blk, h, :off], fmt).astype(F32)
                    codes[blk, h, :off] = to_codes((old * ratio).astype(F32), fmt)
                scale[blk, h] = s
                q = np.zeros_like(rows) if s == 0 else (rows / s).astype(F32)
                codes[blk, h, off:off + r] = to_codes(q, fmt)
            t += r
    return codes, scale


def gather(codes, scale, row, length, fmt):
    """A request's cached values, heads x length x d, float64; blocks outside the pool come back as NaN rows."""
    n_blocks, heads, bs, d = codes.shape
    out = np.full((heads, length, d), np.nan)
    for c in range(-(-length // bs)):
        blk, lo = int(row[c]), c * bs
        hi = min(length, lo + bs)
        if 0 <= blk < n_blocks:
            out[:, lo:hi] = values(codes[blk, :, :hi - lo], fmt) * scale[blk].astype(np.float64)[:, None, None]
    return out


def attend(q, cu, lens, table, kcodes, kscale, vcodes, vscale, fmt, causal, scale, unit=2.0 ** -8):
    """q: tokens x heads x d (float64 holding 16-bit values).  Returns (out, tol): the float64 result and, per
    value, how far a kernel may be off that rounds the weights to fp16 and the result to a type of half step `unit`:
      unit max(|out|, N)              the result's own rounding, N the type's smallest normal number
      (2^-11 + 2 dx + 2^-19) E        weights to fp16; an error dx of a score moves a weight, and the sum of the
                                      weights, by that share; exponentials and sums to 2^-20 each.  E = sum p |v|
      2^-23 (2 |log2 s_v| + |x|) E    the roundings of an exponent x + log2 s_v and of its terms (largest of each)
      T qmax F                        what is lost below fp16's normal numbers, half a step of 2^-24 for each of the T
                                      tokens that the row sees.  The step belongs to weights p s_v taken relative to a
                                      reference 2^6 below the largest one that the row sees, or lower, so F = 2^-31 max p s_v;
                                      2^-144 max p more where all s_v are below 2^-113 (the reference's lower end);
                                      2^-119 max p max s_v for weights below the smallest fp32 number
    with dx = (d 2^-23) scale max_t sum |q| |k|: fp32 products added in any order, and q's own 2^-25."""
    n, heads, d = q.shape
    kv = kcodes.shape[1]
    G = heads // kv
    out, tol = np.zeros((n, heads, d)), np.zeros((n, heads, d))
    for i in range(len(lens)):
        a, e, L = int(cu[i]), int(cu[i + 1]), int(lens[i])
        if e <= a or L <= 0:
            continue
        K, V = gather(kcodes, kscale, table[i], L, fmt), gather(vcodes, vscale, table[i], L, fmt)
        there = ~np.isnan(K[0, :, 0])
        blocks = np.repeat(table[i][:-(-L // kcodes.shape[2])].astype(np.int64), kcodes.shape[2])[:L]
        for h in range(heads):
            k, v = np.nan_to_num(K[h // G]), np.nan_to_num(V[h // G])
            s = q[a:e, h] @ k.T * scale
            seen = np.broadcast_to(there, s.shape).copy()
            if causal:
                seen &= np.arange(L)[None, :] <= L - (e - a) + np.arange(e - a)[:, None]
            s = np.where(seen, s, -np.inf)
            top = s.max(axis=1, keepdims=True)
            p = np.exp(s - np.where(np.isinf(top), 0, top))
            p /= np.maximum(p.sum(axis=1, keepdims=True), 1e-300)
            out[a:e, h] = p @ v
            dx = d * 2.0 ** -23 * abs(scale) * (np.abs(q[a:e, h]) @ np.abs(k).T).max(axis=1, keepdims=True)
            sv = np.where(there, vscale[np.where(there, blocks, 0), h // G].astype(np.float64), 0.0)
            most = lambda w: np.max(np.where(seen, w, 0.0), axis=1, keepdims=True)  # noqa: E731
            lost = 2.0 ** -31 * most(p * sv) + 2.0 ** -144 * most(p) + 2.0 ** -119 * most(p) * most(sv)
            far = 2 * most(np.abs(np.log2(np.where(sv > 0, sv, 1.0)))) + 1.45 * most(np.where(seen, np.abs(s), 0.0))
            tol[a:e, h] = unit * np.maximum(np.abs(out[a:e, h]), NORMAL[unit])
            tol[a:e, h] += (2.0 ** -11 + 2 * dx + 2.0 ** -19 + 2.0 ** -23 * far) * (p @ np.abs(v))
            tol[a:e, h] += seen.sum(axis=1, keepdims=True) * float(QMAX[fmt]) * lost
    return out, tol
