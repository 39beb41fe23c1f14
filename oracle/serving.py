"""Oracle of the serving operators beside the INT4 cache, in numpy: rotary positions (the table in
fp64, the rotation in single fp32 operations), decode attention in fp64 over a shared prefix and own
tokens with every token's weight, and eviction by accumulated weight.  Written from the definitions;
it shares no code with the product path."""
from __future__ import annotations

import math

import numpy as np

from . import f16_bits_to_f64, rotate_f64

PAGE = 16


# ---- rotary positions ---------------------------------------------------------------------------

def rope_table_fp64(first, count, rotary, kind="none", base=10000.0, factor=1.0, original=8192,
                    low=1.0, high=4.0, fast=32.0, slow=1.0, amplitude=0.0) -> np.ndarray:
    """fp64 [count][rotary]: cosines, then sines, of positions first .. first + count - 1."""
    freq = []
    if kind == "ntk":
        base = base * factor ** (rotary / (rotary - 2))
    edge = [rotary * math.log(original / (2 * math.pi * b)) / (2 * math.log(base)) for b in (fast, slow)]
    lo, hi = max(0, math.floor(edge[0])), min(rotary - 1, math.ceil(edge[1]))
    for i in range(rotary // 2):
        f = base ** (-2.0 * i / rotary)
        if kind == "linear":
            f = f / factor
        elif kind == "banded":
            wavelength = 2 * math.pi / f
            if original / wavelength <= low:
                f = f / factor
            elif original / wavelength < high:
                t = (original / wavelength - low) / (high - low)
                f = (1 - t) * f / factor + t * f
        elif kind == "yarn":
            t = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            f = f / factor * t + f * (1 - t)
        freq.append(f)
    if amplitude == 0.0:
        amplitude = 0.1 * math.log(factor) + 1.0 if kind == "yarn" else 1.0
    angle = np.arange(first, first + count, dtype=np.float64)[:, None] * np.array(freq)[None]
    return amplitude * np.concatenate([np.cos(angle), np.sin(angle)], 1)


def bf16_to_f32(bits: np.ndarray) -> np.ndarray:
    return (bits.astype(np.uint32) << 16).view(np.float32)


def f32_to_bf16(x: np.ndarray) -> np.ndarray:
    """Round to nearest, ties to even (finite values)."""
    u = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def rope_bf16(x_bits: np.ndarray, positions: np.ndarray, table: np.ndarray, interleaved: bool) -> np.ndarray:
    """Rotate bf16 head vectors [T][heads][D] by the rows of the fp32 table; bf16 bits out."""
    rotary = table.shape[1]
    half = rotary // 2
    x = bf16_to_f32(x_bits)
    out = x_bits.copy()
    first = np.arange(0, rotary, 2) if interleaved else np.arange(half)
    second = first + 1 if interleaved else first + half
    for t in range(x.shape[0]):
        c, s = table[positions[t], :half], table[positions[t], half:]
        a, b = x[t][:, first], x[t][:, second]
        out[t][:, first] = f32_to_bf16(a * c - b * s)
        out[t][:, second] = f32_to_bf16(b * c + a * s)
    return out


# ---- attention ------------------------------------------------------------------------------------

_F16 = None


def _f16(bits):
    global _F16
    if _F16 is None:
        _F16 = np.array([f16_bits_to_f64(i) for i in range(1 << 16)])
    return _F16[bits]


def rows_fp64(kv_pages, scales, table, n, h, sel) -> np.ndarray:
    """The first n cached vectors (K: sel 0, V: sel 1) of kv head h in the pages of `table`, as
    stored (not rotated back): fp64 [n][D]."""
    t = np.arange(n)
    page, off = np.asarray(table)[t // PAGE], t % PAGE
    packed = kv_pages[page, h, sel, off]
    pair = _f16(scales[page, h, sel, off])
    out = np.empty((n, 2 * kv_pages.shape[-1]))
    out[:, 0::2] = pair[:, 1:] + (packed & 15) * pair[:, :1]
    out[:, 1::2] = pair[:, 1:] + (packed >> 4) * pair[:, :1]
    return out


def decode_rows_fp64(q_bits, kv_pages, scales, parts, *, sm_scale=None, rotate=True):
    """fp64 decode: sequence s attends over the concatenation of its parts[s] = [(page list, tokens),
    ...].  Returns (out [S][Hq][D]; weights[s][h], fp64 [tokens], summed over the query heads of kv
    head h; terms [S][Hkv], a bound on the sum of the magnitudes that make up one logit)."""
    S, Hq, D = q_bits.shape
    Hkv = kv_pages.shape[1]
    G = Hq // Hkv
    sm_scale = 1.0 / math.sqrt(D) if sm_scale is None else sm_scale
    q = bf16_to_f32(q_bits).astype(np.float64)
    if rotate:
        q = rotate_f64(q)
    out = np.zeros((S, Hq, D))
    weights = [[None] * Hkv for _ in range(S)]
    terms = np.zeros((S, Hkv))
    for s in range(S):
        for h in range(Hkv):
            k = np.concatenate([rows_fp64(kv_pages, scales, t, n, h, 0) for t, n in parts[s]])
            v = np.concatenate([rows_fp64(kv_pages, scales, t, n, h, 1) for t, n in parts[s]])
            weights[s][h] = np.zeros(len(k))
            if not len(k):
                continue
            qs = q[s, h * G:(h + 1) * G]
            logits = sm_scale * qs @ k.T
            w = np.exp(logits - logits.max(1, keepdims=True))
            w /= w.sum(1, keepdims=True)
            out[s, h * G:(h + 1) * G] = w @ v
            weights[s][h] = w.sum(0)
            # |q_d| (15 |scale| + |zero|) summed over d, at most: the magnitudes of one logit's terms
            big = 0.0
            for table, n in parts[s]:
                t = np.arange(n)
                pair = np.abs(_f16(scales[np.asarray(table)[t // PAGE], h, 0, t % PAGE]))
                big = max(big, (15 * pair[:, 0] + pair[:, 1]).max(initial=0.0))
            terms[s, h] = sm_scale * np.abs(qs).sum(1).max() * big
    if rotate:
        out = rotate_f64(out)
    return out, weights, terms


# ---- eviction -------------------------------------------------------------------------------------

def evict(kv_pages, scales, mass, block_table, seq_lens, new_table, keep, sink, recent):
    """Evict in place (numpy copies of the cache): returns (new_lens, kept)."""
    S, Hkv = len(seq_lens), kv_pages.shape[1]
    new_lens = np.zeros(S, np.int32)
    kept = np.full((S, Hkv, keep), -1, np.int32)
    moves = []
    for s in range(S):
        L = int(seq_lens[s])
        new_lens[s] = min(L, keep)
        for h in range(Hkv):
            if L <= keep:
                chosen = list(range(L))
            else:
                middle = [(-float(m) if m > 0 else 0.0, t) for t in range(sink, L - recent)
                          for m in [mass[block_table[s, t // PAGE], h, t % PAGE]]]
                chosen = sorted(list(range(sink)) + [t for _, t in sorted(middle)[:keep - sink - recent]] +
                                list(range(L - recent, L)))
            kept[s, h, :len(chosen)] = chosen
            for j, t in enumerate(chosen):
                moves.append((block_table[s, t // PAGE], h, t % PAGE, new_table[s, j // PAGE], j % PAGE))
    old = kv_pages.copy(), scales.copy(), mass.copy()
    for page, h, off, to, to_off in moves:
        kv_pages[to, h, :, to_off] = old[0][page, h, :, off]
        scales[to, h, :, to_off] = old[1][page, h, :, off]
        mass[to, h, to_off] = old[2][page, h, off]
    return new_lens, kept
