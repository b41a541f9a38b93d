"""Float64 CPU oracle for attention over a paged cache of shared latents.

TEST INFRASTRUCTURE ONLY, like the rest of this package. The operators have no
counterpart in the source pages; the functions here state their definitions.

A token's cache row is its latent l (512 values) and its rotated position part r (64),
shared by all heads. Expanded, head h has the key concat(Uk_h l, r) and the value Uv_h l;
absorbed, its query becomes concat(Uk_h^T q, q_r), its key the row itself, its value l, and
the result is mapped by Uv_h afterwards: the scores, and so the weights, are the same.

bf16 tensors are numpy ``uint16`` arrays of raw bits; all arithmetic is float64.
"""

from __future__ import annotations

import math

import numpy as np

from .paged_attention import bf16_bits_to_f64, f64_to_bf16_bits

LATENT, ROTATED = 512, 64
ROW = LATENT + ROTATED


def rotate(x, cos, sin, interleaved):
    """x [..., dims] float64, cos/sin [..., dims / 2]: every pair (a, b) becomes
    (a c - b s, b c + a s); pairs are (x_2j, x_2j+1) or (x_j, x_j+dims/2)."""
    y = np.empty_like(x)
    half = x.shape[-1] // 2
    for j in range(half):
        i0, i1 = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
        a, b, c, s = x[..., i0], x[..., i1], cos[..., j], sin[..., j]
        y[..., i0] = a * c - b * s
        y[..., i1] = b * c + a * s
    return y


def pool_row(table, slot, pos, page_size, num_pages):
    """The pool row of a position, or None where slot, position or entry is out of range."""
    if not 0 <= slot < table.shape[0]:
        return None
    block = pos // page_size
    if pos < 0 or block >= table.shape[1]:
        return None
    page = int(table[slot, block])
    return page * page_size + pos % page_size if 0 <= page < num_pages else None


def append(pool, table, x_new, slots, positions, page_size, cos, sin, interleaved=False,
           weight=None, eps=1e-6):
    """The pool (float64 values of its bf16 rows) after the new tokens' rows have been written,
    unrounded, and the indices of tokens that could not be."""
    pool = pool.copy()
    bad = []
    for i, (slot, pos) in enumerate(zip(slots.tolist(), positions.tolist())):
        if slot == 0:
            continue
        row = pool_row(table, slot, pos, page_size, pool.shape[0] // page_size)
        if row is None or pos >= cos.shape[0]:
            bad.append(i)
            continue
        x = bf16_bits_to_f64(x_new[i])
        lat = x[:LATENT]
        if weight is not None:
            lat = lat / math.sqrt(np.mean(lat * lat) + eps) * weight.astype(np.float64)
        pool[row, :LATENT] = lat
        pool[row, LATENT:] = rotate(x[LATENT:], cos[pos].astype(np.float64),
                                    sin[pos].astype(np.float64), interleaved)
    return pool, bad


def gather(pool, table, slots, starts, out, page_size):
    """``out`` (any row type like the pool's) with the sequences' rows in place."""
    out = out.copy()
    for b, slot in enumerate(slots.tolist()):
        for t in range(int(starts[b + 1]) - int(starts[b])):
            row = pool_row(table, slot, t, page_size, pool.shape[0] // page_size)
            if slot != 0 and row is not None:
                out[int(starts[b]) + t] = pool[row]
    return out


def attend(q, k, v, scale):
    """One query over n keys: (out, lse, sum_t w_t |v_t|, max_t scale sum_d |q_d k_td|), the last
    two for error bounds. No keys: zeros and -inf."""
    if len(k) == 0:
        return np.zeros(v.shape[1]), -math.inf, np.zeros(v.shape[1]), 0.0
    x = scale * (k @ q)
    m = x.max()
    w = np.exp(x - m)
    total = w.sum()
    w /= total
    return w @ v, m + math.log(total), w @ np.abs(v), scale * (np.abs(k) @ np.abs(q)).max()


def decode(q, pool, table, slots, lens, page_size, scale):
    """The absorbed form: q bits [B, n_q, H, 576]. Returns out, lse, and the two bounds of
    ``attend``, all float64 over [B, n_q, H, ...]; rows that are refused have 0 / -inf."""
    B, n_q, H, _ = q.shape
    out, mass = np.zeros((B, n_q, H, LATENT)), np.zeros((B, n_q, H, LATENT))
    lse, size = np.full((B, n_q, H), -math.inf), np.zeros((B, n_q, H))
    for b in range(B):
        slot, n = int(slots[b]), int(lens[b])
        if slot == 0 or not 0 <= slot < table.shape[0] or n < 0 or n > table.shape[1] * page_size:
            continue
        rows = [pool_row(table, slot, t, page_size, pool.shape[0] // page_size) for t in range(n)]
        c = bf16_bits_to_f64(pool[rows]) if n else np.zeros((0, ROW))
        for j in range(n_q):
            end = max(0, n - (n_q - 1 - j))
            for h in range(H):
                out[b, j, h], lse[b, j, h], mass[b, j, h], size[b, j, h] = attend(
                    bf16_bits_to_f64(q[b, j, h]), c[:end], c[:end, :LATENT], scale)
    return out, lse, mass, size


def prefill(q, k_own, k_rot, v, q_starts, k_starts, scale):
    """The expanded form: query i of the n of a sequence with m keys sees keys 0 .. m - n + i.
    Bits q [Tq, H, 192], k_own [Tk, H, 128], k_rot [Tk, 64], v [Tk, H, 128]. Results as
    ``decode``; queries of no sequence stay 0 / -inf."""
    Tq, H, _ = q.shape
    dv = v.shape[2]
    out, mass = np.zeros((Tq, H, dv)), np.zeros((Tq, H, dv))
    lse, size = np.full((Tq, H), -math.inf), np.zeros((Tq, H))
    for s in range(len(q_starts) - 1):
        q0, q1, k0, k1 = (int(x) for x in (q_starts[s], q_starts[s + 1], k_starts[s], k_starts[s + 1]))
        for h in range(H):
            k = np.concatenate([bf16_bits_to_f64(k_own[k0:k1, h]), bf16_bits_to_f64(k_rot[k0:k1])], 1)
            vv = bf16_bits_to_f64(v[k0:k1, h])
            for i in range(q1 - q0):
                end = max(0, (k1 - k0) - (q1 - q0) + i + 1)
                out[q0 + i, h], lse[q0 + i, h], mass[q0 + i, h], size[q0 + i, h] = attend(
                    bf16_bits_to_f64(q[q0 + i, h]), k[:end], vv[:end], scale)
    return out, lse, mass, size


__all__ = ["LATENT", "ROTATED", "ROW", "rotate", "pool_row", "append", "gather", "attend", "decode",
           "prefill", "bf16_bits_to_f64", "f64_to_bf16_bits"]
