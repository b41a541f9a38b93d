"""Inputs and error bounds for the tests of the operators of shared latents."""

from __future__ import annotations

import math

import numpy as np
import torch

import oracle.latent as orl
from paged_kv_gqa_pkv_gb300.workloads import bf16_bits

SCALE = 1 / math.sqrt(192)


def gen(seed):
    return torch.Generator().manual_seed(seed)


def normal(g, *shape, scale=1.0):
    return (torch.randn(shape, generator=g) * scale).to(torch.bfloat16)


def i32(values):
    return torch.as_tensor(values, dtype=torch.int32)


def rope_tables(rows, dims, base=10000.0):
    f = base ** (-torch.arange(0, dims, 2, dtype=torch.float64) / dims)
    a = torch.arange(rows, dtype=torch.float64)[:, None] * f
    return torch.cos(a).float(), torch.sin(a).float()


def cache(g, slots, longest, ps, spare=2, marker=None):
    """A pool and a permuted table of `slots` slots (from 1 on) with room for `longest` tokens each;
    slot 0 and page 0 reserved, the rest of the table -1. `marker` fills the pages of no slot."""
    blocks = -(-longest // ps)
    pages = 1 + slots * blocks + spare
    pool = normal(g, pages * ps, orl.ROW)
    order = torch.randperm(pages - 1, generator=g) + 1
    table = torch.full((slots + 1, blocks + 1), -1, dtype=torch.int32)
    table[1:, :blocks] = order[:slots * blocks].to(torch.int32).view(slots, blocks)
    if marker is not None:
        for p in [0, *order[slots * blocks:].tolist()]:
            pool[p * ps:(p + 1) * ps] = marker
    return pool, table


def attention_bounds(out, lse, mass, size, dims):
    """Bounds on a kernel's out and lse from the definition's values.

    Scores: products of bf16 values are exact in fp32, and each of the `dims` additions loses at
    most 2^-23 of the running sum's bound, so a score is off by at most e = dims 2^-23 size (size =
    scale sum_d |q_d k_d|), plus 2^-22 of it for the scaling. That moves a weight by a factor within
    1 +- 2 (2 e) (numerator and sum). A weight's rounding to bf16 and the result's: 2^-8 each. The
    exponentials, sums and the division in fp32: 2^-16 covers 2^8 roundings."""
    e = (dims * 2.0 ** -23 + 2.0 ** -22) * size
    tol_out = (2.0 ** -8 + 4 * e[..., None] + 2.0 ** -16) * mass + 2.0 ** -8 * np.abs(out) * (1 + 2.0 ** -7) + 1e-30
    tol_lse = e + 2.0 ** -16 + 2.0 ** -22 * np.abs(np.where(np.isinf(lse), 0, lse))
    return tol_out, tol_lse


def check_attention(out_gpu, lse_gpu, want, dims, tag=""):
    """out_gpu, lse_gpu: CPU tensors; want: the oracle's (out, lse, mass, size)."""
    out, lse, mass, size = want
    o, l = out_gpu.double().numpy(), lse_gpu.double().numpy()
    none = np.isneginf(lse)
    assert np.array_equal(np.isneginf(l), none), f"{tag}: rows without keys differ"
    assert not np.isnan(o).any() and not np.isnan(l).any(), f"{tag}: NaN"
    assert (o[none] == 0).all(), f"{tag}: rows without keys are not 0"
    tol_out, tol_lse = attention_bounds(out, lse, mass, size, dims)
    worst = (np.abs(o - out) / tol_out).max() if o.size else 0.0
    assert worst <= 1, f"{tag}: out {worst:.3g} times the bound"
    live = ~none
    if live.any():
        worst = (np.abs(l[live] - lse[live]) / tol_lse[live]).max()
        assert worst <= 1, f"{tag}: lse {worst:.3g} times the bound"


def attend_beside(q, k, v, end, scale, at, place):
    """What one query has to give that sees the keys before `end` of k, of which key `at` holds a
    value that is not finite at k[at, place[0]] and v[at, place[1]] (None: not there): the oracle's
    tuple, with NaN everywhere where the key's score is NaN or +inf, and with the value's product with
    the key's weight (NaN if that is 0) in its place of out."""
    n = v.shape[1]
    if at >= end:
        return orl.attend(q, k[:end], v[:end], scale)
    with np.errstate(invalid="ignore"):
        x = 0.0 if place[0] is None else q[place[0]] * k[at, place[0]]
    if not x < math.inf:
        return np.full(n, math.nan), math.nan, np.zeros(n), 0.0
    finite = v.copy()
    if place[1] is not None:
        finite[at, place[1]] = 0
    keep = [t for t in range(end) if t != at or x != -math.inf]
    out, lse, mass, size = orl.attend(q, k[keep], finite[keep], scale)
    if place[1] is not None:
        out[place[1]] = math.nan if x == -math.inf else v[at, place[1]]
    return out, lse, mass, size


def check_beside(out, lse, want, dims, free, tag=""):
    """out [n, d], lse [n] of a kernel against the rows of attend_beside. free: [n, d], values that may
    be anything (of queries that do not see the key, where the products meet what it holds)."""
    o, l = out.double().numpy().copy(), lse.double().numpy().copy()
    w = [np.stack([np.asarray(r[i]) for r in want]) for i in range(4)]
    o[free] = w[0][free] = 0
    none, odd = np.isnan(w[1]), ~np.isfinite(w[0])
    assert np.array_equal(np.isnan(l), none), f"{tag}: lse is NaN at the wrong places"
    assert np.array_equal(o[odd], w[0][odd], equal_nan=True), f"{tag}: out's values that are not finite"
    o[odd] = w[0][odd] = 0
    if not none.all():
        check_attention(torch.from_numpy(o[~none]), torch.from_numpy(l[~none]), [a[~none] for a in w], dims, tag)


def bits(t):
    return bf16_bits(t)
