"""Inputs and the oracle's results for the tests of the drafted-token and page
operators."""

from __future__ import annotations

import math
from types import SimpleNamespace

import numpy as np
import torch

import oracle.speculative as spec
from paged_kv_gqa_pkv_gb300.workloads import bf16_bits


def rand_parents(rng, B, N, shape="random"):
    p = np.full((B, N), -1, dtype=np.int32)
    for b in range(B):
        for j in range(1, N):
            if shape == "chain":
                p[b, j] = j - 1
            elif shape == "star":
                p[b, j] = 0
            elif shape == "forest":
                p[b, j] = rng.integers(-1, j)
            else:
                p[b, j] = rng.integers(0, j)
    return p


def tree_case(seed, ctx, tree, N, hq=8, hkv=2, ps=16, shape="random", pad=(), fill=float("nan"),
              spare=3):
    """Row b: ctx[b] committed tokens and a tree of tree[b] of N nodes, on
    permuted pages; everything else in the pools is `fill`. Rows in `pad` are
    padding (slot 0)."""
    rng = np.random.default_rng(seed)
    B = len(ctx)
    blocks = [-(-(c + t) // ps) for c, t in zip(ctx, tree)]
    cols = max(max(blocks), 1) + 1
    pages = sum(blocks) + 1 + spare
    order = rng.permutation(np.arange(1, pages))
    table = np.full((B + 2, cols), -1, dtype=np.int32)
    k = np.full((pages * ps, hkv, 128), fill, dtype=np.float32)
    v = k.copy()
    at = 0
    for b in range(B):
        mine = order[at:at + blocks[b]]
        at += blocks[b]
        table[b + 1, :blocks[b]] = mine
        t = np.arange(ctx[b] + tree[b])
        rows = mine[t // ps] * ps + t % ps if len(t) else t
        k[rows] = rng.standard_normal((len(t), hkv, 128))
        v[rows] = rng.standard_normal((len(t), hkv, 128))
    slots = np.arange(1, B + 1, dtype=np.int32)
    slots[list(pad)] = 0
    q = torch.from_numpy(rng.standard_normal((B, N, hq, 128)).astype(np.float32)).bfloat16()
    return SimpleNamespace(
        k=torch.from_numpy(k).bfloat16(), v=torch.from_numpy(v).bfloat16(), table=table, q=q,
        parents=rand_parents(rng, B, N, shape), lens=np.array(tree, dtype=np.int32), slots=slots,
        ctx=np.array(ctx, dtype=np.int32), ps=ps, scale=1 / math.sqrt(128))


def tree_oracle(c):
    return spec.tree_attention(bf16_bits(c.q), bf16_bits(c.k), bf16_bits(c.v), c.table, c.parents,
                               c.lens, c.slots, c.ctx, c.ps, c.scale)


def verify_case(seed, B, N, V, draft=True, kind=torch.float32, shape="random", spread=2.5,
                tree=None):
    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    parents = rand_parents(rng, B, N, shape)
    logits = torch.randn((B, N, V), generator=g) * spread
    target = torch.softmax(logits + 0.7 * torch.randn((B, N, V), generator=g), -1).to(kind)
    probs = torch.softmax(logits, -1)
    tokens = torch.zeros((B, N), dtype=torch.int32)
    for b in range(B):
        for j in range(1, N):
            tokens[b, j] = torch.multinomial(probs[b, max(int(parents[b, j]), 0)], 1, generator=g)
    lens = np.array(tree if tree is not None else rng.integers(1, N + 1, B), dtype=np.int32)
    return SimpleNamespace(
        target=target, draft=probs.to(kind) if draft else None, tokens=tokens, parents=parents,
        lens=lens, u=torch.rand((B, N), generator=g), us=torch.rand((B,), generator=g))


def verify_oracle(c):
    f = lambda t: None if t is None else t.to(torch.float64).numpy()  # noqa: E731
    return spec.verify_tree(f(c.target), f(c.draft), c.tokens.numpy(), c.parents, c.lens,
                            c.u.numpy(), c.us.numpy())


def pool_bits(rng, rows, hkv):
    """Pools of random bit patterns (copies are compared bit for bit)."""
    return [rng.integers(0, 1 << 16, (rows, hkv, 128)).astype(np.uint16) for _ in range(2)]


def from_bits(bits):
    return torch.from_numpy(bits.view(np.int16).copy()).view(torch.bfloat16)


def pages_state(seed, lens, ps, hkv, pages, cols, slots=None, share=()):
    """Slots 1.. hold lens[i] tokens on random pages; `share` lists (slot, of)
    pairs: slot shares every page of slot `of`."""
    rng = np.random.default_rng(seed)
    slots = slots or len(lens) + 1
    order = rng.permutation(np.arange(1, pages))
    table = np.full((slots, cols), -1, dtype=np.int32)
    refs = np.zeros(pages, dtype=np.int32)
    refs[0] = 1
    at = 0
    for i, n in enumerate(lens):
        m = -(-n // ps)
        table[i + 1, :m] = order[at:at + m]
        at += m
    for a, of in share:
        table[a] = table[of]
    for e in table.flatten():
        if e > 0:
            refs[e] += 1
    k, v = pool_bits(rng, pages * ps, hkv)
    return SimpleNamespace(k=k, v=v, table=table, refs=refs, ps=ps)
