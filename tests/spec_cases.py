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


def tree_rows(c, rows):
    """Batch rows `rows` of a case without errors, from the definition in 64 bits,
    whole products at a time: per row (out, lse, A, e) of its live nodes with
    A = sum_t w_t |V[t]|, what an error of the weights relative to themselves moves
    the output by, and e = max_t sum_d |scale q_d K[t]_d|, what rounding errors of the
    scores are relative to."""
    from oracle.paged_attention import bf16_bits_to_f64
    res = []
    for b in rows:
        ctx, n = int(c.ctx[b]), int(c.lens[b])
        t = np.arange(ctx + n)
        at = torch.from_numpy(c.table[int(c.slots[b])][t // c.ps].astype(np.int64) * c.ps + t % c.ps)
        f64 = lambda x: bf16_bits_to_f64(bf16_bits(x))  # noqa: E731
        k, v, q = f64(c.k[at]), f64(c.v[at]), f64(c.q[b, :n])
        sees = np.zeros((n, 1, ctx + n), dtype=bool)
        sees[:, :, :ctx] = True
        for i, kin in enumerate(spec.ancestors(c.parents[b], n)):
            sees[i, 0, [ctx + a for a in kin]] = True
        group = q.shape[1] // k.shape[1]
        out, lse, mass, size = (np.zeros(s) for s in (q.shape, q.shape[:2], q.shape, q.shape[:2]))
        for h in range(k.shape[1]):
            of = slice(h * group, (h + 1) * group)
            x = np.where(sees, c.scale * (q[:, of] @ k[:, h].T), -np.inf)
            m = x.max(-1, keepdims=True)
            w = np.exp(x - m)
            l = w.sum(-1, keepdims=True)
            out[:, of], mass[:, of] = w / l @ v[:, h], w / l @ np.abs(v[:, h])
            lse[:, of] = (m + np.log(l))[..., 0]
            size[:, of] = np.where(sees, c.scale * (np.abs(q[:, of]) @ np.abs(k[:, h]).T), 0).max(-1)
        res.append((out, lse, mass, size))
    return res


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


class Mirror:
    """A cache on the GPU and the oracle's copy of it, driven by the same
    calls. ``equal`` compares every byte of pools, table, counts and lengths."""

    def __init__(self, seed, lens, ps, hkv, pages, cols, slots):
        from paged_kv_gqa_pkv_gb300 import binding
        self.b, self.ps = binding, ps
        self.host = pages_state(seed, lens, ps, hkv, pages, cols, slots=slots)
        rng = np.random.default_rng(seed + 1)
        shape = self.host.k.shape
        self.host.k, self.host.v = (bf16_bits(torch.from_numpy(
            rng.standard_normal(shape).astype(np.float32)).bfloat16()) for _ in range(2))
        self.lens = np.zeros(slots, dtype=np.int32)
        self.lens[1:len(lens) + 1] = lens
        h = self.host
        self.k, self.v = from_bits(h.k).cuda(), from_bits(h.v).cuda()
        self.table, self.refs = torch.from_numpy(h.table.copy()).cuda(), torch.from_numpy(h.refs).cuda()
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def i32(self, x):
        return torch.from_numpy(np.array(x, dtype=np.int32)).cuda()

    def update(self, dst, src, keep, new):
        h = self.host
        self.b.pkv_update_pages(self.k, self.v, self.table, self.refs, self.i32(dst), self.i32(src),
                                self.i32(keep), self.i32(new), self.ps, dev_err=self.err)
        h.k, h.v, h.table, h.refs, err = spec.update_pages(h.k, h.v, h.table, h.refs, dst, src, keep,
                                                           new, self.ps)
        assert err == 0

    def append(self, k_new, v_new, slots, pos):
        import oracle.paged_attention as orc
        h = self.host
        self.b.pkv_append(self.k, self.v, self.table, k_new.cuda(), v_new.cuda(), self.i32(slots),
                          self.i32(pos), self.ps, dev_err=self.err)
        h.k, h.v, bad = orc.append(h.k, h.v, h.table, bf16_bits(k_new), bf16_bits(v_new),
                                   np.array(slots), np.array(pos), self.ps)
        assert not bad

    def compact(self):
        h = self.host
        n = self.b.pkv_compact_pages(self.k, self.v, self.table, self.refs, self.ps,
                                     dev_err=self.err)
        h.k, h.v, h.table, h.refs, want, err = spec.compact_pages(h.k, h.v, h.table, h.refs, self.ps)
        assert err == 0 and int(n.item()) == want
        return want

    def equal(self):
        torch.cuda.synchronize()
        h = self.host
        assert int(self.err.item()) == 0
        assert np.array_equal(self.table.cpu().numpy(), h.table)
        assert np.array_equal(self.refs.cpu().numpy(), h.refs)
        assert np.array_equal(bf16_bits(self.k.cpu()), h.k)
        assert np.array_equal(bf16_bits(self.v.cpu()), h.v)


def draft_step(m, rng, slots, N, hq, V, shape="random"):
    """One step of drafting on the mirror: pages for N nodes, their K/V, tree
    attention, verification against probabilities made from the attention's
    (rounded) output, the accepted path, and the rest given back. Each result
    is compared with the oracle's. Returns the attention's largest error."""
    from tests.parity import assert_attention_close
    B, hkv = len(slots), m.k.shape[1]
    ctx = m.lens[slots].copy()
    m.update(slots, slots, ctx, ctx + N)
    parents = rand_parents(rng, B, N, shape)
    tree = rng.integers(1, N + 1, B).astype(np.int32)
    rows = [(b, a) for b in range(B) for a in range(tree[b])]
    new = lambda: torch.from_numpy(rng.standard_normal(  # noqa: E731
        (len(rows), hkv, 128)).astype(np.float32)).bfloat16()
    m.append(new(), new(), [slots[b] for b, _ in rows], [ctx[b] + a for b, a in rows])
    q = torch.from_numpy(rng.standard_normal((B, N, hq, 128)).astype(np.float32)).bfloat16()
    i32 = m.i32
    par, ln, sl, cx = i32(parents), i32(tree), i32(slots), i32(ctx)
    scale = 1 / math.sqrt(128)
    out, lse = m.b.pkv_tree_attention(m.k, m.v, m.table, q.cuda(), par, ln, sl, cx, m.ps, scale,
                                      dev_err=m.err)
    ro, rl, err, _ = spec.tree_attention(bf16_bits(q), m.host.k, m.host.v, m.host.table, parents,
                                         tree, slots, ctx, m.ps, scale)
    assert err == 0
    worst = assert_attention_close(out.cpu(), lse.cpu(), ro, rl, tag="step")[0]
    # the same bits go to both sides from here
    head = torch.from_numpy(rng.standard_normal((hq * 128, V)).astype(np.float32) * 0.05).cuda()
    target = torch.softmax(out.float().view(B, N, -1) @ head, -1)
    draft = torch.softmax(torch.log(target) +
                          torch.from_numpy(rng.standard_normal((B, N, V)).astype(np.float32)).cuda(),
                          -1)
    tokens = torch.from_numpy(rng.integers(0, V, (B, N)).astype(np.int32)).cuda()
    u, us = (torch.from_numpy(rng.random(s).astype(np.float32)).cuda() for s in ((B, N), (B,)))
    path, toks, n = m.b.pkv_verify_tree(target, tokens, par, ln, u, us, draft_probs=draft,
                                        dev_err=m.err)
    f = lambda t: t.double().cpu().numpy()  # noqa: E731
    want = spec.verify_tree(f(target), f(draft), tokens.cpu().numpy(), parents, tree,
                            f(u), f(us))
    for g, w in zip((path, toks, n), want):
        assert np.array_equal(g.cpu().numpy(), w)
    lens = m.b.pkv_commit_path(m.k, m.v, m.table, path, n, sl, cx, m.ps, dev_err=m.err)
    h = m.host
    h.k, h.v, new_lens, err = spec.commit_path(h.k, h.v, h.table, want[0], want[2], slots, ctx, m.ps)
    assert err == 0 and np.array_equal(lens.cpu().numpy(), new_lens)
    m.lens[slots] = new_lens
    m.update(slots, slots, new_lens, new_lens)   # pages past the accepted tokens go back
    m.equal()
    return worst
