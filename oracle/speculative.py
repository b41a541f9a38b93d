"""CPU oracle of the operators for drafted tokens and for the pages of a cache:
tree attention, verification, the commit of an accepted path, page updates and
pool compaction.

TEST INFRASTRUCTURE ONLY, like the rest of this package: plain loops over the
definitions, numpy float64 for every number, bf16 as raw ``uint16`` patterns.
The source pages have no counterpart of these operators; their definitions
are the comments of the entry points in ``include/pkv.h``.
"""

from __future__ import annotations

import math

import numpy as np

from .paged_attention import bf16_bits_to_f64, physical_slot

BAD_PAGE, BAD_SLOT, BAD_POS, BAD_TREE, NO_PAGES, BAD_PROBS = 0x1, 0x2, 0x4, 0x20, 0x40, 0x80


def ancestors(parents, n):
    """Per node the set of itself and its ancestors, or None for a node that has
    an invalid parent on its way up. ``parents[i]`` is valid in [-1, i)."""
    out = []
    for i in range(n):
        up = int(parents[i])
        if up < -1 or up >= i or (up >= 0 and out[up] is None):
            out.append(None)
        else:
            out.append({i} | (out[up] if up >= 0 else set()))
    return out


def tree_attention(q_bits, k_pool, v_pool, page_table, parents, tree_lens, batch_idx, ctx_lens,
                   page_size, scale):
    """(out f64 [B, N, Hq, D], lse f64 [B, N, Hq], error bits, rows left
    unspecified by a bad page entry)."""
    B, N, hq, d = q_bits.shape
    hkv = k_pool.shape[1]
    num_pages = k_pool.shape[0] // page_size
    out = np.zeros((B, N, hq, d))
    lse = np.full((B, N, hq), -np.inf)
    err, unspecified = 0, []
    for b in range(B):
        slot, ctx, n = int(batch_idx[b]), int(ctx_lens[b]), int(tree_lens[b])
        if slot == 0:
            continue
        if slot < 0 or slot >= page_table.shape[0]:
            err |= BAD_SLOT
            continue
        if n < 0 or n > N:
            err |= BAD_TREE
            continue
        if ctx < 0 or ctx + n > page_table.shape[1] * page_size:
            err |= BAD_POS
            continue
        if n == 0:
            continue
        rows = [physical_slot(page_table, slot, t, page_size, num_pages) for t in range(ctx + n)]
        if any(r is None for r in rows):
            err |= BAD_PAGE
            unspecified.append(b)
            continue
        k, v = bf16_bits_to_f64(k_pool[rows]), bf16_bits_to_f64(v_pool[rows])
        kin = ancestors(parents[b], n)
        for i in range(n):
            if kin[i] is None:
                err |= BAD_TREE
                continue
            seen = list(range(ctx)) + [ctx + a for a in sorted(kin[i])]
            qi = bf16_bits_to_f64(q_bits[b, i])
            for h in range(hq):
                x = scale * (k[seen, h // (hq // hkv)] @ qi[h])
                m = x.max()
                w = np.exp(x - m)
                out[b, i, h] = (w / w.sum()) @ v[seen, h // (hq // hkv)]
                lse[b, i, h] = m + math.log(w.sum())
    return out, lse, err, unspecified


def verify_tree(target, draft, draft_tokens, parents, tree_lens, u_accept, u_sample):
    """target, draft (or None): float64 [B, N, V]. Returns (path, tokens,
    n_accepted, error bits)."""
    B, N, V = target.shape
    path = np.full((B, N), -1, dtype=np.int32)
    tokens = np.full((B, N), -1, dtype=np.int32)
    count = np.zeros(B, dtype=np.int32)
    err = 0
    clean = lambda x: np.where(x > 0, x, 0.0)  # noqa: E731  (negative and NaN count as 0)
    for b in range(B):
        n = int(tree_lens[b])
        if n < 0 or n > N:
            err |= BAD_TREE
            continue
        if n == 0:
            continue
        ok = [True] * n
        for i in range(1, n):
            bad = not -1 <= parents[b, i] < i or not 0 <= draft_tokens[b, i] < V
            if bad:
                err |= BAD_TREE
            ok[i] = not bad and parents[b, i] >= 0
        cur, walked = 0, [0]
        while True:
            p = clean(target[b, cur])
            r, mass = p.copy(), 1.0
            for x in range(1, n):
                if not ok[x] or parents[b, x] != cur:
                    continue
                tok = int(draft_tokens[b, x])
                q_tok = 1.0 if draft is None else float(clean(draft[b, cur, tok]))
                if float(u_accept[b, x]) * q_tok * mass < r[tok]:
                    cur = x
                    walked.append(x)
                    break
                if draft is None:
                    mass = max(mass - r[tok], 0.0)
                    r[tok] = 0.0
                else:
                    r = clean(r - mass * clean(draft[b, cur]))
                    mass = r.sum()
            else:
                break
        if not r.sum() > 0:
            r = p
        total = np.cumsum(r)
        if not (total[-1] > 0 and np.isfinite(total[-1])):
            err |= BAD_PROBS
            drawn = -1
        else:
            at = np.nonzero((total > float(u_sample[b]) * total[-1]) & (r > 0))[0]
            drawn = int(at[0]) if len(at) else int(np.nonzero(r > 0)[0][-1])
        count[b] = len(walked)
        path[b, :len(walked)] = walked
        tokens[b, :len(walked)] = [draft_tokens[b, x] for x in walked[1:]] + [drawn]
    return path, tokens, count, err


def commit_path(k_pool, v_pool, page_table, path, n_accepted, batch_idx, ctx_lens, page_size):
    """(k_pool, v_pool, new_lens, error bits); the pools are copies."""
    k, v = k_pool.copy(), v_pool.copy()
    num_pages = k.shape[0] // page_size
    new = np.array(ctx_lens, dtype=np.int32).copy()
    err = 0
    for b in range(path.shape[0]):
        slot, ctx, n = int(batch_idx[b]), int(ctx_lens[b]), int(n_accepted[b])
        if slot == 0:
            continue
        if slot < 0 or slot >= page_table.shape[0]:
            err |= BAD_SLOT
            continue
        if n < 0 or n > path.shape[1]:
            err |= BAD_TREE
            continue
        if ctx < 0:
            err |= BAD_POS
            continue
        nodes = [int(a) for a in path[b, :n]]
        bad = 0
        moves = []
        for i, a in enumerate(nodes):
            if not 0 <= a < path.shape[1] or (i > 0 and nodes[i - 1] >= a):
                bad |= BAD_TREE
            elif ctx + a >= page_table.shape[1] * page_size:
                bad |= BAD_POS
            elif a != i:
                src = physical_slot(page_table, slot, ctx + a, page_size, num_pages)
                dst = physical_slot(page_table, slot, ctx + i, page_size, num_pages)
                if src is None or dst is None:
                    bad |= BAD_PAGE
                moves.append((src, dst))
        if bad:
            err |= bad
            continue
        for pool, old in ((k, k.copy()), (v, v.copy())):
            for src, dst in moves:
                pool[dst] = old[src]
        new[b] = ctx + n
    return k, v, new, err


def update_pages(k_pool, v_pool, page_table, refs, dst_slots, src_slots, keep_lens, new_lens,
                 page_size):
    """(k_pool, v_pool, page_table, refs, error bits); all copies."""
    k, v, table, count = k_pool.copy(), v_pool.copy(), page_table.copy(), refs.copy()
    num_pages = len(refs)
    max_batch, max_blocks = page_table.shape
    free = [p for p in range(1, num_pages) if refs[p] == 0]
    err, wanted = 0, 0
    real = lambda e: 1 <= e < num_pages  # noqa: E731
    blocks = lambda n: -(-n // page_size)  # noqa: E731
    for i, (d, s, keep, new) in enumerate(zip(*(map(int, x) for x in (dst_slots, src_slots,
                                                                      keep_lens, new_lens)))):
        if d == 0:
            continue
        if not 0 < d < max_batch or not 0 <= s < max_batch or (s == 0 and keep > 0):
            err |= BAD_SLOT
            continue
        if keep < 0 or new < keep or blocks(new) > max_blocks:
            err |= BAD_POS
            continue
        others = [int(x) for j, x in enumerate(dst_slots) if j != i]
        if d in [int(x) for x in dst_slots[:i]] or (s != d and keep > 0 and s in others):
            err |= BAD_SLOT
            continue
        old = [int(e) for e in page_table[d]]
        src = [int(e) for e in page_table[s]]
        if any(real(e) and refs[e] < 1 for e in old) or any(
                not real(src[j]) or refs[src[j]] < 1 for j in range(blocks(keep))):
            err |= BAD_PAGE
            continue
        own = lambda j: s == d and real(old[j]) and refs[old[j]] == 1  # noqa: E731
        fresh = [j for j in range(keep // page_size, blocks(new)) if new > keep and not own(j)]
        wanted += len(fresh)
        if fresh and wanted > len(free):
            err |= NO_PAGES
            continue
        pages = free[wanted - len(fresh):wanted]
        now = []
        for j in range(max_blocks):
            if j in fresh:
                now.append(pages[fresh.index(j)])
            elif j < blocks(keep):
                now.append(src[j])
            elif j < blocks(new) and s == d:
                now.append(old[j])
            else:
                now.append(-1)
        if keep % page_size and keep // page_size in fresh:
            for pool, was in ((k, k_pool), (v, v_pool)):
                a, z = now[keep // page_size] * page_size, src[keep // page_size] * page_size
                pool[a:a + keep % page_size] = was[z:z + keep % page_size]
        for j in range(max_blocks):
            if s == d and now[j] == old[j]:
                continue
            if real(old[j]):
                count[old[j]] -= 1
            if now[j] >= 0:
                count[now[j]] += 1
            table[d, j] = now[j]
    return k, v, table, count, err


def compact_pages(k_pool, v_pool, page_table, refs, page_size):
    """(k_pool, v_pool, page_table, refs, number of live pages, error bits)."""
    k, v, table, count = k_pool.copy(), v_pool.copy(), page_table.copy(), refs.copy()
    num_pages = len(refs)
    live = [p for p in range(num_pages) if p == 0 or refs[p] != 0]
    n = len(live)
    holes = [p for p in range(1, n) if refs[p] == 0]
    to = dict(zip([p for p in live if p >= n], holes))
    err = 0
    for p, h in to.items():
        for pool, was in ((k, k_pool), (v, v_pool)):
            pool[h * page_size:(h + 1) * page_size] = was[p * page_size:(p + 1) * page_size]
        count[h], count[p] = refs[p], 0
    for at, e in np.ndenumerate(page_table):
        e = int(e)
        if n <= e < num_pages:
            if e in to:
                table[at] = to[e]
            else:
                err |= BAD_PAGE
    return k, v, table, count, n, err
