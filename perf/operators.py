"""The speculative-decoding and page operators as workloads: their inputs, their plain form in elementary
torch operations, and the calls of the framework's own kernels (``own``).

* ``tree``: attention of a tree of drafted tokens over the paged cache.
* ``verify``: acceptance of drafted tokens against the target's probabilities, from given random numbers.
* ``commit``: the accepted path's K/V rows moved next to the committed context.
* ``pages``: fork, reserve, copy on write, truncate and free (``fork``: children take over a parent's prefix
  and get room for drafts; ``step``: room for a step's drafts, then the rejected ones' pages dropped).
* ``compact``: the live pages moved to the low end of the pool.

K/V shapes follow the rest of this repository: head dim 128, bf16 pools ``[num_pages * page_size, Hkv, 128]``,
slot 0 and page 0 reserved.
"""

import math

import torch

own = False

D = 128


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one user, a short context, a handful of drafted tokens: latency
        dict(name="tree_one_user", op="tree", B=1, N=8, hq=8, hkv=2, ps=16, lo=200, hi=333),
        # a full decode batch of a 32/8-head layer with small trees: the K/V stream bounds it
        dict(name="tree_batch", op="tree", B=64, N=8, hq=32, hkv=8, ps=128, lo=512, hi=1024),
        # wide trees over longer contexts, ragged tree sizes and padding rows: products and stream together
        dict(name="tree_wide", op="tree", B=32, N=64, hq=32, hkv=8, ps=128, lo=1024, hi=4095),
        # a chain of guessed tokens without draft probabilities (prompt lookup), one user
        dict(name="verify_chain_one", op="verify", B=1, N=6, V=32000, kind="fp32", draft=False, chain=True),
        # small trees of a draft model for an ordinary batch, probabilities in fp32, an odd vocabulary
        dict(name="verify_trees", op="verify", B=12, N=16, V=50257, kind="fp32", draft=True, chain=False),
        # a full batch at a large vocabulary, probabilities kept in bf16
        dict(name="verify_batch", op="verify", B=64, N=16, V=151936, kind="bf16", draft=True, chain=False),
        # the accepted tokens of one user's step
        dict(name="commit_one_user", op="commit", B=1, N=8, hkv=2, ps=16, lo=200, hi=333),
        # deep trees of a large batch
        dict(name="commit_batch", op="commit", B=256, N=64, hkv=8, ps=128, lo=256, hi=600),
        # a step's bookkeeping for a small batch with small pages: room for drafts, then the rejected ones dropped
        dict(name="pages_step", op="pages", mode="step", B=8, N=8, hkv=2, ps=16, lo=100, hi=700, pages=2048),
        # parallel sampling: 16 prompts forked to 8 children each, their partly filled last pages copied
        dict(name="pages_fork", op="pages", mode="fork", B=128, N=8, hkv=8, ps=128, lo=512, hi=1024, pages=2048),
        # a small pool with holes
        dict(name="compact_small", op="compact", B=6, hkv=2, ps=16, lo=100, hi=400, pages=400, gone=3),
        # a pool of a large batch after a third of its sequences have left
        dict(name="compact_pool", op="compact", B=128, hkv=8, ps=128, lo=512, hi=1024, pages=1400, gone=3),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "verify", "verify", "commit", "pages", "compact"])
    if op == "tree":
        # the products and the scores of the plain form stay below the largest listed case's
        while True:
            hkv, g = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 8])
            c = dict(op=op, B=_log(rng, 1, 96), N=_log(rng, 1, 64), hq=hkv * g, hkv=hkv,
                     ps=rng.choice([16, 32, 64, 128, 256]), lo=_log(rng, 1, 2000))
            c["hi"] = c["lo"] + _log(rng, 1, 6000)
            if c["B"] * c["N"] * c["hq"] * c["hi"] < 32 * 64 * 32 * 4095 and c["B"] * c["hkv"] * c["hi"] < 32 * 8 * 4095:
                return c
    if op == "verify":
        while True:
            c = dict(op=op, B=_log(rng, 1, 96), N=_log(rng, 1, 64), V=_log(rng, 2, 200000), kind=rng.choice(["fp32", "bf16"]),
                     draft=rng.random() < 0.7, chain=rng.random() < 0.3)
            if c["B"] * c["N"] * c["V"] < 64 * 16 * 151936:
                return c
    if op == "commit":
        lo = _log(rng, 1, 500)
        return dict(op=op, B=_log(rng, 1, 256), N=_log(rng, 1, 64), hkv=rng.choice([1, 2, 4, 8]), ps=rng.choice([16, 48, 64, 128]),
                    lo=lo, hi=lo + _log(rng, 1, 100))
    if op == "pages":
        lo, ps = _log(rng, 1, 500), rng.choice([16, 32, 64, 128])
        c = dict(op=op, mode=rng.choice(["step", "fork"]), B=8 * _log(rng, 1, 16), N=_log(rng, 1, 64), hkv=rng.choice([1, 2, 8]), ps=ps,
                 lo=lo, hi=lo + _log(rng, 1, 500))
        c["pages"] = 8 + 3 * c["B"] * (-(-(c["hi"] + c["N"]) // ps) + 1)
        return c
    lo, ps = _log(rng, 1, 500), rng.choice([16, 32, 64, 128])
    c = dict(op=op, B=_log(rng, 2, 128), hkv=rng.choice([1, 2, 8]), ps=ps, lo=lo, hi=lo + _log(rng, 1, 500), gone=rng.choice([2, 3, 5]))
    c["pages"] = 2 + int(c["B"] * -(-c["hi"] // ps) * rng.uniform(1.0, 1.5))
    return c


# ----------------------------------------------------------------- inputs --

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _ints(g, lo, hi, shape):
    return torch.randint(lo, hi + 1, shape, generator=g, device="cuda", dtype=torch.int32)


def _pools(g, rows, hkv):
    return [torch.randn((rows, hkv, D), generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2)]


def _permuted_table(g, slots, blocks):
    """Slots 1.. with `blocks` pages each, in a random order of pages 1..; and how many pages that takes."""
    pages = slots * blocks + 1
    table = torch.full((slots + 1, blocks), -1, device="cuda", dtype=torch.int32)
    table[1:] = (torch.randperm(pages - 1, generator=g, device="cuda") + 1).to(torch.int32).view(slots, blocks)
    return table, pages


def _parents(g, B, N, chain=False):
    """Random trees: node 0 is the root, every later node hangs below an earlier one."""
    j = torch.arange(N, device="cuda")
    if chain:
        p = (j - 1).expand(B, N)
    else:
        p = (torch.rand((B, N), generator=g, device="cuda").sqrt() * j).floor().clamp(max=N).minimum(j - 1)
        p[:, 0] = -1
    return p.to(torch.int32).contiguous()


def _prepare_tree(c, g):
    B, N = c["B"], c["N"]
    blocks = -(-(c["hi"] + N) // c["ps"])
    table, pages = _permuted_table(g, B, blocks)
    k, v = _pools(g, pages * c["ps"], c["hkv"])
    pad = B // 16
    batch_idx = torch.arange(1, B + 1, device="cuda", dtype=torch.int32)
    tree_lens = _ints(g, -(-N // 2), N, (B,))
    if pad:  # the unused rows of a padded batch
        batch_idx[-pad:] = 0
        tree_lens[-pad:] = 0
    return dict(k=k, v=v, table=table, ps=c["ps"], scale=1 / math.sqrt(D), parents=_parents(g, B, N), tree_lens=tree_lens,
                batch_idx=batch_idx, ctx=_ints(g, c["lo"], c["hi"], (B,)), longest=c["hi"] + N,
                q=torch.randn((B, N, c["hq"], D), generator=g, device="cuda", dtype=torch.bfloat16))


def _prepare_verify(c, g):
    B, N, V = c["B"], c["N"], c["V"]
    kind = torch.float32 if c["kind"] == "fp32" else torch.bfloat16
    parents = _parents(g, B, N, c["chain"])
    logits = torch.randn((B, N, V), generator=g, device="cuda") * 2.5
    target = torch.softmax(logits + 0.7 * torch.randn((B, N, V), generator=g, device="cuda"), -1).to(kind)
    # each node's token is drawn from the draft's distribution at its parent
    noise = -torch.log(-torch.log(torch.rand((B, N, V), generator=g, device="cuda").clamp(1e-9, 1 - 1e-7)))
    up = parents.clamp(min=0).long()
    noise += torch.gather(logits, 1, up[:, :, None].expand(B, N, V))
    tokens = noise.argmax(-1).to(torch.int32)
    del noise
    draft = torch.softmax(logits, -1).to(kind) if c["draft"] else None
    return dict(target=target, draft=draft, tokens=tokens, parents=parents, tree_lens=_ints(g, -(-N // 2), N, (B,)),
                u_accept=torch.rand((B, N), generator=g, device="cuda"), u_sample=torch.rand((B,), generator=g, device="cuda"))


def _prepare_commit(c, g):
    B, N = c["B"], c["N"]
    blocks = -(-(c["hi"] + N) // c["ps"])
    table, pages = _permuted_table(g, B, blocks)
    k, v = _pools(g, pages * c["ps"], c["hkv"])
    # a path takes the root, then each node with chance one half
    taken = torch.rand((B, N), generator=g, device="cuda") < 0.5
    taken[:, 0] = True
    n = taken.sum(1)
    path = torch.sort(torch.where(taken, torch.arange(N, device="cuda"), N), 1).values
    path = torch.where(path < N, path, -1).to(torch.int32)
    return dict(k=k, v=v, table=table, ps=c["ps"], path=path, n_accepted=n.to(torch.int32),
                batch_idx=torch.arange(1, B + 1, device="cuda", dtype=torch.int32), ctx=_ints(g, c["lo"], c["hi"], (B,)))


def _filled_table(g, lens, rows, cols, ps, pages):
    """A table whose slots 1.. hold ceil(len / ps) pages each, in a random order of the pool's pages, and the pages' counts."""
    need = (lens.long() + ps - 1) // ps
    here = torch.arange(cols, device="cuda") < need[:, None]
    nth = (torch.cumsum(here.flatten().long(), 0) - 1).view_as(here)
    order = (torch.randperm(pages - 1, generator=g, device="cuda") + 1).to(torch.int32)
    table = torch.full((rows, cols), -1, device="cuda", dtype=torch.int32)
    table[1:1 + lens.numel()] = torch.where(here, order[nth.clamp(0, pages - 2)], -1)
    refs = torch.zeros(pages, device="cuda", dtype=torch.int32)
    refs.index_add_(0, table.flatten().clamp(min=0).long(), (table.flatten() >= 0).to(torch.int32))
    refs[0] = 1
    return table, refs


def _prepare_pages(c, g):
    B, N, ps = c["B"], c["N"], c["ps"]
    cols = -(-(c["hi"] + N) // ps) + 1
    if c["mode"] == "step":
        ctx = _ints(g, c["lo"], c["hi"], (B,))
        table, refs = _filled_table(g, ctx, B + 1, cols, ps, c["pages"])
        slots = torch.arange(1, B + 1, device="cuda", dtype=torch.int32)
        left = ctx + _ints(g, 1, N, (B,))
        calls = [(slots, slots, ctx, ctx + N), (slots, slots, left, left)]
    else:
        n = B // 8
        lens = _ints(g, c["lo"], c["hi"], (n,))
        table, refs = _filled_table(g, lens, n + B + 1, cols, ps, c["pages"])
        parents = torch.arange(1, n + 1, device="cuda", dtype=torch.int32).repeat_interleave(8)
        keep = lens.repeat_interleave(8).contiguous()
        calls = [(torch.arange(n + 1, n + B + 1, device="cuda", dtype=torch.int32), parents, keep, keep + N)]
    k, v = _pools(g, c["pages"] * ps, c["hkv"])
    return dict(k=k, v=v, table=table, refs=refs, ps=ps, calls=calls)


def _prepare_compact(c, g):
    B, ps = c["B"], c["ps"]
    lens = _ints(g, c["lo"], c["hi"], (B,))
    table, refs = _filled_table(g, lens, B + 1, -(-c["hi"] // ps), ps, c["pages"])
    gone = torch.arange(1, B + 1, device="cuda") % c["gone"] == 0  # one in so many sequences has left
    out = table[1:][gone].flatten()
    refs.index_add_(0, out.clamp(min=0).long(), -(out >= 0).to(torch.int32))
    table[1:][gone] = -1
    k, v = _pools(g, c["pages"] * ps, c["hkv"])
    return dict(k=k, v=v, table0=table, refs0=refs, table=table.clone(), refs=refs.clone(), ps=ps)


def prepare(case, seed):
    g = _gen(seed)
    make = dict(tree=_prepare_tree, verify=_prepare_verify, commit=_prepare_commit, pages=_prepare_pages, compact=_prepare_compact)
    return dict(make[case["op"]](case, g), op=case["op"])


# ------------------------------------------------------------ plain forms --

def _tree(s):
    q, ps, L = s["q"], s["ps"], s["longest"]
    B, N, hq, _ = q.shape
    hkv = s["k"].shape[1]
    ctx, lens, slot = s["ctx"].long(), s["tree_lens"].long(), s["batch_idx"].long()
    pos = torch.arange(L, device=q.device)
    there = pos < (ctx + lens)[:, None]
    page = s["table"][slot].long()[:, (pos // ps).clamp(max=s["table"].shape[1] - 1)]
    row = torch.where(there, page * ps + pos % ps, 0)
    k = s["k"][row].float().permute(0, 2, 3, 1)
    v = torch.where(there[:, :, None, None], s["v"][row].float(), 0).transpose(1, 2)
    # ancestors: the closure of "is my parent", by squaring
    node = torch.arange(N, device=q.device)
    a = ((node[None, None, :] == s["parents"][:, :, None]) | (node[None, None, :] == node[None, :, None])).float()
    for _ in range(6):
        a = (a @ a).clamp(max=1)
    rel = pos - ctx[:, None]
    inside = (rel >= 0) & (rel < lens[:, None])
    kin = torch.gather(a > 0, 2, rel.clamp(0, N - 1)[:, None, :].expand(B, N, L))
    sees = (rel < 0)[:, None, :] | (inside[:, None, :] & kin)
    sees &= ((node < lens[:, None]) & (slot > 0)[:, None])[:, :, None]
    qh = q.float().view(B, N, hkv, hq // hkv, D).permute(0, 2, 3, 1, 4).reshape(B, hkv, -1, D)
    x = (qh @ k).view(B, hkv, hq // hkv, N, L) * s["scale"]
    x = x.masked_fill(~sees[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0, m)
    p = torch.exp(x - m)
    l = p.sum(-1, keepdim=True)
    o = (p.view(B, hkv, -1, L) @ v).view(B, hkv, hq // hkv, N, D) / torch.where(l > 0, l, 1)
    lse = (m + torch.log(l))[..., 0]
    return dict(out=o.permute(0, 3, 1, 2, 4).reshape(B, N, hq, D).to(q.dtype), lse=lse.permute(0, 3, 1, 2).reshape(B, N, hq))


def _verify(s):
    """In 64 bits: a drawn number next to a border of the cumulated sum must fall on the same side for everybody."""
    target, draft, tokens, parents = s["target"], s["draft"], s["tokens"].long(), s["parents"].long()
    B, N, V = target.shape
    dev = target.device
    b, zero = torch.arange(B, device=dev), torch.zeros(B, device=dev, dtype=torch.float64)
    u = s["u_accept"].double()
    lens = s["tree_lens"].long()
    cur = torch.zeros(B, device=dev, dtype=torch.long)
    count = torch.ones(B, device=dev, dtype=torch.long)
    path = torch.full((B, N), -1, device=dev, dtype=torch.long)
    path[:, 0] = 0
    a, mass = zero, zero + 1
    refused = torch.zeros((B, N), device=dev, dtype=torch.bool)  # siblings at the current node
    row = lambda x: x[b, cur].double().clamp(min=0)  # noqa: E731
    for j in range(1, N):
        asked = (parents[:, j] == cur) & (j < lens)
        px = target[b, cur, tokens[:, j]].double()
        if draft is None:
            again = (refused[:, :j] & (tokens[:, :j] == tokens[:, j:j + 1])).any(1)
            rx = torch.where(again, 0, px)
            ok = asked & (u[:, j] * mass < rx)
        else:
            qx = draft[b, cur, tokens[:, j]].double()
            rx = (px - a * qx).clamp(min=0)
            ok = asked & (u[:, j] * qx * mass < rx)
        no = asked & ~ok
        refused = torch.where(ok[:, None], False, refused)
        refused[:, j] = no
        if draft is None:
            mass = torch.where(no, (mass - rx).clamp(min=0), mass)
        else:
            a = torch.where(no, a + mass, a)
            mass = torch.where(no, (row(target) - a[:, None] * row(draft)).clamp(min=0).sum(1), mass)
        a, mass = torch.where(ok, 0, a), torch.where(ok, 1, mass)
        path[b, count.clamp(max=N - 1)] = torch.where(ok, j, path[b, count.clamp(max=N - 1)])
        count += ok
        cur = torch.where(ok, j, cur)
    p = row(target)
    if draft is None:
        r = p.clone()
        gone = torch.where(refused, tokens, V)
        r = torch.cat([r, r[:, :1]], 1).scatter(1, gone, 0.0)[:, :V]
    else:
        r = (p - a[:, None] * row(draft)).clamp(min=0)
    r = torch.where(r.sum(1, keepdim=True) > 0, r, p)
    c = torch.cumsum(r, 1)
    past = (c > s["u_sample"].double()[:, None] * c[:, -1:]) & (r > 0)
    at = torch.arange(V, device=dev)
    last = torch.where(past.any(1), torch.where(past, at, V).amin(1), torch.where(r > 0, at, -1).amax(1))
    n = torch.arange(N, device=dev)
    follow = torch.gather(tokens, 1, torch.cat([path[:, 1:], path[:, :1]], 1).clamp(min=0))
    out = torch.where(n < (count - 1)[:, None], follow, torch.where(n == (count - 1)[:, None], last[:, None], -1))
    return dict(path=path.to(torch.int32), tokens=out.to(torch.int32), n_accepted=count.to(torch.int32))


def _pool_rows(table, slot, pos, ps):
    page = torch.gather(table[slot].long(), 1, pos // ps)
    return page * ps + pos % ps


def _commit(s):
    path, n, ps = s["path"].long(), s["n_accepted"].long(), s["ps"]
    slot, ctx = s["batch_idx"].long(), s["ctx"].long()
    i = torch.arange(path.shape[1], device=path.device)
    moved = i < n[:, None]
    src = torch.where(moved, _pool_rows(s["table"], slot, ctx[:, None] + path.clamp(min=0), ps), 0)
    dst = torch.where(moved, _pool_rows(s["table"], slot, ctx[:, None] + i, ps), 0)  # the others: row 0 onto itself
    for pool in (s["k"], s["v"]):
        pool[dst] = pool[src]
    return dict(k=s["k"], v=s["v"], new_lens=(ctx + n).to(torch.int32))


def _update(s, dst, src, keep, new):
    table, refs, ps = s["table"], s["refs"], s["ps"]
    d, o, keep, new = dst.long(), src.long(), keep.long()[:, None], new.long()[:, None]
    j = torch.arange(table.shape[1], device=table.device)
    old, have = table[d].long(), table[o].long()
    same = (d == o)[:, None]
    kept = j < (keep + ps - 1) // ps
    written = (j >= keep // ps) & (j < (new + ps - 1) // ps) & (new > keep)
    mine = same & (old >= 0) & (refs[old.clamp(min=0)] == 1)
    fresh = written & ~mine
    free = torch.nonzero(refs == 0)[:, 0]
    nth = (torch.cumsum(fresh.flatten().long(), 0) - 1).clamp(min=0).view_as(fresh)
    now = torch.where(fresh, free[nth.clamp(max=free.numel() - 1)], torch.where(kept | (written & mine), have, -1))
    # the partly filled page that gets written: its kept rows, copied to the fresh page
    tail = torch.where(torch.gather(fresh, 1, keep // ps), keep % ps, 0)
    r = torch.arange(ps, device=table.device)
    get = torch.gather(have, 1, keep // ps).clamp(min=0) * ps + r
    put = torch.gather(now, 1, keep // ps) * ps + r
    copied = r < tail
    get, put = torch.where(copied, get, 0), torch.where(copied, put, 0)
    for pool in (s["k"], s["v"]):
        pool[put] = pool[get]
    left = (old >= 0) & ~(same & (now == old))
    refs.index_add_(0, old.clamp(min=0).flatten(), -left.flatten().to(torch.int32))
    refs.index_add_(0, now.clamp(min=0).flatten(), ((now >= 0) & ~(same & (now == old))).flatten().to(torch.int32))
    table[d] = now.to(torch.int32)


def _pages(s):
    for call in s["calls"]:
        _update(s, *call)
    return dict(table=s["table"], refs=s["refs"], k=s["k"], v=s["v"])


def _compact(s):
    table, refs, ps = s["table"], s["refs"], s["ps"]
    live = refs > 0
    live[0] = True
    n = live.sum()
    page = torch.arange(refs.numel(), device=refs.device)
    movers, holes = torch.nonzero(live & (page >= n))[:, 0], torch.nonzero(~live & (page < n))[:, 0]
    to = page.clone()
    to[movers] = holes
    s["table"].copy_(torch.where(table >= 0, to[table.clamp(min=0).long()].to(torch.int32), table))
    refs[holes] = refs[movers]
    refs[movers] = 0
    for pool in (s["k"], s["v"]):
        p = pool.view(refs.numel(), ps, pool.shape[1], D)
        p[holes] = p[movers]
    return dict(table=s["table"], refs=refs, k=s["k"], v=s["v"], live=n.to(torch.int32).view(1))


# -------------------------------------------------------------- one pass --

def _own(s):
    from paged_kv_gqa_pkv_gb300 import binding
    if s["op"] == "tree":
        out, lse = binding.pkv_tree_attention(s["k"], s["v"], s["table"], s["q"], s["parents"], s["tree_lens"], s["batch_idx"],
                                              s["ctx"], s["ps"], s["scale"])
        return dict(out=out, lse=lse)
    if s["op"] == "verify":
        path, tokens, n = binding.pkv_verify_tree(s["target"], s["tokens"], s["parents"], s["tree_lens"], s["u_accept"],
                                                  s["u_sample"], draft_probs=s["draft"])
        return dict(path=path, tokens=tokens, n_accepted=n)
    if s["op"] == "commit":
        new = binding.pkv_commit_path(s["k"], s["v"], s["table"], s["path"], s["n_accepted"], s["batch_idx"], s["ctx"], s["ps"])
        return dict(k=s["k"], v=s["v"], new_lens=new)
    if s["op"] == "pages":
        for dst, src, keep, new in s["calls"]:
            binding.pkv_update_pages(s["k"], s["v"], s["table"], s["refs"], dst, src, keep, new, s["ps"])
        return dict(table=s["table"], refs=s["refs"], k=s["k"], v=s["v"])
    live = binding.pkv_compact_pages(s["k"], s["v"], s["table"], s["refs"], s["ps"])
    return dict(table=s["table"], refs=s["refs"], k=s["k"], v=s["v"], live=live)


def run(s):
    if s["op"] == "compact":  # a compacted pool has nothing to move: every pass starts from the same table
        s["table"].copy_(s["table0"])
        s["refs"].copy_(s["refs0"])
    if own:
        return _own(s)
    return dict(tree=_tree, verify=_verify, commit=_commit, pages=_pages, compact=_compact)[s["op"]](s)


def work(case):
    """Lengths, tree sizes and paths are random: their mean counts."""
    c = dict(case)
    op, B = c["op"], c["B"]
    mean = (c["lo"] + c["hi"]) / 2 if "lo" in c else 0
    token = 2 * 2 * c["hkv"] * D if "hkv" in c else 0  # bytes of one token's K and V
    if op == "tree":
        live = B - B // 16
        nodes = (-(-c["N"] // 2) + c["N"]) / 2
        return dict(bytes=live * (mean + nodes) * token + live * nodes * c["hq"] * D * 2 + B * c["N"] * c["hq"] * (D * 2 + 4),
                    flops=4 * live * nodes * c["hq"] * D * mean)
    if op == "verify":
        # where the walk ends, the target's row is drawn from, less the draft's where a child was refused there
        row = c["V"] * (4 if c["kind"] == "fp32" else 2)
        return dict(bytes=B * (row * (2 if c["draft"] and c["N"] > 1 else 1) + c["N"] * 28), flops=B * c["V"] * 3)
    if op == "commit":
        # half of the path's rows, on average, are not where they belong
        return dict(bytes=B * max(1, c["N"] - 1) / 2 * token * 2 + B * c["N"] * 4, flops=0)
    if op == "pages":
        copied = B * (c["ps"] - 1) / 2 * token * 2 if c["mode"] == "fork" else 0
        return dict(bytes=copied + 4 * c["pages"] + (2 if c["mode"] == "step" else 1) * B * -(-c["hi"] // c["ps"]) * 8, flops=0)
    used = B * (mean / c["ps"] + 0.5) * (1 - 1 / c["gone"])
    moved = used * max(0.0, 1 - used / c["pages"])
    return dict(bytes=moved * c["ps"] * token * 2 + 8 * c["pages"] + 8 * B * -(-c["hi"] // c["ps"]), flops=0)


def exact(case, seed):
    """The tree attention from its definition in 64 bits, sequence by sequence; the other operators' outputs are whole numbers and copies."""
    if case["op"] != "tree":
        return None
    s = prepare(case, seed)
    B, N, hq, _ = s["q"].shape
    hkv = s["k"].shape[1]
    out = torch.zeros((B, N, hq, D), device="cuda", dtype=torch.float64)
    lse = torch.full((B, N, hq), -math.inf, device="cuda", dtype=torch.float64)
    parents, lens, slots, ctx = (s[k].tolist() for k in ("parents", "tree_lens", "batch_idx", "ctx"))
    for b in range(B):
        n = lens[b]
        if slots[b] == 0 or n == 0:
            continue
        pages = s["table"][slots[b]].long()
        t = torch.arange(ctx[b] + n, device="cuda")
        at = pages[t // s["ps"]] * s["ps"] + t % s["ps"]
        see = torch.zeros((n, ctx[b] + n), dtype=torch.bool)
        see[:, :ctx[b]] = True
        for i in range(n):
            up = i
            while up >= 0:
                see[i, ctx[b] + up] = True
                up = parents[b][up]
        see = see.cuda()
        for h in range(hkv):
            heads = slice(h * (hq // hkv), (h + 1) * (hq // hkv))
            x = torch.einsum("nhd,td->nht", s["q"][b, :n, heads].double(), s["k"][at, h].double()) / math.sqrt(D)
            x = torch.where(see[:, None, :], x, -math.inf)
            z = torch.logsumexp(x, -1)
            out[b, :n, heads] = torch.einsum("nht,td->nhd", torch.exp(x - z[..., None]), s["v"][at, h].double())
            lse[b, :n, heads] = z
    return dict(out=out, lse=lse)
