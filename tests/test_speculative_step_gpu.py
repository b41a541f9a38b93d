"""The drafted-token and page operators as a serving loop uses them: steps of
drafting with forks, freed users and compaction between them, beside the other
operators of the cache; the loop captured once and replayed; calls on two
streams; rows of other users and page 0 left as they were. Whole numbers,
tables and pools have to equal the oracle's; attention keeps the tolerances of
the other attention tests."""

import math

import numpy as np
import pytest
import torch

import oracle.paged_attention as orc
import oracle.speculative as spec
from paged_kv_gqa_pkv_gb300 import binding
from paged_kv_gqa_pkv_gb300.graphs import DecodeGraphs
from paged_kv_gqa_pkv_gb300.workloads import bf16_bits
from tests import spec_cases as S
from tests.parity import assert_attention_close

pytestmark = pytest.mark.gpu


def decode_close(m, rng, slots, hq):
    """One token of decode on each slot, by the framework's own decode."""
    q = torch.from_numpy(rng.standard_normal((len(slots), hq, 128)).astype(np.float32)).bfloat16()
    scale = 1 / math.sqrt(128)
    out, lse = binding.pkv_decode_attention(m.k, m.v, m.table, q.cuda(), m.i32(slots),
                                            m.i32(m.lens[slots]), m.ps, scale, dev_err=m.err)
    ro, rl, bad = orc.decode_attention(bf16_bits(q), m.host.k, m.host.v, m.host.table,
                                       np.array(slots), m.lens[slots], m.ps, scale)
    assert not bad
    assert_attention_close(out.cpu(), lse.cpu(), ro, rl, tag="decode")


@pytest.mark.parametrize("ps,N", [(16, 8), (64, 40)])
def test_a_loop_of_steps(ps, N):
    rng = np.random.default_rng(ps)
    m = S.Mirror(1, [70, 33, 129, 1], ps, 2, 160, -(-800 // ps), slots=9)
    slots = [1, 2, 3, 4]
    for step in range(6):
        S.draft_step(m, rng, slots, N, hq=8, V=97, shape=["random", "chain", "star"][step % 3])
        if step == 1:      # two users branch off user 2, mid-page
            keep = int(m.lens[2])
            m.update([5, 6], [2, 2], [keep, keep - 3], [keep, keep])
            m.lens[5], m.lens[6] = keep, keep - 3
            slots = [1, 2, 3, 4, 5, 6]
        if step == 3:      # one user leaves, the pool is packed
            m.update([3], [0], [0], [0])
            slots = [1, 2, 4, 5, 6]
            live = m.compact()
            assert live == int((m.host.refs > 0).sum())
        decode_close(m, rng, slots, 8)
    m.equal()


@pytest.mark.parametrize("captured", [False, True])
def test_layers_that_share_one_table(captured):
    """Three layers' pools behind one table: all calls but the last on clones of the
    table and counts from before the first. A fork, copies on write, an accepted path
    and a compaction; every layer's bytes, and every clone, equal the oracle's."""
    ps, hkv, pages = 16, 2, 40
    st = S.pages_state(6, [37, 20, 5], ps, hkv, pages, 6, slots=7)
    rng = np.random.default_rng(6)
    bits = [S.pool_bits(rng, pages * ps, hkv) for _ in range(3)]
    pools = [[S.from_bits(x).cuda() for x in b] for b in bits]
    i32 = lambda x: torch.from_numpy(np.array(x, dtype=np.int32)).cuda()  # noqa: E731
    table, refs, err = i32(st.table), i32(st.refs), i32([0])
    calls = [([4, 5], [1, 2], [37, 18], [37, 25]), ([1, 4, 3], [1, 4, 3], [37, 37, 5], [45, 40, 5]),
             ([2], [2], [0], [0])]
    gpu_calls = [[i32(x) for x in call] for call in calls]
    slots, ctx = i32([1, 4]), i32([37, 37])
    path, n = i32([[0, 2, 3, -1], [1, 2, -1, -1]]), i32([3, 2])
    states = lambda: [(table.clone(), refs.clone()) for _ in pools[1:]] + [(table, refs)]  # noqa: E731

    def steps():
        for call in gpu_calls:
            for (k, v), (t, r) in zip(pools, states()):
                binding.pkv_update_pages(k, v, t, r, *call, ps, dev_err=err)
        for i, (k, v) in enumerate(pools):
            binding.pkv_commit_path(k, v, table, path, n, slots, ctx, ps, dev_err=err,
                                    new_lens=ctx if i == len(pools) - 1 else None)
        last = states()
        for (k, v), (t, r) in zip(pools, last):
            binding.pkv_compact_pages(k, v, t, r, ps, dev_err=err)
        return last

    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            last = steps()
        graph.replay()
    else:
        last = steps()
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and ctx.cpu().tolist() == [40, 39]
    for (kb, vb), (k, v) in zip(bits, pools):
        t, r = st.table, st.refs
        for call in calls:
            kb, vb, t, r, e = spec.update_pages(kb, vb, t, r, *call, ps)
            assert e == 0
        kb, vb, _, e = spec.commit_path(kb, vb, t, path.cpu().numpy(), [3, 2], [1, 4], [37, 37], ps)
        assert e == 0
        kb, vb, t, r, _, e = spec.compact_pages(kb, vb, t, r, ps)
        assert e == 0
        assert np.array_equal(bf16_bits(k.cpu()), kb) and np.array_equal(bf16_bits(v.cpu()), vb)
    assert np.array_equal(table.cpu().numpy(), t) and np.array_equal(refs.cpu().numpy(), r)
    for t, r in last[:-1]:
        assert torch.equal(t, table) and torch.equal(r, refs)


def test_steps_between_captured_decode_steps():
    """The table that captured decode steps hold is updated by the page
    operators between replays."""
    rng = np.random.default_rng(5)
    m = S.Mirror(2, [60, 20], 16, 2, 60, 12, slots=5)
    scale = 1 / math.sqrt(128)
    g = DecodeGraphs(m.k, m.v, m.table, 16, 8, scale, buckets=(2, 4))
    slots = [1, 2]
    for step in range(4):
        S.draft_step(m, rng, slots, 6, hq=8, V=50)
        if step == 1:
            m.update([3], [1], [int(m.lens[1])], [int(m.lens[1])])
            m.lens[3] = m.lens[1]
            slots = [1, 2, 3]
        if step == 2:
            m.compact()
        ctx = m.lens[slots].copy()
        m.update(slots, slots, ctx, ctx + 1)
        B = len(slots)
        t = lambda *s: torch.from_numpy(  # noqa: E731
            rng.standard_normal(s).astype(np.float32)).bfloat16()
        q, kn, vn = t(B, 8, 128), t(B, 2, 128), t(B, 2, 128)
        out, lse = g.step(q.cuda(), kn.cuda(), vn.cuda(), m.i32(slots), m.i32(ctx),
                          m.i32(ctx + 1))[:2]
        h = m.host
        h.k, h.v, bad = orc.append(h.k, h.v, h.table, bf16_bits(kn), bf16_bits(vn),
                                   np.array(slots), ctx, 16)
        m.lens[slots] += 1
        ro, rl, bad2 = orc.decode_attention(bf16_bits(q), h.k, h.v, h.table, np.array(slots),
                                            ctx + 1, 16, scale)
        assert not bad and not bad2
        assert_attention_close(out.cpu()[:B], lse.cpu()[:B], ro, rl, tag=f"replay {step}")
        m.equal()


def test_a_step_captured_and_replayed():
    """Reserve, append, attend, verify, commit and truncate in one graph whose
    lengths live on the device; five replays against the oracle."""
    rng = np.random.default_rng(9)
    m = S.Mirror(3, [40, 90, 16], 16, 2, 60, 14, slots=4)
    slots, N, hq, V, B = [1, 2, 3], 7, 8, 61, 3
    scale = 1 / math.sqrt(128)
    h = m.host
    parents = S.rand_parents(rng, B, N)
    sl, par = m.i32(slots), m.i32(parents)
    ctx = m.i32(m.lens[slots])
    lens = m.i32([N] * B)
    f32 = dict(dtype=torch.float32, device="cuda")
    q = torch.zeros((B, N, hq, 128), dtype=torch.bfloat16, device="cuda")
    kn, vn = (torch.zeros((B * N, 2, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    target = torch.zeros((B, N, V), **f32)
    tok = torch.zeros((B, N), dtype=torch.int32, device="cuda")
    u, us = torch.zeros((B, N), **f32), torch.zeros(B, **f32)
    out, lse = torch.empty_like(q), torch.empty((B, N, hq), **f32)
    path, toks = torch.empty_like(tok), torch.empty_like(tok)
    n = torch.empty(B, dtype=torch.int32, device="cuda")
    ws = torch.empty(max(binding.pkv_update_workspace_size(m.k, m.table, 16, B),
                         binding.pkv_tree_workspace_size(m.k, m.table, 16, B, N, hq)),
                     dtype=torch.uint8, device="cuda")   # one for all: the calls are in order
    row_slots = sl.repeat_interleave(N)
    node = torch.arange(N, dtype=torch.int32, device="cuda").repeat(B)

    def step():
        top = ctx + N
        binding.pkv_update_pages(m.k, m.v, m.table, m.refs, sl, sl, ctx, top, 16, workspace=ws,
                                 dev_err=m.err)
        binding.pkv_append(m.k, m.v, m.table, kn, vn, row_slots, ctx.repeat_interleave(N) + node,
                           16, dev_err=m.err)
        binding.pkv_tree_attention(m.k, m.v, m.table, q, par, lens, sl, ctx, 16, scale, out=out,
                                   lse=lse, workspace=ws, dev_err=m.err)
        binding.pkv_verify_tree(target, tok, par, lens, u, us, path=path, tokens=toks,
                                n_accepted=n, dev_err=m.err)
        binding.pkv_commit_path(m.k, m.v, m.table, path, n, sl, ctx, 16, new_lens=ctx,
                                dev_err=m.err)
        binding.pkv_update_pages(m.k, m.v, m.table, m.refs, sl, sl, ctx, ctx, 16, workspace=ws,
                                 dev_err=m.err)

    keep = [t.clone() for t in (m.k, m.v, m.table, m.refs, ctx)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()                      # a warm-up; its state is put back
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t, old in zip((m.k, m.v, m.table, m.refs, ctx), keep):
        t.copy_(old)
    m.err.zero_()
    for replay in range(5):
        g = lambda *s: rng.standard_normal(s).astype(np.float32)  # noqa: E731
        q.copy_(torch.from_numpy(g(B, N, hq, 128)))
        kn.copy_(torch.from_numpy(g(B * N, 2, 128)))
        vn.copy_(torch.from_numpy(g(B * N, 2, 128)))
        target.copy_(torch.softmax(torch.from_numpy(g(B, N, V)), -1))
        tok.copy_(torch.from_numpy(rng.integers(0, V, (B, N)).astype(np.int32)))
        u.copy_(torch.from_numpy(rng.random((B, N)).astype(np.float32) * 0.1))
        us.copy_(torch.from_numpy(rng.random(B).astype(np.float32)))
        old = ctx.cpu().numpy()
        graph.replay()
        torch.cuda.synchronize()
        h.k, h.v, h.table, h.refs, e0 = spec.update_pages(h.k, h.v, h.table, h.refs, slots, slots,
                                                          old, old + N, 16)
        h.k, h.v, bad = orc.append(h.k, h.v, h.table, bf16_bits(kn.cpu()), bf16_bits(vn.cpu()),
                                   row_slots.cpu().numpy(), np.repeat(old, N) + node.cpu().numpy(),
                                   16)
        ro, rl, e1, _ = spec.tree_attention(bf16_bits(q.cpu()), h.k, h.v, h.table, parents,
                                            np.full(B, N), slots, old, 16, scale)
        assert_attention_close(out.cpu(), lse.cpu(), ro, rl, tag=f"replay {replay}")
        wp, wt, wn, e2 = spec.verify_tree(target.double().cpu().numpy(), None, tok.cpu().numpy(),
                                          parents, np.full(B, N), u.double().cpu().numpy(),
                                          us.double().cpu().numpy())
        assert np.array_equal(path.cpu().numpy(), wp) and np.array_equal(toks.cpu().numpy(), wt)
        h.k, h.v, new, e3 = spec.commit_path(h.k, h.v, h.table, wp, wn, slots, old, 16)
        h.k, h.v, h.table, h.refs, e4 = spec.update_pages(h.k, h.v, h.table, h.refs, slots, slots,
                                                          new, new, 16)
        assert not bad and not (e0 | e1 | e2 | e3 | e4)
        assert np.array_equal(ctx.cpu().numpy(), new)
        m.equal()


def test_two_streams_with_their_own_workspaces():
    """Two independent caches worked on at once give the bits that each gives
    alone."""
    cases = [S.tree_case(1, [3000, 700], [30, 64], 64, hq=8, hkv=2, ps=64),
             S.tree_case(2, [500] * 12, [8] * 12, 8, hq=8, hkv=2, ps=16)]
    ver = [S.verify_case(3, 6, 20, 5000), S.verify_case(4, 2, 64, 9000, kind=torch.bfloat16)]
    to = lambda a: (a if isinstance(a, torch.Tensor) else torch.from_numpy(a)).cuda()  # noqa: E731
    ta = [[to(x) for x in (c.k, c.v, c.table, c.q, c.parents, c.lens, c.slots, c.ctx)] +
          [c.ps, c.scale] for c in cases]
    va = [([to(x) for x in (c.target, c.tokens, c.parents, c.lens, c.u, c.us)], to(c.draft))
          for c in ver]
    alone = [binding.pkv_tree_attention(*a) for a in ta] + \
            [binding.pkv_verify_tree(*a, draft_probs=d) for a, d in va]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(8):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got.append((i, binding.pkv_tree_attention(*ta[i])))
                got.append((2 + i, binding.pkv_verify_tree(*va[i][0], draft_probs=va[i][1])))
    torch.cuda.synchronize()
    for which, r in got:
        for x, y in zip(r, alone[which]):
            assert torch.equal(x, y)


def test_a_stream_given_by_name():
    c = S.tree_case(21, [300, 80], [16, 9], 16)
    to = lambda a: (a if isinstance(a, torch.Tensor) else torch.from_numpy(a)).cuda()  # noqa: E731
    args = [to(x) for x in (c.k, c.v, c.table, c.q, c.parents, c.lens, c.slots, c.ctx)] + \
        [c.ps, c.scale]
    want = binding.pkv_tree_attention(*args)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out, lse = (torch.empty_like(x) for x in want)
    ws = torch.empty(binding.pkv_tree_workspace_size(args[0], args[2], c.ps, 2, 16, 8),
                     dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    binding.pkv_tree_attention(*args, out=out, lse=lse, workspace=ws, stream=s)
    # without buffers of its own: they come from the named stream's memory, so
    # nothing that the current stream does meanwhile can reuse them
    more = []
    for _ in range(20):
        more.append(binding.pkv_tree_attention(*args, stream=s))
        torch.full((ws.numel(),), 0xFF, dtype=torch.uint8, device="cuda")
    s.synchronize()
    for o, l in [(out, lse)] + more:
        assert torch.equal(o, want[0]) and torch.equal(l, want[1])


def test_a_context_past_the_reserved_pages_and_a_padded_batch():
    """Rows of padding name arbitrary lengths and trees and touch nothing."""
    c = S.tree_case(22, [100, 64, 30], [8, 8, 8], 8, pad=(1,))
    c.ctx[1], c.lens[1] = -7, 99
    c.parents[1] = 50
    to = lambda a: (a if isinstance(a, torch.Tensor) else torch.from_numpy(a)).cuda()  # noqa: E731
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = binding.pkv_tree_attention(*[to(x) for x in (c.k, c.v, c.table, c.q, c.parents,
                                                            c.lens, c.slots, c.ctx)], c.ps,
                                          c.scale, dev_err=err)
    ro, rl, e, skip = S.tree_oracle(c)
    assert e == int(err.item()) == 0 and not skip
    assert_attention_close(out.cpu(), lse.cpu(), ro, rl)


def test_verification_of_rows_past_32_bits():
    """Probabilities whose offset in elements passes 2^31: the last rows."""
    V, N, B = 1 << 20, 64, 33            # 33 * 64 * 2^20 = 2^31 + 2^26 elements of bf16
    t = torch.zeros((B, N, V), dtype=torch.bfloat16, device="cuda")
    t[:, :, 7] = 0.25
    t[:, :, V - 1] = 0.75
    tok = torch.zeros((B, N), dtype=torch.int32, device="cuda")
    tok[:, 1:] = V - 1
    parents = torch.from_numpy(S.rand_parents(np.random.default_rng(0), B, N, "chain")).cuda()
    lens = torch.full((B,), N, dtype=torch.int32, device="cuda")
    u = torch.full((B, N), 0.5, device="cuda")
    u[:, 40] = 0.9                       # node 40 is refused: 0.9 > 0.75
    path, toks, n = binding.pkv_verify_tree(t, tok, parents, lens, u,
                                            torch.full((B,), 0.5, device="cuda"))
    # nodes 0..39 accepted; without the refused token only token 7 is left
    assert n.cpu().tolist() == [40] * B
    assert torch.equal(path[:, :40].cpu(), torch.arange(40).int().expand(B, 40))
    assert (toks[:, :39] == V - 1).all() and (toks[:, 39] == 7).all()


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [(1 << 29) + 5, (1 << 30) - 1, 1 << 30])
def test_verification_of_the_longest_rows(V, kind):
    """Rows whose bytes, or whose values, pass 31 bits: the largest vocabulary that
    is taken, and borders below it. Four tokens have the mass, at the row's ends, in
    its middle and where the remaining bytes fall under 2^31; the drafted one is
    refused, so the draw is from the other three."""
    at = sorted([0, V // 2, V - (1 << 29) + 1, V - 1])
    t = torch.zeros((2, 2, V), dtype=kind, device="cuda")
    t[:, 0, at] = torch.tensor([0.125, 0.25, 0.125, 0.5], device="cuda").to(kind)
    tok = torch.full((2, 2), V - 1, dtype=torch.int32, device="cuda")
    parents = torch.tensor([[-1, 0]] * 2, dtype=torch.int32, device="cuda")
    lens = torch.full((2,), 2, dtype=torch.int32, device="cuda")
    left = np.cumsum([0.125, 0.25, 0.125])   # 0.75 > 0.5: the last token is refused
    want = lambda u: at[int(np.nonzero(left > u * 0.5)[0][0])]  # noqa: E731
    for u in ((0.0, 0.3), (0.5, 0.99)):
        path, toks, n = binding.pkv_verify_tree(
            t, tok, parents, lens, torch.full((2, 2), 0.75, device="cuda"),
            torch.tensor(u, device="cuda"))
        assert n.cpu().tolist() == [1, 1]
        assert toks[:, 0].cpu().tolist() == [want(x) for x in u]


@pytest.mark.parametrize("how", ["small", "misaligned", "device", "type"])
def test_refused_workspaces_and_outputs(how):
    m = S.Mirror(4, [30], 16, 1, 8, 4, slots=3)
    one = m.i32([1])
    n = binding.pkv_update_workspace_size(m.k, m.table, 16, 1)
    ws = {"small": torch.empty(n - 1, dtype=torch.uint8, device="cuda"),
          "misaligned": torch.empty(n + 64, dtype=torch.uint8, device="cuda")[64:],
          "device": torch.empty(n, dtype=torch.uint8),
          "type": torch.empty(n, dtype=torch.uint8, device="cuda")}[how]
    refs = m.refs.long() if how == "type" else m.refs
    with pytest.raises((ValueError, binding.PkvError)):
        binding.pkv_update_pages(m.k, m.v, m.table, refs, one, one, m.i32([30]), m.i32([40]), 16,
                                 workspace=ws)
    m.equal()


@pytest.mark.parametrize("named", [False, True])
def test_workspaces_without_the_allocators_raw_calls(monkeypatch, named):
    """A PyTorch that lacks the raw allocation calls: workspaces are tensors of the
    call's stream, and the results are the same."""
    c = S.tree_case(23, [900, 80], [16, 9], 16)
    to = lambda a: (a if isinstance(a, torch.Tensor) else torch.from_numpy(a)).cuda()  # noqa: E731
    args = [to(x) for x in (c.k, c.v, c.table, c.q, c.parents, c.lens, c.slots, c.ctx)] + \
        [c.ps, c.scale]
    want = binding.pkv_tree_attention(*args)
    torch.cuda.synchronize()
    monkeypatch.setattr(binding, "_raw_alloc", None)
    stream = torch.cuda.Stream() if named else None
    more = []
    for _ in range(10):
        more.append(binding.pkv_tree_attention(*args, stream=stream))
        torch.full((1 << 24,), 0xFF, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for o, l in more:
        assert torch.equal(o, want[0]) and torch.equal(l, want[1])
    m = S.Mirror(5, [30, 50], 16, 1, 20, 6, slots=4)
    m.update([1, 3], [1, 2], [30, 40], [45, 45])
    m.compact()
    m.equal()


def test_calls_without_buffers_are_captured():
    """Results and workspaces allocated inside the capture; two graphs replayed in
    turn, each with inputs changed in place between replays."""
    to = lambda a: (a if isinstance(a, torch.Tensor) else torch.from_numpy(a)).cuda()  # noqa: E731
    cases = [S.tree_case(31, [900, 40], [12, 7], 12, hq=8, hkv=2),
             S.tree_case(32, [64, 64, 500], [3, 5, 5], 5, hq=4, hkv=2, ps=32)]
    ver = S.verify_case(33, 3, 9, 700)
    graphs = []
    for c in cases:
        a = [to(x) for x in (c.k, c.v, c.table, c.q, c.parents, c.lens, c.slots, c.ctx)]
        vt = [to(x) for x in (ver.target, ver.tokens, ver.parents, ver.lens, ver.u, ver.us)]
        binding.pkv_tree_attention(*a, c.ps, c.scale)
        binding.pkv_verify_tree(*vt)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            r = binding.pkv_tree_attention(*a, c.ps, c.scale) + binding.pkv_verify_tree(*vt)
        graphs.append((g, a, vt, r, c))
    rng = np.random.default_rng(34)
    for _ in range(3):
        for g, a, vt, r, c in graphs:
            c.q = torch.from_numpy(rng.standard_normal(tuple(c.q.shape)).astype(np.float32)).bfloat16()
            ver.u = torch.from_numpy(rng.random(tuple(ver.u.shape)).astype(np.float32))
            a[3].copy_(c.q)
            vt[4].copy_(ver.u)
            g.replay()
            torch.cuda.synchronize()
            ro, rl, err, _ = S.tree_oracle(c)
            assert err == 0
            assert_attention_close(r[0].cpu(), r[1].cpu(), ro, rl)
            f = lambda t: t.double().numpy()  # noqa: E731
            want = spec.verify_tree(f(ver.target), None, ver.tokens.numpy(), ver.parents, ver.lens,
                                    f(ver.u), f(ver.us))
            for x, w in zip(r[2:], want):
                assert np.array_equal(x.cpu().numpy(), w)


def test_a_pool_past_32_bits():
    """4.3 million pages of 16 tokens (8.8e9 elements per pool, more pages than the
    smallest chunks of the page plans): fork, commit, attention and compaction."""
    ps, pages, slots, cols = 16, 4_300_000, 6, 48
    rows = pages * ps
    k = torch.empty((rows, 1, 128), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    mark = torch.arange(rows, dtype=torch.int32, device="cuda")[:, None, None]
    k.view(torch.int32).copy_(mark)          # a row's number, 64 times
    v.view(torch.int32).copy_(-mark)
    del mark
    rng = np.random.default_rng(41)
    table = np.full((slots, cols), -1, dtype=np.int32)
    lens = {1: 500, 2: 333, 3: 700}
    for s, n in lens.items():
        m = -(-n // ps)
        table[s, :m] = rng.choice(np.arange(pages - 5000 * s, pages - 5000 * (s - 1)), m, False)
    refs = np.zeros(pages, dtype=np.int32)
    refs[0] = 1
    refs[1:3_000_000:2] = 1                  # holds of the caller's own
    for e in table[table > 0]:
        refs[e] += 1
    i32 = lambda x: torch.from_numpy(np.array(x, dtype=np.int32)).cuda()  # noqa: E731
    tab, cnt, err = i32(table), i32(refs), i32([0])
    none = np.zeros((rows, 0), dtype=np.uint8)   # the oracle's pools: nothing in them
    row = lambda t, s, n: (t[s, np.arange(n) // ps].astype(np.int64) * ps +  # noqa: E731
                           np.arange(n) % ps)
    held = lambda r: k.view(torch.int32)[torch.from_numpy(r).cuda(), 0, 0].cpu().numpy()  # noqa: E731
    heldv = lambda r: -v.view(torch.int32)[torch.from_numpy(r).cuda(), 0, 63].cpu().numpy()  # noqa: E731

    # slot 4 branches off slot 1 mid-page, slot 3 gets room
    call = ([4, 3], [1, 3], [437, 700], [460, 720])
    binding.pkv_update_pages(k, v, tab, cnt, *map(i32, call), ps, dev_err=err)
    _, _, t2, r2, e2 = spec.update_pages(none, none, table, refs, *call, ps)
    assert e2 == 0 and int(err.item()) == 0
    assert np.array_equal(tab.cpu().numpy(), t2) and np.array_equal(cnt.cpu().numpy(), r2)
    for get in (held, heldv):
        assert np.array_equal(get(row(t2, 4, 437)), row(table, 1, 437))

    # an accepted path of slot 3's last positions
    before = held(row(t2, 3, 720))
    new = binding.pkv_commit_path(k, v, tab, i32([[0, 3, 4, 7, -1, -1, -1, -1]]), i32([4]), i32([3]),
                                  i32([700]), ps, dev_err=err)   # nodes 0 .. 7 of 8
    assert new.item() == 704
    assert np.array_equal(held(row(t2, 3, 704))[700:], before[[700, 703, 704, 707]])

    # attention of a tree behind slot 2, whose rows get numbers that are finite
    update = ([2], [2], [333], [339])
    binding.pkv_update_pages(k, v, tab, cnt, *map(i32, update), ps, dev_err=err)
    _, _, t3, r3, _ = spec.update_pages(none, none, t2, r2, *update, ps)
    at = row(t3, 2, 339)
    kk, vv = (torch.from_numpy(rng.standard_normal((339, 1, 128)).astype(np.float32)).bfloat16()
              for _ in range(2))
    k[torch.from_numpy(at).cuda()], v[torch.from_numpy(at).cuda()] = kk.cuda(), vv.cuda()
    q = torch.from_numpy(rng.standard_normal((1, 6, 4, 128)).astype(np.float32)).bfloat16()
    par = np.array([[-1, 0, 0, 1, 3, 2]], dtype=np.int32)
    out, lse = binding.pkv_tree_attention(k, v, tab, q.cuda(), i32(par), i32([6]), i32([2]),
                                          i32([333]), ps, 0.09, dev_err=err)
    pad = lambda x: bf16_bits(torch.cat([x, torch.zeros(13, 1, 128).bfloat16()]))  # noqa: E731
    small = np.arange(22, dtype=np.int32)[None].repeat(2, 0)
    ro, rl, e, _ = spec.tree_attention(bf16_bits(q), pad(kk), pad(vv), small, par, [6], [1], [333],
                                       ps, 0.09)
    assert e == 0 and int(err.item()) == 0
    assert_attention_close(out.cpu(), lse.cpu(), ro, rl)

    # the caller's holds end, slot 2 leaves, the pool is packed
    cnt[1:3_000_000:2] -= 1
    r3[1:3_000_000:2] -= 1
    gone = ([2], [0], [0], [0])
    binding.pkv_update_pages(k, v, tab, cnt, *map(i32, gone), ps, dev_err=err)
    _, _, t4, r4, _ = spec.update_pages(none, none, t3, r3, *gone, ps)
    was = {s: held(row(t4, s, n)) for s, n in ((1, 500), (3, 704), (4, 437))}
    n = binding.pkv_compact_pages(k, v, tab, cnt, ps, dev_err=err)
    _, _, t5, r5, live, e5 = spec.compact_pages(none, none, t4, r4, ps)
    assert e5 == 0 and int(err.item()) == 0 and n.item() == live
    assert np.array_equal(tab.cpu().numpy(), t5) and np.array_equal(cnt.cpu().numpy(), r5)
    for s, w in was.items():
        assert np.array_equal(held(row(t5, s, len(w))), w)
