"""The operators for drafted tokens and for pages on the GPU, against the
float64 oracle: tree attention, verification, the commit of an accepted path,
page updates and pool compaction.

Tolerances. Attention: those of the other attention tests (max-abs 2e-2,
mean-abs 2e-3, LSE 1e-3): P and the output are each rounded to bf16 (2^-8 of
the value at most per step, values below 4 here), and the sums are fp32. All
other results are whole numbers or byte copies and have to be equal."""

import numpy as np
import pytest
import torch

import oracle.speculative as spec
from paged_kv_gqa_pkv_gb300 import binding
from paged_kv_gqa_pkv_gb300.workloads import bf16_bits
from tests import spec_cases as S
from tests.parity import assert_attention_close, gpu, new_dev_err

pytestmark = pytest.mark.gpu


def dev(a):
    return gpu(a if isinstance(a, torch.Tensor) else torch.from_numpy(np.ascontiguousarray(a)))


def run_tree(c, **kw):
    err = new_dev_err()
    out, lse = binding.pkv_tree_attention(dev(c.k), dev(c.v), dev(c.table), dev(c.q),
                                          dev(c.parents), dev(c.lens), dev(c.slots), dev(c.ctx),
                                          c.ps, c.scale, dev_err=err, **kw)
    torch.cuda.synchronize()
    return out.cpu(), lse.cpu(), int(err.item())


def check_tree(c, tag=""):
    out, lse, err = run_tree(c)
    ro, rl, rerr, skip = S.tree_oracle(c)
    assert err == rerr, (tag, err, rerr)
    rows = [b for b in range(len(c.ctx)) if b not in skip]
    assert_attention_close(out, lse, ro, rl, rows=rows, tag=tag)


@pytest.mark.parametrize("ctx,tree,N", [
    ([0], [1], 1),                       # one node and nothing before it
    ([1], [1], 1),
    ([200], [8], 8),
    ([0, 5, 127, 128, 129], [8, 3, 8, 8, 1], 8),      # borders of a key tile
    ([120, 250, 64], [9, 20, 64], 64),   # trees across a tile border
])
@pytest.mark.parametrize("hq,hkv", [(2, 2), (8, 2)])
def test_tree_small(ctx, tree, N, hq, hkv):
    check_tree(S.tree_case(1, ctx, tree, N, hq=hq, hkv=hkv))


@pytest.mark.parametrize("group", [1, 2, 4, 8])
@pytest.mark.parametrize("N", [1, 5, 16, 17, 32, 33, 64])
def test_tree_groups_and_sizes(group, N):
    """Row counts on both sides of 128 and 256 (two forms and row blocks)."""
    c = S.tree_case(2, [300, 77, 0], [N, max(1, N // 2), N], N, hq=2 * group, hkv=2, ps=32)
    check_tree(c, f"group {group} N {N}")


@pytest.mark.parametrize("ps", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("shape", ["chain", "star", "forest", "random"])
def test_tree_shapes_and_page_sizes(ps, shape):
    check_tree(S.tree_case(3, [190, 40, 383], [40, 24, 11], 40, hq=8, hkv=2, ps=ps, shape=shape))


def test_tree_padding_and_empty_rows():
    c = S.tree_case(4, [100, 50, 30, 0], [8, 0, 5, 0], 8, pad=(2,))
    out, lse, err = run_tree(c)
    assert err == 0
    ro, rl, _, _ = S.tree_oracle(c)
    assert_attention_close(out, lse, ro, rl)
    for b in (1, 2, 3):
        assert torch.all(out[b] == 0) and torch.all(torch.isneginf(lse[b]))


def test_tree_all_rows_empty():
    c = S.tree_case(5, [10, 20], [0, 3], 8, pad=(1,))
    out, lse, err = run_tree(c)
    assert err == 0 and torch.all(out == 0) and torch.all(torch.isneginf(lse))


@pytest.mark.parametrize("N,group", [(8, 4), (64, 4)])
def test_tree_long_context_is_split(N, group):
    """Few items and long contexts: every item is cut over many CTAs and joined."""
    check_tree(S.tree_case(6, [5000, 3333], [N, N - 3], N, hq=2 * group, hkv=2, ps=128))


@pytest.mark.parametrize("N,group", [(8, 1), (8, 4), (16, 4), (32, 4), (64, 4), (64, 8)])
def test_tree_rows_without_keys_of_a_split_item(N, group):
    """Nodes behind an invalid parent and trees much smaller than N, in items that
    are cut over many CTAs, with NaN in the workspace."""
    c = S.tree_case(13, [4000, 2500, 3000], [N, N, max(1, N // 8)], N, hq=2 * group, hkv=2, ps=128)
    half = max(1, N // 4)
    c.parents[0, half] = half                      # names itself
    c.parents[0, half + 1:2 * half] = np.arange(half, 2 * half - 1)
    c.parents[0, 2 * half:] = 0
    k, t = dev(c.k), dev(c.table)
    n = binding.pkv_tree_workspace_size(k, t, c.ps, 3, N, 2 * group)
    out, lse, err = run_tree(c, workspace=torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda"))
    ro, rl, rerr, skip = S.tree_oracle(c)
    assert err == rerr == spec.BAD_TREE and not skip
    assert_attention_close(out, lse, ro, rl)


def test_tree_many_rows():
    """More batch rows than one launch takes, ragged."""
    rng = np.random.default_rng(7)
    B = 300
    c = S.tree_case(7, rng.integers(0, 60, B).tolist(), rng.integers(0, 5, B).tolist(), 4, hq=4,
                    hkv=1, pad=(0, 17, 256, 299))
    check_tree(c)


@pytest.mark.parametrize("N,group,ps", [(1, 1, 16), (1, 8, 128), (2, 4, 64), (3, 2, 32), (8, 1, 16),
                                        (4, 2, 256), (2, 2, 48 * 8), (5, 1, 128)])
def test_tree_many_items_of_few_rows(N, group, ps):
    """Up to 8 query rows of more items than SMs: the warp-level form. Contexts
    around its 16-key tiles, long ones that are cut, dead nodes and padding."""
    rng = np.random.default_rng(N + group)
    B = 90
    ctx = rng.integers(0, 100, B)
    ctx[:8] = [0, 1, 15, 16, 17, 700, 2000, 3000]
    tree = rng.integers(0, N + 1, B)
    tree[:8] = N
    c = S.tree_case(14, ctx.tolist(), tree.tolist(), N, hq=2 * group, hkv=2, ps=ps, pad=(9, 30))
    if N > 1:
        c.parents[5, 1] = 7          # no such parent
    out, lse, err = run_tree(c)
    ro, rl, rerr, skip = S.tree_oracle(c)
    assert err == rerr and not skip
    assert_attention_close(out, lse, ro, rl)


def test_tree_bad_entries():
    c = S.tree_case(8, [100, 50, 60, 40, 33, 70], [6, 6, 6, 6, 6, 6], 6)
    c.slots[1] = 99                # past the table
    c.ctx[2] = 10 ** 6             # past the table
    c.lens[3] = 7                  # more nodes than there are
    c.parents[4] = [-1, 0, 2, 2, 1, 3]  # node 2 names itself; 3 and 5 hang below it
    check_tree(c)
    c = S.tree_case(9, [100, 50], [6, 6], 6)
    c.table[1, 2] = -1             # a block of row 0's context
    out, lse, err = run_tree(c)
    assert err == spec.BAD_PAGE
    ro, rl, _, skip = S.tree_oracle(c)
    assert skip == [0]
    assert_attention_close(out, lse, ro, rl, rows=[1])


def test_tree_large_scores_and_order_of_maxima():
    """Scores that grow along the keys by hundreds: every tile rescales."""
    c = S.tree_case(10, [700], [9], 9, hq=4, hkv=1, ps=64)
    rows = c.table[1][np.arange(709) // 64] * 64 + np.arange(709) % 64
    c.k[torch.from_numpy(rows).long()] *= torch.linspace(0, 40, 709)[:, None, None].bfloat16()
    check_tree(c)


def check_tree_rows(c, rows, out, lse):
    """Against whole products in 64 bits. Tolerances: products of bf16 values are
    exact in fp32 and 128 of them are summed there, an error of at most 2^-23 of the
    sum of magnitudes each (a tensor core truncates), and as much for the scaling to
    log2 units and the exponential's argument: e = 131 * 2^-23 * max sum |scale q K|.
    The weights' errors are e and the roundings of P to bf16, 2^-8 relative at most, the
    output's rounding is 2^-8 of the value; sums of positive terms in fp32 add less than
    (keys) * 2^-24, the exponentials and the logarithm (2^-22 each, of the weights, the
    rescales and the merge) 2^-20. Nodes past the tree give 0 and -inf."""
    for b, (ro, rl, mass, size) in zip(rows, S.tree_rows(c, rows)):
        n, keys = int(c.lens[b]), int(c.ctx[b] + c.lens[b])
        e = 131 * 2.0 ** -23 * size + keys * 2.0 ** -24 + 2.0 ** -20
        o, l = out[b].double().numpy(), lse[b].double().numpy()
        assert (o[n:] == 0).all() and np.isneginf(l[n:]).all()
        bad = np.abs(l[:n] - rl) - (e + 2.0 ** -22 * np.abs(rl))
        assert bad.max() <= 0, (b, "lse", bad.max())
        bad = np.abs(o[:n] - ro) - (2.0 ** -8 * np.abs(ro) + (2.0 ** -8 + 2 * e[..., None]) * mass)
        assert bad.max() <= 0, (b, "out", bad.max())


@pytest.mark.parametrize("N,group", [(1, 1), (2, 4), (3, 4), (8, 4), (16, 4), (17, 4), (32, 4),
                                     (17, 8), (64, 4), (64, 8)])
@pytest.mark.parametrize("scores", ["even", "growing"])
def test_tree_more_tiles_than_workers(N, group, scores):
    """384 items of up to 8 key tiles: every worker's range has several tiles and
    segments, in all forms (up to 8, 64, 128 and 256 query rows, and blocks of 256).
    With growing scores a row's maximum rises by about 14 in log2 units from one
    128-key tile to the next for a third of the rows, by less or hardly for the others;
    without, it never moves by 8. The workspace is full of NaN."""
    rng = np.random.default_rng(N + group)
    B, hkv = 48, 8
    ctx = rng.integers(250, 900, B)
    ctx[::5] = rng.integers(0, 140, len(ctx[::5]))
    tree = rng.integers(max(1, N // 2), N + 1, B)
    c = S.tree_case(15, ctx.tolist(), tree.tolist(), N, hq=hkv * group, hkv=hkv, ps=64, pad=(9,))
    if scores == "growing":
        for b in range(B):
            t = np.arange(ctx[b] + tree[b])
            at = torch.from_numpy(c.table[b + 1][t // 64].astype(np.int64) * 64 + t % 64)
            c.k[at] *= torch.from_numpy(0.5 + t / 32.0).bfloat16()[:, None, None]
        c.q *= torch.from_numpy(rng.choice([0.02, 0.3, 1.0], c.q.shape[:3] + (1,))).bfloat16()
    k, t = dev(c.k), dev(c.table)
    n = binding.pkv_tree_workspace_size(k, t, c.ps, B, N, hkv * group)
    out, lse, err = run_tree(c, workspace=torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda"))
    assert err == 0
    check_tree_rows(c, [0, 1, 2, 20, 33, 46, 47], out, lse)
    assert torch.all(out[9] == 0) and torch.all(torch.isneginf(lse[9]))


def test_tree_same_bits_twice_and_on_a_side_stream():
    c = S.tree_case(11, [1500, 800], [30, 64], 64, hq=8, hkv=2, ps=64)
    a = run_tree(c)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = run_tree(c)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_tree_workspace_refused_when_small():
    c = S.tree_case(12, [10], [4], 4)
    k, t = dev(c.k), dev(c.table)
    n = binding.pkv_tree_workspace_size(k, t, c.ps, 1, 4, 8)
    with pytest.raises(binding.PkvError) as e:
        run_tree(c, workspace=torch.empty(n - 256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 4
    run_tree(c, workspace=torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda"))


# ------------------------------------------------------------------ verify --

def run_verify(c):
    err = new_dev_err()
    r = binding.pkv_verify_tree(dev(c.target), dev(c.tokens), dev(c.parents), dev(c.lens),
                                dev(c.u), dev(c.us),
                                draft_probs=None if c.draft is None else dev(c.draft), dev_err=err)
    torch.cuda.synchronize()
    return [x.cpu().numpy() for x in r] + [int(err.item())]


def check_verify(c):
    got, want = run_verify(c), S.verify_oracle(c)
    for g, w in zip(got, want):
        assert np.array_equal(g, w), (g, w)
    return got


@pytest.mark.parametrize("V", [1, 2, 3, 7, 8, 33, 1000, 4099, 50257])
@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
def test_verify_vocabularies(V, draft, kind):
    check_verify(S.verify_case(V, 3, 9, V, draft=draft, kind=kind))


@pytest.mark.parametrize("shape", ["chain", "star", "random", "forest"])
@pytest.mark.parametrize("draft", [True, False])
def test_verify_shapes(shape, draft):
    for seed in range(4):
        check_verify(S.verify_case(100 + seed, 4, 64, 300, draft=draft, shape=shape))
        check_verify(S.verify_case(200 + seed, 4, 20, 5, draft=draft, shape=shape))


@pytest.mark.parametrize("B,V,kind", [(2, 120001, torch.float32), (2, 230003, torch.bfloat16),
                                      (40, 60001, torch.float32), (40, 110011, torch.bfloat16)])
@pytest.mark.parametrize("draft", [True, False])
def test_verify_rows_larger_than_shared_memory(B, V, kind, draft):
    """Vocabularies whose parts do not fit a CTA's ring, in both CTA sizes, with
    several refusals at one node."""
    c = S.verify_case(V, B, 4, V, draft=draft, kind=kind, shape="star", tree=[4] * B)
    c.u[::2] = 1.5                   # every second row refuses all of its drafts
    check_verify(c)


@pytest.mark.parametrize("V", [4097, 8193, 16385])
@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
def test_verify_many_short_rows_of_several_ctas(V, kind):
    """Many more clusters (of 2, 4 and 8 CTAs) than fit the GPU, each with one
    short pass, every third row padding: the sums that a cluster exchanges come
    right after its CTAs' start."""
    B = 700
    check_verify(S.verify_case(V, B, 1, V, draft=False, kind=kind,
                               tree=[0 if b % 3 == 1 else 1 for b in range(B)]))


def test_verify_one_node_and_padding():
    c = S.verify_case(5, 3, 1, 100, tree=[1, 0, 1])
    got = check_verify(c)
    assert got[2].tolist() == [1, 0, 1] and got[0][1, 0] == -1 and got[1][1, 0] == -1


def test_verify_random_numbers_at_their_ends():
    for u in (0.0, 1.0 - 2.0 ** -24, 1.0, -1.0, float("nan")):
        c = S.verify_case(6, 4, 12, 777, shape="star")
        c.u.fill_(u)
        c.us.fill_(u)
        check_verify(c)


def test_verify_target_without_mass_where_the_draft_was_refused():
    """p <= a q everywhere after the refusal: the next token comes from p."""
    c = S.verify_case(7, 2, 3, 50, shape="star", tree=[3, 3])
    c.draft = c.target.clone()
    c.u.fill_(2.0)   # nothing is accepted
    check_verify(c)


def test_verify_bad_rows():
    c = S.verify_case(8, 6, 8, 64, tree=[8, 8, 8, 9, -1, 8])
    c.tokens[0, 1] = 64
    c.tokens[1, 2] = -5
    c.parents[2, 4] = 6
    c.target[5] = 0.0
    got = check_verify(c)
    assert got[3] == spec.BAD_TREE | spec.BAD_PROBS
    c = S.verify_case(9, 2, 4, 64, tree=[4, 4])
    c.target[0, 0, 3] = float("nan")
    c.target[0, 0, 7] = -1.0
    c.draft[1, 0, 5] = float("nan")
    check_verify(c)
    c.target[:, :, 5] = float("inf")
    assert run_verify(c)[3] == spec.BAD_PROBS


def test_verify_accepts_as_often_as_the_target_says():
    """4000 one-draft rows over five tokens: the first committed token is
    distributed as the target (the bound is five standard deviations)."""
    B, V = 4000, 5
    g = torch.Generator().manual_seed(3)
    p, q = torch.tensor([.4, .3, .2, .1, 0.]), torch.tensor([.1, .1, .1, .3, .4])
    tok = torch.zeros((B, 3), dtype=torch.int32)
    tok[:, 1:] = torch.multinomial(q, 2 * B, replacement=True, generator=g).view(B, 2).int()
    rows = lambda x: x.expand(B, 3, V).contiguous()  # noqa: E731
    parents = torch.tensor([-1, 0, 0], dtype=torch.int32).expand(B, 3).contiguous()
    for draft in (rows(q), None):
        _, tokens, _ = binding.pkv_verify_tree(
            dev(rows(p)), dev(tok), dev(parents), dev(torch.full((B,), 3, dtype=torch.int32)),
            dev(torch.rand((B, 3), generator=g)), dev(torch.rand((B,), generator=g)),
            draft_probs=None if draft is None else dev(draft))
        share = torch.bincount(tokens[:, 0].cpu(), minlength=V).double() / B
        assert torch.all((share - p).abs() <= 5 * (p * (1 - p) / B).sqrt() + 1e-12), share


# ------------------------------------------------------------------ commit --

def run_commit(k, v, table, path, n, slots, ctx, ps, **kw):
    err = new_dev_err()
    kd, vd = dev(S.from_bits(k)), dev(S.from_bits(v))
    new = binding.pkv_commit_path(kd, vd, dev(table), dev(path), dev(n), dev(slots), dev(ctx), ps,
                                  dev_err=err, **kw)
    torch.cuda.synchronize()
    return bf16_bits(kd.cpu()), bf16_bits(vd.cpu()), new.cpu().numpy(), int(err.item())


def rand_paths(rng, B, N):
    path = np.full((B, N), -1, dtype=np.int32)
    n = np.zeros(B, dtype=np.int32)
    for b in range(B):
        taken = np.sort(rng.choice(N, rng.integers(0, N + 1), replace=False))
        n[b] = len(taken)
        path[b, :len(taken)] = taken
    return path, n


@pytest.mark.parametrize("hkv", [1, 2, 8, 17])
@pytest.mark.parametrize("N,ps", [(1, 16), (8, 16), (64, 48), (64, 128)])
def test_commit(hkv, N, ps):
    rng = np.random.default_rng(N + hkv)
    B = 5
    ctx = rng.integers(0, 200, B).astype(np.int32)
    st = S.pages_state(1, (ctx + N).tolist(), ps, hkv, 200, -(-(200 + N) // ps) + 1)
    path, n = rand_paths(rng, B, N)
    slots = np.arange(1, B + 1, dtype=np.int32)
    slots[1] = 0
    got = run_commit(st.k, st.v, st.table, path, n, slots, ctx, ps)
    want = spec.commit_path(st.k, st.v, st.table, path, n, slots, ctx, ps)
    for g, w in zip(got, want):
        assert np.array_equal(g, w)


def test_commit_bad_rows_move_nothing():
    st = S.pages_state(2, [40] * 8, 16, 2, 60, 4)
    path = np.tile(np.array([0, 2, 5, -1], dtype=np.int32), (8, 1))
    path[:, 2] = 3
    n = np.full(8, 3, dtype=np.int32)
    slots = np.arange(1, 9, dtype=np.int32)
    ctx = np.full(8, 30, dtype=np.int32)
    slots[0] = 77
    n[1] = 5
    path[2, 1] = 0          # not increasing
    path[3, 2] = 4          # not a node
    ctx[4] = -1
    ctx[5] = 62             # past the table
    st.table[7, 2] = 60     # no such page
    got = run_commit(st.k, st.v, st.table, path, n, slots, ctx, 16)
    want = spec.commit_path(st.k, st.v, st.table, path, n, slots, ctx, 16)
    for g, w in zip(got, want):
        assert np.array_equal(g, w)
    assert got[3] == spec.BAD_SLOT | spec.BAD_TREE | spec.BAD_POS | spec.BAD_PAGE


def test_commit_lengths_in_place():
    st = S.pages_state(3, [40] * 2, 16, 2, 20, 4)
    ctx = dev(np.array([20, 30], dtype=np.int32))
    path = dev(np.array([[0, 1], [1, -1]], dtype=np.int32))
    out = binding.pkv_commit_path(dev(S.from_bits(st.k)), dev(S.from_bits(st.v)), dev(st.table),
                                  path, dev(np.array([2, 1], dtype=np.int32)),
                                  dev(np.array([1, 2], dtype=np.int32)), ctx, 16, new_lens=ctx)
    assert out is ctx and ctx.cpu().tolist() == [22, 31]


# ------------------------------------------------------------------- pages --

def run_update(st, d, s, keep, new):
    err = new_dev_err()
    k, v, t, r = dev(S.from_bits(st.k)), dev(S.from_bits(st.v)), dev(st.table), dev(st.refs)
    i32 = lambda x: dev(np.array(x, dtype=np.int32))  # noqa: E731
    binding.pkv_update_pages(k, v, t, r, i32(d), i32(s), i32(keep), i32(new), st.ps, dev_err=err)
    torch.cuda.synchronize()
    return bf16_bits(k.cpu()), bf16_bits(v.cpu()), t.cpu().numpy(), r.cpu().numpy(), int(err.item())


def check_update(st, d, s, keep, new):
    got = run_update(st, d, s, keep, new)
    want = spec.update_pages(st.k, st.v, st.table, st.refs, d, s, keep, new, st.ps)
    for name, g, w in zip(("k", "v", "table", "refs", "err"), got, want):
        assert np.array_equal(g, w), (name, g, w)
    st.k, st.v, st.table, st.refs = got[:4]
    # every page's count is the number of entries that name it
    uses = np.bincount(st.table[st.table > 0], minlength=len(st.refs))
    assert np.array_equal(uses[1:], st.refs[1:])
    return got[4]


@pytest.mark.parametrize("ps", [16, 48, 128])
@pytest.mark.parametrize("hkv", [1, 8])
def test_update_life_of_a_cache(ps, hkv):
    """New sequences, forks, reserves with copy on write, truncations, frees."""
    st = S.pages_state(4, [], ps, hkv, 64, 6, slots=12)
    assert check_update(st, [1, 2, 3], [0, 0, 0], [0, 0, 0], [ps + 3, 2 * ps, 1]) == 0
    assert check_update(st, [4, 5, 6], [1, 1, 2], [ps + 3, ps, 2 * ps], [ps + 3, ps, 2 * ps]) == 0
    # all three holders of slot 1's partly filled page write on: all get copies
    assert check_update(st, [1, 4, 5], [1, 4, 5], [ps + 3, ps + 3, ps],
                        [ps + 9, 3 * ps, ps + 1]) == 0
    # fork with room at once; re-fork of a slot that has pages; truncation; free
    assert check_update(st, [7, 6, 2, 3], [4, 1, 2, 3], [ps + 5, 7, ps - 1, 0],
                        [2 * ps + 5, 9, ps - 1, 0]) == 0
    assert check_update(st, [2], [2], [ps - 1], [ps + 2]) == 0   # back into a shared page
    assert check_update(st, [1, 2, 4, 5, 6, 7, 0], [1, 2, 4, 5, 6, 7, 0], [0] * 7, [0] * 7) == 0
    assert st.refs[1:].sum() == 0


def test_update_random_calls():
    rng = np.random.default_rng(5)
    st = S.pages_state(5, [30, 10, 0, 64, 47], 16, 2, 90, 7, slots=14, share=[(6, 1), (7, 4)])
    lens = {1: 30, 2: 10, 3: 0, 4: 64, 5: 47, 6: 30, 7: 64}
    for _ in range(25):
        d = rng.permutation(np.arange(0, 14))[:rng.integers(1, 8)]
        s, keep, new = [], [], []
        for x in d:
            x = int(x)
            src = x if rng.random() < 0.6 else int(rng.integers(0, 14))
            have = lens.get(src, 0) if src else 0
            kp = int(rng.integers(0, have + 1))
            s.append(src)
            keep.append(kp)
            new.append(min(kp + int(rng.integers(0, 40)), 7 * 16))
        before = st.table.copy()
        check_update(st, [int(x) for x in d], s, keep, new)
        for x, a, b in zip(d, keep, new):
            x = int(x)
            if x and not np.array_equal(before[x], st.table[x]) or lens.get(x, 0) > 0:
                # tokens that are surely there: the filled blocks
                lens[x] = min(b, int((st.table[x] > 0).sum()) * 16)


def test_update_bad_rows_change_nothing():
    st = S.pages_state(6, [20, 33, 40, 50], 16, 2, 40, 4, slots=12)
    d = [99, -1, 5, 5, 6, 7, 8, 9, 3, 10, 2, 0]
    s = [1, 1, 0, 1, 0, 3, 1, 77, 3, 11, 2, 99]
    keep = [5, 5, 3, 5, 0, 5, -1, 0, 9, 4, 9, 9]
    new = [5, 5, 3, 5, 65, 5, 4, 3, 8, 4, 9, 9]
    # slot 5 is named twice, slot 3 is a source and a destination
    got = run_update(st, d, s, keep, new)
    want = spec.update_pages(st.k, st.v, st.table, st.refs, d, s, keep, new, 16)
    for g, w in zip(got, want):
        assert np.array_equal(g, w)
    assert got[4] == spec.BAD_SLOT | spec.BAD_POS | spec.BAD_PAGE
    st.refs[st.table[1, 0]] = 0   # a page in use that counts as free
    got = run_update(st, [1, 2], [1, 2], [20, 33], [40, 50])
    want = spec.update_pages(st.k, st.v, st.table, st.refs, [1, 2], [1, 2], [20, 33], [40, 50], 16)
    for g, w in zip(got, want):
        assert np.array_equal(g, w)
    assert got[4] == spec.BAD_PAGE


def test_update_when_pages_run_out():
    """Rows up to the first that does not fit are served; rows that need none too."""
    # 1 + 2 + 2 + 2 + 4 of 15 pages are taken, 4 are free; the rows need 1, 3, 1 and 0
    st = S.pages_state(7, [20, 20, 20, 60], 16, 2, 15, 6)
    err = check_update(st, [1, 2, 3, 4], [1, 2, 3, 4], [20, 20, 20, 10], [36, 80, 36, 10])
    assert err == spec.NO_PAGES
    assert (st.table[1:5] > 0).sum(1).tolist() == [3, 5, 2, 1]


def test_update_many_pages_and_rows():
    """More than one chunk of counts and many rows; free pages far up."""
    pages, ps = 9000, 16
    st = S.pages_state(8, [], ps, 1, pages, 40, slots=260)
    st.refs[1:4200] = 1      # held by the caller
    st.refs[5000:8500] = 1
    d = list(range(1, 257))
    rng = np.random.default_rng(8)
    new = rng.integers(0, 80, 256).tolist()
    got = run_update(st, d, [0] * 256, [0] * 256, new)
    want = spec.update_pages(st.k, st.v, st.table, st.refs, d, [0] * 256, [0] * 256, new, ps)
    for g, w in zip(got, want):
        assert np.array_equal(g, w)


# ----------------------------------------------------------------- compact --

def run_compact(st):
    err = new_dev_err()
    k, v, t, r = dev(S.from_bits(st.k)), dev(S.from_bits(st.v)), dev(st.table), dev(st.refs)
    n = binding.pkv_compact_pages(k, v, t, r, st.ps, dev_err=err)
    torch.cuda.synchronize()
    return (bf16_bits(k.cpu()), bf16_bits(v.cpu()), t.cpu().numpy(), r.cpu().numpy(),
            int(n.item()), int(err.item()))


@pytest.mark.parametrize("ps,hkv,pages", [(16, 1, 1), (16, 2, 9), (48, 3, 100), (16, 1, 9000),
                                          (256, 8, 40)])
@pytest.mark.parametrize("fill", [0.0, 0.3, 0.9, 1.0])
def test_compact(ps, hkv, pages, fill):
    rng = np.random.default_rng(pages)
    st = S.pages_state(9, [], ps, hkv, pages, 8, slots=10)
    used = 1 + rng.permutation(pages - 1)[:int((pages - 1) * fill)]
    st.refs[used] = rng.integers(1, 4, len(used))
    if len(used):
        st.table[1:] = np.where(rng.random((9, 8)) < 0.7, rng.choice(used, (9, 8)), -1)
    got = run_compact(st)
    want = spec.compact_pages(st.k, st.v, st.table, st.refs, ps)
    # rows of pages that were moved from keep what they held: compared as well
    for name, g, w in zip(("k", "v", "table", "refs", "live", "err"), got, want):
        assert np.array_equal(g, w), name


def test_compact_entries_of_free_pages_stay():
    st = S.pages_state(10, [], 16, 1, 20, 4, slots=3)
    st.refs[[3, 15]] = 1
    st.table[1] = [15, 18, 99, -7]    # 18 is free, 99 is no page
    st.table[2] = [3, 1, 2, 15]       # 1 and 2 are free, below the live pages' end or not
    got = run_compact(st)
    want = spec.compact_pages(st.k, st.v, st.table, st.refs, 16)
    for g, w in zip(got, want):
        assert np.array_equal(g, w)
    assert got[5] == spec.BAD_PAGE


def compact_workspace(st, word):
    k, t = dev(S.from_bits(st.k)), dev(st.table)
    n = binding.pkv_compact_workspace_size(k, t, st.ps)
    return torch.full((n // 4,), word, dtype=torch.int32, device="cuda").view(torch.uint8)


def check_compact_in(st, workspace):
    err = new_dev_err()
    k, v, t, r = dev(S.from_bits(st.k)), dev(S.from_bits(st.v)), dev(st.table), dev(st.refs)
    n = binding.pkv_compact_pages(k, v, t, r, st.ps, workspace=workspace, dev_err=err)
    torch.cuda.synchronize()
    got = (bf16_bits(k.cpu()), bf16_bits(v.cpu()), t.cpu().numpy(), r.cpu().numpy(),
           int(n.item()), int(err.item()))
    want = spec.compact_pages(st.k, st.v, st.table, st.refs, st.ps)
    for name, g, w in zip(("k", "v", "table", "refs", "live", "err"), got, want):
        assert np.array_equal(g, w), name
    return got


@pytest.mark.parametrize("dangling", [9, 15, 18, 19])
def test_compact_entries_of_free_pages_whatever_the_workspace_holds(dangling):
    """Every word of the workspace is the number of the free page that an entry
    names, below the highest live page and above it."""
    st = S.pages_state(11, [], 16, 1, 20, 4, slots=3)
    st.refs[[1, 2, 8, 13]] = 1
    st.table[1] = [1, 2, 8, 13]
    st.table[2, 1] = dangling
    got = check_compact_in(st, compact_workspace(st, dangling))
    assert got[5] == spec.BAD_PAGE and got[2][2, 1] == dangling


@pytest.mark.parametrize("dangling", [4000, 4095, 4096, 8100, 8191, 8192, 8999])
def test_compact_entries_of_free_pages_in_several_chunks(dangling):
    """The same over three chunks of counts, with most pages free."""
    st = S.pages_state(12, [], 16, 1, 9000, 8, slots=9)
    rng = np.random.default_rng(dangling)
    used = np.setdiff1d(1 + rng.permutation(8999)[:700], [dangling])
    st.refs[used] = 1
    st.table[1:8] = rng.choice(used, (7, 8))
    st.table[8, 3] = dangling
    got = check_compact_in(st, compact_workspace(st, dangling))
    assert got[5] == spec.BAD_PAGE and got[2][8, 3] == dangling


def test_compact_twice_on_one_workspace():
    """What an earlier call left in the workspace names a page that is free now."""
    st = S.pages_state(13, [], 16, 1, 20, 4, slots=3)
    st.refs[[1, 2, 3, 9]] = 1
    st.table[1] = [1, 2, 3, 9]
    ws = compact_workspace(st, -1)
    assert check_compact_in(st, ws)[5] == 0
    st.refs[[3, 9]], st.refs[8] = 0, 1
    st.table[1] = [1, 2, 8, -1]
    st.table[2, 0] = 9
    got = check_compact_in(st, ws)
    assert got[5] == spec.BAD_PAGE and got[2][2, 0] == 9
