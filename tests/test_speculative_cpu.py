"""The drafted-token and page operators without a GPU: the C entries' and the
binding's refusals, and the oracle against itself and against hand-made cases."""

import ctypes

import numpy as np
import pytest
import torch

import oracle.paged_attention as orc
import oracle.speculative as spec
from paged_kv_gqa_pkv_gb300 import binding
from paged_kv_gqa_pkv_gb300.workloads import bf16_bits
from tests import spec_cases as S

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(binding.LIB_PATH):
        from paged_kv_gqa_pkv_gb300 import build
        build.build()
    return binding.load_library()


def _desc(**kw):
    d = dict(num_pages=32, page_size=16, num_kv_heads=2, head_dim=128, max_batch=5, max_blocks=16)
    d.update(kw)
    return ctypes.byref(binding.CacheDesc(**d))


# ------------------------------------------------------------ the C entries --

def test_tree_refusals(lib):
    def call(desc=None, kp=256, q=256, hq=8, parents=256, B=4, N=8, scale=0.1, out=256, lse=256,
             ws=256, nb=1 << 30, err=0):
        return lib.pkv_tree_attention(
            desc or _desc(), P(kp), P(256), P(256), P(q), hq, P(parents), P(256), P(256), P(256),
            B, N, ctypes.c_float(scale), P(out), P(lse), P(ws), nb, P(err) if err else None, None)
    assert call(B=0) == 0
    for kw in (dict(B=-1), dict(N=0), dict(N=65), dict(hq=6), dict(hq=32), dict(scale=0.0),
               dict(scale=-1.0), dict(scale=float("inf")), dict(scale=float("nan")), dict(kp=0),
               dict(q=0), dict(parents=0), dict(out=0), dict(lse=0), dict(desc=_desc(page_size=48)),
               dict(desc=_desc(head_dim=64)), dict(B=1 << 26, N=64)):
        assert call(**kw) == 1, kw
    for kw in (dict(q=264), dict(kp=264), dict(out=264), dict(lse=258), dict(parents=257),
               dict(err=257)):
        assert call(**kw) == 2, kw
    assert lib.pkv_tree_attention(None, *([P(256)] * 4), 8, *([P(256)] * 4), 4, 8,
                                  ctypes.c_float(0.1), P(256), P(256), P(256), 1, None, None) == 1
    assert lib.pkv_tree_workspace_size(_desc(), 4, 65, 8) == 0
    assert lib.pkv_tree_workspace_size(_desc(), -1, 8, 8) == 0
    assert lib.pkv_tree_workspace_size(_desc(), 4, 8, 6) == 0


def test_verify_refusals(lib):
    def call(t=256, d=0, kind=0, V=100, tok=256, u=256, B=4, N=8, path=256, n=256):
        return lib.pkv_verify_tree(P(t), P(d) if d else None, kind, V, P(tok), P(256), P(256),
                                   P(u), P(256), B, N, P(path), P(256), P(n), None, None)
    assert call(B=0) == 0
    for kw in (dict(kind=2), dict(kind=-1), dict(V=0), dict(V=(1 << 30) + 1), dict(B=-1),
               dict(B=(1 << 24) + 1), dict(N=0), dict(N=65), dict(t=0), dict(tok=0), dict(u=0),
               dict(path=0), dict(n=0)):
        assert call(**kw) == 1, kw
    for kw in (dict(t=264), dict(d=260), dict(tok=257), dict(u=258), dict(path=257), dict(n=258)):
        assert call(**kw) == 2, kw


def test_commit_refusals(lib):
    def call(desc=None, kp=256, path=256, B=4, N=8, new=256):
        return lib.pkv_commit_path(desc or _desc(), P(kp), P(256), P(256), P(path), P(256), P(256),
                                   P(256), B, N, P(new) if new else None, None, None)
    assert call(B=0) == 0
    for kw in (dict(desc=_desc(page_size=24)), dict(kp=0), dict(path=0), dict(B=-1), dict(N=0),
               dict(N=65)):
        assert call(**kw) == 1, kw
    for kw in (dict(kp=264), dict(path=258), dict(new=257)):
        assert call(**kw) == 2, kw


def test_page_refusals(lib):
    def update(desc=None, kp=256, refs=256, dst=256, n=4, ws=256, nb=1 << 30):
        return lib.pkv_update_pages(desc or _desc(), P(kp), P(256), P(256), P(refs), P(dst), P(256),
                                    P(256), P(256), n, P(ws), nb, None, None)
    assert update(n=0) == 0
    for kw in (dict(n=-1), dict(kp=0), dict(refs=0), dict(dst=0), dict(desc=_desc(num_pages=0)),
               dict(desc=_desc(num_pages=2, page_size=1 << 24, max_blocks=1))):
        assert update(**kw) == 1, kw
    for kw in (dict(kp=264), dict(refs=258), dict(dst=257)):
        assert update(**kw) == 2, kw

    def compact(desc=None, kp=256, refs=256, live=256):
        return lib.pkv_compact_pages(desc or _desc(), P(kp), P(256), P(256), P(refs),
                                     P(live) if live else None, P(256), 1 << 30, None, None)
    for kw in (dict(kp=0), dict(refs=0), dict(desc=_desc(head_dim=64))):
        assert compact(**kw) == 1, kw
    for kw in (dict(kp=264), dict(refs=257), dict(live=258)):
        assert compact(**kw) == 2, kw
    assert lib.pkv_update_workspace_size(_desc(), -1) == 0
    assert lib.pkv_update_workspace_size(_desc(page_size=17), 4) == 0
    assert lib.pkv_compact_workspace_size(_desc(max_batch=0)) == 0
    # the counts of every page fit, whatever their number
    for pages in (1, 4096, 4097, 5_000_000):
        d = _desc(num_pages=pages)
        assert lib.pkv_update_workspace_size(d, 3) >= 4 * pages
        assert lib.pkv_compact_workspace_size(d) >= 3 * 4 * pages


def test_without_a_gpu_calls_fail_cleanly(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert lib.pkv_commit_path(_desc(), *([P(256)] * 7), 4, 8, None, None, None) in (5, 6)
    assert lib.pkv_tree_workspace_size(_desc(), 4, 8, 8) == 0


def test_binding_refuses_host_tensors_and_types():
    k = torch.zeros((64, 2, 128), dtype=torch.bfloat16)
    t = torch.zeros((3, 4), dtype=torch.int32)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        binding.pkv_commit_path(k, k, t, t, i, i, i, 16)
    with pytest.raises(ValueError):
        binding.pkv_verify_tree(torch.zeros((1, 2, 3), dtype=torch.float16), i, i, i, i, i)
    with pytest.raises((ValueError, TypeError)):
        binding.pkv_tree_attention(None, k, t, k, t, i, i, i, 16, 1.0)


# --------------------------------------------------------------- the oracle --

def test_a_chain_is_causal_attention():
    """A chain over a context is the tokens of a chunk at consecutive positions."""
    c = S.tree_case(1, [37], [6], 6, hq=4, hkv=2, shape="chain")
    out, lse, err, _ = S.tree_oracle(c)
    pos = np.arange(37, 43, dtype=np.int32)
    ro, rl, bad = orc.paged_prefill_attention(bf16_bits(c.q)[0], bf16_bits(c.k), bf16_bits(c.v),
                                              c.table, np.full(6, 1, dtype=np.int32), pos, c.ps,
                                              c.scale)
    assert err == 0 and not bad
    np.testing.assert_allclose(out[0], ro, atol=1e-12)
    np.testing.assert_allclose(lse[0], rl, atol=1e-12)


def test_siblings_do_not_see_each_other():
    """Each path of a tree gives what the path alone gives."""
    c = S.tree_case(2, [20], [5], 5, hq=2, hkv=1)
    c.parents[0] = [-1, 0, 0, 1, 2]
    out, lse, _, _ = S.tree_oracle(c)
    for path in ([0, 1, 3], [0, 2, 4]):
        k, v = c.k.clone(), c.v.clone()
        rows = [orc.physical_slot(c.table, 1, 20 + a, c.ps, len(c.k) // c.ps) for a in range(5)]
        for i, a in enumerate(path):
            k[rows[i]], v[rows[i]] = c.k[rows[a]], c.v[rows[a]]
        d = S.SimpleNamespace(**{**vars(c), "k": k, "v": v, "q": c.q[:, path],
                                 "parents": np.array([[-1, 0, 1]], dtype=np.int32),
                                 "lens": np.array([3], dtype=np.int32)})
        o, l, _, _ = S.tree_oracle(d)
        np.testing.assert_allclose(o[0], out[0, path], atol=1e-12)
        np.testing.assert_allclose(l[0], lse[0, path], atol=1e-12)


def test_whole_products_equal_the_oracle():
    c = S.tree_case(3, [20, 0, 33], [5, 4, 1], 5, hq=4, hkv=2, shape="forest")
    out, lse, err, _ = S.tree_oracle(c)
    assert err == 0
    for b, (o, l, mass, size) in enumerate(S.tree_rows(c, range(3))):
        n = c.lens[b]
        np.testing.assert_allclose(o, out[b, :n], atol=1e-12)
        np.testing.assert_allclose(l, lse[b, :n], atol=1e-12)
        assert (mass >= np.abs(o)).all() and (size > 0).all()


def test_nested_residuals_collapse():
    """max(max(p - a q, 0) - R q, 0) = max(p - (a + R) q, 0), the kernel's form."""
    rng = np.random.default_rng(0)
    p, q = rng.dirichlet(np.ones(50)), rng.dirichlet(np.ones(50))
    r, mass, a = p, 1.0, 0.0
    for _ in range(5):
        r = np.maximum(r - mass * q, 0)
        a += mass
        mass = r.sum()
        np.testing.assert_allclose(r, np.maximum(p - a * q, 0), atol=1e-15)


def test_oracle_verification_keeps_the_targets_distribution():
    """Exact expectation over u on a grid: one draft over three tokens."""
    p, q = np.array([.5, .3, .2]), np.array([.2, .2, .6])
    share = np.zeros(3)
    grid = (np.arange(100) + .5) / 100
    tok = np.array([[0, 0]], dtype=np.int32)
    par, ln = np.array([[-1, 0]]), [2]
    for d in range(3):
        tok[0, 1] = d
        for u in grid:
            for us in grid[::5]:
                _, t, _, _ = spec.verify_tree(np.tile(p, (1, 2, 1)), np.tile(q, (1, 2, 1)), tok, par,
                                              ln, np.array([[0, u]]), np.array([us]))
                share[t[0, 0]] += q[d] / (100 * 20)
    np.testing.assert_allclose(share, p, atol=0.02)   # grid steps of 1/100 and 1/20 of a third


def test_page_counts_are_the_tables():
    rng = np.random.default_rng(1)
    st = S.pages_state(1, [30, 10, 50], 16, 1, 60, 6, slots=10)
    lens = {1: 30, 2: 10, 3: 50}
    for _ in range(40):
        d = int(rng.integers(1, 10))
        s = d if rng.random() < 0.5 else int(rng.choice(list(lens)))
        keep = int(rng.integers(0, lens.get(s, 0) + 1))
        new = min(keep + int(rng.integers(0, 30)), 96)
        st.k, st.v, st.table, st.refs, err = spec.update_pages(st.k, st.v, st.table, st.refs, [d],
                                                               [s], [keep], [new], 16)
        if not err:
            lens[d] = new
        uses = np.bincount(st.table[st.table > 0], minlength=60)
        assert np.array_equal(uses[1:], st.refs[1:])
    k, v, table, refs, n, err = spec.compact_pages(st.k, st.v, st.table, st.refs, 16)
    assert err == 0 and (refs[:n] > 0).all() and (refs[n:] == 0).all() and table.max() < n
    for slot in range(1, 10):
        for b, e in enumerate(st.table[slot]):
            if e > 0:
                assert np.array_equal(k[table[slot, b] * 16:][:16], st.k[e * 16:][:16])
