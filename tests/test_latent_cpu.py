"""The operators of shared latents without a GPU: the C entries' and the binding's refusals, and
the oracle against closed forms and against itself."""

import ctypes
import math
import os

import numpy as np
import pytest
import torch

import oracle.latent as orl
from paged_kv_gqa_pkv_gb300 import binding
from tests import latent_cases as C

P = ctypes.c_void_p
F = ctypes.c_float


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.LIB_PATH):
        from paged_kv_gqa_pkv_gb300 import build
        build.build()
    return binding.load_library()


def _desc(**kw):
    d = dict(num_pages=32, page_size=16, num_kv_heads=1, head_dim=576, max_batch=5, max_blocks=16)
    d.update(kw)
    return ctypes.byref(binding.CacheDesc(**d))


BAD_CACHES = [dict(head_dim=128), dict(head_dim=512), dict(num_kv_heads=2), dict(num_kv_heads=0), dict(page_size=24),
              dict(page_size=0), dict(num_pages=0), dict(max_batch=0), dict(max_blocks=0),
              dict(num_pages=1 << 28, page_size=128), dict(max_blocks=1 << 28, page_size=128),
              dict(max_batch=1 << 16, max_blocks=1 << 16)]


# ------------------------------------------------------------ the C entries --

def test_rotate_refusals(lib):
    def call(x=256, xt=640, xh=64, out=512, ot=640, oh=64, T=3, H=10, dims=64, inter=0, pos=256, cos=256, sin=256, L=9,
             err=0):
        return lib.pkv_rotate(P(x), xt, xh, P(out), ot, oh, T, H, dims, inter, P(pos), P(cos), P(sin), L,
                              P(err) if err else None, None)
    assert call(T=0) == 0
    for kw in (dict(T=-1), dict(H=0), dict(dims=0), dict(dims=63), dict(dims=-2), dict(L=0), dict(inter=2), dict(inter=-1),
               dict(xt=-1), dict(xh=-8), dict(ot=-1), dict(oh=1 << 41), dict(x=0), dict(out=0), dict(pos=0), dict(cos=0),
               dict(sin=0),
               dict(oh=32), dict(ot=600), dict(ot=32, oh=640), dict(ot=64, oh=128),  # rows of out on one another
               dict(out=256, ot=1280)):                                             # in place with other strides
        assert call(**kw) == 1, kw
    # tokens inside heads, one head, one token: not on one another
    for kw in (dict(ot=64, oh=192), dict(H=1, oh=0), dict(T=1, ot=0), dict(out=256), dict(xt=0, xh=0)):
        assert call(**kw) in (5, 6), kw
    for kw in (dict(x=257), dict(out=513), dict(pos=258), dict(cos=257), dict(sin=258), dict(err=258)):
        assert call(**kw) == 2, kw


def test_append_refusals(lib):
    def call(desc=None, pool=256, table=256, x=256, xt=576, b=256, pos=256, n=4, cos=256, sin=256, L=9, inter=0, w=0, eps=1e-6,
             err=0):
        return lib.pkv_latent_append(desc or _desc(), P(pool), P(table), P(x), xt, P(b), P(pos), n, P(cos), P(sin), L, inter,
                                     P(w) if w else None, F(eps), P(err) if err else None, None)
    assert call(n=0) == 0
    for bad in BAD_CACHES:
        assert call(desc=_desc(**bad)) == 1, bad
    for kw in (dict(n=-1), dict(L=0), dict(inter=3), dict(xt=-8), dict(w=256, eps=-1.0), dict(w=256, eps=float("nan")),
               dict(w=256, eps=float("inf")), dict(pool=0), dict(table=0), dict(x=0), dict(b=0), dict(pos=0), dict(cos=0),
               dict(sin=0)):
        assert call(**kw) == 1, kw
    assert call(eps=-1.0) in (5, 6)  # ignored without a weight
    for kw in (dict(pool=264), dict(x=264), dict(xt=580), dict(cos=260), dict(sin=264), dict(w=260), dict(table=258),
               dict(b=257), dict(pos=258), dict(err=257)):
        assert call(**kw) == 2, kw


def test_gather_refusals(lib):
    def call(desc=None, pool=256, table=256, slots=256, starts=256, n=2, total=9, out=256, err=0):
        return lib.pkv_latent_gather(desc or _desc(), P(pool), P(table), P(slots), P(starts), n, total, P(out),
                                     P(err) if err else None, None)
    assert call(n=0) == 0 and call(total=0) == 0
    for bad in BAD_CACHES:
        assert call(desc=_desc(**bad)) == 1, bad
    for kw in (dict(n=-1), dict(total=-1), dict(pool=0), dict(table=0), dict(slots=0), dict(starts=0), dict(out=0)):
        assert call(**kw) == 1, kw
    for kw in (dict(pool=264), dict(out=264), dict(table=258), dict(slots=257), dict(starts=258), dict(err=257)):
        assert call(**kw) == 2, kw


def test_decode_refusals(lib):
    def call(desc=None, pool=256, table=256, q=256, H=16, b=256, n=256, B=4, nq=1, scale=0.1, out=256, lse=256, ws=256,
             nb=1 << 34, err=0):
        return lib.pkv_latent_decode_attention(desc or _desc(), P(pool), P(table), P(q), H, P(b), P(n), B, nq, F(scale), P(out),
                                               P(lse), P(ws), nb, P(err) if err else None, None)
    assert call(B=0) == 0
    for bad in BAD_CACHES:
        assert call(desc=_desc(**bad)) == 1, bad
    for kw in (dict(B=-1), dict(nq=0), dict(nq=65), dict(H=0), dict(H=1025), dict(B=1 << 24, nq=64, H=1024), dict(scale=0.0),
               dict(scale=-0.1), dict(scale=float("inf")), dict(scale=float("nan")), dict(pool=0), dict(table=0), dict(q=0),
               dict(b=0), dict(n=0), dict(out=0), dict(lse=0)):
        assert call(**kw) == 1, kw
    for kw in (dict(pool=264), dict(q=264), dict(out=264), dict(lse=258), dict(table=257), dict(b=258), dict(n=257),
               dict(ws=264), dict(err=257)):
        assert call(**kw) == 2, kw
    for args in ((4, 0, 16), (4, 65, 16), (4, 1, 0), (4, 1, 1025), (-1, 1, 16)):
        assert lib.pkv_latent_decode_workspace_size(_desc(), *args) == 0
    assert lib.pkv_latent_decode_workspace_size(_desc(head_dim=128), 4, 1, 16) == 0


def test_prefill_refusals(lib):
    def call(q=256, qt=1536, qh=192, k=256, kt=2048, kh=256, r=256, rt=576, v=256, vt=2048, vh=256, H=8, qs=256, ks=256, n=2,
             tq=9, tk=9, scale=0.1, out=256, lse=256, err=0):
        return lib.pkv_latent_prefill_attention(P(q), qt, qh, P(k), kt, kh, P(r), rt, P(v), vt, vh, H, P(qs), P(ks), n, tq, tk,
                                                F(scale), P(out), P(lse), P(err) if err else None, None)
    assert call(n=0) == 0 and call(tq=0) == 0
    for kw in (dict(H=0), dict(H=65536), dict(n=-1), dict(tq=-1), dict(tk=-1), dict(scale=0.0), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(qt=-8), dict(kh=1 << 38), dict(q=0), dict(k=0), dict(r=0), dict(v=0), dict(qs=0),
               dict(ks=0), dict(out=0), dict(lse=0), dict(n=1 << 30, H=8)):
        assert call(**kw) == 1, kw
    for kw in (dict(q=264), dict(k=264), dict(r=264), dict(v=264), dict(out=272), dict(lse=258), dict(qt=1540), dict(rt=580),
               dict(vh=260), dict(qs=257), dict(ks=258), dict(err=257)):
        assert call(**kw) == 2, kw
    assert call(k=0, r=0, v=0, tk=0) in (5, 6)  # no keys at all


# --------------------------------------------------------------- the binding --

def test_binding_refuses_host_tensors_and_wrong_shapes():
    bf, i32, f32 = torch.bfloat16, torch.int32, torch.float32
    pool, table = torch.zeros(64, 576, dtype=bf), torch.zeros(2, 4, dtype=i32)
    cos = torch.zeros(8, 32)
    one = torch.zeros(1, dtype=i32)
    calls = [lambda: binding.pkv_rotate(torch.zeros(1, 2, 64, dtype=bf), one, cos, cos),
             lambda: binding.pkv_rotate(torch.zeros(1, 2, dtype=bf), one, cos, cos),
             lambda: binding.pkv_latent_append(pool, table, torch.zeros(1, 576, dtype=bf), one, one, 16, cos, cos),
             lambda: binding.pkv_latent_gather(pool, table, one, torch.zeros(2, dtype=i32), 4, 16),
             lambda: binding.pkv_latent_decode_attention(pool, table, torch.zeros(1, 4, 576, dtype=bf), one, one, 16, 0.1),
             lambda: binding.pkv_latent_prefill_attention(torch.zeros(1, 2, 192, dtype=bf), torch.zeros(1, 2, 128, dtype=bf),
                                                          torch.zeros(1, 64, dtype=bf), torch.zeros(1, 2, 128, dtype=bf),
                                                          torch.zeros(2, dtype=i32), torch.zeros(2, dtype=i32), 0.1),
             lambda: binding.pkv_latent_prefill_attention(torch.zeros(1, 2, 128, dtype=bf), None, None, None, one, one, 0.1)]
    for call in calls:
        with pytest.raises((ValueError, TypeError)):
            call()
    with pytest.raises(ValueError):
        binding.latent_cache_desc(pool, table, 24)
    with pytest.raises(ValueError):
        binding.latent_cache_desc(pool, table, 0)


def test_a_descriptor_is_the_callers_own():
    """Writing to a descriptor changes neither the next one nor what calls of these sizes use."""
    pool, table = torch.zeros(64, 576, dtype=torch.bfloat16), torch.zeros(2, 4, dtype=torch.int32)
    want = dict(num_pages=4, page_size=16, num_kv_heads=1, head_dim=576, max_batch=2, max_blocks=4)
    fields = lambda d: {n: getattr(d, n) for n, _ in d._fields_}  # noqa: E731
    a = binding.latent_cache_desc(pool, table, 16)
    assert fields(a) == want
    a.num_pages, a.max_blocks = 1 << 20, 1
    assert fields(binding.latent_cache_desc(pool, table, 16)) == want
    assert fields(binding._latent_desc(64, 576, 16, 2, 4)[0]) == want


# ---------------------------------------------------------------- the oracle --

def test_rotation_forms():
    """Interleaved is the halves' form of the values put side by side; position 0 changes nothing; a
    rotation keeps every pair's length."""
    rng = np.random.default_rng(1)
    x = rng.standard_normal((5, 64))
    cos, sin = (t.double().numpy() for t in C.rope_tables(5, 64))
    order = np.concatenate([np.arange(0, 64, 2), np.arange(1, 64, 2)])
    a = orl.rotate(x, cos, sin, True)
    assert np.array_equal(a[:, order], orl.rotate(x[:, order], cos, sin, False))
    assert np.array_equal(a[0], x[0])
    assert np.allclose(a[:, 0::2] ** 2 + a[:, 1::2] ** 2, x[:, 0::2] ** 2 + x[:, 1::2] ** 2, rtol=0, atol=1e-6)


def test_rotated_products_depend_on_the_distance():
    rng = np.random.default_rng(2)
    q, k = rng.standard_normal(64), rng.standard_normal(64)
    f = 10000.0 ** (-np.arange(0, 64, 2) / 64)
    turn = lambda x, p: orl.rotate(x, np.cos(p * f), np.sin(p * f), False)  # noqa: E731
    assert math.isclose(turn(q, 100) @ turn(k, 93), turn(q, 1007) @ turn(k, 1000), rel_tol=0, abs_tol=1e-9)


def test_absorbed_and_expanded_forms_agree():
    """Scores and results through each head's up-projections, and in the latents' space."""
    rng = np.random.default_rng(3)
    n, H = 23, 3
    lat, rot = rng.standard_normal((n, 512)), rng.standard_normal((n, 64))
    q_own, q_rot = rng.standard_normal((H, 128)), rng.standard_normal((H, 64))
    uk, uv = rng.standard_normal((H, 128, 512)) / 20, rng.standard_normal((H, 128, 512)) / 20
    for h in range(H):
        k = np.concatenate([lat @ uk[h].T, rot], 1)
        out, lse, _, _ = orl.attend(np.concatenate([q_own[h], q_rot[h]]), k, lat @ uv[h].T, 0.07)
        absorbed = np.concatenate([q_own[h] @ uk[h], q_rot[h]])
        a_out, a_lse, _, _ = orl.attend(absorbed, np.concatenate([lat, rot], 1), lat, 0.07)
        assert np.allclose(uv[h] @ a_out, out, rtol=0, atol=1e-11) and math.isclose(a_lse, lse, rel_tol=0, abs_tol=1e-11)


def test_attend_closed_forms():
    v = np.array([[1.0, -2.0], [3.0, 4.0], [5.0, 0.5]])
    out, lse, mass, size = orl.attend(np.zeros(4), np.ones((3, 4)), v, 0.5)
    assert np.allclose(out, v.mean(0)) and math.isclose(lse, math.log(3)) and np.allclose(mass, np.abs(v).mean(0)) and size == 0
    out, lse, _, _ = orl.attend(np.ones(4), np.zeros((0, 4)), np.zeros((0, 2)), 0.5)
    assert (out == 0).all() and lse == -math.inf
    # one key far ahead of the others
    out, lse, _, _ = orl.attend(np.array([1.0]), np.array([[0.0], [2000.0], [0.0]]), v, 1.0)
    assert np.array_equal(out, v[1]) and lse == 2000.0


def test_decode_is_prefill_of_the_last_tokens():
    """Heads whose up-projections take the latent as it stands: the absorbed and the expanded forms'
    masks agree token by token."""
    g = C.gen(4)
    pool, table = C.cache(g, 1, 40, 16)
    q = C.normal(g, 1, 3, 1, 576)
    out, lse, _, _ = orl.decode(C.bits(q), C.bits(pool), table.numpy(), np.array([1]), np.array([37]), 16, 0.07)
    rows = [orl.pool_row(table.numpy(), 1, t, 16, pool.shape[0] // 16) for t in range(37)]
    c = orl.bf16_bits_to_f64(C.bits(pool))[rows]
    for j in range(3):
        o, l, _, _ = orl.attend(orl.bf16_bits_to_f64(C.bits(q))[0, j, 0], c[:35 + j], c[:35 + j, :512], 0.07)
        assert np.allclose(o, out[0, j, 0], rtol=0, atol=1e-12) and math.isclose(l, lse[0, j, 0], rel_tol=0, abs_tol=1e-12)


def test_append_then_gather():
    g = C.gen(5)
    pool, table = C.cache(g, 2, 30, 16)
    x = C.normal(g, 5, 576)
    cos, sin = (t.numpy() for t in C.rope_tables(30, 64))
    slots, pos = np.array([1, 1, 2, 0, 2]), np.array([0, 1, 29, 3, 28])
    new, bad = orl.append(orl.bf16_bits_to_f64(C.bits(pool)), table.numpy(), C.bits(x), slots, pos, 16, cos, sin)
    assert bad == []
    got = orl.gather(new, table.numpy(), np.array([2, 1]), np.array([0, 30, 32]), np.zeros((32, 576)), 16)
    assert np.array_equal(got[30, :512], orl.bf16_bits_to_f64(C.bits(x))[0, :512])
    assert np.array_equal(got[28:30, :512], orl.bf16_bits_to_f64(C.bits(x))[[4, 2], :512])
    assert np.array_equal(got[30, 512:], orl.bf16_bits_to_f64(C.bits(x))[0, 512:])  # position 0
    # a latent of equal values: its norm is 1 up to eps
    ones = torch.full((1, 576), 2.0, dtype=torch.bfloat16)
    new, _ = orl.append(orl.bf16_bits_to_f64(C.bits(pool)), table.numpy(), C.bits(ones), np.array([1]), np.array([0]), 16, cos,
                        sin, weight=np.full(512, 3.0), eps=0.0)
    assert np.allclose(new[orl.pool_row(table.numpy(), 1, 0, 16, 99), :512], 3.0, rtol=0, atol=1e-12)


def test_bounds_catch_a_mistake():
    """A kernel that leaves one key of 40 out, or takes one too many, is outside the bounds."""
    g = C.gen(6)
    pool, table = C.cache(g, 1, 40, 16)
    q = C.normal(g, 1, 1, 2, 576)
    want = orl.decode(C.bits(q), C.bits(pool), table.numpy(), np.array([1]), np.array([30]), 16, C.SCALE)
    as_gpu = lambda w: (torch.from_numpy(w[0]).to(torch.bfloat16), torch.from_numpy(w[1]).float())  # noqa: E731
    C.check_attention(*as_gpu(want), want, 576)
    for n in (29, 31):
        wrong = orl.decode(C.bits(q), C.bits(pool), table.numpy(), np.array([1]), np.array([n]), 16, C.SCALE)
        with pytest.raises(AssertionError):
            C.check_attention(*as_gpu(wrong), want, 576)


@pytest.mark.parametrize("place", [(1, 0), (1, None), (None, 2)])
def test_attend_beside_a_value_that_is_not_finite(place):
    """The helper of the GPU tests against numpy's own arithmetic."""
    rng = np.random.default_rng(8)
    q, k, v = rng.standard_normal(4), rng.standard_normal((5, 4)), rng.standard_normal((5, 3))
    for value in (math.nan, math.inf, -math.inf):
        for end in (2, 3, 5):
            k2, v2 = k.copy(), v.copy()
            if place[0] is not None:
                k2[2, place[0]] = value
            if place[1] is not None:
                v2[2, place[1]] = value
            out, lse, _, _ = C.attend_beside(q, k2, v2, end, 0.5, 2, place)
            with np.errstate(invalid="ignore"):
                x = 0.5 * (k2[:end] @ q)
                w = np.exp(x - x.max())
                plain, plain_lse = (w / w.sum()) @ v2[:end], x.max() + np.log(w.sum())
            assert np.allclose(plain, out, rtol=0, atol=1e-12, equal_nan=True)
            assert np.allclose(lse, plain_lse, rtol=0, atol=1e-12, equal_nan=True)
