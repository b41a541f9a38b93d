"""The operators of shared latents together, as a model's layer calls them: prompts in chunks, decode steps with
drafts, graphs, streams, long pools, the calls that the documentation allows and nothing else makes."""

import numpy as np
import pytest
import torch

import oracle.latent as orl
from paged_kv_gqa_pkv_gb300 import binding as pkv
from tests import latent_cases as C

pytestmark = pytest.mark.gpu

H = 4  # heads whose up-projections take a quarter of the latent each: exact in bf16


class Layer:
    """One layer's cache and calls. Head h's keys and values are the values 128 h .. 128 h + 127 of the latent, so the
    expanded tensors and the absorbed queries are exact copies, and both forms see the same numbers."""

    def __init__(self, slots, longest, ps, seed=0):
        g = C.gen(seed)
        pool, table = C.cache(g, slots, longest, ps, marker=float("nan"))
        self.pool, self.table, self.ps = torch.full_like(pool, float("nan")).cuda(), table.cuda(), ps
        self.cos, self.sin = (t.cuda() for t in C.rope_tables(longest, 64))
        self.weight = (1 + 0.1 * torch.randn(512, generator=g)).cuda()
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def append(self, x, slot, pos, **kw):
        pkv.pkv_latent_append(self.pool, self.table, x, slot, pos, self.ps, self.cos, self.sin, norm_weight=self.weight,
                              interleaved=True, dev_err=self.err, **kw)

    def prefill(self, q, pos, slots, q_starts, k_starts, total):
        pkv.pkv_rotate(q[..., 128:], pos, self.cos, self.sin, interleaved=True, out=q[..., 128:], dev_err=self.err)
        rows = pkv.pkv_latent_gather(self.pool, self.table, slots, k_starts, total, self.ps, dev_err=self.err)
        own = rows[:, :512].view(total, H, 128)
        return pkv.pkv_latent_prefill_attention(q, own, rows[:, 512:], own, q_starts, k_starts, C.SCALE, dev_err=self.err)

    def absorb(self, q, pos):
        """[T, H, 192] -> [T, H, 576]: each head's own part at its quarter, the rotated part behind the latent."""
        out = torch.zeros(q.shape[0], H, 576, dtype=q.dtype, device=q.device)
        for h in range(H):
            out[:, h, 128 * h:128 * h + 128] = q[:, h, :128]
        pkv.pkv_rotate(q[..., 128:], pos, self.cos, self.sin, interleaved=True, out=out[..., 512:], dev_err=self.err)
        return out

    def decode(self, q, slot, lens, **kw):
        return pkv.pkv_latent_decode_attention(self.pool, self.table, q, slot, lens, self.ps, C.SCALE, dev_err=self.err, **kw)


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("ps", [16, 64])
def test_prompts_in_chunks_then_steps(ps):
    """Two prompts in chunks through the expanded form, then steps of two tokens through the absorbed one, every result
    against the definition over the cache's own rows; and the last chunk through both forms."""
    g = C.gen(ps)
    lens, chunk = [150, 70], 64
    layer = Layer(2, 200, ps)
    done = [0, 0]
    while any(d < n for d, n in zip(done, lens)):
        take = [min(chunk, n - d) for d, n in zip(done, lens)]
        slot = i32([b + 1 for b in range(2) for _ in range(take[b])])
        pos = i32([done[b] + i for b in range(2) for i in range(take[b])])
        x = C.normal(g, sum(take), 640, scale=2.0).cuda()[:, 32:608]  # a slice of a wider projection
        layer.append(x, slot, pos)
        ends = [done[b] + take[b] for b in range(2)]
        q_starts, k_starts = i32([0, take[0], sum(take)]), i32([0, ends[0], sum(ends)])
        raw = C.normal(g, sum(take), H, 192).cuda()
        q = raw.clone()
        out, lse = layer.prefill(q, pos, i32([1, 2]), q_starts, k_starts, sum(ends))
        assert layer.err.item() == 0
        rows = pkv.pkv_latent_gather(layer.pool, layer.table, i32([1, 2]), k_starts, sum(ends), ps).cpu()
        own = rows[:, :512].reshape(sum(ends), H, 128)
        want = orl.prefill(C.bits(q.cpu()), C.bits(own), C.bits(rows[:, 512:].contiguous()), C.bits(own), q_starts.tolist(),
                           k_starts.tolist(), C.SCALE)
        C.check_attention(out.cpu(), lse.cpu(), want, 192, "chunk")
        done = ends
        # the same queries through the absorbed form, one row of the batch per token
        a = layer.absorb(raw, pos)
        a_out, a_lse = layer.decode(a, slot, pos + 1)
        picked = torch.stack([a_out[:, h, 128 * h:128 * h + 128] for h in range(H)], 1)
        C.check_attention(picked.cpu(), a_lse.cpu(), want, 576, "chunk, absorbed")
    for _ in range(3):  # steps of two tokens a sequence
        slot, pos = i32([1, 1, 2, 2]), i32([done[0], done[0] + 1, done[1], done[1] + 1])
        layer.append(C.normal(g, 4, 576, scale=2.0).cuda(), slot, pos)
        done = [d + 2 for d in done]
        q = layer.absorb(C.normal(g, 4, H, 192).cuda(), pos)
        out, lse = layer.decode(q.view(2, 2, H, 576), i32([1, 2]), i32(done))
        pool = layer.pool.cpu()
        want = orl.decode(C.bits(q.view(2, 2, H, 576).cpu()), C.bits(pool), layer.table.cpu().numpy(), np.array([1, 2]),
                          np.array(done), ps, C.SCALE)
        C.check_attention(out.cpu(), lse.cpu(), want, 576, "step")
    assert layer.err.item() == 0


def _step_inputs(seed, B=5, longest=300):
    g = C.gen(seed)
    lens = torch.randint(1, longest, (B,), generator=g, dtype=torch.int32)
    lens[1] = 0
    return dict(x=C.normal(g, B, 576).cuda(), q=C.normal(g, B, H, 192).cuda(), slot=i32([1, 2, 3, 0, 5][:B]), lens=lens.cuda(),
                pos=(lens - 1).clamp(min=0).cuda())


def _step(layer, s):
    layer.append(s["x"], s["slot"], s["pos"])
    return layer.decode(layer.absorb(s["q"], s["pos"]), s["slot"], s["lens"])


def test_captured_steps():
    """Append, rotation and decode captured without buffers, replayed with other inputs and lengths in the same tensors;
    two graphs whose decodes share a caller's workspace; a prefill beside them."""
    layers = [Layer(5, 300, 16, seed=k) for k in range(2)]
    for layer in layers:
        layer.pool.copy_(C.normal(C.gen(9), *layer.pool.shape).cuda())
    s = _step_inputs(1)
    ws = torch.empty(pkv.pkv_latent_decode_workspace_size(layers[0].pool, layers[0].table, 16, 5, 1, H), dtype=torch.uint8,
                     device="cuda")
    q_starts, k_starts = i32([0, 3, 5]), i32([0, 40, 45])
    kv = C.normal(C.gen(3), 45, H, 256).cuda()
    rows = C.normal(C.gen(4), 45, 576).cuda()

    def calls(layer, **kw):
        layer.append(s["x"], s["slot"], s["pos"])
        a = layer.decode(layer.absorb(s["q"], s["pos"]), s["slot"], s["lens"], **kw)
        b = pkv.pkv_latent_prefill_attention(s["q"], kv[..., :128], rows[:, 512:], kv[..., 128:], q_starts, k_starts, C.SCALE)
        c = pkv.pkv_latent_gather(layer.pool, layer.table, i32_slots, k_starts, 45, 16)
        return (*a, *b, c)

    i32_slots = i32([1, 2])
    graphs, results = [], []
    for k, kw in ((0, {}), (1, dict(workspace=ws)), (0, dict(workspace=ws))):
        calls(layers[k], **kw)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            results.append(calls(layers[k], **kw))
        graphs.append(graph)
    for seed in (5, 6, 7):
        new = _step_inputs(seed)
        for name in s:
            s[name].copy_(new[name])
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for k, got in ((0, results[0]), (1, results[1]), (0, results[2])):
            for a, b in zip(got, calls(layers[k])):
                assert torch.equal(a, b)
        assert layers[0].err.item() == 0


def test_streams():
    """Calls on a named stream while the current one is busy with other tensors: results, buffers and the order of the
    calls belong to the named one."""
    layer = Layer(5, 300, 16)
    layer.pool.copy_(C.normal(C.gen(9), *layer.pool.shape).cuda())
    s = _step_inputs(2)
    want = _step(layer, s)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(5):
        q = layer.absorb(s["q"], s["pos"])
        side.wait_stream(torch.cuda.current_stream())
        got = layer.decode(q, s["slot"], s["lens"], stream=side)
        rot = pkv.pkv_rotate(s["q"][..., 128:], s["pos"], layer.cos, layer.sin, stream=side)
        junk = [torch.full((1 << 20,), float("nan"), device="cuda") for _ in range(4)]  # takes no memory of the calls
        del junk
        side.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert torch.equal(rot, pkv.pkv_rotate(s["q"][..., 128:], s["pos"], layer.cos, layer.sin))
        torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.stream(side):
        got = _step(layer, s)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_two_streams_at_once():
    """Calls without a workspace of the caller's, side by side on two streams."""
    layers = [Layer(5, 300, 16, seed=k) for k in range(2)]
    for k, layer in enumerate(layers):
        layer.pool.copy_(C.normal(C.gen(20 + k), *layer.pool.shape).cuda())
    s = [_step_inputs(30 + k) for k in range(2)]
    q = [layers[k].absorb(s[k]["q"], s[k]["pos"]) for k in range(2)]
    want = [layers[k].decode(q[k], s[k]["slot"], s[k]["lens"]) for k in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        got = [layers[k].decode(q[k], s[k]["slot"], s[k]["lens"], stream=streams[k]) for k in range(2)]
        torch.cuda.synchronize()
        for k in range(2):
            assert torch.equal(got[k][0], want[k][0]) and torch.equal(got[k][1], want[k][1])


def test_long_pool():
    """A pool of 2.6e9 values: rows whose offsets pass 32 bits, written, read back and attended."""
    ps, pages = 64, 71000
    pool = torch.empty(pages * ps, 576, dtype=torch.bfloat16, device="cuda")
    g = C.gen(1)
    table = i32([[-1] * 3, [pages - 1, 5, pages - 7], [pages - 3, pages - 2, 9]])
    cos, sin = (t.cuda() for t in C.rope_tables(192, 64))
    n = 150
    x = C.normal(g, 2 * n, 576)
    slot, pos = i32([1] * n + [2] * n), i32(list(range(n)) * 2)
    pkv.pkv_latent_append(pool, table, x.cuda(), slot, pos, ps, cos, sin)
    rows = pkv.pkv_latent_gather(pool, table, i32([2, 1]), i32([0, n, 2 * n]), 2 * n, ps).cpu()
    assert torch.equal(rows[:n, :512], x[n:, :512]) and torch.equal(rows[n:, :512], x[:n, :512])
    q = C.normal(g, 2, 16, 576)
    out, lse = pkv.pkv_latent_decode_attention(pool, table, q.cuda(), i32([2, 1]), i32([n, n]), ps, C.SCALE)
    for b in range(2):
        c = orl.bf16_bits_to_f64(C.bits(rows[b * n:(b + 1) * n]))
        want = [np.stack(w)[None] for w in zip(*(orl.attend(orl.bf16_bits_to_f64(C.bits(q[b, h])), c, c[:, :512], C.SCALE)
                                                 for h in range(16)))]
        C.check_attention(out[b:b + 1].cpu(), lse[b:b + 1].cpu(), want, 576)


@pytest.mark.parametrize("n_q,heads,lens", [(64, 128, [70, 3]), (1, 1024, [40]), (64, 1, [64, 1, 200]), (7, 37, [9, 500])])
def test_decode_many_query_rows(n_q, heads, lens):
    """Up to 8192 query rows a sequence: many row blocks over the same keys, ragged ones among them."""
    g = C.gen(n_q + heads)
    pool, table = C.cache(g, len(lens), max(lens), 16)
    q = C.normal(g, len(lens), n_q, heads, 576)
    out, lse = pkv.pkv_latent_decode_attention(pool.cuda(), table.cuda(), q.cuda(), i32(range(1, len(lens) + 1)), i32(lens), 16,
                                               C.SCALE)
    want = orl.decode(C.bits(q), C.bits(pool), table.numpy(), np.arange(1, len(lens) + 1), np.array(lens), 16, C.SCALE)
    C.check_attention(out.cpu(), lse.cpu(), want, 576)


@pytest.mark.parametrize("lens", [[4000] * 3 + [5] * 90, [300] * 100, [1] * 200, [129] * 76, [9000], [2000, 2100, 1900, 50]])
def test_decode_schedules(lens):
    """Whole items, parts and ranges: results do not depend on how a batch is cut (each sequence alone gives the same
    numbers within the bounds)."""
    g = C.gen(len(lens))
    B, ps = len(lens), 64
    blocks = -(-max(lens) // ps)
    pool = C.normal(g, (1 + blocks * 4) * ps, 576)
    # all sequences read one of four slots' pages
    table = torch.full((B + 1, blocks), -1, dtype=torch.int32)
    for b in range(B):
        table[b + 1] = 1 + (b % 4) * blocks + torch.arange(blocks, dtype=torch.int32)
    q = C.normal(g, 4, 2, 576)[torch.arange(B) % 4].contiguous()
    out, lse = pkv.pkv_latent_decode_attention(pool.cuda(), table.cuda(), q.cuda(), i32(range(1, B + 1)), i32(lens), ps, C.SCALE)
    out, lse = out.cpu(), lse.cpu()
    seen = {}
    for b in range(B):
        key = (b % 4, lens[b])
        if key not in seen:
            seen[key] = [w[:, 0] for w in orl.decode(C.bits(q[b:b + 1, None]), C.bits(pool), table.numpy(), np.array([b + 1]),
                                                     np.array([lens[b]]), ps, C.SCALE)]
        C.check_attention(out[b:b + 1], lse[b:b + 1], seen[key], 576, f"row {b}")


def test_empty_calls():
    layer = Layer(2, 40, 16)
    bf = torch.bfloat16
    e = lambda *s, dt=bf: torch.empty(s, dtype=dt, device="cuda")  # noqa: E731
    none = e(0, dt=torch.int32)
    assert pkv.pkv_rotate(e(0, 4, 64), none, layer.cos, layer.sin).shape == (0, 4, 64)
    layer.append(e(0, 576), none, none)
    out, lse = layer.decode(e(0, 3, H, 576), none, none)
    assert out.shape == (0, 3, H, 512) and lse.shape == (0, 3, H)
    assert pkv.pkv_latent_gather(layer.pool, layer.table, none, i32([0]), 0, 16).shape == (0, 576)
    out, lse = pkv.pkv_latent_prefill_attention(e(0, H, 192), e(0, H, 128), e(0, 64), e(0, H, 128), i32([0]), i32([0]), 0.1)
    assert out.shape == (0, H, 128)
    # queries without any keys
    out, lse = pkv.pkv_latent_prefill_attention(torch.ones(3, H, 192, dtype=bf, device="cuda"), e(0, H, 128), e(0, 64),
                                                e(0, H, 128), i32([0, 3]), i32([0, 0]), 0.1)
    assert (out == 0).all() and torch.isneginf(lse).all()


def test_binding_refusals_on_the_gpu():
    layer = Layer(2, 40, 16)
    bf = torch.bfloat16
    q = torch.zeros(1, 2, 576, dtype=bf, device="cuda")
    one = i32([1])
    bad = [lambda: layer.decode(q.transpose(0, 1), one, one),                       # shapes
           lambda: layer.decode(q[..., :512], one, one),
           lambda: layer.decode(q.float(), one, one),
           lambda: layer.decode(q, one.long(), one),
           lambda: layer.decode(q, one.cpu(), one),
           lambda: layer.decode(q, one, i32([1, 1])),
           lambda: layer.decode(q, one, one, out=torch.empty(1, 2, 576, dtype=bf, device="cuda")),
           lambda: layer.append(torch.zeros(1, 600, dtype=bf, device="cuda"), one, one),
           lambda: layer.append(torch.zeros(576, 1, dtype=bf, device="cuda").t(), one, one),
           lambda: pkv.pkv_rotate(q[..., ::2], one, layer.cos, layer.sin),
           lambda: pkv.pkv_rotate(q[..., :63], one, layer.cos, layer.sin),
           lambda: pkv.pkv_rotate(q[..., :32], one, layer.cos, layer.sin),          # tables of 64 dims
           lambda: pkv.pkv_rotate(q[..., :64], i32([1, 2]), layer.cos, layer.sin),
           lambda: pkv.pkv_latent_gather(layer.pool, layer.table, one, i32([0, 1, 2]), 2, 16),
           lambda: pkv.pkv_latent_gather(layer.pool[:, :512], layer.table, one, i32([0, 1]), 2, 16),
           lambda: pkv.pkv_latent_gather(layer.pool, layer.table, one, i32([0, 1]), 2, 24)]
    for k, call in enumerate(bad):
        with pytest.raises((ValueError, TypeError, pkv.PkvError)):
            call()
    # a strided view whose rows would lie on one another
    x = torch.zeros(4, 2, 64, dtype=bf, device="cuda")
    with pytest.raises(pkv.PkvError):
        pkv.pkv_rotate(x, i32([0] * 4), layer.cos, layer.sin, out=x[:1].expand(4, 2, 64))
    # strides that no 16-byte load reaches
    wide = torch.zeros(3, H, 196, dtype=bf, device="cuda")[..., :192]
    kv = torch.zeros(3, H, 128, dtype=bf, device="cuda")
    with pytest.raises(pkv.PkvError):
        pkv.pkv_latent_prefill_attention(wide, kv, torch.zeros(3, 64, dtype=bf, device="cuda"), kv, i32([0, 3]), i32([0, 3]), 0.1)


def test_strides_of_single_tokens_and_heads():
    """The strides of an axis of length 1 are whatever the view left there."""
    g = C.gen(5)
    layer = Layer(2, 40, 16)
    odd = lambda t, k: t.as_strided(t.shape, tuple(3 if i == k else s for i, s in enumerate(t.stride())))  # noqa: E731
    x, pos = C.normal(g, 1, 4, 64).cuda(), i32([7])
    want = pkv.pkv_rotate(x, pos, layer.cos, layer.sin)
    assert torch.equal(pkv.pkv_rotate(odd(x, 0), pos, layer.cos, layer.sin), want)
    y = x.clone()
    pkv.pkv_rotate(odd(y, 0), pos, layer.cos, layer.sin, out=y)
    assert torch.equal(y, want)
    assert torch.equal(pkv.pkv_rotate(odd(x[:, :1], 1), pos, layer.cos, layer.sin), want[:, :1])
    q, k, r = C.normal(g, 5, 1, 192).cuda(), C.normal(g, 5, 1, 128).cuda(), C.normal(g, 5, 64).cuda()
    for n in (5, 1):
        a = (q[:n], k[:n], r[:n], k[:n])
        want = pkv.pkv_latent_prefill_attention(*a, i32([0, n]), i32([0, n]), C.SCALE)
        b = [odd(t, 1) if t.dim() == 3 else t for t in a]
        if n == 1:
            b = [odd(t, 0) for t in b]
        got = pkv.pkv_latent_prefill_attention(*b, i32([0, n]), i32([0, n]), C.SCALE)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
