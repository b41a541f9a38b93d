"""The operators of a paged cache of shared latents on the GPU, against the float64 oracle."""

import numpy as np
import pytest
import torch

import oracle.latent as orl
from paged_kv_gqa_pkv_gb300 import binding
from tests import latent_cases as C

pytestmark = pytest.mark.gpu

BAD_PAGE, BAD_SLOT, BAD_POS, LAYOUT = (binding.DEV_ERR_BAD_PAGE, binding.DEV_ERR_BAD_SLOT,
                                       binding.DEV_ERR_BAD_POS, binding.DEV_ERR_LAYOUT)


def new_err():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ rotate --

def check_rotated(y, x, pos, cos, sin, inter):
    """y: the kernel's [T, H, dims]. Products and their sum are off by about an fp32 step of the
    result (2^-22 allows four), the result by half a bf16 step: 2^-8 of it."""
    p = pos.long()
    want = orl.rotate(x.double().numpy(), cos[p].double().numpy()[:, None],
                      sin[p].double().numpy()[:, None], inter)
    err = np.abs(y.double().cpu().numpy() - want)
    assert (err <= (2.0 ** -8 + 2.0 ** -22) * np.abs(want) + 1e-38).all()


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("T,H,dims", [(1, 1, 64), (3, 5, 64), (17, 128, 64), (130, 7, 32), (5, 3, 128),
                                      (9, 4, 2), (6, 2, 10), (4, 9, 24), (2, 1, 8), (33, 6, 256)])
def test_rotate(T, H, dims, inter):
    g = C.gen(T * 1000 + H * 10 + dims)
    x = C.normal(g, T, H, dims)
    pos = torch.randint(0, 500, (T,), generator=g, dtype=torch.int32)
    pos[0] = 499
    cos, sin = C.rope_tables(500, dims)
    y = binding.pkv_rotate(x.cuda(), pos.cuda(), cos.cuda(), sin.cuda(), interleaved=inter)
    check_rotated(y, x, pos, cos, sin, inter)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("off,tail", [(128, 0), (8, 8), (3, 1), (1, 6)])
def test_rotate_part_of_a_head(off, tail, inter):
    """A slice of each head, in place, into another tensor's slice, and through a transposed view;
    the values around it stay."""
    g = C.gen(off * 7 + tail)
    T, H, dims = 21, 6, 64
    full = C.normal(g, T, H, off + dims + tail)
    x = full[..., off:off + dims]
    pos = torch.randint(0, 300, (T,), generator=g, dtype=torch.int32)
    cos, sin = C.rope_tables(300, dims)
    args = (pos.cuda(), cos.cuda(), sin.cuda())
    a = full.cuda()
    binding.pkv_rotate(a[..., off:off + dims], *args, interleaved=inter, out=a[..., off:off + dims])
    check_rotated(a[..., off:off + dims], x, pos, cos, sin, inter)
    assert torch.equal(a[..., :off].cpu(), full[..., :off])
    assert torch.equal(a[..., off + dims:].cpu(), full[..., off + dims:])
    b = torch.full((T, H, 40 + dims), 7.0, dtype=torch.bfloat16, device="cuda")
    y = binding.pkv_rotate(full.cuda()[..., off:off + dims], *args, interleaved=inter, out=b[..., 40:])
    assert y.data_ptr() == b[..., 40:].data_ptr()
    check_rotated(b[..., 40:], x, pos, cos, sin, inter)
    assert (b[..., :40] == 7.0).all()
    # heads outside, tokens inside
    t = x.transpose(0, 1).contiguous().cuda().transpose(0, 1)
    o = torch.empty((H, T, dims), dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    check_rotated(binding.pkv_rotate(t, *args, interleaved=inter, out=o), x, pos, cos, sin, inter)
    # one token's values for all tokens (stride 0)
    r = x[:1].contiguous().cuda().expand(T, H, dims)
    check_rotated(binding.pkv_rotate(r, *args, interleaved=inter), x[:1].expand(T, H, dims), pos, cos, sin, inter)


def test_rotate_cancellation():
    """Pairs whose products nearly cancel keep their relative accuracy."""
    T, dims = 64, 64
    cos, sin = C.rope_tables(T, dims)
    pos = torch.arange(T, dtype=torch.int32)
    x = torch.empty(T, 1, dims)
    x[:, 0, :32] = sin
    x[:, 0, 32:] = cos
    x = x.to(torch.bfloat16)
    y = binding.pkv_rotate(x.cuda(), pos.cuda(), cos.cuda(), sin.cuda())
    check_rotated(y, x, pos, cos, sin, False)


def test_rotate_bad_positions():
    g = C.gen(5)
    x = C.normal(g, 4, 3, 64)
    cos, sin = C.rope_tables(10, 64)
    out = torch.full((4, 3, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    err = new_err()
    pos = C.i32([9, 10, -1, 0])
    binding.pkv_rotate(x.cuda(), pos.cuda(), cos.cuda(), sin.cuda(), out=out, dev_err=err)
    assert err.item() == BAD_POS
    assert (out[1:3] == 5.0).all()
    keep = torch.tensor([0, 3])
    check_rotated(out[keep.cuda()], x[keep], pos[keep], cos, sin, False)


# ------------------------------------------------------------------ append --

@pytest.mark.parametrize("inter,norm", [(False, False), (True, False), (False, True), (True, True)])
@pytest.mark.parametrize("n,ps,stride", [(1, 16, 576), (7, 48, 576), (37, 64, 640), (20, 128, 584)])
def test_append(n, ps, stride, inter, norm):
    g = C.gen(n * 10 + ps)
    slots, longest = 3, 70
    pool, table = C.cache(g, slots, longest, ps)
    pairs = torch.randperm(slots * longest, generator=g)[:n]
    slot, pos = (pairs // longest + 1).to(torch.int32), (pairs % longest).to(torch.int32)
    if n > 5:
        slot[2] = 0  # padding
    wide = C.normal(g, n, stride, scale=3.0)
    weight = 1 + 0.2 * torch.randn(512, generator=g) if norm else None
    cos, sin = C.rope_tables(longest, 64)
    want, bad = orl.append(orl.bf16_bits_to_f64(C.bits(pool)), table.numpy(), C.bits(wide[:, :576].contiguous()),
                           slot.numpy(), pos.numpy(), ps, cos.numpy(), sin.numpy(), inter,
                           None if weight is None else weight.numpy())
    assert not bad
    got, err = pool.cuda(), new_err()
    binding.pkv_latent_append(got, table.cuda(), wide.cuda()[:, :576], slot.cuda(), pos.cuda(), ps, cos.cuda(),
                              sin.cuda(), norm_weight=None if weight is None else weight.cuda(), interleaved=inter,
                              dev_err=err)
    assert err.item() == 0
    got = got.cpu().double().numpy()
    # one rounding to bf16 (2^-8), fp32 before it: the sum of 512 squares in a tree and the root, 2^-20
    assert (np.abs(got - want) <= (2.0 ** -8 + 2.0 ** -20) * np.abs(want) + 1e-38).all()
    touched = (want != orl.bf16_bits_to_f64(C.bits(pool))).any(1)
    assert np.array_equal(got[~touched], pool.double().numpy()[~touched])
    if not norm:
        assert np.array_equal(got[:, :512], want[:, :512])


def test_append_errors():
    g = C.gen(9)
    pool, table = C.cache(g, 2, 64, 16)
    table[2, 1] = pool.shape[0] // 16  # one past the pool
    cos, sin = C.rope_tables(50, 64)
    x = C.normal(g, 7, 576)
    for slot, pos, bit in ((3, 0, BAD_SLOT), (-1, 0, BAD_SLOT), (1, -1, BAD_POS), (1, 80, BAD_POS), (1, 50, BAD_POS),
                           (2, 16, BAD_PAGE)):
        got, err = pool.cuda(), new_err()
        slots, poss = C.i32([1, slot, 2]).cuda(), C.i32([3, pos, 5]).cuda()
        binding.pkv_latent_append(got, table.cuda(), x[:3].cuda(), slots, poss, 16, cos.cuda(), sin.cuda(), dev_err=err)
        assert err.item() == bit, (slot, pos)
        changed = (got.cpu() != pool).any(1).nonzero().flatten().tolist()
        assert changed == sorted([int(table[1, 0]) * 16 + 3, int(table[2, 0]) * 16 + 5])


# ------------------------------------------------------------------ gather --

@pytest.mark.parametrize("ps", [16, 48, 128])
@pytest.mark.parametrize("lens", [[1], [5, 0, 1, 130, 0], [33, 32, 31], [0, 0]])
def test_gather(lens, ps):
    g = C.gen(ps + sum(lens))
    pool, table = C.cache(g, len(lens), max(max(lens), 1), ps)
    slots = C.i32((torch.randperm(len(lens), generator=g) + 1).tolist())
    first = 3
    starts = C.i32([first + sum(lens[:i]) for i in range(len(lens) + 1)])
    total = int(starts[-1]) + 4
    before = C.normal(g, total, 576)
    err = new_err()
    got = binding.pkv_latent_gather(pool.cuda(), table.cuda(), slots.cuda(), starts.cuda(), total, ps, out=before.cuda(),
                                    dev_err=err)
    want = orl.gather(C.bits(pool), table.numpy(), slots.numpy(), starts.numpy(), C.bits(before), ps)
    assert np.array_equal(C.bits(got.cpu()), want)
    assert err.item() == 0


def test_gather_errors():
    g = C.gen(3)
    pool, table = C.cache(g, 3, 40, 16)
    table[2, 1] = -1
    before = C.normal(g, 100, 576)
    # slot 0 stays as it was; a page, a slot and a position out of range; starts that do not ascend
    for slots, starts, bit in (([1, 0, 3], [0, 20, 40, 60], 0), ([1, 2, 3], [0, 20, 40, 60], BAD_PAGE),
                               ([1, 4, 3], [0, 20, 40, 60], BAD_SLOT), ([1, 3, 3], [0, 20, 20, 90], BAD_POS),
                               ([1, 3, 3], [0, 30, 20, 40], LAYOUT), ([1, 3, 3], [0, 20, 40, 101], LAYOUT),
                               ([1, 3, 3], [-5, 20, 40, 60], LAYOUT)):
        err = new_err()
        got = binding.pkv_latent_gather(pool.cuda(), table.cuda(), C.i32(slots).cuda(), C.i32(starts).cuda(), 100, 16,
                                        out=before.cuda(), dev_err=err)
        assert err.item() & bit == bit and (bit or err.item() == 0), (slots, starts)
        if bit != LAYOUT:
            want = orl.gather(C.bits(pool), table.numpy(), np.array(slots), np.array(starts), C.bits(before), 16)
            assert np.array_equal(C.bits(got.cpu()), want)


# ------------------------------------------------------------------ decode --

def run_decode(pool, table, q, slots, lens, ps, **kw):
    err = new_err()
    out, lse = binding.pkv_latent_decode_attention(pool.cuda(), table.cuda(), q.cuda(), slots.cuda(), lens.cuda(), ps,
                                                   C.SCALE, dev_err=err, **kw)
    torch.cuda.synchronize()
    return out.cpu(), lse.cpu(), err.item()


def decode_case(seed, lens, n_q, H, ps, slots=None, marker=float("nan"), q_scale=1.0):
    """Unused rows of the pool hold `marker`."""
    g = C.gen(seed)
    B = len(lens)
    pool, table = C.cache(g, B, max(max(lens), 1), ps, marker=marker)
    for b, n in enumerate(lens):
        blocks = table[b + 1]
        for t in range(n, (table.shape[1] - 1) * ps):
            pool[int(blocks[t // ps]) * ps + t % ps] = marker
    q = C.normal(g, B, n_q, H, 576, scale=q_scale)
    slots = C.i32(list(range(1, B + 1))) if slots is None else C.i32(slots)
    return pool, table, q, slots, C.i32(lens)


def check_decode(case, ps, tag="", **kw):
    pool, table, q, slots, lens = case
    out, lse, err = run_decode(pool, table, q, slots, lens, ps, **kw)
    want = orl.decode(C.bits(q), C.bits(pool), table.numpy(), slots.numpy(), lens.numpy(), ps, C.SCALE)
    C.check_attention(out, lse, want, 576, tag)
    return err


@pytest.mark.parametrize("lens", [[1], [15], [16], [17], [63], [64], [65], [127], [128], [129], [300]])
def test_decode_lengths(lens):
    """Every kind of tile end, one sequence; rows past the end hold NaN."""
    assert check_decode(decode_case(lens[0], lens, 1, 8, 16), 16) == 0


@pytest.mark.parametrize("H", [1, 2, 7, 16, 33, 64, 65, 100, 128])
def test_decode_heads(H):
    assert check_decode(decode_case(H, [77, 200, 5], 1, H, 64), 64) == 0


@pytest.mark.parametrize("n_q,H", [(2, 16), (3, 5), (4, 32), (8, 16), (2, 128), (3, 64), (5, 40), (64, 2)])
def test_decode_drafts(n_q, H):
    """Several tokens a row, also more than 128 rows, and sequences shorter than their drafts."""
    lens = [n_q, 150, 1, 131, 64 + n_q]
    assert check_decode(decode_case(n_q * 100 + H, lens, n_q, H, 32), 32) == 0


@pytest.mark.parametrize("ps", [16, 32, 48, 64, 96, 128, 256])
def test_decode_page_sizes(ps):
    assert check_decode(decode_case(ps, [300, 1, 129], 1, 12, ps), ps) == 0


def test_decode_padding_and_empty_rows():
    """Padding rows, empty sequences and their neighbours; the same slot in two rows."""
    g = C.gen(1)
    pool, table = C.cache(g, 3, 200, 16)
    q = C.normal(g, 7, 1, 16, 576)
    slots, lens = C.i32([0, 1, 2, 0, 3, 1, 2]), C.i32([50, 0, 200, 0, 3, 77, 200])
    assert check_decode((pool, table, q, slots, lens), 16) == 0
    # nothing at all to do
    assert check_decode((pool, table, q, C.i32([0] * 7), lens), 16) == 0


def test_decode_one_token_without_its_axis():
    pool, table, q, slots, lens = decode_case(3, [40, 41], 1, 16, 16)
    a = run_decode(pool, table, q, slots, lens, 16)
    b = run_decode(pool, table, q[:, 0].contiguous(), slots, lens, 16)
    assert b[0].shape == (2, 16, 512) and b[1].shape == (2, 16)
    assert torch.equal(a[0][:, 0], b[0]) and torch.equal(a[1][:, 0], b[1])


def test_decode_large_scores():
    """Scores in the hundreds, whose maximum moves along the sequence: the running maximum has to."""
    pool, table, q, slots, lens = decode_case(11, [700, 650], 1, 16, 16, q_scale=40.0)
    for b in range(2):
        for t in range(int(lens[b])):
            row = int(table[b + 1, t // 16]) * 16 + t % 16
            pool[row] = (pool[row].float() * (0.2 + 2.0 * t / 700)).to(torch.bfloat16)
    assert check_decode((pool, table, q, slots, lens), 16) == 0


def test_decode_many_rows():
    """Ragged lengths over the whole range, split items and whole ones side by side."""
    g = torch.Generator().manual_seed(77)
    lens = torch.randint(0, 1500, (40,), generator=g).tolist()
    assert check_decode(decode_case(5, lens, 1, 4, 64, marker=0.0), 64) == 0


def test_decode_long():
    """A long sequence alone: one item over all the workers."""
    assert check_decode(decode_case(6, [20000], 1, 3, 128, marker=0.0), 128) == 0


def test_decode_more_rows_than_a_launch():
    g = C.gen(2)
    B = 1100
    pool, table = C.cache(g, 5, 40, 16)
    slots = C.i32([1 + i % 5 for i in range(B)])
    lens = C.i32([i % 41 for i in range(B)])
    q = C.normal(g, B, 1, 2, 576)
    assert check_decode((pool, table, q, slots, lens), 16) == 0


def test_decode_errors():
    pool, table, q, slots, lens = decode_case(8, [40, 90, 33, 64], 1, 16, 16, marker=0.0)
    for b, s, n, bit in ((1, 5, 90, BAD_SLOT), (1, -2, 90, BAD_SLOT), (2, 3, -1, BAD_POS), (0, 1, 113, BAD_POS)):
        sl, ln = slots.clone(), lens.clone()
        sl[b], ln[b] = s, n
        assert check_decode((pool, table, q, sl, ln), 16, tag=str((b, s, n))) == bit
    t = table.clone()
    t[2, 3] = -1
    out, lse, err = run_decode(pool, t, q, slots, lens, 16)
    assert err == BAD_PAGE
    want = orl.decode(C.bits(q), C.bits(pool), table.numpy(), slots.numpy(), lens.numpy(), 16, C.SCALE)
    others = [0, 2, 3]
    C.check_attention(out[others], lse[others], [w[others] for w in want], 576)


def test_decode_same_bits_every_time():
    case = decode_case(21, [700, 3, 0, 1200, 64], 2, 16, 64, marker=0.0)
    first = run_decode(*case[:5], 64)
    for _ in range(5):
        again = run_decode(*case[:5], 64)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_decode_workspace():
    """A caller's workspace full of NaN; one that is too small is refused."""
    pool, table, q, slots, lens = decode_case(22, [900, 130], 1, 16, 64, marker=0.0)
    n = binding.pkv_latent_decode_workspace_size(pool.cuda(), table.cuda(), 64, 2, 1, 16)
    ws = torch.full((n // 4,), float("nan"), device="cuda")
    a = run_decode(pool, table, q, slots, lens, 64, workspace=ws)
    b = run_decode(pool, table, q, slots, lens, 64)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    with pytest.raises(binding.PkvError):
        run_decode(pool, table, q, slots, lens, 64, workspace=ws[:n // 4 - 64])
