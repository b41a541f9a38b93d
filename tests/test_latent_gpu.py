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


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dims", [64, 8, 10])
def test_rotated_infinities(dims, inter):
    """Infinite values give what the formula gives (infinities, NaN where it has inf - inf or inf * 0),
    in the rotation and in the append's position part; a NaN stays in its pair."""
    g = C.gen(dims)
    T, inf = 40, float("inf")
    x = C.normal(g, T, 3, dims)
    at = torch.randint(0, dims, (T, 3), generator=g)
    for i in range(1, T):
        x[i, 0, at[i, 0]] = (inf, -inf, float("nan"))[i % 3]
        x[i, 1, at[i, 1]] = x[i, 1, (at[i, 1] + (1 if inter else dims // 2)) % dims] = (inf, -inf)[i % 2]
    pos = torch.arange(T, dtype=torch.int32)
    cos, sin = C.rope_tables(T, dims)
    with np.errstate(invalid="ignore"):
        want = orl.rotate(x.double().numpy(), cos.double().numpy()[:, None], sin.double().numpy()[:, None], inter)
    odd = ~np.isfinite(want)

    def check(y, want, odd):
        y = y.double().cpu().numpy()
        assert np.array_equal(y[odd], want[odd], equal_nan=True)
        ok = np.abs(y[~odd] - want[~odd]) <= (2.0 ** -8 + 2.0 ** -22) * np.abs(want[~odd]) + 1e-38
        assert ok.all()

    check(binding.pkv_rotate(x.cuda(), pos.cuda(), cos.cuda(), sin.cuda(), interleaved=inter), want, odd)
    if dims != 64:
        return
    for h in range(3):
        new = torch.cat((C.normal(g, T, 512), x[:, h]), 1)
        pool, table = C.cache(g, 1, T, 16)
        got = pool.cuda()
        binding.pkv_latent_append(got, table.cuda(), new.cuda(), torch.ones_like(pos).cuda(), pos.cuda(), 16, cos.cuda(),
                                  sin.cuda(), interleaved=inter)
        rows = [orl.pool_row(table.numpy(), 1, t, 16, pool.shape[0] // 16) for t in range(T)]
        check(got[rows, 512:], want[:, h], odd[:, h])


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


@pytest.mark.parametrize("eps", [1e-6, 0.0])
def test_append_norm_of_very_large_and_small_latents(eps):
    """Latents whose squares leave fp32's range have their norm all the same."""
    g = C.gen(14)
    sizes = [1e18, 1e19, 1e25, 1e37, 1e-5, 1e-14, 1e-15, 1e-16, 1e-20, 1e-30, 1e-37]
    n = len(sizes)
    x = torch.cat(((torch.randn(n, 512, generator=g) * torch.tensor(sizes)[:, None]), torch.randn(n, 64, generator=g)), 1)
    x[3] = x[3].clamp(-3e38, 3e38)
    x[2, 7] = 3e38  # one value far ahead of the others
    x = x.to(torch.bfloat16)
    pool, table = C.cache(g, 1, n, 16)
    weight = 1 + 0.2 * torch.randn(512, generator=g)
    cos, sin = C.rope_tables(n, 64)
    pos, slot = torch.arange(n, dtype=torch.int32), torch.ones(n, dtype=torch.int32)
    want, _ = orl.append(orl.bf16_bits_to_f64(C.bits(pool)), table.numpy(), C.bits(x), slot.numpy(), pos.numpy(), 16,
                         cos.numpy(), sin.numpy(), weight=weight.numpy(), eps=eps)
    got = pool.cuda()
    binding.pkv_latent_append(got, table.cuda(), x.cuda(), slot.cuda(), pos.cuda(), 16, cos.cuda(), sin.cuda(),
                              norm_weight=weight.cuda(), norm_eps=eps)
    got = got.cpu().double().numpy()
    assert np.isfinite(want).all()
    # (a value that 2^-70 brings below 2^-126 is off by up to 2^-150, and the root of the mean square that divides
    # it is at least 2^-6: 2^-144, below 1e-38)
    assert (np.abs(got - want) <= (2.0 ** -8 + 2.0 ** -20) * np.abs(want) + 1e-38).all()


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


@pytest.mark.parametrize("short,n_short,long", [(100, 75, 9000), (128, 60, 20000), (1, 10, 5000)])
def test_decode_one_long_sequence_among_short_ones(short, n_short, long):
    """Items that just fill the workers, one of them far longer: equal ranges, not parts."""
    g = C.gen(short + long)
    ps, H = 64, 2
    blocks = -(-long // ps)
    table = torch.full((n_short + 2, blocks), -1, dtype=torch.int32)
    order = torch.randperm(2 * n_short + blocks, generator=g).to(torch.int32) + 1
    table[1:n_short + 1, :2] = order[:2 * n_short].view(-1, 2)
    table[n_short + 1] = order[2 * n_short:]
    pool = C.normal(g, (len(order) + 1) * ps, 576)
    at = n_short // 2
    lens = [short] * n_short
    slots = list(range(1, n_short + 1))
    lens.insert(at, long)
    slots.insert(at, n_short + 1)
    q = C.normal(g, n_short + 1, 1, H, 576)
    assert check_decode((pool, table, q, C.i32(slots), C.i32(lens)), ps) == 0


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


# a whole item; an item of several parts; ranges that begin and end inside items
@pytest.mark.parametrize("lens", [[300, 129, 40], [5000], [700, 90, 800] * 30], ids=["whole", "parts", "ranges"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("back,dim", [(1, 3), (2, 540), (3, 511), (39, 300), (40, 575)])
def test_decode_non_finite_row(lens, value, back, dim):
    """A value of a cached row that is not finite, `back` rows before the end: queries that see it
    tell so (NaN where its score is NaN or +inf), the others' lse and all other sequences are as
    without it."""
    n_q, H = 3, 2
    case = decode_case(len(lens) + dim, lens, n_q, H, 64, marker=0.0)
    pool, table, q, slots, ln = case
    clean = run_decode(*case, 64)
    b = len(lens) // 2
    at = lens[b] - back
    rows = [orl.pool_row(table.numpy(), b + 1, t, 64, pool.shape[0] // 64) for t in range(lens[b])]
    bad = pool.clone()
    bad[rows[at], dim] = value
    out, lse, err = run_decode(bad, table, q, slots, ln, 64)
    assert err == 0
    others = [i for i in range(len(lens)) if i != b]
    assert torch.equal(out[others], clean[0][others]) and torch.equal(lse[others], clean[1][others])
    c, qb = orl.bf16_bits_to_f64(C.bits(bad[rows])), orl.bf16_bits_to_f64(C.bits(q[b]))
    want, free = [], np.zeros((n_q * H, 512), bool)
    for j in range(n_q):
        for h in range(H):
            end = lens[b] - (n_q - 1 - j)
            want.append(C.attend_beside(qb[j, h], c, c[:, :512], end, C.SCALE, at, (dim, dim if dim < 512 else None)))
            if at >= end and dim < 512:
                free[j * H + h, dim] = True
    C.check_beside(out[b].view(-1, 512), lse[b].view(-1), want, 576, free)


@pytest.mark.parametrize("lens", [[300, 40], [5000]])
def test_decode_non_finite_query(lens):
    """One head's query is NaN, one's infinite: their rows are NaN and no other is touched."""
    case = decode_case(4, lens, 2, 5, 64, marker=0.0)
    clean = run_decode(*case, 64)
    q = case[2].clone()
    q[-1, 1, 3, 100], q[-1, 0, 2, 570] = float("nan"), float("inf")  # (rows of both signs: +inf among the scores)
    out, lse, _ = run_decode(case[0], case[1], q, *case[3:], 64)
    for j, h in ((1, 3), (0, 2)):
        assert out[-1, j, h].isnan().all() and lse[-1, j, h].isnan()
        out[-1, j, h], lse[-1, j, h] = clean[0][-1, j, h], clean[1][-1, j, h]
    assert torch.equal(out, clean[0]) and torch.equal(lse, clean[1])


def test_decode_both_ctas_of_a_pair():
    """Heads h and h + 64 with one query: their rows lie in different CTAs of a pair and run through
    the same steps, so one that took weights or values before they were there would differ. Every
    pair busy with several tiles, maxima that move, ragged ends; many calls."""
    g = C.gen(31)
    B, n = 90, 700
    pool, table = C.cache(g, 12, n, 64)
    pool *= torch.rand(pool.shape[0], 1, generator=g).to(torch.bfloat16) * 3
    q = C.normal(g, B, 1, 64, 576, scale=4.0).repeat(1, 1, 2, 1)
    slots = C.i32([1 + b % 12 for b in range(B)])
    lens = torch.randint(n // 2, n + 1, (B,), generator=g).to(torch.int32)
    args = pool.cuda(), table.cuda(), q.cuda(), slots.cuda(), lens.cuda(), 64, C.SCALE
    for _ in range(20):
        out, lse = binding.pkv_latent_decode_attention(*args)
        assert torch.equal(out[:, :, :64], out[:, :, 64:]) and torch.equal(lse[:, :, :64], lse[:, :, 64:])


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


# ----------------------------------------------------------------- prefill --

def prefill_case(seed, lens, H, before=0, after=0, q_scale=1.0):
    """lens: (queries, keys) of each sequence; `before`/`after` rows of no sequence around them."""
    g = C.gen(seed)
    q_starts, k_starts = [before], [before]
    for n, m in lens:
        q_starts.append(q_starts[-1] + n)
        k_starts.append(k_starts[-1] + m)
    tq, tk = q_starts[-1] + after, k_starts[-1] + after
    q = C.normal(g, tq, H, 192, scale=q_scale)
    kv = C.normal(g, tk, H, 256)
    rows = C.normal(g, tk, 576)
    return q, kv, rows, C.i32(q_starts), C.i32(k_starts)


def run_prefill(case, **kw):
    q, kv, rows, q_starts, k_starts = case
    kv, rows, err = kv.cuda(), rows.cuda(), new_err()
    out, lse = binding.pkv_latent_prefill_attention(q.cuda(), kv[..., :128], rows[:, 512:], kv[..., 128:], q_starts.cuda(),
                                                    k_starts.cuda(), C.SCALE, dev_err=err, **kw)
    torch.cuda.synchronize()
    return out.cpu(), lse.cpu(), err.item()


def check_prefill(case, tag="", rows=None, **kw):
    q, kv, lat, q_starts, k_starts = case
    out, lse, err = run_prefill(case, **kw)
    want = orl.prefill(C.bits(q), C.bits(kv[..., :128].contiguous()), C.bits(lat[:, 512:].contiguous()),
                       C.bits(kv[..., 128:].contiguous()), q_starts.tolist(), k_starts.tolist(), C.SCALE)
    a, b = int(q_starts[0]), int(q_starts[-1])
    C.check_attention(out[a:b], lse[a:b], [w[a:b] for w in want], 192, tag)
    return err


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 64, 65, 127, 128, 129, 200, 255, 256, 257, 300, 513])
def test_prefill_lengths(n):
    assert check_prefill(prefill_case(n, [(n, n)], 2)) == 0


@pytest.mark.parametrize("n,m", [(1, 700), (3, 130), (130, 131), (128, 256), (100, 1000), (300, 333), (257, 640)])
def test_prefill_behind_a_prefix(n, m):
    assert check_prefill(prefill_case(n + m, [(n, m)], 2)) == 0


@pytest.mark.parametrize("H", [1, 3, 8, 33])
def test_prefill_heads(H):
    assert check_prefill(prefill_case(H, [(70, 70), (5, 200)], H)) == 0


def test_prefill_packed():
    """Many sequences of all kinds, empty ones among them, rows of none before and behind."""
    lens = [(1, 1), (0, 0), (130, 130), (5, 300), (0, 40), (64, 64), (256, 300), (17, 17), (0, 0), (300, 301), (2, 2)]
    case = prefill_case(4, lens, 3, before=2, after=3)
    out = torch.full((case[0].shape[0], 3, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((case[0].shape[0], 3), 7.0, device="cuda")
    assert check_prefill(case, out=out, lse=lse) == 0
    assert (out[:2] == 7).all() and (out[-3:] == 7).all() and (lse[:2] == 7).all() and (lse[-3:] == 7).all()


def test_prefill_more_queries_than_keys():
    """The first queries see nothing: 0 and -inf."""
    assert check_prefill(prefill_case(5, [(10, 3), (300, 100), (200, 0), (4, 4)], 2)) == 0


def test_prefill_items_of_very_different_cost():
    """Items of one tile beside items of many, more items than SMs."""
    lens = [(700, 2000)] + [(3, 3)] * 40 + [(130, 140)] * 3 + [(1, 1500)] * 5
    assert check_prefill(prefill_case(6, lens, 4)) == 0


def test_prefill_neighbours_are_not_read():
    """NaN in every other sequence's rows, and in rows of none, reaches no result."""
    case = prefill_case(7, [(50, 50), (77, 205), (40, 40)], 2, before=4, after=4)
    q, kv, rows, qs, ks = case
    nan = float("nan")
    for s in range(3):
        kv2, rows2, q2 = kv.clone(), rows.clone(), q.clone()
        keep_k, keep_q = slice(int(ks[s]), int(ks[s + 1])), slice(int(qs[s]), int(qs[s + 1]))
        for t, keep in ((kv2, keep_k), (rows2, keep_k), (q2, keep_q)):
            saved = t[keep].clone()
            t.fill_(nan)
            t[keep] = saved
        a, b = run_prefill(case), run_prefill((q2, kv2, rows2, qs, ks))
        assert torch.equal(a[0][keep_q], b[0][keep_q]) and torch.equal(a[1][keep_q], b[1][keep_q])


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("where", ["own", "rotated", "v"])
@pytest.mark.parametrize("n,m,at", [(5, 5, 2), (140, 300, 170), (300, 300, 0), (300, 300, 299), (130, 400, 128), (1, 140, 139)])
def test_prefill_non_finite_key(n, m, at, where, value):
    """One key's or value's entry is not finite: queries that see it tell so, those before it have the
    same bits as without it (for a value: all but its dim, and lse), and so have other sequences."""
    case = prefill_case(n + m + at, [(20, 30), (n, m), (9, 9)], 2)
    q, kv, rows, qs, ks = case
    clean = run_prefill(case)
    kv2, rows2 = kv.clone(), rows.clone()
    key, dim = int(ks[1]) + at, 37
    if where == "own":
        kv2[key, 1, dim] = value
    elif where == "rotated":
        rows2[key, 512 + dim] = value
    else:
        kv2[key, 1, 128 + dim] = value
    out, lse, err = run_prefill((q, kv2, rows2, qs, ks))
    assert err == 0
    q0, q1, k0, k1 = int(qs[1]), int(qs[2]), int(ks[1]), int(ks[2])
    place = dict(own=(dim, None), rotated=(128 + dim, None), v=(None, dim))[where]
    for h in range(2):
        if where != "rotated" and h == 0:
            assert torch.equal(out[:, h], clean[0][:, h]) and torch.equal(lse[:, h], clean[1][:, h])
            continue
        k = orl.bf16_bits_to_f64(np.concatenate([C.bits(kv2[k0:k1, h, :128].contiguous()),
                                                 C.bits(rows2[k0:k1, 512:].contiguous())], 1))
        v = orl.bf16_bits_to_f64(C.bits(kv2[k0:k1, h, 128:].contiguous()))
        qh = orl.bf16_bits_to_f64(C.bits(q[q0:q1, h].contiguous()))
        want, free = [], np.zeros((n, 128), bool)
        for i in range(n):
            end = m - n + i + 1
            want.append(C.attend_beside(qh[i], k, v, end, C.SCALE, at, place))
            if at >= end:
                same = torch.ones(128, dtype=torch.bool)
                if where == "v":
                    free[i, dim], same[dim] = True, False
                assert torch.equal(out[q0 + i, h, same], clean[0][q0 + i, h, same])
                assert torch.equal(lse[q0 + i, h], clean[1][q0 + i, h])
        C.check_beside(out[q0:q1, h], lse[q0:q1, h], want, 192, free)
    keep = [i for i in range(len(out)) if not q0 <= i < q1]
    assert torch.equal(out[keep], clean[0][keep]) and torch.equal(lse[keep], clean[1][keep])


def test_prefill_non_finite_query():
    """A query that is NaN and one that is infinite: their rows are NaN and no other is touched."""
    case = prefill_case(17, [(140, 150), (20, 20)], 3)
    clean = run_prefill(case)
    q = case[0].clone()
    q[70, 2, 5], q[131, 0, 150] = float("nan"), float("inf")  # (keys of both signs: +inf among the scores)
    out, lse, _ = run_prefill((q, *case[1:]))
    for i, h in ((70, 2), (131, 0)):
        assert out[i, h].isnan().all() and lse[i, h].isnan()
        out[i, h], lse[i, h] = clean[0][i, h], clean[1][i, h]
    assert torch.equal(out, clean[0]) and torch.equal(lse, clean[1])


def test_prefill_large_scores():
    """Scores in the hundreds whose maximum moves along the keys."""
    q, kv, rows, qs, ks = prefill_case(8, [(300, 900)], 2, q_scale=30.0)
    kv = (kv.float() * torch.linspace(0.2, 2.0, 900)[:, None, None]).to(torch.bfloat16)
    assert check_prefill((q, kv, rows, qs, ks)) == 0


def test_prefill_strides():
    """Contiguous tensors, wide rows, heads outside the tokens: one result."""
    case = prefill_case(9, [(140, 200), (30, 30)], 3)
    q, kv, rows, qs, ks = case
    a = run_prefill(case)
    k, v, r = kv[..., :128], kv[..., 128:], rows[:, 512:]
    forms = [(q.cuda(), k.contiguous().cuda(), r.contiguous().cuda(), v.contiguous().cuda()),
             (q.transpose(0, 1).contiguous().cuda().transpose(0, 1), k.transpose(0, 1).contiguous().cuda().transpose(0, 1),
              rows.cuda()[:, 512:], v.cuda())]
    for qf, kf, rf, vf in forms:
        out, lse = binding.pkv_latent_prefill_attention(qf, kf, rf, vf, qs.cuda(), ks.cuda(), C.SCALE)
        assert torch.equal(out.cpu(), a[0]) and torch.equal(lse.cpu(), a[1])
    # one head's keys and values for all heads (stride 0)
    shared = prefill_case(10, [(60, 90)], 1)
    q3 = C.normal(C.gen(11), 60, 3, 192)
    k1, v1, r1 = shared[1][..., :128], shared[1][..., 128:], shared[2][:, 512:]
    out, lse = binding.pkv_latent_prefill_attention(q3.cuda(), k1.cuda().expand(90, 3, 128), r1.cuda(),
                                                    v1.cuda().expand(90, 3, 128), shared[3].cuda(), shared[4].cuda(), C.SCALE)
    for h in range(3):
        o, l = binding.pkv_latent_prefill_attention(q3[:, h:h + 1].cuda(), k1.cuda(), r1.cuda(), v1.cuda(),
                                                    shared[3].cuda(), shared[4].cuda(), C.SCALE)
        assert torch.equal(out[:, h], o[:, 0]) and torch.equal(lse[:, h], l[:, 0])


def test_prefill_bad_starts():
    """Starts that do not ascend or pass the tensors are told, and nothing outside is touched."""
    case = prefill_case(12, [(40, 40), (60, 60), (20, 20)], 2)
    q, kv, rows, qs, ks = case
    for bad_q, bad_k in (([0, 100, 40, 120], None), ([0, 40, 100, 121], None), (None, [0, 40, 100, 121]), (None, [0, 100, 40, 120]),
                         ([-1, 40, 100, 120], None), ([0, 1 << 30, 100, 120], None)):
        c = (q, kv, rows, C.i32(bad_q) if bad_q else qs, C.i32(bad_k) if bad_k else ks)
        assert run_prefill(c)[2] & LAYOUT


def test_prefill_bad_starts_touch_nothing_outside():
    """With starts that do not ascend or pass the tensors, what lies around out and lse stays."""
    case = prefill_case(12, [(40, 40), (60, 60), (20, 20)], 2)
    q, kv, rows, qs, ks = case
    n, pad = 120, 300
    big = 1 << 30
    for bad_q, bad_k in (([0, 100, 40, 120], None), ([0, 40, 100, 121], None), ([0, 40, 100, 100 + 256], None),
                         (None, [0, 40, 100, 121]), (None, [0, 100, 40, 120]), ([-1, 40, 100, 120], None),
                         ([-300, 40, 100, 120], None), ([0, big, 100, 120], None), ([0, 40, 100, big], None),
                         ([0, -big, 100, 120], None), (None, [-5, 40, 100, 120]), (None, [0, 40, 100, big])):
        out = torch.full((pad + n + pad, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((pad + n + pad, 2), 7.0, device="cuda")
        c = (q, kv, rows, C.i32(bad_q) if bad_q else qs, C.i32(bad_k) if bad_k else ks)
        assert run_prefill(c, out=out[pad:pad + n], lse=lse[pad:pad + n])[2] & LAYOUT
        for t in (out, lse):
            assert (t[:pad] == 7).all() and (t[pad + n:] == 7).all(), (bad_q, bad_k)


@pytest.mark.parametrize("places", [767, 768, 769, 1100])
def test_prefill_many_sequences(places):
    """As many places for items as are sorted by cost, one fewer, and more, which are taken as they
    stand: short sequences, empty ones, and a few long ones among them."""
    long = [(300, 300), (257, 500), (1, 700)]
    tq = sum(n for n, _ in long)
    lens, i = [], 0
    while tq // 256 + len(lens) + len(long) < places:
        n = i % 4
        lens.append((n, n + i % 3))
        tq += n
        i += 1
    for k, x in enumerate(long):
        lens.insert((k + 1) * len(lens) // 4, x)
    case = prefill_case(places, lens, 1)
    assert case[0].shape[0] // 256 + len(lens) == places
    assert check_prefill(case) == 0


def test_prefill_items_above_the_costliest_that_are_told_apart():
    """Items of more key tiles than a sorted item's cost can say."""
    lens = [(3, 17000), (5, 5), (2, 33000), (1, 16100), (130, 140), (1, 16000)]
    assert check_prefill(prefill_case(19, lens, 2)) == 0


def test_prefill_same_bits_every_time():
    case = prefill_case(13, [(300, 700), (129, 129), (1, 900)], 4)
    first = run_prefill(case)
    for _ in range(5):
        again = run_prefill(case)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
