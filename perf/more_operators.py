"""The operators of a paged cache of shared latents as workloads: their inputs, their plain form in elementary
torch operations, and the calls of the framework's own kernels (``own``).

* ``rotate``: the rotary embedding of the queries' position part, interleaved or in halves, through strides.
* ``append``: new tokens' latents, normalised, and their rotated position part written through the page table.
* ``gather``: cached rows read back through the page table, for the expanded form's up-projection.
* ``decode``: attention in the absorbed form, over the cache's rows as keys (576) and values (their first 512).
* ``prefill``: attention in the expanded form, causal, sequences packed one after another, with or without a prefix.

A cache row is a latent of 512 and a rotated part of 64 that all heads share, in bf16: pool ``[num_pages * page_size,
576]``, slot 0 and page 0 reserved. Expanded, a head has keys of 128 + 64 and values of 128.
"""

import math

import torch

own = False

R, P = 512, 64        # latent, rotated part
W = R + P             # a cache row
DN, DV = 128, 128     # expanded: a head's own part of a key, a value


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # the queries of a decode batch, read out of the projection's rows, written behind the absorbed part
        dict(name="rotate_step", op="rotate", T=64, H=128, dims=64, inter=True, table=8192, factor=1.0, absorbed=True),
        # the queries of a long prompt, an odd number of tokens, tables scaled for a longer context
        dict(name="rotate_prompt", op="rotate", T=8191, H=32, dims=64, inter=False, table=65536, factor=8.0, absorbed=False),
        # a decode batch's new tokens
        dict(name="append_step", op="append", B=64, n=1, lo=512, hi=1024, ps=64, inter=True, norm=True, table=8192),
        # prompts of ordinary length, all at once
        dict(name="append_prompts", op="append", B=16, n=1024, lo=0, hi=0, ps=128, inter=False, norm=True, table=8192),
        # one user's prefix, small pages
        dict(name="gather_one_user", op="gather", B=1, lo=777, hi=777, ps=16),
        # the prefixes of a step of prompt chunks
        dict(name="gather_prefixes", op="gather", B=16, lo=2048, hi=8191, ps=64),
        # one user, a short context, few heads: latency
        dict(name="decode_one_user", op="decode", B=1, nq=1, H=32, lo=200, hi=333, ps=16),
        # a full decode batch with all heads on one card: stream and products weigh alike
        dict(name="decode_batch", op="decode", B=64, nq=1, H=128, lo=512, hi=1024, ps=64),
        # four drafted tokens a sequence over long contexts, a quarter of the heads
        dict(name="decode_drafts", op="decode", B=16, nq=4, H=32, lo=8192, hi=32767, ps=128),
        # one short prompt of an odd length, few heads: latency
        dict(name="prefill_short", op="prefill", B=1, H=8, lo=333, hi=333, plo=0, phi=0),
        # prompts of a serving step, packed
        dict(name="prefill_packed", op="prefill", B=24, H=32, lo=64, hi=1024, plo=0, phi=0),
        # chunks of longer prompts behind their prefixes
        dict(name="prefill_chunks", op="prefill", B=8, H=32, lo=512, hi=512, plo=512, phi=4096),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotate", "append", "gather", "decode", "decode", "decode", "prefill", "prefill", "prefill"])
    if op == "rotate":
        while True:
            c = dict(op=op, T=_log(rng, 1, 20000), H=_log(rng, 1, 128), dims=rng.choice([32, 64, 64, 64, 128]),
                     inter=rng.random() < 0.5, table=_log(rng, 64, 100000), factor=rng.choice([1.0, 1.0, 4.0, 16.0]),
                     absorbed=rng.random() < 0.5)
            if c["T"] * c["H"] * c["dims"] < 8191 * 32 * 64:
                return c
    if op == "append":
        while True:
            lo = _log(rng, 1, 2000)
            c = dict(op=op, B=_log(rng, 1, 256), n=_log(rng, 1, 2000), lo=lo, hi=lo + _log(rng, 1, 500),
                     ps=rng.choice([16, 48, 64, 128]), inter=rng.random() < 0.5, norm=rng.random() < 0.7)
            c["table"] = c["hi"] + c["n"]
            if c["B"] * c["n"] < 16 * 1024 and c["B"] * (c["hi"] + c["n"]) < 200000:
                return c
    if op == "gather":
        while True:
            lo = _log(rng, 1, 4000)
            c = dict(op=op, B=_log(rng, 1, 128), lo=lo, hi=lo + _log(rng, 1, 4000), ps=rng.choice([16, 48, 64, 128]))
            if c["B"] * c["hi"] < 16 * 5000:
                return c
    if op == "decode":
        while True:
            lo = _log(rng, 1, 20000)
            c = dict(op=op, B=_log(rng, 1, 128), nq=rng.choice([1, 1, 1, 2, 3, 4, 8]), H=_log(rng, 1, 128), lo=lo,
                     hi=lo + _log(rng, 1, 20000), ps=rng.choice([16, 32, 48, 64, 128, 256]))
            rows = c["nq"] * c["H"]
            if c["B"] * c["hi"] < 16 * 20000 and c["B"] * c["hi"] * -(-rows // 128) < 16 * 20000:
                return c
    while True:
        lo, prefix = _log(rng, 1, 2000), rng.random() < 0.5
        c = dict(op=op, B=_log(rng, 1, 32), H=_log(rng, 1, 64), lo=lo, hi=lo + _log(rng, 1, 2000),
                 plo=_log(rng, 1, 2000) if prefix else 0, phi=0)
        if prefix:
            c["phi"] = c["plo"] + _log(rng, 1, 4000)
        if c["B"] * c["H"] * c["hi"] * (c["hi"] + c["phi"]) < 8 * 32 * 512 * 2816 and \
                c["B"] * c["H"] * (c["hi"] + c["phi"]) < 2000000:
            return c


# ----------------------------------------------------------------- inputs --

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _ints(g, lo, hi, shape):
    return torch.randint(lo, hi + 1, shape, generator=g, device="cuda", dtype=torch.int32)


def _normal(g, shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)


def _permuted_table(g, slots, blocks):
    """Slots 1.. with `blocks` pages each, in a random order of pages 1..; and how many pages that takes."""
    pages = slots * blocks + 1
    table = torch.full((slots + 1, blocks), -1, device="cuda", dtype=torch.int32)
    table[1:] = (torch.randperm(pages - 1, generator=g, device="cuda") + 1).to(torch.int32).view(slots, blocks)
    return table, pages


def _rope_tables(rows, dims, factor=1.0):
    """cos and sin of every position's angles, [rows, dims / 2]. For a context `factor` times as long, frequencies
    of few turns over 4096 tokens are divided by the factor, those of many stay, with a ramp between."""
    f = 10000.0 ** (-torch.arange(0, dims, 2, device="cuda", dtype=torch.float64) / dims)
    if factor > 1:
        turns = 4096 * f / (2 * math.pi)
        keep = ((turns - 1) / 31).clamp(0, 1)
        f = f * keep + f / factor * (1 - keep)
    a = torch.arange(rows, device="cuda", dtype=torch.float64)[:, None] * f
    return torch.cos(a).float(), torch.sin(a).float()


def _prepare_rotate(c, g):
    T, H, dims = c["T"], c["H"], c["dims"]
    cos, sin = _rope_tables(c["table"], dims, c["factor"])
    s = dict(q=_normal(g, (T, H, DN + dims)), pos=_ints(g, 0, c["table"] - 1, (T,)), cos=cos, sin=sin, inter=c["inter"], out=None)
    if c["absorbed"]:
        s["out"] = _normal(g, (T, H, R + dims))[..., R:]
    return s


def _prepare_append(c, g):
    B, n, ps = c["B"], c["n"], c["ps"]
    table, pages = _permuted_table(g, B, -(-(c["hi"] + n) // ps))
    cos, sin = _rope_tables(c["table"], P)
    start = _ints(g, c["lo"], c["hi"], (B,))
    pos = (start[:, None] + torch.arange(n, device="cuda", dtype=torch.int32)).flatten().contiguous()
    slot = torch.arange(1, B + 1, device="cuda", dtype=torch.int32).repeat_interleave(n).contiguous()
    weight = 1 + 0.1 * torch.randn((R,), generator=g, device="cuda") if c["norm"] else None
    return dict(pool=_normal(g, (pages * ps, W)), table=table, ps=ps, new=3 * _normal(g, (B * n, W)), slot=slot, pos=pos,
                cos=cos, sin=sin, inter=c["inter"], weight=weight, eps=1e-6)


def _lens(g, lo, hi, n):
    """n lengths spread evenly over lo .. hi, in a random order: their sum is the same for every seed."""
    even = lo + ((hi - lo) * (2 * torch.arange(n, device="cuda") + 1)) // (2 * n)
    return even[torch.randperm(n, generator=g, device="cuda")].to(torch.int32)


def _starts(lens):
    s = torch.zeros((lens.numel() + 1,), device="cuda", dtype=torch.int32)
    s[1:] = torch.cumsum(lens.long(), 0).to(torch.int32)
    return s


def _prepare_gather(c, g):
    B, ps = c["B"], c["ps"]
    table, pages = _permuted_table(g, B, -(-c["hi"] // ps))
    starts = _starts(_lens(g, c["lo"], c["hi"], B))
    slots = (torch.randperm(B, generator=g, device="cuda") + 1).to(torch.int32)
    return dict(pool=_normal(g, (pages * ps, W)), table=table, ps=ps, slots=slots, starts=starts, total=int(starts[-1]))


def _prepare_decode(c, g):
    B, nq, ps = c["B"], c["nq"], c["ps"]
    table, pages = _permuted_table(g, B, -(-c["hi"] // ps))
    slot = torch.arange(1, B + 1, device="cuda", dtype=torch.int32)
    lens = _ints(g, c["lo"], c["hi"], (B,))
    pad = B // 16
    if pad:  # the unused rows of a padded batch
        slot[-pad:] = 0
        lens[-pad:] = 0
    return dict(pool=_normal(g, (pages * ps, W)), table=table, ps=ps, q=_normal(g, (B, nq, c["H"], W)), slot=slot, lens=lens,
                longest=c["hi"], scale=1 / math.sqrt(DN + P))


def _prepare_prefill(c, g):
    B, H = c["B"], c["H"]
    nq = _lens(g, c["lo"], c["hi"], B)
    nk = nq + _lens(g, c["plo"], c["phi"], B)
    q_starts, k_starts = _starts(nq), _starts(nk)
    tq, tk = int(q_starts[-1]), int(k_starts[-1])
    kv = _normal(g, (tk, H, DN + DV))  # as the up-projection leaves it: a head's key part, then its value
    rows = _normal(g, (tk, W))
    return dict(q=_normal(g, (tq, H, DN + P)), k=kv[..., :DN], v=kv[..., DN:], kr=rows[:, R:], q_starts=q_starts,
                k_starts=k_starts, spans=list(zip(q_starts.tolist(), q_starts.tolist()[1:], k_starts.tolist(), k_starts.tolist()[1:])),
                scale=1 / math.sqrt(DN + P))


def prepare(case, seed):
    make = dict(rotate=_prepare_rotate, append=_prepare_append, gather=_prepare_gather, decode=_prepare_decode,
                prefill=_prepare_prefill)
    return dict(make[case["op"]](case, _gen(seed)), op=case["op"])


# ------------------------------------------------------------ plain forms --

def _turn(x, c, s, inter):
    if inter:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    a, b = x.chunk(2, -1)
    return torch.cat((a * c - b * s, b * c + a * s), -1)


def _rotate(s):
    p = s["pos"].long()
    y = _turn(s["q"][..., DN:].float(), s["cos"][p][:, None], s["sin"][p][:, None], s["inter"]).to(s["q"].dtype)
    if s["out"] is None:
        return y
    s["out"].copy_(y)
    return s["out"]


def _append(s):
    x, p = s["new"].float(), s["pos"].long()
    lat = x[:, :R]
    if s["weight"] is not None:
        lat = lat / torch.sqrt((lat * lat).mean(-1, keepdim=True) + s["eps"]) * s["weight"]
    row = torch.cat((lat, _turn(x[:, R:], s["cos"][p], s["sin"][p], s["inter"])), -1)
    s["pool"][s["table"][s["slot"].long(), p // s["ps"]].long() * s["ps"] + p % s["ps"]] = row.to(s["pool"].dtype)
    return s["pool"]


def _gather(s):
    t = torch.arange(s["total"], device="cuda")
    b = torch.searchsorted(s["starts"].long(), t, right=True) - 1
    p = t - s["starts"].long()[b]
    return s["pool"][s["table"][s["slots"].long()[b], p // s["ps"]].long() * s["ps"] + p % s["ps"]]


def _decode(s):
    q, ps = s["q"], s["ps"]
    B, nq, H, _ = q.shape
    t = torch.arange(s["longest"], device=q.device)
    slot, lens = s["slot"].long(), s["lens"].long()
    there = t < lens[:, None]
    row = torch.where(there, s["table"][slot].long()[:, t // ps] * ps + t % ps, 0)
    k = torch.where(there[..., None], s["pool"][row].float(), 0)
    x = (q.float().view(B, nq * H, W) @ k.transpose(1, 2)).view(B, nq, H, -1) * s["scale"]
    end = lens[:, None] - (nq - 1) + torch.arange(nq, device=q.device)
    sees = (t < end[..., None]) & (slot > 0)[:, None, None]
    x = x.masked_fill(~sees[:, :, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0, m)
    p = torch.exp(x - m)
    l = p.sum(-1, keepdim=True)
    o = (p.view(B, nq * H, -1) @ k[..., :R]).view(B, nq, H, R) / torch.where(l > 0, l, 1)
    return dict(out=o.to(q.dtype), lse=(m + torch.log(l))[..., 0])


def _prefill(s):
    tq, H, _ = s["q"].shape
    out = torch.zeros((tq, H, DV), device="cuda", dtype=s["q"].dtype)
    lse = torch.full((tq, H), -math.inf, device="cuda")
    for q0, q1, k0, k1 in s["spans"]:
        n, m = q1 - q0, k1 - k0
        if n == 0 or m == 0:
            continue
        q = s["q"][q0:q1].float().transpose(0, 1)
        k = torch.cat((s["k"][k0:k1].float(), s["kr"][k0:k1].float()[:, None].expand(m, H, P)), -1).permute(1, 2, 0)
        x = (q @ k) * s["scale"]
        ahead = torch.arange(m, device="cuda") > (torch.arange(n, device="cuda") + m - n)[:, None]
        x = x.masked_fill_(ahead, -math.inf)
        top = x.amax(-1, keepdim=True)
        p = torch.exp(x - top)
        l = p.sum(-1, keepdim=True)
        out[q0:q1] = ((p @ s["v"][k0:k1].float().transpose(0, 1)) / l).transpose(0, 1).to(out.dtype)
        lse[q0:q1] = (top + torch.log(l))[..., 0].transpose(0, 1)
    return dict(out=out, lse=lse)


# -------------------------------------------------------------- one pass --

def _own(s):
    from paged_kv_gqa_pkv_gb300 import binding
    if s["op"] == "rotate":
        return binding.pkv_rotate(s["q"][..., DN:], s["pos"], s["cos"], s["sin"], interleaved=s["inter"], out=s["out"])
    if s["op"] == "append":
        binding.pkv_latent_append(s["pool"], s["table"], s["new"], s["slot"], s["pos"], s["ps"], s["cos"], s["sin"],
                                  norm_weight=s["weight"], norm_eps=s["eps"], interleaved=s["inter"])
        return s["pool"]
    if s["op"] == "gather":
        return binding.pkv_latent_gather(s["pool"], s["table"], s["slots"], s["starts"], s["total"], s["ps"])
    if s["op"] == "decode":
        out, lse = binding.pkv_latent_decode_attention(s["pool"], s["table"], s["q"], s["slot"], s["lens"], s["ps"], s["scale"])
        return dict(out=out, lse=lse)
    out, lse = binding.pkv_latent_prefill_attention(s["q"], s["k"], s["kr"], s["v"], s["q_starts"], s["k_starts"], s["scale"])
    return dict(out=out, lse=lse)


def run(s):
    if own:
        return _own(s)
    return dict(rotate=_rotate, append=_append, gather=_gather, decode=_decode, prefill=_prefill)[s["op"]](s)


def work(case):
    """Lengths are random or spread over their range: their mean counts."""
    c = dict(case)
    op = c["op"]
    if op == "rotate":
        n = c["T"] * c["H"] * c["dims"]
        return dict(bytes=4 * n + c["T"] * 4 + min(c["T"], c["table"]) * c["dims"] * 4, flops=3 * n)
    B, mean = c["B"], (c["lo"] + c["hi"]) / 2
    if op == "append":
        rows = B * c["n"]
        places = min(rows, c["hi"] - c["lo"] + c["n"])  # rows of the tables that are read
        return dict(bytes=rows * (2 * 2 * W + 8) + places * P * 4, flops=rows * (3 * R + 3 * P))
    if op == "gather":
        return dict(bytes=B * mean * 2 * 2 * W, flops=0)
    if op == "decode":
        live = B - B // 16
        rows = c["nq"] * c["H"]
        return dict(bytes=live * mean * 2 * W + live * rows * 2 * W + B * rows * (2 * R + 4), flops=2 * live * rows * mean * (W + R))
    pre = (c["plo"] + c["phi"]) / 2
    square = (c["lo"] ** 2 + c["lo"] * c["hi"] + c["hi"] ** 2) / 3  # the mean of a uniform length's square
    seen = B * (mean * pre + (square + mean) / 2)
    return dict(bytes=B * c["H"] * (mean * 2 * (DN + P + DV) + mean * 4 + (mean + pre) * 2 * (DN + DV)) + B * (mean + pre) * 2 * P,
                flops=2 * seen * c["H"] * (DN + P + DV))


# ------------------------------------------------------------ definitions --

def _exact_turn(x, angle_cos, angle_sin, inter):
    """Each pair as a complex number, turned by its angle."""
    z = torch.complex(angle_cos.double(), angle_sin.double())
    half = x.shape[-1] // 2
    first = torch.arange(half, device=x.device) * (2 if inter else 1)
    second = first + (1 if inter else half)
    w = torch.complex(x[..., first], x[..., second]) * z
    y = torch.empty_like(x)
    y[..., first], y[..., second] = w.real, w.imag
    return y


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "rotate":
        at = s["pos"].long()
        return _exact_turn(s["q"][..., DN:].double(), s["cos"][at].unsqueeze(1), s["sin"][at].unsqueeze(1), s["inter"])
    if op == "append":
        pool = s["pool"].double()
        at = s["pos"].long()
        x = s["new"].double()
        if s["weight"] is not None:
            x[:, :R] *= torch.rsqrt(x[:, :R].square().sum(1, keepdim=True) / R + s["eps"]) * s["weight"].double()
        x[:, R:] = _exact_turn(x[:, R:], s["cos"][at], s["sin"][at], s["inter"])
        page = s["table"][s["slot"].long()].long().gather(1, (at // s["ps"]).unsqueeze(1)).squeeze(1)
        pool[page * s["ps"] + at % s["ps"]] = x
        return pool
    if op == "gather":
        out = torch.empty((s["total"], W), device="cuda", dtype=torch.float64)
        starts = s["starts"].tolist()
        for b, slot in enumerate(s["slots"].tolist()):
            t = torch.arange(starts[b + 1] - starts[b], device="cuda")
            out[starts[b]:starts[b + 1]] = s["pool"][s["table"][slot].long()[t // s["ps"]] * s["ps"] + t % s["ps"]].double()
        return out
    if op == "decode":
        B, nq, H, _ = s["q"].shape
        out = torch.zeros((B, nq, H, R), device="cuda", dtype=torch.float64)
        lse = torch.full((B, nq, H), -math.inf, device="cuda", dtype=torch.float64)
        slots, lens = s["slot"].tolist(), s["lens"].tolist()
        for b in range(B):
            if slots[b] == 0:
                continue
            t = torch.arange(lens[b], device="cuda")
            rows = s["pool"][s["table"][slots[b]].long()[t // s["ps"]] * s["ps"] + t % s["ps"]].double()
            for j in range(nq):
                n = lens[b] - (nq - 1 - j)
                if n <= 0:
                    continue
                x = torch.einsum("hd,td->ht", s["q"][b, j].double(), rows[:n]) * s["scale"]
                lse[b, j] = torch.logsumexp(x, 1)
                out[b, j] = torch.einsum("ht,td->hd", torch.exp(x - lse[b, j][:, None]), rows[:n, :R])
        return dict(out=out, lse=lse)
    tq, H, _ = s["q"].shape
    out = torch.zeros((tq, H, DV), device="cuda", dtype=torch.float64)
    lse = torch.full((tq, H), -math.inf, device="cuda", dtype=torch.float64)
    for q0, q1, k0, k1 in s["spans"]:
        n, m = q1 - q0, k1 - k0
        for h in range(H):
            x = torch.einsum("id,jd->ij", s["q"][q0:q1, h, :DN].double(), s["k"][k0:k1, h].double())
            x = (x + torch.einsum("id,jd->ij", s["q"][q0:q1, h, DN:].double(), s["kr"][k0:k1].double())) * s["scale"]
            x = torch.where(torch.ones_like(x, dtype=torch.bool).tril(m - n), x, -math.inf)
            z = torch.logsumexp(x, 1)
            lse[q0:q1, h] = z
            out[q0:q1, h] = torch.einsum("ij,jd->id", torch.exp(x - z[:, None]), s["v"][k0:k1, h].double())
    return dict(out=out, lse=lse)
