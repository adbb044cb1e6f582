"""The paged 8-bit cache on the GPU: block tables and slot maps, storing keys and values, one-token attention.

Tables, slots, scales and codes are compared exactly with plain loops.  Attention is compared with the formula in 64
bits: the softmax's weights are fp16 (half a step is 2^-11, weighted by |v|), the result is rounded to bf16 (2^-8), and
the fp32 steps add less than 2^-12 of the same weights, as in test_gpu_attention.py; queries are exact in fp16 but for
elements 2^-14 below a row's largest, which round at 2^-24 of it.

Weights below fp16's normal range are off by half of its smallest step, 2^-25, instead of by a relative error.  A weight is
C p_j vs_j (probability times value scale), with C such that the largest is at least 2^12, so C >= 2^12 / max_j p_j vs_j,
and sum_j C p_j vs_j code_j is divided by C.  The result is then off by at most
2^-25 sum_j |code_j| / C <= 2^-37 sum_j |code_j| max_j p_j vs_j.
"""
import math

import pytest
import torch

import kda_gated_delta_prefill_b200 as kda

pytestmark = pytest.mark.gpu

E4M3, INT8 = torch.float8_e4m3fn, torch.int8
TOP = {E4M3: 448.0, INT8: 127.0}
FP16, BF16, FP32 = 2.0 ** -11, 2.0 ** -8, 2.0 ** -12


# ------------------------------------------------------------------------------------------------ plan
def plain_plan(ctx, new, table, free, bs, tokens):
    table = [list(r) for r in table]
    used, slots, cu = 0, [], [0]
    for b, (c, n) in enumerate(zip(ctx, new)):
        for k in range(-(-c // bs), -(-(c + n) // bs)):
            if k < len(table[b]):
                table[b][k] = free[used] if used < len(free) else -1
            used += 1
        for p in range(c, c + n):
            k = p // bs
            block = table[b][k] if k < len(table[b]) else -1
            slots.append(block * bs + p % bs if block >= 0 else -1)
        cu.append(cu[-1] + n)
    slots = (slots + [-1] * tokens)[:tokens]
    return table, cu, [c + n for c, n in zip(ctx, new)], slots, min(used, len(free))


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def run_plan(ctx, new, bs, *, pad=0, width=None, free=None, seed=0):
    g = torch.Generator().manual_seed(seed)
    have = [-(-c // bs) for c in ctx]
    need = [-(-(c + n) // bs) for c, n in zip(ctx, new)]
    width = max(need + [1]) if width is None else width
    ids = torch.randperm(sum(have) + sum(need) + 3, generator=g).tolist()
    table, at = [], 0
    for h in have:
        row = ids[at:at + h] + [-7] * width
        table.append(row[:width])
        at += h
    free = ids[at:at + (sum(need) - sum(have) + 2 if free is None else free)]
    tokens = sum(new) + pad
    want = plain_plan(ctx, new, table, free, bs, tokens)
    t = i32(table)
    cu, lens, slots, used = kda.cache_plan(i32(ctx), i32(new), t, i32(free), bs, tokens)
    torch.cuda.synchronize()
    assert t.tolist() == want[0]
    assert cu.tolist() == want[1] and lens.tolist() == want[2] and slots.tolist() == want[3]
    assert used.tolist() == [want[4]]


@pytest.mark.parametrize("ctx,new,bs,pad", [
    ([0], [1], 16, 0),
    ([15, 16, 17, 0, 31], [1, 1, 1, 1, 1], 16, 3),
    ([5, 0, 64, 100], [0, 0, 0, 0], 64, 2),
    ([0, 128, 127, 3], [1000, 0, 129, 77], 128, 10),
    ([7, 9], [3000, 5000], 32, 0),
])
def test_plan(ctx, new, bs, pad):
    run_plan(ctx, new, bs, pad=pad)
    assert kda.device_error() == 0


@pytest.mark.parametrize("rows,most", [(1, 5000), (33, 100), (513, 3), (2000, 40), (16384, 1)])
def test_plan_random(rows, most):
    g = torch.Generator().manual_seed(rows)
    ctx = torch.randint(0, 200, (rows,), generator=g).tolist()
    new = torch.randint(0, most + 1, (rows,), generator=g).tolist()
    run_plan(ctx, new, 16, pad=rows % 7, seed=rows)
    assert kda.device_error() == 0


def test_plan_reports_what_does_not_fit():
    run_plan([10, 20, 0], [30, 30, 40], 16, free=3)            # too few free blocks
    assert kda.device_error() == 32
    run_plan([10, 20, 0], [30, 300, 40], 16, width=5)          # a table row too short
    assert kda.device_error() == 32
    t = i32([[-1, -1]])
    cu, lens, slots, used = kda.cache_plan(i32([0]), i32([20]), t, i32([4, 5]), 16, 7)  # slot map too short
    assert slots.tolist() == [64 + i for i in range(7)] and kda.device_error() == 32
    kda.cache_plan(i32([-4]), i32([-9]), t, i32([4, 5]), 16, 7)  # negative lengths count as zero
    assert kda.device_error() == 0


def test_plan_with_strided_table_rows():
    base = torch.full((3, 10), -3, dtype=torch.int32, device="cuda")
    cu, lens, slots, used = kda.cache_plan(i32([0, 0, 0]), i32([16, 17, 1]), base[:, 2:6], i32([9, 8, 7, 6]), 16, 34)
    assert base[:, :2].eq(-3).all() and base[:, 6:].eq(-3).all()
    assert base[:, 2:6].tolist() == [[9, -3, -3, -3], [8, 7, -3, -3], [6, -3, -3, -3]] and used.item() == 4


# ------------------------------------------------------------------------------------------------ append
def plain_scale(top, dtype):
    """The smallest power of two, 2^-100 at least, whose largest code holds top."""
    e = -100
    while top > TOP[dtype] * 2.0 ** e:
        e += 1
    return 2.0 ** e


def plain_codes(x, s, dtype):
    y = x.double() / s
    if dtype == INT8:
        return torch.nan_to_num(y, nan=0.0).round().clamp(-127, 127).to(torch.int8)
    return torch.where(y.isnan(), y, y.clamp(-448, 448)).float().to(dtype)


def plain_append(x, cache, scale, slots):
    """Token by token in runs, on the CPU; codes as bytes."""
    dtype, bs = cache.dtype, cache.shape[2]
    t = 0
    while t < len(slots):
        if slots[t] < 0:
            t += 1
            continue
        blk, first, e = slots[t] // bs, slots[t] % bs, t
        while e < len(slots) and slots[e] >= 0 and slots[e] // bs == blk:
            e += 1
        for h in range(x.shape[1]):
            v = x[t:e, h].float()
            fine = v[v.isfinite()].abs()
            s = plain_scale(fine.max().item() if fine.numel() else 0.0, dtype)
            if first:
                was = scale[blk, h].item()
                s = max(s, was)
                if s != was:
                    cache[blk, h, :first] = plain_codes(cache[blk, h, :first].float() * was, s, dtype)
            scale[blk, h] = s
            for i in range(t, e):
                cache[blk, h, slots[i] % bs] = plain_codes(x[i, h], s, dtype)
        t = e


def pool(dtype, blocks, HKV, bs, D, seed):
    g = torch.Generator().manual_seed(seed)
    c = torch.randint(0, 256, (blocks, HKV, bs, D), generator=g, dtype=torch.uint8)
    if dtype == E4M3:
        c[(c & 0x7f) == 0x7f] = 0x11
    else:
        c[c == 0x80] = 0x11
    return c.view(dtype), torch.exp2(torch.randint(-9, -4, (blocks, HKV), generator=g).float())


def bits(c):
    return c.cpu().view(torch.uint8)


def wide(seed, *shape):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(*shape, generator=g) * torch.exp2(torch.randint(-12, 12, (*shape[:-1], 1), generator=g).float())
    return x.bfloat16()


@pytest.mark.parametrize("dtype", [E4M3, INT8])
@pytest.mark.parametrize("bs,D,HKV", [(16, 128, 3), (32, 64, 1), (64, 128, 2), (128, 64, 5), (128, 128, 8), (16, 64, 8)])
def test_append_stores_the_same_codes_as_plain_loops(dtype, bs, D, HKV):
    # runs that open a block, that join one, that end inside one, of one token, of a whole block; skipped tokens
    runs = [(3, 0, bs), (0, 5, 1), (1, bs - 1, 1), (None, 0, 3), (6, 0, 1), (2, 3, bs - 3), (5, 1, bs // 2), (4, 0, bs - 1)]
    slots = []
    for blk, first, n in runs:
        slots += [-1] * n if blk is None else [blk * bs + first + i for i in range(n)]
    T = len(slots)
    k, v = wide(1, T, HKV, D), wide(2, T, HKV, D)
    kc, ks = pool(dtype, 8, HKV, bs, D, 3)
    vc, vs = pool(dtype, 8, HKV, bs, D, 4)
    dev = [x.cuda() for x in (k, v, kc, vc, ks, vs)]
    kda.cache_append(*dev, i32(slots))
    torch.cuda.synchronize()
    assert kda.device_error() == 0
    plain_append(k, kc, ks, slots)
    plain_append(v, vc, vs, slots)
    for got, want in zip(dev[2:], (kc, vc, ks, vs)):
        assert torch.equal(bits(got), bits(want))


@pytest.mark.parametrize("dtype", [E4M3, INT8])
def test_append_edges_of_the_scale_and_values_without_one(dtype):
    """Largest magnitudes at and beside the largest code, zeros, tiny and huge values, infinities and NaN."""
    top = TOP[dtype]
    rows = [top, -top, top * 2 ** -9, torch.tensor(top).bfloat16().item() * (1 + 2 ** -7), 0.0, 1e-38, 2.0 ** -100, 3e38,
            math.inf, -math.inf, math.nan]
    x = torch.zeros(len(rows), 1, 64)
    for i, r in enumerate(rows):
        x[i, 0, :3] = torch.tensor([r, 1.0 if abs(r) > 1e-3 and abs(r) < 1e4 else 0.0, r / 3 if math.isfinite(r) else 0.25])
    x = x.bfloat16()
    slots = [16 * i for i in range(len(rows))]
    c, s = pool(dtype, len(rows), 1, 16, 64, 5)
    d = [x.cuda(), x.cuda(), c.cuda(), c.cuda(), s.cuda(), s.cuda()]
    kda.cache_append(*d, i32(slots))
    plain_append(x, c, s, slots)
    assert torch.equal(bits(d[4]), bits(s))
    got, want = d[2].cpu(), c
    if dtype == E4M3:  # NaN of either sign
        nan = want.float().isnan()
        assert torch.equal(got.float().isnan(), nan) and nan[:, 0, 0].sum() == 1
        assert torch.equal(bits(got)[~nan], bits(want)[~nan])
    else:
        assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", [E4M3, INT8])
def test_append_token_by_token_stays_within_one_step(dtype):
    """Tokens that join one by one, growing: rounded again at each doubling, a code is off by less than half a step of the
    last scale for each of them, 1/2 + 1/4 + ... < 1 in all (int8); e4m3 loses nothing but at its smallest steps."""
    bs, D = 32, 128
    x = (torch.randn(bs, 1, D, generator=torch.Generator().manual_seed(0)) * torch.linspace(0.1, 40, bs)[:, None, None])
    x = x.bfloat16()
    c, s = (t.cuda() for t in pool(dtype, 2, 1, bs, D, 6))
    for t in range(bs):
        kda.cache_append(x[t:t + 1].cuda(), x[t:t + 1].cuda(), c, c.clone(), s, s.clone(), i32([bs + t]))
    scale = s[1, 0].item()
    assert scale == plain_scale(x.abs().max().item(), dtype)
    off = (c[1, 0].float().cpu() * scale - x[:, 0].float()).abs()
    if dtype == INT8:
        assert (off <= scale).all()
    else:  # half a step of e4m3 is 2^-4 relative, 2^-10 of the scale for the smallest codes; rounded twice there
        assert (off <= torch.maximum(x[:, 0].float().abs() * 2.0 ** -4, torch.tensor(2.0 ** -9 * scale))).all()


def test_append_strided_rows_interleaved_pools_and_slots_past_the_cache():
    HKV, D, bs = 2, 128, 16
    qkv = wide(7, 40, 8 * D).cuda()
    k, v = qkv[:, 4 * D:6 * D].view(40, HKV, D), qkv[:, 6 * D:].view(40, HKV, D)
    both = torch.zeros(6, 2, HKV, bs, D, dtype=torch.int8, device="cuda")
    ks, vs = torch.zeros(6, HKV, device="cuda"), torch.zeros(6, HKV, device="cuda")
    slots = list(range(16, 50)) + [96, 97, 1 << 30, -1, -5, 5]
    kda.cache_append(k, v, both[:, 0], both[:, 1], ks, vs, i32(slots))
    assert kda.device_error() == 16
    kc, vc = torch.zeros(6, HKV, bs, D, dtype=torch.int8), torch.zeros(6, HKV, bs, D, dtype=torch.int8)
    ks1, vs1 = torch.zeros(6, HKV), torch.zeros(6, HKV)
    slots = [s if s < 96 else -1 for s in slots]
    plain_append(k.cpu(), kc, ks1, slots)
    plain_append(v.cpu(), vc, vs1, slots)
    assert torch.equal(both[:, 0].cpu(), kc) and torch.equal(both[:, 1].cpu(), vc)
    assert torch.equal(ks.cpu(), ks1) and torch.equal(vs.cpu(), vs1)


# ------------------------------------------------------------------------------------------------ decode
def formula(q, kc, vc, ks, vs, table, lens, scale):
    B, H, D = q.shape
    HKV, bs = kc.shape[1], kc.shape[2]
    o = torch.zeros(B, H, D, dtype=torch.float64, device="cuda")
    w, tiny = torch.zeros_like(o), torch.zeros_like(o)
    lse = torch.full((B, H), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        if n <= 0:
            continue
        ids = table[b, :-(-n // bs)].long()
        k, v = ((c.view(torch.uint8)[ids].view(c.dtype).double() * s[ids].double()[..., None, None]).transpose(1, 2)
                .reshape(-1, HKV, D)[:n].transpose(0, 1) for c, s in ((kc, ks), (vc, vs)))
        x = torch.einsum("hgd,hnd->hgn", q[b].double().view(HKV, H // HKV, D), k) * scale
        z = torch.logsumexp(x, 2)
        p = torch.exp(x - z[..., None])
        o[b] = torch.einsum("hgn,hnd->hgd", p, v).reshape(H, D)
        w[b] = torch.einsum("hgn,hnd->hgd", p, v.abs()).reshape(H, D)
        lse[b] = z.reshape(H)
        scales = vs[ids].double().repeat_interleave(bs, 0)[:n].T[:, None]  # [HKV, 1, n]
        codes = (v.abs() / torch.where(scales == 0, 1.0, scales).transpose(1, 2)).sum(1)
        tiny[b] = (2.0 ** -37 * (p * scales).amax(2)[..., None] * codes[:, None]).reshape(H, D)
    return o, lse, w, tiny


def make_decode(dtype, lens, H, HKV, D, bs, seed, width=None):
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // bs) for n in lens]
    width = max(need + [1]) if width is None else width
    blocks = sum(need) + 2
    ids = torch.randperm(blocks, generator=g).tolist()
    table, at = torch.full((len(lens), width), -1, dtype=torch.int32), 0
    for b, m in enumerate(need):
        table[b, :m] = torch.tensor(ids[at:at + m], dtype=torch.int32)
        at += m
    kc, ks = pool(dtype, blocks, HKV, bs, D, seed + 1)
    vc, vs = pool(dtype, blocks, HKV, bs, D, seed + 2)
    for c in (kc, vc):  # what lies behind a request's last token may be anything
        if dtype == E4M3:
            for b, n in enumerate(lens):
                if n % bs:
                    c.view(torch.uint8)[table[b, n // bs].item(), :, n % bs:] = 0x7f
    q = torch.randn(len(lens), H, D, generator=g).bfloat16()
    return [x.cuda() for x in (q, kc, vc, ks, vs, table)]


def check_decode(args, lens, o, lse, scale=None):
    q = args[0]
    f, z, w, tiny = formula(*args, lens, q.shape[2] ** -0.5 if scale is None else scale)
    empty = torch.tensor([n <= 0 for n in lens], device="cuda")
    assert (o[empty] == 0).all() and (lse[empty] == -math.inf).all()
    tol = (FP16 + FP32) * w + BF16 * f.abs() + tiny + 1e-30
    ratio = ((o.double() - f).abs() / tol)[~empty]
    assert ratio.numel() == 0 or ratio.max() <= 1, float(ratio.max())
    dz = (lse.double() - z)[~empty].abs()
    assert dz.numel() == 0 or dz.max() < FP32 * max(1.0, z[~empty].abs().max().item() / 16), float(dz.max())


DECODES = [
    # lens, H, HKV, D, block size
    ([1], 1, 1, 128, 16),
    ([1, 15, 16, 17, 0, 33], 4, 4, 64, 16),
    ([63, 64, 65, 127, 128, 129], 8, 2, 128, 32),
    ([0, 0, 300], 8, 1, 128, 64),
    ([777], 32, 8, 128, 64),
    ([5000, 1, 0, 2500, 130], 10, 2, 128, 128),
    ([1000, 2000, 3], 24, 2, 64, 64),          # 12 heads of a group
    ([1000, 77], 32, 2, 128, 16),              # 16
    ([333, 64], 40, 1, 128, 32),               # 40: several passes over the codes
    ([40000], 8, 8, 64, 128),
    ([200 + 7 * i for i in range(70)], 6, 3, 128, 16),
    ([1 + i % 40 for i in range(700)], 4, 2, 64, 32),
]


@pytest.mark.parametrize("dtype", [E4M3, INT8])
@pytest.mark.parametrize("lens,H,HKV,D,bs", DECODES)
def test_decode_matches_the_formula(dtype, lens, H, HKV, D, bs):
    args = make_decode(dtype, lens, H, HKV, D, bs, 11)
    o, lse = kda.attention_decode(*args, i32(lens))
    torch.cuda.synchronize()
    assert kda.device_error() == 0
    check_decode(args, lens, o, lse)


@pytest.mark.parametrize("lens,H,HKV,D,bs", [
    ([30000], 8, 1, 128, 64),        # one unit over every CTA: its heads are joined by as many CTAs as it has heads
    ([30001], 1, 1, 64, 128),        # ... one head
    ([28300], 5, 1, 128, 16),
    ([27000], 16, 1, 64, 32),
    ([27000], 12, 1, 128, 128),
    ([9000, 3, 21000], 14, 2, 128, 64),
    ([0, 14000, 14000, 1], 6, 3, 64, 64),
])
def test_decode_of_few_long_units(lens, H, HKV, D, bs):
    args = make_decode(E4M3, lens, H, HKV, D, bs, 77)
    got = kda.attention_decode(*args, i32(lens))
    torch.cuda.synchronize()
    assert kda.device_error() == 0
    check_decode(args, lens, *got)
    again = kda.attention_decode(*args, i32(lens))
    assert torch.equal(again[0], got[0]) and torch.equal(again[1], got[1])


def test_decode_rows_of_packed_qkv_scale_and_given_buffers():
    lens, H, HKV, D = [300, 17, 0, 64], 8, 2, 128
    args = make_decode(E4M3, lens, H, HKV, D, 64, 3)
    packed = torch.zeros(4, (H + 2 * HKV) * D, dtype=torch.bfloat16, device="cuda")
    q = packed[:, :H * D].view(4, H, D)
    q.copy_(args[0])
    o = torch.full((4, H, D), math.nan, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((4, H), math.nan, device="cuda")
    ws = torch.full((kda.attention_decode_workspace_size(4, H, HKV, D, args[5].shape[1], 64),), 0xff, dtype=torch.uint8,
                    device="cuda")
    wide = torch.full((4, 40), 1 << 30, dtype=torch.int32, device="cuda")  # a table row inside a wider one
    wide[:, 3:3 + args[5].shape[1]] = args[5]
    table = wide[:, 3:3 + args[5].shape[1]]
    kda.attention_decode(q, *args[1:5], table, i32(lens), scale=0.3, o=o, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    check_decode(args, lens, o, lse, scale=0.3)
    again = kda.attention_decode(args[0], *args[1:], i32(lens), scale=0.3)
    assert torch.equal(again[0], o) and torch.equal(again[1], lse)


@pytest.mark.parametrize("dtype", [E4M3, INT8])
def test_decode_with_scales_far_apart(dtype):
    """Value scales 2^40 apart between blocks (weights ride on their exponents), key scales that make scores of hundreds, and a
    block whose value scale is zero.  Scores of up to S are off by S * 2^-20 or so, which weighs p and lse."""
    lens, H, HKV, D, bs = [900, 40], 8, 2, 128, 16
    q, kc, vc, ks, vs, table = make_decode(dtype, lens, H, HKV, D, bs, 9)
    g = torch.Generator("cuda").manual_seed(1)
    vs.copy_(torch.exp2(torch.randint(-40, 1, vs.shape, generator=g, device="cuda").float()))
    ks.mul_(torch.exp2(torch.randint(-6, 5, ks.shape, generator=g, device="cuda").float()))
    vs[table[0, 3].long()] = 0
    args = (q, kc, vc, ks, vs, table)
    o, lse = kda.attention_decode(*args, i32(lens))
    f, z, w, tiny = formula(*args, lens, D ** -0.5)
    s_max = 0.0
    for b, n in enumerate(lens):
        ids = table[b, :-(-n // bs)].long()
        k = (kc.view(torch.uint8)[ids].view(dtype).double() * ks[ids].double()[..., None, None]).nan_to_num()
        s_max = max(s_max, float((q[b].double().abs().view(HKV, -1, D)[None] @ k.abs().transpose(2, 3)).max()) * D ** -0.5)
    slack = 2 * (FP32 + s_max * 2.0 ** -19)
    assert ((lse.double() - z).abs() <= slack).all()
    assert ((o.double() - f).abs() <= (FP16 + slack) * w + BF16 * f.abs() + tiny).all()


def test_decode_blocks_out_of_range_and_lengths_past_the_table():
    lens, H, HKV, D, bs = [100, 50], 4, 2, 64, 16
    args = make_decode(INT8, lens, H, HKV, D, bs, 4)
    bad = args[5].clone()
    bad[0, 2], bad[0, 5] = args[1].shape[0], -3       # tokens 32..47 and 80..95 do not count
    o, lse = kda.attention_decode(*args[:5], bad, i32(lens))
    assert kda.device_error() == 16
    keep = [i for i in range(100) if i // bs not in (2, 5)]
    ids = args[5][0].long()
    k, v = ((c[ids].double() * s[ids].double()[..., None, None]).transpose(1, 2).reshape(-1, HKV, D)[keep]
            for c, s in ((args[1], args[3]), (args[2], args[4])))
    x = torch.einsum("hgd,nhd->hgn", args[0][0].double().view(HKV, 2, D), k) * D ** -0.5
    want = torch.einsum("hgn,nhd->hgd", torch.softmax(x, 2), v).reshape(H, D)
    weight = torch.einsum("hgn,nhd->hgd", torch.softmax(x, 2), v.abs()).reshape(H, D)
    assert ((o[0].double() - want).abs() <= (FP16 + FP32) * weight + BF16 * want.abs()).all()
    check_decode(tuple(a[1:] if i in (0, 5) else a for i, a in enumerate(args)), lens[1:], o[1:], lse[1:])
    none = torch.full_like(bad, -1)
    o, lse = kda.attention_decode(*args[:5], none, i32(lens))
    assert (o == 0).all() and (lse == -math.inf).all() and kda.device_error() == 16
    o, lse = kda.attention_decode(*args, i32([1000, 50]))  # row 0 is as long as its table
    assert kda.device_error() == 16
    full = bs * args[5].shape[1]
    check_decode(args, [full, 50], *kda.attention_decode(*args, i32([full, 50])))
    assert torch.equal(o[0], kda.attention_decode(*args, i32([full, 50]))[0][0]) and kda.device_error() == 0


def test_decode_same_bits_on_every_run_and_stream():
    lens = [3000, 1, 700, 0, 64, 1500]
    args = make_decode(E4M3, lens, 16, 4, 128, 32, 8)
    n = i32(lens)
    want = kda.attention_decode(*args, n)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    got = []
    for s in streams:
        with torch.cuda.stream(s):
            got.append(kda.attention_decode(*args, n))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for g in got for a, b in zip(g, want))


@pytest.mark.parametrize("dtype", [E4M3, INT8])
@pytest.mark.parametrize("D,bs", [(128, 64), (64, 16)])
def test_a_server_s_steps(dtype, D, bs):
    """Prompts through plan, attention, append; then captured steps of plan, append and decode, replayed while the requests
    grow: every step's attention is the formula's over what the cache holds, and the cache holds what plain loops store."""
    H, HKV, rows, width, blocks = 8, 2, 5, 20, 60
    g = torch.Generator("cuda").manual_seed(3)
    free = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)
    kc, vc = (torch.zeros(blocks, HKV, bs, D, dtype=torch.int8, device="cuda").view(dtype) for _ in range(2))
    ks, vs = (torch.zeros(blocks, HKV, device="cuda") for _ in range(2))
    table = torch.full((rows, width), -1, dtype=torch.int32, device="cuda")
    prompt = [37, 1, 130, 0, 64]
    T = sum(prompt)
    qkv = torch.randn(1, T, H + 2 * HKV, D, generator=g, device="cuda").bfloat16()
    q, k, v = qkv[:, :, :H], qkv[:, :, H:H + HKV], qkv[:, :, H + HKV:]
    cu, lens, slots, used = kda.cache_plan(i32([0] * rows), i32(prompt), table, free, bs, T)
    o, lse = kda.attention_forward(q, k, v, cu)
    kda.cache_append(k[0], v[0], kc, vc, ks, vs, slots)
    plain = [x.cpu().clone() for x in (torch.zeros_like(kc.view(torch.int8)).view(dtype),) * 2] + [torch.zeros(blocks, HKV)] * 2
    plain = [p.clone() for p in plain]
    plain_append(k[0].cpu(), plain[0], plain[2], slots.tolist())
    plain_append(v[0].cpu(), plain[1], plain[3], slots.tolist())

    ctx, one = lens.clone(), i32([1, 1, 1, 1, 0])  # the last request waits
    free_now = free.roll(-int(used.item())).contiguous()
    step_qkv = torch.zeros(4, H + 2 * HKV, D, dtype=torch.bfloat16, device="cuda")
    q_all = torch.zeros(rows, H, D, dtype=torch.bfloat16, device="cuda")

    def step():
        _, n, slot, took = kda.cache_plan(ctx, one, table, free_now, bs, 4)
        kda.cache_append(step_qkv[:, H:H + HKV], step_qkv[:, H + HKV:], kc, vc, ks, vs, slot)
        return (*kda.attention_decode(q_all, kc, vc, ks, vs, table, n), n, slot, took)

    state = [x.clone() for x in (kc.view(torch.uint8), vc.view(torch.uint8), ks, vs, table)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for x, y in zip((kc.view(torch.uint8), vc.view(torch.uint8), ks, vs, table), state):  # as before the trial run
        x.copy_(y)
    for i in range(40):
        step_qkv.copy_(torch.randn(step_qkv.shape, generator=g, device="cuda") * (1 + i / 4))
        q_all.copy_(torch.randn(q_all.shape, generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        o, lse, n, slot, took = out
        plain_append(step_qkv[:, H:H + HKV].cpu(), plain[0], plain[2], slot.tolist())
        plain_append(step_qkv[:, H + HKV:].cpu(), plain[1], plain[3], slot.tolist())
        check_decode((q_all, kc, vc, ks, vs, table), n.tolist(), o, lse)
        ctx.copy_(n)
        free_now.copy_(free_now.roll(-int(took.item())))
    assert n.tolist() == [77, 41, 170, 40, 64] and kda.device_error() == 0
    real = sorted({b for r, m in zip(table.tolist(), n.tolist()) for b in r[:-(-m // bs)]})
    assert len(real) == sum(-(-m // bs) for m in n.tolist())  # no block twice
    for got, want in zip((kc, vc, ks, vs), plain):
        assert torch.equal(bits(got)[real], bits(want)[real])
