"""The softmax-attention operators: their workloads, their plain forms and their definitions in 64 bits.

Stacks of gated delta layers interleave full-attention layers.  Five operators serve those layers: causal attention
over packed prompts ("prefill"), the same with its gradients ("train"), block tables and slot maps from request
lengths ("plan"), storing keys and values in a paged 8-bit cache ("append"), and one-token attention over that cache
("decode").

With ``own`` false, ``run`` computes each one with elementary torch operations in 32 bits; with ``own`` true it makes
the calls that a user of ``kda_gated_delta_prefill_b200`` makes.
"""
import math

import torch

own = False

E4M3, INT8 = "e4m3", "int8"


# ------------------------------------------------------------------------------------------------ the cases
def listed():
    return [
        # a few short requests beside one another, one with a cached prefix of keys and one with fewer keys than
        # queries (its first rows see nothing): launch latency counts
        dict(name="prefill_short", kind="prefill", lens="200,1,77", klens="456,1,50", B=1, H=8, HKV=2, D=128, seed=1),
        # the packed seven-sequence prompt batch, lengths around the tile edges and one long request
        dict(name="prefill_packed", kind="prefill", lens="1,63,64,65,777,2048,8192", klens="", B=1, H=32, HKV=8, D=128,
             seed=2),
        # one long document
        dict(name="prefill_long", kind="prefill", lens="32768", klens="", B=1, H=16, HKV=4, D=128, seed=3),
        # a training step's attention: ragged packed samples with small heads, and a long context with shared heads
        dict(name="train_packed_d64", kind="train", lens="1000,313,2048,1,735", klens="", B=1, H=16, HKV=16, D=64,
             seed=4),
        dict(name="train_long", kind="train", lens="16384", klens="", B=1, H=16, HKV=4, D=128, seed=5),
        # the bookkeeping before a decode step of many requests, and before a step of long prompts
        dict(name="plan_decode", kind="plan", rows=256, most_new=1, most_old=8192, block=64, pad=0, seed=6),
        dict(name="plan_prompts", kind="plan", rows=96, most_new=16384, most_old=4096, block=16, pad=1000, seed=7),
        # one token of each request, and whole prompts, into the cache
        dict(name="append_decode", kind="append", rows=256, most_new=1, most_old=2000, block=64, HKV=8, D=128,
             type=E4M3, seed=8),
        dict(name="append_prompts", kind="append", rows=12, most_new=16384, most_old=300, block=16, HKV=8, D=128,
             type=INT8, seed=9),
        # a single request (latency), a ragged batch, and few very long requests
        dict(name="decode_one", kind="decode", rows=1, least=777, most=777, H=32, HKV=8, D=128, block=64, type=E4M3,
             empty=0, seed=10),
        dict(name="decode_batch", kind="decode", rows=64, least=500, most=12000, H=32, HKV=8, D=128, block=16,
             type=INT8, empty=2, seed=11),
        dict(name="decode_long", kind="decode", rows=4, least=90001, most=131072, H=64, HKV=8, D=128, block=128,
             type=E4M3, empty=0, seed=12),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    kind = rng.choice(["prefill", "prefill", "train", "train", "plan", "append", "decode", "decode"])
    D = rng.choice([64, 128, 128])
    HKV = rng.choice([1, 2, 3, 4, 8])
    seed = rng.randrange(1 << 30)
    if kind in ("prefill", "train"):
        H = HKV * rng.choice([1, 2, 4, 5, 8])
        B = rng.choice([1, 1, 1, 2, 3])
        cap = 8 * 32768 * 32768 * 128 if kind == "prefill" else 8 * 16384 * 16384 * 128
        n = 1 if B > 1 else _log(rng, 1, 24)
        lens = [_log(rng, 1, 32768 if kind == "prefill" else 16384) for _ in range(n)]
        klens = []
        if B == 1 and rng.random() < 0.3:
            klens = [max(1, m + rng.choice([0, 1, -1, rng.randint(-200, 3000)])) for m in lens]
        cost = lambda: B * sum(a * (c + 128) for a, c in zip(lens, klens or lens)) * H * D  # noqa: E731
        while cost() > cap or sum(klens or lens) * B * (H + 2 * HKV) * D > 3e8:
            i = lens.index(max(lens))
            if lens[i] < 64:
                lens, klens = lens[:1], klens[:1]
            lens[i % len(lens)] = max(1, lens[i % len(lens)] * 2 // 3)
            if klens:
                klens[i % len(lens)] = max(1, klens[i % len(lens)] * 2 // 3)
        return dict(kind=kind, lens=",".join(map(str, lens)), klens=",".join(map(str, klens)), B=B, H=H, HKV=HKV, D=D,
                    seed=seed)
    block = rng.choice([16, 32, 64, 128])
    if kind == "plan":
        new = rng.choice([1, 1, _log(rng, 2, 16384)])
        rows = _log(rng, 1, 2048 if new == 1 else max(1, min(2048, 700000 // new)))
        return dict(kind=kind, rows=rows, most_new=new, most_old=_log(rng, 1, 8192), block=block,
                    pad=rng.choice([0, rng.randint(1, 2000)]), seed=seed)
    if kind == "append":
        new = rng.choice([1, _log(rng, 2, 16384)])
        rows = _log(rng, 1, max(1, min(512, 90000 // new)))
        return dict(kind=kind, rows=rows, most_new=new, most_old=_log(rng, 1, 2000), block=block, HKV=HKV, D=D,
                    type=rng.choice([E4M3, INT8]), seed=seed)
    H = HKV * rng.choice([1, 2, 4, 5, 8, 12, 16])
    rows = _log(rng, 1, 256)
    most = _log(rng, 1, max(1, min(131072, 540000 // rows)))
    return dict(kind=kind, rows=rows, least=max(1, most // rng.choice([1, 4, 100])), most=most, H=H, HKV=HKV, D=D,
                block=block, type=rng.choice([E4M3, INT8]), empty=rng.choice([0, 0, 1]), seed=seed)


def _ints(text):
    return [int(x) for x in text.split(",")] if text else None


def _gen(case, seed, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed((case.get("seed", 0) * 1000003 + seed * 7919 + 17) % (1 << 62))
    return g


def _cu(lens):
    return torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda")


def _heads(g, *shape):
    """Activations whose scale differs from head to head, as projections of a normalised stream have."""
    gain = torch.exp(0.4 * torch.randn(*shape[:-3], 1, shape[-2], 1, generator=g, device="cuda"))
    return (gain * torch.randn(*shape, generator=g, device="cuda")).to(torch.bfloat16)


# ------------------------------------------------------------------------------------------------ the inputs
def _fixed(case):
    """A case's host lists (old, new): tokens that each request holds in the cache, and tokens to add; of a decode
    step: its contexts, and nothing."""
    g = _gen(case, 0, "cpu")
    n = case["rows"]
    if case["kind"] == "decode":
        lens = torch.randint(case["least"], case["most"] + 1, (n,), generator=g)
        lens[0] = case["most"]
        if case["empty"] and n > case["empty"]:
            lens[-case["empty"]:] = 0
        return lens, torch.zeros_like(lens)
    old = torch.randint(0, case["most_old"] + 1, (n,), generator=g)
    if case["most_new"] == 1:
        return old, torch.ones_like(old)
    new = torch.randint(0, case["most_new"] + 1, (n,), generator=g)
    new[0] = case["most_new"]
    return old, new


def _lengths(case, seed):
    """The same lengths, another order for another seed, so that sizes stay."""
    g = _gen(case, seed, "cpu")
    old, new = _fixed(case)
    return old[torch.randperm(old.numel(), generator=g)], new[torch.randperm(new.numel(), generator=g)]


def _blocks(case, old, new, g):
    """A block table whose rows hold the blocks of ``old`` tokens (-1 behind them), and the free blocks, in the
    shuffled order that a running server's pool has."""
    bs = case["block"]
    have = (old + bs - 1) // bs
    total = int(have.sum()) + int(((new + bs - 1) // bs).sum()) + 8
    perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    width = max(1, (int(old.max()) + int(new.max()) + bs - 1) // bs)
    cols = torch.arange(width, device="cuda")
    have_d = have.cuda()
    at = (torch.cumsum(have_d, 0) - have_d)[:, None] + cols
    table = torch.where(cols < have_d[:, None], perm[at.clamp(max=total - 1)], -1).to(torch.int32).contiguous()
    return table, perm[int(have.sum()):].contiguous(), total


def _pool(case, blocks, g):
    """A cache in use: random codes and scales, of keys and of values."""
    bs, HKV, D = case["block"], case["HKV"], case["D"]
    out = []
    for _ in range(2):
        if case["type"] == INT8:
            out.append(torch.randint(-127, 128, (blocks, HKV, bs, D), generator=g, device="cuda", dtype=torch.int8))
        else:  # finite codes of either sign: magnitudes 0 .. 448
            c = torch.randint(0, 0x7f, (blocks, HKV, bs, D), generator=g, device="cuda", dtype=torch.uint8)
            s = torch.randint(0, 2, (blocks, HKV, bs, D), generator=g, device="cuda", dtype=torch.uint8)
            out.append((c | (s << 7)).view(torch.float8_e4m3fn))
    top = 127 if case["type"] == INT8 else 448
    for _ in range(2):  # powers of two; values of a few units at most
        e = torch.randint(1, 4, (blocks, HKV), generator=g, device="cuda")
        out.append(torch.exp2(e.float() - math.ceil(math.log2(top))))
    return out


def prepare(case, seed):
    g = _gen(case, seed)
    kind = case["kind"]
    if kind in ("prefill", "train"):
        lens, klens = _ints(case["lens"]), _ints(case["klens"])
        B, H, HKV, D = case["B"], case["H"], case["HKV"], case["D"]
        T, TK = sum(lens), sum(klens or lens)
        s = dict(case=case, q=_heads(g, B, T, H, D), k=_heads(g, B, TK, HKV, D), v=_heads(g, B, TK, HKV, D))
        s["cu"] = _cu(lens) if B == 1 else None
        s["cu_k"] = _cu(klens) if klens else None
        if kind == "train":
            s["dout"] = torch.randn(B, T, H, D, generator=g, device="cuda").to(torch.bfloat16)
        return s
    if kind == "plan":
        old, new = _lengths(case, seed)
        table, free, _ = _blocks(case, old, new, g)
        return dict(case=case, old=old.to(torch.int32).cuda(), new=new.to(torch.int32).cuda(), table=table, free=free,
                    tokens=int(new.sum()) + case["pad"])
    if kind == "append":
        old, new = _lengths(case, seed)
        table, free, total = _blocks(case, old, new, g)
        slots = _plan(old.cuda(), new.cuda(), table, free, case["block"], int(new.sum()))["slot_map"]
        kc, vc, ks, vs = _pool(case, total, g)
        T = int(new.sum())
        return dict(case=case, k=_heads(g, T, case["HKV"], case["D"]), v=_heads(g, T, case["HKV"], case["D"]),
                    k_cache=kc, v_cache=vc, k_scale=ks, v_scale=vs, slots=slots)
    lens, none = _lengths(case, seed)
    table, _, total = _blocks(case, lens, none, g)
    kc, vc, ks, vs = _pool(case, total, g)
    q = _heads(g, case["rows"], case["H"], case["D"])
    return dict(case=case, q=q, k_cache=kc, v_cache=vc, k_scale=ks, v_scale=vs, table=table,
                lens=lens.to(torch.int32).cuda())


# ------------------------------------------------------------------------------------------------ plain forms
_MOST = 1 << 28  # scores held at a time


def _parts(case):
    """(batch row, first query, queries, first key, keys) of every sequence."""
    lens, klens = _ints(case["lens"]), _ints(case["klens"]) or _ints(case["lens"])
    got, a, c = [], 0, 0
    for n, m in zip(lens, klens):
        got += [(b, a, n, c, m) for b in range(case["B"])]
        a, c = a + n, c + m
    return got


def _scores(q, k, first, scale):
    """Scores [HKV, group, rows, keys] of query rows first.. (counted so that row i sees keys 0 .. i)."""
    n, H, D = q.shape
    m, HKV, _ = k.shape
    qh = q.reshape(n, HKV, H // HKV, D).permute(1, 2, 0, 3).reshape(HKV, -1, D)
    s = torch.matmul(qh, k.permute(1, 2, 0)).view(HKV, H // HKV, n, m) * scale
    seen = torch.arange(m, device=q.device) <= (first + torch.arange(n, device=q.device))[:, None]
    return qh, s.masked_fill_(~seen, -math.inf)


def _attention(s, dout=None):
    case = s["case"]
    q, k, v = (s[n].float() for n in ("q", "k", "v"))
    B, T, H, D = q.shape
    HKV, G = case["HKV"], H // case["HKV"]
    scale = D ** -0.5
    o, lse = torch.zeros_like(q), torch.full((B, H, T), -math.inf, device="cuda")
    if dout is not None:
        dout = dout.float()
        dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for b, a, n, c, m in _parts(case):
        step = max(1, min(n, _MOST // (H * m)))
        for r in range(0, n, step):
            e = min(n, r + step)
            hi = max(1, min(m, e + m - n))  # no row of this block sees a later key
            ks, vs = k[b, c:c + hi], v[b, c:c + hi]
            qh, x = _scores(q[b, a + r:a + e], ks, r + m - n, scale)
            top = x.amax(-1, keepdim=True)
            p = torch.exp(x - torch.where(top.isinf(), 0.0, top))
            total = p.sum(-1, keepdim=True)
            p = p / torch.where(total == 0, 1.0, total)
            out = torch.matmul(p.view(HKV, -1, hi), vs.permute(1, 0, 2)).view(HKV, G, e - r, D)
            o[b, a + r:a + e] = out.permute(2, 0, 1, 3).reshape(e - r, H, D)
            lse[b, :, a + r:a + e] = (top + torch.log(total)).view(H, e - r)
            if dout is not None:
                do = dout[b, a + r:a + e].reshape(e - r, HKV, G, D).permute(1, 2, 0, 3)
                delta = (do * out).sum(-1, keepdim=True)
                do = do.reshape(HKV, -1, D)
                ds = (torch.matmul(do, vs.permute(1, 2, 0)).view_as(p) - delta) * p * scale
                p, ds = p.view(HKV, -1, hi), ds.view(HKV, -1, hi)
                dv[b, c:c + hi] += torch.matmul(p.transpose(1, 2), do).permute(1, 0, 2)
                dk[b, c:c + hi] += torch.matmul(ds.transpose(1, 2), qh).permute(1, 0, 2)
                g = torch.matmul(ds, ks.permute(1, 0, 2)).view(HKV, G, e - r, D)
                dq[b, a + r:a + e] = g.permute(2, 0, 1, 3).reshape(e - r, H, D)
    got = dict(o=o.to(torch.bfloat16), lse=lse)
    if dout is not None:
        got.update(dq=dq.to(torch.bfloat16), dk=dk.to(torch.bfloat16), dv=dv.to(torch.bfloat16))
    return got


def _plan(old, new, table, free, bs, tokens):
    old, new = old.long(), new.long()
    cu = torch.cat([new.new_zeros(1), torch.cumsum(new, 0)])
    have, need = (old + bs - 1) // bs, (old + new + bs - 1) // bs
    more = need - have
    start = torch.cumsum(more, 0) - more
    cols = torch.arange(table.shape[1], device=table.device)
    at = (start - have)[:, None] + cols
    fresh = (cols >= have[:, None]) & (cols < need[:, None])
    if free.numel():
        table.copy_(torch.where(fresh, free[at.clamp(0, free.numel() - 1)], table))
    t = torch.arange(tokens, device=table.device)
    row = torch.searchsorted(cu, t, right=True) - 1
    real = t < cu[-1]
    row = row.clamp(max=old.numel() - 1)
    pos = torch.where(real, old[row] + t - cu[row], 0)
    slot = table[row, (pos // bs).clamp(max=table.shape[1] - 1)].long() * bs + pos % bs
    return dict(block_table=table, cu_seqlens=cu.to(torch.int32), seq_lens=(old + new).to(torch.int32),
                slot_map=torch.where(real, slot, -1).to(torch.int32), used=more.sum().to(torch.int32).view(1))


def _code(x, kind):
    """Values over their scale as 8-bit codes: nearest, ties to even."""
    if kind == INT8:
        return x.round().clamp(-127, 127).to(torch.int8)
    return x.clamp(-448, 448).to(torch.float8_e4m3fn)


def _append(x, cache, scale, slots, kind):
    """One power-of-two scale per block and head: the smallest that the block's tokens fit, never smaller than it
    was while the block holds earlier tokens, which are rounded again when it grows."""
    _, HKV, bs, D = cache.shape
    real = slots >= 0
    blk, off = (slots // bs)[real].long(), (slots % bs)[real].long()
    x = x.float()[real]
    blocks, inv = torch.unique(blk, return_inverse=True)
    start = torch.full((blocks.numel(),), bs, device="cuda").scatter_reduce_(0, inv, off, "amin")
    top = torch.zeros(blocks.numel(), HKV, device="cuda")
    top.scatter_reduce_(0, inv[:, None].expand(-1, HKV), x.abs().amax(-1), "amax")
    mant, expo = torch.frexp(top)  # top = mant 2^expo, 1/2 <= mant < 1; the largest code is mant0 2^expo0
    mant0, expo0 = (127 / 128, 7) if kind == INT8 else (448 / 512, 9)
    s = torch.exp2((expo - expo0 + (mant > mant0).int()).clamp(min=-100).float())
    s = torch.where(top == 0, 2.0 ** -100, s)
    old = scale[blocks]
    kept = (start > 0)[:, None]
    s = torch.where(kept, torch.maximum(old, s), s)
    scale[blocks] = s
    was = cache[blocks] if kind == INT8 else cache.view(torch.uint8)[blocks].view(torch.float8_e4m3fn)
    again = _code(was.float() * (old / s)[:, :, None, None], kind).view(torch.uint8)
    earlier = torch.arange(bs, device="cuda") < start[:, None]
    raw = cache.view(torch.uint8)
    raw[blocks] = torch.where(earlier[:, None, :, None], again, was.view(torch.uint8))
    raw[blk, :, off] = _code(x / s[inv][:, :, None], kind).view(torch.uint8)


def _decode(s):
    case, q, lens = s["case"], s["q"].float(), s["lens"].long()
    B, H, D = q.shape
    HKV, bs = case["HKV"], case["block"]
    n = s["table"].shape[1]
    at = s["table"].clamp(min=0).long()

    def gathered(cache, scale):
        x = (cache if case["type"] == INT8 else cache.view(torch.uint8))[at]
        x = (x if case["type"] == INT8 else x.view(torch.float8_e4m3fn)).float()
        x.mul_(scale[at][..., None, None])
        return x.permute(0, 2, 1, 3, 4).reshape(B, HKV, n * bs, D)

    x = torch.matmul(q.view(B, HKV, H // HKV, D), gathered(s["k_cache"], s["k_scale"]).transpose(2, 3)) * D ** -0.5
    x.masked_fill_(torch.arange(n * bs, device="cuda") >= lens[:, None, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top.isinf(), 0.0, top))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total == 0, 1.0, total)
    o = torch.matmul(p, gathered(s["v_cache"], s["v_scale"]))
    return dict(o=o.view(B, H, D).to(torch.bfloat16), lse=(top + torch.log(total)).view(B, H))


def run(state):
    s, case = state, state["case"]
    kind = case["kind"]
    if own:
        import kda_gated_delta_prefill_b200 as kda
        if kind == "prefill":
            o, lse = kda.attention_forward(s["q"], s["k"], s["v"], s["cu"], s["cu_k"])
            return dict(o=o, lse=lse)
        if kind == "train":
            o, lse = kda.attention_forward(s["q"], s["k"], s["v"], s["cu"], s["cu_k"])
            dq, dk, dv = kda.attention_backward(s["q"], s["k"], s["v"], o, lse, s["dout"], s["cu"], s["cu_k"])
            return dict(o=o, lse=lse, dq=dq, dk=dk, dv=dv)
        if kind == "plan":
            cu, lens, slots, used = kda.cache_plan(s["old"], s["new"], s["table"], s["free"], case["block"],
                                                   s["tokens"])
            return dict(block_table=s["table"], cu_seqlens=cu, seq_lens=lens, slot_map=slots, used=used)
        if kind == "append":
            kda.cache_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["slots"])
            return {n: s[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale")}
        o, lse = kda.attention_decode(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"],
                                      s["lens"])
        return dict(o=o, lse=lse)
    if kind == "prefill":
        return _attention(s)
    if kind == "train":
        return _attention(s, s["dout"])
    if kind == "plan":
        return _plan(s["old"], s["new"], s["table"], s["free"], case["block"], s["tokens"])
    if kind == "append":
        _append(s["k"], s["k_cache"], s["k_scale"], s["slots"], case["type"])
        _append(s["v"], s["v_cache"], s["v_scale"], s["slots"], case["type"])
        return {n: s[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale")}
    return _decode(s)


# ------------------------------------------------------------------------------------------------ floors
def work(case):
    kind = case["kind"]
    if kind in ("prefill", "train"):
        lens, klens = _ints(case["lens"]), _ints(case["klens"]) or _ints(case["lens"])
        B, H, HKV, D = case["B"], case["H"], case["HKV"], case["D"]
        pairs = 0
        for n, m in zip(lens, klens):  # row i sees i + 1 + m - n keys, where that is positive
            first = max(1, 1 + m - n)
            rows = m - first + 1
            pairs += (first + m) * rows // 2 if rows > 0 else 0
        pairs *= B * H
        q, kv, stat = B * sum(lens) * H * D * 2, B * sum(klens) * HKV * D * 2, B * sum(lens) * H * 4
        if kind == "prefill":
            return {"bytes": 2 * q + 2 * kv + stat, "flops": 4 * D * pairs}
        return {"bytes": 4 * q + 4 * kv + stat, "flops": 14 * D * pairs}
    if kind in ("plan", "append"):
        old, new = _lengths(case, 1)
        bs, T = case["block"], int(new.sum())
        more = int(((old + new + bs - 1) // bs - (old + bs - 1) // bs).sum())
        if kind == "plan":
            return {"bytes": 4 * (4 * case["rows"] + 2 + 2 * more + T + case["pad"]), "flops": 0}
        touched = int(torch.where(new > 0, (old + new + bs - 1) // bs - old // bs, 0).sum())
        return {"bytes": 2 * (3 * T * case["HKV"] * case["D"] + 8 * touched * case["HKV"]) + 4 * T, "flops": 0}
    lens, _ = _fixed(case)
    n, blocks = int(lens.sum()), int(((lens + case["block"] - 1) // case["block"]).sum())
    return {"bytes": 2 * n * case["HKV"] * case["D"] + blocks * (8 * case["HKV"] + 4) + case["rows"] * case["H"] *
            (4 * case["D"] + 4), "flops": 4 * n * case["H"] * case["D"]}


# ------------------------------------------------------------------------------------------------ 64 bits
def _exact_attention(s, train):
    """Head by head: softmax(q k^T / sqrt(D) + mask) v and its derivative, every matrix written out."""
    case = s["case"]
    q, k, v = (s[n].double() for n in ("q", "k", "v"))
    B, T, H, D = q.shape
    group = H // case["HKV"]
    o, lse = torch.zeros_like(q), torch.full((B, H, T), -math.inf, dtype=torch.float64, device="cuda")
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for b, a, n, c, m in _parts(case):
        rows = max(1, min(n, (1 << 27) // m))
        for h in range(H):
            K, V = k[b, c:c + m, h // group], v[b, c:c + m, h // group]
            for r in range(0, n, rows):
                e = min(n, r + rows)
                Q = q[b, a + r:a + e, h]
                last = torch.arange(r, e, device="cuda") + (m - n)
                x = (Q @ K.T) / math.sqrt(D)
                hidden = torch.arange(m, device="cuda")[None, :] > last[:, None]
                z = torch.logsumexp(x.masked_fill(hidden, -math.inf), 1)
                p = torch.exp(x - torch.where(last < 0, 0.0, z)[:, None]).masked_fill(hidden, 0.0)
                o[b, a + r:a + e, h] = p @ V
                lse[b, h, a + r:a + e] = z
                if train:
                    do = s["dout"][b, a + r:a + e, h].double()
                    dp = do @ V.T
                    dx = p * (dp - (p * dp).sum(1, keepdim=True)) / math.sqrt(D)
                    dq[b, a + r:a + e, h] = dx @ K
                    dk[b, c:c + m, h // group] += dx.T @ Q
                    dv[b, c:c + m, h // group] += p.T @ do
    return dict(o=o, lse=lse, dq=dq, dk=dk, dv=dv) if train else dict(o=o, lse=lse)


def exact(case, seed):
    kind = case["kind"]
    s = prepare(case, seed)
    if kind in ("prefill", "train"):
        return _exact_attention(s, kind == "train")
    if kind == "plan":
        return None
    if kind == "append":
        got = {}
        bs = case["block"]
        slots = s["slots"].long()
        blocks, at = torch.unique_consecutive(slots // bs, return_inverse=True)
        begin = torch.full((blocks.numel(),), bs, device="cuda").index_reduce_(0, at, slots % bs, "amin")
        for n, most in (("k", 127.0 if case["type"] == INT8 else 448.0), ("v", 127.0 if case["type"] == INT8 else 448.0)):
            x = s[n].double()
            top = torch.zeros(blocks.numel(), case["HKV"], dtype=torch.float64, device="cuda")
            top.index_reduce_(0, at, x.abs().amax(2), "amax")
            low = torch.ldexp(torch.ones_like(top), torch.frexp((top / most).clamp(min=2.0 ** -99))[1] - 2)
            need = torch.where(top <= most * low, low, torch.where(top <= most * 2 * low, 2 * low, 4 * low))
            was = s[n + "_scale"].double()
            now = torch.where((begin > 0)[:, None], torch.maximum(need, was[blocks]), need)
            whole = was.clone()
            whole[blocks] = now
            got[n + "_scale"] = whole
            if case["type"] == INT8:
                got[n + "_cache"] = None
                continue
            pool = s[n + "_cache"].double()
            ratio = torch.ones_like(was)
            ratio[blocks] = was[blocks] / now
            first = torch.full((pool.shape[0],), 0, device="cuda")
            first[blocks] = begin
            early = (torch.arange(bs, device="cuda") < first[:, None])[:, None, :, None]
            pool *= torch.where(early, ratio[:, :, None, None], 1.0)
            pool[slots // bs, :, slots % bs] = x / now[at][:, :, None]
            got[n + "_cache"] = pool
        return got
    B, H, D = s["q"].shape
    o = torch.zeros(B, H, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, H), -math.inf, dtype=torch.float64, device="cuda")
    group, bs = H // case["HKV"], case["block"]
    if case["rows"] > 300:
        return None
    for b, n in enumerate(s["lens"].tolist()):
        if n == 0:
            continue
        ids = s["table"][b, :(n + bs - 1) // bs].tolist()
        ids = torch.tensor(ids, device="cuda")
        raw = {}
        for x in ("k", "v"):
            c = s[x + "_cache"].view(torch.uint8)[ids].view(s[x + "_cache"].dtype).double()
            c = c * s[x + "_scale"][ids].double()[:, :, None, None]
            raw[x] = c.transpose(1, 2).reshape(-1, case["HKV"], D)[:n].transpose(0, 1)
        x = torch.einsum("hgd,hnd->hgn", s["q"][b].double().view(-1, group, D), raw["k"]) / math.sqrt(D)
        z = torch.logsumexp(x, 2)
        o[b] = torch.einsum("hgn,hnd->hgd", torch.exp(x - z[..., None]), raw["v"]).reshape(H, D)
        lse[b] = z.reshape(H)
    return dict(o=o, lse=lse)
