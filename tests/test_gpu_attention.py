"""Causal softmax attention over whole prompts on the GPU against the formula in 64 bits.

Tolerances.  The products are bf16 with fp32 accumulation, so an output differs from the formula by the roundings to
bf16 on the way (half a step each, 2^-8 relative): of the probabilities, weighted by |v|, and of the result.  The
fp32 steps (scores summed over at most 128 products, exponentials, sums) add less than 2^-12 of the same weights at
these sizes: an error d in a score of size up to 60 is below 60 * 128 * 2^-24, and exp carries it on as a factor.
"""
import math

import pytest
import torch

import kda_gated_delta_prefill_b200 as kda

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -8  # bf16: half a step, relative
FP32 = 2.0 ** -12


def cu_of(lens, device="cuda"):
    return torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device=device)


def heads(seed, *shape, gain=0.4):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(*shape, generator=g, device="cuda")
    return (x * torch.exp(gain * torch.randn(*shape[:-3], 1, shape[-2], 1, generator=g, device="cuda"))).bfloat16()


def formula(q, k, v, scale, dout=None):
    """One sequence in float64: q [n,H,D], k and v [m,HKV,D].  Returns o, lse and sum p |v|; with dout also the
    gradients and the weights that their roundings are counted in."""
    n, H, D = q.shape
    m, HKV, _ = k.shape
    G = H // HKV
    q, k, v = q.double(), k.double(), v.double()
    kk, vv = (x.repeat_interleave(G, 1).transpose(0, 1) for x in (k, v))  # [H, m, D]
    qq = q.transpose(0, 1)
    seen = torch.arange(m, device=q.device)[None] <= torch.arange(n, device=q.device)[:, None] + m - n
    s = (qq @ kk.transpose(1, 2) * scale).masked_fill(~seen, -math.inf)
    if m == 0:
        s = s.new_zeros(H, n, 0)
    lse = torch.logsumexp(s, -1) if m else s.new_full((H, n), -math.inf)
    p = torch.where(seen, torch.exp(s - torch.where(lse.isinf(), 0.0, lse)[..., None]), 0.0)
    o = p @ vv
    out = dict(o=o.transpose(0, 1), lse=lse, o_w=(p @ vv.abs()).transpose(0, 1))
    if dout is not None:
        do = dout.double().transpose(0, 1)
        delta = (do * o).sum(-1, keepdim=True)
        dp = do @ vv.transpose(1, 2)
        ds = p * (dp - delta) * scale
        # what ds is off by, in half steps: its own rounding, that of delta (from an o that is off by half a step of
        # itself and of sum p |v|), and the fp32 sums of dp (2^-12 = 2^-4 half steps of the products)
        o_w = p @ vv.abs()
        ds_w = ds.abs() + p * scale * ((do.abs() * (o.abs() + o_w)).sum(-1, keepdim=True) +
                                       2.0 ** -4 * (do.abs() @ vv.abs().transpose(1, 2)))
        share = lambda x: x.view(HKV, G, m, D).sum(1).transpose(0, 1)  # noqa: E731
        out.update(dq=(ds @ kk).transpose(0, 1), dq_w=(ds_w @ kk.abs()).transpose(0, 1),
                   dk=share(ds.transpose(1, 2) @ qq), dk_w=share(ds_w.transpose(1, 2) @ qq.abs()),
                   dv=share(p.transpose(1, 2) @ do), dv_w=share(p.transpose(1, 2) @ do.abs()))
    return out


def sequences(B, T, Tk, lens, klens):
    if lens is None:
        return [(b, 0, T, 0, Tk) for b in range(B)]
    klens = klens or lens
    return [(0, sum(lens[:i]), lens[i], sum(klens[:i]), klens[i]) for i in range(len(lens))]


def check_forward(q, k, v, o, lse, lens=None, klens=None, scale=None):
    B, T, H, D = q.shape
    scale = D ** -0.5 if scale is None else scale
    for b, a, n, c, m in sequences(B, T, k.shape[1], lens, klens):
        if n == 0:
            continue
        f = formula(q[b, a:a + n], k[b, c:c + m], v[b, c:c + m], scale)
        got, z = o[b, a:a + n].double(), lse[b, :, a:a + n].double()
        assert torch.equal(torch.isinf(z), torch.isinf(f["lse"])) and not torch.isnan(z).any()
        none = torch.isinf(f["lse"]).T
        assert (got[none] == 0).all()
        dz = (z - f["lse"])[~torch.isinf(z)].abs()
        assert dz.numel() == 0 or dz.max() < FP32, (a, n, m, dz.max())
        tol = (HALF + FP32) * f["o_w"] + HALF * f["o"].abs() + 1e-30
        ratio = ((got - f["o"]).abs() / tol).max()
        assert ratio <= 1, (a, n, m, float(ratio))


CASES = [
    # B, T, Tk, H, HKV, D, lens, klens
    (1, 1, 1, 1, 1, 128, None, None),
    (2, 127, 127, 2, 1, 64, None, None),
    (1, 128, 128, 1, 1, 128, None, None),
    (3, 129, 129, 3, 3, 128, None, None),
    (1, 255, 255, 2, 2, 64, None, None),
    (2, 256, 256, 2, 1, 128, None, None),
    (1, 257, 257, 5, 1, 128, None, None),
    (1, 1000, 1000, 8, 2, 128, None, None),
    (1, 1000, 1000, 4, 4, 64, None, None),
    (2, 40, 300, 4, 2, 128, None, None),      # a prefix of keys
    (2, 300, 40, 4, 2, 128, None, None),      # rows that see nothing
    (1, 300, 44, 2, 2, 64, None, None),       # the whole first block sees nothing
    (1, 2500, 2500, 2, 1, 128, None, None),
    (1, 2100, 2100, 3, 1, 64, None, None),    # the second half of the last block is empty, its first sees 17 key tiles
    (1, 2350, 2350, 2, 2, 64, None, None),
    (1, 4000, 4000, 2, 1, 64, [1700, 80, 1300, 130, 790], None),
    (1, 100, 3000, 4, 2, 64, None, None),
    (1, 100, 3000, 4, 2, 128, None, None),
    (1, 905, 905, 8, 2, 128, [1, 63, 64, 65, 0, 127, 128, 129, 328], None),
    (1, 1025, 1025, 4, 1, 64, [512, 1, 511, 0, 1], None),
    (1, 278, 707, 8, 2, 128, [200, 1, 0, 77], [456, 1, 200, 50]),
    (1, 300, 600, 2, 1, 64, [150, 150], [0, 600]),
    (1, 700, 5, 2, 1, 128, [600, 100], [3, 2]),
]


@pytest.mark.parametrize("B,T,Tk,H,HKV,D,lens,klens", CASES)
def test_forward_matches_the_formula(B, T, Tk, H, HKV, D, lens, klens):
    q, k, v = heads(1, B, T, H, D), heads(2, B, Tk, HKV, D), heads(3, B, Tk, HKV, D)
    cu = None if lens is None else cu_of(lens)
    cu_k = None if klens is None else cu_of(klens)
    o, lse = kda.attention_forward(q, k, v, cu, cu_k)
    torch.cuda.synchronize()
    assert kda.device_error() == 0
    check_forward(q, k, v, o, lse, lens, klens)


def check_backward(q, k, v, dout, grads, lens=None, klens=None, scale=None):
    B, T, H, D = q.shape
    scale = D ** -0.5 if scale is None else scale
    for b, a, n, c, m in sequences(B, T, k.shape[1], lens, klens):
        if n == 0 or m == 0:
            continue
        f = formula(q[b, a:a + n], k[b, c:c + m], v[b, c:c + m], scale, dout[b, a:a + n])
        for name, g, x, e in (("dq", grads[0], a, a + n), ("dk", grads[1], c, c + m), ("dv", grads[2], c, c + m)):
            tol = (HALF + FP32) * f[name + "_w"] + HALF * f[name].abs() + 1e-30
            ratio = ((g[b, x:e].double() - f[name]).abs() / tol).max()
            assert ratio <= 1, (name, a, n, m, float(ratio))


@pytest.mark.parametrize("B,T,Tk,H,HKV,D,lens,klens", CASES)
def test_backward_matches_the_formula(B, T, Tk, H, HKV, D, lens, klens):
    q, k, v = heads(1, B, T, H, D), heads(2, B, Tk, HKV, D), heads(3, B, Tk, HKV, D)
    dout = heads(4, B, T, H, D, gain=0.0)
    cu = None if lens is None else cu_of(lens)
    cu_k = None if klens is None else cu_of(klens)
    o, lse = kda.attention_forward(q, k, v, cu, cu_k)
    grads = kda.attention_backward(q, k, v, o, lse, dout, cu, cu_k)
    torch.cuda.synchronize()
    assert kda.device_error() == 0
    check_backward(q, k, v, dout, grads, lens, klens)
    # rows without a counterpart have no gradient
    for b, a, n, c, m in sequences(B, T, Tk, lens, klens):
        if m == 0:
            assert (grads[0][b, a:a + n] == 0).all()
        if n == 0:
            assert (grads[1][b, c:c + m] == 0).all() and (grads[2][b, c:c + m] == 0).all()


def run(q, k, v, dout, cu=None, cu_k=None, **kw):
    o, lse = kda.attention_forward(q, k, v, cu, cu_k, **kw)
    return (o, lse, *kda.attention_backward(q, k, v, o, lse, dout, cu, cu_k, **kw))


@pytest.mark.parametrize("D", [64, 128])
def test_rows_of_packed_qkv_and_strided_dout(D):
    """Views of one packed tensor give the same bits as compact tensors."""
    B, T, H, HKV = 2, 300, 4, 2
    qkv = heads(5, B, T, H + 2 * HKV, D)
    q, k, v = qkv[:, :, :H], qkv[:, :, H:H + HKV], qkv[:, :, H + HKV:]
    wide = heads(6, B, T, 2 * H, D)
    dout = wide[:, :, H:]
    got = run(q, k, v, dout)
    want = run(q.contiguous(), k.contiguous(), v.contiguous(), dout.contiguous())
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    check_forward(q, k, v, got[0], got[1])
    check_backward(q, k, v, dout, got[2:])


@pytest.mark.parametrize("D", [64, 128])
def test_rows_of_no_sequence(D):
    """Rows before, between and behind the sequences hold NaN and infinities: outputs there stay as they were, and
    nothing of them reaches a result; a workspace of NaN does not either."""
    lens, klens, H, HKV = [70, 0, 200], [100, 30, 150], 4, 2
    pad_q, pad_k = 90, 60
    T, TK = sum(lens) + pad_q, sum(klens) + pad_k
    q, k, v, dout = heads(1, 1, T, H, D), heads(2, 1, TK, HKV, D), heads(3, 1, TK, HKV, D), heads(4, 1, T, H, D)
    for x, n in ((q, sum(lens)), (k, sum(klens)), (v, sum(klens)), (dout, sum(lens))):
        x[:, n:] = math.nan
        x[:, n::2] = math.inf
    cu, cu_k = cu_of(lens), cu_of(klens)
    o = torch.full((1, T, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((1, H, T), 7.0, device="cuda")
    kda.attention_forward(q, k, v, cu, cu_k, o=o, lse=lse)
    n = sum(lens)
    assert (o[:, n:] == 7).all() and (lse[:, :, n:] == 7).all()
    check_forward(q, k, v, o, lse, lens, klens)
    ws = torch.full((kda.attention_backward_workspace_size(1, T, H, 3),), 0xff, dtype=torch.uint8, device="cuda")
    o[:, n:] = math.nan
    grads = kda.attention_backward(q, k, v, o, lse, dout, cu, cu_k, workspace=ws)
    torch.cuda.synchronize()
    assert kda.device_error() == 0
    check_backward(q, k, v, dout, grads, lens, klens)
    # offsets past the tensors are cut off at them
    far = cu.clone()
    far[-1] += 10000
    o2, lse2 = kda.attention_forward(q[:, :n], k, v, far, cu_k)
    assert torch.equal(o2, o[:, :n]) and torch.equal(lse2, lse[:, :, :n])


@pytest.mark.parametrize("D,scale", [(64, 0.5), (128, 3.0), (128, 1e-6), (64, 1.0)])
def test_scores_far_apart(D, scale):
    """Maxima that grow by hundreds from key tile to key tile, and scores hundreds below them.  Scores of up to S are
    off by about S * 128 * 2^-24 here, which weighs p and lse: the bounds grow with it."""
    T, H = 700, 2
    q, k, v = heads(1, 1, T, H, D), heads(2, 1, T, H, D), heads(3, 1, T, H, D)
    k *= torch.linspace(0.1, 12, T, device="cuda")[None, :, None, None]
    k[:, 130:260] *= -1
    k = k.bfloat16()
    o, lse = kda.attention_forward(q, k, v, scale=scale)
    f = formula(q[0], k[0], v[0], scale)
    top = float((q[0].double().abs().transpose(0, 1) @ k[0].double().abs().permute(1, 2, 0)).max()) * scale
    slack = 2 * (FP32 + top * 2.0 ** -19)
    assert ((lse[0].double() - f["lse"]).abs() <= slack).all()
    tol = (HALF + slack) * f["o_w"] + HALF * f["o"].abs() + slack * 8 * v.abs().max().double()
    assert ((o[0].double() - f["o"]).abs() <= tol).all()


@pytest.mark.parametrize("D", [64, 128])
def test_gradients_against_differences(D):
    """The directional derivative of sum(o * dout) by central differences of the formula in 64 bits."""
    T, H, HKV, e = 150, 4, 2, 1e-5
    q, k, v, dout = heads(1, 1, T, H, D), heads(2, 1, T, HKV, D), heads(3, 1, T, HKV, D), heads(4, 1, T, H, D)
    grads = run(q, k, v, dout)[2:]
    loss = lambda *x: (formula(*(y[0] for y in x), D ** -0.5)["o"] * dout[0].double()).sum()  # noqa: E731
    x = [q.double(), k.double(), v.double()]
    f = formula(q[0], k[0], v[0], D ** -0.5, dout[0])
    for i, name in enumerate(("dq", "dk", "dv")):
        u = torch.randn(x[i].shape, generator=torch.Generator("cuda").manual_seed(i), device="cuda", dtype=torch.float64)
        step = lambda s: loss(*(y + s * e * u if j == i else y for j, y in enumerate(x)))  # noqa: E731
        want = (step(1) - step(-1)) / (2 * e)
        got = (grads[i].double() * u).sum()
        tol = (((HALF + FP32) * f[name + "_w"] + HALF * f[name].abs()) * u[0].abs()).sum()  # every rounding the same way
        assert (got - want).abs() <= tol and tol < 0.5 * (grads[i].double() * u).abs().sum()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,klens", [([1, 2, 3, 2, 16, 2, 5, 2, 2, 11, 2], None),
                                        ([3, 20, 2, 140], [16, 10, 1, 5])])
def test_gradients_of_rows_that_see_few_keys(D, lens, klens):
    """There P (dP - delta) is a small difference of large numbers, and delta = o . dout with its rounded o too coarse.
    The tolerance counts the roundings of P, dS and the results, and for dP and delta those of fp32 sums of D products alone:
    D 2^-24 <= 2^-17 of the products' sizes, twice that for the tensor cores' additions, so 2^-8 half steps of bf16."""
    klens = klens or lens
    H, HKV, scale = 8, 2, D ** -0.5
    q, dout = heads(11, 1, sum(lens), H, D, gain=1.0), heads(12, 1, sum(lens), H, D)
    k, v = heads(13, 1, sum(klens), HKV, D, gain=1.0), heads(14, 1, sum(klens), HKV, D)
    grads = run(q, k, v, dout, cu_of(lens), cu_of(klens))[2:]
    for _, a, n, c, m in sequences(1, 0, 0, lens, klens):
        x = [t[0, a:a + n].double().transpose(0, 1) for t in (q, dout)]
        kk, vv = (t[0, c:c + m].double().repeat_interleave(H // HKV, 1).transpose(0, 1) for t in (k, v))
        f = formula(q[0, a:a + n], k[0, c:c + m], v[0, c:c + m], scale, dout[0, a:a + n])
        seen = torch.arange(m, device="cuda")[None] <= torch.arange(n, device="cuda")[:, None] + m - n
        p = torch.exp((x[0] @ kk.transpose(1, 2) * scale) - f["lse"].nan_to_num(0, 0, 0)[..., None]) * seen
        dp, dp_w = x[1] @ vv.transpose(1, 2), x[1].abs() @ vv.abs().transpose(1, 2)
        ds = p * (dp - (p * dp).sum(-1, keepdim=True)) * scale
        w = ds.abs() + p * scale * 2.0 ** -8 * (dp_w + (p * dp_w).sum(-1, keepdim=True))
        dk_w = (w.transpose(1, 2) @ x[0].abs()).view(HKV, H // HKV, m, D).sum(1).transpose(0, 1)
        for got, want, weight in ((grads[0][0, a:a + n], f["dq"], (w @ kk.abs()).transpose(0, 1)),
                                  (grads[1][0, c:c + m], f["dk"], dk_w)):
            tol = (HALF + FP32) * weight + HALF * want.abs() + 1e-30
            assert ((got.double() - want).abs() <= tol).all(), (a, n, m)


def test_same_bits_on_every_run_and_stream():
    q, k, v, dout = heads(1, 1, 2000, 8, 128), heads(2, 1, 2000, 2, 128), heads(3, 1, 2000, 2, 128), heads(4, 1, 2000, 8, 128)
    cu = cu_of([700, 1, 1299])
    want = run(q, k, v, dout, cu)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for s in streams:  # at the same time, each with its own workspace; once by argument, else by the current stream
        with torch.cuda.stream(s):
            got.append(run(q, k, v, dout, cu) if s is not streams[0] else None)
    got[0] = run(q, k, v, dout, cu, stream=streams[0])
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want))


def test_a_stream_s_results_are_in_memory_of_that_stream():
    """What a call on another stream allocates must not be memory that the current stream has yet to write to: work is
    pending there on tensors that are already given back, of the sizes of the call's results and workspace."""
    q, k, v, dout = heads(1, 1, 1024, 4, 64), heads(2, 1, 1024, 4, 64), heads(3, 1, 1024, 4, 64), heads(4, 1, 1024, 4, 64)
    want = run(q, k, v, dout)
    ws = torch.empty(kda.attention_backward_workspace_size(1, 1024, 4), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    late = [torch.empty_like(x).fill_(6) for x in (*want, ws)]  # (loads the kernels: that would wait for the pending work)
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    for x in late:
        x.fill_(7)
    del late, x
    got = run(q, k, v, dout, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("T,H,HKV,D", [(4096, 32, 4, 128), (700, 16, 2, 128), (2100, 16, 4, 64)])
def test_same_bits_over_many_runs(T, H, HKV, D):
    """The warps of a CTA meet at barriers whose phases must not run ahead of a slow one: hundreds of launches of thousands
    of CTAs, back to back."""
    q, k, v, dout = heads(1, 1, T, H, D), heads(2, 1, T, HKV, D), heads(3, 1, T, HKV, D), heads(4, 1, T, H, D)
    want = run(q, k, v, dout)
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(150):
        for a, b in zip(run(q, k, v, dout), want):
            wrong += (a != b).sum()
    assert wrong.item() == 0 and kda.device_error() == 0


def test_captured_forward_and_backward_follow_new_inputs_and_lengths():
    """A graph of the pass replays on new values and new offsets of the same tensors."""
    T, H, HKV, D = 600, 4, 1, 128
    q, k, v, dout = (torch.empty(1, T, h, D, dtype=torch.bfloat16, device="cuda") for h in (H, HKV, HKV, H))
    cu = cu_of([100, 500])

    def fill(seed, lens):
        for i, x in enumerate((q, k, v, dout)):
            x.copy_(heads(seed + i, *x.shape))
        cu.copy_(cu_of(lens))

    fill(1, [100, 500])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(q, k, v, dout, cu)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run(q, k, v, dout, cu)
    for seed, lens in ((10, [333, 267]), (20, [1, 599]), (30, [600, 0])):
        fill(seed, lens)
        g.replay()
        torch.cuda.synchronize()
        check_forward(q, k, v, out[0], out[1], lens)
        check_backward(q, k, v, dout, out[2:], lens)
    assert kda.device_error() == 0


def test_many_sequences():
    """More sequences than a search step covers, of every length from zero up."""
    lens = [i % 37 for i in range(1500)]
    T = sum(lens)
    q, k, v, dout = heads(1, 1, T, 2, 64), heads(2, 1, T, 1, 64), heads(3, 1, T, 1, 64), heads(4, 1, T, 2, 64)
    out = run(q, k, v, dout, cu_of(lens))
    torch.cuda.synchronize()
    some = [i for i in range(1500) if i % 97 in (0, 1, 2)]
    for i in some:
        a, n = sum(lens[:i]), lens[i]
        check_forward(q[:, a:a + n], k[:, a:a + n], v[:, a:a + n], out[0][:, a:a + n], out[1][:, :, a:a + n])
        check_backward(q[:, a:a + n], k[:, a:a + n], v[:, a:a + n], dout[:, a:a + n],
                       [out[2][:, a:a + n], out[3][:, a:a + n], out[4][:, a:a + n]])
    assert kda.device_error() == 0


def test_no_queries_or_no_keys():
    q, k = heads(1, 2, 50, 4, 64), heads(2, 2, 30, 2, 64)
    none_k, none_q = k[:, :0], q[:, :0]
    o, lse = kda.attention_forward(q, none_k, none_k)
    assert (o == 0).all() and (lse == -math.inf).all()
    dq, dk, dv = kda.attention_backward(q, none_k, none_k, o, lse, q)
    assert (dq == 0).all() and dk.numel() == 0
    o, lse = kda.attention_forward(none_q, k, k)
    assert o.numel() == 0
    dq, dk, dv = kda.attention_backward(none_q, k, k, o, lse, none_q)
    assert (dk == 0).all() and (dv == 0).all()
    torch.cuda.synchronize()
    assert kda.device_error() == 0


def test_split_keys_join_by_lse():
    """The first query's attention over the prefix and over its own key, joined by their lse, is its attention over both."""
    n, m, D = 200, 500, 128
    q, k, v = heads(1, 1, n, 2, D), heads(2, 1, m, 2, D), heads(3, 1, m, 2, D)
    oa, la = kda.attention_forward(q[:, :1], k[:, :m - n], v[:, :m - n])
    ob, lb = kda.attention_forward(q[:, :1], k[:, m - n:m - n + 1], v[:, m - n:m - n + 1])
    w = torch.softmax(torch.stack([la, lb]), 0)[..., None]
    both = (w[0] * oa[0].transpose(0, 1) + w[1] * ob[0].transpose(0, 1)).float()
    f = formula(q[0], k[0], v[0], D ** -0.5)
    assert (both[0, :, 0].double() - f["o"][0]).abs().max() <= (4 * HALF * f["o_w"][0]).max()
