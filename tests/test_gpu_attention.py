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
