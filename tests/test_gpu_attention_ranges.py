"""Causal softmax attention over whole prompts on the GPU: batches at the ends of what the calls allow.  Formula and
tolerances as in test_gpu_attention.py."""
import math

import pytest
import torch

import kda_gated_delta_prefill_b200 as kda
from tests.test_gpu_attention import HALF, check_backward, check_forward, cu_of, formula, heads, sequences

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,N", [(64, 3), (128, 3), (64, 200)])
def test_a_backward_without_any_key_is_over_when_the_next_work_starts(D, N):
    """Packed sequences that all have no keys, in a key tensor that has rows: no launch of the call may still write the
    workspace when what follows in the stream does."""
    lens, H, HKV, Tk = [90] * N + [20000], 8, 4, 300
    T = sum(lens)
    q, dout = heads(1, 1, T, H, D), heads(2, 1, T, H, D)
    k = heads(3, 1, Tk, HKV, D)
    cu, cu_k = cu_of(lens), cu_of([0] * len(lens))
    o, lse = kda.attention_forward(q, k, k, cu, cu_k)
    assert (o == 0).all() and (lse == -math.inf).all()
    ws = torch.empty(kda.attention_backward_workspace_size(1, T, H, len(lens)), dtype=torch.uint8, device="cuda")
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(50):
        dq, _, _ = kda.attention_backward(q, k, k, o, lse, dout, cu, cu_k, workspace=ws)
        ws.fill_(0x55)
        wrong += (dq != 0).sum() + (ws != 0x55).sum()
    assert wrong.item() == 0 and kda.device_error() == 0


def concentrated(kind, n, H, HKV, D, gain):
    """q, k, v, dout with rows whose probability is mostly one key's: their own, the first (a sink), or any."""
    g = torch.Generator("cuda").manual_seed(n + D)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    k, v, dout = r(1, n, HKV, D), r(1, n, HKV, D), r(1, n, H, D)
    like = k.repeat_interleave(H // HKV, 2)
    q = gain * (like if kind == "own" else like[:, :1] if kind == "first" else r(1, n, H, D)) + 0.3 * r(1, n, H, D)
    return [x.bfloat16() for x in (q, k, v, dout)]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kind,gain", [("own", 1.0), ("own", 1.4), ("first", 1.0), ("first", 1.4), ("any", 3.0), ("any", 7.0)])
@pytest.mark.parametrize("n,H,HKV", [(600, 4, 2), (2050, 2, 2), (515, 8, 1)])
def test_gradients_of_rows_with_most_probability_on_one_key(D, kind, gain, n, H, HKV):
    """There dS = P (dP - delta) is a small difference of large numbers, and delta = o . dout of a rounded o is too coarse.

    What the gradients may be off by, in the 2-norm; roundings fall independently, so sums of them count as the root of the
    sum of their squares.  dS is rounded to bf16, by half a step.  delta, off by d (half a step of each element of o, and of
    each P that o is formed with), is corrected by the sum of the row's dS: wholly in dK, and in dQ at the key with more
    than half of the probability, so that d sum_j P_j (k_j - k_top) is left, or d sum_j P_j k_j where there is none.  dP
    and the row's sum are off by D roundings of 2^-24 of their products' sizes, or twice that for the tensor cores'
    additions: 2 sqrt(D) 2^-24 < 2^-11 half steps, in the same direction for all of a row's keys or not.  The result is
    rounded by half a step."""
    q, k, v, dout = concentrated(kind, n, H, HKV, D, gain * (1.5 if D == 64 and kind != "any" else 1.0))
    o, lse = kda.attention_forward(q, k, v)
    dq, dk, dv = kda.attention_backward(q, k, v, o, lse, dout)
    assert kda.device_error() == 0
    G, scale = H // HKV, D ** -0.5
    f = formula(q[0], k[0], v[0], scale, dout[0])
    qq, do = (x[0].double().transpose(0, 1) for x in (q, dout))
    kk, vv = (x[0].double().repeat_interleave(G, 1).transpose(0, 1) for x in (k, v))
    seen = torch.ones(n, n, device="cuda", dtype=torch.bool).tril()
    p = torch.exp(qq @ kk.transpose(1, 2) * scale - f["lse"][..., None]).masked_fill(~seen, 0.0)
    dp, dp_w = do @ vv.transpose(1, 2), do.abs() @ vv.abs().transpose(1, 2)
    ds = p * (dp - (p * dp).sum(-1, keepdim=True)) * scale
    fine = 2.0 ** -11 * p * scale * (dp_w + (p * dp_w).sum(-1, keepdim=True))
    d = scale * ((do * (p @ vv)).square().sum(-1, keepdim=True) + (p * dp).square().sum(-1, keepdim=True)).sqrt()
    most, top = p.max(-1, keepdim=True)
    k_top = torch.gather(kk, 1, top.expand(-1, -1, D))
    left = torch.where(most > 0.5, p @ kk - k_top, p @ kk).abs()
    off_q = (ds.square() @ kk.square()).sqrt() + d * left + fine @ kk.abs() + f["dq"].transpose(0, 1).abs()
    off_k = (ds.square().transpose(1, 2) @ qq.square()).view(HKV, G, n, D).sum(1).sqrt() + \
        (fine.square().transpose(1, 2) @ qq.square()).view(HKV, G, n, D).sum(1).sqrt() + f["dk"].transpose(0, 1).abs()
    if kind != "any":
        assert p.amax(-1).median() > 0.9
    for name, got, off in (("dq", dq, off_q), ("dk", dk, off_k)):
        ratio = (got[0].double() - f[name]).norm() / (HALF * off.norm())
        assert ratio <= 1, (name, float(ratio))


def test_gradients_of_one_key_among_packed_sequences_and_strided_rows():
    """The key that a row's correction is taken from is the sequence's, head's and stride's."""
    lens, H, HKV, D = [300, 1, 0, 140, 600], 4, 2, 128
    T = sum(lens)
    qkv = torch.randn(1, T, H + 2 * HKV, D, generator=torch.Generator("cuda").manual_seed(1), device="cuda").bfloat16()
    q, k, v = qkv[:, :, :H], qkv[:, :, H:H + HKV], qkv[:, :, H + HKV:]
    q.copy_(k.repeat_interleave(2, 2) * 1.3)
    dout = heads(2, 1, T, H, D, gain=0.0)
    cu = cu_of(lens)
    o, lse = kda.attention_forward(q, k, v, cu)
    got = kda.attention_backward(q, k, v, o, lse, dout, cu)
    for i, n in enumerate(lens):
        if n == 0:
            continue
        a, e = sum(lens[:i]), sum(lens[:i]) + n
        part = [x[:, a:e].contiguous() for x in (q, k, v, dout)]
        oi, li = kda.attention_forward(*part[:3])
        want = kda.attention_backward(*part[:3], oi, li, part[3])
        assert all(torch.equal(x[:, a:e], y) for x, y in zip(got, want))
    assert kda.device_error() == 0


MIXED = [0, 1, 127, 128, 129, 255, 256, 257, 600, 64, 3, 40]
RANGES = [
    # T, H, HKV, D, lens, klens
    (None, 2, 1, 64, [MIXED[i * 5 % 12] for i in range(150)], [MIXED[(i * 7 + 3) % 12] for i in range(150)]),  # the slot search
    (None, 2, 2, 128, [MIXED[i * 5 % 12] for i in range(150)], None),
    (None, 4, 2, 128, [MIXED[i * 7 % 12] for i in range(129)], [MIXED[(i * 7 + 1) % 12] for i in range(129)]),
    (None, 2, 1, 128, [MIXED[i * 7 % 12] for i in range(128)], [MIXED[(i * 5 + 2) % 12] for i in range(128)]),  # levels
    (None, 2, 1, 64, [MIXED[i * 7 % 12] for i in range(70)], None),
    (None, 4, 1, 64, [MIXED[i * 11 % 12] for i in range(33)], [MIXED[(i * 11 + 5) % 12] for i in range(33)]),
    (300, 8, 1, 128, None, None),    # eight CTAs to a key tile
    (700, 16, 2, 64, None, None),
    (700, 16, 2, 128, None, None),
    (None, 8, 1, 64, [130, 300, 1], [300, 140, 20]),
    (300, 24, 3, 128, None, None),
    (200, 12, 1, 128, None, None),   # four of three heads
    (6100, 2, 1, 128, None, None),   # long prompts
    (9000, 1, 1, 64, None, None),
    (None, 2, 2, 128, [5000, 3, 1300], [5500, 3, 1200]),
]


@pytest.mark.parametrize("T,H,HKV,D,lens,klens", RANGES)
def test_many_sequences_and_heads_and_long_prompts_match_the_formula(T, H, HKV, D, lens, klens):
    T = sum(lens) if T is None else T
    Tk = T if klens is None else sum(klens)
    q, k, v = heads(1, 1, T, H, D), heads(2, 1, Tk, HKV, D), heads(3, 1, Tk, HKV, D)
    dout = heads(4, 1, T, H, D, gain=0.0)
    cu = None if lens is None else cu_of(lens)
    cu_k = None if klens is None else cu_of(klens)
    o, lse = kda.attention_forward(q, k, v, cu, cu_k)
    grads = kda.attention_backward(q, k, v, o, lse, dout, cu, cu_k)
    torch.cuda.synchronize()
    assert kda.device_error() == 0
    check_forward(q, k, v, o, lse, lens, klens)
    check_backward(q, k, v, dout, grads, lens, klens)
    for _, a, n, c, m in sequences(1, T, Tk, lens, klens):
        if m == 0:
            assert (grads[0][:, a:a + n] == 0).all()
        if n == 0:
            assert (grads[1][:, c:c + m] == 0).all() and (grads[2][:, c:c + m] == 0).all()
