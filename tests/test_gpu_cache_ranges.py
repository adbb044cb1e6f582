"""The paged 8-bit cache on the GPU at the ends of its ranges: value scales, lengths.  Tolerances as in test_gpu_cache.py,
whose formula in 64 bits this uses; a score of up to S is off by S * 2^-19 at most (fp32 sums of 128 products and its own
rounding), which weighs p and lse."""
import math

import pytest
import torch

import kda_gated_delta_prefill_b200 as kda
from tests.test_gpu_cache import BF16, E4M3, FP16, FP32, INT8, check_decode, formula, i32, make_decode

pytestmark = pytest.mark.gpu


def top_score(args, lens):
    """The largest sum of |q| |k| over the dims, scaled: bounds every score."""
    q, kc, _, ks, _, table = args
    most = 0.0
    for b, n in enumerate(lens):
        ids = table[b, :-(-n // kc.shape[2])].long()
        k = (kc.view(torch.uint8)[ids].view(kc.dtype).double() * ks[ids].double()[..., None, None]).nan_to_num()
        qh = q[b].double().abs().view(kc.shape[1], -1, q.shape[2])
        most = max(most, float((qh[None] @ k.abs().transpose(2, 3)).max()))
    return most * q.shape[2] ** -0.5


def check_scales(args, lens):
    n = i32(lens)
    o, lse = kda.attention_decode(*args, n)
    f, z, w, tiny = formula(*args, lens, args[0].shape[2] ** -0.5)
    slack = 2 * (FP32 + top_score(args, lens) * 2.0 ** -19)
    assert ((lse.double() - z).abs() <= slack).all(), float((lse.double() - z).abs().max())
    # (below 2^-126 bf16 has steps of 2^-133, and fp32 of 2^-149)
    assert ((o.double() - f).abs() <= (FP16 + slack) * w + BF16 * f.abs() + tiny + 2.0 ** -134 + 2.0 ** -149).all()
    assert kda.device_error() == 0


@pytest.mark.parametrize("dtype", [E4M3, INT8])
@pytest.mark.parametrize("D,bs,H,HKV,n", [(128, 128, 8, 1, 70000), (64, 64, 16, 1, 131072), (128, 16, 2, 2, 3000),
                                          (64, 32, 4, 2, 65536)])
def test_decode_of_a_cache_of_zeros(dtype, D, bs, H, HKV, n):
    """Zero keys and values as cache_append stores them, at scale 2^-100: o is 0 and lse the logarithm of the length."""
    blocks = 4
    kc, vc = (torch.ones(blocks, HKV, bs, D, device="cuda").to(dtype) for _ in range(2))
    ks, vs = torch.ones(blocks, HKV, device="cuda"), torch.ones(blocks, HKV, device="cuda")
    zero = torch.zeros(blocks * bs, HKV, D, dtype=torch.bfloat16, device="cuda")
    kda.cache_append(zero, zero, kc, vc, ks, vs, torch.arange(blocks * bs, dtype=torch.int32, device="cuda"))
    assert (vs == 2.0 ** -100).all()
    table = (torch.arange(-(-n // bs), device="cuda") % blocks).to(torch.int32)[None].repeat(2, 1)
    q = torch.randn(2, H, D, generator=torch.Generator("cuda").manual_seed(0), device="cuda").bfloat16()
    lens = [n, n // 2 + 1]
    o, lse = kda.attention_decode(q, kc, vc, ks, vs, table, i32(lens))
    assert (o == 0).all()
    want = torch.tensor([math.log(m) for m in lens], dtype=torch.float64, device="cuda")[:, None]
    assert ((lse.double() - want).abs() < FP32).all(), lse
    assert kda.device_error() == 0


@pytest.mark.parametrize("dtype", [E4M3, INT8])
@pytest.mark.parametrize("D,bs", [(128, 16), (128, 64), (64, 16), (64, 128)])
@pytest.mark.parametrize("lens,H,HKV,width", [([900, 40], 8, 2, None), ([9000, 300], 12, 1, None), ([900, 40], 8, 2, 2000)])
@pytest.mark.parametrize("low,high", [(-120, -120), (-100, -5), (-120, 100), (-60, 60), (110, 110), (-149, -140)])
def test_decode_of_any_value_scale(dtype, D, bs, lens, H, HKV, width, low, high):
    """Value scales between 2^low and 2^high, block by block: alone, next to ordinary ones, and further apart than fp32's
    exponents reach; in a narrow table (one launch) and in a wide one."""
    args = list(make_decode(dtype, lens, H, HKV, D, bs, 21, width=width and width * 16 // bs))
    g = torch.Generator("cuda").manual_seed(5)
    some = torch.rand(args[4].shape, generator=g, device="cuda") < 0.5
    args[4] = torch.tensor([2.0 ** high, 2.0 ** low], device="cuda")[some.long()]
    check_scales(args, lens)


@pytest.mark.parametrize("first,then", [(-100, 100), (100, -100)])
def test_decode_of_value_scales_that_jump(first, then):
    """Pieces of a unit whose scales are 2^200 apart: the sum of either counts in both."""
    lens, H, HKV, D, bs = [60000], 4, 1, 128, 64
    args = list(make_decode(E4M3, lens, H, HKV, D, bs, 22))
    half = args[5][0, :400].long()
    args[4].fill_(2.0 ** then)
    args[4][half] = 2.0 ** first
    check_scales(args, lens)


def test_decode_of_all_scales_zero():
    lens, H, HKV, D, bs = [500, 17], 4, 2, 64, 16
    args = list(make_decode(E4M3, lens, H, HKV, D, bs, 23))
    args[4].zero_()
    o, lse = kda.attention_decode(*args, i32(lens))
    assert (o == 0).all()
    args[4].fill_(1.0)
    check_decode(args, lens, *kda.attention_decode(*args, i32(lens)))
    assert torch.equal(lse, kda.attention_decode(*args, i32(lens))[1])


def test_plan_reports_tokens_of_a_held_block_that_is_missing():
    """What an earlier call could not supply stays missing when its lengths are carried on: its tokens have no slot, which
    the error word says again; so do held entries and free blocks that name no block."""
    table = i32([[3, -7, -7, -7], [5, -7, -7, -7]])
    _, lens, slots, used = kda.cache_plan(i32([10, 16]), i32([30, 1]), table, i32([4]), 16, 31)
    assert used.tolist() == [1] and table.tolist() == [[3, 4, -1, -7], [5, -1, -7, -7]]
    assert slots.tolist() == [*range(58, 64), *range(64, 80), *[-1] * 9] and kda.device_error() == 32
    _, lens, slots, used = kda.cache_plan(lens, i32([10, 0]), table, i32([8, 9]), 16, 10)
    assert used.tolist() == [1] and lens.tolist() == [50, 17] and table.tolist() == [[3, 4, -1, 8], [5, -1, -7, -7]]
    assert slots.tolist() == [-1] * 8 + [128, 129] and kda.device_error() == 32
    kda.cache_plan(lens, i32([1, 0]), table, i32([8, 9]), 16, 1)  # the other row's block is not asked for
    assert kda.device_error() == 0
    _, _, slots, _ = kda.cache_plan(i32([20]), i32([13]), i32([[3, 1 << 30, 0]]), i32([-2]), 16, 13)
    assert slots.tolist() == [-1] * 13 and kda.device_error() == 32
    # from the length before the row is planned anew
    _, lens, slots, used = kda.cache_plan(i32([32, 16]), i32([8, 1]), table, i32([6, 7]), 16, 9)
    assert table.tolist() == [[3, 4, 6, 8], [5, 7, -7, -7]] and slots.tolist() == [*range(96, 104), 112]
    assert kda.device_error() == 0


def test_plan_of_lengths_whose_sums_pass_32_bits():
    """Lengths that are no lengths (of a row not in use, say) give no slot and no block of another row: sums stop at
    2^31 - 1."""
    top = 2 ** 31 - 1
    table = i32([[1, 2], [-7, -7]])
    cu, lens, slots, used = kda.cache_plan(i32([top, 0]), i32([1, 20]), table, i32([4, 5]), 16, 20)
    assert cu.tolist() == [0, 0, 20] and lens.tolist() == [top, 20] and used.tolist() == [2]
    assert table.tolist() == [[1, 2], [4, 5]] and slots.tolist() == list(range(64, 84)) and kda.device_error() == 32
    table = i32([[-7], [3], [-7]])
    cu, lens, slots, used = kda.cache_plan(i32([0, 5, 0]), i32([top, top, 7]), table, i32([4, 5, 6]), 16, 40)
    assert cu.tolist() == [0, top, top, top] and lens.tolist() == [top, top, 7] and used.tolist() == [3]
    assert table.tolist() == [[4], [3], [-1]] and slots.tolist() == [*range(64, 80), *[-1] * 24]
    assert kda.device_error() == 32
    rows = 700  # blocks, too, pass 2^31
    table = torch.full((rows, 3), -7, dtype=torch.int32, device="cuda")
    cu, lens, slots, used = kda.cache_plan(i32([0] * rows), i32([17] + [top] * (rows - 1)), table, i32([9, 8, 7, 6]), 16, 50)
    assert cu[:3].tolist() == [0, 17, top] and (cu[2:] == top).all() and used.tolist() == [4]
    assert table[:2].tolist() == [[9, 8, -7], [7, 6, -1]] and (table[2:] == -1).all()
    assert slots.tolist() == [*range(144, 160), 128, *range(112, 128), *range(96, 112), -1] and kda.device_error() == 32


def test_decode_of_a_length_near_2_31():
    """One block, 2^24 times in a row of the table.  444 CTAs take 37,800 tiles each, and a lane adds two terms a tile to its
    sums, which rounds them by 2^-24 of themselves at most: 75,600 * 2^-24 < 2^-7."""
    H, D, bs, width = 2, 64, 128, 1 << 24
    q, kc, vc, ks, vs, _ = make_decode(INT8, [128], H, 1, D, bs, 31)
    table = torch.zeros(1, width, dtype=torch.int32, device="cuda")
    f, z, w, _ = formula(q, kc, vc, ks, vs, torch.zeros(1, 1, dtype=torch.int32, device="cuda"), [128], D ** -0.5)
    for n, cut, err in ((2 ** 31 - 4096, 0, 0), (2 ** 31 - 64, 4032, 16), (2 ** 31 - 1, 4095, 16)):
        o, lse = kda.attention_decode(q, kc, vc, ks, vs, table, i32([n]))
        assert kda.device_error() == err
        assert ((lse.double() - z - math.log((n - cut) / 128)).abs() < 2.0 ** -7).all()
        assert ((o.double() - f).abs() <= (2.0 ** -6 + FP16) * w + BF16 * f.abs()).all()
