"""What the softmax-attention entry points refuse, on the host: the C library's status codes and the binding's
errors, before anything is launched (no GPU)."""
import ctypes

import pytest
import torch

import kda_gated_delta_prefill_b200 as kda
from kda_gated_delta_prefill_b200 import build as kbuild

FAKE, STEP = 1 << 20, 1 << 36  # addresses far apart that are never dereferenced
INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = 1, 2, 3, 4


@pytest.fixture(scope="module")
def L():
    kbuild.build()
    return kda.lib()


def ptr(i):
    return None if i is None else FAKE + int(i * STEP)


BYTE = 1 / STEP


def forward(L, q=1, qs=None, k=2, ks=None, v=3, vs=None, cu=None, cu_k=None, n=0, B=2, T=100, Tk=120, H=4, HKV=2, D=128,
            scale=0.1, o=4, lse=5):
    qs, ks, vs = (H * D if qs is None else qs), (HKV * D if ks is None else ks), (HKV * D if vs is None else vs)
    return L.kda_attention_forward(ptr(q), qs, ptr(k), ks, ptr(v), vs, ptr(cu), ptr(cu_k), n, B, T, Tk, H, HKV, D, scale,
                                   ptr(o), ptr(lse), None)


PACKED = dict(B=1, cu=6, cu_k=7, n=3)
SHAPES = [
    (dict(B=0), INVALID), (dict(T=-1), INVALID), (dict(Tk=-1), INVALID), (dict(H=0), INVALID), (dict(HKV=0), INVALID),
    (dict(H=3), INVALID), (dict(D=96), UNSUPPORTED), (dict(D=256), UNSUPPORTED), (dict(scale=0.0), INVALID),
    (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(cu=6), INVALID), (dict(cu=6, cu_k=7, n=0, B=1), INVALID), (dict(n=2), INVALID), (dict(PACKED, B=2), INVALID),
    (dict(PACKED, cu_k=None), INVALID), (dict(PACKED, cu=6 + 2 * BYTE), MISALIGNED),
    (dict(B=1 << 15, T=1 << 16), UNSUPPORTED), (dict(B=1 << 15, Tk=1 << 16), UNSUPPORTED),
    (dict(B=1, T=1 << 30, H=1 << 12, HKV=1), UNSUPPORTED),
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(q=1 + 8 * BYTE), MISALIGNED), (dict(k=2 + 2 * BYTE), MISALIGNED), (dict(vs=2 * 128 + 4), MISALIGNED),
    (dict(qs=128), INVALID), (dict(ks=0), INVALID),
]


@pytest.mark.parametrize("over,code", SHAPES + [
    (dict(o=None), INVALID), (dict(lse=None), INVALID), (dict(o=4 + 8 * BYTE), MISALIGNED), (dict(lse=5 + 2 * BYTE), MISALIGNED),
    (dict(o=1), INVALID), (dict(o=3 + 1024 * BYTE), INVALID), (dict(lse=2), INVALID), (dict(lse=4), INVALID),
    (dict(PACKED, lse=6), INVALID), (dict(PACKED, o=7), INVALID),
])
def test_forward_refuses(L, over, code):
    assert forward(L, **over) == code


def test_forward_without_queries_is_a_no_op(L):
    assert forward(L, T=0, q=None, o=None, lse=None) == 0


def backward(L, q=1, qs=None, k=2, ks=None, v=3, vs=None, o=4, lse=5, do=8, dos=None, cu=None, cu_k=None, n=0, B=2, T=100,
             Tk=120, H=4, HKV=2, D=128, scale=0.1, dq=9, dk=10, dv=11, ws=12, nbytes=None):
    qs, ks, vs = (H * D if qs is None else qs), (HKV * D if ks is None else ks), (HKV * D if vs is None else vs)
    nbytes = L.kda_attention_backward_workspace_size(B, T, H, n) if nbytes is None else nbytes
    return L.kda_attention_backward(ptr(q), qs, ptr(k), ks, ptr(v), vs, ptr(o), ptr(lse), ptr(do),
                                    H * D if dos is None else dos, ptr(cu), ptr(cu_k), n, B, T, Tk, H, HKV, D, scale,
                                    ptr(dq), ptr(dk), ptr(dv), ptr(ws), nbytes, None)


@pytest.mark.parametrize("over,code", SHAPES + [
    (dict(o=None), INVALID), (dict(lse=None), INVALID), (dict(do=None), INVALID), (dict(dq=None), INVALID),
    (dict(dk=None), INVALID), (dict(dv=None), INVALID), (dict(ws=None), INVALID), (dict(nbytes=100), WORKSPACE),
    (dict(dos=4 * 128 + 2), MISALIGNED), (dict(dq=9 + 8 * BYTE), MISALIGNED), (dict(ws=12 + 4 * BYTE), MISALIGNED),
    (dict(dq=1), INVALID), (dict(dk=10, dv=10), INVALID), (dict(ws=8), INVALID), (dict(dv=4), INVALID),
])
def test_backward_refuses(L, over, code):
    assert backward(L, **over) == code


def test_backward_of_nothing_is_a_no_op(L):
    assert backward(L, T=0, Tk=0, q=None, k=None, v=None, o=None, lse=None, do=None, dq=None, dk=None, dv=None, ws=None) == 0


def test_backward_workspace_size(L):
    f = L.kda_attention_backward_workspace_size
    assert f(2, 100, 4, 0) == 2 * 4 * 1024            # a tile of statistics per sequence and head
    assert f(1, 1000, 4, 3) == (1000 // 128 + 3) * 4 * 1024
    assert f(0, 100, 4, 0) == f(2, 100, 4, 1) == f(1, -1, 4, 0) == 0


def plan(L, ctx=1, new=2, B=4, table=3, stride=10, width=10, free=4, nfree=5, bs=64, cu=5, lens=6, slots=7, tokens=9, used=8):
    return L.kda_cache_plan(ptr(ctx), ptr(new), B, ptr(table), stride, width, ptr(free), nfree, bs, ptr(cu), ptr(lens),
                            ptr(slots), tokens, ptr(used), None)


@pytest.mark.parametrize("over,code", [
    (dict(B=0), INVALID), (dict(B=16385), UNSUPPORTED), (dict(width=0), INVALID), (dict(stride=9), INVALID),
    (dict(nfree=-1), INVALID), (dict(tokens=-1), INVALID), (dict(bs=48), UNSUPPORTED), (dict(bs=8), UNSUPPORTED),
    (dict(bs=0), UNSUPPORTED), (dict(ctx=None), INVALID), (dict(table=None), INVALID), (dict(free=None), INVALID),
    (dict(slots=None), INVALID), (dict(used=None), INVALID), (dict(cu=5 + BYTE), MISALIGNED),
    (dict(table=1), INVALID), (dict(slots=4), INVALID), (dict(lens=5), INVALID), (dict(used=2), INVALID),
])
def test_plan_refuses(L, over, code):
    assert plan(L, **over) == code


def append(L, k=1, ks=256, v=2, vs=256, kc=3, vc=4, stride=2 * 64 * 128, sk=5, sv=6, code=0, blocks=7, bs=64, slots=8, T=9, HKV=2,
           D=128):
    return L.kda_cache_append(ptr(k), ks, ptr(v), vs, ptr(kc), ptr(vc), stride, ptr(sk), ptr(sv), code, blocks, bs,
                              ptr(slots), T, HKV, D, None)


CACHE = [(dict(code=2), UNSUPPORTED), (dict(blocks=0), INVALID), (dict(bs=96), UNSUPPORTED), (dict(bs=-1), INVALID),
         (dict(HKV=0), INVALID), (dict(D=80), UNSUPPORTED), (dict(stride=64 * 128), INVALID),
         (dict(stride=2 * 64 * 128 + 8), MISALIGNED), (dict(blocks=1 << 26), UNSUPPORTED), (dict(kc=None), INVALID),
         (dict(vc=None), INVALID), (dict(sk=None), INVALID), (dict(kc=3 + 8 * BYTE), MISALIGNED),
         (dict(sv=6 + 2 * BYTE), MISALIGNED)]


@pytest.mark.parametrize("over,code", CACHE + [
    (dict(T=-1), INVALID), (dict(k=None), INVALID), (dict(ks=128), INVALID), (dict(vs=258), MISALIGNED),
    (dict(slots=None), INVALID), (dict(kc=4), INVALID), (dict(vc=3 + 64 * 128 * BYTE), INVALID),
    (dict(kc=1), INVALID), (dict(sk=6), INVALID), (dict(sk=3), INVALID), (dict(sv=8), INVALID),
    (dict(stride=4 * 64 * 128, vc=3 + 64 * 128 * BYTE), INVALID),   # interleaved, but the blocks overlap
])
def test_append_refuses(L, over, code):
    assert append(L, **over) == code


def test_append_of_nothing_is_a_no_op(L):
    assert append(L, T=0, k=None, slots=None) == 0


def decode(L, q=1, qs=None, kc=3, vc=4, stride=2 * 64 * 128, sk=5, sv=6, code=0, blocks=7, bs=64, table=7, ts=3, width=3, lens=8,
           B=5, H=4, HKV=2, D=128, scale=0.1, o=9, lse=10, ws=11, nbytes=None):
    nbytes = L.kda_attention_decode_workspace_size(B, H, HKV, D, width, bs) if nbytes is None else nbytes
    return L.kda_attention_decode(ptr(q), H * D if qs is None else qs, ptr(kc), ptr(vc), stride, ptr(sk), ptr(sv), code,
                                  blocks, bs, ptr(table), ts, width, ptr(lens), B, H, HKV, D, scale, ptr(o), ptr(lse),
                                  ptr(ws), nbytes, None)


@pytest.mark.parametrize("over,code", CACHE + [
    (dict(B=-1), INVALID), (dict(H=3), INVALID), (dict(width=0), INVALID), (dict(ts=2), INVALID), (dict(scale=0.0), INVALID),
    (dict(q=None), INVALID), (dict(qs=256), INVALID), (dict(qs=4 * 128 + 4), MISALIGNED), (dict(table=None), INVALID),
    (dict(lens=None), INVALID), (dict(o=None), INVALID), (dict(lse=None), INVALID), (dict(ws=None), WORKSPACE),
    (dict(nbytes=16), WORKSPACE), (dict(ws=11 + 8 * BYTE), MISALIGNED), (dict(o=1), INVALID), (dict(lse=3), INVALID),
    (dict(ws=4), INVALID), (dict(o=9, lse=9), INVALID), (dict(B=1 << 30), UNSUPPORTED),
])
def test_decode_refuses(L, over, code):
    assert decode(L, **over) == code


def test_decode_of_no_rows_is_a_no_op(L):
    assert decode(L, B=0, q=None, ws=None) == 0


def test_decode_workspace_size(L):
    f = L.kda_attention_decode_workspace_size
    one = f(1, 8, 2, 128, 1, 64)   # one tile a unit: two CTAs
    assert one >= 2 * 2 * 8 * (128 + 2) * 4
    assert f(1 << 12, 64, 8, 128, 1 << 20, 128) == f(1 << 13, 64, 8, 128, 1 << 20, 128)  # the CTAs are bounded
    assert f(1, 8, 3, 128, 1, 64) == f(1, 8, 2, 96, 1, 64) == f(1, 8, 2, 128, 0, 64) == f(1, 8, 2, 128, 1, 63) == 0


# ------------------------------------------------------------------------------------------------ the binding
BF, I32 = torch.bfloat16, torch.int32


def z(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype)


@pytest.mark.parametrize("q,k,v,cu,cu_k,msg", [
    (z(1, 8, 4), z(1, 8, 2, 64), z(1, 8, 2, 64), None, None, "q must be"),
    (z(1, 8, 4, 64), z(1, 8, 2, 128), z(1, 8, 2, 128), None, None, "q must be"),
    (z(2, 8, 4, 64), z(1, 8, 2, 64), z(1, 8, 2, 64), None, None, "q must be"),
    (z(1, 8, 4, 64), z(1, 8, 2, 64), z(1, 9, 2, 64), None, None, "q must be"),
    (z(1, 8, 4, 64), z(1, 8, 2, 64), z(1, 8, 2, 64), None, z(2, dtype=I32), "needs cu_seqlens"),
    (z(1, 8, 4, 64), z(1, 8, 2, 64), z(1, 8, 2, 64), z(1, dtype=I32), None, "at least 2"),
    (z(1, 8, 4, 64), z(1, 9, 2, 64), z(1, 9, 2, 64), z(3, dtype=I32), None, "need cu_seqlens_k"),
    (z(1, 8, 4, 64), z(1, 9, 2, 64), z(1, 9, 2, 64), z(3, dtype=I32), z(2, dtype=I32), "must hold 3"),
    (z(1, 8, 4, 64), z(1, 8, 2, 64), z(1, 8, 2, 64), z(3, dtype=torch.int64), None, "torch.int32"),
    (z(1, 8, 4, 64, dtype=torch.float16), z(1, 8, 2, 64), z(1, 8, 2, 64), None, None, "q must be torch.bfloat16"),
    (z(1, 8, 4, 64), z(1, 8, 2, 64), z(1, 8, 2, 64, dtype=torch.float32), None, None, "v must be torch.bfloat16"),
    (z(1, 8, 4, 64), z(1, 8, 2, 64), z(1, 8, 2, 64), None, None, "must be a CUDA tensor"),
])
def test_binding_refuses_prompts(q, k, v, cu, cu_k, msg):
    with pytest.raises(ValueError, match=msg):
        kda.attention_forward(q, k, v, cu, cu_k)
    with pytest.raises(ValueError, match=msg):
        kda.attention_backward(q, k, v, z(*q.shape), z(1, dtype=torch.float32).expand(q.shape[0], q.shape[2] if q.dim() > 2
                               else 1, q.shape[1]).contiguous(), z(*q.shape), cu, cu_k)


def test_binding_reads_row_strides():
    shape = lambda t: (t.shape, t.stride())  # noqa: E731
    qkv = z(2, 10, 8 * 64)
    q = qkv[..., :4 * 64].view(2, 10, 4, 64)
    assert kda._row_stride("q", *shape(q)) == 512
    assert kda._row_stride("q", *shape(q[0])) == 512
    assert kda._row_stride("q", *shape(z(3, 1, 4, 64))) == 256 and kda._row_stride("q", *shape(z(1, 1, 4, 64))) == 256
    assert kda._row_stride("q", *shape(q[:, :1])) == 5120
    with pytest.raises(ValueError, match="evenly spaced"):
        kda._row_stride("q", *shape(q[:, :5]))
    with pytest.raises(ValueError, match="compact rows"):
        kda._row_stride("q", *shape(z(2, 4, 10, 64).transpose(1, 2)))
    with pytest.raises(ValueError, match="compact rows"):
        kda._row_stride("q", *shape(z(2, 10, 4, 128)[..., ::2]))


def test_binding_refuses_caches():
    f8 = torch.float8_e4m3fn
    kc, s = torch.zeros(4, 2, 16, 64, dtype=f8), z(4, 2, dtype=torch.float32)
    k, slots = z(3, 2, 64), z(3, dtype=I32)
    bad = [
        ((z(3, 2, 64, 1), k, kc, kc, s, s, slots), "k and v must be"),
        ((k, z(2, 2, 64), kc, kc, s, s, slots), "k and v must be"),
        ((k, k, kc[0], kc[0], s, s, slots), "k_cache and v_cache must be"),
        ((k, k, kc, kc[:3], s, s, slots), "k_cache and v_cache must be"),
        ((k, k, kc.float(), kc.float(), s, s, slots), "float8_e4m3fn or torch.int8"),
        ((k, k, kc, kc.view(torch.int8), s, s, slots), "v_cache must be"),
        ((k, k, kc, kc, s[:3], s, slots), "k_scale must hold"),
        ((k, k, kc, kc, s, s.double(), slots), "v_scale must be"),
        ((k, k, kc, kc, s, s, slots[:2]), "slot_map must hold"),
        ((k, k, kc, kc, s, s, slots.long()), "slot_map must be"),
        ((k, k, kc, kc, s, s, slots), "must be a CUDA tensor"),
    ]
    for args, msg in bad:
        with pytest.raises(ValueError, match=msg):
            kda.cache_append(*args)
    q, table, lens = z(3, 4, 64), z(3, 5, dtype=I32), z(3, dtype=I32)
    for args, msg in [((q[0], kc, kc, s, s, table, lens), "q must be"), ((q, kc, kc, s, s, table[:2], lens), "q must be"),
                      ((q, kc, kc, s, s, table, lens[:2]), "seq_lens must hold"),
                      ((q, kc, kc, s, s, table.long(), lens), "block_table must be"),
                      ((q.float(), kc, kc, s, s, table, lens), "q must be torch.bfloat16"),
                      ((q, kc, kc, s, s, table, lens), "must be a CUDA tensor")]:
        with pytest.raises(ValueError, match=msg):
            kda.attention_decode(*args)
    for args, msg in [((lens, lens, table[:2], slots, 16, 9), "block_table must be"),
                      ((lens, lens[:2], table, slots, 16, 9), "new_lens must hold"),
                      ((lens, lens, table, slots.long(), 16, 9), "free_blocks must be"),
                      ((lens, lens, table, slots, 16, -1), "num_tokens"),
                      ((lens, lens, table, slots, 16, 9), "must be a CUDA tensor")]:
        with pytest.raises(ValueError, match=msg):
            kda.cache_plan(*args)


def test_a_stream_of_another_device_is_refused():
    class Stream:
        device = torch.device("cuda", 1)

    q = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16)
    n = torch.zeros(2, dtype=torch.int32)
    for call in (lambda s: kda.attention_forward(q, q, q, stream=s),
                 lambda s: kda.attention_backward(q, q, q, q, q, q, stream=s),
                 lambda s: kda.cache_plan(n, n, n[:, None], n, 16, 4, stream=s),
                 lambda s: kda.cache_append(q[0], q[0], q, q, n, n, n, stream=s),
                 lambda s: kda.attention_decode(q[0], q, q, n, n, n[:, None], n, stream=s)):
        with pytest.raises(ValueError, match="stream is on"):
            call(Stream())
