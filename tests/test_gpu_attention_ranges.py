"""Causal softmax attention over whole prompts on the GPU: batches at the ends of what the calls allow.  Formula and
tolerances as in test_gpu_attention.py."""
import math

import pytest
import torch

import kda_gated_delta_prefill_b200 as kda
from tests.test_gpu_attention import cu_of, heads

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
