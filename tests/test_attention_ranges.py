"""What the softmax-attention entry points refuse at the ends of their ranges, on the host (no GPU)."""
import pytest
import torch

import kda_gated_delta_prefill_b200 as kda
from tests.test_attention_refusals import L, UNSUPPORTED, plan  # noqa: F401 (L is a fixture)


def test_plan_refuses_slot_maps_near_2_31(L):  # noqa: F811
    for tokens in (2 ** 31 - 2 ** 20, 2 ** 31 - 1):
        assert plan(L, tokens=tokens) == UNSUPPORTED
    n = torch.zeros(2, dtype=torch.int32)
    for tokens in (2 ** 31, 2 ** 32 + 5):  # (an int would drop the upper bits)
        with pytest.raises(ValueError, match="num_tokens must be below"):
            kda.cache_plan(n, n, n[:, None], n, 16, tokens)
