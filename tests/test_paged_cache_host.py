"""PagedKVCache used out of order (no GPU needed)."""
import pytest
import torch

import flashattention_backward_preprocess_gb300 as fa


def test_attend_before_begin_is_refused():
    cache = fa.PagedKVCache(1, 4, 16, 2, 64, 1, 4, device="cpu")
    q, k = torch.zeros(5, 4, 64, dtype=torch.bfloat16), torch.zeros(5, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(fa.FaError, match="begin"):
        cache.attend(0, q, k, k)
