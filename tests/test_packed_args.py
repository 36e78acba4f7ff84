"""Whole numbers past 32 bits are refused (no GPU needed)."""
import pytest
import torch

import flashattention_backward_preprocess_gb300 as fa
from flashattention_backward_preprocess_gb300 import build, packed


@pytest.fixture
def calls(monkeypatch):
    """The torch calls with host tensors: the device check is taken out and the library's calls recorded."""
    build.build()
    seen = []

    class Lib:
        def __getattr__(self, name):
            f = getattr(fa.load_library(), name)

            def call(*a):
                if "workspace_bytes" in name:
                    return f(*a)
                seen.append([c(x).value for c, x in zip(f.argtypes, a) if isinstance(x, int)])  # as C sees them
                return 0
            return call

    monkeypatch.setattr(packed, "load_library", lambda: Lib())
    monkeypatch.setattr(packed, "_device", lambda first, *rest: first.device)
    monkeypatch.setattr(packed, "_call", lambda dev, stream, body: body(0))
    return seen


q, k = torch.zeros(5, 4, 64, dtype=torch.bfloat16), torch.zeros(5, 2, 64, dtype=torch.bfloat16)
cu = torch.tensor([0, 5], dtype=torch.int32)
cache, table, lens = torch.zeros(3, 16, 2, 64, dtype=torch.bfloat16), torch.zeros(1, 2, dtype=torch.int32), torch.tensor([5], dtype=torch.int32)
WINDOWED = {
    "fwd": lambda w: fa.fa_varlen_fwd(q, k, k, cu, cu, window_size=w),
    "bwd": lambda w: fa.fa_varlen_bwd(q, q, k, k, q, torch.zeros(4, 5), cu, cu, window_size=w),
    "paged": lambda w: fa.fa_paged_fwd(q, cache, cache, table, cu, lens, window_size=w),
}


@pytest.mark.parametrize("which", list(WINDOWED))
def test_windows_past_32_bits(calls, which):
    """A window is never another window modulo 2^32."""
    WINDOWED[which](7)
    assert 7 in calls[-1]
    for w in (2 ** 31, 2 ** 32 + 7, 2 ** 32, -2 ** 32 + 7):
        n = len(calls)
        with pytest.raises(fa.FaError, match="window_size"):
            WINDOWED[which](w)
        assert len(calls) == n


def test_page_sizes_past_32_bits(calls):
    for page in (2 ** 32 + 16, 2 ** 31, -2 ** 32 + 16):
        with pytest.raises(fa.FaError, match="page_size"):
            fa.fa_page_slots(lens, cu, table, lens, lens, page, 5)
    with pytest.raises(fa.FaError, match="tokens"):
        fa.fa_page_slots(lens, cu, table, lens, lens, 16, 2 ** 32 + 5)
    assert not calls
