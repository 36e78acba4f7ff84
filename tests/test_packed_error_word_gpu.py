"""fa_check_device while calls on another stream are still reporting: no report is lost."""
import pytest
import torch

import flashattention_backward_preprocess_gb300 as fa
from tests.test_packed_gpu import _cu, _rand

pytestmark = pytest.mark.gpu


def _said():
    try:
        fa.fa_check_device()
    except fa.FaError as e:
        return str(e)
    return ""


def test_no_report_is_lost():
    """One stream reports a bad slot while the check reads and clears a report of bad lengths.  The delay
    between the two is swept over the time of the check, so that the report falls on each part of it."""
    K = _rand(1, (1, 1, 64), torch.bfloat16)
    cache = torch.zeros(2, 8, 1, 64, dtype=torch.bfloat16, device="cuda")
    slot = torch.tensor([99], device="cuda")
    Q, bad = _rand(2, (4, 1, 64), torch.bfloat16), torch.tensor([0, 9], dtype=torch.int32, device="cuda")
    other = torch.cuda.Stream()
    fa.fa_varlen_fwd(Q, Q, Q, bad, _cu([4]))
    fa.fa_paged_write(K, K, slot, cache, cache, stream=other)
    torch.cuda.synchronize()
    assert "lengths" in _said() and _said() == ""
    lost = []
    for i in range(1500):
        fa.fa_varlen_fwd(Q, Q, Q, bad, _cu([4]))
        torch.cuda.current_stream().synchronize()
        with torch.cuda.stream(other):
            torch.cuda._sleep(100 * (i % 750))  # up to about 40 us
        fa.fa_paged_write(K, K, slot, cache, cache, stream=other)
        first = _said()
        torch.cuda.synchronize()
        said = first + _said()
        assert "lengths" in said
        if "page or slot" not in said:
            lost.append(i)
    assert not lost, f"{len(lost)} of 1500 reports lost"
