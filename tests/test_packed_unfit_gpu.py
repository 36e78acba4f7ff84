"""Lengths that do not fit the tensors: outputs that the call itself allocates hold no stray memory."""
import math

import pytest
import torch

import flashattention_backward_preprocess_gb300 as fa
from tests.test_packed_gpu import DT, _cu, _paged, _rand

pytestmark = pytest.mark.gpu
BAD = [[0, 15, 10], [-1, 5, 20], [0, 10, 21], [0, 10, 2 ** 31 - 1], [3, 2, 20]]


def _stale(*shapes_types):
    """Leaves 7s in the blocks that the allocator hands out next."""
    for _ in range(4):
        for shape, dt in shapes_types:
            x = [torch.full(shape, 7, dtype=dt, device="cuda") for _ in range(3)]
            del x


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [2, 1200])  # planned by every CTA, and by one block
def test_forward_rows_are_set(dtype, N):
    dt, T = DT[dtype], 20
    Q, K, V = (_rand(i, (T, 2, 64), dt) for i in range(3))
    good = torch.cat([_cu([10, 10]), torch.full((N - 2,), 20, dtype=torch.int32, device="cuda")])
    for cu in BAD:
        bad = good.clone()
        bad[:3] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        for q, k in ((bad, good), (good, bad)):
            _stale(((T, 2, 64), dt), ((2, T), torch.float32))
            O, LSE = fa.fa_varlen_fwd(Q, K, V, q, k)
            torch.cuda.synchronize()
            with pytest.raises(fa.FaError, match="sequence lengths"):
                fa.fa_check_device()
            assert (O == 0).all() and (LSE == -math.inf).all(), cu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradient_rows_are_set(dtype):
    dt, T = DT[dtype], 20
    dO, Q, K, V = (_rand(i, (T, 2, 64), dt) for i in range(4))
    good = _cu([10, 10])
    O, LSE = fa.fa_varlen_fwd(Q, K, V, good, good)
    for cu in BAD:
        bad = torch.tensor(cu, dtype=torch.int32, device="cuda")
        for q, k in ((bad, good), (good, bad)):
            _stale(((T, 2, 64), dt))
            grads = fa.fa_varlen_bwd(dO, Q, K, V, O, LSE, q, k)
            torch.cuda.synchronize()
            with pytest.raises(fa.FaError, match="sequence lengths"):
                fa.fa_check_device()
            assert all((x == 0).all() for x in grads), cu


@pytest.mark.parametrize("dtype,page", [("bf16", 16), ("bf16", 5)])
def test_paged_rows_are_set(dtype, page):
    dt, new, total = DT[dtype], [1, 5], [40, 33]
    Q, K, V, table, lens = _paged(2, new, total, 2, 1, 64, page, dt)
    for cu, n in (([0, 1, 7], lens), ([0, 1, 6], torch.tensor([-1, 33], dtype=torch.int32, device="cuda"))):
        _stale(((6, 2, 64), dt), ((2, 6), torch.float32))
        O, LSE = fa.fa_paged_fwd(Q, K, V, table, torch.tensor(cu, dtype=torch.int32, device="cuda"), n)
        torch.cuda.synchronize()
        with pytest.raises(fa.FaError, match="sequence lengths"):
            fa.fa_check_device()
        assert (O == 0).all() and (LSE == -math.inf).all()
