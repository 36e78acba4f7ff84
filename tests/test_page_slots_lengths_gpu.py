"""fa_page_slots with lengths that do not fit: nothing is handed out, what the requests hold stays as it
is, no slot of the step may be written, and the check names it."""
import pytest
import torch

import flashattention_backward_preprocess_gb300 as fa
from tests.test_packed_gpu import _cu

pytestmark = pytest.mark.gpu
I32 = dict(dtype=torch.int32, device="cuda")


def _i32(x):
    return torch.tensor(x, **I32)


@pytest.mark.parametrize("cu,ctx", [
    ([0, 5, 9, 40], [3, 17, 0]),             # past the rows of the step
    ([0, 5, 3, 9], [3, 17, 0]),              # decreasing
    ([-2, 5, 6, 9], [3, 17, 0]),             # negative
    ([0, 5, 6, 9], [3, -1, 0]),              # negative context
    ([0, 5, 6, 9], [3, 17, 2 ** 31 - 1]),    # context out of range
    ([0, 4, 8, 2 ** 31 - 1], [3, 17, 0]),
])
@pytest.mark.parametrize("front", [0, 300])  # requests before them, over a block border
def test_bad_lengths_hand_out_nothing(cu, ctx, front):
    N, page, cols, T = front + 3, 8, 8, 20 + front
    cu = _i32([i for i in range(front)] + [front + c if -1 < c < 2 ** 30 else c for c in cu])
    ctx = _i32([8] * front + ctx)
    table = torch.arange(N * cols, **I32).view(N, cols) + 1000
    before = table.clone()
    free, start = torch.arange(4000, 4400, **I32), _i32([2])
    slots, pos, lens, nxt = fa.fa_page_slots(ctx, cu, table, free, start, page, T)
    torch.cuda.synchronize()
    with pytest.raises(fa.FaError, match="sequence lengths"):
        fa.fa_check_device()
    fa.fa_check_device()
    assert (slots == -1).all() and (pos == -1).all()
    assert torch.equal(lens, ctx) and torch.equal(nxt, start) and torch.equal(table, before)


def test_cache_survives_a_bad_step():
    """Too small a token count: the step is lost, the cache is what it was, and goes on."""
    rows, H_kv, d, page = 3, 2, 64, 16
    a, b = (fa.PagedKVCache(1, 24, page, H_kv, d, rows, 8) for _ in range(2))
    gen = torch.Generator().manual_seed(2)
    r = lambda n, h: torch.randn(n, h, d, generator=gen).bfloat16().cuda()
    K, V, Q = r(60, H_kv), r(60, H_kv), r(60, 4)
    for c in (a, b):
        c.begin(_cu([30, 10, 20]), 60)
        c.attend(0, Q, K, V)
    torch.cuda.synchronize()
    fa.fa_check_device()
    held = [x.clone() for x in (a.lens, a.free_start, a.block_table, a.K[0], a.V[0])]
    a.begin(_cu([4, 1, 9]), 9)  # 14 tokens announced as 9
    a.attend(0, Q[:9], K[:9], V[:9])
    torch.cuda.synchronize()
    with pytest.raises(fa.FaError, match="sequence lengths"):
        fa.fa_check_device()
    for x, y in zip(held, (a.lens, a.free_start, a.block_table, a.K[0], a.V[0])):
        assert torch.equal(x, y)
    out = []
    for c in (a, b):
        c.begin(_cu([4, 1, 9]), 14)
        out.append(c.attend(0, Q[:14], K[:14], V[:14]))
    torch.cuda.synchronize()
    fa.fa_check_device()
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])
