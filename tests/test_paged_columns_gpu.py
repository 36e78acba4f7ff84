"""A request that outgrows its row of the table: its tokens behind the last column are not cached and are
reported, no page is lost, and the other requests go on as if it were not there."""
import pytest
import torch

import flashattention_backward_preprocess_gb300 as fa
from tests import packed_ref as ref
from tests.test_packed_gpu import _cu

pytestmark = pytest.mark.gpu
I32 = dict(dtype=torch.int32, device="cuda")


def _errors():
    torch.cuda.synchronize()
    try:
        fa.fa_check_device()
    except fa.FaError as e:
        assert e.status == 1
        return str(e)
    return ""


def test_pages_that_cannot_be_entered_stay_free():
    """The pages behind the table's last column are not taken from the list, so the next request has them."""
    table = torch.full((4, 3), -1, **I32)
    table[1, :2] = torch.tensor([50, 51], **I32)
    ctx, new, page = [0, 30, 0, 0], [5, 40, 17, 1], 16  # request 1 holds 30 of 48 tokens and brings 40
    free = torch.arange(20, **I32)
    slots, pos, lens, nxt = fa.fa_page_slots(torch.tensor(ctx, **I32), _cu(new), table, free, torch.zeros(1, **I32), page, sum(new))
    assert "columns" in _errors()
    assert table.tolist() == [[0, -1, -1], [50, 51, 1], [2, 3, -1], [4, -1, -1]]
    assert nxt.tolist() == [5]
    want = list(range(5)) + [51 * 16 + 14, 51 * 16 + 15] + [16 + i for i in range(16)] + [-1] * 22
    want += [32 + i for i in range(16)] + [48] + [64]
    assert slots.tolist() == want
    assert pos.tolist() == [c + i for c, m in zip(ctx, new) for i in range(m)]


@pytest.mark.parametrize("dtype,page", [(torch.bfloat16, 16), (torch.bfloat16, 6), (torch.float32, 16)])
def test_other_rows_go_on(dtype, page):
    rows, H, H_kv, d, cols = 3, 4, 2, 64, 4
    cap = cols * page
    cache = fa.PagedKVCache(1, 12, page, H_kv, d, rows, cols, dtype=dtype)
    gen = torch.Generator().manual_seed(4)
    kv = [[torch.zeros(0, H_kv, d, dtype=dtype)] * 2 for _ in range(rows)]

    def step(new):
        T, at = sum(new), 0
        Q, K, V = (torch.randn(T, h, d, generator=gen).to(dtype) for h in (H, H_kv, H_kv))
        cache.begin(_cu(new), T)
        O, LSE = cache.attend(0, Q.cuda(), K.cuda(), V.cuda())
        said = _errors()
        for r, n in enumerate(new):
            held = kv[r][0].shape[0]
            kv[r] = [torch.cat([old, x[at:at + n]]) for old, x in zip(kv[r], (K, V))]
            m = min(max(cap - held, 0), n)  # the new tokens that the row has room for
            k, v = (x.double() for x in kv[r])
            # the others see all that is cached
            for a, b, keys, causal in ((at, at + m, held + m, True), (at + m, at + n, cap, False)):
                if a < b:
                    o, lse, mag, e = ref.attend(Q[a:b].double(), k[:keys], v[:keys], causal, 0, d ** -0.5)
                    ref.check(f"row {r}", O[a:b], o, mag, e, dtype)
                    ref.check_lse(LSE[:, a:b], lse, e)
            at += n
        return said

    assert step([cap - 3, 7, 2]) == ""
    assert step([3, 1, 1]) == ""          # row 0 is full
    assert "columns" in step([1, 5, 1])   # and outgrows its table
    for _ in range(3):
        assert "columns" in step([1, 1, 2 * page - 1])  # row 2 outgrows it too
    assert _errors() == ""
    used = cache.block_table[cache.block_table >= 0].tolist()
    free = cache.free_pages[cache.free_start.item():].tolist()
    assert sorted(used + free) == list(range(12))
    cache.release(0)
    kv[0] = [torch.zeros(0, H_kv, d, dtype=dtype)] * 2
    used = cache.block_table[cache.block_table >= 0].tolist()
    assert sorted(used + cache.free_pages[cache.free_start.item():].tolist()) == list(range(12))
    assert step([5, 1, 0]) == ""
