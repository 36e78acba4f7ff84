"""PagedKVCache.accept with a request whose path or count does not fit: it keeps what it has, the others are accepted."""
import pytest
import torch

import flashattention_backward_preprocess_gb300 as fa
from tests.test_draft_tree_gpu import I32
from tests.test_packed_gpu import _cu, _rand
from tests.test_paged_q8_gpu import _errors

pytestmark = pytest.mark.gpu
PAGE, NEW, HELD = 8, [12, 20, 9], [5, 30, 16]
PATHS = [[0, 4, 11], [1, 2, 9, 19], [0, 8]]


def _step(quantised, paths, counts, entries=None):
    """A cache of three requests after a drafted step, its rows before accept(), and the error reported."""
    H, H_kv, d, layers = 4, 2, 64, 2
    cache = fa.PagedKVCache(layers, 40, PAGE, H_kv, d, 3, 12, quantised=quantised)
    for n, (new, parents) in enumerate(((HELD, None), (NEW, [i - 1 for m in NEW for i in range(m)]))):
        T = sum(new)
        cache.begin(_cu(new), T, parents=None if parents is None else torch.tensor(parents, **I32))
        for layer in range(layers):
            x = [_rand(10 * n + layer, (T, h, d), torch.bfloat16) for h in (H, H_kv, H_kv)]
            cache.attend(layer, *x)
    before = _rows(cache, [a + b for a, b in zip(HELD, NEW)])
    path = sum((p + [0] * (m - len(p)) for p, m in zip(paths, NEW)), [])
    cache.accept(torch.tensor(path[:entries], **I32), torch.tensor(counts, **I32))
    return cache, before, _errors()


def _rows(cache, lens):
    """Of each request: its first lens[n] rows of every layer's tensors."""
    out = []
    for n, m in enumerate(lens):
        j = torch.arange(m, device="cuda")
        pg, row = cache.block_table[n].long()[j // PAGE], j % PAGE
        ts = [t.view(torch.uint8)[pg, row] if t.dtype == torch.float8_e4m3fn else t[pg, row] for t in cache.K + cache.V]
        out.append(ts + [t[pg, :, row] for t in (cache.K_exp or []) + (cache.V_exp or [])])
    return out


@pytest.mark.parametrize("quantised", [False, True])
@pytest.mark.parametrize("path,count,entries", [
    (PATHS[1], 21, None), (PATHS[1], -1, None), ([1, 2, 2, 19], 4, None), ([1, 9, 2, 19], 4, None), ([1, 2, 9, 20], 4, None),
    ([-1, 2, 9, 19], 4, None), (PATHS[1], 4, 31),
])
def test_one_bad_request(quantised, path, count, entries):
    """entries: the path's tensor ends inside the rows of the last two requests."""
    good, before, said = _step(quantised, PATHS, [3, 4, 2])
    assert said == ""
    assert good.lens.tolist() == [8, 34, 18]
    left = [1] if entries is None else [1, 2]
    cache, before, said = _step(quantised, [PATHS[0], path, PATHS[2]], [3, count, 2], entries)
    assert "path" in said
    lens = [HELD[n] + (NEW[n] if n in left else [3, 4, 2][n]) for n in range(3)]
    assert cache.lens.tolist() == lens
    want = _rows(good, good.lens.tolist())
    for n, rows in enumerate(_rows(cache, lens)):
        for got, w in zip(rows, before[n] if n in left else want[n]):
            assert torch.equal(got, w), n
    used = [int(x) for row, m in zip(cache.block_table, lens) for x in row[: -(-m // PAGE)]]
    assert sorted(used + cache.free_pages[cache.free_start.item():].tolist()) == list(range(40))


def test_trim_judges_a_path_as_keep_does():
    """count 0, a path behind it, equal lengths, no new tokens; running the call again changes nothing."""
    cu, lens = _cu([8, 3, 0, 5]), torch.tensor([10, 12, 7, 2], **I32)  # the last has more new tokens than it holds
    table = torch.arange(12, **I32).view(4, 3)
    path = torch.tensor([0, 3, 99, 0, 0, 0, 0, 0] + [-5, 0, 0] + [0, 1, 2, 3, 4], **I32)
    count = torch.tensor([2, 0, 0, 1], **I32)
    free, start = torch.arange(100, 120, **I32), torch.tensor([10], **I32)
    for _ in range(2):
        out, nxt = fa.fa_page_trim(count, cu, lens, table, free, start, 4, path=path)
        assert "path" in _errors()
        assert out.tolist() == [4, 9, 7, 2]
        assert nxt.tolist() == [8] and free[8:10].tolist() == [1, 2]
    # offsets of one request that make no sense
    out, nxt = fa.fa_page_trim(count, torch.tensor([0, 8, 7, 11, 40], **I32), lens, table, free, start, 4, path=path)
    assert "path" in _errors()
    assert out.tolist() == [4, 12, 3, 2]


@pytest.mark.parametrize("parents,words", [([-1, 0, 1], 1), ([-1, 0, 1, 2, 3], 1), ([-1, 0, 1, 2], 1025)])
def test_a_refused_begin_changes_nothing(parents, words):
    """The step before it can go on: same tables, slots and results."""
    cache = fa.PagedKVCache(1, 8, PAGE, 2, 64, 1, 6)
    cu, x = _cu([7]), [_rand(i, (7, h, 64), torch.bfloat16) for i, h in enumerate((4, 2, 2))]
    cache.begin(cu, 7)
    want = cache.attend(0, *x)
    held = [t.clone() for t in (cache.block_table, cache.lens, cache.free_start, cache.slots, cache.positions)]
    with pytest.raises(fa.FaError):
        cache.begin(_cu([4]), 4, parents=torch.tensor(parents, **I32), words=words)
    for a, b in zip(held, (cache.block_table, cache.lens, cache.free_start, cache.slots, cache.positions)):
        assert torch.equal(a, b)
    assert cache.tree is None and cache.cu_q is cu
    for a, b in zip(cache.attend(0, *x), want):
        assert torch.equal(a, b)
    assert _errors() == ""
