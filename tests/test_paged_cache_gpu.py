"""The paged cache end to end: prompts in chunks, single tokens, releases and reuse of pages, each
step against plain 64-bit attention over everything the request has sent so far."""
import math

import pytest
import torch

import flashattention_backward_preprocess_gb300 as fa
from tests import packed_ref as ref
from tests.test_packed_gpu import DT, _cu

pytestmark = pytest.mark.gpu


class _Run:
    def __init__(self, rows, H, H_kv, d, page, dtype, pages, window=0, layers=2):
        self.H, self.H_kv, self.d, self.dt, self.window, self.layers = H, H_kv, d, DT[dtype], window, layers
        self.cache = fa.PagedKVCache(layers, pages, page, H_kv, d, rows, -(-600 // page), dtype=self.dt)
        self.kv = [[[], []] for _ in range(rows)]  # per row: K, V pieces [layers, n, H_kv, d]
        self.gen = torch.Generator().manual_seed(7)

    def rand(self, *shape):
        return torch.randn(*shape, generator=self.gen).to(self.dt)

    def step(self, new, pad=0):
        T = sum(new) + pad
        cu = _cu(new)
        pos = self.cache.begin(cu, T)
        held = [sum(p.shape[1] for p in kv[0]) for kv in self.kv]
        want = [held[r] + i for r, n in enumerate(new) for i in range(n)] + [-1] * pad
        assert pos.tolist() == want
        Q, K, V = self.rand(self.layers, T, self.H, self.d), self.rand(self.layers, T, self.H_kv, self.d), self.rand(self.layers, T, self.H_kv, self.d)
        a = 0
        for r, n in enumerate(new):
            self.kv[r][0].append(K[:, a:a + n])
            self.kv[r][1].append(V[:, a:a + n])
            a += n
        for layer in range(self.layers):
            O, LSE = self.cache.attend(layer, Q[layer].cuda(), K[layer].cuda(), V[layer].cuda(), window_size=self.window)
            torch.cuda.synchronize()
            fa.fa_check_device()
            a = 0
            for r, n in enumerate(new):
                k, v = (torch.cat(x, 1)[layer].double() for x in self.kv[r])
                o, lse, mag, e = ref.attend(Q[layer, a:a + n].double(), k, v, True, self.window, 1 / math.sqrt(self.d))
                ref.check(f"layer {layer} row {r}", O[a:a + n], o, mag, e, self.dt)
                ref.check_lse(LSE[:, a:a + n], lse, e)
                a += n
            assert (O[a:] == 0).all() and (LSE[:, a:] == -math.inf).all()


@pytest.mark.parametrize("dtype,H,H_kv,d,page,window", [("bf16", 8, 2, 128, 16, 0), ("f16", 4, 4, 64, 32, 40), ("f32", 4, 1, 32, 5, 0)])
def test_chunks_then_tokens(dtype, H, H_kv, d, page, window):
    run = _Run(3, H, H_kv, d, page, dtype, pages=-(-600 // page) * 3, window=window)
    run.step([70, 0, 5], pad=3)
    run.step([1, 130, 1])
    run.step([64, 33, 0])
    for _ in range(3):
        run.step([1, 1, 1], pad=5)
    assert run.cache.lens.tolist() == [138, 166, 9]


def test_release_and_reuse():
    run = _Run(3, 4, 2, 64, 16, "bf16", pages=24, layers=1)
    run.step([100, 60, 33])
    run.cache.release(1)
    run.kv[1] = [[], []]
    run.step([1, 200, 1])  # takes the pages given back
    used = run.cache.block_table[run.cache.block_table >= 0].tolist()
    assert len(used) == len(set(used)) == 7 + 13 + 3
    run.cache.release(0)
    run.kv[0] = [[], []]
    run.step([40, 0, 1])
    # a step that needs more pages than there are is reported
    run.cache.begin(_cu([300, 0, 0]), 300)
    torch.cuda.synchronize()
    with pytest.raises(fa.FaError, match="free pages"):
        fa.fa_check_device()
    # afterwards a release gives back what the rows really hold
    free = 24 - int((run.cache.block_table >= 0).sum())
    run.cache.release(0)
    assert free == 0 and run.cache.free_start.item() == int((run.cache.block_table >= 0).sum())
    assert sorted(run.cache.free_pages[run.cache.free_start.item():].tolist() +
                  run.cache.block_table[run.cache.block_table >= 0].tolist()) == list(range(24))


def test_step_is_capturable():
    """A decode step captured once and replayed with the lengths it finds."""
    rows, H, H_kv, d, page = 4, 8, 2, 64, 16
    cache = fa.PagedKVCache(1, 64, page, H_kv, d, rows, 8)
    eager = fa.PagedKVCache(1, 64, page, H_kv, d, rows, 8)
    gen = torch.Generator().manual_seed(1)
    r = lambda h, n=rows: torch.randn(n, h, d, generator=gen).bfloat16().cuda()
    cu = _cu([1] * rows)
    first = _cu([20, 1, 16, 7])
    K0, V0, Q0 = r(H_kv, 44), r(H_kv, 44), r(H, 44)
    for c in (cache, eager):
        c.begin(first, 44)
        c.attend(0, Q0, K0, V0)
    lens, start = cache.lens.clone(), cache.free_start.clone()
    Q, K, V = r(H), r(H_kv), r(H_kv)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cache.lens, cache.free_start = lens, start
        cache.begin(cu, rows)
        O, LSE = cache.attend(0, Q, K, V)
        lens.copy_(cache.lens)
        start.copy_(cache.free_start)
    for _ in range(20):
        for t, h in ((Q, H), (K, H_kv), (V, H_kv)):
            t.copy_(r(h))
        g.replay()
        eager.begin(cu, rows)
        want = eager.attend(0, Q, K, V)
        torch.cuda.synchronize()
        fa.fa_check_device()
        assert torch.equal(O, want[0]) and torch.equal(LSE, want[1])
    assert lens.tolist() == [40, 21, 36, 27]


def test_replays_of_a_step_go_on():
    """Nothing but the step is captured; eager steps and a release come between replays."""
    rows, H, H_kv, d, page = 3, 4, 2, 64, 8
    a, b = (fa.PagedKVCache(1, 40, page, H_kv, d, rows, 8) for _ in range(2))
    gen = torch.Generator().manual_seed(3)
    r = lambda h: torch.randn(rows, h, d, generator=gen).bfloat16().cuda()
    cu = _cu([1] * rows)
    Q, K, V = r(H), r(H_kv), r(H_kv)
    for c in (a, b):
        c.begin(cu, rows)
        c.attend(0, Q, K, V)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.begin(cu, rows)
        O, LSE = a.attend(0, Q, K, V)
    for i in range(24):
        for t, h in ((Q, H), (K, H_kv), (V, H_kv)):
            t.copy_(r(h))
        if i % 7 == 3:
            got = (a.begin(cu, rows), a.attend(0, Q, K, V))[1]
        else:
            g.replay()
            got = O, LSE
        b.begin(cu, rows)
        want = b.attend(0, Q, K, V)
        torch.cuda.synchronize()
        fa.fa_check_device()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), i
        if i == 12:
            a.release(1)
            b.release(1)
        assert a.lens.tolist() == b.lens.tolist() and a.free_start.tolist() == b.free_start.tolist()
    assert a.lens.tolist() == [25, 11, 25]
