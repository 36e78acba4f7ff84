"""Scratch of the packed backward: it follows the tokens, not the number of sequences (no GPU needed)."""
import pytest

import flashattention_backward_preprocess_gb300 as fa
from flashattention_backward_preprocess_gb300 import build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return fa.load_library()


@pytest.mark.parametrize("dtype", [fa.FA_BF16, fa.FA_F32])
@pytest.mark.parametrize("N,T,H,H_kv,d", [(4096, 65536, 32, 8, 128), (4096, 16384, 32, 8, 128), (1024, 32768, 32, 8, 128),
                                          (40960, 655360, 32, 8, 128), (5000, 40000, 16, 16, 64), (3000, 9000, 8, 2, 256)])
def test_short_sequences_do_not_multiply_the_scratch(lib, dtype, N, T, H, H_kv, d):
    """Beside the fp32 accumulator of T rows: D, the LSE copy and the order's counters of whole 128-row tiles
    (T / 128 + N of them at most), a few hundred bytes of plan per sequence and tile, the parts of cut tiles."""
    got = lib.fa_varlen_workspace_bytes(N, T, T, H, H_kv, d, dtype, 1)
    tiles = T // 128 + N
    want = T * H * d * 4 + tiles * H * (128 * 8 + 4) + (N + tiles) * 1024
    parts = 2 * (2 * 160 // H_kv + 1) * H_kv * 2 * 128 * d * 4  # 160: more than the SMs there are
    assert T * H * d * 4 < got <= want + parts + 65536
