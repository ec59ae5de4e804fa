"""How many blocks the few-token layer runs on a device of so many SMs, without
a GPU: it refuses devices with fewer SMs than row pairs of y, and where it runs
every block's share of the down projection lies in two row pairs at most (what
its kernel has room for)."""
import pytest

from fp8_block_scaled_pow2_b200 import moe


def row_pairs(H):
    return (H // 128 + 1) // 2


@pytest.mark.parametrize("H", [128, 256, 384, 4096, 7168, 7296, 8064, 8192])
def test_refused_with_fewer_sms_than_row_pairs(H):
    rp = row_pairs(H)
    for sms in range(1, 200):
        n = moe.moe_layer_few_blocks(4, H, 2048, 64, 6, 1, sms)
        assert (n == 0) == (sms < rp), sms
        assert n <= min(sms, 160)
    assert moe.moe_layer_few_blocks(4, H, 2048, 64, 6, 1, 148) == 148      # a whole B200


def test_refused_sizes():
    assert moe.moe_layer_few_blocks(1, 256, 128, 8, 2, 1, 148) == 1 * 3 * 1       # one row pair, two experts and the shared one
    for bad in ((17, 256, 128, 8, 2, 1, 148), (1, 8320, 128, 8, 2, 1, 148), (1, 200, 128, 8, 2, 1, 148),
                (1, 256, 128, 8, 2, 1, 0), (1, 256, 128, 8, 2, 1, -4)):
        assert moe.moe_layer_few_blocks(*bad) == 0, bad


@pytest.mark.parametrize("T,H,I,E,k,shared", [(1, 8192, 128, 8, 1, 0), (1, 8192, 2048, 256, 6, 1), (16, 7168, 2048, 384, 16, 1),
                                              (3, 384, 128, 4, 2, 1), (2, 8064, 896, 40, 3, 0)])
def test_shares_lie_in_two_row_pairs(T, H, I, E, k, shared):
    rp = row_pairs(H)
    for sms in sorted({rp, rp + 1, 33, 64, 100, 132, 148, 160}):
        grid = moe.moe_layer_few_blocks(T, H, I, E, k, shared, sms)
        assert (grid > 0) == (sms >= rp)
        for n in {1, 2, k + shared, min(E, T * k) + shared} if grid else ():
            total = n * (I // 128)                           # steps of a row pair
            Z = rp * total
            blocks = min(grid, Z)
            for c in range(blocks):
                lo, hi = Z * c // blocks, Z * (c + 1) // blocks
                assert lo < hi and (hi - 1) // total - lo // total <= 1
