"""4-bit matrix-vector products whose rows of x do not fit a block at once, so
that the call streams the weights several times, on matrices with several sets
of tiles per block.  Bounds: those of test_gpu_matvec."""
import pytest
import torch

from tests.test_gpu_matvec import DT, FMTS, activations, call, check, weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K,xt", [(16, 5003, 8192, "f32"), (16, 4999, 8192, "bf16"), (13, 2700, 16384, "f16"),
                                      (9, 6007, 4096, "f32"), (5, 2501, 12288, "f32")])
def test_several_passes_and_sets(lib, fmt, M, N, K, xt):
    wt, w, mag = weights(fmt, M + K, N, K)
    x = activations(N, M, K, xt)
    room = torch.full((M + 1, N + 3), 7.0, device="cuda")
    out = room[:M, 1:N + 1]
    call(lib, fmt, x, wt, out)
    check(out.contiguous(), x, w, mag)
    keep = torch.ones_like(room, dtype=torch.bool)
    keep[:M, 1:N + 1] = False
    assert (room[keep] == 7.0).all()


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_several_passes_with_ragged_scales(lib, fmt):
    """K a multiple of 32 only: scale rows at any byte, over several copies and passes."""
    M, N, K = 16, 3001, 8224
    wt, w, mag = weights(fmt, 17, N, K)
    x = activations(17, M, K, "f32")
    out = torch.full((M, N), float("nan"), device="cuda")
    call(lib, fmt, x, wt, out)
    check(out, x, w, mag)
    assert DT["f32"] == out.dtype
