"""4-bit matrix-vector products at the ends of float32's range: a result is
finite and as exact as elsewhere wherever it fits float32, whatever the other
rows of x are.

Tolerance, as for ordinary sizes: x within 2^-39 of its row's largest value
(float32: and 2^-22 of its own), at most 256 + K / 128 float32 additions a term
passes through, each off by at most 2^-23 of the magnitudes summed, one
rounding.  Besides, each addition (and the last product) is off by at most
2^-149, the step of float32's subnormals.
"""
import numpy as np
import pytest
import torch

import synth
from oracle import ffn
from oracle.formats import decode_e2m1_packed, decode_e4m3

pytestmark = pytest.mark.gpu

FMTS = ("mxfp4", "nvfp4", "int4")


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def weights(fmt, seed, N, K, size):
    """Weights of about 2^size: (device arrays of the call, float64 [N, K])."""
    nib = synth.random_bytes(seed, 1, (N, K // 2))
    if fmt == "mxfp4":
        s = np.clip(synth.random_bytes(seed, 2, (N, K // 32), 0, 4).astype(np.int64) + size + 125, 0, 254).astype(np.uint8)
        return (dev(nib), dev(s)), ffn.dequant_mxfp4(nib, s)
    if fmt == "nvfp4":
        s = synth.random_e4m3(seed, 2, (N, K // 16)) & 0x7F
        g = np.array([2.0 ** (size - 8) * 1.1], np.float32)
        w = decode_e2m1_packed(nib) * np.repeat(decode_e4m3(s), 16, -1) * float(g[0])
        return (dev(nib), dev(s), dev(g)), w
    s = ((1 + synth.uniform(seed, 2, N * (K // 128))) * 2.0 ** size).astype(np.float32).reshape(N, K // 128)
    return (dev(nib.view(np.int8)), dev(s)), ffn.dequant_int4g128(nib, s)


def call(lib, fmt, x, wt):
    out = torch.full((x.shape[0], wt[0].shape[0]), float("nan"), device="cuda")
    {"mxfp4": lib.moe_matvec_mxfp4, "nvfp4": lib.moe_matvec_nvfp4, "int4": lib.moe_matvec_int4g128}[fmt](x, *wt, out)
    return out


def check(out, x, w):
    K = w.shape[1]
    x64, mag = x.double().cpu().numpy(), np.abs(w)
    ref = x64 @ w.T
    tol = (256 + K / 128) * (2.0 ** -23 * (np.abs(x64) @ mag.T) + 2.0 ** -149)
    tol += 2.0 ** -39 * np.abs(x64).max(-1)[:, None] * mag.sum(-1)
    if x.dtype == torch.float32:
        tol += 2.0 ** -22 * (np.abs(x64) @ mag.T)
    tol += 2.0 ** -24 * np.abs(ref)
    fits = np.abs(ref) + tol < torch.finfo(torch.float32).max
    assert fits.all()
    got = out.double().cpu().numpy()
    assert np.isfinite(got).all()
    assert (np.abs(got - ref) <= tol).all(), np.argwhere(np.abs(got - ref) > tol)[:4]


def rows(seed, K, sizes, xt):
    x = synth.normal(seed, 3, len(sizes) * K).reshape(len(sizes), K) * np.exp2(np.array(sizes, np.float64))[:, None]
    return torch.from_numpy(x.astype(np.float32)).to(xt).cuda()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("xt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("K", [256, 4096, 8192])
@pytest.mark.parametrize("sizes,weight", [
    ((0, 0), 108),                  # large weights, ordinary x: the sums of x scaled to 2^14 would pass 2^128
    ((-30, -60, -90), 112),         # and small x
    ((0, -12, -30), -118),          # small weights, beside rows of x that are smaller still
    ((60, 30, 0), -110),
    ((100, 20), -105),
    ((-110, -40, 0), 100),
    ((0, -13, -40), -127),          # the smallest scales of all
])
def test_results_within_float32(lib, fmt, xt, K, sizes, weight):
    if fmt == "int4" and weight < -110:
        weight = -110               # float32 scales: products with them stay normal
    wt, w = weights(fmt, K + weight, 37, K, weight)
    x = rows(K, K, sizes, xt)
    check(call(lib, fmt, x, wt), x, w)


def test_mxfp4_positive_weights_of_the_largest_scales(lib):
    """Sums that only grow, at the largest E8M0 scale, times small x."""
    N, K = 20, 8192
    nib = synth.random_bytes(5, 1, (N, K // 2)) & 0x77
    s = np.full((N, K // 32), 254, np.uint8)
    x = rows(5, K, (-30, -50), torch.bfloat16).abs()
    check(call(lib, "mxfp4", x, (dev(nib), dev(s))), x, ffn.dequant_mxfp4(nib, s))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("xt", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("weight", [-127, -110, 0, 60])
def test_a_row_does_not_depend_on_its_neighbours(lib, fmt, xt, weight):
    """The same bits alone and beside rows of any size (up to 8 columns of the
    products: the same cut of the work)."""
    N, K = 53, 2048
    wt, _ = weights(fmt, 3, N, K, weight)
    sizes = (0, -13, 9, -3) if xt == torch.float16 else (0, -40, 40, -10)
    x = rows(8, K, sizes, xt)
    together = call(lib, fmt, x, wt)
    for m in range(len(sizes)):
        assert torch.equal(call(lib, fmt, x[m:m + 1], wt)[0], together[m]), m
