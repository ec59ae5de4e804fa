"""4-bit matrix-vector products against the oracle's dequantisation and a
float64 product.

Tolerances, from the arithmetic.  Element by element: the products of a 4-bit
weight with x are exact in the kernel's operands up to x's own representation
there, which is within 2^-39 of the largest |x| of its row (float32: and 2^-22
of its value, two roundings to 11 bits); sums are float32 and a term passes
through at most 256 + K / 128 additions, each off by at most 2^-23 of the
magnitudes summed (a tensor-core addition may truncate); the result is rounded
once, by at most half a step.  And over a whole float32 result (where roundings
do not hide it): a value is the sum of at most 16 + 16 partial sums one after
another (MMAs of a warp, warps; longer K add float32 sums of such), which grow
evenly to its size, so that truncations of 2^-24 on average come to
32 * 2^-24 / 2 = 2^-20 of the norm.
"""
import numpy as np
import pytest
import torch

import synth
from oracle import ffn
from oracle import repack as RP
from oracle.formats import decode_e2m1_packed, decode_e4m3

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
FMTS = ("mxfp4", "nvfp4", "int4")


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def weights(fmt, seed, N, K, e_lo=110, e_hi=130):
    """(device arrays the call takes, float64 [N, K], float64 magnitudes of the summed weights)."""
    nib = synth.random_bytes(seed, 1, (N, K // 2))
    if fmt == "mxfp4":
        s = synth.random_bytes(seed, 2, (N, K // 32), e_lo, e_hi)
        w = ffn.dequant_mxfp4(nib, s)
        return (dev(nib), dev(s)), w, np.abs(w)
    if fmt == "nvfp4":
        s = synth.random_e4m3(seed, 2, (N, K // 16)) & 0x7F
        g = np.array([3.1e-4], np.float32)
        w = decode_e2m1_packed(nib) * np.repeat(decode_e4m3(s), 16, -1) * float(g[0])
        return (dev(nib), dev(s), dev(g)), w, np.abs(w)
    s = (0.001 + synth.uniform(seed, 2, N * (K // 128))).astype(np.float32).reshape(N, K // 128)
    w = ffn.dequant_int4g128(nib, s)
    return (dev(nib.view(np.int8)), dev(s)), w, np.abs(w)


def activations(seed, M, K, xt):
    x = synth.normal(seed, 3, M * K).reshape(M, K)
    x[synth.uniform(seed, 4, M * K).reshape(M, K) < 1e-2] *= 20
    return torch.from_numpy(x.astype(np.float32)).to(DT[xt]).cuda()


def call(lib, fmt, x, wt, out, stream=None):
    fn = {"mxfp4": lib.moe_matvec_mxfp4, "nvfp4": lib.moe_matvec_nvfp4, "int4": lib.moe_matvec_int4g128}[fmt]
    fn(x, *wt, out, stream=stream)


def check(out, x, w, mag):
    K = w.shape[1]
    x64 = x.double().cpu().numpy()
    ref = x64 @ w.T
    tol = (256 + K / 128) * 2.0 ** -23 * (np.abs(x64) @ mag.T)
    tol += 2.0 ** -39 * np.abs(x64).max(-1)[:, None] * mag.sum(-1)
    if x.dtype == torch.float32:
        tol += 2.0 ** -22 * (np.abs(x64) @ mag.T)
    tol += torch.finfo(out.dtype).eps / 2 * (np.abs(ref) + tol) + torch.finfo(out.dtype).tiny
    got = out.double().cpu().numpy()
    big = np.abs(ref) > torch.finfo(out.dtype).max
    assert np.isfinite(got[~big]).all()
    err = np.abs(got - ref)
    assert (err[~big] <= tol[~big]).all(), (np.nanmax((err / tol)[~big]), np.argwhere((err > tol) & ~big)[:4])
    return np.linalg.norm(err) / max(np.linalg.norm(ref), 1e-300)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K", [(1, 1, 128), (1, 4096, 2048), (1, 2048, 4096), (2, 37, 256), (3, 1001, 1408),
                                   (5, 16, 8192), (8, 300, 640), (9, 129, 4096), (16, 1000, 1024), (16, 40, 8192),
                                   (13, 2375, 384)])
@pytest.mark.parametrize("xt,ot", [("bf16", "f32"), ("f16", "f16"), ("f32", "bf16")])
def test_matvec(lib, fmt, M, N, K, xt, ot):
    wt, w, mag = weights(fmt, M + N + K, N, K)
    x = activations(K + M, M, K, xt)
    if ot == "f16":
        x = x * 1e-3 if fmt == "mxfp4" else x
    out = torch.full((M, N), float("nan"), dtype=DT[ot], device="cuda")
    call(lib, fmt, x, wt, out)
    check(out, x, w, mag)
    again = torch.empty_like(out)
    call(lib, fmt, x, wt, again)
    assert torch.equal(out, again)                                # the same bits each time


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("K", [32, 64, 96, 160, 1056, 2016])
def test_matvec_ragged_groups(lib, fmt, K):
    """K a multiple of 32 but not of 128: the last step is partial and the
    scale rows start at any byte."""
    for M, N, xt in ((1, 77, "bf16"), (7, 30, "f16"), (16, 5, "f32")):
        wt, w, mag = weights(fmt, K + M, N, K)
        x = activations(K + M, M, K, xt)
        out = torch.full((M, N), float("nan"), device="cuda")
        call(lib, fmt, x, wt, out)
        check(out, x, w, mag)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K,xt", [(4, 2605, 4224, "bf16"), (2, 2400, 4608, "f16"), (16, 100, 6272, "f32"),
                                      (9, 20011, 256, "bf16"), (1, 9000, 1408, "f32"), (3, 40003, 128, "f16")])
def test_matvec_cuts(lib, fmt, M, N, K, xt):
    """Long rows in several copies (whole and partial ones, scale rows of any
    length) and short ones with many tiles a visit, several visits a block."""
    wt, w, mag = weights(fmt, K + M, N, K)
    x = activations(K + M, M, K, xt)
    out = torch.full((M, N), float("nan"), device="cuda")
    call(lib, fmt, x, wt, out)
    check(out, x, w, mag)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("K", [4128, 8160])
def test_matvec_long_ragged_groups(lib, fmt, K):
    wt, w, mag = weights(fmt, K, 333, K)
    x = activations(K, 5, K, "bf16")
    out = torch.full((5, 333), float("nan"), device="cuda")
    call(lib, fmt, x, wt, out)
    check(out, x, w, mag)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("xt", ["bf16", "f16", "f32"])
def test_matvec_strides_and_neighbours(lib, fmt, xt):
    """Row strides of x and out (odd ones, an odd first element); what lies
    between and behind out's rows stays as it was."""
    M, N, K = 5, 133, 512
    wt, w, mag = weights(fmt, 9, N, K)
    base = torch.zeros(M + 1, K + 7, dtype=DT[xt], device="cuda")
    x = base[1:, 3:3 + K]
    x.copy_(activations(3, M, K, xt))
    room = torch.full((M + 2, N + 5), 7.0, dtype=DT[xt], device="cuda")
    out = room[1:M + 1, 2:2 + N]
    call(lib, fmt, x, wt, out)
    check(out.contiguous(), x, w, mag)
    keep = torch.ones_like(room, dtype=torch.bool)
    keep[1:M + 1, 2:2 + N] = False
    assert (room[keep] == 7.0).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_matvec_wide_range_of_x(lib, fmt):
    """Rows and groups of very different size, zeros, subnormals and the
    types' largest values."""
    M, N, K = 4, 64, 1024
    for xt, big, small in (("bf16", 1e37, 1e-38), ("f16", 6e4, 6e-8), ("f32", 1e37, 1e-38)):
        wt, w, mag = weights(fmt, 5, N, K, 118, 122)
        x = activations(8, M, K, "f32")
        x[0] = 0
        x[1, 256:384] *= small / 4
        x[2] *= small
        x[3, ::7] = 0
        x[3, 5] = big / 1e3
        x = x.to(DT[xt])
        out = torch.empty(M, N, device="cuda")
        call(lib, fmt, x, wt, out)
        assert (out[0] == 0).all()
        check(out[1:], x[1:], w, mag)


def test_matvec_mxfp4_scale_range(lib):
    """Every E8M0 byte: the smallest (2^-127) and large ones are exact; a NaN
    scale (255) reaches its own row only."""
    N, K = 256, 128
    nib = synth.random_bytes(1, 1, (N, K // 2))
    s = np.repeat(np.arange(N, dtype=np.uint8)[:, None], K // 32, 1)
    w = ffn.dequant_mxfp4(nib, np.minimum(s, 254))
    x = torch.zeros(2, K, device="cuda")
    x[0, :32] = torch.randn(32, device="cuda").sign() * 2.0 ** -6
    x[1, 64:96] = 2.0 ** -3
    out = torch.empty(2, N, device="cuda")
    lib.moe_matvec_mxfp4(x, dev(nib), dev(s), out)
    ref = x.double().cpu().numpy() @ w.T
    got = out.double().cpu().numpy()
    # powers of two times codes: sums are exact, the result is rounded once (subnormal results to 2^-149)
    ok = np.abs(ref) < 3e38
    ok[:, 255] = False
    assert (np.abs(got - ref)[ok] <= 2.0 ** -24 * np.abs(ref)[ok] + 2.0 ** -147).all()
    assert np.isnan(got[:, 255]).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_matvec_non_finite_rows_stay_apart(lib, fmt):
    M, N, K = 6, 50, 256
    wt, w, mag = weights(fmt, 2, N, K)
    x = activations(2, M, K, "bf16")
    ref = torch.empty(M, N, device="cuda")
    call(lib, fmt, x, wt, ref)
    x[1, 3], x[4, 200], x[5, 0] = float("nan"), float("inf"), float("-inf")
    out = torch.empty(M, N, device="cuda")
    call(lib, fmt, x, wt, out)
    for m in (0, 2, 3):
        assert torch.equal(out[m], ref[m])


def test_matvec_of_the_repacks(lib):
    """The repacks' own outputs, as a user chains them: MXFP4 -> NVFP4 gives the
    same product, MXFP4 -> INT4 the product of the INT4 weights."""
    N, K, M = 384, 1024, 3
    nib, s = synth.quantize_mxfp4(synth.normal(4, 1, N * K).reshape(N, K) * 0.02)
    dn, ds = dev(nib)[None], dev(s)[None]
    x = activations(4, M, K, "bf16")
    y0, y1, y2 = (torch.empty(M, N, device="cuda") for _ in range(3))
    lib.moe_matvec_mxfp4(x, dn[0], ds[0], y0)
    q, e4, g = torch.empty_like(dn), torch.empty((1, N, K // 16), dtype=torch.uint8, device="cuda"), \
        torch.empty(1, device="cuda")
    lib.repack_mxfp4_to_nvfp4(dn, ds, q, e4, g)
    lib.moe_matvec_nvfp4(x, q[0], e4[0], g, y1)
    i4, sinv = torch.empty((1, N, K // 2), dtype=torch.int8, device="cuda"), torch.empty((1, N, K // 128), device="cuda")
    lib.repack_mxfp4_to_int4g128(dn, ds, i4, sinv)
    lib.moe_matvec_int4g128(x, i4[0], sinv[0], y2)
    w = ffn.dequant_mxfp4(nib, s)
    check(y0, x, w, np.abs(w))
    check(y1, x, w, np.abs(w))
    qi, si = RP.repack_mxfp4_to_int4g128(nib, s)
    wi = ffn.dequant_int4g128(qi, si)
    check(y2, x, wi, wi + 16 * np.repeat(si.astype(np.float64), 128, -1))
    assert lib.moe_get_device_error() == 0


@pytest.mark.parametrize("fmt", FMTS)
def test_matvec_streams_and_graphs(lib, fmt):
    """Another stream, two calls at once on two streams, and a captured call
    replayed on new inputs."""
    M, N, K = 2, 700, 2048
    wt, w, mag = weights(fmt, 6, N, K)
    x = [activations(20 + i, M, K, "bf16") for i in range(3)]
    ref = [torch.empty(M, N, device="cuda") for _ in x]
    for i in range(3):
        call(lib, fmt, x[i], wt, ref[i])
    torch.cuda.synchronize()
    st = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.zeros(M, N, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            call(lib, fmt, x[i], wt, outs[i], stream=st[i])
    torch.cuda.synchronize()
    assert torch.equal(outs[0], ref[0]) and torch.equal(outs[1], ref[1])
    xin, out = x[0].clone(), torch.zeros(M, N, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(lib, fmt, xin, wt, out)
    for i in (1, 2, 0):
        xin.copy_(x[i])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref[i])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,xt", [(1, "f32"), (3, "bf16"), (16, "f16"), (16, "f32")])
def test_matvec_widest(lib, fmt, M, xt):
    """The largest K; several rows of x then take several passes."""
    N, K = 48, lib.MOE_MATVEC_MAX_K
    wt, w, mag = weights(fmt, 7, N, K)
    x = activations(7, M, K, xt)
    out = torch.full((M, N), float("nan"), device="cuda")
    call(lib, fmt, x, wt, out)
    check(out, x, w, mag)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_matvec_scales_at_any_byte(lib, fmt):
    """Scale arrays that start at an odd address."""
    M, N, K = 3, 40, 512
    wt, w, mag = weights(fmt, 11, N, K)
    room = torch.empty(wt[1].numel() + 1, dtype=torch.uint8, device="cuda")
    odd = room[1:].view(wt[1].shape)
    odd.copy_(wt[1])
    x = activations(11, M, K, "bf16")
    out = torch.empty((M, N), device="cuda")
    call(lib, fmt, x, (wt[0], odd) + tuple(wt[2:]), out)
    check(out, x, w, mag)


def test_matvec_offsets_past_32_bits(lib):
    """A matrix of more than 2^32 nibbles: its last rows."""
    N, K = 1_050_000, 4096
    nib = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda")
    s = torch.full((N, K // 32), 120, dtype=torch.uint8, device="cuda")
    x = activations(1, 1, K, "bf16")
    out = torch.empty(1, N, device="cuda")
    lib.moe_matvec_mxfp4(x, nib, s, out)
    for r in (0, N // 2, N - 3):
        w = ffn.dequant_mxfp4(nib[r:r + 3].cpu().numpy(), s[r:r + 3].cpu().numpy())
        check(out[:, r:r + 3], x, w, np.abs(w))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("xt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("size", [1.0, 2.0 ** -20])
def test_matvec_keeps_float32_precision(lib, fmt, xt, size):
    """Sums lose nothing to the operands' form: INT4 codes, and rows of x among
    float16's subnormals."""
    for M, N, K in ((7, 1203, 1408), (1, 512, 4096), (3, 64, 32768)):
        wt, w, mag = weights(fmt, 13, N, K, 118, 122)
        x = (activations(13, M, K, "f32") * size).to(DT[xt])
        out = torch.empty((M, N), device="cuda")
        call(lib, fmt, x, wt, out)
        assert check(out, x, w, mag) <= 2.0 ** -20
