"""The few-token layer token by token and element by element against the
float64 oracle, with tokens of very different size in one call.

Tolerance of an element of y, from the steps (g, u: the float32 sums of the
gate and up products of a pair; E: its expert):
  g, u   within H / 32 * 2^-22 of the magnitudes summed: each MMA adds 32 exact
         products and the float32 sum so far, and may truncate twice by 2^-23;
  h      |silu'| <= 1.1 carries that through the SwiGLU, whose own arithmetic is
         within 24 ulp;
  codes  an element of h may take any code that the interval h +- dh reaches,
         under any group scale that its group's largest value +- dh reaches;
  o      the sum over I of |change of h| * |w2|, and I / 32 * 2^-22 of the magnitudes;
  y      the weighted sum of these over a token's pairs, 2^-20 of the magnitudes
         for the router weights and the sum of the parts, one bfloat16 rounding.
"""
import numpy as np
import pytest
import torch

import synth
from oracle import ffn, quant
from oracle.formats import decode_e4m3, encode_e4m3_rne_sat

from tests.test_gpu_few_layer import Case, dev

pytestmark = pytest.mark.gpu


def reached(h, dh):
    """Largest change of a requantised element of h [rows, I] when h moves by up to dh."""
    R, I = h.shape
    g, d = h.reshape(R, I // 128, 128), dh.reshape(R, I // 128, 128)
    scale = lambda a: quant.pow2_scale_exponent(a.astype(np.float32))[..., None]
    codes = lambda v, k: decode_e4m3(encode_e4m3_rne_sat(v * np.ldexp(1.0, -k))) * np.ldexp(1.0, k)
    k = scale(np.abs(g).max(-1))
    ref = codes(g.astype(np.float32).astype(np.float64), k)
    lo, hi = np.maximum(np.abs(g) - d, 0).max(-1), (np.abs(g) + d).max(-1)
    step = np.zeros_like(g)
    for kk in (k, scale(lo), scale(hi)):
        for v in (g - d, g + d):
            step = np.maximum(step, np.abs(codes(v, kk) - ref))
    return step.reshape(R, I)


def tolerance(c, ref, T, k):
    """float64 [T, H]."""
    H, I = c.H, c.I
    x = quant.dequantize_fp8_pow2(ref["xq_perm"], ref["sx_perm"])
    h = ffn.swiglu_clamp(ref["gu"], I)
    hd = quant.dequantize_fp8_pow2(ref["hq"], ref["sh"])
    per_row, mag = np.zeros((len(x), H)), np.zeros((len(x), H))
    for e in range(c.E + c.shared):
        r = slice(int(ref["offsets"][e]), int(ref["offsets"][e + 1]))
        if r.start == r.stop:
            continue
        sums = np.abs(x[r]) @ np.abs(ffn.dequant_mxfp4(c.w13[e], c.s13[e])).T * (H / 32 * 2.0 ** -22)
        gc, uc = np.clip(ref["gu"][r, :I], -10, 10), np.clip(ref["gu"][r, I:], -10, 10)
        dg, du = sums[:, :I], sums[:, I:]
        dh = 1.1 * dg * np.abs(uc) + np.abs(ffn.silu(gc)) * du + 1.1 * dg * du + 24 * 2.0 ** -23 * np.abs(h[r])
        w2 = np.abs(ffn.dequant_mxfp4(c.w2[e], c.s2[e])).T
        step = reached(h[r], dh)
        mag[r] = (np.abs(hd[r]) + step) @ w2
        per_row[r] = step @ w2 + I / 32 * 2.0 ** -22 * mag[r]
    tol, total = np.zeros((T, H)), np.zeros((T, H))
    inv = ref["inv"].reshape(T, k)
    for j in range(k):
        tol += ref["w"][:, j:j + 1] * per_row[inv[:, j]]
        total += ref["w"][:, j:j + 1] * mag[inv[:, j]]
    if c.shared:
        s = int(ref["offsets"][c.E]) + np.arange(T)
        tol += per_row[s]
        total += mag[s]
    tol += 2.0 ** -20 * total
    return tol + 2.0 ** -8 * (np.abs(ref["y"]) + tol) + 2.0 ** -130


@pytest.mark.parametrize("T,H,I,E,k,shared", [(1, 256, 128, 8, 2, 1), (16, 256, 128, 8, 2, 1), (5, 512, 256, 24, 4, 1),
                                              (9, 1408, 640, 12, 6, 0), (16, 640, 384, 30, 3, 1), (3, 2048, 512, 9, 2, 1)])
@pytest.mark.parametrize("spread", [0, 2])
def test_every_token_within_its_own_bound(lib, T, H, I, E, k, shared, spread):
    c = Case(lib, T + H + I, H, I, E, shared)
    x = synth.normal(T + E, 5, T * H).reshape(T, H) * np.exp2(-spread * np.arange(T))[:, None]
    xb = synth.to_bf16_bits(x)
    z = synth.normal(T + E, 6, T * E).reshape(T, E).astype(np.float32)
    out = c.run(lib, dev(xb.view(np.int16)), dev(z), k)
    ref = c.ref(xb, z, k)
    np.testing.assert_array_equal(out["idx"].cpu().numpy(), ref["idx"])
    tol = tolerance(c, ref, T, k)
    err = np.abs(out["y"].double().cpu().numpy() - ref["y"])
    assert np.isfinite(err).all()
    worst = (err / tol).max(-1)
    assert (err <= tol).all(), worst
    # the bound says something about every token, the smallest ones too
    assert (np.linalg.norm(tol, axis=-1) < 0.25 * np.linalg.norm(ref["y"], axis=-1)).all()
