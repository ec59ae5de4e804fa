"""The few-token layer (moe_layer_few_mxfp4) against the float64 oracle of the
same steps, and against the library's own calls for the routing (bit-equal).

Tolerance of y, that of the layer's other paths: max |gpu - oracle| <= 1e-2 *
max |oracle| and sum |gpu - oracle| / sum |oracle| <= 2e-3.  It covers one
bfloat16 rounding (2^-8 of a value at most, half of that on average) and the
few E4M3 codes of h that float32 sums move across a rounding boundary.
"""
import numpy as np
import pytest
import torch

import synth
from fp8_block_scaled_pow2_b200.layer import MoeLayer
from oracle import ffn

pytestmark = pytest.mark.gpu

MAX_TOL, MEAN_TOL = 1e-2, 2e-3


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def check_y(y, ref):
    y = y.double().cpu().numpy()
    assert np.isfinite(y).all()
    err = np.abs(y - ref)
    assert err.max() <= MAX_TOL * np.abs(ref).max(), (err.max(), np.abs(ref).max())
    assert err.sum() / np.abs(ref).sum() <= MEAN_TOL, err.sum() / np.abs(ref).sum()


class Case:
    """One layer's weights on the host and the device."""

    def __init__(self, lib, seed, H, I, E, shared=1):
        G = E + shared
        self.H, self.I, self.E, self.shared = H, I, E, shared
        self.w13, self.s13 = synth.quantize_mxfp4(synth.normal(seed, 1, G * 2 * I * H).reshape(G * 2 * I, H) * 0.02)
        self.w2, self.s2 = synth.quantize_mxfp4(synth.normal(seed, 2, G * H * I).reshape(G * H, I) * 0.02)
        self.w13, self.s13 = self.w13.reshape(G, 2 * I, H // 2), self.s13.reshape(G, 2 * I, H // 32)
        self.w2, self.s2 = self.w2.reshape(G, H, I // 2), self.s2.reshape(G, H, I // 32)
        self.p13 = torch.empty(lib.moe_prepared_weights_size(G, 2 * I, H), dtype=torch.uint8, device="cuda")
        lib.moe_prepare_weights(dev(self.w13), dev(self.s13), self.p13, paired=True)
        self.p2 = torch.empty(lib.moe_prepared_weights_size(G, H, I), dtype=torch.uint8, device="cuda")
        lib.moe_prepare_weights(dev(self.w2), dev(self.s2), self.p2)

    def out(self, lib, T, k):
        ws = torch.full((lib.moe_layer_few_workspace_size(T, self.H, self.I, self.E, k, self.shared),), 0xFF,
                        dtype=torch.uint8, device="cuda")                # float32 NaN everywhere
        return dict(idx=torch.full((T, k), -7, dtype=torch.int32, device="cuda"),
                    w=torch.full((T, k), -7.0, device="cuda"),
                    y=torch.full((T, self.H), -7.0, dtype=torch.bfloat16, device="cuda"), workspace=ws)

    def run(self, lib, x, logits, k, out=None, norm=1, stream=None, tok=None, table=None):
        out = out or self.out(lib, x.shape[0], k)
        lib.moe_layer_few_mxfp4(x, logits, self.p13, self.p2, self.I, out["idx"], out["w"], out["y"],
                                out["workspace"], 1.5, 10.0, self.shared, norm, token_ids=tok, tid2eid=table,
                                stream=stream)
        return out

    def ref(self, x_bits, logits, k, norm=1, tok=None, table=None):
        return ffn.moe_layer(x_bits, logits, self.w13, self.s13, self.w2, self.s2, k, 1.5, 10.0, self.shared, norm,
                             token_ids=tok, tid2eid=table)


def inputs(seed, T, H, E):
    x = synth.to_bf16_bits(synth.normal(seed, 5, T * H).reshape(T, H))
    z = (synth.normal(seed, 6, T * E).reshape(T, E)).astype(np.float32)
    return x, z


@pytest.mark.parametrize("T,H,I,E,k,shared,norm", [
    (1, 256, 128, 8, 2, 1, 1), (16, 256, 128, 8, 2, 1, 1), (1, 128, 128, 1, 1, 0, 0), (2, 1408, 640, 40, 3, 1, 0),
    (3, 640, 1408, 12, 6, 0, 1), (5, 512, 384, 100, 16, 1, 1), (8, 1024, 256, 16, 8, 1, 1), (9, 384, 256, 4, 4, 1, 1),
    (16, 896, 128, 1, 1, 1, 1), (13, 256, 896, 33, 5, 0, 1), (16, 2048, 512, 64, 6, 1, 1), (4, 128, 2048, 20, 2, 1, 1),
    (7, 4096, 128, 9, 3, 1, 1),
])
def test_few_layer(lib, T, H, I, E, k, shared, norm):
    c = Case(lib, T + H + I, H, I, E, shared)
    xb, z = inputs(T * 31 + E, T, H, E)
    x = dev(xb.view(np.int16)).view(torch.bfloat16)
    out = c.run(lib, x, dev(z), k, norm=norm)
    ref = c.ref(xb, z, k, norm)
    np.testing.assert_array_equal(out["idx"].cpu().numpy(), ref["idx"])
    i2, w2 = torch.empty_like(out["idx"]), torch.empty_like(out["w"])
    lib.moe_route_topk(dev(z), k, i2, w2, 1.5, norm)
    assert torch.equal(out["idx"], i2) and torch.equal(out["w"], w2)
    check_y(out["y"], ref["y"])
    again = c.run(lib, x, dev(z), k, norm=norm)
    assert all(torch.equal(out[n], again[n]) for n in ("idx", "w", "y"))
    assert lib.moe_get_device_error() == 0


@pytest.mark.parametrize("T", [1, 2, 6, 16])
def test_few_layer_all_tokens_on_the_same_experts(lib, T):
    """Every token picks the same experts, so each expert has T rows."""
    H, I, E, k = 512, 256, 24, 4
    c = Case(lib, 3, H, I, E)
    xb, z = inputs(T, T, H, E)
    z[:, [3, 23, 0, 11]] += 50
    out = c.run(lib, dev(xb.view(np.int16)), dev(z), k)
    ref = c.ref(xb, z, k)
    np.testing.assert_array_equal(out["idx"].cpu().numpy(), ref["idx"])
    check_y(out["y"], ref["y"])


def test_few_layer_equal_and_masked_logits(lib):
    """Ties go to the lower index; experts masked with -inf or the lowest
    float32 are chosen last and weigh nothing."""
    T, H, I, E, k = 6, 256, 128, 70, 4
    c = Case(lib, 8, H, I, E)
    xb, z = inputs(8, T, H, E)
    z[0] = 0.25
    z[1, ::2] = 1.0
    z[2, 2:] = -np.inf
    z[3, 3:] = np.finfo(np.float32).min
    z[4] = np.repeat([1.0, 2.0], 35)
    out = c.run(lib, dev(xb.view(np.int16)), dev(z), k)
    ref = c.ref(xb, np.maximum(z, -1e30), k)
    np.testing.assert_array_equal(out["idx"].cpu().numpy(), ref["idx"])
    assert out["idx"][0].tolist() == [0, 1, 2, 3]
    w = out["w"].cpu().numpy()
    np.testing.assert_allclose(w, ref["w"], rtol=1e-6, atol=1e-30)
    assert (w[2, 2:] == 0).all() and (w[3, 3:] == 0).all()
    check_y(out["y"], ref["y"])


def test_few_layer_nan_logits_are_never_chosen(lib):
    T, H, I, E, k = 3, 256, 128, 40, 3
    c = Case(lib, 9, H, I, E)
    xb, z = inputs(9, T, H, E)
    z[:, ::3] = np.nan
    z[2, 2:] = np.nan                                     # one finite logit (index 1) for three slots
    out = c.run(lib, dev(xb.view(np.int16)), dev(z), k)
    assert lib.moe_get_device_error() == -1               # MOE_ERR_INVALID: slots without an expert
    idx = out["idx"].cpu().numpy()
    ref = c.ref(xb[:2], np.where(np.isnan(z[:2]), -1e30, z[:2]), k)
    np.testing.assert_array_equal(idx[:2], ref["idx"])
    check_y(out["y"][:2], ref["y"])
    assert idx[2].tolist() == [1, -1, -1] and out["w"][2].tolist() == [1.5, 0, 0]


@pytest.mark.parametrize("T,k,shared", [(1, 6, 1), (3, 3, 0), (16, 4, 1)])
def test_few_layer_hash_routing(lib, T, k, shared):
    H, I, E, V = 640, 256, 30, 50
    c = Case(lib, 12, H, I, E, shared)
    xb, z = inputs(T, T, H, E)
    table = synth.hash_table(5, V, E, k).astype(np.int32)
    tok = synth.token_ids(6, T, V).astype(np.int32)
    out = c.run(lib, dev(xb.view(np.int16)), dev(z), k, tok=dev(tok), table=dev(table))
    ref = c.ref(xb, z, k, tok=tok, table=table)
    np.testing.assert_array_equal(out["idx"].cpu().numpy(), ref["idx"])
    i2, w2 = torch.empty_like(out["idx"]), torch.empty_like(out["w"])
    lib.moe_route_hash(dev(tok), dev(table), dev(z), i2, w2)
    assert torch.equal(out["idx"], i2) and torch.equal(out["w"], w2)
    check_y(out["y"], ref["y"])
    assert lib.moe_get_device_error() == 0


def test_few_layer_hash_bad_ids_and_repeated_experts(lib):
    """A token id past the table, a table entry past E and an expert twice in
    one row: the bad slots add nothing, the others are as they should be."""
    T, H, I, E, V, k = 5, 256, 128, 6, 8, 3
    c = Case(lib, 14, H, I, E)
    xb, z = inputs(14, T, H, E)
    table = synth.hash_table(7, V, E, k).astype(np.int32)
    table[2] = [4, 4, 1]
    table[3] = [5, E, 0]
    tok = np.array([2, V, 3, 0, -1], np.int32)
    out = c.run(lib, dev(xb.view(np.int16)), dev(z), k, tok=dev(tok), table=dev(table))
    assert lib.moe_get_device_error() == -1
    idx, w = out["idx"].cpu().numpy(), out["w"].double().cpu().numpy()
    assert (idx[1] == -1).all() and (idx[4] == -1).all() and idx[2].tolist() == [5, -1, 0]
    assert idx[0].tolist() == [4, 4, 1] and (w[[1, 4]] == 0).all() and w[2, 1] == 0
    # the oracle expert by expert: with one expert per token and no normalisation w is a plain factor
    y = np.zeros((T, H))
    for t in range(T):
        for j in range(k):
            if idx[t, j] >= 0:
                one = ffn.moe_layer(xb[t:t + 1], z[t:t + 1], c.w13, c.s13, c.w2, c.s2, 1, 1.0, 10.0, 1, 1,
                                    token_ids=np.zeros(1, np.int32), tid2eid=idx[t:t + 1, j:j + 1])
                y[t] += w[t, j] * one["o"][0]
                shared = one["o"][1]
            elif j == 0:
                shared = ffn.moe_layer(xb[t:t + 1], z[t:t + 1], c.w13, c.s13, c.w2, c.s2, 1)["o"][1]
        y[t] += shared
    check_y(out["y"], y)


def test_few_layer_clamp_and_zero_rows(lib):
    """A zero token gives zero, and gate / up values far past the clamp."""
    T, H, I, E, k = 4, 256, 128, 8, 2
    c = Case(lib, 15, H, I, E)
    xb, z = inputs(15, T, H, E)
    xb[1] = 0
    xb[2] = synth.to_bf16_bits(synth.bf16_bits_to_f32(xb[2]) * 300)
    out = c.run(lib, dev(xb.view(np.int16)), dev(z), k)
    ref = c.ref(xb, z, k)
    assert (out["y"][1] == 0).all()
    check_y(out["y"], ref["y"])


def test_few_layer_streams_graphs_and_neighbours(lib):
    """Two calls at once on two streams, captured calls that share a workspace
    and replay on new inputs, and rows behind the last token left alone."""
    T, H, I, E, k = 3, 512, 256, 32, 4
    c = Case(lib, 16, H, I, E)
    ins = [inputs(40 + i, T, H, E) for i in range(4)]
    xs = [dev(a.view(np.int16)) for a, _ in ins]
    zs = [dev(b) for _, b in ins]
    ref = [c.run(lib, xs[i], zs[i], k)["y"].clone() for i in range(4)]
    torch.cuda.synchronize()
    st = [torch.cuda.Stream() for _ in range(2)]
    outs = [c.out(lib, T, k) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            c.run(lib, xs[i], zs[i], k, out=outs[i], stream=st[i])
    torch.cuda.synchronize()
    assert torch.equal(outs[0]["y"], ref[0]) and torch.equal(outs[1]["y"], ref[1])
    xin, zin = xs[0].clone(), zs[0].clone()
    o1, o2 = c.out(lib, T, k), c.out(lib, T, k)
    o2["workspace"] = o1["workspace"]
    graphs = []
    for o in (o1, o2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run(lib, xin, zin, k, out=o)
        graphs.append(g)
    for i in (2, 1, 3):
        xin.copy_(xs[i])
        zin.copy_(zs[i])
        for g, o in zip(graphs, (o1, o2)):
            o["y"].fill_(0)
            g.replay()
        for _ in range(10):
            graphs[0].replay()
            graphs[1].replay()
        torch.cuda.synchronize()
        assert torch.equal(o1["y"], ref[i]) and torch.equal(o2["y"], ref[i])
    big = c.out(lib, T + 2, k)
    part = dict(idx=big["idx"][:T], w=big["w"][:T], y=big["y"][:T], workspace=big["workspace"])
    c.run(lib, xs[0], zs[0], k, out=part)
    assert torch.equal(big["y"][:T], ref[0])
    assert (big["y"][T:] == -7).all() and (big["idx"][T:] == -7).all() and (big["w"][T:] == -7).all()


def test_few_layer_through_moe_layer(lib):
    """MoeLayer.forward_few beside MoeLayer.forward, alternating on one stream
    with producers and consumers of its buffers; refusals."""
    H, I, E, k = 512, 256, 16, 4
    c = Case(lib, 17, H, I, E)
    layer = MoeLayer(c.w13, c.s13, c.w2, c.s2, k)
    for T in (1, 4, 16):
        buf, full = layer.alloc_few(T), layer.alloc(T)
        for i in range(3):
            xb, z = inputs(60 + T + i, T, H, E)
            x, zd = dev(xb.view(np.int16)), dev(z)
            x2 = torch.zeros_like(x)
            x2 += x                                      # x written by the kernel just before the call
            y = layer.forward_few(x2, zd, buf).clone()
            x2.zero_()                                   # and overwritten just after it
            yf = layer.forward(x, zd, full)
            assert torch.equal(buf.idx, full.idx) and torch.equal(buf.w, full.w)
            ref = c.ref(xb, z, k)["y"]
            check_y(y, ref)
            check_y(yf, ref)
            check_y(layer.forward_few(x, zd), ref)        # buffers of its own
    assert layer.alloc_few(0).y.shape == (0, H)
    layer.forward_few(torch.empty((0, H), dtype=torch.int16, device="cuda"), torch.empty((0, E), device="cuda"))
    with pytest.raises(ValueError):
        layer.alloc_few(17)
    with pytest.raises(ValueError):
        MoeLayer(c.w13, c.s13, c.w2, c.s2, k, weights="ptpc").alloc_few(1)
    table = synth.hash_table(1, 20, E, k).astype(np.int32)
    hashed = MoeLayer(c.w13, c.s13, c.w2, c.s2, k, tid2eid=table)
    xb, z = inputs(99, 2, H, E)
    tok = np.array([3, 19], np.int32)
    y = hashed.forward_few(dev(xb.view(np.int16)), dev(z), token_ids=dev(tok))
    check_y(y, c.ref(xb, z, k, tok=tok, table=table)["y"])
    with pytest.raises(ValueError):
        hashed.forward_few(dev(xb.view(np.int16)), dev(z))


def test_few_layer_widest(lib):
    """The widest supported rows with the most tokens."""
    T, H, I, E, k = 16, lib.MOE_FEW_MAX_WIDTH, 256, 2, 1
    c = Case(lib, 18, H, I, E)
    xb, z = inputs(18, T, H, E)
    check_y(c.run(lib, dev(xb.view(np.int16)), dev(z), k)["y"], c.ref(xb, z, k)["y"])
    H, I = 256, lib.MOE_FEW_MAX_WIDTH
    c = Case(lib, 19, H, I, E)
    xb, z = inputs(19, T, H, E)
    check_y(c.run(lib, dev(xb.view(np.int16)), dev(z), k)["y"], c.ref(xb, z, k)["y"])


@pytest.mark.parametrize("T", [1, 5])
def test_few_layer_decode_size(lib, T):
    """The decode configuration's sizes (hidden 4096, intermediate 2048, 256 + 1
    experts sharing a few prototypes) against the oracle."""
    H, I, E, k = 4096, 2048, 256, 6
    w13, s13, w2, s2 = synth.expert_views(21, E + 1, H, I, 3)
    layer = MoeLayer(w13[:], s13[:], w2[:], s2[:], k)
    xb, z = inputs(22, T, H, E)
    y = layer.forward_few(dev(xb.view(np.int16)), dev(z))
    check_y(y, ffn.moe_layer(xb, z, w13, s13, w2, s2, k, cache={})["y"])
